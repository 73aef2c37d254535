// Linear attention with a decay for each head: gradients.
//
// With dS_t the gradient of the state after token t (from the outputs and the last
// state's),
//   dS_{t-1} = e^g_t dS_t + scale q_{t-1} do_{t-1}^T
//   dq_t = scale S_t do_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t
// which are three more linear attentions: dq forward in time with do, v, k in the
// places of q, k, v; dk backward with v, do, q; dv backward with k, q, do.  So no
// states are kept from the forward pass: the walks make them again from rows that
// they read anyway.
//
// dg_t = <dS_t, e^g_t S_{t-1}> is the sum over all pairs s < t <= u of
// W_us = scale e^(g_{s+1} + .. + g_u) (q_u.k_s)(do_u.v_s).  As a difference of sums
// of q.dq and k.dk it would lose what strong decays leave of it.  So by chunks:
//   s before the chunk, u in it:  sum over u >= t of q_u . (dq_u's part with S0)
//   s in it, u behind:            sum over s < t of k_s . (dk_s's part with X)
//   both in it:                   sums of W over rectangles
//   s before, u behind:           A = e^Dc <X, S0>, the same for the whole chunk
// A follows from the next chunk's: A + (s in it, u behind) by all tokens = A' + (s
// before, u in the next) by all of its, 0 where e^Dc leaves nothing in fp32.
#include "fftconv_decay_walk.h"

namespace fftconv {
namespace {

template <int IO, int DA>
struct Back {
    static constexpr int C = IO == IO_F32 || DA > 128 ? 32 : 64;
    static constexpr int RW = DA <= 64 ? 2 : 4;          // waves of a role
    static constexpr int kTile = C * DA * Kind<IO>::kB;
    static constexpr int kP = Scores<IO, C>::kBytes;
    static constexpr int kBytes = 4 * kTile + 2 * kP;
};

// Scores of dk (rows of v against do) as make_scores() makes them, and the sums over
// rectangles of W: part[qt][t] for the sixteen s of the wave.
template <int IO, int DA, int C, int NW>
__device__ __forceinline__ void make_scores_and_sums(const char* V, const char* DO, const char* K,
                                                     const char* Q, char* P, float* back,
                                                     const Factors<C>& F, float scale, int wave,
                                                     float (*part)[C]) {
    constexpr int KT = C / 16;
    const int lane = fresh_lane(), g = lane >> 4, c = lane & 15;
    const RowReader<IO, DA, 16> rows(lane);
    if (NW > KT && wave >= KT) return;
#pragma unroll
    for (int j = 0; j < (KT + NW - 1) / NW; ++j) {
        const int qt = wave + NW * j;
        dfloat4 vd[KT], kq[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) vd[kt] = kq[kt] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DA / 32; ++kb) {
            const Frag<IO> b = rows.get(V, 16 * qt, 32 * kb);
            const Frag<IO> b2 = rows.get(K, 16 * qt, 32 * kb);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                vd[kt] = mma16<IO>(rows.get(DO, 16 * kt, 32 * kb), b, vd[kt]);
                kq[kt] = mma16<IO>(rows.get(Q, 16 * kt, 32 * kb), b2, kq[kt]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        products_done();
        const int i = 16 * qt + c, iw = F.whole[i];
        const float ir = F.rest[i];
        float largest = 0.f, carry = 0.f;
#pragma unroll
        for (int kt = KT - 1; kt >= 0; --kt) {
            const int s0 = 16 * kt + 4 * g;
            const int4 sw = *(const int4*)&F.whole[s0];
            const float4 sr = *(const float4*)&F.rest[s0];
            const int w[4] = {sw.x, sw.y, sw.z, sw.w};
            const float r[4] = {sr.x, sr.y, sr.z, sr.w};
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = scale * exp2_of(w[e] - iw, r[e] - ir) * vd[kt][e];
                vd[kt][e] = s0 + e >= i ? x : 0.f;
                y[e] = s0 + e > i ? x * kq[kt][e] : 0.f;
                if (IO == IO_F16) largest = fmaxf(largest, fabsf(vd[kt][e]));
            }
            // of the tokens u from t on
            y[2] += y[3];
            y[1] += y[2];
            y[0] += y[1];
            float a = y[0], b = __shfl_down(a, 16);
            a += g < 3 ? b : 0.f;
            b = __shfl_down(a, 32);
            a += g < 2 ? b : 0.f;
            b = __shfl_down(a, 16);
            const float behind = (g < 3 ? b : 0.f) + carry;
            carry += __shfl(a, c);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = s0 + e > i ? y[e] + behind : 0.f;
            const float sum = sums16_of4(y);
            if ((c & 3) == 0) part[qt][s0 + (c >> 2)] = sum;
        }
        float to = 1.f;
        if constexpr (IO == IO_F16) {
            const Scale sc = scale_to(fmaxf(max_groups(largest), 0x1p-40f));
            to = sc.to;
            if (g == 0) back[i] = sc.back;
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) put_scores<IO, C>(P, lane, qt, kt, to, vd[kt]);
    }
}

// dk and dv: a workgroup of two roles of RW waves each walks over a segment's
// chunks backward in time, with the gradient X of the state, columns of Dv in the
// first role's waves (dv) and, transposed, columns of Dk in the second's (dk).
template <int IO, int DA>
__global__ __launch_bounds__((DA <= 64 ? 256 : 512), 1) void decay_back_kernel(DecayGradParams p,
                                                                             int slices) {
    typedef Back<IO, DA> L;
    constexpr int C = L::C, RW = L::RW, N = 128 * RW, kB = Kind<IO>::kB;
    const DecayParams& f = p.f;
    const unsigned units = (unsigned)(f.sp.segs * f.Hv * slices), u = xcd_unit(blockIdx.x, units);
    if (u >= units) return;
    const int slice = (int)(u % slices), h = (int)(u / slices % f.Hv);
    const unsigned seg = u / slices / f.Hv;
    DecaySpan s;
    if (!segment_of(f.sp, seg, s)) return;
    const int tid = threadIdx.x, lane = tid & 63, place = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = place & (RW - 1);
    const bool keys = place >= RW;      // the role
    const int first = slice * 32 * RW, mine = first + 32 * wave, col = mine + (lane & 31);
    const int cols = keys ? f.Dk : f.Dv, rows = keys ? f.Dv : f.Dk;
    const bool ok = col < cols, wide = keys && p.dk_heads;
    if (s.index == 0 && f.sp.cu) {
        const int nk = min(f.Dk - first, 32 * RW), nv = min(f.Dv - first, 32 * RW);
        if (nk > 0)
            clear_unheld(f.sp, s, p.dk_heads ? p.dk_heads : p.dk, p.dk_heads ? 4 : kB, f.Hv, f.Dk, h,
                         first, nk);
        if (nv > 0) clear_unheld(f.sp, s, p.dv, kB, f.Hv, f.Dv, h, first, nv);
    }
    const long long size = (long long)f.Dk * f.Dv;
    const long long rs = keys ? 1 : f.Dv, cs = keys ? f.Dv : 1, at_col = ok ? col * cs : 0;
    State<DA> X;
    X.clear();
    if (p.seg_back) X.load(p.seg_back + (seg * (long long)f.Hv + h) * size + at_col, rs, ok, rows);
    else if (p.dfin) X.load(p.dfin + (s.seq * (long long)f.Hv + h) * size + at_col, rs, ok, rows);

    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const Q = lds;
    char* const K = lds + L::kTile;
    char* const V = lds + 2 * L::kTile;
    char* const DO = lds + 3 * L::kTile;
    char* const P = lds + 4 * L::kTile + (keys ? L::kP : 0);
    __shared__ __attribute__((aligned(16))) Factors<C> F[2];
    __shared__ __attribute__((aligned(16))) float back[2][C];
    __shared__ __attribute__((aligned(16))) float part[C / 16][C];
    __shared__ float dots[RW][C];
    const int chunks = (s.to - s.from + C - 1) / C;
    const Tokens q = rows_of<IO>(f.q, s, h), k = rows_of<IO>(f.k, s, h), v = rows_of<IO>(f.v, s, h),
                 d = rows_of<IO>(p.d_o, s, h);
    const int kp = f.Dk * kB / 16, vp = f.Dv * kB / 16;
    const float* gates = f.fixed ? f.g + h : f.g + (s.b * f.sp.T + s.t0) * f.Hv + h;
    const auto log_decay = [&](int at, int n) {
        return f.fixed ? gates[0] : gates[(long long)(at + (lane < n ? lane : n - 1)) * f.Hv];
    };
    const long long token0 = s.b * f.sp.T + s.t0;
    const long long slot0 = f.sp.cu ? s.t0 / C + s.seq : s.b * ((f.sp.T + C - 1) / C);
    Moving<IO, DA, C, N> mq, mk, mv, md;
    const auto fetch = [&](int at, int n) {
        mq.load(q, at, n, kp, tid);
        mk.load(k, at, n, kp, tid);
        mv.load(v, at, n, vp, tid);
        md.load(d, at, n, vp, tid);
    };
    const auto put = [&](Factors<C>& F, int n) {
        mq.clear(n, kp, tid);
        mk.clear(n, kp, tid);
        mv.clear(n, vp, tid);
        md.clear(n, vp, tid);
        mq.store(Q, tid);
        mk.store(K, tid);
        mv.store(V, tid);
        md.store(DO, tid);
        if (mq.unbounded() || md.unbounded()) F.unbounded = 1;
    };
    const auto factors = [&](Factors<C>& F, float g, int n) {
        put_factors<C, true>(F, decays_to<C>(g, f.fixed, n), 1.f, f.scale);
        if (lane == 0) F.unbounded = 0;
    };
    if (chunks) {
        const int at = s.from + (chunks - 1) * C, n = s.to - at;
        fetch(at, n);
        if (tid < 64) factors(F[0], log_decay(at, n), n);
        __syncthreads();
        put(F[0], n);
        __syncthreads();
    }
    for (int i = 0; i < chunks; ++i) {
        const Factors<C>& fac = F[i & 1];
        const int ch = chunks - 1 - i, at = s.from + ch * C, n = s.to - at < C ? s.to - at : C;
        const bool more = ch > 0;
        float g = 0.f;
        if (more) {
            fetch(at - C, C);
            if (tid < 64) g = log_decay(at - C, C);
        }
        dfloat16 acc[C / 32];
        if (keys) {
            make_scores_and_sums<IO, DA, C, RW>(V, DO, K, Q, P, back[1], fac, f.scale, wave, part);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C, IO == IO_BF16 ? 2 : Kind<IO>::NS>(V, X, fac, acc);
        } else {
            make_scores<IO, DA, C, RW, true>(K, Q, P, back[0], fac, f.scale, wave);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C, Kind<IO>::NS>(K, X, fac, acc);
            __builtin_amdgcn_sched_barrier(0);
            row_dots<IO, DA, C>(V, mine < DA ? mine : 0, acc, dots[wave]);
        }
        __syncthreads();
        if (tid < 64 && first < f.Dv) {
            // s in the chunk before t
            double x = 0, r = 0;
            if (lane < C) {
#pragma unroll
                for (int w = 0; w < RW; ++w) x += dots[w][lane];
#pragma unroll
                for (int w = 0; w < C / 16; ++w) r += part[w][lane];
            }
            const double to = prefix_sum(x), all = __shfl(to, 63);
            double before = __shfl_up(to, 1);
            if (lane == 0) before = 0;
            if (lane < n)
                p.behind[((long long)slice * f.Hv + h) * p.B * f.sp.T + token0 + at + lane] =
                    (float)(before + (slice == 0 ? r : 0));
            if (lane == 0)
                p.chunks[(slice * p.slots + slot0 + at / C) * f.Hv + h] = make_float2((float)all, fac.all);
        }
        Frag<IO> val[C / 16];
        const int from = mine < DA ? mine : 0;
        const ColReader<IO, DA, false> vcols(fresh_lane());
#pragma unroll
        for (int kb = 0; kb < C / 16; ++kb) val[kb] = vcols.get(keys ? Q : DO, 16 * kb, from);
        scores_product<IO, C, true>(P, back[keys], val, fac.unbounded, acc);
        __builtin_amdgcn_sched_barrier(0);
        // K's and V's tiles are done with
        const int ob = wide ? 4 : kB;
        const long long row = (long long)f.Hv * cols * ob;
        store_rows<IO, DA, C>(keys ? V : K, from, acc,
                              (char*)(keys ? (wide ? (void*)p.dk_heads : p.dk) : p.dv) +
                                  (token0 + at) * row + (long long)(h * cols + mine) * ob,
                              row, (cols - mine) * ob / 16, wide, n);
        __builtin_amdgcn_sched_barrier(0);
        update_state<IO, DA, C>(keys ? DO : Q, val, fac, X);
        if (tid < 64 && more) factors(F[(i + 1) & 1], g, C);
        __syncthreads();
        if (more) put(F[(i + 1) & 1], C);
        __syncthreads();
    }
    if (!keys && s.index == 0 && p.dinit)
        X.store(p.dinit + (s.seq * (long long)f.Hv + h) * size + col * cs, rs, ok, rows);
}

// dg from its parts, kDgChunks chunks of C tokens a workgroup.
__global__ __launch_bounds__(256) void decay_dg_kernel(DecayGradParams p, DecaySpans sp, int C,
                                                       int ks, int vs, int ends) {
    const DecayParams& f = p.f;
    const int h = (int)(blockIdx.x % f.Hv), lane = threadIdx.x & 63;
    const unsigned part = blockIdx.x / f.Hv;
    __shared__ float A[kDgChunks];
    __shared__ double sums[4];
    DecaySpan s;
    double sum = 0;
    const bool held = segment_of(sp, part, s);
    if (held) {
        const long long token0 = s.b * sp.T + s.t0, tokens = p.B * sp.T;
        const int nc = (s.len + C - 1) / C, mine = s.from / C;
        const long long slot0 = sp.cu ? s.t0 / C + s.seq : s.b * ((sp.T + C - 1) / C);
        if (threadIdx.x < 64) {
            // A of the chunks from the sequence's last to the workgroup's first
            double next = 0;
            for (int top = (nc - 1) / kDgChunks * kDgChunks; top >= mine; top -= kDgChunks) {
                const int c = top + kDgChunks - 1 - lane;      // lanes: from the last on
                double b = 0;
                int keep = 1;
                if (c < nc) {
                    for (int i = 0; i < vs; ++i) {
                        // a slice's sum is its part of the chunk's
                        const float2 x = p.chunks[(i * p.slots + slot0 + c) * f.Hv + h];
                        b -= x.x;
                        keep = x.y >= 0x1p-24f;
                    }
                    if (c + 1 < nc) {
                        for (int i = 0; i < ks; ++i)
                            b += p.before[((long long)i * f.Hv + h) * tokens + token0 +
                                          (long long)(c + 1) * C];
                    } else {
                        for (int i = 0; i < ends; ++i)
                            b += p.ends[(s.seq * (long long)f.Hv + h) * ends + i];
                    }
                    if (!keep) b = 0;
                }
                // the lane's chunk on top of the later ones': A = keep A' + b
                for (int m = 1; m < 64; m <<= 1) {
                    const double x = __shfl_up(b, m);
                    const int y = __shfl_up(keep, m);
                    if (lane >= m) {
                        if (keep) b += x;
                        keep &= y;
                    }
                }
                if (keep) b += next;
                next = __shfl(b, 63);
                if (top == mine) A[kDgChunks - 1 - lane] = (float)b;
            }
        }
        __syncthreads();
        for (int t = s.from + threadIdx.x; t < s.to; t += 256) {
            const long long at = token0 + t;
            float x = A[(t - s.from) / C], y = 0;
            for (int i = 0; i < ks; ++i) y += p.before[((long long)i * f.Hv + h) * tokens + at];
            for (int i = 0; i < vs; ++i) y += p.behind[((long long)i * f.Hv + h) * tokens + at];
            if (f.fixed) sum += (double)x + (double)y;
            else p.dg[at * f.Hv + h] = x + y;
        }
        if (!f.fixed && sp.cu && s.index == 0) {
            const long long end = s.t0 + s.len;
            if (s.seq == 0)
                for (long long t = threadIdx.x; t < s.t0; t += 256) p.dg[t * f.Hv + h] = 0.f;
            if (s.seq + 1 == sp.nseq)
                for (long long t = end + threadIdx.x; t < sp.T; t += 256) p.dg[t * f.Hv + h] = 0.f;
        }
    }
    if (!f.fixed) return;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (lane == 0) sums[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        p.sums[(long long)part * f.Hv + h] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}
// dg of a head, one decay for all its tokens
__global__ __launch_bounds__(256) void decay_dg_sum_kernel(const double* part, long long n, int Hv,
                                                           float* dg) {
    __shared__ double sums[4];
    double a = 0;
    for (long long i = threadIdx.x; i < n; i += 256) a += part[i * Hv + blockIdx.x];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) a += __shfl_xor(a, m);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = a;
    __syncthreads();
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)((sums[0] + sums[1]) + (sums[2] + sums[3]));
}

// Gradients of heads that value heads share: four elements a thread.
template <int IO>
__global__ __launch_bounds__(256) void decay_share_kernel(const float* x, void* y, long long n, int D,
                                                          int group) {
    const long long i = 4 * ((long long)blockIdx.x * 256 + threadIdx.x);
    if (i >= n) return;
    const long long head = i / D, e = i - head * D;
    dfloat4 a = {0, 0, 0, 0};
    for (int j = 0; j < group; ++j) a += *(const dfloat4*)(x + (head * group + j) * D + e);
    store4<IO>(y, i, a);
}

template <int IO, int DA>
hipError_t back_launch(const DecayGradParams& p, hipStream_t s) {
    typedef Back<IO, DA> L;
    const auto kernel = decay_back_kernel<IO, DA>;
    const hipError_t e = hipFuncSetAttribute((const void*)kernel,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != hipSuccess) return e;
    const int widest = p.f.Dk > p.f.Dv ? p.f.Dk : p.f.Dv;
    const int slices = (widest + 32 * L::RW - 1) / (32 * L::RW);
    hipLaunchKernelGGL(kernel, dim3((unsigned)xcd_blocks(p.f.sp.segs * p.f.Hv * slices)),
                       dim3(128 * L::RW), L::kBytes, s, p, slices);
    return hipGetLastError();
}

template <int IO>
hipError_t bwd_io(const DecayGradParams& p, hipStream_t s) {
    const DecayParams& f = p.f;
    hipError_t e;
    DecayWalk w = DecayWalk();
    w.sp = f.sp;
    w.Hv = f.Hv;
    w.fixed = f.fixed;
    w.g = f.g;
    w.seg_g = f.seg_g;
    w.tokens = p.B * f.sp.T;
    if (f.seg && f.sp.nseq) {
        // the first states of the segments and the gradients of their last
        w.rows = f.Dk;
        w.cols = f.Dv;
        w.rs = f.Dv;
        w.cs = 1;
        w.b = f.k;
        w.v = f.v;
        w.sw = 1.f;
        w.seg = f.seg;
        if ((e = decay_walk_io<IO, kEffects>(w, s)) != hipSuccess) return e;
        if ((e = launch_decay_join(f, f.init, false, s)) != hipSuccess) return e;
        w.b = f.q;
        w.v = p.d_o;
        w.sw = f.scale;
        w.seg = p.seg_back;
        if ((e = decay_walk_io<IO, kEffectsBack>(w, s)) != hipSuccess) return e;
        DecayParams r = f;
        r.seg = p.seg_back;
        if ((e = launch_decay_join(r, p.dfin, true, s)) != hipSuccess) return e;
    }
    w.rows = f.Dv;
    w.cols = f.Dk;
    w.rs = 1;
    w.cs = f.Dv;
    w.a = p.d_o;
    w.b = f.v;
    w.v = f.k;
    w.x = f.q;
    w.sf = w.ss = f.scale;
    w.sw = 1.f;
    w.init = f.init;
    w.seg = f.seg;
    w.out = p.dq_heads ? p.dq_heads : p.dq;
    w.wide = p.dq_heads != nullptr;
    w.clear = 1;
    w.before = p.before;
    w.dfin = p.dfin;
    w.ends = p.ends;
    const int widest = f.Dk > f.Dv ? f.Dk : f.Dv;
    if (f.sp.nseq) {
        if ((e = decay_walk_io<IO, kQueries>(w, s)) != hipSuccess) return e;
        e = widest <= 64    ? back_launch<IO, 64>(p, s)
            : widest <= 128 ? back_launch<IO, 128>(p, s)
                            : back_launch<IO, 256>(p, s);
        if (e != hipSuccess) return e;
    }
    const int C = decay_chunk(IO, widest), ks = (f.Dk + 127) / 128, vs = (f.Dv + 127) / 128;
    DecaySpans sp = f.sp;
    sp.seg_tokens = kDgChunks * C;
    sp.segs = (long long)decay_dg_units(sp.T, sp.nseq, sp.cu != nullptr, C);
    sp.per = sp.cu ? 1 : (int)(sp.T ? (sp.T + sp.seg_tokens - 1) / sp.seg_tokens : 1);
    if (sp.segs)
        hipLaunchKernelGGL(decay_dg_kernel, dim3((unsigned)(sp.segs * f.Hv)), dim3(256), 0, s, p, sp,
                           C, ks, vs, 4 * ks);
    if (f.fixed)
        hipLaunchKernelGGL(decay_dg_sum_kernel, dim3(f.Hv), dim3(256), 0, s, p.sums, sp.segs, f.Hv,
                           p.dg);
    if (p.dq_heads && w.tokens) {
        const int Hk = f.Hv / f.q.group;
        const long long n = w.tokens * Hk * f.Dk;
        const dim3 grid((unsigned)((n / 4 + 255) / 256));
        hipLaunchKernelGGL((decay_share_kernel<IO>), grid, dim3(256), 0, s, p.dq_heads, p.dq, n, f.Dk,
                           f.q.group);
        hipLaunchKernelGGL((decay_share_kernel<IO>), grid, dim3(256), 0, s, p.dk_heads, p.dk, n, f.Dk,
                           f.q.group);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decay_bwd(int io, const DecayGradParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return bwd_io<IO_F32>(p, s);
    case IO_F16: return bwd_io<IO_F16>(p, s);
    default: return bwd_io<IO_BF16>(p, s);
    }
}

}  // namespace fftconv
