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
// The walk of dq leaves S0 of every eighth chunk for A.  Between them A follows from
// the next chunk's A': A + (s in it, u behind) by all tokens = A' + (s before, u in the
// next) by all of its; it is taken as 0 where e^Dc is below 2^-22, which the terms'
// own errors reach.  A fixed decay's dg sums A over all tokens, so its errors too: it
// has S0 of every second.  (With chains to the sequence's end dg of 2 x 1501 tokens of
// one decay a head was off by 1.4e-5.)
#include "fftconv_decay_walk.h"

namespace fftconv {
namespace {

template <int IO, int DA>
struct Back {
    static constexpr int C = kDecayChunk;
    static constexpr int RW = 4;                         // waves of a role
    static constexpr int kTile = C * DA * Kind<IO>::kB;
    static constexpr int kP = Scores<IO, C>::kBytes;
    static constexpr int kBytes = 4 * kTile + 2 * kP;
};

// Scores of dk (rows of v against do) as make_scores() makes them, and the sums over
// rectangles of W: sums[unit][t] for the sixteen s and the u of the unit.
template <int IO, int DA, int C, int NW>
__device__ __forceinline__ void make_scores_and_sums(const RowReader<IO, DA>& rows, int lane,
                                                     const char* V, const char* DO, const char* K,
                                                     const char* Q, char* P, float* back,
                                                     const Factors<C>& F, float scale, int wave,
                                                     float (*sums)[C]) {
    typedef Scores<IO, C> L;
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int j = 0; j < (L::kUnits + NW - 1) / NW; ++j) {
        const int unit = wave + NW * j, qt = unit % L::M, part = unit / L::M, k0 = part * L::kTiles;
        if (NW > L::kUnits && unit >= L::kUnits) continue;
        if (k0 + L::kTiles - 1 < (qt & ~1)) {
            if (lane < C) sums[unit][lane] = 0.f;
            continue;
        }
        dfloat4 vd[L::kTiles], kq[L::kTiles];
#pragma unroll
        for (int x = 0; x < L::kTiles; ++x) vd[x] = kq[x] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DA / 32; ++kb) {
            constexpr int kTile = 16 * Rows<IO, DA>::kRow;
            const Frag<IO> b = rows.get(V + qt * kTile, 0, 32 * kb);
            const Frag<IO> b2 = rows.get(K + qt * kTile, 0, 32 * kb);
#pragma unroll
            for (int x = 0; x < L::kTiles; ++x) {
                vd[x] = mma16<IO>(rows.get(DO + k0 * kTile, 16 * x, 32 * kb), b, vd[x]);
                kq[x] = mma16<IO>(rows.get(Q + k0 * kTile, 16 * x, 32 * kb), b2, kq[x]);
            }
        }
        products_done();
        const int i = 16 * qt + c, whole = F.whole[i];
        const float rest = F.rest[i];
        float largest = 0.f, carry = 0.f;
#pragma unroll
        for (int x = L::kTiles - 1; x >= 0; --x) {
            const int s0 = 16 * (k0 + x) + 4 * g;
            float gam[4], y[4];
            decays_between<C, true>(F, s0, whole, rest, gam);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = scale * gam[e] * vd[x][e];
                vd[x][e] = s0 + e >= i ? p : 0.f;
                y[e] = s0 + e > i ? p * kq[x][e] : 0.f;
                if (IO == IO_F16) largest = fmaxf(largest, fabsf(vd[x][e]));
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
            if ((c & 3) == 0) sums[unit][s0 + (c >> 2)] = sum;
        }
        // t before and behind the unit's u
#pragma unroll
        for (int kt = 0; kt < L::M; ++kt) {
            if (kt >= k0 && kt < k0 + L::kTiles) continue;
            const int s0 = 16 * kt + 4 * g;
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = kt < k0 && s0 + e > i ? carry : 0.f;
            const float sum = sums16_of4(y);
            if ((c & 3) == 0) sums[unit][s0 + (c >> 2)] = sum;
        }
        const float to = L::scale(largest, back, lane, qt, part);
#pragma unroll
        for (int x = 0; x < L::kTiles; ++x) L::put(P, lane, qt, k0 + x, to, vd[x]);
    }
}

// dk and dv: a workgroup of two roles of RW waves each walks over a segment's
// chunks backward in time, with the gradient X of the state, columns of Dv in the
// first role's waves (dv) and, transposed, columns of Dk in the second's (dk).
//
// 64 x 1024 tokens of 6 heads of 128 in bf16 take 405 us in a trace (the walk of dq 204,
// dg 16, outputs 161; a call of the forward pass and all gradients takes 700 without one).
// Vector instructions take 58 % of the cycles, matrix instructions 22 %, and waves wait 46 %
// of their time for the chunk's barriers, LDS and loads (the walk of dq: 55, 22 and 41 %).
// With two terms of the state for dk and of scores it took 366; at that time both
// products in one role of four waves, which need 64 more state registers, took 454 with
// two waves a SIMD and 1000 with registers spilled, the chains in three rounds of half
// their length 381.
template <int IO, int DA>
__global__ __launch_bounds__(512, (DA > 128 || (IO == IO_F32 && DA > 64) ? 2 : 4)) void decay_back_kernel(DecayGradParams p,
                                                                               int slices) {
    typedef Back<IO, DA> L;
    constexpr int C = L::C, RW = L::RW, N = 128 * RW, kB = Kind<IO>::kB, kCols = 16 * RW;
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
    const int first = slice * kCols, mine = first + 16 * wave, col = mine + (lane & 15);
    const int cols = keys ? f.Dk : f.Dv, rows = keys ? f.Dv : f.Dk;
    const bool ok = col < cols, wide = p.dk_heads != nullptr;
    // what there is of the slice's columns
    const int nk = min(f.Dk - first, kCols), nv = min(f.Dv - first, kCols);
    if (s.index == 0 && f.sp.cu) {
        if (nk > 0)
            clear_unheld(f.sp, s, wide ? p.dk_heads : p.dk, wide ? 4 : kB, f.Hv, f.Dk, h, first, nk);
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
    __shared__ __attribute__((aligned(16))) Factors<C> F[8];
    __shared__ __attribute__((aligned(16))) float back[2][C / 32 * C];
    __shared__ float sums[Scores<IO, C>::kUnits][C];
    __shared__ float dots[RW][C];
    __shared__ int unbounded[2];
    __shared__ double products[RW];
    const int chunks = (s.to - s.from + C - 1) / C;
    const Tokens q = rows_of<IO>(f.q, s, h), k = rows_of<IO>(f.k, s, h), v = rows_of<IO>(f.v, s, h),
                 d = rows_of<IO>(p.d_o, s, h);
    const int kp = f.Dk * kB / 16, vp = f.Dv * kB / 16;
    const float* gates = f.fixed ? f.g + h : f.g + (s.b * f.sp.T + s.t0) * f.Hv + h;
    const long long token0 = s.b * f.sp.T + s.t0;
    const long long slot0 = f.sp.cu ? s.t0 / C + s.seq : s.b * ((f.sp.T + C - 1) / C);
    // the first token of the walk's chunk i, and its tokens
    const auto start = [&](int i) { return s.from + (chunks - 1 - i) * C; };
    const auto count = [&](int i) { return min(C, s.to - start(i)); };
    const auto log_decays = [&](int i) {
        const int n = place < 4 && i + place < chunks ? count(i + place) : 0;
        if (n <= 0) return 0.f;
        if (f.fixed) return gates[0];
        return gates[(long long)(start(i + place) + min(lane, n - 1)) * f.Hv];
    };
    const auto factors = [&](int i, float g) {
        if (place >= 4 || i + place >= chunks) return;
        put_factors<C, true>(F[(i + place) & 7], decays_to<C>(g, f.fixed, count(i + place)), 1.f,
                             f.scale);
    };
    typedef Moving<IO, DA, C, N> Move;
    Move mq, mk, mv, md;
    const int last = s.from + (chunks - 1) * C;
    Source sq = Move::source(q, last, tid), sk = Move::source(k, last, tid),
           sv = Move::source(v, last, tid), sd = Move::source(d, last, tid);
    const uint32_t piece = Move::place(tid);
    // n: tokens of the chunk
    const auto fetch = [&](int n) {
        const int lk = Move::left(tid, n, kp), lv = Move::left(tid, n, vp);
        mq.load(sq, lk);
        mk.load(sk, lk);
        mv.load(sv, lv);
        md.load(sd, lv);
        sq.p -= C * (long long)sq.stride;
        sk.p -= C * (long long)sk.stride;
        sv.p -= C * (long long)sv.stride;
        sd.p -= C * (long long)sd.stride;
    };
    const auto put = [&](int n, int* bad) {
        if (n < C || kp < Move::kPieces || vp < Move::kPieces) {
            const int lk = Move::left(tid, n, kp), lv = Move::left(tid, n, vp);
            mq.clear(lk);
            mk.clear(lk);
            mv.clear(lv);
            md.clear(lv);
        }
        mq.store(Q, piece, tid);
        mk.store(K, piece, tid);
        mv.store(V, piece, tid);
        md.store(DO, piece, tid);
        if (mq.unbounded() || md.unbounded()) *bad = 1;
    };
    const int kb = wide ? 4 : kB, p0 = first * kB / 16;
    const uint32_t krow = (uint32_t)(f.Hv * f.Dk * kb), vrow = (uint32_t)(f.Hv * f.Dv * kB);
    char* dk = (char*)(wide ? (void*)p.dk_heads : p.dk) + (token0 + last) * krow +
               (long long)(h * f.Dk + first) * kb;
    char* dv = (char*)p.dv + (token0 + last) * vrow + (long long)(h * f.Dv + first) * kB;
    Drift drift;
    float g = 0.f;
    if (chunks) {
        fetch(count(0));
        factors(0, log_decays(0));
        g = log_decays(4);
        if (tid < 2) unbounded[tid] = 0;
        __syncthreads();
        put(count(0), &unbounded[0]);
        __syncthreads();
    }
    const int tile = mine < DA ? wave + first / 16 : 0;        // columns that are in the tiles
    Places<IO, DA, DA> places(lane, 16 * tile);
    for (int i = 0; i < chunks; ++i) {
        const Factors<C>& fac = F[i & 7];
        const int at = start(i), n = count(i);
        places.fresh();
        const bool more = i + 1 < chunks;
        if ((i & 3) == 0) {
            factors(i + 4, g);
            g = log_decays(i + 8);
        }
        const bool anchor = (at / C & ((1 << p.anchor_shift) - 1)) == 0;
        if (anchor && keys) {
            double x = 0;
            if (mine < f.Dk) {
                const int tiles = 2 * ((f.Dv + 31) / 32);
                x = X.times_tiles(p.anchors +
                                      (anchor_of(f.sp, s, C, p.anchor_shift, at / C) * f.Hv + h) *
                                          p.anchor_floats +
                                      (long long)(mine / 16) * tiles * 256,
                                  tiles);
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
            if (lane == 0) products[wave] = x;
        }
        if (more) fetch(C);
        dfloat4 acc[C / 16];
        if (keys) {
            // the sums once for a head
            if (slice == 0)
                make_scores_and_sums<IO, DA, C, RW>(places.rows, places.lane, V, DO, K, Q, P, back[1],
                                                    fac, f.scale, wave, sums);
            else
                make_scores<IO, DA, C, RW, true>(places.rows, places.lane, V, DO, P, back[1], fac,
                                                 f.scale, wave);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C>(places.rows, places.lane, V, X, fac, acc);
        } else {
            make_scores<IO, DA, C, RW, true>(places.rows, places.lane, K, Q, P, back[0], fac, f.scale,
                                             wave);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C>(places.rows, places.lane, K, X, fac, acc);
            __builtin_amdgcn_sched_barrier(0);
            row_dots<IO, DA, C>(places.cells, places.lane, V, acc, dots[wave]);
        }
        __syncthreads();
        if (place == RW - 1 && nv > 0) {
            // s in the chunk before t
            double x = 0, r = 0;
            if (lane < C) {
#pragma unroll
                for (int w = 0; w < RW; ++w) x += dots[w][lane];
                if (slice == 0)
#pragma unroll
                    for (int w = 0; w < Scores<IO, C>::kUnits; ++w) r += sums[w][lane];
            }
            const double to = prefix_sum(x), all = __shfl(to, 63);
            double before = __shfl_up(to, 1);
            if (lane == 0) before = 0;
            if (lane < n)
                p.behind[((long long)slice * f.Hv + h) * p.B * f.sp.T + token0 + at + lane] =
                    (float)(before + r);
            if (lane == 0)
                p.chunks[(slice * p.slots + slot0 + at / C) * f.Hv + h] = make_double2(all, fac.all);
        }
        if (anchor && tid == 0 && nk > 0) {
            double x = 0;
#pragma unroll
            for (int w = 0; w < RW; ++w) x += products[w];
            p.anchor_dg[(slice * p.anchor_count + anchor_of(f.sp, s, C, p.anchor_shift, at / C)) *
                            f.Hv + h] = fac.all * x;
        }
        Frag<IO> val[C / 32];
#pragma unroll
        for (int j = 0; j < C / 32; ++j) val[j] = places.values.get(keys ? Q : DO, 32 * j, tile);
        scores_product<IO, C, true>(P, back[keys], places.lane, val, unbounded[i & 1], acc);
        __builtin_amdgcn_sched_barrier(0);
        // K's and V's tiles are done with
        if (keys && wide) rows_to_memory<C>(places.lane, dk + 64 * wave, krow, ok, n, acc);
        else if (mine < DA) rows_to_tile<IO, DA, C>(places.cells, keys ? V : K, acc);
        __builtin_amdgcn_sched_barrier(0);
        update_state<IO, DA, C, 2>(places.elements, places.lane, keys ? DO : Q, val, fac, X);
        drift.after(fac.err, i, !more, X);
        if (tid == 0) unbounded[(i + 1) & 1] = 0;
        __syncthreads();
        Move rows_k, rows_v;
        rows_v.take(K, piece, tid);
        rows_k.take(V, piece, tid);
        if (more) put(C, &unbounded[(i + 1) & 1]);
        // the thread's piece among the slice's columns
        const int id = fresh_thread(), at_piece = id % Move::kPieces - p0, t0 = id / Move::kPieces;
        const bool mine_k = at_piece >= 0 && at_piece < nk * kB / 16,
                   mine_v = at_piece >= 0 && at_piece < nv * kB / 16;
        rows_v.write(dv, (uint32_t)t0 * vrow + 16u * at_piece, vrow, mine_v ? n - t0 : 0, tid);
        if (!wide) rows_k.write(dk, (uint32_t)t0 * krow + 16u * at_piece, krow, mine_k ? n - t0 : 0, tid);
        dk -= C * (long long)krow;
        dv -= C * (long long)vrow;
        __syncthreads();
    }
    if (!keys && s.index == 0 && p.dinit)
        X.store(p.dinit + (s.seq * (long long)f.Hv + h) * size + at_col, rs, ok, rows);
}

// dg from its parts, kDgChunks chunks a workgroup.  Parts by columns: ks of Dk, vs of Dv.
// Its time grows with the tokens of a head as the number of workgroups does: 2^20 tokens
// of one head of 64 take 14.5 us, 32768 take 9.9.
__global__ __launch_bounds__(256) void decay_dg_kernel(DecayGradParams p, DecaySpans sp, int ks,
                                                       int vs) {
    constexpr int C = kDecayChunk;
    const DecayParams& f = p.f;
    const int h = (int)(blockIdx.x % f.Hv), lane = threadIdx.x & 63;
    const unsigned part = blockIdx.x / f.Hv;
    __shared__ double A[kDgChunks];
    __shared__ double sums[4];
    DecaySpan s;
    double sum = 0;
    const bool held = segment_of(sp, part, s);
    if (held) {
        const long long token0 = s.b * sp.T + s.t0, tokens = p.B * sp.T;
        const int nc = (s.len + C - 1) / C, mine = s.from / C;
        const long long slot0 = sp.cu ? s.t0 / C + s.seq : s.b * ((sp.T + C - 1) / C);
        if (threadIdx.x < 64) {
            // A of the workgroup's chunks, from the last one in lane 0 on
            const auto anchored = [&](int c) {
                const long long a = anchor_of(sp, s, C, p.anchor_shift, c);
                double x = 0;
                for (int i = 0; i < ks; ++i) x += p.anchor_dg[(i * p.anchor_count + a) * f.Hv + h];
                return x;
            };
            const int c = mine + kDgChunks - 1 - lane;
            double b = 0;
            int keep = 1;                       // by way of the next chunk
            if (c < nc) {
                if ((c & ((1 << p.anchor_shift) - 1)) == 0) {
                    keep = 0;
                    b = anchored(c);
                } else {
                    for (int i = 0; i < vs; ++i) {
                        const double2 x = p.chunks[(i * p.slots + slot0 + c) * f.Hv + h];
                        b -= x.x;
                        keep = x.y >= 0x1p-22;
                    }
                    if (c + 1 < nc) {
                        for (int i = 0; i < ks; ++i)
                            b += p.before_all[(i * p.slots + slot0 + c + 1) * f.Hv + h];
                    } else {
                        for (int i = 0; i < 4 * ks; ++i)
                            b += p.ends[(s.seq * (long long)f.Hv + h) * 4 * ks + i];
                    }
                    if (!keep) b = 0;
                }
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
            // the chunk behind the workgroup's has an anchor
            if (keep && mine + kDgChunks < nc) b += anchored(mine + kDgChunks);
            A[kDgChunks - 1 - lane] = b;
        }
        __syncthreads();
        for (int t = s.from + threadIdx.x; t < s.to; t += 256) {
            const long long at = token0 + t;
            double x = A[(t - s.from) / C];
            for (int i = 0; i < ks; ++i) x += p.before[((long long)i * f.Hv + h) * tokens + at];
            for (int i = 0; i < vs; ++i) x += p.behind[((long long)i * f.Hv + h) * tokens + at];
            if (f.fixed) sum += x;
            else p.dg[at * f.Hv + h] = (float)x;
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
    const int slices = (widest + kDecayCols - 1) / kDecayCols;
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
    w.before_all = p.before_all;
    w.slots = p.slots;
    w.anchor_shift = p.anchor_shift;
    w.anchors = p.anchors;
    w.anchor_floats = p.anchor_floats;
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
    const int ks = (f.Dk + kDecayCols - 1) / kDecayCols, vs = (f.Dv + kDecayCols - 1) / kDecayCols;
    DecaySpans sp = f.sp;
    sp.seg_tokens = kDgChunks * kDecayChunk;
    sp.segs = (long long)decay_dg_units(sp.T, sp.nseq, sp.cu != nullptr);
    sp.per = sp.cu ? 1 : (int)(sp.T ? (sp.T + sp.seg_tokens - 1) / sp.seg_tokens : 1);
    if (sp.segs)
        hipLaunchKernelGGL(decay_dg_kernel, dim3((unsigned)(sp.segs * f.Hv)), dim3(256), 0, s, p, sp,
                           ks, vs);
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
