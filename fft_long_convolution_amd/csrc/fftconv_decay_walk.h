// The walk of linear attention forward in time: the outputs, the gradients of the
// queries (the same with other rows in the places of q, k and v), and what a
// segment does to the state.  See fftconv_decay_dev.h for the mathematics.
#pragma once

#include "fftconv_decay_dev.h"

namespace fftconv {

struct DecayWalk {
    DecaySpans sp;
    int Hv, rows, cols;              // heads; elements of a and b, columns of v
    int slices;                      // workgroups that share a head's columns
    bool fixed;
    const float* g;
    DecayRows a, b, v;
    float sf, ss, sw;                // factors of the state's product, scores, values
    // states: element e and column c of a head at e * rs + c * cs
    long long rs, cs;
    const float* init;               // [nseq][Hv] states or null
    float* seg;                      // [segs][Hv] states, or null for one segment each
    double* seg_g;
    float* fin;                      // [nseq][Hv] or null
    void* out;                       // [B][T][Hv][cols]
    bool wide;                       // of fp32 whatever the rows' type
    int clear;
    // gradients of queries: the queries themselves, what their part with the state
    // owes (before), and the last state's part of <d final state, final state>
    DecayRows x;
    float* before;                   // [slices][Hv][B T]
    long long tokens;                // B T
    const float* dfin;
    float* ends;                     // [nseq][Hv][4 slices]
};

enum WalkMode { kOutputs, kEffects, kEffectsBack, kQueries };

template <int IO, int DA, int C, int W, int MODE>
struct WalkLds {
    static constexpr int kB = Kind<IO>::kB;
    static constexpr bool kOut = MODE == kOutputs || MODE == kQueries;
    static constexpr int kA = kOut ? C * DA * kB : 0, kBm = C * DA * kB, kV = C * 32 * W * kB;
    static constexpr int kP = kOut ? Scores<IO, C>::kBytes : 0;
    static constexpr int kX = MODE == kQueries ? kV : 0;
    static constexpr int kAtB = kA, kAtV = kAtB + kBm, kAtP = kAtV + kV, kAtX = kAtP + kP;
    static constexpr int kBytes = kAtX + kX;
};

template <int IO, int DA, int C, int W, int MODE>
__global__ __launch_bounds__(64 * W, DA > 128 || (DA == 128 && W == 2) ? 1 : 2) void decay_walk_kernel(DecayWalk p) {
    typedef WalkLds<IO, DA, C, W, MODE> L;
    constexpr int N = 64 * W, kB = Kind<IO>::kB;
    constexpr bool OUT = L::kOut, REV = MODE == kEffectsBack, DOT = MODE == kQueries;
    const unsigned units = (unsigned)(p.sp.segs * p.Hv * p.slices), u = xcd_unit(blockIdx.x, units);
    if (u >= units) return;
    const int slice = (int)(u % p.slices), h = (int)(u / p.slices % p.Hv);
    const unsigned seg = u / p.slices / p.Hv;
    DecaySpan s;
    if (!segment_of(p.sp, seg, s)) return;
    if (MODE == kEffects && s.last) return;
    if (MODE == kEffectsBack && s.index == 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int first = slice * 32 * W, col = first + 32 * wave + (lane & 31);
    const bool ok = col < p.cols;
    const int here = p.cols - first < 32 * W ? p.cols - first : 32 * W;
    if (OUT && p.clear && s.index == 0 && p.sp.cu) {
        // tokens before the first sequence and behind the last
        clear_unheld(p.sp, s, p.out, DOT && p.wide ? 4 : kB, p.Hv, p.cols, h, first, here);
    }
    const long long size = (long long)p.rows * p.cols;
    State<DA> S;
    S.clear();
    if (OUT) {
        if (p.seg) S.load(p.seg + (seg * (long long)p.Hv + h) * size + (ok ? col * p.cs : 0), p.rs, ok, p.rows);
        else if (p.init)
            S.load(p.init + (s.seq * (long long)p.Hv + h) * size + (ok ? col * p.cs : 0), p.rs, ok, p.rows);
    }

    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* A = lds;
    char* B = lds + L::kAtB;
    char* V = lds + L::kAtV;
    char* P = lds + L::kAtP;
    __shared__ __attribute__((aligned(16))) Factors<C> F[2];
    __shared__ __attribute__((aligned(16))) float back[C];
    const int chunks = (s.to - s.from + C - 1) / C;
    const Tokens a = rows_of<IO>(p.a, s, h), b = rows_of<IO>(p.b, s, h), v = rows_of<IO>(p.v, s, h);
    const int pieces = p.rows * kB / 16, vpieces = here * kB / 16;
    const long long vcol = (long long)first * kB;
    const Tokens vs = {v.base + vcol, v.bytes};
    const float* gates = p.fixed ? p.g + h : p.g + (s.b * p.sp.T + s.t0) * p.Hv + h;
    const auto log_decay = [&](int at, int n) {
        return p.fixed ? gates[0] : gates[(long long)(at + (lane < n ? lane : n - 1)) * p.Hv];
    };
    double sum = 0;
    Moving<IO, DA, C, N> ma, mb;
    Moving<IO, 32 * W, C, N> mv, mx;
    Tokens x = vs;
    if (DOT) {
        x = rows_of<IO>(p.x, s, h);
        x.base += vcol;
    }
    __shared__ float dots[DOT ? W : 1][DOT ? C : 1];
    const auto fetch = [&](int at, int n) {
        if (OUT) ma.load(a, at, n, pieces, tid);
        mb.load(b, at, n, pieces, tid);
        mv.load(vs, at, n, vpieces, tid);
        if (DOT) mx.load(x, at, n, vpieces, tid);
    };
    const auto put = [&](Factors<C>& f, int n) {
        if (OUT) ma.clear(n, pieces, tid);
        mb.clear(n, pieces, tid);
        mv.clear(n, vpieces, tid);
        if (DOT) mx.clear(n, vpieces, tid);
        if (OUT) ma.store(A, tid);
        mb.store(B, tid);
        mv.store(V, tid);
        if (DOT) mx.store(lds + L::kAtX, tid);
        if (OUT && mv.unbounded()) f.unbounded = 1;
    };
    const auto factors = [&](Factors<C>& f, float g, int n) {
        const double D = decays_to<C>(g, p.fixed, n);
        put_factors<C, REV>(f, D, p.sf, p.sw);
        sum += __shfl(D, C - 1);
        if (lane == 0) f.unbounded = 0;
    };
    if (chunks) {
        const int at = s.from, n = s.to - at < C ? s.to - at : C;
        fetch(at, n);
        if (wave == 0) factors(F[0], log_decay(at, n), n);
        __syncthreads();
        put(F[0], n);
        __syncthreads();
    }
    for (int ch = 0; ch < chunks; ++ch) {
        const Factors<C>& f = F[ch & 1];
        const int at = s.from + ch * C, n = s.to - at < C ? s.to - at : C;
        const bool more = ch + 1 < chunks;
        const int next = more ? at + C : at, m = s.to - next < C ? s.to - next : C;
        float g = 0.f;
        if (more) {
            fetch(next, m);
            if (wave == 0) g = log_decay(next, m);
        }
        dfloat16 acc[C / 32];
        if (OUT) {
            make_scores<IO, DA, C, W, false>(A, B, P, back, f, p.ss, wave);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C, IO == IO_BF16 && !DOT ? 2 : Kind<IO>::NS>(A, S, f, acc);
            __builtin_amdgcn_sched_barrier(0);
            if (DOT) row_dots<IO, 32 * W, C>(lds + L::kAtX, 32 * wave, acc, dots[wave]);
            __syncthreads();
        }
        if (DOT && wave == 0) {
            // from the chunk's last token on
            double d = 0;
            if (lane < C)
#pragma unroll
                for (int w = 0; w < W; ++w) d += dots[w][C - 1 - lane];
            d = prefix_sum(d);
            const int t = C - 1 - lane;
            if (t >= 0 && t < n)
                p.before[((long long)slice * p.Hv + h) * p.tokens + s.b * p.sp.T + s.t0 + at + t] = (float)d;
        }
        Frag<IO> vf[C / 16];
        const ColReader<IO, 32 * W, false> vcols(fresh_lane());
#pragma unroll
        for (int kb = 0; kb < C / 16; ++kb) vf[kb] = vcols.get(V, 16 * kb, 32 * wave);
        if (OUT) {
            scores_product<IO, C, false>(P, back, vf, f.unbounded, acc);
            __builtin_amdgcn_sched_barrier(0);
            const bool wide = DOT && p.wide;
            const int ob = wide ? 4 : kB;
            const long long row = (long long)p.Hv * p.cols * ob;
            store_rows<IO, 32 * W, C>(
                V, 32 * wave, acc,
                (char*)p.out + (s.b * p.sp.T + s.t0 + at) * row + (long long)(h * p.cols + first + 32 * wave) * ob,
                row, (here - 32 * wave) * ob / 16, wide, n);
        }
        __builtin_amdgcn_sched_barrier(0);
        update_state<IO, DA, C>(B, vf, f, S);
        if (wave == 0 && more) factors(F[(ch + 1) & 1], g, m);
        __syncthreads();
        if (more) put(F[(ch + 1) & 1], m);
        __syncthreads();
    }
    if (OUT) {
        if (s.last && p.fin)
            S.store(p.fin + (s.seq * (long long)p.Hv + h) * size + col * p.cs, p.rs, ok, p.rows);
        if (DOT && s.last) {
            double d = 0;
            if (p.dfin) {
                const float* df = p.dfin + (s.seq * (long long)p.Hv + h) * size + col * p.cs;
#pragma unroll
                for (int i = 0; i < DA / 32; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int e = State<DA>::element(i, r, lane >> 5);
                        if (ok && e < p.rows) d += (double)df[e * p.rs] * S.t[i][r];
                    }
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) d += __shfl_xor(d, m);
            if (lane < 4 / W)
                p.ends[(s.seq * (long long)p.Hv + h) * 4 * p.slices + 4 * slice + wave + W * lane] =
                    lane ? 0.f : (float)d;
        }
    } else {
        S.store(p.seg + (seg * (long long)p.Hv + h) * size + col * p.cs, p.rs, ok, p.rows);
        if (slice == 0 && tid == 0) p.seg_g[seg * (long long)p.Hv + h] = sum;
    }
}

template <int IO, int DA, int C, int W, int MODE>
hipError_t decay_walk_launch(const DecayWalk& p, hipStream_t s) {
    constexpr int bytes = WalkLds<IO, DA, C, W, MODE>::kBytes;
    const auto kernel = decay_walk_kernel<IO, DA, C, W, MODE>;
    const hipError_t e = hipFuncSetAttribute((const void*)kernel,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    DecayWalk w = p;
    w.slices = (p.cols + 32 * W - 1) / (32 * W);
    const long long units = p.sp.segs * p.Hv * w.slices;
    hipLaunchKernelGGL(kernel, dim3((unsigned)xcd_blocks(units)), dim3(64 * W), bytes, s, w);
    return hipGetLastError();
}
template <int IO, int DA, int MODE>
hipError_t decay_walk_cols(const DecayWalk& p, hipStream_t s) {
    constexpr int C = IO == IO_F32 || DA > 128 ? 32 : 64;
    // the chunks of the gradients' other walk, which has wide rows then
    if constexpr (MODE == kQueries && C == 64)
        if (p.cols > 128) return decay_walk_launch<IO, DA, 32, 4, MODE>(p, s);
    // two waves where four would have nothing to do
    return p.cols <= 64 ? decay_walk_launch<IO, DA, C, 2, MODE>(p, s)
                        : decay_walk_launch<IO, DA, C, 4, MODE>(p, s);
}
template <int IO, int MODE>
hipError_t decay_walk_io(const DecayWalk& p, hipStream_t s) {
    return p.rows <= 64    ? decay_walk_cols<IO, 64, MODE>(p, s)
           : p.rows <= 128 ? decay_walk_cols<IO, 128, MODE>(p, s)
                           : decay_walk_cols<IO, 256, MODE>(p, s);
}

}  // namespace fftconv
