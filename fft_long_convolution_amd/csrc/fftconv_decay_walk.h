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
    double* before_all;              // [slices][slots][Hv]
    long long slots;
    double* ends;                    // [nseq][Hv][slices][4]
    int anchor_shift;
    float* anchors;
    long long anchor_floats;         // of a head's anchor
};

enum WalkMode { kOutputs, kEffects, kEffectsBack, kQueries };

template <int IO, int DA, int C, int W, int MODE>
struct WalkLds {
    static constexpr int kB = Kind<IO>::kB;
    static constexpr bool kOut = MODE == kOutputs || MODE == kQueries;
    static constexpr int kA = kOut ? C * DA * kB : 0, kBm = C * DA * kB, kV = C * 16 * W * kB;
    static constexpr int kP = kOut ? Scores<IO, C>::kBytes : 0;
    static constexpr int kX = MODE == kQueries ? kV : 0;
    static constexpr int kAtB = kA, kAtV = kAtB + kBm, kAtP = kAtV + kV, kAtX = kAtP + kP;
    static constexpr int kBytes = kAtX + kX;
};

// Waves of a SIMD that the walk leaves registers for.
template <int IO, int DA>
constexpr int kWalkWaves = DA > 128 ? 2 : DA > 64 ? (IO == IO_F32 ? 2 : 3) : 4;

// A workgroup takes 16 W columns of a segment of one head.  A chunk goes in two
// halves: scores and the state's product (with A and B), then what has V in it; the
// rows of the next chunk are on their way in registers all the time, and go to LDS
// when the chunk is done, where its outputs, brought to V's place, come out.
//
// 64 x 1024 tokens of 6 heads of 128 in bf16 take 150 us, 428 MB or 2.9 TB/s.  By the
// counters vector instructions take 59 % of the cycles (490 for 58 matrix instructions
// of a wave and chunk: terms of the state, factors, addresses), matrix instructions 28 %,
// and waves wait 31 % of their time, at the chunk's three barriers and for LDS: the tiles
// are there once, so a chunk's rows go in when the one before is done.  With two bf16
// terms of states and scores, 17 bits, it took 134.  Then chunks of 64 tokens on tiles of
// 32 x 32 took 154, eight waves of 16 columns no less; with chunks of 32 the scores
// outside the triangle are few and three workgroups share a CU.
template <int IO, int DA, int C, int W, int MODE>
__global__ __launch_bounds__(64 * W, (kWalkWaves<IO, DA>)) void decay_walk_kernel(DecayWalk p) {
    typedef WalkLds<IO, DA, C, W, MODE> L;
    constexpr int N = 64 * W, kB = Kind<IO>::kB, kCols = 16 * W;
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
    const int first = slice * kCols, col = first + 16 * wave + (lane & 15);
    const bool ok = col < p.cols, wide = DOT && p.wide;
    const int here = p.cols - first < kCols ? p.cols - first : kCols;
    if (OUT && p.clear && s.index == 0 && p.sp.cu) {
        // tokens before the first sequence and behind the last
        clear_unheld(p.sp, s, p.out, wide ? 4 : kB, p.Hv, p.cols, h, first, here);
    }
    const long long size = (long long)p.rows * p.cols, at_col = ok ? col * p.cs : 0;
    State<DA> S;
    S.clear();
    if (OUT) {
        if (p.seg) S.load(p.seg + (seg * (long long)p.Hv + h) * size + at_col, p.rs, ok, p.rows);
        else if (p.init)
            S.load(p.init + (s.seq * (long long)p.Hv + h) * size + at_col, p.rs, ok, p.rows);
    }

    extern __shared__ __attribute__((aligned(16))) char lds[];
    char* const A = lds;
    char* const B = lds + L::kAtB;
    char* const V = lds + L::kAtV;
    char* const P = lds + L::kAtP;
    __shared__ __attribute__((aligned(16))) Factors<C> F[8];
    __shared__ __attribute__((aligned(16))) float back[C / 32 * C];
    __shared__ float dots[DOT ? W : 1][DOT ? C : 1];
    __shared__ int unbounded[2];
    __shared__ double sums[4];
    const int chunks = (s.to - s.from + C - 1) / C;
    const Tokens a = rows_of<IO>(p.a, s, h), b = rows_of<IO>(p.b, s, h), v = rows_of<IO>(p.v, s, h);
    const int pieces = p.rows * kB / 16, vpieces = here * kB / 16;
    const Tokens vs = {v.base + first * kB, v.bytes};
    Tokens x = vs;
    if (DOT) {
        x = rows_of<IO>(p.x, s, h);
        x.base += first * kB;
    }
    const float* gates = p.fixed ? p.g + h : p.g + (s.b * p.sp.T + s.t0) * p.Hv + h;
    // the first token of chunk number i of the walk in the segment, and its tokens
    const auto start = [&](int i) { return (REV ? chunks - 1 - i : i) * C; };
    const auto count = [&](int i) { return i < chunks ? min(C, s.to - s.from - start(i)) : 0; };
    double sum = 0;
    // of chunks i .. i + 3, by the first four waves
    const auto log_decays = [&](int i) {
        const int n = wave < 4 ? count(i + wave) : 0;
        if (n <= 0) return 0.f;
        if (p.fixed) return gates[0];
        return gates[(long long)(s.from + start(i + wave) + min(lane, n - 1)) * p.Hv];
    };
    const auto factors = [&](int i, float g) {
        const int n = wave < 4 ? count(i + wave) : 0;
        if (n <= 0) return;
        const double D = decays_to<C>(g, p.fixed, n);
        put_factors<C, REV>(F[(i + wave) & 7], D, p.sf, p.sw);
        if (!OUT) sum += __shfl(D, C - 1);
    };
    typedef Moving<IO, DA, C, N> MoveA;
    typedef Moving<IO, kCols, C, N> MoveV;
    MoveA ma, mb;
    MoveV mv, mx, mo;
    const long long token = s.from + (chunks ? start(0) : 0);
    Source sa = MoveA::source(a, token, tid), sb = MoveA::source(b, token, tid),
           sv = MoveV::source(vs, token, tid), sx = MoveV::source(x, token, tid);
    const uint32_t pa = MoveA::place(tid), pv = MoveV::place(tid);
    const bool aligned = pieces >= MoveA::kPieces && vpieces >= MoveV::kPieces;
    // n: tokens of the chunk
    const auto fetch = [&](int n) {
        const int la = MoveA::left(tid, n, pieces), lv = MoveV::left(tid, n, vpieces);
        if (OUT) ma.load(sa, la);
        mb.load(sb, la);
        mv.load(sv, lv);
        if (DOT) mx.load(sx, lv);
        constexpr long long kOn = REV ? -C : C;
        sa.p += kOn * sa.stride;
        sb.p += kOn * sb.stride;
        sv.p += kOn * sv.stride;
        if (DOT) sx.p += kOn * sx.stride;
    };
    const auto put = [&](int n, int* bad) {
        if (n < C || !aligned) {
            const int la = MoveA::left(tid, n, pieces), lv = MoveV::left(tid, n, vpieces);
            if (OUT) ma.clear(la);
            mb.clear(la);
            mv.clear(lv);
            if (DOT) mx.clear(lv);
        }
        if (OUT) ma.store(A, pa, tid);
        mb.store(B, pa, tid);
        mv.store(V, pv, tid);
        if (DOT) mx.store(lds + L::kAtX, pv, tid);
        if (OUT && mv.unbounded()) *bad = 1;
    };
    const int ob = wide ? 4 : kB;
    const uint32_t row = (uint32_t)(p.Hv * p.cols * ob);
    char* out = (char*)p.out + (s.b * p.sp.T + s.t0 + s.from) * row +
                (long long)(h * p.cols + first) * ob;
    const uint32_t omine = tid / MoveV::kPieces * row + 16u * (tid % MoveV::kPieces);
    Places<IO, DA, kCols> at(lane, 16 * wave);
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
    for (int i = 0; i < chunks; ++i) {
        const Factors<C>& f = F[i & 7];
        const int n = count(i), ahead = count(i + 1);
        at.fresh();
        if ((i & 3) == 0) {
            factors(i + 4, g);
            g = log_decays(i + 8);
        }
        if (DOT) {
            const int chunk = s.from / C + i;
            if ((chunk & ((1 << p.anchor_shift) - 1)) == 0 && first + 16 * wave < p.cols) {
                const int tiles = 2 * ((p.rows + 31) / 32);
                S.store_tiles(p.anchors +
                                  (anchor_of(p.sp, s, C, p.anchor_shift, chunk) * p.Hv + h) *
                                      p.anchor_floats +
                                  (long long)(first / 16 + wave) * tiles * 256,
                              tiles);
            }
        }
        if (ahead) fetch(ahead);
        dfloat4 acc[C / 16];
        if (OUT) {
            make_scores<IO, DA, C, W, false>(at.rows, at.lane, A, B, P, back, f, p.ss, wave);
            __builtin_amdgcn_sched_barrier(0);
            state_product<IO, DA, C>(at.rows, at.lane, A, S, f, acc);
            __builtin_amdgcn_sched_barrier(0);
            if (DOT) row_dots<IO, kCols, C>(at.cells, at.lane, lds + L::kAtX, acc, dots[wave]);
            __syncthreads();
        }
        if (DOT && wave == W - 1) {
            // from the chunk's last token on
            double d = 0;
            if (lane < C)
#pragma unroll
                for (int w = 0; w < W; ++w) d += dots[w][C - 1 - lane];
            d = prefix_sum(d);
            const int t = C - 1 - lane;
            if (t == 0) {
                const long long slot0 = p.sp.cu ? s.t0 / C + s.seq : s.b * ((p.sp.T + C - 1) / C);
                p.before_all[(slice * p.slots + slot0 + s.from / C + i) * p.Hv + h] = d;
            }
            if (t >= 0 && t < n)
                p.before[((long long)slice * p.Hv + h) * p.tokens + s.b * p.sp.T + s.t0 + s.from +
                         i * C + t] = (float)d;
        }
        Frag<IO> vf[C / 32];
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) vf[kb] = at.values.get(V, 32 * kb, wave);
        if (OUT) {
            scores_product<IO, C, false>(P, back, at.lane, vf, unbounded[i & 1], acc);
            __builtin_amdgcn_sched_barrier(0);
            if (wide) rows_to_memory<C>(at.lane, out + 64 * wave, row, ok, n, acc);
            else rows_to_tile<IO, kCols, C>(at.cells, V, acc);
        }
        __builtin_amdgcn_sched_barrier(0);
        update_state<IO, DA, C, 4>(at.elements, at.lane, B, vf, f, S);
        drift.after(f.err, i, ahead == 0, S);
        if (tid == 0) unbounded[(i + 1) & 1] = 0;
        __syncthreads();
        if (OUT && !wide) mo.take(V, pv, tid);
        if (ahead) put(ahead, &unbounded[(i + 1) & 1]);
        if (OUT && !wide) mo.write(out, omine, row, MoveV::left(tid, n, vpieces), tid);
        out += C * (long long)row;
        __syncthreads();
    }
    if (OUT) {
        if (s.last && p.fin)
            S.store(p.fin + (s.seq * (long long)p.Hv + h) * size + at_col, p.rs, ok, p.rows);
        if (DOT && s.last) {
            double d = 0;
            if (p.dfin) {
                const float* df = p.dfin + (s.seq * (long long)p.Hv + h) * size + at_col;
#pragma unroll
                for (int i = 0; i < State<DA>::N; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int e = State<DA>::element(i, r, lane >> 4);
                        if (ok && e < p.rows) d += (double)df[e * p.rs] * S.t[i][r];
                    }
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) d += __shfl_xor(d, m);
            if (lane == 0)
                p.ends[((s.seq * (long long)p.Hv + h) * p.slices + slice) * W + wave] = d;
        }
    } else {
        S.store(p.seg + (seg * (long long)p.Hv + h) * size + at_col, p.rs, ok, p.rows);
        if (slice == 0) {
            if (lane == 0 && wave < 4) sums[wave] = sum;
            __syncthreads();
            if (tid == 0)
                p.seg_g[seg * (long long)p.Hv + h] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        }
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
    w.slices = (p.cols + 16 * W - 1) / (16 * W);
    const long long units = p.sp.segs * p.Hv * w.slices;
    hipLaunchKernelGGL(kernel, dim3((unsigned)xcd_blocks(units)), dim3(64 * W), bytes, s, w);
    return hipGetLastError();
}
template <int IO, int MODE>
hipError_t decay_walk_io(const DecayWalk& p, hipStream_t s) {
    return p.rows <= 64    ? decay_walk_launch<IO, 64, kDecayChunk, 4, MODE>(p, s)
           : p.rows <= 128 ? decay_walk_launch<IO, 128, kDecayChunk, 4, MODE>(p, s)
                           : decay_walk_launch<IO, 256, kDecayChunk, 4, MODE>(p, s);
}

}  // namespace fftconv
