// The gated delta rule, forward: one token against a pool of states, and
// whole sequences in chunks.
//
// A value head h keeps a state S (Dk x Dv).  A token with key k, value v,
// query q, log decay g and write strength beta does
//   S <- a S,  a = e^g
//   u  = beta (v - S^T k)          what the key should read, less what it does
//   S <- S + k u^T,   o = scale S^T q
//
// In a chunk of 64 tokens, with G_i the sum of the log decays up to token i,
// S0 the chunk's first state and Gam_ij = e^(G_i - G_j), j <= i:
//   A_ij = beta_i Gam_ij k_i.k_j  (j < i),  T = (I + A)^-1
//   X = V - e^G o (K S0),  U = T (beta o X)
//   O = scale e^G o (Q S0) + P U,  P_ij = scale Gam_ij q_i.k_j
//   S1 = e^Gc S0 + K^T (e^(Gc-G) o U)
// T and P need no state: delta_prep_kernel makes them for all chunks at
// once.  delta_scan_kernel then walks over a sequence's chunks.
#include "fftconv_delta_dev.h"

namespace fftconv {
namespace {

// ------------------------------------------------------------ one token

// A workgroup takes 32 columns of one state: 8 lanes x 4 columns, 32 row
// groups of R rows, all in registers.  S^T k and S^T q are summed in one
// pass over the old state, for o = scale (a S^T q + (q.k) u) needs no second
// one: each state is read and written once, and HBM bounds the call (192
// requests x 8 heads of 128 x 128: 203 MB in 32 us, 6.3 TB/s, what a streaming
// copy reaches; one request: 4 us, a launch).  All arithmetic is fp32, o is
// rounded once.
template <int IO, int R>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
    const int tiles = (p.Dv + 31) / 32;
    unsigned id = blockIdx.x;
    const int tile = (int)(id % tiles);
    id /= tiles;
    const int h = (int)(id % p.Hv);
    const long long n = id / p.Hv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = tile * 32 + 4 * (lane & 7);
    const int row0 = (wave * 8 + (lane >> 3)) * R;
    const bool cok = col < p.Dv;
    const long long slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.pool) {
        // no state: a row of padding
        if (threadIdx.x < 32 && tile * 32 + threadIdx.x < p.Dv)
            io_store<IO>(p.o, (n * p.Hv + h) * p.Dv + tile * 32 + threadIdx.x, 0.f);
        return;
    }
    const long long at = (slot * p.Hv + h) * p.Dk * (long long)p.Dv + col;
    float* S = p.state + at;
    const int hk = h / (p.Hv / p.Hk);
    float4 s[R];
    float k[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool ok = row0 + i < p.Dk;
        float x[4];
        load4<IO_F32>(p.state, at + (long long)(row0 + i) * p.Dv, cok && ok, x);
        s[i] = make_float4(x[0], x[1], x[2], x[3]);
        k[i] = io_load_if<IO>(p.k, n * p.ks[0] + hk * p.ks[1] + row0 + i, ok);
        q[i] = io_load_if<IO>(p.q, n * p.qs[0] + hk * p.qs[1] + row0 + i, ok);
    }
    const float a = expf(p.g[n * p.Hv + h]), beta = p.beta[n * p.Hv + h];
    float v[4];
    load4<IO>(p.v, n * p.vs[0] + h * p.vs[1] + col, cok, v);
    // sums over the rows: S^T k, S^T q (four columns each) and q.k
    float r[9] = {0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float x[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            r[j] += k[i] * x[j];
            r[4 + j] += q[i] * x[j];
        }
        r[8] += q[i] * k[i];
    }
#pragma unroll
    for (int j = 0; j < 9; ++j) r[j] = sum_groups(r[j] + row_ror<8>(r[j]));
    __shared__ float sums[4][8][9];
    if (lane < 8)
#pragma unroll
        for (int j = 0; j < 9; ++j) sums[wave][lane][j] = r[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 9; ++j)
        r[j] = (sums[0][lane & 7][j] + sums[1][lane & 7][j]) +
               (sums[2][lane & 7][j] + sums[3][lane & 7][j]);
    if (!cok) return;
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        u[j] = beta * (v[j] - a * r[j]);
    if (row0 == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            io_store<IO>(p.o, (n * p.Hv + h) * p.Dv + col + j,
                         p.scale * (a * r[4 + j] + r[8] * u[j]));
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (row0 + i < p.Dk)
            *(float4*)(S + (long long)(row0 + i) * p.Dv) =
                make_float4(a * s[i].x + k[i] * u[0], a * s[i].y + k[i] * u[1],
                            a * s[i].z + k[i] * u[2], a * s[i].w + k[i] * u[3]);
}

// ------------------------------------- what a chunk needs before its state

__device__ __forceinline__ dfloat4 mma_f32(float a, float b, dfloat4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Turns the strict lower triangle a (64 x 64 in LDS) into t = (I + a)^-1 by
// halves: 16 x 16 diagonal blocks by forward substitution (a lane a column),
// then [T11 0; -T22 A21 T11 T22] for 32 and 64, on the fp32 matrix cores.
// Above the diagonal t is 0 within 32 x 32 blocks and not written beyond.  The
// four waves of the workgroup call it together; returns the largest magnitude
// of what the lane made.
__device__ float invert_unit_lower(const float (*a)[kLd], float (*t)[kLd]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    float big = 1.f;                         // the diagonal
    {
        const int o = 16 * wave;
        if (!(wave & 1))                     // the block to the right
            *(float4*)&t[o + (lane >> 2)][o + 16 + 4 * (lane & 3)] = make_float4(0, 0, 0, 0);
        if (lane < 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // four sums side by side: each step waits for the one before
                float s[4] = {i == c ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int l = 0; l < i; ++l)
                    s[(i - 1 - l) & 3] = fmaf(-a[o + i][o + l], x[l], s[(i - 1 - l) & 3]);
                x[i] = (s[3] + s[2]) + (s[1] + s[0]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                t[o + i][o + c] = x[i];
                big = fmaxf(big, fabsf(x[i]));
            }
        }
    }
    __syncthreads();
    if (wave < 2) {
        const int o = 32 * wave;
        dfloat4 m = {0, 0, 0, 0}, r = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 4; ++s)
            m = mma_f32(a[o + 16 + c][o + 4 * s + g], t[o + 4 * s + g][o + c], m);
        // the lane's rows 4g + s of m are the k of step s
#pragma unroll
        for (int s = 0; s < 4; ++s) r = mma_f32(t[o + 16 + c][o + 16 + 4 * g + s], m[s], r);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            t[o + 16 + 4 * g + s][o + c] = -r[s];
            big = fmaxf(big, fabsf(r[s]));
        }
    }
    __syncthreads();
    {
        const int col = 16 * (wave & 1), row = 32 + 16 * (wave >> 1);
        dfloat4 m[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, r = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                m[i] = mma_f32(a[32 + 16 * i + c][4 * s + g], t[4 * s + g][col + c], m[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int s = 0; s < 4; ++s)
                r = mma_f32(t[row + c][32 + 16 * i + 4 * g + s], m[i][s], r);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            t[row + 4 * g + s][col + c] = -r[s];
            big = fmaxf(big, fabsf(r[s]));
        }
    }
    return big;
}

// Writes a lower triangle from LDS as two terms in operand order: tile (m, kb),
// lane (g, c), element i holds [tile_row(m, c)][32 kb + 8 g + i].  Rows are
// multiplied with their scale.
__device__ __forceinline__ void store_tri(const float (*t)[kLd], const float* scale, uint4* dst) {
    for (int i = threadIdx.x; i < kTriTiles * 64; i += blockDim.x) {
        const int tile = i >> 6, l = i & 63;
        const int m = tile < 2 ? tile : 2 + ((tile - 2) >> 1);
        const int kb = tile < 2 ? 0 : (tile - 2) & 1;
        const int row = tile_row(m, l & 15);
        const float* s = &t[row][32 * kb + 8 * (l >> 4)];
        const float4 a = *(const float4*)s, b = *(const float4*)(s + 4);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint4 w[2];
        split8h<2>(x, scale[row], w);
#pragma unroll
        for (int j = 0; j < 2; ++j) dst[j * kTerm + i] = w[j];
    }
}
// The same triangle's transpose, an upper one: tile (m, kb), kb >= m / 2.
__device__ __forceinline__ void store_tri_transposed(const float (*t)[kLd], const float* scale,
                                                     uint4* dst) {
    for (int i = threadIdx.x; i < kTriTiles * 64; i += blockDim.x) {
        const int tile = i >> 6, l = i & 63;
        const int m = tile < 4 ? tile >> 1 : tile - 2;
        const int kb = tile < 4 ? tile & 1 : 1;
        const int col = tile_row(m, l & 15), row = 32 * kb + 8 * (l >> 4);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = t[row + j][col];
        uint4 w[2];
        split8h<2>(x, scale[col], w);
#pragma unroll
        for (int j = 0; j < 2; ++j) dst[j * kTerm + i] = w[j];
    }
}

template <int IO, int DK>
struct PrepLds {
    static constexpr int NT = IO == IO_F32 ? 3 : 1;                 // plain terms
    static constexpr int kRows = NT * 4 * (DK / 32) * 64;           // uint4
    static constexpr int kMat = kChunk * kLd / 4;
    static constexpr int kBytes = 32 * (kRows > kMat ? kRows : kMat);
};
// One workgroup of four waves per chunk and value head: a wave makes 16 rows of
// K K^T and Q K^T (16-bit operands exact, fp32 in three bf16 terms), the decays
// turn them into A and P, then T is made from A in LDS.  Writes T, P and the
// chunk's factors as the walk takes them, 27 KB for the 32 KB of keys and queries
// of a chunk at D_k = 128 in bf16.  It is latency, of barriers, LDS (31 % of its
// cycles bank conflicts) and the substitution's 16 steps, that other workgroups of
// the CU only partly fill: 64 x 1024 tokens of 6 heads of 128 in bf16, 6144
// workgroups, take 100 to 110 us (0.36 GB), with the transposes for the backward
// pass 125 to 145 (0.53 GB).  (The
// bound of two workgroups a CU keeps the compiler from accumulating in registers
// apart, which cost it 290 moves in 1460 instructions.)
template <int IO, int DK>
__global__ __launch_bounds__(256, 2) void delta_prep_kernel(DeltaParams p) {
    typedef PrepLds<IO, DK> L;
    constexpr int NT = L::NT, KB = DK / 32;
    const unsigned units = (unsigned)p.slots * p.Hv, u = xcd_unit(blockIdx.x, units);
    if (u >= units) return;
    const unsigned slot = u / p.Hv;
    const int h = (int)(u - slot * p.Hv);
    const long long id = u;
    const unsigned seq = seq_of(p, slot, 1);
    const Span sp = span_of(p, seq);
    const long long at = ((long long)slot - sp.slot0) * kChunk;
    if (p.clear)
        unheld_tokens(p, sp, seq, slot, [&](long long token, int rows) {
            constexpr int kB = Io<IO>::kB;
            clear_rows((char*)p.o + (token * p.Hv + h) * p.Dv * kB, (long long)p.Hv * p.Dv * kB,
                       rows, p.Dv * kB);
        });
    if (at < 0 || at >= sp.len) return;      // a slot between two sequences
    const int n = (int)(sp.len - at < kChunk ? sp.len - at : kChunk);
    const long long tok = sp.t0 + at;

    // keys and queries first, then the 64 x 64 matrices
    extern __shared__ uint4 lds[];
    float (*A)[kLd] = (float (*)[kLd])lds;
    float (*P)[kLd] = A + kChunk;
    __shared__ double G[kChunk];
    __shared__ float bet[kChunk], rowp[kChunk], colp[kChunk];
    __shared__ uint32_t big[4][kChunk];      // largest of K, Q, columns of P, T
    __shared__ float spoil[kChunk];          // NaN for a token with a score that is not finite
    __shared__ int spoilt;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g4 = lane >> 4, rslot = 16 * g4 + (c ^ (4 * g4));
    const int hk = h / p.group;
    big[wave][lane] = 0;
    if (wave == 1) spoil[lane] = 0.f;
    if (threadIdx.x == 0) spoilt = 0;
    RowTiles<IO, DK, 4> rk, rq;
    rk.load(tokens_of<IO>(p.k, sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2], p.ks[1]), 0, n, p.Dk);
    rq.load(tokens_of<IO>(p.q, sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2], p.qs[1]), 0, n, p.Dk);
    double mine = 0, last = 0;               // sums of log decays
    if (wave == 0) {
        const long long gi = (sp.b * p.T + tok + (lane < n ? lane : 0)) * p.Hv + h;
        const float gv = p.g[gi], bv = p.beta[gi];
        mine = decay_sum(lane < n ? gv : 0.f);
        last = __shfl(mine, 63);
        G[lane] = mine;
        bet[lane] = lane < n ? bv : 0.f;
    }
    rk.store_plain(lds);
    rq.store_plain(lds + L::kRows);
    __syncthreads();
    if (IO != IO_F16) {
        rk.max_rows(big[0]);
        rq.max_rows(big[1]);
    }
    // scores of the wave's tokens, tile_row(wave, .), against those of the
    // tiles up to it
    dfloat4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
    const int jtiles = wave < 2 ? 2 : 4;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        uint4 a[2][NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            a[0][i] = lds[((i * 4 + wave) * KB + kb) * 64 + rslot];
            a[1][i] = lds[L::kRows + ((i * 4 + wave) * KB + kb) * 64 + rslot];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < jtiles) {
                uint4 b[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) b[i] = lds[((i * 4 + j) * KB + kb) * 64 + rslot];
                dfloat4 x[2] = {kk[j], qk[j]};
                if constexpr (IO == IO_F16) mma_tiles(a, b, x);
                else mma_bf_tiles(a, b, x);
                kk[j] = x[0];
                qk[j] = x[1];
            }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < jtiles) {
            const int col = tile_row(j, c);
            float big_p = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(wave, 4 * g4 + r);
                const float gam = row >= col ? decay(G[row] - G[col]) : 0.f;
                const float pv = row >= col ? p.scale * gam * qk[j][r] : 0.f;
                float av = row > col ? bet[row] * gam * kk[j][r] : 0.f;
                if (!finite(av)) {
                    // The inverse would spread it over its zeros, to tokens
                    // before this one.  The token itself is lost, by its beta.
                    av = 0.f;
                    spoil[row] = __uint_as_float(0x7fc00000u);
                    spoilt = 1;
                }
                A[row][col] = av;
                P[row][col] = pv;
                qk[j][r] = fabsf(pv);
                big_p = fmaxf(big_p, qk[j][r]);
            }
            if (p.bpack) {
                big_p = max_groups(big_p);
                if (g4 == 0) atomicMax(&big[2][col], __float_as_uint(big_p));
            }
        }
    // rows of P: largest over the wave's tiles, 16 lanes a row
    float back_row[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = tile_row(wave, 4 * g4 + r);
        float a = fmaxf(qk[0][r], qk[1][r]);
        if (jtiles == 4) a = fmaxf(a, fmaxf(qk[2][r], qk[3][r]));
        const Scale s = scale_to(max16(a));
        back_row[r] = s.back;
        if (c == 0) rowp[row] = s.to;
    }
    __syncthreads();
    uint4* pack = p.pack + id * kPack;
    uint4* back = p.bpack ? p.bpack + id * kPack : nullptr;
    if (wave == 0) {
        const Scale one = {1.f, 1.f};
        const Scale sk = IO == IO_F16 ? one : scale_to(__uint_as_float(big[0][lane]));
        const Scale sq = IO == IO_F16 ? one : scale_to(__uint_as_float(big[1][lane]));
        const Scale sc = scale_to(__uint_as_float(big[2][lane]));
        colp[lane] = sc.to;
        const float eg = decay(mine), ee = decay(last - mine);
        for (uint4* d : {pack, back})
            if (d) {
                float* f = (float*)(d + kDec);
                f[kDecayK + lane] = eg * sk.back;
                f[kDecayQ + lane] = p.scale * eg * sq.back;
                f[kEndK + lane] = ee * sk.back;
                f[kBeta + lane] = bet[lane] + spoil[lane];
                f[kScaleK + lane] = sk.to;
                f[kScaleQ + lane] = sq.to;
                if (lane == 0) f[kDecayAll] = decay(last);
            }
        if (back) ((float*)(back + kDec))[kBackP + lane] = sc.back;
    }
    if (c == 0)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            ((float*)(pack + kDec))[kBackP + tile_row(wave, 4 * g4 + r)] = back_row[r];
    store_tri(P, rowp, pack + kPm);
    if (back) {
        __syncthreads();
        store_tri_transposed(P, colp, back + kPm);
    }
    __syncthreads();
    // one scale for T
    const float big_t = max_groups(max16(invert_unit_lower(A, P)));
    if (lane == 0) big[3][wave] = __float_as_uint(big_t);
    __syncthreads();
    {
        float a = __uint_as_float(big[3][0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) a = fmaxf(a, __uint_as_float(big[3][i]));
        const Scale s = scale_to(a);
        if (threadIdx.x < 64) rowp[threadIdx.x] = s.to;
        if (threadIdx.x == 0) {
            ((float*)(pack + kDec))[kBackT] = s.back;
            // backward a lost token's gradients are those of all before it
            if (back) ((float*)(back + kDec))[kBackT] = spoilt ? __uint_as_float(0x7fc00000u) : s.back;
        }
    }
    __syncthreads();
    store_tri(P, rowp, pack);
    if (back) store_tri_transposed(P, rowp, back);
}

// ------------------------------------------------- the walk over the chunks

// LDS of the walk, in uint4.  Operands of the next chunk are put into a second
// buffer while the present one is worked on, where the CU's 160 KB hold two
// (fp32's at D_k = 128 do not fit, but for K alone).
template <int IO, int DK, bool FULL>
struct ScanLds {
    static constexpr int kRows = Io<IO>::NA * 4 * (DK / 32) * 64;
    static constexpr int kPackU4 = FULL ? kPack : kPm;
    static constexpr int kK = 0, kQ = kRows, kTri = kQ + (FULL ? kRows : 0);
    static constexpr int kSize = kTri + kPackU4;
    static constexpr int kBufs = 2 * kSize * 16 <= kLdsBytes ? 2 : 1;
    static constexpr int kBytes = kBufs * kSize * 16;
};

// What a walk does.  kEffect: a segment's effect on the state alone: its last
// state from the first (the first segment of a sequence) or from 0, and, in
// columns of their own, the matrix its first state is multiplied with (the
// last state from the identity, without v).  kOutputs: outputs and final
// state; kSaving: and what the backward pass reads.
enum ScanMode { kEffect, kOutputs, kSaving };

// A workgroup's walk over the chunks of one segment.  CAREFUL: tokens are kept from
// values that are not finite in the ones behind them.  Such a value meets the
// zeros of T and P on its way through a chunk and takes tokens before it along;
// it also stays in the state, so the plain walk needs no test in its steps.  True,
// and nothing stored of the state, where one of the workgroup's states ends so.
template <int IO, int DK, int W, int MODE, bool CAREFUL>
__device__ __forceinline__ bool delta_walk(const DeltaParams& p, const Span& sp, long long seq,
                                           long long seg, int sn, int h, int cb, bool matrix,
                                           bool pieces, uint4* lds) {
    constexpr bool FULL = MODE != kEffect;
    typedef ScanLds<IO, DK, FULL> L;
    constexpr int NA = Io<IO>::NA, KB = DK / 32, ST = DK / 16;
    constexpr int kCols = 16 * W, kB = Io<IO>::kB;
    const int chunks = (sp.len + kChunk - 1) / kChunk, first = sn * p.seg_chunks;
    const int last = chunks - first > p.seg_chunks ? first + p.seg_chunks : chunks;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int slot = 16 * g + (c ^ (4 * g));             // of a row operand
    const int col = cb * kCols + wave * 16 + c;
    const int width = matrix ? p.Dk : p.Dv;
    const bool cok = col < width;
    const int colv = cok && !matrix ? col : 0;           // to read from
    const int hk = h / p.group;
    const long long state = p.Dk * (long long)p.Dv;
    const Tokens tk = tokens_of<IO>(p.k, sp.b * p.ks[0] + sp.t0 * p.ks[1] + hk * p.ks[2], p.ks[1]);
    const Tokens tq = tokens_of<IO>(p.q, sp.b * p.qs[0] + sp.t0 * p.qs[1] + hk * p.qs[2], p.qs[1]);
    const Tokens tv = tokens_of<IO>(p.v, sp.b * p.vs[0] + sp.t0 * p.vs[1] + h * p.vs[2], p.vs[1]);
    const Tokens to = tokens_of<IO>(p.o, (sp.b * p.T + sp.t0) * p.Hv * p.Dv + h * p.Dv,
                                    (long long)p.Hv * p.Dv);
    const uint32_t vlane = (uint32_t)(8 * g) * (uint32_t)tv.bytes + colv * kB;
    const uint32_t olane = (uint32_t)(8 * g) * (uint32_t)to.bytes + col * kB;
    const uint4* pack = p.pack + (sp.slot0 * p.Hv + h) * kPack;
    const long long pack_step = (long long)p.Hv * kPack;

    if (__builtin_amdgcn_readfirstlane(wave) >= W) {
        RowTiles<IO, DK, kLoaders> rk, rq;
        Block<L::kPackU4 / 64, kLoaders> rp;
        const auto load = [&](int ch) __attribute__((always_inline)) {
            const int n = sp.len - ch * kChunk;
            const uint4* next_pack = pack + ch * pack_step;
            const float* f = (const float*)(next_pack + kDec);
            rk.load(tk, ch * kChunk, n, p.Dk, f + kScaleK);
            if (FULL) rq.load(tq, ch * kChunk, n, p.Dk, f + kScaleQ);
            rp.load(next_pack);
        };
        const auto store = [&](uint4* d) __attribute__((always_inline)) {
            rk.store(d + L::kK);
            if (FULL) rq.store(d + L::kQ);
            rp.store(d + L::kTri);
        };
        if (first < last) {
            load(first);
            store(lds);
        }
        __syncthreads();
        for (int ch = first, buf = 0; ch < last; ++ch) {
            load(ch + 1 < last ? ch + 1 : ch);
            if (L::kBufs == 2) {
                buf ^= 1;
                store(lds + buf * L::kSize);
                __syncthreads();
            } else {
                __syncthreads();
                store(lds);
                __syncthreads();
            }
        }
        return FULL && !CAREFUL && __syncthreads_or(0);
    }

    dfloat4 S[ST];
    {
        const float* s = nullptr;
        if (sn == 0) s = p.init ? p.init + (seq * p.Hv + h) * state + col : nullptr;
        else if (FULL) s = p.seg_n + ((pieces ? seq : seg - 1) * p.Hv + h) * state + col;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(t, 4 * g + r);
                S[t][r] = matrix ? (row == col ? 1.f : 0.f)
                                 : (s && cok && row < p.Dk ? s[(long long)row * p.Dv] : 0.f);
            }
    }
    Column<IO> v;
    if (first < last) v.load(tv, first * kChunk, vlane, sp.len - first * kChunk);
    __syncthreads();
    int buf = 0;
    for (int ch = first; ch < last; ++ch) {
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        const int n = sp.len - ch * kChunk;
        const int ahead = ch + 1 < last ? ch + 1 : ch;
        const uint4* now = lds + buf * L::kSize;
        const float* fac = (const float*)(now + L::kTri + kDec);
        const uint4* tri = now + L::kTri;
        const float big_s = max_column(S);
        const Scale ss = scale_to(big_s);
        if (MODE == kSaving && cok) save_columns<KB>(p.states, ci, p.Dv, col, S, big_s);
        // K S and Q S
        dfloat4 X[4], O[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) X[m] = O[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint4 a[4][NA], q[4][NA];
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    a[m][i] = now[L::kK + ((i * 4 + m) * KB + kb) * 64 + slot];
                    if (FULL) q[m][i] = now[L::kQ + ((i * 4 + m) * KB + kb) * 64 + slot];
                }
            uint4 st[2];
            split_acc<2>(S[2 * kb], S[2 * kb + 1], ss.to, st);
            mma_tiles(a, st, X);
            if (FULL) mma_tiles(q, st, O);
        }
        // X = beta o (V - e^G o K S);  O = scale e^G o Q S
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int row = tile_row(m, 4 * g);
            const float4 e = *(const float4*)(fac + kDecayK + row);
            const float4 b = *(const float4*)(fac + kBeta + row);
            const float4 f = *(const float4*)(fac + kDecayQ + row);
            const float ev[4] = {e.x, e.y, e.z, e.w}, bv[4] = {b.x, b.y, b.z, b.w};
            const float fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                X[m][r] = bv[r] * fmaf(-(ev[r] * ss.back), X[m][r], matrix ? 0.f : v.get(m, r));
                if (FULL) O[m][r] = (fv[r] * ss.back) * O[m][r];
            }
        }
        v.load(tv, ahead * kChunk, vlane, sp.len - ahead * kChunk);
        // Tokens of the lane's column from the first value that is not finite
        // on: their outputs and the state become NaN, and x 0, for what follows
        // multiplies it with the zeros of T and P.
        const auto lose = [&](dfloat4 (&x)[4]) __attribute__((always_inline)) {
            const float nan = __uint_as_float(0x7fc00000u);
            int at = kChunk;
#pragma unroll
            for (int m = 3; m >= 0; --m)
#pragma unroll
                for (int r = 3; r >= 0; --r)
                    if (!finite(x[m][r])) at = tile_row(m, 4 * g + r);
            at = min(at, __shfl_xor(at, 16));
            at = min(at, __shfl_xor(at, 32));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (tile_row(m, 4 * g + r) >= at) {
                        x[m][r] = 0.f;
                        O[m][r] = nan;
                    }
            if (at < kChunk)
#pragma unroll
                for (int t = 0; t < ST; ++t) S[t] = dfloat4{nan, nan, nan, nan};
        };
        // U = T X
        dfloat4 U[4];
        if (CAREFUL) lose(X);
        const Scale sx = scale_to(max_column(X));
#pragma unroll
        for (int m = 0; m < 4; ++m) U[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 xt[2];
            split_acc<2>(X[2 * kb], X[2 * kb + 1], sx.to, xt);
#pragma unroll
            for (int m0 = 2 * kb; m0 < 4; m0 += 2) {
                uint4 a[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        a[m][i] = tri[i * kTerm + tri_tile(m0 + m, kb) * 64 + lane];
                mma_tiles(a, xt, *(dfloat4 (*)[2])&U[m0]);
            }
        }
        {
            const float back = sx.back * fac[kBackT];
#pragma unroll
            for (int m = 0; m < 4; ++m) U[m] *= back;
        }
        if (FULL) {
            if (CAREFUL) lose(U);
            const float big_u = max_column(U);
            // (an infinite largest value: a chunk with lost tokens has no gradients)
            if (MODE == kSaving && cok)
                save_columns<2>(p.us, ci, p.Dv, col, U,
                                CAREFUL && S[0][0] != S[0][0] ? INFINITY : big_u);
            // O += P U
            const Scale su = scale_to(big_u);
            dfloat4 PU[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) PU[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                uint4 ut[2];
                split_acc<2>(U[2 * kb], U[2 * kb + 1], su.to, ut);
#pragma unroll
                for (int m0 = 2 * kb; m0 < 4; m0 += 2) {
                    uint4 a[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            a[m][i] = tri[kPm + i * kTerm + tri_tile(m0 + m, kb) * 64 + lane];
                    mma_tiles(a, ut, *(dfloat4 (*)[2])&PU[m0]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float4 e = *(const float4*)(fac + kBackP + tile_row(m, 4 * g));
                const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) O[m][r] = fmaf(ev[r] * su.back, PU[m][r], O[m][r]);
            }
            if (cok) store_column<IO>((char*)to.at(ch * kChunk), to.bytes, olane, n, O);
        }
        // e^(Gc-G) o U
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = *(const float4*)(fac + kEndK + tile_row(m, 4 * g));
            U[m][0] *= e.x;
            U[m][1] *= e.y;
            U[m][2] *= e.z;
            U[m][3] *= e.w;
        }
        const float ec = fac[kDecayAll];
        // S = e^Gc S + K^T U
        const Scale se = scale_to(max_column(U));
        uint4 ut[2][2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) split_acc<2>(U[2 * tb], U[2 * tb + 1], se.to, ut[tb]);
#pragma unroll
        for (int t0 = 0; t0 < ST; t0 += 4) {
            dfloat4 a[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = dfloat4{0, 0, 0, 0};
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                uint4 x[4][NA];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < NA; ++i)
                        x[t][i] = read_cols<DK>(now + L::kK + i * 4 * KB * 64, t0 + t, tb);
                mma_tiles(x, ut[tb], a);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[t0 + t][r] = fmaf(se.back, a[t][r], ec * S[t0 + t][r]);
        }
        __syncthreads();
        if (L::kBufs == 2) buf ^= 1;
        else __syncthreads();
    }
    if (FULL && !CAREFUL && __syncthreads_or(first < last && !finite(S[0][0]))) return true;
    if (!cok) return false;
    float* d = nullptr;
    if (FULL && last == chunks) d = p.fin ? p.fin + (seq * p.Hv + h) * state : nullptr;
    else if (FULL) d = pieces ? p.seg_n + (seq * p.Hv + h) * state : nullptr;
    else if (matrix) d = p.seg_m + (seg * p.Hv + h) * p.Dk * (long long)p.Dk;
    else d = p.seg_n + (seg * p.Hv + h) * state;
    if (d) store_state<ST>((char*)d, width * 4, (uint32_t)(8 * g * width + col) * 4, p.Dk, S);
    return false;
}

// A wave owns 16 columns of the state: its accumulators hold S (Dk x 16), and
// every product of the chunk, K S, T X, P U, K^T U, takes the last one's
// accumulators as its B operand, so the chain of a chunk has no exchange and
// no barrier of its own.  The W waves of a workgroup share the operands that
// do not depend on the state (K, Q, T, P) through LDS, K^T being K read
// transposed; four further waves bring the next chunk's, in step by a barrier a
// chunk.  The chain is latency: a step's vector work, its products and their
// operands wait for one another, and what else a wave did would add to it (with
// the loads in the chain's waves: 23 sequences of 9001 tokens in f16 103 us, so
// 82 when both were tried; on eight waves, which hide more of it, 205 and 199).  With
// 256 CUs taken a chunk of bf16 at D_k = 128 takes 6.9 us on eight waves and 4.5 on
// four: 64 x 1024 tokens of 6 heads of 128 are 384 chains of 16 chunks, three
// launches of 256 workgroups and 8 chunks, 63 to 69 us each, with what the backward
// pass reads 88 to 100.  The vector unit (scales and terms) is busy 46 % of the
// time, the matrix cores 21 %, and 30 % of the LDS cycles are bank conflicts.
template <int IO, int DK, int W, int MODE>
__global__ __launch_bounds__(64 * (W + kLoaders)) void delta_scan_kernel(DeltaParams p) {
    constexpr bool FULL = MODE != kEffect;
    constexpr int kCols = 16 * W;
    extern __shared__ uint4 lds[];
    const int vcols = (p.Dv + kCols - 1) / kCols;
    const int cols = vcols + (FULL ? 0 : (p.Dk + kCols - 1) / kCols);
    const bool pieces = FULL && p.pieces > 1;
    int sn = 0;                                          // segment of the sequence
    unsigned id;
    if (pieces) {
        if (!piece_of(p, (unsigned)p.nseq * p.Hv * cols, &id, &sn)) return;
    } else {
        const unsigned units = (unsigned)p.segs * p.Hv * cols;
        id = xcd_unit(blockIdx.x, units);
        if (id >= units) return;
    }
    int cb = (int)(id % cols);
    id /= cols;
    const int h = (int)(id % p.Hv);
    id /= p.Hv;
    const long long seq = pieces ? id : seq_of(p, id, p.seg_chunks);
    const Span sp = span_of(p, seq);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const unsigned seg0 = seg_of(p, sp, (unsigned)seq, p.seg_chunks);
    if (!pieces) sn = (int)(id - seg0);
    const long long seg = (long long)seg0 + sn;
    const long long first_ = (long long)sn * p.seg_chunks;
    if (sn < 0 || (sn != 0 && first_ >= chunks)) return;   // no such segment
    const int first = (int)first_;
    const int last = chunks - first > p.seg_chunks ? first + p.seg_chunks : chunks;
    if (!FULL && (last == chunks || (sn == 0 && cb >= vcols))) return;
    const bool matrix = !FULL && cb >= vcols;
    if (matrix) cb -= vcols;

    const bool lost =
        delta_walk<IO, DK, W, MODE, false>(p, sp, seq, seg, sn, h, cb, matrix, pieces, lds);
    if constexpr (FULL)
        if (lost) delta_walk<IO, DK, W, MODE, true>(p, sp, seq, seg, sn, h, cb, false, pieces, lds);
}

// Joins the segments of a sequence: with N the last state of a segment from 0
// and M the matrix of the segment, the state after it is M S + N.  Leaves in
// place of N the state after each segment but the last (the backward walk's
// segments go from the last on, all but the first).  The eight waves of a
// workgroup take 16 columns each, as in the walk, and share M through LDS, the
// next one's loads in flight.  States of a sequence's end go through every M, so
// here both are in three bf16 terms, 24 bits.  A step at heads of 128 brings 64 KB
// of M and 64 KB of N through one CU, splits M and reads it from LDS eight times,
// one after the other for the most part: 6 to 7 us a step, 95 to 104 us for 16
// segments of 4 x 32768 tokens of 4 heads; 2.2 a step at D_k = 64.
template <int DK>
struct JoinLds {
    static constexpr int kHalves = DK / 64;             // 64 rows of M each
    static constexpr int kRows = 3 * 4 * (DK / 32) * 64;
    static constexpr int kBytes = kHalves * kRows * 16;
};
template <int DK>
__global__ __launch_bounds__(512) void delta_join_kernel(DeltaParams p, bool reverse) {
    typedef JoinLds<DK> L;
    constexpr int KB = DK / 32, ST = DK / 16;
    extern __shared__ uint4 lds[];
    const int cols = (p.Dv + 127) / 128;
    unsigned id = blockIdx.x;
    const int cb = (int)(id % cols);
    id /= cols;
    const int h = (int)(id % p.Hv);
    const long long seq = id / p.Hv;
    const Span sp = span_of(p, seq);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const int n = (chunks + p.seg_chunks - 1) / p.seg_chunks;   // segments
    if (n < 3) return;           // the first one's state is already whole
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4, slot = 16 * g + (c ^ (4 * g));
    const int col = cb * 128 + wave * 16 + c;
    const bool cok = col < p.Dv;
    const long long state = p.Dk * (long long)p.Dv, square = p.Dk * (long long)p.Dk;
    const long long seg0 = seg_of(p, sp, (unsigned)seq, p.seg_chunks);
    // the i-th segment on the way
    const auto seg = [&](int i) { return (seg0 + (reverse ? n - 1 - i : i)) * p.Hv + h; };
    const uint32_t slane = (uint32_t)(8 * g * p.Dv + col) * 4;
    dfloat4 S[ST], R[ST];
    RowTiles<IO_F32, DK, 8> rm[L::kHalves];
    const auto load = [&](int i, dfloat4 (&x)[ST]) __attribute__((always_inline)) {
        const long long at = seg(i) * state;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(t, 4 * g + r);
                x[t][r] = io_load_if<IO_F32>(p.seg_n, at + (long long)row * p.Dv + col,
                                             cok && row < p.Dk);
            }
    };
    const auto load_m = [&](int i) __attribute__((always_inline)) {
        const Tokens m = tokens_of<IO_F32>(p.seg_m, seg(i) * square, p.Dk);
#pragma unroll
        for (int j = 0; j < L::kHalves; ++j) {
            const int rows = p.Dk - 64 * j;
            rm[j].load(m, rows > 0 ? 64 * j : 0, rows > 0 ? rows : 0, p.Dk);
        }
    };
    load(0, S);
    load_m(1);
    load(1, R);
    for (int i = 1; i + 1 < n; ++i) {
#pragma unroll
        for (int j = 0; j < L::kHalves; ++j) rm[j].store_plain(lds + j * L::kRows);
        __syncthreads();
        const int ahead = i + 2 < n ? i + 1 : i;
        load_m(ahead);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint4 b[3];
            const dfloat4 lo = S[2 * kb], hi = S[2 * kb + 1];
            const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            split8<3>(x, b);
#pragma unroll
            for (int t0 = 0; t0 < ST; t0 += 2) {
                uint4 a[2][3];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        a[t][j] = lds[((t0 + t) >> 2) * L::kRows +
                                      ((j * 4 + ((t0 + t) & 3)) * KB + kb) * 64 + slot];
                mma_bf_tiles(a, b, *(dfloat4 (*)[2])&R[t0]);
            }
        }
#pragma unroll
        for (int t = 0; t < ST; ++t) S[t] = R[t];
        if (cok)
            store_state<ST>((char*)(p.seg_n + seg(i) * state), p.Dv * 4, slane, p.Dk, S);
        load(ahead, R);
        __syncthreads();
    }
}

template <int IO>
hipError_t step_io(const DeltaStepParams& p, hipStream_t s) {
    const long long blocks = (long long)p.N * p.Hv * ((p.Dv + 31) / 32);
    if (p.Dk <= 64)
        hipLaunchKernelGGL((delta_step_kernel<IO, 2>), dim3((unsigned)blocks), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((delta_step_kernel<IO, 4>), dim3((unsigned)blocks), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int IO, int DK, int W, int MODE>
hipError_t scan_launch(const DeltaParams& p, const WalkGrid& w, hipStream_t s) {
    const int bytes = ScanLds<IO, DK, MODE != kEffect>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_scan_kernel<IO, DK, W, MODE>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    DeltaParams r = p;
    do {
        hipLaunchKernelGGL((delta_scan_kernel<IO, DK, W, MODE>), dim3((unsigned)w.blocks()),
                           dim3(w.threads()), bytes, s, r);
    } while (MODE != kEffect && p.pieces > 1 && ++r.round < r.rounds);
    return hipGetLastError();
}

template <int IO, int DK, int MODE>
hipError_t scan_mode(const DeltaParams& p, hipStream_t s) {
    const WalkGrid w = walk_grid(p, MODE == kEffect);
    return w.waves == 4 ? scan_launch<IO, DK, 4, MODE>(p, w, s)
                        : scan_launch<IO, DK, 8, MODE>(p, w, s);
}
template <int IO, int DK>
hipError_t scan_io(const DeltaParams& p, hipStream_t s) {
    if (p.seg_m) {
        hipError_t e = scan_mode<IO, DK, kEffect>(p, s);
        if (e == hipSuccess) e = launch_delta_join(p, false, s);
        if (e != hipSuccess) return e;
    }
    return p.states ? scan_mode<IO, DK, kSaving>(p, s) : scan_mode<IO, DK, kOutputs>(p, s);
}
template <int DK>
hipError_t join_launch(const DeltaParams& p, bool reverse, hipStream_t s) {
    const int bytes = JoinLds<DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_join_kernel<DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const long long joins = p.nseq * p.Hv * ((p.Dv + 127) / 128);
    hipLaunchKernelGGL((delta_join_kernel<DK>), dim3((unsigned)joins), dim3(512), bytes, s, p,
                       reverse);
    return hipGetLastError();
}

template <int IO, int DK>
hipError_t prep_io(const DeltaParams& p, hipStream_t s) {
    const int bytes = PrepLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_prep_kernel<IO, DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_prep_kernel<IO, DK>), dim3((unsigned)xcd_blocks(p.slots * p.Hv)),
                       dim3(256), bytes, s, p);
    return hipGetLastError();
}

}  // namespace

int delta_pack_uint4() { return kPack; }

hipError_t launch_delta_step(int io, const DeltaStepParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return step_io<IO_F32>(p, s);
    case IO_F16: return step_io<IO_F16>(p, s);
    default: return step_io<IO_BF16>(p, s);
    }
}

hipError_t launch_delta_prep(int io, const DeltaParams& p, hipStream_t s) {
    const bool d64 = p.Dk <= 64;
    switch (io) {
    case IO_F32: return d64 ? prep_io<IO_F32, 64>(p, s) : prep_io<IO_F32, 128>(p, s);
    case IO_F16: return d64 ? prep_io<IO_F16, 64>(p, s) : prep_io<IO_F16, 128>(p, s);
    default: return d64 ? prep_io<IO_BF16, 64>(p, s) : prep_io<IO_BF16, 128>(p, s);
    }
}

hipError_t launch_delta_join(const DeltaParams& p, bool reverse, hipStream_t s) {
    return p.Dk <= 64 ? join_launch<64>(p, reverse, s) : join_launch<128>(p, reverse, s);
}

hipError_t launch_delta_scan(int io, const DeltaParams& p, hipStream_t s) {
    const bool d64 = p.Dk <= 64;
    switch (io) {
    case IO_F32: return d64 ? scan_io<IO_F32, 64>(p, s) : scan_io<IO_F32, 128>(p, s);
    case IO_F16: return d64 ? scan_io<IO_F16, 64>(p, s) : scan_io<IO_F16, 128>(p, s);
    default: return d64 ? scan_io<IO_BF16, 64>(p, s) : scan_io<IO_BF16, 128>(p, s);
    }
}

}  // namespace fftconv
