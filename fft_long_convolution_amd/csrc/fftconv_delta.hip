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
// one: each state is read and written once, and HBM bounds the call.
template <int IO, int R>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepParams p) {
    const int tiles = (p.Dv + 31) / 32;
    long long id = blockIdx.x;
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
    float* S = p.state + (slot * p.Hv + h) * p.Dk * (long long)p.Dv + col;
    const int hk = h / (p.Hv / p.Hk);
    float4 s[R];
    float k[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool ok = row0 + i < p.Dk;
        s[i] = cok && ok ? *(const float4*)(S + (long long)(row0 + i) * p.Dv)
                         : make_float4(0, 0, 0, 0);
        k[i] = ok ? io_load<IO>(p.k, n * p.ks[0] + hk * p.ks[1] + row0 + i) : 0.f;
        q[i] = ok ? io_load<IO>(p.q, n * p.qs[0] + hk * p.qs[1] + row0 + i) : 0.f;
    }
    const float a = expf(p.g[n * p.Hv + h]), beta = p.beta[n * p.Hv + h];
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
    for (int j = 0; j < 9; ++j)
#pragma unroll
        for (int m = 8; m < 64; m <<= 1) r[j] += __shfl_xor(r[j], m);
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
        u[j] = beta * (io_load<IO>(p.v, n * p.vs[0] + h * p.vs[1] + col + j) - a * r[j]);
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
// The four waves of the workgroup call it together.
__device__ void invert_unit_lower(const float (*a)[kLd], float (*t)[kLd]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    {
        // zero the blocks above the diagonal, invert those on it
        const int o = 16 * wave;
        for (int i = lane; i < 16 * 64; i += 64) {
            const int row = o + (i >> 6), col = i & 63;
            if (col >= o + 16) t[row][col] = 0.f;
        }
        if (lane < 16) {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == c ? 1.f : 0.f;
#pragma unroll
                for (int l = 0; l < i; ++l) s -= a[o + i][o + l] * x[l];
                x[i] = s;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) t[o + i][o + c] = x[i];
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
        for (int s = 0; s < 4; ++s) t[o + 16 + 4 * g + s][o + c] = -r[s];
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
        for (int s = 0; s < 4; ++s) t[row + 4 * g + s][col + c] = -r[s];
    }
    __syncthreads();
}

// Writes a lower triangle from LDS in operand order: tile (m, kb), lane
// (g, c), element i holds [tile_row(m, c)][32 kb + 8 g + i].
__device__ __forceinline__ void store_tri(const float (*t)[kLd], float* dst) {
    for (int i = threadIdx.x; i < kTriTiles * 64; i += blockDim.x) {
        const int tile = i >> 6, l = i & 63;
        const int m = tile < 2 ? tile : 2 + ((tile - 2) >> 1);
        const int kb = tile < 2 ? 0 : (tile - 2) & 1;
        const float* s = &t[tile_row(m, l & 15)][32 * kb + 8 * (l >> 4)];
        float4* d = (float4*)(dst + (long long)i * 8);
        d[0] = *(const float4*)s;
        d[1] = *(const float4*)(s + 4);
    }
}

// The same triangle's transpose, an upper one: tile (m, kb), kb >= m / 2.
__device__ __forceinline__ void store_tri_transposed(const float (*t)[kLd], float* dst) {
    for (int i = threadIdx.x; i < kTriTiles * 64; i += blockDim.x) {
        const int tile = i >> 6, l = i & 63;
        const int m = tile < 4 ? tile >> 1 : tile - 2;
        const int kb = tile < 4 ? tile & 1 : 1;
        const int col = tile_row(m, l & 15), row = 32 * kb + 8 * (l >> 4);
        float4* d = (float4*)(dst + (long long)i * 8);
        d[0] = make_float4(t[row][col], t[row + 1][col], t[row + 2][col], t[row + 3][col]);
        d[1] = make_float4(t[row + 4][col], t[row + 5][col], t[row + 6][col], t[row + 7][col]);
    }
}

// One workgroup per chunk and value head.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaParams p) {
    constexpr int NA = IoTerms<IO>::n, KB = DK / 32;
    const long long id = xcd_unit(blockIdx.x, p.slots * p.Hv);
    if (id >= p.slots * p.Hv) return;
    const long long slot = id / p.Hv;
    const int h = (int)(id - slot * p.Hv);
    const long long seq = seq_of(p, slot);
    const Span sp = span_of(p, seq);
    const long long at = (slot - sp.slot0) * kChunk;
    if (at < 0 || at >= sp.len) return;      // a slot between two sequences
    const int n = (int)(sp.len - at < kChunk ? sp.len - at : kChunk);
    const long long tok = sp.t0 + at;

    __shared__ __align__(16) float A[kChunk][kLd], P[kChunk][kLd];
    __shared__ double G[kChunk];
    __shared__ float bet[kChunk];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g4 = lane >> 4;
    if (wave == 0) {
        const long long gi = (sp.b * p.T + tok + lane) * p.Hv + h;
        const float gv = lane < n ? p.g[gi] : 0.f;
        const float bv = lane < n ? p.beta[gi] : 0.f;
        const double s = decay_sum(gv);
        G[lane] = s;
        bet[lane] = bv;
        const double last = __shfl(s, 63);
        float* dec = p.dec + id * kDecFloats;
        dec[lane] = expf((float)s);
        dec[64 + lane] = expf((float)(last - s));
        dec[128 + lane] = bv;
        if (lane == 0) dec[192] = expf((float)last);
    }
    // scores of the 16 rows of the wave against the columns up to them
    const int hk = h / p.group;
    const long long kbase = sp.b * p.ks[0] + hk * p.ks[2];
    const long long qbase = sp.b * p.qs[0] + hk * p.qs[2];
    dfloat4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int e = 32 * kb + 8 * g4;
        uint4 ka[NA], qa[NA];
        const int row = 16 * wave + c;
        const bool ok = row < n && e < p.Dk;
        load_terms<IO>(p.k, kbase + (tok + row) * p.ks[1] + e, ok, ka);
        load_terms<IO>(p.q, qbase + (tok + row) * p.qs[1] + e, ok, qa);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) {
                uint4 b[NA];
                const int col = 16 * j + c;
                load_terms<IO>(p.k, kbase + (tok + col) * p.ks[1] + e, col < n && e < p.Dk, b);
                kk[j] = mma_terms<3>(ka, b, kk[j]);
                qk[j] = mma_terms<3>(qa, b, qk[j]);
            }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * wave + 4 * g4 + r, col = 16 * j + c;
            const float gam = row >= col ? expf((float)(G[row] - G[col])) : 0.f;
            A[row][col] = row > col ? bet[row] * gam * kk[j][r] : 0.f;
            P[row][col] = row >= col ? p.scale * gam * qk[j][r] : 0.f;
        }
    __syncthreads();
    store_tri(P, p.pm + id * kTriFloats);
    if (p.pmt) store_tri_transposed(P, p.pmt + id * kTriFloats);
    __syncthreads();
    invert_unit_lower(A, P);
    store_tri(P, p.tri + id * kTriFloats);
    if (p.trit) store_tri_transposed(P, p.trit + id * kTriFloats);
}

// ------------------------------------------------- the walk over the chunks

template <int IO, int DK>
struct ScanLds {
    static constexpr int NA = IoTerms<IO>::n;
    static constexpr int NP = IO == IO_F32 ? 3 : 2;   // terms of P and of U in P U
    // fp32 operands fill the LDS: the transposed keys take the place of the
    // keys once those are used
    static constexpr bool kShare = NA == 3;
    static constexpr int kRows = NA * 4 * (DK / 32) * 64;     // uint4
    static constexpr int kK = 0, kQ = kRows, kT = kShare ? 0 : 2 * kRows;
    static constexpr int kTri = kShare ? 2 * kRows : 3 * kRows;
    static constexpr int kP = kTri + 3 * kTriTiles * 64;
    static constexpr int kDec = kP + NP * kTriTiles * 64;
    static constexpr int kBytes = (kDec + kDecFloats / 4) * 16;
};

// A wave owns 16 columns of the state: its accumulators hold S (Dk x 16), and
// every product of the chunk, K S, T X, P U, K^T U, takes the last one's
// accumulators as its B operand, so the chain of a chunk has no exchange and
// no barrier of its own.  The four waves of a workgroup share the operands
// that do not depend on the state (K, Q, K^T, T, P) through LDS.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_scan_kernel(DeltaParams p) {
    typedef ScanLds<IO, DK> L;
    constexpr int NA = L::NA, KB = DK / 32, ST = DK / 16, NP = L::NP;
    extern __shared__ uint4 lds[];
    const float* dec = (const float*)(lds + L::kDec);
    const int cols = (p.Dv + 63) / 64;
    const long long units = p.nseq * p.Hv * cols;
    long long id = xcd_unit(blockIdx.x, units);
    if (id >= units) return;
    const int cb = (int)(id % cols);
    id /= cols;
    const int h = (int)(id % p.Hv);
    const long long seq = id / p.Hv;
    const Span sp = span_of(p, seq);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int col = cb * 64 + wave * 16 + c;
    const bool cok = col < p.Dv;
    const int hk = h / p.group;
    const long long sbase = (seq * p.Hv + h) * p.Dk * (long long)p.Dv + col;
    dfloat4 S[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = tile_row(t, 4 * g + r);
            S[t][r] = p.init && cok && row < p.Dk ? p.init[sbase + (long long)row * p.Dv] : 0.f;
        }
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    for (int ch = 0; ch < chunks; ++ch) {
        const long long tok = sp.t0 + (long long)ch * kChunk;
        const int left = sp.len - ch * kChunk, n = left < kChunk ? left : kChunk;
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        const long long kbase = sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2];
        const long long qbase = sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2];
        fill_rows<IO, DK>(lds + L::kK, p.k, kbase, p.ks[1], n, p.Dk);
        fill_rows<IO, DK>(lds + L::kQ, p.q, qbase, p.qs[1], n, p.Dk);
        if (!L::kShare) fill_cols<IO, DK>(lds + L::kT, p.k, kbase, p.ks[1], n, p.Dk);
        fill_tri<3>(lds + L::kTri, p.tri + ci * kTriFloats);
        fill_tri<NP>(lds + L::kP, p.pm + ci * kTriFloats);
        if (threadIdx.x < kDecFloats / 4)
            lds[L::kDec + threadIdx.x] = ((const uint4*)(p.dec + ci * kDecFloats))[threadIdx.x];
        float v[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(m, 4 * g + r);
                v[m][r] = cok && row < n
                              ? io_load<IO>(p.v, sp.b * p.vs[0] + (tok + row) * p.vs[1] +
                                                     h * p.vs[2] + col)
                              : 0.f;
            }
        if (p.states && cok) {
            float* d = p.states + ci * p.Dk * (long long)p.Dv + col;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = tile_row(t, 4 * g + r);
                    if (row < p.Dk) d[(long long)row * p.Dv] = S[t][r];
                }
        }
        __syncthreads();
        // K S and Q S
        dfloat4 X[4], O[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) X[m] = O[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint4 st[3];
            split_acc<3>(S[2 * kb], S[2 * kb + 1], st);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint4 a[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = lds[L::kK + ((i * 4 + m) * KB + kb) * 64 + lane];
                X[m] = mma_terms<3>(a, st, X[m]);
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = lds[L::kQ + ((i * 4 + m) * KB + kb) * 64 + lane];
                O[m] = mma_terms<NP>(a, st, O[m]);
            }
        }
        // X = beta o (V - e^G o K S);  O = scale e^G o Q S
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int row = tile_row(m, 4 * g);
            const float4 e = *(const float4*)(dec + row), b = *(const float4*)(dec + 128 + row);
            const float ev[4] = {e.x, e.y, e.z, e.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                X[m][r] = bv[r] * (v[m][r] - ev[r] * X[m][r]);
                O[m][r] = p.scale * ev[r] * O[m][r];
            }
        }
        // U = T X
        dfloat4 U[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) U[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 xt[3];
            split_acc<3>(X[2 * kb], X[2 * kb + 1], xt);
#pragma unroll
            for (int m = 2 * kb; m < 4; ++m) {
                uint4 a[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    a[i] = lds[L::kTri + (i * kTriTiles + tri_tile(m, kb)) * 64 + lane];
                U[m] = mma_terms<3>(a, xt, U[m]);
            }
        }
        if (p.us && cok) {
            float* d = p.us + ci * kChunk * p.Dv + col;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = tile_row(m, 4 * g + r);
                    d[(long long)row * p.Dv] = U[m][r];
                }
        }
        // O += P U
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 ut[NP];
            split_acc<NP>(U[2 * kb], U[2 * kb + 1], ut);
#pragma unroll
            for (int m = 2 * kb; m < 4; ++m) {
                uint4 a[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    a[i] = lds[L::kP + (i * kTriTiles + tri_tile(m, kb)) * 64 + lane];
                O[m] = mma_terms<NP>(a, ut, O[m]);
            }
        }
        if (cok)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = tile_row(m, 4 * g + r);
                    if (row < n)
                        io_store<IO>(p.o, ((sp.b * p.T + tok + row) * p.Hv + h) * p.Dv + col,
                                     O[m][r]);
                }
        if (L::kShare) {
            __syncthreads();
            fill_cols<IO, DK>(lds + L::kT, p.k, kbase, p.ks[1], n, p.Dk);
            __syncthreads();
        }
        // S = e^Gc S + K^T (e^(Gc-G) o U)
        const float ec = dec[192];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] *= ec;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            const int row = 32 * tb + 8 * g;
            const float4 e0 = *(const float4*)(dec + 64 + row);
            const float4 e1 = *(const float4*)(dec + 68 + row);
            const float x[8] = {e0.x * U[2 * tb][0],     e0.y * U[2 * tb][1],
                                e0.z * U[2 * tb][2],     e0.w * U[2 * tb][3],
                                e1.x * U[2 * tb + 1][0], e1.y * U[2 * tb + 1][1],
                                e1.z * U[2 * tb + 1][2], e1.w * U[2 * tb + 1][3]};
            uint4 ut[3];
            split8<3>(x, ut);
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                uint4 a[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = lds[L::kT + ((i * ST + t) * 2 + tb) * 64 + lane];
                S[t] = mma_terms<3>(a, ut, S[t]);
            }
        }
        __syncthreads();
    }
    if (p.fin && cok)
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(t, 4 * g + r);
                if (row < p.Dk) p.fin[sbase + (long long)row * p.Dv] = S[t][r];
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

template <int IO, int DK>
hipError_t scan_io(const DeltaParams& p, hipStream_t s) {
    const int bytes = ScanLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_scan_kernel<IO, DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const long long units = p.nseq * p.Hv * ((p.Dv + 63) / 64);
    hipLaunchKernelGGL((delta_scan_kernel<IO, DK>), dim3((unsigned)xcd_blocks(units)), dim3(256),
                       bytes, s, p);
    return hipGetLastError();
}

template <int IO>
hipError_t prep_io(const DeltaParams& p, hipStream_t s) {
    const dim3 grid((unsigned)xcd_blocks(p.slots * p.Hv));
    if (p.Dk <= 64)
        hipLaunchKernelGGL((delta_prep_kernel<IO, 64>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((delta_prep_kernel<IO, 128>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_step(int io, const DeltaStepParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return step_io<IO_F32>(p, s);
    case IO_F16: return step_io<IO_F16>(p, s);
    default: return step_io<IO_BF16>(p, s);
    }
}

hipError_t launch_delta_prep(int io, const DeltaParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return prep_io<IO_F32>(p, s);
    case IO_F16: return prep_io<IO_F16>(p, s);
    default: return prep_io<IO_BF16>(p, s);
    }
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
