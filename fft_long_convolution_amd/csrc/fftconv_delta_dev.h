// Device helpers of the gated delta rule kernels: spans of sequences, loads
// of the I/O types, products on the bf16 matrix cores at 24 bits.
//
// Matrix products.  States, solutions and gradients have to keep fp32
// accuracy over thousands of chunks, and gfx950's fp32 matrix rate is 1/16 of
// its bf16 rate.  So an fp32 operand x is written as three bf16 terms,
// x = h + m + l with h the leading 8 bits of x, m those of x - h and l those
// of the rest (24 bits), and a product is the sum of the term products whose
// weight is not below 2^-24 of the whole: with an operand that is exact in
// bf16 three matrix instructions, with one of f16 (two terms) five, of fp32
// six.
//
// Operand order.  v_mfma_f32_16x16x32_bf16 takes from lane (g = l/16, c =
// l%16) A[row c][k = 8g + i] and B[k = 8g + i][col c], i < 8, and leaves
// D[row 4g + r][col c], r < 4.  Rows of a 16-row tile m stand for index
// tile_row(m, row) = 32 (m/2) + 8 (row/4) + 4 (m%2) + row%4 of the matrix, so
// the accumulators of tiles 2b and 2b+1 in a lane are exactly the eight
// k = 32b + 8g + i that the lane feeds as B of the next product: results go
// from one product into the next without leaving their registers.
#pragma once

#include "fftconv_delta.h"

namespace fftconv {

typedef __bf16 dbf8 __attribute__((ext_vector_type(8)));
typedef float dfloat4 __attribute__((ext_vector_type(4)));

template <int IO>
struct IoTerms { static constexpr int n = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3; };

__device__ __forceinline__ int tile_row(int m, int row) {
    return 32 * (m >> 1) + 8 * (row >> 2) + 4 * (m & 1) + (row & 3);
}
// tile (m, kb) of a lower triangle of 64 x 64, kb <= m / 2
__device__ __forceinline__ constexpr int tri_tile(int m, int kb) {
    return m < 2 ? m : 2 + 2 * (m - 2) + kb;
}

// tile (m, kb) of an upper triangle, kb >= m / 2
__device__ __forceinline__ constexpr int upper_tile(int m, int kb) {
    return m < 2 ? 2 * m + kb : 2 + m;
}

struct Span {
    long long b, t0, slot0;
    int len;
};
// Bounds that are not ascending within [0, T] are clamped to it: nothing
// outside the tensors is ever addressed.
__device__ __forceinline__ Span span_of(const DeltaParams& p, long long i) {
    Span s;
    if (p.cu) {
        long long a = p.cu[i], z = p.cu[i + 1];
        a = a < 0 ? 0 : a > p.T ? p.T : a;
        z = z < a ? a : z > p.T ? p.T : z;
        s.b = 0;
        s.t0 = a;
        s.len = (int)(z - a);
        s.slot0 = a / kChunk + i;
    } else {
        s.b = i;
        s.t0 = 0;
        s.len = (int)p.T;
        s.slot0 = i * p.nch;
    }
    return s;
}
// the sequence whose chunk a slot is (its span may end before the slot)
__device__ __forceinline__ long long seq_of(const DeltaParams& p, long long slot) {
    if (!p.cu) return slot / p.nch;
    long long lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const long long mid = (lo + hi + 1) / 2;
        long long a = p.cu[mid];
        a = a < 0 ? 0 : a > p.T ? p.T : a;
        if (a / kChunk + mid <= slot) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int IO>
__device__ __forceinline__ float io_load(const void* p, long long i) {
    if constexpr (IO == IO_F32) return ((const float*)p)[i];
    else if constexpr (IO == IO_F16) return (float)((const _Float16*)p)[i];
    else return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}
template <int IO>
__device__ __forceinline__ void io_store(void* p, long long i, float x) {
    if constexpr (IO == IO_F32) ((float*)p)[i] = x;
    else if constexpr (IO == IO_F16) ((_Float16*)p)[i] = (_Float16)x;
    else ((__bf16*)p)[i] = (__bf16)x;
}

// the upper halves of a and b, a in the low one
__device__ __forceinline__ uint32_t hi_pair(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ float top16(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
// x[8] as N bf16 terms
template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], uint4 (&t)[N]) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = x[i];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        t[n] = make_uint4(hi_pair(a[0], a[1]), hi_pair(a[2], a[3]), hi_pair(a[4], a[5]),
                          hi_pair(a[6], a[7]));
        if (n + 1 < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] -= top16(a[i]);
        }
    }
}
template <int N>
__device__ __forceinline__ void split_acc(dfloat4 lo, dfloat4 hi, uint4 (&t)[N]) {
    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    split8<N>(x, t);
}

__device__ __forceinline__ dfloat4 mma(uint4 a, uint4 b, dfloat4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(dbf8, a),
                                                   __builtin_bit_cast(dbf8, b), c, 0, 0, 0);
}
// c += a b over the term products of weight above 2^-8 LIM, small ones first
template <int LIM, int NA, int NB>
__device__ __forceinline__ dfloat4 mma_terms(const uint4 (&a)[NA], const uint4 (&b)[NB], dfloat4 c) {
#pragma unroll
    for (int w = LIM - 1; w >= 0; --w)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = w - i;
            if (j >= 0 && j < NB) c = mma(a[i], b[j], c);
        }
    return c;
}

// eight consecutive elements of the I/O type as NA bf16 terms
template <int IO>
__device__ __forceinline__ void load_terms(const void* p, long long i, bool ok,
                                           uint4 (&t)[IoTerms<IO>::n]) {
    if constexpr (IO == IO_BF16) {
        t[0] = ok ? *(const uint4*)((const uint16_t*)p + i) : make_uint4(0, 0, 0, 0);
    } else {
        float x[8];
        if constexpr (IO == IO_F16) {
            typedef _Float16 h8 __attribute__((ext_vector_type(8)));
            const uint4 r = ok ? *(const uint4*)((const uint16_t*)p + i) : make_uint4(0, 0, 0, 0);
            const h8 h = __builtin_bit_cast(h8, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)h[j];
        } else {
            float4 a = make_float4(0, 0, 0, 0), b = a;
            if (ok) {
                a = *(const float4*)((const float*)p + i);
                b = *(const float4*)((const float*)p + i + 4);
            }
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
        split8<IoTerms<IO>::n>(x, t);
    }
}

// The 8 x 8 transpose of 16-bit elements held as rows of eight.
__device__ __forceinline__ void transpose8(const uint4 (&r)[8], uint4 (&c)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t ra[4] = {r[2 * i].x, r[2 * i].y, r[2 * i].z, r[2 * i].w};
            const uint32_t rb[4] = {r[2 * i + 1].x, r[2 * i + 1].y, r[2 * i + 1].z,
                                    r[2 * i + 1].w};
            w[i] = __builtin_amdgcn_perm(rb[j >> 1], ra[j >> 1],
                                         (j & 1) ? 0x07060302u : 0x05040100u);
        }
        c[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Fills the A operands of 64 tokens x DK of a head in LDS: tile (m, kb),
// lane (g, c) holds [token tile_row(m, c)][32 kb + 8 g + i].
template <int IO, int DK>
__device__ __forceinline__ void fill_rows(uint4* dst, const void* src, long long base,
                                          long long stride, int n, int Dk) {
    constexpr int NA = IoTerms<IO>::n, KB = DK / 32;
    for (int i = threadIdx.x; i < 4 * KB * 64; i += 256) {
        const int tile = i >> 6, l = i & 63;
        const int m = tile / KB, kb = tile - m * KB;
        const int row = tile_row(m, l & 15), e = 32 * kb + 8 * (l >> 4);
        uint4 t[NA];
        load_terms<IO>(src, base + row * stride + e, row < n && e < Dk, t);
#pragma unroll
        for (int a = 0; a < NA; ++a) dst[a * 4 * KB * 64 + i] = t[a];
    }
}
// The same tokens' transpose: tile (t, tb), lane (g, c) holds
// [element tile_row(t, c)][token 32 tb + 8 g + i].
template <int IO, int DK>
__device__ __forceinline__ void fill_cols(uint4* dst, const void* src, long long base,
                                          long long stride, int n, int Dk) {
    constexpr int NA = IoTerms<IO>::n;
    for (int i = threadIdx.x; i < 8 * (DK / 8); i += 256) {
        // eight tokens x eight elements
        const int tg = i & 7, ec = i >> 3;
        uint4 t[8][NA];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            load_terms<IO>(src, base + (8 * tg + j) * stride + 8 * ec,
                           8 * tg + j < n && 8 * ec < Dk, t[j]);
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            uint4 r[8], col[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = t[j][a];
            transpose8(r, col);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // element 8 ec + j: tile and row that stand for it
                const int tile = 2 * (ec >> 2) + (j >> 2), row = 4 * (ec & 3) + (j & 3);
                dst[((a * (DK / 16) + tile) * 2 + (tg >> 2)) * 64 + 16 * (tg & 3) + row] = col[j];
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void fill_tri(uint4* dst, const float* src) {
    for (int i = threadIdx.x; i < kTriTiles * 64; i += 256) {
        const float4 a = *(const float4*)(src + i * 8), b = *(const float4*)(src + i * 8 + 4);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint4 t[N];
        split8<N>(x, t);
#pragma unroll
        for (int j = 0; j < N; ++j) dst[j * kTriTiles * 64 + i] = t[j];
    }
}

constexpr int kLd = 68;   // floats between rows of the 64 x 64 matrices in LDS

// Sum of the log decays up to the lane's token.  Sums are fp64, so
// e^(G_i - G_j) is right to fp32 however much the chunk has decayed before;
// decays below -1e4 count as -1e4 (their factor is 0 in fp32 either way), so
// a reset (g = -inf) does not meet itself as inf - inf.  NaN stays NaN.
__device__ __forceinline__ double decay_sum(float g) {
    const int lane = threadIdx.x & 63;
    double s = g < -1e4f ? -1e4f : g;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(s, m);
        if (lane >= m) s += o;
    }
    return s;
}

// Workgroups are dealt round robin over the 8 XCDs; this gives each XCD a
// run of consecutive units, so the units that share a head's rows share an
// L2.  Returns n where there is no unit.
__device__ __forceinline__ long long xcd_unit(long long block, long long n) {
    const long long per = (n + 7) / 8;
    const long long u = (block & 7) * per + (block >> 3);
    return (block >> 3) < per && u < n ? u : n;
}
inline long long xcd_blocks(long long n) { return (n + 7) / 8 * 8; }

}  // namespace fftconv
