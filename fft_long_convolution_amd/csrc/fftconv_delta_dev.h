// Device helpers of the gated delta rule kernels: spans of sequences, loads
// of the I/O types, products on the 16-bit matrix cores at fp32 accuracy.
//
// Matrix products.  States, solutions and gradients have to keep fp32
// accuracy over thousands of chunks, and gfx950's fp32 matrix rate is 1/16 of
// its 16-bit rate.  So an fp32 operand x is written as two f16 terms, h = f16(x)
// and l = f16(x - h), 22 bits, and a product is the sum of the term products
// but the smallest: two matrix instructions with an operand that is exact in
// one term, three otherwise.  (Three bf16 terms, 24 bits, need three and six,
// and twice the vector work.)  f16 has little range, so operands are scaled by
// powers of two that take their largest value to 2^14: the fp32 one column by
// column, a column staying in one lane of each group of 16 from operand to
// result; the other one row by row, by factors that the chunk's preparation
// folds into the decays the rows are multiplied with anyway.  What is 2^-16
// of the largest value still has all its 22 bits.
//
// Operand order.  v_mfma_f32_16x16x32_f16 takes from lane (g = l/16, c =
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
// Registers that hold loads in flight are of clang's own vector type: copies
// of HIP's, a struct, end up in scratch memory here.
typedef uint32_t du4 __attribute__((ext_vector_type(4)));

// Terms: NA of an operand of the I/O type, whose 16-bit values are exact in one.
// All others take two, also where only outputs of 16 bits follow: an output is
// a sum whose terms may cancel, so an operand's rounding has to be small
// beside the output's after they did.
template <int IO>
struct Io {
    static constexpr int NA = IO == IO_F32 ? 2 : 1;
    static constexpr int kB = IO == IO_F32 ? 4 : 2;
};

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

// tile_row(m, 4 g + r) = 8 g + tile_base(m) + r
__device__ __forceinline__ constexpr int tile_base(int m) { return 32 * (m >> 1) + 4 * (m & 1); }

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
// Units of work, slots, segments and tokens of a row are below 2^31, so their
// divisions are of 32 bits.
// index of the first segment (of L chunks; L = 1: chunk) of a sequence
__device__ __forceinline__ unsigned seg_of(const DeltaParams& p, const Span& s, unsigned i,
                                           unsigned L) {
    const unsigned nch = (unsigned)p.nch;
    return p.cu ? (unsigned)s.t0 / kChunk / L + i : i * (nch ? (nch + L - 1) / L : 1);
}
// the sequence whose segment (of L chunks) number `seg` is; its span may end
// before the segment
__device__ __forceinline__ unsigned seq_of(const DeltaParams& p, unsigned seg, unsigned L) {
    const unsigned nch = (unsigned)p.nch;
    if (!p.cu) return seg / (nch ? (nch + L - 1) / L : 1);
    unsigned lo = 0, hi = (unsigned)p.nseq - 1;
    while (lo < hi) {
        const unsigned mid = lo + (hi - lo + 1) / 2;
        long long a = p.cu[mid];
        a = a < 0 ? 0 : a > p.T ? p.T : a;
        if ((unsigned)a / kChunk / L + mid <= seg) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Tokens of a packed row that no sequence holds, for the workgroups of slots: those
// before the first bound go to the slots up to the first sequence's, those
// behind the last to the slots that its chunks leave.  do_rows(token, n).
template <typename F>
__device__ __forceinline__ void unheld_tokens(const DeltaParams& p, const Span& sp, unsigned seq,
                                              unsigned slot, F do_rows) {
    if (!p.cu) return;
    if (seq == 0 && slot <= sp.slot0) {
        const long long from = (long long)slot * kChunk;
        if (from < sp.t0) do_rows(from, (int)(sp.t0 - from < kChunk ? sp.t0 - from : kChunk));
    }
    const long long left = slot - sp.slot0 - (sp.len + kChunk - 1) / kChunk;
    if (seq + 1 == p.nseq && left >= 0) {
        const long long from = sp.t0 + sp.len + left * kChunk;
        if (from < p.T) do_rows(from, (int)(p.T - from < kChunk ? p.T - from : kChunk));
    }
}
// rows of `bytes` (a multiple of 16) set to 0, `step` bytes apart, by the workgroup
__device__ __forceinline__ void clear_rows(void* first, long long step, int rows, int bytes) {
    const int per = bytes / 16;
    for (int i = threadIdx.x; i < rows * per; i += blockDim.x)
        *(uint4*)((char*)first + i / per * step + i % per * 16) = make_uint4(0, 0, 0, 0);
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

// four consecutive elements (the place a multiple of four)
template <int IO>
__device__ __forceinline__ void load4(const void* p, long long i, bool ok, float (&x)[4]) {
    if constexpr (IO == IO_F32) {
        const float4 a = *(const float4*)((const float*)p + (ok ? i : 0));
        x[0] = ok ? a.x : 0.f; x[1] = ok ? a.y : 0.f;
        x[2] = ok ? a.z : 0.f; x[3] = ok ? a.w : 0.f;
    } else {
        const uint2 a = *(const uint2*)((const uint16_t*)p + (ok ? i : 0));
        const uint32_t u[2] = {ok ? a.x : 0, ok ? a.y : 0};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (IO == IO_BF16) {
                x[2 * j] = __uint_as_float(u[j] << 16);
                x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const h2 h = __builtin_bit_cast(h2, u[j]);
                x[2 * j] = (float)h.x;
                x[2 * j + 1] = (float)h.y;
            }
        }
    }
}
template <int IO>
__device__ __forceinline__ void store4(void* p, long long i, dfloat4 x) {
    if constexpr (IO == IO_F32) {
        *(float4*)((float*)p + i) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (IO == IO_BF16) {
        __bf16 h[4] = {(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
        *(uint2*)((uint16_t*)p + i) = __builtin_bit_cast(uint2, h);
    } else {
        _Float16 h[4] = {(_Float16)x[0], (_Float16)x[1], (_Float16)x[2], (_Float16)x[3]};
        *(uint2*)((uint16_t*)p + i) = __builtin_bit_cast(uint2, h);
    }
}

// ------------------------------------------------------------ bf16 terms
// x = h + m + l, h the leading 8 bits of x, m those of x - h, l those of the
// rest: 24 bits, and fp32's range without a scale.  For the products that
// come before the scales are known, and the join of segments.

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
__device__ __forceinline__ dfloat4 mma_bf(uint4 a, uint4 b, dfloat4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(dbf8, a),
                                                   __builtin_bit_cast(dbf8, b), c, 0, 0, 0);
}
// c[m] += a[m] b for M tiles over the bf16 term products of weight above
// 2^-24, small ones first, consecutive instructions on different accumulators
template <int M, int NA, int NB>
__device__ __forceinline__ void mma_bf_tiles(const uint4 (&a)[M][NA], const uint4 (&b)[NB],
                                             dfloat4 (&c)[M]) {
#pragma unroll
    for (int w = 2; w >= 0; --w)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = w - i;
            if (j >= 0 && j < NB)
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mma_bf(a[m][i], b[j], c[m]);
        }
}

// ------------------------------------------------------------- f16 terms

typedef _Float16 dh8 __attribute__((ext_vector_type(8)));
typedef _Float16 dh2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ dfloat4 mma_h(uint4 a, uint4 b, dfloat4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(dh8, a),
                                                  __builtin_bit_cast(dh8, b), c, 0, 0, 0);
}
// x[8] times s as N terms
template <int N>
__device__ __forceinline__ void split8h(const float (&x)[8], float s, uint4 (&t)[N]) {
    uint32_t u[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i] * s, b = x[2 * i + 1] * s;
        const dh2 h = {(_Float16)a, (_Float16)b};
        u[0][i] = __builtin_bit_cast(uint32_t, h);
        if (N == 2) {
            const dh2 l = {(_Float16)(a - (float)h.x), (_Float16)(b - (float)h.y)};
            u[1][i] = __builtin_bit_cast(uint32_t, l);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) t[n] = make_uint4(u[n][0], u[n][1], u[n][2], u[n][3]);
}
template <int N>
__device__ __forceinline__ void split_acc(dfloat4 lo, dfloat4 hi, float s, uint4 (&t)[N]) {
    const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    split8h<N>(x, s, t);
}
// c[m] += a[m] b for M tiles: all term products but low by low, small ones
// first, consecutive instructions on different accumulators
template <int M, int NA, int NB>
__device__ __forceinline__ void mma_tiles(const uint4 (&a)[M][NA], const uint4 (&b)[NB],
                                          dfloat4 (&c)[M]) {
#pragma unroll
    for (int w = 1; w >= 0; --w)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = w - i;
            if (j >= 0 && j < NB)
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mma_h(a[m][i], b[j], c[m]);
        }
}
template <int NA, int NB>
__device__ __forceinline__ dfloat4 mma_prod(const uint4 (&a)[NA], const uint4 (&b)[NB], dfloat4 c) {
#pragma unroll
    for (int w = 1; w >= 0; --w)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = w - i;
            if (j >= 0 && j < NB) c = mma_h(a[i], b[j], c);
        }
    return c;
}

// A power of two and its inverse, both normal numbers.  Where the largest value
// is not finite the others would vanish beside it, so the inverse is NaN: what
// such a row or column is part of never looks like a result.
struct Scale { float to, back; };
__device__ __forceinline__ Scale scale_to(float largest) {
    int e = (int)(__float_as_uint(largest) >> 23) & 255;
    e = e < 28 ? 28 : e;
    return {__uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23),
            e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e - 14) << 23)};
}
// Reductions in the vector unit; a shuffle through LDS would take some 100
// cycles a step.  All-reduce over the 16 lanes of a group, by rotations:
template <int N>
__device__ __forceinline__ float row_ror(float a) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(a), 0x120 + N, 15, 15, true));
}
__device__ __forceinline__ float max16(float a) {
    a = fmaxf(a, row_ror<8>(a));
    a = fmaxf(a, row_ror<4>(a));
    a = fmaxf(a, row_ror<2>(a));
    return fmaxf(a, row_ror<1>(a));
}
__device__ __forceinline__ float sum16(float a) {
    a += row_ror<8>(a);
    a += row_ror<4>(a);
    a += row_ror<2>(a);
    return a + row_ror<1>(a);
}
// over the four groups at the lane's place
__device__ __forceinline__ float sum_groups(float a) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    a = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}
// Sums in 64 bits.
template <int DPP>
__device__ __forceinline__ float moved(float a) {
    return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(a), DPP, 15, 15, true));
}
template <int DPP>
__device__ __forceinline__ double moved(double a) {
    const uint64_t u = __builtin_bit_cast(uint64_t, a);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((uint32_t)u, DPP, 15, 15, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((uint32_t)(u >> 32), DPP, 15, 15, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Of four values over the 16 lanes of a group: lane c gets the sum of t[c / 4].  Half
// of them go to the lanes half a group away, then half of the rest.
__device__ __forceinline__ double sum16_of4(const float (&t)[4]) {
    const int c = threadIdx.x & 15;
    const bool up = c & 8, odd = c & 4;
    const float s0 = up ? t[0] : t[2], s1 = up ? t[1] : t[3];
    const double a = (double)(up ? t[2] : t[0]) + moved<0x128>(s0);
    const double b = (double)(up ? t[3] : t[1]) + moved<0x128>(s1);
    double x = (odd ? b : a) + moved<0x141>(odd ? a : b);     // the mirrored eight
    x += moved<0xb1>(x);                                       // and its four lanes
    return x + moved<0x4e>(x);
}
__device__ __forceinline__ double sum_groups(double a) {
    a += __shfl_xor(a, 32);
    return a + __shfl_xor(a, 16);
}
// The larger magnitude; NaN where one of them is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
    return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ bool finite(float a) { return fabsf(a) <= 3.402823466e38f; }
// the larger value of the lane and of the other groups of 16 at its place
__device__ __forceinline__ float max_groups(float a) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    a = max_nan(__uint_as_float(x[0]), __uint_as_float(x[1]));
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    return max_nan(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
// largest magnitude in the lane's column of N tiles, NaN if one is there
template <int N>
__device__ __forceinline__ float max_column(const dfloat4 (&x)[N]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; r += 2)
            a = max_nan(max_nan(a, fabsf(x[i][r])), fabsf(x[i][r + 1]));
    return max_groups(a);
}

// Loads under a condition read the tensor's first elements where it does not
// hold and drop them: a load inside a branch would have to arrive before the
// branch ends, one latency after the other.
template <int IO>
__device__ __forceinline__ float io_load_if(const void* p, long long i, bool ok) {
    const float x = io_load<IO>(p, ok ? i : 0);
    return ok ? x : 0.f;
}

// eight elements from their bits (two vectors of an fp32 type, else one)
template <int IO>
__device__ __forceinline__ void unpack8(const du4* r, float (&x)[8]) {
    if constexpr (IO == IO_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[j >> 2][j & 3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = r[0][j];
            if constexpr (IO == IO_BF16) {
                x[2 * j] = __uint_as_float(u << 16);
                x[2 * j + 1] = __uint_as_float(u & 0xffff0000u);
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const h2 h = __builtin_bit_cast(h2, u);
                x[2 * j] = (float)h.x;
                x[2 * j + 1] = (float)h.y;
            }
        }
    }
}
// The tokens of one head: a base for the whole workgroup and byte offsets of
// the lanes below 2^32 (the host keeps token strides below 2^24 elements), so
// that addresses cost a lane one 32-bit register.
struct Tokens {
    const char* base;        // first token of the sequence
    long long bytes;         // between tokens
    __device__ __forceinline__ const char* at(long long token) const {
        return base + token * bytes;
    }
};
template <int IO>
__device__ __forceinline__ Tokens tokens_of(const void* p, long long first, long long stride) {
    constexpr int kB = IO == IO_F32 ? 4 : 2;
    return {(const char*)p + first * kB, stride * kB};
}

// Operands go from global memory to LDS through registers: the loads of the
// next chunk are in flight while the present one is worked on.  (Loads
// straight to LDS were tried: the compiler lets no later LDS read pass them,
// as they might write what it reads, and each chunk waited for its own
// prefetch.)

// The A operands of 64 tokens x DK of a head, by W waves (those whose number
// modulo W is 0 .. W - 1).  In LDS, tile
// (m, kb), place 16 g + (c ^ 4 g) holds [token tile_row(m, c)][32 kb + 8 g +
// i], i < 8; the exclusive or spreads the four groups over the banks for the
// transposed reads.  Tokens from n on and elements from Dk on are 0.
template <int IO, int DK, int W>
struct RowTiles {
    static constexpr int KB = DK / 32, kTiles = 4 * KB;
    static constexpr int kMine = (kTiles + W - 1) / W;
    static constexpr int kWords = IO == IO_F32 ? 2 : 1;
    static constexpr int kB = IO == IO_F32 ? 4 : 2;
    du4 r[kMine][kWords];
    float s[kMine];
    __device__ __forceinline__ void load(const Tokens& x, long long token, int n, int Dk) {
        const int wave = (threadIdx.x >> 6) & (W - 1), lane = threadIdx.x & 63;
        const int g = lane >> 4, c = (lane & 15) ^ (4 * g);
        const char* p = x.at(token);
        const uint32_t stride = (uint32_t)x.bytes;
        const bool whole = n >= kChunk && Dk == DK;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int tile = W * j + wave, m = tile / KB, kb = tile % KB;
            const uint32_t row = tile_row(m, c), e = 32 * kb + 8 * g;
            const bool ok = whole || ((int)row < n && (int)e < Dk);
            const uint32_t at = ok ? row * stride + e * kB : 0;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                r[j][w] = *(const du4*)(p + at + 16 * w);
            }
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                const int tile = W * j + wave, m = tile / KB, kb = tile % KB;
                const bool ok = tile_row(m, c) < n && 32 * kb + 8 * g < Dk;
#pragma unroll
                for (int w = 0; w < kWords; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[j][w][i] = ok ? r[j][w][i] : 0;
            }
        }
    }
    // and the rows' scales (f16 needs none)
    __device__ __forceinline__ void load(const Tokens& x, long long token, int n, int Dk,
                                         const float* scales) {
        load(x, token, n, Dk);
        if (IO == IO_F16) return;
        const int wave = (threadIdx.x >> 6) & (W - 1), lane = threadIdx.x & 63;
        const int c = (lane & 15) ^ (4 * (lane >> 4));
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int tile = W * j + wave;
            s[j] = scales[tile_row((kTiles % W ? tile % kTiles : tile) / KB, c)];
        }
    }
    // as f16 terms, Io<IO>::NA of them
    __device__ __forceinline__ void store(uint4* dst) const {
        constexpr int NA = Io<IO>::NA;
        const int wave = (threadIdx.x >> 6) & (W - 1), lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int at = (W * j + wave) * 64 + lane;
            if (kTiles % W && W * j + wave >= kTiles) continue;
            if constexpr (IO == IO_F16) {
                ((du4*)dst)[at] = r[j][0];
            } else {
                float x[8];
                uint4 t[NA];
                unpack8<IO>(r[j], x);
                split8h<NA>(x, s[j], t);
#pragma unroll
                for (int i = 0; i < NA; ++i) dst[i * kTiles * 64 + at] = t[i];
            }
        }
    }
    // as they are, fp32 in three bf16 terms
    __device__ __forceinline__ void store_plain(uint4* dst) const {
        const int wave = (threadIdx.x >> 6) & (W - 1), lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int at = (W * j + wave) * 64 + lane;
            if (kTiles % W && W * j + wave >= kTiles) continue;
            if constexpr (IO == IO_F32) {
                float x[8];
                unpack8<IO>(r[j], x);
                uint4 t[3];
                split8<3>(x, t);
#pragma unroll
                for (int i = 0; i < 3; ++i) dst[i * kTiles * 64 + at] = t[i];
            } else {
                ((du4*)dst)[at] = r[j][0];
            }
        }
    }
    // largest magnitudes of the rows, joined into `largest` in LDS (the bits
    // of a magnitude grow with it)
    __device__ __forceinline__ void max_rows(uint32_t* largest) const {
        const int wave = (threadIdx.x >> 6) & (W - 1), lane = threadIdx.x & 63;
        const int c = (lane & 15) ^ (4 * (lane >> 4));
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int tile = W * j + wave;
            if (kTiles % W && tile >= kTiles) continue;
            float x[8];
            unpack8<IO>(r[j], x);
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
                a = a > u ? a : u;
            }
            atomicMax(&largest[tile_row(tile / KB, c)], a);
        }
    }
};
// N KiB of consecutive memory, by W waves; those without a last piece of
// their own move the last one too, with the same values.
template <int N, int W>
struct Block {
    static constexpr int kMine = (N + W - 1) / W;
    du4 r[kMine];
    static __device__ __forceinline__ int place(int j) {
        const int i = W * j + ((threadIdx.x >> 6) & (W - 1));
        return (i < N ? i : N - 1) * 64 + (threadIdx.x & 63);
    }
    __device__ __forceinline__ void load(const uint4* src) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) r[j] = ((const du4*)src)[place(j)];
    }
    __device__ __forceinline__ void store(uint4* dst) const {
#pragma unroll
        for (int j = 0; j < kMine; ++j) ((du4*)dst)[place(j)] = r[j];
    }
};
// Elements [8 g + tile_base(m) + r] of one column of 64 tokens, as a lane's
// accumulators have them.  The bits as loaded, made numbers where they are used:
// loads that are in flight for a chunk may meet neither an instruction nor the end
// of a branch.
template <int IO>
struct Column {
    uint32_t raw[4][4];
    // lane: byte offset of the column and the group's first token.  Tokens from n
    // on read the last one: nothing that is made of them is kept.
    __device__ __forceinline__ void load(const Tokens& x, long long token, uint32_t lane, int n) {
        const char* s = x.at(token);
        const int g = (threadIdx.x >> 4) & 3, left = n - 8 * g;
        const uint32_t bytes = (uint32_t)x.bytes, last = lane + (uint32_t)(left - 1) * bytes;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t at = tile_base(m) + r < left ? lane + (tile_base(m) + r) * bytes : last;
                if constexpr (IO == IO_F32) raw[m][r] = *(const uint32_t*)(s + at);
                else raw[m][r] = *(const uint16_t*)(s + at);
            }
    }
    __device__ __forceinline__ float get(int m, int r) const {
        if constexpr (IO == IO_F32) return __uint_as_float(raw[m][r]);
        else if constexpr (IO == IO_BF16) return __uint_as_float(raw[m][r] << 16);
        else return (float)__builtin_bit_cast(_Float16, (uint16_t)raw[m][r]);
    }
};
template <int IO>
__device__ __forceinline__ void store_column(char* s, long long bytes, uint32_t lane, int n,
                                             const dfloat4 (&v)[4]) {
    if (n >= kChunk) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                io_store<IO>(s + (tile_base(m) + r) * bytes + lane, 0, v[m][r]);
    } else {
        const int left = n - 8 * ((threadIdx.x >> 4) & 3);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (tile_base(m) + r < left)
                    io_store<IO>(s + (tile_base(m) + r) * bytes + lane, 0, v[m][r]);
    }
}
// A column of an fp32 matrix of 16 ST rows (rows of `bytes`): rows from Dk on
// are left out.
template <int ST>
__device__ __forceinline__ void store_state(char* s, uint32_t bytes, uint32_t lane, int Dk,
                                            const dfloat4 (&S)[ST]) {
    if (Dk == 16 * ST) {
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *(float*)(s + (tile_base(t) + r) * bytes + lane) = S[t][r];
    } else {
        const int left = Dk - 8 * ((threadIdx.x >> 4) & 3);
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (tile_base(t) + r < left)
                    *(float*)(s + (tile_base(t) + r) * bytes + lane) = S[t][r];
    }
}
// Saved matrices (states and their gradients, U, dY): rows x Dv of fp32 for a
// chunk and head, rows a multiple of 32, columns padded to 16, and behind them
// the largest magnitude of each column (and, with dY, of dO's).  Sixteen
// columns together: block kb, half j, place 16 g + (c ^ 4 g) holds rows
// 32 kb + 8 g + 4 j + i, i < 4, of column c: a lane's accumulators in two
// 16-byte stores, each of them 1 KiB in a row for the wave (with a lane's two
// side by side the walks of 64 x 1024 tokens of 6 heads of 128 took 368 and 392
// us, so 346 and 360 when both were tried), and what RowTiles puts into LDS for
// transposed reads.
__host__ __device__ __forceinline__ long long saved_floats(int rows, int Dv) {
    const int cols = (Dv + 15) / 16 * 16;
    return (long long)(rows + 2) * cols;
}
template <int KB>
__device__ __forceinline__ void save_columns(float* all, long long ci, int Dv, int col,
                                             const dfloat4 (&x)[2 * KB], float largest,
                                             float other = 0.f) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    float* base = all + ci * saved_floats(32 * KB, Dv);
    dfloat4* d = (dfloat4*)(base + (long long)(col - c) * (32 * KB)) + 16 * g + (c ^ (4 * g));
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) d[64 * i] = x[i];
    if (g == 0) {
        const int cols = (Dv + 15) / 16 * 16;
        float* m = base + (long long)cols * (32 * KB) + col;
        m[0] = largest;
        m[cols] = other;
    }
}

// The transposed operand from rows so filled: tile (t, tb), the lane's
// [element tile_row(t, c)][token 32 tb + 8 g + i], i < 8.  Each transposed
// read takes four tokens x 16 elements for 16 lanes.
template <int DK>
__device__ __forceinline__ uint4 read_cols(const uint4* rows, int t, int tb) {
    typedef short s4 __attribute__((ext_vector_type(4)));
    constexpr int KB = DK / 32;
    const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
    const int a = j & 3, c = 4 * g + (j >> 2);
    uint2 r[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4* s = rows + ((2 * tb + half) * KB + (t >> 1)) * 64 + 16 * a + (c ^ (4 * a));
        const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4*)((const char*)s + 8 * (t & 1)));
        r[half] = __builtin_bit_cast(uint2, x);
    }
    return make_uint4(r[0].x, r[0].y, r[1].x, r[1].y);
}

// Four consecutive elements (el a multiple of four) of token tile_row(m, c)
// from rows stored by RowTiles in NA f16 terms.
template <int NA, int DK>
__device__ __forceinline__ void row4(const uint4* rows, int m, int c, int el, float (&x)[4]) {
    constexpr int KB = DK / 32;
    const int g = (el >> 3) & 3;
    const int at = (m * KB + (el >> 5)) * 64 + 16 * g + (c ^ (4 * g));
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 0.f;
#pragma unroll
    for (int a = NA - 1; a >= 0; --a) {
        const uint2 r = ((const uint2*)(rows + a * 4 * KB * 64 + at))[(el >> 2) & 1];
        const uint32_t u[2] = {r.x, r.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const dh2 h = __builtin_bit_cast(dh2, u[j]);
            x[2 * j] += (float)h.x;
            x[2 * j + 1] += (float)h.y;
        }
    }
}

// A chunk's pack, in uint4: T (two terms), the factors below, P (two terms).
// For the backward pass: T^T, factors, P^T.
constexpr int kLdsBytes = 160 * 1024;              // of a CU
constexpr int kTerm = kTriTiles * 64;             // one term of a triangle
constexpr int kDec = 2 * kTerm, kDecU4 = 128, kPm = kDec + kDecU4;
constexpr int kPack = kPm + 2 * kTerm;
// Factors of the chunk's tokens, 64 floats each.  With rk, rq the scales of
// the rows of K and Q and G, beta as in the formulas:
enum Factor {
    kDecayK = 0,      // e^G / rk
    kDecayQ = 64,     // scale e^G / rq
    kEndK = 128,      // e^(Gc-G) / rk
    kBeta = 192,
    kBackP = 256,     // inverse scales of the rows of P (backward: of P^T)
    kScaleK = 320,    // rk
    kScaleQ = 384,    // rq
    kDecayAll = 448,  // e^Gc
    kBackT = 449,     // inverse scale of T
};

constexpr int kLd = 68;   // floats between rows of the 64 x 64 matrices in LDS

// x of the lane that is so many places before in the group of 16, or 0
template <int DPP>
__device__ __forceinline__ double shifted(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)u, DPP, 15, 15, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(u >> 32), DPP, 15, 15, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum of the log decays up to the lane's token, in units of log 2 (decay()
// makes factors of them).  Sums are fp64, so e^(G_i - G_j) is right to fp32
// however much the chunk has decayed before; decays below -1e4 count as -1e4
// (their factor is 0 in fp32 either way), so a reset (g = -inf) does not meet
// itself as inf - inf.  NaN stays NaN.
__device__ __forceinline__ double decay_sum(float g) {
    double s = g < -1e4f ? -1e4f : g;
    // within each group of 16, then the groups before
    s += shifted<0x111>(s);
    s += shifted<0x112>(s);
    s += shifted<0x114>(s);
    s += shifted<0x118>(s);
    const int lane = threadIdx.x & 63;
    const double a = __shfl(s, 15), b = __shfl(s, 31), c = __shfl(s, 47);
    if (lane >= 16) s += a;
    if (lane >= 32) s += b;
    if (lane >= 48) s += c;
    return s * 1.4426950408889634074;
}
__device__ __forceinline__ float decay(double g) { return __builtin_amdgcn_exp2f((float)g); }

// Workgroups are dealt round robin over the 8 XCDs; this gives each XCD a
// run of consecutive units, so the units that share a head's rows share an
// L2.  Returns n where there is no unit.
__device__ __forceinline__ unsigned xcd_unit(unsigned block, unsigned n) {
    const unsigned per = (n + 7) / 8;
    const unsigned u = (block & 7) * per + (block >> 3);
    return (block >> 3) < per && u < n ? u : n;
}
inline long long xcd_blocks(long long n) { return (n + 7) / 8 * 8; }

// The piece of a chain that a workgroup takes in the present round.  All pieces
// in a row, `pieces` a chain, are dealt to the machines (a workgroup of every
// round) `rounds` at a time, so no two of a chain meet in one round; its first
// piece is the one of its earliest round.  False: nothing to do.
__device__ __forceinline__ bool piece_of(const DeltaParams& p, unsigned chains, unsigned* chain,
                                         int* piece) {
    const unsigned n = p.pieces, rounds = p.rounds, round = p.round;
    const unsigned machines = (chains * n + rounds - 1) / rounds;
    const unsigned m = xcd_unit(blockIdx.x, machines);
    if (m >= machines) return false;
    const unsigned at = m * rounds + round;
    *chain = at / n;
    if (*chain >= chains) return false;
    // its rounds are start .. start + n - 1, modulo `rounds`
    const unsigned start = *chain * n % rounds, end = start + n;
    const unsigned early = end > rounds ? end - rounds : 0;
    *piece = (int)(round < early ? round : early + round - start);
    return true;
}

}  // namespace fftconv
