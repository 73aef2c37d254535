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
// Registers that hold loads in flight are of clang's own vector type: copies
// of HIP's, a struct, end up in scratch memory here.
typedef uint32_t du4 __attribute__((ext_vector_type(4)));

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
// index of the first segment (of L chunks; L = 1: chunk) of a sequence
__device__ __forceinline__ long long seg_first(long long t0, long long i, long long nch, long long L,
                                               bool packed) {
    return packed ? t0 / (kChunk * L) + i : i * (nch ? (nch + L - 1) / L : 1);
}
__device__ __forceinline__ long long seg_of(const DeltaParams& p, const Span& s, long long i) {
    return seg_first(s.t0, i, p.nch, p.seg_chunks, p.cu != nullptr);
}
// the sequence whose segment (of L chunks) number `seg` is; its span may end
// before the segment
__device__ __forceinline__ long long seq_of(const DeltaParams& p, long long seg, long long L) {
    if (!p.cu) {
        return seg / (p.nch ? (p.nch + L - 1) / L : 1);
    }
    long long lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const long long mid = (lo + hi + 1) / 2;
        long long a = p.cu[mid];
        a = a < 0 ? 0 : a > p.T ? p.T : a;
        if (a / (kChunk * L) + mid <= seg) lo = mid; else hi = mid - 1;
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

// c[m] += a[m] b for M tiles: the same products, but consecutive instructions
// go to different accumulators
template <int LIM, int M, int NA, int NB>
__device__ __forceinline__ void mma_tiles(const uint4 (&a)[M][NA], const uint4 (&b)[NB],
                                          dfloat4 (&c)[M]) {
#pragma unroll
    for (int w = LIM - 1; w >= 0; --w)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = w - i;
            if (j >= 0 && j < NB)
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mma(a[m][i], b[j], c[m]);
        }
}

// Loads under a condition read the tensor's first elements where it does not
// hold and drop them: a load inside a branch would have to arrive before the
// branch ends, one latency after the other.
__device__ __forceinline__ uint4 keep(bool ok, uint4 x) {
    return make_uint4(ok ? x.x : 0, ok ? x.y : 0, ok ? x.z : 0, ok ? x.w : 0);
}
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
// eight consecutive elements
template <int IO>
__device__ __forceinline__ void load8(const void* p, long long i, bool ok, float (&x)[8]) {
    constexpr int kB = IO == IO_F32 ? 4 : 2;
    const du4* s = (const du4*)((const char*)p + (ok ? i : 0) * kB);
    du4 r[2];
    r[0] = s[0];
    if (IO == IO_F32) r[1] = s[1];
    unpack8<IO>(r, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = ok ? x[j] : 0.f;
}
// the same as bf16 terms
template <int IO>
__device__ __forceinline__ void load_terms(const void* p, long long i, bool ok,
                                           uint4 (&t)[IoTerms<IO>::n]) {
    if constexpr (IO == IO_BF16) {
        t[0] = keep(ok, *(const uint4*)((const uint16_t*)p + (ok ? i : 0)));
    } else {
        float x[8];
        load8<IO>(p, i, ok, x);
        split8<IoTerms<IO>::n>(x, t);
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

// The A operands of 64 tokens x DK of a head, by W waves.  In LDS, tile
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
    __device__ __forceinline__ void load(const Tokens& x, long long token, int n, int Dk) {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        const int g = lane >> 4, c = (lane & 15) ^ (4 * g);
        const char* s = x.at(token);
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
                r[j][w] = *(const du4*)(s + at + 16 * w);
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
    __device__ __forceinline__ void store(uint4* dst) const {
        const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int at = (W * j + wave) * 64 + lane;
            if (kTiles % W && W * j + wave >= kTiles) continue;
            if constexpr (IO == IO_F32) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[j][i >> 2][i & 3]);
                uint4 t[3];
                split8<3>(x, t);
#pragma unroll
                for (int i = 0; i < 3; ++i) dst[i * kTiles * 64 + at] = t[i];
            } else {
                ((du4*)dst)[at] = r[j][0];
            }
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
        const int i = W * j + (threadIdx.x >> 6);
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
// accumulators have them; `lane`: byte offset of the column and the group's
// first token.  Tokens from n on read the last one: nothing that is made of
// them is kept.
template <int IO>
__device__ __forceinline__ void load_column(const Tokens& x, long long token, uint32_t lane, int n,
                                            dfloat4 (&v)[4]) {
    const char* s = x.at(token);
    if (n >= kChunk) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[m][r] = io_load<IO>(s + (tile_base(m) + r) * x.bytes + lane, 0);
    } else {
        const int g = (threadIdx.x >> 4) & 3;
        const uint32_t col = lane - 8 * g * (uint32_t)x.bytes;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 8 * g + tile_base(m) + r;
                v[m][r] = io_load<IO>(s + (row < n ? row : n - 1) * (uint32_t)x.bytes + col, 0);
            }
    }
}
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
// from rows filled by RowTiles.
template <int IO, int DK>
__device__ __forceinline__ void row4(const uint4* rows, int m, int c, int el, float (&x)[4]) {
    constexpr int KB = DK / 32, NA = IO == IO_F32 ? 3 : 1;
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
            if constexpr (IO == IO_F16) {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const h2 h = __builtin_bit_cast(h2, u[j]);
                x[2 * j] = (float)h.x;
                x[2 * j + 1] = (float)h.y;
            } else {
                x[2 * j] += __uint_as_float(u[j] << 16);
                x[2 * j + 1] += __uint_as_float(u[j] & 0xffff0000u);
            }
        }
    }
}

// Products of an operand of the I/O type with an fp32 one.
//   bf16: exact in one term, times three bf16 terms;
//   fp32: three terms, times three (the six products above 2^-24);
//   f16: exact in one f16 term, times two f16 terms, 22 bits.  f16 has little
//     range, so each column of the fp32 operand is first multiplied with the
//     power of two that takes its largest value to 2^14; a column stays in
//     one lane of each group of 16 from operand to result.
struct ColScale { float to, back; };
template <int IO>
struct Operand {
    static constexpr int NA = IO == IO_F32 ? 3 : 1, NB = IO == IO_F16 ? 2 : 3;
    static constexpr bool kScaled = IO == IO_F16;
    // terms of P and U in the outputs' P U: 16 bits are enough for a 16-bit
    // output, whose rounding is 2^-9 or 2^-12 of it
    static constexpr int NP = IO == IO_F32 ? 3 : 2;
    // uint4 of a chunk's pack: T (three terms), decays, P
    static constexpr int kPack = (3 * kTriTiles + 1 + NP * kTriTiles) * 64;

    template <int N>
    static __device__ __forceinline__ ColScale scale_of(const dfloat4 (&x)[N]) {
        if constexpr (!kScaled) return {1.f, 1.f};
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) a = fmaxf(a, fabsf(x[i][r]));
        a = fmaxf(a, __shfl_xor(a, 16));
        a = fmaxf(a, __shfl_xor(a, 32));
        // exponents where both factors are normal numbers
        int e = (int)(__float_as_uint(a) >> 23);
        e = e < 28 ? 28 : e > 240 ? 240 : e;
        return {__uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23),
                __uint_as_float((uint32_t)(e - 14) << 23)};
    }
    static __device__ __forceinline__ void split(dfloat4 lo, dfloat4 hi, const ColScale& s,
                                                 uint4 (&t)[NB]) {
        if constexpr (kScaled) {
            typedef _Float16 h8 __attribute__((ext_vector_type(8)));
            h8 a, b;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = (i < 4 ? lo[i & 3] : hi[i & 3]) * s.to;
                a[i] = (_Float16)x;
                b[i] = (_Float16)(x - (float)a[i]);
            }
            t[0] = __builtin_bit_cast(uint4, a);
            t[1] = __builtin_bit_cast(uint4, b);
        } else {
            split_acc<NB>(lo, hi, t);
        }
    }
    static __device__ __forceinline__ dfloat4 mma(const uint4 (&a)[NA], const uint4 (&b)[NB],
                                                  dfloat4 c) {
        if constexpr (kScaled) return mma_h(a[0], b[0], mma_h(a[0], b[1], c));
        else return mma_terms<3>(a, b, c);
    }
    template <int M>
    static __device__ __forceinline__ void mma_all(const uint4 (&a)[M][NA], const uint4 (&b)[NB],
                                                   dfloat4 (&c)[M]) {
        if constexpr (kScaled) {
#pragma unroll
            for (int i = 1; i >= 0; --i)
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mma_h(a[m][0], b[i], c[m]);
        } else {
            mma_tiles<3>(a, b, c);
        }
    }
    template <int M>
    static __device__ __forceinline__ void mma_all_out(const uint4 (&a)[M][NA],
                                                       const uint4 (&b)[NB], dfloat4 (&c)[M]) {
        if constexpr (kScaled) mma_all(a, b, c);
        else mma_tiles<NP>(a, b, c);
    }
    // both operands of the I/O type
    static __device__ __forceinline__ dfloat4 mma_io(const uint4 (&a)[NA], const uint4 (&b)[NA],
                                                     dfloat4 c) {
        if constexpr (kScaled) return mma_h(a[0], b[0], c);
        else return mma_terms<3>(a, b, c);
    }
    // where a 16-bit output is all that follows, 16 bits of b
    static __device__ __forceinline__ dfloat4 mma_out(const uint4 (&a)[NA], const uint4 (&b)[NB],
                                                      dfloat4 c) {
        if constexpr (kScaled) return mma(a, b, c);
        else return mma_terms<NP>(a, b, c);
    }
    static __device__ __forceinline__ dfloat4 mma_h(uint4 a, uint4 b, dfloat4 c) {
        typedef _Float16 h8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                      __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
};
// uint4 of a chunk's pack for the backward: T^T and P^T (three terms each)
// around the decays
constexpr int kBackPack = (6 * kTriTiles + 1) * 64;

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
