// Device helpers of linear attention with a decay for each head: spans of
// sequences, token matrices in LDS, products on the matrix cores, and the steps
// of a chunk that the forward and the backward walks share.
//
// A walk takes a sequence's chunks of C tokens one after the other with a state
// S (DA x columns) in the accumulators of its waves, 16 columns a wave.  With rows
// A, B of DA elements and rows V of the columns, and D_t the sum of the log decays
// from the chunk's first token to t:
//   out = f o (A S) + P V,   P_ts = Gam_ts A_t.B_s
//   S  <- e^Dc S + B^T (w o V)
// forward in time f = e^D, w = e^(Dc-D), Gam_ts = e^(D_t-D_s) for s <= t; backward
// f = e^(Dc-D), w = e^D, Gam_ts = e^(D_s-D_t) for s >= t (and constant factors).
//
// Matrix products.  16-bit rows are exact operands.  An fp32 operand (states, scores,
// weighted values) is written in terms of that type, each the rounding of what the ones
// before leave: of bf16 three (26 bits), with fp32's range; of f16 two (22 bits), with a
// power of two for each column (states, weighted values) or row of 32 scores that takes
// the largest to 2^14.  So the rounding of an output is the only one to fewer bits, also
// where most of a sum cancels.
// fp32 rows go to the fp32 matrix instructions as they are, which have 1/16 of
// the rate, and so have all operands 24 bits.
//
// Operand order.  The 16 x 16 instructions take 32 k at a time: lane (g = l/16, c
// = l%16) gives A[row c][k = 8g + i], B[k = 8g + i][col c], i < 8, and has D[row
// 4g + r][col c], r < 4.  Row 4g + r of a 16-row tile i of the state stands for
// element 32 (i/2) + 8g + 4 (i%2) + r, so that a lane's accumulators of two tiles
// are the eight k that it gives as B of the next product.  fp32: the same places,
// eight instructions of four k.
#pragma once

#include "fftconv_decay.h"
#include "fftconv_delta_dev.h"

namespace fftconv {

template <int IO>
struct Kind {
    static constexpr int kB = IO == IO_F32 ? 4 : 2;
    static constexpr int NT = IO == IO_BF16 ? 3 : IO == IO_F16 ? 2 : 1;   // terms of an operand
};

// ------------------------------------------------------------------- spans

struct DecaySpan {
    long long b, t0;         // batch row, first token
    int len, from, to;       // tokens of the sequence, of the segment in it
    unsigned seq, index;     // the segment's place among the sequence's
    bool last;               // segment
};
// Bounds that are not ascending within [0, T] are clamped to it.
__device__ __forceinline__ long long bound_of(const DecaySpans& p, long long i) {
    const long long a = p.cu[i];
    return a < 0 ? 0 : a > p.T ? p.T : a;
}
// False for a number that no segment has.  An empty sequence has one.
__device__ __forceinline__ bool segment_of(const DecaySpans& p, unsigned seg, DecaySpan& s) {
    const unsigned L = (unsigned)p.seg_tokens;
    if (p.cu) {
        unsigned lo = 0, hi = (unsigned)p.nseq - 1;
        while (lo < hi) {
            const unsigned mid = lo + (hi - lo + 1) / 2;
            if ((unsigned)bound_of(p, mid) / L + mid <= seg) lo = mid; else hi = mid - 1;
        }
        const long long a = bound_of(p, lo);
        long long z = bound_of(p, lo + 1);
        z = z < a ? a : z;
        s.seq = lo;
        s.b = 0;
        s.t0 = a;
        s.len = (int)(z - a);
        const unsigned first = (unsigned)a / L + lo;
        if (seg < first) return false;
        s.index = seg - first;
    } else {
        s.seq = seg / (unsigned)p.per;
        s.index = seg - s.seq * (unsigned)p.per;
        s.b = s.seq;
        s.t0 = 0;
        s.len = (int)p.T;
    }
    // the same for all lanes: kept in scalar registers
    s.seq = __builtin_amdgcn_readfirstlane(s.seq);
    s.index = __builtin_amdgcn_readfirstlane(s.index);
    s.len = __builtin_amdgcn_readfirstlane(s.len);
    s.b = __builtin_amdgcn_readfirstlane((uint32_t)s.b);
    s.t0 = __builtin_amdgcn_readfirstlane((uint32_t)s.t0);
    const long long from = (long long)s.index * L;
    if (from >= s.len && s.index) return false;
    s.from = (int)from;
    s.last = from + L >= s.len;
    s.to = s.last ? s.len : (int)(from + L);
    return true;
}

// ---------------------------------------------------- token matrices in LDS

// Which 16-byte piece of a token's row holds piece u: u ^ swirl(token).  Sixteen
// tokens at one piece (row reads) and four tokens by 32 bytes of two neighbouring
// 16-element groups (transposed reads of the values) each meet all banks.  Single cells of
// 16 columns of 16-bit rows do not: tokens 8 apart exchange two neighbouring pieces, so
// four tokens meet each bank twice; nor do the transposed reads of the state's elements,
// which take the same half of all pieces.  A third of the walks' LDS cycles are such
// conflicts.
template <int PIECES>
__device__ __forceinline__ uint32_t swirl(uint32_t t) {
    if constexpr (PIECES == 8) return ((t >> 3) & 1) | ((t >> 1) & 2) | ((t << 1) & 4);
    else return ((t >> 3) & 1) | ((t >> 1) & 2) | ((t & 1) << 2) | ((t & 2) << 2);
}
// Bases are of a lane; which of its pieces is read is then an exclusive or with a
// constant, which token an immediate offset: swirl() is linear and sees four bits.
template <int IO, int D>
struct Rows {
    static constexpr int kB = Kind<IO>::kB, kPieces = D * kB / 16, kRow = D * kB;
    // byte offset of piece u of a token
    static __device__ __forceinline__ uint32_t at(uint32_t token, uint32_t u) {
        return token * kRow + ((u ^ swirl<kPieces>(token)) << 4);
    }
};
// x, unknown to the compiler from here on: what follows from a lane's base is made
// where it is used instead of being kept in registers over the whole walk.
__device__ __forceinline__ void forget(uint32_t& x) { asm volatile("" : "+v"(x)); }
__device__ __forceinline__ int fresh_thread() {
    uint32_t x = threadIdx.x;
    forget(x);
    return (int)x;
}

// Eight consecutive elements or k, as an operand.
template <int IO>
struct Frag { du4 v; };
template <>
struct Frag<IO_F32> { dfloat4 a, b; };

template <int IO>
__device__ __forceinline__ void unpack_frag(const Frag<IO>& f, float (&x)[8]) {
    if constexpr (IO == IO_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = f.a[i]; x[4 + i] = f.b[i]; }
    } else {
        unpack8<IO>(&f.v, x);
    }
}
// Rows as operands with k along the elements: lane (g, c) has token t0 + c at
// elements e0 + 8g + i, i < 8; t0 a multiple of 16, e0 of 32.
template <int IO, int D>
struct RowReader {
    uint32_t base;
    __device__ __forceinline__ explicit RowReader(int lane)
        : base(Rows<IO, D>::at(lane & 15, (lane >> 4) * (IO == IO_F32 ? 2 : 1))) {}
    __device__ __forceinline__ Frag<IO> get(const char* m, int t0, int e0) const {
        Frag<IO> f;
        if constexpr (IO == IO_F32) {
            const char* s = m + t0 * Rows<IO, D>::kRow;
            f.a = *(const dfloat4*)(s + (base ^ (uint32_t)(e0 << 2)));
            f.b = *(const dfloat4*)(s + (base ^ (uint32_t)(e0 << 2 | 16)));
        } else {
            f.v = *(const du4*)(m + t0 * Rows<IO, D>::kRow + (base ^ (uint32_t)(e0 << 1)));
        }
        return f;
    }
};
// Rows as operands with k along the tokens: lane (g, c) has tokens t0 + 8g + i, i < 8,
// at element 16 i + c, or, STATE, at the element that row c of tile i of the state
// stands for; t0 a multiple of 32.
template <int IO, int D, bool STATE>
struct ColReader {
    typedef Rows<IO, D> R;
    uint32_t base;
    __device__ __forceinline__ explicit ColReader(int lane) {
        const int g = lane >> 4, j = lane & 15;
        if constexpr (IO == IO_F32) {
            base = R::at(8 * g, STATE ? 2 * (j >> 2) : j >> 2) + 4 * (j & 3);
        } else {
            // each read takes, from 16 lanes, four tokens by four pieces of four
            // elements, and gives lane j the four tokens' element j of the pieces in
            // the lanes' order
            base = STATE ? R::at(8 * g + (j >> 2), j & 3)
                         : R::at(8 * g + (j >> 2), (j & 3) >> 1) + 8 * (j & 1);
        }
    }
    __device__ __forceinline__ Frag<IO> get(const char* m, int t0, int i) const {
        const uint32_t at = base ^ (uint32_t)(STATE ? 32 * (i >> 1) * R::kB : 16 * i * R::kB);
        const char* s = m + t0 * R::kRow;
        Frag<IO> f;
        if constexpr (IO == IO_F32) {
            const uint32_t half = STATE ? 16 * (i & 1) : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x = *(const float*)(
                    s + k * R::kRow + (at ^ half ^ (swirl<R::kPieces>(k) << 4)));
                if (k < 4) f.a[k & 3] = x; else f.b[k & 3] = x;
            }
        } else {
            typedef short s4 __attribute__((ext_vector_type(4)));
            uint2 r[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const char* x = s + 4 * k * R::kRow + (STATE ? 8 * (i & 1) : 0) +
                                (at ^ (swirl<R::kPieces>(4 * k) << 4));
                r[k] = __builtin_bit_cast(
                    uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                               (__attribute__((address_space(3))) s4*)x));
            }
            f.v = du4{r[0].x, r[0].y, r[1].x, r[1].y};
        }
        return f;
    }
};

// Single elements of a tile in accumulator order: lane (g, c) has token t0 + 4g + r, r < 4,
// at column first + c; t0 a multiple of 16.
template <int IO, int D>
struct CellPlaces {
    typedef Rows<IO, D> R;
    uint32_t base;
    __device__ __forceinline__ CellPlaces(int lane, int first) {
        constexpr int kPer = 16 / R::kB;
        const int e = first + (lane & 15);
        base = R::at(4 * (lane >> 4), e / kPer) + e % kPer * R::kB;
    }
    __device__ __forceinline__ uint32_t at(int t0, int r) const {
        return (t0 + r) * R::kRow + (base ^ (swirl<R::kPieces>(r) << 4));
    }
};
// The bases of a lane.  Columns of the values are `first` and so on in tiles of DV.
template <int IO, int DA, int DV>
struct Places {
    RowReader<IO, DA> rows;
    ColReader<IO, DA, true> elements;
    ColReader<IO, DV, false> values;
    CellPlaces<IO, DV> cells;
    int lane;
    __device__ __forceinline__ Places(int lane, int first)
        : rows(lane), elements(lane), values(lane), cells(lane, first), lane(lane) {}
    __device__ __forceinline__ void fresh() {
        forget(rows.base);
        forget(elements.base);
        forget(values.base);
        forget(cells.base);
        lane = fresh_thread() & 63;
    }
};

// Rows of one head on their way: the walk's present ones (a uniform address) and the
// thread's part of them.
struct Source {
    const char* p;
    uint32_t stride, mine;
};
// C tokens of rows on their way from memory to LDS (or back), by N threads, each of
// which keeps to its pieces: tokens from n on and pieces from the row's end on are 0.
template <int IO, int D, int C, int N>
struct Moving {
    static constexpr int kPieces = Rows<IO, D>::kPieces, kAll = C * kPieces;
    static constexpr int kMine = (kAll + N - 1) / N, kStep = N / kPieces;
    static_assert(N % kPieces == 0 && (kAll % N == 0 || kAll < N), "threads share evenly");
    du4 r[kMine];
    static __device__ __forceinline__ bool idle(int tid) { return kAll < N && tid >= kAll; }
    // of the thread's first piece, in a tile
    static __device__ __forceinline__ uint32_t place(int tid) {
        return Rows<IO, D>::at(tid / kPieces, tid % kPieces);
    }
    static __device__ __forceinline__ uint32_t next(uint32_t place, int j) {
        return (place ^ (swirl<kPieces>(j * kStep) << 4)) + j * kStep * Rows<IO, D>::kRow;
    }
    // tokens of the thread's, counted from its first one
    static __device__ __forceinline__ int left(int tid, int n, int pieces) {
        return tid % kPieces < pieces ? n - tid / kPieces : 0;
    }
    static __device__ __forceinline__ Source source(const Tokens& x, long long token, int tid) {
        return {x.at(token), (uint32_t)x.bytes,
                (uint32_t)(tid / kPieces) * (uint32_t)x.bytes + 16u * (tid % kPieces)};
    }
    // Loads in flight may meet neither an instruction nor the end of a branch: those
    // of what is not there read the first piece, and are dropped by clear().
    __device__ __forceinline__ void load(const Source& s, int left) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            r[j] = *(const du4*)(s.p + (j * kStep < left ? s.mine + j * kStep * s.stride : 0u));
    }
    __device__ __forceinline__ void clear(int left) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) r[j][w] = j * kStep < left ? r[j][w] : 0;
    }
    __device__ __forceinline__ void store(char* m, uint32_t place, int tid) const {
        if (idle(tid)) return;
#pragma unroll
        for (int j = 0; j < kMine; ++j) *(du4*)(m + next(place, j)) = r[j];
    }
    __device__ __forceinline__ void take(const char* m, uint32_t place, int tid) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) r[j] = *(const du4*)(m + (idle(tid) ? 0 : next(place, j)));
    }
    // to rows `row` bytes apart, the thread's first piece at mine
    __device__ __forceinline__ void write(char* out, uint32_t mine, uint32_t row, int left,
                                          int tid) const {
        if (idle(tid)) return;
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            if (j * kStep < left) *(du4*)(out + (j * kStep * row + mine)) = r[j];
    }
    // whether an element is infinite or NaN
    __device__ __forceinline__ bool unbounded() const {
        if constexpr (IO == IO_F32) {
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < kMine; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w) most = max(most, r[j][w] & 0x7fffffffu);
            return most >= 0x7f800000u;
        } else {
            typedef uint16_t u2 __attribute__((ext_vector_type(2)));
            u2 most = {0, 0};
#pragma unroll
            for (int j = 0; j < kMine; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    most = __builtin_elementwise_max(most, __builtin_bit_cast(u2, r[j][w] & 0x7fff7fffu));
            return max(most.x, most.y) >= (IO == IO_F16 ? 0x7c00 : 0x7f80);
        }
    }
};

// ---------------------------------------------------------------- products

template <int IO>
__device__ __forceinline__ dfloat4 mma16(const Frag<IO>& a, const Frag<IO>& b, dfloat4 c) {
    if constexpr (IO == IO_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.a[i], b.a[i], c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.b[i], b.b[i], c, 0, 0, 0);
        return c;
    } else if constexpr (IO == IO_F16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(dh8, a.v),
                                                      __builtin_bit_cast(dh8, b.v), c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(dbf8, a.v),
                                                       __builtin_bit_cast(dbf8, b.v), c, 0, 0, 0);
    }
}
// After a run of matrix instructions: time for the last of them to write its result.
// The compiler puts the waits that are needed before what reads it in the same
// block, but a block that a branch leads to may begin with such a read: one did (an
// accumulator's copy right behind the branch), and got the old value.
__device__ __forceinline__ void products_done() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 7");
    __builtin_amdgcn_sched_barrier(0);
}
// x[8] times s (f16; a power of two) as N terms
template <int IO, int N>
__device__ __forceinline__ void terms(const float (&x)[8], float s, Frag<IO> (&t)[N]) {
    if constexpr (IO == IO_F32) {
        t[0].a = dfloat4{x[0], x[1], x[2], x[3]};
        t[0].b = dfloat4{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = x[2 * i], b = x[2 * i + 1];
            if constexpr (IO == IO_F16) { a *= s; b *= s; }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if constexpr (IO == IO_F16) {
                    const dh2 h = {(_Float16)a, (_Float16)b};
                    t[n].v[i] = __builtin_bit_cast(uint32_t, h);
                    if (n + 1 < N) { a -= (float)h.x; b -= (float)h.y; }
                } else {
                    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
                    const b2 h = {(__bf16)a, (__bf16)b};
                    uint32_t u = __builtin_bit_cast(uint32_t, h);
                    asm("" : "+v"(u));       // one conversion of two values
                    t[n].v[i] = u;
                    if (n + 1 < N) {
                        a -= __uint_as_float(u << 16);
                        b -= __uint_as_float(u & 0xffff0000u);
                    }
                }
            }
        }
    }
}

// the larger (smaller) of the lane's value and those of the other groups at its place
__device__ __forceinline__ int max_all(int a) {
    a = max(a, __shfl_xor(a, 32));
    return max(a, __shfl_xor(a, 16));
}
__device__ __forceinline__ int min_all(int a) {
    a = min(a, __shfl_xor(a, 32));
    return min(a, __shfl_xor(a, 16));
}

// -------------------------------------------------------- factors of a chunk

// Sums of log decays in units of log 2, as a whole number and a rest of at most a
// half: their differences are right to 2^-24 however large the sums are.
template <int C>
struct Factors {
    int whole[C];
    float rest[C];
    float f[C], w[C];        // of the rows of the state's product, of the values
    float all, err;          // e^Dc, and what its rounding left of it, in parts of it
    float none[2];
};
struct Power { int whole; float rest; };
__device__ __forceinline__ Power power_of(double x) {
    const double n = __builtin_rint(x);
    return {(int)n, (float)(x - n)};
}
__device__ __forceinline__ float exp2_of(int whole, float rest) {
    return __builtin_ldexpf(__builtin_amdgcn_exp2f(rest), whole);
}
// 2^x rounded to fp32 once: of a chunk's factors, which all elements of a row and the
// whole state share, so that their errors do not average out.  With y = rest log 2,
// at most 0.35: 1 + y in 64 bits and the Taylor terms from y^2 / 2 on, below 0.07, in
// 32 (off by 2^-28), up to y^9 / 9! (2e-10).
// left: the exact value is (1 + left) times the result.
__device__ __forceinline__ float exact_exp2(double x, float& left) {
    const double n = __builtin_rint(x), y = (x - n) * 0.6931471805599453;
    const float z = (float)y;
    float e = 1.f / 362880;
    e = fmaf(e, z, 1.f / 40320);
    e = fmaf(e, z, 1.f / 5040);
    e = fmaf(e, z, 1.f / 720);
    e = fmaf(e, z, 1.f / 120);
    e = fmaf(e, z, 1.f / 24);
    e = fmaf(e, z, 1.f / 6);
    e = fmaf(e, z, 0.5f);
    const double exact = 1.0 + (y + (double)(e * z * z));
    const float near = (float)exact;
    left = (float)(exact - near) / near;
    return __builtin_ldexpf(near, (int)n);
}
__device__ __forceinline__ float exact_exp2(double x) {
    float left;
    return exact_exp2(x, left);
}
// By the 64 lanes of one wave: D of the lane's token (n tokens, those behind have the
// last one's), in units of log 2.  g: the token's log decay (0 behind the last).
template <int C>
__device__ __forceinline__ double decays_to(float g, bool fixed, int n) {
    const int lane = threadIdx.x & 63;
    if (fixed) {
        const float a = g < -1e4f ? -1e4f : g;
        return (double)a * (double)(lane < n ? lane + 1 : n) * 1.4426950408889634074;
    }
    return decay_sum(lane < n ? g : 0.f);
}
// f and w for a walk forward in time (REV: backward), times sf and sw.
template <int C, bool REV>
__device__ __forceinline__ void put_factors(Factors<C>& F, double D, float sf, float sw) {
    const int lane = threadIdx.x & 63;
    const double all = __shfl(D, C - 1);
    const Power p = power_of(D);
    float left;
    const float to = exact_exp2(D, left), from = exact_exp2(all - D);
    if (lane < C) {
        F.whole[lane] = p.whole;
        F.rest[lane] = p.rest;
        F.f[lane] = sf * (REV ? from : to);
        F.w[lane] = sw * (REV ? to : from);
        if (lane == C - 1) {
            F.all = to;
            F.err = left;
        }
    }
}

// ------------------------------------------------------- the steps of a chunk

// Scores P (rows A against rows B) as operands of 16 rows x 32 k: block (m, kb) of
// term i at ((i * C/16 + m) * C/32 + kb) * 64 + lane.  f16: 32 scores of a row have
// a scale, back[kb][row] holds its inverse.  A wave makes kTiles blocks of 16 x 16 of
// a row tile together.
template <int IO, int C>
struct Scores {
    static constexpr int kBlock = 64 * (int)sizeof(Frag<IO>), M = C / 16, KB = C / 32;
    static constexpr int kTerm = kBlock * M * KB, kBytes = kTerm * Kind<IO>::NT;
    static constexpr int kTiles = C == 64 || IO == IO_F16 ? 2 : 1;
    static constexpr int kParts = M / kTiles, kUnits = M * kParts;
    static __device__ __forceinline__ Frag<IO> get(const char* P, int lane, int term, int m, int kb) {
        return *(const Frag<IO>*)(P + term * kTerm + (m * KB + kb) * kBlock +
                                  lane * (int)sizeof(Frag<IO>));
    }
    // the lane's rows 16 kt + 4 g + r of B, r < 4, for its row 16 qt + c of A
    static __device__ __forceinline__ void put(char* P, int lane, int qt, int kt, float to, dfloat4 p) {
        const int g = lane >> 4, c = lane & 15;
        const int place = (qt * KB + (kt >> 1)) * 64 + (2 * (kt & 1) + (g >> 1)) * 16 + c;
        if constexpr (IO == IO_F32) {
            *(dfloat4*)(P + place * 32 + (g & 1) * 16) = p;
        } else {
            const float x[8] = {p[0], p[1], p[2], p[3], 0, 0, 0, 0};
            Frag<IO> t[Kind<IO>::NT];
            terms<IO, Kind<IO>::NT>(x, to, t);
#pragma unroll
            for (int n = 0; n < Kind<IO>::NT; ++n)
                *(uint2*)(P + n * kTerm + place * 16 + (g & 1) * 8) = make_uint2(t[n].v[0], t[n].v[1]);
        }
    }
    // the scale of a row, from the largest of the lane's scores of it: at most 2^54, as
    // scores below 2^-40 do not reach an f16 output
    static __device__ __forceinline__ float scale(float largest, float* back, int lane, int qt, int part) {
        if constexpr (IO == IO_F16) {
            const Scale sc = scale_to(fmaxf(max_groups(largest), 0x1p-40f));
            if (lane < 16) back[part * C + 16 * qt + lane] = sc.back;
            return sc.to;
        }
        return 1.f;
    }
};
// Decays between the lane's token (whole, rest) and tokens s0 .. s0 + 3.
template <int C, bool REV>
__device__ __forceinline__ void decays_between(const Factors<C>& F, int s0, int whole, float rest,
                                               float (&gam)[4]) {
    const int4 sw = *(const int4*)&F.whole[s0];
    const float4 sr = *(const float4*)&F.rest[s0];
    const int w[4] = {sw.x, sw.y, sw.z, sw.w};
    const float r[4] = {sr.x, sr.y, sr.z, sr.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        gam[e] = REV ? exp2_of(w[e] - whole, r[e] - rest) : exp2_of(whole - w[e], rest - r[e]);
}
template <int IO, int DA, int C, int NW, bool REV>
__device__ __forceinline__ void make_scores(const RowReader<IO, DA>& rows, int lane, const char* A,
                                            const char* B, char* P, float* back,
                                            const Factors<C>& F, float scale, int wave) {
    typedef Scores<IO, C> L;
    const int g = lane >> 4, c = lane & 15;
#pragma unroll
    for (int j = 0; j < (L::kUnits + NW - 1) / NW; ++j) {
        const int unit = wave + NW * j, qt = unit % L::M, part = unit / L::M, k0 = part * L::kTiles;
        // blocks of 32 k that meet no 1 of the triangle are not read
        if ((NW > L::kUnits && unit >= L::kUnits) ||
            (REV ? k0 + L::kTiles - 1 < (qt & ~1) : k0 > (qt | 1)))
            continue;
        dfloat4 acc[L::kTiles];
#pragma unroll
        for (int x = 0; x < L::kTiles; ++x) acc[x] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DA / 32; ++kb) {
            const Frag<IO> b = rows.get(A + qt * 16 * Rows<IO, DA>::kRow, 0, 32 * kb);
#pragma unroll
            for (int x = 0; x < L::kTiles; ++x)
                acc[x] = mma16<IO>(rows.get(B + k0 * 16 * Rows<IO, DA>::kRow, 16 * x, 32 * kb), b, acc[x]);
        }
        products_done();
        const int i = 16 * qt + c, whole = F.whole[i];
        const float rest = F.rest[i];
        float largest = 0.f;
#pragma unroll
        for (int x = 0; x < L::kTiles; ++x) {
            const int s0 = 16 * (k0 + x) + 4 * g;
            float gam[4];
            decays_between<C, REV>(F, s0, whole, rest, gam);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = scale * gam[e] * acc[x][e];
                acc[x][e] = (REV ? s0 + e >= i : s0 + e <= i) ? p : 0.f;
                if (IO == IO_F16) largest = fmaxf(largest, fabsf(acc[x][e]));
            }
        }
        const float to = L::scale(largest, back, lane, qt, part);
#pragma unroll
        for (int x = 0; x < L::kTiles; ++x) L::put(P, lane, qt, k0 + x, to, acc[x]);
    }
}

// The lane's column of the state: tiles of 16 elements.
template <int DA>
struct State {
    static constexpr int N = DA / 16;
    dfloat4 t[N];
    // largest magnitude of the column that is finite
    __device__ __forceinline__ float largest() const {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) a = fmaxf(a, fabsf(t[i][r]));
        a = max_groups(a);
        return finite(a) ? a : 0.f;
    }
    // element of register r of tile i for the lane's group g
    static __device__ __forceinline__ int element(int i, int r, int g) {
        return 32 * (i >> 1) + 8 * g + 4 * (i & 1) + r;
    }
    // base[element * rs], elements below rows, where ok
    __device__ __forceinline__ void load(const float* base, long long rs, bool ok, int rows) {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = element(i, r, g);
                const bool here = ok && e < rows;
                const float x = base[here ? e * rs : 0];
                t[i][r] = here ? x : 0.f;
            }
    }
    __device__ __forceinline__ void store(float* base, long long rs, bool ok, int rows) const {
        const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int e = element(i, r, g);
                if (ok && e < rows) base[e * rs] = t[i][r];
            }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = dfloat4{0, 0, 0, 0};
    }
    // times 1 + x
    __device__ __forceinline__ void correct(float x) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) t[i][r] = fmaf(x, t[i][r], t[i][r]);
    }
    // as it is, `tiles` of its tiles
    __device__ __forceinline__ void store_tiles(float* to, int tiles) const {
        dfloat4* d = (dfloat4*)to + (threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < tiles) d[64 * i] = t[i];
    }
    // sum of the products with tiles so stored, of the lane
    __device__ __forceinline__ float times_tiles(const float* from, int tiles) const {
        const dfloat4* d = (const dfloat4*)from + (threadIdx.x & 63);
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < tiles) {
                const dfloat4 x = d[64 * i];
#pragma unroll
                for (int r = 0; r < 4; ++r) a += t[i][r] * x[r];
            }
        return a;
    }
};
// The anchor before a sequence's chunk number `chunk` of C tokens (a multiple of 1 << shift)
__device__ __forceinline__ long long anchor_of(const DecaySpans& p, const DecaySpan& s, int C,
                                               int shift, int chunk) {
    const long long n = (long long)C << shift;
    return (p.cu ? s.t0 / n + s.seq : s.b * ((p.T + n - 1) / n)) + (chunk >> shift);
}

// acc[m] = f o (rows A times S) for the row tiles m
template <int IO, int DA, int C>
__device__ __forceinline__ void state_product(const RowReader<IO, DA>& rows, int lane, const char* A,
                                              const State<DA>& S, const Factors<C>& F,
                                              dfloat4 (&acc)[C / 16]) {
    constexpr int M = C / 16, N = Kind<IO>::NT;
    const int g = lane >> 4;
    float back = 1.f, to = 1.f;
    if constexpr (IO == IO_F16) {
        const Scale sc = scale_to(S.largest());
        to = sc.to;
        back = sc.back;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) acc[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < DA / 32; ++kb) {
        Frag<IO> a[M], b[N];
#pragma unroll
        for (int m = 0; m < M; ++m) a[m] = rows.get(A, 16 * m, 32 * kb);
        const float s[8] = {S.t[2 * kb][0], S.t[2 * kb][1], S.t[2 * kb][2], S.t[2 * kb][3],
                            S.t[2 * kb + 1][0], S.t[2 * kb + 1][1], S.t[2 * kb + 1][2],
                            S.t[2 * kb + 1][3]};
        terms<IO, N>(s, to, b);
        if constexpr (IO == IO_F32) {
            // a chain of additions for each block of k: fewer roundings in a row
#pragma unroll
            for (int m = 0; m < M; ++m)
                acc[m] += mma16<IO>(a[m], b[0], dfloat4{0, 0, 0, 0});
        } else {
#pragma unroll
            for (int n = N - 1; n >= 0; --n)
#pragma unroll
                for (int m = 0; m < M; ++m) acc[m] = mma16<IO>(a[m], b[n], acc[m]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const float4 f = *(const float4*)&F.f[16 * m + 4 * g];
        acc[m][0] *= f.x * back;
        acc[m][1] *= f.y * back;
        acc[m][2] *= f.z * back;
        acc[m][3] *= f.w * back;
    }
}

// The values with 0 for those that are infinite or NaN; bad: the first (REV: last) of
// their tokens, t the first of the eight.
template <int IO, bool REV>
__device__ __forceinline__ Frag<IO> bounded(const Frag<IO>& v, int t, int& bad) {
    Frag<IO> x = v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bool ok;
        if constexpr (IO == IO_F32) {
            float& e = i < 4 ? ((float*)&x.a)[i & 3] : ((float*)&x.b)[i & 3];
            ok = finite(e);
            e = ok ? e : 0.f;
        } else {
            constexpr uint32_t top = IO == IO_F16 ? 0x7c00u : 0x7f80u;
            const int shift = 16 * (i & 1);
            ok = (x.v[i >> 1] >> shift & top) != top;
            if (!ok) x.v[i >> 1] &= 0xffff0000u >> shift;
        }
        if (!ok) bad = REV ? max(bad, t + i) : min(bad, t + i);
    }
    return x;
}
// acc += P V: values holds the column of V, block kb the tokens 32 kb ...  unbounded: one
// of V's values is infinite or NaN.  Those are left out, as they would meet the
// zeros of P, and the column's rows that see one become NaN.
template <int IO, int C, bool REV>
__device__ __forceinline__ void scores_product(const char* P, const float* back, int lane,
                                               const Frag<IO> (&values)[C / 32], bool unbounded,
                                               dfloat4 (&acc)[C / 16]) {
    typedef Scores<IO, C> L;
    constexpr int N = Kind<IO>::NT;
    const int g = lane >> 4;
    int bad = REV ? -1 : C;
#pragma unroll
    for (int kb = 0; kb < L::KB; ++kb) {
        Frag<IO> v = values[kb];
        if (unbounded) v = bounded<IO, REV>(v, 32 * kb + 8 * g, bad);
        dfloat4 s[L::M];
#pragma unroll
        for (int m = 0; m < L::M; ++m)
            s[m] = IO == IO_F16 ? dfloat4{0, 0, 0, 0} : acc[m];
#pragma unroll
        for (int n = N - 1; n >= 0; --n)
#pragma unroll
            for (int m = 0; m < L::M; ++m)
                if (REV ? kb >= m / 2 : kb <= m / 2)
                    s[m] = mma16<IO>(L::get(P, lane, n, m, kb), v, s[m]);
        products_done();
#pragma unroll
        for (int m = 0; m < L::M; ++m) {
            if constexpr (IO == IO_F16) {
                if (!(REV ? kb >= m / 2 : kb <= m / 2)) continue;
                const float4 f = *(const float4*)&back[kb * C + 16 * m + 4 * g];
                acc[m][0] += s[m][0] * f.x;
                acc[m][1] += s[m][1] * f.y;
                acc[m][2] += s[m][2] * f.z;
                acc[m][3] += s[m][3] * f.w;
            } else {
                acc[m] = s[m];
            }
        }
    }
    if (!unbounded) return;
    bad = REV ? max_all(bad) : min_all(bad);
#pragma unroll
    for (int m = 0; m < C / 16; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * m + 4 * g + r;
            if (REV ? t <= bad : t >= bad) acc[m][r] = __uint_as_float(0x7fc00000u);
        }
}

// eight values of the tokens t .. t + 7 times their w
template <int IO, int C>
__device__ __forceinline__ void weighted(const Frag<IO>& v, const Factors<C>& F, int t, float (&x)[8]) {
    unpack_frag<IO>(v, x);
    const float4 a = *(const float4*)&F.w[t], b = *(const float4*)&F.w[t + 4];
    x[0] *= a.x; x[1] *= a.y; x[2] *= a.z; x[3] *= a.w;
    x[4] *= b.x; x[5] *= b.y; x[6] *= b.z; x[7] *= b.w;
}
// What the roundings of e^Dc left of a state, in parts of it.  With equal decays that
// is the same number chunk after chunk, up to 2^-25: over the 1024 chunks of a slow
// decay 3e-5 of the state, where its own roundings, either way, come to 1e-6.  So it is
// summed and given back every eighth chunk (2^-22 at most by then), which costs an
// eighth of a vector instruction for each element and chunk.
struct Drift {
    float sum = 0.f;
    template <int DA>
    __device__ __forceinline__ void after(float err, int chunk, bool last, State<DA>& S) {
        sum += err;
        if ((chunk & 7) != 7 && !last) return;
        S.correct(sum);
        sum = 0.f;
    }
};
// S <- e^Dc S + B^T (w o V).  The chunk's part is summed by itself: one rounding of the
// state a chunk.  G: tiles at a time.
template <int IO, int DA, int C, int G>
__device__ __forceinline__ void update_state(const ColReader<IO, DA, true>& cols, int lane,
                                             const char* B, const Frag<IO> (&values)[C / 32],
                                             const Factors<C>& F, State<DA>& S) {
    constexpr int N = Kind<IO>::NT, KB = C / 32;
    const int g = lane >> 4;
    const float all = F.all;
    float to = 1.f, back = 1.f;
    if constexpr (IO == IO_F16) {
        float largest = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            float x[8];
            weighted<IO, C>(values[kb], F, 32 * kb + 8 * g, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) largest = fmaxf(largest, fabsf(x[i]));
        }
        largest = max_groups(largest);
        const Scale sc = scale_to(finite(largest) ? largest : 0.f);
        to = sc.to;
        back = sc.back;
    }
    Frag<IO> v[KB][N];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        float x[8];
        weighted<IO, C>(values[kb], F, 32 * kb + 8 * g, x);
        terms<IO, N>(x, to, v[kb]);
    }
#pragma unroll
    for (int i = 0; i < State<DA>::N; i += G) {
        dfloat4 part[G];
#pragma unroll
        for (int j = 0; j < G; ++j) part[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            Frag<IO> a[G];
#pragma unroll
            for (int j = 0; j < G; ++j) a[j] = cols.get(B, 32 * kb, i + j);
#pragma unroll
            for (int n = N - 1; n >= 0; --n)
#pragma unroll
                for (int j = 0; j < G; ++j) part[j] = mma16<IO>(a[j], v[kb][n], part[j]);
        }
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                S.t[i + j][r] = IO == IO_F16 ? fmaf(all, S.t[i + j][r], back * part[j][r])
                                             : fmaf(all, S.t[i + j][r], part[j][r]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The wave's 16 columns of the rows to their places in a tile, in the I/O type, for
// threads that then take whole pieces of it.
template <int IO, int D, int C>
__device__ __forceinline__ void rows_to_tile(const CellPlaces<IO, D>& cells, char* tile,
                                             const dfloat4 (&acc)[C / 16]) {
#pragma unroll
    for (int m = 0; m < C / 16; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) io_store<IO>(tile + cells.at(16 * m, r), 0, acc[m][r]);
}
// The rows below n to fp32 memory, `row` bytes apart.
template <int C>
__device__ __forceinline__ void rows_to_memory(int lane, char* out, uint32_t row, bool ok, int n,
                                               const dfloat4 (&acc)[C / 16]) {
    const int left = ok ? n - 4 * (lane >> 4) : 0;
    const uint32_t mine = (uint32_t)(4 * (lane >> 4)) * row + 4u * (lane & 15);
#pragma unroll
    for (int m = 0; m < C / 16; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (16 * m + r < left) *(float*)(out + ((16 * m + r) * row + mine)) = acc[m][r];
}

// Sums over the 16 lanes of a group: lane c gets that of t[c / 4].
__device__ __forceinline__ float sums16_of4(const float (&t)[4]) {
    const int c = threadIdx.x & 15;
    const bool up = c & 8, odd = c & 4;
    const float a = (up ? t[2] : t[0]) + moved<0x128>(up ? t[0] : t[2]);
    const float b = (up ? t[3] : t[1]) + moved<0x128>(up ? t[1] : t[3]);
    float x = (odd ? b : a) + moved<0x141>(odd ? a : b);
    x += moved<0xb1>(x);
    return x + moved<0x4e>(x);
}
// dots[t] = sum over the wave's 16 columns of acc and the rows X there
template <int IO, int D, int C>
__device__ __forceinline__ void row_dots(const CellPlaces<IO, D>& cells, int lane, const char* X,
                                         const dfloat4 (&acc)[C / 16], float* dots) {
#pragma unroll
    for (int m = 0; m < C / 16; ++m) {
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = acc[m][r] * io_load<IO>(X + cells.at(16 * m, r), 0);
        const float d = sums16_of4(x);
        if ((lane & 3) == 0) dots[16 * m + 4 * (lane >> 4) + ((lane & 15) >> 2)] = d;
    }
}

// Columns first .. first + n of the tokens that no sequence holds become 0, by the
// workgroups of the first and the last sequence's first segments.
__device__ __forceinline__ void clear_unheld(const DecaySpans& p, const DecaySpan& s, void* out,
                                             int bytes, int H, int cols, int h, int first, int n) {
    const long long step = (long long)H * cols * bytes;
    char* o = (char*)out + ((long long)h * cols + first) * bytes;
    if (s.seq == 0) clear_rows(o, step, (int)s.t0, n * bytes);
    const long long end = s.t0 + s.len;
    if (s.seq + 1 == p.nseq) clear_rows(o + end * step, step, (int)(p.T - end), n * bytes);
}

// Token matrices of one head of a span.
template <int IO>
__device__ __forceinline__ Tokens rows_of(const DecayRows& x, const DecaySpan& s, int h) {
    return tokens_of<IO>(x.p, s.b * x.st[0] + s.t0 * x.st[1] + (h / x.group) * x.st[2], x.st[1]);
}

}  // namespace fftconv
