// Device helpers of linear attention with a decay for each head: spans of
// sequences, token matrices in LDS, products on the matrix cores, and the steps
// of a chunk that the forward and the backward walks share.
//
// A walk takes a sequence's chunks of C tokens one after the other with a state
// S (DA x columns) in the accumulators of its waves, 32 columns a wave.  With rows
// A, B of DA elements and rows V of the columns, and D_t the sum of the log decays
// from the chunk's first token to t:
//   out = f o (A S) + P V,   P_ts = Gam_ts A_t.B_s
//   S  <- e^Dc S + B^T (w o V)
// forward in time f = e^D, w = e^(Dc-D), Gam_ts = e^(D_t-D_s) for s <= t; backward
// f = e^(Dc-D), w = e^D, Gam_ts = e^(D_s-D_t) for s >= t (and constant factors).
//
// Matrix products.  16-bit rows are exact operands.  An fp32 operand is written
// in terms of that type, each the rounding of what the ones before leave: of
// bf16 three for states (26 bits) and two for scores (17 bits: they meet outputs of 8),
// with fp32's range; of f16 two (22 bits), with a power of two for each column
// (states, weighted values) or row (scores) that takes the largest to 2^14.
// fp32 rows go to the fp32 matrix instructions as they are, which have 1/16 of
// the rate, and so have all operands 24 bits.
//
// Operand order.  The 32 x 32 instructions take 16 k at a time: lane (g = l/32, c
// = l%32) gives A[row c][k = 8g + i], B[k = 8g + i][col c], i < 8, and has D[row
// 8a + 4g + b][col c] in register 4a + b.  Row 8a + 4g + b of a 32-row tile of
// the state stands for element 16 (a/2) + 8g + 4 (a%2) + b, so that a lane's
// accumulators are the eight k that it gives as B of the next product.  fp32:
// the same places, eight instructions of two k.
#pragma once

#include "fftconv_decay.h"
#include "fftconv_delta_dev.h"

namespace fftconv {

typedef float dfloat16 __attribute__((ext_vector_type(16)));

template <int IO>
struct Kind {
    static constexpr int kB = IO == IO_F32 ? 4 : 2;
    static constexpr int NS = IO == IO_BF16 ? 3 : IO == IO_F16 ? 2 : 1;   // terms of a state
    static constexpr int NP = IO == IO_F32 ? 1 : 2;                       // of scores
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
// 16-element groups (transposed reads) each meet all banks.
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
// The lane, unknown to the compiler: what follows from it is made where it is
// used instead of being kept in registers over the whole walk.
__device__ __forceinline__ int fresh_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
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
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Rows as operands with k along the elements: lane (g, c), of lanes in groups of G,
// has token t0 + c at elements e0 + 8g + i, i < 8; t0 a multiple of 16, e0 of 16.
template <int IO, int D, int G>
struct RowReader {
    uint32_t base;
    __device__ __forceinline__ explicit RowReader(int lane)
        : base(Rows<IO, D>::at(lane & (G - 1), (lane / G) * (IO == IO_F32 ? 2 : 1))) {}
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
// at element e0 + c, or, STATE, at the element that row c of a tile of the state
// stands for; t0 a multiple of 16, e0 of 32.
template <int IO, int D, bool STATE>
struct ColReader {
    typedef Rows<IO, D> R;
    uint32_t base;
    __device__ __forceinline__ explicit ColReader(int lane) {
        if constexpr (IO == IO_F32) {
            const int c = lane & 31;
            const int e = STATE ? (c & 19) | ((c & 8) >> 1) | ((c & 4) << 1) : c;
            base = R::at(8 * (lane >> 5), e >> 2) + 4 * (e & 3);
        } else {
            // each read takes, from 16 lanes, four tokens by four pieces of four
            // elements, and gives lane j the four tokens' element j of the pieces in
            // the lanes' order: the state's order swaps the middle two
            const int j = lane & 15;
            int piece = j & 3;
            if (STATE) piece = (piece >> 1) | ((piece & 1) << 1);
            base = R::at(8 * (lane >> 5) + (j >> 2), 2 * ((lane >> 4) & 1) + (piece >> 1)) +
                   8 * (piece & 1);
        }
    }
    __device__ __forceinline__ Frag<IO> get(const char* m, int t0, int e0) const {
        const char* s = m + t0 * R::kRow;
        Frag<IO> f;
        if constexpr (IO == IO_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = *(const float*)(
                    s + i * R::kRow + (base ^ (uint32_t)(e0 << 2) ^ (swirl<R::kPieces>(i) << 4)));
                if (i < 4) f.a[i & 3] = x; else f.b[i & 3] = x;
            }
        } else {
            typedef short s4 __attribute__((ext_vector_type(4)));
            uint2 r[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const char* x = s + 4 * half * R::kRow +
                                (base ^ (uint32_t)(e0 << 1) ^ (swirl<R::kPieces>(4 * half) << 4));
                r[half] = __builtin_bit_cast(
                    uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                               (__attribute__((address_space(3))) s4*)x));
            }
            f.v = du4{r[0].x, r[0].y, r[1].x, r[1].y};
        }
        return f;
    }
};

// C tokens of rows on their way from memory to LDS, by N threads (tid < N):
// tokens from n on and pieces from the row's end on are 0.
template <int IO, int D, int C, int N>
struct Moving {
    static constexpr int kPieces = Rows<IO, D>::kPieces, kMine = C * kPieces / N;
    static_assert(C * kPieces % N == 0, "threads share the pieces evenly");
    du4 r[kMine];
    static constexpr int kStep = N / kPieces;           // tokens between a thread's pieces
    static_assert(N % kPieces == 0, "a thread keeps its piece");
    // Loads in flight may meet neither an instruction nor the end of a branch: those
    // of what is not there read the first piece, and are dropped by clear().
    __device__ __forceinline__ void load(const Tokens& x, long long token, int n, int pieces,
                                         int tid) {
        const char* p = x.at(token);
        const uint32_t stride = (uint32_t)x.bytes;
        tid = fresh(tid);
        const int u = tid % kPieces, left = u < pieces ? n - tid / kPieces : 0;
        const uint32_t mine = (uint32_t)(tid / kPieces) * stride + 16u * u;
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            r[j] = *(const du4*)(p + (j * kStep < left ? mine + j * kStep * stride : 0u));
    }
    __device__ __forceinline__ void clear(int n, int pieces, int tid) {
        if (n >= C && pieces >= kPieces) return;
        tid = fresh(tid);
        const int left = tid % kPieces < pieces ? n - tid / kPieces : 0;
#pragma unroll
        for (int j = 0; j < kMine; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) r[j][w] = j * kStep < left ? r[j][w] : 0;
    }
    __device__ __forceinline__ void store(char* m, int tid) const {
        tid = fresh(tid);
#pragma unroll
        for (int j = 0; j < kMine; ++j)
            *(du4*)(m + Rows<IO, D>::at(j * kStep + tid / kPieces, tid % kPieces)) = r[j];
    }
    // whether an element is infinite or NaN
    __device__ __forceinline__ bool unbounded() const {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < kMine; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t u = r[j][w];
                if constexpr (IO == IO_F32) {
                    most = max(most, u & 0x7fffffffu);
                } else {
                    most = max(most, max((u & 0x7fffu) << 16, u & 0x7fff0000u));
                }
            }
        return most >= (IO == IO_F16 ? 0x7c000000u : 0x7f800000u);
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
template <int IO>
__device__ __forceinline__ dfloat16 mma32(const Frag<IO>& a, const Frag<IO>& b, dfloat16 c) {
    if constexpr (IO == IO_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.a[i], b.a[i], c, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.b[i], b.b[i], c, 0, 0, 0);
        return c;
    } else if constexpr (IO == IO_F16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(dh8, a.v),
                                                      __builtin_bit_cast(dh8, b.v), c, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(dbf8, a.v),
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
                    const uint32_t u = __builtin_bit_cast(uint32_t, h);
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

// the larger of the lane's value and that of the other half of the wave
__device__ __forceinline__ float max_halves(float a) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
__device__ __forceinline__ int min_halves(int a) {
    const auto x = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)a, false, false);
    return min((int)x[0], (int)x[1]);
}
__device__ __forceinline__ int max_halves(int a) {
    const auto x = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)a, false, false);
    return max((int)x[0], (int)x[1]);
}

// -------------------------------------------------------- factors of a chunk

// Sums of log decays in units of log 2, as a whole number and a rest of at most a
// half: their differences are right to 2^-24 however large the sums are.
template <int C>
struct Factors {
    int whole[C];
    float rest[C];
    float f[C], w[C];        // of the rows of the state's product, of the values
    float all;               // e^Dc
    int unbounded;           // an infinite or NaN value in the chunk
};
struct Power { int whole; float rest; };
__device__ __forceinline__ Power power_of(double x) {
    const double n = __builtin_rint(x);
    return {(int)n, (float)(x - n)};
}
__device__ __forceinline__ float exp2_of(int whole, float rest) {
    return __builtin_ldexpf(__builtin_amdgcn_exp2f(rest), whole);
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
    const Power p = power_of(D), r = power_of(all - D);
    const float to = exp2_of(p.whole, p.rest), from = exp2_of(r.whole, r.rest);
    if (lane < C) {
        F.whole[lane] = p.whole;
        F.rest[lane] = p.rest;
        F.f[lane] = sf * (REV ? from : to);
        F.w[lane] = sw * (REV ? to : from);
        if (lane == C - 1) F.all = to;
    }
}

// ------------------------------------------------------- the steps of a chunk

// Scores P (rows A against rows B) by NW waves, as operands of 32 rows x 16 k: block
// (m, kb) of term i at ((i * C/32 + m) * C/16 + kb) * 64 + lane.  f16: rows scaled, back
// holds the inverse scales.
template <int IO, int C>
struct Scores {
    static constexpr int kBlock = 64 * (IO == IO_F32 ? 32 : 16), kBlocks = (C / 32) * (C / 16);
    static constexpr int kTerm = kBlock * kBlocks, kBytes = kTerm * Kind<IO>::NP;
    static __device__ __forceinline__ Frag<IO> get(const char* P, int lane, int term, int m, int kb) {
        return *(const Frag<IO>*)(P + term * kTerm + (m * (C / 16) + kb) * kBlock +
                                  lane * (int)sizeof(Frag<IO>));
    }
};
// The lane's rows 16 kt + 4 g + r of B, r < 4, for its row 16 qt + c of A.
template <int IO, int C>
__device__ __forceinline__ void put_scores(char* P, int lane, int qt, int kt, float to,
                                           dfloat4 p) {
    constexpr int NP = Kind<IO>::NP;
    const int g = lane >> 4, c = lane & 15;
    const int place = ((qt >> 1) * (C / 16) + kt) * 64 + (g >> 1) * 32 + 16 * (qt & 1) + c;
    if constexpr (IO == IO_F32) {
        *(dfloat4*)(P + place * 32 + (g & 1) * 16) = p;
    } else {
        const float x[8] = {p[0], p[1], p[2], p[3], 0, 0, 0, 0};
        Frag<IO> t[NP];
        terms<IO, NP>(x, to, t);
#pragma unroll
        for (int n = 0; n < NP; ++n)
            *(uint2*)(P + n * Scores<IO, C>::kTerm + place * 16 + (g & 1) * 8) =
                make_uint2(t[n].v[0], t[n].v[1]);
    }
}
template <int IO, int DA, int C, int NW, bool REV>
__device__ __forceinline__ void make_scores(const char* A, const char* B, char* P, float* back,
                                            const Factors<C>& F, float scale, int wave) {
    constexpr int KT = C / 16;
    const int lane = fresh_lane(), g = lane >> 4, c = lane & 15;
    const RowReader<IO, DA, 16> rows(lane);
    if (NW > KT && wave >= KT) return;
#pragma unroll
    for (int j = 0; j < (KT + NW - 1) / NW; ++j) {
        const int qt = wave + NW * j;
        dfloat4 acc[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) acc[kt] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < DA / 32; ++kb) {
            const Frag<IO> b = rows.get(A, 16 * qt, 32 * kb);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                acc[kt] = mma16<IO>(rows.get(B, 16 * kt, 32 * kb), b, acc[kt]);
            __builtin_amdgcn_sched_barrier(0);
        }
        products_done();
        const int i = 16 * qt + c, iw = F.whole[i];
        const float ir = F.rest[i];
        float largest = 0.f;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            const int s0 = 16 * kt + 4 * g;
            const int4 sw = *(const int4*)&F.whole[s0];
            const float4 sr = *(const float4*)&F.rest[s0];
            const int w[4] = {sw.x, sw.y, sw.z, sw.w};
            const float r[4] = {sr.x, sr.y, sr.z, sr.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float gam = REV ? exp2_of(w[e] - iw, r[e] - ir) : exp2_of(iw - w[e], ir - r[e]);
                const bool on = REV ? s0 + e >= i : s0 + e <= i;
                acc[kt][e] = on ? scale * gam * acc[kt][e] : 0.f;
                if (IO == IO_F16) largest = fmaxf(largest, fabsf(acc[kt][e]));
            }
        }
        float to = 1.f;
        if constexpr (IO == IO_F16) {
            // at most 2^54: scores below 2^-40 do not reach an f16 output
            const Scale sc = scale_to(fmaxf(max_groups(largest), 0x1p-40f));
            to = sc.to;
            if (g == 0) back[i] = sc.back;
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) put_scores<IO, C>(P, lane, qt, kt, to, acc[kt]);
    }
}

// The lane's columns of the state: tiles of 32 elements.
template <int DA>
struct State {
    dfloat16 t[DA / 32];
    // largest magnitude of the column that is finite
    __device__ __forceinline__ float largest() const {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < DA / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) a = fmaxf(a, fabsf(t[i][r]));
        a = max_halves(a);
        return finite(a) ? a : 0.f;
    }
    // element of register r of tile i for the lane's half g
    static __device__ __forceinline__ int element(int i, int r, int g) {
        return 32 * i + 16 * (r >> 3) + 8 * g + (r & 7);
    }
    // base[element * rs + column * cs], elements below rows, where ok
    __device__ __forceinline__ void load(const float* base, long long rs, bool ok, int rows) {
        const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int i = 0; i < DA / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int e = element(i, r, g);
                const bool here = ok && e < rows;
                const float x = base[here ? e * rs : 0];
                t[i][r] = here ? x : 0.f;
            }
    }
    __device__ __forceinline__ void store(float* base, long long rs, bool ok, int rows) const {
        const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int i = 0; i < DA / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int e = element(i, r, g);
                if (ok && e < rows) base[e * rs] = t[i][r];
            }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < DA / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) t[i][r] = 0.f;
    }
};

// acc[m] = f o (rows A times S) for the 32-row tiles m
template <int IO, int DA, int C, int NS>
__device__ __forceinline__ void state_product(const char* A, const State<DA>& S, const Factors<C>& F,
                                              dfloat16 (&acc)[C / 32]) {
    const int lane = fresh_lane(), g = lane >> 5;
    const RowReader<IO, DA, 32> rows(lane);
    float back = 1.f, to = 1.f;
    if constexpr (IO == IO_F16) {
        const Scale sc = scale_to(S.largest());
        to = sc.to;
        back = sc.back;
    }
#pragma unroll
    for (int m = 0; m < C / 32; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[m][r] = 0.f;
#pragma unroll
    for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float s[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) s[r] = S.t[i][8 * x + r];
            Frag<IO> b[NS];
            terms<IO, NS>(s, to, b);
            Frag<IO> a[C / 32];
#pragma unroll
            for (int m = 0; m < C / 32; ++m)
                a[m] = rows.get(A, 32 * m, 32 * i + 16 * x);
#pragma unroll
            for (int n = NS - 1; n >= 0; --n)
#pragma unroll
                for (int m = 0; m < C / 32; ++m) acc[m] = mma32<IO>(a[m], b[n], acc[m]);
            __builtin_amdgcn_sched_barrier(0);
        }
    products_done();
#pragma unroll
    for (int m = 0; m < C / 32; ++m)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const float4 f = *(const float4*)&F.f[32 * m + 8 * a + 4 * g];
            acc[m][4 * a] *= f.x * back;
            acc[m][4 * a + 1] *= f.y * back;
            acc[m][4 * a + 2] *= f.z * back;
            acc[m][4 * a + 3] *= f.w * back;
        }
}

// acc += P V: v holds the columns of V, block kb the tokens 16 kb ...
template <int IO, int C, bool REV>
__device__ __forceinline__ void add_scores(const char* P, const float* back, int lane,
                                           const Frag<IO> (&v)[C / 16], dfloat16 (&acc)[C / 32]) {
    constexpr int NP = Kind<IO>::NP, KB = C / 16;
    const int g = lane >> 5;
#pragma unroll
    for (int m = 0; m < C / 32; ++m) {
        dfloat16 s;
        if constexpr (IO == IO_F16)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = 0.f;
        else s = acc[m];
#pragma unroll
        for (int n = NP - 1; n >= 0; --n)
#pragma unroll
            for (int kb = REV ? 2 * m : 0; kb < (REV ? KB : 2 * m + 2); ++kb)
                s = mma32<IO>(Scores<IO, C>::get(P, lane, n, m, kb), v[kb], s);
        products_done();
        if constexpr (IO == IO_F16) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float4 f = *(const float4*)&back[32 * m + 8 * a + 4 * g];
                acc[m][4 * a] += s[4 * a] * f.x;
                acc[m][4 * a + 1] += s[4 * a + 1] * f.y;
                acc[m][4 * a + 2] += s[4 * a + 2] * f.z;
                acc[m][4 * a + 3] += s[4 * a + 3] * f.w;
            }
        } else {
            acc[m] = s;
        }
    }
}
// The same where V may hold a value that is infinite or NaN: it is left out, as it
// would meet the zeros of P, and the column's rows that see it become NaN.
template <int IO, int C, bool REV>
__device__ __forceinline__ void scores_product(const char* P, const float* back,
                                               const Frag<IO> (&values)[C / 16], bool unbounded,
                                               dfloat16 (&acc)[C / 32]) {
    constexpr int KB = C / 16;
    const int lane = fresh_lane(), g = lane >> 5;
    if (!unbounded) {
        add_scores<IO, C, REV>(P, back, lane, values, acc);
        return;
    }
    Frag<IO> v[KB];
    int bad = REV ? -1 : C;            // the first (last) such token of the column
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        float x[8];
        unpack_frag<IO>(values[kb], x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!finite(x[i])) {
                const int t = 16 * kb + 8 * g + i;
                bad = REV ? max(bad, t) : min(bad, t);
                x[i] = 0.f;
            }
        Frag<IO> t[1];
        terms<IO, 1>(x, 1.f, t);       // exact: they are of the type
        v[kb] = t[0];
    }
    bad = REV ? max_halves(bad) : min_halves(bad);
    add_scores<IO, C, REV>(P, back, lane, v, acc);
#pragma unroll
    for (int m = 0; m < C / 32; ++m)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int t = 32 * m + 8 * (r >> 2) + 4 * g + (r & 3);
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
// S <- e^Dc S + B^T (w o V)
template <int IO, int DA, int C>
__device__ __forceinline__ void update_state(const char* B, const Frag<IO> (&values)[C / 16],
                                             const Factors<C>& F, State<DA>& S) {
    constexpr int NS = Kind<IO>::NS, KB = C / 16;
    const int lane = fresh_lane(), g = lane >> 5;
    const ColReader<IO, DA, true> cols(lane);
    float all = F.all, to = 1.f, back = 1.f;
    if constexpr (IO == IO_F16) {
        // the column's scale; values of less than 2^-24 of the state do not
        // reach it, and so do not ask for a larger one
        float largest = 0.f;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            float x[8];
            weighted<IO, C>(values[kb], F, 16 * kb + 8 * g, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) largest = fmaxf(largest, fabsf(x[i]));
        }
        largest = max_halves(largest);
        const Scale sc = scale_to(fmaxf(finite(largest) ? largest : 0.f, S.largest() * all * 0x1p-24f));
        to = sc.to;
        back = sc.back;
        all *= to;
    }
#pragma unroll
    for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) S.t[i][r] *= all;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        float x[8];
        Frag<IO> v[NS];
        weighted<IO, C>(values[kb], F, 16 * kb + 8 * g, x);
        terms<IO, NS>(x, to, v);
        Frag<IO> a[DA / 32];
#pragma unroll
        for (int i = 0; i < DA / 32; ++i) a[i] = cols.get(B, 16 * kb, 32 * i);
#pragma unroll
        for (int n = NS - 1; n >= 0; --n)
#pragma unroll
            for (int i = 0; i < DA / 32; ++i) S.t[i] = mma32<IO>(a[i], v[n], S.t[i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    products_done();
    if constexpr (IO == IO_F16)
#pragma unroll
        for (int i = 0; i < DA / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) S.t[i][r] *= back;
}

// The wave's 32 columns of the rows below n to memory, `row` bytes apart, through the
// places of its columns in a tile that nobody else uses (columns first .. first + 32):
// stores of 16 bytes, four or eight lanes a row, where the accumulators would give
// 32 of two.  pieces: 16-byte pieces that there are.  wide: fp32 whatever the type.
template <int IO, int D, int C>
__device__ __forceinline__ void store_rows(char* tile, int first, const dfloat16 (&acc)[C / 32],
                                           char* out, long long row, int pieces, bool wide, int n) {
    typedef Rows<IO, D> R;
    constexpr int kB = R::kB, kPer = 16 / kB;
    const int lane = fresh_lane(), g = lane >> 5, c = lane & 31;
    const auto drain = [&](int t0, int tokens, int per, auto place) {
        asm volatile("" ::: "memory");
        const int u = lane % per, left = u < pieces ? n - t0 - lane / per : 0;
        char* to = out + t0 * row;
        const uint32_t mine = (uint32_t)(lane / per) * (uint32_t)row + 16u * u;
#pragma unroll
        for (int j = 0; j < tokens * per / 64; ++j) {
            const int t = j * (64 / per);
            const du4 x = *(const du4*)(tile + place(t + lane / per, u));
            if (t < left) *(du4*)(to + t * row + mine) = x;
        }
        asm volatile("" ::: "memory");
    };
    if (IO == IO_F32 || !wide) {
        const uint32_t base = R::at(4 * g, (first + c) / kPer) + (first + c) % kPer * kB;
#pragma unroll
        for (int m = 0; m < C / 32; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = 8 * (r >> 2) + (r & 3);
                io_store<IO>(tile + (32 * m + t) * R::kRow + (base ^ (swirl<R::kPieces>(t) << 4)), 0,
                             acc[m][r]);
            }
        drain(0, C, 32 / kPer, [&](int t, int u) { return R::at(t, first / kPer + u); });
    } else {
        // half of the tokens at a time: a row's upper 16 columns C/2 rows on
        const uint32_t base = R::at(4 * g + (c >> 4) * (C / 2), first / kPer + ((c >> 2) & 3)) +
                              4 * (c & 3);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int f = half * C / 4; f < (half + 1) * C / 4; ++f) {
                const int t = (32 * (f >> 4) + 8 * ((f & 15) >> 2) + (f & 3)) % (C / 2);
                *(float*)(tile + t * R::kRow + (base ^ (swirl<R::kPieces>(t) << 4))) =
                    acc[f >> 4][f & 15];
            }
            drain(half * (C / 2), C / 2, 8, [&](int t, int u) {
                return R::at(t + (u >> 2) * (C / 2), first / kPer + (u & 3));
            });
        }
    }
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
// sum of the lane's value and its neighbour group's of 16 in the half of the wave
__device__ __forceinline__ float sum_pair(float a) {
    const auto y = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false,
                                                    false);
    return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}
// dots[t] = sum over the wave's 32 columns of acc and the rows X at column first
template <int IO, int D, int C>
__device__ __forceinline__ void row_dots(const char* X, int first, const dfloat16 (&acc)[C / 32],
                                         float* dots) {
    typedef Rows<IO, D> R;
    const int lane = fresh_lane(), g = lane >> 5, e = first + (lane & 31);
    constexpr int kPer = 16 / Kind<IO>::kB;
    const uint32_t base = R::at(4 * g, e / kPer) + e % kPer * Kind<IO>::kB;
#pragma unroll
    for (int m = 0; m < C / 32; ++m)
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float x[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                x[b] = acc[m][4 * a + b] *
                       io_load<IO>(X + (32 * m + 8 * a + b) * R::kRow +
                                       (base ^ (swirl<R::kPieces>(8 * a + b) << 4)), 0);
            const float d = sum_pair(sums16_of4(x));
            if ((lane & 19) == 0) dots[32 * m + 8 * a + 4 * g + ((lane & 15) >> 2)] = d;
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
