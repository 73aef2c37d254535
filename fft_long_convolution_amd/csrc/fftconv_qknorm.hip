// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward.
//
// For a head x of D elements, with r = (c sum_i x_i^2 + eps)^(-1/2) and
// c = 1/D (root mean square) or 1 (2-norm):
//   n = w x r,   y = Rot(n)
// where Rot turns the pairs (i, i + R/2) or (2i, 2i+1) of the first R
// elements by the angle whose cosine and sine stand in the token's row of
// the tables.  Backward, with m = Rot^T(dy):
//   dw = sum over tokens and heads of m x r
//   dx = r (w m) - c r^3 x <x, w m>
// All arithmetic is fp32; the only rounding is the one of the outputs to the
// I/O type.
//
// The pass moves each element once in and once out and does some ten
// operations on it, so HBM bounds it: 64 x 1024 tokens of 12 heads of 128 in
// bf16, 403 MB, take 76 us (5.3 TB/s; a streaming copy reaches 6.0); fp32, 268 MB
// of q and k, 107 us forward and 159 backward (5.0 and 5.1).  A lane
// holds 8 consecutive elements (one 16-byte access at 16 bits, two at 32), the
// lanes of a head (D/8, rounded up to a power of two) sum by shuffles, and a
// group of lanes walks over heads of ONE token, so the token's cosines and
// sines are read once and stay in registers.
#include "fftconv_delta.h"

namespace fftconv {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;     // heads in flight in a group of lanes

typedef uint32_t qu4 __attribute__((ext_vector_type(4)));
template <int IO>
struct Raw8 { qu4 v; };
template <>
struct Raw8<IO_F32> { qu4 v, w; };

// NT: past the caches, for tensors that do not stay there anyway
template <bool NT>
__device__ __forceinline__ qu4 load16(const void* p) {
    return NT ? __builtin_nontemporal_load((const qu4*)p) : *(const qu4*)p;
}
template <bool NT>
__device__ __forceinline__ void store16(void* p, qu4 x) {
    if (NT) __builtin_nontemporal_store(x, (qu4*)p);
    else *(qu4*)p = x;
}

template <int IO, bool NT>
__device__ __forceinline__ Raw8<IO> load8(const void* p, long long i) {
    Raw8<IO> r;
    if constexpr (IO == IO_F32) {
        r.v = load16<NT>((const float*)p + i);
        r.w = load16<NT>((const float*)p + i + 4);
    } else {
        r.v = load16<NT>((const uint16_t*)p + i);
    }
    return r;
}

template <int IO>
__device__ __forceinline__ void unpack8(const Raw8<IO>& r, float (&x)[8]) {
    if constexpr (IO == IO_F32) {
        const uint32_t u[8] = {r.v.x, r.v.y, r.v.z, r.v.w, r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (IO == IO_BF16) {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                const h2 h = __builtin_bit_cast(h2, u[i]);
                x[2 * i] = (float)h.x;
                x[2 * i + 1] = (float)h.y;
            }
        }
    }
}

template <int IO, bool NT>
__device__ __forceinline__ void store8(void* p, long long i, const float (&x)[8]) {
    if constexpr (IO == IO_F32) {
        qu4 u[2];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j >> 2][j & 3] = __float_as_uint(x[j]);
        store16<NT>((float*)p + i, u[0]);
        store16<NT>((float*)p + i + 4, u[1]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (IO == IO_BF16) {
                __bf16 h[2] = {(__bf16)x[2 * j], (__bf16)x[2 * j + 1]};
                u[j] = __builtin_bit_cast(uint32_t, h);
            } else {
                _Float16 h[2] = {(_Float16)x[2 * j], (_Float16)x[2 * j + 1]};
                u[j] = __builtin_bit_cast(uint32_t, h);
            }
        }
        store16<NT>((uint16_t*)p + i, qu4{u[0], u[1], u[2], u[3]});
    }
}

// What a lane keeps for its token: its chunk's cosines and sines (the sine
// signed for the lane's side of the pair) and the lane that holds the other
// side.  interleaved: entry j turns the lane's pair (2j, 2j+1).
struct Turn {
    float c[8], s[8];
    int other;
    bool on;
};

// sgn = +1 turns forward, -1 back (the transpose).
template <int LPR>
__device__ __forceinline__ void load_turn(const QkNormParams& p, long long token, int c, float sgn,
                                          Turn& t) {
    t.on = c < (p.R >> 3);
    t.other = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) { t.c[i] = 1.f; t.s[i] = 0.f; }
    if (p.R == 0) return;
    const int lane = threadIdx.x & 63;
    const int half = p.R >> 4;             // chunks in half of the rotated part
    const bool lower = c < half;
    // lanes beyond the rotated part shuffle with themselves
    t.other = p.interleaved || !t.on ? lane : (lower ? lane + half : lane - half);
    if (!t.on) return;
    const long long row = p.pos[token];
    const float bad = __uint_as_float(0x7fc00000u);
    if (row < 0 || row >= p.P) {
        // no such row: the rotated elements become NaN, nothing is read
#pragma unroll
        for (int i = 0; i < 8; ++i) t.c[i] = t.s[i] = bad;
        return;
    }
    const float* cs = p.cs + row * (p.R >> 1);
    const float* sn = p.sn + row * (p.R >> 1);
    if (p.interleaved) {
        const float4 a = *(const float4*)(cs + 4 * c), b = *(const float4*)(sn + 4 * c);
        t.c[0] = a.x; t.c[1] = a.y; t.c[2] = a.z; t.c[3] = a.w;
        t.s[0] = sgn * b.x; t.s[1] = sgn * b.y; t.s[2] = sgn * b.z; t.s[3] = sgn * b.w;
    } else {
        const int e = 8 * (lower ? c : c - half);
        const float sg = lower ? -sgn : sgn;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 a = *(const float4*)(cs + e + 4 * j), b = *(const float4*)(sn + e + 4 * j);
            t.c[4 * j] = a.x; t.c[4 * j + 1] = a.y; t.c[4 * j + 2] = a.z; t.c[4 * j + 3] = a.w;
            t.s[4 * j] = sg * b.x; t.s[4 * j + 1] = sg * b.y;
            t.s[4 * j + 2] = sg * b.z; t.s[4 * j + 3] = sg * b.w;
        }
    }
}

__device__ __forceinline__ void turn8(const QkNormParams& p, const Turn& t, float (&x)[8]) {
    if (p.R == 0) return;
    if (p.interleaved) {
        if (!t.on) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * t.c[j] - b * t.s[j];
            x[2 * j + 1] = b * t.c[j] + a * t.s[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl(x[i], t.other);
            x[i] = t.on ? x[i] * t.c[i] + o * t.s[i] : x[i];
        }
    }
}

template <int LPR>
__device__ __forceinline__ float sum_row(float a) {
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) a += __shfl_xor(a, m);
    return a;
}

__device__ __forceinline__ void load_weight(const float* w, int c, bool have, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
    if (!w || !have) return;
    const float4 a = *(const float4*)(w + 8 * c), b = *(const float4*)(w + 8 * c + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// A group of LPR lanes takes (token, part): the heads part, part + parts, ...
// of the token's Hq + Hk.  All lanes of a wave run the same trip counts, so
// every shuffle has its partners; a lane without work holds zeros.
template <int IO, int LPR, bool NT>
__global__ __launch_bounds__(kThreads) void qknorm_fwd_kernel(QkNormParams p) {
    const int c = threadIdx.x & (LPR - 1);
    const long long unit = ((long long)blockIdx.x * kThreads + threadIdx.x) / LPR;
    const long long token = unit / p.parts;
    const int part = (int)(unit - token * p.parts);
    const bool have = token < p.tokens && 8 * c < p.D;
    const int H = p.Hq + p.Hk;
    Turn t;
    load_turn<LPR>(p, have ? token : 0, have ? c : p.D, 1.f, t);
    float wq[8], wk[8];
    load_weight(p.wq, c, have, wq);
    load_weight(p.wk, c, have, wk);
    const long long b = have ? token / p.T : 0, at = have ? token - b * p.T : 0;
    const long long qb = b * p.qs[0] + at * p.qs[1] + 8 * c;
    const long long kb = b * p.ks[0] + at * p.ks[1] + 8 * c;
    // trips of the part with the most heads, the same for all lanes
    const int trips = (H + p.parts - 1) / p.parts;
    for (int i0 = 0; i0 < trips; i0 += kUnroll) {
        Raw8<IO> raw[kUnroll];
        bool ok[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int h = part + (i0 + j) * p.parts;
            ok[j] = have && h < H;
            raw[j] = Raw8<IO>{};
            if (ok[j])
                raw[j] = h < p.Hq ? load8<IO, NT>(p.q, qb + h * p.qs[2])
                                  : load8<IO, NT>(p.k, kb + (h - p.Hq) * p.ks[2]);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (i0 + j >= trips) break;
            const int h = part + (i0 + j) * p.parts;
            float x[8];
            unpack8<IO>(raw[j], x);
            float a = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) a += x[i] * x[i];
            a = sum_row<LPR>(a);
            const float r = 1.f / sqrtf(p.c * a + p.eps);
            const bool isq = h < p.Hq;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (isq ? wq[i] : wk[i]);
            turn8(p, t, x);
            if (ok[j]) {
                if (isq) store8<IO, NT>(p.qo, (token * p.Hq + h) * p.D + 8 * c, x);
                else store8<IO, NT>(p.ko, (token * p.Hk + (h - p.Hq)) * p.D + 8 * c, x);
            }
        }
    }
}

template <int IO, int LPR, bool NT>
__global__ __launch_bounds__(kThreads) void qknorm_bwd_kernel(QkNormParams p) {
    const int c = threadIdx.x & (LPR - 1);
    const int H = p.Hq + p.Hk;
    const bool col = 8 * c < p.D;
    float wq[8], wk[8], gq[8], gk[8];
    load_weight(p.wq, c, col, wq);
    load_weight(p.wk, c, col, wk);
#pragma unroll
    for (int i = 0; i < 8; ++i) gq[i] = gk[i] = 0.f;
    constexpr int kGroups = kThreads / LPR;
    const long long units = p.tokens * p.parts;
    const int trips = (H + p.parts - 1) / p.parts;
    for (long long u0 = (long long)blockIdx.x * kGroups; u0 < units;
         u0 += (long long)gridDim.x * kGroups) {
        const long long unit = u0 + threadIdx.x / LPR;
        const long long token = unit / p.parts;
        const int part = (int)(unit - token * p.parts);
        const bool have = token < p.tokens && col;
        Turn t;
        load_turn<LPR>(p, have ? token : 0, have ? c : p.D, -1.f, t);
        const long long b = have ? token / p.T : 0, at = have ? token - b * p.T : 0;
        const long long qb = b * p.qs[0] + at * p.qs[1] + 8 * c;
        const long long kb = b * p.ks[0] + at * p.ks[1] + 8 * c;
        for (int i0 = 0; i0 < trips; i0 += kUnroll) {
            Raw8<IO> rx[kUnroll], rd[kUnroll];
            bool ok[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int h = part + (i0 + j) * p.parts;
                ok[j] = have && h < H;
                rx[j] = rd[j] = Raw8<IO>{};
                if (ok[j]) {
                    if (h < p.Hq) {
                        rx[j] = load8<IO, NT>(p.q, qb + h * p.qs[2]);
                        rd[j] = load8<IO, NT>(p.dqo, (token * p.Hq + h) * p.D + 8 * c);
                    } else {
                        rx[j] = load8<IO, NT>(p.k, kb + (h - p.Hq) * p.ks[2]);
                        rd[j] = load8<IO, NT>(p.dko, (token * p.Hk + (h - p.Hq)) * p.D + 8 * c);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                if (i0 + j >= trips) break;
                const int h = part + (i0 + j) * p.parts;
                const bool isq = h < p.Hq;
                float x[8], m[8];
                unpack8<IO>(rx[j], x);
                unpack8<IO>(rd[j], m);
                turn8(p, t, m);
                float a = 0.f, d = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a += x[i] * x[i];
                    d += x[i] * (m[i] * (isq ? wq[i] : wk[i]));
                }
                a = sum_row<LPR>(a);
                d = sum_row<LPR>(d);
                const float r = 1.f / sqrtf(p.c * a + p.eps);
                const float e = p.c * (r * d) * r * r;   // r^3 alone may overflow
                if (ok[j]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xr = x[i] * r * m[i];
                        if (isq) gq[i] += xr; else gk[i] += xr;
                        x[i] = r * (m[i] * (isq ? wq[i] : wk[i])) - x[i] * e;
                    }
                    if (isq) store8<IO, NT>(p.dq, (token * p.Hq + h) * p.D + 8 * c, x);
                    else store8<IO, NT>(p.dk, (token * p.Hk + (h - p.Hq)) * p.D + 8 * c, x);
                }
            }
        }
    }
    if (!p.part) return;
    // weight gradients of the block: the groups of a wave by shuffles, the
    // waves through LDS, in a fixed order
    __shared__ float sums[kThreads / 64][2][LPR * 8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int m = LPR; m < 64; m <<= 1) {
            gq[i] += __shfl_xor(gq[i], m);
            gk[i] += __shfl_xor(gk[i], m);
        }
    }
    if ((threadIdx.x & 63) < LPR) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sums[threadIdx.x >> 6][0][8 * c + i] = gq[i];
            sums[threadIdx.x >> 6][1][8 * c + i] = gk[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        const int w = i / p.D, e = i - w * p.D;
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < kThreads / 64; ++j) a += sums[j][w][e];
        p.part[(long long)blockIdx.x * 2 * p.D + i] = a;
    }
}

// Sums the blocks' weight gradients: a workgroup takes four columns, 64 threads
// a column, in a fixed order.
__global__ __launch_bounds__(256) void qknorm_dw_kernel(QkNormParams p) {
    __shared__ float sums[64][5];
    const int col = threadIdx.x & 3, row = threadIdx.x >> 2;
    const int i = blockIdx.x * 4 + col;          // 2 D is a multiple of four
    float a = 0.f;
#pragma unroll 4
    for (int b = row; b < p.blocks; b += 64) a += p.part[(long long)b * 2 * p.D + i];
    sums[row][col] = a;
    __syncthreads();
    if (row < 8) {
        a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a += sums[8 * row + j][col];
    }
    __syncthreads();
    if (row < 8) sums[row][col] = a;
    __syncthreads();
    if (row == 0) {
#pragma unroll
        for (int j = 1; j < 8; ++j) a += sums[j][col];
        float* d = i < p.D ? p.dwq : p.dwk;
        if (d) d[i < p.D ? i : i - p.D] = a;
    }
}

template <int IO, bool NT>
hipError_t fwd_nt(const QkNormParams& p, hipStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    const long long units = p.tokens * p.parts;
    const long long per = kThreads / lanes;
    const dim3 grid((unsigned)((units + per - 1) / per));
    switch (lanes) {
    case 8: hipLaunchKernelGGL((qknorm_fwd_kernel<IO, 8, NT>), grid, kThreads, 0, s, p); break;
    case 16: hipLaunchKernelGGL((qknorm_fwd_kernel<IO, 16, NT>), grid, kThreads, 0, s, p); break;
    default: hipLaunchKernelGGL((qknorm_fwd_kernel<IO, 32, NT>), grid, kThreads, 0, s, p); break;
    }
    return hipGetLastError();
}

template <int IO, bool NT>
hipError_t bwd_nt(const QkNormParams& p, hipStream_t s) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    const dim3 grid(p.blocks);
    switch (lanes) {
    case 8: hipLaunchKernelGGL((qknorm_bwd_kernel<IO, 8, NT>), grid, kThreads, 0, s, p); break;
    case 16: hipLaunchKernelGGL((qknorm_bwd_kernel<IO, 16, NT>), grid, kThreads, 0, s, p); break;
    default: hipLaunchKernelGGL((qknorm_bwd_kernel<IO, 32, NT>), grid, kThreads, 0, s, p); break;
    }
    return hipGetLastError();
}

// Whether q and k are so large that little of them is still in a cache (256 MB
// in all) when they are read again.  16 bits, 12 heads of 128, through the caches
// and past them: 128 MB forward 47 and 54 us, backward 87 and 81; 192 MB 80 and 75,
// 122 and 114; 256 MB 102 and 96, 161 and 152; 64 MB 29 and 32, 46 and 47.  fp32 is
// slower past them at every size (192 MB: 82 and 87, 122 and 130).
bool streams(const QkNormParams& p) {
    return p.tokens * (p.Hq + p.Hk) * p.D * 2 > (160ll << 20);
}
template <int IO>
hipError_t fwd_io(const QkNormParams& p, hipStream_t s) {
    if constexpr (IO != IO_F32)
        if (streams(p)) return fwd_nt<IO, true>(p, s);
    return fwd_nt<IO, false>(p, s);
}
template <int IO>
hipError_t bwd_io(const QkNormParams& p, hipStream_t s) {
    if constexpr (IO != IO_F32)
        if (streams(p)) return bwd_nt<IO, true>(p, s);
    return bwd_nt<IO, false>(p, s);
}

}  // namespace

// Workgroups of the backward pass: they keep their weight-gradient sums to
// the end, so as many as run at once, three on each of the 256 CUs (their
// registers allow no more; 1024 leave a second round of a third: 168 us where
// 768 take 152).
int qknorm_bwd_blocks(long long tokens) {
    const long long n = (tokens + 3) / 4;
    return (int)(n < 1 ? 1 : n > 768 ? 768 : n);
}

hipError_t launch_qknorm_fwd(int io, const QkNormParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return fwd_io<IO_F32>(p, s);
    case IO_F16: return fwd_io<IO_F16>(p, s);
    default: return fwd_io<IO_BF16>(p, s);
    }
}

hipError_t launch_qknorm_bwd(int io, const QkNormParams& p, hipStream_t s) {
    hipError_t e;
    switch (io) {
    case IO_F32: e = bwd_io<IO_F32>(p, s); break;
    case IO_F16: e = bwd_io<IO_F16>(p, s); break;
    default: e = bwd_io<IO_BF16>(p, s); break;
    }
    if (e != hipSuccess || !p.part) return e;
    hipLaunchKernelGGL(qknorm_dw_kernel, dim3(2 * p.D / 4), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace fftconv
