// Layer norm of token rows, forward and backward.
//
// For a row x of D elements, with m its mean, s the mean of (x - m)^2 and
// r = (s + eps)^(-1/2):
//   n = (x - m) r,   y = w n + b
// Backward, with h = w dy:
//   dx = r (h - mean(h) - n mean(h n)),   dw = sum over rows of dy n,   db = of dy
// All arithmetic is fp32; the only rounding is the one of the outputs to the I/O
// type.  A row stays in registers between its sums: s is of differences
// already taken, and m and r are not kept for the backward pass, which has the
// row in hand anyway.
//
// Each element moves once in and once out (backward twice in) with some ten operations:
// HBM bounds both passes.  64 x 1024 rows of 768 in bf16, 201 MB, take 31 us and a call 38
// (6.5 and 5.2 TB/s: part of so many bytes stays in the 256 MB of caches; a streaming copy
// of 2 GB reaches 5.9), 16 x 8192 of 768 in f16 forward and backward, 1.0 GB, 198 us
// (5.1).  A lane of a row's group holds its pieces of eight elements from the load to the
// store; the sums go by shuffles, of rows of more than 2048 through LDS.
#include "fftconv_decay.h"
#include "fftconv_delta_dev.h"

namespace fftconv {
namespace {

// Groups of LPR lanes take a row each, every lane V pieces of 8 elements: WIDE,
// eight in a row (16-byte accesses), else LPR apart (rows that are not aligned).
template <int LPR>
constexpr int kGroupThreads = LPR > 256 ? LPR : 256;

template <int LPR, bool WIDE>
__device__ __forceinline__ int place(int v, int c) {
    return WIDE ? 8 * (v * LPR + c) : 8 * v * LPR + c;
}
// A piece as loaded.
template <int IO, bool WIDE>
struct Piece {
    static constexpr int kWords = WIDE ? (IO == IO_F32 ? 2 : 1) : 8;
    du4 wide[WIDE ? kWords : 1];
    float each[WIDE ? 1 : 8];
};
// A piece that is used at once: what is not there is 0.
template <int IO, int LPR, bool WIDE>
__device__ __forceinline__ void load_now(const void* p, long long at, int v, int c, int D, bool have,
                                         float (&x)[8]) {
    const int e = place<LPR, WIDE>(v, c);
    if constexpr (WIDE) {
        const bool ok = have && e < D;
        constexpr int n = IO == IO_F32 ? 2 : 1;
        du4 r[n];
#pragma unroll
        for (int j = 0; j < n; ++j) {
            r[j] = du4{0, 0, 0, 0};
            if (ok) r[j] = *(const du4*)((const char*)p + (at + e) * (IO == IO_F32 ? 4 : 2) + 16 * j);
        }
        unpack8<IO>(r, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool ok = have && e + i * LPR < D;
            x[i] = 0.f;
            if (ok) x[i] = io_load<IO>(p, at + e + i * LPR);
        }
    }
}
// One that stays in flight: what is not there reads the row's first elements, as it may
// meet no branch's end, and is dropped by unpack_piece().
template <int IO, int LPR, bool WIDE>
__device__ __forceinline__ void load_piece(const void* p, long long at, int v, int c, int D,
                                           Piece<IO, WIDE>& x) {
    const int e = place<LPR, WIDE>(v, c);
    if constexpr (WIDE) {
        constexpr int kB = IO == IO_F32 ? 4 : 2;
#pragma unroll
        for (int j = 0; j < Piece<IO, WIDE>::kWords; ++j)
            x.wide[j] = *(const du4*)((const char*)p + (at + (e < D ? e : 0)) * kB + 16 * j);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x.each[i] = io_load<IO>(p, at + (e + i * LPR < D ? e + i * LPR : 0));
    }
}
template <int IO, int LPR, bool WIDE>
__device__ __forceinline__ void unpack_piece(const Piece<IO, WIDE>& p, int v, int c, int D, bool have,
                                             float (&x)[8]) {
    const int e = place<LPR, WIDE>(v, c);
    if constexpr (WIDE) unpack8<IO>(p.wide, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool ok = have && (WIDE ? e : e + i * LPR) < D;
        x[i] = ok ? (WIDE ? x[i] : p.each[i]) : 0.f;
    }
}
// past: by the caches
template <int IO, int LPR, bool WIDE>
__device__ __forceinline__ void store_piece(void* p, long long at, int v, int c, int D,
                                            const float (&x)[8], bool past = false) {
    const int e = place<LPR, WIDE>(v, c);
    if constexpr (WIDE) {
        if (e >= D) return;
        if constexpr (IO == IO_F32) {
            store4<IO>(p, at + e, dfloat4{x[0], x[1], x[2], x[3]});
            store4<IO>(p, at + e + 4, dfloat4{x[4], x[5], x[6], x[7]});
        } else {
            du4 u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (IO == IO_BF16) {
                    const __bf16 h[2] = {(__bf16)x[2 * j], (__bf16)x[2 * j + 1]};
                    u[j] = __builtin_bit_cast(uint32_t, h);
                } else {
                    const dh2 h = {(_Float16)x[2 * j], (_Float16)x[2 * j + 1]};
                    u[j] = __builtin_bit_cast(uint32_t, h);
                }
            }
            du4* const to = (du4*)((char*)p + (at + e) * 2);
            if (past) __builtin_nontemporal_store(u, to);
            else *to = u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i * LPR < D) io_store<IO>(p, at + e + i * LPR, x[i]);
    }
}
template <int LPR, bool WIDE>
__device__ __forceinline__ bool inside(int v, int c, int i, int D) {
    return place<LPR, WIDE>(v, c) + (WIDE ? i : i * LPR) < D;
}

// sums over the group; of more than a wave, through LDS (all its waves call it)
template <int LPR>
__device__ __forceinline__ void sum_group(float& a, float& b, float2* lds) {
#pragma unroll
    for (int m = 1; m < (LPR < 64 ? LPR : 64); m <<= 1) {
        a += __shfl_xor(a, m);
        b += __shfl_xor(b, m);
    }
    if constexpr (LPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int i = 0; i < LPR / 64; ++i) {
            a += lds[i].x;
            b += lds[i].y;
        }
    }
}
template <int LPR>
__device__ __forceinline__ float sum_group(float a, float2* lds) {
    float none = 0.f;
    sum_group<LPR>(a, none, lds);
    return a;
}

// x becomes x - m; returns r
template <int LPR, int V, bool WIDE>
__device__ __forceinline__ float normal(const LayerNormParams& p, int c, float (&x)[V][8], float2* lds) {
    const float each = 1.f / (float)p.D;
    float a = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) a += x[v][i];
    const float mean = sum_group<LPR>(a, lds) * each;
    float sum = 0.f, square = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[v][i] = inside<LPR, WIDE>(v, c, i, p.D) ? x[v][i] - mean : 0.f;
            sum += x[v][i];
            square += x[v][i] * x[v][i];
        }
    sum_group<LPR>(sum, square, lds);
    // what the mean's rounding left of it (as much as the spread where the mean
    // is 2^24 times as large)
    const float rest = sum * each;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[v][i] = inside<LPR, WIDE>(v, c, i, p.D) ? x[v][i] - rest : 0.f;
    return 1.f / sqrtf(fmaxf(square * each - rest * rest, 0.f) + p.eps);
}

template <int LPR, int V, bool WIDE>
__device__ __forceinline__ void load_weights(const float* w, int c, int D, float other,
                                             float (&x)[V][8]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (w) {
            load_now<IO_F32, LPR, WIDE>(w, 0, v, c, D, true, x[v]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[v][i] = other;
        }
    }
}

template <int IO, int LPR, int V, bool WIDE>
__global__ __launch_bounds__(kGroupThreads<LPR>) void layernorm_fwd_kernel(LayerNormParams p) {
    __shared__ float2 lds[kGroupThreads<LPR> / 64];
    const int c = threadIdx.x & (LPR - 1);
    const long long row = (long long)blockIdx.x * (kGroupThreads<LPR> / LPR) + threadIdx.x / LPR;
    const bool have = row < p.rows;
    float x[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
        load_now<IO, LPR, WIDE>(p.x, (have ? row : 0) * p.stride, v, c, p.D, have, x[v]);
    float w[V][8], b[V][8];
    load_weights<LPR, V, WIDE>(p.w, c, p.D, 1.f, w);
    load_weights<LPR, V, WIDE>(p.b, c, p.D, 0.f, b);
    const float r = normal<LPR, V, WIDE>(p, c, x, lds);
    if (!have) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] = x[v][i] * r * w[v][i] + b[v][i];
        store_piece<IO, LPR, WIDE>(p.y, row * p.D, v, c, p.D, x[v], p.past);
    }
}

template <int IO, int LPR, int V, bool WIDE>
__global__ __launch_bounds__(kGroupThreads<LPR>) void layernorm_bwd_kernel(LayerNormParams p) {
    constexpr int N = kGroupThreads<LPR>, kGroups = N / LPR;
    __shared__ float2 lds[N / 64];
    const int c = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR;
    const float each = 1.f / (float)p.D;
    float w[V][8], gw[V][8], gb[V][8];
    load_weights<LPR, V, WIDE>(p.w, c, p.D, 1.f, w);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) gw[v][i] = gb[v][i] = 0.f;
    // the next row is on its way while this one is worked on, where that is few registers
    constexpr bool kAhead = WIDE && IO != IO_F32;
    Piece<IO, WIDE> rx[V], rd[V];
    const long long step = (long long)gridDim.x * kGroups;
    const auto fetch = [&](long long row) {
        row = row < p.rows ? row : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            load_piece<IO, LPR, WIDE>(p.x, row * p.stride, v, c, p.D, rx[v]);
            load_piece<IO, LPR, WIDE>(p.dy, row * p.D, v, c, p.D, rd[v]);
        }
    };
    if (kAhead && p.rows) fetch((long long)blockIdx.x * kGroups + group);
    for (long long row0 = (long long)blockIdx.x * kGroups; row0 < p.rows; row0 += step) {
        const long long row = row0 + group;
        const bool have = row < p.rows;
        float x[V][8], d[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (kAhead) {
                unpack_piece<IO, LPR, WIDE>(rx[v], v, c, p.D, have, x[v]);
                unpack_piece<IO, LPR, WIDE>(rd[v], v, c, p.D, have, d[v]);
            } else {
                load_now<IO, LPR, WIDE>(p.x, (have ? row : 0) * p.stride, v, c, p.D, have, x[v]);
                load_now<IO, LPR, WIDE>(p.dy, (have ? row : 0) * p.D, v, c, p.D, have, d[v]);
            }
        }
        if (kAhead) fetch(row + step);
        const float r = normal<LPR, V, WIDE>(p, c, x, lds);
        float h = 0.f, hn = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[v][i] *= r;
                // rows that are not there and places behind the end hold zeros
                if (have) {
                    gw[v][i] += d[v][i] * x[v][i];
                    gb[v][i] += d[v][i];
                }
                d[v][i] *= w[v][i];
                h += d[v][i];
                hn += d[v][i] * x[v][i];
            }
        sum_group<LPR>(h, hn, lds);
        h *= each;
        hn *= each;
        if (!have) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[v][i] = r * (d[v][i] - h - x[v][i] * hn);
            store_piece<IO, LPR, WIDE>(p.dx, row * p.D, v, c, p.D, x[v], p.past);
        }
    }
    if (!p.part) return;
    float* part = p.part + (long long)blockIdx.x * 2 * p.D;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            store_piece<IO_F32, LPR, WIDE>(part, 0, v, c, p.D, gw[v]);
            store_piece<IO_F32, LPR, WIDE>(part, p.D, v, c, p.D, gb[v]);
        }
    } else {
        // the groups of a wave by shuffles, then the waves, in a fixed order
        __shared__ float sums[N / 64][LPR][8];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                float(&g)[8] = which ? gb[v] : gw[v];
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int m = LPR; m < 64; m <<= 1) g[i] += __shfl_xor(g[i], m);
                __syncthreads();
                if ((threadIdx.x & 63) < LPR)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sums[threadIdx.x >> 6][c][i] = g[i];
                __syncthreads();
                if (threadIdx.x < LPR) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        g[i] = 0.f;
#pragma unroll
                        for (int j = 0; j < N / 64; ++j) g[i] += sums[j][c][i];
                    }
                    store_piece<IO_F32, LPR, WIDE>(part, which * (long long)p.D, v, c, p.D, g);
                }
            }
    }
}

// Sums the blocks' parts: a workgroup takes 16 of the 2 D columns, 16 threads a
// column, in a fixed order.
__global__ __launch_bounds__(256) void layernorm_sum_kernel(LayerNormParams p) {
    __shared__ float sums[16][17];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4, i = blockIdx.x * 16 + col;
    float a = 0.f;
    if (i < 2 * p.D)
#pragma unroll 8
        for (int b = row; b < p.blocks; b += 16) a += p.part[(long long)b * 2 * p.D + i];
    sums[row][col] = a;
    __syncthreads();
    if (row || i >= 2 * p.D) return;
    a = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) a += sums[j][col];
    float* d = i < p.D ? p.dw : p.db;
    if (d) d[i < p.D ? i : i - p.D] = a;
}

// Lanes of a row: up to four pieces a lane forward; backward, where a lane holds sums,
// weights and two rows too, up to two as far as that goes.
int lanes_of(int D, bool back) {
    const int n = (D + 7) / 8 * (back ? 2 : 1);
    return n <= 64 ? 16 : n <= 128 ? 32 : n <= 256 ? 64 : n <= 1024 ? 256 : 512;
}

template <int IO, int LPR, int V, bool WIDE>
hipError_t launch(const LayerNormParams& p, bool back, hipStream_t s) {
    constexpr int N = kGroupThreads<LPR>, kGroups = N / LPR;
    if (back) {
        hipLaunchKernelGGL((layernorm_bwd_kernel<IO, LPR, V, WIDE>), dim3(p.blocks), dim3(N), 0, s, p);
    } else {
        // a launch takes fewer than 2^32 threads
        constexpr long long most = 0xffffffffll / N * kGroups, kB = IO == IO_F32 ? 4 : 2;
        LayerNormParams part = p;
        for (long long left = p.rows; left > 0; left -= most) {
            part.rows = left < most ? left : most;
            const dim3 grid((unsigned)((part.rows + kGroups - 1) / kGroups));
            hipLaunchKernelGGL((layernorm_fwd_kernel<IO, LPR, V, WIDE>), grid, dim3(N), 0, s, part);
            part.x = (const char*)part.x + most * p.stride * kB;
            part.y = (char*)part.y + most * p.D * kB;
        }
    }
    return hipGetLastError();
}
template <int IO, int LPR, bool WIDE>
hipError_t pieces(const LayerNormParams& p, bool back, hipStream_t s) {
    switch (((p.D + 7) / 8 + LPR - 1) / LPR) {
    case 1: return launch<IO, LPR, 1, WIDE>(p, back, s);
    case 2: return launch<IO, LPR, 2, WIDE>(p, back, s);
    case 3: return launch<IO, LPR, 3, WIDE>(p, back, s);
    default: return launch<IO, LPR, 4, WIDE>(p, back, s);
    }
}
template <int IO, bool WIDE>
hipError_t lanes(const LayerNormParams& p, bool back, hipStream_t s) {
    switch (lanes_of(p.D, back)) {
    case 16: return pieces<IO, 16, WIDE>(p, back, s);
    case 32: return pieces<IO, 32, WIDE>(p, back, s);
    case 64: return pieces<IO, 64, WIDE>(p, back, s);
    case 256: return pieces<IO, 256, WIDE>(p, back, s);
    default: return pieces<IO, 512, WIDE>(p, back, s);
    }
}
// Outputs of 160 MB and more do not stay in the caches (256 MB in all) until they are
// read again, and past them they leave the input there: 16 x 8192 rows of 768 in f16,
// 201 MB each, forward and backward 193 us, through the caches 200 (in turn).
hipError_t any(int io, LayerNormParams p, bool back, hipStream_t s) {
    p.past = p.rows * p.D * 2 >= (160ll << 20);
    switch (io) {
    case IO_F32: return p.wide ? lanes<IO_F32, true>(p, back, s) : lanes<IO_F32, false>(p, back, s);
    case IO_F16: return p.wide ? lanes<IO_F16, true>(p, back, s) : lanes<IO_F16, false>(p, back, s);
    default: return p.wide ? lanes<IO_BF16, true>(p, back, s) : lanes<IO_BF16, false>(p, back, s);
    }
}

}  // namespace

// Workgroups of the backward pass: they keep their sums to the end, so about as many as
// run at once (at two pieces a lane, three of 256 threads on each of the 256 CUs).  With few
// wide rows their sums are more than the rows: of 1000 x 8192 in bf16, 49 MB in and out,
// they are 50 MB, written and read (45 us in all).
int layernorm_bwd_blocks(long long rows, int D) {
    const int lpr = lanes_of(D, true), groups = lpr > 256 ? 1 : 256 / lpr;
    const long long n = (rows + groups - 1) / groups;
    return (int)(n < 1 ? 1 : n > 768 ? 768 : n);
}

hipError_t launch_layernorm_fwd(int io, const LayerNormParams& p, hipStream_t s) {
    return any(io, p, false, s);
}

hipError_t launch_layernorm_bwd(int io, const LayerNormParams& p, hipStream_t s) {
    const hipError_t e = any(io, p, true, s);
    if (e != hipSuccess || !p.part) return e;
    hipLaunchKernelGGL(layernorm_sum_kernel, dim3((2 * p.D + 15) / 16), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace fftconv
