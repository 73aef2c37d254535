// Linear attention with a decay for each head, forward: one token against a
// pool of states, and whole sequences in chunks.
//
// A value head h keeps a state S (Dk x Dv).  A token with key k, value v, query q
// and log decay g does
//   S <- e^g S + k v^T,   o = scale S^T q
#include "fftconv_decay_walk.h"

namespace fftconv {
namespace {

// ------------------------------------------------------------ one token

// A workgroup takes 32 columns of one state: 8 lanes x 4 columns, 32 row
// groups of R rows, all in registers: each state is read and written once.  All
// arithmetic is fp32, o is rounded once.  HBM bounds it: 192 requests of 8 heads of
// 128 x 128 move 203 MB in 38 us (5.4 TB/s; a streaming copy reaches 5.9); one
// request takes the launch's time, 10 us.
template <int IO, int R>
__global__ __launch_bounds__(256) void decay_step_kernel(DecayStepParams p) {
    const unsigned tiles = (p.Dv + 31) / 32;
    const unsigned tile = blockIdx.x % tiles, h = blockIdx.x / tiles % p.Hv;
    const long long n = blockIdx.x / tiles / p.Hv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = tile * 32 + 4 * (lane & 7);
    const int row0 = (wave * 8 + (lane >> 3)) * R;
    const bool cok = col < p.Dv;
    const long long slot = p.slots ? p.slots[n] : n;
    if (slot < 0 || slot >= p.pool) {
        // no state: a row of padding
        if (threadIdx.x < 32 && tile * 32 + threadIdx.x < (unsigned)p.Dv)
            io_store<IO>(p.o, (n * p.Hv + h) * p.Dv + tile * 32 + threadIdx.x, 0.f);
        return;
    }
    const long long at = (slot * p.Hv + h) * p.Dk * (long long)p.Dv + col;
    const int hk = h / (p.Hv / p.Hk);
    float s[R][4], k[R], q[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool ok = row0 + i < p.Dk;
        load4<IO_F32>(p.state, at + (long long)(row0 + i) * p.Dv, cok && ok, s[i]);
        k[i] = io_load_if<IO>(p.k, n * p.ks[0] + hk * p.ks[1] + row0 + i, ok);
        q[i] = io_load_if<IO>(p.q, n * p.qs[0] + hk * p.qs[1] + row0 + i, ok);
    }
    const float a = expf(p.g[p.fixed ? h : n * p.Hv + h]);
    float v[4], o[4] = {0, 0, 0, 0};
    load4<IO>(p.v, n * p.vs[0] + h * p.vs[1] + col, cok, v);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool ok = cok && row0 + i < p.Dk;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] = a * s[i][j] + k[i] * v[j];
            o[j] += ok ? q[i] * s[i][j] : 0.f;
        }
        if (ok)
            *(float4*)(p.state + at + (long long)(row0 + i) * p.Dv) =
                make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    }
    // over the row groups
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = sum_groups(o[j] + row_ror<8>(o[j]));
    __shared__ float sums[4][8][4];
    if (lane < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[wave][lane][j] = o[j];
    __syncthreads();
    if (threadIdx.x < 32 && tile * 32 + threadIdx.x < (unsigned)p.Dv) {
        const int x = threadIdx.x >> 2, j = threadIdx.x & 3;
        io_store<IO>(p.o, (n * p.Hv + h) * p.Dv + tile * 32 + threadIdx.x,
                     p.scale * ((sums[0][x][j] + sums[1][x][j]) + (sums[2][x][j] + sums[3][x][j])));
    }
}

template <int IO>
hipError_t step_io(const DecayStepParams& p, hipStream_t s) {
    const dim3 grid((unsigned)((long long)p.N * p.Hv * ((p.Dv + 31) / 32)));
    if (p.Dk <= 64) hipLaunchKernelGGL((decay_step_kernel<IO, 2>), grid, dim3(256), 0, s, p);
    else if (p.Dk <= 128) hipLaunchKernelGGL((decay_step_kernel<IO, 4>), grid, dim3(256), 0, s, p);
    else hipLaunchKernelGGL((decay_step_kernel<IO, 8>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int IO>
hipError_t fwd_io(const DecayParams& p, hipStream_t s) {
    DecayWalk w = DecayWalk();
    w.sp = p.sp;
    w.Hv = p.Hv;
    w.rows = p.Dk;
    w.cols = p.Dv;
    w.fixed = p.fixed;
    w.g = p.g;
    w.a = p.q;
    w.b = p.k;
    w.v = p.v;
    w.sf = w.ss = p.scale;
    w.sw = 1.f;
    w.rs = p.Dv;
    w.cs = 1;
    w.init = p.init;
    w.seg = p.seg;
    w.seg_g = p.seg_g;
    w.fin = p.fin;
    w.out = p.o;
    w.clear = p.clear;
    if (p.seg) {
        hipError_t e = decay_walk_io<IO, kEffects>(w, s);
        if (e == hipSuccess) e = launch_decay_join(p, p.init, false, s);
        if (e != hipSuccess) return e;
    }
    return decay_walk_io<IO, kOutputs>(w, s);
}

// ------------------------------------------------------------------- segments

// The segments' effects on the state become their first states: a thread takes V
// elements of one sequence's state.  back: from the last segment to the first.
// A chain of loads, so eight segments' effects are on their way at once (the last
// segment's is not made); sixteen were no faster.
template <int V>
__global__ __launch_bounds__(256) void decay_join_kernel(DecaySpans p, int Hv, unsigned size,
                                                         const float* init, float* seg,
                                                         const double* seg_g, bool back) {
    typedef float Part __attribute__((ext_vector_type(V)));
    const unsigned per = (size + 256 * V - 1) / (256 * V), block = blockIdx.x / per;
    const unsigned e = ((blockIdx.x - block * per) * 256 + threadIdx.x) * V;
    const unsigned seq = block / (unsigned)Hv, h = block - seq * Hv;
    if (e >= size) return;
    long long first = (long long)seq * p.per;
    int n = p.per;
    if (p.cu) {
        const unsigned a = (unsigned)bound_of(p, seq), z = (unsigned)bound_of(p, seq + 1);
        first = a / (unsigned)p.seg_tokens + seq;
        n = z > a ? (int)((z - a + p.seg_tokens - 1) / (unsigned)p.seg_tokens) : 1;
    }
    const auto part = [&](const float* x, long long i) { return *(const Part*)(x + i * size + e); };
    Part S;
#pragma unroll
    for (int v = 0; v < V; ++v) S[v] = 0.f;
    if (init) S = part(init, (long long)seq * Hv + h);
    const auto at = [&](int j) { return (first + (back ? n - 1 - j : j)) * Hv + h; };
    constexpr int kAhead = 8;
    for (int j0 = 0; j0 + 1 < n; j0 += kAhead) {
        Part effect[kAhead];
        double g[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const long long i = at(j0 + j + 1 < n ? j0 + j : n - 2);
            effect[j] = part(seg, i);
            g[j] = seg_g[i];
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j0 + j + 1 < n) {
                *(Part*)(seg + at(j0 + j) * size + e) = S;
                // the rounding of a, the same for equal segments, goes with it
                float left;
                const float a = exact_exp2(g[j], left);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    S[v] = fmaf(a, S[v], fmaf(a * left, S[v], effect[j][v]));
            }
    }
    *(Part*)(seg + at(n - 1) * size + e) = S;
}
template <int V>
hipError_t join_launch(const DecayParams& p, const float* init, bool back, hipStream_t s) {
    const unsigned size = (unsigned)(p.Dk * p.Dv), per = (size + 256 * V - 1) / (256 * V);
    hipLaunchKernelGGL((decay_join_kernel<V>), dim3((unsigned)(p.sp.nseq * p.Hv * per)),
                       dim3(256), 0, s, p.sp, p.Hv, size, init, p.seg, p.seg_g, back);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decay_join(const DecayParams& p, const float* init, bool back, hipStream_t s) {
    // Four elements a thread where that leaves a workgroup for each CU.  With one and with
    // four: 5888 workgroups of single elements 18.0 and 8.3 us, 1024 (4 x 32768 tokens of 4
    // heads of 128) 12.8 and 9.2, 128 (2 x 1501 of 4 heads of 64) 7.2 and 8.1.
    const long long blocks = p.sp.nseq * p.Hv * ((p.Dk * p.Dv + 255) / 256);
    return blocks >= 1024 ? join_launch<4>(p, init, back, s) : join_launch<1>(p, init, back, s);
}

hipError_t launch_decay_fwd(int io, const DecayParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return fwd_io<IO_F32>(p, s);
    case IO_F16: return fwd_io<IO_F16>(p, s);
    default: return fwd_io<IO_BF16>(p, s);
    }
}
hipError_t launch_decay_step(int io, const DecayStepParams& p, hipStream_t s) {
    switch (io) {
    case IO_F32: return step_io<IO_F32>(p, s);
    case IO_F16: return step_io<IO_F16>(p, s);
    default: return step_io<IO_BF16>(p, s);
    }
}

}  // namespace fftconv
