// The gated delta rule, backward.  With the names of the forward pass
// (Y = beta o X, U = T Y, P with the output scale in it) and D the gradient
// of a chunk's last state:
//   dU = P^T dO + e^(Gc-G) o (K D),  dY = T^T dU,  dX = dV = beta o dY
//   dS0 = e^Gc D + Q^T (scale e^G o dO) - K^T (e^G o dX)
// (delta_rscan_kernel, from the last chunk of a sequence to the first), then
// for all chunks at once (delta_grads_kernel), with R1 = dO S0^T,
// R2 = dY S0^T, R3 = U D^T, Dp = dO U^T, Dy = dY U^T,
//   W_ij = scale Gam_ij Dp_ij (j <= i),  E_ij = -beta_i Gam_ij Dy_ij (j < i):
//   dQ = scale e^G o R1 + W K
//   dK = e^(Gc-G) o R3 - beta e^G o R2 + W^T Q + (E + E^T) K
//   dbeta_i = dY_i.V_i - e^G_i k_i.R2_i - sum_j Gam_ij Dy_ij k_i.k_j
//   dG_i = scale e^G_i q_i.R1_i - beta_i e^G_i k_i.R2_i - e^(Gc-G_i) k_i.R3_i
//        + sum_j (W_ij q_i.k_j + E_ij k_i.k_j) - sum_j (W_ji q_j.k_i + E_ji k_j.k_i)
//   dGc += e^Gc <S0, D> + sum_i e^(Gc-G_i) k_i.R3_i
// and dg is dG summed from the chunk's end.  beta is never divided by.
#include "fftconv_delta_dev.h"

namespace fftconv {
namespace {

template <int IO, int DK>
struct RscanLds {
    static constexpr int NA = IoTerms<IO>::n;
    // fp32 operands fill the LDS: the transposed queries take the place of
    // the keys, the transposed keys that of the queries
    static constexpr bool kShare = NA == 3;
    static constexpr int kRows = NA * 4 * (DK / 32) * 64;
    static constexpr int kK = 0, kKt = kShare ? 0 : kRows, kQt = kShare ? kRows : 2 * kRows;
    static constexpr int kTri = kShare ? 2 * kRows : 3 * kRows;
    static constexpr int kP = kTri + 3 * kTriTiles * 64;
    static constexpr int kDec = kP + 3 * kTriTiles * 64;
    static constexpr int kBytes = (kDec + kDecFloats / 4) * 16;
};

// The mirror of the forward walk: a wave owns 16 columns of D and goes
// through K D, T^T dU and the two transposed products without an exchange.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_rscan_kernel(DeltaGradParams gp) {
    typedef RscanLds<IO, DK> L;
    const DeltaParams& p = gp.f;
    constexpr int NA = L::NA, KB = DK / 32, ST = DK / 16;
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
    dfloat4 D[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = tile_row(t, 4 * g + r);
            D[t][r] = gp.dfin && cok && row < p.Dk ? gp.dfin[sbase + (long long)row * p.Dv] : 0.f;
        }
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const long long tok = sp.t0 + (long long)ch * kChunk;
        const int left = sp.len - ch * kChunk, n = left < kChunk ? left : kChunk;
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        const long long kbase = sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2];
        const long long qbase = sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2];
        fill_rows<IO, DK>(lds + L::kK, p.k, kbase, p.ks[1], n, p.Dk);
        fill_cols<IO, DK>(lds + L::kQt, p.q, qbase, p.qs[1], n, p.Dk);
        if (!L::kShare) fill_cols<IO, DK>(lds + L::kKt, p.k, kbase, p.ks[1], n, p.Dk);
        fill_tri<3>(lds + L::kTri, p.trit + ci * kTriFloats);
        fill_tri<3>(lds + L::kP, p.pmt + ci * kTriFloats);
        if (threadIdx.x < kDecFloats / 4)
            lds[L::kDec + threadIdx.x] = ((const uint4*)(p.dec + ci * kDecFloats))[threadIdx.x];
        const long long obase = ((sp.b * p.T + tok) * p.Hv + h) * p.Dv + col;
        dfloat4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(m, 4 * g + r);
                dO[m][r] = cok && row < n
                               ? io_load<IO>(gp.dout, obase + (long long)row * p.Hv * p.Dv) : 0.f;
            }
        if (cok) {
            float* d = gp.dstates + ci * p.Dk * (long long)p.Dv + col;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = tile_row(t, 4 * g + r);
                    if (row < p.Dk) d[(long long)row * p.Dv] = D[t][r];
                }
        }
        __syncthreads();
        // dU = e^(Gc-G) o K D + P^T dO
        dfloat4 dU[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dU[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint4 dt[3];
            split_acc<3>(D[2 * kb], D[2 * kb + 1], dt);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint4 a[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) a[i] = lds[L::kK + ((i * 4 + m) * KB + kb) * 64 + lane];
                dU[m] = mma_terms<3>(a, dt, dU[m]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = *(const float4*)(dec + 64 + tile_row(m, 4 * g));
            dU[m][0] *= e.x;
            dU[m][1] *= e.y;
            dU[m][2] *= e.z;
            dU[m][3] *= e.w;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 ot[NA];
            split_acc<NA>(dO[2 * kb], dO[2 * kb + 1], ot);
#pragma unroll
            for (int m = 0; m < 2 * kb + 2; ++m) {
                uint4 a[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    a[i] = lds[L::kP + (i * kTriTiles + upper_tile(m, kb)) * 64 + lane];
                dU[m] = mma_terms<3>(a, ot, dU[m]);
            }
        }
        // dY = T^T dU
        dfloat4 dY[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dY[m] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 ut[3];
            split_acc<3>(dU[2 * kb], dU[2 * kb + 1], ut);
#pragma unroll
            for (int m = 0; m < 2 * kb + 2; ++m) {
                uint4 a[3];
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    a[i] = lds[L::kTri + (i * kTriTiles + upper_tile(m, kb)) * 64 + lane];
                dY[m] = mma_terms<3>(a, ut, dY[m]);
            }
        }
        // dV = beta o dY; what goes back to the state through K and Q
        float* yd = gp.dys + ci * kChunk * p.Dv + col;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int r0 = tile_row(m, 4 * g);
            const float4 e = *(const float4*)(dec + r0), b = *(const float4*)(dec + 128 + r0);
            const float ev[4] = {e.x, e.y, e.z, e.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (cok) yd[(long long)(r0 + r) * p.Dv] = dY[m][r];
                const float dx = bv[r] * dY[m][r];
                if (cok && r0 + r < n)
                    io_store<IO>(gp.dv, obase + (long long)(r0 + r) * p.Hv * p.Dv, dx);
                dY[m][r] = -ev[r] * dx;
                dO[m][r] *= p.scale * ev[r];
            }
        }
        if (L::kShare) {
            __syncthreads();
            fill_cols<IO, DK>(lds + L::kKt, p.k, kbase, p.ks[1], n, p.Dk);
            __syncthreads();
        }
        const float ec = dec[192];
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) D[t][r] *= ec;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            uint4 yt[3], ot[3];
            split_acc<3>(dY[2 * tb], dY[2 * tb + 1], yt);
            split_acc<3>(dO[2 * tb], dO[2 * tb + 1], ot);
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                uint4 a[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    a[i] = lds[L::kKt + ((i * ST + t) * 2 + tb) * 64 + lane];
                D[t] = mma_terms<3>(a, yt, D[t]);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    a[i] = lds[L::kQt + ((i * ST + t) * 2 + tb) * 64 + lane];
                D[t] = mma_terms<3>(a, ot, D[t]);
            }
        }
        __syncthreads();
    }
    if (gp.dinit && cok)
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(t, 4 * g + r);
                if (row < p.Dk) gp.dinit[sbase + (long long)row * p.Dv] = D[t][r];
            }
}

// ------------------------------------------------ the gradients of a chunk

// LDS of delta_grads_kernel.  The slices of S0, D and U (32 columns, three
// terms) and the transposed keys and queries are never live together.
template <int IO, int DK>
struct GradsLds {
    static constexpr int NA = IoTerms<IO>::n;
    static constexpr int ST = DK / 16;
    static constexpr int kS = 0, kD = 3 * ST * 64, kU = 2 * kD;   // uint4
    static constexpr int kSlices = kU + 3 * 4 * 64;
    static constexpr int kKt = 0, kQt = NA * ST * 2 * 64, kCols = 2 * kQt;
    static constexpr int kBig = kSlices > kCols ? kSlices : kCols;
    static constexpr int kW = kBig, kF = kW + kChunk * kLd / 4;
    static constexpr int kBytes = (kF + kChunk * kLd / 4) * 16;
};

// eight consecutive fp32 values as three terms
__device__ __forceinline__ void load_f32_terms(const float* p, bool ok, uint4 (&t)[3]) {
    load_terms<IO_F32>(p, 0, ok, t);
}

// One workgroup per chunk and key head; a wave owns 16 tokens.  The value
// heads that share the key head follow one another and their parts of dQ and
// dK are summed in registers, in a fixed order.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_grads_kernel(DeltaGradParams gp) {
    typedef GradsLds<IO, DK> L;
    const DeltaParams& p = gp.f;
    constexpr int NA = L::NA, KB = DK / 32, ST = L::ST;
    constexpr int NW = NA == 3 ? 3 : 2;      // terms of W and E
    extern __shared__ uint4 lds[];
    __shared__ double G[kChunk];
    __shared__ float bet[kChunk], colsum[4][kChunk], rowG[kChunk], rowB[kChunk];
    __shared__ float rowV[kChunk], red[4], red3[4];
    const long long units = p.slots * p.Hk;
    const long long id = xcd_unit(blockIdx.x, units);
    if (id >= units) return;
    const long long slot = id / p.Hk;
    const int hk = (int)(id - slot * p.Hk);
    const long long seq = seq_of(p, slot);
    const Span sp = span_of(p, seq);
    const long long at = (slot - sp.slot0) * kChunk;
    if (at < 0 || at >= sp.len) return;
    const int n = (int)(sp.len - at < kChunk ? sp.len - at : kChunk);
    const long long tok = sp.t0 + at;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const long long kbase = sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2];
    const long long qbase = sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2];
    const int arow = 16 * wave + c;          // the lane's token in A operands
    float (*W)[kLd] = (float (*)[kLd])(lds + L::kW);
    float (*F)[kLd] = (float (*)[kLd])(lds + L::kF);

    // scores of the wave's tokens against those up to them
    dfloat4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int e = 32 * kb + 8 * g;
        uint4 ka[NA], qa[NA];
        const bool ok = arow < n && e < p.Dk;
        load_terms<IO>(p.k, kbase + arow * p.ks[1] + e, ok, ka);
        load_terms<IO>(p.q, qbase + arow * p.qs[1] + e, ok, qa);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= wave) {
                uint4 b[NA];
                const int col = 16 * j + c;
                load_terms<IO>(p.k, kbase + col * p.ks[1] + e, col < n && e < p.Dk, b);
                kk[j] = mma_terms<3>(ka, b, kk[j]);
                qk[j] = mma_terms<3>(qa, b, qk[j]);
            }
    }
    dfloat4 dQ[ST], dK[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t) dQ[t] = dK[t] = dfloat4{0, 0, 0, 0};

    for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
        const long long ci = slot * p.Hv + h;
        __syncthreads();
        if (wave == 0) {
            const long long gi = (sp.b * p.T + tok + lane) * p.Hv + h;
            G[lane] = decay_sum(lane < n ? p.g[gi] : 0.f);
            bet[lane] = lane < n ? p.beta[gi] : 0.f;
        }
        // products over the columns of the state, 32 at a time
        dfloat4 R1[ST], R2[ST], R3[ST], Dp[4], Dy[4];
#pragma unroll
        for (int t = 0; t < ST; ++t) R1[t] = R2[t] = R3[t] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) Dp[j] = Dy[j] = dfloat4{0, 0, 0, 0};
        float sd = 0.f, yv = 0.f;
        const float* S0 = p.states + ci * p.Dk * (long long)p.Dv;
        const float* D = gp.dstates + ci * p.Dk * (long long)p.Dv;
        const float* U = p.us + ci * kChunk * (long long)p.Dv;
        const float* Y = gp.dys + ci * kChunk * (long long)p.Dv;
        for (int d0 = 0; d0 < p.Dv; d0 += 32) {
            const int e = d0 + 8 * g;
            __syncthreads();
            // B operands: tile t, lane (g, c) holds [16 t + c][d0 + 8 g + i]
            for (int i = threadIdx.x; i < ST * 64; i += 256) {
                const int row = 16 * (i >> 6) + (i & 15), el = d0 + 8 * ((i >> 4) & 3);
                const bool ok = row < p.Dk && el < p.Dv;
                const float* s = S0 + (long long)row * p.Dv + el;
                const float* d = D + (long long)row * p.Dv + el;
                uint4 ts[3], td[3];
                load_f32_terms(s, ok, ts);
                load_f32_terms(d, ok, td);
                if (ok)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sd += s[j] * d[j];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    lds[L::kS + j * ST * 64 + i] = ts[j];
                    lds[L::kD + j * ST * 64 + i] = td[j];
                }
            }
            {
                const int i = threadIdx.x;
                const int row = 16 * (i >> 6) + (i & 15), el = d0 + 8 * ((i >> 4) & 3);
                uint4 tu[3];
                load_f32_terms(U + (long long)row * p.Dv + el, el < p.Dv, tu);
#pragma unroll
                for (int j = 0; j < 3; ++j) lds[L::kU + j * 256 + i] = tu[j];
            }
            // A operands of the wave's tokens
            uint4 oa[NA], ya[3], ua[3];
            load_terms<IO>(gp.dout, ((sp.b * p.T + tok + arow) * p.Hv + h) * p.Dv + e,
                           arow < n && e < p.Dv, oa);
            const float* yp = Y + (long long)arow * p.Dv + e;
            load_f32_terms(yp, e < p.Dv, ya);
            load_f32_terms(U + (long long)arow * p.Dv + e, e < p.Dv, ua);
            if (arow < n && e < p.Dv) {
                const long long vi = sp.b * p.vs[0] + (tok + arow) * p.vs[1] + h * p.vs[2] + e;
#pragma unroll
                for (int j = 0; j < 8; ++j) yv += yp[j] * io_load<IO>(p.v, vi + j);
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                uint4 b[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) b[j] = lds[L::kS + (j * ST + t) * 64 + lane];
                R1[t] = mma_terms<3>(oa, b, R1[t]);
                R2[t] = mma_terms<3>(ya, b, R2[t]);
#pragma unroll
                for (int j = 0; j < 3; ++j) b[j] = lds[L::kD + (j * ST + t) * 64 + lane];
                R3[t] = mma_terms<3>(ua, b, R3[t]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= wave) {
                    uint4 b[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i) b[i] = lds[L::kU + i * 256 + j * 64 + lane];
                    Dp[j] = mma_terms<3>(oa, b, Dp[j]);
                    Dy[j] = mma_terms<3>(ya, b, Dy[j]);
                }
        }
        __syncthreads();
        // transposed keys and queries take the slices' place
        fill_cols<IO, DK>(lds + L::kKt, p.k, kbase, p.ks[1], n, p.Dk);
        fill_cols<IO, DK>(lds + L::kQt, p.q, qbase, p.qs[1], n, p.Dk);
        // <S0, D>, and dY.V of the lane's token
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) sd += __shfl_xor(sd, m);
        if (lane == 0) red[wave] = sd;
#pragma unroll
        for (int m = 16; m < 64; m <<= 1) yv += __shfl_xor(yv, m);
        if (g == 0) rowV[arow] = yv;
        const double last = G[kChunk - 1];
        // sums over the elements of a head: rows 16 wave + 4 g + r
        float a1[4], a2[4], a3[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * wave + 4 * g + r;
            const double Gr = G[row];
            const float eg = expf((float)Gr), ee = expf((float)(last - Gr)), b = bet[row];
            float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                const int el = 16 * t + c;
                const bool ok = row < n && el < p.Dk;
                const float qv = ok ? io_load<IO>(p.q, qbase + row * p.qs[1] + el) : 0.f;
                const float kv = ok ? io_load<IO>(p.k, kbase + row * p.ks[1] + el) : 0.f;
                s1 += qv * R1[t][r];
                s2 += kv * R2[t][r];
                s3 += kv * R3[t][r];
                dQ[t][r] += p.scale * eg * R1[t][r];
                dK[t][r] += ee * R3[t][r] - b * eg * R2[t][r];
            }
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) {
                s1 += __shfl_xor(s1, m);
                s2 += __shfl_xor(s2, m);
                s3 += __shfl_xor(s3, m);
            }
            a1[r] = p.scale * eg * s1;
            a2[r] = eg * s2;
            a3[r] = ee * s3;
        }
        // the 64 x 64 part
        float cs[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * wave + 4 * g + r;
            const double Gr = G[row];
            const float b = bet[row];
            float sg = 0.f, sb = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 16 * j + c;
                float w = 0.f, f = 0.f;
                if (row >= col) {
                    const float gam = expf((float)(Gr - G[col]));
                    w = p.scale * gam * Dp[j][r];
                    const float x = row > col ? gam * Dy[j][r] : 0.f;
                    f = -b * x;
                    const float t = w * qk[j][r] + f * kk[j][r];
                    sg += t;
                    cs[j] += t;
                    sb -= x * kk[j][r];
                    if (row > col) F[col][row] = f;
                }
                if (row >= col) F[row][col] = f;
                W[row][col] = w;
            }
#pragma unroll
            for (int m = 1; m < 16; m <<= 1) {
                sg += __shfl_xor(sg, m);
                sb += __shfl_xor(sb, m);
            }
            if (c == 0) {
                rowG[row] = sg + a1[r] - b * a2[r] - a3[r];
                rowB[row] = sb - a2[r];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int m = 16; m < 64; m <<= 1) cs[j] += __shfl_xor(cs[j], m);
            if (g == 0) colsum[wave][16 * j + c] = cs[j];
        }
        // the chunk's last decay: sum of a3 over all tokens
        float s3 = c == 0 ? a3[0] + a3[1] + a3[2] + a3[3] : 0.f;
#pragma unroll
        for (int m = 16; m < 64; m <<= 1) s3 += __shfl_xor(s3, m);
        if (lane == 0) red3[wave] = s3;
        __syncthreads();
        if (wave == 0) {
            double x = (double)rowG[lane] - (colsum[0][lane] + colsum[1][lane] +
                                             colsum[2][lane] + colsum[3][lane]);
            if (lane == 63)
                x += (red3[0] + red3[1] + red3[2] + red3[3]) +
                     expf((float)last) * (red[0] + red[1] + red[2] + red[3]);
            // sums from the end
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double o = __shfl_down(x, m);
                if (lane + m < 64) x += o;
            }
            const long long gi = (sp.b * p.T + tok + lane) * p.Hv + h;
            if (lane < n) {
                // a factor of 0 has the gradient 0, which the difference of
                // sums above meets only up to their rounding
                gp.dg[gi] = expf(p.g[gi]) == 0.f ? 0.f : (float)x;
                gp.dbeta[gi] = rowV[lane] + rowB[lane];
            }
        }
        // dQ += W K, dK += W^T Q + F K
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int e = 32 * kb + 8 * g;
            float x[8];
            uint4 wa[NW], wt[NW], fa[NW];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = W[arow][e + i];
            split8<NW>(x, wa);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = W[e + i][arow];
            split8<NW>(x, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = F[arow][e + i];
            split8<NW>(x, fa);
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                // the lane's column of tile t is element 16 t + c
                const int el = 16 * t + c;
                const int tile = 2 * (el >> 5) + ((el >> 2) & 1);
                const int row = 4 * ((el >> 3) & 3) + (el & 3);
                uint4 b[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    b[i] = lds[L::kKt + ((i * ST + tile) * 2 + kb) * 64 + 16 * g + row];
                dQ[t] = mma_terms<NW>(wa, b, dQ[t]);
                dK[t] = mma_terms<NW>(fa, b, dK[t]);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    b[i] = lds[L::kQt + ((i * ST + tile) * 2 + kb) * 64 + 16 * g + row];
                dK[t] = mma_terms<NW>(wt, b, dK[t]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int row = 16 * wave + 4 * g + r;
        if (row >= n) continue;
        const long long o = ((sp.b * p.T + tok + row) * p.Hk + hk) * p.Dk;
#pragma unroll
        for (int t = 0; t < ST; ++t)
            if (16 * t + c < p.Dk) {
                io_store<IO>(gp.dq, o + 16 * t + c, dQ[t][r]);
                io_store<IO>(gp.dk, o + 16 * t + c, dK[t][r]);
            }
    }
}

template <int IO, int DK>
hipError_t rscan_io(const DeltaGradParams& p, hipStream_t s) {
    const int bytes = RscanLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_rscan_kernel<IO, DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const long long units = p.f.nseq * p.f.Hv * ((p.f.Dv + 63) / 64);
    hipLaunchKernelGGL((delta_rscan_kernel<IO, DK>), dim3((unsigned)xcd_blocks(units)), dim3(256),
                       bytes, s, p);
    return hipGetLastError();
}

template <int IO, int DK>
hipError_t grads_io(const DeltaGradParams& p, hipStream_t s) {
    const int bytes = GradsLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_grads_kernel<IO, DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_grads_kernel<IO, DK>), dim3((unsigned)xcd_blocks(p.f.slots * p.f.Hk)),
                       dim3(256), bytes, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_rscan(int io, const DeltaGradParams& p, hipStream_t s) {
    const bool d64 = p.f.Dk <= 64;
    switch (io) {
    case IO_F32: return d64 ? rscan_io<IO_F32, 64>(p, s) : rscan_io<IO_F32, 128>(p, s);
    case IO_F16: return d64 ? rscan_io<IO_F16, 64>(p, s) : rscan_io<IO_F16, 128>(p, s);
    default: return d64 ? rscan_io<IO_BF16, 64>(p, s) : rscan_io<IO_BF16, 128>(p, s);
    }
}

hipError_t launch_delta_grads(int io, const DeltaGradParams& p, hipStream_t s) {
    const bool d64 = p.f.Dk <= 64;
    switch (io) {
    case IO_F32: return d64 ? grads_io<IO_F32, 64>(p, s) : grads_io<IO_F32, 128>(p, s);
    case IO_F16: return d64 ? grads_io<IO_F16, 64>(p, s) : grads_io<IO_F16, 128>(p, s);
    default: return d64 ? grads_io<IO_BF16, 64>(p, s) : grads_io<IO_BF16, 128>(p, s);
    }
}

}  // namespace fftconv
