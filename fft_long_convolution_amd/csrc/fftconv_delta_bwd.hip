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
    static constexpr int kRows = Operand<IO>::NA * 4 * (DK / 32) * 64;     // uint4
    static constexpr int kK = 0, kQ = kRows, kPack = 2 * kRows;
    static constexpr int kTri = kPack, kDec = kTri + 3 * kTriTiles * 64, kP = kDec + 64;
    static constexpr int kBytes = (kPack + kBackPack) * 16;
};

// The mirror of the forward walk: a wave owns 16 columns of D and goes
// through K D, T^T dU and the two transposed products without an exchange.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_rscan_kernel(DeltaGradParams gp) {
    typedef RscanLds<IO, DK> L;
    typedef Operand<IO> Op;
    const DeltaParams& p = gp.f;
    constexpr int NA = Op::NA, NB = Op::NB, KB = DK / 32, ST = DK / 16, NO = IoTerms<IO>::n;
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
    const int slot = 16 * g + (c ^ (4 * g));             // of a row operand
    const int col = cb * 64 + wave * 16 + c;
    const bool cok = col < p.Dv;
    const int hk = h / p.group;
    const long long state = p.Dk * (long long)p.Dv;
    const long long sbase = (seq * p.Hv + h) * state + col;
    dfloat4 D[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = tile_row(t, 4 * g + r);
            D[t][r] = gp.dfin && cok && row < p.Dk ? gp.dfin[sbase + (long long)row * p.Dv] : 0.f;
        }
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const long long kbase = sp.b * p.ks[0] + sp.t0 * p.ks[1] + hk * p.ks[2];
    const long long qbase = sp.b * p.qs[0] + sp.t0 * p.qs[1] + hk * p.qs[2];
    const long long obase = ((sp.b * p.T + sp.t0) * p.Hv + h) * p.Dv + col;
    const long long ostride = (long long)p.Hv * p.Dv;
    RowTiles<IO, DK> rk, rq;
    Block<kBackPack / 64> rp;
    const auto load = [&](int ch) __attribute__((always_inline)) {
        const int n = sp.len - ch * kChunk;
        rk.load(p.k, kbase + ch * (kChunk * p.ks[1]), p.ks[1], n, p.Dk);
        rq.load(p.q, qbase + ch * (kChunk * p.qs[1]), p.qs[1], n, p.Dk);
        rp.load(p.bpack + ((sp.slot0 + ch) * p.Hv + h) * kBackPack);
    };
    const auto store = [&](uint4* d) __attribute__((always_inline)) {
        rk.store(d + L::kK);
        rq.store(d + L::kQ);
        rp.store(d + L::kPack);
    };
    dfloat4 dN[4];                       // dO of the next chunk
    const auto load_do = [&](int ch) __attribute__((always_inline)) {
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = ch * kChunk + tile_row(m, 4 * g + r);
                dN[m][r] = io_load_if<IO>(gp.dout, obase + row * ostride, cok && row < sp.len);
            }
    };
    if (chunks > 0) {
        load(chunks - 1);
        load_do(chunks - 1);
        store(lds);
    }
    __syncthreads();
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        dfloat4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dO[m] = dN[m];
        const int ahead = ch > 0 ? ch - 1 : 0;
        load(ahead);
        if (cok) {
            float* d = gp.dstates + ci * state + col;
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = tile_row(t, 4 * g + r);
                    if (row < p.Dk) d[(long long)row * p.Dv] = D[t][r];
                }
        }
        // dU = e^(Gc-G) o K D + P^T dO
        dfloat4 dU[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dU[m] = dfloat4{0, 0, 0, 0};
        {
            const ColScale sc = Op::template scale_of<ST>(D);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint4 dt[NB];
                Op::split(D[2 * kb], D[2 * kb + 1], sc, dt);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint4 a[NA];
#pragma unroll
                    for (int i = 0; i < NA; ++i)
                        a[i] = lds[L::kK + ((i * 4 + m) * KB + kb) * 64 + slot];
                    dU[m] = Op::mma(a, dt, dU[m]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float4 e = *(const float4*)(dec + 64 + tile_row(m, 4 * g));
                dU[m][0] *= e.x * sc.back;
                dU[m][1] *= e.y * sc.back;
                dU[m][2] *= e.z * sc.back;
                dU[m][3] *= e.w * sc.back;
            }
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 ot[NO];
            split_acc<NO>(dO[2 * kb], dO[2 * kb + 1], ot);
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
                const int row = ch * kChunk + r0 + r;
                if (cok && row < sp.len) io_store<IO>(gp.dv, obase + row * ostride, dx);
                dY[m][r] = -ev[r] * dx;
                dO[m][r] *= p.scale * ev[r];
            }
        }
        const float ec = dec[192];
        load_do(ahead);
        const ColScale sy = Op::template scale_of<4>(dY), so = Op::template scale_of<4>(dO);
        uint4 yt[2][NB], ot[2][NB];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            Op::split(dY[2 * tb], dY[2 * tb + 1], sy, yt[tb]);
            Op::split(dO[2 * tb], dO[2 * tb + 1], so, ot[tb]);
        }
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            dfloat4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
            if (!Op::kScaled)
#pragma unroll
                for (int r = 0; r < 4; ++r) a[r] = ec * D[t][r];
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                uint4 x[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    x[i] = read_cols<DK>(lds + L::kK + i * 4 * KB * 64, t, tb);
                a = Op::mma(x, yt[tb], a);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    x[i] = read_cols<DK>(lds + L::kQ + i * 4 * KB * 64, t, tb);
                b = Op::mma(x, ot[tb], b);
            }
            if (Op::kScaled)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    D[t][r] = ec * D[t][r] + (sy.back * a[r] + so.back * b[r]);
            else
                D[t] = a + b;
        }
        __syncthreads();
        store(lds);
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

// LDS of delta_grads_kernel, in uint4.  The slices of S0, D and U (32
// columns, three terms) are used up before the keys, queries and the 64 x 64
// matrices take their place.
template <int IO, int DK>
struct GradsLds {
    static constexpr int ST = DK / 16;
    static constexpr int kS = 0, kD = 3 * ST * 64, kU = 2 * kD, kSlices = kU + 3 * 4 * 64;
    static constexpr int kRows = Operand<IO>::NA * 4 * (DK / 32) * 64;
    static constexpr int kK = 0, kQ = kRows, kW = 2 * kRows, kF = kW + kChunk * kLd / 4;
    static constexpr int kTail = kF + kChunk * kLd / 4;
    static constexpr int kBytes = (kSlices > kTail ? kSlices : kTail) * 16;
};

// Sum over the four groups of 16 lanes.
__device__ __forceinline__ float sum_groups(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// One workgroup per chunk and key head; a wave owns 16 tokens as the columns
// of its products, R^T = S0 dO^T and so on, so a lane has one token: what
// belongs to it (decays, row sums) is a scalar of the lane, and sums over a
// head's elements are sums in the lane and over four groups.  The value heads
// that share the key head follow one another, and their parts of dQ and dK
// are summed in registers, in a fixed order.
template <int IO, int DK>
__global__ __launch_bounds__(256) void delta_grads_kernel(DeltaGradParams gp) {
    typedef GradsLds<IO, DK> L;
    typedef Operand<IO> Op;
    const DeltaParams& p = gp.f;
    constexpr int NA = Op::NA, NB = Op::NB, NO = IoTerms<IO>::n, KB = DK / 32, ST = L::ST;
    extern __shared__ uint4 lds[];
    __shared__ double G[kChunk];
    __shared__ float bet[kChunk], colsum[4][kChunk], rowG[kChunk], rowB[kChunk], red[4], red3[4];
    const long long units = p.slots * p.Hk;
    const long long id = xcd_unit(blockIdx.x, units);
    if (id >= units) return;
    const long long slot = id / p.Hk;
    const int hk = (int)(id - slot * p.Hk);
    const long long seq = seq_of(p, slot, 1);
    const Span sp = span_of(p, seq);
    const long long at = (slot - sp.slot0) * kChunk;
    if (at < 0 || at >= sp.len) return;
    const int n = (int)(sp.len - at < kChunk ? sp.len - at : kChunk);
    const long long tok = sp.t0 + at;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const long long kbase = sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2];
    const long long qbase = sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2];
    const int mine = 16 * wave + c;          // the lane's token
    const int jtiles = wave < 2 ? 2 : 4;     // tiles of tokens up to the wave's
    float (*W)[kLd] = (float (*)[kLd])(lds + L::kW);   // [j][i]: W_ij
    float (*F)[kLd] = (float (*)[kLd])(lds + L::kF);   // E + E^T

    // q.k and k.k of the lane's token with those of tile j
    dfloat4 kk[4], qk[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        const int e = 32 * kb + 8 * g;
        uint4 kb_[NO], qb_[NO];
        const bool ok = mine < n && e < p.Dk;
        load_terms<IO>(p.k, kbase + mine * p.ks[1] + e, ok, kb_);
        load_terms<IO>(p.q, qbase + mine * p.qs[1] + e, ok, qb_);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < jtiles) {
                uint4 a[NO];
                const int row = tile_row(j, c);
                load_terms<IO>(p.k, kbase + row * p.ks[1] + e, row < n && e < p.Dk, a);
                kk[j] = mma_terms<3>(a, kb_, kk[j]);
                qk[j] = mma_terms<3>(a, qb_, qk[j]);
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
            // A operands: tile t, lane (g, c) holds [tile_row(t, c)][d0 + 8 g + i]
#pragma unroll
            for (int i = threadIdx.x; i < ST * 64; i += 256) {
                const int row = tile_row(i >> 6, i & 15), el = d0 + 8 * ((i >> 4) & 3);
                const bool ok = row < p.Dk && el < p.Dv;
                const long long at = ok ? (long long)row * p.Dv + el : 0;
                float s[8], d[8];
                load8<IO_F32>(S0, at, ok, s);
                load8<IO_F32>(D, at, ok, d);
                uint4 ts[3], td[3];
                split8<3>(s, ts);
                split8<3>(d, td);
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
                const int row = tile_row(i >> 6, i & 15), el = d0 + 8 * ((i >> 4) & 3);
                uint4 tu[3];
                load_terms<IO_F32>(U, (long long)row * p.Dv + el, el < p.Dv, tu);
#pragma unroll
                for (int j = 0; j < 3; ++j) lds[L::kU + j * 256 + i] = tu[j];
            }
            // B operands: columns of the wave's tokens
            uint4 ob[NO], yb[3], ub[3];
            const bool ok = mine < n && e < p.Dv;
            load_terms<IO>(gp.dout, ((sp.b * p.T + tok + mine) * p.Hv + h) * p.Dv + e, ok, ob);
            float y[8], v[8];
            load8<IO_F32>(Y, (long long)mine * p.Dv + e, e < p.Dv, y);
            load8<IO>(p.v, sp.b * p.vs[0] + (tok + mine) * p.vs[1] + h * p.vs[2] + e, ok, v);
            load_terms<IO_F32>(U, (long long)mine * p.Dv + e, e < p.Dv, ub);
            split8<3>(y, yb);
#pragma unroll
            for (int j = 0; j < 8; ++j) yv += y[j] * v[j];
            __syncthreads();
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                uint4 a[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) a[j] = lds[L::kS + (j * ST + t) * 64 + lane];
                R1[t] = mma_terms<3>(a, ob, R1[t]);
                R2[t] = mma_terms<3>(a, yb, R2[t]);
#pragma unroll
                for (int j = 0; j < 3; ++j) a[j] = lds[L::kD + (j * ST + t) * 64 + lane];
                R3[t] = mma_terms<3>(a, ub, R3[t]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < jtiles) {
                    uint4 a[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i) a[i] = lds[L::kU + i * 256 + j * 64 + lane];
                    Dp[j] = mma_terms<3>(a, ob, Dp[j]);
                    Dy[j] = mma_terms<3>(a, yb, Dy[j]);
                }
        }
        __syncthreads();
        // keys and queries take the slices' place
        {
            RowTiles<IO, DK> rk, rq;
            rk.load(p.k, kbase, p.ks[1], n, p.Dk);
            rq.load(p.q, qbase, p.qs[1], n, p.Dk);
            rk.store(lds + L::kK);
            rq.store(lds + L::kQ);
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) sd += __shfl_xor(sd, m);
        yv = sum_groups(yv);
        const double last = G[kChunk - 1], Gi = G[mine];
        const float eg = expf((float)Gi), ee = expf((float)(last - Gi)), b = bet[mine];
        // sums over the elements of a head
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const int el = tile_row(t, 4 * g);
            const bool ok = mine < n && el < p.Dk;
            float qv[4], kv[4];
            load4<IO>(p.q, qbase + mine * p.qs[1] + el, ok, qv);
            load4<IO>(p.k, kbase + mine * p.ks[1] + el, ok, kv);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s1 += qv[r] * R1[t][r];
                s2 += kv[r] * R2[t][r];
                s3 += kv[r] * R3[t][r];
                dQ[t][r] += p.scale * eg * R1[t][r];
                dK[t][r] += ee * R3[t][r] - b * eg * R2[t][r];
            }
        }
        s1 = p.scale * eg * sum_groups(s1);
        s2 = eg * sum_groups(s2);
        s3 = ee * sum_groups(s3);
        // the 64 x 64 part: the lane's token is i, tile j's row 4 g + r is j
        float sg = 0.f, sb = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int j0 = tile_row(j, 4 * g);
            float cs[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float w = 0.f, f = 0.f, t = 0.f;
                if (j < jtiles && mine >= j0 + r) {
                    const float gam = expf((float)(Gi - G[j0 + r]));
                    w = p.scale * gam * Dp[j][r];
                    const float x = mine > j0 + r ? gam * Dy[j][r] : 0.f;
                    f = -b * x;
                    t = w * qk[j][r] + f * kk[j][r];
                    sg += t;
                    sb -= x * kk[j][r];
                    F[mine][j0 + r] = f;
                    if (mine > j0 + r) F[j0 + r][mine] = f;
                }
                W[j0 + r][mine] = w;
                Dp[j][r] = w;                 // the lane's row of W
                cs[r] = t;
            }
            // sums over the wave's tokens
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) cs[r] += __shfl_xor(cs[r], m);
                if (c == 0) colsum[wave][j0 + r] = cs[r];
            }
        }
        sg = sum_groups(sg);
        sb = sum_groups(sb);
        if (g == 0) {
            rowG[mine] = sg + s1 - b * s2 - s3;
            rowB[mine] = yv + sb - s2;
        }
        // the chunk's last decay
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) s3 += __shfl_xor(s3, m);
        if (lane == 0) {
            red[wave] = sd;
            red3[wave] = s3;
        }
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
                gp.dbeta[gi] = rowB[lane];
            }
        }
        // dQ^T += K^T W^T, dK^T += Q^T W + K^T F
        dfloat4 wt[4], ft[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            wt[m] = *(const dfloat4*)&W[mine][tile_row(m, 4 * g)];
            ft[m] = *(const dfloat4*)&F[mine][tile_row(m, 4 * g)];
        }
        const ColScale sw = Op::template scale_of<4>(Dp), st = Op::template scale_of<4>(wt),
                       sf = Op::template scale_of<4>(ft);
        uint4 wb[2][NB], tb_[2][NB], fb[2][NB];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            Op::split(Dp[2 * tb], Dp[2 * tb + 1], sw, wb[tb]);
            Op::split(wt[2 * tb], wt[2 * tb + 1], st, tb_[tb]);
            Op::split(ft[2 * tb], ft[2 * tb + 1], sf, fb[tb]);
        }
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            dfloat4 a = {0, 0, 0, 0}, x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                uint4 kt[NA], qt[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    kt[i] = read_cols<DK>(lds + L::kK + i * 4 * KB * 64, t, tb);
                    qt[i] = read_cols<DK>(lds + L::kQ + i * 4 * KB * 64, t, tb);
                }
                a = Op::mma_out(kt, wb[tb], a);
                x = Op::mma_out(qt, tb_[tb], x);
                y = Op::mma_out(kt, fb[tb], y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dQ[t][r] += sw.back * a[r];
                dK[t][r] += st.back * x[r] + sf.back * y[r];
            }
        }
    }
    if (mine >= n) return;
    const long long o = ((sp.b * p.T + tok + mine) * p.Hk + hk) * p.Dk;
#pragma unroll
    for (int t = 0; t < ST; ++t) {
        const int el = tile_row(t, 4 * g);
        if (el < p.Dk) {
            store4<IO>(gp.dq, o + el, dQ[t]);
            store4<IO>(gp.dk, o + el, dK[t]);
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
