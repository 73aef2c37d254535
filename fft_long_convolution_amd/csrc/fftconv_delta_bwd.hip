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
    static constexpr int kSize = kPack + kBackPack;
    static constexpr int kBufs = Operand<IO>::NA == 1 ? 2 : 1;
    static constexpr int kBytes = kBufs * kSize * 16;
};

// The mirror of the forward walk: a wave owns 16 columns of D and goes
// through K D, T^T dU and the two transposed products without an exchange.
template <int IO, int DK, int W>
__global__ __launch_bounds__(64 * W) void delta_rscan_kernel(DeltaGradParams gp) {
    typedef RscanLds<IO, DK> L;
    typedef Operand<IO> Op;
    const DeltaParams& p = gp.f;
    constexpr int NA = Op::NA, NB = Op::NB, KB = DK / 32, ST = DK / 16, NO = IoTerms<IO>::n;
    extern __shared__ uint4 lds[];
    constexpr int kCols = 16 * W, kB = IO == IO_F32 ? 4 : 2;
    const int cols = (p.Dv + kCols - 1) / kCols;
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
    const int col = cb * kCols + wave * 16 + c;
    const bool cok = col < p.Dv;
    const int hk = h / p.group;
    const long long state = p.Dk * (long long)p.Dv;
    const int colv = cok ? col : 0;                      // to read from
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
    const Tokens tk = tokens_of<IO>(p.k, sp.b * p.ks[0] + sp.t0 * p.ks[1] + hk * p.ks[2], p.ks[1]);
    const Tokens tq = tokens_of<IO>(p.q, sp.b * p.qs[0] + sp.t0 * p.qs[1] + hk * p.qs[2], p.qs[1]);
    const long long ofirst = (sp.b * p.T + sp.t0) * p.Hv * p.Dv + h * p.Dv;
    const Tokens to = tokens_of<IO>(gp.dout, ofirst, (long long)p.Hv * p.Dv);
    const Tokens tv = tokens_of<IO>(gp.dv, ofirst, (long long)p.Hv * p.Dv);
    const uint32_t olane = (uint32_t)(8 * g) * (uint32_t)to.bytes + colv * kB;
    const uint32_t slane = (uint32_t)(8 * g * p.Dv + col) * 4;
    const uint4* pack = p.bpack + (sp.slot0 * p.Hv + h) * kBackPack;
    const long long pack_step = (long long)p.Hv * kBackPack;
    RowTiles<IO, DK, W> rk, rq;
    Block<kBackPack / 64, W> rp;
    const auto load = [&](int ch) __attribute__((always_inline)) {
        const int n = sp.len - ch * kChunk;
        rk.load(tk, ch * kChunk, n, p.Dk);
        rq.load(tq, ch * kChunk, n, p.Dk);
        rp.load(pack + ch * pack_step);
    };
    const auto store = [&](uint4* d) __attribute__((always_inline)) {
        rk.store(d + L::kK);
        rq.store(d + L::kQ);
        rp.store(d + L::kPack);
    };
    // dO of the next chunk.  The tokens from n on that repeat the last one
    // meet columns of P^T and rows of Q that are 0.
    dfloat4 dN[4];
    const auto load_do = [&](int ch) __attribute__((always_inline)) {
        load_column<IO>(to, ch * kChunk, olane, sp.len - ch * kChunk, dN);
    };
    if (chunks > 0) {
        load(chunks - 1);
        load_do(chunks - 1);
        store(lds);
    }
    __syncthreads();
    uint4* now = lds;
    uint4* next = lds + (L::kBufs == 2 ? L::kSize : 0);
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        const float* dec = (const float*)(now + L::kDec);
        dfloat4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dO[m] = dN[m];
        const int ahead = ch > 0 ? ch - 1 : 0;
        load(ahead);
        if (cok) store_state<ST>((char*)(gp.dstates + ci * state), p.Dv * 4, slane, p.Dk, D);
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
                        a[i] = now[L::kK + ((i * 4 + m) * KB + kb) * 64 + slot];
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
                    a[i] = now[L::kP + (i * kTriTiles + upper_tile(m, kb)) * 64 + lane];
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
                    a[i] = now[L::kTri + (i * kTriTiles + upper_tile(m, kb)) * 64 + lane];
                dY[m] = mma_terms<3>(a, ut, dY[m]);
            }
        }
        if (cok)
            store_column<IO_F32>((char*)(gp.dys + ci * kChunk * p.Dv), p.Dv * 4, slane, kChunk, dY);
        // dV = beta o dY; what goes back to the state through K and Q
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 b = *(const float4*)(dec + 128 + tile_row(m, 4 * g));
            dY[m][0] *= b.x;
            dY[m][1] *= b.y;
            dY[m][2] *= b.z;
            dY[m][3] *= b.w;
        }
        if (cok)
            store_column<IO>((char*)tv.at(ch * kChunk), tv.bytes, olane, sp.len - ch * kChunk, dY);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = *(const float4*)(dec + tile_row(m, 4 * g));
            const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dY[m][r] *= -ev[r];
                dO[m][r] *= p.scale * ev[r];
            }
        }
        const float ec = dec[192];
        if (L::kBufs == 2) store(next);
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
                    x[i] = read_cols<DK>(now + L::kK + i * 4 * KB * 64, t, tb);
                a = Op::mma(x, yt[tb], a);
#pragma unroll
                for (int i = 0; i < NA; ++i)
                    x[i] = read_cols<DK>(now + L::kQ + i * 4 * KB * 64, t, tb);
                b = Op::mma(x, ot[tb], b);
            }
            if (Op::kScaled)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    D[t][r] = fmaf(sy.back, a[r], fmaf(so.back, b[r], ec * D[t][r]));
            else
                D[t] = a + b;
        }
        __syncthreads();
        if (L::kBufs == 2) {
            uint4* x = now;
            now = next;
            next = x;
        } else {
            store(lds);
            __syncthreads();
        }
    }
    if (gp.dinit && cok)
        store_state<ST>((char*)(gp.dinit + (seq * p.Hv + h) * state), p.Dv * 4, slane, p.Dk, D);
}

// ------------------------------------------------ the gradients of a chunk

// LDS of delta_grads_kernel, in uint4.  The slices of S0, D, U and dY (32
// columns, three terms; two buffers) are used up before the keys, queries and
// the 64 x 64 matrices take their place.
template <int IO, int DK>
struct GradsLds {
    static constexpr int ST = DK / 16;
    static constexpr int kS = 0, kD = 3 * ST * 64, kU = 2 * kD, kY = kU + 3 * 4 * 64;
    static constexpr int kSlice = kY + 3 * 4 * 64;
    static constexpr int kRows = Operand<IO>::NA * 4 * (DK / 32) * 64;
    static constexpr int kMat = kChunk * kLd / 4;
    static constexpr int kK = 0, kQ = kRows, kW = 2 * kRows, kWt = kW + kMat, kF = kWt + kMat;
    static constexpr int kTail = kF + kMat;
    static constexpr int kBytes = (2 * kSlice > kTail ? 2 * kSlice : kTail) * 16;
};

// Sum over the four groups of 16 lanes.
__device__ __forceinline__ float sum_groups(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// What a thread has in flight of a slice: eight elements of S0 and D, of U
// (waves 0..3) or dY and V (4..7) and of its wave's token's dO.
struct SliceRegs {
    du4 s[2], d[2], u[2], v[2], o[2];
};

// One workgroup of eight waves per chunk and key head.  A wave owns 16 tokens
// (tile w % 4) as the columns of its products, R^T = S0 dO^T and so on, and
// half of their rows (w / 4): half of a head's elements, and of the other
// tokens in the 64 x 64 part.  So a lane has one token: what belongs to it
// (decays, row sums) is a scalar of the lane, and sums over a head's elements
// are sums in the lane and over four groups.  The value heads that share the
// key head follow one another, and their parts of dQ and dK are summed in
// registers, in a fixed order.
template <int IO, int DK>
__global__ __launch_bounds__(512) void delta_grads_kernel(DeltaGradParams gp) {
    typedef GradsLds<IO, DK> L;
    typedef Operand<IO> Op;
    const DeltaParams& p = gp.f;
    constexpr int NA = Op::NA, NB = Op::NB, NO = IoTerms<IO>::n, KB = DK / 32, ST = L::ST;
    constexpr int HT = ST / 2;               // a wave's tiles of a head's elements
    constexpr int kB = IO == IO_F32 ? 4 : 2;
    extern __shared__ uint4 lds[];
    __shared__ double G[kChunk];
    __shared__ float bet[kChunk], colsum[4][kChunk], rowG[2][kChunk], rowB[2][kChunk];
    __shared__ float red[8], red3[8];
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
    const int tile = wave & 3, half = wave >> 2;
    const int rslot = 16 * g + (c ^ (4 * g));        // of a row operand
    const int mine = tile_row(tile, c);              // the lane's token
    const int have = mine < n ? mine : n - 1;        // one to read from
    const bool jwork = half <= tile >> 1;            // tokens up to the wave's
    const Tokens tk = tokens_of<IO>(p.k, sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2], p.ks[1]);
    const Tokens tq = tokens_of<IO>(p.q, sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2], p.qs[1]);
    float (*W)[kLd] = (float (*)[kLd])(lds + L::kW);     // [i][j]: W_ij
    float (*Wt)[kLd] = (float (*)[kLd])(lds + L::kWt);   // [j][i]: W_ij
    float (*F)[kLd] = (float (*)[kLd])(lds + L::kF);     // E + E^T

    dfloat4 dQ[HT], dK[HT];
#pragma unroll
    for (int t = 0; t < HT; ++t) dQ[t] = dK[t] = dfloat4{0, 0, 0, 0};

    for (int h = hk * p.group; h < (hk + 1) * p.group; ++h) {
        const long long ci = slot * p.Hv + h;
        if (wave == 0) {
            const long long gi = (sp.b * p.T + tok + (lane < n ? lane : 0)) * p.Hv + h;
            const float gv = p.g[gi], bv = p.beta[gi];
            G[lane] = decay_sum(lane < n ? gv : 0.f);
            bet[lane] = lane < n ? bv : 0.f;
        }
        // products over the columns of the state, 32 at a time
        dfloat4 R1[HT], R2[HT], R3[HT], Dp[2], Dy[2];
#pragma unroll
        for (int t = 0; t < HT; ++t) R1[t] = R2[t] = R3[t] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j) Dp[j] = Dy[j] = dfloat4{0, 0, 0, 0};
        float sd = 0.f, yv = 0.f;
        const float* S0 = p.states + ci * p.Dk * (long long)p.Dv;
        const float* D = gp.dstates + ci * p.Dk * (long long)p.Dv;
        const float* U = p.us + ci * kChunk * (long long)p.Dv;
        const float* Y = gp.dys + ci * kChunk * (long long)p.Dv;
        const char* dO = (const char*)gp.dout +
                         (((sp.b * p.T + tok + have) * p.Hv + h) * (long long)p.Dv) * kB;
        const long long vat = sp.b * p.vs[0] + (tok + have) * p.vs[1] + h * p.vs[2];
        // operands: tile t, lane (g, c) holds [tile_row(t, c)][d0 + 8 g + i];
        // the thread's are those of tile `wave` of S0 and D, of tile `tile` of
        // U or dY
        const int arow = tile_row(wave, c);
        const float* UY = half == 0 ? U : Y;
        const auto load = [&](SliceRegs& x, int d0) __attribute__((always_inline)) {
            const int e = d0 + 8 * g < p.Dv ? d0 + 8 * g : 0;
            const long long sa = (long long)(arow < p.Dk ? arow : 0) * p.Dv + e;
            const du4* s = (const du4*)(S0 + sa);
            const du4* d = (const du4*)(D + sa);
            const du4* u = (const du4*)(UY + (long long)mine * p.Dv + e);
            const du4* v = (const du4*)((const char*)p.v + (vat + e) * kB);
            const du4* o = (const du4*)(dO + e * kB);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x.s[j] = s[j];
                x.d[j] = d[j];
                x.u[j] = u[j];
            }
            x.v[0] = v[0];
            x.o[0] = o[0];
            if (IO == IO_F32) {
                x.v[1] = v[1];
                x.o[1] = o[1];
            }
        };
        const auto store = [&](const SliceRegs& x, int d0, uint4* to) __attribute__((always_inline)) {
            const bool ok = d0 + 8 * g < p.Dv;
            if (wave < ST) {
                const bool in = ok && arow < p.Dk;
                float s[8], d[8];
                uint4 ts[3], td[3];
                unpack8<IO_F32>(x.s, s);
                unpack8<IO_F32>(x.d, d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j] = in ? s[j] : 0.f;
                    d[j] = in ? d[j] : 0.f;
                    sd += s[j] * d[j];
                }
                split8<3>(s, ts);
                split8<3>(d, td);
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    to[L::kS + j * ST * 64 + threadIdx.x] = ts[j];
                    to[L::kD + j * ST * 64 + threadIdx.x] = td[j];
                }
            }
            float u[8], v[8];
            uint4 tu[3];
            unpack8<IO_F32>(x.u, u);
            unpack8<IO>(x.v, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[j] = ok ? u[j] : 0.f;
                yv += half == 1 && ok && mine < n ? u[j] * v[j] : 0.f;
            }
            split8<3>(u, tu);
#pragma unroll
            for (int j = 0; j < 3; ++j)
                to[(half == 0 ? L::kU : L::kY) + j * 256 + tile * 64 + lane] = tu[j];
        };
        SliceRegs x;
        load(x, 0);
        __syncthreads();             // the last head's matrices are used up
        store(x, 0, lds);
        __syncthreads();
        for (int d0 = 0, b = 0; d0 < p.Dv; d0 += 32, b ^= 1) {
            const uint4* now = lds + b * L::kSlice;
            const bool ok = d0 + 8 * g < p.Dv;
            // B operands: columns of the wave's tokens
            uint4 ob[NO], yb[3], ub[3];
            if constexpr (IO == IO_BF16) {
                ob[0] = keep(ok && mine < n, __builtin_bit_cast(uint4, x.o[0]));
            } else {
                float o[8];
                unpack8<IO>(x.o, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = ok && mine < n ? o[j] : 0.f;
                split8<NO>(o, ob);
            }
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                ub[j] = now[L::kU + j * 256 + tile * 64 + lane];
                yb[j] = now[L::kY + j * 256 + tile * 64 + lane];
            }
            load(x, d0 + 32 < p.Dv ? d0 + 32 : 0);
#pragma unroll
            for (int t = 0; t < HT; ++t) {
                uint4 a[3], d[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    a[j] = now[L::kS + (j * ST + half * HT + t) * 64 + lane];
                    d[j] = now[L::kD + (j * ST + half * HT + t) * 64 + lane];
                }
                R1[t] = mma_terms<3>(a, ob, R1[t]);
                R2[t] = mma_terms<3>(a, yb, R2[t]);
                R3[t] = mma_terms<3>(d, ub, R3[t]);
            }
            if (jwork)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint4 a[3];
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        a[i] = now[L::kU + i * 256 + (2 * half + j) * 64 + lane];
                    Dp[j] = mma_terms<3>(a, ob, Dp[j]);
                    Dy[j] = mma_terms<3>(a, yb, Dy[j]);
                }
            if (d0 + 32 < p.Dv) store(x, d0 + 32, lds + (b ^ 1) * L::kSlice);
            __syncthreads();
        }
        // keys and queries take the slices' place
        {
            RowTiles<IO, DK, 8> rk, rq;
            rk.load(tk, 0, n, p.Dk);
            rq.load(tq, 0, n, p.Dk);
            rk.store(lds + L::kK);
            rq.store(lds + L::kQ);
        }
        __syncthreads();
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) sd += __shfl_xor(sd, m);
        const double last = G[kChunk - 1], Gi = G[mine];
        const float eg = expf((float)Gi), ee = expf((float)(last - Gi)), b = bet[mine];
        // sums over the wave's elements of the head
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            // four elements of the token's key and query, from LDS
            float qv[4], kv[4];
            row4<IO, DK>(lds + L::kQ, tile, c, tile_row(half * HT + t, 4 * g), qv);
            row4<IO, DK>(lds + L::kK, tile, c, tile_row(half * HT + t, 4 * g), kv);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                s1 += qv[r] * R1[t][r];
                s2 += kv[r] * R2[t][r];
                s3 += kv[r] * R3[t][r];
                dQ[t][r] += p.scale * eg * R1[t][r];
                dK[t][r] += ee * R3[t][r] - b * eg * R2[t][r];
            }
        }
        s1 = p.scale * eg * s1;
        s2 = eg * s2;
        s3 = ee * s3;
        // the 64 x 64 part: the lane's token is i, tile j's row 4 g + r is j
        float sg = 0.f, sb = yv;
        if (jwork) {
            dfloat4 kk[2], qk[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint4 ko[NA], qo[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    ko[i] = lds[L::kK + ((i * 4 + tile) * KB + kb) * 64 + rslot];
                    qo[i] = lds[L::kQ + ((i * 4 + tile) * KB + kb) * 64 + rslot];
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint4 a[NA];
#pragma unroll
                    for (int i = 0; i < NA; ++i)
                        a[i] = lds[L::kK + ((i * 4 + 2 * half + j) * KB + kb) * 64 + rslot];
                    kk[j] = Op::mma_io(a, ko, kk[j]);
                    qk[j] = Op::mma_io(a, qo, qk[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int j0 = tile_row(2 * half + j, 4 * g);
                float cs[4];
                dfloat4 wr;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float w = 0.f, f = 0.f, t = 0.f;
                    if (mine >= j0 + r) {
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
                    wr[r] = w;
                    Wt[j0 + r][mine] = w;
                    cs[r] = t;
                }
                *(dfloat4*)&W[mine][j0] = wr;
                // sums over the wave's tokens
#pragma unroll
                for (int r = 0; r < 4; ++r) {
#pragma unroll
                    for (int m = 1; m < 16; m <<= 1) cs[r] += __shfl_xor(cs[r], m);
                    if (c == 0) colsum[tile][j0 + r] = cs[r];
                }
            }
        } else {
            // tokens after the wave's
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int j0 = tile_row(2 * half + j, 4 * g);
                *(dfloat4*)&W[mine][j0] = dfloat4{0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    Wt[j0 + r][mine] = 0.f;
                    if (c == 0) colsum[tile][j0 + r] = 0.f;
                }
            }
        }
        const float rg = sum_groups(sg + s1 - b * s2 - s3), rb = sum_groups(sb - s2);
        s3 = sum_groups(s3);
        if (g == 0) {
            rowG[half][mine] = rg;
            rowB[half][mine] = rb;
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
            double x = ((double)rowG[0][lane] + rowG[1][lane]) -
                       (colsum[0][lane] + colsum[1][lane] + colsum[2][lane] + colsum[3][lane]);
            if (lane == 63) {
                float s = 0.f, d = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s += red3[j];
                    d += red[j];
                }
                x += s + expf((float)last) * d;
            }
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
                gp.dbeta[gi] = rowB[0][lane] + rowB[1][lane];
            }
        }
        // dQ^T += K^T W^T, dK^T += Q^T W + K^T F
        dfloat4 wr[4], wt[4], ft[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            wr[m] = *(const dfloat4*)&W[mine][tile_row(m, 4 * g)];
            wt[m] = *(const dfloat4*)&Wt[mine][tile_row(m, 4 * g)];
            ft[m] = *(const dfloat4*)&F[mine][tile_row(m, 4 * g)];
        }
        const ColScale sw = Op::template scale_of<4>(wr), st = Op::template scale_of<4>(wt),
                       sf = Op::template scale_of<4>(ft);
        uint4 wb[2][NB], tb_[2][NB], fb[2][NB];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            Op::split(wr[2 * tb], wr[2 * tb + 1], sw, wb[tb]);
            Op::split(wt[2 * tb], wt[2 * tb + 1], st, tb_[tb]);
            Op::split(ft[2 * tb], ft[2 * tb + 1], sf, fb[tb]);
        }
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            dfloat4 a = {0, 0, 0, 0}, x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                uint4 kt[NA], qt[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    kt[i] = read_cols<DK>(lds + L::kK + i * 4 * KB * 64, half * HT + t, tb);
                    qt[i] = read_cols<DK>(lds + L::kQ + i * 4 * KB * 64, half * HT + t, tb);
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
        __syncthreads();
    }
    if (mine >= n) return;
    const long long o = ((sp.b * p.T + tok + mine) * p.Hk + hk) * p.Dk;
#pragma unroll
    for (int t = 0; t < HT; ++t) {
        const int el = tile_row(half * HT + t, 4 * g);
        if (el < p.Dk) {
            store4<IO>(gp.dq, o + el, dQ[t]);
            store4<IO>(gp.dk, o + el, dK[t]);
        }
    }
}

template <int IO, int DK, int W>
hipError_t rscan_w(const DeltaGradParams& p, hipStream_t s) {
    const int bytes = RscanLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_rscan_kernel<IO, DK, W>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const long long units = p.f.nseq * p.f.Hv * ((p.f.Dv + 16 * W - 1) / (16 * W));
    hipLaunchKernelGGL((delta_rscan_kernel<IO, DK, W>), dim3((unsigned)xcd_blocks(units)),
                       dim3(64 * W), bytes, s, p);
    return hipGetLastError();
}
template <int IO, int DK>
hipError_t rscan_io(const DeltaGradParams& p, hipStream_t s) {
    return p.f.Dv <= 64 ? rscan_w<IO, DK, 4>(p, s) : rscan_w<IO, DK, 8>(p, s);
}

template <int IO, int DK>
hipError_t grads_io(const DeltaGradParams& p, hipStream_t s) {
    const int bytes = GradsLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_grads_kernel<IO, DK>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_grads_kernel<IO, DK>), dim3((unsigned)xcd_blocks(p.f.slots * p.f.Hk)),
                       dim3(512), bytes, s, p);
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
