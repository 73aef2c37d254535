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
    static constexpr int kRows = Io<IO>::NA * 4 * (DK / 32) * 64;     // uint4
    static constexpr int kK = 0, kQ = kRows, kTri = 2 * kRows, kSize = kTri + kPack;
    static constexpr int kBufs = 2 * kSize * 16 <= kLdsBytes ? 2 : 1;
    static constexpr int kBytes = kBufs * kSize * 16;
};

// The mirror of the forward walk: a wave owns 16 columns of D and goes
// through K D, T^T dU and the two transposed products without an exchange.
// FULL false: a segment's effect on D alone, from the gradient of the final
// state (the last segment of a sequence) or from 0, and in columns of their own
// the matrix D is multiplied with (from the identity, without dO).  Bound as
// the forward walk is: 64 x 1024 tokens of 6 heads of 128 in bf16 take three
// launches of 92 to 98 us, 0.7 GB of D, dY and dV written.
template <int IO, int DK, int W, bool FULL>
__global__ __launch_bounds__(64 * (W + kLoaders)) void delta_rscan_kernel(DeltaGradParams gp) {
    typedef RscanLds<IO, DK> L;
    const DeltaParams& p = gp.f;
    constexpr int NA = Io<IO>::NA, KB = DK / 32, ST = DK / 16, kB = Io<IO>::kB, kCols = 16 * W;
    extern __shared__ uint4 lds[];
    const int vcols = (p.Dv + kCols - 1) / kCols;
    const int cols = vcols + (FULL ? 0 : (p.Dk + kCols - 1) / kCols);
    const bool pieces = FULL && p.pieces > 1;
    int sn = 0;                                          // segment of the sequence
    unsigned id;
    if (pieces) {
        if (!piece_of(p, (unsigned)p.nseq * p.Hv * cols, &id, &sn)) return;
    } else {
        const unsigned units = (unsigned)p.segs * p.Hv * cols;
        id = xcd_unit(blockIdx.x, units);
        if (id >= units) return;
    }
    int cb = (int)(id % cols);
    id /= cols;
    const int h = (int)(id % p.Hv);
    id /= p.Hv;
    const long long seq = pieces ? id : seq_of(p, id, p.seg_chunks);
    const Span sp = span_of(p, seq);
    const int chunks = (sp.len + kChunk - 1) / kChunk;
    const unsigned seg0 = seg_of(p, sp, (unsigned)seq, p.seg_chunks);
    if (pieces) sn = p.pieces - 1 - sn;                  // from the end
    else sn = (int)(id - seg0);
    const long long seg = (long long)seg0 + sn;
    const long long first_ = (long long)sn * p.seg_chunks;
    if (sn < 0 || (sn != 0 && first_ >= chunks)) return;   // no such segment
    const int first = (int)first_;
    const int last = chunks - first > p.seg_chunks ? first + p.seg_chunks : chunks;
    if (!FULL && (sn == 0 || (last == chunks && cb >= vcols))) return;
    const bool matrix = !FULL && cb >= vcols;
    if (matrix) cb -= vcols;

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int slot = 16 * g + (c ^ (4 * g));             // of a row operand
    const int col = cb * kCols + wave * 16 + c;
    const int width = matrix ? p.Dk : p.Dv;
    const bool cok = col < width;
    const int colv = cok && !matrix ? col : 0;           // to read from
    const int hk = h / p.group;
    const long long state = p.Dk * (long long)p.Dv;
    dfloat4 D[ST];
    {
        const float* s = nullptr;
        if (last == chunks) s = gp.dfin ? gp.dfin + (seq * p.Hv + h) * state + col : nullptr;
        else if (FULL) s = p.seg_n + ((pieces ? seq : seg + 1) * p.Hv + h) * state + col;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = tile_row(t, 4 * g + r);
                D[t][r] = matrix ? (row == col ? 1.f : 0.f)
                                 : (s && cok && row < p.Dk ? s[(long long)row * p.Dv] : 0.f);
            }
    }
    const Tokens tk = tokens_of<IO>(p.k, sp.b * p.ks[0] + sp.t0 * p.ks[1] + hk * p.ks[2], p.ks[1]);
    const Tokens tq = tokens_of<IO>(p.q, sp.b * p.qs[0] + sp.t0 * p.qs[1] + hk * p.qs[2], p.qs[1]);
    const long long ofirst = (sp.b * p.T + sp.t0) * p.Hv * p.Dv + h * p.Dv;
    const Tokens to = tokens_of<IO>(gp.dout, ofirst, (long long)p.Hv * p.Dv);
    const Tokens tv = tokens_of<IO>(gp.dv, ofirst, (long long)p.Hv * p.Dv);
    const uint32_t olane = (uint32_t)(8 * g) * (uint32_t)to.bytes + colv * kB;
    const uint4* pack = p.bpack + (sp.slot0 * p.Hv + h) * kPack;
    const long long pack_step = (long long)p.Hv * kPack;
    if (__builtin_amdgcn_readfirstlane(wave) >= W) {
        RowTiles<IO, DK, kLoaders> rk, rq;
        Block<kPack / 64, kLoaders> rp;
        const auto load = [&](int ch) __attribute__((always_inline)) {
            const int n = sp.len - ch * kChunk;
            const uint4* next_pack = pack + ch * pack_step;
            const float* f = (const float*)(next_pack + kDec);
            rk.load(tk, ch * kChunk, n, p.Dk, f + kScaleK);
            rq.load(tq, ch * kChunk, n, p.Dk, f + kScaleQ);
            rp.load(next_pack);
        };
        const auto store = [&](uint4* d) __attribute__((always_inline)) {
            rk.store(d + L::kK);
            rq.store(d + L::kQ);
            rp.store(d + L::kTri);
        };
        if (first < last) {
            load(last - 1);
            store(lds);
        }
        __syncthreads();
        for (int ch = last - 1, buf = 0; ch >= first; --ch) {
            load(ch > first ? ch - 1 : first);
            if (L::kBufs == 2) {
                buf ^= 1;
                store(lds + buf * L::kSize);
                __syncthreads();
            } else {
                __syncthreads();
                store(lds);
                __syncthreads();
            }
        }
        return;
    }
    // dO of the next chunk.  The tokens from n on that repeat the last one
    // meet columns of P^T and rows of Q that are 0.
    Column<IO> next;
    if (first < last) next.load(to, (last - 1) * kChunk, olane, sp.len - (last - 1) * kChunk);
    __syncthreads();
    int buf = 0;
    for (int ch = last - 1; ch >= first; --ch) {
        const long long ci = (sp.slot0 + ch) * p.Hv + h;
        const uint4* now = lds + buf * L::kSize;
        const float* fac = (const float*)(now + L::kTri + kDec);
        const uint4* tri = now + L::kTri;
        dfloat4 dO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) dO[m][r] = matrix ? 0.f : next.get(m, r);
        const int ahead = ch > first ? ch - 1 : first;
        const float big_d = max_column(D);
        if (FULL && cok) save_columns<KB>(gp.dstates, ci, p.Dv, col, D, big_d);
        // dU = e^(Gc-G) o K D + P^T dO
        dfloat4 dU[4], PO[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dU[m] = PO[m] = dfloat4{0, 0, 0, 0};
        const float big_o = max_column(dO);
        const Scale sd = scale_to(big_d), so = scale_to(big_o);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint4 dt[2], a[4][NA];
            split_acc<2>(D[2 * kb], D[2 * kb + 1], sd.to, dt);
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < NA; ++i) a[m][i] = now[L::kK + ((i * 4 + m) * KB + kb) * 64 + slot];
            mma_tiles(a, dt, dU);
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint4 ot[NA];
            split_acc<NA>(dO[2 * kb], dO[2 * kb + 1], so.to, ot);
#pragma unroll
            for (int m0 = 0; m0 < 2 * kb + 2; m0 += 2) {
                uint4 a[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        a[m][i] = tri[kPm + i * kTerm + upper_tile(m0 + m, kb) * 64 + lane];
                mma_tiles(a, ot, *(dfloat4 (*)[2])&PO[m0]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = *(const float4*)(fac + kEndK + tile_row(m, 4 * g));
            const float4 f = *(const float4*)(fac + kBackP + tile_row(m, 4 * g));
            const float ev[4] = {e.x, e.y, e.z, e.w}, fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int r = 0; r < 4; ++r)
                dU[m][r] = fmaf(fv[r] * so.back, PO[m][r], (ev[r] * sd.back) * dU[m][r]);
        }
        // dY = T^T dU
        dfloat4 dY[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) dY[m] = dfloat4{0, 0, 0, 0};
        {
            const Scale su = scale_to(max_column(dU));
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                uint4 ut[2];
                split_acc<2>(dU[2 * kb], dU[2 * kb + 1], su.to, ut);
#pragma unroll
                for (int m0 = 0; m0 < 2 * kb + 2; m0 += 2) {
                    uint4 a[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            a[m][i] = tri[i * kTerm + upper_tile(m0 + m, kb) * 64 + lane];
                    mma_tiles(a, ut, *(dfloat4 (*)[2])&dY[m0]);
                }
            }
            const float back = su.back * fac[kBackT];
#pragma unroll
            for (int m = 0; m < 4; ++m) dY[m] *= back;
        }
        if (FULL) {
            const float big_y = max_column(dY);
            if (cok) save_columns<2>(gp.dys, ci, p.Dv, col, dY, big_y, big_o);
        }
        // dV = beta o dY; what goes back to the state through K and Q
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 b = *(const float4*)(fac + kBeta + tile_row(m, 4 * g));
            dY[m][0] *= b.x;
            dY[m][1] *= b.y;
            dY[m][2] *= b.z;
            dY[m][3] *= b.w;
        }
        if (FULL && cok)
            store_column<IO>((char*)tv.at(ch * kChunk), tv.bytes, olane, sp.len - ch * kChunk, dY);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 e = *(const float4*)(fac + kDecayK + tile_row(m, 4 * g));
            const float4 f = *(const float4*)(fac + kDecayQ + tile_row(m, 4 * g));
            const float ev[4] = {e.x, e.y, e.z, e.w}, fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dY[m][r] *= -ev[r];
                dO[m][r] *= fv[r];
            }
        }
        const float ec = fac[kDecayAll];
        next.load(to, ahead * kChunk, olane, sp.len - ahead * kChunk);
        const Scale sy = scale_to(max_column(dY)), sq = scale_to(max_column(dO));
        uint4 yt[2][2], ot[2][2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            split_acc<2>(dY[2 * tb], dY[2 * tb + 1], sy.to, yt[tb]);
            split_acc<2>(dO[2 * tb], dO[2 * tb + 1], sq.to, ot[tb]);
        }
#pragma unroll
        for (int t0 = 0; t0 < ST; t0 += 2) {
            dfloat4 a[2], b[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) a[t] = b[t] = dfloat4{0, 0, 0, 0};
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                uint4 x[2][NA], z[2][NA];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < NA; ++i) {
                        x[t][i] = read_cols<DK>(now + L::kK + i * 4 * KB * 64, t0 + t, tb);
                        z[t][i] = read_cols<DK>(now + L::kQ + i * 4 * KB * 64, t0 + t, tb);
                    }
                mma_tiles(x, yt[tb], a);
                mma_tiles(z, ot[tb], b);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    D[t0 + t][r] =
                        fmaf(sy.back, a[t][r], fmaf(sq.back, b[t][r], ec * D[t0 + t][r]));
        }
        __syncthreads();
        if (L::kBufs == 2) buf ^= 1;
        else __syncthreads();
    }
    if (!cok) return;
    float* d = nullptr;
    if (FULL && sn == 0) d = gp.dinit ? gp.dinit + (seq * p.Hv + h) * state : nullptr;
    else if (FULL) d = pieces ? p.seg_n + (seq * p.Hv + h) * state : nullptr;
    else if (matrix) d = p.seg_m + (seg * p.Hv + h) * p.Dk * (long long)p.Dk;
    else d = p.seg_n + (seg * p.Hv + h) * state;
    if (d) store_state<ST>((char*)d, width * 4, (uint32_t)(8 * g * width + col) * 4, p.Dk, D);
}

// ------------------------------------------------ the gradients of a chunk

// LDS of delta_grads_kernel, in uint4: a slice (32 columns, two terms) of S0, D,
// U and dY; after the last one, in its place, the chunk's keys and queries and
// two 64 x 64 matrices.  Where two workgroups fit a CU, their waits and work
// overlap.
template <int IO, int DK>
struct GradsLds {
    static constexpr int ST = DK / 16, KB = DK / 32;
    static constexpr int kRows = Io<IO>::NA * 4 * KB * 64;
    static constexpr int kSTerm = 2 * KB * 64, kUTerm = 4 * 64;      // one term of a slice
    static constexpr int kS = 0, kD = 2 * kSTerm, kU = 2 * kD, kY = kU + 2 * kUTerm;
    static constexpr int kSlice = kY + 2 * kUTerm;
    static constexpr int kMat = kChunk * kLd / 4;
    static constexpr int kK = 0, kQ = kRows, kWt = 2 * kRows, kF = kWt + kMat;
    static constexpr int kTail = kF + kMat;
    static constexpr int kBytes = (kSlice > kTail ? kSlice : kTail) * 16;
};

// What a thread has in flight of a slice: eights of S0, D, U and dY, and eight
// elements of its wave's token's dO and V in two pieces of four.
template <int IO, int DK>
struct SliceRegs {
    typedef uint32_t piece __attribute__((ext_vector_type(IO == IO_F32 ? 4 : 2)));
    static constexpr int NS = DK / 64;
    du4 s[NS][2], d[NS][2], u[2], y[2];
    piece o[2], v[2];
};
template <int IO, typename P>
__device__ __forceinline__ void unpack_pieces(const P (&x)[2], bool ok0, bool ok1, float (&y)[8]) {
    du4 r[2];
    if constexpr (IO == IO_F32) {
        r[0] = x[0];
        r[1] = x[1];
    } else {
        r[0] = du4{x[0][0], x[0][1], x[1][0], x[1][1]};
    }
    unpack8<IO>(r, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (i < 4 ? ok0 : ok1) ? y[i] : 0.f;
}

// Workgroups on a CU: two where 256 registers a lane hold what it needs, nearly.
// Backward calls with two and with one: 32 x 1024 tokens of 6 heads of 64, 3 key
// heads, bf16 (20 registers spilled) 206 and 237 us, 6 key heads, fp32 (none) 232 and
// 297; 64 x 1024 of 6 heads of 128, bf16 (6 spilled) 764 and 930, with 3 key heads
// (134 spilled) 1020 and 885.  fp32 with shared heads of 64 (46 spilled): 271 and 280
// at 768 workgroups, but 85 and 78 at 96, which have a CU each.
template <int IO, int DK, bool GROUP>
constexpr int grads_per_cu() {
    return DK > 64 ? (GROUP || IO == IO_F32 ? 1 : 2) : (GROUP && IO == IO_F32 ? 1 : 2);
}

// One workgroup of four waves per chunk and key head.  A wave owns 16 tokens as
// the columns of its products, R^T = S0 dO^T and so on.  So a lane has one
// token: what belongs to it (decays, row sums) is a scalar of the lane, and
// sums over a head's elements are sums in the lane and over four groups; W_ij
// with the lane's token as i is in its registers as the B operand of W K.  S0,
// D, U and dY come as the walks saved them, eight rows of a column together,
// and are read transposed: position i of the lane's eight columns is
// d0 + 16 (i/4) + 4 g + i%4.  They and dO have one scale each.  The value heads
// that share the key head follow one another, and their parts of dQ and dK are
// summed in registers, in a fixed order; with one (GROUP false) R1 and R3 become
// dQ and dK.  64 x 1024 tokens of 6 heads of 128 in bf16 take 510 to 560 us for
// the 1.6 GB it reads (S0 and D, in fp32 for dg's sums, are 0.8 of them, U and dY
// 0.4) and the 0.2 it writes, 3.2 to 3.5 TB/s: its registers allow two workgroups a
// CU, which wait 38 % of the time; the vector unit (the f16 terms) is busy 38 %, the
// matrix cores 15 %, and 41 % of the LDS cycles are bank conflicts.
template <int IO, int DK, bool GROUP>
__global__ __launch_bounds__(256, (grads_per_cu<IO, DK, GROUP>()))
void delta_grads_kernel(DeltaGradParams gp) {
    typedef GradsLds<IO, DK> L;
    typedef SliceRegs<IO, DK> Regs;
    const DeltaParams& p = gp.f;
    constexpr int NA = Io<IO>::NA, KB = DK / 32, ST = L::ST, kB = Io<IO>::kB;
    constexpr int NS = Regs::NS, GT = GROUP ? ST : 1;
    extern __shared__ uint4 lds[];
    __shared__ double G[kChunk];
    __shared__ double colsum[4][kChunk], rowG[kChunk], red3[4];
    __shared__ float bet[kChunk], rowB[kChunk];
    __shared__ float backK[kChunk], backQ[kChunk];
    __shared__ float red[4], big[5];
    const unsigned units = (unsigned)p.slots * p.Hk, id = xcd_unit(blockIdx.x, units);
    if (id >= units) return;
    const long long slot = id / p.Hk;
    const int hk = (int)(id - (unsigned)slot * p.Hk);
    const unsigned seq = seq_of(p, (unsigned)slot, 1);
    const Span sp = span_of(p, seq);
    const long long at = (slot - sp.slot0) * kChunk;
    unheld_tokens(p, sp, seq, (unsigned)slot, [&](long long token, int rows) {
        const long long k = (token * p.Hk + hk) * p.Dk * kB, kstep = (long long)p.Hk * p.Dk * kB;
        clear_rows((char*)gp.dq + k, kstep, rows, p.Dk * kB);
        clear_rows((char*)gp.dk + k, kstep, rows, p.Dk * kB);
        const long long first = token * p.Hv + hk * p.group;
        clear_rows((char*)gp.dv + first * p.Dv * kB, (long long)p.Hv * p.Dv * kB, rows,
                   p.group * p.Dv * kB);
        for (int i = threadIdx.x; i < rows * p.group; i += blockDim.x) {
            const long long gi = first + (long long)(i / p.group) * p.Hv + i % p.group;
            gp.dg[gi] = 0.f;
            gp.dbeta[gi] = 0.f;
        }
    });
    if (at < 0 || at >= sp.len) return;
    const int n = (int)(sp.len - at < kChunk ? sp.len - at : kChunk);
    const long long tok = sp.t0 + at;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int rslot = 16 * g + (c ^ (4 * g));        // of a row operand
    const int mine = tile_row(wave, c);              // the lane's token
    const int have = mine < n ? mine : n - 1;        // one to read from
    const int jtiles = wave < 2 ? 2 : 4;             // tiles of tokens up to the wave's
    float (*Wt)[kLd] = (float (*)[kLd])(lds + L::kWt);   // [j][i]: W_ij / rq_i
    float (*F)[kLd] = (float (*)[kLd])(lds + L::kF);     // [i][j]: (E + E^T)_ij / rk_j
    const Tokens tk = tokens_of<IO>(p.k, sp.b * p.ks[0] + tok * p.ks[1] + hk * p.ks[2], p.ks[1]);
    const Tokens tq = tokens_of<IO>(p.q, sp.b * p.qs[0] + tok * p.qs[1] + hk * p.qs[2], p.qs[1]);
    const float* fac = (const float*)(p.bpack + (slot * p.Hv + hk * p.group) * kPack + kDec);

    dfloat4 dQ[GT], dK[GT];
#pragma unroll
    for (int t = 0; t < GT; ++t) dQ[t] = dK[t] = dfloat4{0, 0, 0, 0};
    const int padded = (p.Dv + 15) / 16 * 16;
    const int hn = GROUP ? p.group : 1;

    for (int hi = 0; hi < hn; ++hi) {
        const int h = hk * p.group + hi;
        const long long ci = slot * p.Hv + h;
        const float* S0 = p.states + ci * saved_floats(DK, p.Dv);
        const float* D = gp.dstates + ci * saved_floats(DK, p.Dv);
        const float* U = p.us + ci * saved_floats(kChunk, p.Dv);
        const float* Y = gp.dys + ci * saved_floats(kChunk, p.Dv);
        const char* dO = (const char*)gp.dout +
                         ((sp.b * p.T + tok + have) * p.Hv + h) * (long long)p.Dv * kB;
        const char* V = (const char*)p.v +
                        (sp.b * p.vs[0] + (tok + have) * p.vs[1] + h * p.vs[2]) * kB;
        // the thread's eights of a slice: of U and dY number threadIdx.x, of
        // S0 and D that and 256 further
        const int u_tile = threadIdx.x >> 7, u_in = threadIdx.x & 127;
        const int pc = c ^ (4 * g);          // their column within 16
        const auto load = [&](Regs& x, int d0) __attribute__((always_inline)) {
            typedef typename Regs::piece piece;
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int i = threadIdx.x + 256 * k, t = i / (KB * 64), in = i % (KB * 64);
                const int ds = d0 + 16 * t < padded ? d0 + 16 * t : 0;
                const int first = (in & ~63) * 2 + (in & 63);        // 16-byte piece
                const du4* s = (const du4*)(S0 + (long long)ds * DK) + first;
                const du4* d = (const du4*)(D + (long long)ds * DK) + first;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    x.s[k][j] = s[64 * j];
                    x.d[k][j] = d[64 * j];
                }
            }
            const int du = d0 + 16 * u_tile < padded ? d0 + 16 * u_tile : 0;
            const int first = (u_in & ~63) * 2 + (u_in & 63);
            const du4* u = (const du4*)(U + (long long)du * kChunk) + first;
            const du4* y = (const du4*)(Y + (long long)du * kChunk) + first;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                x.u[j] = u[64 * j];
                x.y[j] = y[64 * j];
                const int e = d0 + 16 * j + 4 * g < p.Dv ? d0 + 16 * j + 4 * g : 0;
                x.o[j] = *(const piece*)(dO + e * kB);
                x.v[j] = *(const piece*)(V + e * kB);
            }
        };
        Regs x;
        load(x, 0);
        // scales: largest of S0, D, U, dY and dO over their columns
        {
            const float* m = wave == 0 ? S0 + (long long)DK * padded
                             : wave == 1 ? D + (long long)DK * padded
                             : wave == 2 ? U + (long long)kChunk * padded
                                         : Y + (long long)kChunk * padded;
            float a = 0.f, o = 0.f;
            for (int i = lane; i < p.Dv; i += 64) {
                a = fmaxf(a, m[i]);
                if (wave == 3) o = fmaxf(o, m[padded + i]);
            }
            a = max_groups(max16(a));
            o = max_groups(max16(o));
            if (lane == 0) {
                big[wave] = a;
                if (wave == 3) big[4] = o;
            }
        }
        if (wave == 0) {
            const long long gi = (sp.b * p.T + tok + (lane < n ? lane : 0)) * p.Hv + h;
            const float gv = p.g[gi], bv = p.beta[gi];
            G[lane] = decay_sum(lane < n ? gv : 0.f);
            bet[lane] = lane < n ? bv : 0.f;
        } else if (wave == 1) {
            backK[lane] = 1.f / fac[kScaleK + lane];
            backQ[lane] = 1.f / fac[kScaleQ + lane];
        }
        __syncthreads();             // and the last head's matrices are used up
        const Scale sS = scale_to(big[0]), sD = scale_to(big[1]), sU = scale_to(big[2]),
                    sY = scale_to(big[3]), sO = scale_to(big[4]);
        float sd = 0.f, yv = 0.f;
        const auto store = [&](const Regs& x, int d0) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int i = threadIdx.x + 256 * k, t = i / (KB * 64);
                const bool ok = d0 + 16 * t + pc < p.Dv;
                float s[8], d[8];
                uint4 ts[2], td[2];
                unpack8<IO_F32>(x.s[k], s);
                unpack8<IO_F32>(x.d[k], d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j] = ok ? s[j] : 0.f;
                    d[j] = ok ? d[j] : 0.f;
                    sd += s[j] * d[j];
                }
                split8h<2>(s, sS.to, ts);
                split8h<2>(d, sD.to, td);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lds[L::kS + j * L::kSTerm + i] = ts[j];
                    lds[L::kD + j * L::kSTerm + i] = td[j];
                }
            }
            float u[8], y[8];
            uint4 tu[2], ty[2];
            unpack8<IO_F32>(x.u, u);
            unpack8<IO_F32>(x.y, y);
            const bool ok = d0 + 16 * u_tile + pc < p.Dv;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[j] = ok ? u[j] : 0.f;
                y[j] = ok ? y[j] : 0.f;
            }
            split8h<2>(u, sU.to, tu);
            split8h<2>(y, sY.to, ty);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                lds[L::kU + j * L::kUTerm + threadIdx.x] = tu[j];
                lds[L::kY + j * L::kUTerm + threadIdx.x] = ty[j];
            }
        };
        // products over the columns of the state, 32 at a time
        dfloat4 R1[ST], R2[ST], R3[ST], Dp[4], Dy[4];
#pragma unroll
        for (int t = 0; t < ST; ++t) R1[t] = R2[t] = R3[t] = dfloat4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) Dp[j] = Dy[j] = dfloat4{0, 0, 0, 0};
        for (int d0 = 0; d0 < p.Dv; d0 += 32) {
            store(x, d0);
            // B operands: columns of the wave's tokens
            uint4 ob[NA], yb[2], ub[2];
            float v[8];
            {
                const bool ok0 = mine < n && d0 + 4 * g < p.Dv;
                const bool ok1 = mine < n && d0 + 16 + 4 * g < p.Dv;
                float o[8];
                unpack_pieces<IO>(x.o, ok0, ok1, o);
                split8h<NA>(o, sO.to, ob);
                unpack_pieces<IO>(x.v, ok0, ok1, v);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ub[j] = read_cols<64>(lds + L::kU + j * L::kUTerm, wave, 0);
                yb[j] = read_cols<64>(lds + L::kY + j * L::kUTerm, wave, 0);
            }
            {
                const dh8 y0 = __builtin_bit_cast(dh8, yb[0]), y1 = __builtin_bit_cast(dh8, yb[1]);
#pragma unroll
                for (int j = 0; j < 8; ++j) yv += ((float)y0[j] + (float)y1[j]) * v[j];
            }
#pragma unroll
            for (int t0 = 0; t0 < ST; t0 += 2) {
                uint4 a[2][2], d[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        a[t][j] = read_cols<DK>(lds + L::kS + j * L::kSTerm, t0 + t, 0);
                        d[t][j] = read_cols<DK>(lds + L::kD + j * L::kSTerm, t0 + t, 0);
                    }
                mma_tiles(a, ob, *(dfloat4 (*)[2])&R1[t0]);
                mma_tiles(a, yb, *(dfloat4 (*)[2])&R2[t0]);
                mma_tiles(d, ub, *(dfloat4 (*)[2])&R3[t0]);
            }
#pragma unroll
            for (int j0 = 0; j0 < 4; j0 += 2)
                if (j0 < jtiles) {
                    uint4 a[2][2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            a[j][i] = read_cols<64>(lds + L::kU + i * L::kUTerm, j0 + j, 0);
                    mma_tiles(a, ob, *(dfloat4 (*)[2])&Dp[j0]);
                    mma_tiles(a, yb, *(dfloat4 (*)[2])&Dy[j0]);
                }
            load(x, d0 + 32 < p.Dv ? d0 + 32 : 0);
            __syncthreads();
        }
        {
            RowTiles<IO, DK, 4> rk, rq;
            rk.load(tk, 0, n, p.Dk, fac + kScaleK);
            rq.load(tq, 0, n, p.Dk, fac + kScaleQ);
            rk.store(lds + L::kK);
            rq.store(lds + L::kQ);
        }
        __syncthreads();
        sd = sum_groups(sum16(sd));
        yv *= sY.back;
        const double last = G[kChunk - 1], Gi = G[mine];
        const float eg = decay(Gi), ee = decay(last - Gi), b = bet[mine];
        const float bk = backK[mine], bq = backQ[mine];
        // sums over the elements of a head
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        {
            const float f1 = p.scale * eg * (sS.back * sO.back), f2 = eg * (sS.back * sY.back),
                        f3 = ee * (sD.back * sU.back);
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                // four elements of the token's key and query
                float qv[4], kv[4];
                row4<NA, DK>(lds + L::kQ, wave, c, tile_row(t, 4 * g), qv);
                row4<NA, DK>(lds + L::kK, wave, c, tile_row(t, 4 * g), kv);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float r1 = f1 * R1[t][r], r2 = f2 * R2[t][r], r3 = f3 * R3[t][r];
                    s1 += qv[r] * r1;
                    s2 += kv[r] * r2;
                    s3 += kv[r] * r3;
                    R1[t][r] = r1;
                    R3[t][r] = r3 - b * r2;
                }
            }
        }
        s1 *= bq;
        s2 *= bk;
        s3 *= bk;
        // The 64 x 64 part: the lane's token is i, tile j's row 4 g + r is j.
        // dg is dG summed from the end, where a term of tokens i and j counts
        // for the g between them alone: in all others it stands in a row and in
        // a column, and has to leave nothing.  So these sums are of 64 bits; in
        // 32 dg was off by 1e-7 of the terms, all of it where e^g is as small.
        double sg = 0.;
        float sb = yv;
        {
            dfloat4 kk[4], qk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) kk[j] = qk[j] = dfloat4{0, 0, 0, 0};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint4 ko[NA], qo[NA];
#pragma unroll
                for (int i = 0; i < NA; ++i) {
                    ko[i] = lds[L::kK + ((i * 4 + wave) * KB + kb) * 64 + rslot];
                    qo[i] = lds[L::kQ + ((i * 4 + wave) * KB + kb) * 64 + rslot];
                }
#pragma unroll
                for (int j0 = 0; j0 < 4; j0 += 2)
                    if (j0 < jtiles) {
                        uint4 a[2][NA];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < NA; ++i)
                                a[j][i] = lds[L::kK + ((i * 4 + j0 + j) * KB + kb) * 64 + rslot];
                        mma_tiles(a, ko, *(dfloat4 (*)[2])&kk[j0]);
                        mma_tiles(a, qo, *(dfloat4 (*)[2])&qk[j0]);
                    }
            }
            const float fp = p.scale * (sU.back * sO.back), fy = sU.back * sY.back;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int j0 = tile_row(j, 4 * g);
                float t[4];
                const dfloat4 bj = *(const dfloat4*)&backK[j0];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float w = 0.f, f = 0.f;
                    t[r] = 0.f;
                    if (j < jtiles && mine >= j0 + r) {
                        const float gam = decay(Gi - G[j0 + r]);
                        const float kij = kk[j][r] * (bk * bj[r]);
                        w = gam * (fp * Dp[j][r]);
                        const float x = mine > j0 + r ? gam * (fy * Dy[j][r]) : 0.f;
                        f = -b * x;
                        t[r] = w * (qk[j][r] * (bq * bj[r])) + f * kij;
                        sg += t[r];
                        sb -= x * kij;
                        F[mine][j0 + r] = f * bj[r];
                        if (mine > j0 + r) F[j0 + r][mine] = f * bk;
                    }
                    Dp[j][r] = w * bj[r];        // the lane's row of W
                    Wt[j0 + r][mine] = w * bq;
                }
                // over the wave's tokens
                const double cs = sum16_of4(t);
                if ((c & 3) == 0) colsum[wave][j0 + (c >> 2)] = cs;
            }
        }
        const double s3_all = sum_groups((double)s3);
        const double rg = sum_groups(sg + (s1 - b * s2)) - s3_all;
        const float rb = sum_groups(sb - s2);
        if (g == 0) {
            rowG[mine] = rg;
            rowB[mine] = rb;
        }
        // the chunk's last decay
        double s3_wave = s3_all + moved<0x128>(s3_all);
        s3_wave += moved<0x141>(s3_wave);
        s3_wave += moved<0xb1>(s3_wave);
        s3_wave += moved<0x4e>(s3_wave);
        if (lane == 0) {
            red[wave] = sd;
            red3[wave] = s3_wave;
        }
        __syncthreads();
        if (wave == 0) {
            double x = rowG[lane] -
                       (colsum[0][lane] + colsum[1][lane] + colsum[2][lane] + colsum[3][lane]);
            if (lane == 63)
                x += (red3[0] + red3[1] + red3[2] + red3[3]) +
                     decay(last) * (red[0] + red[1] + red[2] + red[3]);
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
            wt[m] = *(const dfloat4*)&Wt[mine][tile_row(m, 4 * g)];
            ft[m] = *(const dfloat4*)&F[mine][tile_row(m, 4 * g)];
        }
        const Scale sw = scale_to(max_column(Dp)), st = scale_to(max_column(wt)),
                    sf = scale_to(max_column(ft));
        uint4 wb[2][2], tb_[2][2], fb[2][2];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
            split_acc<2>(Dp[2 * tb], Dp[2 * tb + 1], sw.to, wb[tb]);
            split_acc<2>(wt[2 * tb], wt[2 * tb + 1], st.to, tb_[tb]);
            split_acc<2>(ft[2 * tb], ft[2 * tb + 1], sf.to, fb[tb]);
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
                a = mma_prod(kt, wb[tb], a);
                x = mma_prod(qt, tb_[tb], x);
                y = mma_prod(kt, fb[tb], y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                R1[t][r] += sw.back * a[r];
                R3[t][r] += st.back * x[r] + sf.back * y[r];
            }
            if (GROUP) {
                dQ[t % GT] += R1[t];
                dK[t % GT] += R3[t];
            }
        }
        if (!GROUP || hi + 1 == hn) {
            if (mine < n) {
                const long long o = ((sp.b * p.T + tok + mine) * p.Hk + hk) * p.Dk;
#pragma unroll
                for (int t = 0; t < ST; ++t) {
                    const int el = tile_row(t, 4 * g);
                    if (el < p.Dk) {
                        store4<IO>(gp.dq, o + el, GROUP ? dQ[t % GT] : R1[t]);
                        store4<IO>(gp.dk, o + el, GROUP ? dK[t % GT] : R3[t]);
                    }
                }
            }
        }
        // the next head's slices take the matrices' place only behind the
        // barrier that follows its scales
    }
}

template <int IO, int DK, int W, bool FULL>
hipError_t rscan_launch(const DeltaGradParams& p, const WalkGrid& w, hipStream_t s) {
    const int bytes = RscanLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_rscan_kernel<IO, DK, W, FULL>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    DeltaGradParams r = p;
    do {
        hipLaunchKernelGGL((delta_rscan_kernel<IO, DK, W, FULL>), dim3((unsigned)w.blocks()),
                           dim3(w.threads()), bytes, s, r);
    } while (FULL && p.f.pieces > 1 && ++r.f.round < r.f.rounds);
    return hipGetLastError();
}
template <int IO, int DK, bool FULL>
hipError_t rscan_mode(const DeltaGradParams& p, hipStream_t s) {
    const WalkGrid w = walk_grid(p.f, !FULL);
    return w.waves == 4 ? rscan_launch<IO, DK, 4, FULL>(p, w, s)
                        : rscan_launch<IO, DK, 8, FULL>(p, w, s);
}
template <int IO, int DK>
hipError_t rscan_io(const DeltaGradParams& p, hipStream_t s) {
    if (p.f.seg_m) {
        hipError_t e = rscan_mode<IO, DK, false>(p, s);
        if (e == hipSuccess) e = launch_delta_join(p.f, true, s);
        if (e != hipSuccess) return e;
    }
    return rscan_mode<IO, DK, true>(p, s);
}

template <int IO, int DK, bool GROUP>
hipError_t grads_launch(const DeltaGradParams& p, hipStream_t s) {
    const int bytes = GradsLds<IO, DK>::kBytes;
    const hipError_t e = hipFuncSetAttribute((const void*)delta_grads_kernel<IO, DK, GROUP>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_grads_kernel<IO, DK, GROUP>),
                       dim3((unsigned)xcd_blocks(p.f.slots * p.f.Hk)), dim3(256), bytes, s, p);
    return hipGetLastError();
}
template <int IO, int DK>
hipError_t grads_io(const DeltaGradParams& p, hipStream_t s) {
    return p.f.group == 1 ? grads_launch<IO, DK, false>(p, s) : grads_launch<IO, DK, true>(p, s);
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
