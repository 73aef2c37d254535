// Internal declarations of the token-mixer operators that stand next to the
// long convolution: norms of queries and keys with the position rotation
// (fftconv_qknorm.hip) and the gated delta rule (fftconv_delta.hip,
// fftconv_delta_bwd.hip).  Host checks and the C ABI: fftconv_delta_host.cpp.
// Not part of the public ABI.
#pragma once

#include "fftconv_internal.h"

namespace fftconv {

// ------------------------------------------------------------- q/k norms

struct QkNormParams {
    long long tokens;         // B * T
    long long T;
    int Hq, Hk, D, R;         // R: rotated elements of a head
    int interleaved;
    int parts;                // threads groups a token's heads are dealt to
    float c, eps;             // r = rsqrt(c sum x^2 + eps)
    long long P;              // rows of the tables
    long long qs[3], ks[3];   // element strides (batch, token, head) of q, k
    const void* q;
    const void* k;
    const float* wq;          // [D] or null
    const float* wk;
    const float* cs;          // [P][R/2]
    const float* sn;
    const long long* pos;     // [B][T]
    void* qo;                 // forward: outputs, [B][T][H][D]
    void* ko;
    const void* dqo;          // backward: gradients of the outputs
    const void* dko;
    void* dq;
    void* dk;
    float* part;              // backward: [blocks][2][D] weight-gradient sums
    float* dwq;
    float* dwk;
    int blocks;
};
hipError_t launch_qknorm_fwd(int io, const QkNormParams& p, hipStream_t s);
hipError_t launch_qknorm_bwd(int io, const QkNormParams& p, hipStream_t s);
int qknorm_bwd_blocks(long long tokens);

// ------------------------------------------------------- gated delta rule

struct DeltaStepParams {
    int N, Hk, Hv, Dk, Dv;
    float scale;
    long long pool;
    long long qs[2], ks[2], vs[2];   // element strides (request, head)
    const void* q;
    const void* k;
    const void* v;
    const float* g;                  // [N][Hv]
    const float* beta;
    float* state;                    // [pool][Hv][Dk][Dv]
    const long long* slots;          // [N] or null
    void* o;                         // [N][Hv][Dv]
};
hipError_t launch_delta_step(int io, const DeltaStepParams& p, hipStream_t s);

// Sequences in chunks of kChunk tokens.  Equal lengths: sequence i is batch
// row i, its chunks are slots i * nch ...  Packed: sequence i is the tokens
// cu[i] .. cu[i+1] of the one batch row, its chunks are slots
// cu[i] / kChunk + i ..., which never reach those of sequence i + 1.
constexpr int kChunk = 64;
constexpr int kTriTiles = 6;               // 16 x 32 tiles of a 64 x 64 triangle
// What a chunk and value head needs besides its tokens, in matrix-operand
// order, one uint4 a lane: (I + A)^-1 in two f16 terms, the chunk's factors
// (decays, beta, scales), the decayed scores P.
int delta_pack_uint4();                    // the pack of its transposes alike

// Time of a walk for each chunk of its longest chain, in us, by the number of
// workgroups that take 64 or 128 columns (four or eight waves for the chain):
// alone on a card and with all 256 CUs taken, for heads of 128 at 16 bits.  (The
// outputs' are 3.0 and 4.5 with four and 4.9 and 6.9 with eight now, f16 within 6 %;
// effects 2.2 and 2.5, 3.1 and 4.0.)  Heads of 64 take 0.75 to 0.85 of it and fp32
// 1.4 to 1.65, with four and eight alike, so they choose alike.  A workgroup has a CU to itself, so more than 256 run in rounds;
// packed sequences differ in length, and about half of a further round is hidden
// behind the longest of them.  *waves: the better of four and eight.
//
// Held against 45 measured calls, 13 of equal and 32 of packed sequences (half of
// them of lengths as of chance), 1 to 100 rows, heads of 64 to 128 x 64 to 256, all
// types: what this and delta_cut() choose is within 5 % of the best of whole and
// cut walks on average, 22 % at most.  The most by a length that the host does not
// know.  Four or eight waves: 23 sequences of 9001 tokens, 8 heads of 64 x 128, f16,
// 98 us with four (chosen) and 112 with eight, of equal lengths 76 and 63; 30 of
// 12000, 12 heads of 128, bf16, 178 and 202 (chosen), of equal ones 135 and 142; 38 of
// 16000, 6 heads of 128 x 256, 226 and 199 (chosen), 149 and 130.  Segments: 10 of
// 16000, 2 heads of 128, in 5 chunks (chosen) 152 us and in 12, 129; 5 of 4000, 3 of 96,
// fp32, in 3 (chosen) 128 and in 4, 106.
inline double walk_us(double units64, double units128, bool effect, bool packed, int* waves) {
    const double cus = 256.0;
    const auto time = [&](double units, double alone, double full) {
        const double load = units / cus;
        const double rounds = load <= 1 ? 1
                              : packed  ? 0.5 + 0.5 * load
                                        : (double)(long long)(load + 0.999999);
        return rounds * (alone + (full - alone) * (load < 1 ? load : 1));
    };
    const double four = effect ? time(units64, 2.5, 3.25) : time(units64, 3.4, 4.7);
    const double eight = effect ? time(units128, 3.6, 4.7) : time(units128, 4.7, 6.2);
    if (waves) *waves = four <= eight ? 4 : 8;
    return four <= eight ? four : eight;
}

struct DeltaParams {
    int Hk, Hv, group, Dk, Dv;
    float scale;
    long long T;
    long long qs[3], ks[3], vs[3];   // element strides (batch, token, head)
    const long long* cu;             // [nseq + 1] or null
    bool packed;                     // cu is given
    int clear;                       // o of tokens that no sequence holds
    long long nseq, nch, slots;
    const void* q;
    const void* k;
    const void* v;
    const float* g;                  // [B][T][Hv]
    const float* beta;
    const float* init;               // [nseq][Hv][Dk][Dv] or null
    void* o;                         // [B][T][Hv][Dv]
    float* fin;                      // [nseq][Hv][Dk][Dv] or null
    uint4* pack;                     // [slots][Hv] packs
    uint4* bpack;                    // the transposes' packs, or null
    // sequences longer than seg_chunks chunks are cut into segments, numbered
    // like the slots of chunks, where seg_m is given
    long long segs;
    int seg_chunks;
    float* seg_n;                    // [segs][Hv][Dk][Dv]; pieces: [nseq] ...
    float* seg_m;                    // [segs][Hv][Dk][Dk]
    // > 1: a walk's chains go in so many pieces (the segments), seg_n handed from
    // one to the next, `rounds` launches of workgroups of `waves` chain waves
    int pieces, rounds, round, waves;
    // for the backward, or null: each chunk's first state and U, [slots][Hv]
    // matrices in the layout of saved_floats()
    float* states;
    float* us;
};
constexpr int kLoaders = 4;   // waves of a walk that bring the operands
// A walk's launch: waves for the chain and workgroups.  effect: of the walk that
// makes the segments' effects on the state, with columns for the matrices too.
struct WalkGrid {
    int waves;
    long long units;
    int threads() const { return 64 * (waves + kLoaders); }
    // dealt to the XCDs in eights; the threads of a launch are a 32-bit number
    long long blocks() const { return (units + 7) / 8 * 8; }
    bool fits() const { return blocks() * threads() <= 0xffffffffll; }
};
inline WalkGrid walk_grid(const DeltaParams& p, bool effect) {
    const auto columns = [&](int width) {
        return (p.Dv + width - 1) / width + (effect ? (p.Dk + width - 1) / width : 0);
    };
    WalkGrid w;
    if (p.pieces > 1 && !effect) {
        // workgroups that take one of the chains' pieces in each round
        w.waves = p.waves;
        w.units = (p.nseq * p.Hv * columns(16 * w.waves) * p.pieces + p.rounds - 1) / p.rounds;
        return w;
    }
    const double chains = (double)p.segs * p.Hv;
    walk_us(chains * columns(64), chains * columns(128), effect, p.packed, &w.waves);
    w.units = p.segs * p.Hv * columns(16 * w.waves);
    return w;
}

struct DeltaGradParams {
    DeltaParams f;                   // inputs, bpack, states, us, segments
    const void* dout;                // [B][T][Hv][Dv]
    const float* dfin;               // [nseq][Hv][Dk][Dv] or null
    float* dstates;                  // [slots][Hv] saved matrices: gradient of
    float* dys;                      // each chunk's last state, T^T dU
    void* dq;                        // [B][T][Hk][Dk]
    void* dk;
    void* dv;                        // [B][T][Hv][Dv]
    float* dg;                       // [B][T][Hv]
    float* dbeta;
    float* dinit;                    // [nseq][Hv][Dk][Dv] or null
};
// reverse: the segments' effects on the gradient of the state, from the last on
hipError_t launch_delta_join(const DeltaParams& p, bool reverse, hipStream_t s);
hipError_t launch_delta_rscan(int io, const DeltaGradParams& p, hipStream_t s);
hipError_t launch_delta_grads(int io, const DeltaGradParams& p, hipStream_t s);
hipError_t launch_delta_prep(int io, const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_scan(int io, const DeltaParams& p, hipStream_t s);

}  // namespace fftconv
