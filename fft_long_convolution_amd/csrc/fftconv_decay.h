// Internal declarations of linear attention with a decay for each head
// (fftconv_decay.hip, fftconv_decay_bwd.hip) and of layer norm
// (fftconv_layernorm.hip).  Host checks and the C ABI: fftconv_decay_host.cpp.
// Not part of the public ABI.
#pragma once

#include "fftconv_internal.h"

namespace fftconv {

// ------------------------------------------------------------- layer norm

struct LayerNormParams {
    long long rows;
    int D;
    float eps;
    long long stride;         // elements between rows of x
    bool wide;                // rows in 16-byte pieces: sizes and strides allow it
    bool past;                // outputs past the caches
    const void* x;
    const float* w;           // [D] or null
    const float* b;
    void* y;                  // forward: [rows][D]
    const void* dy;           // backward: [rows][D]
    void* dx;
    float* part;              // backward: [blocks][2][D] sums of dy n and dy
    float* dw;
    float* db;
    int blocks;
};
hipError_t launch_layernorm_fwd(int io, const LayerNormParams& p, hipStream_t s);
hipError_t launch_layernorm_bwd(int io, const LayerNormParams& p, hipStream_t s);
int layernorm_bwd_blocks(long long rows, int D);

// ------------------------------------------- linear attention with decays

struct DecayStepParams {
    int N, Hk, Hv, Dk, Dv;
    float scale;
    bool fixed;                      // g is [Hv]
    long long pool;
    long long qs[2], ks[2], vs[2];   // element strides (request, head)
    const void* q;
    const void* k;
    const void* v;
    const float* g;                  // [N][Hv] or [Hv]
    float* state;                    // [pool][Hv][Dk][Dv]
    const long long* slots;          // [N] or null
    void* o;                         // [N][Hv][Dv]
};
hipError_t launch_decay_step(int io, const DecayStepParams& p, hipStream_t s);

constexpr int kDecayChunk = 32;      // tokens
constexpr int kDecayCols = 64;       // columns of a head that a workgroup takes
constexpr int kSegAlign = 64;        // segments are cut at multiples of it

// A token matrix, [B][T][H][D] with strides in elements; value head h reads
// head h / group.
struct DecayRows {
    const void* p;
    long long st[3];                 // batch, token, head
    int group;
};
// Sequences, and their segments of seg_tokens tokens (a multiple of
// kSegAlign).  Equal lengths: sequence i is batch row i, its segments are
// numbers i * per ...  Packed: sequence i is the tokens cu[i] .. cu[i+1] of the
// one batch row, its segments are numbers cu[i] / seg_tokens + i ..., which
// never reach those of sequence i + 1.
struct DecaySpans {
    long long T, nseq, segs;
    int seg_tokens, per;
    const long long* cu;             // [nseq + 1] or null
};
struct DecayParams {
    DecaySpans sp;
    int Hv, Dk, Dv;
    float scale;
    bool fixed;                      // g is [Hv]
    int clear;                       // outputs of tokens that no sequence holds
    DecayRows q, k, v;
    const float* g;                  // [B][T][Hv] or [Hv]
    const float* init;               // [nseq][Hv][Dk][Dv] or null
    void* o;                         // [B][T][Hv][Dv]
    float* fin;                      // [nseq][Hv][Dk][Dv] or null
    // where a sequence may have several segments: their effects on the state and
    // then their first states, [segs][Hv][Dk][Dv], and sums of log decays
    float* seg;
    double* seg_g;                   // [segs][Hv]
};
// the segments' effects on the state (back: on its gradient) to first states
hipError_t launch_decay_join(const DecayParams& p, const float* init, bool back, hipStream_t s);
hipError_t launch_decay_fwd(int io, const DecayParams& p, hipStream_t s);

struct DecayGradParams {
    DecayParams f;                   // inputs, segments
    long long B;
    DecayRows d_o;
    const float* dfin;               // [nseq][Hv][Dk][Dv] or null
    float* seg_back;                 // effects on the gradient of the state, first ones
    // dg_t is the sum over pairs s < t <= u of what u's output owes to s.  before:
    // s before the chunk, u in it; behind: s in it, u in it or behind; both [parts
    // of the columns][Hv][B T].  ends: <d final state, final state> in parts;
    // before_all, chunks: by all tokens of a chunk what is before it, and what is
    // behind and the chunk's e^Dc, [parts of the columns][slots][Hv], a packed
    // sequence's slots from cu / chunk + its number on.  What all tokens of a chunk
    // share is in 64 bits: a fixed decay's dg sums it over all of them.
    float* before;
    float* behind;
    double* ends;
    double* before_all;
    double2* chunks;
    long long slots;
    // every 1 << anchor_shift chunks of a sequence from the first on: the state before the
    // chunk (as accumulators of its transpose, [anchors][Hv][16 columns of Dk][tiles
    // of Dv][lane]), and e^Dc times its product with the gradient of the chunk's last
    int anchor_shift;
    long long anchor_floats;         // of a head's anchor
    float* anchors;
    double* anchor_dg;               // [parts of the columns of Dk][anchors][Hv]
    long long anchor_count;
    double* sums;                    // dg of the parts of the tokens (fixed decays)
    float* dq_heads;                 // [B][T][Hv][Dk], or null where Hv = Hk
    float* dk_heads;
    void* dq;                        // [B][T][Hk][Dk]
    void* dk;
    void* dv;                        // [B][T][Hv][Dv]
    float* dg;                       // [B][T][Hv] or [Hv]
    float* dinit;                    // [nseq][Hv][Dk][Dv] or null
};
hipError_t launch_decay_bwd(int io, const DecayGradParams& p, hipStream_t s);
// Chunks between anchors.  A decay for each token: every eighth, 8 KB of states
// written and read for each chunk of a head of 128.  A fixed decay's dg sums what
// all tokens of a chunk share, and its error with it: every second.
inline int decay_anchor_shift(bool fixed) { return fixed ? 1 : 3; }
// Anchors in all; a packed sequence's start at cu / (so many chunks) + its number.
inline size_t decay_anchors(size_t T, size_t nseq, bool packed, size_t n) {
    return packed ? T / n + nseq : nseq * ((T + n - 1) / n);
}
// accumulators of an anchor, in floats
inline size_t decay_anchor_floats(int Dk, int Dv) {
    return (size_t)(Dk + 15) / 16 * ((size_t)(Dv + 31) / 32) * 512;
}
// Workgroups of the last pass over dg take so many chunks of a sequence, a multiple of
// those between anchors: none looks further than the chunk behind its own.
constexpr int kDgChunks = 64;
inline size_t decay_dg_units(size_t T, size_t nseq, bool packed) {
    const size_t n = (size_t)kDgChunks * kDecayChunk;
    return packed ? T / n + nseq : nseq * (T ? (T + n - 1) / n : 1);
}

}  // namespace fftconv
