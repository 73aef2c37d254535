// Host side of the token-mixer operators: argument checks, buffer layouts and
// the C ABI declared in include/fftconv.h.
#include <stdint.h>

#include "../../include/fftconv.h"
#include "fftconv_delta.h"

using namespace fftconv;

namespace {

constexpr size_t kMaxCount = 0x7fffffff;      // of any one dimension
constexpr size_t kMaxElems = (size_t)1 << 46; // of any one tensor
constexpr size_t kMaxGrid = 0xfffff0;         // workgroups of 256 threads of a launch

constexpr size_t kMaxTokenStride = (size_t)1 << 24;  // elements, gated delta rule

// a byte range of the caller's memory
struct Range {
    const void* p;
    size_t n;
};

bool meet(const Range& a, const Range& b) {
    if (!a.p || !b.p || !a.n || !b.n) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + b.n && y < x + a.n;
}
// no output may meet an input or another output
template <size_t NO, size_t NI>
bool outputs_clear(const Range (&out)[NO], const Range (&in)[NI]) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return false;
        for (size_t j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return false;
    }
    return true;
}
// a missing pointer or one that is not 16-byte aligned
fftconv_status check_ptr(const void* p, size_t bytes, bool needed = true) {
    if (!p) return needed && bytes ? FFTCONV_ERR_INVALID_ARG : FFTCONV_OK;
    return ((uintptr_t)p & 15) ? FFTCONV_ERR_ALIGNMENT : FFTCONV_OK;
}

bool dtype_ok(fftconv_dtype t) {
    return t == FFTCONV_F32 || t == FFTCONV_F16 || t == FFTCONV_BF16;
}
size_t elem(fftconv_dtype t) { return t == FFTCONV_F32 ? 4 : 2; }

// a * b * c * d, false beyond kMaxElems
bool product(size_t a, size_t b, size_t c, size_t d, size_t* out) {
    size_t r = 1;
    const size_t f[4] = {a, b, c, d};
    for (size_t x : f)
        if (x == 0) { *out = 0; return true; }
    for (size_t x : f) {
        if (x > kMaxElems / r) return false;
        r *= x;
    }
    *out = r;
    return true;
}

// Bytes a strided [B][T][H][D] tensor spans, or an error.
fftconv_status span_bytes(size_t B, size_t T, size_t H, size_t D, const long long st[3],
                          fftconv_dtype t, size_t* bytes) {
    *bytes = 0;
    const long long step = (long long)(16 / elem(t));
    const size_t n[3] = {B, T, H};
    size_t last = 0;
    if (!B || !T || !H || !D) return FFTCONV_OK;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || (size_t)st[i] > kMaxElems) return FFTCONV_ERR_INVALID_ARG;
        if (n[i] > 1 && st[i] % step) return FFTCONV_ERR_ALIGNMENT;
        if (n[i] > 1 && (size_t)st[i] > kMaxElems / (n[i] - 1)) return FFTCONV_ERR_INVALID_ARG;
        last += (n[i] - 1) * (size_t)st[i];
    }
    if (last > kMaxElems) return FFTCONV_ERR_INVALID_ARG;
    *bytes = (last + D) * elem(t);
    return FFTCONV_OK;
}

#define CHECK(expr)                                      \
    do {                                                 \
        const fftconv_status status_ = (expr);           \
        if (status_ != FFTCONV_OK) return status_;       \
    } while (0)

fftconv_status launched(hipError_t e) { return e == hipSuccess ? FFTCONV_OK : FFTCONV_ERR_HIP; }

// ------------------------------------------------------------- q/k norms

fftconv_status qknorm_sizes(const fftconv_qknorm_desc* d) {
    if (!d) return FFTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return FFTCONV_ERR_UNSUPPORTED;
    if (d->norm != FFTCONV_NORM_RMS && d->norm != FFTCONV_NORM_L2) return FFTCONV_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f)) return FFTCONV_ERR_INVALID_ARG;
    if (d->D == 0 || d->D % 8 || d->D > 256) return FFTCONV_ERR_UNSUPPORTED;
    if (d->rotary_dim > d->D) return FFTCONV_ERR_INVALID_ARG;
    if (d->rotary_dim % (d->interleaved ? 8 : 16)) return FFTCONV_ERR_UNSUPPORTED;
    if (d->B > kMaxCount || d->T > kMaxCount || d->Hq > 65536 || d->Hk > 65536)
        return FFTCONV_ERR_UNSUPPORTED;
    size_t n;
    if (!product(d->B, d->T, d->Hq + d->Hk, d->D, &n)) return FFTCONV_ERR_UNSUPPORTED;
    if (d->table_rows > kMaxCount) return FFTCONV_ERR_UNSUPPORTED;
    return FFTCONV_OK;
}

struct QkNormArgs {
    const void *q, *k;
    const float *wq, *wk, *cos, *sin;
    const long long* pos;
};

// Checks what both directions read and fills the kernels' parameters.
fftconv_status qknorm_inputs(const fftconv_qknorm_desc* d, const QkNormArgs& a, QkNormParams& p,
                             Range (&in)[7]) {
    CHECK(qknorm_sizes(d));
    size_t qb, kb;
    CHECK(span_bytes(d->B, d->T, d->Hq, d->D, d->q_stride, d->dtype, &qb));
    CHECK(span_bytes(d->B, d->T, d->Hk, d->D, d->k_stride, d->dtype, &kb));
    const size_t tokens = d->B * d->T, work = tokens * (d->Hq + d->Hk);
    const size_t table = work && d->rotary_dim ? d->table_rows * (d->rotary_dim / 2) * 4 : 0;
    const size_t posb = work && d->rotary_dim ? tokens * 8 : 0;
    CHECK(check_ptr(a.q, qb));
    CHECK(check_ptr(a.k, kb));
    CHECK(check_ptr(a.wq, 0, false));
    CHECK(check_ptr(a.wk, 0, false));
    if (posb && (!a.cos || !a.sin || !a.pos) && d->table_rows) return FFTCONV_ERR_INVALID_ARG;
    if (posb && !a.pos) return FFTCONV_ERR_INVALID_ARG;
    CHECK(check_ptr(a.cos, table));
    CHECK(check_ptr(a.sin, table));
    if ((uintptr_t)a.pos & 7) return FFTCONV_ERR_ALIGNMENT;
    in[0] = {a.q, qb};
    in[1] = {a.k, kb};
    in[2] = {a.wq, d->D * 4};
    in[3] = {a.wk, d->D * 4};
    in[4] = {a.cos, table};
    in[5] = {a.sin, table};
    in[6] = {a.pos, posb};
    p = QkNormParams();
    p.tokens = (long long)tokens;
    p.T = (long long)d->T;
    p.Hq = (int)d->Hq;
    p.Hk = (int)d->Hk;
    p.D = (int)d->D;
    p.R = (int)d->rotary_dim;
    p.interleaved = d->interleaved != 0;
    p.c = d->norm == FFTCONV_NORM_RMS ? 1.f / (float)d->D : 1.f;
    p.eps = d->eps;
    p.P = (long long)d->table_rows;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = d->q_stride[i];
        p.ks[i] = d->k_stride[i];
    }
    p.q = a.q;
    p.k = a.k;
    p.wq = a.wq;
    p.wk = a.wk;
    p.cs = a.cos;
    p.sn = a.sin;
    p.pos = a.pos;
    // Heads of a token are dealt to several groups of lanes while there are
    // too few tokens to fill the card (some 16 groups for each SIMD).
    const size_t H = d->Hq + d->Hk, want = 16384;
    size_t parts = tokens ? (want + tokens - 1) / tokens : 1;
    if (parts > H) parts = H;
    p.parts = (int)(parts ? parts : 1);
    if (tokens * (size_t)p.parts / 8 > kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    return FFTCONV_OK;
}

// ------------------------------------------------------- gated delta rule

fftconv_status delta_sizes(const fftconv_delta_desc* d) {
    if (!d) return FFTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return FFTCONV_ERR_UNSUPPORTED;
    if (!d->Dk || d->Dk % 8 || d->Dk > 128 || !d->Dv || d->Dv % 8 || d->Dv > 1024)
        return FFTCONV_ERR_UNSUPPORTED;
    if (!d->Hk || d->Hv % d->Hk || !d->Hv) return FFTCONV_ERR_INVALID_ARG;
    if (d->Hv > 65536 || d->B > kMaxCount || d->T > kMaxCount - 64 || d->sequences > kMaxCount)
        return FFTCONV_ERR_UNSUPPORTED;
    if (d->sequences && d->B != 1) return FFTCONV_ERR_INVALID_ARG;
    size_t n;
    if (!product(d->B, d->T, d->Hv, d->Dv, &n) || !product(d->B, d->T, d->Hk, d->Dk, &n))
        return FFTCONV_ERR_UNSUPPORTED;
    const size_t rows = d->sequences ? d->sequences : d->B;
    if (!product(rows, d->Hv, d->Dk, d->Dv, &n)) return FFTCONV_ERR_UNSUPPORTED;
    return FFTCONV_OK;
}

size_t delta_slots(const fftconv_delta_desc* d) {
    const size_t per = (d->T + kChunk - 1) / kChunk;
    return d->sequences ? per + d->sequences : d->B * per;
}

// Chunks of a segment.  A sequence is a chain of chunks; where the heads and
// columns leave CUs idle, sequences are cut into segments that are walked side
// by side: once for their effects on the state, and, after a join, for the
// outputs; the backward walk likewise.  The number of segments is the one of
// least time by walk_us() and the steps of the join (2.5 us at D_k = 64, 7 at
// 128), 1 where that is least.  bf16, forward: 4 x 32768 tokens of 4 heads of
// 128, 16 segments, 0.73 ms, uncut 1.75; 1 x 4096 x 8: 8, 0.12 ms, uncut 0.22;
// 16 x 8192 x 6: uncut 0.63, in three 1.06.  With the gradients, fp32, 2 x 1501
// tokens of 4 heads of 64: 8 segments, 137 us, uncut 229.
//
// Where the chains are more than the CUs, a last round of few would take as
// long as a full one.  So equal chains are cut into pieces, which launches of
// at most one workgroup a CU take round by round (piece_of() in the kernels).  A
// round costs some 7 us beside its chunks.  Of calls, bf16 and heads of 128, in
// pieces and whole: 64 x 1024 tokens of 6 heads, 384 chains in halves, 309 and
// 322 us (with gradients 1188 and 1198); 33 x 4096 of 8, 264 chains, 0.84 and
// 1.01 ms (3.24 and 3.61); 10 x 8192 of 32 in f16, 320 chains, 1.69 and 2.01
// (7.3 and 8.3).
struct Cut {
    size_t per;             // chunks of a segment or piece
    int pieces, rounds, waves;
};
Cut delta_cut(const fftconv_delta_desc* d) {
    const size_t nch = (d->T + kChunk - 1) / kChunk;
    const size_t rows = d->sequences ? d->sequences : d->B;
    const size_t chunks = d->sequences ? nch : d->B * nch;
    Cut cut = {nch + 1, 1, 1, 0};           // one segment a sequence
    const size_t L = rows ? chunks / rows : 0;      // of a sequence, on average
    const bool packed = d->sequences != 0;
    const double heads = (double)rows * d->Hv;
    const size_t v64 = (d->Dv + 63) / 64, v128 = (d->Dv + 127) / 128;
    const size_t k64 = (d->Dk + 63) / 64, k128 = (d->Dk + 127) / 128;
    // a chunk of fp32 against one of 16 bits; a step of the join
    const double chunk = d->dtype == FFTCONV_F32 ? 1.35 : 1.0;
    const double join = d->Dk <= 64 ? 2.5 : 7.0;
    double best = chunk * L * walk_us(heads * v64, heads * v128, false, packed, nullptr);
    for (size_t n = 3; n <= 64 && n * 2 <= L; ++n) {
        const size_t p = (L + n - 1) / n;
        if (L < 8 || (L + p - 1) / p != n) continue;
        const double full = walk_us(heads * n * v64, heads * n * v128, false, packed, nullptr);
        const double effect = walk_us(heads * ((n - 1) * v64 + (n - 2) * k64),
                                      heads * ((n - 1) * v128 + (n - 2) * k128), true, packed,
                                      nullptr);
        const double t = chunk * p * (full + effect) + join * (n - 2) + 12.0;
        if (t < best) {
            best = t;
            cut.per = p;
        }
    }
    for (int waves = 4; waves <= 8 && !packed; waves += 4) {
        const double chains = heads * (waves == 4 ? v64 : v128);
        if (chains <= 256 || chains > 1e6) continue;
        const double us = walk_us(waves == 4 ? 256 : 1e9, waves == 4 ? 1e9 : 256, false, false,
                                  nullptr);
        for (size_t n = 2; n <= 16 && n <= L; ++n) {
            const size_t p = (L + n - 1) / n;
            if ((L + p - 1) / p != n) continue;
            const size_t rounds = ((size_t)chains * n + 255) / 256;
            const double t = rounds * (chunk * p * us + 7.0);
            if (t < best) {
                best = t;
                cut = {p, (int)n, (int)rounds, waves};
            }
        }
    }
    return cut;
}
size_t delta_segs(const fftconv_delta_desc* d, size_t per) {
    const size_t nch = (d->T + kChunk - 1) / kChunk;
    if (d->sequences) return d->T / (kChunk * per) + d->sequences;
    return d->B * (nch ? (nch + per - 1) / per : 1);
}

// Bytes of the buffers of a call, each a multiple of 16.
struct DeltaLayout {
    Cut cut;
    size_t pack, seg_n, seg_m;      // forward workspace
    size_t bpack, states, us;       // saved
    size_t workspace() const { return pack + seg_n + seg_m; }
    size_t saved() const { return bpack + states + us; }
    // dstates, dys and the segments
    size_t backward() const { return states + us + seg_n + seg_m; }
};
// What the walks' launches follow from.
void delta_geometry(const fftconv_delta_desc* d, const Cut& c, DeltaParams& p) {
    p.Dk = (int)d->Dk;
    p.Dv = (int)d->Dv;
    p.Hv = (int)d->Hv;
    p.packed = d->sequences != 0;
    p.nseq = (long long)(d->sequences ? d->sequences : d->B);
    p.seg_chunks = (int)c.per;
    p.segs = (long long)delta_segs(d, c.per);
    p.pieces = c.pieces;
    p.rounds = c.rounds;
    p.waves = c.waves;
}
bool delta_layout(const fftconv_delta_desc* d, DeltaLayout* l) {
    size_t n, x, y, m;
    const Cut c = delta_cut(d);
    const size_t per = c.per;
    l->cut = c;
    if (!product(delta_slots(d), d->Hv, 1, 1, &n) || n > kMaxGrid) return false;
    // saved matrices: rows for the largest magnitudes, columns padded to 16
    const size_t cols = (d->Dv + 15) / 16 * 16, rows = d->Dk <= 64 ? 64 : 128;
    if (!product(n, rows + 2, cols, 1, &x) || !product(n, kChunk + 2, cols, 1, &y)) return false;
    const bool cut = per <= (d->T + kChunk - 1) / kChunk;
    const size_t segs = delta_segs(d, per);
    if (!product(segs, d->Hv, (d->Dv + d->Dk + 15) / 16, 1, &m) || m > kMaxGrid) return false;
    l->pack = n * (size_t)delta_pack_uint4() * 16;
    // pieces: one state a chain, which each of them takes over from the last
    const size_t held = c.pieces > 1 ? (d->sequences ? d->sequences : d->B) : segs;
    l->seg_n = cut ? held * d->Hv * d->Dk * d->Dv * 4 : 0;
    l->seg_m = cut && c.pieces == 1 ? segs * d->Hv * d->Dk * d->Dk * 4 : 0;
    l->bpack = n * (size_t)delta_pack_uint4() * 16;
    l->states = x * 4;
    l->us = y * 4;
    DeltaParams p = DeltaParams();
    delta_geometry(d, c, p);
    return walk_grid(p, false).fits() && (!l->seg_m || walk_grid(p, true).fits());
}

struct DeltaArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    const long long* cu;
    const float* init;
};

// Checks what both directions read and fills the kernels' parameters.
fftconv_status delta_inputs(const fftconv_delta_desc* d, const DeltaArgs& a, DeltaParams& p,
                            Range (&in)[7]) {
    CHECK(delta_sizes(d));
    size_t qb, kb, vb;
    CHECK(span_bytes(d->B, d->T, d->Hk, d->Dk, d->q_stride, d->dtype, &qb));
    CHECK(span_bytes(d->B, d->T, d->Hk, d->Dk, d->k_stride, d->dtype, &kb));
    CHECK(span_bytes(d->B, d->T, d->Hv, d->Dv, d->v_stride, d->dtype, &vb));
    // the kernels' byte offsets within 64 tokens are 32-bit numbers
    const size_t far = kMaxTokenStride;
    if (d->T > 1 && ((size_t)d->q_stride[1] >= far || (size_t)d->k_stride[1] >= far ||
                     (size_t)d->v_stride[1] >= far))
        return FFTCONV_ERR_UNSUPPORTED;
    if (d->Hv * d->Dv >= far) return FFTCONV_ERR_UNSUPPORTED;
    const size_t gates = d->B * d->T * d->Hv * 4;
    const size_t rows = d->sequences ? d->sequences : d->B;
    const size_t state = rows * d->Hv * d->Dk * d->Dv * 4;
    CHECK(check_ptr(a.q, qb));
    CHECK(check_ptr(a.k, kb));
    CHECK(check_ptr(a.v, vb));
    CHECK(check_ptr(a.g, gates));
    CHECK(check_ptr(a.beta, gates));
    CHECK(check_ptr(a.init, state, false));
    if (d->sequences ? !a.cu : a.cu != nullptr) return FFTCONV_ERR_INVALID_ARG;
    if ((uintptr_t)a.cu & 7) return FFTCONV_ERR_ALIGNMENT;
    in[0] = {a.q, qb};
    in[1] = {a.k, kb};
    in[2] = {a.v, vb};
    in[3] = {a.g, gates};
    in[4] = {a.beta, gates};
    in[5] = {a.init, state};
    in[6] = {a.cu, a.cu ? (d->sequences + 1) * 8 : 0};
    p = DeltaParams();
    p.Hk = (int)d->Hk;
    p.Hv = (int)d->Hv;
    p.group = (int)(d->Hv / d->Hk);
    p.Dk = (int)d->Dk;
    p.Dv = (int)d->Dv;
    p.scale = d->scale;
    p.T = (long long)d->T;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = d->q_stride[i];
        p.ks[i] = d->k_stride[i];
        p.vs[i] = d->v_stride[i];
    }
    p.cu = a.cu;
    p.nseq = (long long)rows;
    p.nch = (long long)((d->T + kChunk - 1) / kChunk);
    p.slots = (long long)delta_slots(d);
    p.q = a.q;
    p.k = a.k;
    p.v = a.v;
    p.g = a.g;
    p.beta = a.beta;
    p.init = a.init;
    if (rows * d->Hv * ((d->Dv + 15) / 16) > kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    return FFTCONV_OK;
}

void delta_place_segments(const fftconv_delta_desc* d, const DeltaLayout& l, char* at,
                          DeltaParams& p) {
    delta_geometry(d, l.cut, p);
    if (l.seg_n) p.seg_n = (float*)at;
    if (l.seg_m) p.seg_m = (float*)(at + l.seg_n);
}
void delta_place_saved(const DeltaLayout& l, void* saved, DeltaParams& p) {
    char* f = (char*)saved;
    p.bpack = (uint4*)f;
    p.states = (float*)(f + l.bpack);
    p.us = (float*)(f + l.bpack + l.states);
}

}  // namespace

extern "C" {

fftconv_status fftconv_qknorm_forward(const fftconv_qknorm_desc* d, const void* q, const void* k,
                                      const float* q_weight, const float* k_weight,
                                      const float* cos, const float* sin,
                                      const long long* positions, void* q_out, void* k_out,
                                      void* stream) {
    QkNormParams p;
    Range in[7];
    CHECK(qknorm_inputs(d, {q, k, q_weight, k_weight, cos, sin, positions}, p, in));
    const size_t qn = d->B * d->T * d->Hq * d->D * elem(d->dtype);
    const size_t kn = d->B * d->T * d->Hk * d->D * elem(d->dtype);
    CHECK(check_ptr(q_out, qn));
    CHECK(check_ptr(k_out, kn));
    const Range out[] = {{q_out, qn}, {k_out, kn}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (!(qn + kn)) return FFTCONV_OK;
    p.qo = q_out;
    p.ko = k_out;
    return launched(launch_qknorm_fwd(d->dtype, p, (hipStream_t)stream));
}

size_t fftconv_qknorm_workspace_bytes(const fftconv_qknorm_desc* d) {
    if (qknorm_sizes(d) != FFTCONV_OK) return 0;
    return (size_t)qknorm_bwd_blocks((long long)(d->B * d->T)) * 2 * d->D * 4;
}

fftconv_status fftconv_qknorm_backward(const fftconv_qknorm_desc* d, const void* q, const void* k,
                                       const float* q_weight, const float* k_weight,
                                       const float* cos, const float* sin,
                                       const long long* positions, const void* dq_out,
                                       const void* dk_out, void* dq, void* dk, float* dq_weight,
                                       float* dk_weight, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    QkNormParams p;
    Range in[7];
    CHECK(qknorm_inputs(d, {q, k, q_weight, k_weight, cos, sin, positions}, p, in));
    const size_t qn = d->B * d->T * d->Hq * d->D * elem(d->dtype);
    const size_t kn = d->B * d->T * d->Hk * d->D * elem(d->dtype);
    CHECK(check_ptr(dq_out, qn));
    CHECK(check_ptr(dk_out, kn));
    CHECK(check_ptr(dq, qn));
    CHECK(check_ptr(dk, kn));
    CHECK(check_ptr(dq_weight, 0, false));
    CHECK(check_ptr(dk_weight, 0, false));
    const size_t need = dq_weight || dk_weight ? fftconv_qknorm_workspace_bytes(d) : 0;
    if (need) {
        if (!workspace || workspace_bytes < need) return FFTCONV_ERR_WORKSPACE;
        if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    }
    const Range more[] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], {dq_out, qn},
                          {dk_out, kn}};
    const Range out[] = {{dq, qn}, {dk, kn}, {dq_weight, d->D * 4}, {dk_weight, d->D * 4},
                         {workspace, need}};
    if (!outputs_clear(out, more)) return FFTCONV_ERR_INVALID_ARG;
    if (!(qn + kn)) {
        if (!need) return FFTCONV_OK;
        p.tokens = 0;      // no heads: the weights' gradients are 0, no token is read
    }
    p.dqo = dq_out;
    p.dko = dk_out;
    p.dq = dq;
    p.dk = dk;
    p.part = need ? (float*)workspace : nullptr;
    p.dwq = dq_weight;
    p.dwk = dk_weight;
    p.blocks = qknorm_bwd_blocks(p.tokens);
    return launched(launch_qknorm_bwd(d->dtype, p, (hipStream_t)stream));
}

size_t fftconv_delta_workspace_bytes(const fftconv_delta_desc* d) {
    DeltaLayout l;
    if (delta_sizes(d) != FFTCONV_OK || !delta_layout(d, &l)) return 0;
    return l.workspace();
}

size_t fftconv_delta_saved_bytes(const fftconv_delta_desc* d) {
    DeltaLayout l;
    if (delta_sizes(d) != FFTCONV_OK || !delta_layout(d, &l)) return 0;
    return l.saved();
}

fftconv_status fftconv_delta_forward(const fftconv_delta_desc* d, const void* q, const void* k,
                                     const void* v, const float* g, const float* beta,
                                     const long long* cu_seqlens, const float* initial_state,
                                     void* o, float* final_state, void* saved, size_t saved_bytes,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    DeltaParams p;
    Range in[7];
    CHECK(delta_inputs(d, {q, k, v, g, beta, cu_seqlens, initial_state}, p, in));
    DeltaLayout l;
    if (!delta_layout(d, &l)) return FFTCONV_ERR_UNSUPPORTED;
    const size_t on = d->B * d->T * d->Hv * d->Dv * elem(d->dtype);
    const size_t state = (size_t)p.nseq * d->Hv * d->Dk * d->Dv * 4;
    const size_t need = l.workspace(), keep = saved ? l.saved() : 0;
    CHECK(check_ptr(o, on));
    CHECK(check_ptr(final_state, state, false));
    CHECK(check_ptr(saved, keep, false));
    if (saved_bytes < keep) return FFTCONV_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    const Range out[] = {{o, on}, {final_state, state}, {saved, keep}, {workspace, need}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (!p.nseq) return FFTCONV_OK;
    p.o = o;
    p.fin = final_state;
    p.pack = (uint4*)workspace;
    p.clear = d->clear_unheld != 0;
    if (keep) delta_place_saved(l, saved, p);
    delta_place_segments(d, l, (char*)workspace + l.pack, p);
    hipStream_t s = (hipStream_t)stream;
    if (d->B * d->T) CHECK(launched(launch_delta_prep(d->dtype, p, s)));
    return launched(launch_delta_scan(d->dtype, p, s));
}

size_t fftconv_delta_backward_workspace_bytes(const fftconv_delta_desc* d) {
    DeltaLayout l;
    if (delta_sizes(d) != FFTCONV_OK || !delta_layout(d, &l)) return 0;
    return l.backward();
}

fftconv_status fftconv_delta_backward(const fftconv_delta_desc* d, const void* q, const void* k,
                                      const void* v, const float* g, const float* beta,
                                      const long long* cu_seqlens, const void* saved,
                                      size_t saved_bytes, const void* d_o,
                                      const float* d_final_state, void* dq, void* dk, void* dv,
                                      float* dg, float* dbeta, float* d_initial_state,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    DeltaGradParams p = DeltaGradParams();
    Range in[7];
    CHECK(delta_inputs(d, {q, k, v, g, beta, cu_seqlens, nullptr}, p.f, in));
    DeltaLayout l;
    if (!delta_layout(d, &l)) return FFTCONV_ERR_UNSUPPORTED;
    const size_t n = d->B * d->T, e = elem(d->dtype);
    const size_t on = n * d->Hv * d->Dv * e, kn = n * d->Hk * d->Dk * e, gn = n * d->Hv * 4;
    const size_t state = (size_t)p.f.nseq * d->Hv * d->Dk * d->Dv * 4;
    CHECK(check_ptr(d_o, on));
    CHECK(check_ptr(d_final_state, state, false));
    CHECK(check_ptr(dq, kn));
    CHECK(check_ptr(dk, kn));
    CHECK(check_ptr(dv, on));
    CHECK(check_ptr(dg, gn));
    CHECK(check_ptr(dbeta, gn));
    CHECK(check_ptr(d_initial_state, state, false));
    CHECK(check_ptr(saved, l.saved()));
    if (saved_bytes < l.saved()) return FFTCONV_ERR_INVALID_ARG;
    const size_t need = l.backward();
    if (need && (!workspace || workspace_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    in[5] = {saved, l.saved()};
    const Range more[] = {in[0], in[1], in[2], in[3], in[4], in[5], in[6], {d_o, on},
                          {d_final_state, state}};
    const Range out[] = {{dq, kn}, {dk, kn}, {dv, on}, {dg, gn}, {dbeta, gn},
                         {d_initial_state, state}, {workspace, need}};
    if (!outputs_clear(out, more)) return FFTCONV_ERR_INVALID_ARG;
    if (!p.f.nseq) return FFTCONV_OK;
    delta_place_saved(l, (void*)saved, p.f);     // only read here
    p.dout = d_o;
    p.dfin = d_final_state;
    p.dstates = (float*)workspace;
    p.dys = (float*)((char*)workspace + l.states);
    delta_place_segments(d, l, (char*)workspace + l.states + l.us, p.f);
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dg = dg;
    p.dbeta = dbeta;
    p.dinit = d_initial_state;
    hipStream_t s = (hipStream_t)stream;
    CHECK(launched(launch_delta_rscan(d->dtype, p, s)));
    return n ? launched(launch_delta_grads(d->dtype, p, s)) : FFTCONV_OK;
}

fftconv_status fftconv_delta_step(const fftconv_delta_desc* d, const void* q, const void* k,
                                  const void* v, const float* g, const float* beta, float* state,
                                  size_t pool, const long long* slots, void* o, void* stream) {
    DeltaParams c;
    Range in[7];
    if (d && (d->T != 1 || d->sequences)) return FFTCONV_ERR_INVALID_ARG;
    CHECK(delta_inputs(d, {q, k, v, g, beta, nullptr, nullptr}, c, in));
    size_t n;
    if (pool > kMaxCount || !product(pool, d->Hv, d->Dk, d->Dv, &n))
        return FFTCONV_ERR_UNSUPPORTED;
    const size_t on = d->B * d->Hv * d->Dv * elem(d->dtype);
    if (!d->B) return FFTCONV_OK;
    CHECK(check_ptr(state, n * 4));
    CHECK(check_ptr(o, on));
    if ((uintptr_t)slots & 7) return FFTCONV_ERR_ALIGNMENT;
    if (!slots && pool < d->B) return FFTCONV_ERR_INVALID_ARG;
    in[6] = {slots, slots ? d->B * 8 : 0};
    const Range out[] = {{o, on}, {state, n * 4}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (d->B * d->Hv * ((d->Dv + 31) / 32) > kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    DeltaStepParams p = DeltaStepParams();
    p.N = (int)d->B;
    p.Hk = c.Hk;
    p.Hv = c.Hv;
    p.Dk = c.Dk;
    p.Dv = c.Dv;
    p.scale = c.scale;
    p.pool = (long long)pool;
    p.qs[0] = c.qs[0]; p.qs[1] = c.qs[2];
    p.ks[0] = c.ks[0]; p.ks[1] = c.ks[2];
    p.vs[0] = c.vs[0]; p.vs[1] = c.vs[2];
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.state = state;
    p.slots = slots;
    p.o = o;
    return launched(launch_delta_step(d->dtype, p, (hipStream_t)stream));
}

}  // extern "C"
