// Host side of linear attention with a decay for each head and of layer norm:
// argument checks, buffer layouts and the C ABI declared in include/fftconv.h.
#include <stdint.h>

#include "../../include/fftconv.h"
#include "fftconv_decay.h"
#include "fftconv_mixer_host.h"

using namespace fftconv;

namespace {

// ------------------------------------------------------------- layer norm

fftconv_status layernorm_sizes(const fftconv_layernorm_desc* d) {
    if (!d) return FFTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return FFTCONV_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f)) return FFTCONV_ERR_INVALID_ARG;
    if (!d->D) return FFTCONV_ERR_INVALID_ARG;
    if (d->D > 16384 || d->rows > kMaxCount) return FFTCONV_ERR_UNSUPPORTED;
    if (d->rows > 1 && (d->x_stride < (long long)d->D || (size_t)d->x_stride > kMaxElems / d->rows))
        return FFTCONV_ERR_INVALID_ARG;
    return FFTCONV_OK;
}

fftconv_status layernorm_inputs(const fftconv_layernorm_desc* d, const void* x, const float* w,
                                const float* b, LayerNormParams& p, Range (&in)[3]) {
    CHECK(layernorm_sizes(d));
    const size_t e = elem(d->dtype);
    const size_t xb = d->rows ? ((d->rows - 1) * (size_t)(d->rows > 1 ? d->x_stride : 0) + d->D) * e : 0;
    CHECK(check_ptr(x, xb));
    CHECK(check_ptr(w, 0, false));
    CHECK(check_ptr(b, 0, false));
    in[0] = {x, xb};
    in[1] = {w, d->D * 4};
    in[2] = {b, d->D * 4};
    p = LayerNormParams();
    p.rows = (long long)d->rows;
    p.D = (int)d->D;
    p.eps = d->eps;
    p.stride = d->rows > 1 ? d->x_stride : (long long)d->D;
    p.wide = d->D % 8 == 0 && p.stride % (16 / (long long)e) == 0;
    p.x = x;
    p.w = w;
    p.b = b;
    return FFTCONV_OK;
}

// ------------------------------------------- linear attention with decays

fftconv_status decay_sizes(const fftconv_decay_desc* d) {
    if (!d) return FFTCONV_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return FFTCONV_ERR_UNSUPPORTED;
    if (!d->Dk || d->Dk % 8 || d->Dk > 256 || !d->Dv || d->Dv % 8 || d->Dv > 1024)
        return FFTCONV_ERR_UNSUPPORTED;
    if (!d->Hk || !d->Hv || d->Hv % d->Hk) return FFTCONV_ERR_INVALID_ARG;
    if (d->Hv > 65536 || d->B > kMaxCount || d->T > kMaxCount - 64 || d->sequences > kMaxCount)
        return FFTCONV_ERR_UNSUPPORTED;
    if (d->sequences && d->B != 1) return FFTCONV_ERR_INVALID_ARG;
    size_t n;
    if (!product(d->B, d->T, d->Hv, d->Dv, &n) || !product(d->B, d->T, d->Hv, d->Dk, &n))
        return FFTCONV_ERR_UNSUPPORTED;
    const size_t rows = d->sequences ? d->sequences : d->B;
    if (!product(rows, d->Hv, d->Dk, d->Dv, &n)) return FFTCONV_ERR_UNSUPPORTED;
    // units of a launch, and of one that goes over states
    if (n / 1024 > kMaxGrid || rows * d->Hv * 8 > kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    return FFTCONV_OK;
}

// Tokens of a segment.  A sequence is a chain of chunks; where the heads and columns
// leave CUs idle, sequences are cut into segments that are walked side by side: once
// for their effects on the state, and, after a join, for the outputs.  The length is
// the one of least time by the model below, a whole sequence where that is least.
//
// Measured, bf16 and heads of 128, whole, as chosen and the best of ten lengths from 64
// tokens on: 4 x 32768 tokens of 4 heads 2545, 310 and 292 us; 16 x 8192 of 6, 623, 406
// and 405; 1 x 4096 of 8, 310, 49 and 50; 16 x 1024 of 6, 84, 84 (whole) and 71; with
// gradients 8 x 2048 of 4, 687, 243 and 238.  23 packed sequences of 9001 tokens, 8 heads
// of 64 x 128 in f16, 102, 65 and 61.  The device alone knows the bounds of packed
// sequences: 16384 tokens in 40 of 6 heads, walked whole, take 57 us where they are of equal
// length and 1254 where one holds nearly all (in segments of 256 tokens 100 and 135).
size_t decay_segment(const fftconv_decay_desc* d) {
    const size_t blocks = (d->T + kSegAlign - 1) / kSegAlign;
    const size_t whole = (blocks + 1) * kSegAlign;
    const size_t rows = d->sequences ? d->sequences : d->B;
    if (!rows || !blocks) return whole;
    // workgroups of the join
    if (rows * d->Hv * ((d->Dk * d->Dv + 255) / 256) > kMaxGrid) return whole;
    const double vs = (double)((d->Dv + kDecayCols - 1) / kDecayCols);
    const double heads = (double)rows * d->Hv * vs;
    // us of 64 tokens in a walk of so many workgroups: the latency of one, or what the
    // CU with the most of them takes; the same for the effects
    const double wide = (d->dtype == FFTCONV_F32 ? 2.0 : 1.0) * (d->Dk > 128 ? 2.0 : d->Dk > 64 ? 1.0 : 0.7);
    const auto time = [&](double units, double one, double each) {
        const double load = units / 256 < 8 ? (double)(size_t)(units / 256 + 0.999) : units / 256;
        return wide * (one > each * load ? one : each * load);
    };
    // packed sequences: some are longer than the average
    const double mean = (double)blocks / (d->sequences ? rows : 1);
    const double longest = d->sequences ? (mean * 3 < blocks ? mean * 3 : (double)blocks) : mean;
    double best = longest * time(heads, 4.3, 2.75);
    size_t most = whole;
    for (size_t per = 1, step = 1; per < blocks && per < longest; per += step) {
        while (step * 16 <= per) step *= 2;
        const double n = (double)(size_t)(longest / per + 0.999);
        const double all = heads * (d->sequences ? mean / per + 0.5 : n);
        if (n > 256) continue;
        // those of the walks
        const size_t segs = d->sequences ? blocks / per + rows : rows * ((blocks + per - 1) / per);
        if (segs * d->Hv * 32 > kMaxGrid) continue;
        // two more launches, the join's steps, states made, joined and read at 5 TB/s
        const double states = all / vs * d->Dk * d->Dv * 16 / 5e6;
        const double t = per * (time(all, 4.3, 2.75) + time(all, 2.3, 1.45)) + 14.0 + 0.3 * n + states;
        if (t < best) {
            best = t;
            most = per * kSegAlign;
        }
    }
    return most;
}

struct DecayLayout {
    size_t L, per, segs;          // tokens of a segment; segments of a sequence, in all
    size_t seg, seg_g;            // bytes
    // backward: parts of dg by columns of dk and of dv, of the last states, of
    // chunks, of workgroups; dq and dk of the value heads where they share heads
    size_t before, behind, ends, before_all, chunks, anchors, anchor_dg, sums, shared, slots, anchor_count;
    size_t forward() const { return seg + seg_g; }
    size_t backward() const {
        return 2 * seg + seg_g + before + behind + ends + before_all + chunks + anchors + anchor_dg +
               sums + 2 * shared;
    }
};
size_t up16(size_t n) { return (n + 15) / 16 * 16; }
bool decay_layout(const fftconv_decay_desc* d, DecayLayout* l) {
    l->L = decay_segment(d);
    l->per = (d->T + l->L - 1) / l->L;
    if (!l->per) l->per = 1;
    l->segs = d->sequences ? d->T / l->L + d->sequences : d->B * l->per;
    const bool cut = l->L < d->T;
    size_t n;
    if (!product(l->segs, d->Hv, d->Dk, d->Dv, &n) || !product(l->segs, d->Hv, 32, 1, &n) ||
        n > kMaxGrid)
        return false;
    l->seg = cut ? l->segs * d->Hv * d->Dk * d->Dv * 4 : 0;
    l->seg_g = cut ? up16(l->segs * d->Hv * 8) : 0;
    const size_t tokens = d->B * d->T, rows = d->sequences ? d->sequences : d->B;
    const size_t C = kDecayChunk;
    // parts by columns, of Dk and of Dv
    const size_t ks = (d->Dk + kDecayCols - 1) / kDecayCols, vs = (d->Dv + kDecayCols - 1) / kDecayCols;
    l->slots = d->sequences ? d->T / C + d->sequences : d->B * ((d->T + C - 1) / C);
    l->before = up16(ks * d->Hv * tokens * 4);
    l->behind = up16(vs * d->Hv * tokens * 4);
    l->ends = up16(rows * d->Hv * ks * 4 * 8);
    l->before_all = up16(ks * l->slots * d->Hv * 8);
    l->chunks = up16(vs * l->slots * d->Hv * 16);
    const size_t anchors = decay_anchors(d->T, rows, d->sequences != 0,
                                         C << decay_anchor_shift(d->fixed_decay != 0));
    l->anchors = anchors * d->Hv * decay_anchor_floats((int)d->Dk, (int)d->Dv) * 4;
    l->anchor_dg = up16(ks * anchors * d->Hv * 8);
    l->anchor_count = anchors;
    l->sums = d->fixed_decay ? up16(decay_dg_units(d->T, rows, d->sequences != 0) * d->Hv * 8) : 0;
    l->shared = d->Hv > d->Hk ? up16(tokens * d->Hv * d->Dk * 4) : 0;
    return true;
}

struct DecayArgs {
    const void *q, *k, *v;
    const float* g;
    const long long* cu;
    const float* init;
};

// Checks what both directions read and fills the kernels' parameters.
fftconv_status decay_inputs(const fftconv_decay_desc* d, const DecayArgs& a, const DecayLayout& l,
                            DecayParams& p, Range (&in)[6]) {
    size_t qb, kb, vb;
    CHECK(span_bytes(d->B, d->T, d->Hk, d->Dk, d->q_stride, d->dtype, &qb));
    CHECK(span_bytes(d->B, d->T, d->Hk, d->Dk, d->k_stride, d->dtype, &kb));
    CHECK(span_bytes(d->B, d->T, d->Hv, d->Dv, d->v_stride, d->dtype, &vb));
    // the kernels' byte offsets within a chunk are 32-bit numbers
    const size_t far = kMaxTokenStride;
    if (d->T > 1 && ((size_t)d->q_stride[1] >= far || (size_t)d->k_stride[1] >= far ||
                     (size_t)d->v_stride[1] >= far))
        return FFTCONV_ERR_UNSUPPORTED;
    if (d->Hv * d->Dv >= far || d->Hv * d->Dk >= far) return FFTCONV_ERR_UNSUPPORTED;
    const size_t gates = (d->fixed_decay ? 1 : d->B * d->T) * d->Hv * 4;
    const size_t rows = d->sequences ? d->sequences : d->B;
    const size_t state = rows * d->Hv * d->Dk * d->Dv * 4;
    CHECK(check_ptr(a.q, qb));
    CHECK(check_ptr(a.k, kb));
    CHECK(check_ptr(a.v, vb));
    CHECK(check_ptr(a.g, gates));
    CHECK(check_ptr(a.init, state, false));
    if (d->sequences ? !a.cu : a.cu != nullptr) return FFTCONV_ERR_INVALID_ARG;
    if ((uintptr_t)a.cu & 7) return FFTCONV_ERR_ALIGNMENT;
    in[0] = {a.q, qb};
    in[1] = {a.k, kb};
    in[2] = {a.v, vb};
    in[3] = {a.g, gates};
    in[4] = {a.init, state};
    in[5] = {a.cu, a.cu ? (d->sequences + 1) * 8 : 0};
    p = DecayParams();
    p.sp.T = (long long)d->T;
    p.sp.nseq = (long long)rows;
    p.sp.segs = (long long)l.segs;
    p.sp.seg_tokens = (int)l.L;
    p.sp.per = (int)l.per;
    p.sp.cu = a.cu;
    p.Hv = (int)d->Hv;
    p.Dk = (int)d->Dk;
    p.Dv = (int)d->Dv;
    p.scale = d->scale;
    p.fixed = d->fixed_decay != 0;
    p.clear = d->clear_unheld != 0;
    const int group = (int)(d->Hv / d->Hk);
    p.q = {a.q, {d->q_stride[0], d->q_stride[1], d->q_stride[2]}, group};
    p.k = {a.k, {d->k_stride[0], d->k_stride[1], d->k_stride[2]}, group};
    p.v = {a.v, {d->v_stride[0], d->v_stride[1], d->v_stride[2]}, 1};
    p.g = a.g;
    p.init = a.init;
    return FFTCONV_OK;
}

}  // namespace

extern "C" {

fftconv_status fftconv_layernorm_forward(const fftconv_layernorm_desc* d, const void* x,
                                         const float* weight, const float* bias, void* y,
                                         void* stream) {
    LayerNormParams p;
    Range in[3];
    CHECK(layernorm_inputs(d, x, weight, bias, p, in));
    const size_t n = d->rows * d->D * elem(d->dtype);
    CHECK(check_ptr(y, n));
    const Range out[] = {{y, n}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (!n) return FFTCONV_OK;
    p.y = y;
    return launched(launch_layernorm_fwd(d->dtype, p, (hipStream_t)stream));
}

size_t fftconv_layernorm_workspace_bytes(const fftconv_layernorm_desc* d) {
    if (layernorm_sizes(d) != FFTCONV_OK) return 0;
    return (size_t)layernorm_bwd_blocks((long long)d->rows, (int)d->D) * 2 * d->D * 4;
}

fftconv_status fftconv_layernorm_backward(const fftconv_layernorm_desc* d, const void* x,
                                          const float* weight, const void* dy, void* dx,
                                          float* dweight, float* dbias, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    LayerNormParams p;
    Range in[3];
    CHECK(layernorm_inputs(d, x, weight, nullptr, p, in));
    const size_t n = d->rows * d->D * elem(d->dtype);
    CHECK(check_ptr(dy, n));
    CHECK(check_ptr(dx, n));
    CHECK(check_ptr(dweight, 0, false));
    CHECK(check_ptr(dbias, 0, false));
    const size_t need = dweight || dbias ? fftconv_layernorm_workspace_bytes(d) : 0;
    if (need) {
        if (!workspace || workspace_bytes < need) return FFTCONV_ERR_WORKSPACE;
        if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    }
    const Range more[] = {in[0], in[1], {dy, n}};
    const Range out[] = {{dx, n}, {dweight, d->D * 4}, {dbias, d->D * 4}, {workspace, need}};
    if (!outputs_clear(out, more)) return FFTCONV_ERR_INVALID_ARG;
    if (!n && !need) return FFTCONV_OK;
    p.dy = dy;
    p.dx = dx;
    p.part = need ? (float*)workspace : nullptr;
    p.dw = dweight;
    p.db = dbias;
    p.blocks = layernorm_bwd_blocks(p.rows, p.D);
    return launched(launch_layernorm_bwd(d->dtype, p, (hipStream_t)stream));
}

size_t fftconv_decay_workspace_bytes(const fftconv_decay_desc* d) {
    DecayLayout l;
    if (decay_sizes(d) != FFTCONV_OK || !decay_layout(d, &l)) return 0;
    return l.forward();
}

fftconv_status fftconv_decay_forward(const fftconv_decay_desc* d, const void* q, const void* k,
                                     const void* v, const float* g, const long long* cu_seqlens,
                                     const float* initial_state, void* o, float* final_state,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    DecayParams p;
    DecayLayout l;
    Range in[6];
    CHECK(decay_sizes(d));
    if (!decay_layout(d, &l)) return FFTCONV_ERR_UNSUPPORTED;
    CHECK(decay_inputs(d, {q, k, v, g, cu_seqlens, initial_state}, l, p, in));
    const size_t on = d->B * d->T * d->Hv * d->Dv * elem(d->dtype);
    const size_t state = (size_t)p.sp.nseq * d->Hv * d->Dk * d->Dv * 4;
    const size_t need = l.forward();
    CHECK(check_ptr(o, on));
    CHECK(check_ptr(final_state, state, false));
    if (need && (!workspace || workspace_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    const Range out[] = {{o, on}, {final_state, state}, {workspace, need}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (!p.sp.nseq) return FFTCONV_OK;
    p.o = o;
    p.fin = final_state;
    if (l.seg) {
        p.seg = (float*)workspace;
        p.seg_g = (double*)((char*)workspace + l.seg);
    }
    return launched(launch_decay_fwd(d->dtype, p, (hipStream_t)stream));
}

size_t fftconv_decay_backward_workspace_bytes(const fftconv_decay_desc* d) {
    DecayLayout l;
    if (decay_sizes(d) != FFTCONV_OK || d->Dv > 256 || !decay_layout(d, &l)) return 0;
    return l.backward();
}

fftconv_status fftconv_decay_backward(const fftconv_decay_desc* d, const void* q, const void* k,
                                      const void* v, const float* g, const long long* cu_seqlens,
                                      const float* initial_state, const void* d_o,
                                      const float* d_final_state, void* dq, void* dk, void* dv,
                                      float* dg, float* d_initial_state, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    DecayGradParams p = DecayGradParams();
    DecayLayout l;
    Range in[6];
    CHECK(decay_sizes(d));
    if (d->Dv > 256 || !decay_layout(d, &l)) return FFTCONV_ERR_UNSUPPORTED;
    CHECK(decay_inputs(d, {q, k, v, g, cu_seqlens, initial_state}, l, p.f, in));
    const size_t n = d->B * d->T, e = elem(d->dtype);
    if (l.shared && n * d->Hk * d->Dk / 1024 >= kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    const size_t on = n * d->Hv * d->Dv * e, kn = n * d->Hk * d->Dk * e;
    const size_t gn = (d->fixed_decay ? 1 : n) * d->Hv * 4;
    const size_t state = (size_t)p.f.sp.nseq * d->Hv * d->Dk * d->Dv * 4;
    CHECK(check_ptr(d_o, on));
    CHECK(check_ptr(d_final_state, state, false));
    CHECK(check_ptr(dq, kn));
    CHECK(check_ptr(dk, kn));
    CHECK(check_ptr(dv, on));
    CHECK(check_ptr(dg, gn));
    CHECK(check_ptr(d_initial_state, state, false));
    const size_t need = l.backward();
    if (need && (!workspace || workspace_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15) return FFTCONV_ERR_ALIGNMENT;
    const Range more[] = {in[0], in[1], in[2], in[3], in[4], in[5], {d_o, on},
                          {d_final_state, state}};
    const Range out[] = {{dq, kn}, {dk, kn}, {dv, on}, {dg, gn}, {d_initial_state, state},
                         {workspace, need}};
    if (!outputs_clear(out, more)) return FFTCONV_ERR_INVALID_ARG;
    if (!p.f.sp.nseq && !d->fixed_decay) return FFTCONV_OK;
    p.B = (long long)d->B;
    p.d_o = {d_o,
             {(long long)(d->T * d->Hv * d->Dv), (long long)(d->Hv * d->Dv), (long long)d->Dv},
             1};
    p.dfin = d_final_state;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.dg = dg;
    p.dinit = d_initial_state;
    char* at = (char*)workspace;
    const auto take = [&](size_t bytes) {
        char* x = at;
        at += bytes;
        return x;
    };
    if (l.seg) {
        p.f.seg = (float*)take(l.seg);
        p.seg_back = (float*)take(l.seg);
        p.f.seg_g = (double*)take(l.seg_g);
    }
    p.before = (float*)take(l.before);
    p.behind = (float*)take(l.behind);
    p.ends = (double*)take(l.ends);
    p.before_all = (double*)take(l.before_all);
    p.chunks = (double2*)take(l.chunks);
    p.slots = (long long)l.slots;
    p.anchor_shift = decay_anchor_shift(p.f.fixed);
    p.anchor_floats = (long long)decay_anchor_floats(p.f.Dk, p.f.Dv);
    p.anchors = (float*)take(l.anchors);
    p.anchor_dg = (double*)take(l.anchor_dg);
    p.anchor_count = (long long)l.anchor_count;
    if (l.sums) p.sums = (double*)take(l.sums);
    if (l.shared) {
        p.dq_heads = (float*)take(l.shared);
        p.dk_heads = (float*)take(l.shared);
    }
    return launched(launch_decay_bwd(d->dtype, p, (hipStream_t)stream));
}

fftconv_status fftconv_decay_step(const fftconv_decay_desc* d, const void* q, const void* k,
                                  const void* v, const float* g, float* state, size_t pool,
                                  const long long* slots, void* o, void* stream) {
    DecayParams c;
    DecayLayout l;
    Range in[6];
    CHECK(decay_sizes(d));
    if (d->T != 1 || d->sequences) return FFTCONV_ERR_INVALID_ARG;
    if (!decay_layout(d, &l)) return FFTCONV_ERR_UNSUPPORTED;
    CHECK(decay_inputs(d, {q, k, v, g, nullptr, nullptr}, l, c, in));
    size_t n;
    if (pool > kMaxCount || !product(pool, d->Hv, d->Dk, d->Dv, &n))
        return FFTCONV_ERR_UNSUPPORTED;
    const size_t on = d->B * d->Hv * d->Dv * elem(d->dtype);
    if (!d->B) return FFTCONV_OK;
    CHECK(check_ptr(state, n * 4));
    CHECK(check_ptr(o, on));
    if ((uintptr_t)slots & 7) return FFTCONV_ERR_ALIGNMENT;
    if (!slots && pool < d->B) return FFTCONV_ERR_INVALID_ARG;
    in[5] = {slots, slots ? d->B * 8 : 0};
    const Range out[] = {{o, on}, {state, n * 4}};
    if (!outputs_clear(out, in)) return FFTCONV_ERR_INVALID_ARG;
    if (d->B * d->Hv * ((d->Dv + 31) / 32) > kMaxGrid) return FFTCONV_ERR_UNSUPPORTED;
    DecayStepParams p = DecayStepParams();
    p.N = (int)d->B;
    p.Hk = (int)d->Hk;
    p.Hv = c.Hv;
    p.Dk = c.Dk;
    p.Dv = c.Dv;
    p.scale = c.scale;
    p.fixed = c.fixed;
    p.pool = (long long)pool;
    p.qs[0] = c.q.st[0]; p.qs[1] = c.q.st[2];
    p.ks[0] = c.k.st[0]; p.ks[1] = c.k.st[2];
    p.vs[0] = c.v.st[0]; p.vs[1] = c.v.st[2];
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.state = state;
    p.slots = slots;
    p.o = o;
    return launched(launch_decay_step(d->dtype, p, (hipStream_t)stream));
}

}  // extern "C"
