// Checks of arguments that the host sides of the token mixers share.
#pragma once

#include <stdint.h>

#include "../../include/fftconv.h"
#include "fftconv_internal.h"

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

}  // namespace
