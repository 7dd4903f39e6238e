// heads.cuh -- host checks of mxfp4_heads descriptors, shared by the operators on queries, keys and
// values (rotation, attention).
#pragma once

#include <algorithm>
#include <cstdlib>

#include "step_ops.cuh"

namespace mx {

// 3D tensor map over bf16 heads (mxfp4_api.cu): box = 64 elements x box_heads heads x box_tokens tokens,
// 128-byte swizzle.
bool encode_heads_map(CUtensorMap* map, const void* p, int64_t tokens, int64_t heads, int64_t dim, int64_t token_stride,
                      int64_t head_stride, uint32_t box_heads, uint32_t box_tokens);

// A descriptor whose strides have a meaning: that of a single token or head is the row itself.
struct Heads {
    void* data;
    int64_t token_stride, head_stride;  // elements
    int32_t heads, dtype;
};

inline int64_t heads_esize(int dtype) { return dtype == MXFP4_OUT_BF16 ? 2 : 4; }

// Checks `h`, heads of [tokens, heads, dim], and writes it to *out.  `written`: no two of its rows may overlap.
inline mxfp4_status check_heads(const char* what, const char* name, const mxfp4_heads* h, int64_t tokens, int64_t dim,
                                bool written, Heads* out) {
    if (!h) return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
    if (h->heads < 1 || h->heads > 65535)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: %s has %d heads (1 to 65535)", what, name, h->heads);
    if (h->dtype != MXFP4_OUT_F32 && h->dtype != MXFP4_OUT_BF16)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: bad dtype %d of %s", what, h->dtype, name);
    Heads r{h->data, h->token_stride, h->head_stride, h->heads, h->dtype};
    if (tokens <= 1) r.token_stride = 0;
    if (r.heads == 1) r.head_stride = 0;
    if (tokens > 0) {
        if (!r.data) return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s is NULL", what, name);
        if (reinterpret_cast<uintptr_t>(r.data) % heads_esize(r.dtype))
            return record_error(MXFP4_ERR_MISALIGNED, "%s: %s not aligned to its element type", what, name);
    }
    const int64_t most = int64_t(1) << 38;
    if ((tokens > 1 && (r.token_stride < dim || r.token_stride > most)) ||
        (r.heads > 1 && (r.head_stride < dim || r.head_stride > most)))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: a stride of %s is below head_dim or above 2^38", what, name);
    // tokens of heads, or heads of tokens, one behind the other
    if (written && tokens > 1 && r.heads > 1 && r.token_stride < (r.heads - 1) * r.head_stride + dim &&
        r.head_stride < (tokens - 1) * r.token_stride + dim)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: rows of %s overlap", what, name);
    *out = r;
    return MXFP4_OK;
}

// Whether every row starts on a multiple of `bytes`.
inline bool heads_aligned(const Heads& h, int64_t bytes) {
    const int64_t e = heads_esize(h.dtype);
    return reinterpret_cast<uintptr_t>(h.data) % bytes == 0 && h.token_stride * e % bytes == 0 &&
           h.head_stride * e % bytes == 0;
}

// Whether two checked tensors of one type share an element.  Exact where their token strides and their head strides are the
// same (slices of one buffer, a tensor and itself); of others that lie in each other's range only a common start is seen.
inline bool heads_overlap(const Heads& a, int64_t tokens_a, const Heads& b, int64_t tokens_b, int64_t dim) {
    if (tokens_a <= 0 || tokens_b <= 0 || !a.data || !b.data) return false;
    const int64_t size = heads_esize(a.dtype), width = dim * size;
    auto extent = [&](const Heads& h, int64_t tokens) {  // a stride without a meaning is 0
        return ((tokens - 1) * h.token_stride + (h.heads - 1) * h.head_stride) * size + width;
    };
    const int64_t at_a = (int64_t)reinterpret_cast<uintptr_t>(a.data), at_b = (int64_t)reinterpret_cast<uintptr_t>(b.data);
    if (at_a + extent(a, tokens_a) <= at_b || at_b + extent(b, tokens_b) <= at_a) return false;
    const int64_t token = (tokens_a > 1 ? a.token_stride : b.token_stride) * size;
    const int64_t head = (a.heads > 1 ? a.head_stride : b.head_stride) * size;
    if ((tokens_b > 1 && b.token_stride * size != token) || (b.heads > 1 && b.head_stride * size != head)) return at_a == at_b;
    // Row (t, h) of b lies `by` + n * token bytes behind row (t - n, h - m) of a: the n that brings them closest.
    for (int64_t m = 1 - a.heads; m < b.heads; ++m) {
        const int64_t by = at_b - at_a + m * head, low = 1 - tokens_a, high = tokens_b - 1;
        int64_t n = token > 0 ? -by / token : 0;
        for (int64_t i = n - 1; i <= n + 1; ++i)
            if (std::llabs(by + std::min(std::max(i, low), high) * token) < width) return true;
    }
    return false;
}
inline bool same_heads(const Heads& a, const Heads& b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride && a.heads == b.heads;
}

}  // namespace mx
