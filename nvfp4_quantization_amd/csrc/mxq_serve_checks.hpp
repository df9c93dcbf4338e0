// mxq_serve_checks.hpp -- argument checks that the serving calls' host entry points share
// (mxq_serve_api.cpp, mxq_pages_api.cpp).
#pragma once

#include "mxq.h"

#include <hip/hip_runtime_api.h>

#include "mxq_serve.hpp"

namespace {

constexpr int64_t kMaxGridThreads = 0xFFFFFFFFll;    // 1-D grids only; threads per launch < 2^32
constexpr int64_t kMaxRows = (1ll << 31) - 128;
constexpr int64_t kMaxElems = 1ll << 40;
constexpr int64_t kMaxTokenStride = 1ll << 24;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// a * b < lim for a, b >= 0 and lim >= 1, without forming the product.
bool product_below(int64_t a, int64_t b, int64_t lim) { return a == 0 || b <= (lim - 1) / a; }

// A [rows][ld] array whose rows hold len elements spans fewer than kMaxElems.
bool extent_ok(int64_t rows, int64_t ld, int64_t len) {
    return len < kMaxElems && product_below(rows - 1, ld, kMaxElems - len);
}

// The largest index of a [rows][cols] array addressed as r * s_r + c * s_c is below
// kMaxElems (rows, cols >= 1; s_r, s_c >= 0).
bool index2_ok(int64_t rows, int64_t s_r, int64_t cols, int64_t s_c) {
    if (!product_below(rows - 1, s_r, kMaxElems) || !product_below(cols - 1, s_c, kMaxElems)) return false;
    return (rows - 1) * s_r < kMaxElems - (cols - 1) * s_c;
}

// The three strides of a cache array: its last row's first byte is below kMaxElems.
bool index3_ok(int64_t a, int64_t sa, int64_t b, int64_t sb, int64_t c, int64_t sc) {
    if (!index2_ok(a, sa, b, sb) || !product_below(c - 1, sc, kMaxElems)) return false;
    return (a - 1) * sa + (b - 1) * sb < kMaxElems - (c - 1) * sc;
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

mxq_status check_cache(const mxq_nvfp4_kv* c, mxq::KvCache* out) {
    if (!c || c->num_pages < 0 || c->kv_heads < 1 || c->page_size < 1 || c->head_dim < 1)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (!c->k_global || !c->v_global) return MXQ_ERR_INVALID_ARGUMENT;
    if (c->num_pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales))
        return MXQ_ERR_INVALID_ARGUMENT;
    if (c->head_dim != 64 && c->head_dim != 128) return MXQ_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)))
        return MXQ_ERR_UNSUPPORTED;
    if (c->num_pages > kMaxRows) return MXQ_ERR_UNSUPPORTED;
    const int64_t cs[3] = {c->code_stride_page, c->code_stride_head, c->code_stride_token};
    const int64_t ss[3] = {c->scale_stride_page, c->scale_stride_head, c->scale_stride_token};
    for (int i = 0; i < 3; ++i) {
        if (cs[i] < 0 || ss[i] < 0) return MXQ_ERR_INVALID_ARGUMENT;
        if (cs[i] % 16 != 0 || ss[i] % (c->head_dim / 16) != 0) return MXQ_ERR_MISALIGNED;
    }
    // (the kernels address the rows of a 64-token tile with 32-bit offsets)
    if (cs[2] > kMaxTokenStride || ss[2] > kMaxTokenStride) return MXQ_ERR_UNSUPPORTED;
    if (cs[2] < c->head_dim / 2 || ss[2] < c->head_dim / 16) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 8) || !aligned(c->v_scales, 8) ||
        !aligned(c->k_global, 4) || !aligned(c->v_global, 4))
        return MXQ_ERR_MISALIGNED;
    if (c->num_pages > 0 && (!index3_ok(c->num_pages, cs[0], c->kv_heads, cs[1], c->page_size, cs[2]) ||
                             !index3_ok(c->num_pages, ss[0], c->kv_heads, ss[1], c->page_size, ss[2])))
        return MXQ_ERR_UNSUPPORTED;
    int shift = 4;
    while ((1 << shift) < c->page_size) ++shift;
    *out = mxq::KvCache{c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->k_global, c->v_global, c->num_pages,
                        cs[0], cs[1], cs[2], ss[0], ss[1], ss[2], shift, c->kv_heads, c->head_dim};
    return MXQ_OK;
}

}  // namespace
