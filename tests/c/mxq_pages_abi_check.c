/* mxq_pages_abi_check.c -- a C11 caller of the calls for long and shared contexts of
 * include/mxq.h: each through the header's own prototypes and types, on paths that the
 * library answers on the host before anything is enqueued (empty calls, argument errors,
 * the size queries).  The device addresses are fake and never dereferenced; the program is
 * run where no GPU is visible.  Exit status: the number of failed checks. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mxq.h"

static int failures = 0;

#define CHECK(cond)                                                                      \
    do {                                                                                 \
        if (!(cond)) {                                                                   \
            fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond);     \
            ++failures;                                                                  \
        }                                                                                \
    } while (0)

/* A 256-byte aligned address that no buffer holds. */
#define DEV(T) ((T*)(uintptr_t)(1u << 20))
#define DEV_OFF(T, off) ((T*)(uintptr_t)((1u << 20) + (off)))

static mxq_nvfp4_kv cache_of(void) {
    mxq_nvfp4_kv c;
    c.k_codes = c.k_scales = c.v_codes = c.v_scales = DEV(uint8_t);
    c.k_global = c.v_global = DEV(const float);
    c.num_pages = 10;
    c.page_size = 16;
    c.kv_heads = 2;
    c.head_dim = 128;
    c.code_stride_token = 64;
    c.code_stride_head = 16 * 64;
    c.code_stride_page = 2 * 16 * 64;
    c.scale_stride_token = 8;
    c.scale_stride_head = 16 * 8;
    c.scale_stride_page = 2 * 16 * 8;
    return c;
}

static mxq_page_keys keys_of(void) {
    mxq_page_keys k;
    k.codes = DEV(int8_t);
    k.scales = DEV(float);
    k.num_pages = 10;
    k.page_size = 16;
    k.kv_heads = 2;
    k.head_dim = 128;
    return k;
}

static mxq_status prefix(const mxq_nvfp4_kv* c, int64_t total_q, int64_t groups, int64_t max_prefix, void* workspace,
                         size_t bytes) {
    return mxq_attention_prefix_nvfp4(DEV(const uint16_t), 4096, 8, total_q, DEV(uint16_t), 4096, NULL, c,
                                      DEV(const int32_t), 100, 100, DEV(const int32_t), DEV(const int32_t), 4,
                                      DEV(const int32_t), DEV(const int32_t), groups, 1, max_prefix, 100, 0.125f,
                                      workspace, bytes, NULL);
}

static mxq_status select_pages(const mxq_page_keys* k, int64_t total_q, int64_t max_len, int32_t top, int32_t first,
                               int32_t last, void* workspace, size_t bytes) {
    return mxq_select_pages_nvfp4(DEV(const uint16_t), 4096, 8, total_q, k, DEV(const int32_t), 5000, 5000,
                                  DEV(const int32_t), DEV(const int32_t), 1, max_len, top, first, last, DEV(int32_t),
                                  workspace, bytes, NULL);
}

static mxq_status attend(const mxq_nvfp4_kv* c, int64_t total_q, int32_t top, float scale, void* workspace, size_t bytes) {
    return mxq_attention_pages_nvfp4(DEV(const uint16_t), 4096, 8, total_q, DEV(uint16_t), 4096, NULL, c,
                                     DEV(const int32_t), 100, 100, DEV(const int32_t), DEV(const int32_t), 1,
                                     DEV(const int32_t), top, scale, workspace, bytes, NULL);
}

int main(void) {
    const mxq_nvfp4_kv cache = cache_of();
    const mxq_page_keys keys = keys_of();
    mxq_page_keys other = keys;
    size_t need;

    CHECK(mxq_page_keys_nvfp4(&cache, NULL, 0, &keys, NULL) == MXQ_OK);
    CHECK(mxq_page_keys_nvfp4(&cache, NULL, 1, &keys, NULL) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(mxq_page_keys_nvfp4(&cache, DEV_OFF(const int64_t, 4), 1, &keys, NULL) == MXQ_ERR_MISALIGNED);
    other.num_pages = 11;
    CHECK(mxq_page_keys_nvfp4(&cache, DEV(const int64_t), 1, &other, NULL) == MXQ_ERR_INVALID_ARGUMENT);
    other = keys;
    other.codes = DEV_OFF(int8_t, 8);
    CHECK(mxq_page_keys_nvfp4(&cache, DEV(const int64_t), 1, &other, NULL) == MXQ_ERR_MISALIGNED);

    /* one query's many candidates are scored by more work-groups, few are not */
    need = mxq_select_pages_nvfp4_workspace_size(8, 2, 16, 1, 1, 65536);
    CHECK(need > 0 && need % 256 == 0);
    CHECK(mxq_select_pages_nvfp4_workspace_size(8, 2, 16, 1, 1, 64) == 0);
    CHECK(select_pages(&keys, 0, 65536, 8, 1, 2, NULL, 0) == MXQ_OK);
    CHECK(select_pages(&keys, 1, 65536, 8, 1, 0, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(select_pages(&keys, 1, 65536, 8, 6, 3, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(select_pages(&keys, 1, 65536, 8, 1, 2, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(select_pages(&keys, 1, 65536, 8, 1, 2, DEV(void), need - 1) == MXQ_ERR_WORKSPACE_TOO_SMALL);
    CHECK(select_pages(&keys, 1, 65536, 8, 1, 2, DEV_OFF(void, 16), need) == MXQ_ERR_MISALIGNED);
    CHECK(select_pages(NULL, 1, 65536, 8, 1, 2, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);

    need = mxq_attention_pages_nvfp4_workspace_size(8, 2, 128, 16, 1, 64);
    CHECK(need > 0 && need % 256 == 0);
    CHECK(mxq_attention_pages_nvfp4_workspace_size(8, 2, 128, 16, 1, 4) == 0);
    CHECK(mxq_attention_pages_nvfp4_workspace_size(8, 3, 128, 16, 1, 64) == 0);
    CHECK(attend(&cache, 0, 64, 0.125f, NULL, 0) == MXQ_OK);
    CHECK(attend(&cache, 1, 0, 0.125f, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&cache, 1, 64, NAN, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&cache, 1, 64, 0.125f, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&cache, 1, 64, 0.125f, DEV(void), need - 1) == MXQ_ERR_WORKSPACE_TOO_SMALL);
    CHECK(attend(&cache, 1, 64, 0.125f, DEV_OFF(void, 16), need) == MXQ_ERR_MISALIGNED);
    CHECK(attend(NULL, 1, 64, 0.125f, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);

    need = mxq_attention_prefix_nvfp4_workspace_size(8, 2, 128, 4, 2, 4, 1, 1000, 100);
    CHECK(need > 0 && need % 256 == 0);
    CHECK(mxq_attention_prefix_nvfp4_workspace_size(8, 2, 128, 4, 0, 4, 1, 1000, 100) == 0);
    CHECK(prefix(&cache, 0, 2, 1000, NULL, 0) == MXQ_OK);
    CHECK(prefix(&cache, 4, 0, 1000, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(prefix(&cache, 4, 2, -1, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(prefix(&cache, 4, 2, 1000, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(prefix(&cache, 4, 2, 1000, DEV(void), need - 1) == MXQ_ERR_WORKSPACE_TOO_SMALL);
    CHECK(prefix(&cache, 4, 2, 1000, DEV_OFF(void, 16), need) == MXQ_ERR_MISALIGNED);
    CHECK(prefix(NULL, 4, 2, 1000, DEV(void), need) == MXQ_ERR_INVALID_ARGUMENT);

    if (failures == 0) printf("all checks passed\n");
    return failures;
}
