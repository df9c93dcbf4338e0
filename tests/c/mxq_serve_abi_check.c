/* mxq_serve_abi_check.c -- a C11 caller of the serving calls of include/mxq.h: each is
 * called through the header's own prototypes and types on paths that the library answers
 * on the host before anything is enqueued (empty calls, argument errors, the size query).
 * The device addresses are fake and never dereferenced; the program is run where no GPU is
 * visible.  Exit status: 0 when every check holds, else the number of failed checks. */
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

static mxq_status norm(int64_t m, int64_t n, float eps, uint32_t options) {
    return mxq_add_rmsnorm_quant_fp8(DEV(const uint16_t), n, NULL, 0, NULL, 0, DEV(const uint16_t), eps, m, n, options,
                                     NULL, 0, DEV(uint8_t), n, DEV(float), n / 128, 1, NULL);
}

static mxq_status append(const mxq_rope* rope, const mxq_nvfp4_kv* c, int64_t tokens) {
    return mxq_rope_append_nvfp4(DEV(const uint16_t), 512, 4, DEV(uint16_t), 512, DEV(const uint16_t), 256,
                                 DEV(const uint16_t), 256, tokens, DEV(const int32_t), DEV(const int64_t), rope, c, NULL,
                                 NULL, NULL);
}

static mxq_status attend(const mxq_nvfp4_kv* c, int32_t q_heads, int64_t total_q, int64_t max_len, int32_t window,
                         void* workspace, size_t bytes) {
    return mxq_attention_nvfp4(DEV(const uint16_t), 4096, q_heads, total_q, DEV(uint16_t), 4096, NULL, c,
                               DEV(const int32_t), 100, 100, DEV(const int32_t), DEV(const int32_t), 1, 1, max_len,
                               0.125f, window, 0, workspace, bytes, NULL);
}

int main(void) {
    const mxq_nvfp4_kv good = cache_of();
    mxq_nvfp4_kv bad;
    mxq_rope rope = {DEV(const double), 64, MXQ_ROPE_INTERLEAVED, 1.0};
    size_t need;

    CHECK(norm(0, 7168, 1e-6f, 0) == MXQ_OK);
    CHECK(norm(4, 200, 1e-6f, 0) == MXQ_ERR_MISALIGNED);
    CHECK(norm(4, 7168, NAN, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, 7168, 1e-6f, 0x80000000u) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(norm(4, MXQ_RMSNORM_MAX_N + 128, 1e-6f, 0) == MXQ_ERR_UNSUPPORTED);

    CHECK(append(&rope, &good, 0) == MXQ_OK);
    CHECK(append(NULL, &good, 1) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(append(&rope, NULL, 1) == MXQ_ERR_INVALID_ARGUMENT);
    rope.rot_dim = 40;
    CHECK(append(&rope, &good, 1) == MXQ_ERR_MISALIGNED);
    bad = good;
    bad.page_size = 24;
    rope.rot_dim = 64;
    CHECK(append(&rope, &bad, 1) == MXQ_ERR_UNSUPPORTED);
    bad = good;
    bad.k_scales = DEV_OFF(uint8_t, 4);
    CHECK(append(&rope, &bad, 1) == MXQ_ERR_MISALIGNED);

    /* one sequence of 65536 tokens is cut over the chip, one of 64 is not */
    need = mxq_attention_nvfp4_workspace_size(8, 2, 128, 1, 1, 1, 65536, 0, 0);
    CHECK(need > 0 && need % 256 == 0);
    CHECK(mxq_attention_nvfp4_workspace_size(8, 2, 128, 1, 1, 1, 64, 0, 0) == 0);
    CHECK(mxq_attention_nvfp4_workspace_size(8, 3, 128, 1, 1, 1, 65536, 0, 0) == 0);
    CHECK(attend(&good, 8, 0, 65536, 0, NULL, 0) == MXQ_OK);
    CHECK(attend(&good, 7, 1, 65536, 0, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&good, 8, 1, 65536, -1, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&good, 8, 1, 65536, 0, NULL, 0) == MXQ_ERR_INVALID_ARGUMENT);
    CHECK(attend(&good, 8, 1, 65536, 0, DEV(void), need - 1) == MXQ_ERR_WORKSPACE_TOO_SMALL);
    CHECK(attend(&good, 8, 1, 65536, 0, DEV_OFF(void, 16), need) == MXQ_ERR_MISALIGNED);
    bad = good;
    bad.code_stride_token = 8;
    CHECK(attend(&bad, 8, 1, 65536, 0, DEV(void), need) == MXQ_ERR_MISALIGNED);

    if (failures == 0) printf("all checks passed\n");
    return failures;
}
