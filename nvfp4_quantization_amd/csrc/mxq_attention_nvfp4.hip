// mxq_attention_nvfp4.hip -- causal attention over the paged NVFP4 cache (gfx950).
//
// The plain form: one wave per (query, head), 64 cached tokens a step.  Lane i forms the
// score of token i of the step; the running maximum and sum of the softmax are kept in
// FP32, and the wave then holds 1 (head_dim 64) or 2 output elements per lane.
#include "mxq_device.hpp"
#include "mxq_serve.hpp"

namespace mxq {

namespace {

__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * (float)m : __builtin_bit_cast(float, (126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return (c & 8u) ? -v : v;
}

// The page of token t (-1: none that may be read).
__device__ __forceinline__ int64_t page_of(const AttnArgs& a, int b, int t) {
    const int i = t >> a.c.page_shift;
    if (i >= a.table_pages) return -1;
    const int32_t p = a.table[(int64_t)b * a.ld_table + i];
    return p >= 0 && p < a.c.num_pages ? p : -1;
}

}  // namespace

template <int D>
__global__ __launch_bounds__(64) void k_attention_plain(const AttnArgs a) {
    const int lane = (int)threadIdx.x;
    const int64_t item = blockIdx.x;
    const int qi = (int)(item / a.q_heads), head = (int)(item % a.q_heads), kvh = head / a.group;
    // the sequence of query qi
    int b = -1, start = 0, end = 0;
    for (int i = 0; i < a.batch; ++i) {
        const int s = a.q_starts[i], e = a.q_starts[i + 1];
        if (qi >= s && qi < e) b = i, start = s, end = e;
    }
    if (b < 0 || qi - start >= a.max_q_len) return;
    const int64_t cap = (int64_t)a.table_pages << a.c.page_shift;
    int64_t len64 = a.seq_lens[b];
    len64 = len64 < 0 ? 0 : len64 > cap ? cap : len64;
    const int len = (int)(len64 > 0x7FFFFF00ll ? 0x7FFFFF00ll : len64);
    const int pos = len - (end - start) + (qi - start);
    const uint16_t* q = a.q + qi * a.ld_q + (int64_t)head * D;
    const float kg = a.c.kg[kvh], vg = a.c.vg[kvh];
    float m = -1e30f, l = 0.0f, o[D / 64] = {};
    for (int t0 = 0; t0 <= pos; t0 += 64) {
        if (a.window && t0 >= a.sinks && t0 + 63 <= pos - a.window) continue;
        const int t = t0 + lane;
        const bool see = t <= pos && (!a.window || t > pos - a.window || t < a.sinks);
        float x = -__builtin_inff();
        int64_t page = -1;
        if (see) {
            page = page_of(a, b, t);
            x = __builtin_nanf("");
            if (page >= 0) {
                const int64_t off = t & ((1 << a.c.page_shift) - 1);
                const uint8_t* kc = a.c.kc + page * a.c.cs_page + kvh * a.c.cs_head + off * a.c.cs_tok;
                const uint8_t* ks = a.c.ks + page * a.c.ss_page + kvh * a.c.ss_head + off * a.c.ss_tok;
                float acc = 0.0f;
                for (int g = 0; g < D / 16; ++g) {
                    float part = 0.0f;
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = kc[g * 8 + i];
                        const uint32_t qq = *reinterpret_cast<const uint32_t*>(q + g * 16 + 2 * i);
                        part += e2m1_value(w) * lo_bf16(qq);
                        part += e2m1_value(w >> 4) * hi_bf16(qq);
                    }
                    acc += part * e4m3_value(ks[g]);
                }
                x = acc * kg * a.scale_log2;
            }
        }
        float top = x;
        for (int i = 1; i < 64; i <<= 1) top = __builtin_fmaxf(top, shfl_xor_f32(top, i));
        const float m1 = __builtin_fmaxf(m, top);
        const float keep = __builtin_amdgcn_exp2f(m - m1);
        const float p = see ? __builtin_amdgcn_exp2f(x - m1) : 0.0f;
        m = m1;
        l = l * keep + p;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) o[j] *= keep;
        for (int i = 0; i < 64; ++i) {
            const float pi = __shfl(p, i, 64);
            const int64_t pg = __shfl(page, i, 64);
            if (pi == 0.0f || pg < 0) continue;                    // (uniform) unseen, or a NaN score in l
            const int64_t off = (t0 + i) & ((1 << a.c.page_shift) - 1);
            const uint8_t* vc = a.c.vc + pg * a.c.cs_page + kvh * a.c.cs_head + off * a.c.cs_tok;
            const uint8_t* vs = a.c.vs + pg * a.c.ss_page + kvh * a.c.ss_head + off * a.c.ss_tok;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const int d = lane + 64 * j;
                const uint32_t c = vc[d >> 1] >> (4 * (d & 1));
                o[j] += pi * (e2m1_value(c) * e4m3_value(vs[d >> 4]));
            }
        }
    }
    for (int i = 1; i < 64; i <<= 1) l += shfl_xor_f32(l, i);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
        const float v = l == 0.0f ? 0.0f : o[j] * vg / l;
        a.out[qi * a.ld_out + (int64_t)head * D + lane + 64 * j] = (uint16_t)(pack_bf16(v, v) & 0xFFFFu);
    }
    if (a.lse && lane == 0)
        a.lse[item] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
}

hipError_t launch_attention_nvfp4(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.total_q * a.q_heads));
    if (a.c.head_dim == 128)
        hipLaunchKernelGGL(k_attention_plain<128>, grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL(k_attention_plain<64>, grid, dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
