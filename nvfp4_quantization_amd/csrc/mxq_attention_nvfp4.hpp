// mxq_attention_nvfp4.hpp -- what the attention kernels share (gfx950): sequences and the
// tiles of tokens that a set of query rows sees, dequantization into FP16 operands, one
// softmax step, and how finished rows are stored.
#pragma once

#include "mxq_device.hpp"
#include "mxq_serve.hpp"

namespace mxq {

namespace {

typedef _Float16 f16;
typedef f16 f16x2 __attribute__((ext_vector_type(2)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

constexpr float kFloor = -0x1.fffffep+127f;     // the running maximum before any score (finite: no inf - inf)
constexpr float kBias = 9.0f;         // weights are 2^(s - m + kBias): at most 2^(kSlack + kBias) = 2^14
constexpr float kSlack = 5.0f;        // how far scores may exceed m before it is raised

// ---------------------------------------------------------------- sequences and tiles
struct Seq {
    int len;                          // cached tokens that may be read
    int start;                        // first query row
    int nq;                           // queries (their positions end at len - 1)
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
    Seq s;
    const int64_t cap = min((int64_t)a.table_pages << a.c.page_shift, (int64_t)0x7FFFFF00);
    s.len = (int)min((int64_t)max(a.seq_lens[b], 0), cap);
    const int64_t q0 = min(max(a.q_starts[b], 0), a.total_q), q1 = min(max(a.q_starts[b + 1], 0), a.total_q);
    s.start = (int)q0;
    s.nq = (int)max(q1 - q0, (int64_t)0);
    return s;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);       // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true);       // lane 15 of the row before, rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, true);       // lane 31, rows 2 and 3
    return v;
}

// The sequence, the position and the place in its run of one query (b = -1: a row of no
// sequence), searched by a whole wave, 64 sequences a step.
struct Query {
    int b, pos, index;
    int len, left;                    // the sequence's length; queries of its run from this one on
};
template <typename Args>
__device__ __forceinline__ Query query_of(const Args& a, int page_shift, int row) {
    const int lane = (int)threadIdx.x & 63;
    // A query a sequence, or one sequence, is usual: that place is looked at beside the first
    // step's (a memory latency less where it is right).
    const int guess = min(row, a.batch - 1);
    int lo = 0, n = a.batch, s0 = a.q_starts[guess], s1 = a.q_starts[guess + 1], held = a.seq_lens[guess];
    int start = a.q_starts[min(lane * ((n + 63) >> 6), n)];
    if (row < s0 || row >= s1) {
        for (int step = 64; step > 1;) {                     // the last one that starts at or before row
            step = (n + 63) >> 6;
            if (n < a.batch) start = a.q_starts[min(lo + lane * step, a.batch)];
            const int k = __popcll(__ballot(lane * step < n && start <= row));
            if (k == 0) return Query{-1, -1, 0, 0, 0};
            lo += (k - 1) * step;
            n = min(step, n - (k - 1) * step);
        }
        s0 = a.q_starts[lo], s1 = a.q_starts[lo + 1], held = a.seq_lens[lo];
    } else {
        lo = guess;
    }
    const int64_t q0 = min(max(s0, 0), a.total_q), q1 = min(max(s1, 0), a.total_q);
    if (row < q0 || row >= q1) return Query{-1, -1, 0, 0, 0};
    const int64_t cap = min((int64_t)a.table_pages << page_shift, (int64_t)0x7FFFFF00);
    const int64_t len = min((int64_t)max(held, 0), cap);
    Query r;
    r.b = __builtin_amdgcn_readfirstlane(lo);
    r.pos = __builtin_amdgcn_readfirstlane((int)max(len - (q1 - row), (int64_t)-1));
    r.index = __builtin_amdgcn_readfirstlane((int)(row - q0));
    r.len = __builtin_amdgcn_readfirstlane((int)len);
    r.left = __builtin_amdgcn_readfirstlane((int)(q1 - row));
    return r;
}

// The 64-token tiles that queries q_first .. q_last of a sequence see: with a window the
// tiles of the first `sinks` tokens, then those from the first query's window on.
struct Span {
    int head;                         // tiles 0 .. head - 1, then
    int body;                         // tile body and following ones
    int n;                            // tiles in all
    int p_lo, p_hi;                   // positions of the first and last query (>= -1)
    __device__ __forceinline__ int tile(int i) const { return i < head ? i : body + (i - head); }
};
__device__ __forceinline__ Span tile_span(const AttnArgs& a, const Seq& s, int q_first, int q_last) {
    Span r;
    r.p_lo = max(s.len - s.nq + q_first, -1);
    r.p_hi = max(s.len - s.nq + q_last, -1);
    const int end = (int)(((int64_t)r.p_hi + 64) >> 6);                  // ceil((p_hi + 1) / 64)
    const int64_t from = a.window ? max((int64_t)r.p_lo - a.window + 1, (int64_t)0) : 0;
    r.body = (int)(from >> 6);
    r.head = a.window ? (int)min((min((int64_t)a.sinks, from) + 63) >> 6, (int64_t)r.body) : 0;
    r.n = r.head + max(end - r.body, 0);
    return r;
}
__device__ __forceinline__ int splits_used(const AttnArgs& a, int tiles) {
    return max(min((tiles + a.chunk - 1) / a.chunk, a.splits), 1);
}

// The query at position p sees token t (p < t: never; window and sinks are >= 0).
__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int t) {
    return t <= p && (!a.window || t > p - a.window || t < a.sinks);
}

// keep(e, seen) for N of a lane's tokens, token t0 + at(e), for the query at position p: sees()
// in vector instructions (unsigned: tokens ahead of the query wrap to far behind it).
template <int N, typename At, typename Keep>
__device__ __forceinline__ void each_seen(const AttnArgs& a, int p, int t0, At&& at, Keep&& keep) {
    constexpr uint32_t kAll = 0x80000000u;
    const uint32_t window = a.window ? (uint32_t)a.window : kAll;
    int ago = p - t0, first = a.sinks - t0;
    asm("" : "+v"(ago), "+v"(first));                        // (or p - at(e) is held for every e across the tiles)
#pragma unroll
    for (int e = 0; e < N; ++e) keep(e, (uint32_t)(ago - at(e)) < (at(e) < first ? kAll : window));
}

// ---------------------------------------------------------------- FP16 operands
// 8 E2M1 codes of a dword.
__device__ __forceinline__ f16x8 e2m1_8(uint32_t w) {
    const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
    const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
    const f16x2 c = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
    const f16x2 d = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// Two E4M3 codes (the low or the high half of w) as FP16 (exact; NaN stays NaN).
__device__ __forceinline__ f16x2 e4m3_pair(uint32_t w, bool high) {
    return high ? __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))
                : __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
}
// D / 4 elements of a K row (D / 32 dwords) with their D / 64 block scales.
template <int D>
using KWords = uint32_t __attribute__((ext_vector_type(D / 32)));
template <int D>
__device__ __forceinline__ void dequant_row(KWords<D> w, uint32_t scales, f16x8 (&k)[D / 32]) {
    const f16x2 s = e4m3_pair(scales, false);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const f16 f = (D == 128 && c >= 2) ? s.y : s.x;
        k[c] = e2m1_8(w[c]) * f16x8{f, f, f, f, f, f, f, f};
    }
}
// Q's power of two from the BF16 bits of its row's largest magnitude: returns 2^(14 - e) for a
// largest element in [2^e, 2^(e + 1)), and its inverse.  e is held to [-100, 127], where
// both are normal; a row below 2^-100 only uses fewer bits, an infinite one stays infinite.
__device__ __forceinline__ float q_power(uint32_t top, float& inverse) {
    const int e = min(max((int)(top >> 7) - 127, -100), 127);
    inverse = __builtin_bit_cast(float, (uint32_t)(e - 14 + 127) << 23);
    return __builtin_bit_cast(float, (uint32_t)(14 - e + 127) << 23);
}
// The factor on a row's scores: in binary64, since two of the three may leave binary32's range
// where their product with the third does not.  Kept normal and finite: a masked score is -inf,
// and times zero (queries of zeros under a small tensor scale) it would be NaN.  A factor raised
// to 2^-126 stands for scores below 2^-90.
__device__ __forceinline__ float score_factor(const AttnArgs& a, float inverse, float kg) {
    return __builtin_fminf(__builtin_fmaxf((float)(inverse * (kg * a.scale_log2)), 0x1p-126f), 0x1.fffffep+127f);
}
__device__ __forceinline__ f16x8 q_operand(const u32x4v& w, float up) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = (f16)(lo_bf16(p[i]) * up);
        r[2 * i + 1] = (f16)(hi_bf16(p[i]) * up);
    }
    return r;
}

// A byte of w is an E4M3 NaN (0x7F or 0xFF).
__device__ __forceinline__ bool has_nan_scale(uint32_t w) {
    return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// ---------------------------------------------------------------- softmax
// A row's maximum after a tile whose largest score is top (over all of the row's lanes).  By the
// row itself, though the wave raises all its rows at once: another row's scores, which may be of
// tokens that this one does not see, must not change a bit of it.
__device__ __forceinline__ float raise(float m, float top) { return top > m + kSlack ? top : m; }

// Weights are 2^fma(x, factor, kBias - m): one rounding, of a small number, but m itself is a
// rounded product, and from 2^24 on its rounding alone (all of a row's weights times 2 and more)
// would leave FP16's range.  There the rounded product is taken for every score, as it was for
// m: weights of a row with far() are 2^(fl(x factor) - m + kBias), the difference formed in place
// of x.  (The floor and infinities stay out.)  The test costs a tile of heads of 64 1.5 to 2 %.
__device__ __forceinline__ bool far(float m) {
    constexpr uint32_t kNear = 0x4A800000u;                              // 2^22
    return (__builtin_bit_cast(uint32_t, m) & 0x7FFFFFFFu) - kNear < 0x7F7FFFFFu - kNear;
}

// One step of 64 tokens for 16 query rows: raw scores x (lane column = row, 16 tokens a
// lane) to FP16 weights p, with the row's maximum, its lane's share of the sum and, when
// the maximum is raised, the outputs.  factor > 0 turns raw scores into base-2 exponents.
// The four lanes of a row always hold the same m.
template <int D>
__device__ __forceinline__ void softmax_step(f32x4 (&x)[4], float factor, float& m, float& l, f32x4 (&o)[D / 16],
                                             f16x8 (&p)[2]) {
    float top = x[0][0];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __builtin_fmaxf(top, x[t][e]);
    top *= factor;
    if (__any(top > m + kSlack)) {
        top = __builtin_fmaxf(top, shfl_xor_f32(top, 16));
        top = __builtin_fmaxf(top, shfl_xor_f32(top, 32));
        const float raised = raise(m, top);
        const float f = __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) o[dt] *= f;
    }
    float shift = kBias - m;
    if (__builtin_expect(__any(far(m)), 0)) {
        const bool is_far = far(m);
        const float by = is_far ? factor : 1.0f, less = is_far ? m : 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = x[t][e] * by - less;
        factor = is_far ? 1.0f : factor;
        shift = is_far ? kBias : shift;
    }
    float part[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][e], factor, shift));
        part[t] = (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const f32x2 pair = {w[e], w[e + 1]};
            const f16x2 h = __builtin_convertvector(pair, f16x2);
            p[t >> 1][4 * (t & 1) + e] = h.x;
            p[t >> 1][4 * (t & 1) + e + 1] = h.y;
        }
    }
    l += (part[0] + part[1]) + (part[2] + part[3]);
}

// ---------------------------------------------------------------- results
// Natural logarithm of the sum of exponentials of a row with maximum m (base 2) and biased sum.
__device__ __forceinline__ float row_lse(float m, float sum) {
    return sum == 0.0f ? -__builtin_inff() : ((m - kBias) + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

// Four elements d0 .. d0 + 3 of row r of a sequence's rows of one cached head, finished (o:
// unnormalized) ...
template <int D>
__device__ __forceinline__ void store_finished(const AttnArgs& a, const Seq& seq, int kvh, int64_t r, int d0, const f32x4& o,
                                               float m, float sum, float vg) {
    const int qi = (int)(r / a.group), head = kvh * a.group + (int)(r - (int64_t)qi * a.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;       // (vg / sum could leave the normal range)
    uint16_t* dst = a.out + (int64_t)(seq.start + qi) * a.ld_out + (int64_t)head * D + d0;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0] * inv * vg, o[1] * inv * vg), pack_bf16(o[2] * inv * vg, o[3] * inv * vg));
    if (a.lse && d0 == 0) a.lse[(int64_t)(seq.start + qi) * a.q_heads + head] = row_lse(m, sum);
}
// ... or as one part of it, in row `at` of the workspace.
template <int D>
__device__ __forceinline__ void store_part(const AttnArgs& a, int64_t at, int d0, const f32x4& o, float m, float sum) {
    *reinterpret_cast<f32x4*>(a.part_o + at * D + d0) = o;
    if (d0 == 0) a.part_ml[at] = make_float2(m, sum);
}

}  // namespace

}  // namespace mxq
