// mxq_pages.hip -- which pages of the paged NVFP4 cache a query attends (gfx950): the mean
// key of every page that an append has filled, in 8-bit integers, and the selection of the
// pages whose mean keys score highest.
//
// Mean keys.  E2M1 times E4M3 is a whole multiple of 2^-10 of at most 2688, so a page's sum
// of them is a whole number below 2^31 (up to 512 tokens): formed exactly, in FP32 while four
// tokens add up (below 2^24), in 32-bit integers from there on, whatever the order.  The codes
// are then the nearest whole numbers of S * 127 / max |S|: in binary64 the quotient is a
// half only where it is one exactly.
//
// Scores.  Products of 8-bit integers in 32 bits (v_mfma_i32_16x16x64_i8: 16 query rows by 16
// pages, 64 elements each), then two stated FP32 products; so the selection is the same
// whatever the order of the work.
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- mean keys
// One page of one head, by a wave: D / 32 lanes hold a token's 32 codes each.
template <int D>
__device__ __forceinline__ void page_key(const PageKeysArgs& a, int page, int head, int lane) {
    constexpr int kLanes = D / 32, kStep = 64 / kLanes;     // lanes of a token, tokens of a load
    const int size = 1 << a.c.page_shift;
    const uint8_t* const codes = a.c.kc + page * a.c.cs_page + head * a.c.cs_head + 16 * (lane % kLanes);
    const uint8_t* const scales = a.c.ks + page * a.c.ss_page + head * a.c.ss_head + 2 * (lane % kLanes);
    const float g = a.c.kg[head];
    int sum[32] = {};
    bool bad = false;
    for (int t0 = 0; t0 < size; t0 += 4 * kStep) {
        u32x4v w[4];
        uint32_t s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = min(t0 + kStep * i + lane / kLanes, size - 1);
            w[i] = *reinterpret_cast<const u32x4v*>(codes + t * a.c.cs_tok);
            s[i] = *reinterpret_cast<const uint16_t*>(scales + t * a.c.ss_tok);
        }
        float part[32] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = t0 + kStep * i + lane / kLanes < size;
            bad |= (((s[i] & 0x7F7Fu) + 0x0101u) & 0x8080u) != 0;
            const f16x2 f = e4m3_pair(in ? s[i] : 0u, false);
            const uint32_t p[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const f16x8 e = e2m1_8(p[c]);
                const f16 by = c < 2 ? f.x : f.y;
#pragma unroll
                for (int j = 0; j < 8; ++j) part[8 * c + j] = __builtin_fmaf((float)e[j], (float)by, part[8 * c + j]);
            }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) sum[e] += (int)(part[e] * 1024.0f);
    }
    // over the lanes of the same elements, half of the elements handed over at each step
    int first = 32 * (lane % kLanes);
#pragma unroll
    for (int bit = 32, n = 16; bit >= kLanes; bit >>= 1, n >>= 1) {
        const bool upper = lane & bit;
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const int mine = upper ? sum[e + n] : sum[e], other = upper ? sum[e] : sum[e + n];
            sum[e] = mine + __shfl_xor(other, bit, 64);
        }
        first += upper ? n : 0;
    }
    constexpr int kMine = D / 64;
    int top = 0;
#pragma unroll
    for (int e = 0; e < kMine; ++e) top = max(top, abs(sum[e]));
#pragma unroll
    for (int bit = 1; bit < 64; bit <<= 1) top = max(top, __shfl_xor(top, bit, 64));
    bad = __any(bad);
    const int64_t at = (int64_t)page * a.c.kv_heads + head;
    uint32_t out = 0;
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
        const int code = bad || top == 0 ? 0 : (int)__builtin_rint((double)sum[e] * 127.0 / (double)top);
        out |= ((uint32_t)code & 0xFFu) << (8 * e);
    }
    if constexpr (kMine == 2)
        *reinterpret_cast<uint16_t*>(a.codes + at * D + first) = (uint16_t)out;
    else
        a.codes[at * D + first] = (int8_t)out;
    if (lane == 0) a.scales[at] = bad ? __builtin_nanf("") : (float)((double)top * (double)g * (1.0 / (130048.0 * size)));
}

}  // namespace

// A wave per `chunk` slots and head: the pages whose last row is among them.
template <int D>
__global__ __launch_bounds__(256) void k_page_keys(const PageKeysArgs a) {
    const int lane = (int)threadIdx.x & 63;
    const int64_t item = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t first = item / a.c.kv_heads * a.chunk;
    const int head = (int)(item % a.c.kv_heads);
    if (first >= a.tokens) return;
    const int64_t slot = lane < a.chunk && first + lane < a.tokens ? a.slots[first + lane] : -1;
    const int64_t last_row = ((int64_t)1 << a.c.page_shift) - 1;
    const bool full = slot >= 0 && (slot & last_row) == last_row && (slot >> a.c.page_shift) < a.c.num_pages;
    const int page = (int)(slot >> a.c.page_shift);
    for (uint64_t todo = __ballot(full); todo; todo &= todo - 1)
        page_key<D>(a, __builtin_amdgcn_readlane(page, __builtin_ctzll(todo)), head, lane);
}

hipError_t launch_page_keys(const PageKeysArgs& a, hipStream_t stream) {
    const int64_t waves = (a.tokens + a.chunk - 1) / a.chunk * a.c.kv_heads;
    const dim3 grid((unsigned)((waves + 3) / 4));
    if (a.c.head_dim == 128)
        hipLaunchKernelGGL(k_page_keys<128>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(k_page_keys<64>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- selection
namespace {

// A score as a whole number of the same order; NaN below all.
__device__ __forceinline__ uint32_t order_of(float score) {
    const uint32_t u = __builtin_bit_cast(uint32_t, score + 0.0f);       // (-0 is 0)
    return score != score ? 0u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

// Sum over the work-group of a value per wave.
__device__ __forceinline__ int wave_counts(int count, int wave, int* shared) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[wave] = count;
    __syncthreads();
    return (shared[0] + shared[1]) + (shared[2] + shared[3]);
}

}  // namespace

// A work-group per (query, cached head).  The scores of `window` candidates at a time are held
// in LDS, as order_of(); where a query has more, every pass forms them again.
template <int D>
__global__ __launch_bounds__(256) void k_select_pages(const SelectArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ int counts[4];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int token = (int)(blockIdx.x / (unsigned)a.kv_heads), kvh = (int)(blockIdx.x % (unsigned)a.kv_heads);
    const Query at = query_of(a, a.page_shift, token);
    if (at.b < 0) return;
    int32_t* const out = a.out + ((int64_t)token * a.kv_heads + kvh) * a.top;
    const int current = at.pos < 0 ? -1 : at.pos >> a.page_shift;
    if (current < a.top) {                                   // all there are
        for (int i = tid; i < a.top; i += 256) out[i] = i <= current ? i : -1;
        return;
    }
    for (int i = tid; i < a.first; i += 256) out[i] = i;
    for (int i = tid; i < a.last; i += 256) out[a.top - a.last + i] = current - a.last + 1 + i;
    const int n = current + 1 - a.first - a.last, wanted = a.top - a.first - a.last;
    if (wanted == 0) return;                                 // (n > wanted)
    const int32_t* const table = a.table + (int64_t)at.b * a.ld_table + a.first;

    // scores of the candidates w0 .. w1 - 1: 16 pages a wave and step
    const auto score = [&](int w0, int w1) {
        __syncthreads();
        for (int r0 = 0; r0 < a.group; r0 += 16) {
            // 16 query rows (the last again past the group) as 8-bit integers
            const int row = min(r0 + col, a.group - 1);
            const uint16_t* const src = a.q + (int64_t)token * a.ld_q + (int64_t)(kvh * a.group + row) * D + 16 * g;
            u32x4v w[D / 32];
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                w[c] = *reinterpret_cast<const u32x4v*>(src + 64 * (c >> 1) + 8 * (c & 1));
                top = absmax_pk(absmax_pk(absmax_pk(absmax_pk(top, w[c].x), w[c].y), w[c].z), w[c].w);
            }
            top = fold_pk(top);
            top = max(top, shfl_xor_u32(top, 16));
            top = max(top, shfl_xor_u32(top, 32));
            const float step = top >= 0x7F80u ? 0.0f : bf16_mag(top) * (1.0f / 127.0f);
            i32x4 q[D / 64];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                const uint32_t p[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t word = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = e & 1 ? hi_bf16(p[2 * i + (e >> 1)]) : lo_bf16(p[2 * i + (e >> 1)]);
                        const float y = step > 0.0f ? __builtin_rintf(x / step) : 0.0f;
                        word |= ((uint32_t)(int)__builtin_fminf(__builtin_fmaxf(y, -127.0f), 127.0f) & 0xFFu) << (8 * e);
                    }
                    q[c >> 1][2 * (c & 1) + i] = (int)word;
                }
            }
            float by[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) by[e] = __shfl(step, 4 * g + e, 64);
            for (int j0 = w0 + 16 * wave; j0 < w1; j0 += 64) {
                const int j = min(j0 + col, w1 - 1);
                const int32_t entry = table[j];
                const bool ok = (uint32_t)entry < (uint32_t)a.num_pages;
                const int64_t page = (ok ? (int64_t)entry : 0) * a.kv_heads + kvh;
                i32x4 k[D / 64], x = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 64; ++c) k[c] = *reinterpret_cast<const i32x4*>(a.codes + page * D + 64 * c + 16 * g);
                const float scale = a.scales[page];
#pragma unroll
                for (int c = 0; c < D / 64; ++c) x = __builtin_amdgcn_mfma_i32_16x16x64_i8(q[c], k[c], x, 0, 0, 0);
                float best = (float)x[0] * by[0];
#pragma unroll
                for (int e = 1; e < 4; ++e) best = __builtin_fmaxf(best, (float)x[e] * by[e]);
                best = __builtin_fmaxf(best, shfl_xor_f32(best, 16));
                best = __builtin_fmaxf(best, shfl_xor_f32(best, 32));
                if (g == 0 && j0 + col < w1) {
                    if (r0 > 0) best = __builtin_fmaxf(best, __builtin_bit_cast(float, keys[j - w0]));
                    const bool last = r0 + 16 >= a.group;
                    keys[j - w0] = !last ? __builtin_bit_cast(uint32_t, best) : ok ? order_of(best * scale) : 0u;
                }
            }
        }
        __syncthreads();
    };
    const bool once = n <= a.window;
    if (once) score(0, n);
    // visit(candidate or -1, its key), all threads together, in candidates' order
    const auto each = [&](auto&& visit) {
        for (int w0 = 0; w0 < n; w0 += a.window) {
            const int w1 = min(w0 + a.window, n);
            if (!once) score(w0, w1);
            for (int j = w0; j < w1; j += 256) {
                const bool in = j + tid < w1;
                visit(in ? j + tid : -1, in ? keys[j + tid - w0] : 0u);
            }
        }
    };
    // the wanted-th largest key, bit by bit; or any that exactly `wanted` reach
    uint32_t least = 0;
    int ties = wanted;                                       // of keys equal to it
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t t = least | 1u << bit;
        int count = 0;
        each([&](int j, uint32_t key) { count += __popcll(__ballot(j >= 0 && key >= t)); });
        count = wave_counts(count, wave, counts);
        if (count >= wanted) least = t;
        if (count == wanted) break;
    }
    {
        int above = 0;
        each([&](int j, uint32_t key) { above += __popcll(__ballot(j >= 0 && key > least)); });
        ties = wanted - wave_counts(above, wave, counts);
    }
    // them, in order
    int done = 0, equal = 0;                                 // written so far; of them ties
    __shared__ int2 sums[4];
    each([&](int j, uint32_t key) {
        const uint64_t up = __ballot(j >= 0 && key > least), tie = __ballot(j >= 0 && key == least);
        __syncthreads();
        if (lane == 0) sums[wave] = make_int2(__popcll(up), __popcll(tie));
        __syncthreads();
        int ups = 0, before = equal, all_ups = 0, all_ties = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) ups += sums[w].x, before += sums[w].y;
            all_ups += sums[w].x, all_ties += sums[w].y;
        }
        const uint64_t below = (1ull << lane) - 1;
        const int my_ups = ups + __popcll(up & below), my_ties = before + __popcll(tie & below);
        // written before this one: every key above and the first ties
        const int place = done + my_ups + min(my_ties, ties);
        if ((up >> lane & 1) || ((tie >> lane & 1) && my_ties < ties)) out[a.first + place] = a.first + j;
        done += all_ups;
        equal += all_ties;
    });
}

hipError_t launch_select_pages(const SelectArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.total_q * a.kv_heads));
    const unsigned bytes = (unsigned)a.window * 4;
    if (a.head_dim == 128)
        hipLaunchKernelGGL(k_select_pages<128>, grid, dim3(256), bytes, stream, a);
    else
        hipLaunchKernelGGL(k_select_pages<64>, grid, dim3(256), bytes, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
