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
// What bounds it: the vector unit beside memory.  131000 tokens of 8 heads of 128 (77 MB of K) take
// 17.5 us, 4.5 TB/s where a plain read reaches 7.0; a SIMD's vector unit is busy 14 of them (a
// conversion for two codes, an FMA a code, two instructions for each four of those sums to become
// an integer).
//
// Scores.  Products of 8-bit integers in 32 bits (v_mfma_i32_16x16x64_i8: 16 query rows by 16
// pages, 64 elements each), then two stated FP32 products; so the selection is the same
// whatever the order of the work.  A group's best head is found in the registers of its rows, and
// over lanes by swaps of rows of 16 lanes, two scores at a time.
//
// The largest of them: kept in LDS as integers of the same order.  A bound that a few more than
// wanted reach comes from the largest of 64 to 256 columns of them; those few are listed in order
// and one wave finishes with them in registers (64 candidates a pass over LDS until then, two passes
// in all).  Long selections and heaps of equal scores are halved by value instead.
//
// What bounds it: latency, mostly.  One query of 8 cached heads over 2048 pages takes 12.2 us, in two
// launches (4 and 8): lengths, page numbers, keys and scores come one after another, then the
// search's ballots (16 waves of 128 registers a work-group, of which heads of 128 spill up to 33).  64
// queries over up to 512 pages, 64 query heads over 8 (21 MB), 12.4 us in one launch.  2000 queries of 24 heads of 64 over 1250 short pages 34 us: 48 of some 80 k cycles
// of a SIMD are vector instructions.
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// The maximum over aligned sets of N lanes (8 or 16), in all of them.
template <int N>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
    static_assert(N == 8 || N == 16, "");
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));            // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));            // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));           // mirrored halves of 16
    if constexpr (N == 16) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
    return v;
}
// The maximum over a wave (uniform).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_lanes<16>(v);
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, true));     // the row before, rows 1 and 3
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, true));     // lane 31, rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// ---------------------------------------------------------------- mean keys
// One page of one head, by a wave: D / 16 lanes hold a token's 16-element blocks.
template <int D>
__device__ __forceinline__ void page_key(const PageKeysArgs& a, int page, int head, int lane) {
    constexpr int kLanes = D / 16, kStep = 64 / kLanes;     // lanes of a token, tokens of a load
    const int size = 1 << a.c.page_shift;
    const uint8_t* const codes = a.c.kc + page * a.c.cs_page + head * a.c.cs_head;
    const uint8_t* const scales = a.c.ks + page * a.c.ss_page + head * a.c.ss_head;
    const uint32_t code_at = (uint32_t)(lane / kLanes) * (uint32_t)a.c.cs_tok + 8 * (lane % kLanes);
    const uint32_t scale_at = (uint32_t)(lane / kLanes) * (uint32_t)a.c.ss_tok + lane % kLanes;
    const float g = a.c.kg[head];
    int sum[16] = {};
    float scale_sum = 0.0f;
    // eight tokens a lane at a time, all of their loads at once (a page holds whole multiples of
    // kStep tokens; past its end the last ones again, with zero scales)
    for (int t0 = 0; t0 < size; t0 += 8 * kStep) {
        u32x2v w[8];
        uint32_t s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = min(t0 + kStep * i, size - kStep);
            w[i] = *reinterpret_cast<const u32x2v*>(codes + t * a.c.cs_tok + code_at);
            s[i] = (scales + t * a.c.ss_tok)[scale_at];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float part[16] = {};
#pragma unroll
            for (int i = 4 * half; i < 4 * half + 4; ++i) {
                const float f = (float)e4m3_pair(t0 + kStep * i < size ? s[i] : 0u, false).x * 1024.0f;
                scale_sum += f;                             // (NaN with any of them)
                const f16x8 lo = e2m1_8(w[i].x), hi = e2m1_8(w[i].y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    part[j] = __builtin_fmaf((float)lo[j], f, part[j]);
                    part[8 + j] = __builtin_fmaf((float)hi[j], f, part[8 + j]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e] += (int)part[e];
        }
    }
    // over the lanes of the same elements, half of the elements handed over at each step
    int first = 16 * (lane % kLanes);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)sum[e], (uint32_t)sum[e + 8], false, false);
        sum[e] = (int)(r[0] + r[1]);
    }
    first += lane & 32 ? 8 : 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)sum[e], (uint32_t)sum[e + 4], false, false);
        sum[e] = (int)(r[0] + r[1]);
    }
    first += lane & 16 ? 4 : 0;
    // (two steps written out: a loop over them would index the sums by a variable)
    const auto hand_over = [&](int bit, int& a0, int& b0) {
        const bool upper = lane & bit;
        const int mine = upper ? b0 : a0, other = upper ? a0 : b0;
        a0 = mine + __shfl_xor(other, bit, 64);
    };
    hand_over(8, sum[0], sum[2]);
    hand_over(8, sum[1], sum[3]);
    first += lane & 8 ? 2 : 0;
    if constexpr (kLanes == 4) {
        hand_over(4, sum[0], sum[1]);
        first += lane & 4 ? 1 : 0;
    }
    constexpr int kMine = D / 64;
    int top = 0;
#pragma unroll
    for (int e = 0; e < kMine; ++e) top = max(top, abs(sum[e]));
    top = (int)wave_max((uint32_t)top);
    const bool bad = __any(scale_sum != scale_sum);
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
    if (lane == 0) a.scales[at] = bad ? __builtin_nanf("") : (float)((double)top * (double)g * a.inverse);
}

}  // namespace

// A wave per `chunk` slots and head: the pages whose last row is among them.
template <int D>
__global__ __launch_bounds__(256) void k_page_keys(const PageKeysArgs a) {
    const int lane = (int)threadIdx.x & 63;
    const unsigned item = blockIdx.x * 4 + (unsigned)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);      // (below 2^26)
    const unsigned part = item / (unsigned)a.c.kv_heads;
    const int64_t first = (int64_t)part * a.chunk;
    const int head = (int)(item - part * (unsigned)a.c.kv_heads);
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

// ---------------------------------------------------------------- scores
namespace {

// A score as a whole number of the same order; NaN below all.
__device__ __forceinline__ uint32_t order_of(float score) {
    const uint32_t u = __builtin_bit_cast(uint32_t, score + 0.0f);       // (-0 is 0)
    return score != score ? 0u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t order) {
    return __builtin_bit_cast(float, order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

// Rows of 16 lanes: a's maxima over rows 0, 1 and 2, 3 in rows 0 and 2, b's in rows 1 and 3.
__device__ __forceinline__ float max_rows16(float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    // (by way of two words: a bit cast of r[1] itself is compiled as one of r[0])
    const uint32_t x = r[0], y = r[1];
    return __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
// a's maxima over rows 0, 2 and 1, 3 in rows 0 and 1, b's in rows 2 and 3.
__device__ __forceinline__ float max_rows32(float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}

// Query rows as 8-bit integers, and their steps.
template <int D, int R>
struct IntRows {
    static constexpr int kPitch = D + 16;                    // 16 rows in different banks
    __attribute__((aligned(16))) uint8_t row[16 * R * kPitch];
    float step[16 * R];
};

// Mean keys of 64 candidates, lane l's scale that of the l-th.
template <int D>
struct KeyStep {
    i32x4 k[4][D / 64];                                      // 16 u + col, elements 64 c + 16 g ..
    float scale;
};
template <int D>
__device__ __forceinline__ KeyStep<D> load_keys(const SelectArgs& a, int kvh, int32_t entry, int col, int g) {
    const bool ok = (uint32_t)entry < (uint32_t)a.num_pages;
    const int mine = ok ? entry : 0;
    KeyStep<D> s;
    s.scale = a.scales[(int64_t)mine * a.kv_heads + kvh];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t page = (int64_t)__shfl(mine, 16 * u + col, 64) * a.kv_heads + kvh;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) s.k[u][c] = *reinterpret_cast<const i32x4*>(a.codes + page * D + 64 * c + 16 * g);
    }
    s.scale = ok ? s.scale : __builtin_nanf("");
    return s;
}

// Scores of the candidates w0 .. w1 - 1 of `run` queries from t on, for one cached head, by W
// waves together: store(query of the run, candidate, its order) once for each below end(query).
// Groups of more than 16 heads (one query): several times, before(candidate) hands back the last.
// table: of the first candidate.
template <int D, int GP, int R, int W, typename End, typename Store, typename Before>
__device__ __forceinline__ void score_pages(const SelectArgs& a, int t, int run, int kvh, const int32_t* table, int w0, int w1,
                                            IntRows<D, R>& ints, End&& end, Store&& store, Before&& before) {
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const bool many = GP == 16 && a.group > 16;              // heads: several tiles of one query
    for (int h0 = 0; h0 < a.group; h0 += GP < 16 ? GP : 16 * R) {
        // Loads come back in order: the first page numbers, the queries, the first mean keys.
        const auto entry_of = [&](int j) { return table[min(j + lane, w1 - 1)]; };
        const int first = w0 + 64 * wave;
        const int32_t e0 = entry_of(first);
        int32_t entry = entry_of(first + 64 * W);
        // 16 R query rows as 8-bit integers, D / 8 threads a row, by way of LDS
        const int tiles = many ? min((a.group - h0 + 15) / 16, R) : (run * GP + 15) / 16;
        constexpr int kRounds = 16 * R * (D / 8) / (64 * W) > 0 ? 16 * R * (D / 8) / (64 * W) : 1;
        u32x4v w[kRounds];
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
            const int e = min(tid + 64 * W * n, tiles * 16 * (D / 8) - 1), row = e / (D / 8);
            const int i = many ? 0 : min(row / GP, run - 1), head = min(many ? h0 + row : row % GP, a.group - 1);
            w[n] = *reinterpret_cast<const u32x4v*>(a.q + (int64_t)(t + i) * a.ld_q + (int64_t)(kvh * a.group + head) * D +
                                                    8 * (e % (D / 8)));
        }
        __builtin_amdgcn_sched_barrier(0);
        KeyStep<D> now = load_keys<D>(a, kvh, e0, col, g);
        if (h0 > 0) __syncthreads();
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
            const int e = tid + 64 * W * n, row = e / (D / 8);
            if (e >= tiles * 16 * (D / 8)) break;            // (whole rows)
            const uint32_t top =
                max_lanes<D / 8>(fold_pk(absmax_pk(absmax_pk(absmax_pk(absmax_pk(0u, w[n].x), w[n].y), w[n].z), w[n].w)));
            const float step = top >= 0x7F80u ? 0.0f : bf16_mag(top) * (1.0f / 127.0f);
            const uint32_t p[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
            // the stated quotients: by the reciprocal and one correction where all of it is normal
            const bool plain = step >= 0x1p-90f && step <= 0x1p+110f;
            const float inverse = 1.0f / step;
            uint32_t word[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float x = c & 1 ? hi_bf16(p[c >> 1]) : lo_bf16(p[c >> 1]);
                float y = div_rn(x, step, inverse);
                if (!plain) y = step > 0.0f ? x / step : 0.0f;
                y = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(y), -127.0f), 127.0f);
                word[c >> 2] |= ((uint32_t)(int)y & 0xFFu) << (8 * (c & 3));
            }
            *reinterpret_cast<uint2*>(ints.row + row * ints.kPitch + 8 * (e % (D / 8))) = make_uint2(word[0], word[1]);
            if (e % (D / 8) == 0) ints.step[row] = step;
        }
        __syncthreads();
        i32x4 q[R][D / 64];
        float by[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= tiles) break;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                q[r][c] = *reinterpret_cast<const i32x4*>(ints.row + (r * 16 + col) * ints.kPitch + 64 * c + 16 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) by[r][e] = ints.step[r * 16 + 4 * g + e];
        }
        // of a step's 64 candidates a lane finishes kTimes, for kOut queries of its four rows of a tile
        constexpr int kTimes = GP == 16 ? 1 : GP == 8 ? 2 : 4, kOut = GP >= 4 ? 1 : 4 / GP;
        int ends[R][kOut];                                   // of their candidates
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < kOut; ++e) {
                const int i = many ? 0 : (r * 16 + 4 * g) / GP + e;
                ends[r][e] = i < run ? min(end(i), w1) : 0;
            }
        // (one tile of rows: the next step's keys are on their way; more hide their own latency)
        constexpr bool kNext = R == 1;
        for (int j0 = first; j0 < w1; j0 += 64 * W) {
            KeyStep<D> next;
            if constexpr (kNext) {
                next = load_keys<D>(a, kvh, entry, col, g);  // (past the end the last again)
                entry = entry_of(j0 + 128 * W);
            }
            int at[kTimes];
            float of[kTimes];
#pragma unroll
            for (int n = 0; n < kTimes; ++n) {
                at[n] = GP == 16 ? lane : GP == 8 ? 32 * n + (lane & 31) : 16 * n + col;
                of[n] = GP == 16 ? now.scale : __shfl(now.scale, at[n], 64);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= tiles) break;
                float s[4][4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    i32x4 x = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) x = __builtin_amdgcn_mfma_i32_16x16x64_i8(q[r][c], now.k[u][c], x, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][e] = (float)x[e] * by[r][e];
                    // the best head: rows 4 g + e of the tile are heads % GP of query / GP
                    if constexpr (GP >= 2) {
                        s[u][0] = __builtin_fmaxf(s[u][0], s[u][1]);
                        s[u][2] = __builtin_fmaxf(s[u][2], s[u][3]);
                    }
                    if constexpr (GP >= 4) s[u][0] = __builtin_fmaxf(s[u][0], s[u][2]);
                }
                if constexpr (GP >= 8) {
                    s[0][0] = max_rows16(s[0][0], s[1][0]);
                    s[1][0] = max_rows16(s[2][0], s[3][0]);
                }
                if constexpr (GP >= 16) s[0][0] = max_rows32(s[0][0], s[1][0]);
#pragma unroll
                for (int e = 0; e < kOut; ++e) {
                    const int i = many ? 0 : (r * 16 + 4 * g) / GP + e;
#pragma unroll
                    for (int n = 0; n < kTimes; ++n) {
                        const int j = j0 + at[n];
                        if (j >= ends[r][e]) continue;
                        float best = s[n][e * (4 / kOut)];
                        if (many && h0 + r > 0) best = __builtin_fmaxf(best, before(j));
                        if (many && h0 + 16 * (r + 1) < a.group)
                            store(i, j, __builtin_bit_cast(uint32_t, best));
                        else
                            store(i, j, order_of(best * of[n]));
                    }
                }
            }
            if constexpr (kNext) {
                now = next;
            } else {
                now = load_keys<D>(a, kvh, entry, col, g);
                entry = entry_of(j0 + 128 * W);
            }
        }
    }
}

// ---------------------------------------------------------------- selection
// What the waves of a work-group hand each other, and the shortlist of a row (of each wave's
// row, one each).
constexpr int kShort = 256;
template <int W>
struct RowShared {
    int count[16];
    int2 pair[16];
    uint32_t column[256];
    uint32_t least;
    uint16_t list[W * kShort];        // places, ascending
};
template <int NW>
__device__ __forceinline__ int sum_waves(int v, int wave, int (&shared)[16]) {
    if constexpr (NW == 1) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[wave] = v;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += shared[w];
    return sum;
}

// Of a wave's 64 N orders, none above `top` and at least `wanted` from `from` on: the largest that
// `wanted` reach, or any that at most `enough` do as well; two bits at a time.
template <int N>
__device__ __forceinline__ int count_reach(const uint32_t (&x)[4], uint32_t t) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(x[i] >= t));
    return n;
}
template <int N>
__device__ __forceinline__ uint32_t edge_of(const uint32_t (&x)[4], int wanted, int enough, uint32_t from, uint32_t top) {
    const int bits = from == top ? 0 : (33 - __builtin_clz(from ^ top)) & ~1;                // even
    uint32_t edge = bits == 32 ? 0u : from >> bits << bits;
    for (int bit = bits - 2; bit >= 0; bit -= 2) {
        const uint32_t one = 1u << bit;
        const int n1 = count_reach<N>(x, edge + one), n2 = count_reach<N>(x, edge + 2 * one), n3 = count_reach<N>(x, edge + 3 * one);
        const int n = n3 >= wanted ? n3 : n2 >= wanted ? n2 : n1;
        edge += n3 >= wanted ? 3 * one : n2 >= wanted ? 2 * one : n1 >= wanted ? one : 0u;
        if (n >= wanted && n <= enough) break;
    }
    return edge;
}
// The edge of a row's columns, a little more than `wanted` of them from it on.  From a half, a
// quarter or an eighth of the largest score, if that is a number above zero and one of them is low
// enough (most of an order's upper bits are the exponent).
template <int N>
__device__ __forceinline__ uint32_t column_edge(const uint32_t (&x)[4], int wanted, uint32_t top) {
    constexpr uint32_t kOne = 1u << 23;
    uint32_t from = 0;
    if (top >= 0x80000000u + 4 * kOne) {
        const int n1 = count_reach<N>(x, top - kOne), n2 = count_reach<N>(x, top - 2 * kOne), n3 = count_reach<N>(x, top - 3 * kOne);
        from = n1 >= wanted ? top - kOne : n2 >= wanted ? top - 2 * kOne : n3 >= wanted ? top - 3 * kOne : 0;
    }
    return edge_of<N>(x, wanted, wanted + wanted / 8 + 4, from, top);
}

// The `wanted` largest of n orders (n > wanted >= 1), lower places first among equal ones, by NW
// waves: their places plus `add` to out, ascending.  keys: the orders of places w0 .. w0 +
// window - 1 once prepare(w0) has returned (all of them at the start if n <= window), zeros up to
// a multiple of 256.
template <int NW, typename Prepare, typename Shared>
__device__ __forceinline__ void select_row(const uint32_t* keys, int n, int wanted, int window, Prepare&& prepare, int32_t* out,
                                           int add, int wave, Shared& shared) {
    const int lane = (int)threadIdx.x & 63;
    // The wanted-th largest of 64 to 256 columns' largest orders is reached by that many orders at
    // least, and by few more (about 80 for 59 with 128 columns), unless many are equal: those are put
    // on a list, in their places' order, and one wave finishes there.
    if (wanted <= 200 && n <= window) {
        uint16_t* const list = shared.list + (NW == 1 ? (int)(threadIdx.x >> 6) * kShort : 0);
        uint32_t column[4] = {0, 0, 0, 0};
        for (int j = 256 * wave; j < n; j += 256 * NW) {
            const u32x4v k = *reinterpret_cast<const u32x4v*>(keys + j + 4 * lane);
            column[0] = max(column[0], k.x), column[1] = max(column[1], k.y);
            column[2] = max(column[2], k.z), column[3] = max(column[3], k.w);
        }
        if constexpr (NW > 1) {
            if (wave == 0)                                   // (words: the columns lie on no 16-byte boundary)
#pragma unroll
                for (int e = 0; e < 4; ++e) shared.column[64 * e + lane] = 0;
            __syncthreads();
            if (256 * wave < n)
#pragma unroll
                for (int e = 0; e < 4; ++e) atomicMax(&shared.column[64 * e + lane], column[e]);
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 4; ++e) column[e] = shared.column[64 * e + lane];
        }
        const uint32_t top = wave_max(max(max(column[0], column[1]), max(column[2], column[3])));
        // (1 at least: not the zeros behind n.  Those of NaN scores then are too few)
        uint32_t least = 1;
        if (NW <= 4 || wave == 0) {                          // (64 columns of several candidates do for few)
            if (n > 256 && wanted <= 40) {
                column[0] = max(max(column[0], column[1]), max(column[2], column[3]));
                least = max(column_edge<1>(column, wanted, top), 1u);
            } else if (n > 256 && wanted <= 100) {
                column[0] = max(column[0], column[1]), column[1] = max(column[2], column[3]);
                least = max(column_edge<2>(column, wanted, top), 1u);
            } else {
                least = max(column_edge<4>(column, wanted, top), 1u);
            }
        }
        if constexpr (NW > 4) {                              // (the others would only be in its way)
            if (wave == 0 && lane == 0) shared.least = least;
            __syncthreads();
            least = shared.least;
        }
        const int share = NW == 1 ? n : ((n + NW - 1) / NW + 255) & ~255, j0 = min(share * wave, n), j1 = min(j0 + share, n);
        int m = 0, mine = 0;
        if constexpr (NW > 1) {
            for (int j = j0; j < j1; j += 256) {
                const u32x4v k = *reinterpret_cast<const u32x4v*>(keys + j + 4 * lane);
                mine += __popcll(__ballot(k.x >= least)) + __popcll(__ballot(k.y >= least)) + __popcll(__ballot(k.z >= least)) +
                        __popcll(__ballot(k.w >= least));
            }
            if (lane == 0) shared.count[wave] = mine;
            __syncthreads();
            mine = 0;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                mine += w < wave ? shared.count[w] : 0;
                m += shared.count[w];
            }
        }
        if (NW == 1 || (m >= wanted && m <= kShort)) {
            for (int j = j0; j < j1; j += 256) {
                uint32_t k[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) k[e] = keys[j + 64 * e + lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t in = __ballot(k[e] >= least);
                    const int place = mine + __popcll(in & ((1ull << lane) - 1));
                    if (k[e] >= least && place < kShort) list[place] = (uint16_t)(j + 64 * e + lane);
                    mine += __popcll(in);
                }
            }
            if constexpr (NW == 1) m = mine;
        }
        if constexpr (NW > 1) __syncthreads();
        if (m >= wanted && m <= kShort) {
            if (wave != 0) return;
            uint32_t k[4];
            int place[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                place[e] = list[min(64 * e + lane, m - 1)];
                k[e] = 64 * e + lane < m ? keys[place[e]] : 0u;          // (those of the list are 1 and more)
            }
            const uint32_t edge = m <= 128 ? edge_of<2>(k, wanted, wanted, least, top) : edge_of<4>(k, wanted, wanted, least, top);
            int ties = wanted;
#pragma unroll
            for (int e = 0; e < 4; ++e) ties -= __popcll(__ballot(k[e] > edge));
            int done = 0, equal = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool up = k[e] > edge, tie = k[e] == edge;
                const uint64_t ups = __ballot(up), same = __ballot(tie), below = (1ull << lane) - 1;
                const int my_ties = equal + __popcll(same & below);
                // written before this one: every larger one and the first ties
                if (up || (tie && my_ties < ties)) out[done + __popcll(ups & below) + min(my_ties, ties)] = place[e] + add;
                done += __popcll(ups);
                equal += __popcll(same);
            }
            return;
        }
    }

    const auto windows = [&](auto&& visit) {
        for (int w0 = 0; w0 < n; w0 += window) {
            if (n > window) prepare(w0);
            visit(w0, min(window, n - w0));
        }
    };
    const auto count_from = [&](uint32_t t) {               // t >= 1
        int count = 0;
        windows([&](int, int size) {
            for (int j = 256 * wave; j < size; j += 256 * NW) {
                const u32x4v k = *reinterpret_cast<const u32x4v*>(keys + j + 4 * lane);
                count += __popcll(__ballot(k.x >= t)) + __popcll(__ballot(k.y >= t)) + __popcll(__ballot(k.z >= t)) +
                         __popcll(__ballot(k.w >= t));
            }
        });
        return sum_waves<NW>(count, wave, shared.count);
    };
    // The largest order that `wanted` reach, between lo (which at least `wanted` reach) and hi
    // (which `above` do, fewer).  Halfway by value first: scores lie like a bell, so that
    // halves of their orders would be spent on the smallest numbers.  Any order that exactly
    // `wanted` reach does as well.
    uint32_t lo = 0, hi = 0xFFFFFFFFu;                       // (an order is below 2^32 - 1)
    int above = 0;
    bool exact = false;
    for (int step = 0; hi - lo > 1; ++step) {
        uint32_t t = lo + ((hi - lo) >> 1);
        if (step < 24) {
            const uint32_t by_value = order_of(0.5f * value_of(max(lo, 0x00800000u)) + 0.5f * value_of(min(hi, 0xFF7FFFFFu)));
            if (by_value > lo && by_value < hi) t = by_value;
        }
        t = (uint32_t)__builtin_amdgcn_readfirstlane((int)t);
        const int count = count_from(t);
        if (count < wanted) {
            hi = t;
            above = count;
        } else {
            lo = t;
            if (count == wanted) {
                exact = true;
                break;
            }
        }
    }
    const uint32_t all_from = exact ? lo : lo + 1;           // every order from here on, and ...
    const int ties = exact ? 0 : wanted - above;             // ... the first of those equal to lo
    int done = 0, equal = 0;
    windows([&](int w0, int size) {
        // contiguous places a wave
        const int share = ((size + NW - 1) / NW + 63) & ~63, j0 = min(share * wave, size), j1 = min(j0 + share, size);
        int next_done = done, next_equal = equal;
        if constexpr (NW > 1) {
            int ups = 0, same = 0;
            for (int j = j0; j < j1; j += 64) {
                const uint32_t k = keys[min(j + lane, size - 1)];
                ups += __popcll(__ballot(j + lane < j1 && k >= all_from));
                same += __popcll(__ballot(j + lane < j1 && k == lo));
            }
            __syncthreads();
            if (lane == 0) shared.pair[wave] = make_int2(ups, same);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const int2 p = shared.pair[w];
                if (w < wave) done += p.x, equal += p.y;
                next_done += p.x, next_equal += p.y;
            }
        }
        for (int j = j0; j < j1; j += 64) {
            const uint32_t k = keys[min(j + lane, size - 1)];
            const bool in = j + lane < j1, up = in && k >= all_from, tie = in && k == lo;
            const uint64_t ups = __ballot(up), same = __ballot(tie), below = (1ull << lane) - 1;
            const int my_ties = equal + __popcll(same & below);
            if (up || (tie && my_ties < ties)) out[done + __popcll(ups & below) + min(my_ties, ties)] = w0 + j + lane + add;
            done += __popcll(ups);
            equal += __popcll(same);
        }
        if constexpr (NW > 1) done = next_done, equal = next_equal;
    });
}

// The page of the i-th query from `at` on (-1: before the sequence).
__device__ __forceinline__ int page_of_query(const SelectArgs& a, const Query& at, int i) {
    const int p = at.len - at.left + i;
    return p < 0 ? -1 : p >> a.page_shift;
}

}  // namespace

// Few queries with many candidates: their scores by work-groups of their own (a row's 256 to 512
// candidates each), as order_of(), to a.orders.
template <int D, int GP>
__global__ __launch_bounds__(256) void k_score_pages(const SelectArgs a) {
    __shared__ IntRows<D, 1> ints;
    const unsigned unit = blockIdx.x / (unsigned)a.splits, split = blockIdx.x - unit * (unsigned)a.splits;
    const int t = (int)(unit / (unsigned)a.kv_heads), kvh = (int)(unit - (unsigned)t * (unsigned)a.kv_heads);
    const Query at = query_of(a, a.page_shift, t);
    if (at.b < 0) return;
    const int current = page_of_query(a, at, 0), n = current + 1 - a.first - a.last;
    if (current < a.top || a.top == a.first + a.last || n > a.order_stride) return;
    const int share = ((n + a.splits - 1) / a.splits + 255) & ~255;
    const int w0 = min((int)split * share, n), w1 = min(w0 + share, n);
    if (w0 >= w1) return;
    uint32_t* const orders = a.orders + (int64_t)unit * a.order_stride;
    score_pages<D, GP, 1, 4>(
        a, t, 1, kvh, a.table + (int64_t)at.b * a.ld_table + a.first, w0, w1, ints, [&](int) { return n; },
        [&](int, int j, uint32_t order) { orders[j] = order; }, [&](int j) { return __builtin_bit_cast(float, orders[j]); });
}

// W waves take `tokens` consecutive queries for one cached head, run by run of one sequence:
// their scores share each mean key that is read.  GP: the group's heads, rounded up to a
// power of two (16 for more); R: tiles of 16 query rows (16 / GP queries each) held at a time.
// Scores of `window` candidates a query are held in LDS, as order_of(); a query with more takes
// all of LDS, and where that is too little every pass over its scores forms them again.
template <int D, int GP, int R, int W>
__global__ __launch_bounds__(64 * W, W == 4 ? 2 : 4) void k_select_pages(const SelectArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t keys[];
    __shared__ RowShared<R == 1 ? 1 : W> shared;
    __shared__ IntRows<D, R> ints;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kvh = (int)(blockIdx.x % (unsigned)a.kv_heads);
    const int t_end = (int)min((int64_t)(blockIdx.x / (unsigned)a.kv_heads + 1) * a.tokens, (int64_t)a.total_q);
    const int wanted = a.top - a.first - a.last;

    for (int t = (int)(blockIdx.x / (unsigned)a.kv_heads) * a.tokens, run; t < t_end; t += run) {
        const Query at = query_of(a, a.page_shift, t);
        run = 1;
        if (at.b < 0) continue;
        run = min(at.left, t_end - t);
        int window = a.window;
        if (run > 1 && page_of_query(a, at, run - 1) + 1 - a.first - a.last > window) run = 1;
        if (run == 1) window = a.window * a.tokens;
        const int n_most = page_of_query(a, at, run - 1) + 1 - a.first - a.last;
        const int32_t* const table = a.table + (int64_t)at.b * a.ld_table + a.first;

        // what needs no scores
        for (int i = wave; i < run; i += W) {
            const int current = page_of_query(a, at, i);
            int32_t* const out = a.out + ((int64_t)(t + i) * a.kv_heads + kvh) * a.top;
            if (current < a.top) {                           // all there are
                for (int e = lane; e < a.top; e += 64) out[e] = e <= current ? e : -1;
            } else {
                for (int e = lane; e < a.first; e += 64) out[e] = e;
                for (int e = lane; e < a.last; e += 64) out[a.top - a.last + e] = current - a.last + 1 + e;
            }
        }
        if (wanted == 0 || page_of_query(a, at, run - 1) < a.top) continue;

        const auto score = [&](int w0) {
            const int w1 = min(w0 + window, n_most);
            __syncthreads();
            for (int i = wave; i < run; i += W) {            // zeros behind each query's own
                const int n = max(page_of_query(a, at, i) + 1 - a.first - a.last - w0, 0);
                for (int j = n + lane; j < min((w1 - w0 + 255) & ~255, window); j += 64) keys[i * window + j] = 0;
            }
            if (a.orders && n_most <= min(a.order_stride, window)) {
                const uint32_t* const orders = a.orders + (int64_t)blockIdx.x * a.order_stride;
                for (int j = tid; j < n_most; j += 64 * W) keys[j] = orders[j];
            } else {
                score_pages<D, GP, R, W>(
                    a, t, run, kvh, table, w0, w1, ints,
                    [&](int i) { return page_of_query(a, at, i) + 1 - a.first - a.last; },
                    [&](int i, int j, uint32_t order) { keys[i * window + (j - w0)] = order; },
                    [&](int j) { return __builtin_bit_cast(float, keys[j - w0]); });
            }
            __syncthreads();
        };
        if (n_most <= window) score(0);
        if (R > 1 && run >= W) {
            // a wave a query (their scores fit: runs of several do)
            for (int i = wave; i < run; i += W) {
                if (page_of_query(a, at, i) < a.top) continue;
                select_row<1>(keys + i * window, page_of_query(a, at, i) + 1 - a.first - a.last, wanted, window, [](int) {},
                              a.out + ((int64_t)(t + i) * a.kv_heads + kvh) * a.top + a.first, a.first, 0, shared);
            }
        } else {
            for (int i = 0; i < run; ++i) {
                if (page_of_query(a, at, i) < a.top) continue;
                select_row<W>(keys + i * window, page_of_query(a, at, i) + 1 - a.first - a.last, wanted, window, score,
                              a.out + ((int64_t)(t + i) * a.kv_heads + kvh) * a.top + a.first, a.first, wave, shared);
            }
        }
        __syncthreads();                                     // before the next run's scores
    }
}

template <int D, int GP>
static void launch_select(const SelectArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.total_q + a.tokens - 1) / a.tokens * a.kv_heads));
    const unsigned bytes = (unsigned)a.window * (unsigned)a.tokens * 4;
    if (a.orders)
        hipLaunchKernelGGL((k_score_pages<D, GP>), dim3((unsigned)((int64_t)a.total_q * a.kv_heads * a.splits)), dim3(256), 0, stream, a);
    if (a.waves == 16)
        hipLaunchKernelGGL((k_select_pages<D, GP, 1, 16>), grid, dim3(1024), bytes, stream, a);
    else if (a.tokens == 1)
        hipLaunchKernelGGL((k_select_pages<D, GP, 1, 4>), grid, dim3(256), bytes, stream, a);
    else
        hipLaunchKernelGGL((k_select_pages<D, GP, (GP == 16 ? 4 : 2), 4>), grid, dim3(256), bytes, stream, a);
}
template <int D>
static void launch_select_group(const SelectArgs& a, hipStream_t stream) {
    if (a.group == 1)
        launch_select<D, 1>(a, stream);
    else if (a.group == 2)
        launch_select<D, 2>(a, stream);
    else if (a.group <= 4)
        launch_select<D, 4>(a, stream);
    else if (a.group <= 8)
        launch_select<D, 8>(a, stream);
    else
        launch_select<D, 16>(a, stream);
}
hipError_t launch_select_pages(const SelectArgs& a, hipStream_t stream) {
    if (a.head_dim == 128)
        launch_select_group<128>(a, stream);
    else
        launch_select_group<64>(a, stream);
    return hipGetLastError();
}

}  // namespace mxq
