// mxq_attention_ranges.hpp -- the units of attention with shared prefixes (gfx950): which
// query rows, through which pages, over which tokens.
//
// A row at position p of a sequence whose first P tokens are shared sees the tokens 0 ..
// min(P, p + 1) - 1 in the prefix's unit, through the pages of its group's first sequence, and
// P .. p in its sequence's own.  In both a row's tokens are hi - count + 1 .. hi.
//
// What bounds it: 32 sequences, 64 query heads over 8 of 128, on 65536 shared tokens take 94 to 96
// us, 719 to 740 TFLOP/s: the vector and matrix instructions of the form for many rows (66 k cycles of
// products a SIMD, 91 k of vector ones), then the parts, written and joined in FP32 (36 MB each way). 64
// sequences on 8192 tokens with 200 to 1500 of their own take 45 us: each of 256 work-groups has 16
// tiles of the prefix, 22 us, between a start of 5 (groups, runs, lengths, page table, queries and first
// tile, one after another) and its parts, while the sequences' own tokens (60 MB) pass beside them.
// Four sequences on 2048 tokens take 10.8 us: 7.8 the units, 3.3 to 4 of them until the first tile, and
// a launch that joins.
#pragma once

#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

// The shared tokens of a sequence, at most what a row of the table holds.
__device__ __forceinline__ int shared_tokens(const PrefixAttnArgs& a, int b) {
    const int64_t cap = min((int64_t)a.table_pages << a.c.page_shift, (int64_t)0x7FFFFF00);
    return (int)min((int64_t)max(a.prefix_lens[b], 0), cap);
}
// The first sequence of a group (the first group's is 0, that after the last `batch`).
__device__ __forceinline__ int group_start(const PrefixAttnArgs& a, int g) {
    return g <= 0 ? 0 : g >= a.groups ? a.batch : min(max(a.group_starts[g], 0), a.batch);
}
__device__ __forceinline__ int query_start(const AttnArgs& a, int b) { return min(max(a.q_starts[b], 0), a.total_q); }

// A unit's piece; uniform over the work-group.  rows <= 0: none.
struct RangeUnit {
    const int32_t* table;
    int start;                        // query row of the run's first query
    int len;                          // tokens that may be read
    int kvh, part;
    int q0, in_group;                 // its first row: query of the run and head of the group
    int rows;
    int low, first_pos;               // own tokens: from `low` on, position of the run's first query (may be negative)
    bool shared;
    int min_hi;                       // the least of the rows' last tokens
    int body, first, last;            // tiles body + first .. body + last - 1
};

// limits: LDS for a prefix's rows, kRows tokens: how many tokens each query sees.
template <int kRows>
__device__ __forceinline__ RangeUnit range_unit(const PrefixAttnArgs& a, int block, int* limits) {
    const int tid = (int)threadIdx.x, lane = tid & 63;
    RangeUnit u;
    u.shared = block < a.prefix_blocks;
    const int splits = u.shared ? a.prefix_splits : a.own_splits;
    const unsigned at = (unsigned)(u.shared ? block : block - a.prefix_blocks);
    const unsigned unit = at / (unsigned)splits, split = at - unit * (unsigned)splits;
    const unsigned tile = unit / (unsigned)a.c.kv_heads;
    u.kvh = (int)(unit - tile * (unsigned)a.c.kv_heads);
    u.part = (int)split + (u.shared ? a.own_splits : 0);
    u.rows = 0;
    u.low = u.first_pos = 0;
    int n = 0;
    if (!u.shared) {
        const int b = (int)(tile / (unsigned)a.row_tiles), rt = (int)(tile - (unsigned)b * (unsigned)a.row_tiles);
        const Seq s = sequence(a, b);
        const int64_t r0 = (int64_t)rt * kRows;
        u.rows = (int)min((int64_t)min(s.nq, a.max_q_len) * a.group - r0, (int64_t)kRows);
        if (u.rows <= 0) return u;
        u.q0 = (int)(r0 / a.group), u.in_group = (int)(r0 - (int64_t)u.q0 * a.group);
        u.table = a.table + (int64_t)b * a.ld_table;
        u.start = s.start;
        u.len = s.len;
        u.low = shared_tokens(a, b);
        u.first_pos = s.len - s.nq;
        u.min_hi = max(u.first_pos + u.q0, -1);
        const int max_hi = u.first_pos + u.q0 + (u.in_group + u.rows - 1) / a.group;
        u.body = u.low >> 6;
        n = max_hi >= u.low ? (max_hi >> 6) - u.body + 1 : 0;
    } else {
        // the group whose row tiles hold this one, 64 groups a step
        int g = -1;
        unsigned left = tile;
        for (int g0 = 0; g0 < a.groups; g0 += 64) {
            uint32_t tiles = 0;
            if (g0 + lane < a.groups) {
                const int q0 = query_start(a, group_start(a, g0 + lane)), q1 = query_start(a, group_start(a, g0 + lane + 1));
                tiles = (uint32_t)(((int64_t)max(q1 - q0, 0) * a.group + kRows - 1) / kRows);
            }
            const uint32_t upto = wave_scan(tiles);
            const uint64_t past = __ballot(upto > left);
            if (past) {
                const int j = __builtin_ctzll(past);
                left -= (unsigned)__builtin_amdgcn_readlane((int)(upto - tiles), j);
                g = g0 + j;
                break;
            }
            left -= (unsigned)__builtin_amdgcn_readlane((int)upto, 63);
        }
        if (g < 0) return u;
        const int b0 = __builtin_amdgcn_readfirstlane(group_start(a, g)), b1 = __builtin_amdgcn_readfirstlane(group_start(a, g + 1));
        u.start = __builtin_amdgcn_readfirstlane(query_start(a, b0));
        const int64_t all = (int64_t)(__builtin_amdgcn_readfirstlane(query_start(a, b1)) - u.start) * a.group;
        const int64_t r0 = (int64_t)left * kRows;
        u.rows = (int)min(all - r0, (int64_t)kRows);
        if (u.rows <= 0) return u;
        u.q0 = (int)(r0 / a.group), u.in_group = (int)(r0 - (int64_t)u.q0 * a.group);
        // what the tile's queries see
        const int q_first = u.start + u.q0, q_last = q_first + (u.in_group + u.rows - 1) / a.group;
        for (int i = tid; i < kRows; i += (int)blockDim.x) limits[i] = 0;
        __syncthreads();
        for (int b = b0 + tid; b < b1; b += (int)blockDim.x) {
            const Seq s = sequence(a, b);
            const int shared = shared_tokens(a, b);
            for (int q = max(s.start, q_first); q <= min(s.start + s.nq - 1, q_last); ++q)
                limits[q - q_first] = min(shared, max(s.len - s.nq + (q - s.start), -1) + 1);
        }
        __syncthreads();
        int most = 0, least = 0x7FFFFFFF;
        for (int i = lane; i <= q_last - q_first; i += 64) most = max(most, limits[i]), least = min(least, limits[i]);
#pragma unroll
        for (int bit = 1; bit < 64; bit <<= 1) {
            most = max(most, __shfl_xor(most, bit, 64));
            least = min(least, __shfl_xor(least, bit, 64));
        }
        u.table = a.table + (int64_t)b0 * a.ld_table;
        u.len = __builtin_amdgcn_readfirstlane(most);
        u.min_hi = __builtin_amdgcn_readfirstlane(least) - 1;
        u.body = 0;
        n = (int)(((int64_t)u.len + 63) >> 6);
    }
    const int chunk = (n + splits - 1) / splits;
    u.first = min((int)split * chunk, n);
    u.last = min(u.first + chunk, n);
    return u;
}

// Row r of a unit (row 0 past the last): its query, head, last token and number of tokens.
struct RangeRow {
    int query, head, hi, count;
};
__device__ __forceinline__ RangeRow range_row(const PrefixAttnArgs& a, const RangeUnit& u, const int* limits, int r) {
    const bool live = r < u.rows;
    const int at = u.in_group + (live ? r : 0), qi = at / a.group;
    RangeRow row;
    row.query = u.start + u.q0 + qi;
    row.head = u.kvh * a.group + (at - qi * a.group);
    row.hi = u.shared ? limits[qi] - 1 : max(u.first_pos + u.q0 + qi, -1);
    row.count = live ? max(row.hi + 1 - u.low, 0) : 0;
    return row;
}
__device__ __forceinline__ bool in_range(int hi, int count, int t) { return (uint32_t)(hi - t) < (uint32_t)count; }

}  // namespace

}  // namespace mxq
