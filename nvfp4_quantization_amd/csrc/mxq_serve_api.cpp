// mxq_serve_api.cpp -- the C ABI of the serving calls of include/mxq.h (RMS norm ->
// FP8, rotary append to the NVFP4 cache, attention over it): argument checks, launch
// planning and kernel launches.  Host code only; nothing here allocates, synchronizes,
// memsets or reads the environment.
#include <cmath>

#include "mxq_serve_checks.hpp"

namespace {

// How the attention call splits its work.  A unit is (sequence, row tile, cached head).
//   rows form    up to 32 query rows per cached head: a decoding step or a draft.  One row
//                tile of 16 or 32.  A work-group takes a unit, or, where that leaves too
//                much of the chip idle too long (pays_line), kRowsGroups work-groups (what
//                the chip holds at once) share the line of all units' tiles evenly.
//   prompt form  more rows, 128 a unit, whose waves share the dequantized tiles.  A unit's
//                tiles are cut into chunks only where there are fewer units than
//                kPromptGroups work-groups (two fit a CU).
constexpr int64_t kRowsGroups = 256 * 2;
constexpr int64_t kLineUnits = 1024;           // the line's units, and so its sequences, are fewer
constexpr int64_t kMaxUnits = 1ll << 24;       // a launch's work-groups, 256 threads each, are fewer
constexpr int64_t kPromptGroups = 256 * 2;
static_assert(kRowsGroups <= mxq::kMaxParts, "a unit may be cut by every work-group");

// Whether the line is worth its join and its cut units, about 40 tiles of a CU's time (11 us).
// With a work-group a unit the fullest CU has ceil(units / 256) units' tiles, with the line
// every CU has units / 256; up to 256 units, where all start at once, sequences are taken to
// fill three quarters of the longest.  Measured, line / unit in us (8 query rows a cached head,
// pages of 64; batches of equal lengths; of lengths from an eighth to the whole):
//                 head_dim 128                     head_dim 64
//   units  tiles  equal          ragged            equal          ragged          taken
//       8     36   14.5 / 14.4    14.2 / 14.3       12.5 / 10.9    12.5 / 10.7    unit
//       8     56   14.2 / 19.6    14.2 / 19.6       12.5 / 14.4    12.4 / 14.3    line
//      64     44   17.7 / 17.0    16.3 / 16.8       15.0 / 12.4    14.4 / 12.1    unit
//      64     72   19.9 / 24.4    19.6 / 24.1       15.8 / 17.4    16.0 / 17.1    line
//     128     56   23.4 / 20.7    21.9 / 20.5       18.1 / 14.8    17.3 / 14.7    unit
//     128     72   27.5 / 24.8    23.2 / 24.2       20.0 / 17.5    18.5 / 17.2    line
//     256     96   49.2 / 41.2    32.0 / 32.8       31.5 / 24.5    23.3 / 21.8    unit
//     256    192   83.1 / 74.7    54.6 / 59.9       51.6 / 43.3    35.1 / 38.0    line
//     384    192  119.0 / 121.0   78.1 / 90.7       70.6 / 72.0    48.4 / 58.1    line
//     512     24   34.2 / 24.6    29.6 / 20.2       24.8 / 14.5    22.9 / 13.7    unit
//     512    192  153.4 / 142.8  101.1 / 109.4      92.3 / 82.2    62.8 / 63.7    unit
//     768     96  122.1 / 111.1   80.8 / 88.8       76.1 / 61.0    51.5 / 47.5    unit
//    1024     96  150.0 / 144.3  102.8 / 101.7     100.6 / 80.2    66.3 / 60.3    unit
//    2048     48  157.7 / 149.4  111.9 / 100.7     101.4 / 81.9    74.8 / 58.0    unit
// With 32 rows a head (head_dim 128) both take longer: 128 x 72 40.5 / 35.0 and 36.6 / 34.3, 384 x
// 192 161 / 158 and 111 / 118.  So the rule is off by up to a seventh near its threshold (128 x
// 72), and it sees lengths only as max_seq_len: it loses a tenth for 256 equal sequences'
// units, and without bound where 512, 768 or from 1024 units on hold one far longer sequence
// (262144 tokens among 63 of 1000, 64 heads over 8: 1335 us; among 62, 504 units, 78).
bool pays_line(int64_t units, int64_t tiles) {
    if (units >= kLineUnits) return false;
    const int64_t idle = units <= 256 ? 256 - units * 3 / 4 : (units + 255) / 256 * 256 - units;     // CUs
    return tiles * idle > 40 * 256;
}
struct AttnPlan {
    int32_t tile_rows, row_tiles, splits, chunk;
    int64_t units;
    size_t ml_offset, desc_offset, bytes;      // workspace: parts, maxima and sums, unit descriptors
};

bool plan_attention(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t batch, int64_t total_q, int64_t max_q,
                    int64_t max_len, int64_t window, int64_t sinks, AttnPlan* p) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (d != 64 && d != 128) || batch < 1 || batch > 65535 ||
        total_q < 1 || max_q < 1 || max_len < 0 || window < 0 || sinks < 0 || !product_below(total_q, q_heads, 1ll << 31))
        return false;
    if (max_q > total_q) max_q = total_q;
    if (max_len > (1ll << 31)) max_len = 1ll << 31;
    const int64_t group = q_heads / kv_heads, rows = max_q * group;
    p->tile_rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
    p->row_tiles = (int32_t)((rows + p->tile_rows - 1) / p->tile_rows);
    p->units = batch * p->row_tiles * kv_heads;                     // (below 2^48)
    if (p->units >= kMaxUnits) return false;
    int64_t tiles = (max_len + 63) / 64;
    if (window > 0) {
        const int64_t near = (window + p->tile_rows / group + 62) / 64 + 1, far = (sinks + 63) / 64;
        tiles = tiles < near + far ? tiles : near + far;
    }
    if (tiles < 1) tiles = 1;
    int64_t parts = 0;
    p->ml_offset = p->desc_offset = p->bytes = 0;
    if (p->tile_rows < 128) {
        const bool line = pays_line(p->units, tiles);
        const int64_t most = product_below(p->units, tiles, 4 * kRowsGroups) ? (p->units * tiles + 3) / 4 : kRowsGroups;
        p->splits = (int32_t)(!line ? p->units : most < kRowsGroups ? most : kRowsGroups);
        p->chunk = 0;
        parts = line ? 2 * (int64_t)p->splits : 0;
    } else {
        int64_t chunk = product_below(p->units, tiles, 1ll << 62) ? (p->units * tiles + kPromptGroups - 1) / kPromptGroups : tiles;
        if (p->units * 2 > kPromptGroups || chunk > tiles) chunk = tiles;
        if (chunk < 4) chunk = 4;
        p->chunk = (int32_t)chunk;
        p->splits = (int32_t)((tiles + chunk - 1) / chunk);
        if (p->splits > mxq::kMaxParts) return false;        // (units >= 1 and kPromptGroups chunks: never)
        parts = p->splits > 1 ? p->units * p->splits : 0;
    }
    if (parts > 0) {
        p->ml_offset = (size_t)(parts * p->tile_rows * d * 4);
        p->desc_offset = p->ml_offset + (size_t)(parts * p->tile_rows * 8);
        p->bytes = (size_t)round256((int64_t)p->desc_offset + (p->tile_rows < 128 ? p->units * 8 : 0));
    }
    return true;
}

}  // namespace

extern "C" {

mxq_status mxq_add_rmsnorm_quant_fp8(const uint16_t* x_bf16, int64_t ldx, const uint16_t* residual, int64_t ld_res,
                                     uint16_t* residual_out, int64_t ld_res_out, const uint16_t* weight_bf16,
                                     float eps, int64_t m, int64_t n, uint32_t options,
                                     uint16_t* y_bf16, int64_t ld_y, uint8_t* q_e4m3, int64_t ldq,
                                     float* scales, int64_t scale_stride_row, int64_t scale_stride_group,
                                     void* stream) {
    if (options & ~(uint32_t)MXQ_FP8_UE8M0) return MXQ_ERR_INVALID_ARGUMENT;
    if (m < 0 || n <= 0 || ldx < n || ldq < n || scale_stride_row < 0 || scale_stride_group < 0)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return MXQ_ERR_INVALID_ARGUMENT;
    if ((residual != nullptr) != (residual_out != nullptr)) return MXQ_ERR_INVALID_ARGUMENT;
    if (residual && (ld_res < n || ld_res_out < n)) return MXQ_ERR_INVALID_ARGUMENT;
    if (y_bf16 && ld_y < n) return MXQ_ERR_INVALID_ARGUMENT;
    if (n % 128 != 0 || ldx % 8 != 0 || ldq % 16 != 0) return MXQ_ERR_MISALIGNED;
    if ((residual && (ld_res % 8 != 0 || ld_res_out % 8 != 0)) || (y_bf16 && ld_y % 8 != 0)) return MXQ_ERR_MISALIGNED;
    if (n > MXQ_RMSNORM_MAX_N) return MXQ_ERR_UNSUPPORTED;
    if (m == 0) return MXQ_OK;
    if (!x_bf16 || !weight_bf16 || !q_e4m3 || !scales) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(x_bf16, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) || !aligned(weight_bf16, 16) ||
        !aligned(y_bf16, 16) || !aligned(q_e4m3, 16) || !aligned(scales, 4))
        return MXQ_ERR_MISALIGNED;
    if (m > kMaxRows || !extent_ok(m, ldx, n) || !extent_ok(m, ldq, n) ||
        (residual && (!extent_ok(m, ld_res, n) || !extent_ok(m, ld_res_out, n))) || (y_bf16 && !extent_ok(m, ld_y, n)) ||
        !index2_ok(m, scale_stride_row, n / 128, scale_stride_group))
        return MXQ_ERR_UNSUPPORTED;
    if (!product_below(m, 1024, kMaxGridThreads)) return MXQ_ERR_UNSUPPORTED;
    mxq::RmsNormArgs a{x_bf16, residual, residual_out, weight_bf16, y_bf16, q_e4m3, scales, ldx, ld_res, ld_res_out,
                       ld_y, ldq, scale_stride_row, scale_stride_group, m, (int32_t)n, eps};
    return mxq::launch_add_rmsnorm_quant_fp8(a, (options & MXQ_FP8_UE8M0) != 0, static_cast<hipStream_t>(stream)) ==
                   hipSuccess
               ? MXQ_OK
               : MXQ_ERR_HIP;
}

mxq_status mxq_rope_append_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, uint16_t* q_out, int64_t ld_q_out,
                                 const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, int64_t tokens,
                                 const int32_t* positions, const int64_t* slots, const mxq_rope* rope,
                                 const mxq_nvfp4_kv* cache, uint16_t* k_values, uint16_t* v_values, void* stream) {
    mxq::KvCache c;
    const mxq_status st = check_cache(cache, &c);
    if (st != MXQ_OK) return st;
    if (!rope || (rope->flags & ~(uint32_t)MXQ_ROPE_INTERLEAVED)) return MXQ_ERR_INVALID_ARGUMENT;
    if (tokens < 0 || q_heads < 0 || rope->rot_dim < 0 || rope->rot_dim > c.head_dim) return MXQ_ERR_INVALID_ARGUMENT;
    if (rope->rot_dim % 16 != 0) return MXQ_ERR_MISALIGNED;
    if (!std::isfinite(rope->factor) || (rope->rot_dim > 0 && !rope->inv_freq)) return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t qw = (int64_t)q_heads * c.head_dim, kw = (int64_t)c.kv_heads * c.head_dim;
    if ((q_heads > 0 && (ld_q < qw || ld_q_out < qw)) || ld_k < kw || ld_v < kw) return MXQ_ERR_INVALID_ARGUMENT;
    if ((q_heads > 0 && (ld_q % 8 != 0 || ld_q_out % 8 != 0)) || ld_k % 8 != 0 || ld_v % 8 != 0)
        return MXQ_ERR_MISALIGNED;
    if (tokens == 0) return MXQ_OK;
    if ((q_heads > 0 && (!q || !q_out)) || !k || !v || !positions || !slots) return MXQ_ERR_INVALID_ARGUMENT;
    if ((q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16))) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(positions, 4) || !aligned(slots, 8) || !aligned(rope->inv_freq, 8) || !aligned(k_values, 16) ||
        !aligned(v_values, 16))
        return MXQ_ERR_MISALIGNED;
    if (q_heads > (1 << 20) || c.kv_heads > (1 << 20) || tokens > kMaxRows ||
        (q_heads > 0 && (!extent_ok(tokens, ld_q, qw) || !extent_ok(tokens, ld_q_out, qw))) ||
        !extent_ok(tokens, ld_k, kw) || !extent_ok(tokens, ld_v, kw) || !extent_ok(tokens, kw, kw))
        return MXQ_ERR_UNSUPPORTED;
    // at most one 256-thread work-group per 16 * 8 elements of every token
    const int64_t rows = q_heads + 2ll * c.kv_heads;
    if (!product_below(tokens, (rows * (c.head_dim / 8) + 255) / 256 * 256, kMaxGridThreads)) return MXQ_ERR_UNSUPPORTED;
    mxq::RopeAppendArgs a{q, q_out, k, v, ld_q, ld_q_out, ld_k, ld_v, tokens, positions, slots, rope->inv_freq,
                          rope->factor, rope->rot_dim, q_heads, k_values, v_values, c};
    return mxq::launch_rope_append_nvfp4(a, (rope->flags & MXQ_ROPE_INTERLEAVED) != 0,
                                         static_cast<hipStream_t>(stream)) == hipSuccess
               ? MXQ_OK
               : MXQ_ERR_HIP;
}

size_t mxq_attention_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t batch,
                                          int64_t total_q, int64_t max_q_len, int64_t max_seq_len,
                                          int32_t window, int32_t sinks) {
    AttnPlan p;
    if (!plan_attention(q_heads, kv_heads, head_dim, batch, total_q, max_q_len, max_seq_len, window, sinks, &p)) return 0;
    return p.bytes;
}

mxq_status mxq_attention_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q,
                               uint16_t* out, int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache,
                               const int32_t* block_table, int64_t ld_table, int64_t table_pages,
                               const int32_t* seq_lens, const int32_t* q_starts, int64_t batch,
                               int64_t max_q_len, int64_t max_seq_len, float softmax_scale,
                               int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                               void* stream) {
    mxq::KvCache c;
    const mxq_status st = check_cache(cache, &c);
    if (st != MXQ_OK) return st;
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || total_q < 0 || batch < 1 || max_q_len < 0 || max_seq_len < 0 ||
        table_pages < 0 || ld_table < table_pages || window < 0 || sinks < 0)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)q_heads * c.head_dim;
    if (ld_q < width || ld_out < width) return MXQ_ERR_INVALID_ARGUMENT;
    if (ld_q % 8 != 0 || ld_out % 8 != 0) return MXQ_ERR_MISALIGNED;
    if (batch > 65535 || !product_below(total_q, q_heads, 1ll << 31) || max_q_len > kMaxRows || max_seq_len > kMaxRows)
        return MXQ_ERR_UNSUPPORTED;
    if (total_q == 0 || max_q_len == 0) return MXQ_OK;
    if (!q || !out || !seq_lens || !q_starts || (table_pages > 0 && !block_table)) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(q_starts, 4))
        return MXQ_ERR_MISALIGNED;
    if (!extent_ok(total_q, ld_q, width) || !extent_ok(total_q, ld_out, width) ||
        !extent_ok(batch, ld_table, table_pages) || table_pages > kMaxRows)
        return MXQ_ERR_UNSUPPORTED;
    // (units bound every grid: 512 threads each only up to kWideUnits; parts and the join only
    // of fewer than kLineUnits units, or kPromptGroups / 2 at most)
    AttnPlan p;
    if (!plan_attention(q_heads, c.kv_heads, c.head_dim, batch, total_q, max_q_len, max_seq_len, window, sinks, &p))
        return MXQ_ERR_UNSUPPORTED;
    if (p.bytes > 0) {
        if (!workspace) return MXQ_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < p.bytes) return MXQ_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return MXQ_ERR_MISALIGNED;
    }
    mxq::AttnArgs a{};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.table = block_table;
    a.ld_table = ld_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.table_pages = (int32_t)table_pages;
    a.batch = (int32_t)batch;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.total_q = (int32_t)total_q;
    a.max_q_len = (int32_t)(max_q_len < total_q ? max_q_len : total_q);
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = (double)softmax_scale * 1.44269504088896341;
    a.c = c;
    if (c.num_pages == 0) a.table_pages = 0;                 // no page can be read: no tokens
    a.tile_rows = p.tile_rows;
    a.row_tiles = p.row_tiles;
    a.splits = p.splits;
    a.chunk = p.chunk;
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    a.part_o = p.bytes ? reinterpret_cast<float*>(ws) : nullptr;
    a.part_ml = p.bytes ? reinterpret_cast<float2*>(ws + p.ml_offset) : nullptr;
    a.desc = p.bytes && p.tile_rows < 128 ? reinterpret_cast<int2*>(ws + p.desc_offset) : nullptr;
    hipStream_t const hs = static_cast<hipStream_t>(stream);
    if ((p.tile_rows == 128 ? mxq::launch_attention_prompt(a, hs) : mxq::launch_attention_rows(a, hs)) != hipSuccess)
        return MXQ_ERR_HIP;
    if (p.bytes > 0 && mxq::launch_attention_join(a, hs) != hipSuccess) return MXQ_ERR_HIP;
    return MXQ_OK;
}

}  // extern "C"
