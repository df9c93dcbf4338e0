// mxq_serve.hpp -- launch descriptors of the serving calls (RMS norm -> FP8, rotary
// append, attention over the NVFP4 cache, page selection), shared by the host entry points
// (mxq_serve_api.cpp, mxq_pages_api.cpp) and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// ---------------------------------------------------------------- RMS norm -> FP8 1x128
struct RmsNormArgs {
    const uint16_t* x;
    const uint16_t* res;              // null: no residual
    uint16_t* res_out;
    const uint16_t* w;
    uint16_t* y;                      // null: not wanted
    uint8_t* q;
    float* scales;
    int64_t ldx, ld_res, ld_res_out, ld_y, ldq, srow, sgroup, m;
    int32_t n;
    float eps;
};
hipError_t launch_add_rmsnorm_quant_fp8(const RmsNormArgs& a, bool ue8m0, hipStream_t stream);

// ---------------------------------------------------------------- the paged NVFP4 cache
struct KvCache {
    uint8_t* kc;
    uint8_t* ks;
    uint8_t* vc;
    uint8_t* vs;
    const float* kg;
    const float* vg;
    int64_t num_pages;
    int64_t cs_page, cs_head, cs_tok; // strides of the codes, bytes
    int64_t ss_page, ss_head, ss_tok; // strides of the scales, bytes
    int32_t page_shift;               // log2(page_size)
    int32_t kv_heads;
    int32_t head_dim;
};

// ---------------------------------------------------------------- rotary append
struct RopeAppendArgs {
    const uint16_t* q;
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    int64_t ld_q, ld_q_out, ld_k, ld_v, tokens;
    const int32_t* positions;
    const int64_t* slots;
    const double* inv_freq;
    double factor;
    int32_t rot_dim;
    int32_t q_heads;
    uint16_t* k_values;               // null: not wanted
    uint16_t* v_values;
    KvCache c;
};
hipError_t launch_rope_append_nvfp4(const RopeAppendArgs& a, bool interleaved, hipStream_t stream);

// ---------------------------------------------------------------- attention
constexpr int kMaxParts = 512;        // parts of one unit that the join adds (and work-groups of the rows form)
struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    float* lse;                       // null: not wanted
    int64_t ld_q, ld_out;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* seq_lens;
    const int32_t* q_starts;
    int32_t table_pages;
    int32_t batch;
    int32_t q_heads;
    int32_t group;                    // q_heads / kv_heads
    int32_t total_q;
    int32_t max_q_len;
    int32_t window, sinks;
    double scale_log2;                // softmax_scale * log2(e)
    KvCache c;
    // the plan: a unit is (sequence, row tile, cached head) with tile_rows query rows.
    // Rows form: `splits` work-groups share the line of all units' tiles (one row tile);
    // form for many rows: each unit's visible tiles in at most `splits` chunks of `chunk`
    // (the last takes the rest).
    int32_t tile_rows, row_tiles;
    int32_t splits, chunk;
    float* part_o;                    // workspace: parts, [part][tile_rows][head_dim]
    float2* part_ml;                  // workspace: [part][tile_rows] (maximum, sum)
    int2* desc;                       // workspace, rows form: [unit] (first work-group, parts or 0)
};
hipError_t launch_attention_rows(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_prompt(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_join(const AttnArgs& a, hipStream_t stream);

// ---------------------------------------------------------------- pages: mean keys, selection
struct PageKeysArgs {
    KvCache c;
    const int64_t* slots;
    int64_t tokens;
    int8_t* codes;                    // [num_pages][kv_heads][head_dim]
    float* scales;                    // [num_pages][kv_heads]
    int32_t chunk;                    // slots a wave looks at, 1 .. 64
    double inverse;                   // of 130048 page_size
};
hipError_t launch_page_keys(const PageKeysArgs& a, hipStream_t stream);

struct SelectArgs {
    const uint16_t* q;
    int64_t ld_q;
    const int8_t* codes;
    const float* scales;
    int64_t num_pages;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* seq_lens;
    const int32_t* q_starts;
    int32_t* out;                     // [total_q][kv_heads][top]
    int32_t table_pages, batch, total_q;
    int32_t kv_heads, head_dim, group, page_shift;
    int32_t top, first, last;
    int32_t window;                   // candidates whose scores are held of a query at a time, a multiple of 256
    int32_t tokens;                   // queries of a work-group
    int32_t waves;                    // of a work-group: 4, or 16 for one query
    uint32_t* orders;                 // null, or workspace: [query][cached head][order_stride] scores, made
    int32_t order_stride, splits;     // by `splits` work-groups each where there are no more candidates
};
hipError_t launch_select_pages(const SelectArgs& a, hipStream_t stream);

// Attention over listed pages: a unit is (query, cached head, tile of tile_rows rows of its
// group), its list in `splits` pieces.  Parts: [piece][query row][head].
struct PagesAttnArgs : AttnArgs {
    const int32_t* pages;             // [total_q][kv_heads][top]
    int32_t top;
    int32_t waves;                    // of a work-group
};
hipError_t launch_attention_pages(const PagesAttnArgs& a, hipStream_t stream);

// Attention with shared prefixes: per group of sequences, its rows over the first tokens that
// they share, read through its first sequence's pages (units (group, row tile, cached head)
// first), and per sequence its own tokens from there on (units (sequence, row tile, cached
// head)), each in pieces.  Parts: [own pieces, then prefix pieces][query row][head]; splits
// counts both.
struct PrefixAttnArgs : AttnArgs {
    const int32_t* group_starts;
    const int32_t* prefix_lens;       // per sequence
    int32_t groups;
    int32_t own_splits, prefix_splits;
    int32_t prefix_blocks;            // the launch's first work-groups take units of the prefixes ...
    int32_t own_blocks;               // ... and these units of sequences' own tokens
};
hipError_t launch_attention_ranges_rows(const PrefixAttnArgs& a, hipStream_t stream);
hipError_t launch_attention_ranges_prompt(const PrefixAttnArgs& a, hipStream_t stream);

// Joins `splits` parts of every query row and head, [part][query row][head].
hipError_t launch_attention_join_rows(const AttnArgs& a, hipStream_t stream);

}  // namespace mxq
