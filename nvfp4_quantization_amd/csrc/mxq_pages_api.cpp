// mxq_pages_api.cpp -- the C ABI of the calls of include/mxq.h around long and shared
// contexts (mean keys of pages, page selection, attention over listed pages, attention with
// shared prefixes): argument checks, launch planning and kernel launches.  Host code only; nothing here allocates,
// synchronizes, memsets or reads the environment.
#include <cmath>

#include "mxq_serve_checks.hpp"

namespace {

constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxBlocks = 1 << 24;        // of 256 threads
constexpr int64_t kGroups = 512;               // work-groups that the chip holds at once
constexpr int64_t kMaxPageTokens = 512;        // whose exact sums stay below 2^31
constexpr int64_t kMaxTop = 1 << 16;
constexpr int64_t kMaxListed = 1 << 30;        // tokens of a list's pages

// The mean keys' layout; num_pages 0 needs no arrays.
mxq_status check_keys(const mxq_page_keys* k) {
    if (!k || k->num_pages < 0 || k->kv_heads < 1 || k->page_size < 1 || k->head_dim < 1) return MXQ_ERR_INVALID_ARGUMENT;
    if (k->num_pages > 0 && (!k->codes || !k->scales)) return MXQ_ERR_INVALID_ARGUMENT;
    if (k->head_dim != 64 && k->head_dim != 128) return MXQ_ERR_UNSUPPORTED;
    if (k->page_size < 16 || k->page_size > kMaxPageTokens || (k->page_size & (k->page_size - 1))) return MXQ_ERR_UNSUPPORTED;
    if (!aligned(k->codes, 16) || !aligned(k->scales, 4)) return MXQ_ERR_MISALIGNED;
    if (k->num_pages > kMaxRows || !product_below(k->num_pages * k->head_dim, k->kv_heads, kMaxElems)) return MXQ_ERR_UNSUPPORTED;
    return MXQ_OK;
}

// The sequences of a call: MXQ_OK, or what is wrong with them.
mxq_status check_sequences(int64_t total_q, int64_t q_heads, const int32_t* block_table, int64_t ld_table, int64_t table_pages,
                           const int32_t* seq_lens, const int32_t* q_starts, int64_t batch) {
    if (!seq_lens || !q_starts || (table_pages > 0 && !block_table)) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(q_starts, 4)) return MXQ_ERR_MISALIGNED;
    if (batch > kMaxBatch || !product_below(total_q, q_heads, 1ll << 31) || table_pages > kMaxRows ||
        !extent_ok(batch, ld_table, table_pages))
        return MXQ_ERR_UNSUPPORTED;
    return MXQ_OK;
}

int32_t log2_of(int32_t page_size) {
    int32_t shift = 4;
    while ((1 << shift) < page_size) ++shift;
    return shift;
}

// How the selection spreads its work: queries of a work-group (for one cached head), and what is
// held of their scores in LDS.  Several where sequences have long runs of queries, which then
// share the mean keys that are read: two tiles of 16 rows, four of groups of more than 8 heads
// (a query a wave then: 2000 queries over 1024 pages, 16 heads over 2 of 128, 28.4 us against 30.4
// with four tiles, 16 over 4 of 64 22.9 against 30.3; 32 over 2 of 64 over 938 pages 19.8 with four,
// 32.9 with two).  Few queries with many candidates: their scores are made by more work-groups,
// through the workspace (one query, 8 cached heads: 2048 candidates 12.2 us against 17.0, 8192 15.4
// against 45.5).
constexpr int64_t kHeldScores = 14336;         // 56 KB, of one query
constexpr int64_t kHeldScoresRun = 12288;      // 48 KB, of several (whose waves need more beside them)
struct SelectPlan {
    int32_t window, tokens, waves, splits;
    int64_t order_stride;
    size_t bytes;
};
SelectPlan plan_select(int64_t group, int64_t kv_heads, int64_t page_size, int64_t batch, int64_t total_q, int64_t max_seq_len) {
    SelectPlan p{};
    const int64_t most = ((max_seq_len + page_size - 1) / page_size + 255) / 256 * 256;
    const int64_t window = most < 256 ? 256 : most > kHeldScores ? kHeldScores : most;
    int64_t padded = 1;
    while (padded < group && padded < 16) padded *= 2;
    int64_t tokens = group > 16 ? 1 : group > 8 ? 4 : 32 / padded;
    while (tokens > 1 && (tokens * batch > total_q || tokens * window > kHeldScoresRun || total_q * kv_heads < tokens * 512)) tokens /= 2;
    const int64_t units = total_q * kv_heads;
    p.window = (int32_t)window;
    p.tokens = (int32_t)tokens;
    p.waves = tokens == 1 && units <= 256 ? 16 : 4;
    if (p.waves == 16 && units <= 64 && window >= 1024) {
        p.order_stride = window;
        p.splits = (int32_t)(512 / units < window / 256 ? 512 / units : window / 256);
        p.bytes = (size_t)round256(units * window * 4);
    }
    return p;
}

// How attention over listed pages splits its work: a unit is (query, cached head, 16 or 32 rows
// of its group).  Few units go over several work-groups, a tile a wave where a CU each is enough
// for them, else two (4 sequences, 8 cached heads, 64 pages of 64 in 8 pieces 12.0 us, in 16
// 13.7; one sequence's 32 pages in 8 pieces 9.9, in 4 11.3).  From 2048 units on a wave takes one
// alone: 8000 of 24 tiles 241 us against 267 by four waves each, which have to meet.
struct PagesPlan {
    int32_t tile_rows, row_tiles, waves, splits;
    size_t ml_offset, bytes;
};
bool plan_pages(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t page_size, int64_t total_q, int64_t top, PagesPlan* p) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (d != 64 && d != 128) || page_size < 16 ||
        page_size > (1 << 20) || (page_size & (page_size - 1)) || total_q < 1 || top < 1 || top > kMaxTop ||
        top * page_size > kMaxListed || !product_below(total_q, q_heads, 1ll << 31))
        return false;
    const int64_t group = q_heads / kv_heads;
    p->tile_rows = group <= 16 ? 16 : 32;
    p->row_tiles = (int32_t)((group + p->tile_rows - 1) / p->tile_rows);
    const int64_t units = total_q * kv_heads * p->row_tiles, tiles = (top * page_size + 63) / 64;
    p->waves = units >= 2048 ? 1 : 4;
    int64_t splits = (tiles + 3) / 4;
    if (units * splits > 256) splits = (tiles + 7) / 8;
    if (splits > kGroups / units) splits = kGroups / units;
    p->splits = (int32_t)(splits < 1 ? 1 : splits);
    if (units >= kMaxBlocks) return false;
    p->ml_offset = p->bytes = 0;
    if (p->splits > 1) {
        const int64_t parts = total_q * q_heads * p->splits;
        p->ml_offset = (size_t)(parts * d * 4);
        p->bytes = (size_t)round256((int64_t)p->ml_offset + parts * 8);
    }
    return true;
}

// How attention with shared prefixes splits its work.  A group's rows over its prefix, and a
// sequence's over its own tokens, come in tiles of 16, 32 or 128: the first two by the waves'
// own tiles, 128 by the form for many rows, all in one launch.  Pieces of both until it fills the
// chip, all by the mean group and the longest estimates (32 sequences on 65536 tokens beside 32
// without a prefix, 64 query heads over 8 of 128: 110 us in two groups, 350 in 33).  Of the
// prefixes, in the form for many rows, a work-group a CU, where two would have few tiles each
// (their rows' parts have to be written, read and joined) or the sequences' own tokens are as much
// work, which then runs beside them.  Measured, one a CU / two, us (64 query heads over 8 of 128,
// own tokens 50 to 400, the last row 500 to 4000):
//   sequences  shared tokens                         taken
//          16   16384    31.3 / 35.0                  one
//          64    4096    33.0 / 39.6                  one
//          64   16384    59.6 / 64.0                  one
//          32   32768    58.6 / 61.2                  one
//          32   65536   100.4 / 94.5                  two
//          64   65536   179.5 / 161.6                 two
//          64   32768   115.0 / 126.7 (much of own)   one
constexpr int64_t kMaxGroups = 4096;
constexpr int64_t kMaxRowParts = 256;          // of a prefix and of a sequence's own tokens together
struct PrefixPlan {
    int32_t prefix_rows, own_rows, row_tiles, prefix_splits, own_splits;
    int64_t prefix_blocks, own_blocks;
    size_t ml_offset, bytes;
};
int64_t pieces(int64_t units, int64_t tiles, int64_t least, int64_t most) {
    int64_t s = kGroups / units;
    if (s > tiles / least) s = tiles / least;
    return s < 1 ? 1 : s > most ? most : s;
}
bool plan_prefix(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t batch, int64_t groups, int64_t total_q, int64_t max_q,
                 int64_t max_prefix, int64_t max_own, PrefixPlan* p) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || (d != 64 && d != 128) || batch < 1 || batch > kMaxBatch ||
        groups < 1 || groups > kMaxGroups || total_q < 1 || max_q < 1 || max_prefix < 0 || max_own < 0 ||
        !product_below(total_q, q_heads, 4 * kMaxBlocks - 3))           // (the launch that joins: a wave a row)
        return false;
    if (max_q > total_q) max_q = total_q;
    if (max_prefix > (1ll << 31)) max_prefix = 1ll << 31;
    if (max_own > (1ll << 31)) max_own = 1ll << 31;
    const auto size = [](int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 128; };
    const int64_t group = q_heads / kv_heads, per_group = (total_q * group + groups - 1) / groups;
    p->own_rows = size(max_q * group);
    p->prefix_rows = p->own_rows == 128 ? 128 : size(per_group);
    if (p->prefix_rows < 128) p->prefix_rows = p->own_rows = p->prefix_rows > p->own_rows ? p->prefix_rows : p->own_rows;
    p->row_tiles = (int32_t)((max_q * group + p->own_rows - 1) / p->own_rows);
    const int64_t own_units = batch * p->row_tiles * kv_heads;                                  // (below 2^48)
    const int64_t prefix_units = (total_q * group / p->prefix_rows + groups) * kv_heads;        // at most
    const int64_t usual = (per_group + p->prefix_rows - 1) / p->prefix_rows * groups * kv_heads;
    if (own_units >= kMaxBlocks || prefix_units >= kMaxBlocks) return false;
    const int64_t tiles = (max_prefix + 63) / 64, own_tiles = (max_own + 63) / 64 + 1;
    const bool half = p->prefix_rows == 128 && (!product_below(usual, tiles, 1ll << 60) || usual * tiles < 80 * d ||
                                                own_units * own_tiles > usual * tiles);
    p->own_splits = (int32_t)pieces(own_units, own_tiles, 4, kMaxRowParts / 2);
    p->prefix_splits = (int32_t)pieces(half ? 2 * usual : usual, tiles, 4, kMaxRowParts - p->own_splits);
    p->prefix_blocks = prefix_units * p->prefix_splits;
    p->own_blocks = own_units * p->own_splits;
    if (p->prefix_blocks + p->own_blocks >= kMaxBlocks) return false;
    const int64_t parts = total_q * q_heads * (p->prefix_splits + p->own_splits);
    p->ml_offset = (size_t)(parts * d * 4);
    p->bytes = (size_t)round256((int64_t)p->ml_offset + parts * 8);
    return true;
}

}  // namespace

extern "C" {

mxq_status mxq_page_keys_nvfp4(const mxq_nvfp4_kv* cache, const int64_t* slots, int64_t tokens, const mxq_page_keys* keys,
                               void* stream) {
    mxq::KvCache c;
    mxq_status st = check_cache(cache, &c);
    if (st == MXQ_OK) st = check_keys(keys);
    if (st != MXQ_OK) return st;
    if (tokens < 0 || keys->num_pages != c.num_pages || keys->page_size != cache->page_size || keys->kv_heads != c.kv_heads ||
        keys->head_dim != c.head_dim)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return MXQ_OK;
    if (!slots) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(slots, 8)) return MXQ_ERR_MISALIGNED;
    // a wave per slot and head while those are few: each may have filled its page
    const bool few = tokens <= kMaxRows && product_below(tokens, c.kv_heads, 8192 + 1);
    const int64_t chunk = few ? 1 : keys->page_size < 64 ? keys->page_size : 64;
    if (tokens > kMaxRows || !product_below((tokens + chunk - 1) / chunk, 64ll * c.kv_heads, kMaxGridThreads - 255))
        return MXQ_ERR_UNSUPPORTED;
    mxq::PageKeysArgs a{c, slots, tokens, keys->codes, keys->scales, (int32_t)chunk, 1.0 / (130048.0 * keys->page_size)};
    return mxq::launch_page_keys(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}

size_t mxq_select_pages_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t page_size, int64_t batch,
                                             int64_t total_q, int64_t max_seq_len) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 || page_size < 16 || page_size > kMaxPageTokens ||
        (page_size & (page_size - 1)) || batch < 1 || batch > kMaxBatch || total_q < 1 || max_seq_len < 0 ||
        max_seq_len > kMaxRows || !product_below(total_q, q_heads, 1ll << 31))
        return 0;
    return plan_select(q_heads / kv_heads, kv_heads, page_size, batch, total_q, max_seq_len).bytes;
}

mxq_status mxq_select_pages_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q, const mxq_page_keys* keys,
                                  const int32_t* block_table, int64_t ld_table, int64_t table_pages, const int32_t* seq_lens,
                                  const int32_t* q_starts, int64_t batch, int64_t max_seq_len, int32_t top, int32_t first,
                                  int32_t last, int32_t* pages, void* workspace, size_t workspace_bytes, void* stream) {
    mxq_status st = check_keys(keys);
    if (st != MXQ_OK) return st;
    if (q_heads < 1 || q_heads % keys->kv_heads != 0 || total_q < 0 || batch < 1 || max_seq_len < 0 || table_pages < 0 ||
        ld_table < table_pages || first < 0 || last < 1 || top < 1 || (int64_t)first + last > top)
        return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)q_heads * keys->head_dim;
    if (ld_q < width) return MXQ_ERR_INVALID_ARGUMENT;
    if (ld_q % 8 != 0) return MXQ_ERR_MISALIGNED;
    if (top > kMaxTop) return MXQ_ERR_UNSUPPORTED;
    if (total_q == 0) return MXQ_OK;
    if (!q || !pages) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(pages, 4)) return MXQ_ERR_MISALIGNED;
    st = check_sequences(total_q, q_heads, block_table, ld_table, table_pages, seq_lens, q_starts, batch);
    if (st != MXQ_OK) return st;
    if (!extent_ok(total_q, ld_q, width) || !product_below(total_q * keys->kv_heads, top, kMaxElems) ||
        max_seq_len > kMaxRows || !product_below(total_q, 256ll * keys->kv_heads, kMaxGridThreads))  // (1024 threads only for few)
        return MXQ_ERR_UNSUPPORTED;
    const SelectPlan p = plan_select(q_heads / keys->kv_heads, keys->kv_heads, keys->page_size, batch, total_q, max_seq_len);
    if (p.bytes > 0) {
        if (!workspace) return MXQ_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < p.bytes) return MXQ_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return MXQ_ERR_MISALIGNED;
    }
    mxq::SelectArgs a{};
    a.q = q;
    a.ld_q = ld_q;
    a.codes = keys->codes;
    a.scales = keys->scales;
    a.num_pages = keys->num_pages;
    a.table = block_table;
    a.ld_table = ld_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.out = pages;
    a.table_pages = keys->num_pages == 0 ? 0 : (int32_t)table_pages;     // no page: no tokens
    a.batch = (int32_t)batch;
    a.total_q = (int32_t)total_q;
    a.kv_heads = keys->kv_heads;
    a.head_dim = keys->head_dim;
    a.group = q_heads / keys->kv_heads;
    a.page_shift = log2_of(keys->page_size);
    a.top = top;
    a.first = first;
    a.last = last;
    a.window = p.window;
    a.tokens = p.tokens;
    a.waves = p.waves;
    a.orders = static_cast<uint32_t*>(p.bytes ? workspace : nullptr);
    a.order_stride = (int32_t)p.order_stride;
    a.splits = p.splits;
    return mxq::launch_select_pages(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}

size_t mxq_attention_pages_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t page_size,
                                                int64_t total_q, int32_t top) {
    PagesPlan p;
    return plan_pages(q_heads, kv_heads, head_dim, page_size, total_q, top, &p) ? p.bytes : 0;
}

mxq_status mxq_attention_pages_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q, uint16_t* out,
                                     int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache, const int32_t* block_table,
                                     int64_t ld_table, int64_t table_pages, const int32_t* seq_lens, const int32_t* q_starts,
                                     int64_t batch, const int32_t* pages, int32_t top, float softmax_scale, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    mxq::KvCache c;
    mxq_status st = check_cache(cache, &c);
    if (st != MXQ_OK) return st;
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || total_q < 0 || batch < 1 || table_pages < 0 || ld_table < table_pages || top < 1)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)q_heads * c.head_dim;
    if (ld_q < width || ld_out < width) return MXQ_ERR_INVALID_ARGUMENT;
    if (ld_q % 8 != 0 || ld_out % 8 != 0) return MXQ_ERR_MISALIGNED;
    if (total_q == 0) return MXQ_OK;
    if (!q || !out || !pages) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(pages, 4)) return MXQ_ERR_MISALIGNED;
    st = check_sequences(total_q, q_heads, block_table, ld_table, table_pages, seq_lens, q_starts, batch);
    if (st != MXQ_OK) return st;
    PagesPlan p;
    if (!extent_ok(total_q, ld_q, width) || !extent_ok(total_q, ld_out, width) ||
        !product_below(total_q * c.kv_heads, top, kMaxElems) ||
        !plan_pages(q_heads, c.kv_heads, c.head_dim, cache->page_size, total_q, top, &p))
        return MXQ_ERR_UNSUPPORTED;
    if (p.bytes > 0) {
        if (!workspace) return MXQ_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < p.bytes) return MXQ_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned(workspace, 256)) return MXQ_ERR_MISALIGNED;
    }
    mxq::PagesAttnArgs a{};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.table = block_table;
    a.ld_table = ld_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.table_pages = c.num_pages == 0 ? 0 : (int32_t)table_pages;         // no page: no tokens
    a.batch = (int32_t)batch;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.total_q = a.max_q_len = (int32_t)total_q;
    a.scale_log2 = (double)softmax_scale * 1.44269504088896341;
    a.c = c;
    a.tile_rows = p.tile_rows;
    a.row_tiles = p.row_tiles;
    a.splits = p.splits;
    a.part_o = static_cast<float*>(p.bytes ? workspace : nullptr);
    a.part_ml = p.bytes ? reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.ml_offset) : nullptr;
    a.pages = pages;
    a.top = top;
    a.waves = p.waves;
    hipStream_t const hs = static_cast<hipStream_t>(stream);
    if (mxq::launch_attention_pages(a, hs) != hipSuccess) return MXQ_ERR_HIP;
    if (p.splits > 1 && mxq::launch_attention_join_rows(a, hs) != hipSuccess) return MXQ_ERR_HIP;
    return MXQ_OK;
}

size_t mxq_attention_prefix_nvfp4_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t batch,
                                                 int64_t groups, int64_t total_q, int64_t max_q_len, int64_t max_prefix_len,
                                                 int64_t max_own_len) {
    PrefixPlan p;
    return plan_prefix(q_heads, kv_heads, head_dim, batch, groups, total_q, max_q_len, max_prefix_len, max_own_len, &p) ? p.bytes
                                                                                                                         : 0;
}

mxq_status mxq_attention_prefix_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q, uint16_t* out,
                                      int64_t ld_out, float* lse, const mxq_nvfp4_kv* cache, const int32_t* block_table,
                                      int64_t ld_table, int64_t table_pages, const int32_t* seq_lens, const int32_t* q_starts,
                                      int64_t batch, const int32_t* group_starts, const int32_t* prefix_lens, int64_t groups,
                                      int64_t max_q_len, int64_t max_prefix_len, int64_t max_own_len, float softmax_scale,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    mxq::KvCache c;
    mxq_status st = check_cache(cache, &c);
    if (st != MXQ_OK) return st;
    if (q_heads < 1 || q_heads % c.kv_heads != 0 || total_q < 0 || batch < 1 || groups < 1 || max_q_len < 0 ||
        max_prefix_len < 0 || max_own_len < 0 || table_pages < 0 || ld_table < table_pages)
        return MXQ_ERR_INVALID_ARGUMENT;
    if (!(softmax_scale > 0.0f) || !std::isfinite(softmax_scale)) return MXQ_ERR_INVALID_ARGUMENT;
    const int64_t width = (int64_t)q_heads * c.head_dim;
    if (ld_q < width || ld_out < width) return MXQ_ERR_INVALID_ARGUMENT;
    if (ld_q % 8 != 0 || ld_out % 8 != 0) return MXQ_ERR_MISALIGNED;
    if (total_q == 0 || max_q_len == 0) return MXQ_OK;
    if (!q || !out || !group_starts || !prefix_lens) return MXQ_ERR_INVALID_ARGUMENT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(group_starts, 4) || !aligned(prefix_lens, 4))
        return MXQ_ERR_MISALIGNED;
    st = check_sequences(total_q, q_heads, block_table, ld_table, table_pages, seq_lens, q_starts, batch);
    if (st != MXQ_OK) return st;
    PrefixPlan p;
    if (!extent_ok(total_q, ld_q, width) || !extent_ok(total_q, ld_out, width) || max_q_len > kMaxRows ||
        !plan_prefix(q_heads, c.kv_heads, c.head_dim, batch, groups, total_q, max_q_len, max_prefix_len, max_own_len, &p))
        return MXQ_ERR_UNSUPPORTED;
    if (!workspace) return MXQ_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < p.bytes) return MXQ_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 256)) return MXQ_ERR_MISALIGNED;
    mxq::PrefixAttnArgs a{};
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ld_q = ld_q;
    a.ld_out = ld_out;
    a.table = block_table;
    a.ld_table = ld_table;
    a.seq_lens = seq_lens;
    a.q_starts = q_starts;
    a.table_pages = c.num_pages == 0 ? 0 : (int32_t)table_pages;         // no page: no tokens
    a.batch = (int32_t)batch;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.total_q = (int32_t)total_q;
    a.max_q_len = (int32_t)(max_q_len < total_q ? max_q_len : total_q);
    a.scale_log2 = (double)softmax_scale * 1.44269504088896341;
    a.c = c;
    a.row_tiles = p.row_tiles;
    a.splits = p.own_splits + p.prefix_splits;
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + p.ml_offset);
    a.group_starts = group_starts;
    a.prefix_lens = prefix_lens;
    a.groups = (int32_t)groups;
    a.own_splits = p.own_splits;
    a.prefix_splits = p.prefix_splits;
    a.prefix_blocks = (int32_t)p.prefix_blocks;
    a.own_blocks = (int32_t)p.own_blocks;
    a.tile_rows = p.own_rows;
    hipStream_t const hs = static_cast<hipStream_t>(stream);
    if ((p.prefix_rows == 128 ? mxq::launch_attention_ranges_prompt(a, hs) : mxq::launch_attention_ranges_rows(a, hs)) != hipSuccess)
        return MXQ_ERR_HIP;
    return mxq::launch_attention_join_rows(a, hs) == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}

}  // extern "C"
