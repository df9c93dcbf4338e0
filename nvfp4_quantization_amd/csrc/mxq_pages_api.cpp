// mxq_pages_api.cpp -- the C ABI of the calls of include/mxq.h around long and shared
// contexts (mean keys of pages, page selection, attention over listed pages): argument
// checks, launch planning and kernel launches.  Host code only; nothing here allocates,
// synchronizes, memsets or reads the environment.
#include <cmath>

#include "mxq_serve_checks.hpp"

namespace {

constexpr int64_t kMaxBatch = 65535;
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

// How attention over listed pages splits its work: a unit is (query, cached head, 16 or 32 rows
// of its group).
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
    int64_t splits = 512 / units;
    if (splits > (tiles + 7) / 8) splits = (tiles + 7) / 8;
    p->splits = (int32_t)(splits < 1 ? 1 : splits);
    if (!product_below(units * p->splits, 64 * p->waves, kMaxGridThreads)) return false;
    p->ml_offset = p->bytes = 0;
    if (p->splits > 1) {
        const int64_t parts = total_q * q_heads * p->splits;
        p->ml_offset = (size_t)(parts * d * 4);
        p->bytes = (size_t)round256((int64_t)p->ml_offset + parts * 8);
    }
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
    mxq::PageKeysArgs a{c, slots, tokens, keys->codes, keys->scales, (int32_t)chunk};
    return mxq::launch_page_keys(a, static_cast<hipStream_t>(stream)) == hipSuccess ? MXQ_OK : MXQ_ERR_HIP;
}

mxq_status mxq_select_pages_nvfp4(const uint16_t* q, int64_t ld_q, int32_t q_heads, int64_t total_q, const mxq_page_keys* keys,
                                  const int32_t* block_table, int64_t ld_table, int64_t table_pages, const int32_t* seq_lens,
                                  const int32_t* q_starts, int64_t batch, int64_t max_seq_len, int32_t top, int32_t first,
                                  int32_t last, int32_t* pages, void* stream) {
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
        !product_below(total_q, 256ll * keys->kv_heads, kMaxGridThreads))
        return MXQ_ERR_UNSUPPORTED;
    int64_t window = (max_seq_len + keys->page_size - 1) / keys->page_size;
    if (window > table_pages) window = table_pages;
    window = window < 256 ? 256 : window > 15360 ? 15360 : window;      // 60 KB
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
    a.window = (int32_t)window;
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
    a.total_q = (int32_t)total_q;
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

}  // extern "C"
