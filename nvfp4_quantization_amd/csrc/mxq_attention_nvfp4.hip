// mxq_attention_nvfp4.hip -- causal attention over the paged NVFP4 cache (gfx950): few
// query rows per cached head (decoding steps, drafts), and the join of split work.
//
// The cache is read once, straight into the operands of the matrix instructions: scores
// S^T = K Q^T and outputs O^T = V^T P^T, 64 cached tokens a step, one wave per step.
//
//  * An E2M1 value times its E4M3 block scale has at most six significant bits and lies
//    in [2^-10, 2688], so the dequantized K and V are exact in FP16: one conversion and
//    one packed FP16 product per two elements.  Q is BF16 times a power of two per row
//    (its largest element in [2^14, 2^15)): exact in FP16 down to 2^-31 of the row's largest,
//    off by half its smallest step, 2^-39 of it, below.  Scores and outputs accumulate in FP32.
//  * The tensor scales, the softmax scale and Q's power of two are one FP32 factor on the
//    scores and one on the outputs.
//  * Softmax: running maximum per row in FP32, raised only when a score exceeds it by more
//    than kSlack (the outputs are then rescaled); the weights 2^(s - m + kBias) are rounded to
//    FP16 (nearest-even) for the product with V, their FP32 values are summed.  With
//    kBias = 9 a weight keeps all 11 bits down to 2^-23 of the row's largest and adds in
//    down to 2^-33 of it.
//  * S^T leaves the matrix unit with a query row per lane column and, in lane group g of 16,
//    tokens 16 t + 4 g + e (score tile t, register e): P^T's operand layout for the second
//    product when its k index 8 g + j of half u stands for token 16 (2 u + j / 4) + 4 g +
//    j % 4.  The weights never leave their registers.
//  * V is staged per wave in LDS as it lies in the cache (two codes a byte, a token per
//    row) and read back transposed (ds_read_b64_tr_b4): a lane gets the 16 tokens of one
//    output element.  Its scales are staged as FP16, a token pair per dword.
//
// Work split: a work-group per unit (sequence, cached head), whose waves take its 64-token
// tiles in turn and join through LDS; or, where that would leave much of the chip idle, the
// tiles of all units on one line, of which every work-group takes an equal stretch, however
// ragged the lengths are: a unit inside one stretch is finished there, one cut by a stretch's
// end leaves partial outputs (maximum, sum, unnormalized FP32 rows) in the workspace for the
// join.
//
// What bounds it: two sequences of 262144 tokens, 8 heads of 128 (604 MB of cache) take 103 us, 5
// of them the join and about 6 the start (sequences, page table, first tile: three memory
// latencies one after another), so the cache streams at 6.6 TB/s of the 7.0 that a plain read
// reaches; 256 work-groups instead of 512 cost a third more, three a CU spill.  64 sequences
// of up to 8192 tokens take 70 us (333 MB): there the longest units end last, and from 512 such
// units on one far longer than the others is walked by one work-group a head, whatever it
// takes (262144 tokens among 63 of 1000: 1335 us for 375 MB).  Few or short
// sequences are latency: one of 1000 tokens takes 9.6 us on 8 CUs, 2 of them until lengths,
// page table and queries are there, 5 for two tiles a wave (the two waves of a SIMD take turns).
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

struct Lane {
    int lane, g, col;                 // g = lane / 16, col = lane % 16
};

// ---------------------------------------------------------------- a tile's loads
// A tile's 64 tokens lie in G groups that share a page each: one where pages hold 64 tokens
// or more, else four of 16 (a page of 32 holds two).  The group addresses are uniform.
//
// The table entries of a tile's groups, group lane % 4 in each lane (past the sequence the
// last token's page: nothing of such tokens is used).
__device__ __forceinline__ int32_t page_entries(const AttnArgs& a, const int32_t* table, int len, int tile, const Lane& L) {
    return table[min(tile * 64 + 16 * (L.lane & 3), len - 1) >> a.c.page_shift];
}

// Where the groups lie (page 0 for a page that may not be read).
template <int G>
struct Place {
    int64_t codes[G], scales[G];
    uint32_t bad;                     // bit t: group t's page may not be read
};
template <int G>
__device__ __forceinline__ Place<G> place(const AttnArgs& a, int32_t entries, int tile, const Lane& L) {
    Place<G> p;
    if constexpr (G == 1) {
        const int32_t e = __builtin_amdgcn_readfirstlane(entries);
        const bool ok = (uint32_t)e < (uint32_t)a.c.num_pages;
        const int64_t page = ok ? e : 0, row = (tile * 64) & ((1 << a.c.page_shift) - 1);
        p.bad = ok ? 0u : 1u;
        p.codes[0] = page * a.c.cs_page + row * a.c.cs_tok;
        p.scales[0] = page * a.c.ss_page + row * a.c.ss_tok;
    } else {
        // each lane its own group's offsets, then read from the first four: four times the
        // above took 170 scalar instructions a tile, and drafts on pages of 16 25.1 us, not
        // 22.7; one group's are as fast in the scalar unit
        const bool ok = (uint32_t)entries < (uint32_t)a.c.num_pages;
        const uint32_t page = ok ? (uint32_t)entries : 0u;
        const uint32_t row = (uint32_t)(tile * 64 + 16 * (L.lane & 3)) & ((1u << a.c.page_shift) - 1);
        const uint64_t codes = page * (uint64_t)a.c.cs_page + (uint64_t)row * (uint32_t)a.c.cs_tok;
        const uint64_t scales = page * (uint64_t)a.c.ss_page + (uint64_t)row * (uint32_t)a.c.ss_tok;
        p.bad = (uint32_t)__ballot(!ok) & 15u;
#pragma unroll
        for (int t = 0; t < G; ++t) {
            p.codes[t] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)codes, t) |
                                   (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(codes >> 32), t) << 32);
            p.scales[t] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)scales, t) |
                                    (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(scales >> 32), t) << 32);
        }
    }
    return p;
}

// The cached head's arrays.
struct Base {
    const uint8_t *kc, *ks, *vc, *vs;
};

// This lane's bytes inside a group: K's codes D / 4 g .. of token col (of the tile's 16 t +
// col with one group) and their scales; V's 16 codes-bytes of token lane / 4 (D = 64: lane /
// 2) and load j's; the scales of token `lane`.
template <int D, int G>
struct Offsets {
    uint32_t k[5 - G], ks[5 - G], v[G == 1 ? D / 32 : 1], vs;
    __device__ __forceinline__ Offsets(const AttnArgs& a, const Lane& L) {
        const uint32_t cs = (uint32_t)a.c.cs_tok, ss = (uint32_t)a.c.ss_tok;
#pragma unroll
        for (int t = 0; t < 5 - G; ++t) {
            k[t] = (uint32_t)(16 * t + L.col) * cs + L.g * (D / 8);
            ks[t] = (uint32_t)(16 * t + L.col) * ss + (D == 128 ? 4 * (L.g >> 1) : 0);
        }
        const int tok = D == 128 ? L.lane >> 2 : (L.lane >> 1) & (G == 1 ? 31 : 15);
#pragma unroll
        for (int j = 0; j < (G == 1 ? D / 32 : 1); ++j)
            v[j] = (uint32_t)((D == 128 ? 16 : 32) * j + tok) * cs + 16 * (L.lane & (D == 128 ? 3 : 1));
        vs = (uint32_t)(G == 1 ? L.lane : L.col) * ss;
    }
};

// A lane's offset that the compiler does not know: it would widen it once, ahead of the loop,
// and hold and add 64 bits in vector registers instead of the load's own base and offset.
__device__ __forceinline__ uint32_t here(uint32_t off) {
    asm("" : "+v"(off));
    return off;
}
// The cache's codes are mostly read once, by one work-group: loads that pass them through the L2
// without keeping them ("non-temporal") take 97 us instead of 110 for 64 sequences of 8192
// tokens (604 MB).  Where 7168 of those are pages that all sequences share (84 MB in all),
// loads that keep them are a little faster: 73 us against 76.
template <typename T>
__device__ __forceinline__ T stream(const uint8_t* base, uint32_t off) {
    return __builtin_nontemporal_load(reinterpret_cast<const T*>(base + here(off)));
}

// (Named members: an array indexed in the score loop would end up in scratch.)
template <int D>
struct KRegs {
    KWords<D> w0, w1, w2, w3;
    uint32_t s0, s1, s2, s3;
};
// A dword with the scales (D = 128: of lanes g and g ^ 1; D = 64: of all four), shifted down
// at its use: the compiler would copy the result of a smaller load, and wait for it there.
__device__ __forceinline__ uint32_t k_scales(const uint8_t* p, uint32_t off) {
    return *reinterpret_cast<const uint32_t*>(p + here(off));
}
template <int D, int G>
__device__ __forceinline__ void load_k(const Base& a, const Place<G>& p, const Offsets<D, G>& o, KRegs<D>& r) {
    // (which group and which offset: one of the two is always the first)
    constexpr bool kOne = G == 1;
    r.w0 = stream<KWords<D>>(a.kc + p.codes[0], o.k[0]);
    r.w1 = stream<KWords<D>>(a.kc + p.codes[kOne ? 0 : 1], o.k[kOne ? 1 : 0]);
    r.w2 = stream<KWords<D>>(a.kc + p.codes[kOne ? 0 : 2], o.k[kOne ? 2 : 0]);
    r.w3 = stream<KWords<D>>(a.kc + p.codes[kOne ? 0 : 3], o.k[kOne ? 3 : 0]);
    r.s0 = k_scales(a.ks + p.scales[0], o.ks[0]);
    r.s1 = k_scales(a.ks + p.scales[kOne ? 0 : 1], o.ks[kOne ? 1 : 0]);
    r.s2 = k_scales(a.ks + p.scales[kOne ? 0 : 2], o.ks[kOne ? 2 : 0]);
    r.s3 = k_scales(a.ks + p.scales[kOne ? 0 : 3], o.ks[kOne ? 3 : 0]);
}

template <int D>
struct VRegs {
    u32x4v w[D / 32];
    uint32_t s[D / 64];
};
template <int D, int G>
__device__ __forceinline__ void load_v(const Base& a, const Place<G>& p, const Offsets<D, G>& o, const Lane& L, VRegs<D>& r) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        if constexpr (G == 1)
            r.w[j] = stream<u32x4v>(a.vc + p.codes[0], o.v[j]);
        else if constexpr (D == 128)
            r.w[j] = stream<u32x4v>(a.vc + p.codes[j], o.v[0]);
        else
            r.w[j] = stream<u32x4v>(a.vc + (L.lane < 32 ? p.codes[2 * j] : p.codes[2 * j + 1]), o.v[0]);
    }
    int64_t s = p.scales[0];
    if constexpr (G == 4) {
        const int64_t lo = L.g & 1 ? p.scales[1] : p.scales[0], hi = L.g & 1 ? p.scales[3] : p.scales[2];
        s = L.g & 2 ? hi : lo;
    }
    const uint8_t* vs = a.vs + s + here(o.vs);
    if constexpr (D == 128) {
        const u32x2v w = *reinterpret_cast<const u32x2v*>(vs);
        r.s[0] = w.x, r.s[1] = w.y;
    } else {
        r.s[0] = *reinterpret_cast<const uint32_t*>(vs);
    }
}

// ---------------------------------------------------------------- LDS of one wave
// V codes: load j's 64 x 16 bytes at j * kVJ (16 bytes of padding keep the tokens that a
// transposing read touches in different banks); V scales as FP16 [D/16][64 tokens], lane
// group g's 16 tokens together; a byte per token for NaN V blocks.
constexpr int kVJ = 1024 + 16;
template <int D>
struct WaveLds {
    static constexpr int kScales = (D / 32) * kVJ;
    static constexpr int kNan = kScales + (D / 16) * 128;
    static constexpr int kBytes = kNan + 64;
};
// The byte of V's LDS image where element tile dt of lane group g's token k starts.
template <int D>
__device__ __forceinline__ int v_addr(int g, int k, int dt) {
    const int token = 16 * (k >> 2) + 4 * g + (k & 3);
    if constexpr (D == 128) return (token >> 4) * kVJ + (token & 15) * 64 + 8 * dt;
    return (token >> 5) * kVJ + (token & 31) * 32 + 8 * dt;
}

// The 16 tokens of element 16 dt + col of lane group g: codes, and the scales of half u.
template <int D>
__device__ __forceinline__ i32x2 v_codes(uint8_t* lds, const Lane& L, int dt) {
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i32x2*)(lds + v_addr<D>(L.g, L.col, dt)));
}
template <int D>
__device__ __forceinline__ f16x8 v_scales(const uint8_t* lds, const Lane& L, int dt, int u) {
    return *reinterpret_cast<const f16x8*>(lds + WaveLds<D>::kScales + dt * 128 + L.g * 32 + u * 16);
}

// FP16 scales of this lane's token into LDS (zero for a token that is not valid).
template <int D>
__device__ __forceinline__ void stage_scales(uint8_t* lds, const uint32_t (&vs)[D / 64], bool valid, const Lane& L) {
    f16* const p = reinterpret_cast<f16*>(lds + WaveLds<D>::kScales) + 16 * ((L.lane >> 2) & 3) + 4 * L.g + (L.lane & 3);
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
        const uint32_t s = valid ? vs[w] : 0u;
        const f16x2 a = e4m3_pair(s, false), b = e4m3_pair(s, true);
        p[(4 * w + 0) * 64] = a.x;
        p[(4 * w + 1) * 64] = a.y;
        p[(4 * w + 2) * 64] = b.x;
        p[(4 * w + 3) * 64] = b.y;
    }
}

// ---------------------------------------------------------------- the line of tiles
constexpr int kWideUnits = 256;       // units of their own that get a CU, and eight waves, each
constexpr int kLineSeqs = 1024;       // sequences of a call whose units share the line: fewer
// A unit's length on the line: its tiles and kUnitCost more for what a unit costs beside them
// (queries, the first loads' latency, the join of the waves: about one round of four
// tiles), so that stretches of many short units are not longer in time.  0 without queries.
constexpr int kUnitCost = 6;
__device__ __forceinline__ int unit_length(const AttnArgs& a, const Seq& s) {
    const int nq = min(s.nq, a.max_q_len);
    return nq > 0 ? tile_span(a, s, 0, nq - 1).n + kUnitCost : 0;
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

}  // namespace

// LINE: the units lie on the line.  (A kernel apart from units of their own, which then need
// 40 registers less: 64 drafts of four 55 -> 51 us.)
template <int D, int NT, int G, int W, bool LINE>
__global__ __launch_bounds__(64 * W, 8 / W) void k_attention_rows(const AttnArgs a) {
    constexpr int kWave = WaveLds<D>::kBytes;
    constexpr int kJoin = (D / 16) * 64 * 16;               // a wave's outputs of one column tile
    constexpr int kLds = W * (kWave > kJoin ? kWave : kJoin);
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    __shared__ float2 join[W][NT * 16];
    // of the sequences on the line: length, first query row, queries, a unit's length on it
    __shared__ int4 seqs[LINE ? kLineSeqs : 1];
    __shared__ int64_t wave_length[4];
    __shared__ int found;
    __shared__ int64_t found_before;

    const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Lane L;
    L.lane = tid & 63;
    L.g = L.lane >> 4, L.col = L.lane & 15;

    // ---- this work-group's stretch of the line [at, end), and the sequence it starts in
    int64_t at = 0, end, share = 0, before = 0;             // before: the line up to sequence b
    int b, own_head = 0;
    if constexpr (!LINE) {                                  // a unit of its own
        b = (int)(blockIdx.x / (unsigned)a.c.kv_heads);
        own_head = (int)(blockIdx.x - (unsigned)b * (unsigned)a.c.kv_heads);
        const Seq s = sequence(a, b);
        const int n = unit_length(a, s);
        if (n == 0) return;
        seqs[0] = make_int4(s.len, s.start, s.nq, n);       // (every thread the same)
        end = n;
    } else {
        // four consecutive sequences a thread
        uint32_t n[4], sum = 0;                             // (a unit is shorter than 2^26)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[j] = 0;
            if (4 * tid + j < a.batch) {
                const Seq s = sequence(a, 4 * tid + j);
                n[j] = (uint32_t)unit_length(a, s);
                seqs[4 * tid + j] = make_int4(s.len, s.start, s.nq, (int)n[j]);
            }
            sum += n[j];
        }
        const int64_t upto = wave_scan(sum & 0xFFFFu) + ((int64_t)wave_scan(sum >> 16) << 16);
        if (L.lane == 63) wave_length[wave] = upto;
        __syncthreads();
        int64_t mine = 0, line = 0;                         // before this thread's sequences; all
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w < wave) mine += wave_length[w];
            line += wave_length[w];
        }
        line *= a.c.kv_heads;
        // equal stretches of whole rounds of four waves
        share = line >> 31 ? (line + gridDim.x - 1) / gridDim.x : (int64_t)(((uint32_t)line + gridDim.x - 1) / gridDim.x);
        share = max((share + 3) / 4 * 4, (int64_t)8);
        at = (int64_t)blockIdx.x * share;
        end = min(at + share, line);
        if (at >= end) return;
        mine = (mine + (upto - sum)) * a.c.kv_heads;
        if (at >= mine && at < mine + (int64_t)sum * a.c.kv_heads) {
            int j = 0;
            while (at >= mine + (int64_t)n[j] * a.c.kv_heads) mine += (int64_t)n[j++] * a.c.kv_heads;
            found = 4 * tid + j;
            found_before = mine;
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(found);
        before = found_before;
    }

    const Offsets<D, G> off(a, L);
    const int scale_shift = D == 128 ? 16 * (L.g & 1) : 8 * L.g;         // of this lane's K scales in their dword
    uint8_t* const mine = lds + wave * kWave;

    // ---- segment by segment: the part of one unit inside the stretch
    while (at < end) {
        const int4 info = seqs[LINE ? b : 0];
        const int n_unit = info.w;
        if (n_unit == 0) {                                  // (a sequence without queries)
            ++b;
            continue;
        }
        int kvh = own_head, first = 0;
        if constexpr (LINE) {
            const int64_t ahead = at - before;
            kvh = __builtin_amdgcn_readfirstlane(ahead >> 32 ? (int)(ahead / n_unit) : (int)((uint32_t)ahead / (uint32_t)n_unit));
            first = __builtin_amdgcn_readfirstlane((int)(ahead - (int64_t)kvh * n_unit));
        }
        const int last = __builtin_amdgcn_readfirstlane((int)min((int64_t)n_unit, first + (end - at)));
        Seq seq;
        seq.len = __builtin_amdgcn_readfirstlane(info.x);
        seq.start = __builtin_amdgcn_readfirstlane(info.y);
        seq.nq = __builtin_amdgcn_readfirstlane(info.z);
        const int rows = min(seq.nq, a.max_q_len) * a.group;
        const Span span = tile_span(a, seq, 0, (rows - 1) / a.group);
        const int stop = min(last, span.n);
        const Base head{a.c.kc + kvh * a.c.cs_head, a.c.ks + kvh * a.c.ss_head, a.c.vc + kvh * a.c.cs_head,
                        a.c.vs + kvh * a.c.ss_head};

        // Loads run one round ahead of the tile that uses them (V's registers are free once
        // it is in LDS, K's after the scores), page table entries two.
        const int32_t* const table = a.table + (int64_t)b * a.ld_table;
        KRegs<D> k;
        VRegs<D> v;
        int32_t entries = 0;
        uint32_t bad = 0;                                   // groups of the loaded tile that may not be read
        int i = first + wave;
        const auto tile_of = [&](int j) { return span.tile(min(j, stop - 1)); };
        const auto entries_of = [&](int j) { return page_entries(a, table, seq.len, tile_of(j), L); };
        // Q as the second operand of S^T = K Q^T: lane (col, g) holds elements D/4 g .. of
        // row col (row 0 again past the last), scaled to FP16 by the row's power of two
        f16x8 q[NT][D / 32];
        float factor[NT];
        int pos[NT];
        const float vg = a.c.vg[kvh];
        if (first < stop) {
            // The queries are asked for ahead of the first tile, which has to wait for its page
            // table entries: loads come back in order, and so the queries are made ready while
            // the tile is on its way.
            const int32_t e = entries_of(i);
            entries = entries_of(i + W);
            u32x4v w[NT][D / 32];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = n * 16 + L.col < rows ? n * 16 + L.col : 0;
                const int qi = r / a.group, h = kvh * a.group + (r - qi * a.group);
                pos[n] = n * 16 + L.col < rows ? max(seq.len - seq.nq + qi, -1) : -1;
                const uint16_t* src = a.q + (int64_t)(seq.start + qi) * a.ld_q + (int64_t)h * D + L.g * (D / 4);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) w[n][c] = reinterpret_cast<const u32x4v*>(src)[c];
            }
            const float kg = a.c.kg[kvh];
            __builtin_amdgcn_sched_barrier(0);
            const Place<G> where = place<G>(a, e, tile_of(i), L);
            load_v<D, G>(head, where, off, L, v);
            load_k<D, G>(head, where, off, k);
            bad = where.bad;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    top = absmax_pk(absmax_pk(absmax_pk(absmax_pk(top, w[n][c].x), w[n][c].y), w[n][c].z), w[n][c].w);
                top = fold_pk(top);
                top = max(top, shfl_xor_u32(top, 16));
                top = max(top, shfl_xor_u32(top, 32));
                const float up = q_power(top, factor[n]);
                factor[n] = score_factor(a, factor[n], kg);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) q[n][c] = q_operand(w[n][c], up);
            }
        }

        f32x4 o[NT][D / 16];
        float m[NT], l[NT];
        uint32_t nan_blocks[NT];                            // V blocks that this lane's tokens make NaN
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n] = kFloor;
            l[n] = 0.0f;
            nan_blocks[n] = 0;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) o[n][dt] = f32x4{0, 0, 0, 0};
        }

        for (; i < stop; i += W) {
            const int t0 = span.tile(i) * 64;
            // V and its scales to LDS; tokens past the sequence or of unreadable pages get
            // zero scales, so whatever lies there stays out
            const uint32_t unread = bad;
            const bool valid = !((unread >> (G == 1 ? 0 : L.g)) & 1) && t0 + L.lane < seq.len;
            bool nan_here = false;
#pragma unroll
            for (int w = 0; w < D / 64; ++w) nan_here |= has_nan_scale(v.s[w]);
            if (__any(nan_here && valid)) {                 // (rare) note NaN V blocks, stage them as zero
                uint32_t blocks = 0;
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    const uint32_t hit = (((v.s[w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
                    v.s[w] &= ~(hit * 0xFFu);
                    blocks |= ((hit | hit >> 7 | hit >> 14 | hit >> 21) & 0xFu) << (4 * w);
                }
                mine[WaveLds<D>::kNan + L.lane] = (uint8_t)(valid ? blocks : 0u);
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {
                    const int tok = 16 * (j >> 2) + 4 * L.g + (j & 3);
                    const uint32_t x = mine[WaveLds<D>::kNan + tok];
#pragma unroll
                    for (int n = 0; n < NT; ++n) nan_blocks[n] |= sees(a, pos[n], t0 + tok) ? x : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) *reinterpret_cast<u32x4v*>(mine + j * kVJ + L.lane * 16) = v.w[j];
            stage_scales<D>(mine, v.s, valid, L);
            // (past the stretch the last tile again: a branch around a load would make every
            // later wait for loads a wait for all of them)
            const Place<G> where = place<G>(a, entries, tile_of(i + W), L);
            load_v<D, G>(head, where, off, L, v);
            entries = entries_of(i + 2 * W);
            bad = where.bad;

            // scores of 64 tokens
            f32x4 x[NT][4];
            const auto score = [&](int t, KWords<D> w, uint32_t scales) {
                // a page that may not be read: NaN scales, so that rows that see its tokens are NaN
                f16x8 kk[D / 32];
                dequant_row<D>(w, (unread >> (G == 1 ? 0 : t)) & 1 ? 0x7F7Fu : scales >> scale_shift, kk);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    x[n][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < D / 32; ++c)
                        x[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk[c], q[n][c], x[n][t], 0, 0, 0);
                }
            };
            score(0, k.w0, k.s0);
            __builtin_amdgcn_sched_barrier(0);
            score(1, k.w1, k.s1);
            __builtin_amdgcn_sched_barrier(0);
            score(2, k.w2, k.s2);
            __builtin_amdgcn_sched_barrier(0);
            score(3, k.w3, k.s3);
            __builtin_amdgcn_sched_barrier(0);
            load_k<D, G>(head, where, off, k);

            // masks only where an edge crosses the tile (uniform)
            if (t0 + 63 > span.p_lo || (a.window && t0 <= (int64_t)span.p_hi - a.window)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    each_seen<16>(a, pos[n], t0 + 4 * L.g, [](int e) { return 16 * (e >> 2) + (e & 3); }, [&](int e, bool seen) {
                        x[n][e >> 2][e & 3] = seen ? x[n][e >> 2][e & 3] : -__builtin_inff();
                    });
            }
            f16x8 p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) softmax_step<D>(x[n], factor[n], m[n], l[n], o[n], p[n]);

            // O^T += V^T P^T, the operands of kAhead element tiles read before they are used
            // (the order is fixed: the compiler would read all of them first, and spill)
            constexpr int kAhead = NT == 1 ? 2 : 1;
            i32x2 c[kAhead];
            f16x8 s0[kAhead], s1[kAhead];
#pragma unroll
            for (int dt = 0; dt < kAhead; ++dt) {
                c[dt] = v_codes<D>(mine, L, dt);
                s0[dt] = v_scales<D>(mine, L, dt, 0);
                s1[dt] = v_scales<D>(mine, L, dt, 1);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                const int z = dt % kAhead;
                const f16x8 v0 = e2m1_8(c[z].x) * s0[z], v1 = e2m1_8(c[z].y) * s1[z];
                if (dt + kAhead < D / 16) {
                    c[z] = v_codes<D>(mine, L, dt + kAhead);
                    s0[z] = v_scales<D>(mine, L, dt + kAhead, 0);
                    s1[z] = v_scales<D>(mine, L, dt + kAhead, 1);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, p[n][0], o[n][dt], 0, 0, 0);
                    o[n][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, p[n][1], o[n][dt], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }

        // ---- join the waves
        __syncthreads();                                    // the staging areas are free
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n] += shfl_xor_f32(l[n], 16);
            l[n] += shfl_xor_f32(l[n], 32);
            nan_blocks[n] |= shfl_xor_u32(nan_blocks[n], 16);
            nan_blocks[n] |= shfl_xor_u32(nan_blocks[n], 32);
            if (__any(nan_blocks[n] != 0)) {
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt)
                    if ((nan_blocks[n] >> dt) & 1) o[n][dt] = f32x4{0, 0, 0, 0} + __builtin_nanf("");
            }
            if (L.g == 0) join[wave][n * 16 + L.col] = make_float2(m[n], l[n]);
        }
        const bool whole = first == 0 && last == n_unit;
        // a cut unit's part: slot 1 of the work-group where it begins, slot 0 of those it goes on in
        const int64_t slot = 2 * (int64_t)blockIdx.x + (first == 0 ? 1 : 0);
        if (LINE && first == 0 && tid == 0) {
            const int64_t rest = before + (int64_t)(kvh + 1) * n_unit - end;                 // past this stretch
            a.desc[(int64_t)b * a.c.kv_heads + kvh] =
                make_int2((int)blockIdx.x, whole ? 0 : (int)((rest + share - 1) / share) + 1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4* const all = reinterpret_cast<f32x4*>(lds);
            if (n) __syncthreads();
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) all[(wave * (D / 16) + dt) * 64 + L.lane] = o[n][dt];
            __syncthreads();
            float top = kFloor, total = 0.0f, f[W];
#pragma unroll
            for (int w = 0; w < W; ++w) top = __builtin_fmaxf(top, join[w][n * 16 + L.col].x);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                f[w] = __builtin_amdgcn_exp2f(join[w][n * 16 + L.col].x - top);
                total += join[w][n * 16 + L.col].y * f[w];
            }
            const int r = n * 16 + L.col;
            const bool live = r < rows;
#pragma unroll
            for (int j = 0; j < (D / 16 + W - 1) / W; ++j) {
                const int dt = wave * (D / 16 >= W ? D / 16 / W : 1) + j;
                if (dt >= D / 16) break;
                f32x4 y = all[dt * 64 + L.lane] * f[0];
#pragma unroll
                for (int w = 1; w < W; ++w) y += all[(w * (D / 16) + dt) * 64 + L.lane] * f[w];
                const int d0 = 16 * dt + 4 * L.g;
                if (!live) continue;
                if (whole)
                    store_finished<D>(a, seq, kvh, r, d0, y, top, total, vg);
                else
                    store_part<D>(a, slot * (NT * 16) + r, d0, y, top, total);
            }
        }
        __syncthreads();                                    // before the next segment's staging
        at += last - first;
        if (last == n_unit && kvh == a.c.kv_heads - 1) {
            before += (int64_t)n_unit * a.c.kv_heads;
            ++b;
        }
    }
}

// Joins a query row's parts: W waves per row (a work-group has four).  Lanes first turn the
// parts' maxima and sums into weights (LDS), then each wave adds every W-th part, all of a
// lane's loads independent of one another.  parts: at most kMaxParts; part 0 at `first`, the
// others `step` apart from `rest` on (rows).
template <int D, int W>
__device__ __forceinline__ void join_row(const AttnArgs& a, const Seq& seq, int kvh, int64_t r, int parts, int64_t first,
                                         int64_t rest, int64_t step) {
    constexpr int kRows = 4 / W;                             // rows of a work-group
    __shared__ float weight[kRows][kMaxParts];
    __shared__ float wave_sum[4], wave_top[4];
    __shared__ float part[4][D];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int mine = tid / (64 * W), t = tid % (64 * W), w0 = wave % W;
    const auto row_of = [&](int s) { return s == 0 ? first : rest + (s - 1) * step; };
    // (the first parts' rows are on their way while the weights are made)
    constexpr int kAhead = 8;
    float ahead[kAhead][D / 64];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const float* src = a.part_o + row_of(min(w0 + W * j, parts - 1)) * D + lane * (D / 64);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) ahead[j][e] = src[e];
    }
    const float vg = a.c.vg[kvh];
    float2 ml[kMaxParts / (64 * W)];
    float top = kFloor;
#pragma unroll
    for (int j = 0; j < kMaxParts / (64 * W); ++j) {
        const int s = t + 64 * W * j;
        ml[j] = s < parts ? a.part_ml[row_of(s)] : make_float2(kFloor, 0.0f);
        top = __builtin_fmaxf(top, ml[j].x);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = __builtin_fmaxf(top, shfl_xor_f32(top, o));
    if (W > 1) {
        if (lane == 0) wave_top[wave] = top;
        __syncthreads();
        top = __builtin_fmaxf(__builtin_fmaxf(wave_top[0], wave_top[1]), __builtin_fmaxf(wave_top[2], wave_top[3]));
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxParts / (64 * W); ++j) {
        const float f = __builtin_amdgcn_exp2f(ml[j].x - top);
        weight[mine][t + 64 * W * j] = f;
        sum += ml[j].y * f;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += shfl_xor_f32(sum, o);
    if (W > 1) {
        if (lane == 0) wave_sum[wave] = sum;
        __syncthreads();
        sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
    }
    float v[D / 64] = {};
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
        const float w = w0 + W * j < parts ? weight[mine][w0 + W * j] : 0.0f;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) v[e] += w0 + W * j < parts ? ahead[j][e] * w : 0.0f;
    }
#pragma unroll 8
    for (int s = w0 + W * kAhead; s < parts; s += W) {
        const float w = weight[mine][s];
        const float* src = a.part_o + row_of(s) * D + lane * (D / 64);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) v[j] += src[j] * w;
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) part[wave][lane * (D / 64) + j] = v[j];
    if (W > 1) __syncthreads();
    if (t >= D / 4) return;
    f32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = 4 * t + j;
        y[j] = W > 1 ? (part[0][d] + part[1][d]) + (part[2][d] + part[3][d]) : part[wave][d];
    }
    store_finished<D>(a, seq, kvh, r, 4 * t, y, top, sum, vg);
}

// Rows of a unit on the line that can hold queries, a multiple of 4.
__host__ __device__ __forceinline__ int join_rows(const AttnArgs& a) {
    const int64_t rows = ((int64_t)a.max_q_len * a.group + 3) / 4 * 4;
    return rows < a.tile_rows ? (int)rows : a.tile_rows;
}

// The units that the line's stretches cut (desc: where the unit begins, and its parts).
// W = 4: a work-group per row; W = 1: a wave.
template <int D, int W>
__global__ __launch_bounds__(256) void k_attention_join_units(const AttnArgs a) {
    const int64_t item = (int64_t)blockIdx.x * (4 / W) + (threadIdx.x >> 6) / W;
    const int rows = join_rows(a);
    const int64_t unit = item / rows;
    const int r = (int)(item - unit * rows);
    int2 d = a.desc[unit];
    const int b = (int)(unit / a.c.kv_heads), kvh = (int)(unit - (int64_t)b * a.c.kv_heads);
    const Seq seq = sequence(a, b);
    if (r >= min(seq.nq, a.max_q_len) * a.group) return;
    d.x = min(max(d.x, 0), a.splits - 1);                    // (in bounds whatever the workspace holds)
    d.y = min(max(d.y, 0), a.splits - d.x);
    if (d.y == 0) return;                                    // finished by its work-group
    const int64_t at = 2 * (int64_t)d.x;
    const int parts = d.y;
    join_row<D, W>(a, seq, kvh, r, parts, (at + 1) * a.tile_rows + r, (at + 2) * a.tile_rows + r, 2 * (int64_t)a.tile_rows);
}

// The units that the form for many rows split.  W as above.
template <int D, int W>
__global__ __launch_bounds__(256) void k_attention_join_splits(const AttnArgs a) {
    const int64_t item = (int64_t)blockIdx.x * (4 / W) + (threadIdx.x >> 6) / W;
    const int64_t unit = item / a.tile_rows;
    const int r = (int)(item - unit * a.tile_rows);
    const int64_t bt = unit / a.c.kv_heads;
    const int kvh = (int)(unit - bt * a.c.kv_heads);
    const int b = (int)(bt / a.row_tiles), rt = (int)(bt - (int64_t)b * a.row_tiles);
    const Seq seq = sequence(a, b);
    const int64_t rows = min((int64_t)seq.nq, (int64_t)a.max_q_len) * a.group;
    const int64_t r0 = (int64_t)rt * a.tile_rows;
    if (r0 + r >= rows) return;
    const int64_t r1 = min(r0 + a.tile_rows, rows) - 1;
    const int used = splits_used(a, tile_span(a, seq, (int)(r0 / a.group), (int)(r1 / a.group)).n);
    if (used <= 1) return;                                   // written by the first kernel
    const int64_t at = unit * a.splits * a.tile_rows + r;
    join_row<D, W>(a, seq, kvh, r0 + r, used, at, at + a.tile_rows, a.tile_rows);
}

// Units of their own get eight waves each while there is a CU for each: 256 units of 96
// ragged tiles 34 us instead of 39, 8 units of 32 tiles 14.5 instead of 15.7; but 512 units of
// 16 tiles 23 instead of 18.
template <int D, int NT, int G>
static void launch_rows_pages(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.splits);
    if (a.desc)
        hipLaunchKernelGGL((k_attention_rows<D, NT, G, 4, true>), grid, dim3(256), 0, stream, a);
    else if (a.splits <= kWideUnits)
        hipLaunchKernelGGL((k_attention_rows<D, NT, G, 8, false>), grid, dim3(512), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attention_rows<D, NT, G, 4, false>), grid, dim3(256), 0, stream, a);
}
template <int D, int NT>
static void launch_rows(const AttnArgs& a, hipStream_t stream) {
    if (a.c.page_shift >= 6)
        launch_rows_pages<D, NT, 1>(a, stream);
    else
        launch_rows_pages<D, NT, 4>(a, stream);
}
hipError_t launch_attention_rows(const AttnArgs& a, hipStream_t stream) {
    if (a.c.head_dim == 128) {
        if (a.tile_rows == 16)
            launch_rows<128, 1>(a, stream);
        else
            launch_rows<128, 2>(a, stream);
    } else {
        if (a.tile_rows == 16)
            launch_rows<64, 1>(a, stream);
        else
            launch_rows<64, 2>(a, stream);
    }
    return hipGetLastError();
}

// A row has at most `splits` parts, or on the line gridDim / units on average.  Few are added
// by a wave alone, with a fourth of the work-groups (a chunk of 512 queries in 4 parts: 12 us
// against 38; the other way round two sequences in 32 parts each: 5 us against 8).
constexpr int kWaveParts = 4;
template <int D>
static void launch_join(const AttnArgs& a, hipStream_t stream) {
    const int64_t units = (int64_t)a.batch * a.row_tiles * a.c.kv_heads, rows = units * (a.desc ? join_rows(a) : a.tile_rows);
    const dim3 each((unsigned)rows), four((unsigned)(rows / 4));
    if (a.desc && units * kWaveParts < a.splits)
        hipLaunchKernelGGL((k_attention_join_units<D, 4>), each, dim3(256), 0, stream, a);
    else if (a.desc)
        hipLaunchKernelGGL((k_attention_join_units<D, 1>), four, dim3(256), 0, stream, a);
    else if (a.splits > kWaveParts)
        hipLaunchKernelGGL((k_attention_join_splits<D, 4>), each, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attention_join_splits<D, 1>), four, dim3(256), 0, stream, a);
}
hipError_t launch_attention_join(const AttnArgs& a, hipStream_t stream) {
    if (a.c.head_dim == 128)
        launch_join<128>(a, stream);
    else
        launch_join<64>(a, stream);
    return hipGetLastError();
}

}  // namespace mxq
