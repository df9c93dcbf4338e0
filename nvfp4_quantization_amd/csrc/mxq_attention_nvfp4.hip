// mxq_attention_nvfp4.hip -- causal attention over the paged NVFP4 cache (gfx950): few
// query rows per cached head (decoding steps, drafts), and the join of split work.
//
// The cache is read once, straight into the operands of the matrix instructions: scores
// S^T = K Q^T and outputs O^T = V^T P^T, 64 cached tokens a step, one wave per step.
//
//  * An E2M1 value times its E4M3 block scale has at most six significant bits and lies
//    in [2^-10, 2688], so the dequantized K and V are exact in FP16: one conversion and
//    one packed FP16 product per two elements.  Q is BF16 times a power of two per row
//    (its largest element in [2^14, 2^15)), exact in FP16 but for elements 2^-28 below the
//    row's largest.  Scores and outputs accumulate in FP32.
//  * The tensor scales, the softmax scale and Q's power of two are one FP32 factor on the
//    scores and one on the outputs.
//  * Softmax: running maximum per row in FP32, raised only when a score exceeds it by more
//    than 2^kSlack (the outputs are then rescaled); the weights 2^(s - m + kBias) are rounded to
//    FP16 (nearest-even) for the product with V, their FP32 values are summed.  With
//    kBias = 9 a weight keeps all 11 bits down to 2^-23 of the row's largest and adds in
//    down to 2^-33 of it.
//  * S^T leaves the matrix unit with a query row per lane column and four tokens per lane
//    register group, which is P^T's operand layout for the second product when score
//    tile t row 4g + i is token 16 g + 4 t + i: K's rows are loaded in that order, and
//    the weights never leave their registers.
//  * V is staged per wave in LDS as it lies in the cache (two codes a byte, a token per
//    row) and read back transposed (ds_read_b64_tr_b4): a lane gets the 16 tokens of one
//    output element.  Its scales are staged as FP16, a token pair per dword.
//
// A work-group of four waves takes one chunk of one (sequence, cached head, rows of
// queries) and interleaves its 64-token tiles over the waves; the waves join through LDS.
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

// ---------------------------------------------------------------- a step's loads
struct Lane {
    int lane, g, q, low;              // g = lane / 16, q = (lane / 4) % 4, low = lane % 4
};

// The page of the 16 tokens 16 q .. of a tile that this lane loads, raw from the table
// (0 past the sequence: nothing of such tokens is used).
__device__ __forceinline__ int32_t page_entry(const AttnArgs& a, const int32_t* table, int len, int tile, const Lane& L) {
    const int tg = tile * 64 + 16 * L.q;
    return tg < len ? table[tg >> a.c.page_shift] : 0;
}

// Where those tokens' codes and scales lie (page 0 for a page that may not be read).
struct Place {
    int64_t codes, scales;
    bool ok;
};
__device__ __forceinline__ Place place(const AttnArgs& a, int32_t entry, int tile, int kvh, const Lane& L) {
    Place p;
    p.ok = (uint32_t)entry < (uint32_t)a.c.num_pages;
    const int64_t page = p.ok ? entry : 0;
    const int64_t row = (tile * 64 + 16 * L.q) & ((1 << a.c.page_shift) - 1);
    p.codes = page * a.c.cs_page + kvh * a.c.cs_head + row * a.c.cs_tok;
    p.scales = page * a.c.ss_page + kvh * a.c.ss_head + row * a.c.ss_tok;
    return p;
}

// (Named members: an array indexed in the long score loop would end up in scratch.)
template <int D>
struct KRegs {
    KWords<D> w0, w1, w2, w3;         // codes of this lane's K rows (score tile t): D / 4 elements each
    uint32_t s0, s1, s2, s3;          // their scales (D / 64 bytes)
};
template <int D>
__device__ __forceinline__ uint32_t k_scales(const uint8_t* p) {
    if constexpr (D == 128) return *reinterpret_cast<const uint16_t*>(p);
    return *p;
}
template <int D>
__device__ __forceinline__ void load_k(const AttnArgs& a, const Place& p, const Lane& L, KRegs<D>& r) {
    const uint8_t* kc = a.c.kc + p.codes + L.low * a.c.cs_tok + L.g * (D / 8);
    const uint8_t* ks = a.c.ks + p.scales + L.low * a.c.ss_tok + L.g * (D / 64);
    r.w0 = *reinterpret_cast<const KWords<D>*>(kc);
    r.w1 = *reinterpret_cast<const KWords<D>*>(kc + 4 * a.c.cs_tok);
    r.w2 = *reinterpret_cast<const KWords<D>*>(kc + 8 * a.c.cs_tok);
    r.w3 = *reinterpret_cast<const KWords<D>*>(kc + 12 * a.c.cs_tok);
    r.s0 = k_scales<D>(ks);
    r.s1 = k_scales<D>(ks + 4 * a.c.ss_tok);
    r.s2 = k_scales<D>(ks + 8 * a.c.ss_tok);
    r.s3 = k_scales<D>(ks + 12 * a.c.ss_tok);
}

template <int D>
struct VRegs {
    u32x4v w[D / 32];                 // codes on their way to LDS
    uint32_t s[D / 64];               // scales of this lane's token
    bool ok;
};
template <int D>
__device__ __forceinline__ void load_v(const AttnArgs& a, const Place& p, const Lane& L, VRegs<D>& r) {
    const uint8_t* vc = a.c.vc + p.codes;
    const int sw = L.low ^ L.g;                             // 16-byte chunk order of the staging
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const int tok = D == 128 ? 4 * j + L.g : 8 * j + 2 * L.g + (sw >> 1);
        const int chunk = D == 128 ? sw : sw & 1;
        r.w[j] = *reinterpret_cast<const u32x4v*>(vc + tok * a.c.cs_tok + 16 * chunk);
    }
    const uint8_t* vs = a.c.vs + p.scales + (4 * L.g + L.low) * a.c.ss_tok;
    if constexpr (D == 128) {
        const u32x2v w = *reinterpret_cast<const u32x2v*>(vs);
        r.s[0] = w.x, r.s[1] = w.y;
    } else {
        r.s[0] = *reinterpret_cast<const uint32_t*>(vs);
    }
    r.ok = p.ok;
}

// ---------------------------------------------------------------- LDS of one wave
// V codes: load j's 64 x 16 bytes at j * kVJ (64 bytes of padding keep the 16 tokens that
// a transposing read touches in different banks); V scales as FP16 [D/16][64 tokens].
constexpr int kVJ = 1024 + 64;
template <int D>
struct WaveLds {
    static constexpr int kScales = (D / 32) * kVJ;
    static constexpr int kBytes = kScales + (D / 16) * 128;
};
// The byte of V's LDS image where token k of lane group G starts its element tile dt.
template <int D>
__device__ __forceinline__ int v_addr(int G, int k, int dt) {
    if constexpr (D == 128) return (k >> 2) * kVJ + 256 * (k & 3) + 64 * G + 16 * ((dt >> 1) ^ (k & 3)) + 8 * (dt & 1);
    const int g = (k >> 1) & 3;
    return (k >> 3) * kVJ + 256 * g + 64 * G + 16 * ((2 * (k & 1) + (dt >> 1)) ^ g) + 8 * (dt & 1);
}

// FP16 scales of this lane's token into LDS (zero for a token that is not valid).
template <int D>
__device__ __forceinline__ void stage_scales(uint8_t* lds, const uint32_t (&vs)[D / 64], bool valid, const Lane& L) {
    f16* const p = reinterpret_cast<f16*>(lds + WaveLds<D>::kScales) + 16 * L.q + 4 * L.g + L.low;
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
        const f16x2 a = e4m3_pair(vs[w], false), b = e4m3_pair(vs[w], true);
        const f16 z = (f16)0.0f;
        p[(4 * w + 0) * 64] = valid ? a.x : z;
        p[(4 * w + 1) * 64] = valid ? a.y : z;
        p[(4 * w + 2) * 64] = valid ? b.x : z;
        p[(4 * w + 3) * 64] = valid ? b.y : z;
    }
}

// This lane's staged scales with NaN ones replaced by zero.
template <int D>
__device__ __forceinline__ void clean_scales(uint8_t* lds, const Lane& L) {
    f16* const p = reinterpret_cast<f16*>(lds + WaveLds<D>::kScales) + 16 * L.q + 4 * L.g + L.low;
#pragma unroll
    for (int b = 0; b < D / 16; ++b) {
        const f16 v = p[b * 64];
        p[b * 64] = v != v ? (f16)0.0f : v;
    }
}

}  // namespace

template <int D, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 3 : 2) void k_attention_rows(const AttnArgs a) {
    constexpr int kWave = WaveLds<D>::kBytes;
    constexpr int kJoin = (D / 16) * 64 * 16;               // a wave's outputs of one column tile
    constexpr int kLds = 4 * kWave > 4 * kJoin ? 4 * kWave : 4 * kJoin;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    __shared__ float2 join[4][NT * 16];

    const int wave = (int)threadIdx.x >> 6;
    Lane L;
    L.lane = (int)threadIdx.x & 63;
    L.g = L.lane >> 4, L.q = (L.lane >> 2) & 3, L.low = L.lane & 3;
    const int col = L.lane & 15;

    const int split = (int)(blockIdx.x % (unsigned)a.splits);
    const int unit = (int)(blockIdx.x / (unsigned)a.splits);
    const int kvh = unit % a.c.kv_heads, bt = unit / a.c.kv_heads;
    const int b = bt / a.row_tiles, r0 = (bt - b * a.row_tiles) * (NT * 16);
    const Seq seq = sequence(a, b);
    const int rows = min(min(seq.nq, a.max_q_len) * a.group - r0, NT * 16);      // of this unit
    if (rows <= 0) return;
    const Span span = tile_span(a, seq, r0 / a.group, (r0 + rows - 1) / a.group);
    const int used = splits_used(a, span.n);
    if (split >= used) return;
    const int first = split * a.chunk, last = split == used - 1 ? span.n : first + a.chunk;

    // Q as the second operand of S^T = K Q^T: lane (col, g) holds elements D/4 g .. of row
    // col, scaled to FP16 by the row's power of two
    f16x8 q[NT][D / 32];
    float factor[NT];
    int pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = n * 16 + col;
        const bool live = r < rows;
        const int qi = live ? (r0 + r) / a.group : 0, head = kvh * a.group + (live ? r0 + r - qi * a.group : 0);
        pos[n] = live ? max(seq.len - seq.nq + qi, -1) : -1;
        const uint16_t* src = a.q + (int64_t)(seq.start + qi) * a.ld_q + (int64_t)head * D + L.g * (D / 4);
        u32x4v w[D / 32];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            w[i] = live ? reinterpret_cast<const u32x4v*>(src)[i] : u32x4v{0, 0, 0, 0};
            top = absmax_pk(absmax_pk(absmax_pk(absmax_pk(top, w[i].x), w[i].y), w[i].z), w[i].w);
        }
        top = fold_pk(top);
        top = max(top, shfl_xor_u32(top, 16));
        top = max(top, shfl_xor_u32(top, 32));
        const float up = q_power(top, factor[n]);
        factor[n] *= a.scale_log2 * a.c.kg[kvh];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) q[n][i] = q_operand(w[i], up);
    }

    f32x4 o[NT][D / 16];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kFloor;
        l[n] = 0.0f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) o[n][dt] = f32x4{0, 0, 0, 0};
    }
    uint8_t* const mine = lds + wave * kWave;
    const int32_t* const table = a.table + (int64_t)b * a.ld_table;

    // Loads run ahead of the step that uses them: the page table entry by two steps, V by
    // one (its registers are free once it is in LDS), K by one (after its use).
    KRegs<D> k;
    VRegs<D> v;
    int i = first + wave;
    int32_t entry = 0;
    if (i < last) {
        const Place at = place(a, page_entry(a, table, seq.len, span.tile(i), L), span.tile(i), kvh, L);
        load_v<D>(a, at, L, v);
        load_k<D>(a, at, L, k);
        if (i + 4 < last) entry = page_entry(a, table, seq.len, span.tile(i + 4), L);
    }
    while (i < last) {
        const int tile = span.tile(i), t0 = tile * 64;
        // V and its scales to LDS; tokens past the sequence or of unreadable pages get
        // zero scales, so whatever lies there stays out
        const bool v_valid = v.ok && t0 + 16 * L.q + 4 * L.g + L.low < seq.len;
        const uint64_t bad = __ballot(!v.ok);
        bool nan_here = false;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) nan_here |= has_nan_scale(v.s[w]);
        const bool nan_v = __any(nan_here && v_valid);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) *reinterpret_cast<u32x4v*>(mine + j * kVJ + L.lane * 16) = v.w[j];
        stage_scales<D>(mine, v.s, v_valid, L);
        const int next = i + 4;
        Place at;
        if (next < last) {
            at = place(a, entry, span.tile(next), kvh, L);
            load_v<D>(a, at, L, v);
            if (next + 4 < last) entry = page_entry(a, table, seq.len, span.tile(next + 4), L);
        }

        // scores of 64 tokens: tile t row 4 g' + i' is token 16 g' + 4 t + i'
        f32x4 x[NT][4];
        const auto score = [&](int t, KWords<D> w, uint32_t scales) {
            f16x8 kk[D / 32];
            dequant_row<D>(w, scales, kk);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    x[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk[c], q[n][c], x[n][t], 0, 0, 0);
            }
        };
        score(0, k.w0, k.s0);
        score(1, k.w1, k.s1);
        score(2, k.w2, k.s2);
        score(3, k.w3, k.s3);
        if (next < last) load_k<D>(a, at, L, k);

        f16x8 p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // masks only where an edge crosses the tile (uniform over the wave)
            const bool edge = t0 + 63 > span.p_lo || (a.window && t0 <= (int64_t)span.p_hi - a.window) || bad != 0;
            if (edge) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = t0 + 16 * L.g + 4 * t + e;
                        const bool see = tok <= pos[n] && (!a.window || tok > pos[n] - a.window || tok < a.sinks);
                        if ((bad >> (4 * L.g)) & 1) x[n][t][e] = __builtin_nanf("");
                        x[n][t][e] = see ? x[n][t][e] : -__builtin_inff();
                    }
            }
            softmax_step<D>(x[n], factor[n], m[n], l[n], o[n], p[n]);
        }

        if (nan_v) {
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                const f16x8* sc = reinterpret_cast<const f16x8*>(mine + WaveLds<D>::kScales + dt * 128 + L.g * 32);
                f16x8 hit[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const f16x8 s = sc[u];
#pragma unroll
                    for (int j = 0; j < 8; ++j) hit[u][j] = s[j] != s[j] ? (f16)1.0f : (f16)0.0f;
                }
                spread_nan<NT, D / 16>(hit, dt, p, o);
            }
            clean_scales<D>(mine, L);
        }
        // O^T += V^T P^T
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
            const i32x2 c = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                (__attribute__((address_space(3))) i32x2*)(mine + v_addr<D>(L.g, col, dt)));
            const f16x8* sc = reinterpret_cast<const f16x8*>(mine + WaveLds<D>::kScales + dt * 128 + L.g * 32);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const f16x8 vv = e2m1_8(u ? c.y : c.x) * sc[u];
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    o[n][dt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[n][u], o[n][dt], 0, 0, 0);
            }
        }
        i = next;
    }

    // join the four waves
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        l[n] += shfl_xor_f32(l[n], 16);
        l[n] += shfl_xor_f32(l[n], 32);
        if (L.g == 0) join[wave][n * 16 + col] = make_float2(m[n], l[n]);
    }
    const float vg = a.c.vg[kvh];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        __syncthreads();
        float top = kFloor, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, join[w][n * 16 + col].x);
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += join[w][n * 16 + col].y * __builtin_amdgcn_exp2f(join[w][n * 16 + col].x - top);
        const float f = __builtin_amdgcn_exp2f(m[n] - top);
        f32x4* const all = reinterpret_cast<f32x4*>(lds);
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) all[(wave * (D / 16) + dt) * 64 + L.lane] = o[n][dt] * f;
        __syncthreads();
        const int r = n * 16 + col;
        const bool live = r < rows;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            const int dt = wave * (D / 64) + j;
            f32x4 v = all[dt * 64 + L.lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) v += all[(w * (D / 16) + dt) * 64 + L.lane];
            if (live) store_rows<D>(a, seq, unit, kvh, split, used, NT * 16, r0 + r, 16 * dt + 4 * L.g, v, top, sum, vg);
        }
    }
}

// Joins the splits of every query row: a work-group per row.  Its lanes first turn the
// splits' maxima and sums into weights (LDS), then each wave adds every fourth split, all
// of a lane's loads independent of one another.
template <int D>
__global__ __launch_bounds__(256) void k_attention_join(const AttnArgs a) {
    __shared__ float weight[kMaxSplits];
    __shared__ float wave_sum[4], wave_top[4];
    __shared__ float part[4][D];
    const int64_t unit = blockIdx.x / (unsigned)a.tile_rows;
    const int r = (int)(blockIdx.x % (unsigned)a.tile_rows);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int kvh = (int)(unit % a.c.kv_heads);
    const int64_t bt = unit / a.c.kv_heads;
    const int b = (int)(bt / a.row_tiles), rt = (int)(bt - (int64_t)b * a.row_tiles);
    const Seq seq = sequence(a, b);
    const int64_t rows = min((int64_t)seq.nq, (int64_t)a.max_q_len) * a.group;
    const int64_t r0 = (int64_t)rt * a.tile_rows;
    if (r0 + r >= rows) return;
    const int64_t r1 = min(r0 + a.tile_rows, rows) - 1;
    const Span span = tile_span(a, seq, (int)(r0 / a.group), (int)(r1 / a.group));
    const int used = splits_used(a, span.n);
    if (used <= 1) return;                                   // written by the first kernel
    const int64_t at = unit * a.splits * a.tile_rows + r;
    const int mine = (int)threadIdx.x;
    const float2 ml = mine < used ? a.part_ml[at + (int64_t)mine * a.tile_rows] : make_float2(kFloor, 0.0f);
    float top = ml.x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = __builtin_fmaxf(top, shfl_xor_f32(top, o));
    if (lane == 0) wave_top[wave] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(wave_top[0], wave_top[1]), __builtin_fmaxf(wave_top[2], wave_top[3]));
    const float f = __builtin_amdgcn_exp2f(ml.x - top);
    weight[mine] = f;
    float sum = ml.y * f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += shfl_xor_f32(sum, o);
    if (lane == 0) wave_sum[wave] = sum;
    __syncthreads();
    sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
    const float* po = a.part_o + at * D + lane * (D / 64);
    float v[D / 64] = {};
#pragma unroll 8
    for (int s = wave; s < used; s += 4) {
        const float w = weight[s];
        const float* src = po + (int64_t)s * a.tile_rows * D;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) v[j] += src[j] * w;
    }
#pragma unroll
    for (int j = 0; j < D / 64; ++j) part[wave][lane * (D / 64) + j] = v[j];
    __syncthreads();
    if ((int)threadIdx.x >= D / 2) return;
    const int qi = (int)((r0 + r) / a.group), head = kvh * a.group + (int)((r0 + r) - (int64_t)qi * a.group);
    const float inv = sum == 0.0f ? 0.0f : a.c.vg[kvh] / sum;
    float x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int d = 2 * (int)threadIdx.x + j;
        x[j] = ((part[0][d] + part[1][d]) + (part[2][d] + part[3][d])) * inv;
    }
    uint16_t* dst = a.out + (int64_t)(seq.start + qi) * a.ld_out + (int64_t)head * D;
    reinterpret_cast<uint32_t*>(dst)[threadIdx.x] = pack_bf16(x[0], x[1]);
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)(seq.start + qi) * a.q_heads + head] = row_lse(top, sum);
}

hipError_t launch_attention_rows(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.batch * a.row_tiles * a.c.kv_heads * a.splits));
    if (a.c.head_dim == 128) {
        if (a.tile_rows == 16)
            hipLaunchKernelGGL((k_attention_rows<128, 1>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((k_attention_rows<128, 2>), grid, dim3(256), 0, stream, a);
    } else {
        if (a.tile_rows == 16)
            hipLaunchKernelGGL((k_attention_rows<64, 1>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((k_attention_rows<64, 2>), grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_attention_join(const AttnArgs& a, hipStream_t stream) {
    const int64_t items = (int64_t)a.batch * a.row_tiles * a.c.kv_heads * a.tile_rows;
    const dim3 grid((unsigned)items);
    if (a.c.head_dim == 128)
        hipLaunchKernelGGL(k_attention_join<128>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(k_attention_join<64>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
