// mxq_attention_prompt.hip -- causal attention over the paged NVFP4 cache (gfx950) for
// many query rows per cached head: prompts and chunks of them.
//
// The operands and the arithmetic are those of the form for few rows
// (mxq_attention_nvfp4.hip: S^T = K Q^T, O^T = V^T P^T in FP16 with FP32 accumulators, K and
// V dequantized exactly), but a work-group's four waves share every 64-token tile, 32
// query rows each: the tile is dequantized once, into LDS, instead of once per 32 rows.
// A thread turns 32 codes (head_dim 128) of K and of V of one token into FP16 per tile; two
// tiles of LDS let that overlap the products of the tile before, one barrier a tile.
//  * K's rows are read as operands with 16-byte loads, V's with ds_read_b64_tr_b16 (four
//    tokens of one element a lane).  Both images are row-major: K's rows lie 16 bytes apart
//    in the 64 banks, so 16 rows' chunks of a read meet in none; V's chunks are permuted
//    by row, so that neither four rows' 64 bytes (a read) nor four rows' four quarters (a
//    write) do.
//  * What must not reach a row: codes past the sequence's end get a zero scale (V) or are
//    masked (K); an unreadable page's K scales are NaN, so that only rows that see it are.
//    A NaN V scale is staged as zero and noted; rows that see its token put NaN into that
//    block at the end.
//
// Instructions are placed so that the matrix unit runs beside the rest: the next tile's
// dequantization between the products with K, the weights between those with V, operands
// read from LDS some products ahead.  The tile loop is unrolled over the two LDS images, as
// separate arrays: with one array and a dynamic buffer index the compiler orders every read
// after the other image's writes.
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kRowTile = 128;         // query rows of a work-group

__device__ __forceinline__ f32x16 zero16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

// Row pitch of K's LDS image, bytes, and the byte of 16-byte chunk c of row t of V's.
template <int D>
constexpr int kPitchK = 2 * D + 16;
template <int D>
__device__ __forceinline__ int v_byte(int t, int c) {
    return t * (2 * D) + 16 * (c ^ 5 * (D == 128 ? t & 3 : (t >> 1) & 1));
}

template <int D>
struct TileRegs {
    KWords<D> k, v;                   // D / 4 codes of this thread's token
    uint32_t ks, vs;                  // their scales (D / 64 bytes)
    bool ok;                          // the token's page may be read
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs& a, int32_t entry, int t, int kvh, int part, TileRegs<D>& r) {
    r.ok = (uint32_t)entry < (uint32_t)a.c.num_pages;
    const int64_t page = r.ok ? entry : 0, row = t & ((1 << a.c.page_shift) - 1);
    const int64_t oc = page * a.c.cs_page + kvh * a.c.cs_head + row * a.c.cs_tok + part * (D / 8);
    const int64_t os = page * a.c.ss_page + kvh * a.c.ss_head + row * a.c.ss_tok + part * (D / 64);
    r.k = *reinterpret_cast<const KWords<D>*>(a.c.kc + oc);
    r.v = *reinterpret_cast<const KWords<D>*>(a.c.vc + oc);
    if constexpr (D == 128) {
        r.ks = *reinterpret_cast<const uint16_t*>(a.c.ks + os);
        r.vs = *reinterpret_cast<const uint16_t*>(a.c.vs + os);
    } else {
        r.ks = a.c.ks[os];
        r.vs = a.c.vs[os];
    }
}

template <int D>
struct TileLds {
    alignas(16) uint8_t k[64 * kPitchK<D>];
    alignas(16) uint8_t v[64 * 2 * D];
    alignas(16) uint8_t nan[64 * 4];                   // per token and quarter: its V blocks with a NaN scale
    alignas(16) int any_nan[4];                        // per storing wave: one of them is not zero
};

// The thread's share of a tile into LDS.
template <int D>
__device__ __forceinline__ void store_tile(TileLds<D>& lds, const TileRegs<D>& r, int t, bool valid, int part) {
    const uint32_t nan = D == 128 ? 0x7F7Fu : 0x7Fu;
    f16x8 x[D / 32];
    dequant_row<D>(r.k, r.ok ? r.ks : nan, x);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        *reinterpret_cast<f16x8*>(lds.k + t * kPitchK<D> + part * (D / 2) + 16 * c) = x[c];
    const uint32_t vs = valid && r.ok ? r.vs : 0u;
    // a NaN scale byte keeps its seven bits only in `hit` (bit 0: its low block, bit 8: its high one)
    const uint32_t hit = (((vs & 0x7F7Fu) + 0x0101u) & 0x8080u) >> 7;
    dequant_row<D>(r.v, vs & ~(hit * 0xFFu), x);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        *reinterpret_cast<f16x8*>(lds.v + v_byte<D>(t, part * (D / 32) + c)) = x[c];
    lds.nan[t * 4 + part] = (uint8_t)((hit | hit >> 7) & 3u);
    const int any = __any(hit != 0);
    if ((t & 15) == 0 && part == 0) lds.any_nan[t >> 4] = any;
}

}  // namespace

template <int D>
__global__ __launch_bounds__(256, 2) void k_attention_prompt(const AttnArgs a) {
    __shared__ TileLds<D> image0, image1;

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int col = lane & 31, h = lane >> 5;
    // work-groups of one (sequence, cached head) run together; later rows (more tiles) first
    const int split = (int)(blockIdx.x % (unsigned)a.splits);
    const int order = (int)(blockIdx.x / (unsigned)a.splits);
    const int rt = a.row_tiles - 1 - order % a.row_tiles, bh = order / a.row_tiles;
    const int b = bh / a.c.kv_heads, kvh = bh - b * a.c.kv_heads;
    const int64_t unit = ((int64_t)b * a.row_tiles + rt) * a.c.kv_heads + kvh;
    const Seq seq = sequence(a, b);
    const int64_t r0 = (int64_t)rt * kRowTile;
    const int rows = (int)min(min((int64_t)seq.nq, (int64_t)a.max_q_len) * a.group - r0, (int64_t)kRowTile);
    if (rows <= 0) return;
    const Span span = tile_span(a, seq, (int)(r0 / a.group), (int)((r0 + rows - 1) / a.group));
    const int used = splits_used(a, span.n);
    if (split >= used) return;
    const int first = split * a.chunk, last = split == used - 1 ? span.n : first + a.chunk;

    // Q as the second operand of S^T = K Q^T: lane (col, h) holds elements 16 c + 8 h .. + 7
    f16x8 q[D / 16];
    const int my_row = wave * 32 + col;
    const bool live = my_row < rows;
    const int qi = live ? (int)((r0 + my_row) / a.group) : 0;
    const int head = kvh * a.group + (live ? (int)(r0 + my_row - (int64_t)qi * a.group) : 0);
    const int pos = live ? max(seq.len - seq.nq + qi, -1) : -1;
    float factor;
    {
        const uint16_t* src = a.q + (int64_t)(seq.start + qi) * a.ld_q + (int64_t)head * D + h * 8;
        u32x4v w[D / 16];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            w[c] = live ? *reinterpret_cast<const u32x4v*>(src + 16 * c) : u32x4v{0, 0, 0, 0};
            top = absmax_pk(absmax_pk(absmax_pk(absmax_pk(top, w[c].x), w[c].y), w[c].z), w[c].w);
        }
        top = fold_pk(top);
        top = max(top, shfl_xor_u32(top, 32));
        const float up = q_power(top, factor);
        factor *= a.scale_log2 * a.c.kg[kvh];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) q[c] = q_operand(w[c], up);
    }

    f32x16 o[D / 32];
    float m = kFloor, l = 0.0f;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();

    const int32_t* const table = a.table + (int64_t)b * a.ld_table;
    const int my_tok = tid >> 2, part = tid & 3;
    const auto entry_of = [&](int i) {
        const int t = span.tile(i) * 64 + my_tok;
        return t < seq.len ? table[t >> a.c.page_shift] : 0;
    };
    // the positions of this wave's rows, for its masks
    const int w_lo = max(seq.len - seq.nq + (int)((r0 + wave * 32) / a.group), -1);
    const int w_hi = max(seq.len - seq.nq + (int)((r0 + min(wave * 32 + 31, rows - 1)) / a.group), -1);

    TileRegs<D> regs;
    int32_t entry = 0;
    uint32_t nan_blocks = 0;                           // V blocks that this lane's tokens make NaN
    if (first < last) {
        load_tile<D>(a, entry_of(first), span.tile(first) * 64 + my_tok, kvh, part, regs);
        if (first + 1 < last) entry = entry_of(first + 1);
        store_tile<D>(image0, regs, my_tok, span.tile(first) * 64 + my_tok < seq.len, part);
        if (first + 1 < last) {
            load_tile<D>(a, entry, span.tile(first + 1) * 64 + my_tok, kvh, part, regs);
            if (first + 2 < last) entry = entry_of(first + 2);
        }
    }
    const int k_lane = col * kPitchK<D> + 16 * h;
    int v_lane[D / 32];                                // (rows 8 apart keep the chunk order)
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
        v_lane[dt] = v_byte<D>(4 * h + ((lane & 15) >> 2), 4 * dt + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) + 8 * (lane & 1);

    // One tile: its products from `now`, the next tile into `then`.
    const auto step = [&](int i, TileLds<D>& now, TileLds<D>& then) {
        __syncthreads();                               // this tile is whole; the other image is free
        const int t0 = span.tile(i) * 64;
        const u32x4v noted = *reinterpret_cast<const u32x4v*>(now.any_nan);

        // Scores: token 32 T + 8 (e / 4) + 4 h + e % 4 in x[T][e].  The next tile's
        // dequantization (the last one's again at the end: that image is not read) runs
        // between the products.
        f32x16 x[2];
#pragma unroll
        for (int T = 0; T < 2; ++T) {
            x[T] = zero16();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const f16x8 k = *reinterpret_cast<const f16x8*>(now.k + k_lane + 32 * T * kPitchK<D> + 32 * c);
                x[T] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[c], x[T], 0, 0, 0);
            }
        }
        const int next = min(i + 1, last - 1);
        store_tile<D>(then, regs, my_tok, span.tile(next) * 64 + my_tok < seq.len, part);
        if (i + 2 < last) {
            load_tile<D>(a, entry, span.tile(i + 2) * 64 + my_tok, kvh, part, regs);
            if (i + 3 < last) entry = entry_of(i + 3);
        }

        // masks only where an edge crosses the tile for this wave's rows
        if (t0 + 63 > w_lo || (a.window && t0 <= (int64_t)w_hi - a.window)) {
#pragma unroll
            for (int T = 0; T < 2; ++T)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int tok = t0 + 32 * T + 8 * (e >> 2) + 4 * h + (e & 3);
                    const bool see = tok <= pos && (!a.window || tok > pos - a.window || tok < a.sinks);
                    x[T][e] = see ? x[T][e] : -__builtin_inff();
                }
        }
        if (noted.x | noted.y | noted.z | noted.w) {   // (rare) note the NaN V blocks this lane sees
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
                const int tok = t0 + 8 * (e >> 2) + 4 * h + (e & 3);
                const bool see = tok <= pos && (!a.window || tok > pos - a.window || tok < a.sinks);
                const uint32_t w = *reinterpret_cast<const uint32_t*>(now.nan + 4 * (tok - t0));
                const uint32_t blocks = D == 128 ? (w & 3u) | (w >> 6 & 0xCu) | (w >> 12 & 0x30u) | (w >> 18 & 0xC0u)
                                                 : (w & 1u) | (w >> 7 & 2u) | (w >> 14 & 4u) | (w >> 21 & 8u);
                nan_blocks |= see ? blocks : 0u;
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int T = 0; T < 2; ++T)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = __builtin_fmaxf(top, x[T][e]);
        top *= factor;
        if (__any(top > m + kSlack)) {
            top = __builtin_fmaxf(top, shfl_xor_f32(top, 32));
            const float raised = __builtin_fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f(m - raised);
            m = raised;
            l *= f;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= f;
        }

        // Weights of 16 tokens at a time and their products with V: the weights and V
        // operands of the next 16 are formed between the products.
        const float shift = kBias - m;
        const auto weights = [&](int f) {
            float w[8];
            f16x8 p;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[f >> 1][8 * (f & 1) + e], factor, shift));
            l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const f32x2 pair = {w[e], w[e + 1]};
                const f16x2 r = __builtin_convertvector(pair, f16x2);
                p[e] = r.x;
                p[e + 1] = r.y;
            }
            return p;
        };
        const auto v_operand = [&](int f, int dt) {
            s16x4 v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                v[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
                    now.v + v_lane[dt] + (16 * f + 8 * e) * (2 * D)));
            return __builtin_bit_cast(f16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        };
        f16x8 v[2][D / 32], p[2];
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) v[0][dt] = v_operand(0, dt);
        p[0] = weights(0);
        __builtin_amdgcn_sched_group_barrier(0x100, D / 16, 0);            // reads
        __builtin_amdgcn_sched_group_barrier(0x002, 48, 0);                // vector instructions
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            if (f < 3) {
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) v[(f + 1) & 1][dt] = v_operand(f + 1, dt);
                p[(f + 1) & 1] = weights(f + 1);
                __builtin_amdgcn_sched_group_barrier(0x100, D / 16, 0);
            }
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) {
                o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[f & 1][dt], p[f & 1], o[dt], 0, 0, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);         // a product
                if (f < 3) __builtin_amdgcn_sched_group_barrier(0x002, 40 / (D / 32), 0);
            }
        }
    };
    for (int i = first; i < last; i += 2) {
        step(i, image0, image1);
        if (i + 1 < last) step(i + 1, image1, image0);
    }

    l += shfl_xor_f32(l, 32);
    nan_blocks |= shfl_xor_u32(nan_blocks, 32);
    if (!live) return;
    if (nan_blocks) {
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int e = 0; e < 16; ++e)               // element 32 dt + 8 (e / 4) + ..: block 2 dt + e / 8
                if ((nan_blocks >> (2 * dt + (e >> 3))) & 1) o[dt][e] = __builtin_nanf("");
    }
    const float vg = a.c.vg[kvh];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            store_rows<D>(a, seq, unit, kvh, split, used, kRowTile, r0 + my_row, 32 * dt + 2 * e + 4 * h,
                          f32x4{o[dt][e], o[dt][e + 1], o[dt][e + 2], o[dt][e + 3]}, m, l, vg);
}

hipError_t launch_attention_prompt(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.batch * a.row_tiles * a.c.kv_heads * a.splits));
    if (a.c.head_dim == 128)
        hipLaunchKernelGGL(k_attention_prompt<128>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(k_attention_prompt<64>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxq
