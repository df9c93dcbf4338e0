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
// dequantization between the products with K, weights between the products with V, operands
// read from LDS some products ahead.  The tile loop is unrolled over the two LDS
// images, as separate arrays: with one array and a dynamic buffer index the compiler orders
// every read after the other image's writes.
//
// What bounds it: a tile costs a wave 1024 cycles of matrix instructions and 1180 of vector
// ones (half of it the 32 exponentials and their sums, a quarter the dequantization), of which
// a matrix instruction hides all but its own issue, some 12 cycles; a CU's LDS is busy two
// thirds of the time, an operand read from it feeding 32 rows.  512 queries of 32 heads of 128
// over 65536 tokens take 570 us, 961 TFLOP/s (a plain FP16 product of 8192^3: 1074 to 1109, by
// card); two prompts of 4096 tokens 300 to 308 us, 892 to 916 TFLOP/s, and a quarter more when
// the tiles of a sequence ran together, so that the last sequence's longest rows started last.
// 64 rows a wave (half the operand reads, one wave a SIMD) were slower.
#include "mxq_attention_nvfp4.hpp"

namespace mxq {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 zero16() { return f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0}; }

// Row pitch of K's LDS image, bytes, and the byte of 16-byte chunk c of row t of V's.
template <int D>
constexpr int kPitchK = 2 * D + 16;
template <int D>
__device__ __forceinline__ int v_byte(int t, int c) {
    return t * (2 * D) + 16 * (c ^ 5 * (D == 128 ? t & 3 : (t >> 1) & 1));
}

// A thread's share of one tile's K or V: D / 4 codes of one token and their scales.
template <int D>
struct Part {
    KWords<D> w;
    uint32_t s;                       // D / 64 bytes
    bool ok;                          // the token's page may be read
};
// Where the 16 tokens of a wave lie (they share a page: everything here is uniform).
struct Spot {
    int64_t codes, scales;
    bool ok;
};
__device__ __forceinline__ Spot spot(const AttnArgs& a, int32_t entry, int t, int kvh) {
    Spot r;
    r.ok = (uint32_t)entry < (uint32_t)a.c.num_pages;
    const int64_t page = r.ok ? entry : 0, row = t & ((1 << a.c.page_shift) - 1);
    r.codes = page * a.c.cs_page + kvh * a.c.cs_head + row * a.c.cs_tok;
    r.scales = page * a.c.ss_page + kvh * a.c.ss_head + row * a.c.ss_tok;
    return r;
}
// code_at, scale_at: this lane's bytes inside the 16 rows.
template <int D>
__device__ __forceinline__ void load_part(const uint8_t* codes, const uint8_t* scales, const Spot& at, uint32_t code_at,
                                          uint32_t scale_at, Part<D>& r) {
    r.w = *reinterpret_cast<const KWords<D>*>(codes + at.codes + code_at);
    if constexpr (D == 128)
        r.s = *reinterpret_cast<const uint16_t*>(scales + at.scales + scale_at);
    else
        r.s = (scales + at.scales)[scale_at];
    r.ok = at.ok;
}

template <int D>
struct KImage {
    alignas(16) uint8_t b[64 * kPitchK<D>];
};
template <int D>
struct VImage {
    alignas(16) uint8_t b[64 * 2 * D];
    alignas(16) uint8_t nan[64 * 4];                   // per token and quarter: its V blocks with a NaN scale
    alignas(16) int any_nan[4];                        // per storing wave: one of them is not zero
};

// The scales a part is dequantized with, as FP16: K's are NaN where the page may not be
// read; V's are zero there, past the sequence and where they are NaN, and the latter are
// noted (a byte per thread, a word per wave).
template <int D>
__device__ __forceinline__ f16x2 k_factors(const Part<D>& r) {
    return e4m3_pair(r.ok ? r.s : (D == 128 ? 0x7F7Fu : 0x7Fu), false);
}
template <int D>
__device__ __forceinline__ f16x2 v_factors(const Part<D>& r, bool valid, VImage<D>& lds, int t, int part) {
    const uint32_t s = valid && r.ok ? r.s : 0u;
    const uint32_t hit = (((s & 0x7F7Fu) + 0x0101u) & 0x8080u) >> 7;     // bit 0: the low block, bit 8: the high one
    lds.nan[t * 4 + part] = (uint8_t)((hit | hit >> 7) & 3u);
    const int any = __any(hit != 0);
    lds.any_nan[t >> 4] = any;                                           // (the whole wave writes one word)
    return e4m3_pair(s & ~(hit * 0xFFu), false);
}
// Four elements: the low or high half of code dword c of a part.
template <int D>
__device__ __forceinline__ f16x4 dequant_half(const KWords<D>& w, f16x2 factors, int c, int half) {
    const f16 f = (D == 128 && c >= 2) ? factors.y : factors.x;
    const f16x2 a = __builtin_bit_cast(f16x2, half ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[c], 1.0f, 2)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[c], 1.0f, 0));
    const f16x2 b = __builtin_bit_cast(f16x2, half ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[c], 1.0f, 3)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w[c], 1.0f, 1));
    return f16x4{a.x, a.y, b.x, b.y} * f16x4{f, f, f, f};
}
template <int D>
__device__ __forceinline__ void store_chunk_k(KImage<D>& lds, int t, int part, int c, const f16x8& x) {
    *reinterpret_cast<f16x8*>(lds.b + t * kPitchK<D> + part * (D / 2) + 16 * c) = x;
}
template <int D>
__device__ __forceinline__ void store_chunk_v(VImage<D>& lds, int t, int part, int c, const f16x8& x) {
    *reinterpret_cast<f16x8*>(lds.b + v_byte<D>(t, part * (D / 32) + c)) = x;
}
template <int D>
__device__ __forceinline__ void store_k(KImage<D>& lds, const Part<D>& r, int t, int part) {
    const f16x2 f = k_factors<D>(r);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        store_chunk_k<D>(lds, t, part, c,
                         __builtin_shufflevector(dequant_half<D>(r.w, f, c, 0), dequant_half<D>(r.w, f, c, 1), 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int D>
__device__ __forceinline__ void store_v(VImage<D>& lds, const Part<D>& r, int t, bool valid, int part) {
    const f16x2 f = v_factors<D>(r, valid, lds, t, part);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
        store_chunk_v<D>(lds, t, part, c,
                         __builtin_shufflevector(dequant_half<D>(r.w, f, c, 0), dequant_half<D>(r.w, f, c, 1), 0, 1, 2, 3, 4, 5, 6, 7));
}

}  // namespace

// A wave holds 32 query rows (lane column = row), a work-group 128.
template <int D>
__global__ __launch_bounds__(256, 2) void k_attention_prompt(const AttnArgs a) {
    constexpr int kWaveRows = 32, kRowTile = 4 * kWaveRows;
    __shared__ KImage<D> k0, k1;
    __shared__ VImage<D> v0, v1;

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, h = lane >> 5;
    // later rows, which see more tiles, first for all sequences and heads: the last to start are
    // the shortest (two prompts of 4096 tokens 298 us against 368 when it was brought in)
    const int split = (int)(blockIdx.x % (unsigned)a.splits);
    const int order = (int)(blockIdx.x / (unsigned)a.splits);
    const int bhs = a.batch * a.c.kv_heads;
    const int rt = a.row_tiles - 1 - order / bhs, bh = order % bhs;
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

    // Q as the second operand of S^T = K Q^T: lane (col, h) holds elements 16 c + 8 h .. + 7 of
    // its row (the first row again past the last)
    f16x8 q[D / 16];
    const int row = wave * kWaveRows + col;
    const bool live = row < rows;
    const int qi = (int)((r0 + (live ? row : 0)) / a.group);
    const int head = kvh * a.group + (int)(r0 + (live ? row : 0) - (int64_t)qi * a.group);
    const int pos = live ? max(seq.len - seq.nq + qi, -1) : -1;
    float factor = 0.0f;

    f32x16 o[D / 32];
    float m = kFloor, l = 0.0f;
    uint32_t nan_blocks = 0;                           // V blocks that this lane's tokens make NaN
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();

    const int32_t* const table = a.table + (int64_t)b * a.ld_table;
    const int my_tok = tid >> 2, part = tid & 3;
    const uint32_t code_at = (uint32_t)((my_tok & 15) * a.c.cs_tok + part * (D / 8));
    const uint32_t scale_at = (uint32_t)((my_tok & 15) * a.c.ss_tok + part * (D / 64));
    // the first token of tile i (the last tile past the end) that this wave stages, and its
    // page's table entry; both uniform over the wave
    const int wave16 = wave * 16;
    const auto token = [&](int i) { return span.tile(min(i, last - 1)) * 64 + wave16; };
    const auto entry_of = [&](int i) { return table[min(token(i), seq.len - 1) >> a.c.page_shift]; };
    const auto spot_of = [&](int32_t entry, int i) { return spot(a, __builtin_amdgcn_readfirstlane(entry), token(i), kvh); };
    const auto valid = [&](int i) { return token(i) + (my_tok & 15) < seq.len; };
    // the positions of this wave's rows, for its masks
    const int w_lo = max(seq.len - seq.nq + (int)((r0 + wave * kWaveRows) / a.group), -1);
    const int w_hi = max(seq.len - seq.nq + (int)((r0 + min(wave * kWaveRows + kWaveRows - 1, rows - 1)) / a.group), -1);

    constexpr int kProducts = D / 8, kAhead = 4;       // with K, and with V, per tile
    const int k_lane = col * kPitchK<D> + 16 * h;
    int v_lane[D / 32];                                // (rows 8 apart keep the chunk order)
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
        v_lane[dt] = v_byte<D>(4 * h + ((lane & 15) >> 2), 4 * dt + 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) + 8 * (lane & 1);

    // Scores of a tile: token 32 T + 8 (e / 4) + 4 h + e % 4 in x[T][e].  Product n adds the
    // 16 elements n / 2 to half T = n % 2.
    f32x16 x[2];
    const auto k_operand = [&](const KImage<D>& k, int n) {
        return *reinterpret_cast<const f16x8*>(k.b + k_lane + 32 * (n & 1) * kPitchK<D> + 32 * (n >> 1));
    };
    const auto v_operand = [&](const VImage<D>& v, int n) {            // 16 tokens n / (D / 32), elements 32 (n % (D / 32)) ..
        const int f = n / (D / 32), dt = n % (D / 32);
        s16x4 r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            r[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
                v.b + v_lane[dt] + (16 * f + 8 * e) * (2 * D)));
        return __builtin_bit_cast(f16x8, __builtin_shufflevector(r[0], r[1], 0, 1, 2, 3, 4, 5, 6, 7));
    };

    // The queries are asked for ahead of the first tile, which has to wait for its page table
    // entry: loads come back in order, and so they are made ready while the tile is on its way.
    Part<D> kr, vr;
    int32_t entry = 0;
    if (first < last) {
        const int32_t e0 = entry_of(first), e1 = entry_of(first + 1);
        entry = entry_of(first + 2);
        const uint16_t* src = a.q + (int64_t)(seq.start + qi) * a.ld_q + (int64_t)head * D + h * 8;
        u32x4v w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) w[c] = *reinterpret_cast<const u32x4v*>(src + 16 * c);
        const float kg = a.c.kg[kvh];
        __builtin_amdgcn_sched_barrier(0);
        Spot at = spot_of(e0, first);
        load_part<D>(a.c.kc, a.c.ks, at, code_at, scale_at, kr);
        load_part<D>(a.c.vc, a.c.vs, at, code_at, scale_at, vr);
        __builtin_amdgcn_sched_barrier(0);
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
            top = absmax_pk(absmax_pk(absmax_pk(absmax_pk(top, w[c].x), w[c].y), w[c].z), w[c].w);
        top = fold_pk(top);
        top = max(top, shfl_xor_u32(top, 32));
        const float up = q_power(top, factor);
        factor = score_factor(a, factor, kg);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) q[c] = q_operand(w[c], up);
        store_k<D>(k0, kr, my_tok, part);
        store_v<D>(v0, vr, my_tok, valid(first), part);
        at = spot_of(e1, first + 1);
        load_part<D>(a.c.kc, a.c.ks, at, code_at, scale_at, kr);
        load_part<D>(a.c.vc, a.c.vs, at, code_at, scale_at, vr);
    }

    // One tile: kn, vn its images; kf, vf the next one's (the last tile's again at the end).
    // The order of the products and what stands between them is fixed by hand: left alone,
    // the compiler forms all weights first and reads each operand right before its product.
    const auto step = [&](int i, const KImage<D>& kn, KImage<D>& kf, const VImage<D>& vn, VImage<D>& vf) {
        __syncthreads();                               // kn and vn are whole; kf and vf are free
        const int t0 = span.tile(i) * 64;
        const u32x4v noted = *reinterpret_cast<const u32x4v*>(vn.any_nan);
        f16x8 ahead[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) ahead[n] = k_operand(kn, n);
        f16x4 low = {};
        f16x2 fk, fv;
        x[0] = x[1] = zero16();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
            x[n & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ahead[n % kAhead], q[n >> 1], x[n & 1], 0, 0, 0);
            ahead[n % kAhead] = n + kAhead < kProducts ? k_operand(kn, n + kAhead) : v_operand(vn, n + kAhead - kProducts);
            const int c = (n >> 1) % (D / 32);
            const bool is_v = n >= kProducts / 2;
            if (n == 0) fk = k_factors<D>(kr);
            if (n == kProducts / 2) fv = v_factors<D>(vr, valid(i + 1), vf, my_tok, part);
            const f16x4 half = is_v ? dequant_half<D>(vr.w, fv, c, n & 1) : dequant_half<D>(kr.w, fk, c, n & 1);
            if (n & 1) {
                const f16x8 whole = __builtin_shufflevector(low, half, 0, 1, 2, 3, 4, 5, 6, 7);
                if (is_v)
                    store_chunk_v<D>(vf, my_tok, part, c, whole);
                else
                    store_chunk_k<D>(kf, my_tok, part, c, whole);
            } else {
                low = half;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        {
            const Spot at = spot_of(entry, i + 2);
            load_part<D>(a.c.kc, a.c.ks, at, code_at, scale_at, kr);
            load_part<D>(a.c.vc, a.c.vs, at, code_at, scale_at, vr);
            entry = entry_of(i + 3);
        }
        // masks only where an edge crosses the tile for this wave's rows
        if (t0 + 63 > w_lo || (a.window && t0 <= (int64_t)w_hi - a.window))
            each_seen<32>(a, pos, t0 + 4 * h, [](int e) { return 8 * (e >> 2) + (e & 3); },
                          [&](int e, bool seen) { x[e >> 4][e & 15] = seen ? x[e >> 4][e & 15] : -__builtin_inff(); });
        if (noted.x | noted.y | noted.z | noted.w) {   // (rare) note the NaN V blocks this lane sees
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
                const int tok = t0 + 8 * (e >> 2) + 4 * h + (e & 3);
                const uint32_t w = *reinterpret_cast<const uint32_t*>(vn.nan + 4 * (tok - t0));
                const uint32_t blocks = D == 128 ? (w & 3u) | (w >> 6 & 0xCu) | (w >> 12 & 0x30u) | (w >> 18 & 0xC0u)
                                                 : (w & 1u) | (w >> 7 & 2u) | (w >> 14 & 4u) | (w >> 21 & 8u);
                nan_blocks |= sees(a, pos, tok) ? blocks : 0u;
            }
        }
        float top = x[0][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top = __builtin_fmaxf(top, x[e >> 4][e & 15]);
        top *= factor;
        if (__any(top > m + kSlack)) {
            top = __builtin_fmaxf(top, shfl_xor_f32(top, 32));
            const float raised = raise(m, top);
            const float f = __builtin_amdgcn_exp2f(m - raised);
            m = raised;
            l *= f;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) o[dt] *= f;
        }

        // Weights of 16 tokens at a time; their products with V between the weights of the
        // next 16.
        float shift = kBias - m, scale = factor;
        if (__builtin_expect(__any(far(m)), 0)) {
            const bool is_far = far(m);
            const float by = is_far ? factor : 1.0f, less = is_far ? m : 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e >> 4][e & 15] = x[e >> 4][e & 15] * by - less;
            scale = is_far ? 1.0f : factor;
            shift = is_far ? kBias : shift;
        }
        f16x8 p[2];
        const auto weights = [&](int f, int e) {                           // two of them
            const int k = 8 * f + e;
            const f32x2 w = {__builtin_amdgcn_exp2f(__builtin_fmaf(x[k >> 4][k & 15], scale, shift)),
                             __builtin_amdgcn_exp2f(__builtin_fmaf(x[k >> 4][(k & 15) + 1], scale, shift))};
            l += w.x + w.y;                            // before the rounding: lse is an output
            const f16x2 b = __builtin_convertvector(w, f16x2);
            p[f & 1][e] = b.x;
            p[f & 1][e + 1] = b.y;
        };
#pragma unroll
        for (int e = 0; e < 8; e += 2) weights(0, e);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kProducts; ++n) {
            const int f = n / (D / 32), dt = n % (D / 32);
            o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ahead[n % kAhead], p[f & 1], o[dt], 0, 0, 0);
            if (n + kAhead < kProducts) ahead[n % kAhead] = v_operand(vn, n + kAhead);
            if (f < 3) {
#pragma unroll
                for (int e = 0; e < 8 / (D / 32); e += 2) weights(f + 1, dt * (8 / (D / 32)) + e);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // A wave without rows only stages its share of the next tile (64 ragged sequences of up to
    // 8192 tokens with 40 rows a unit: 211 us against 257).  The other two of four waves then do
    // all products, so that these 336 MB take four times as long as their bytes.
    const auto stage = [&](int i, KImage<D>& kf, VImage<D>& vf) {
        __syncthreads();
        store_k<D>(kf, kr, my_tok, part);
        store_v<D>(vf, vr, my_tok, valid(i + 1), part);
        const Spot at = spot_of(entry, i + 2);
        load_part<D>(a.c.kc, a.c.ks, at, code_at, scale_at, kr);
        load_part<D>(a.c.vc, a.c.vs, at, code_at, scale_at, vr);
        entry = entry_of(i + 3);
    };
    if (wave * kWaveRows < rows) {
        for (int i = first; i < last; i += 2) {
            step(i, k0, k1, v0, v1);
            if (i + 1 < last) step(i + 1, k1, k0, v1, v0);
        }
    } else {
        for (int i = first; i < last; i += 2) {
            stage(i, k1, v1);
            if (i + 1 < last) stage(i + 1, k0, v0);
        }
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
        for (int e = 0; e < 16; e += 4) {
            const f32x4 y = {o[dt][e], o[dt][e + 1], o[dt][e + 2], o[dt][e + 3]};
            if (used == 1)
                store_finished<D>(a, seq, kvh, r0 + row, 32 * dt + 2 * e + 4 * h, y, m, l, vg);
            else
                store_part<D>(a, (unit * a.splits + split) * kRowTile + row, 32 * dt + 2 * e + 4 * h, y, m, l);
        }
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
