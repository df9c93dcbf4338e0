// mxq_attention_tile.hpp -- one 64-token tile of the paged NVFP4 cache against up to 32 query
// rows of a wave (gfx950): where its tokens lie, its loads, V in LDS, scores, softmax and the
// product with V; and the join of a work-group's waves.  The arithmetic is described in
// mxq_attention_nvfp4.hip.
#pragma once

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

// ---------------------------------------------------------------- one tile
// Adds the loaded tile (k, v; bit t of unread: group t's page may not be read; valid: this
// lane's token of V's scales is one of the sequence) to the rows' running softmax.  next_v and
// next_k load the following tile when V's and K's registers are free; mask(x) hides what rows
// do not see (token 16 t + 4 g + e of the tile in x[n][t][e]); sees_token(n, t, i): token 16 t + i.
template <int D, int NT, int G, typename NextV, typename NextK, typename Mask, typename Sees>
__device__ __forceinline__ void rows_step(uint8_t* mine, const Lane& L, uint32_t unread, bool valid, int scale_shift,
                                          KRegs<D>& k, VRegs<D>& v, const f16x8 (&q)[NT][D / 32], const float (&factor)[NT],
                                          float (&m)[NT], float (&l)[NT], f32x4 (&o)[NT][D / 16], uint32_t (&nan_blocks)[NT],
                                          NextV&& next_v, NextK&& next_k, Mask&& mask, Sees&& sees_token) {
    // V and its scales to LDS; tokens past the sequence or of unreadable pages get
    // zero scales, so whatever lies there stays out
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
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll 1
            for (int i = 4 * L.g; i < 4 * L.g + 4; ++i) {
                const uint32_t x = mine[WaveLds<D>::kNan + 16 * t + i];
#pragma unroll
                for (int n = 0; n < NT; ++n) nan_blocks[n] |= sees_token(n, t, i) ? x : 0u;
            }
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j) *reinterpret_cast<u32x4v*>(mine + j * kVJ + L.lane * 16) = v.w[j];
    stage_scales<D>(mine, v.s, valid, L);
    next_v();

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
    next_k();

    mask(x);
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

// ---------------------------------------------------------------- the join of the waves
// A wave's rows, summed over its lanes, to LDS; then (after what the caller does in between)
// each wave adds its element tiles of all waves (join is whole behind a barrier): store(row, d0, four elements d0 .., maximum, sum).
template <int D, int NT, int W>
__device__ __forceinline__ void waves_meet(int wave, const Lane& L, const float (&m)[NT], float (&l)[NT], f32x4 (&o)[NT][D / 16],
                                           uint32_t (&nan_blocks)[NT], float2 (&join)[W][NT * 16]) {
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
}
// area(wave): LDS of D / 16 KB each.
template <int D, int NT, int W, typename Area, typename Store>
__device__ __forceinline__ void waves_join(Area&& area, int wave, const Lane& L, int rows, const f32x4 (&o)[NT][D / 16],
                                           const float2 (&join)[W][NT * 16], Store&& store) {
    if constexpr (W == 1) {                                  // (a wave alone: from its registers)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 ml = join[0][n * 16 + L.col];
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
                if (n * 16 + L.col < rows) store(n * 16 + L.col, 16 * dt + 4 * L.g, o[n][dt], ml.x, ml.y);
        }
        return;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const auto at = [&](int w, int dt) { return reinterpret_cast<f32x4*>(area(w)) + dt * 64 + L.lane; };
        if (n) __syncthreads();
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) *at(wave, dt) = o[n][dt];
        __syncthreads();
        float top = kFloor, total = 0.0f, f[W];
#pragma unroll
        for (int w = 0; w < W; ++w) top = __builtin_fmaxf(top, join[w][n * 16 + L.col].x);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            f[w] = __builtin_amdgcn_exp2f(join[w][n * 16 + L.col].x - top);
            total += join[w][n * 16 + L.col].y * f[w];
        }
#pragma unroll
        for (int j = 0; j < (D / 16 + W - 1) / W; ++j) {
            const int dt = wave * (D / 16 >= W ? D / 16 / W : 1) + j;
            if (dt >= D / 16) break;
            f32x4 y = *at(0, dt) * f[0];
#pragma unroll
            for (int w = 1; w < W; ++w) y += *at(w, dt) * f[w];
            const int d0 = 16 * dt + 4 * L.g;
            if (n * 16 + L.col < rows) store(n * 16 + L.col, d0, y, top, total);
        }
    }
}

}  // namespace

}  // namespace mxq
