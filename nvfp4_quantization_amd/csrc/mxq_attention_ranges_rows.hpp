// mxq_attention_ranges_rows.hpp -- a unit of up to 32 query rows of attention with shared prefixes
// (gfx950): every 64-token tile by one wave, as in mxq_attention_nvfp4.hip.
#pragma once

#include "mxq_attention_ranges.hpp"
#include "mxq_attention_tile.hpp"

namespace mxq {

namespace {

// By a work-group of W waves; area(wave): LDS of its own, 16-byte aligned, WaveLds<D>::kBytes or
// D / 16 KB, whichever is more.
template <int D, int NT, int G, int W, typename Area>
__device__ __forceinline__ void range_rows(const PrefixAttnArgs& a, const RangeUnit& u, const int* limits, Area&& area,
                                           float2 (&join)[W][NT * 16]) {
    const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Lane L;
    L.lane = tid & 63;
    L.g = L.lane >> 4, L.col = L.lane & 15;
    uint8_t* const mine = area(wave);
    const int kvh = u.kvh, stop = u.last;

    const Offsets<D, G> off(a, L);
    const int scale_shift = D == 128 ? 16 * (L.g & 1) : 8 * L.g;
    const Base head{a.c.kc + kvh * a.c.cs_head, a.c.ks + kvh * a.c.ss_head, a.c.vc + kvh * a.c.cs_head,
                    a.c.vs + kvh * a.c.ss_head};

    // loads run one round ahead of the tile that uses them, page table entries two
    KRegs<D> k;
    VRegs<D> v;
    int32_t entries = 0;
    uint32_t bad = 0;
    int i = u.first + wave;
    const auto tile_of = [&](int j) { return u.body + min(j, stop - 1); };
    const auto entries_of = [&](int j) { return page_entries(a, u.table, u.len, tile_of(j), L); };
    f16x8 q[NT][D / 32];
    float factor[NT];
    int hi[NT], count[NT];
    if (u.first < stop) {
        const int32_t e = entries_of(i);
        entries = entries_of(i + W);
        u32x4v w[NT][D / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const RangeRow row = range_row(a, u, limits, n * 16 + L.col);
            hi[n] = row.hi, count[n] = row.count;
            const uint16_t* src = a.q + (int64_t)row.query * a.ld_q + (int64_t)row.head * D + L.g * (D / 4);
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
    uint32_t nan_blocks[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = kFloor;
        l[n] = 0.0f;
        nan_blocks[n] = 0;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) o[n][dt] = f32x4{0, 0, 0, 0};
    }

    for (; i < stop; i += W) {
        const int t0 = (u.body + i) * 64;
        const uint32_t unread = bad;
        const bool valid = !((unread >> (G == 1 ? 0 : L.g)) & 1) && t0 + L.lane < u.len;
        Place<G> where;
        rows_step<D, NT, G>(
            mine, L, unread, valid, scale_shift, k, v, q, factor, m, l, o, nan_blocks,
            [&] {
                where = place<G>(a, entries, tile_of(i + W), L);
                load_v<D, G>(head, where, off, L, v);
                entries = entries_of(i + 2 * W);
                bad = where.bad;
            },
            [&] { load_k<D, G>(head, where, off, k); },
            [&](f32x4 (&x)[NT][4]) {
                if (t0 + 63 > u.min_hi || t0 < u.low) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        int ago = hi[n] - t0 - 4 * L.g;
                        asm("" : "+v"(ago));                 // (or a difference per element is held across the tiles)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const bool seen = (uint32_t)(ago - (16 * (e >> 2) + (e & 3))) < (uint32_t)count[n];
                            x[n][e >> 2][e & 3] = seen ? x[n][e >> 2][e & 3] : -__builtin_inff();
                        }
                    }
                }
            },
            [&](int n, int t, int i) { return in_range(hi[n], count[n], t0 + 16 * t + i); });
    }

    waves_meet<D, NT, W>(wave, L, m, l, o, nan_blocks, join);
    waves_join<D, NT, W>(area, wave, L, u.rows, o, join, [&](int r, int d0, const f32x4& y, float top, float total) {
        const RangeRow row = range_row(a, u, limits, r);
        store_part<D>(a, ((int64_t)u.part * a.total_q + row.query) * a.q_heads + row.head, d0, y, top, total);
    });
}

}  // namespace

}  // namespace mxq
