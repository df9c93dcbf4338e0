// mxq_attention_pages.hip -- causal attention over listed pages of the paged NVFP4 cache
// (gfx950): each query and cached head has a list of pages of its own.
//
// The tiles, the operands and the arithmetic are those of the call over whole sequences
// (mxq_attention_nvfp4.hip); a tile's 64 tokens are the next 64 of the list's pages, one
// after another.  The rows of a unit are the query heads of one cached head, so all of them
// share the position up to which they see.
//
// Few units go over several work-groups, whose parts meet in the workspace; many take a wave each, so
// that no waves have to meet.  Page numbers are read two rounds ahead of a tile, list entries three.
//
// What bounds it: 64 queries of 64 pages of 64, 64 query heads over 8 of 128 (304 MB) take 53 us,
// 5.8 TB/s: memory, and 4 us until the first tile (sequence, list, page table, tile: four memory
// latencies).  1000 queries of 48 pages of 32, 32 query heads over 8 (1.8 GB by way of the L2, 0.6 of
// it from beyond) take 239 us: a tile costs a wave some 430 vector instructions, 256 of them to
// dequantize it for the group's four rows alone, 168 of the 239 us on every SIMD, and 40 of matrix
// ones beside them.  Sharing a dequantized tile takes queries that list the same pages.
#include "mxq_attention_tile.hpp"

namespace mxq {

namespace {

constexpr int kAbsent = 0x7FFFFFC0;   // the first token of a tile's group that no entry names: past every position

// First tokens of a tile's groups (uniform) from the lanes' own (group lane % 4).  (Named members:
// an array indexed by a lane's group would end up in scratch.)
template <int G>
struct Starts {
    int t0, t1, t2, t3;
    __device__ __forceinline__ explicit Starts(int mine) {
        t0 = __builtin_amdgcn_readlane(mine, 0);
        t1 = G == 1 ? t0 + 16 : __builtin_amdgcn_readlane(mine, 1);
        t2 = G == 1 ? t0 + 32 : __builtin_amdgcn_readlane(mine, 2);
        t3 = G == 1 ? t0 + 48 : __builtin_amdgcn_readlane(mine, 3);
    }
    __device__ __forceinline__ int of(int group) const {     // of a lane's group
        if constexpr (G == 1) return t0 + 16 * group;
        const int lo = group & 1 ? t1 : t0, hi = group & 1 ? t3 : t2;
        return group & 2 ? hi : lo;
    }
    __device__ __forceinline__ int last() const { return max(max(t0, t1), max(t2, t3)) + 15; }           // the tile's last token
};

}  // namespace

template <int D, int NT, int G, int W>
__global__ __launch_bounds__(64 * W, W == 1 ? 2 : 8 / W) void k_attention_pages(const PagesAttnArgs a) {
    constexpr int kWave = WaveLds<D>::kBytes;
    constexpr int kJoin = W == 1 ? 0 : (D / 16) * 64 * 16;
    constexpr int kLds = W * (kWave > kJoin ? kWave : kJoin);
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    __shared__ float2 join[W][NT * 16];

    const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Lane L;
    L.lane = tid & 63;
    L.g = L.lane >> 4, L.col = L.lane & 15;
    const int split = (int)(blockIdx.x % (unsigned)a.splits);
    const unsigned unit = blockIdx.x / (unsigned)a.splits;
    const int rt = (int)(unit % (unsigned)a.row_tiles);
    const unsigned tk = unit / (unsigned)a.row_tiles;
    const int token = (int)(tk / (unsigned)a.c.kv_heads), kvh = (int)(tk - (unsigned)token * (unsigned)a.c.kv_heads);
    const int32_t* const list = a.pages + (int64_t)tk * a.top;
    const Query at = query_of(a, a.c.page_shift, token);
    if (at.b < 0) return;
    const int rows = min(a.group - rt * (NT * 16), NT * 16);
    const int shift = a.c.page_shift, current = at.pos < 0 ? -1 : at.pos >> shift;

    // entries up to the last that names a page with something to see; tiles of those
    int entries = 0;
    for (int e0 = 0; e0 < a.top; e0 += 64) {
        const int j = e0 + L.lane < a.top ? list[e0 + L.lane] : -1;
        const uint64_t there = __ballot(j >= 0 && j <= current);
        if (there) entries = e0 + 64 - __builtin_clzll(there);
    }
    const int tiles = (int)((((int64_t)entries << shift) + 63) >> 6);
    const int chunk = (tiles + a.splits - 1) / a.splits;
    const int first = min(split * chunk, tiles), stop = min(first + chunk, tiles);

    const Offsets<D, G> off(a, L);
    const int scale_shift = D == 128 ? 16 * (L.g & 1) : 8 * L.g;
    uint8_t* const mine = lds + wave * kWave;
    const Base head{a.c.kc + kvh * a.c.cs_head, a.c.ks + kvh * a.c.ss_head, a.c.vc + kvh * a.c.cs_head,
                    a.c.vs + kvh * a.c.ss_head};
    const int32_t* const table = a.table + (int64_t)at.b * a.ld_table;

    // Loads run one round ahead of the tile that uses them, page table entries two, list
    // entries three.
    int i = first + wave;
    const auto tile_of = [&](int j) { return min(j, stop - 1); };
    const auto token_of = [&](int j) {                       // of the list, of this lane's group
        return (int64_t)tile_of(j) * 64 + (G == 1 ? 0 : 16 * (L.lane & 3));
    };
    const auto listed = [&](int j) { return list[min((int)(token_of(j) >> shift), entries - 1)]; };
    const auto there = [&](int page, int j) { return page >= 0 && page <= current && (token_of(j) >> shift) < entries; };
    const auto page_of = [&](int page) { return table[page >= 0 && page <= current ? page : 0]; };
    const auto start_of = [&](int page, int j) {
        return there(page, j) ? (page << shift) + (int)(token_of(j) & ((1 << shift) - 1)) : kAbsent;
    };
    KRegs<D> k;
    VRegs<D> v;
    int32_t entry = 0;
    int list1 = 0, list2 = 0, start = kAbsent;
    uint32_t bad = 0;
    f16x8 q[NT][D / 32];
    float factor[NT];
    const float vg = a.c.vg[kvh];
    if (first < stop) {
        const int list0 = listed(i);
        list1 = listed(i + W);
        list2 = listed(i + 2 * W);
        u32x4v w[NT][D / 32];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = rt * (NT * 16) + (n * 16 + L.col < rows ? n * 16 + L.col : 0);
            const uint16_t* src = a.q + (int64_t)token * a.ld_q + (int64_t)(kvh * a.group + r) * D + L.g * (D / 4);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) w[n][c] = reinterpret_cast<const u32x4v*>(src)[c];
        }
        const float kg = a.c.kg[kvh];
        const int32_t e = page_of(list0);
        entry = page_of(list1);
        start = start_of(list0, i);
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
        const Starts<G> from(start);
        const uint32_t unread = bad;
        const bool valid = !((unread >> (G == 1 ? 0 : L.g)) & 1) && from.of(L.g) + L.col <= at.pos;
        Place<G> where;
        rows_step<D, NT, G>(
            mine, L, unread, valid, scale_shift, k, v, q, factor, m, l, o, nan_blocks,
            [&] {
                where = place<G>(a, entry, tile_of(i + W), L);
                load_v<D, G>(head, where, off, L, v);
                start = start_of(list1, i + W);
                bad = where.bad;
                entry = page_of(list2);
                list1 = list2;
                list2 = listed(i + 3 * W);
            },
            [&] { load_k<D, G>(head, where, off, k); },
            [&](f32x4 (&x)[NT][4]) {
                if (from.last() > at.pos) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int start = t == 0 ? from.t0 : t == 1 ? from.t1 : t == 2 ? from.t2 : from.t3;
                            const bool seen = start + 4 * L.g + e <= at.pos;
#pragma unroll
                            for (int n = 0; n < NT; ++n) x[n][t][e] = seen ? x[n][t][e] : -__builtin_inff();
                        }
                }
            },
            [&](int, int t, int i) { return (t == 0 ? from.t0 : t == 1 ? from.t1 : t == 2 ? from.t2 : from.t3) + i <= at.pos; });
    }

    waves_meet<D, NT, W>(wave, L, m, l, o, nan_blocks, join);
    if constexpr (W == 1) __syncthreads();
    const Seq seq{0, token, 1};
    waves_join<D, NT, W>([&](int w) { return lds + w * kJoin; }, wave, L, rows, o, join, [&](int r, int d0, const f32x4& y, float top, float total) {
        const int in_group = rt * (NT * 16) + r;
        if (a.splits == 1)
            store_finished<D>(a, seq, kvh, in_group, d0, y, top, total, vg);
        else
            store_part<D>(a, ((int64_t)split * a.total_q + token) * a.q_heads + kvh * a.group + in_group, d0, y, top, total);
    });
}

// The parts of a query row and head, by a wave: D / 8 lanes a part (elements 4 l .. and D / 2 + 4 l .. of
// it), kPer parts a load, BLOCK such loads on their way at once (9: as many as 128 registers hold).
template <int D, int BLOCK>
__global__ __launch_bounds__(256) void k_attention_join_rows(const AttnArgs a) {
    constexpr int kLanes = D / 8, kPer = 64 / kLanes;
    const int lane = (int)threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t all = (int64_t)a.total_q * a.q_heads;
    if (row >= all) return;
    const int token = (int)(row / a.q_heads), head = (int)(row - (int64_t)token * a.q_heads), kvh = head / a.group;
    const float vg = a.c.vg[kvh];
    f32x4 o[BLOCK][2];
    float2 ml[BLOCK];
    const auto load = [&](int s0) {                          // parts s0 .. (past the last it again)
#pragma unroll
        for (int j = 0; j < BLOCK; ++j) {
            const int64_t at = min(s0 + kPer * j + lane / kLanes, a.splits - 1) * all + row;
            const float* const src = a.part_o + at * D + 4 * (lane % kLanes);
            ml[j] = a.part_ml[at];
            o[j][0] = *reinterpret_cast<const f32x4*>(src);
            o[j][1] = *reinterpret_cast<const f32x4*>(src + D / 2);
        }
    };
    load(0);
    const Query at = query_of(a, a.c.page_shift, token);
    if (at.b < 0 || at.index >= a.max_q_len) return;
    float top = kFloor, sum = 0.0f;
    f32x4 y[2] = {};
    for (int s0 = 0; s0 < a.splits; s0 += BLOCK * kPer) {
        if (s0 > 0) load(s0);
        float most = top;
#pragma unroll
        for (int j = 0; j < BLOCK; ++j) most = __builtin_fmaxf(most, ml[j].x);
#pragma unroll
        for (int bit = kLanes; bit < 64; bit <<= 1) most = __builtin_fmaxf(most, shfl_xor_f32(most, bit));
        const float f = __builtin_amdgcn_exp2f(top - most);
        top = most;
        sum *= f;
        y[0] *= f;
        y[1] *= f;
#pragma unroll
        for (int j = 0; j < BLOCK; ++j) {
            const bool there = s0 + kPer * j + lane / kLanes < a.splits;
            const float w = __builtin_amdgcn_exp2f(ml[j].x - top);
            sum = there ? __builtin_fmaf(ml[j].y, w, sum) : sum;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] = there ? __builtin_fmaf(o[j][e >> 2][e & 3], w, y[e >> 2][e & 3]) : y[e >> 2][e & 3];
        }
    }
#pragma unroll
    for (int bit = kLanes; bit < 64; bit <<= 1) {
        sum += shfl_xor_f32(sum, bit);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] += shfl_xor_f32(y[e >> 2][e & 3], bit);
    }
    if (lane >= kLanes) return;
    const Seq seq{0, token, 1};
    store_finished<D>(a, seq, kvh, head - kvh * a.group, 4 * lane, y[0], top, sum, vg);
    store_finished<D>(a, seq, kvh, head - kvh * a.group, D / 2 + 4 * lane, y[1], top, sum, vg);
}

template <int D>
static void launch_join_rows(const AttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.total_q * a.q_heads + 3) / 4));
    if (a.splits <= 4 * (64 / (D / 8)))
        hipLaunchKernelGGL((k_attention_join_rows<D, 4>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attention_join_rows<D, 9>), grid, dim3(256), 0, stream, a);
}
hipError_t launch_attention_join_rows(const AttnArgs& a, hipStream_t stream) {
    if (a.c.head_dim == 128)
        launch_join_rows<128>(a, stream);
    else
        launch_join_rows<64>(a, stream);
    return hipGetLastError();
}

template <int D, int NT, int G>
static void launch_pages_waves(const PagesAttnArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.total_q * a.c.kv_heads * a.row_tiles * a.splits));
    if (a.waves == 1)
        hipLaunchKernelGGL((k_attention_pages<D, NT, G, 1>), grid, dim3(64), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attention_pages<D, NT, G, 4>), grid, dim3(256), 0, stream, a);
}
template <int D>
static void launch_pages(const PagesAttnArgs& a, hipStream_t stream) {
    if (a.tile_rows == 16)
        a.c.page_shift >= 6 ? launch_pages_waves<D, 1, 1>(a, stream) : launch_pages_waves<D, 1, 4>(a, stream);
    else
        a.c.page_shift >= 6 ? launch_pages_waves<D, 2, 1>(a, stream) : launch_pages_waves<D, 2, 4>(a, stream);
}
hipError_t launch_attention_pages(const PagesAttnArgs& a, hipStream_t stream) {
    if (a.c.head_dim == 128)
        launch_pages<128>(a, stream);
    else
        launch_pages<64>(a, stream);
    return hipGetLastError();
}

}  // namespace mxq
