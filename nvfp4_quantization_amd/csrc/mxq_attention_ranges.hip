// mxq_attention_ranges.hip -- attention with shared prefixes over the paged NVFP4 cache
// (gfx950) for few query rows: up to 32 of a group's over its prefix, or of a sequence's over
// its own tokens, every 64-token tile by one wave as in mxq_attention_nvfp4.hip.
#include "mxq_attention_ranges_rows.hpp"

namespace mxq {

template <int D, int NT, int G, int W>
__global__ __launch_bounds__(64 * W, 8 / W) void k_attention_ranges(const PrefixAttnArgs a) {
    constexpr int kWave = WaveLds<D>::kBytes;
    constexpr int kJoin = (D / 16) * 64 * 16;
    constexpr int kArea = kWave > kJoin ? kWave : kJoin;
    __shared__ __attribute__((aligned(16))) uint8_t lds[W * kArea];
    __shared__ float2 join[W][NT * 16];
    __shared__ int limits[NT * 16];
    const RangeUnit u = range_unit<NT * 16>(a, (int)blockIdx.x, limits);
    if (u.rows > 0) range_rows<D, NT, G, W>(a, u, limits, [&](int w) { return lds + w * kArea; }, join);
}

template <int D, int NT, int G>
static void launch_ranges_waves(const PrefixAttnArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((k_attention_ranges<D, NT, G, 4>), dim3((unsigned)(a.prefix_blocks + a.own_blocks)), dim3(256), 0, stream, a);
}
template <int D>
static void launch_ranges(const PrefixAttnArgs& a, hipStream_t stream) {
    if (a.tile_rows == 16)
        a.c.page_shift >= 6 ? launch_ranges_waves<D, 1, 1>(a, stream) : launch_ranges_waves<D, 1, 4>(a, stream);
    else
        a.c.page_shift >= 6 ? launch_ranges_waves<D, 2, 1>(a, stream) : launch_ranges_waves<D, 2, 4>(a, stream);
}
hipError_t launch_attention_ranges_rows(const PrefixAttnArgs& a, hipStream_t stream) {
    if (a.c.head_dim == 128)
        launch_ranges<128>(a, stream);
    else
        launch_ranges<64>(a, stream);
    return hipGetLastError();
}

}  // namespace mxq
