// mxq_rmsnorm_fp8.hip -- residual addition + RMS norm -> FP8 1x128 (gfx950).
//
// z = BF16(x + res); r = F(1 / sqrt(sum z^2 / n + eps)), in binary64 up to the one
// round of r; y = fl(fl(z r) w) in FP32, and the FP8 recipe of onnxruntime PR #33644
// (Description) on y with no round in between: s = max(amax, 1e-10) * F(1/448) per
// 1x128 group, y / s by FP32 division, saturating nearest-even E4M3.
//
// The sum is carried in binary64: a square of a BF16 value has 16 significant bits, so
// 53 bits hold the sums of a row's squares to 2^-38 or better in any order, and r (and
// with it every code) does not depend on how the row is spread over the threads.
//
// What bounds it: memory.  16384 x 7168 with a residual (1.06 GB in and out) take 183 us, 5.8
// TB/s (a kernel that moves the same bytes without the arithmetic: 193); a row stays in
// registers between the sum and the encode.
#include "mxq_device.hpp"
#include "mxq_serve.hpp"

namespace mxq {

namespace {

// Bytes equal to 0xFF (the conversion's code for a NaN input) become 0x7F.
__device__ __forceinline__ uint32_t nan_codes_to_7f(uint32_t c) {
    const uint32_t ff =
        c & (c >> 1) & (c >> 2) & (c >> 3) & (c >> 4) & (c >> 5) & (c >> 6) & (c >> 7) & 0x01010101u;
    return c ^ (ff * 0x80u);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

}  // namespace

// One work-group per row; thread t holds the 8-element chunks t, t + threads, ... (J of
// them), so 16 consecutive lanes hold one 1x128 group.
template <int J, bool RES, bool UE8M0>
__global__ __launch_bounds__(1024) void k_add_rmsnorm_quant_fp8(const RmsNormArgs a) {
    __shared__ double part[16];
    const int64_t row = blockIdx.x;
    const int chunks = a.n >> 3;
    uint4 z[J];
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (int)threadIdx.x + j * (int)blockDim.x;
        z[j] = make_uint4(0, 0, 0, 0);
        if (c < chunks) {
            z[j] = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + c * 8);
            if (RES) {
                const uint4 r = *reinterpret_cast<const uint4*>(a.res + row * a.ld_res + c * 8);
                z[j].x = pack_bf16(lo_bf16(z[j].x) + lo_bf16(r.x), hi_bf16(z[j].x) + hi_bf16(r.x));
                z[j].y = pack_bf16(lo_bf16(z[j].y) + lo_bf16(r.y), hi_bf16(z[j].y) + hi_bf16(r.y));
                z[j].z = pack_bf16(lo_bf16(z[j].z) + lo_bf16(r.z), hi_bf16(z[j].z) + hi_bf16(r.z));
                z[j].w = pack_bf16(lo_bf16(z[j].w) + lo_bf16(r.w), hi_bf16(z[j].w) + hi_bf16(r.w));
                *reinterpret_cast<uint4*>(a.res_out + row * a.ld_res_out + c * 8) = z[j];
            }
        }
        const uint32_t w[4] = {z[j].x, z[j].y, z[j].z, z[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double lo = lo_bf16(w[i]), hi = hi_bf16(w[i]);
            sum = __builtin_fma(lo, lo, sum);
            sum = __builtin_fma(hi, hi, sum);
        }
    }
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) sum += part[i];
    const float r = (float)(1.0 / __builtin_sqrt(sum / (double)a.n + (double)a.eps));

#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (int)threadIdx.x + j * (int)blockDim.x;
        const bool live = c < chunks;
        uint4 wv = make_uint4(0, 0, 0, 0);
        if (live) wv = *reinterpret_cast<const uint4*>(a.w + c * 8);
        const uint32_t zw[4] = {z[j].x, z[j].y, z[j].z, z[j].w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = (lo_bf16(zw[i]) * r) * lo_bf16(ww[i]);
            y[2 * i + 1] = (hi_bf16(zw[i]) * r) * hi_bf16(ww[i]);
        }
        float m = 0.0f;
        bool has_nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m = __builtin_fmaxf(m, __builtin_fabsf(y[i]));
            has_nan |= y[i] != y[i];
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) m = __builtin_fmaxf(m, shfl_xor_f32(m, o));
        float s = (m > k_floor() ? m : k_floor()) * k_inv448();
        if (UE8M0) s = pow2_ceil(s);
        const float inv = 1.0f / s, sd = fp8_divisor(s);
        const bool fix = has_nan || s == __builtin_inff();
        uint32_t q[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            q[i] = e4m3_pack4(div_rn(y[4 * i], sd, inv), div_rn(y[4 * i + 1], sd, inv), div_rn(y[4 * i + 2], sd, inv),
                              div_rn(y[4 * i + 3], sd, inv));
            if (fix) q[i] = nan_codes_to_7f(q[i]);
        }
        if (live) {
            *reinterpret_cast<uint2*>(a.q + row * a.ldq + c * 8) = make_uint2(q[0], q[1]);
            if ((c & 15) == 0) a.scales[row * a.srow + (int64_t)(c >> 4) * a.sgroup] = s;
            if (a.y)
                *reinterpret_cast<uint4*>(a.y + row * a.ld_y + c * 8) =
                    make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                               pack_bf16(y[6], y[7]));
        }
    }
}

template <int J>
static hipError_t launch_j(const RmsNormArgs& a, bool ue8m0, int waves, hipStream_t stream) {
    const dim3 grid((unsigned)a.m), block((unsigned)(64 * waves));
    if (a.res) {
        if (ue8m0)
            hipLaunchKernelGGL((k_add_rmsnorm_quant_fp8<J, true, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((k_add_rmsnorm_quant_fp8<J, true, false>), grid, block, 0, stream, a);
    } else {
        if (ue8m0)
            hipLaunchKernelGGL((k_add_rmsnorm_quant_fp8<J, false, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((k_add_rmsnorm_quant_fp8<J, false, false>), grid, block, 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_add_rmsnorm_quant_fp8(const RmsNormArgs& a, bool ue8m0, hipStream_t stream) {
    // Two chunks a thread hide more of each other's latency than twice the waves, which the
    // barrier stops together; past 16 steps four chunks keep the work-group within 16 waves.
    // 8192 rows with a residual, in us, for one / two / four chunks: n = 4096 49.5 / 46.8 / -,
    // 7168 91.0 / 77.0 / 79.7, 8192 95.9 / 83.1 / 87.9, 16384 - / 168.5 / 164.3.
    const int steps = (a.n / 8 + 63) / 64;                     // wave-wide chunks of a row: 1 .. 64
    if (steps <= 4) return launch_j<1>(a, ue8m0, steps, stream);
    if (steps <= 16) return launch_j<2>(a, ue8m0, (steps + 1) / 2, stream);
    return launch_j<4>(a, ue8m0, (steps + 3) / 4, stream);
}

}  // namespace mxq
