// mxq_rope_append.hip -- rotary positions on Q and K, then K and V into the paged NVFP4
// cache (gfx950).
//
// Angles are formed in binary64 (theta = fl(position * inv_freq), so a position of a
// million keeps its place on the circle to 2^-33) and reduced by Cody and Waite's method
// (Software Manual for the Elementary Functions, 1980) with pi/2 in two parts: the FMA
// keeps k * part exact, so the remainder in [-pi/4, pi/4] carries an error below 2^-52 for
// |theta| < 2^45 (others become NaN);
// sine and cosine are their Taylor polynomials to r^17 and r^16, whose first left-out
// terms are below 2^-56.  cos and sin are rounded to FP32 once, and one work-group's
// heads share them through LDS.
//
// The cache rows are the row-wise NVFP4 encode of the grouped call (TransformerEngine
// PR #2564: 1x16 E2M1 blocks with E4M3 scales) with a caller-supplied tensor scale per
// head.
//
// What bounds it: memory.  8191 tokens of 32 + 8 + 8 heads of 128 with the values written
// (211 MB) take 44 us, 4.8 TB/s, where a large copy reaches 5.4; a decoding step's 64
// tokens take 4.3 us on the GPU, less than a call.
#include "mxq_nvfp4_impl.hpp"
#include "mxq_serve.hpp"

namespace mxq {

namespace {

constexpr int kMaxPairs = 64;         // rot_dim / 2 at head_dim 128

// cos and sin of theta; NaN unless |theta| < 2^45 (past 2^50 the multiple of pi/2 would not be
// the nearest one any more, past 2^53 not a whole number's).
__device__ __forceinline__ void sincos_stated(double theta, double& c, double& s) {
    if (!(__builtin_fabs(theta) < 0x1p45)) theta = __builtin_nan("");
    const double k = __builtin_rint(theta * 0x1.45f306dc9c883p-1);              // 2/pi
    double r = __builtin_fma(-k, 0x1.921fb54442d18p+0, theta);                  // pi/2, high part
    r = __builtin_fma(-k, 0x1.1a62633145c07p-54, r);                            // and the rest
    const double t = r * r;
    double p = 1.0 / 355687428096000.0;                                         // 1/17!
    p = __builtin_fma(p, t, -1.0 / 1307674368000.0);
    p = __builtin_fma(p, t, 1.0 / 6227020800.0);
    p = __builtin_fma(p, t, -1.0 / 39916800.0);
    p = __builtin_fma(p, t, 1.0 / 362880.0);
    p = __builtin_fma(p, t, -1.0 / 5040.0);
    p = __builtin_fma(p, t, 1.0 / 120.0);
    p = __builtin_fma(p, t, -1.0 / 6.0);
    const double sn = __builtin_fma(p * t, r, r);
    double u = 1.0 / 20922789888000.0;                                          // 1/16!
    u = __builtin_fma(u, t, -1.0 / 87178291200.0);
    u = __builtin_fma(u, t, 1.0 / 479001600.0);
    u = __builtin_fma(u, t, -1.0 / 3628800.0);
    u = __builtin_fma(u, t, 1.0 / 40320.0);
    u = __builtin_fma(u, t, -1.0 / 720.0);
    u = __builtin_fma(u, t, 1.0 / 24.0);
    u = __builtin_fma(u, t, -0.5);
    const double cs = __builtin_fma(u, t, 1.0);
    const double quad = k - 4.0 * __builtin_floor(k * 0.25);                    // 0, 1, 2 or 3, exactly
    const bool swap = quad == 1.0 || quad == 3.0;
    c = swap ? sn : cs;
    s = swap ? cs : sn;
    if (quad == 1.0 || quad == 2.0) c = -c;
    if (quad >= 2.0) s = -s;
}

// 16 bytes of an output that the call does not read again, past the L2 (8191 tokens of 48
// head rows: 44.6 us against 48.1 with ordinary stores).
typedef uint32_t u32x4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void put16(uint16_t* p, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    __builtin_nontemporal_store(u32x4s{x, y, z, w}, reinterpret_cast<u32x4s*>(p));
}

// 8 BF16 values of a chunk.
__device__ __forceinline__ void widen8(const uint4& w, float (&v)[8]) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_bf16(p[i]);
        v[2 * i + 1] = hi_bf16(p[i]);
    }
}

// The divisions' corrected quotients need steps, inverses and residuals that are normal.  Under
// a tensor scale g outside [2^-64, 2^64] both operands of each are brought there by this power
// of two first: exactly, after their own roundings, or with a result (a scale or a code of
// zero, or a saturated one) that no rounding can change.
__device__ __forceinline__ float mid_power(float g) { return g < 0x1p-64f ? 0x1p64f : g > 0x1p64f ? 0x1p-64f : 1.0f; }
// block_code() of a scaled fl(a * F(1/6)) and g.
__device__ __forceinline__ uint32_t scale_code(float a6, float g, float yg) {
    return e4m3_code(__builtin_elementwise_minimum(div_ieee(a6, g, yg), 448.0f)) & 0x7Fu;
}

// E2M1 value of a code's magnitude bits, signed.
__device__ __forceinline__ float e2m1_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2 ? 0.5f * (float)m : __builtin_bit_cast(float, (126u + (m >> 1)) << 23 | (m & 1u) << 22);
    return (c & 8u) ? -v : v;
}

}  // namespace

// A head row is held by head_dim / 8 consecutive lanes, 8 elements each; a row's lanes
// never leave their wave, so Q may be rotated in place (every lane has read its own and
// its pair's elements before any lane of the wave stores).  Rows of a token: q_heads of
// Q, kv_heads of K, kv_heads of V.
template <int D, bool INTERLEAVED>
__global__ __launch_bounds__(256) void k_rope_append_nvfp4(const RopeAppendArgs a, int splits) {
    constexpr int kLanes = D / 8, kRows = 256 / kLanes;
    __shared__ float2 cs[kMaxPairs];
    const int64_t t = blockIdx.x / (unsigned)splits;
    const int split = (int)(blockIdx.x % (unsigned)splits);
    const int half = a.rot_dim >> 1;
    if ((int)threadIdx.x < half) {
        double c, s;
        sincos_stated((double)a.positions[t] * a.inv_freq[threadIdx.x], c, s);
        cs[threadIdx.x] = make_float2((float)(a.factor * c), (float)(a.factor * s));
    }
    __syncthreads();
    const int rows = a.q_heads + 2 * a.c.kv_heads;
    const int e0 = ((int)threadIdx.x % kLanes) * 8;
    const int64_t slot = a.slots[t];
    const bool keep = slot >= 0 && slot < (a.c.num_pages << a.c.page_shift);
    const int64_t page = slot >> a.c.page_shift, off = slot & ((1ll << a.c.page_shift) - 1);

    for (int row = split * kRows + (int)threadIdx.x / kLanes; row < rows; row += splits * kRows) {
        const bool is_q = row < a.q_heads, is_v = row >= a.q_heads + a.c.kv_heads;
        const int head = is_q ? row : is_v ? row - a.q_heads - a.c.kv_heads : row - a.q_heads;
        const uint16_t* src = (is_q ? a.q + t * a.ld_q : is_v ? a.v + t * a.ld_v : a.k + t * a.ld_k) + head * D;
        uint4 w = *reinterpret_cast<const uint4*>(src + e0);
        if (!is_v && e0 < a.rot_dim) {
            float x[8], o[8];
            widen8(w, x);
            if (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = cs[e0 / 2 + i];
                    o[2 * i] = x[2 * i] * f.x - x[2 * i + 1] * f.y;
                    o[2 * i + 1] = x[2 * i + 1] * f.x + x[2 * i] * f.y;
                }
            } else {
                const bool second = e0 >= half;
                const int p0 = second ? e0 - half : e0;
                float other[8];
                widen8(*reinterpret_cast<const uint4*>(src + (second ? e0 - half : e0 + half)), other);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 f = cs[p0 + i];
                    o[i] = second ? x[i] * f.x + other[i] * f.y : x[i] * f.x - other[i] * f.y;
                }
            }
            w = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
        }
        if (is_q) {
            put16(a.q_out + t * a.ld_q_out + head * D + e0, w.x, w.y, w.z, w.w);
            continue;
        }
        // K or V: two lanes share a 1x16 block
        float y[8];
        widen8(w, y);
        float m = 0.0f;                              // NaN when the block holds one
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __builtin_elementwise_maximum(m, __builtin_fabsf(y[i]));
        m = __builtin_elementwise_maximum(m, shfl_xor_f32(m, 1));
        const float g = (is_v ? a.c.vg : a.c.kg)[head];
        const float up = mid_power(g), gu = g * up;
        const uint32_t sc = scale_code(m * k_inv6() * up, gu, 1.0f / gu);
        const float d = e4m3_value(sc) * g, du = d * up;
        float yu[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) yu[i] = y[i] * up;
        const u32x4 none = {0, 0, 0, 0};
        uint32_t codes = encode8<Enc::Div, true>(yu, du, 1.0f / du, none, 0);
        if (sc == 0 || sc == 0x7Fu) codes = 0;
        if (keep) {
            uint8_t* cp = (is_v ? a.c.vc : a.c.kc) + page * a.c.cs_page + head * a.c.cs_head + off * a.c.cs_tok;
            uint8_t* sp = (is_v ? a.c.vs : a.c.ks) + page * a.c.ss_page + head * a.c.ss_head + off * a.c.ss_tok;
            *reinterpret_cast<uint32_t*>(cp + e0 / 2) = codes;
            if ((e0 & 8) == 0) sp[e0 >> 4] = (uint8_t)sc;
        }
        uint16_t* values = is_v ? a.v_values : a.k_values;
        if (values) {
            uint32_t p[4];
            const float sv = e4m3_value(sc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                p[i] = pack_bf16((e2m1_value(codes >> (8 * i)) * sv) * g, (e2m1_value(codes >> (8 * i + 4)) * sv) * g);
            put16(values + (t * a.c.kv_heads + head) * D + e0, p[0], p[1], p[2], p[3]);
        }
    }
}

hipError_t launch_rope_append_nvfp4(const RopeAppendArgs& a, bool interleaved, hipStream_t stream) {
    const int rows = a.q_heads + 2 * a.c.kv_heads, per = 256 / (a.c.head_dim / 8);
    const int steps = (rows + per - 1) / per;
    // few tokens: a work-group per 256 lanes of each, which forms the angles again (48 head
    // rows, kernel times in us for one / several, with the values written: 64 tokens 5.0 / 4.3,
    // 512 6.1 / 6.0, 1024 8.3 / 9.0, 8191 44.6 / 51.3; without them 4.7 / 3.8, 5.6 / 5.2,
    // 7.3 / 8.4, 38.3 / 44.9)
    const int splits = a.tokens >= 1024 ? 1 : steps;
    const dim3 grid((unsigned)(a.tokens * splits));
    if (a.c.head_dim == 128) {
        if (interleaved)
            hipLaunchKernelGGL((k_rope_append_nvfp4<128, true>), grid, dim3(256), 0, stream, a, splits);
        else
            hipLaunchKernelGGL((k_rope_append_nvfp4<128, false>), grid, dim3(256), 0, stream, a, splits);
    } else {
        if (interleaved)
            hipLaunchKernelGGL((k_rope_append_nvfp4<64, true>), grid, dim3(256), 0, stream, a, splits);
        else
            hipLaunchKernelGGL((k_rope_append_nvfp4<64, false>), grid, dim3(256), 0, stream, a, splits);
    }
    return hipGetLastError();
}

}  // namespace mxq
