// f64 helpers: sums over a wavefront, and the reciprocal, reciprocal square root
// and exponential from the hardware's estimates and the series, without the
// special cases that the callers keep away.
#pragma once

#include "device_common.h"

namespace q4k {

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v)
{
    const u32x2 b = bitcast<u32x2>(v);
    return bitcast<double>((u32x2){(uint32_t)__builtin_amdgcn_mov_dpp((int)b.x, CTRL, 0xF, 0xF, false),
                                   (uint32_t)__builtin_amdgcn_mov_dpp((int)b.y, CTRL, 0xF, 0xF, false)});
}

__device__ __forceinline__ double readlane_f64(double v, int lane)
{
    const u32x2 b = bitcast<u32x2>(v);
    return bitcast<double>((u32x2){(uint32_t)__builtin_amdgcn_readlane((int)b.x, lane),
                                   (uint32_t)__builtin_amdgcn_readlane((int)b.y, lane)});
}

// The sum over the wavefront, in every lane, in a fixed order.
__device__ __forceinline__ double wave_sum_f64(double v)
{
    v += dpp_f64<0xB1>(v);    // quad_perm 1,0,3,2
    v += dpp_f64<0x4E>(v);    // quad_perm 2,3,0,1
    v += dpp_f64<0x141>(v);   // row_half_mirror
    v += dpp_f64<0x140>(v);   // row_mirror
    return (readlane_f64(v, 0) + readlane_f64(v, 16)) + (readlane_f64(v, 32) + readlane_f64(v, 48));
}

// The same over each 16 or 32 neighbouring lanes.
template <int L>
__device__ __forceinline__ double lanes_sum_f64(double v)
{
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    if constexpr (L == 32) {
        // Rows of 16 lanes 0 and 1, and 2 and 3, change places.
        const u32x2 b = bitcast<u32x2>(v);
        const auto lo = __builtin_amdgcn_permlane16_swap(b.x, b.x, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(b.y, b.y, false, false);
        v = bitcast<double>((u32x2){lo[0], hi[0]}) + bitcast<double>((u32x2){lo[1], hi[1]});
    }
    return v;
}

// 1 / sqrt(v) for normal v > 0: each Newton step squares the estimate's error
// (2^-14 at most at the start), to within 2^-51.
__device__ __forceinline__ double rsqrt_f64(double v)
{
    double r = __builtin_amdgcn_rsq(v);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = fma(r * 0.5, fma(-v * r, r, 1.0), r);
    return r;
}

// 1 / v for normal v with a normal reciprocal, to within 2^-51.
__device__ __forceinline__ double rcp_f64(double v)
{
    double r = __builtin_amdgcn_rcp(v);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = fma(r, fma(-v, r, 1.0), r);
    return r;
}

// exp(x) for |x| <= 700, to within 2^-51: x = n ln 2 + r, |r| <= 0.35 (ln 2 in two
// parts, the upper one of 42 bits, so that its product with n is exact), and the Taylor series of
// exp(r), whose first term left out is r^14 / 14! < 2^-57.
__device__ __forceinline__ double exp_f64(double x)
{
    const double n = __builtin_rint(x * 1.4426950408889634074);
    double r = fma(-n, 0x1.62e42fefa3800p-1, x);
    r = fma(-n, 0x1.ef35793c76730p-45, r);
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

}  // namespace q4k
