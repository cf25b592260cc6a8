// 2^x on the FMA and integer pipes, for a share of the serving kernels' exponentials.
#pragma once

#include "ptx_sm100.cuh"

namespace gqa {

// 2^x on two lanes at once on the FMA pipe: x = j + f with j the nearest integer, 2^f by the
// degree-4 polynomial with constant term 1 that has the least relative error on [-1/2, 1/2]
// (2.8e-6, a thousandth of the half step 2^-8 that P is rounded by next; an LSE moves by at most as
// much), and j added to the exponent.  x is at most 8 here; below -126 it counts as -126.  A NaN does
// not pass: the caller keeps account of those.
__device__ __forceinline__ void exp2_poly4(float x0, float x1, float& y0, float& y1) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it leaves j in the low bits
    constexpr float c1 = 0.6931241750717163f, c2 = 0.24024099111557007f, c3 = 0.055906426161527634f,
                    c4 = 0.009582853876054287f;
    x0 = fmaxf(x0, -126.f);
    x1 = fmaxf(x1, -126.f);
    float t0, t1, r0, r1, f0, f1, q0, q1;
    ptx::add2(x0, x1, kRound, kRound, t0, t1);
    ptx::add2(t0, t1, -kRound, -kRound, r0, r1);
    ptx::add2(x0, x1, -r0, -r1, f0, f1);
    ptx::fma2(f0, f1, c4, c4, c3, c3, q0, q1);
    ptx::fma2(q0, q1, f0, f1, c2, c2, q0, q1);
    ptx::fma2(q0, q1, f0, f1, c1, c1, q0, q1);
    ptx::fma2(q0, q1, f0, f1, 1.f, 1.f, q0, q1);
    y0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
    y1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}

}  // namespace gqa
