// quant8.cuh -- 8-bit codes of fp16 values, shared by the token quantiser and
// the key/value cache.
//
// A code is rint(fp32(x / s)), both in IEEE fp32.  It is computed without a
// division: with inv = fp32(1 / s), r = x inv rounded to an integer by adding
// 1.5 2^23 in one fused step, and the distance x inv - r.  |x / s| <= 127 (1 +
// 2^-24), so x inv is off the quotient, and the quotient off its rounding to
// fp32, by 7.6e-6 each at most: where the distance is at most 0.49998 both round
// to r.  Elsewhere (one value in 25,000) the quotient is divided out.  An IEEE
// division for every value made these kernels ALU-bound.
#pragma once

#include "common.cuh"

namespace glowq {

__device__ __forceinline__ uint32_t code8_exact(float x, float s) {
    return __float_as_uint(rintf(__fdiv_rn(x, s)) + 12582912.f);
}
// Codes of 8 consecutive values (s > 0 finite, |x| <= 127 s (1 + 2^-24)).
__device__ __forceinline__ uint2 codes8(const uint4& u, float s, float inv) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float far = 0.f;
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        const float t0 = fmaf(f.x, inv, 12582912.f), t1 = fmaf(f.y, inv, 12582912.f);
        far = max3(far, fabsf(fmaf(f.x, inv, 12582912.f - t0)), fabsf(fmaf(f.y, inv, 12582912.f - t1)));
        m[2 * i] = __float_as_uint(t0);
        m[2 * i + 1] = __float_as_uint(t1);
    }
    if (far > 0.49998f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(u32_as_h2(w[i]));
            m[2 * i] = code8_exact(f.x, s);
            m[2 * i + 1] = code8_exact(f.y, s);
        }
    }
    return make_uint2(__byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410));
}
// Largest magnitude of 8 values, taken into `amax`; NaN stays NaN.
__device__ __forceinline__ void amax8(const uint4& u, __half2& amax) {
    const __half2 a = __hmax2_nan(__habs2(u32_as_h2(u.x)), __habs2(u32_as_h2(u.y)));
    const __half2 b = __hmax2_nan(__habs2(u32_as_h2(u.z)), __habs2(u32_as_h2(u.w)));
    amax = __hmax2_nan(amax, __hmax2_nan(a, b));
}
// The larger of the two, as fp32: infinity or NaN where a value was not finite.
__device__ __forceinline__ float amax_float(__half2 amax) {
    return __half2float(__hmax_nan(__low2half(amax), __high2half(amax)));
}

}  // namespace glowq
