// fp8.cuh — e4m3 values and the power-of-two scales of a cache that holds them.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace gbattn {

// Scales are 2^-48 to 2^48 (a float whose mantissa is zero): wide enough for any
// activation, and weights of two blocks can be added up in fp32 whatever their scales.
constexpr int kLeastScale = -48, kMostScale = 48;

// Two e4m3 values (low byte first) to two fp16, which hold every e4m3 exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return r;
}

// Sixteen e4m3 values to eight pairs of fp16.
__device__ __forceinline__ void e4m3x16_to_f16(const uint4& v, uint32_t (&w)[8]) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
            : "r"(x[i]));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 2^e as a float, e in [-126, 127].
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Exponent of a scale given by its bits (sign and mantissa ignored), within the range.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    return min(max(static_cast<int>((bits >> 23) & 0xffu) - 127, kLeastScale), kMostScale);
}
// A float that is not a power of two (or zero, as a cache never written to has).
__device__ __forceinline__ bool bad_scale(uint32_t bits) {
    return (bits & 0x807fffffu) != 0 || bits == 0x7f800000u;
}

// A factor of scores, kept in fp32's normal numbers: a masked score (-inf) times 0 would be
// NaN, and so would a score of 0 times infinity.  What it moves at either end is a
// score below 2^-90 or far past what exp2 can tell apart.
__device__ __forceinline__ float score_factor(float f) { return fminf(fmaxf(f, 0x1p-126f), 3.402823466e38f); }

// The smallest exponent e in range with x <= 448 2^e, x >= 0 given by its bits:
// 448 = 1.75 x 2^8, so one more than x's own exponent less 8 where its mantissa exceeds 1.75.
__device__ __forceinline__ int fit_exponent(uint32_t bits) {
    return min(max(static_cast<int>((bits + 0x1fffffu) >> 23) - 135, kLeastScale), kMostScale);
}

}  // namespace gbattn
