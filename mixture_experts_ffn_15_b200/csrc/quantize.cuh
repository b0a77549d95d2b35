// Rounding of a row to int8 with one scale (the arithmetic and its exactness: quantize.cu).
#pragma once

#include "common.cuh"

namespace moe {

struct RowQuant {
    float scale;   // amax / 127; NaN for a row with an infinity or a NaN
    float pre;     // a power of two that keeps 254 x and 127 / amax normal (1 for most rows)
    float amax;    // amax * pre
    float inv;     // 127 / (amax * pre) rounded up; 0 for a row without a finite, non-zero maximum
};

// From the bits of max |x| of the row (a NaN's are above an infinity's).
__device__ __forceinline__ RowQuant row_quant(uint32_t amax_bits) {
    RowQuant r;
    const float amax = __uint_as_float(amax_bits);
    r.scale = __fdiv_rn(amax, 127.f);
    r.pre = amax < 1e-30f ? 0x1p64f : amax > 1e36f ? 0x1p-20f : 1.f;
    r.amax = amax * r.pre;
    r.inv = __fdiv_ru(127.f, r.amax);
    if (amax_bits == 0u) r.inv = 0.f;
    if (amax_bits >= 0x7f800000u) {
        r.scale = __uint_as_float(0x7fc00000u);
        r.inv = 0.f;
    }
    return r;
}

// An ordinary row: 127 / amax and 254 x are normal numbers and nothing in it is infinite.
__device__ __forceinline__ bool ordinary(const RowQuant& r) { return r.pre == 1.f && r.inv != 0.f; }

// v = m + 1/2 + (a little): the whole number nearest 127 |x| / amax, ties to even, from the
// sign of 254 |x| - (2 m + 1) amax; signed as x.  Both products (at most 8 x 24 bits) as an
// unevaluated sum of two floats: the high parts are within a factor of 2 of each other and
// the low parts hold at most 8 bits, so that both differences and their sum are exact.
__device__ __forceinline__ int round_near_half(float x, float v, float amax) {
    const float a = fabsf(x);
    const int m = static_cast<int>(fabsf(v));
    const float w = static_cast<float>(2 * m + 1);
    const float h1 = 254.f * a, h2 = w * amax;
    const float d = (h1 - h2) + (fmaf(254.f, a, -h1) - fmaf(w, amax, -h2));
    const int k = m + ((d > 0.f || (d == 0.f && (m & 1))) ? 1 : 0);
    return x < 0.f ? -k : k;
}

// v is within |v| 2^-23 (the rounding of 127 / amax) of the exact quotient, at most 1.6e-5,
// and its distance from a whole number is computed exactly: at or below this distance the
// whole number is the nearest one.
constexpr float kSureDistance = 0.49998f;

// bf16 values need no look at that distance.  Where 254 x = (2 m + 1) amax does not hold, the
// quotient is at least 2^-16 of itself away from a half (the difference of two products of
// 8-bit significands is at least one unit), far more than v's error.  Where it does, 127
// divides 2 m + 1, so that m = 63, or amax's significand: for m = 63 (x = amax / 2) the even
// neighbour is the one above in magnitude, which 127 / amax rounded up gives; rows whose
// amax has the significand 254 are the exception.
__device__ __forceinline__ bool bf16_exception(uint32_t amax_bits) { return ((amax_bits >> 16) & 0x7fu) == 0x7eu; }

// The whole number nearest x inv, in the low byte of the result, and *far raised to its
// distance from x inv.  PLAIN: the row is ordinary (pre = 1).
template <bool PLAIN>
__device__ __forceinline__ uint32_t quantize_fast(float x, float pre, float inv, float* far) {
    // x inv + 1.5 * 2^23, rounded once, holds round-to-nearest-even of x inv in its low bits
    constexpr float kMagic = 12582912.f;
    if (!PLAIN) x *= pre;
    const float t = fmaf(x, inv, kMagic);
    *far = fmaxf(*far, fabsf(fmaf(x, inv, kMagic - t)));
    return __float_as_uint(t);
}

// The exact one, for any row; amax = r.amax of the row.
__device__ __forceinline__ uint32_t quantize_exact(float x, float pre, float inv, float amax) {
    if (inv == 0.f) return 0u;   // zeros; an infinity or a NaN times 0 is no whole number
    float far = 0.f;
    const uint32_t n = quantize_fast<false>(x, pre, inv, &far);
    x *= pre;
    return far > kSureDistance ? static_cast<uint32_t>(round_near_half(x, x * inv, amax)) : n;
}

// Low bytes of four words, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_s8x4(const uint32_t* n) {
    return __byte_perm(__byte_perm(n[0], n[1], 0x0040u), __byte_perm(n[2], n[3], 0x0040u), 0x5410u);
}

}  // namespace moe
