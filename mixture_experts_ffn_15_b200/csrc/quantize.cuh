// Rounding of a row to int8 with one scale (the arithmetic and its exactness: quantize.cu).
#pragma once

#include "common.cuh"

namespace moe {

struct RowQuant {
    float scale;   // amax / 127; NaN for a row with an infinity or a NaN
    float pre;     // a power of two that keeps 254 x and 127 / amax normal (1 for most rows)
    float amax;    // amax * pre
    float inv;     // 127 / (amax * pre); 0 for a row without a finite, non-zero maximum
};

// From the bits of max |x| of the row (a NaN's are above an infinity's).
__device__ __forceinline__ RowQuant row_quant(uint32_t amax_bits) {
    RowQuant r;
    const float amax = __uint_as_float(amax_bits);
    r.scale = __fdiv_rn(amax, 127.f);
    r.pre = amax < 1e-30f ? 0x1p64f : amax > 1e36f ? 0x1p-20f : 1.f;
    r.amax = amax * r.pre;
    r.inv = __fdiv_rn(127.f, r.amax);
    if (amax_bits == 0u) r.inv = 0.f;
    if (amax_bits >= 0x7f800000u) {
        r.scale = __uint_as_float(0x7fc00000u);
        r.inv = 0.f;
    }
    return r;
}

// v = m + 1/2 + (a little): the whole number nearest 127 |x| / amax, ties to even, from the
// sign of 254 |x| - (2 m + 1) amax, exact in float64 (32-bit products), for bf16 values
// already in float32 (16-bit products); signed as x.
template <bool BF16>
__device__ __forceinline__ int round_near_half(float x, float v, float amax) {
    const float a = fabsf(x);
    const int m = static_cast<int>(fabsf(v));
    bool up, tie;
    if constexpr (BF16) {
        const float l = 254.f * a, h = static_cast<float>(2 * m + 1) * amax;
        up = l > h;
        tie = l == h;
    } else {
        const double l = 254.0 * static_cast<double>(a);
        const double h = static_cast<double>(2 * m + 1) * static_cast<double>(amax);
        up = l > h;
        tie = l == h;
    }
    const int k = m + ((up || (tie && (m & 1))) ? 1 : 0);
    return x < 0.f ? -k : k;
}

// N values -> N whole numbers (in the low bytes of n).
template <bool BF16, int N>
__device__ __forceinline__ void quantize_n(const float* f, const RowQuant& r, uint32_t* n) {
    // x inv + 1.5 * 2^23, rounded once, holds the nearest whole number of x inv in its low
    // bits (two's complement)
    constexpr float kMagic = 12582912.f;
    bool near = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float x = f[i] * r.pre;
        const float t = fmaf(x, r.inv, kMagic);
        n[i] = __float_as_uint(t);
        near = near || fabsf(fmaf(x, r.inv, kMagic - t)) > 0.4999f;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = f[i] * r.pre;
            if (fabsf(fmaf(x, r.inv, kMagic - __uint_as_float(n[i]))) > 0.4999f)
                n[i] = static_cast<uint32_t>(round_near_half<BF16>(x, x * r.inv, r.amax));
        }
    }
    if (r.inv == 0.f) {   // an infinity or a NaN times 0 is no whole number
#pragma unroll
        for (int i = 0; i < N; ++i) n[i] = 0;
    }
}

// Low bytes of four words, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_s8x4(const uint32_t* n) {
    return __byte_perm(__byte_perm(n[0], n[1], 0x0040u), __byte_perm(n[2], n[3], 0x0040u), 0x5410u);
}

template <bool BF16>
__device__ __forceinline__ uint2 quantize8(const float* f, const RowQuant& r) {
    uint32_t n[8];
    quantize_n<BF16, 8>(f, r, n);
    return make_uint2(pack_s8x4(n), pack_s8x4(n + 4));
}

}  // namespace moe
