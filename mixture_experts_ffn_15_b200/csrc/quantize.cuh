// Rounding of a row to int8 with one scale (the arithmetic and its exactness: quantize.cu).
#pragma once

#include "common.cuh"

namespace moe {

struct RowQuant {
    float scale;   // amax / 127; NaN for a row with an infinity or a NaN
    float inv;     // 127 / amax
    float amax;
    bool plain;    // amax in the range where float32 products keep their full precision
};

// From the bits of max |x| of the row (a NaN's are above an infinity's).
__device__ __forceinline__ RowQuant row_quant(uint32_t amax_bits) {
    RowQuant r;
    r.amax = __uint_as_float(amax_bits);
    r.scale = __fdiv_rn(r.amax, 127.f);
    r.inv = __fdiv_rn(127.f, r.amax);
    // outside: zero rows, rows of subnormals, rows beyond float32 (127 / amax subnormal)
    r.plain = r.amax > 1e-30f && r.amax < 1e37f;
    if (amax_bits >= 0x7f800000u) {
        r.scale = __uint_as_float(0x7fc00000u);
        r.amax = 0.f;
    }
    return r;
}

// One value by its float64 quotient (0 for a row without a finite, non-zero maximum).
__device__ __noinline__ int quantize_exact(float x, float amax) {
    if (!(amax > 0.f)) return 0;
    return __double2int_rn(127.0 * static_cast<double>(x) / static_cast<double>(amax));
}

// Eight values -> eight int8, the first in the lowest byte.
__device__ __forceinline__ uint2 quantize8(const float* f, const RowQuant& r) {
    // v + 1.5 * 2^23 leaves round-to-nearest-even of v in the low bits (two's complement)
    constexpr float kMagic = 12582912.f;
    uint32_t n[8];
    bool near = !r.plain;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = f[i] * r.inv;
        const float t = v + kMagic;
        n[i] = __float_as_uint(t);
        near = near || fabsf(v - (t - kMagic)) > 0.4999f;
    }
    if (near) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) n[i] = static_cast<uint32_t>(quantize_exact(f[i], r.amax));
    }
    uint2 o;
    o.x = __byte_perm(__byte_perm(n[0], n[1], 0x0040u), __byte_perm(n[2], n[3], 0x0040u), 0x5410u);
    o.y = __byte_perm(__byte_perm(n[4], n[5], 0x0040u), __byte_perm(n[6], n[7], 0x0040u), 0x5410u);
    return o;
}

}  // namespace moe
