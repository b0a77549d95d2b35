// int8 rows with one float32 scale each (symmetric, per token):
//   amax_r = max_k |x[r, k]|,  scale[r] = amax_r / 127 (float32 division),
//   q[r, k] = 127 x[r, k] / amax_r rounded to the nearest whole number, ties to even.
// A row of zeros has scale 0 and q = 0; a row that holds an infinity or a NaN has scale
// NaN and q = 0, so that whatever is multiplied with it comes out NaN, as it would in
// floating point.
//
// The whole number is the exact one, for every float32 and bf16 input.  v = x (127 / amax) in
// float32 is within 1.6e-5 of the exact quotient, so its rounding can be wrong only where v
// lies within that distance of a half.  A thread that meets such a float32 value (one value
// in 25000 is within 2e-5 of a half) does its part of the row again, deciding each such value
// by the sign of 254 |x| - (2 m + 1) amax, m the whole part, exact in pairs of floats.  For
// bf16 the first rounding is exact (quantize.cuh says why), which matters: x = amax / 2 is a
// half, and one value in 600 of a normal row is.
//
// With perm_dst, row t's int8 row and scale go to every row perm_dst[t k + j] instead (the
// permuted rows of the layer: the token rows are read and rounded once, not k times).
//
// One pass over the row: a row's threads keep their vectors of 8 elements in registers
// between the maximum and the rounding (rows longer than kRegVec vectors a thread read the
// rest again, from L2).  Bound by HBM: rows K (2 or 4) bytes read, rows (K + 4) written.
// Measured: 65536 x 2816 bf16 88 us, 6.3 TB/s; 65536 x 704 float32 38 us, 6.1 TB/s (65536 x
// 2816 in an earlier form of 100 us: the quotient in float64 309 us, a branch a value for those
// near a half 130 us).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "quantize.cuh"

namespace moe {
namespace {

constexpr int kMaxTpr = 256;
// Threads of a block: 64 where a row's threads are no more, since a small block's registers
// go to the next one as soon as its rows are out (blocks of 256: 65536 x 1536 float32 91 us
// instead of 74, 65536 x 704 55 instead of 41).  Short float32 rows are held to 64 registers
// a thread for more rows in flight (65536 x 704: 38 us; longer ones would spill, 74 -> 87 us).
__host__ __device__ constexpr int block_threads(int tpr) { return tpr > 64 ? tpr : 64; }
constexpr int kFew = 4;                  // vectors a thread of a short row
__host__ __device__ constexpr int min_blocks(bool bf16, int tpr, int vec) {
    return !bf16 && vec == kFew ? 1024 / block_threads(tpr) : 1;
}

template <bool BF16>
struct Vec8 {
    uint4 a, b;   // bf16: a only
    __device__ __forceinline__ void load(const void* x, size_t row, int nvec, int v) {
        if constexpr (BF16) {
            a = __ldg(reinterpret_cast<const uint4*>(x) + row * nvec + v);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(x) + (row * nvec + v) * 2;
            a = __ldg(p);
            b = __ldg(p + 1);
        }
    }
    __device__ __forceinline__ void get(float* f) const {
        if constexpr (BF16) {
            unpack_bf16x8(a, f);
        } else {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        }
    }
    // bits of the largest |element|, as float32 (a NaN is larger than an infinity)
    __device__ __forceinline__ uint32_t amax() const {
        if constexpr (BF16) {
            // two 16-bit magnitudes at a time
            const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu),
                                        __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
            return max(m & 0xffff0000u, m << 16);
        } else {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
    }
};

// TPR threads (a power of two, 32 .. 256) share a row, kRegVec vectors a thread in registers.
template <bool BF16, int TPR, int kRegVec, bool SCATTER>
__global__ void __launch_bounds__(block_threads(TPR), min_blocks(BF16, TPR, kRegVec))
quantize_rows_kernel(const void* __restrict__ x, int rows, int K, int8_t* __restrict__ q, int ldq,
                     float* __restrict__ scale, const int32_t* __restrict__ perm_dst, int k, int rows_out,
                     int32_t* __restrict__ clear, int clear_words) {
    constexpr int kQThreads = block_threads(TPR), kRows = kQThreads / TPR;   // rows of a block
    __shared__ uint32_t s_max[kQThreads / 32];
    pdl_wait();
    pdl_trigger();
    // 64 bits: 2^30 rows make more than 2^31 threads
    for (long long i = static_cast<long long>(blockIdx.x) * kQThreads + threadIdx.x; i < clear_words;
         i += static_cast<long long>(gridDim.x) * kQThreads)
        clear[i] = 0;
    const int nvec = K / 8;
    const int t = threadIdx.x % TPR;
    const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
    const bool live = row < rows;
    Vec8<BF16> r[kRegVec];
    uint32_t m = 0;
    if (live) {
#pragma unroll
        for (int j = 0; j < kRegVec; ++j)
            if (t + j * TPR < nvec) r[j].load(x, row, nvec, t + j * TPR);
#pragma unroll
        for (int j = 0; j < kRegVec; ++j)
            if (t + j * TPR < nvec) m = max(m, r[j].amax());
        for (int v = t + kRegVec * TPR; v < nvec; v += TPR) {
            Vec8<BF16> w;
            w.load(x, row, nvec, v);
            m = max(m, w.amax());
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
        __syncthreads();
        const int w0 = (threadIdx.x / TPR) * (TPR / 32);
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) m = max(m, s_max[w0 + i]);
    }
    if (!live) return;
    const RowQuant rq = row_quant(m);
    // copies of the row: k permuted ones, or itself
    auto each = [&](auto fn) {
        if constexpr (!SCATTER) {
            fn(row);
            return;
        }
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int to = __ldg(perm_dst + row * k + j);
            if (static_cast<unsigned>(to) < static_cast<unsigned>(rows_out)) fn(static_cast<long long>(to));
        }
    };
    if (t == 0) each([&](long long to) { scale[to] = rq.scale; });
    uint2* out = reinterpret_cast<uint2*>(q);
    const int ldv = ldq / 8;
    bool sure = ordinary(rq) && !(BF16 && bf16_exception(m));
    if (sure) {
        float far = 0.f, f[8];
        auto put = [&](const Vec8<BF16>& w, int v) {
            uint32_t n[8];
            w.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = quantize_fast<true>(f[i], 1.f, rq.inv, &far);
            if (BF16) far = 0.f;
            const uint2 o = make_uint2(pack_s8x4(n), pack_s8x4(n + 4));
            each([&](long long to) { out[to * ldv + v] = o; });
        };
#pragma unroll
        for (int j = 0; j < kRegVec; ++j)
            if (t + j * TPR < nvec) put(r[j], t + j * TPR);
        for (int v = t + kRegVec * TPR; v < nvec; v += TPR) {
            Vec8<BF16> w;
            w.load(x, row, nvec, v);
            put(w, v);
        }
        sure = far <= kSureDistance;
    }
    if (!sure) {
#pragma unroll 1
        for (int v = t; v < nvec; v += TPR) {
            Vec8<BF16> w;
            float f[8];
            uint32_t n[8];
            w.load(x, row, nvec, v);
            w.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = quantize_exact(f[i], rq.pre, rq.inv, rq.amax);
            const uint2 o = make_uint2(pack_s8x4(n), pack_s8x4(n + 4));
            each([&](long long to) { out[to * ldv + v] = o; });
        }
    }
}

template <bool BF16>
cudaError_t launch(const QuantizeArgs& a, cudaStream_t s) {
    const int rows = a.rows, K = a.K;
    const int nvec = K / 8;
    auto go = [&](auto kern, int tpr) {
        const int threads = block_threads(tpr), per = threads / tpr;
        return launch_k(kern, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(threads), 0, s, a.x,
                        rows, K, a.q, a.ldq ? a.ldq : K, a.scale, a.perm_dst, a.k, a.rows_out, a.clear, a.clear_words);
    };
    // Many rows: as few threads a row as hold it in registers, for many loads in flight and
    // no barrier.  Few rows (less than 1024 threads an SM): spread a row, for latency.
    constexpr int kReg = BF16 ? 12 : 6;
    const long long sms = device_sm_count();
    int tpr = 32;
    while (tpr < kMaxTpr && (tpr * kReg < nvec || (tpr < nvec && static_cast<long long>(rows) * tpr < 1024 * sms)))
        tpr *= 2;
    const bool few = tpr * kFew >= nvec;
    auto pick = [&](auto scatter) {
        constexpr bool S = decltype(scatter)::value;
        switch (tpr) {
            case 32: return few ? go(quantize_rows_kernel<BF16, 32, kFew, S>, 32) : go(quantize_rows_kernel<BF16, 32, kReg, S>, 32);
            case 64: return few ? go(quantize_rows_kernel<BF16, 64, kFew, S>, 64) : go(quantize_rows_kernel<BF16, 64, kReg, S>, 64);
            case 128:
                return few ? go(quantize_rows_kernel<BF16, 128, kFew, S>, 128) : go(quantize_rows_kernel<BF16, 128, kReg, S>, 128);
            default:
                return few ? go(quantize_rows_kernel<BF16, 256, kFew, S>, 256) : go(quantize_rows_kernel<BF16, 256, kReg, S>, 256);
        }
    };
    if constexpr (BF16) {
        if (a.perm_dst) return pick(std::true_type());
    } else if (a.perm_dst) {
        return cudaErrorInvalidValue;   // the layer's input is bf16
    }
    return pick(std::false_type());
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantizeArgs& a, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    return a.bf16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
