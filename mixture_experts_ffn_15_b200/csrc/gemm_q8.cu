// Grouped products of int8 rows with int8 weights, scales per token and per channel:
//   out[r, n] = (sum_k a[r, k] w[e, n, k]) sa[r] sw[e, n] + bias[e, n]
// for the rows r of expert e (one expert and no offsets: a dense product).  The sum is
// exact in int32 (K <= 65536: |sum| <= 2^30); it is rounded to float32 once, scaled by the
// product of the two scales and, after the bias, rounded once to the output's type.
// With SwiGLU (fc1 of the expert FFN) the (gate, up) pairs of rows give one float32
// activation each.
#include "common.cuh"
#include "kernels.h"
#include "tile_map.cuh"

namespace moe {
namespace {

constexpr int QBM = 32, QBN = 64, QBK = 32;   // rows, columns, K words of 4 bytes

enum OutMode : int { OUT_F32 = 0, OUT_BF16 = 1, OUT_SWIGLU = 2 };

template <int MODE>
__global__ void __launch_bounds__(256)
q8_gemm_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa, const int8_t* __restrict__ W,
               const float* __restrict__ sw, const void* __restrict__ bias, const int32_t* offsets,
               int rows, int K, int E, int N, void* __restrict__ out, int32_t* err, SwigluAttr act,
               bool chunked) {
    __shared__ int sA[QBM][QBK + 1];
    __shared__ __align__(16) int sW[QBK][QBN + 4];
    __shared__ int s_off[kMaxExperts + 1];
    __shared__ int s_pre[kMaxExperts + 1];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (tid < 32) build_group_tiles(offsets, rows, err, E, QBM, s_off, s_pre, tid);
    __syncthreads();
    const int NT = (N + QBN - 1) / QBN;
    const long long total = static_cast<long long>(s_pre[E]) * NT;
    const int tx = tid & 15, ty = tid >> 4;
    const int KW = K / 4;
    for (long long u = blockIdx.x; u < total; u += gridDim.x) {
        const int mt = static_cast<int>(u / NT), nt = static_cast<int>(u - static_cast<long long>(mt) * NT);
        const int e = tile_group(mt, E, s_pre);
        const int row0 = s_off[e] + (mt - s_pre[e]) * QBM;
        const int nrows = min(QBM, s_off[e + 1] - row0);
        const int* We = reinterpret_cast<const int*>(W) + static_cast<size_t>(e) * N * KW;
        const int* Aw = reinterpret_cast<const int*>(A);
        int acc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        for (int k0 = 0; k0 < KW; k0 += QBK) {
            for (int i = tid; i < QBM * QBK; i += 256) {
                const int r = i / QBK, c = i % QBK;
                sA[r][c] = (r < nrows && k0 + c < KW) ? Aw[static_cast<size_t>(row0 + r) * KW + k0 + c] : 0;
            }
            for (int i = tid; i < QBN * QBK; i += 256) {
                const int n = i / QBK, c = i % QBK, wn = nt * QBN + n;
                const int wr = MODE == OUT_SWIGLU ? fc1_row(wn, N / 2, chunked) : wn;
                sW[c][n] = (wn < N && k0 + c < KW) ? We[static_cast<size_t>(wr) * KW + k0 + c] : 0;
            }
            __syncthreads();
#pragma unroll 8
            for (int c = 0; c < QBK; ++c) {
                const int a0 = sA[ty * 2][c], a1 = sA[ty * 2 + 1][c];
                const int4 w4 = *reinterpret_cast<const int4*>(&sW[c][tx * 4]);
                const int w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[0][j] = __dp4a(a0, w[j], acc[0][j]);
                    acc[1][j] = __dp4a(a1, w[j], acc[1][j]);
                }
            }
            __syncthreads();
        }
        const int n0 = nt * QBN + tx * 4;
        if (n0 >= N) continue;   // N is a multiple of 4: a thread's columns are all valid or none
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            const int r = ty * 2 + rr;
            if (r >= nrows) continue;
            const float s = sa[row0 + r];
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int wr = MODE == OUT_SWIGLU ? fc1_row(n0 + j, N / 2, chunked) : n0 + j;
                const size_t wi = static_cast<size_t>(e) * N + wr;
                float b = 0.f;
                if (bias) b = MODE == OUT_F32 ? static_cast<const float*>(bias)[wi]
                                              : bf16_at(static_cast<const __nv_bfloat16*>(bias), wi);
                y[j] = fmaf(static_cast<float>(acc[rr][j]), s * sw[wi], b);
            }
            const size_t o = static_cast<size_t>(row0 + r) * (MODE == OUT_SWIGLU ? N / 2 : N);
            if constexpr (MODE == OUT_SWIGLU) {
                *reinterpret_cast<float2*>(static_cast<float*>(out) + o + n0 / 2) =
                    make_float2(swiglu_attr(y[0], y[1], act), swiglu_attr(y[2], y[3], act));
            } else if constexpr (MODE == OUT_BF16) {
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + o + n0) =
                    make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(out) + o + n0) =
                    make_float4(y[0], y[1], y[2], y[3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    const long long bound = (static_cast<long long>((a.rows + QBM - 1) / QBM) + a.E) * ((a.N + QBN - 1) / QBN);
    const long long cap = static_cast<long long>(device_sm_count()) * 8;
    const dim3 grid(static_cast<unsigned>(bound < cap ? bound : cap)), block(256);
    auto go = [&](auto kern) {
        return launch_k(kern, grid, block, 0, s, a.a_q, a.a_scale, a.w_q, a.w_scale, a.bias, a.offsets,
                        a.rows, a.K, a.E, a.N, a.out, a.err, a.act, a.fc1_chunked);
    };
    if (a.swiglu) return go(q8_gemm_kernel<OUT_SWIGLU>);
    return a.out_bf16 ? go(q8_gemm_kernel<OUT_BF16>) : go(q8_gemm_kernel<OUT_F32>);
}

}  // namespace moe
