// Products of int8 rows with int8 weights on the tensor cores (tcgen05 kind::i8), scales
// per row and per channel, grouped by expert (one expert and no offsets: a dense product):
//   out[r, n] = (sum_k a[r, k] w[e, n, k]) sa[r] sw[e, n] + bias[e, n]
// The sum is exact in int32 (K <= 65536: |sum| <= 2^30); it is rounded to float32 once,
// scaled by the product of the two scales and, after the bias, rounded once to the output's
// type.  With SwiGLU (fc1 of the expert FFN) the (gate, up) pairs of rows give one float32
// activation each, not rounded further: it is cut to 8 bits next, and 16-bit activations
// would move one in ten of those whole numbers.
//
// Both kernels put the WEIGHT rows on the MMA's M side and the tokens on N, so that a few
// tokens cost a few columns, not a tile of rows:
//   q8_stream_kernel  128 weight rows x up to 64 tokens per CTA: few rows per expert, each
//                     weight byte read once, bound by HBM
//   q8_pair_kernel    256 weight rows x up to 256 tokens per pair of CTAs: many rows per
//                     expert, bound by what an SM takes in from L2
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tile_map.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kBK = tmap::kBoxK8;    // K per ring slot: one 128-byte row
constexpr uint64_t kWaitNs = 2000000000ull;

enum OutMode : int { OUT_F32 = 0, OUT_BF16 = 1, OUT_SWIGLU = 2 };

struct Q8Params {
    const int32_t* offsets;   // [E+1] device, or nullptr: one group of `rows` rows
    int E, rows, K, N;
    const float* sa;          // [rows]
    const float* sw;          // [E, N]
    const void* bias;         // [E, N] or nullptr
    void* out;                // [rows, N] (SwiGLU: [rows, N / 2] float32)
    int32_t* err;
    SwigluAttr act;
    bool chunked;             // SwiGLU: scales and bias in the chunked layout
};

// Scale and bias of weight row wr (SwiGLU: in interleaved order) of expert g.
template <int MODE>
__device__ __forceinline__ void channel(const Q8Params& p, int g, int wr, float* scale, float* bias) {
    const int row = MODE == OUT_SWIGLU ? fc1_row(wr, p.N / 2, p.chunked) : wr;
    const size_t i = static_cast<size_t>(g) * p.N + row;
    *scale = p.sw[i];
    *bias = 0.f;
    if (p.bias)
        *bias = MODE == OUT_F32 ? static_cast<const float*>(p.bias)[i]
                                : bf16_at(static_cast<const __nv_bfloat16*>(p.bias), i);
}

// Output of one weight row and one token.
template <int MODE>
__device__ __forceinline__ void store_one(const Q8Params& p, int row, int wr, float y, bool valid) {
    if (!valid) return;
    const size_t o = static_cast<size_t>(row) * p.N + wr;
    if constexpr (MODE == OUT_BF16) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(y);
    else static_cast<float*>(p.out)[o] = y;
}

// --------------------------------------------------------------------- few rows: stream
// Six warps a CTA: 0 the TMA producer, 1 the MMA issuer, 2-5 the epilogue (warp w reads
// tensor-memory lanes 32 (w % 4) .. +31, one weight row a lane).  Units (64-token chunk x
// 128 weight rows) are strided over the clusters.  A cluster of CS CTAs shares one unit
// along K when there are too few units for the SMs (one unit a cluster then): every CTA
// accumulates its slices, sends its partial sums to the CTA that owns those tokens (whole
// numbers: any order gives the same sum) and finishes its own tokens.
constexpr int kSTok = 64;                       // tokens per chunk
constexpr int kSBox = 16;                       // token rows per TMA box
constexpr int kSWRows = 128;
constexpr int kSSub = 2;                        // slots per barrier stage
constexpr int kSMaxStages = 4;
// ring slots: what fits (a split unit has few K slices a CTA, and needs room for the sums)
__host__ __device__ constexpr int stream_slots(bool split) { return kSSub * (split ? 3 : kSMaxStages); }
constexpr int kSABytes = kSWRows * kBK;
constexpr int kSBBytes = kSTok * kBK;
constexpr int kSThreads = 192;
// partial sums of one unit (cs > 1): for each source CTA and weight row the 64 / cs tokens of
// this CTA, rows padded by 16 bytes against bank conflicts (cs = 8: 8 x 128 x 12 words)
constexpr int kSPartBytes = 8 * kSWRows * (kSTok / 8 + 4) * 4;
constexpr int kSMiscBytes = (2 * kSMaxStages + 4) * 8 + 16 + 2 * (kMaxExperts + 1) * 4 + 64;

constexpr int stream_smem(bool split) {
    return 1024 + stream_slots(split) * (kSABytes + kSBBytes) + (split ? kSPartBytes : 0) + kSMiscBytes;
}
static_assert(stream_smem(true) <= 227 * 1024, "shared memory");

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(kSThreads, 1)
q8_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                 const Q8Params p, const int cs) {
    constexpr int kSSlots = stream_slots(SPLIT), kSStages = kSSlots / kSSub;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kSSlots * kSABytes;
    int* s_part = reinterpret_cast<int*>(sB + kSSlots * kSBBytes);   // SPLIT
    uint64_t* full = reinterpret_cast<uint64_t*>(sB + kSSlots * kSBBytes + (SPLIT ? kSPartBytes : 0));
    uint64_t* empty = full + kSStages;
    uint64_t* tfull = empty + kSStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
    int* s_pre = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kSStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 2 * kSTok);
        tmem_relinquish();
    }
    // the prologue above touches no global memory; everything below may
    pdl_wait();
    pdl_trigger();
    if (warp == 2) build_group_tiles(p.offsets, p.rows, p.err, p.E, kSTok, s_off, s_pre, lane);
    tc_fence_before();
    __syncthreads();
    if (SPLIT) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int MT = (p.N + kSWRows - 1) / kSWRows;
    const long long units = static_cast<long long>(s_pre[p.E]) * MT;
    const int first = static_cast<int>(blockIdx.x) / cs, step = static_cast<int>(gridDim.x) / cs;
    const int nk_all = (p.K + kBK - 1) / kBK;
    const int kb_lo = static_cast<int>(static_cast<long long>(rank) * nk_all / cs);
    const int kb_hi = static_cast<int>(static_cast<long long>(rank + 1) * nk_all / cs);

    auto unit = [&](long long u, int* g, int* row0, int* nrows) {
        const int tile = static_cast<int>(u / MT);
        *g = tile_group(tile, p.E, s_pre);
        *row0 = s_off[*g] + (tile - s_pre[*g]) * kSTok;
        *nrows = min(kSTok, s_off[*g + 1] - *row0);
        return static_cast<int>(u - static_cast<long long>(tile) * MT);
    };

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0;
        for (long long u = first; u < units; u += step) {
            int g, row0, nrows;
            const int mt = unit(u, &g, &row0, &nrows);
            const int nl = (nrows + kSBox - 1) / kSBox;
            const uint32_t bytes = static_cast<uint32_t>(kSABytes + nl * kSBox * kBK);
            bool ok = true;
            for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += kSSub) {
                const int ns = min(kSSub, kb_hi - kb0);
                if (lane == 0) {
                    ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs);
                    if (ok) mbar_arrive_expect_tx(smem_u32(&full[stage]), static_cast<uint32_t>(ns) * bytes);
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[stage]);
                for (int j = 0; j < ns; ++j) {
                    const int sl = stage * kSSub + j, k0 = (kb0 + j) * kBK;
                    if (lane == 0) tma_load_4d(smem_u32(sA + sl * kSABytes), &tmW, fb, k0, 0, mt * (kSWRows / 2), g);
                    if (lane < nl)
                        tma_load_2d(smem_u32(sB + sl * kSBBytes) + lane * kSBox * kBK, &tmX, fb, k0, row0 + lane * kSBox);
                }
                if (++stage == kSStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            for (long long u = first; u < units && !*abort_flag; u += step) {
                int g, row0, nrows;
                unit(u, &g, &row0, &nrows);
                const uint32_t idesc = idesc_s8_s32(kSWRows, ((nrows + 15) / 16) * 16);
                if (!mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, kWaitNs)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kSTok);
                bool ok = true;
                for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += kSSub) {
                    const int ns = min(kSSub, kb_hi - kb0);
                    if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, kWaitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int j = 0; j < ns; ++j) {
                        const int sl = stage * kSSub + j;
                        const uint32_t a0 = smem_u32(sA + sl * kSABytes), b0 = smem_u32(sB + sl * kSBBytes);
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)
                            umma_s8(d_tmem, smem_desc_sw128(a0 + kk * 32), smem_desc_sw128(b0 + kk * 32), idesc,
                                    (kb0 + j > kb_lo || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(smem_u32(&empty[stage]));
                    if (++stage == kSStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit(smem_u32(&tfull[acc]));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
    }
    const int quad = warp & 3, r = quad * 32 + lane;
    const int per_log2 = 31 - __clz(kSTok / cs), per = 1 << per_log2;   // tokens a CTA of the cluster finishes
    if (warp >= 2) {
        int acc = 0;
        uint32_t acc_phase = 0;
        for (long long u = first; u < units; u += step) {
            int g, row0, nrows;
            const int mt = unit(u, &g, &row0, &nrows);
            const int wr = mt * kSWRows + r;
            const bool wvalid = wr < p.N;
            float sw = 0.f, bias = 0.f;
            if (!SPLIT && wvalid) channel<MODE>(p, g, wr, &sw, &bias);
            if (!mbar_wait_warp(smem_u32(&tfull[acc]), acc_phase, abort_flag, kWaitNs)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * kSTok);
#pragma unroll 1
            for (int c = 0; c < nrows; c += 16) {
                uint32_t v[16];
                float sa[16];
                tmem_ld_32x32b_x16(tb + c, v);
                if constexpr (!SPLIT) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) sa[i] = __ldg(p.sa + row0 + min(c + i, nrows - 1));
                }
                tmem_wait_ld();
                if constexpr (SPLIT) {
                    // four tokens of a weight row at a time, to the CTA that finishes them
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const int n = c + i, dst = n >> per_log2;
                        if (n < nrows)
                            st_shared_cluster_v4(mapa_shared(smem_u32(s_part + (rank * kSWRows + r) * (per + 4) + n - (dst << per_log2)),
                                                             static_cast<uint32_t>(dst)),
                                                 __uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                                 __uint_as_float(v[i + 3]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int n = c + i;
                        const float y = fmaf(static_cast<float>(static_cast<int>(v[i])), sa[i] * sw, bias);
                        store_one<MODE>(p, row0 + n, wr, y, n < nrows && wvalid);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&tempty[acc]));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }
    if constexpr (SPLIT) {
        __syncwarp();
        // the finishing CTA's channel and token scales (at most 32 tokens), behind the barrier
        int g = 0, row0 = 0, nrows = 0, mt = 0;
        if (warp >= 2 && first < units) mt = unit(first, &g, &row0, &nrows);
        const int wr = mt * kSWRows + r, n0 = rank * per, n1 = min(n0 + per, nrows);
        const bool wvalid = wr < p.N;
        float sw = 0.f, bias = 0.f, sa_lane = 0.f;
        if (n0 < n1) {
            if (wvalid) channel<MODE>(p, g, wr, &sw, &bias);
            if (n0 + lane < n1) sa_lane = p.sa[row0 + n0 + lane];
        }
        cluster_sync();   // every partial sum of the cluster's unit has arrived
        for (int n = n0; n < n1; n += 4) {
            int sum[4] = {0, 0, 0, 0};
            for (int q = 0; q < cs; ++q) {
                const int4 v = *reinterpret_cast<const int4*>(s_part + (q * kSWRows + r) * (per + 4) + n - n0);
                sum[0] += v.x;
                sum[1] += v.y;
                sum[2] += v.z;
                sum[3] += v.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sa = __shfl_sync(0xffffffffu, sa_lane, (n - n0 + i) & 31);
                store_one<MODE>(p, row0 + n + i, wr, fmaf(static_cast<float>(sum[i]), sa * sw, bias), wvalid && n + i < n1);
            }
        }
    }
    if (*abort_flag) {
        // copies already issued may still land: give them time before the CTA exits
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 2 * kSTok);
    }
    if (threadIdx.x == 0 && *abort_flag && p.err) atomicOr(p.err, kErrTimeout);
}

// --------------------------------------------------------------------- many rows: pairs
// A cluster of two CTAs runs one unit (expert, up to 256 tokens, 256 weight rows) as one
// M = 256 MMA: each CTA loads its own 128 weight rows and half of the tokens, and holds its
// 128 weight rows x all tokens of the unit in tensor memory (two accumulators of 256
// columns).  The weight rows are loaded in fragment order (lane 8 q + j of a 32-lane
// quadrant holds the quadrant's row 4 j + q), so that a 16x256b accumulator fragment gives a
// thread four consecutive weight rows of two tokens, stored straight from registers.
// A CTA's warps: 0 the TMA producer, 1 the MMA issuer (even CTA), 2-17 the epilogue, 18 works
// out the units a few ahead, 19 brings the next unit's scales and biases into shared memory.
// While the MMAs run, their operand reads leave the shared memory's other users waiting (a
// load or a shuffle takes ~330 cycles): the search for a unit's expert by the MMA thread
// itself cost 3000 cycles a unit (of 14800 at K = 2816, of 5900 at K = 704), the scales
// loaded by the epilogue 4200.  16 warps of epilogue instead of 8 halve its time a unit (4900
// -> 2200 cycles at N = 256): it waits for tensor memory and for stores, not for issue slots.
// A slot (128 bytes of K: 16 KB of weights and up to 16 KB of tokens a CTA) takes 654 cycles
// at N = 256 where its four MMAs take 512: an SM takes in about 50 bytes a cycle from L2.
// Barriers a slot instead of two slots: 745 cycles.  Weight tiles kept in shared memory for
// several token tiles change nothing at K = 704 (171.5 us against 175.5, 176.6 against
// 175.9): of the ~5400 cycles a unit takes there, intake accounts for 3900, beside the
// epilogue's 2200; which wait holds the rest has not been measured.  Measured: 8191 rows, 4096 -> 4096,
// 95 us (2896 TOP/s); E = 128, 65536 rows: 2816 -> 2 x 704 with SwiGLU 284 us, 704 -> 2816
// 178 us (369 MB of outputs), the clock held to ~1.45 GHz by the power cap.
constexpr int kPEpi = 16;
constexpr int kPThreads = 128 + 32 * kPEpi;
constexpr int kPPlan = 8;                // units worked out ahead
constexpr int kPWRows = 128;
constexpr int kPTok = 256;
constexpr int kPSlots = 6;
constexpr int kPSub = 2;
constexpr int kPStages = kPSlots / kPSub;
constexpr int kPABytes = kPWRows * kBK;
constexpr int kPBox = 32;                // token rows per TMA box
constexpr int kPBBytes = kPTok / 2 * kBK;
constexpr int kPAccCols = 256;
struct PScales {
    float sa[kPTok];         // of the unit's tokens
    float sw[kPWRows];       // of the CTA's weight rows
    float bias[kPWRows];
};
constexpr int kPMiscBytes = 2 * static_cast<int>(sizeof(PScales)) + kPPlan * 32 + (2 * kPStages + 8) * 8 + 16 +
                            2 * (kMaxExperts + 1) * 4 + 64;
constexpr int kPSmemBytes = 1024 + kPSlots * (kPABytes + kPBBytes) + kPMiscBytes;
static_assert(kPSmemBytes <= 227 * 1024, "shared memory");

// A unit as the planning warp hands it on: expert, first row, rows, weight tile.  The MMA's N
// is rows rounded up to 32 (each CTA's half: a multiple of 16 rows).
struct __align__(16) PUnit {
    int g, row0, nrows, mt;
};
__device__ __forceinline__ int unit_n(int nrows) { return (nrows + 31) / 32 * 32; }

template <int MODE>
__global__ void __launch_bounds__(kPThreads, 1)
q8_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
               const Q8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kPSlots * kPABytes;
    PScales* s_scales = reinterpret_cast<PScales*>(sB + kPSlots * kPBBytes);   // [2]
    PUnit* s_unit = reinterpret_cast<PUnit*>(s_scales + 2);   // [kPPlan]
    uint64_t* ufull = reinterpret_cast<uint64_t*>(s_unit + kPPlan);
    uint64_t* uempty = ufull + kPPlan;
    uint64_t* full = uempty + kPPlan;
    uint64_t* empty = full + kPStages;
    uint64_t* tfull = empty + kPStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* sfull = tempty + 2;
    uint64_t* sempty = sfull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
    int* s_pre = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool lead = rank == 0;
    const int G = p.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kPStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);    // the even CTA's producer (expect_tx)
            mbar_init(smem_u32(&empty[s]), 1);   // the pair MMA's commit
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 2 * kPEpi);   // both CTAs'
            mbar_init(smem_u32(&sfull[a]), 1);
            mbar_init(smem_u32(&sempty[a]), kPEpi);
        }
        for (int q = 0; q < kPPlan; ++q) {
            mbar_init(smem_u32(&ufull[q]), 1);
            mbar_init(smem_u32(&uempty[q]), kPEpi + (lead ? 3 : 2));   // producer, scales, epilogue, MMA
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 2 * kPAccCols);
        tmem_relinquish_pair();
    }
    // the prologue above touches no global memory; everything below may
    pdl_wait();
    pdl_trigger();
    if (warp == 2) build_group_tiles(p.offsets, p.rows, p.err, G, kPTok, s_off, s_pre, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers and tensor memory exist before any signal
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int MT = (p.N + 2 * kPWRows - 1) / (2 * kPWRows);
    const long long units = static_cast<long long>(s_pre[G]) * MT;
    const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
    const int nk = (p.K + kBK - 1) / kBK;

    // the planned units, as every role reads them: wait, read; free the slot once done
    struct Plan {
        int slot = 0;
        uint32_t phase = 0;
        __device__ __forceinline__ void next() {
            if (++slot == kPPlan) {
                slot = 0;
                phase ^= 1u;
            }
        }
    } plan;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (long long u = pair; u < units && !*abort_flag; u += npairs, plan.next()) {
                if (!mbar_wait(smem_u32(&ufull[plan.slot]), plan.phase, abort_flag, kWaitNs)) break;
                const PUnit d = s_unit[plan.slot];
                mbar_arrive(smem_u32(&uempty[plan.slot]));
                const int trow0 = d.row0 + static_cast<int>(rank) * (unit_n(d.nrows) / 2);
                // weight views: plain (k, j, q, Q, e) at (k, 0, 0, w_in / 32, g); chunked fc1
                // (k, j, s, qq, X) at (k, 0, 0, 0, g I / 8 + w_in / 32)
                const int w_in = d.mt * 2 * kPWRows + static_cast<int>(rank) * kPWRows;
                const bool chunked = MODE == OUT_SWIGLU && p.chunked;
                const int wc3 = chunked ? 0 : w_in / 32;
                const int wc4 = chunked ? d.g * (p.N / 16) + w_in / 32 : d.g;
                // the CTA's half of the tokens in boxes of 32 rows: a slot's time goes by the
                // bytes that come in, so no rows past the tile
                const int nb = (unit_n(d.nrows) / 2 + kPBox - 1) / kPBox;
                const uint32_t bytes = static_cast<uint32_t>(2 * (kPABytes + nb * kPBox * kBK));
                bool ok = true;
                for (int kb0 = 0; kb0 < nk; kb0 += kPSub) {
                    const int ns = min(kPSub, nk - kb0);
                    ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs);
                    if (!ok) break;
                    if (lead) mbar_arrive_expect_tx(smem_u32(&full[stage]), static_cast<uint32_t>(ns) * bytes);
                    const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);   // the even CTA's
                    for (int j = 0; j < ns; ++j) {
                        const int sl = stage * kPSub + j, k0 = (kb0 + j) * kBK;
                        tma_load_5d_pair(smem_u32(sA + sl * kPABytes), &tmW, fb, k0, 0, 0, wc3, wc4);
                        for (int i = 0; i < nb; ++i)
                            tma_load_2d_pair(smem_u32(sB + sl * kPBBytes) + i * kPBox * kBK, &tmX, fb, k0, trow0 + i * kPBox);
                    }
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp walks the units in step, one elected lane issues.
        if (lead) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            auto rows_of_next = [&]() {   // the next unit's rows, 0 if the wait gave up
                int n = 0;
                if (mbar_wait_warp(smem_u32(&ufull[plan.slot]), plan.phase, abort_flag, kWaitNs)) n = s_unit[plan.slot].nrows;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&uempty[plan.slot]));
                plan.next();
                return n;
            };
            const uint64_t a_desc = smem_desc_sw128(smem_u32(sA)), b_desc = smem_desc_sw128(smem_u32(sB));
            const uint32_t a_lo = static_cast<uint32_t>(a_desc), b_lo = static_cast<uint32_t>(b_desc);
            const uint32_t hi = static_cast<uint32_t>(a_desc >> 32);
            const int steps = (p.K + 31) / 32;            // MMAs of a unit: none past K
            constexpr int kStep = kPSub * (kBK / 32);     // of a whole stage
            int nrows = pair < units ? rows_of_next() : 0, nrows_next = 0;
            for (long long u = pair; u < units && nrows > 0; u += npairs) {
                const uint32_t idesc = idesc_s8_s32(2 * kPWRows, unit_n(nrows));
                if (!mbar_wait_warp(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, kWaitNs)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kPAccCols);
                bool ok = true;
                for (int s0 = 0; s0 < steps; s0 += kStep) {
                    if (!mbar_wait_warp(smem_u32(&full[stage]), phase, abort_flag, kWaitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t la = a_lo + static_cast<uint32_t>(stage * (kPSub * kPABytes >> 4));
                    const uint32_t lb = b_lo + static_cast<uint32_t>(stage * (kPSub * kPBBytes >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kStep; ++i)
                            if (s0 + i < steps)
                                umma_s8_pair_lo(d_tmem, la + (i / 4) * (kPABytes >> 4) + (i % 4) * 2,
                                                lb + (i / 4) * (kPBBytes >> 4) + (i % 4) * 2, hi, idesc,
                                                i > 0 ? 1u : (s0 > 0 ? 1u : 0u));
                        umma_commit_pair(smem_u32(&empty[stage]), 0x3);
                    }
                    __syncwarp();
                    if (++stage == kPStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    // read behind the first MMAs, used after the last
                    if (s0 == 0 && u + npairs < units) nrows_next = rows_of_next();
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair(smem_u32(&tfull[acc]), 0x3);
                __syncwarp();
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
                nrows = nrows_next;
            }
        }
    } else if (warp == 2 + kPEpi) {
        // ------------------------------------------------------------ the units, ahead
        if (lane == 0) {
            for (long long u = pair; u < units && !*abort_flag; u += npairs, plan.next()) {
                const int tile = static_cast<int>(u / MT);
                PUnit d;
                d.mt = static_cast<int>(u - static_cast<long long>(tile) * MT);
                d.g = tile_group(tile, G, s_pre);
                d.row0 = s_off[d.g] + (tile - s_pre[d.g]) * kPTok;
                d.nrows = min(kPTok, s_off[d.g + 1] - d.row0);
                if (!mbar_wait(smem_u32(&uempty[plan.slot]), plan.phase ^ 1u, abort_flag, kWaitNs)) break;
                s_unit[plan.slot] = d;
                mbar_arrive(smem_u32(&ufull[plan.slot]));
            }
        }
    } else if (warp == 3 + kPEpi) {
        // ------------------------------------------------------------ scales, a unit ahead
        int acc = 0;
        uint32_t acc_phase = 0;
        for (long long u = pair; u < units; u += npairs, plan.next()) {
            if (!mbar_wait_warp(smem_u32(&ufull[plan.slot]), plan.phase, abort_flag, kWaitNs)) break;
            const PUnit d = s_unit[plan.slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&uempty[plan.slot]));
            const int w0 = d.mt * 2 * kPWRows + static_cast<int>(rank) * kPWRows;
            float a8[kPTok / 32], w8[kPWRows / 32], b8[kPWRows / 32];
#pragma unroll
            for (int i = 0; i < kPTok / 32; ++i) a8[i] = __ldg(p.sa + d.row0 + min(lane + 32 * i, d.nrows - 1));
#pragma unroll
            for (int i = 0; i < kPWRows / 32; ++i) {
                w8[i] = b8[i] = 0.f;
                if (w0 + 32 * i < p.N) channel<MODE>(p, d.g, w0 + lane + 32 * i, &w8[i], &b8[i]);
            }
            if (!mbar_wait_warp(smem_u32(&sempty[acc]), acc_phase ^ 1u, abort_flag, kWaitNs)) break;
            PScales& sc = s_scales[acc];
#pragma unroll
            for (int i = 0; i < kPTok / 32; ++i) sc.sa[lane + 32 * i] = a8[i];
#pragma unroll
            for (int i = 0; i < kPWRows / 32; ++i) {
                sc.sw[lane + 32 * i] = w8[i];
                sc.bias[lane + 32 * i] = b8[i];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sfull[acc]));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread (fj, ft) = (lane / 4, lane % 4) of a 16x256b fragment holds weight rows
        // 4 fj .. 4 fj + 3 of its quadrant for tokens 8 m + 2 ft + e of a 32-token chunk.
        const int quad = warp & 3;
        const int part = (warp - 2) >> 2;
        constexpr int kParts = kPEpi / 4;
        const int fj = lane >> 2, ft = lane & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        // the unit after the current one, read behind the current one's first loads
        auto read_unit = [&](PUnit* d) {
            if (!mbar_wait_warp(smem_u32(&ufull[plan.slot]), plan.phase, abort_flag, kWaitNs)) return false;
            *d = s_unit[plan.slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&uempty[plan.slot]));
            plan.next();
            return true;
        };
        PUnit d, d_next{0, 0, 0, 0};
        bool ok = pair >= units || read_unit(&d);
        for (long long u = pair; ok && u < units; u += npairs) {
            const int w0 = d.mt * 2 * kPWRows + static_cast<int>(rank) * kPWRows + quad * 32;
            const bool wvalid = w0 < p.N;   // N is a multiple of 32: the warp's rows are all valid or none
            const int wr = w0 + 4 * fj;
            constexpr int kChunks = kPTok / (32 * kParts);
            if (!mbar_wait_warp(smem_u32(&sfull[acc]), acc_phase, abort_flag, kWaitNs)) break;
            const PScales& sc = s_scales[acc];
            if (!mbar_wait_warp(smem_u32(&tfull[acc]), acc_phase, abort_flag, kWaitNs)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                                static_cast<uint32_t>(acc * kPAccCols);
            float4 sw, bias;
#pragma unroll
            for (int ci = 0; ci < kChunks; ++ci) {
                const int c = 32 * (part + ci * kParts);
                uint32_t lo[16], hi[16];
                if (c < d.nrows) {
                    tmem_ld_16x256b_x4(tb + c, lo);                  // rows 4 fj, 4 fj + 1
                    tmem_ld_16x256b_x4(tb + (16u << 16) + c, hi);    // rows 4 fj + 2, 4 fj + 3
                }
                if (ci == 0) {
                    sw = *reinterpret_cast<const float4*>(sc.sw + quad * 32 + 4 * fj);
                    bias = *reinterpret_cast<const float4*>(sc.bias + quad * 32 + 4 * fj);
                    if (u + npairs < units) ok = read_unit(&d_next);
                }
                float2 sa2[4];
                if (c < d.nrows) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) sa2[m] = *reinterpret_cast<const float2*>(sc.sa + c + 8 * m + 2 * ft);
                    tmem_wait_ld();
                }
                if (c + 32 * kParts >= d.nrows || ci == kChunks - 1) {
                    // this warp's last values are in registers: the accumulator and the scales
                    // are free before the stores go out, which a release arrival behind them
                    // would wait for (2800 cycles a unit; the bound at K = 704)
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[acc]), 0));
                        mbar_arrive(smem_u32(&sempty[acc]));
                    }
                    if (c >= d.nrows) break;
                }
                if (!wvalid) {
                    if (c + 32 * kParts >= d.nrows) break;
                    continue;
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = c + 8 * m + 2 * ft + e;
                        const float s = e ? sa2[m].y : sa2[m].x;
                        const float x0 = fmaf(static_cast<float>(static_cast<int>(lo[4 * m + e])), s * sw.x, bias.x);
                        const float x1 = fmaf(static_cast<float>(static_cast<int>(lo[4 * m + 2 + e])), s * sw.y, bias.y);
                        const float x2 = fmaf(static_cast<float>(static_cast<int>(hi[4 * m + e])), s * sw.z, bias.z);
                        const float x3 = fmaf(static_cast<float>(static_cast<int>(hi[4 * m + 2 + e])), s * sw.w, bias.w);
                        if (tok < d.nrows) {
                            const size_t row = static_cast<size_t>(d.row0 + tok);
                            if constexpr (MODE == OUT_SWIGLU)
                                *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * (p.N / 2) + (wr >> 1)) =
                                    make_float2(swiglu_attr_fast(x0, x1, p.act), swiglu_attr_fast(x2, x3, p.act));
                            else if constexpr (MODE == OUT_BF16)
                                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * p.N + wr) =
                                    make_uint2(pack_bf16x2(x0, x1), pack_bf16x2(x2, x3));
                            else
                                *reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * p.N + wr) =
                                    make_float4(x0, x1, x2, x3);
                        }
                    }
                }
                if (c + 32 * kParts >= d.nrows) break;
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            d = d_next;
        }
    }

    if (*abort_flag) {
        // copies already issued may still land: give them time before the pair exits
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 200000ull) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // no CTA leaves while its partner may still read its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 2 * kPAccCols);
    }
    if (threadIdx.x == 0 && *abort_flag && p.err) atomicOr(p.err, kErrTimeout);
}

// ------------------------------------------------------------------------ host side

// Launch in clusters of `cs` CTAs, programmatic stream serialisation allowed.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), int ctas, int cs, int threads, int smem, cudaStream_t s,
                            Args&&... args) {
    cudaLaunchAttribute attr[2];
    int n = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (cs > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cs);
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(n);
    count_launch();
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// The kernel's shared-memory limit, once per device.
template <typename K>
cudaError_t set_smem(K* kern, int bytes, bool* done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

template <int MODE, bool SPLIT>
cudaError_t launch_stream(const CUtensorMap& w, const CUtensorMap& x, const Q8Params& p, int clusters, int cs,
                          cudaStream_t s) {
    static bool done[64] = {false};
    const cudaError_t e = set_smem(q8_stream_kernel<MODE, SPLIT>, stream_smem(SPLIT), done);
    if (e != cudaSuccess) return e;
    return launch_clusters(q8_stream_kernel<MODE, SPLIT>, clusters * cs, cs, kSThreads, stream_smem(SPLIT), s, w, x, p, cs);
}

// Pairs of CTAs that fit on the device at once, asked once per device.
template <int MODE>
cudaError_t max_pairs(int* pairs) {
    static int most[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (most[dev] == 0) {
        cudaError_t e = cudaFuncSetAttribute(q8_pair_kernel<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmemBytes);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (device_sm_count() / 2));
        cfg.blockDim = dim3(kPThreads);
        cfg.dynamicSmemBytes = kPSmemBytes;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, q8_pair_kernel<MODE>, &cfg);
        if (e != cudaSuccess) return e;
        most[dev] = n > 0 ? n : 1;
    }
    *pairs = most[dev];
    return cudaSuccess;
}

template <int MODE>
cudaError_t launch_pair(const CUtensorMap& w, const CUtensorMap& x, const Q8Params& p, long long units, cudaStream_t s) {
    int most = 0;
    const cudaError_t e = max_pairs<MODE>(&most);
    if (e != cudaSuccess) return e;
    const int pairs = units < most ? static_cast<int>(units) : most;
    return launch_clusters(q8_pair_kernel<MODE>, 2 * pairs, 2, kPThreads, kPSmemBytes, s, w, x, p);
}

// The streaming kernel runs for up to 56 rows per expert on average, and wherever its units
// fit on the GPU at once.  Measured (stream / pair, us): grouped, E = 128, 2816 -> 1408, 48
// rows per expert 88.2 / 96.8, 64 rows 100.8 / 98.1, 128 rows 162.6 / 108.8; dense, 2816 ->
// 1408, 128 rows 8.8 / 12.7, 768 rows (132 units) 12.1 / 14.0, 1024 rows (176) 18.1 / 14.0;
// 4096 -> 4096, 256 rows (128 units) 14.6 / 17.3, 384 rows (192) 23.4 / 17.4.
constexpr int kStreamRows = 56;

// Upper bound of the 64-row chunks: one per 64 rows, one more for every expert, at most one a
// row (dense: exactly one per 64 rows).
long long stream_units(const Q8GemmArgs& a) {
    long long chunks = (a.rows + kSTok - 1LL) / kSTok;
    if (a.offsets) chunks = a.rows < chunks + a.E ? a.rows : chunks + a.E;
    return chunks * ((a.N + kSWRows - 1) / kSWRows);
}

bool use_stream(const Q8GemmArgs& a) {
    return static_cast<long long>(a.rows) <= static_cast<long long>(kStreamRows) * a.E ||
           stream_units(a) <= device_sm_count();
}

template <int MODE>
cudaError_t stream_product(const Q8GemmArgs& a, const Q8Params& p, cudaStream_t s) {
    CUtensorMap w, x;
    if (!tmap::pairs8(&w, a.w_q, a.E, a.N, a.K, kSWRows / 2, false)) return cudaErrorInvalidValue;
    if (!tmap::matrix8(&x, a.a_q, a.rows, a.K, kSBox, a.lda ? a.lda : a.K)) return cudaErrorInvalidValue;
    const long long units = stream_units(a);
    const int sms = device_sm_count(), nk = (a.K + kBK - 1) / kBK;
    int cs = 8;
    while (cs > 1 && (units * cs > sms || cs > nk)) cs /= 2;
    if (cs > 1) return launch_stream<MODE, true>(w, x, p, static_cast<int>(units), cs, s);
    return launch_stream<MODE, false>(w, x, p, static_cast<int>(units < sms ? units : sms), 1, s);
}

template <int MODE>
cudaError_t product(const Q8GemmArgs& a, const Q8Params& p, cudaStream_t s) {
    CUtensorMap w, x;
    const bool chunked = a.swiglu && a.fc1_chunked;
    if (MODE == OUT_SWIGLU || !use_stream(a)) {
        if (!tmap::quads8(&w, a.w_q, a.E, a.N, a.K, chunked)) return cudaErrorInvalidValue;
        if (!tmap::matrix8(&x, a.a_q, a.rows, a.K, kPBox, a.lda ? a.lda : a.K)) return cudaErrorInvalidValue;
        const long long units = ((a.rows + kPTok - 1LL) / kPTok + a.E) *
                                ((a.N + 2 * kPWRows - 1) / (2 * kPWRows));
        return launch_pair<MODE>(w, x, p, units, s);
    }
    // (fc1 alone has many rows: the FFN of few is one launch, ffn_q8.cu)
    if constexpr (MODE == OUT_SWIGLU) return cudaErrorInvalidValue;
    else return stream_product<MODE>(a, p, s);
}
}  // namespace

cudaError_t launch_q8_gemm(const Q8GemmArgs& a, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    const Q8Params p{a.offsets, a.E, a.rows, a.K, a.N, a.a_scale, a.w_scale, a.bias, a.out, a.err, a.act,
                     a.fc1_chunked};
    if (a.swiglu) return product<OUT_SWIGLU>(a, p, s);
    return a.out_bf16 ? product<OUT_BF16>(a, p, s) : product<OUT_F32>(a, p, s);
}

}  // namespace moe
