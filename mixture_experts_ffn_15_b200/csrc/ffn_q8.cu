// Expert FFN with int8 activations and weights for few rows per expert, in one launch:
//   fc1 (int8 x int8) + SwiGLU -> rows cut to int8 -> fc2 (int8 x int8)
// The arithmetic is that of gemm_q8.cu and quantize.cu; x_perm arrives as int8 rows.
//
// 128 weight rows on the MMA's M side, a chunk of up to 64 token rows of one expert on N, so
// that every weight byte streams from HBM once; bound by that stream.  The unit list holds
// every fc1 unit (chunk x 128 rows of fc1), then every fc2 unit.  A CTA's first unit is unit
// blockIdx.x, later ones come in list order from a counter (starting at the grid size), so
// the long fc1 units go first and the short fc2 units even out the end.
//
// Warps of a CTA:
//   0    claims the units and streams their weights (TMA) into the ring.  Weights depend on
//        nothing this launch or the quantiser in front of it writes: the first unit's loads
//        start before that kernel has finished, and those of an fc2 unit before its
//        activations exist.
//   1    issues the MMAs (tcgen05 kind::i8) into one of two accumulators
//   2-5  epilogue.  fc1: the activations in float32 to scratch, counted per chunk.  fc2:
//        scales, bias, bf16 outputs.
//   6    streams the token rows: x's, or a chunk's activations once they are published
//   7    brings each unit's channel scales and biases, and its rows' scales, into shared
//        memory ahead of the epilogue (which waited 2.5 us a unit for them in turn, more
//        than an fc2 unit's weights take)
//   8-11 cut activations to int8, two rows at a time, as soon as their chunk's count is
//        complete.  Row pairs are strided over the CTAs, apart from the units: rounding as
//        units of the list, taken by the epilogue in its turn, came up to 8 us late for the
//        last chunks (E = 128, H = 2816, I = 704: 50 us instead of 46 at 32 rows, 168 instead
//        of 148 at 2048), and by the warp that completes a chunk it took 576 us at 2048 rows.
// The launch is cooperative (every CTA resident), so a unit waited for is some running CTA's.
// Every wait is bounded (2 s) and reports MOE_DEVERR_TIMEOUT.
// Measured with the row quantiser in front: E = 128, H = 2816, I = 704, 32 rows (170 MB of the
// used experts' weights) 43 us, 2048 rows (786 MB) 137 us, 5.7 TB/s.
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "quantize.cuh"
#include "sm100.cuh"
#include "tile_map.cuh"
#include "tmap.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kBK = tmap::kBoxK8;
constexpr int kTok = 64;                 // token rows per chunk
constexpr int kBox = 16;                 // token rows per TMA box
constexpr int kWRows = 128;
constexpr int kSub = 2;                  // ring slots per barrier stage
constexpr int kStages = 4;
constexpr int kSlots = kStages * kSub;
constexpr int kABytes = kWRows * kBK;
constexpr int kBBytes = kTok * kBK;
constexpr int kRing = 8;                 // claimed units handed to the other warps
constexpr int kRoundWarps = 4;
constexpr int kThreads = 32 * (8 + kRoundWarps);
constexpr uint64_t kWaitNs = 2000000000ull;
struct Scales {
    float sw[kWRows], bias[kWRows], sa[kTok];
};
constexpr int kMiscBytes = kRing * (32 + static_cast<int>(sizeof(Scales))) + (2 * kStages + 4 + 3 * kRing) * 8 + 16 +
                           2 * (kMaxExperts + 1) * 4 + 64;
constexpr int kSmemBytes = 1024 + kSlots * (kABytes + kBBytes) + kMiscBytes;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Params {
    const int32_t* offsets;   // [E+1] device
    int E, rows, H, I;
    const float* xs;          // [rows] scales of the int8 rows of x
    const float* s1;          // [E, 2I]
    const float* s2;          // [E, H]
    const __nv_bfloat16* b1;  // [E, 2I] or nullptr
    const __nv_bfloat16* b2;  // [E, H] or nullptr
    float* act;               // [rows, I] scratch
    int8_t* aq;               // [rows, I] scratch, rows lda bytes apart
    int lda;
    float* as;                // [rows] scratch
    __nv_bfloat16* y;         // [rows, H]
    int32_t* done;            // [chunks] finished fc1 epilogue warps, zero on entry
    int32_t* ready;           // [chunks] rows whose int8 activations are there, zero on entry
    int32_t* sched;           // units claimed past the first gridDim.x, zero on entry
    int32_t* err;
    SwigluAttr attr;
    bool chunked;
};

struct __align__(16) Unit {
    int g, row0, nrows, mt;   // expert, first row, rows, weight tile
    int chunk, kind;
    int pad[2];
};
enum Kind : int { kNone = -1, kFc2 = 0, kFc1 = 1 };

// The int8 rows of activation rows row and row + 1 (if `two`), by one warp.
__device__ __forceinline__ void round_rows(const Params& p, int row, bool two, int lane) {
    const int nvec = p.I / 4, ldw = p.lda / 4;
    const float4* x0 = reinterpret_cast<const float4*>(p.act + static_cast<size_t>(row) * p.I);
    const float4* x1 = two ? x0 + nvec : x0;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.aq + static_cast<size_t>(row) * p.lda);
    auto top = [](const float4& v) {
        return max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
                   max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
    };
    float far = 0.f;
    auto fast = [&](const float4& v, const RowQuant& q) {
        const uint32_t n[4] = {quantize_fast<true>(v.x, 1.f, q.inv, &far), quantize_fast<true>(v.y, 1.f, q.inv, &far),
                               quantize_fast<true>(v.z, 1.f, q.inv, &far), quantize_fast<true>(v.w, 1.f, q.inv, &far)};
        return pack_s8x4(n);
    };
    // up to kHold vectors a lane stay in registers between the maximum and the rounding; the
    // rest of a longer row is read again
    constexpr int kHold = 8;
    float4 h0[kHold], h1[kHold];
    uint32_t m0 = 0, m1 = 0;
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (lane + 32 * j < nvec) {
            h0[j] = __ldcg(x0 + lane + 32 * j);
            h1[j] = __ldcg(x1 + lane + 32 * j);
        }
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (lane + 32 * j < nvec) {
            m0 = max(m0, top(h0[j]));
            m1 = max(m1, top(h1[j]));
        }
#pragma unroll 4
    for (int v = lane + 32 * kHold; v < nvec; v += 32) {
        m0 = max(m0, top(__ldcg(x0 + v)));
        m1 = max(m1, top(__ldcg(x1 + v)));
    }
    const RowQuant q0 = row_quant(__reduce_max_sync(0xffffffffu, m0));
    const RowQuant q1 = row_quant(__reduce_max_sync(0xffffffffu, m1));
#pragma unroll
    for (int j = 0; j < kHold; ++j)
        if (lane + 32 * j < nvec) {
            out[lane + 32 * j] = fast(h0[j], q0);
            if (two) out[ldw + lane + 32 * j] = fast(h1[j], q1);
        }
#pragma unroll 4
    for (int v = lane + 32 * kHold; v < nvec; v += 32) {
        out[v] = fast(__ldcg(x0 + v), q0);
        if (two) out[ldw + v] = fast(__ldcg(x1 + v), q1);
    }
    if (!ordinary(q0) || !ordinary(q1) || !(far <= kSureDistance)) {   // this lane's values again, exactly
        auto exact = [](const float4& v, const RowQuant& q) {
            const uint32_t n[4] = {quantize_exact(v.x, q.pre, q.inv, q.amax), quantize_exact(v.y, q.pre, q.inv, q.amax),
                                   quantize_exact(v.z, q.pre, q.inv, q.amax), quantize_exact(v.w, q.pre, q.inv, q.amax)};
            return pack_s8x4(n);
        };
#pragma unroll 1
        for (int v = lane; v < nvec; v += 32) {
            out[v] = exact(__ldcg(x0 + v), q0);
            if (two) out[ldw + v] = exact(__ldcg(x1 + v), q1);
        }
    }
    if (lane == 0) {
        p.as[row] = q0.scale;
        if (two) p.as[row + 1] = q1.scale;
    }
}

__global__ void __launch_bounds__(kThreads, 1)
q8_ffn_kernel(const __grid_constant__ CUtensorMap tmW1, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ CUtensorMap tmW2, const __grid_constant__ CUtensorMap tmA, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kSlots * kABytes;
    Unit* s_unit = reinterpret_cast<Unit*>(sB + kSlots * kBBytes);   // [kRing]
    Scales* s_scales = reinterpret_cast<Scales*>(s_unit + kRing);    // [kRing]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_scales + kRing);
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* ufull = tempty + 2;
    uint64_t* uempty = ufull + kRing;
    uint64_t* sfull = uempty + kRing;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sfull + kRing);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_off = reinterpret_cast<int*>(tmem_slot + 4);
    int* s_pre = s_off + (kMaxExperts + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 2);    // the weights' and the tokens' producer
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 4);
        }
        for (int q = 0; q < kRing; ++q) {
            mbar_init(smem_u32(&ufull[q]), 1);
            mbar_init(smem_u32(&uempty[q]), 7);  // MMA, tokens, scales, 4 epilogue warps
            mbar_init(smem_u32(&sfull[q]), 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW1);
        tma_prefetch_desc(&tmW2);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmA);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 2 * kTok);
        tmem_relinquish();
    }
    // The kernel in front is the row quantiser of the same call, which lets this one start
    // only after all work before it has completed: the offsets and the weights are final.
    // What the quantiser writes (int8 rows, scales, cleared counters, the error word) is
    // read, and anything is written, only after pdl_wait.
    pdl_trigger();
    if (warp == 2) build_group_tiles(p.offsets, p.rows, nullptr, p.E, kTok, s_off, s_pre, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    const int MT1 = (2 * p.I + kWRows - 1) / kWRows, MT2 = (p.H + kWRows - 1) / kWRows;
    const int chunks = s_pre[p.E];
    const int U1 = chunks * MT1, U = U1 + chunks * MT2;
    const int nk1 = (p.H + kBK - 1) / kBK, nk2 = (p.I + kBK - 1) / kBK;

    int slot = 0;
    uint32_t uphase = 0;
    auto next_slot = [&]() {
        if (++slot == kRing) {
            slot = 0;
            uphase ^= 1u;
        }
    };
    // the next claimed unit, as the MMA's and the tokens' lane read it
    auto next_unit = [&](Unit* d) {
        if (!mbar_wait(smem_u32(&ufull[slot]), uphase, abort_flag, kWaitNs)) return false;
        *d = s_unit[slot];
        mbar_arrive(smem_u32(&uempty[slot]));
        next_slot();
        return d->kind != kNone;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ claims, weights
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool waited = false;
            // the next claim is made while the current unit's loads go out: the counter's
            // round trip (1 us) is half of what an fc2 unit's weights take
            int u = static_cast<int>(blockIdx.x), u_next = 0;
            auto claim = [&]() {
                if (!waited) pdl_wait();   // the counter is cleared by then
                waited = true;
                u_next = static_cast<int>(gridDim.x) + atomicAdd(p.sched, 1);
            };
            for (;; u = u_next) {
                Unit d;
                d.kind = u >= U ? kNone : u < U1 ? kFc1 : kFc2;
                if (d.kind != kNone) {
                    const int v = d.kind == kFc1 ? u : u - U1, MT = d.kind == kFc1 ? MT1 : MT2;
                    d.chunk = v / MT;
                    d.mt = v - d.chunk * MT;
                    d.g = tile_group(d.chunk, p.E, s_pre);
                    d.row0 = s_off[d.g] + (d.chunk - s_pre[d.g]) * kTok;
                    d.nrows = min(kTok, s_off[d.g + 1] - d.row0);
                }
                if (!mbar_wait(smem_u32(&uempty[slot]), uphase ^ 1u, abort_flag, kWaitNs)) break;
                s_unit[slot] = d;
                mbar_arrive(smem_u32(&ufull[slot]));
                next_slot();
                if (d.kind == kNone) break;
                // one load instruction for both weight tensors, its map chosen at run time
                const CUtensorMap* mw = d.kind == kFc1 ? &tmW1 : &tmW2;
                const int nk = d.kind == kFc1 ? nk1 : nk2;
                // behind the first unit's first ring of loads, any other unit's first stage
                const int claim_at = waited ? 0 : min((nk - 1) / kSub, kStages - 1) * kSub;
                bool ok = true;
                for (int kb0 = 0; kb0 < nk; kb0 += kSub) {
                    const int ns = min(kSub, nk - kb0);
                    ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(ns * kABytes));
                    for (int j = 0; j < ns; ++j)
                        tma_load_4d(smem_u32(sA + (stage * kSub + j) * kABytes), mw, fb, (kb0 + j) * kBK, 0,
                                    d.mt * (kWRows / 2), d.g);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (kb0 == claim_at) claim();
                }
                if (!ok) break;
            }
            if (!waited) pdl_wait();
        }
    } else if (warp == 6) {
        // ------------------------------------------------------------ token rows
        if (lane == 0) {
            pdl_wait();
            int stage = 0;
            uint32_t phase = 0;
            Unit d;
            while (next_unit(&d)) {
                const CUtensorMap* mx = d.kind == kFc1 ? &tmX : &tmA;
                const int nk = d.kind == kFc1 ? nk1 : nk2;
                if (d.kind == kFc2) {
                    if (!wait_count(p.ready + d.chunk, d.nrows, abort_flag, kWaitNs)) break;
                    fence_proxy_async_global();
                }
                const int nl = (d.nrows + kBox - 1) / kBox;
                bool ok = true;
                for (int kb0 = 0; kb0 < nk; kb0 += kSub) {
                    const int ns = min(kSub, nk - kb0);
                    ok = mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kWaitNs);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(ns * nl * kBox * kBK));
                    for (int j = 0; j < ns; ++j)
                        for (int i = 0; i < nl; ++i)
                            tma_load_2d(smem_u32(sB + (stage * kSub + j) * kBBytes) + i * kBox * kBK, mx, fb,
                                        (kb0 + j) * kBK, d.row0 + i * kBox);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            Unit d;
            while (next_unit(&d)) {
                const int nk = d.kind == kFc1 ? nk1 : nk2, K = d.kind == kFc1 ? p.H : p.I;
                const uint32_t idesc = idesc_s8_s32(kWRows, ((d.nrows + 15) / 16) * 16);
                if (!mbar_wait(smem_u32(&tempty[acc]), acc_phase ^ 1u, abort_flag, kWaitNs)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTok);
                bool ok = true;
                for (int kb0 = 0; kb0 < nk; kb0 += kSub) {
                    const int ns = min(kSub, nk - kb0);
                    if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, kWaitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int j = 0; j < ns; ++j) {
                        const int sl = stage * kSub + j;
                        const uint32_t a0 = smem_u32(sA + sl * kABytes), b0 = smem_u32(sB + sl * kBBytes);
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)
                            if ((kb0 + j) * kBK + kk * 32 < K)   // nothing but zeros past K
                                umma_s8(d_tmem, smem_desc_sw128(a0 + kk * 32), smem_desc_sw128(b0 + kk * 32), idesc,
                                        (kb0 + j > 0 || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(smem_u32(&empty[stage]));
                    if (++stage == kStages) {
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
    } else if (warp == 7) {
        // ------------------------------------------------------------ scales
        pdl_wait();
        for (;;) {
            const int at = slot;
            if (!mbar_wait_warp(smem_u32(&ufull[at]), uphase, abort_flag, kWaitNs)) break;
            const Unit d = s_unit[at];
            if (d.kind == kNone) break;
            const bool f1 = d.kind == kFc1;
            const int n_out = f1 ? 2 * p.I : p.H;
            const float* s = f1 ? p.s1 : p.s2;
            const __nv_bfloat16* b = f1 ? p.b1 : p.b2;
            float sw[kWRows / 32], bias[kWRows / 32];
#pragma unroll
            for (int i = 0; i < kWRows / 32; ++i) {
                const int wr = d.mt * kWRows + 32 * i + lane;
                sw[i] = bias[i] = 0.f;
                if (wr < n_out) {
                    const size_t j = static_cast<size_t>(d.g) * n_out + (f1 ? fc1_row(wr, p.I, p.chunked) : wr);
                    sw[i] = s[j];
                    if (b) bias[i] = bf16_at(b, j);
                }
            }
            if (!f1 && !wait_count_warp(p.ready + d.chunk, d.nrows, abort_flag, kWaitNs, lane)) break;
            Scales& sc = s_scales[at];
#pragma unroll
            for (int i = 0; i < kTok / 32; ++i)
                if (lane + 32 * i < d.nrows) sc.sa[lane + 32 * i] = __ldcg((f1 ? p.xs : p.as) + d.row0 + lane + 32 * i);
#pragma unroll
            for (int i = 0; i < kWRows / 32; ++i) {
                sc.sw[32 * i + lane] = sw[i];
                sc.bias[32 * i + lane] = bias[i];
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sfull[at]));
                mbar_arrive(smem_u32(&uempty[at]));
            }
            next_slot();
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ activations to int8
        pdl_wait();
        constexpr int kPairs = kTok / 2;
        // neighbouring pairs on different CTAs: a chunk's rows are rounded at once
        const int w0 = (warp - 8) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
        for (int v = w0; v < chunks * kPairs; v += kRoundWarps * static_cast<int>(gridDim.x)) {
            const int chunk = v / kPairs, r0 = 2 * (v - chunk * kPairs);
            const int g = tile_group(chunk, p.E, s_pre);
            const int row0 = s_off[g] + (chunk - s_pre[g]) * kTok;
            const int n = min(2, min(kTok, s_off[g + 1] - row0) - r0);
            if (n <= 0) continue;
            if (!wait_count_warp(p.done + chunk, 4 * MT1, abort_flag, kWaitNs, lane)) break;
            round_rows(p, row0 + r0, n == 2, lane);
            fence_proxy_async_global();   // read by TMA
            __threadfence();
            __syncwarp();
            if (lane == 0) atomicAdd(p.ready + chunk, n);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        pdl_wait();
        const int quad = warp & 3, r = quad * 32 + lane;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (;;) {
            const int at = slot;
            if (!mbar_wait_warp(smem_u32(&ufull[at]), uphase, abort_flag, kWaitNs)) break;
            const Unit d = s_unit[at];
            if (d.kind == kNone) break;
            const bool f1 = d.kind == kFc1;
            const int wr = d.mt * kWRows + r;
            const bool wvalid = wr < (f1 ? 2 * p.I : p.H);   // even: a (gate, up) pair is valid or not as one
            if (!mbar_wait_warp(smem_u32(&sfull[at]), uphase, abort_flag, kWaitNs)) break;
            const Scales& sc = s_scales[at];
            const float sw = sc.sw[r], bias = sc.bias[r];
            if (!mbar_wait_warp(smem_u32(&tfull[acc]), acc_phase, abort_flag, kWaitNs)) break;
            tc_fence_after();
            const uint32_t tb = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * kTok);
#pragma unroll 1
            for (int c = 0; c < d.nrows; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tb + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int n = c + i;   // past the chunk: a stale scale, nothing stored
                    const float x = fmaf(static_cast<float>(static_cast<int>(v[i])), sc.sa[n] * sw, bias);
                    if (f1) {
                        const float up = __shfl_xor_sync(0xffffffffu, x, 1);
                        if (!(lane & 1) && wvalid && n < d.nrows)
                            p.act[static_cast<size_t>(d.row0 + n) * p.I + (wr >> 1)] = swiglu_attr_fast(x, up, p.attr);
                    } else if (wvalid && n < d.nrows) {
                        p.y[static_cast<size_t>(d.row0 + n) * p.H + wr] = __float2bfloat16_rn(x);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&tempty[acc]));
                mbar_arrive(smem_u32(&uempty[at]));
            }
            if (f1) {
                __threadfence();
                __syncwarp();
                if (lane == 0) atomicAdd(p.done + d.chunk, 1);
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
            next_slot();
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
        tmem_dealloc(tmem_base, 2 * kTok);
    }
    // errors: a wait that ran out, offsets out of order (found again for the report, behind
    // pdl_wait; block 0)
    if (threadIdx.x == 0) {
        pdl_wait();
        if (*abort_flag) atomicOr(p.err, kErrTimeout);
    }
    if (blockIdx.x == 0 && warp == 2) build_group_tiles(p.offsets, p.rows, p.err, p.E, kTok, s_off, s_pre, lane);
}

}  // namespace

// One launch for up to 48 rows per expert on average; with 8 rows and more, only where fc1 has
// more than two rounds of units for the CTA pairs (E ceil(2I / 256) > SMs), since the separate
// kernels (row quantiser, fc1, row quantiser, fc2) then have no stream to lose between them
// and shorter waits.  Measured (one launch / separate, us): E = 128, H = 2816, I = 704: 32
// rows 41.8 / 54.3, 1024 rows 127.0 / 158.1, 48 rows per expert 180.7 / 186.1, 64 per expert
// 239.0 / 193.7; E = 32, H = 1024, I = 512 (128 units): 4 rows per expert 24.7 / 24.9, 32 per
// expert 37.2 / 26.8; E = 8, H = 2816, I = 704: 1 row per expert 24.9 / 25.1, 32 per expert
// 35.2 / 29.3.
constexpr int kMostPerExpert = 48;

bool q8_ffn_supported(int rows, int E, int I) {
    const long long r = rows;
    return r <= static_cast<long long>(kMostPerExpert) * E && (r < 8LL * E || static_cast<long long>(E) * ((2 * I + 255) / 256) > device_sm_count());
}

// Two words per chunk and the scheduler's; for more rows than the kernel takes, those of the most.
int q8_ffn_counters(int rows, int E) {
    const int most = kMostPerExpert * E;
    return 2 * ((rows < most ? rows : most) / kTok + E + 1) + 1;
}

cudaError_t launch_q8_ffn(const Q8FfnArgs& a, cudaStream_t s) {
    if (a.rows <= 0) return cudaSuccess;
    CUtensorMap w1, x, w2, act;
    if (!tmap::pairs8(&w1, a.fc1_q, a.E, 2 * a.I, a.H, kWRows / 2, a.ep.fc1_chunked)) return cudaErrorInvalidValue;
    if (!tmap::pairs8(&w2, a.fc2_q, a.E, a.H, a.I, kWRows / 2, false)) return cudaErrorInvalidValue;
    if (!tmap::matrix8(&x, a.x_q, a.rows, a.H, kBox, a.ldx)) return cudaErrorInvalidValue;
    if (!tmap::matrix8(&act, a.act_q, a.rows, a.I, kBox, a.lda)) return cudaErrorInvalidValue;
    const int chunks = a.rows / kTok + a.E + 1;
    const Params p{a.offsets, a.E, a.rows, a.H, a.I, a.x_scale, a.ep.fc1_scale, a.ep.fc2_scale,
                   static_cast<const __nv_bfloat16*>(a.ep.fc1_bias), static_cast<const __nv_bfloat16*>(a.ep.fc2_bias),
                   a.act, a.act_q, a.lda, a.act_scale, static_cast<__nv_bfloat16*>(a.y), a.counters, a.counters + chunks,
                   a.counters + 2 * chunks, a.err, a.ep.act, a.ep.fc1_chunked};
    static bool done[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(q8_ffn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    // chunks: at most one a row, and one per 64 rows and one more for every expert
    const long long most = a.rows < a.rows / kTok + a.E ? a.rows : a.rows / kTok + a.E;
    const long long units = most * ((2 * a.I + kWRows - 1) / kWRows + (a.H + kWRows - 1) / kWRows);
    const int sms = device_sm_count();
    return launch_k_coop(q8_ffn_kernel, dim3(static_cast<unsigned>(units < sms ? units : sms)), dim3(kThreads),
                         static_cast<size_t>(kSmemBytes), s, true, w1, x, w2, act, p);
}

}  // namespace moe
