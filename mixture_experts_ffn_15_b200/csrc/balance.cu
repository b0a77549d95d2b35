// Load-balance loss of the routing, its per-expert counts, and its gradient.
//
// For every sequence s (a range of tokens; the whole batch is one by default) with n valid
// tokens, p_t = softmax(logits_t), c_e the number of (token, slot) pairs that chose e:
//   f_e = c_e / (n k),  P_e = (1 / n) sum_t p_te,  loss = (coef / S) sum_s E sum_e f_e P_e
// and, the counts being constants,
//   d loss / d logit_te = coef E / (S n) p_te (f_e - sum_j f_j p_tj).
// sum_j p_tj = 1, so f may be replaced by f - 1/E there: with balanced experts both terms
// are close to 1/E and their difference would lose its leading digits.  (c_e E - n k is
// formed in whole numbers, so the difference itself is exact.)
//
// Forward: the blocks take equal ranges of tokens; a block writes one row of partial sums
// and counts for every sequence that its range meets, into slot b + s (walking along the
// tokens either the block or the sequence advances, so slots are unique).  A second launch
// adds each sequence's slots in order: no floating-point atomics, the same bits every time.
// A batch that one block holds as one sequence is finished in the first launch.
//
// Batches of one sequence have kernels of their own (RAGGED false) without the walk (131071 x 256
// 38.2 us forward instead of 39.1, 64 tokens 3.4 instead of 3.6).
//
// A row's E logits are spread over LPR lanes with 8 each (two 16-byte vectors where E is a
// multiple of 4), 32 / LPR rows to a warp, the loads of the next two rows issued before the
// current one is used.  Bound by HBM: 4 T E bytes read, the gradient as much again and written.
// Measured, 131071 x 256, k = 8: forward 38 us (138 MB of logits, ids and mask; 6 us of it the
// second launch), gradient 49 us (268 MB, 5.5 TB/s).
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBThreads = 1024;
constexpr int kBWarps = kBThreads / 32;
constexpr int kGThreads = 384;           // two blocks an SM at 80 registers
constexpr int kPer = 8;                  // logits a lane holds
constexpr int kTokensPerBlockMin = 64;
constexpr int kOneBlockTokens = 256;     // up to here one block takes the batch
constexpr int kFold = 32;                // rows a lane adds up before it adds the sum to its longer one
constexpr int kMostRows = kFold * kFold; // rows a lane takes

// Sequence s is the tokens [M_s, M_{s+1}) with M_i the largest of the offsets 0 .. i, each
// clamped to [0, T]: offsets that decrease make empty sequences, and every token lies in one
// sequence at most whatever the offsets hold.  Valid offsets are their own M.

// Offset s clamped to [0, T] (nullptr: one sequence, the batch).
__device__ __forceinline__ int seq_offset(const int32_t* seq, int s, int T) {
    return seq ? min(max(seq[s], 0), T) : (s == 0 ? 0 : T);
}

// First i >= from with M_i > t (the first offset that is), S + 1 if there is none; by the whole
// block.  A search of every offset, not by halves: they may decrease.
__device__ __forceinline__ int first_behind(const int32_t* seq, int S, int from, int t, int T, int* s_first) {
    int at = S + 1;
    if (S < 32) {   // every warp by itself
        const int i = static_cast<int>(threadIdx.x) & 31;
        const unsigned hits = __ballot_sync(0xffffffffu, i >= from && i <= S && seq_offset(seq, min(i, S), T) > t);
        return hits ? __ffs(hits) - 1 : S + 1;
    }
    if (threadIdx.x == 0) *s_first = S + 1;
    __syncthreads();
    constexpr int kBatch = 16;   // loads in flight; most searches need one
    for (int i0 = from + threadIdx.x; i0 <= S && at > S; i0 += kBatch * blockDim.x) {
#pragma unroll
        for (int u = kBatch - 1; u >= 0; --u) {
            const int i = i0 + u * static_cast<int>(blockDim.x);
            if (i <= S && seq_offset(seq, i, T) > t) at = i;
        }
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if ((threadIdx.x & 31) == 0 && at <= S) atomicMin(s_first, at);
    __syncthreads();
    at = *s_first;
    __syncthreads();   // it may be searched again
    return at;
}

// The 8 logits of lane l (of LPR) of a row: with VEC, experts 4 l .. 4 l + 3 and
// 4 LPR + 4 l .. + 3, else l + LPR i.
template <int LPR, bool VEC>
struct Row {
    float v[kPer];
    static __device__ __forceinline__ int expert(int l, int i) {
        return VEC ? (i >> 2) * 4 * LPR + 4 * l + (i & 3) : l + LPR * i;
    }
    __device__ __forceinline__ void load(const float* __restrict__ row, int E, int l, bool live) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = -INFINITY;
        if (!live) return;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                if (expert(l, i) < E) {
                    const float4 x = __ldg(reinterpret_cast<const float4*>(row + expert(l, i)));
                    v[i] = x.x;
                    v[i + 1] = x.y;
                    v[i + 2] = x.z;
                    v[i + 3] = x.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (expert(l, i) < E) v[i] = __ldg(row + expert(l, i));
        }
    }
    __device__ __forceinline__ void store(float* __restrict__ row, int E, int l) const {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                if (expert(l, i) < E)
                    *reinterpret_cast<float4*>(row + expert(l, i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (expert(l, i) < E) row[expert(l, i)] = v[i];
        }
    }
    // logits -> probabilities.  fmaxf drops a NaN, but the NaN's own exponential reaches the
    // sum; a row of -inf alone gives zeros.
    __device__ __forceinline__ void softmax() {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i) m = fmaxf(m, v[i]);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // without a maximum: exp(-inf - 0) = 0 for a row of -inf, NaN for a NaN
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            v[i] = __expf(v[i] - base);   // |logit - max| 2^-23 and 2 ulp: a few instructions of ten
            sum += v[i];
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] *= inv;
    }
};

struct BalanceParams {
    const float* logits;
    const int32_t* idx;
    const uint8_t* mask;
    const int32_t* seq;
    int T, E, k, S, per_block, blocks;
    float coef;
    int32_t* bad;          // are the sequence offsets not their own M?
    float* part_p;         // [blocks + S, E]
    int32_t* part_c;       // [blocks + S, E]
    int32_t* part_n;       // [blocks + S]
    int32_t* ticket;
    double* seq_loss;      // [S, ceil(E / 32)]
    float* loss;
    int32_t* counts;
    float* probs;
    int32_t* tokens;
    int32_t* err;
};

// Sum of one double per thread, in a fixed order; the result on thread 0.
__device__ __forceinline__ double block_sum(double v, double* s) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) s[warp] = v;
    __syncthreads();
    if (warp == 0) {
        v = lane < static_cast<int>(blockDim.x >> 5) ? s[lane] : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
}

// Counts, mean probability and E f P of one expert of one sequence.
__device__ __forceinline__ double finish_expert(const BalanceParams& p, int s, int e, double sum, long long c, int n) {
    const double P = n > 0 ? sum / n : 0.0;
    p.counts[static_cast<size_t>(s) * p.E + e] = static_cast<int32_t>(c);
    p.probs[static_cast<size_t>(s) * p.E + e] = static_cast<float>(P);
    return n > 0 ? static_cast<double>(c) / (static_cast<double>(n) * p.k) * P * p.E : 0.0;
}

template <int LPR, bool VEC, bool RAGGED>
__global__ void __launch_bounds__(kBThreads, 1)
balance_partial_kernel(const BalanceParams p) {
    constexpr int kRows = 32 / LPR;     // rows of a warp
    __shared__ float s_p[kBWarps][kMaxExperts];   // folded sums of the lanes, then sums of the warps
    static_assert(kMaxExperts == 32 * kPer, "a warp's folded sums");
    __shared__ int s_c[kMaxExperts];
    __shared__ int s_n, s_first;
    __shared__ double s_red[kBWarps];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane & (LPR - 1), sub = lane / LPR;
    const int b = blockIdx.x, E = p.E, T = p.T, S = RAGGED ? p.S : 1;
    if (b == 0) {
        if (threadIdx.x == 0) *p.ticket = 0;
        if (RAGGED) {
            // reported, not trusted: every use below is clamped
            bool bad = threadIdx.x == 0 && p.seq[0] != 0;
            for (int s = threadIdx.x; s < S; s += kBThreads)
                bad = bad || p.seq[s + 1] < p.seq[s] || p.seq[s + 1] > T;
            bad = __syncthreads_or(bad);
            if (threadIdx.x == 0) {
                *p.bad = bad;
                if (bad && p.err) atomicOr(p.err, kErrBadExpert);
            }
        }
    }
    const int t0 = static_cast<int>(min(static_cast<long long>(b) * p.per_block, static_cast<long long>(T)));
    const int t1 = static_cast<int>(min(static_cast<long long>(t0) + p.per_block, static_cast<long long>(T)));
    const bool single = p.blocks <= 1 && S == 1;   // one block finishes the batch
    // The walk starts with token t0's sequence, the one before the first bound behind t0 (its
    // own bound is at or before t0: lo = t0 stands for it).
    const int i1 = RAGGED ? first_behind(p.seq, S, 0, t0, T, &s_first) : 1;
    int lo = RAGGED && i1 == 0 ? seq_offset(p.seq, 0, T) : t0, empty = 0;
    for (int s = single ? 0 : max(i1 - 1, 0); s < S; ++s) {
        int a = t0, z = t1;
        if (RAGGED) {
            if (lo >= t1 && !single) break;
            a = max(lo, t0);
            lo = max(lo, seq_offset(p.seq, s + 1, T));
            z = min(lo, t1);
            if (a >= z && !single) {
                // over a long run of empty sequences in one search
                if (++empty % 16 == 0) s = first_behind(p.seq, S, s + 1, lo, T, &s_first) - 2;
                continue;
            }
        }
        for (int e = threadIdx.x; e < E; e += kBThreads) s_c[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
        int n = 0;
        constexpr int kStep = kBWarps * kRows;
        // ids: the range's pairs in order over all threads (row by row, each row would wait
        // for its ids: 46.6 us instead of 39.8 at 131071 x 256)
        const long long q0 = static_cast<long long>(a) * p.k, q1 = static_cast<long long>(z) * p.k;
#pragma unroll 4
        for (long long q = q0 + threadIdx.x; q < q1; q += kBThreads) {
            const int e = p.idx[q];
            if (p.mask && p.mask[q / p.k] == 0) continue;
            if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(&s_c[e], 1);
            else if (p.err) atomicOr(p.err, kErrBadExpert);
        }
        auto row = [&](int t) { return p.logits + static_cast<size_t>(t) * E; };
        auto mask_of = [&](int t) { return t < z && p.mask ? p.mask[t] : static_cast<uint8_t>(1); };
        int t = a + warp * kRows + sub;
        Row<LPR, VEC> r, next, next2;
        uint8_t m = mask_of(t), m1 = mask_of(t + kStep);
        r.load(row(t), E, l, t < z);
        next.load(row(t + kStep), E, l, t + kStep < z);
        const int trips = (z - a - warp * kRows + kStep - 1) / kStep;   // of this warp
        for (int it0 = 0; it0 < trips; it0 += kFold) {
            const int end = min(it0 + kFold, trips);
#pragma unroll 1
            for (int it = it0; it < end; ++it) {
                const uint8_t m2 = mask_of(t + 2 * kStep);
                next2.load(row(t + 2 * kStep), E, l, t + 2 * kStep < z);
                const bool live = t < z && m != 0;
                r.softmax();   // a row past the end holds -inf: zeros
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc[i] += live ? r.v[i] : 0.f;
                n += live && l == 0;
                t += kStep;
                m = m1;
                m1 = m2;
                r = next;
                next = next2;
            }
            if (end < trips) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    s_p[warp][32 * i + lane] = (it0 == 0 ? 0.f : s_p[warp][32 * i + lane]) + acc[i];
                    acc[i] = 0.f;
                }
            }
        }
        if (trips > kFold) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += s_p[warp][32 * i + lane];
            __syncwarp();
        }
        // the warp's rows, then the warps, in order
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (Row<LPR, VEC>::expert(l, i) < E) s_p[warp][Row<LPR, VEC>::expert(l, i)] = acc[i];
        }
        if (lane == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        const int e = threadIdx.x;
        float v = 0.f;
        if (e < E) {
#pragma unroll
            for (int w = 0; w < kBWarps; ++w) v += s_p[w][e];
        }
        if (single) {
            // the whole batch is here
            double term = 0.0;
            if (e < E) term = finish_expert(p, 0, e, static_cast<double>(v), s_c[e], s_n);
            term = block_sum(term, s_red);
            if (threadIdx.x == 0) {
                p.tokens[0] = s_n;
                *p.loss = static_cast<float>(term * static_cast<double>(p.coef));
            }
            return;
        }
        const size_t slot = static_cast<size_t>(b) + s;
        if (e < E) {
            p.part_p[slot * E + e] = v;
            p.part_c[slot * E + e] = s_c[e];
        }
        if (threadIdx.x == 0) p.part_n[slot] = s_n;
        __syncthreads();
    }
}

// One block per sequence and 32 experts adds its slots (32 strips of threads take every 32nd
// one, then the strips in order); the last block to finish adds the blocks' terms.
constexpr int kRExperts = 32;

__global__ void __launch_bounds__(kBThreads)
balance_reduce_kernel(const BalanceParams p) {
    __shared__ double s_sum[kBThreads];
    __shared__ int s_cnt[kBThreads];
    __shared__ double s_red[kBWarps];
    __shared__ int s_n, s_last;
    if (threadIdx.x == 0) s_n = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int s = blockIdx.x, E = p.E, nb = gridDim.y;
    const int e = static_cast<int>(blockIdx.y) * kRExperts + (threadIdx.x & 31), st = threadIdx.x >> 5;
    int lo = 0, hi = p.T;
    if (p.seq) {
        lo = seq_offset(p.seq, s, p.T);
        hi = seq_offset(p.seq, s + 1, p.T);
        if (*p.bad) {   // M_s and M_{s+1}
            for (int i = threadIdx.x; i < s; i += kBThreads) lo = max(lo, seq_offset(p.seq, i, p.T));
            lo = __reduce_max_sync(0xffffffffu, lo);
            if ((threadIdx.x & 31) == 0) s_cnt[threadIdx.x >> 5] = lo;
            __syncthreads();
            for (int i = 0; i < kBWarps; ++i) lo = max(lo, s_cnt[i]);
            __syncthreads();
            hi = max(lo, hi);
        }
    }
    const int b0 = lo / p.per_block, b1 = hi > lo ? (hi - 1) / p.per_block + 1 : b0;
    int n = 0;
    for (int b = b0 + threadIdx.x; b < b1; b += kBThreads) n += p.part_n[b + s];
    if (n) atomicAdd(&s_n, n);
    double sum = 0.0;
    int c = 0;
    if (e < E) {
#pragma unroll 4
        for (int b = b0 + st; b < b1; b += kBWarps) {
            sum += static_cast<double>(p.part_p[static_cast<size_t>(b + s) * E + e]);
            c += p.part_c[static_cast<size_t>(b + s) * E + e];
        }
    }
    s_sum[threadIdx.x] = sum;
    s_cnt[threadIdx.x] = c;
    __syncthreads();
    double v = 0.0;
    if (st == 0 && e < E) {
        long long cc = c;
#pragma unroll 8
        for (int i = 1; i < kBWarps; ++i) {
            sum += s_sum[i * kRExperts + threadIdx.x];
            cc += s_cnt[i * kRExperts + threadIdx.x];
        }
        v = finish_expert(p, s, e, sum, cc, s_n);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) p.tokens[s] = s_n;
    if (st == 0) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (threadIdx.x == 0) {
            p.seq_loss[static_cast<size_t>(s) * nb + blockIdx.y] = v;
            __threadfence();
            s_last = atomicAdd(p.ticket, 1) == p.S * nb - 1;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    v = 0.0;
    for (int i = threadIdx.x; i < p.S * nb; i += kBThreads) v += __ldcg(p.seq_loss + i);
    v = block_sum(v, s_red);
    if (threadIdx.x == 0) *p.loss = static_cast<float>(v * static_cast<double>(p.coef) / p.S);
}

template <int LPR, bool VEC>
__global__ void __launch_bounds__(kGThreads, 2)
balance_grad_kernel(const BalanceGradArgs a, int per_block) {
    constexpr int kRows = 32 / LPR, kStep = (kGThreads / 32) * kRows;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane & (LPR - 1), sub = lane / LPR;
    const int T = a.T, E = a.E;
    const float g = a.coef * (a.grad_loss ? *a.grad_loss : 1.f);
    const int t0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * per_block, static_cast<long long>(T)));
    const int t1 = static_cast<int>(min(static_cast<long long>(t0) + per_block, static_cast<long long>(T)));
    int t = t0 + warp * kRows + sub;
    // the lane group's sequence: its bounds (M), shares less 1/E and scale; t only grows.  It
    // starts with the block's first token, as the forward's walk does.
    __shared__ int s_first;
    const int i1 = !a.seq_offsets ? 1 : first_behind(a.seq_offsets, a.S, 0, t0, T, &s_first);
    int s = min(max(i1 - 1, 0), a.S - 1);
    int lo = i1 == 0 ? seq_offset(a.seq_offsets, 0, T) : t0;
    int hi = i1 > a.S ? t0 : max(lo, seq_offset(a.seq_offsets, s + 1, T));
    int have = -1;
    float f[kPer], scale = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) f[i] = 0.f;
    auto row = [&](int u) { return a.logits + static_cast<size_t>(u) * E; };
    auto mask_of = [&](int u) { return u < t1 && a.mask ? a.mask[u] : static_cast<uint8_t>(1); };
    uint8_t m = mask_of(t);
    Row<LPR, VEC> r, next, next2;
    uint8_t m1 = mask_of(t + kStep);
    r.load(row(t), E, l, t < t1);
    next.load(row(t + kStep), E, l, t + kStep < t1);
    const int trips = (t1 - t0 - warp * kRows + kStep - 1) / kStep;
    for (int it = 0; it < trips; ++it) {
        const int tn = t + kStep;
        const uint8_t m2 = mask_of(t + 2 * kStep);
        next2.load(row(t + 2 * kStep), E, l, t + 2 * kStep < t1);
        while (t >= hi && s + 1 < a.S && t < t1) {
            ++s;
            lo = hi;
            hi = max(lo, seq_offset(a.seq_offsets, s + 1, T));
        }
        const bool live = t < t1 && m != 0 && t >= lo && t < hi;
        if (live && s != have) {
            have = s;
            const int n = a.tokens[s];
            const double nd = n > 0 ? static_cast<double>(n) : 1.0;
            scale = static_cast<float>(static_cast<double>(g) * E / (nd * a.S));
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = Row<LPR, VEC>::expert(l, i);
                f[i] = 0.f;
                if (e < E) {
                    const long long c = a.counts[static_cast<size_t>(s) * E + e];
                    f[i] = static_cast<float>(static_cast<double>(c * E - static_cast<long long>(n) * a.k) / (nd * a.k * E));
                }
            }
        }
        r.softmax();
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) dot = fmaf(f[i], r.v[i], dot);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
#pragma unroll
        for (int i = 0; i < kPer; ++i) r.v[i] = live ? scale * (r.v[i] * (f[i] - dot)) : 0.f;
        if (t < t1) r.store(a.dlogits + static_cast<size_t>(t) * E, E, l);
        t = tn;
        m = m1;
        m1 = m2;
        r = next;
        next = next2;
    }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BalanceLayout {
    int blocks, per_block;
    size_t ticket, bad, seq_loss, part_n, part_c, part_p, total;
};

// Lanes of a row: the smallest power of two that holds E logits at 8 a lane.
int lanes_per_row(int E) {
    int n = 1;
    while (n * kPer < E) n *= 2;
    return n;
}

// One block an SM, as many times over as it takes for ranges of at most kMostRows rows a lane.
// With the sums folded every kFold rows, a float32 probability goes through at most 31 + 32
// additions of a lane, 5 of the lanes and 31 of the warps in front of the second launch's
// float64, whatever T is.  (400000 x 256 forward: 88 us, one long sum a lane 86, ranges of
// kFold rows instead 97.)
BalanceLayout balance_layout(int T, int E, int S) {
    BalanceLayout L;
    // a fixed count: the same cut, so the same bits, on any GPU, and sizes that need no device
    const int sms = 148, range = kMostRows * kBWarps * (32 / lanes_per_row(E));
    const int each = (T + sms - 1) / sms;
    const int most = sms * (each > range ? (each + range - 1) / range : 1);
    L.per_block = (T + most - 1) / most;
    if (L.per_block < kTokensPerBlockMin) L.per_block = kTokensPerBlockMin;
    if (T <= kOneBlockTokens) L.per_block = kOneBlockTokens;
    L.blocks = (T + L.per_block - 1) / L.per_block;
    // the blocks' upper bound, which grows with T as their number does not
    const int finest = (T + kTokensPerBlockMin - 1) / kTokensPerBlockMin;
    const size_t slots = static_cast<size_t>(finest < most ? finest : most) + S;
    L.ticket = 0;
    L.bad = 4;
    L.seq_loss = 256;
    L.part_n = L.seq_loss + align256(static_cast<size_t>(S) * ((E + kRExperts - 1) / kRExperts) * 8);
    L.part_c = L.part_n + align256(slots * 4);
    L.part_p = L.part_c + align256(slots * E * 4);
    L.total = L.part_p + align256(slots * E * 4);
    return L;
}

// fn(lanes per row, vector loads).
template <typename F>
cudaError_t by_experts(int E, F fn) {
    const bool vec = E % 4 == 0;
    auto go = [&](auto lpr) {
        constexpr int L = decltype(lpr)::value;
        return vec ? fn(lpr, std::true_type()) : fn(std::integral_constant<int, L>(), std::false_type());
    };
    switch (lanes_per_row(E)) {
        case 1: return go(std::integral_constant<int, 1>());
        case 2: return go(std::integral_constant<int, 2>());
        case 4: return go(std::integral_constant<int, 4>());
        case 8: return go(std::integral_constant<int, 8>());
        case 16: return go(std::integral_constant<int, 16>());
        default: return go(std::integral_constant<int, 32>());
    }
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
    const BalanceLayout L = balance_layout(a.T, a.E, a.S);
    char* ws = static_cast<char*>(a.workspace);
    const BalanceParams p{a.logits, a.topk_idx, a.mask, a.seq_offsets, a.T, a.E, a.k, a.S, L.per_block, L.blocks,
                          a.coef, reinterpret_cast<int32_t*>(ws + L.bad), reinterpret_cast<float*>(ws + L.part_p), reinterpret_cast<int32_t*>(ws + L.part_c),
                          reinterpret_cast<int32_t*>(ws + L.part_n), reinterpret_cast<int32_t*>(ws + L.ticket),
                          reinterpret_cast<double*>(ws + L.seq_loss), a.loss, a.counts, a.probs, a.tokens, a.err};
    const dim3 grid(L.blocks > 0 ? L.blocks : 1), block(kBThreads);
    const cudaError_t e = by_experts(a.E, [&](auto lpr, auto vec) {
        constexpr int lanes = decltype(lpr)::value;
        constexpr bool V = decltype(vec)::value;
        return a.seq_offsets ? launch_k(balance_partial_kernel<lanes, V, true>, grid, block, 0, s, p)
                             : launch_k(balance_partial_kernel<lanes, V, false>, grid, block, 0, s, p);
    });
    if (e != cudaSuccess || (L.blocks <= 1 && a.S == 1)) return e;
    return launch_k(balance_reduce_kernel, dim3(a.S, (a.E + kRExperts - 1) / kRExperts), block, 0, s, p);
}

cudaError_t launch_balance_grad(const BalanceGradArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    const int most = 2 * device_sm_count();
    int per_block = (a.T + most - 1) / most;
    if (per_block < 16) per_block = 16;
    const dim3 grid((a.T + per_block - 1) / per_block), block(kGThreads);
    return by_experts(a.E, [&](auto lpr, auto vec) {
        return launch_k(balance_grad_kernel<decltype(lpr)::value, decltype(vec)::value>, grid, block, 0, s, a, per_block);
    });
}

}  // namespace moe
