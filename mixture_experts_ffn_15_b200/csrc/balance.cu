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
// Forward: B blocks take equal ranges of tokens; a block writes one row of partial sums
// and counts for every sequence that its range meets, into slot b + s (walking along the
// tokens either the block or the sequence advances, so slots are unique).  A second launch
// adds each sequence's slots in order: no floating-point atomics, the same bits every time.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBThreads = 256;
constexpr int kBWarps = kBThreads / 32;
constexpr int kPer = kMaxExperts / 32;   // logits a lane holds
constexpr int kTokensPerBlockMin = 64;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Sequence bounds with offsets clamped to [0, T] (nullptr: one sequence, the batch).
__device__ __forceinline__ int seq_bound(const int32_t* seq, int s, int T) {
    return seq ? min(max(seq[s], 0), T) : (s == 0 ? 0 : T);
}

// Last sequence whose first token is at or before t (0 if none is).
__device__ __forceinline__ int seq_at(const int32_t* seq, int S, int t, int T) {
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_bound(seq, mid, T) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Softmax of one row, lane l holding logits l + 32 i.  fmaxf drops a NaN, but the
// exponential of the NaN itself reaches the sum; a row of -inf alone gives zeros.
__device__ __forceinline__ void row_softmax(const float* __restrict__ lg, int E, int lane, float* p) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        p[i] = e < E ? lg[e] : -INFINITY;
        m = fmaxf(m, p[i]);
    }
    m = warp_max(m);
    const bool none = m == -INFINITY;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        p[i] = (none && p[i] == -INFINITY) ? 0.f : expf(p[i] - m);
        sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) p[i] *= inv;
}

__global__ void __launch_bounds__(kBThreads)
balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                       const uint8_t* __restrict__ mask, const int32_t* __restrict__ seq, int T, int E,
                       int k, int S, int per_block, float* __restrict__ part_p,
                       int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                       int32_t* __restrict__ ticket, int32_t* __restrict__ err) {
    __shared__ float s_p[kBWarps][kMaxExperts];
    __shared__ int s_c[kMaxExperts];
    __shared__ int s_n;
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x;
    if (b == 0) {
        if (threadIdx.x == 0) *ticket = 0;
        if (seq && err) {
            // reported, not trusted: every use below is clamped
            bool bad = threadIdx.x == 0 && seq[0] != 0;
            for (int s = threadIdx.x; s < S; s += kBThreads)
                bad = bad || seq[s + 1] < seq[s] || seq[s + 1] > T;
            if (bad) atomicOr(err, kErrBadExpert);
        }
    }
    const int t0 = static_cast<int>(min(static_cast<long long>(b) * per_block, static_cast<long long>(T)));
    const int t1 = static_cast<int>(min(static_cast<long long>(t0) + per_block, static_cast<long long>(T)));
    for (int s = seq_at(seq, S, t0, T); s < S; ++s) {
        const int a = max(seq_bound(seq, s, T), t0), z = min(seq_bound(seq, s + 1, T), t1);
        if (seq_bound(seq, s, T) >= t1) break;
        if (a >= z) continue;
        for (int e = threadIdx.x; e < E; e += kBThreads) s_c[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
        int n = 0;
        for (int t = a + warp; t < z; t += kBWarps) {
            if (mask && !mask[t]) continue;
            ++n;
            float p[kPer];
            row_softmax(logits + static_cast<size_t>(t) * E, E, lane, p);
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += p[i];
            for (int j = lane; j < k; j += 32) {
                const int e = idx[static_cast<size_t>(t) * k + j];
                if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(&s_c[e], 1);
                else if (err) atomicOr(err, kErrBadExpert);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < E) s_p[warp][lane + 32 * i] = acc[i];
        if (lane == 0) atomicAdd(&s_n, n);
        __syncthreads();
        const size_t slot = static_cast<size_t>(b) + s;
        for (int e = threadIdx.x; e < E; e += kBThreads) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kBWarps; ++w) v += s_p[w][e];
            part_p[slot * E + e] = v;
            part_c[slot * E + e] = s_c[e];
        }
        if (threadIdx.x == 0) part_n[slot] = s_n;
        __syncthreads();
    }
}

// One block per sequence adds its slots; the last block to finish adds the sequences.
__global__ void __launch_bounds__(kBThreads)
balance_reduce_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                      const int32_t* __restrict__ part_n, const int32_t* __restrict__ seq, int T, int E,
                      int k, int S, int per_block, float coef, int32_t* __restrict__ ticket,
                      double* __restrict__ seq_loss, float* __restrict__ loss,
                      int32_t* __restrict__ counts, float* __restrict__ probs,
                      int32_t* __restrict__ tokens) {
    __shared__ double s_sum[kBThreads];
    __shared__ int s_last;
    pdl_wait();
    pdl_trigger();
    const int s = blockIdx.x, e = threadIdx.x;
    const int lo = seq_bound(seq, s, T), hi = seq_bound(seq, s + 1, T);
    const int b0 = lo / per_block, b1 = hi > lo ? (hi - 1) / per_block + 1 : b0;
    int n = 0;
    for (int b = b0; b < b1; ++b) n += part_n[b + s];
    double v = 0.0;
    if (e < E) {
        double sum = 0.0;
        long long c = 0;
        for (int b = b0; b < b1; ++b) {
            sum += static_cast<double>(part_p[static_cast<size_t>(b + s) * E + e]);
            c += part_c[static_cast<size_t>(b + s) * E + e];
        }
        const double P = n > 0 ? sum / n : 0.0;
        counts[static_cast<size_t>(s) * E + e] = static_cast<int32_t>(c);
        probs[static_cast<size_t>(s) * E + e] = static_cast<float>(P);
        if (n > 0) v = static_cast<double>(c) / (static_cast<double>(n) * k) * P * E;
    }
    if (e == 0) tokens[s] = n;
    s_sum[threadIdx.x] = v;
    for (int d = kBThreads / 2; d > 0; d >>= 1) {
        __syncthreads();
        if (threadIdx.x < d) s_sum[threadIdx.x] += s_sum[threadIdx.x + d];
    }
    if (threadIdx.x == 0) {
        seq_loss[s] = s_sum[0];
        __threadfence();
        s_last = atomicAdd(ticket, 1) == S - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last block: sequences in a fixed order
    v = 0.0;
    for (int i = threadIdx.x; i < S; i += kBThreads) v += __ldcg(seq_loss + i);
    s_sum[threadIdx.x] = v;
    for (int d = kBThreads / 2; d > 0; d >>= 1) {
        __syncthreads();
        if (threadIdx.x < d) s_sum[threadIdx.x] += s_sum[threadIdx.x + d];
    }
    if (threadIdx.x == 0) *loss = static_cast<float>(s_sum[0] * static_cast<double>(coef) / S);
}

__global__ void __launch_bounds__(kBThreads)
balance_grad_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ mask,
                    const int32_t* __restrict__ seq, const int32_t* __restrict__ counts,
                    const int32_t* __restrict__ tokens, int T, int E, int k, int S, float coef,
                    const float* __restrict__ grad_loss, float* __restrict__ dlogits) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float g = coef * (grad_loss ? *grad_loss : 1.f);
    int have = -1;
    float f[kPer], scale = 0.f;
    for (long long t = static_cast<long long>(blockIdx.x) * kBWarps + warp; t < T;
         t += static_cast<long long>(gridDim.x) * kBWarps) {
        float* d = dlogits + t * E;
        const int s = seq_at(seq, S, static_cast<int>(t), T);
        bool valid = t >= seq_bound(seq, s, T) && t < seq_bound(seq, s + 1, T);
        if (valid && mask) valid = mask[t] != 0;
        if (!valid) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < E) d[lane + 32 * i] = 0.f;
            continue;
        }
        if (s != have) {
            have = s;
            const double n = tokens[s] > 0 ? static_cast<double>(tokens[s]) : 1.0;
            scale = static_cast<float>(static_cast<double>(g) * E / (n * S));
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = lane + 32 * i;
                f[i] = 0.f;
                if (e < E) {
                    const long long c = counts[static_cast<size_t>(s) * E + e];
                    f[i] = static_cast<float>(static_cast<double>(c * E - static_cast<long long>(tokens[s]) * k) /
                                              (n * k * E));
                }
            }
        }
        float p[kPer], dot = 0.f;
        row_softmax(logits + t * E, E, lane, p);
#pragma unroll
        for (int i = 0; i < kPer; ++i) dot = fmaf(f[i], p[i], dot);
        dot = warp_sum(dot);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < E) d[lane + 32 * i] = scale * (p[i] * (f[i] - dot));
    }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct BalanceLayout {
    int blocks, per_block;
    size_t ticket, seq_loss, part_n, part_c, part_p, total;
};

BalanceLayout balance_layout(int T, int E, int S) {
    BalanceLayout L;
    const int most = 2 * 148;
    L.per_block = (T + most - 1) / most;
    if (L.per_block < kTokensPerBlockMin) L.per_block = kTokensPerBlockMin;
    L.blocks = (T + L.per_block - 1) / L.per_block;
    const size_t slots = static_cast<size_t>(L.blocks) + S;
    L.ticket = 0;
    L.seq_loss = 256;
    L.part_n = L.seq_loss + align256(static_cast<size_t>(S) * 8);
    L.part_c = L.part_n + align256(slots * 4);
    L.part_p = L.part_c + align256(slots * E * 4);
    L.total = L.part_p + align256(slots * E * 4);
    return L;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

cudaError_t launch_balance_loss(const BalanceArgs& a, cudaStream_t s) {
    const BalanceLayout L = balance_layout(a.T, a.E, a.S);
    char* ws = static_cast<char*>(a.workspace);
    int32_t* ticket = reinterpret_cast<int32_t*>(ws + L.ticket);
    double* seq_loss = reinterpret_cast<double*>(ws + L.seq_loss);
    int32_t* part_n = reinterpret_cast<int32_t*>(ws + L.part_n);
    int32_t* part_c = reinterpret_cast<int32_t*>(ws + L.part_c);
    float* part_p = reinterpret_cast<float*>(ws + L.part_p);
    cudaError_t e = launch_k(balance_partial_kernel, dim3(L.blocks > 0 ? L.blocks : 1), dim3(kBThreads), 0, s,
                             a.logits, a.topk_idx, a.mask, a.seq_offsets, a.T, a.E, a.k, a.S, L.per_block,
                             part_p, part_c, part_n, ticket, a.err);
    if (e != cudaSuccess) return e;
    return launch_k(balance_reduce_kernel, dim3(a.S), dim3(kBThreads), 0, s,
                    static_cast<const float*>(part_p), static_cast<const int32_t*>(part_c),
                    static_cast<const int32_t*>(part_n), a.seq_offsets, a.T, a.E, a.k, a.S, L.per_block,
                    a.coef, ticket, seq_loss, a.loss, a.counts, a.probs, a.tokens);
}

cudaError_t launch_balance_grad(const BalanceGradArgs& a, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    const long long want = (a.T + kBWarps - 1) / kBWarps, most = static_cast<long long>(device_sm_count()) * 8;
    return launch_k(balance_grad_kernel, dim3(static_cast<unsigned>(want < most ? want : most)),
                    dim3(kBThreads), 0, s, a.logits, a.mask, a.seq_offsets, a.counts, a.tokens, a.T, a.E,
                    a.k, a.S, a.coef, a.grad_loss, a.dlogits);
}

}  // namespace moe
