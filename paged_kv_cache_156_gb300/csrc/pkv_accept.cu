// speculative_accept: drafted tokens accepted or refused against the target's
// probabilities, and the token that follows, from given random numbers.
//
// Draft i (token x_i, drawn from q_i) is kept while u_i q_i(x_i) < p_i(x_i);
// after a kept draft the next is looked at.  At the first refusal, position a,
// the next token is drawn from the weights max(p_a - q_a, 0); when every draft
// is kept, from the target's next row.  So the tokens follow the target's
// distribution whatever the draft's.  A draft without probabilities (q null) is
// taken as certain: kept while u_i < p_i(x_i), and refused, x_i leaves the row.
//
// The draw is the inverse of the cumulative sum, and the answer is a whole
// number, so the sum must not depend on its order.  Each weight is therefore
// cut to whole units of 2^-44 (fp32 times 2^44 is exact; what is cut off a row
// of 2^18 tokens is below 2^-26 of it, less than the rounding of the
// probabilities themselves) and summed in 64-bit integers: with T the total,
// the token is the first whose inclusive sum exceeds floor(u T).
//
// One cluster a sequence: its CTAs take a contiguous piece of the row each, a
// warp a contiguous piece of that, held in registers, so the row is read once;
// totals go round through distributed shared memory, and the warp that holds
// the mark scans its registers.  Rows of more than kHeld weights a cluster are
// summed in several rounds and the round that holds the mark is read again.
// Bound by latency at a few sequences (some dependent loads: draft token, its
// probabilities, the row), by HBM at many.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kIters = 8;                           // groups of 128 weights a warp holds
constexpr int kHeld = kCluster * kWarps * kIters * 128;     // weights of a round
constexpr float kUnit = 17592186044416.0f;          // 2^44

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (std::is_same<T, float>::value) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}

// Four consecutive probabilities from element i of a row (0 past its end).
template <typename T>
__device__ __forceinline__ void load4(const T* row, int64_t i, int64_t vocab, bool vec, float (&x)[4]) {
    if (vec && i + 4 <= vocab) {
        if constexpr (std::is_same<T, float>::value) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(row + i));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(row + i));
            const float2 lo = Mma<T>::unpack(v.x), hi = Mma<T>::unpack(v.y);
            x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e < vocab ? to_f32(row[i + e]) : 0.0f;
    }
}

__device__ __forceinline__ unsigned long long units(float w) {
    return w > 0.0f ? static_cast<unsigned long long>(__float2ull_rz(fminf(w, 1.0f) * kUnit)) : 0ull;   // (NaN: none)
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) accept_kernel(const AcceptArgs a) {
    __shared__ unsigned long long warp_total[kWarps];
    __shared__ unsigned long long cta_total[2][kCluster];   // every CTA's total of a round (alternating rounds)
    __shared__ int s_kept;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / kCluster;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    auto started = cluster.barrier_arrive();        // (waited for before the first write into another CTA)
    grid_dependency_wait();
    launch_dependents();
    const int K = a.max_drafts;
    const int64_t V = a.vocab;
    const T* target = static_cast<const T*>(a.target_probs) + static_cast<int64_t>(b) * (K + 1) * V;
    const T* draft = a.draft_probs ? static_cast<const T*>(a.draft_probs) + static_cast<int64_t>(b) * K * V : nullptr;
    const int64_t* drafts = a.draft_tokens + static_cast<int64_t>(b) * K;
    const float* uniform = a.uniform + static_cast<int64_t>(b) * (K + 1);

    // ---- the first refused draft, by the first warp of every CTA
    int n = K;
    if (a.num_drafts) {
        n = __ldcg(a.num_drafts + b);
        if (n < 0 || n > K) {
            if (rank == 0 && t == 0) raise_error(a.err, kErrBounds);
            n = min(max(n, 0), K);
        }
    }
    if (warp == 0) {
        int kept = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + lane;
            bool keep = false;
            if (i < n) {
                const int64_t x = __ldcg(drafts + i);
                if (x >= 0 && x < V) {
                    // (both factors have 24 bits: the fp64 product is exact)
                    const double q = draft ? static_cast<double>(to_f32(draft[i * V + x])) : 1.0;
                    keep = static_cast<double>(__ldcg(uniform + i)) * q < static_cast<double>(to_f32(target[i * V + x]));
                } else if (rank == 0) {
                    raise_error(a.err, kErrBounds);
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, keep);
            const int run = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            kept += run;
            if (run < 32) break;
        }
        kept = min(kept, n);
        if (lane == 0) s_kept = kept;
        if (rank == 0) {
            for (int i = lane; i <= K; i += 32)
                if (i != kept) a.tokens[static_cast<int64_t>(b) * (K + 1) + i] = i < kept ? __ldcg(drafts + i) : -1;
            if (lane == 0) a.num_accepted[b] = kept;
        }
    }
    __syncthreads();
    const int kept = s_kept;
    const bool refused = kept < n;
    const T* prow = target + static_cast<int64_t>(kept) * V;
    const T* qrow = refused && draft ? draft + static_cast<int64_t>(kept) * V : nullptr;
    const int64_t out_x = refused && !draft ? __ldcg(drafts + kept) : -1;      // the weight that leaves the row
    const float u = __ldcg(uniform + K);
    constexpr int kVec = std::is_same<T, float>::value ? 16 : 8;
    const bool vec = ((reinterpret_cast<uintptr_t>(prow) | (qrow ? reinterpret_cast<uintptr_t>(qrow) : 0)) & (kVec - 1)) == 0;
    const int rounds = static_cast<int>((V + kHeld - 1) / kHeld);
    // a warp's weights of a round: per groups of 128 from `first`
    const int64_t per = ((min(V, static_cast<int64_t>(kHeld)) + kCluster * kWarps * 128 - 1) / (kCluster * kWarps * 128)) * 128;
    const int iters = static_cast<int>(per / 128);

    float w[kIters][4];
    unsigned flips = 0;                             // which half of cta_total this exchange uses
    auto load = [&](int round, bool residual) {     // this warp's weights and their total
        const int64_t first = static_cast<int64_t>(round) * kHeld + (static_cast<int64_t>(rank) * kWarps + warp) * per + 4 * lane;
        float p[kIters][4], q[kIters][4];
#pragma unroll
        for (int k = 0; k < kIters; ++k)
            if (k < iters) load4(prow, first + 128 * k, V, vec, p[k]);
        if (residual && qrow) {
#pragma unroll
            for (int k = 0; k < kIters; ++k)
                if (k < iters) load4(qrow, first + 128 * k, V, vec, q[k]);
        }
        unsigned long long sum = 0;
#pragma unroll
        for (int k = 0; k < kIters; ++k) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = k < iters ? p[k][e] : 0.0f;
                if (residual && qrow && k < iters) x -= q[k][e];
                if (residual && first + 128 * k + e == out_x) x = 0.0f;
                w[k][e] = x;
                sum += units(x);
            }
        }
        return warp_sum(sum);
    };
    auto exchange = [&](unsigned long long mine) {  // every CTA's total into cta_total[flips]; this CTA's warps' into warp_total
        __syncthreads();                            // (warp_total is no longer read)
        if (lane == 0) warp_total[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long sum = warp_sum(lane < kWarps ? warp_total[lane] : 0ull);
            if (lane < kCluster) *cluster.map_shared_rank(&cta_total[flips][rank], lane) = sum;
        }
        cluster.sync();
    };

    cluster.barrier_wait(std::move(started));
    for (int pass = 0; pass < 2; ++pass) {
        const bool residual = pass == 0;
        unsigned long long total = 0, before_round = 0;
        for (int round = 0; round < rounds; ++round) {
            exchange(load(round, residual));
#pragma unroll
            for (int c = 0; c < kCluster; ++c) total += cta_total[flips][c];
            flips ^= 1u;
        }
        if (total == 0) {
            if (pass == 0) continue;                // nothing left of the row: draw from the target's itself
            if (rank == 0 && t == 0) a.tokens[static_cast<int64_t>(b) * (K + 1) + kept] = -1;
            break;
        }
        const double z = (u > 0.0f ? static_cast<double>(u) : 0.0) * static_cast<double>(total);
        const unsigned long long mark = min(__double2ull_rz(z), total - 1);
        for (int round = 0; round < rounds; ++round) {
            if (rounds > 1) {
                exchange(load(round, residual));
                flips ^= 1u;
            }
            // the totals before this warp's weights, in the row's order
            unsigned long long before = before_round, all = 0;
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                const unsigned long long x = cta_total[flips ^ 1u][c];
                before += c < rank ? x : 0ull;
                all += x;
            }
            for (int v = 0; v < warp; ++v) before += warp_total[v];
            if (mark >= before && mark < before + warp_total[warp]) {
                const int64_t first = static_cast<int64_t>(round) * kHeld + (static_cast<int64_t>(rank) * kWarps + warp) * per + 4 * lane;
                unsigned long long at = before;
#pragma unroll
                for (int k = 0; k < kIters; ++k) {
                    if (k >= iters) break;
                    unsigned long long c[4];
                    c[0] = units(w[k][0]);
                    c[1] = c[0] + units(w[k][1]);
                    c[2] = c[1] + units(w[k][2]);
                    c[3] = c[2] + units(w[k][3]);
                    unsigned long long inc = c[3];
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
                        if (lane >= o) inc += y;
                    }
                    const unsigned long long mine = at + inc - c[3];     // before this lane's four
                    if (mark >= mine && mark < mine + c[3]) {
                        const int e = mark < mine + c[0] ? 0 : mark < mine + c[1] ? 1 : mark < mine + c[2] ? 2 : 3;
                        a.tokens[static_cast<int64_t>(b) * (K + 1) + kept] = first + 128 * k + e;
                    }
                    at += __shfl_sync(0xffffffffu, inc, 31);
                }
            }
            before_round += all;
            if (mark < before_round) break;         // (the same in every thread of the cluster)
        }
        break;
    }
    cluster.sync();                                 // no CTA leaves while another may still write its shared memory
}

template <typename T>
cudaError_t launch(const AcceptArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, accept_kernel<T>, a);
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, int dtype, cudaStream_t s) {
    if (a.num_seqs <= 0) return cudaSuccess;
    if (dtype == 0) return launch<__half>(a, s);
    if (dtype == 1) return launch<__nv_bfloat16>(a, s);
    return launch<float>(a, s);
}

}  // namespace pkv
