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
// cut to whole units of 2^-44 (fp32 times 2^44 is exact) and summed in 64-bit
// integers: with T the total, the token is the first whose inclusive sum exceeds
// floor(u T).  What is cut off a row is below 2^-44 a token, 2^-25 at the largest
// vocabulary, of a target row that sums to 1.  Of a residual max(p - q, 0) that
// sums to R it may be a larger share, up to all of it (the target's own row is
// then drawn from), but a refusal is itself only as likely as R: a token's
// probability over both stays within 2^-25.
//
// One cluster a sequence: its CTAs take a contiguous piece of the row each, a
// warp a contiguous piece of that, so the row is read once; totals go round
// through distributed shared memory.  Every lane keeps its sum of each batch of
// 512 weights in shared memory, so the warp that holds the mark finds the batch
// from there and reads those 512 weights again.  (Weights held in registers
// instead spilled at two CTAs an SM: 36 us for 64 sequences of 128000 tokens.
// The float32 form still spills 44 bytes a thread at its 64 registers.)
// Bound by latency: at a few sequences by dependent loads (draft token, its
// probabilities, the row: 5.1 us for one of 32000 tokens), at many by those and
// the exchange (64 sequences of 128000 float32, 41 MB read: 9.8 us with the rows
// in L2 from the call before, of which they take 5; 12.0 us with the rows in HBM,
// 50% of the copy rate.  A prefetch of the pieces into L2 ahead of the loop made
// the first of these 11.6).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;                           // groups of 128 weights whose loads are in flight together
constexpr int kMaxBatches = (PKV_ACCEPT_MAX_VOCAB + 3 + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128);

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (std::is_same<T, float>::value) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}

// Four probabilities, as one vector load brings them.
template <typename T>
struct Four {
    static constexpr int kWords = 2;
    static __device__ __forceinline__ void unpack(const uint32_t (&v)[2], float (&x)[4]) {
        const float2 lo = Mma<T>::unpack(v[0]), hi = Mma<T>::unpack(v[1]);
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    }
    // elements d to d + 3 of v and the vector after it, n (d: 1 to 3)
    static __device__ __forceinline__ void shift(uint32_t (&v)[2], const uint32_t (&n)[2], int d) {
        const uint32_t a = d >= 2 ? v[1] : v[0], b = d >= 2 ? n[0] : v[1], c = d >= 2 ? n[1] : n[0];
        v[0] = (d & 1) ? __funnelshift_r(a, b, 16) : a;
        v[1] = (d & 1) ? __funnelshift_r(b, c, 16) : b;
    }
    static __device__ __forceinline__ void load(uint32_t (&v)[2], const T* p) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
        v[0] = r.x; v[1] = r.y;
    }
};
template <>
struct Four<float> {
    static constexpr int kWords = 4;
    static __device__ __forceinline__ void unpack(const uint32_t (&v)[4], float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(v[e]);
    }
    static __device__ __forceinline__ void shift(uint32_t (&v)[4], const uint32_t (&n)[4], int d) {
        const uint32_t x[7] = {v[0], v[1], v[2], v[3], n[0], n[1], n[2]};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = d == 1 ? x[e + 1] : d == 2 ? x[e + 2] : x[e + 3];
    }
    static __device__ __forceinline__ void load(uint32_t (&v)[4], const float* p) {
        const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    }
};

// Whole units of a weight in [0, 1] (clipped as it is formed, NaN to 0), floor(w 2^44), as two 22-bit halves added
// to hi and lo: w + 2 rounded towards zero holds floor(w 2^22) in its significand's last bits, what is left of w
// (exact) plus 2^-21 the next 22.  Seven single-rate instructions a weight with its clipped difference; a shift by
// the exponent took twice that, the conversion to 64-bit integers runs at a sixteenth of the rate.
__device__ __forceinline__ void add_units(float w, uint32_t& hi, uint32_t& lo) {
    const float y = __fadd_rz(w, 2.0f);
    const float rest = __fsub_rn(w, __fsub_rn(y, 2.0f));
    hi += __float_as_uint(y) - 0x40000000u;
    lo += __float_as_uint(__fadd_rz(rest, 0x1p-21f)) - 0x35000000u;
}
__device__ __forceinline__ unsigned long long join(uint32_t hi, uint32_t lo) {      // (of up to 512 weights)
    return (static_cast<unsigned long long>(hi) << 22) + lo;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4) accept_kernel(const AcceptArgs a) {
    __shared__ unsigned long long warp_total[kWarps];
    __shared__ unsigned long long cta_total[2][kCluster];   // every CTA's total, one for each pass
    __shared__ unsigned long long batch_sum[kMaxBatches][kThreads];
    __shared__ int s_kept;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / kCluster;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    auto started = cluster.barrier_arrive();        // (waited for before the first write into another CTA)
    grid_dependency_wait();
    launch_dependents();
    const int K = a.max_drafts;
    const int V = static_cast<int>(a.vocab);
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
                    const double q = draft ? static_cast<double>(to_f32(draft[static_cast<int64_t>(i) * V + x])) : 1.0;
                    keep = static_cast<double>(__ldcg(uniform + i)) * q < static_cast<double>(to_f32(target[static_cast<int64_t>(i) * V + x]));
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
    // The row is cut at the target row's boundaries of four: its first vector may hold elements before it.  The
    // draft's row may stand otherwise there (by qoff): a lane then joins its vector with the next lane's.
    auto offset = [](const T* row) {                // elements past a boundary of four
        return static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
    };
    const int poff = offset(prow), qoff = qrow ? (offset(qrow) - poff) & 3 : 0;
    // a warp's piece of the row: whole batches
    const int batches = (V + poff + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128);
    const int first = (rank * kWarps + warp) * batches * kBatch * 128 - poff;

    float w[kBatch][4];
    auto load = [&](int batch, bool residual) {     // this lane's weights of a batch
        constexpr int W = Four<T>::kWords;
        const int i0 = first + batch * kBatch * 128;             // (warp-uniform, as the branches below)
        const int i = i0 + 4 * lane;
        const bool sub = residual && qrow != nullptr;
        if (i0 >= qoff && i0 + kBatch * 128 + (qoff ? 4 : 0) <= V) {
            // every load before the first use: a branch between them would wait for each in turn
            uint32_t p[kBatch][W], q[kBatch][W];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Four<T>::load(p[k], prow + i + 128 * k);
            if (sub) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k) Four<T>::load(q[k], qrow + i + 128 * k - qoff);
                if (qoff != 0) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        uint32_t last[W] = {}, next[W];
                        if (lane == 31) Four<T>::load(last, qrow + i + 128 * k - qoff + 4);
#pragma unroll
                        for (int e = 0; e < W; ++e) {
                            next[e] = __shfl_down_sync(0xffffffffu, q[k][e], 1);
                            if (lane == 31) next[e] = last[e];
                        }
                        Four<T>::shift(q[k], next, qoff);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float y[4];
                Four<T>::unpack(p[k], w[k]);
                if (sub) Four<T>::unpack(q[k], y);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k][e] = __saturatef(sub ? w[k][e] - y[e] : w[k][e]);
            }
        } else {                                    // a batch at the row's ends
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = i + 128 * k + e;
                    w[k][e] = 0.0f;
                    if (at >= 0 && at < V) {
                        const float x = to_f32(prow[at]);
                        w[k][e] = __saturatef(sub ? x - to_f32(qrow[at]) : x);
                    }
                }
        }
        if (residual && out_x >= 0) {
            const int gone = static_cast<int>(min(out_x, static_cast<int64_t>(V))) - i;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k][e] = gone == 128 * k + e ? 0.0f : w[k][e];
        }
    };

    cluster.barrier_wait(std::move(started));
    for (int pass = 0; pass < 2; ++pass) {
        const bool residual = pass == 0;
        unsigned long long mine = 0;
#pragma unroll 1
        for (int batch = 0; batch < batches; ++batch) {
            uint32_t hi = 0, lo = 0;
            if (first + batch * kBatch * 128 < V) {
                load(batch, residual);
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) add_units(w[k][e], hi, lo);
            }
            const unsigned long long sum = join(hi, lo);
            batch_sum[batch][t] = sum;
            mine += sum;
        }
        mine = warp_sum(mine);
        if (lane == 0) warp_total[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long sum = warp_sum(lane < kWarps ? warp_total[lane] : 0ull);
            if (lane < kCluster) *cluster.map_shared_rank(&cta_total[pass][rank], lane) = sum;
        }
        cluster.sync();
        unsigned long long total = 0, before = 0;   // of the row; of what stands before this warp's piece
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const unsigned long long x = cta_total[pass][c];
            before += c < rank ? x : 0ull;
            total += x;
        }
        if (total == 0) {
            if (pass == 0) continue;                // nothing left of the row: draw from the target's itself
            if (rank == 0 && t == 0) a.tokens[static_cast<int64_t>(b) * (K + 1) + kept] = -1;
            break;
        }
        const double z = (u > 0.0f ? static_cast<double>(u) : 0.0) * static_cast<double>(total);
        const unsigned long long mark = min(__double2ull_rz(z), total - 1);
        for (int v = 0; v < warp; ++v) before += warp_total[v];
        if (mark < before || mark >= before + mine) break;       // another warp's
        // the batch that holds the mark: four batches' sums at a time, side by side
        int batch = 0;
        for (int b0 = 0; b0 < batches; b0 += 4) {
            unsigned long long sum[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = b0 + e < batches ? batch_sum[b0 + e][t] : 0ull;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = warp_sum(sum[e]);
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (here) continue;
                batch = b0 + e;
                here = mark < before + sum[e];
                if (!here) before += sum[e];
            }
            if (here) break;
        }
        load(batch, residual);
        unsigned long long own[kBatch], inc[kBatch];              // a lane's four weights, and up to and with them
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) add_units(w[k][e], hi, lo);
            own[k] = inc[k] = join(hi, lo);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, inc[k], o);
                if (lane >= o) inc[k] += y;
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            unsigned long long at = before + inc[k] - own[k];     // before this lane's four
            if (mark >= at && mark < at + own[k]) {
                int e = 0;
#pragma unroll
                for (int f = 0; f < 3; ++f) {
                    uint32_t hi = 0, lo = 0;
                    add_units(w[k][f], hi, lo);
                    at += join(hi, lo);
                    e += mark >= at;
                }
                a.tokens[static_cast<int64_t>(b) * (K + 1) + kept] = first + (batch * kBatch + k) * 128 + 4 * lane + e;
            }
            before += __shfl_sync(0xffffffffu, inc[k], 31);
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
