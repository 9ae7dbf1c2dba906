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
// warp a contiguous piece of that, so the row is read once; totals go round
// through distributed shared memory.  Every lane keeps its sum of each batch of
// 512 weights in shared memory, so the warp that holds the mark finds the batch
// from there and reads those 512 weights again.  (Weights held in registers
// instead spilled at two CTAs an SM: 36 us for 64 sequences of 128000 tokens.)
// Bound by latency at a few sequences (dependent loads: draft token, its
// probabilities, the row), by HBM at many.
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
constexpr int kMaxBatches = (PKV_ACCEPT_MAX_VOCAB + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128);

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (std::is_same<T, float>::value) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}

// Four consecutive probabilities from element i of a row (0 past its end), `off` elements past a vector's
// boundary (the row's base and so every fourth element are): the two aligned vectors that hold them, shifted
// together, where both lie inside the row; element by element at its ends.
template <typename T>
__device__ __forceinline__ void load4(const T* row, int i, int vocab, int off, float (&x)[4]) {
    const int at = i - off;
    if (off == 0 ? i + 4 <= vocab : at >= 0 && at + 8 <= vocab) {
        if constexpr (std::is_same<T, float>::value) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(row + at));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            if (off != 0) {
                const float4 n = __ldcs(reinterpret_cast<const float4*>(row + at) + 1);
                x[0] = off == 1 ? v.y : off == 2 ? v.z : v.w;
                x[1] = off == 1 ? v.z : off == 2 ? v.w : n.x;
                x[2] = off == 1 ? v.w : off == 2 ? n.x : n.y;
                x[3] = off == 1 ? n.x : off == 2 ? n.y : n.z;
            }
        } else {
            uint2 v = __ldcs(reinterpret_cast<const uint2*>(row + at));
            if (off != 0) {
                const uint2 n = __ldcs(reinterpret_cast<const uint2*>(row + at) + 1);
                const uint32_t a = off >= 2 ? v.y : v.x, b = off >= 2 ? n.x : v.y, c = off >= 2 ? n.y : n.x;
                v = (off & 1) ? make_uint2(__funnelshift_r(a, b, 16), __funnelshift_r(b, c, 16)) : make_uint2(a, b);
            }
            const float2 lo = Mma<T>::unpack(v.x), hi = Mma<T>::unpack(v.y);
            x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e < vocab ? to_f32(row[i + e]) : 0.0f;
    }
}

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
    auto offset = [](const T* row) {                // elements past a boundary of four
        return static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
    };
    const int poff = offset(prow), qoff = qrow ? offset(qrow) : 0;
    // a warp's piece of the row: whole batches
    const int batches = static_cast<int>((V + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128));
    const int first = (rank * kWarps + warp) * batches * kBatch * 128 + 4 * lane;

    float w[kBatch][4];
    auto load = [&](int batch, bool residual) {     // this lane's weights of a batch
        const int i0 = first + batch * kBatch * 128;
        float q[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            load4(prow, i0 + 128 * k, V, poff, w[k]);
            if (residual && qrow) load4(qrow, i0 + 128 * k, V, qoff, q[k]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[k][e] = __saturatef(residual && qrow ? w[k][e] - q[k][e] : w[k][e]);
        if (residual && out_x >= 0) {
            const int gone = static_cast<int>(min(out_x, static_cast<int64_t>(V))) - i0;
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
            if (first - 4 * lane + batch * kBatch * 128 < V) {
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
        int batch = 0;
        for (; batch + 1 < batches; ++batch) {
            const unsigned long long sum = warp_sum(batch_sum[batch][t]);
            if (mark < before + sum) break;
            before += sum;
        }
        load(batch, residual);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            unsigned long long c[4];
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                add_units(w[k][e], hi, lo);
                c[e] = join(hi, lo);
            }
            unsigned long long inc = c[3];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned long long at = before + inc - c[3];   // before this lane's four
            if (mark >= at && mark < at + c[3]) {
                const int e = mark < at + c[0] ? 0 : mark < at + c[1] ? 1 : mark < at + c[2] ? 2 : 3;
                a.tokens[static_cast<int64_t>(b) * (K + 1) + kept] = first + (batch * kBatch + k) * 128 + e;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
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
