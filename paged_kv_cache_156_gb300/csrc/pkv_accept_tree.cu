// speculative_accept_tree: the path through a tree of drafted tokens that
// follows the target's distribution, and the token after it.
//
// The walk starts at the root (the sequence's last token, of whose successors
// row 0 holds the target's probabilities).  At a node a token y is drawn from
// the node's own row with the node's own random number; the walk goes on to the
// child that drafted y, and where there is none y is the sequence's new token.
// So every token of the path is a draw from the target, whatever was drafted.
//
// The draw is the one of pkv_accept.cu: weights in whole units of 2^-44, the
// first token whose inclusive sum exceeds floor(u T), exact whatever the order.
//
// One cluster of 8 CTAs a sequence, as there: a row is cut into a piece a warp;
// the CTAs' totals go round through distributed shared memory; the warp that
// holds the mark reads its batch of 512 weights again, finds the token and hands
// it to every CTA, each of which looks the child up in its own copy of the tree.
// Rows depend on one another: bound by latency, a row after another.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_draw.cuh"
#include "pkv_internal.h"

namespace cg = cooperative_groups;

namespace pkv {
namespace {

using draw::add_units;
using draw::Four;
using draw::join;
using draw::to_f32;
using draw::warp_sum;

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;                           // groups of 128 weights whose loads are in flight together
constexpr int kMaxBatches = (PKV_ACCEPT_MAX_VOCAB + 3 + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128);
constexpr int kNodes = PKV_TREE_MAX_NODES;
static_assert(kNodes == 64, "a warp looks a child up two nodes a lane");

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4) accept_tree_kernel(const AcceptTreeArgs a) {
    __shared__ unsigned long long warp_total[kWarps];
    __shared__ unsigned long long cta_total[kCluster];       // every CTA's total of the row
    __shared__ unsigned long long batch_sum[kMaxBatches][kThreads];
    __shared__ int s_parent[kNodes];
    __shared__ int s_draft[kNodes];
    __shared__ int s_drawn;                                   // the row's token, from the CTA that found it
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int b = blockIdx.x / kCluster;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    auto started = cluster.barrier_arrive();        // (waited for before the first write into another CTA)
    grid_dependency_wait();
    launch_dependents();
    const int V = static_cast<int>(a.vocab);
    const int W = a.width;
    const int first = __ldcg(a.query_starts + b), end = __ldcg(a.query_starts + b + 1);
    const bool valid = first >= 0 && end >= first && end <= a.num_tokens && end - first <= kNodes;
    const int n = valid ? end - first : 0;
    if (t < kNodes) {
        int parent = -1, token = -1;
        if (t > 0 && t < n) {
            parent = __ldcg(a.parents + first + t);
            const int64_t x = __ldcg(a.draft_tokens + first + t);
            token = x >= 0 && x < V ? static_cast<int>(x) : -1;
            if (parent < 0 || parent >= t) {        // no node before it: nobody's child
                if (rank == 0) raise_error(a.err, kErrBounds);
                parent = -1;
            }
        }
        s_parent[t] = parent;
        s_draft[t] = token;
    }
    if (!valid && rank == 0 && t == 0) raise_error(a.err, kErrBounds);
    __syncthreads();
    int64_t* tokens = a.tokens + static_cast<int64_t>(b) * W;
    int32_t* path = a.path + static_cast<int64_t>(b) * W;
    cluster.barrier_wait(std::move(started));

    int node = 0, steps = 0;                        // (the same in every thread of the cluster)
    for (; steps < W && n > 0; ++steps) {
        if (rank == 0 && t == 0) path[steps] = node;
        const T* row = static_cast<const T*>(a.target_probs) + static_cast<int64_t>(first + node) * V;
        const float u = __ldcg(a.uniform + first + node);
        // the row is cut at its boundaries of four: its first vector may hold elements before it
        const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) / sizeof(T)) & 3);
        const int batches = (V + off + kCluster * kWarps * kBatch * 128 - 1) / (kCluster * kWarps * kBatch * 128);
        const int piece = (rank * kWarps + warp) * batches * kBatch * 128 - off;

        constexpr int kWords = Four<T>::kWords;
        const T* mine_at = row + piece + 4 * lane;
        // (warp-uniform: a batch wholly in the row; one of the row's ends is read weight by weight)
        auto inside = [&](int batch) { return piece + batch * kBatch * 128 >= 0 && piece + (batch + 1) * kBatch * 128 <= V; };
        auto load = [&](int batch, uint32_t (&p)[kBatch][kWords]) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) Four<T>::load(p[k], mine_at + (batch * kBatch + k) * 128);
        };
        auto at_ends = [&](int batch, int k, int e) {
            const int at = piece + (batch * kBatch + k) * 128 + 4 * lane + e;
            return at >= 0 && at < V ? __saturatef(to_f32(row[at])) : 0.0f;
        };
        auto units_of = [&](const uint32_t (&p)[kBatch][kWords]) {            // of a batch's 16 weights
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float w[4];
                Four<T>::unpack(p[k], w);
#pragma unroll
                for (int e = 0; e < 4; ++e) add_units(__saturatef(w[e]), hi, lo);
            }
            return join(hi, lo);
        };
        auto units_at_ends = [&](int batch) {
            uint32_t hi = 0, lo = 0;
            if (piece + batch * kBatch * 128 < V) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) add_units(at_ends(batch, k, e), hi, lo);
            }
            return join(hi, lo);
        };

        // ---- the row's total, two batches in flight: a sequence whose neighbours are through has its SMs to itself, and
        // what its eight warps a CTA have in flight sets its pace
        unsigned long long mine = 0;
        int batch = 0;
#pragma unroll 1
        for (; batch + 2 <= batches && inside(batch) && inside(batch + 1); batch += 2) {
            uint32_t p[2][kBatch][kWords];
            load(batch, p[0]);
            load(batch + 1, p[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned long long sum = units_of(p[i]);
                batch_sum[batch + i][t] = sum;
                mine += sum;
            }
        }
#pragma unroll 1
        for (; batch < batches; ++batch) {
            unsigned long long sum;
            if (inside(batch)) {
                uint32_t p[kBatch][kWords];
                load(batch, p);
                sum = units_of(p);
            } else {
                sum = units_at_ends(batch);
            }
            batch_sum[batch][t] = sum;
            mine += sum;
        }
        mine = warp_sum(mine);
        if (lane == 0) warp_total[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long sum = warp_sum(lane < kWarps ? warp_total[lane] : 0ull);
            if (lane < kCluster) *cluster.map_shared_rank(&cta_total[rank], lane) = sum;
        }
        cluster.sync();
        unsigned long long total = 0, before = 0;   // of the row; of what stands before this warp's piece
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const unsigned long long x = cta_total[c];
            before += c < rank ? x : 0ull;
            total += x;
        }
        int drawn = -1;
        if (total != 0) {
            const double z = (u > 0.0f ? static_cast<double>(u) : 0.0) * static_cast<double>(total);
            const unsigned long long mark = min(__double2ull_rz(z), total - 1);
            for (int v = 0; v < warp; ++v) before += warp_total[v];
            if (mark >= before && mark < before + mine) {
                // the batch that holds the mark: four batches' sums at a time, side by side
                batch = 0;
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
                float w[kBatch][4];
                if (inside(batch)) {
                    uint32_t p[kBatch][kWords];
                    load(batch, p);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        Four<T>::unpack(p[k], w[k]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[k][e] = __saturatef(w[k][e]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[k][e] = at_ends(batch, k, e);
                }
                unsigned long long own[kBatch], inc[kBatch];      // a lane's four weights, and up to and with them
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
                        const int y = piece + (batch * kBatch + k) * 128 + 4 * lane + e;
                        for (int c = 0; c < kCluster; ++c) *cluster.map_shared_rank(&s_drawn, c) = y;
                    }
                    before += __shfl_sync(0xffffffffu, inc[k], 31);
                }
            }
            cluster.sync();
            drawn = s_drawn;
        }
        if (rank == 0 && t == 0) tokens[steps] = drawn;
        // the first child that drafted it
        const unsigned low = __ballot_sync(0xffffffffu, drawn >= 0 && s_parent[lane] == node && s_draft[lane] == drawn);
        const unsigned high = __ballot_sync(0xffffffffu, drawn >= 0 && s_parent[32 + lane] == node && s_draft[32 + lane] == drawn);
        if ((low | high) == 0 || steps + 1 == W) break;
        node = low ? __ffs(low) - 1 : 31 + __ffs(high);
    }
    // (steps: the place of the last token written; without nodes nothing was)
    if (rank == 0) {
        for (int i = (n > 0 ? steps + 1 : 0) + t; i < W; i += kThreads) tokens[i] = path[i] = -1;
        if (t == 0) a.num_accepted[b] = steps;
    }
    cluster.sync();                                 // no CTA leaves while another may still write its shared memory
}

template <typename T>
cudaError_t launch(const AcceptTreeArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, accept_tree_kernel<T>, a);
}

}  // namespace

cudaError_t launch_accept_tree(const AcceptTreeArgs& a, int dtype, cudaStream_t s) {
    if (a.num_seqs <= 0) return cudaSuccess;
    if (dtype == 0) return launch<__half>(a, s);
    if (dtype == 1) return launch<__nv_bfloat16>(a, s);
    return launch<float>(a, s);
}

}  // namespace pkv
