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
// One cluster of 8 CTAs a sequence, as there (one CTA over small vocabularies): a
// row is cut into a piece a warp; the CTAs' totals go round through distributed
// shared memory, and with them, for each child of the node, the units before its
// token: whether the walk goes on to a child is then known in every CTA.  Only the
// walk's last token is searched for, by the warp that holds the mark, which reads
// its batch of 512 weights again.
// Rows depend on one another: bound by latency, a row after another.  64 trees of
// 16 over 128000 float32 tokens: 26.7 us, of which the longest path's five or six
// rows take 4 us each (1.8 us of loads, the rest the totals, their exchange and the
// decision).  One batch in flight a thread instead of four took 35 us, a search after
// every row 30; an asynchronous ring of eleven vectors, waited for one by one, 46; a
// child's row prefetched in hope 28 to 30.  One tree over 32000 float16 tokens: 6.6 us.
// Rows off their boundary of four are a little slower, the first and last batch being
// read weight by weight (128001 float32 tokens: 29 us).  The children of a node whose
// tokens lie in one warp's piece are added up one after another, which shows where wide
// trees meet small vocabularies: 32 roots of 63 children (bfloat16) take 11.5 us at
// 128000 tokens, 9.8 at 32000, 16 at 8000 and 39 at 129, of one child 7.3, 6.1, 4.6, 4.5.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
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

// Rows up to so long are one CTA's, longer ones a cluster's (32 trees of 16, bfloat16, one CTA / eight: 12.3 / 14.3 us at 8000
// tokens, 15.4 / 15.6 at 16000, 20.8 / 15.8 at 32000; 14.9 / 20.8 at 1000).
constexpr int kSmallVocab = 8192;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;                           // groups of 128 weights whose loads are in flight together
// Batches of every warp that so many weights fill, over a cluster of CTAs.
__host__ __device__ constexpr int batches_of(int weights, int cluster) {
    return (weights + cluster * kWarps * kBatch * 128 - 1) / (cluster * kWarps * kBatch * 128);
}
// Batches of a warp at most, and of them those that come by way of shared memory (one CTA's rows have no fourth batch).
__host__ __device__ constexpr int max_batches(int cluster) {
    return batches_of((cluster == 1 ? kSmallVocab : PKV_ACCEPT_MAX_VOCAB) + 3, cluster);
}
__host__ __device__ constexpr int late_batches(int cluster) { return max_batches(cluster) >= 4 ? 2 : 0; }
constexpr int kNodes = PKV_TREE_MAX_NODES;
static_assert(kNodes == 64, "a warp looks the children up two nodes a lane");

// Four weights of a row into shared memory, asynchronously.
template <int BYTES>
__device__ __forceinline__ void copy_vector(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16) cp_async_16(dst, src);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// The units of a warp's weights (up to 16 a lane: each half's sum stays below 2^31).
__device__ __forceinline__ unsigned long long warp_units(uint32_t hi, uint32_t lo) {
    return join(__reduce_add_sync(0xffffffffu, hi), __reduce_add_sync(0xffffffffu, lo));
}

template <typename T, int kCluster>
__global__ void __launch_bounds__(kThreads, 4) accept_tree_kernel(const AcceptTreeArgs a) {
    constexpr int kMaxBatches = max_batches(kCluster);
    static_assert(kMaxBatches <= 32, "a batch a lane");
    __shared__ unsigned long long warp_total[kWarps];
    // (two of each, for the rows in turn: a CTA may still read a row's when another writes the next one's)
    __shared__ unsigned long long s_total[2][kCluster];      // every CTA's total of the row
    __shared__ unsigned long long s_before[2][kNodes];       // of a child's token: the units before it in its CTA's piece,
    __shared__ unsigned long long s_units[2][kNodes];        // and its own
    __shared__ unsigned long long batch_total[kWarps][kMaxBatches];
    struct alignas(4 * sizeof(T)) Vector {
        uint32_t w[Four<T>::kWords];
    };
    // a thread's own places: the vectors of two batches, and of a child's
    extern __shared__ __align__(16) uint8_t dynamic[];
    Vector* later = reinterpret_cast<Vector*>(dynamic);
    Vector* kid_batch = later + late_batches(kCluster) * kBatch * kThreads;
    __shared__ int s_parent[kNodes];
    __shared__ int s_draft[kNodes];
    __shared__ int s_owner[kNodes];                           // the warp of the cluster whose piece of the parent's row holds it
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = kCluster == 1 ? 0 : static_cast<int>(cluster.block_rank());
    auto sync = [&] {
        if constexpr (kCluster == 1) __syncthreads();
        else cluster.sync();
    };
    auto put = [&](unsigned long long* at, unsigned long long x) {            // lane r: into CTA r's shared memory
        if constexpr (kCluster == 1) {
            if (lane == 0) *at = x;
        } else {
            if (lane < kCluster) *cluster.map_shared_rank(at, lane) = x;
        }
    };
    const int b = blockIdx.x / kCluster;
    auto started = cluster.barrier_arrive();        // (waited for before the first write into another CTA)
    grid_dependency_wait();
    launch_dependents();
    const int V = static_cast<int>(a.vocab);
    const int W = a.width;
    const int first = __ldcg(a.query_starts + b), end = __ldcg(a.query_starts + b + 1);
    const bool valid = first >= 0 && end >= first && end <= a.num_tokens && end - first <= kNodes;
    const int n = valid ? end - first : 0;
    // the rows are cut at their boundaries of four: a row's first vector may hold elements before it
    auto row_of = [&](int r) { return static_cast<const T*>(a.target_probs) + static_cast<int64_t>(r) * V; };
    auto offset_of = [&](int r) { return static_cast<int>((reinterpret_cast<uintptr_t>(row_of(r)) / sizeof(T)) & 3); };
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
        int owner = -1;
        if (parent >= 0 && token >= 0) {
            const int off = offset_of(first + parent);
            owner = (token + off) / (batches_of(V + off, kCluster) * kBatch * 128);
        }
        s_parent[t] = parent;
        s_draft[t] = token;
        s_owner[t] = owner;
    }
    if (!valid && rank == 0 && t == 0) raise_error(a.err, kErrBounds);
    __syncthreads();
    int64_t* tokens = a.tokens + static_cast<int64_t>(b) * W;
    int32_t* path = a.path + static_cast<int64_t>(b) * W;
    cluster.barrier_wait(std::move(started));

    int node = 0, steps = 0;                        // (the same in every thread of the cluster)
    for (; steps < W && n > 0; ++steps) {
        if (rank == 0 && t == 0) path[steps] = node;
        const T* row = row_of(first + node);
        const float u = __ldcg(a.uniform + first + node);
        const int off = offset_of(first + node);
        const int batches = batches_of(V + off, kCluster);
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
            return warp_units(hi, lo);
        };
        auto units_at_ends = [&](int batch) {
            uint32_t hi = 0, lo = 0;
            if (piece + batch * kBatch * 128 < V) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) add_units(at_ends(batch, k, e), hi, lo);
            }
            return warp_units(hi, lo);
        };

        // The third and fourth batch come by way of shared memory, so that four are in flight (128000 float32 tokens: all),
        // where the first four are whole: the pass below then always takes them up.
        const bool more = late_batches(kCluster) && batches >= 4 && inside(0) && inside(3);
        if (more) {
#pragma unroll
            for (int k = 0; k < 2 * kBatch; ++k)
                copy_vector<4 * sizeof(T)>(smem_u32(later + k * kThreads + t), mine_at + (2 * kBatch + k) * 128);
            cp_async_commit();
        }
        // The node's children.  Whether the mark falls on the token of one is known as soon as the totals are, if the units
        // before that token are, which its warp adds up.  So a row whose token a child drafted needs no search.  Lane l looks
        // after nodes l and 32 + l.
        int owner[2];
        unsigned here[2];                           // the children whose token lies in this warp's piece
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            owner[h] = s_parent[32 * h + lane] == node ? s_owner[32 * h + lane] : -1;
            here[h] = __ballot_sync(0xffffffffu, owner[h] == rank * kWarps + warp);
        }
        // the batch of the first of them is fetched beside the pass
        const int ahead = here[0] ? __ffs(here[0]) - 1 : here[1] ? 31 + __ffs(here[1]) : -1;
        const uint32_t saved = smem_u32(kid_batch) + threadIdx.x * sizeof(kid_batch[0]);
        if (ahead >= 0) {
            const int kb = (s_draft[ahead] - piece) / (kBatch * 128);
            if (inside(kb)) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    copy_vector<4 * sizeof(T)>(saved + k * kThreads * static_cast<uint32_t>(sizeof(kid_batch[0])), mine_at + (kb * kBatch + k) * 128);
            }
            cp_async_commit();
        }
        // ---- the row's total, two batches in flight and two on their way: a sequence whose neighbours are through has its
        // SMs to itself, and what its eight warps a CTA have in flight sets its pace
        unsigned long long mine = 0;
        const int head = piece < 0;                 // (a row off its boundary starts inside a batch, which comes last)
        int batch = head;
#pragma unroll 1
        for (; batch + 2 <= batches && inside(batch) && inside(batch + 1); batch += 2) {
            uint32_t p[2][kBatch][kWords];
            load(batch, p[0]);
            load(batch + 1, p[1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned long long sum = units_of(p[i]);
                if (lane == 0) batch_total[warp][batch + i] = sum;
                mine += sum;
            }
            if (batch == 0 && more) {
                cp_async_wait_all();
                batch = 2;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t hi = 0, lo = 0;
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const Vector v = later[(i * kBatch + k) * kThreads + t];
                        float w[4];
                        Four<T>::unpack(v.w, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) add_units(__saturatef(w[e]), hi, lo);
                    }
                    const unsigned long long sum = warp_units(hi, lo);
                    if (lane == 0) batch_total[warp][batch + i] = sum;
                    mine += sum;
                }
            }
        }
#pragma unroll 1
        for (; batch < batches + head; ++batch) {
            const int i = batch < batches ? batch : 0;
            unsigned long long sum;
            if (inside(i)) {
                uint32_t p[kBatch][kWords];
                load(i, p);
                sum = units_of(p);
            } else {
                sum = units_at_ends(i);
            }
            if (lane == 0) batch_total[warp][i] = sum;
            mine += sum;
        }
        if (ahead >= 0) cp_async_wait_all();
        __syncwarp();
#pragma unroll 1
        for (unsigned long long m = static_cast<unsigned long long>(here[1]) << 32 | here[0]; m; m &= m - 1) {
            const int c = __ffsll(m) - 1, kb = (s_draft[c] - piece) / (kBatch * 128);
            const int at = s_draft[c] - piece - kb * kBatch * 128;            // in its batch
            uint32_t hi = 0, lo = 0;
            float x = 0.0f;                         // the token's own weight, in its lane
#pragma unroll 1
            for (int k = 0; k < kBatch; ++k) {
                float w[4];
                if (c == ahead && inside(kb)) {
                    const Vector v = kid_batch[k * kThreads + t];
                    Four<T>::unpack(v.w, w);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = at_ends(kb, k, e);
                }
                const int i = at - k * 128 - 4 * lane;            // this lane's weights before it: i of these four
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    add_units(e < i ? __saturatef(w[e]) : 0.0f, hi, lo);
                    x = e == i ? __saturatef(w[e]) : x;
                }
            }
            unsigned long long before = warp_units(hi, lo);
            hi = lo = 0;
            add_units(x, hi, lo);
            const unsigned long long own = warp_units(hi, lo);
            for (int i = 0; i < kb; ++i) before += batch_total[warp][i];
            if (lane == 0) {
                s_before[steps & 1][c] = before;
                s_units[steps & 1][c] = own;
            }
        }
        if (lane == 0) warp_total[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const unsigned long long sum = warp_sum(lane < kWarps ? warp_total[lane] : 0ull);
            put(&s_total[steps & 1][rank], sum);
        }
#pragma unroll 1
        for (unsigned long long m = static_cast<unsigned long long>(here[1]) << 32 | here[0]; m; m &= m - 1) {
            const int c = __ffsll(m) - 1;
            unsigned long long before = s_before[steps & 1][c];
            const unsigned long long own = s_units[steps & 1][c];
            for (int v = 0; v < warp; ++v) before += warp_total[v];
            __syncwarp();
            put(&s_before[steps & 1][c], before);
            put(&s_units[steps & 1][c], own);
        }
        sync();
        unsigned long long total = 0;               // of the row
        unsigned long long before = 0, kid[2] = {0, 0};      // of what stands before this CTA's piece; before a lane's children's
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const unsigned long long x = s_total[steps & 1][c];
            total += x;
            before += c < rank ? x : 0ull;
#pragma unroll
            for (int h = 0; h < 2; ++h) kid[h] += c < owner[h] / kWarps ? x : 0ull;
        }
        if (total == 0) {                           // nothing to draw from
            if (rank == 0 && t == 0) tokens[steps] = -1;
            break;
        }
        const double z = (u > 0.0f ? static_cast<double>(u) : 0.0) * static_cast<double>(total);
        const unsigned long long mark = min(__double2ull_rz(z), total - 1);
        unsigned holds[2];                          // the children whose token holds the mark: the first is gone to
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bool on = owner[h] >= 0;
            if (on) {
                const unsigned long long from = kid[h] + s_before[steps & 1][32 * h + lane];
                on = mark >= from && mark < from + s_units[steps & 1][32 * h + lane];
            }
            holds[h] = __ballot_sync(0xffffffffu, on);
        }
        const int next = holds[0] ? __ffs(holds[0]) - 1 : holds[1] ? 31 + __ffs(holds[1]) : -1;
        if (next >= 0) {
            if (rank == 0 && t == 0) tokens[steps] = s_draft[next];
            if (steps + 1 == W) break;
            node = next;
            continue;
        }
        // ---- no child's: the warp whose piece holds the mark finds the token
        for (int v = 0; v < warp; ++v) before += warp_total[v];
        if (mark >= before && mark < before + mine) {
            // the batch that holds the mark
            unsigned long long sums = lane < batches ? batch_total[warp][lane] : 0ull, upto = sums;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            batch = __ffs(__ballot_sync(0xffffffffu, mark < before + upto)) - 1;
            before += __shfl_sync(0xffffffffu, upto - sums, batch);
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
            // its group of 128, then the lane, then the weight
            unsigned long long own = 0;             // this lane's units of the group
            float mine4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            int group = -1;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) add_units(w[k][e], hi, lo);
                const unsigned long long all = warp_units(hi, lo);
                if (group < 0 && mark < before + all) {
                    group = k;
                    own = join(hi, lo);
#pragma unroll
                    for (int e = 0; e < 4; ++e) mine4[e] = w[k][e];
                }
                before += group < 0 ? all : 0ull;
            }
            unsigned long long inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            unsigned long long at = before + inc - own;           // before this lane's four
            if (mark >= at && mark < at + own) {
                int e = 0;
#pragma unroll
                for (int f = 0; f < 3; ++f) {
                    uint32_t hi = 0, lo = 0;
                    add_units(mine4[f], hi, lo);
                    at += join(hi, lo);
                    e += mark >= at;
                }
                tokens[steps] = piece + (batch * kBatch + group) * 128 + 4 * lane + e;
            }
        }
        break;
    }
    // (steps: the place of the last token written; without nodes nothing was)
    if (rank == 0) {
        for (int i = (n > 0 ? steps + 1 : 0) + t; i < W; i += kThreads) tokens[i] = path[i] = -1;
        if (t == 0) a.num_accepted[b] = steps;
    }
    sync();                                         // no CTA leaves while another may still write its shared memory
}

template <typename T, int kCluster>
cudaError_t launch(const AcceptTreeArgs& a, cudaStream_t s) {
    constexpr int kShared = (late_batches(kCluster) + 1) * kBatch * kThreads * 4 * sizeof(T);
    static std::atomic<uint64_t> ready{0};          // devices on which the kernel may take that much
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        e = cudaFuncSetAttribute(accept_tree_kernel<T, kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs) * kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, accept_tree_kernel<T, kCluster>, a);
}

template <typename T>
cudaError_t launch_by_vocab(const AcceptTreeArgs& a, cudaStream_t s) {
    return a.vocab <= kSmallVocab ? launch<T, 1>(a, s) : launch<T, 8>(a, s);
}

}  // namespace

cudaError_t launch_accept_tree(const AcceptTreeArgs& a, int dtype, cudaStream_t s) {
    if (a.num_seqs <= 0) return cudaSuccess;
    if (dtype == 0) return launch_by_vocab<__half>(a, s);
    if (dtype == 1) return launch_by_vocab<__nv_bfloat16>(a, s);
    return launch_by_vocab<float>(a, s);
}

}  // namespace pkv
