// paged_kv_keep_path: the accepted path's rows of the cache moved to the places
// that a sequence without branches has.
//
// Sequence s's last n_s positions hold a tree's nodes; the path 0 = p_0 < p_1 <
// .. < p_a is kept:  row base + i = row base + p_i,  base = L - n_s, in every
// layer's K and V pool, bit for bit.  The moves overlap (a node's place may be
// another's source), but p_i >= i: a thread that takes its 16-byte column of the
// moves in rising order, a run of loads before the run's stores, reads no row
// that an earlier store has overwritten, and no other thread touches the column.
//
// Bound by latency: lengths, path and table are three dependent reads before the
// first row.  A CTA takes one sequence and a few pools, two at a time; with a CTA
// a pool those reads were made 4096 times in 2.7 waves and 32 layers of 64
// sequences, 5 rows each (84 MB), took 20.8 us instead of 16.8 (12.4 at the copy
// rate; 128 threads 18.3, one pool at a time 19.2).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/pkv.h"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 64;
constexpr int kMoves = 8;                           // rows of a thread in flight together,
constexpr int kAtOnce = 2;                          // in so many pools
constexpr int kCtas = 152 * 12;                     // of the grid
constexpr int kNodes = PKV_TREE_MAX_NODES;

__global__ void __launch_bounds__(kThreads) keep_path_kernel(const __grid_constant__ KeepPathArgs a) {
    __shared__ int64_t s_src[kNodes], s_dst[kNodes];
    grid_dependency_wait();
    launch_dependents();
    const int b = blockIdx.x, t = threadIdx.x;
    const int first = __ldcg(a.query_starts + b), end = __ldcg(a.query_starts + b + 1);
    const int len = __ldcg(a.seq_lens + b), kept = __ldcg(a.num_accepted + b);
    const bool valid = first >= 0 && end >= first && end - first <= kNodes && kept >= 0 && kept < min(a.width, kNodes) &&
                       len >= end - first && len <= static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
    const int n = end - first;
    // moves from the first node that is not in its place on
    int node = 0, prev = -1;
    if (valid && n > 0 && t <= kept) {
        node = __ldcg(a.path + static_cast<int64_t>(b) * a.width + t);
        prev = t > 0 ? __ldcg(a.path + static_cast<int64_t>(b) * a.width + t - 1) : -1;
    }
    const bool listed = valid && n > 0 && t <= kept;
    const bool wrong = !valid || kept >= max(n, 1) || (listed && (node <= prev || node >= n || (t == 0 && node != 0)));
    const bool moved = listed && node != t;
    if (__syncthreads_or(wrong)) {
        if (t == 0 && blockIdx.y == 0) raise_error(a.err, kErrBounds);
        return;
    }
    const int moves = __syncthreads_count(moved);   // (the last `moves` of the path: once off its place, always off)
    if (moves == 0) return;
    const int at = t - (kept + 1 - moves);
    if (moved) {
        const int src = len - n + node, dst = len - n + t;
        const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq;
        const int sb = __ldcg(table + src / a.block_size), db = __ldcg(table + dst / a.block_size);
        const bool in = sb >= 0 && sb < a.num_blocks && db >= 0 && db < a.num_blocks;
        if (!in && blockIdx.y == 0) raise_error(a.err, kErrBounds);
        s_src[at] = in ? static_cast<int64_t>(sb) * a.block_size + src % a.block_size : -1;
        s_dst[at] = in ? static_cast<int64_t>(db) * a.block_size + dst % a.block_size : -1;
    }
    __syncthreads();
    // every (pool, column) of the CTA, kAtOnce at a time
    const int pools = 2 * a.num_layers, y = gridDim.y;
    const int wide = (a.row_vecs + kThreads - 1) / kThreads;                  // columns of a thread in a pool
    const int all = (pools - static_cast<int>(blockIdx.y) + y - 1) / y * wide;
    for (int k0 = 0; k0 < all; k0 += kAtOnce) {
        uint4* column[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int p = (k0 + k) / wide, c = (k0 + k) % wide * kThreads + t;
            column[k] = k0 + k < all && c < a.row_vecs ? a.pools[blockIdx.y + p * y] + c : nullptr;
        }
        for (int m0 = 0; m0 < moves; m0 += kMoves) {
            uint4 x[kAtOnce][kMoves];
#pragma unroll
            for (int i = 0; i < kMoves; ++i) {
                const int64_t src = m0 + i < moves ? s_src[m0 + i] : -1;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (src >= 0 && column[k]) x[k][i] = __ldcg(column[k] + src * a.row_vecs);
            }
#pragma unroll
            for (int i = 0; i < kMoves; ++i) {
                const int64_t dst = m0 + i < moves ? s_dst[m0 + i] : -1;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    if (dst >= 0 && column[k]) column[k][dst * a.row_vecs] = x[k][i];
            }
        }
    }
}

}  // namespace

cudaError_t launch_keep_path(const KeepPathArgs& a, cudaStream_t s) {
    if (a.num_seqs <= 0 || a.num_layers <= 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_seqs),
                       static_cast<unsigned>(std::min(2 * a.num_layers, (kCtas - 1) / a.num_seqs + 1)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, keep_path_kernel, a);
}

}  // namespace pkv
