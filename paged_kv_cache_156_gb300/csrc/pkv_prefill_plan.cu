// Prefill work plan: one small kernel that turns a ragged batch's lengths into
// the work list of the prefill kernel (pkv_prefill.cu).
//
// A tile is 256 query rows of a sequence (rows are (token, query head of the
// KV head's group) pairs), and its work is the number of 128-position steps
// its last row sees.  Tiles are listed longest first, so that the persistent
// CTAs, which take items round robin, end at about the same time.  When a few
// long tiles would leave SMs idle (a handful of rows over a long cache), every
// tile is cut into parts whose partial softmax states a merge kernel joins
// (pf::choose_part).  The order of equally long items, and which partial slot a
// tile gets, vary from run to run; no result depends on either, since the merge
// sums parts in part order.
//
// A single call over a batch of moderate size does not run this kernel: every
// CTA of the prefill kernel makes the same plan by itself.  This one serves the
// calls that share a plan (a step's layers) and the largest batches.
//
// One CTA: a few bytes per sequence, latency-bound.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv_prefill_common.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBuckets = 32;         // (one a lane of the scan)

using pf::load_seq;
using pf::parts_of;
using pf::Seq;
using pf::tile_steps;
using pf::warp_scan;

constexpr int kCached = 2048;        // tiles whose steps stay in shared memory between the phases

struct Shared {
    int start[kThreads], n[kThreads], len[kThreads];
    int first[kThreads + 1];                                 // first tile of each of this chunk's sequences
    int scan[kWarps];
    int steps[kCached], seq[kCached];
    int wmax[kWarps];
    unsigned long long wsum[kWarps];
    pf::Choice choice;
    int bucket[kBuckets], at[kBuckets];
    int next_slot, next_merge;
};

// (The kernel runs every instruction about once, so it is bound by fetching them: what is used twice is a function,
// and no loop is unrolled.  Inlined and unrolled it was 45 KB and took 7 us.)

// Loads a chunk of sequences and their tile offsets.
__device__ __noinline__ void load_chunk(const PrefillArgs& a, Shared& sh, int base, bool report) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int s = base + t;
    Seq q{0, 0, 0};
    if (s < a.num_seqs) q = load_seq(a, s, report);
    __syncthreads();
    sh.start[t] = q.start;
    sh.n[t] = q.n;
    sh.len[t] = q.len;
    const int mine = pf::tiles_of(q, a.group);
    const int inc = warp_scan(mine);
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    const int w = warp_scan(sh.scan[lane]);                  // (every warp scans the warps' totals)
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    sh.first[t + 1] = inc + (warp > 0 ? before : 0);
    if (t == 0) sh.first[0] = 0;
    __syncthreads();
}

// The chunk's sequence (0 .. 1023) that holds a tile.
__device__ __forceinline__ int find_seq(const Shared& sh, int tile) {
    int lo = 0;
#pragma unroll 1
    for (int w = kThreads / 2; w > 0; w >>= 1)
        if (sh.first[lo + w] <= tile) lo += w;
    return lo;
}

// Tile i of the current chunk: its sequence and steps.
__device__ __noinline__ int tile_of(const PrefillArgs& a, const Shared& sh, int i, int* k) {
    *k = find_seq(sh, i);
    return tile_steps(a, Seq{sh.start[*k], sh.n[*k], sh.len[*k]}, i - sh.first[*k]);
}

__global__ void __launch_bounds__(kThreads) prefill_plan_kernel(const __grid_constant__ PrefillArgs a) {
    __shared__ Shared sh;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    grid_dependency_wait();
    launch_dependents();
    if (t == 0) sh.next_slot = sh.next_merge = 0;
    if (t < kBuckets) sh.bucket[t] = 0;
    const bool one_chunk = a.num_seqs <= kThreads;
    // ---- tiles, their steps' sum and maximum
    int mx = 0;
    long long tiles_all = 0;
    unsigned long long sum = 0;
#pragma unroll 1
    for (int base = 0; base < a.num_seqs; base += kThreads) {
        load_chunk(a, sh, base, true);
        const int tiles = sh.first[kThreads];
        const bool keep = one_chunk && tiles <= kCached;
#pragma unroll 1
        for (int i = t; i < tiles; i += kThreads) {
            int k;
            const int st = tile_of(a, sh, i, &k);
            if (keep) {
                sh.steps[i] = st;
                sh.seq[i] = k;
            }
            mx = max(mx, st);
            sum += st;
        }
        tiles_all += tiles;
    }
    const bool cached = one_chunk && tiles_all <= kCached;
    mx = __reduce_max_sync(0xffffffffu, mx);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
        sh.wmax[warp] = mx;
        sh.wsum[warp] = sum;
    }
    __syncthreads();
    const int maxs = __reduce_max_sync(0xffffffffu, sh.wmax[lane]);
    unsigned long long steps = sh.wsum[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, o);

    // ---- the part length (a batch that the plan would have to reload is not split)
    const int P = cached ? pf::choose_part<kWarps>(a, sh.choice, sh.steps, static_cast<int>(tiles_all), maxs, static_cast<float>(steps))
                         : max(1, maxs);
    const int top = min(P, max(1, maxs));                    // the longest item

    // ---- items by length: count, offsets, write
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int base = 0; base < a.num_seqs; base += kThreads) {
            if (!one_chunk) load_chunk(a, sh, base, false);
            const int tiles = sh.first[kThreads];
#pragma unroll 1
        for (int i = t; i < tiles; i += kThreads) {
                int k;
                const int st = cached ? sh.steps[i] : tile_of(a, sh, i, &k);
                if (cached) k = sh.seq[i];
                const int tile = i - sh.first[k];
                const int parts = parts_of(st, P);
                const int len = pf::part_len(st, parts);            // equal parts
                int slot = 0;
                if (pass == 1 && parts > 1) {
                    slot = atomicAdd(&sh.next_slot, parts);
                    a.merges[atomicAdd(&sh.next_merge, 1)] = make_int4(prefill_split(parts, 0, slot), tile, sh.start[k], sh.n[k]);
                }
#pragma unroll 1
                for (int p = 0; p < parts; ++p) {
                    const int s0 = min(st, p * len), s1 = min(st, s0 + len);
                    const int b = min(kBuckets - 1, (top - (s1 - s0)) * kBuckets / (top + 1));
                    if (pass == 0) {
                        atomicAdd(&sh.bucket[b], 1);
                    } else {
                        const int at = atomicAdd(&sh.at[b], 1);
                        if (at < a.capacity) {
                            a.items[2 * at] = make_int4(base + k, tile, s0, s1);
                            a.items[2 * at + 1] =
                                make_int4(sh.start[k], sh.n[k], sh.len[k], parts > 1 ? prefill_split(parts, p, slot) : 0);
                        }
                    }
                }
            }
        }
        __syncthreads();
        if (pass == 0) {
            if (warp == 0) {
                const int v = sh.bucket[lane], inc = warp_scan(v);
                sh.at[lane] = inc - v;
                if (lane == 31) a.header[0] = min(inc, a.capacity);
            }
        } else if (t == 0) {
            a.header[1] = sh.next_merge;
        }
        __syncthreads();
    }
}

}  // namespace

PrefillWorkspace prefill_workspace_layout(int num_seqs, int64_t num_tokens, int num_heads, int num_kv_heads,
                                          int head_dim, int slots) {
    PrefillWorkspace w{};
    auto pad = [](size_t x) { return (x + 255) / 256 * 256; };
    const int64_t rows = num_tokens * (num_heads / num_kv_heads);
    w.part_rows = static_cast<int>((std::min<int64_t>(kPrefillRows, std::max<int64_t>(rows, 1)) + 31) / 32 * 32);
    // two parts for every CTA over all KV heads, at least 16 a head: what a KV head's split tiles share, and so the most
    // parts of one tile too
    w.part_cap = std::max((2 * slots + num_kv_heads - 1) / num_kv_heads, 16);
    w.capacity = static_cast<int>(rows / kPrefillRows + std::min<int64_t>(num_seqs, rows) + w.part_cap);
    const size_t parts = static_cast<size_t>(num_kv_heads) * w.part_cap;
    w.items = 256;
    w.merges = w.items + pad(static_cast<size_t>(w.capacity) * 32);
    w.ml = w.merges + pad(static_cast<size_t>(w.part_cap) * 8);
    w.o = w.ml + pad(parts * w.part_rows * sizeof(float2));
    w.total = w.o + pad(parts * w.part_rows * head_dim * sizeof(float));
    return w;
}

bool prefill_may_split(int64_t num_tokens, int max_seq_len, int num_heads, int num_kv_heads, int slots) {
    const int64_t tiles = num_tokens * (num_heads / num_kv_heads) / kPrefillRows;       // at least
    return max_seq_len > kPrefillNoSplit * kPrefillStep && tiles * num_kv_heads < 8ll * slots;
}

bool prefill_direct(int num_seqs, int64_t num_tokens, int max_seq_len, int num_heads, int num_kv_heads, int slots) {
    const int64_t rows = num_tokens * (num_heads / num_kv_heads);
    return num_seqs <= 128 && (rows / kPrefillRows + std::min<int64_t>(num_seqs, rows)) * num_kv_heads <= slots &&
           !prefill_may_split(num_tokens, max_seq_len, num_heads, num_kv_heads, slots);
}

bool prefill_local(int num_seqs, int64_t num_tokens, int num_heads, int num_kv_heads, int slots,
                   const PrefillWorkspace& w) {
    const int64_t rows = num_tokens * (num_heads / num_kv_heads);
    const int64_t tiles = rows / kPrefillRows + std::min<int64_t>(num_seqs, rows);        // at most
    // (an item a lane of the plan warp, 32 rounds)
    return num_seqs <= kPrefillLocal && tiles <= kPrefillLocal && tiles + w.part_cap <= kPrefillLocalItems &&
           (tiles + w.part_cap) * num_kv_heads <= 32ll * slots;
}

cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_plan_kernel, a);
}

}  // namespace pkv
