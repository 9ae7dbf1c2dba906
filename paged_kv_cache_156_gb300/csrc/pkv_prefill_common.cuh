// What the prefill plan and the prefill kernel share: a sequence's bounds, its tiles, and whether and how far tiles are
// split.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace pf {

struct Seq {
    int start, n, len;               // first query row, new tokens (0 where the starts are not a range), positions
};

__device__ __forceinline__ Seq load_seq(const PrefillArgs& a, int s, bool report) {
    Seq q{__ldcg(a.query_starts + s), 0, __ldcg(a.seq_lens + s)};
    const int end = __ldcg(a.query_starts + s + 1);
    if (q.len > a.max_seq_len) {
        if (report) raise_error(a.err, kErrBounds);
        q.len = a.max_seq_len;
    }
    q.len = max(q.len, 0);
    if (q.start < 0 || end < q.start || end > a.num_tokens) {
        if (report) raise_error(a.err, kErrBounds);
    } else {
        q.n = end - q.start;
    }
    return q;
}

__device__ __forceinline__ int tiles_of(const Seq& q, int group) { return (q.n * group + kPrefillRows - 1) / kPrefillRows; }

// (An integer division by a number the compiler does not know is some thirty instructions, and the planning code runs
// each of its own about once: it is bound by fetching them.)
__device__ __forceinline__ int div(int n, FastDiv d) {       // 0 <= n < 2^31
    return static_cast<int>((__umulhi(d.mul, static_cast<unsigned>(n)) + static_cast<unsigned>(n)) >> d.shift);
}

// Steps the last row of a tile sees.
__device__ __forceinline__ int tile_steps(const PrefillArgs& a, const Seq& q, int tile) {
    const int rows = q.n * a.group;
    const int last = min(rows, (tile + 1) * kPrefillRows) - 1;
    const int lim = min(q.len, max(0, q.len - q.n + div(last, a.by_group) + 1));
    return (lim + kPrefillStep - 1) / kPrefillStep;
}

__device__ __forceinline__ int warp_scan(int v) {            // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// ceil(steps / P), at least 1, where that is a small number (a tile has up to kPrefillMaxParts parts): the quotient in
// single precision is then off by one at most, which the remainder shows.
__device__ __forceinline__ int parts_of(int steps, int P) {
    const int n = steps + P - 1;
    int q = __float2int_rz(__fdividef(static_cast<float>(n), static_cast<float>(P)));
    const int r = n - q * P;
    q += (r >= P) - (r < 0);
    return max(1, q);
}
// Steps of each of a tile's parts.
__device__ __forceinline__ int part_len(int steps, int parts) { return parts > 1 ? (steps + parts - 1) / parts : steps; }

constexpr int kCand = 32;            // (a lane each)
// Parts that candidate c cuts the longest tile into: 1 .. 20, then ever wider apart up to kPrefillMaxParts.
__device__ __forceinline__ int cand_parts(int c) {
    return c < 20 ? c + 1 : 20 + ((c - 19) * (c - 19) * (kPrefillMaxParts - 20) + 72) / 144;
}
static_assert((kCand - 20) * (kCand - 20) == 144, "the last candidate: kPrefillMaxParts");
constexpr int kItemCost = 2;         // steps' worth of an item's query load and epilogue
constexpr int kSplitCost = 3;        // and of a part's partial output and its share of the merge

struct Choice {
    int items[kCand], parts[kCand];  // per candidate: all items; parts of split tiles
};

// The part length P of a batch whose tiles' steps are in `steps`, by a block of WARPS warps: the longest tile's
// length (no split), or the candidate with the smallest estimated end,
//
//     (steps + kItemCost * items + kSplitCost * parts) * KV heads / SMs
//         + half the largest item             when the items outnumber the SMs,
//     the largest item                        otherwise
//
// (the first line is the average load plus the expected overhang of a longest-first schedule).  Tiles are not split
// when there are many for every SM (8 and more: one much longer than the rest then keeps its KV heads' CTAs after the
// others are done), nor when the longest is well below what every CTA has to do anyway.
template <int WARPS>
__device__ __forceinline__ int choose_part(const PrefillArgs& a, Choice& ch, const int* steps, int tiles, int maxs, float sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float nh = static_cast<float>(a.num_kv_heads), slots = static_cast<float>(a.slots);
    const float each = (sum + kItemCost * static_cast<float>(tiles)) * nh / slots;
    if (!a.may_split || maxs <= kPrefillMinPart || tiles * nh >= 8.0f * slots || maxs + kItemCost <= 0.6f * each)
        return max(1, maxs);
#pragma unroll 1
    for (int c = warp; c < kCand; c += WARPS) {
        const int k = cand_parts(c), P = max(kPrefillMinPart, (maxs + k - 1) / k);
        int all = 0, split = 0;
#pragma unroll 1
        for (int i = lane; i < tiles; i += 32) {
            const int parts = parts_of(steps[i], P);
            all += parts;
            split += parts > 1 ? parts : 0;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        split = __reduce_add_sync(0xffffffffu, split);
        if (lane == 0) {
            ch.items[c] = all;
            ch.parts[c] = split;
        }
    }
    __syncthreads();
    // (every warp chooses for itself)
    unsigned best = 0xffffffffu;
    int P = max(1, maxs);
    {
        const int k = cand_parts(lane);
        if (lane > 0) P = max(kPrefillMinPart, (maxs + k - 1) / k);
        const int items = ch.items[lane], parts = ch.parts[lane];
        const float top = static_cast<float>(min(P, maxs) + kItemCost + (parts > 0 ? kSplitCost : 0));
        const float load = (sum + kItemCost * static_cast<float>(items) + kSplitCost * static_cast<float>(parts)) * nh / slots;
        const float est = items * nh <= slots ? top : fmaxf(top, load + 0.5f * top);
        // (positive floats order as their bits)
        if (parts <= a.part_cap && tiles + parts <= a.capacity && (maxs + P - 1) / P <= kPrefillMaxParts) best = __float_as_uint(est);
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, best);
    const unsigned m = __ballot_sync(0xffffffffu, best == least);
    const int win = least == 0xffffffffu ? 0 : __ffs(m) - 1;              // ties: fewer parts
    return least == 0xffffffffu ? max(1, maxs) : __shfl_sync(0xffffffffu, P, win);
}

}  // namespace pf
}  // namespace pkv
