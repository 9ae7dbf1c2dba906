// What the prefill plan and the prefill kernel share: a sequence's bounds, and its tiles.
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

__device__ __forceinline__ int warp_scan(int v) {            // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

}  // namespace pf
}  // namespace pkv
