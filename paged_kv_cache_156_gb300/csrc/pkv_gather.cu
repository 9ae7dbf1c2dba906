// paged_kv_gather: the cached K/V of a batch read back into dense rows.
//
//     k_out[row_starts[s] + t] = K_t, v_out likewise,  t < seq_lens[s],
//
// K_t being the pool's row itself, or, over an E4M3 pool, each code's value
// times its KV head's scale in fp32, rounded once to the output type.  The
// inverse of the slot writes (pkv_append.cu): what a dense kernel, another
// process or a prefix store takes from the cache.
//
// HBM-bound: every byte is read once and written once.  The grid covers the
// output's rows (the one size the host knows), kRows a CTA; the CTA finds the
// sequence of its first row by counting the starts at or below it (no search
// loop: one load a thread for up to 256 sequences), walks on from there, and
// then moves its rows 16 bytes a lane, every load of a thread issued before its
// stores.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;                            // output rows a CTA
constexpr int kUnroll = 4;                          // 16-byte loads of K and of V in flight a thread

template <typename T>
__device__ __forceinline__ uint4 expand8(uint2 c, float scale) {        // 8 codes -> 8 elements
    uint32_t w[4];
    const uint32_t in[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(in[i]), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        w[i] = Mma<T>::pack(f.x * scale, f.y * scale);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// T: the output's type over an E4M3 pool (KV8); 16-bit rows are moved as they are.
template <typename T, bool KV8>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherArgs a) {
    __shared__ int64_t src_row[kRows];              // the output row's row in the pools (-1: not written)
    grid_dependency_wait();
    launch_dependents();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows;
    const int t = threadIdx.x;
    // ---- the last sequence that starts at or before the first row (the starts do not decrease)
    int mine = 0;
    for (int i = t; i < a.num_seqs; i += kThreads) mine += __ldcg(a.row_starts + i) <= row0 ? 1 : 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    __shared__ int part[kThreads / 32];
    if ((t & 31) == 0) part[t >> 5] = mine;
    __syncthreads();
    if (t < kRows) {
        int s = -1;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += part[w];
        const int64_t row = row0 + t;
        int64_t src = -1;
        s = max(s, 0);
        while (s + 1 < a.num_seqs && __ldcg(a.row_starts + s + 1) <= row) ++s;
        const int start = __ldcg(a.row_starts + s), end = __ldcg(a.row_starts + s + 1), len = __ldcg(a.seq_lens + s);
        if (row < a.num_rows && start >= 0 && start <= row && row < end && row - start < len) {
            const int pos = static_cast<int>(row - start), lb = pos / a.block_size;
            if (lb < a.max_blocks_per_seq) {
                const int pb = __ldcg(a.block_tables + static_cast<int64_t>(s) * a.max_blocks_per_seq + lb);
                if (pb >= 0 && pb < a.num_blocks) src = static_cast<int64_t>(pb) * a.block_size + (pos - lb * a.block_size);
            }
            if (src < 0) raise_error(a.err, kErrBounds);
        }
        src_row[t] = src;
    }
    // the batch's lengths and starts, checked by the first CTA
    if (blockIdx.x == 0)
        for (int i = t; i < a.num_seqs; i += kThreads) {
            const int start = __ldcg(a.row_starts + i), end = __ldcg(a.row_starts + i + 1), len = __ldcg(a.seq_lens + i);
            if (start < 0 || end < start || end > a.num_rows || len > end - start) raise_error(a.err, kErrBounds);
        }
    __syncthreads();

    const int rv = a.row_vecs;                      // output vectors of a row (8 elements each)
    const int total = kRows * rv;
    for (int i0 = t; i0 < total; i0 += kThreads * kUnroll) {
        if constexpr (KV8) {
            uint2 x[kUnroll], y[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads, r = i / rv;
                const int64_t src = i < total ? src_row[r] : -1;
                if (src >= 0) {
                    x[u] = __ldcs(static_cast<const uint2*>(a.key_cache) + src * rv + (i - r * rv));
                    y[u] = __ldcs(static_cast<const uint2*>(a.value_cache) + src * rv + (i - r * rv));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads, r = i / rv;
                if (i >= total || src_row[r] < 0) continue;
                const int h = (i - r * rv) / a.head_vecs;
                a.k_out[row0 * rv + i] = expand8<T>(x[u], __ldcg(a.k_scale + h));
                a.v_out[row0 * rv + i] = expand8<T>(y[u], __ldcg(a.v_scale + h));
            }
        } else {
            uint4 x[kUnroll], y[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads, r = i / rv;
                const int64_t src = i < total ? src_row[r] : -1;
                if (src >= 0) {
                    x[u] = __ldcs(static_cast<const uint4*>(a.key_cache) + src * rv + (i - r * rv));
                    y[u] = __ldcs(static_cast<const uint4*>(a.value_cache) + src * rv + (i - r * rv));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int i = i0 + u * kThreads, r = i / rv;
                if (i >= total || src_row[r] < 0) continue;
                a.k_out[row0 * rv + i] = x[u];
                a.v_out[row0 * rv + i] = y[u];
            }
        }
    }
}

template <typename T, bool KV8>
cudaError_t launch(const GatherArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.num_rows + kRows - 1) / kRows));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_kernel<T, KV8>, a);
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t s) {
    if (a.num_rows <= 0 || a.num_seqs <= 0) return cudaSuccess;
    if (!a.k_scale) return launch<__half, false>(a, s);
    return a.bf16 ? launch<__nv_bfloat16, true>(a, s) : launch<__half, true>(a, s);
}

}  // namespace pkv
