// paged_kv_gather: the cached K/V of a batch read back into dense rows.
//
//     k_out[row_starts[s] + t] = K_t, v_out likewise,  t < seq_lens[s],
//
// K_t being the pool's row itself, or, over an E4M3 pool, each code's value
// times its KV head's scale in fp32, rounded once to the output type.  The
// inverse of the slot writes (pkv_append.cu): what a dense kernel, another
// process or a prefix store takes from the cache.
//
// HBM-bound: every byte is read once and written once (64 sequences of 512 to 4096
// positions, 8 heads of 128, bf16: 177 us, 6.71 TB/s, 99% of a plain copy; 100 of 1
// to 1500 over E4M3 pools: 77 us, 6.53 TB/s).  The grid covers the
// output's rows (the one size the host knows), so many a CTA that each thread has
// kUnroll loads of K and of V; the CTA finds the sequence of its first row by
// counting the starts at or below it (no search loop: one load a thread for up to
// 256 sequences), every thread walks on from there to a row of its own, and then
// the rows are moved 16 bytes a load, a thread's loads before its stores.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = kThreads;                  // output rows a CTA at most
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

// The neighbouring lane's first 8 codes for an even lane, its last 8 for an odd one.
__device__ __forceinline__ uint2 swap_half(bool odd, const uint4& x) {
    uint2 g = odd ? make_uint2(x.x, x.y) : make_uint2(x.z, x.w);
    g.x = __shfl_xor_sync(0xffffffffu, g.x, 1);
    g.y = __shfl_xor_sync(0xffffffffu, g.y, 1);
    return g;
}

// T: the output's type over an E4M3 pool (KV8); 16-bit rows are moved as they are.  WIDE: 16 codes a load (head_dim
// a multiple of 16, an even number of loads a row and 16-byte aligned pools), else 8.
template <typename T, bool KV8, bool WIDE>
__global__ void __launch_bounds__(kThreads, 4) gather_kernel(const GatherArgs a) {
    __shared__ int64_t src_row[kMaxRows];           // the output row's row in the pools (-1: not written)
    grid_dependency_wait();
    launch_dependents();
    const int rows = a.cta_rows;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows;
    const int t = threadIdx.x;
    // ---- the last sequence that starts at or before the first row (the starts do not decrease)
    int mine = 0;
    for (int i = t; i < a.num_seqs; i += kThreads) mine += __ldcg(a.row_starts + i) <= row0 ? 1 : 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    __shared__ int part[kThreads / 32];
    if ((t & 31) == 0) part[t >> 5] = mine;
    __syncthreads();
    if (t < rows) {
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
    // the heads' scales, once a CTA (from L2 for every vector they cost as much as the codes)
    extern __shared__ float scales[];               // [K | V][heads]
    const int heads = KV8 ? a.row_vecs / a.head_vecs : 0;
    for (int i = t; i < heads; i += kThreads) {
        scales[i] = __ldcg(a.k_scale + i);
        scales[heads + i] = __ldcg(a.v_scale + i);
    }
    // the batch's lengths and starts, checked by the first CTA
    if (blockIdx.x == 0)
        for (int i = t; i < a.num_seqs; i += kThreads) {
            const int start = __ldcg(a.row_starts + i), end = __ldcg(a.row_starts + i + 1), len = __ldcg(a.seq_lens + i);
            if (start < 0 || end < start || end > a.num_rows || len > end - start) raise_error(a.err, kErrBounds);
        }
    __syncthreads();

    // A thread's row and place advance by constants, without a division a vector.
    using Vec = std::conditional_t<KV8 && !WIDE, uint2, uint4>;
    constexpr int kOut = KV8 && WIDE ? 2 : 1;       // output vectors a load gives
    const int rv = a.row_vecs / kOut;               // loads a row
    const int step_r = kThreads / rv, step_c = kThreads - step_r * rv;
    const int hv = KV8 ? a.head_vecs / kOut : 1;
    const int trips = (rows * rv + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    int r = t / rv, c = t - r * rv;
    for (int trip = 0; trip < trips; ++trip) {
        Vec x[kUnroll], y[kUnroll];
        int rr[kUnroll], cc[kUnroll];
        bool live[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            rr[u] = r;
            cc[u] = c;
            const int64_t src = r < rows ? src_row[r] : -1;
            live[u] = src >= 0;
            if (live[u]) {
                x[u] = __ldcs(static_cast<const Vec*>(a.key_cache) + src * rv + c);
                y[u] = __ldcs(static_cast<const Vec*>(a.value_cache) + src * rv + c);
            }
            r += step_r;
            c += step_c;
            if (c >= rv) {
                c -= rv;
                ++r;
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if constexpr (KV8 && WIDE) {
                // 16 codes are two output vectors: lane pairs swap halves, so that a pair's store fills a
                // 32-byte sector (each lane's two vectors stored by itself filled half of one at a time and
                // cost 15% more)
                const bool odd = threadIdx.x & 1;
                const uint2 kx = swap_half(odd, x[u]), vx = swap_half(odd, y[u]);
                if (!live[u]) continue;
                const int ce = cc[u] & ~1, h0 = ce / hv, h1 = (ce + 1) / hv;
                const int64_t at = ((row0 + rr[u]) * rv + ce) * 2 + odd;
                a.k_out[at] = expand8<T>(odd ? kx : make_uint2(x[u].x, x[u].y), scales[h0]);
                a.v_out[at] = expand8<T>(odd ? vx : make_uint2(y[u].x, y[u].y), scales[heads + h0]);
                a.k_out[at + 2] = expand8<T>(odd ? make_uint2(x[u].z, x[u].w) : kx, scales[h1]);
                a.v_out[at + 2] = expand8<T>(odd ? make_uint2(y[u].z, y[u].w) : vx, scales[heads + h1]);
            } else if (live[u]) {
                const int64_t at = (row0 + rr[u]) * rv + cc[u];
                if constexpr (KV8) {
                    const int h = cc[u] / hv;
                    a.k_out[at] = expand8<T>(x[u], scales[h]);
                    a.v_out[at] = expand8<T>(y[u], scales[heads + h]);
                } else {
                    a.k_out[at] = x[u];
                    a.v_out[at] = y[u];
                }
            }
        }
    }
}

template <typename T, bool KV8, bool WIDE>
cudaError_t launch(GatherArgs a, cudaStream_t s) {
    const int loads = a.row_vecs / (KV8 && WIDE ? 2 : 1);                // a row
    a.cta_rows = std::min(kMaxRows, std::max(4, kThreads * kUnroll / loads));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.num_rows + a.cta_rows - 1) / a.cta_rows));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = KV8 ? 2 * sizeof(float) * static_cast<size_t>(a.row_vecs / a.head_vecs) : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_kernel<T, KV8, WIDE>, a);
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t s) {
    if (a.num_rows <= 0 || a.num_seqs <= 0) return cudaSuccess;
    if (!a.k_scale) return launch<__half, false, true>(a, s);
    const bool wide = a.head_vecs % 2 == 0 && a.row_vecs % 4 == 0 &&
                      ((reinterpret_cast<uintptr_t>(a.key_cache) | reinterpret_cast<uintptr_t>(a.value_cache)) & 15u) == 0;
    if (a.bf16) return wide ? launch<__nv_bfloat16, true, true>(a, s) : launch<__nv_bfloat16, true, false>(a, s);
    return wide ? launch<__half, true, true>(a, s) : launch<__half, true, false>(a, s);
}

}  // namespace pkv
