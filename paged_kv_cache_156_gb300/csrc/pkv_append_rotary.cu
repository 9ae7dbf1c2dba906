// paged_kv_append_rotary: a step's queries and keys turned to their positions,
// keys and values written into their slots.
//
// A head's first r elements are r / 2 pairs, (i, i + r / 2) or, interleaved,
// (2 i, 2 i + 1); the pair (x, y) becomes (x c - y s, y c + x s) with c and s
// the cosine and sine of the position's angle i, read from a table.  Each
// product and sum is rounded to fp32 by itself (no fused multiply-add), then the
// result once to its own type: the 16-bit type of q_out and of a 16-bit pool, or
// an E4M3 pool's code (divided by the head's scale first).
//
// Bound by HBM: every element is read once and written once.  One CTA a token;
// a thread takes two 16-byte pieces of a row (a row: a head of q, k or v), the
// two halves of eight pairs, and the same two of further rows, so that it reads
// its cosines and sines once.  All of a thread's loads stand before its first
// store, and before what the token's slot and position decide (66 to 58 us).
// 8192 tokens of 64 heads over 8, bf16: 51.7 us, 6.6 TB/s, 97% of the measured
// copy (256 threads 58 us, 64 threads 52, five rows a thread 53); 1037 tokens
// into an E4M3 pool 5.5 us (256 threads 9.0), launch and dependent reads.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;                       // (heads of more than 2048 elements: twice as many)
constexpr int kRows = 3;                            // rows of a thread whose loads are in flight together

// (ld.cg, never ld.nc: q_out may be q, and the compiler may move an ld.nc above the wait for the kernel that writes it)
__device__ __forceinline__ uint4 load16(const void* p) { return __ldcg(static_cast<const uint4*>(p)); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
    if constexpr (BF16) return Mma<__nv_bfloat16>::pack(x, y);
    else return Mma<__half>::pack(x, y);
}

template <bool BF16>
__device__ __forceinline__ void widen(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = pair_to_float2<BF16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
    return make_uint4(pack_pair<BF16>(x[0], x[1]), pack_pair<BF16>(x[2], x[3]), pack_pair<BF16>(x[4], x[5]),
                      pack_pair<BF16>(x[6], x[7]));
}
__device__ __forceinline__ uint2 quantize8f(const float (&x)[8], float scale) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}

template <bool BF16, bool KV8>
__global__ void __launch_bounds__(2 * kThreads) append_rotary_kernel(const __grid_constant__ AppendRotaryArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const int64_t tok = blockIdx.x;
    const int units = a.head_dim / 16;              // of a row: two 16-byte pieces each
    const int step = blockDim.x / units;             // rows the CTA takes side by side
    const int u = threadIdx.x % units, r0 = threadIdx.x / units;
    if (r0 >= step) return;
    const int half = a.rotary_dim / 2;
    const bool turns = u < a.rotary_dim / 16;
    const bool apart = turns && !a.interleaved;     // its pieces stand half the rotated elements apart
    const int e0 = apart ? 8 * u : 16 * u, e1 = apart ? e0 + half : e0 + 8;      // their first elements
    const int hq = a.num_heads, hk = a.num_kv_heads, d = a.head_dim;
    const int rows = hq + 2 * hk;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + tok * a.q_stride;
    const uint16_t* k = static_cast<const uint16_t*>(a.k) + tok * a.k_stride;
    const uint16_t* v = static_cast<const uint16_t*>(a.v) + tok * a.v_stride;
    uint16_t* q_out = static_cast<uint16_t*>(a.q_out) + tok * a.q_out_stride;
    uint4 x[kRows][2];
    auto load = [&](int base) {                     // (whatever becomes of the token: its rows are there)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = base + i * step;
            if (r < rows) {
                const uint16_t* src = r < hq ? q + r * d : r < hq + hk ? k + (r - hq) * d : v + (r - hq - hk) * d;
                x[i][0] = load16(src + e0);
                x[i][1] = load16(src + e1);
            }
        }
    };
    const int64_t slot = __ldcg(a.slots + tok);
    const int pos = __ldcg(a.positions + tok);
    load(r0);
    if (pos < 0 || pos >= a.num_positions) {        // nothing to turn by: the token is left out
        if (threadIdx.x == 0 && !(pos < 0 && slot < 0)) raise_error(a.err, kErrBounds);
        return;
    }
    bool store_kv = slot >= 0;                      // (a negative slot: nothing to write there)
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) raise_error(a.err, kErrBounds);
        store_kv = false;
    }
    float c[8], s[8];
    if (turns) {
        const float4* cp = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + 8 * u);
        const float4* sp = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * a.rotary_dim + half + 8 * u);
        const float4 c0 = __ldcg(cp), c1 = __ldcg(cp + 1), s0 = __ldcg(sp), s1 = __ldcg(sp + 1);
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
#pragma unroll 1
    for (int base = r0;;) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = base + i * step;
            if (!(r < hq || (r < rows && store_kv))) continue;
            const bool is_v = r >= hq + hk;
            const int h = r < hq ? r : is_v ? r - hq - hk : r - hq;
            const int64_t at = slot * hk * d + h * d;            // (in the pool)
            if (!turns || is_v) {
                if (!KV8 || r < hq) {
                    uint16_t* dst = r < hq ? q_out + h * d : static_cast<uint16_t*>(is_v ? a.value_cache : a.key_cache) + at;
                    *reinterpret_cast<uint4*>(dst + e0) = x[i][0];
                    *reinterpret_cast<uint4*>(dst + e1) = x[i][1];
                    continue;
                }
            }
            float lo[8], hi[8];
            widen<BF16>(x[i][0], lo);
            widen<BF16>(x[i][1], hi);
            if (turns && !is_v) {
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        turn(lo[2 * e], lo[2 * e + 1], c[e], s[e]);
                        turn(hi[2 * e], hi[2 * e + 1], c[4 + e], s[4 + e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) turn(lo[e], hi[e], c[e], s[e]);
                }
            }
            if (!KV8 || r < hq) {
                uint16_t* dst = r < hq ? q_out + h * d : static_cast<uint16_t*>(a.key_cache) + at;
                *reinterpret_cast<uint4*>(dst + e0) = narrow<BF16>(lo);
                *reinterpret_cast<uint4*>(dst + e1) = narrow<BF16>(hi);
            } else {
                const float scale = __ldcg((is_v ? a.v_scale : a.k_scale) + h);
                uint8_t* dst = static_cast<uint8_t*>(is_v ? a.value_cache : a.key_cache) + at;
                *reinterpret_cast<uint2*>(dst + e0) = quantize8f(lo, scale);
                *reinterpret_cast<uint2*>(dst + e1) = quantize8f(hi, scale);
            }
        }
        base += kRows * step;
        if (base >= rows) break;
        load(base);
    }
}

template <bool BF16, bool KV8>
cudaError_t launch(const AppendRotaryArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.num_tokens));
    cfg.blockDim = dim3(a.head_dim / 16 > kThreads ? 2 * kThreads : kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_rotary_kernel<BF16, KV8>, a);
}

}  // namespace

cudaError_t launch_append_rotary(const AppendRotaryArgs& a, bool bf16, bool kv8, cudaStream_t s) {
    if (a.num_tokens <= 0) return cudaSuccess;
    if (bf16) return kv8 ? launch<true, true>(a, s) : launch<true, false>(a, s);
    return kv8 ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace pkv
