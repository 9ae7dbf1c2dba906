// Draws from a row of probabilities by whole units: what the acceptance kernels share.
//
// Each weight is cut to whole units of 2^-44 (fp32 times 2^44 is exact) and summed in 64-bit integers, so that a sum
// does not depend on its order (pkv_accept.cu says what the cut costs).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pkv_device.cuh"

namespace pkv {
namespace draw {

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (std::is_same<T, float>::value) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}

// Four probabilities, as one vector load brings them.
template <typename T>
struct Four {
    static constexpr int kWords = 2;
    static __device__ __forceinline__ void unpack(const uint32_t (&v)[2], float (&x)[4]) {
        const float2 lo = Mma<T>::unpack(v[0]), hi = Mma<T>::unpack(v[1]);
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    }
    // elements d to d + 3 of v and the vector after it, n (d: 1 to 3)
    static __device__ __forceinline__ void shift(uint32_t (&v)[2], const uint32_t (&n)[2], int d) {
        const uint32_t a = d >= 2 ? v[1] : v[0], b = d >= 2 ? n[0] : v[1], c = d >= 2 ? n[1] : n[0];
        v[0] = (d & 1) ? __funnelshift_r(a, b, 16) : a;
        v[1] = (d & 1) ? __funnelshift_r(b, c, 16) : b;
    }
    static __device__ __forceinline__ void load(uint32_t (&v)[2], const T* p) {
        const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
        v[0] = r.x; v[1] = r.y;
    }
};
template <>
struct Four<float> {
    static constexpr int kWords = 4;
    static __device__ __forceinline__ void unpack(const uint32_t (&v)[4], float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(v[e]);
    }
    static __device__ __forceinline__ void shift(uint32_t (&v)[4], const uint32_t (&n)[4], int d) {
        const uint32_t x[7] = {v[0], v[1], v[2], v[3], n[0], n[1], n[2]};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = d == 1 ? x[e + 1] : d == 2 ? x[e + 2] : x[e + 3];
    }
    static __device__ __forceinline__ void load(uint32_t (&v)[4], const float* p) {
        const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
        v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
    }
};

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

}  // namespace draw
}  // namespace pkv
