// mxq_elem.cuh -- element access shared by the operators around the GEMMs
// (routing, row permutation, layer norm, gradient clipping): BF16 and FP32
// values in vectors of 16 bytes or one by one, and reductions over a warp.
// Values are held in FP32; a store rounds once, to nearest even.
#pragma once

#include <cstdint>

#include "mxq_device.cuh"

namespace mxq {

// Storage types: BF16 as its bits, FP32 as float.
using bf16_bits = unsigned short;

__device__ __forceinline__ float to_float(bf16_bits v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_bits from_float<bf16_bits>(float v) {
    return static_cast<bf16_bits>(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
}

// Elements of a 16-byte vector.
template <typename T>
constexpr int kVec16 = 16 / static_cast<int>(sizeof(T));

// V consecutive elements as floats.  V * sizeof(T) is 16 (p 16-byte aligned),
// or V is 1.
template <typename T, int V>
__device__ __forceinline__ void unpack(const uint4 w, float (&f)[V]) {
    static_assert(V * sizeof(T) == 16, "a 16-byte vector");
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(u[i]);
    }
}

template <typename T, int V>
__device__ __forceinline__ uint4 pack(const float (&f)[V]) {
    static_assert(V * sizeof(T) == 16, "a 16-byte vector");
    if constexpr (sizeof(T) == 2)
        return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                          cvt_bf16x2(f[6], f[7]));
    else
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
}

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
    if constexpr (V == 1)
        f[0] = to_float(*p);
    else
        unpack<T, V>(*reinterpret_cast<const uint4*>(p), f);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    if constexpr (V == 1)
        *p = from_float<T>(f[0]);
    else
        *reinterpret_cast<uint4*>(p) = pack<T, V>(f);
}

// Sum over the warp, the same order on every call, the result in all lanes.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

}  // namespace mxq
