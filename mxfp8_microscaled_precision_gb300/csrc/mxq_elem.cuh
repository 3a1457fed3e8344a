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

// 16 bytes as kVec16<T> floats and back (a store rounds to nearest even).
template <typename T>
__device__ __forceinline__ void unpack(const uint4 w, float (&f)[kVec16<T>]) {
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

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec16<T>]) {
    if constexpr (sizeof(T) == 2)
        return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                          cvt_bf16x2(f[6], f[7]));
    else
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
}

// ---- rows that start at any element ------------------------------------------------
//
// A row whose length is odd leaves the next one off the 16-byte grid.  Element by element such rows
// move at a third of the bandwidth (64 bytes a request), so they are moved in
// vectors too: a load takes the two aligned vectors that its elements lie in
// and shifts them together, a store gets the missing elements of an aligned
// vector from the next lane.  Only a row's first and last vectors go element by
// element, so nothing outside the row is touched.

// Bytes off .. off + 15 of the 32 bytes a, b (off even, the same for most lanes).
__device__ __forceinline__ uint4 shift16(const uint4 a, const uint4 b, unsigned off) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (off & 2u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [i, i + V) of a row of n as 16 bytes, zeros from n on (i a multiple
// of V = 16 / kSize).  kAny: the row may start at any element; otherwise it is
// 16-byte aligned and n a multiple of V.
template <int kSize, bool kAny>
__device__ __forceinline__ uint4 load16(const void* row, int64_t i, int64_t n) {
    constexpr int V = 16 / kSize;
    const unsigned char* p = static_cast<const unsigned char*>(row) + i * kSize;
    if (i >= n) return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!kAny) {
        return *reinterpret_cast<const uint4*>(p);
    } else {
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15u);
        if (off == 0u && i + V <= n) return *reinterpret_cast<const uint4*>(p);
        if (i > 0 && i + 2 * V - static_cast<int>(off) / kSize <= n) {
            const uint4* q = reinterpret_cast<const uint4*>(p - off);
            return shift16(q[0], q[1], off);
        }
        uint32_t w[4] = {};
#pragma unroll
        for (int c = 0; c < V; ++c) {
            if (i + c < n) {
                if constexpr (kSize == 2)
                    w[c / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(p)[c]) << (16 * (c & 1));
                else
                    w[c] = reinterpret_cast<const uint32_t*>(p)[c];
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Elements a .. b - 1 (of the V that v holds) to p, one by one.
template <int kSize>
__device__ __forceinline__ void store_some(unsigned char* p, const uint4 v, int a, int b) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 16 / kSize; ++c) {
        if (c >= a && c < b) {
            if constexpr (kSize == 2)
                reinterpret_cast<unsigned short*>(p)[c] = static_cast<unsigned short>(w[c / 2] >> (16 * (c & 1)));
            else
                reinterpret_cast<uint32_t*>(p)[c] = w[c];
        }
    }
}

// Stores elements [i, i + V) of a row of n.  With kAny every lane of the warp
// takes part (a lane with nothing to store has i >= n), and within each `width` lanes
// (a power of two) lane l + 1 holds the V elements after lane l's of the same row.
template <int kSize, bool kAny>
__device__ __forceinline__ void store16(void* row, int64_t i, int64_t n, const uint4 v, int width = 32) {
    constexpr int V = 16 / kSize;
    unsigned char* p = static_cast<unsigned char*>(row) + i * kSize;
    if constexpr (!kAny) {
        if (i < n) *reinterpret_cast<uint4*>(p) = v;
    } else {
        const int lane = static_cast<int>(threadIdx.x) & (width - 1);
        uint4 next;
        next.x = __shfl_down_sync(0xFFFFFFFFu, v.x, 1);
        next.y = __shfl_down_sync(0xFFFFFFFFu, v.y, 1);
        next.z = __shfl_down_sync(0xFFFFFFFFu, v.z, 1);
        next.w = __shfl_down_sync(0xFFFFFFFFu, v.w, 1);
        const int m = i >= n ? 0 : (n - i < V ? static_cast<int>(n - i) : V);   // elements of this lane
        const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15u);
        if (off == 0u) {
            if (m == V) *reinterpret_cast<uint4*>(p) = v;
            else store_some<kSize>(p, v, 0, m);
            return;
        }
        const int head = V - static_cast<int>(off) / kSize;   // elements before the aligned vector
        if (m == V && lane < width - 1 && n - i - V >= head)
            *reinterpret_cast<uint4*>(p + (16u - off)) = shift16(v, next, 16u - off);
        else
            store_some<kSize>(p, v, head, m);
        if (lane == 0 || m < head)   // not in the vector that the lane before stored
            store_some<kSize>(p, v, 0, m < head ? m : head);
    }
}

// V = kVec16<T> parameters [i, i + V) of W (weights and the like, n of them, read
// by many rows) as floats; `otherwise` without a tensor.  kAny as for load16; the tensor
// starts on 16 bytes otherwise.
template <typename W, int V, bool kAny>
__device__ __forceinline__ void load_params(const W* p, int64_t i, int64_t n, float otherwise, float (&f)[V]) {
    if (p == nullptr) {
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = otherwise;
    } else if constexpr (V * sizeof(W) == 16) {
        unpack<W>(load16<sizeof(W), kAny>(p, i, n), f);
    } else if constexpr (V * sizeof(W) == 32) {   // 8 FP32 parameters of 8 BF16 elements
        float lo[4], hi[4];
        unpack<W>(load16<sizeof(W), kAny>(p, i, n), lo);
        unpack<W>(load16<sizeof(W), kAny>(p, i + 4, n), hi);
#pragma unroll
        for (int c = 0; c < 4; ++c) f[c] = lo[c], f[c + 4] = hi[c];
    } else {   // 4 BF16 parameters of 4 FP32 elements
        static_assert(V * sizeof(W) == 8, "vectors of 4 or 8");
        if (!kAny && i < n) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + i);
            f[0] = __uint_as_float(w.x << 16), f[1] = __uint_as_float(w.x & 0xFFFF0000u);
            f[2] = __uint_as_float(w.y << 16), f[3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) f[c] = i + c < n ? to_float(p[i + c]) : 0.0f;
        }
    }
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
