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

// ---- pairs of floats -----------------------------------------------------------------
//
// Two FP32 values in one 64-bit register: sm_103 adds, multiplies and fuses pairs in one
// instruction (each half rounded as the scalar instruction rounds it).

using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    return static_cast<f32x2>(__float_as_uint(lo)) | (static_cast<f32x2>(__float_as_uint(hi)) << 32);
}
__device__ __forceinline__ float lo_of(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi_of(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 16 bytes as pairs and back.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4 w, f32x2 (&f)[kVec16<T> / 2]) {
    float s[kVec16<T>];
    unpack<T>(w, s);
#pragma unroll
    for (int i = 0; i < kVec16<T> / 2; ++i) f[i] = pair(s[2 * i], s[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const f32x2 (&f)[kVec16<T> / 2]) {
    float s[kVec16<T>];
#pragma unroll
    for (int i = 0; i < kVec16<T> / 2; ++i) s[2 * i] = lo_of(f[i]), s[2 * i + 1] = hi_of(f[i]);
    return pack<T>(s);
}

// ---- rows that start at any element ------------------------------------------------
//
// A row whose length is odd leaves the next one off the 16-byte grid.  Element by element such rows
// move at a third of the bandwidth (64 bytes a request), so they are moved in vectors
// too, on the 16-byte grid of the memory itself: with `lead` the elements between the last
// boundary and the row's first one, vector q holds the elements [q V - lead, q V - lead + V).  Only a row's
// first and last vectors, which it shares with its neighbours, go element by element,
// so nothing outside the row is touched.  Where another tensor's row has another lead, the two
// aligned vectors that the wanted elements lie in are loaded and shifted together.

// Elements of the row at p before its first one on the 16-byte grid.
template <int kSize>
__device__ __forceinline__ int lead_of(const void* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u) / kSize;
}

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

// Elements [i, i + V) (V = 16 / kSize) of a row of n, one by one; 0 outside the row.
template <int kSize>
__device__ __noinline__ uint4 load_ends(const void* row, int i, int n) {
    uint32_t w[4] = {};
#pragma unroll
    for (int c = 0; c < 16 / kSize; ++c) {
        if (i + c >= 0 && i + c < n) {
            if constexpr (kSize == 2)
                w[c / 2] |= static_cast<uint32_t>(static_cast<const unsigned short*>(row)[i + c]) << (16 * (c & 1));
            else
                w[c] = static_cast<const uint32_t*>(row)[i + c];
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kSize>
__device__ __noinline__ void store_ends(void* row, int i, int n, const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 16 / kSize; ++c) {
        if (i + c >= 0 && i + c < n) {
            if constexpr (kSize == 2)
                static_cast<unsigned short*>(row)[i + c] = static_cast<unsigned short>(w[c / 2] >> (16 * (c & 1)));
            else
                static_cast<uint32_t*>(row)[i + c] = w[c];
        }
    }
}

// v with the elements outside [0, n) set to 0; i: index of its first element.
template <int kSize>
__device__ __forceinline__ uint4 inside(const uint4 v, int i, int n) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if constexpr (kSize == 2) {
            const int e = i + 2 * c;
            w[c] &= (e >= 0 && e < n ? 0xFFFFu : 0u) | (e + 1 >= 0 && e + 1 < n ? 0xFFFF0000u : 0u);
        } else {
            w[c] = i + c >= 0 && i + c < n ? w[c] : 0u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Whether rows of n, of which this is one, lie before and after it in memory, so that a
// vector (or two) that it has a part of can be loaded whole.  Element by element the ends of a row cost
// its threads a second latency.
template <int kSize>
__device__ __forceinline__ bool is_between(int64_t row, int64_t rows, int n) {
    return row > 0 && row < rows - 1 && n >= 2 * (16 / kSize);
}

// Elements [i, i + V) of a row of n, where element i lies on the 16-byte grid; 0 outside the
// row.  Without kAny the row holds whole vectors, from its first element on.
template <int kSize, bool kAny>
__device__ __forceinline__ uint4 load16(const void* row, int i, int n, bool between = false) {
    const void* p = static_cast<const unsigned char*>(row) + static_cast<int64_t>(i) * kSize;
    if (kAny && between) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < n) v = *static_cast<const uint4*>(p);
        if (i < 0 || i + 16 / kSize > n) v = inside<kSize>(v, i, n);
        return v;
    }
    if (kAny ? i >= 0 && i + 16 / kSize <= n : i < n) return *static_cast<const uint4*>(p);
    if (kAny && i < n) return load_ends<kSize>(row, i, n);
    return make_uint4(0u, 0u, 0u, 0u);
}

// alike: element i lies on the 16-byte grid of this row too (kAny only).
template <int kSize, bool kAny>
__device__ __forceinline__ void store16(void* row, int i, int n, const uint4 v, bool alike = true) {
    void* p = static_cast<unsigned char*>(row) + static_cast<int64_t>(i) * kSize;
    if (kAny ? alike && i >= 0 && i + 16 / kSize <= n : i < n) *static_cast<uint4*>(p) = v;
    else if (kAny && i < n) store_ends<kSize>(row, i, n, v);
}

// Whether the elements [i, i + V) of rows of n with any lead can be loaded by two vectors
// each without leaving the row.
template <int kSize>
__device__ __forceinline__ bool is_inner(int i, int n) {
    constexpr int V = 16 / kSize;
    return i >= V - 1 && i + 2 * V <= n;
}

// Elements [i, i + V) of a row with any lead (is_inner holds).
template <int kSize>
__device__ __forceinline__ uint4 load_inner(const void* row, int i) {
    const unsigned char* p = static_cast<const unsigned char*>(row) + static_cast<int64_t>(i) * kSize;
    const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15u);
    const uint4* q = reinterpret_cast<const uint4*>(p - off);
    return shift16(q[0], q[1], off);
}

// The same of any row, i < n; 0 outside it.
template <int kSize>
__device__ __forceinline__ uint4 load_shifted(const void* row, int i, int n, bool between) {
    if (!between && !is_inner<kSize>(i, n)) return load_ends<kSize>(row, i, n);
    uint4 v = load_inner<kSize>(row, i);
    if (i < 0 || i + 16 / kSize > n) v = inside<kSize>(v, i, n);
    return v;
}

// V parameters [i, i + V) of W (weights and the like, n of them, read by many rows) as
// pairs; `otherwise` without a tensor, 0 outside it.  Without kAny the tensor starts on 16 bytes and
// i is a multiple of V.
template <typename W, int V, bool kAny>
__device__ __forceinline__ void load_params2(const W* p, int i, int n, float otherwise, f32x2 (&f)[V / 2]) {
    if (p == nullptr) {
#pragma unroll
        for (int c = 0; c < V / 2; ++c) f[c] = pair(otherwise, otherwise);
    } else if constexpr (V * sizeof(W) == 8) {   // 4 BF16 parameters of 4 FP32 elements
        uint2 w = make_uint2(0u, 0u);
        if (!kAny) {
            if (i < n) w = *reinterpret_cast<const uint2*>(p + i);
        } else {
            const uint4 v = load_ends<2>(p, i, i + 4 < n ? i + 4 : n);
            w = make_uint2(v.x, v.y);
        }
        f[0] = pair(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
        f[1] = pair(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        constexpr int kPer = kVec16<W>;   // parameters of 16 bytes: V, or half of it
#pragma unroll
        for (int k = 0; k < V / kPer; ++k) {
            const int at = i + k * kPer;
            uint4 v;
            if (!kAny) v = load16<sizeof(W), false>(p, at, n);
            else v = is_inner<sizeof(W)>(at, n) ? load_inner<sizeof(W)>(p, at) : load_ends<sizeof(W)>(p, at, n);
            f32x2 s[kPer / 2];
            unpack2<W>(v, s);
#pragma unroll
            for (int c = 0; c < kPer / 2; ++c) f[k * kPer / 2 + c] = s[c];
        }
    }
}

// V parameters of a thread's columns in the registers of their own type, for a loop over rows.
template <typename W, int V>
struct Params {
    uint32_t u[V * sizeof(W) / 4];
    template <bool kAny>
    __device__ __forceinline__ void load(const W* p, int i, int n, float otherwise) {
        f32x2 f[V / 2];
        load_params2<W, V, kAny>(p, i, n, otherwise, f);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
            if constexpr (sizeof(W) == 2) {
                u[c] = cvt_bf16x2(lo_of(f[c]), hi_of(f[c]));   // exact: 0, 1 or a BF16 value
            } else {
                u[2 * c] = __float_as_uint(lo_of(f[c]));
                u[2 * c + 1] = __float_as_uint(hi_of(f[c]));
            }
        }
    }
    __device__ __forceinline__ void get(f32x2 (&f)[V / 2]) const {
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
            if constexpr (sizeof(W) == 2)
                f[c] = pair(__uint_as_float(u[c] << 16), __uint_as_float(u[c] & 0xFFFF0000u));
            else
                f[c] = pair(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]));
        }
    }
};

// The same in shared memory, n vectors of V a thread, each thread's its own (nobody else reads
// them): [n][16-byte parts of V parameters][threads].
template <typename W, int V>
struct ParamSlots {
    static constexpr int kWords = V * static_cast<int>(sizeof(W)) / 4;   // 2, 4 or 8
    static constexpr int kPart = kWords < 4 ? kWords : 4;
    uint32_t* mine;
    int threads;
    static constexpr int64_t bytes_of(int64_t n, int64_t threads) { return n * threads * V * sizeof(W); }
    __device__ __forceinline__ ParamSlots(void* memory, int thread, int threads)
        : mine(static_cast<uint32_t*>(memory) + thread * kPart), threads(threads) {}
    __device__ __forceinline__ uint32_t* part(int n, int k) const {
        return mine + (n * (kWords / kPart) + k) * threads * kPart;
    }
    __device__ __forceinline__ void put(int n, const Params<W, V>& p) const {
#pragma unroll
        for (int c = 0; c < kWords; ++c) part(n, c / kPart)[c % kPart] = p.u[c];
    }
    __device__ __forceinline__ void get(int n, f32x2 (&f)[V / 2]) const {
        Params<W, V> p;
#pragma unroll
        for (int k = 0; k < kWords / kPart; ++k) {
            if constexpr (kPart == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(part(n, k));
                p.u[4 * k] = v.x, p.u[4 * k + 1] = v.y, p.u[4 * k + 2] = v.z, p.u[4 * k + 3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(part(n, k));
                p.u[0] = v.x, p.u[1] = v.y;
            }
        }
        p.get(f);
    }
};

// Asynchronous copy of 16 bytes to shared memory (both sides aligned), of which `bytes` are read and the others set to 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Four bytes, or zeros (bytes = 0).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// In a kernel launched by launch_behind: returns when the kernel before it has ended and its
// results are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// In any kernel: a kernel launched behind it by launch_behind may be put on the device from now on, as far as there is
// room; what it reads still waits for this one's end.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
