// act.cu -- the (gated) activation between two products, and its gradients from an input kept in 8 bits.
//
//   y = f(g) u  (without a gate: f(g)),  f(g) = g / (1 + exp(-g))  or  g (1 + erf(g / sqrt 2)) / 2
//   checkpoint: g and u in E4M3, one E8M0 scale per 32 elements of a row (each of the two on its own)
//   backward, from the checkpoint's values:  dg = dy u f'(g),  du = dy f(g),  y = f(g) u
//
// Memory-bound: every tensor is read or written once.  Two forms of each kernel.  Rows that hold whole 16-byte
// vectors (inter a multiple of 8, all rows aligned): a thread has eight elements of g and the eight of
// u in the same places, the four threads of a group of 32 sit side by side.  Any other rows: a lane has one
// element of a group, a warp several groups, so that its accesses are contiguous wherever a row starts.
// Arithmetic in FP32, one rounding.
//
// 131072 x 2 x 2048 BF16, SiLU with a gate: 351 us forward (91% of the copy rate), 228 us without a checkpoint, 386 us
// backward; GELU 423, 271 and 425 us (forward by its instructions).  65536 x 2 x 2048 FP32: SiLU 270, 226 and 371 us, GELU 272, 226
// and 359 us (the copy rate, but for SiLU backward, 96%).  BF16 rows of 2047: 652, 286 and 717 us, the checkpoint
// by single bytes; FP32 SiLU 364, 227 and 466 us.  Tried on such rows without gain: eight elements a lane from shifted vectors, results
// through shared memory onto the 16-byte grid of their rows (673, 424 and 813 us; 4099 x 1111 FP32 GELU forward 14.8 us when the
// kernel took 14.6 us, now 12.6).

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"
#include "mxq_quant_math.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kSilu = 0, kGelu = 1;
constexpr int kSpan = 8;   // groups of 32 that a warp of the second form has at once

// exp(-(x + rest)), x in [0, 200], rest small.  What the product x log2(e) loses to its rounding (Dekker's exact product, by
// one fused operation), log2(e)'s own next digits and rest come back as a factor 1 + d ln 2.
__device__ __forceinline__ float exp_minus(float x, float rest) {
    constexpr float kLog2e = 1.44269502162933349609375f, kLow = 1.9259629911266175e-8f, kLn2 = 0.693147182464599609375f;
    const float t = x * -kLog2e, d = fmaf(x, -kLow, fmaf(x, -kLog2e, -t)), e = exp2f(t);
    return fmaf(e, fmaf(d, kLn2, -rest), e);
}

// f(g) and, where asked for, f'(g), as precise as results of T show.  BF16: the fast exponential, whose argument's rounding costs
// |g| (GELU: g^2 / 2) roundings in the tails, 63 units of 2^-24 at -80 and 124 at -12; a result rounds by 2^16 of them.  FP32:
// exp_minus, 6 and 10 units at most, for which rows that start anywhere pay (65536 x 2 x 2047 kept, SiLU 336 us to 363 us, GELU
// 373 us to 396 us; 4099 x 1111 GELU 11.8 us to 12.6 us).  CUDA's expf and division cost more there (408, 447 and 14.5 us).
template <typename T, int kKind, bool kSlope>
__device__ __forceinline__ float act(float g, float* slope) {
    constexpr bool kFull = sizeof(T) == 4;
    if constexpr (kKind == kSilu) {
        // from exp(-|g|), which neither overflows nor loses the far side's digits to 1 - sig
        const float e = kFull ? exp_minus(fminf(fabsf(g), 200.0f), 0.0f) : __expf(-fabsf(g));
        const float r = __fdividef(1.0f, 1.0f + e), far = e * r;
        const float sig = g < 0.0f ? far : r;
        if (kSlope) *slope = sig * (1.0f + g * (g < 0.0f ? r : far));   // f' = s(g) (1 + g s(-g))
        return g * sig;
    } else {
        // The normal distribution's far side, exp(-g^2/2) h(|g|) with h(a) = exp(a^2/2) erfc(a / sqrt 2) / 2: the bell
        // that the slope needs too times a smooth function, here t P(t), t = k / (a + k), P by least squares on
        // Chebyshev points of [0, 15] weighted towards equal relative errors: 4.4e-8 at most with these coefficients.
        constexpr float kP[9] = {0.10640031844377518f, 0.10602681338787079f, 0.10231088101863861f,
                                 0.06455493718385696f, 0.12730126082897186f, -0.10002311319112778f,
                                 0.20164304971694946f, -0.1384870558977127f, 0.030272917822003365f};
        const float a = fabsf(g), t = __fdividef(3.75f, a + 3.75f);
        float e;
        if constexpr (kFull) {   // at 20 it is zero already
            const float b = fminf(a, 20.0f), half = 0.5f * b, square = half * b;
            e = exp_minus(square, fmaf(half, b, -square));
        } else {
            e = __expf(-0.5f * g * g);
        }
        float h = kP[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) h = fmaf(h, t, kP[i]);
        const float far = e * (h * t), cdf = g < 0.0f ? far : 1.0f - far;
        if (kSlope) *slope = fmaf(g * e, 0.39894228040143268f, cdf);
        return g * cdf;
    }
}

// Scale code and factor 2^-e of a group whose largest |x| has these bits; false: NaN or infinity in it.
__device__ __forceinline__ bool e4m3_scale(uint32_t amax, uint32_t* code, float* factor) {
    if (amax >= kInfBits) {
        *code = 0xFFu;
        return false;
    }
    const int e = rceil_exponent_f32<kE4M3>(amax);
    *code = static_cast<uint32_t>(e + 127);
    *factor = pow2_neg(e);
    return true;
}

// ---- rows of whole vectors -----------------------------------------------------------------------

// Eight elements of a row.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
    // FP32 without the hint that they are read once: two loads take the halves of a thread's sectors, and the hint lets go of
    // some between them (L1 hits 38% instead of 50%; SiLU not kept, 65536 x 2 x 2048: 251 us, 226 us without it)
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            const uint4* from = reinterpret_cast<const uint4*>(p) + i;
            w[i] = sizeof(T) == 2 ? __ldcs(from) : *from;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            float s[kVec16<T>];
            unpack<T>(w[i], s);
#pragma unroll
            for (int j = 0; j < kVec16<T>; ++j) f[i * kVec16<T> + j] = s[j];
        }
    }
    // largest |x| of the group (four threads), as FP32 bits
    __device__ __forceinline__ uint32_t group_amax() const {
        uint32_t m;
        if constexpr (sizeof(T) == 2) {
            m = amax8_bits(w[0]) << 16;
        } else {
            m = 0u;
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
        }
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    // E4M3 of the eight (group_amax over the group's four threads); *code: the group's scale
    __device__ __forceinline__ uint2 e4m3(uint32_t* code) const {
        float factor;
        float f[8];
        get(f);
        uint32_t o[4];
        if (e4m3_scale(group_amax(), code, &factor)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = cvt_e4m3x2(f[2 * i] * factor, f[2 * i + 1] * factor);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = 0x7F7Fu | ((__float_as_uint(f[2 * i]) >> 24) & 0x80u) | ((__float_as_uint(f[2 * i + 1]) >> 16) & 0x8000u);
        }
        return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
        float s[kVec16<T>];
#pragma unroll
        for (int j = 0; j < kVec16<T>; ++j) s[j] = f[i * kVec16<T> + j];
        reinterpret_cast<uint4*>(p)[i] = pack<T>(s);   // what follows reads it; the checkpoint, read much later, streams
    }
}

// Blocks of kThreads >> log_row rows by 1 << log_row threads.
struct Place {
    int64_t row;
    int64_t col;
};
__device__ __forceinline__ Place place_of(int log_row) {
    const int t = threadIdx.x;
    return {static_cast<int64_t>(blockIdx.x) * (kThreads >> log_row) + (t >> log_row),
            ((static_cast<int64_t>(blockIdx.y) << log_row) + (t & ((1 << log_row) - 1))) * 8};
}

template <typename T, int kKind, bool kGated, bool kKeep>
__global__ void __launch_bounds__(kThreads) act_kernel(const ActArgs a, int log_row) {
    const Place at = place_of(log_row);
    const bool in = at.row < a.rows && at.col < a.inter;
    Eight<T> g, u;
    g.clear();
    u.clear();
    const T* z = static_cast<const T*>(a.z) + at.row * a.ldz + at.col;
    if (in) {
        g.load(z);
        if (kGated) u.load(z + a.inter);
        float fg[8], fu[8], y[8];
        g.get(fg);
        u.get(fu);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float f = act<T, kKind, false>(fg[k], nullptr);
            y[k] = kGated ? f * fu[k] : f;
        }
        store8(static_cast<T*>(a.y) + at.row * a.ldy + at.col, y);
    }
    if constexpr (kKeep) {
        constexpr int kParts = kGated ? 2 : 1;
        const int64_t groups = (a.inter + 31) >> 5;
        uint8_t* q = static_cast<uint8_t*>(a.q) + at.row * kParts * a.inter + at.col;
        uint8_t* s = static_cast<uint8_t*>(a.s) + at.row * kParts * groups + (at.col >> 5);
        const bool first = in && (at.col & 31) == 0;
        uint32_t code;
        const uint2 qg = g.e4m3(&code);
        if (in) __stcs(reinterpret_cast<uint2*>(q), qg);
        if (first) s[0] = static_cast<uint8_t>(code);
        if constexpr (kGated) {
            const uint2 qu = u.e4m3(&code);
            if (in) __stcs(reinterpret_cast<uint2*>(q + a.inter), qu);
            if (first) s[groups] = static_cast<uint8_t>(code);
        }
    }
}

__device__ __forceinline__ void restore8(const uint2 v, float s, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = cvt_f16_fp8x2<kE4M3>(((i < 2 ? v.x : v.y) >> (16 * (i & 1))) & 0xFFFFu);
        f[2 * i] = f16_lo(h) * s;
        f[2 * i + 1] = f16_hi(h) * s;
    }
}

template <typename T, int kKind, bool kGated>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(const ActBackwardArgs a, int log_row) {
    const Place at = place_of(log_row);
    if (at.row >= a.rows || at.col >= a.inter) return;
    constexpr int kParts = kGated ? 2 : 1;
    const int64_t groups = (a.inter + 31) >> 5;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + at.row * kParts * a.inter + at.col;
    const uint8_t* s = static_cast<const uint8_t*>(a.s) + at.row * kParts * groups + (at.col >> 5);
    Eight<T> d;
    d.load(static_cast<const T*>(a.dy) + at.row * a.lddy + at.col);
    const uint2 qg = __ldcs(reinterpret_cast<const uint2*>(q));
    const uint2 qu = kGated ? __ldcs(reinterpret_cast<const uint2*>(q + a.inter)) : make_uint2(0u, 0u);
    const float sg = scale_of(s[0]), su = kGated ? scale_of(s[groups]) : 0.0f;
    float g[8], u[8], dy[8], dg[8], du[8], y[8];
    restore8(qg, sg, g);
    restore8(qu, su, u);
    d.get(dy);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float slope;
        const float f = act<T, kKind, true>(g[k], &slope);
        y[k] = kGated ? f * u[k] : f;
        dg[k] = (kGated ? dy[k] * u[k] : dy[k]) * slope;
        du[k] = dy[k] * f;
    }
    T* dz = static_cast<T*>(a.dz) + at.row * a.lddz + at.col;
    store8(dz, dg);
    if (kGated) store8(dz + a.inter, du);
    if (a.y != nullptr) store8(static_cast<T*>(a.y) + at.row * a.ldy + at.col, y);
}

// ---- rows that start anywhere --------------------------------------------------------------------

// E4M3 of a group that a warp holds, one element a lane.
__device__ __forceinline__ uint32_t lane_e4m3(float f, uint32_t* code) {
    float factor;
    if (e4m3_scale(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(f) & 0x7FFFFFFFu), code, &factor))
        return cvt_e4m3x2(f * factor, 0.0f) & 0xFFu;
    return 0x7Fu | ((__float_as_uint(f) >> 24) & 0x80u);
}

// The first group and the row of a warp: kSpan groups, `per_row` such warps a row, row after row.
struct Span {
    int64_t row, group;
};
__device__ __forceinline__ Span span_of(int per_row) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5), row = w / per_row;
    return {row, (w - row * per_row) * kSpan};
}

template <typename T, int kKind, bool kGated, bool kKeep>
__global__ void __launch_bounds__(kThreads) act_any_kernel(const ActArgs a, int per_row) {
    const Span at = span_of(per_row);
    if (at.row >= a.rows) return;   // a whole warp
    constexpr int kParts = kGated ? 2 : 1;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (a.inter + 31) >> 5, c0 = at.group * 32 + lane;
    const T* z = static_cast<const T*>(a.z) + at.row * a.ldz;
    float g[kSpan], u[kSpan];
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        const int64_t c = c0 + 32 * i;
        g[i] = c < a.inter ? to_float(z[c]) : 0.0f;
        if (kGated) u[i] = c < a.inter ? to_float(z[a.inter + c]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        const int64_t c = c0 + 32 * i;
        const float f = act<T, kKind, false>(g[i], nullptr);
        if (c < a.inter) static_cast<T*>(a.y)[at.row * a.ldy + c] = from_float<T>(kGated ? f * u[i] : f);
        if constexpr (kKeep) {
            uint8_t* q = static_cast<uint8_t*>(a.q) + at.row * kParts * a.inter + c;
            uint8_t* s = static_cast<uint8_t*>(a.s) + at.row * kParts * groups + at.group + i;
            const bool first = lane == 0 && at.group + i < groups;
            uint32_t code;
            uint32_t o = lane_e4m3(g[i], &code);
            if (c < a.inter) *q = static_cast<uint8_t>(o);
            if (first) s[0] = static_cast<uint8_t>(code);
            if constexpr (kGated) {
                o = lane_e4m3(u[i], &code);
                if (c < a.inter) q[a.inter] = static_cast<uint8_t>(o);
                if (first) s[groups] = static_cast<uint8_t>(code);
            }
        }
    }
}

template <typename T, int kKind, bool kGated>
__global__ void __launch_bounds__(kThreads) act_backward_any_kernel(const ActBackwardArgs a, int per_row) {
    const Span at = span_of(per_row);
    if (at.row >= a.rows) return;
    constexpr int kParts = kGated ? 2 : 1;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (a.inter + 31) >> 5, c0 = at.group * 32 + lane;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + at.row * kParts * a.inter;
    const uint8_t* s = static_cast<const uint8_t*>(a.s) + at.row * kParts * groups + at.group;
    const T* d = static_cast<const T*>(a.dy) + at.row * a.lddy;
    uint32_t qg[kSpan], qu[kSpan], sg[kSpan], su[kSpan];
    float dy[kSpan];
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        const int64_t c = c0 + 32 * i;
        const bool in = c < a.inter;
        qg[i] = in ? q[c] : 0u;
        sg[i] = in ? s[i] : 0u;
        if (kGated) qu[i] = in ? q[a.inter + c] : 0u, su[i] = in ? s[groups + i] : 0u;
        dy[i] = in ? to_float(d[c]) : 0.0f;
    }
    T* dz = static_cast<T*>(a.dz) + at.row * a.lddz;
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        const int64_t c = c0 + 32 * i;
        if (c >= a.inter) break;
        const float g = f16_lo(cvt_f16_fp8x2<kE4M3>(qg[i])) * scale_of(sg[i]);
        const float u = kGated ? f16_lo(cvt_f16_fp8x2<kE4M3>(qu[i])) * scale_of(su[i]) : 1.0f;
        float slope;
        const float f = act<T, kKind, true>(g, &slope);
        dz[c] = from_float<T>((kGated ? dy[i] * u : dy[i]) * slope);
        if (kGated) dz[a.inter + c] = from_float<T>(dy[i] * f);
        if (a.y != nullptr) static_cast<T*>(a.y)[at.row * a.ldy + c] = from_float<T>(kGated ? f * u : f);
    }
}

// ---- host ----------------------------------------------------------------------------------------

// Whole vectors: 1 << log_row of a block's threads lie along a row, the least power of two that holds it or all.
struct Grid {
    dim3 blocks;
    int log_row;
    bool fits;
    Grid(int64_t rows, int64_t inter, int least_log) : log_row(least_log) {
        const int64_t units = inter / 8;
        while ((1 << log_row) < kThreads && (1 << log_row) < units) ++log_row;
        const int64_t down = kThreads >> log_row, x = (rows + down - 1) / down, y = (units + (1 << log_row) - 1) >> log_row;
        fits = x <= 0x7FFFFFFF && y <= 65535;
        blocks = dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
    }
};

// Any rows: warps of kSpan groups, row after row.
struct AnyGrid {
    unsigned blocks;
    int per_row;
    bool fits;
    AnyGrid(int64_t rows, int64_t inter) : per_row(static_cast<int>((inter + 32 * kSpan - 1) / (32 * kSpan))) {
        const int64_t n = (rows * per_row + kThreads / 32 - 1) / (kThreads / 32);
        fits = n <= 0x7FFFFFFF;
        blocks = static_cast<unsigned>(n);
    }
};

inline bool whole(const void* p, int64_t ld, int64_t size) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * size % 16 == 0;
}

template <typename T, int kKind, bool kGated>
cudaError_t launch_act_t(const ActArgs& a, cudaStream_t stream) {
    constexpr int64_t kSize = sizeof(T);
    if (a.inter % 8 == 0 && whole(a.z, a.ldz, kSize) && whole(a.y, a.ldy, kSize)) {
        const Grid grid(a.rows, a.inter, 2);   // a group's four threads in one row
        if (!grid.fits) return cudaErrorInvalidValue;
        if (a.q != nullptr) act_kernel<T, kKind, kGated, true><<<grid.blocks, kThreads, 0, stream>>>(a, grid.log_row);
        else act_kernel<T, kKind, kGated, false><<<grid.blocks, kThreads, 0, stream>>>(a, grid.log_row);
    } else {
        const AnyGrid grid(a.rows, a.inter);
        if (!grid.fits) return cudaErrorInvalidValue;
        if (a.q != nullptr) act_any_kernel<T, kKind, kGated, true><<<grid.blocks, kThreads, 0, stream>>>(a, grid.per_row);
        else act_any_kernel<T, kKind, kGated, false><<<grid.blocks, kThreads, 0, stream>>>(a, grid.per_row);
    }
    return cudaGetLastError();
}

template <typename T, int kKind, bool kGated>
cudaError_t launch_backward_t(const ActBackwardArgs& a, cudaStream_t stream) {
    constexpr int64_t kSize = sizeof(T);
    if (a.inter % 8 == 0 && whole(a.dy, a.lddy, kSize) && whole(a.dz, a.lddz, kSize) &&
        (a.y == nullptr || whole(a.y, a.ldy, kSize))) {
        const Grid grid(a.rows, a.inter, 0);
        if (!grid.fits) return cudaErrorInvalidValue;
        act_backward_kernel<T, kKind, kGated><<<grid.blocks, kThreads, 0, stream>>>(a, grid.log_row);
    } else {
        const AnyGrid grid(a.rows, a.inter);
        if (!grid.fits) return cudaErrorInvalidValue;
        act_backward_any_kernel<T, kKind, kGated><<<grid.blocks, kThreads, 0, stream>>>(a, grid.per_row);
    }
    return cudaGetLastError();
}

template <int kKind>
cudaError_t launch_act_of(const ActArgs& a, bool f32, bool gated, cudaStream_t stream) {
    if (f32) return gated ? launch_act_t<float, kKind, true>(a, stream) : launch_act_t<float, kKind, false>(a, stream);
    return gated ? launch_act_t<bf16_bits, kKind, true>(a, stream) : launch_act_t<bf16_bits, kKind, false>(a, stream);
}

template <int kKind>
cudaError_t launch_backward_of(const ActBackwardArgs& a, bool f32, bool gated, cudaStream_t stream) {
    if (f32) return gated ? launch_backward_t<float, kKind, true>(a, stream) : launch_backward_t<float, kKind, false>(a, stream);
    return gated ? launch_backward_t<bf16_bits, kKind, true>(a, stream) : launch_backward_t<bf16_bits, kKind, false>(a, stream);
}

}  // namespace

cudaError_t launch_activation(const ActArgs& a, bool f32, int kind, bool gated, cudaStream_t stream) {
    return kind == kSilu ? launch_act_of<kSilu>(a, f32, gated, stream) : launch_act_of<kGelu>(a, f32, gated, stream);
}

cudaError_t launch_activation_backward(const ActBackwardArgs& a, bool f32, int kind, bool gated, cudaStream_t stream) {
    return kind == kSilu ? launch_backward_of<kSilu>(a, f32, gated, stream) : launch_backward_of<kGelu>(a, f32, gated, stream);
}

}  // namespace mxq
