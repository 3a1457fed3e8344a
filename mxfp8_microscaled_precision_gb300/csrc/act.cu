// act.cu -- the (gated) activation between two products, and its gradients from an input kept in 8 bits.
//
//   y = f(g) u  (without a gate: f(g)),  f(g) = g / (1 + exp(-g))  or  g (1 + erf(g / sqrt 2)) / 2
//   checkpoint: g and u in E4M3, one E8M0 scale per 32 elements of a row (each of the two on its own)
//   backward, from the checkpoint's values:  dg = dy u f'(g),  du = dy f(g),  y = f(g) u
//
// A thread has eight elements of g and the eight of u in the same places; the four threads of a group of
// 32 sit side by side.  Arithmetic in FP32, one rounding.

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"
#include "mxq_quant_math.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kSilu = 0, kGelu = 1;

// f(g) and, where asked for, f'(g).
template <int kKind, bool kSlope>
__device__ __forceinline__ float act(float g, float* slope) {
    if constexpr (kKind == kSilu) {
        // from exp(-|g|), which neither overflows nor loses the far side's digits to 1 - sig
        const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e), far = e * r;
        const float sig = g < 0.0f ? far : r, other = g < 0.0f ? r : far;   // sigmoid of g and of -g
        if (kSlope) *slope = sig * (1.0f + g * other);
        return g * sig;
    } else {
        const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);   // 1 + erf would lose the bits of a negative g
        if (kSlope) *slope = cdf + g * expf(-0.5f * g * g) * 0.39894228040143268f;
        return g * cdf;
    }
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t c, int64_t n, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < n ? to_float(p[c + i]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t c, int64_t n, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < n) p[c + i] = from_float<T>(f[i]);
}

// E4M3 of eight elements of a group spread over four neighbouring threads.
__device__ __forceinline__ uint2 quant8_e4m3(const float (&f)[8], uint32_t* code) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    uint32_t o[4];
    if (m >= kInfBits) {
        *code = 0xFFu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = 0x7F7Fu | ((__float_as_uint(f[2 * i]) >> 24) & 0x80u) | ((__float_as_uint(f[2 * i + 1]) >> 16) & 0x8000u);
    } else {
        const int e = rceil_exponent_f32<kE4M3>(m);
        *code = static_cast<uint32_t>(e + 127);
        const float s = pow2_neg(e);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = cvt_e4m3x2(f[2 * i] * s, f[2 * i + 1] * s);
    }
    return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

__device__ __forceinline__ void store_q8(uint8_t* q, int64_t c, int64_t n, uint2 v) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < n) q[c + i] = static_cast<uint8_t>((i < 4 ? v.x : v.y) >> (8 * (i & 3)));
}

template <typename T, int kKind, bool kGated, bool kKeep>
__global__ void __launch_bounds__(kThreads) act_kernel(const ActArgs a, int64_t per_row) {
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    int64_t r = i / per_row;
    const int64_t c = (i - r * per_row) * 8;
    const bool in = r < a.rows;   // the threads of a group are in or out together
    if (!in) r = a.rows - 1;
    const T* z = static_cast<const T*>(a.z) + r * a.ldz;
    float g[8], u[8], y[8];
    load8(z, c, a.inter, g);
    if (kGated) load8(z + a.inter, c, a.inter, u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float f = act<kKind, false>(g[k], nullptr);
        y[k] = kGated ? f * u[k] : f;
    }
    if (in) store8(static_cast<T*>(a.y) + r * a.ldy, c, a.inter, y);
    if constexpr (kKeep) {
        const int64_t groups = (a.inter + 31) >> 5, width = kGated ? 2 : 1;
        uint8_t* q = static_cast<uint8_t*>(a.q) + r * width * a.inter;
        uint8_t* s = static_cast<uint8_t*>(a.s) + r * width * groups + (c >> 5);
        uint32_t code;
        const uint2 qg = quant8_e4m3(g, &code);
        if (in) store_q8(q, c, a.inter, qg);
        if (in && (c & 31) == 0) *s = static_cast<uint8_t>(code);
        if constexpr (kGated) {
            const uint2 qu = quant8_e4m3(u, &code);
            if (in) store_q8(q + a.inter, c, a.inter, qu);
            if (in && (c & 31) == 0) s[groups] = static_cast<uint8_t>(code);
        }
    }
}

__device__ __forceinline__ void load_q8(const uint8_t* q, int64_t c, int64_t n, float s, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t h = cvt_f16_fp8x2<kE4M3>((c + i < n ? q[c + i] : 0) | (c + i + 1 < n ? q[c + i + 1] << 8 : 0));
        f[i] = f16_lo(h) * s;
        f[i + 1] = f16_hi(h) * s;
    }
}

template <typename T, int kKind, bool kGated>
__global__ void __launch_bounds__(kThreads) act_backward_kernel(const ActBackwardArgs a, int64_t per_row) {
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    if (r >= a.rows) return;
    const int64_t groups = (a.inter + 31) >> 5, width = kGated ? 2 : 1;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + r * width * a.inter;
    const uint8_t* s = static_cast<const uint8_t*>(a.s) + r * width * groups + (c >> 5);
    float g[8], u[8], dy[8], dg[8], du[8], y[8];
    load_q8(q, c, a.inter, scale_of(s[0]), g);
    if (kGated) load_q8(q + a.inter, c, a.inter, scale_of(s[groups]), u);
    load8(static_cast<const T*>(a.dy) + r * a.lddy, c, a.inter, dy);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float slope;
        const float f = act<kKind, true>(g[k], &slope);
        y[k] = kGated ? f * u[k] : f;
        dg[k] = (kGated ? dy[k] * u[k] : dy[k]) * slope;
        du[k] = dy[k] * f;
    }
    T* dz = static_cast<T*>(a.dz) + r * a.lddz;
    store8(dz, c, a.inter, dg);
    if (kGated) store8(dz + a.inter, c, a.inter, du);
    if (a.y != nullptr) store8(static_cast<T*>(a.y) + r * a.ldy, c, a.inter, y);
}

// per_row: threads of a row, a multiple of 4, so that no group spans two warps
template <typename T, int kKind, bool kGated>
cudaError_t launch_act_t(const ActArgs& a, cudaStream_t stream) {
    const int64_t per_row = (a.inter + 31) / 32 * 4, blocks = (a.rows * per_row + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (a.q != nullptr) act_kernel<T, kKind, kGated, true><<<grid, kThreads, 0, stream>>>(a, per_row);
    else act_kernel<T, kKind, kGated, false><<<grid, kThreads, 0, stream>>>(a, per_row);
    return cudaGetLastError();
}

template <typename T, int kKind, bool kGated>
cudaError_t launch_backward_t(const ActBackwardArgs& a, cudaStream_t stream) {
    const int64_t per_row = (a.inter + 31) / 32 * 4, blocks = (a.rows * per_row + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    act_backward_kernel<T, kKind, kGated><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, per_row);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_activation(const ActArgs& a, bool f32, int kind, bool gated, cudaStream_t stream) {
    if (f32) {
        if (kind == kSilu) return gated ? launch_act_t<float, kSilu, true>(a, stream) : launch_act_t<float, kSilu, false>(a, stream);
        return gated ? launch_act_t<float, kGelu, true>(a, stream) : launch_act_t<float, kGelu, false>(a, stream);
    }
    if (kind == kSilu)
        return gated ? launch_act_t<bf16_bits, kSilu, true>(a, stream) : launch_act_t<bf16_bits, kSilu, false>(a, stream);
    return gated ? launch_act_t<bf16_bits, kGelu, true>(a, stream) : launch_act_t<bf16_bits, kGelu, false>(a, stream);
}

cudaError_t launch_activation_backward(const ActBackwardArgs& a, bool f32, int kind, bool gated, cudaStream_t stream) {
    if (f32) {
        if (kind == kSilu)
            return gated ? launch_backward_t<float, kSilu, true>(a, stream) : launch_backward_t<float, kSilu, false>(a, stream);
        return gated ? launch_backward_t<float, kGelu, true>(a, stream) : launch_backward_t<float, kGelu, false>(a, stream);
    }
    if (kind == kSilu)
        return gated ? launch_backward_t<bf16_bits, kSilu, true>(a, stream) : launch_backward_t<bf16_bits, kSilu, false>(a, stream);
    return gated ? launch_backward_t<bf16_bits, kGelu, true>(a, stream) : launch_backward_t<bf16_bits, kGelu, false>(a, stream);
}

}  // namespace mxq
