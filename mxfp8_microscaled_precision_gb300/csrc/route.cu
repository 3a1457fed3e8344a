// route.cu -- routing of tokens to experts: scores, the k best experts of each
// token and their weights (route_kernel), and the gradient of the weights by
// the router's logits (route_backward_kernel).
//
//   s = softmax(x) or 1 / (1 + exp(-x)),  c = s + bias (without a bias the
//   order of c is that of x, and x itself is compared: no rounding decides),
//   ids = the k largest c, largest first, ties to the lowest expert,
//   w_j = scale * s_j  [ / (sum_i s_i + 1e-20) ].
//
// One warp per token: expert e sits in lane e % 32, register e / 32, so loads
// are coalesced for any number of experts, and a round of the selection is a
// scan of the lane's registers and two warp-wide integer reductions (the
// largest key, then the lowest expert that has it).

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr float kRenormEps = 1e-20f;   // keeps a token whose chosen scores are all 0 finite
constexpr int kWarps = 4;              // tokens per block

// Order of choice values as unsigned keys: 0 = out (-inf), 1 = NaN (below every
// number, so that the chosen experts are always distinct and exist), then the
// numbers in ascending order.
constexpr uint32_t kOut = 0u;
__device__ __forceinline__ uint32_t choice_key(float c) {
    if (c != c) return 1u;
    const uint32_t u = __float_as_uint(c + 0.0f);   // -0 and +0 are equal
    const uint32_t key = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return c == -INFINITY ? kOut : key;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Largest logit of the token as the softmax subtracts it: 0 if every logit is
// -inf (no expert is eligible then, and exp(-inf) stays 0 instead of NaN).
template <int kPer>
__device__ __forceinline__ float softmax_max(const float (&x)[kPer]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    return m == -INFINITY ? 0.0f : m;
}

template <typename T, int kPer, bool kSoftmax>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const T* logits, RouteArgs a) {
    extern __shared__ float smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.tokens) return;
    int32_t* ids = a.ids + t * a.topk;
    float* weights = a.weights + t * a.topk;
    if (a.token_mask != nullptr && a.token_mask[t] == 0) {   // a padding token: its logits are not read
        if (lane < a.topk) {
            ids[lane] = -1;
            weights[lane] = 0.0f;
        }
        return;
    }
    const T* row = logits + t * a.ld;
    const int E = a.experts;
    float x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < E ? to_float(row[e]) : -INFINITY;
    }
    float m = 0.0f, z = 1.0f;
    if constexpr (kSoftmax) {
        m = softmax_max(x);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) z += expf(x[i] - m);   // -inf adds 0
        z = warp_sum(z);
    }
    // Score of a logit; a logit of -inf is out whatever its score.
    auto score = [&](float v) { return kSoftmax ? expf(v - m) / z : sigmoid(v); };

    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = lane + 32 * i;
        float c = x[i];
        if (a.bias != nullptr && e < E && x[i] != -INFINITY) c = score(x[i]) + a.bias[e];
        key[i] = choice_key(c);
    }

    if (a.n_group > 1) {
        // Every expert's value to shared memory; lane g scans group g.
        float* sh = smem + warp * E;
        const bool sums = a.top2sum != 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            if (e >= E) continue;
            float c = x[i];
            if (c != -INFINITY && (a.bias != nullptr || sums)) {
                c = score(x[i]);
                if (a.bias != nullptr) c += a.bias[e];
            }
            sh[e] = c;
        }
        __syncwarp();
        const int per = E / a.n_group;
        uint32_t gkey = kOut;
        if (lane < a.n_group) {
            const float* g = sh + lane * per;
            uint32_t k1 = kOut, k2 = kOut;
            float v1 = 0.0f, v2 = 0.0f;
            for (int i = 0; i < per; ++i) {
                const float v = g[i];
                const uint32_t kk = choice_key(v);
                if (kk > k1) {
                    k2 = k1, v2 = v1;
                    k1 = kk, v1 = v;
                } else if (kk > k2) {
                    k2 = kk, v2 = v;
                }
            }
            gkey = k1;
            if (sums && k2 != kOut) gkey = choice_key(v1 + v2);
            if (k1 != kOut && gkey == kOut) gkey = 1u;   // a sum that overflowed to -inf: still has experts
        }
        int before = 0;   // groups that stand before this lane's
        for (int h = 0; h < a.n_group; ++h) {
            const uint32_t other = __shfl_sync(0xFFFFFFFFu, gkey, h);
            before += (other > gkey || (other == gkey && h < lane)) ? 1 : 0;
        }
        const uint32_t stays = __ballot_sync(0xFFFFFFFFu, lane < a.n_group && gkey != kOut && before < a.topk_group);
        // e / per for e < 1024 by a 20-bit reciprocal (exact: e * (error < per) < 2^20)
        const uint32_t inv = ((1u << 20) + per - 1) / per;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t e = lane + 32 * i;
            if (((stays >> ((e * inv >> 20) & 31u)) & 1u) == 0u) key[i] = kOut;
        }
    }

    int chosen = -1;   // of slot `lane`
    for (int j = 0; j < a.topk; ++j) {
        uint32_t best = kOut;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) best = key[i], at = i;   // the lowest of equal ones
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
        if (top == kOut) break;   // nothing left: the remaining slots stay -1
        const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == top ? lane + 32u * at : 0xFFFFFFFFu);
        if (lane == j) chosen = static_cast<int>(e);
        if ((e & 31u) == static_cast<uint32_t>(lane)) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i == static_cast<int>(e >> 5)) key[i] = kOut;
        }
    }
    float s = chosen >= 0 ? score(to_float(row[chosen])) : 0.0f;
    float w = a.scale * s;
    if (a.renorm) w = w / (warp_sum(s) + kRenormEps);
    if (lane < a.topk) {
        ids[lane] = chosen;
        weights[lane] = chosen >= 0 ? w : 0.0f;
    }
}

// dlogits from dweights.  With S = sum_i s_i + 1e-20 over the chosen experts:
//   ds_j = (scale dw_j - sum_i dw_i w_i) / S   (renorm)   or   scale dw_j,
//   sigmoid: dx_j = ds_j s_j (1 - s_j), 0 at experts not chosen;
//   softmax: dx_e = s_e (ds_e [chosen] - sum_j ds_j s_j).
template <typename T, int kPer, bool kSoftmax>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(const T* logits, T* dlogits, RouteBackwardArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.tokens) return;
    const T* row = logits + t * a.ld;
    T* out = dlogits + t * a.ld_out;
    const int E = a.experts;
    int id = -1;
    float dw = 0.0f;
    if (lane < a.topk) {
        id = a.ids[t * a.topk + lane];
        if (id < 0 || id >= E) id = -1;
        else dw = a.dweights[t * a.topk + lane];
    }
    const bool any = __any_sync(0xFFFFFFFFu, id >= 0);   // no expert (a padding token): zeros, logits not read
    const float xc = id >= 0 ? to_float(row[id]) : 0.0f;
    float m = 0.0f, z = 1.0f;
    float x[kPer];
    if (kSoftmax && any) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            x[i] = e < E ? to_float(row[e]) : -INFINITY;
        }
        m = softmax_max(x);
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            x[i] = expf(x[i] - m);
            z += x[i];
        }
        z = warp_sum(z);
    }
    float s = 0.0f, slope = 0.0f;   // slope: ds/dx of a sigmoid score
    if (id >= 0) {
        if (kSoftmax) {
            s = expf(xc - m) / z;
        } else {
            // s (1 - s) = q / (1 + q)^2 with q = exp(-|x|): no cancellation near s = 1
            const float q = expf(-fabsf(xc));
            s = sigmoid(xc);
            slope = q / ((1.0f + q) * (1.0f + q));
        }
    }
    float ds = a.scale * dw;
    if (a.renorm) {
        const float total = warp_sum(s) + kRenormEps;
        const float dot = warp_sum(dw * (a.scale * s / total));
        ds = (a.scale * dw - dot) / total;
    }
    if (id < 0) ds = 0.0f;
    if constexpr (kSoftmax) {
        const float d = warp_sum(ds * s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            if (e < E) out[e] = from_float<T>(any ? -(x[i] / z) * d : 0.0f);
        }
        __syncwarp();   // the chosen experts' values replace what the row's pass wrote
        if (id >= 0) out[id] = from_float<T>(s * (ds - d));
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 32 * i;
            if (e < E) out[e] = from_float<T>(0.0f);
        }
        __syncwarp();
        if (id >= 0) out[id] = from_float<T>(ds * slope);
    }
}

template <typename T, int kPer>
cudaError_t route_launch(const void* logits, const RouteArgs& a, bool softmax, cudaStream_t stream) {
    const int64_t blocks = (a.tokens + kWarps - 1) / kWarps;
    const size_t smem = a.n_group > 1 ? sizeof(float) * kWarps * a.experts : 0;
    const T* x = static_cast<const T*>(logits);
    if (softmax)
        route_kernel<T, kPer, true><<<static_cast<unsigned>(blocks), 32 * kWarps, smem, stream>>>(x, a);
    else
        route_kernel<T, kPer, false><<<static_cast<unsigned>(blocks), 32 * kWarps, smem, stream>>>(x, a);
    return cudaGetLastError();
}

template <typename T, int kPer>
cudaError_t route_backward_launch(const void* logits, void* dlogits, const RouteBackwardArgs& a, bool softmax,
                                  cudaStream_t stream) {
    const int64_t blocks = (a.tokens + kWarps - 1) / kWarps;
    const T* x = static_cast<const T*>(logits);
    T* dx = static_cast<T*>(dlogits);
    if (softmax)
        route_backward_kernel<T, kPer, true><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, stream>>>(x, dx, a);
    else
        route_backward_kernel<T, kPer, false><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, stream>>>(x, dx, a);
    return cudaGetLastError();
}

// The registers of a lane that hold a token's experts: the next power of two.
template <typename F>
cudaError_t by_experts(int experts, F f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const void* logits, bool f32, const RouteArgs& a, bool softmax, cudaStream_t stream) {
    return by_experts(a.experts, [&](auto per) {
        return f32 ? route_launch<float, per.value>(logits, a, softmax, stream)
                   : route_launch<bf16_bits, per.value>(logits, a, softmax, stream);
    });
}

cudaError_t launch_route_backward(const void* logits, void* dlogits, bool f32, const RouteBackwardArgs& a,
                                  bool softmax, cudaStream_t stream) {
    return by_experts(a.experts, [&](auto per) {
        return f32 ? route_backward_launch<float, per.value>(logits, dlogits, a, softmax, stream)
                   : route_backward_launch<bf16_bits, per.value>(logits, dlogits, a, softmax, stream);
    });
}

}  // namespace mxq
