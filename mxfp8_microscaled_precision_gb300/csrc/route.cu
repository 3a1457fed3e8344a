// route.cu -- routing of tokens to experts: scores, the k best experts of each
// token and their weights (route_kernel), and the gradient of the weights by
// the router's logits (route_backward_kernel).
//
//   s = softmax(x) or 1 / (1 + exp(-x)),  c = s + bias (without a bias the
//   order of c is that of x, and x itself is compared: no rounding decides),
//   ids = the k largest c, largest first, ties to the lowest expert,
//   w_j = scale * s_j  [ / (sum_i s_i + 1e-20) ].
//
// One warp per token: lane l holds the experts [l N, (l + 1) N), N = the next power of
// two of experts / 32, so a lane's logits are one vector, of equal values the
// lowest lane has the lowest expert, and a group of experts is mostly a few neighbouring lanes.  A round of
// the selection is a scan of the lane's registers, the largest key of the warp and a vote
// on who has it.
//
// Bound by instructions, not by memory (some 500 a token of 128 experts; the rounds are a
// chain of reductions).  Measured: 16384 tokens x 128 experts FP32, softmax, top 8: 12 us (the
// logits alone would take 1.4 us), backward 7.5 us (2.6); 8191 x 256 BF16, sigmoid with bias,
// 4 of 8 groups: 12 us, backward 4.1 us; 4096 x 1024 BF16: 12 us and 8.0 us; 4 tokens 2.6 us.
// The first form (an expert every 32, groups scanned by a lane each) took 13.4 us and 22 us.

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr float kRenormEps = 1e-20f;   // keeps a token whose chosen scores are all 0 finite
constexpr int kWarps = 8;              // tokens per block

// Order of choice values as unsigned keys: 0 = out (-inf), 1 = NaN (below every
// number, so that the chosen experts are always distinct and exist), then the
// numbers in ascending order.
constexpr uint32_t kOut = 0u, kNaN = 1u;
__device__ __forceinline__ uint32_t choice_key(float c) {
    if (c != c) return kNaN;
    if (c == -INFINITY) return kOut;
    const uint32_t u = __float_as_uint(c + 0.0f);   // -0 and +0 are equal
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {   // of a key that is not kOut
    return key == kNaN ? __uint_as_float(0x7FC00000u) : __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Score of a group from the keys of its two best values (k1 >= k2).
__device__ __forceinline__ uint32_t group_key(uint32_t k1, uint32_t k2, bool sums) {
    if (!sums || k2 == kOut) return k1;
    const uint32_t key = choice_key(value_of(k1) + value_of(k2));
    return key == kOut ? kNaN : key;   // a sum that overflowed to -inf: the group still has experts
}

__device__ __forceinline__ void keep_two(uint32_t k, uint32_t& k1, uint32_t& k2) {
    const uint32_t low = k < k1 ? k : k1;
    k1 = k < k1 ? k1 : k;
    k2 = low < k2 ? k2 : low;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Largest logit of the token as the softmax subtracts it: 0 if every logit is
// -inf (no expert is eligible then, and exp(-inf) stays 0 instead of NaN).
template <int kN>
__device__ __forceinline__ float softmax_max(const float (&x)[kN]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    return m == -INFINITY ? 0.0f : m;
}

// The lane's kN elements of a row of n from `first` on; `otherwise` past the row.  kVec: whole
// vectors of up to 16 bytes (n a multiple of kN, rows aligned to them); else the row goes
// through the warp's kStage words of shared memory, so that neighbouring lanes read neighbouring
// elements (element e at e + e / kN: no two lanes of a step in one bank).
template <int kN>
constexpr int kStage = 32 * (kN + 1);

template <typename T, int kN, bool kVec>
__device__ __forceinline__ void load_lane(const T* row, int first, int n, float otherwise, float* sh, float (&x)[kN]) {
    if constexpr (!kVec) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = 32 * i + lane;
            sh[e + e / kN] = e < n ? to_float(row[e]) : otherwise;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = sh[lane * (kN + 1) + i];
        __syncwarp();
    } else {
        constexpr int kPer = kN * sizeof(T) >= 16 ? kVec16<T> : kN;   // elements of a load
        struct alignas(kPer * sizeof(T)) Vec {
            T v[kPer];
        };
#pragma unroll
        for (int i = 0; i < kN; i += kPer) {
            Vec v;
            if (first < n) v = *reinterpret_cast<const Vec*>(row + first + i);
#pragma unroll
            for (int c = 0; c < kPer; ++c) x[i + c] = first < n ? to_float(v.v[c]) : otherwise;
        }
    }
}

template <typename T, int kN, bool kVec>
__device__ __forceinline__ void store_lane(T* row, int first, int n, float* sh, const float (&x)[kN]) {
    if constexpr (!kVec) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kN; ++i) sh[lane * (kN + 1) + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = 32 * i + lane;
            if (e < n) row[e] = from_float<T>(sh[e + e / kN]);
        }
    } else if (first < n) {
        constexpr int kPer = kN * sizeof(T) >= 16 ? kVec16<T> : kN;
        struct alignas(kPer * sizeof(T)) Vec {
            T v[kPer];
        };
#pragma unroll
        for (int i = 0; i < kN; i += kPer) {
            Vec v;
#pragma unroll
            for (int c = 0; c < kPer; ++c) v.v[c] = from_float<T>(x[i + c]);
            *reinterpret_cast<Vec*>(row + first + i) = v;
        }
    }
}

template <typename T, int kN, bool kSoftmax, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const T* logits, const RouteArgs a) {
    extern __shared__ uint32_t smem[];
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
    const int E = a.experts, first = lane * kN;
    float x[kN];
    load_lane<T, kN, kVec>(row, first, E, -INFINITY, reinterpret_cast<float*>(smem) + warp * kStage<kN>, x);
    float m = 0.0f, over_z = 1.0f;
    if constexpr (kSoftmax) {
        m = softmax_max(x);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i) z += expf(x[i] - m);   // -inf adds 0
        over_z = 1.0f / warp_sum(z);
    }
    // Score of a logit; a logit of -inf is out whatever its score.
    auto score = [&](float v) { return kSoftmax ? expf(v - m) * over_z : sigmoid(v); };

    // The choice's keys, and the keys that groups are scored by (they differ where sums are formed without a bias).
    const bool sums = a.top2sum != 0, biased = a.bias != nullptr;
    uint32_t key[kN];
    if (biased) {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            key[i] = first + i < E && x[i] != -INFINITY ? choice_key(score(x[i]) + a.bias[first + i]) : kOut;
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) key[i] = choice_key(x[i]);
    }

    if (a.n_group > 1) {
        const int per = E / a.n_group;
        auto by = [&](int i) {
            return sums && !biased && key[i] != kOut ? choice_key(score(x[i])) : key[i];
        };
        const int span = per / kN;   // lanes of a group
        uint32_t gkey = kOut;        // of group `lane`
        if (span * kN == per && (span & (span - 1)) == 0) {
            uint32_t k1 = kOut, k2 = kOut;
#pragma unroll
            for (int i = 0; i < kN; ++i) keep_two(by(i), k1, k2);
            for (int d = 1; d < span; d <<= 1) {   // both lists are this lane's and its partner's: the two best of four
                const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, k1, d), o2 = __shfl_xor_sync(0xFFFFFFFFu, k2, d);
                keep_two(o1, k1, k2);
                keep_two(o2, k1, k2);
            }
            gkey = group_key(k1, k2, sums);
            gkey = __shfl_sync(0xFFFFFFFFu, gkey, (lane * span) & 31);
            if (lane >= a.n_group) gkey = kOut;
        } else {   // through shared memory: lane g scans group g
            uint32_t* sh = smem + warp * kStage<kN>;
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (first + i < E) sh[first + i] = by(i);
            __syncwarp();
            if (lane < a.n_group) {
                uint32_t k1 = kOut, k2 = kOut;
                for (int i = 0; i < per; ++i) keep_two(sh[lane * per + i], k1, k2);
                gkey = group_key(k1, k2, sums);
            }
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
        for (int i = 0; i < kN; ++i) {
            const uint32_t e = first + i;
            if (((stays >> ((e * inv >> 20) & 31u)) & 1u) == 0u) key[i] = kOut;
        }
    }

    // The lane's best, by blocks of up to 4 registers: the place of a chosen expert is the same number
    // of registers into every lane, so one block is scanned again, in all lanes, and the
    // blocks' bests are compared.
    constexpr int kBlock = kN < 4 ? kN : 4, kBlocks = kN / kBlock;
    uint32_t best[kBlocks];
    int at[kBlocks];
    auto scan = [&](int b) {
        best[b] = key[b * kBlock];
        at[b] = b * kBlock;
#pragma unroll
        for (int i = b * kBlock + 1; i < (b + 1) * kBlock; ++i)
            if (key[i] > best[b]) best[b] = key[i], at[b] = i;   // the lowest of equal ones
    };
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) scan(b);
    int chosen = -1;   // of slot `lane`
    for (int j = 0; j < a.topk; ++j) {
        uint32_t mine = best[0];
        int place = at[0];
#pragma unroll
        for (int b = 1; b < kBlocks; ++b)
            if (best[b] > mine) mine = best[b], place = at[b];
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mine);
        if (top == kOut) break;   // nothing left: the remaining slots stay -1
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, mine == top)) - 1;   // the lowest lane: the lowest expert
        const int e = __shfl_sync(0xFFFFFFFFu, first + place, from);
        if (lane == j) chosen = e;
        const int block = (e & (kN - 1)) / kBlock;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            if (block != b) continue;
#pragma unroll
            for (int i = b * kBlock; i < (b + 1) * kBlock; ++i)
                if (first + i == e) key[i] = kOut;
            scan(b);
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
//   ds_j = scale (dw_j - sum_i dw_i s_i / S) / S   (renorm)   or   scale dw_j,
//   sigmoid: dx_j = ds_j s_j (1 - s_j), 0 at experts not chosen;
//   softmax: dx_e = s_e (ds_e [chosen] - sum_j ds_j s_j).
template <typename T, int kN, bool kSoftmax, bool kVec>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(const T* logits, T* dlogits, const RouteBackwardArgs a) {
    extern __shared__ float stage[];   // without kVec
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    if (t >= a.tokens) return;
    const T* row = logits + t * a.ld;
    T* out = dlogits + t * a.ld_out;
    const int E = a.experts, first = lane * kN;
    int id = -1;
    float dw = 0.0f;
    if (lane < a.topk) {
        id = a.ids[t * a.topk + lane];
        if (id < 0 || id >= E) id = -1;
        else dw = a.dweights[t * a.topk + lane];
    }
    const bool any = __any_sync(0xFFFFFFFFu, id >= 0);   // no expert (a padding token): zeros, logits not read
    const float xc = id >= 0 ? to_float(row[id]) : 0.0f;
    float m = 0.0f, over_z = 1.0f;
    float x[kN] = {};
    if (kSoftmax && any) {
        load_lane<T, kN, kVec>(row, first, E, -INFINITY, stage + warp * kStage<kN>, x);
        m = softmax_max(x);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            x[i] = expf(x[i] - m);
            z += x[i];
        }
        over_z = 1.0f / warp_sum(z);
    }
    float s = 0.0f, slope = 0.0f;   // slope: ds/dx of a sigmoid score
    if (id >= 0) {
        if (kSoftmax) {
            s = expf(xc - m) * over_z;
        } else {
            // s (1 - s) = q / (1 + q)^2 with q = exp(-|x|): no cancellation near s = 1
            const float q = expf(-fabsf(xc));
            s = sigmoid(xc);
            slope = q / ((1.0f + q) * (1.0f + q));
        }
    }
    float ds = a.scale * dw;
    if (a.renorm) {
        // the scale comes last and the products are rounded: where one expert is all there is, its share is
        // 1 and the difference 0, whatever a scale that is no power of two would have rounded
        const float total = warp_sum(s) + kRenormEps;
        const float dot = warp_sum(__fmul_rn(dw, s / total));
        ds = a.scale * (dw - dot) / total;
    }
    if (id < 0) ds = 0.0f;
    const float d = kSoftmax ? warp_sum(ds * s) : 0.0f;
    if (kSoftmax && any) {
        const float scale = -over_z * d;
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] *= scale;
    }
    store_lane<T, kN, kVec>(out, first, E, stage + warp * kStage<kN>, x);
    __syncwarp();   // the chosen experts' values replace what the row's pass wrote
    if (id >= 0) out[id] = from_float<T>(kSoftmax ? s * (ds - d) : ds * slope);
}

// f(kN, kVec) for the experts and the alignment of the rows.
template <typename T, typename F>
cudaError_t by_experts(int experts, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds, F f) {
    auto go = [&](auto count) {
        constexpr int kN = count.value;
        constexpr size_t kBytes = kN * sizeof(T) < 16 ? kN * sizeof(T) : 16;
        bool vec = experts % kN == 0;
        for (const void* p : ptrs) vec = vec && reinterpret_cast<uintptr_t>(p) % kBytes == 0;
        for (int64_t ld : lds) vec = vec && ld * sizeof(T) % kBytes == 0;
        return vec ? f(count, std::true_type{}) : f(count, std::false_type{});
    };
    if (experts <= 32) return go(std::integral_constant<int, 1>{});
    if (experts <= 64) return go(std::integral_constant<int, 2>{});
    if (experts <= 128) return go(std::integral_constant<int, 4>{});
    if (experts <= 256) return go(std::integral_constant<int, 8>{});
    if (experts <= 512) return go(std::integral_constant<int, 16>{});
    return go(std::integral_constant<int, 32>{});
}

template <typename T>
cudaError_t route_launch(const void* logits, const RouteArgs& a, bool softmax, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((a.tokens + kWarps - 1) / kWarps);
    const T* x = static_cast<const T*>(logits);
    return by_experts<T>(a.experts, {logits}, {a.ld}, [&](auto n, auto vec) {
        const size_t smem = vec.value && a.n_group == 1 ? 0 : sizeof(uint32_t) * kWarps * kStage<n.value>;
        if (softmax) route_kernel<T, n.value, true, vec.value><<<blocks, 32 * kWarps, smem, stream>>>(x, a);
        else route_kernel<T, n.value, false, vec.value><<<blocks, 32 * kWarps, smem, stream>>>(x, a);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t route_backward_launch(const void* logits, void* dlogits, const RouteBackwardArgs& a, bool softmax,
                                  cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((a.tokens + kWarps - 1) / kWarps);
    const T* x = static_cast<const T*>(logits);
    T* dx = static_cast<T*>(dlogits);
    return by_experts<T>(a.experts, {logits, dlogits}, {a.ld, a.ld_out}, [&](auto n, auto vec) {
        const size_t smem = vec.value ? 0 : sizeof(float) * kWarps * kStage<n.value>;
        if (softmax) route_backward_kernel<T, n.value, true, vec.value><<<blocks, 32 * kWarps, smem, stream>>>(x, dx, a);
        else route_backward_kernel<T, n.value, false, vec.value><<<blocks, 32 * kWarps, smem, stream>>>(x, dx, a);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_route(const void* logits, bool f32, const RouteArgs& a, bool softmax, cudaStream_t stream) {
    return f32 ? route_launch<float>(logits, a, softmax, stream) : route_launch<bf16_bits>(logits, a, softmax, stream);
}

cudaError_t launch_route_backward(const void* logits, void* dlogits, bool f32, const RouteBackwardArgs& a,
                                  bool softmax, cudaStream_t stream) {
    return f32 ? route_backward_launch<float>(logits, dlogits, a, softmax, stream)
               : route_backward_launch<bf16_bits>(logits, dlogits, a, softmax, stream);
}

}  // namespace mxq
