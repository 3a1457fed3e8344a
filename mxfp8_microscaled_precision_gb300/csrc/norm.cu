// norm.cu -- layer norm over the rows of a matrix and its backward pass.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r w + b
//   h = (x - mu) r, u = dy w:
//   dx = r (u - mean(u) - h mean(u h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// The mean and the variance are two passes over a row held in registers: the
// variance is that of the centred values, without the cancellation of
// mean(x^2) - mu^2.

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

// Values of a row that a thread holds at most, and so the longest row of the
// register kernels (1024 threads); longer rows are read again in each pass.
constexpr int kHeld = 32;
constexpr int kMaxHeldCols = 1024 * kHeld;

// Sum over the block, the same order on every call, the result in all threads.
// sh: 33 floats that no earlier call's reader still needs (two barriers inside).
__device__ __forceinline__ float block_sum(float v, float* sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (warps == 1) return v;
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = lane < warps ? sh[lane] : 0.0f;
    v = warp_sum(v);
    __syncthreads();
    return v;
}

__device__ __forceinline__ float2 block_sum2(float2 v, float2* sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (warps == 1) return v;
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = lane < warps ? sh[lane] : make_float2(0.0f, 0.0f);
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    __syncthreads();
    return v;
}

// w[i .. i+V) and the like as floats; `otherwise` where there is no tensor.
template <typename W, int V>
__device__ __forceinline__ void load_param(const W* p, int64_t i, float otherwise, float (&f)[V]) {
#pragma unroll
    for (int c = 0; c < V; ++c) f[c] = p != nullptr ? to_float(p[i + c]) : otherwise;
}

// One row per block.  Thread i holds the vectors i, i + threads, ... of the row.
template <typename T, typename W, int V, int kN>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs a) {
    __shared__ float sh[33];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.shift);
    float v[kN][V];
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
        if (i < a.cols) {
            load_vec<T, V>(x + i, v[n]);
#pragma unroll
            for (int c = 0; c < V; ++c) sum += v[n][c];
        }
    }
    const float mu = block_sum(sum, sh) / static_cast<float>(a.cols);
    float sq = 0.0f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
        if (i < a.cols) {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                v[n][c] -= mu;
                sq = fmaf(v[n][c], v[n][c], sq);
            }
        }
    }
    const float var = block_sum(sq, sh) / static_cast<float>(a.cols);
    const float r = 1.0f / sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
        if (i < a.cols) {
            float fw[V], fb[V];
            load_param<W, V>(w, i, 1.0f, fw);
            load_param<W, V>(b, i, 0.0f, fb);
#pragma unroll
            for (int c = 0; c < V; ++c) v[n][c] = fmaf(v[n][c] * r, fw[c], fb[c]);
            store_vec<T, V>(y + i, v[n]);
        }
    }
}

// Rows longer than the registers hold: read again in each pass.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_long_kernel(NormArgs a) {
    __shared__ float sh[33];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.shift);
    float sum = 0.0f, sq = 0.0f;
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) sum += to_float(x[i]);
    const float mu = block_sum(sum, sh) / static_cast<float>(a.cols);
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
        const float d = to_float(x[i]) - mu;
        sq = fmaf(d, d, sq);
    }
    const float r = 1.0f / sqrtf(block_sum(sq, sh) / static_cast<float>(a.cols) + a.eps);
    if (threadIdx.x == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x)
        y[i] = from_float<T>(fmaf((to_float(x[i]) - mu) * r, w ? to_float(w[i]) : 1.0f, b ? to_float(b[i]) : 0.0f));
}

// Block p takes the rows p, p + grid, ... and keeps its share of dw and db in
// registers (each thread owns the same columns in every row); the shares go to
// the workspace [grid][2][cols] and norm_reduce_kernel adds them up in order.
template <typename T, typename W, int V, int kN>
__global__ void __launch_bounds__(1024) norm_backward_kernel(NormBackwardArgs a) {
    __shared__ float2 sh[33];
    const W* w = static_cast<const W*>(a.weight);
    const float inv = 1.0f / static_cast<float>(a.cols);
    float dw[kN][V] = {}, db[kN][V] = {};
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
        const float mu = a.mean[row], r = a.rstd[row];
        float h[kN][V], u[kN][V];
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
            if (i < a.cols) {
                float fw[V];
                load_vec<T, V>(x + i, h[n]);
                load_vec<T, V>(dy + i, u[n]);
                load_param<W, V>(w, i, 1.0f, fw);
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    h[n][c] = (h[n][c] - mu) * r;
                    dw[n][c] = fmaf(u[n][c], h[n][c], dw[n][c]);
                    db[n][c] += u[n][c];
                    u[n][c] *= fw[c];
                    sum.x += u[n][c];
                    sum.y = fmaf(u[n][c], h[n][c], sum.y);
                }
            }
        }
        sum = block_sum2(sum, sh);
        const float m1 = sum.x * inv, m2 = sum.y * inv;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
            if (i < a.cols) {
#pragma unroll
                for (int c = 0; c < V; ++c) u[n][c] = r * (u[n][c] - m1 - h[n][c] * m2);
                store_vec<T, V>(dx + i, u[n]);
            }
        }
    }
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int64_t i = (static_cast<int64_t>(n) * blockDim.x + threadIdx.x) * V;
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (i + c < a.cols) {
                part[i + c] = dw[n][c];
                part[a.cols + i + c] = db[n][c];
            }
    }
}

// Long rows: dw and db by columns, one thread each, over the block's rows (their
// shares in the workspace), then dx from two passes over each row.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(NormBackwardArgs a) {
    __shared__ float2 sh[33];
    const W* w = static_cast<const W*>(a.weight);
    const float inv = 1.0f / static_cast<float>(a.cols);
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
        float dw = 0.0f, db = 0.0f;
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
            const float g = to_float(static_cast<const T*>(a.dy)[row * a.lddy + i]);
            dw = fmaf(g, (to_float(static_cast<const T*>(a.x)[row * a.ldx + i]) - a.mean[row]) * a.rstd[row], dw);
            db += g;
        }
        part[i] = dw;
        part[a.cols + i] = db;
    }
    __syncthreads();   // dx may be dy itself: the sums by columns have read it
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
        const float mu = a.mean[row], r = a.rstd[row];
        float2 sum = make_float2(0.0f, 0.0f);
        for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
            const float u = to_float(dy[i]) * (w ? to_float(w[i]) : 1.0f);
            sum.x += u;
            sum.y = fmaf(u, (to_float(x[i]) - mu) * r, sum.y);
        }
        sum = block_sum2(sum, sh);
        const float m1 = sum.x * inv, m2 = sum.y * inv;
        for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
            const float u = to_float(dy[i]) * (w ? to_float(w[i]) : 1.0f);
            dx[i] = from_float<T>(r * (u - m1 - (to_float(x[i]) - mu) * r * m2));
        }
    }
}

// Column i of dw (and of db): the blocks' shares in their order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* partial, int parts, int64_t cols, float* dw,
                                                          float* db) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= 2 * cols) return;
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += partial[static_cast<int64_t>(p) * 2 * cols + i];
    float* out = i < cols ? dw : db;
    if (out != nullptr) out[i < cols ? i : i - cols] = s;
}

bool vectors16(int64_t cols, size_t size, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    if (cols * size % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    for (int64_t ld : lds)
        if (ld * size % 16 != 0) return false;
    return true;
}

// f(vector width, vectors per thread) and the threads of a block for a row.
template <typename T, typename F>
cudaError_t by_cols(int64_t cols, bool vec, F f) {
    auto go = [&](auto v, auto n) {
        const int64_t vectors = (cols + v.value - 1) / v.value;
        const int64_t threads = ((vectors + n.value - 1) / n.value + 31) / 32 * 32;
        return f(v, n, static_cast<int>(threads));
    };
    constexpr int kV = kVec16<T>;
    using std::integral_constant;
    if (vec) {
        const int64_t vectors = cols / kV;
        if (vectors <= 512) return go(integral_constant<int, kV>{}, integral_constant<int, 1>{});
        if (vectors <= 1024) return go(integral_constant<int, kV>{}, integral_constant<int, 2>{});
        return go(integral_constant<int, kV>{}, integral_constant<int, kHeld / kV>{});
    }
    if (cols <= 1024) return go(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    if (cols <= 4096) return go(integral_constant<int, 1>{}, integral_constant<int, 8>{});
    return go(integral_constant<int, 1>{}, integral_constant<int, kHeld>{});
}

template <typename T, typename W>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(a.rows);
    if (a.cols > kMaxHeldCols) {
        norm_long_kernel<T, W><<<grid, 1024, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const bool vec = vectors16(a.cols, sizeof(T), {a.x, a.y}, {a.ldx, a.ldy});
    return by_cols<T>(a.cols, vec, [&](auto v, auto n, int threads) {
        norm_kernel<T, W, v.value, n.value><<<grid, threads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

template <typename T, typename W>
cudaError_t norm_backward_launch(const NormBackwardArgs& a, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(norm_partials(a.rows));
    cudaError_t e;
    if (a.cols > kMaxHeldCols) {
        norm_backward_long_kernel<T, W><<<grid, 1024, 0, stream>>>(a);
        e = cudaGetLastError();
    } else {
        const bool vec = vectors16(a.cols, sizeof(T), {a.x, a.dy, a.dx}, {a.ldx, a.lddy, a.lddx});
        e = by_cols<T>(a.cols, vec, [&](auto v, auto n, int threads) {
            norm_backward_kernel<T, W, v.value, n.value><<<grid, threads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    }
    if (e != cudaSuccess || (a.dweight == nullptr && a.dshift == nullptr)) return e;
    norm_reduce_kernel<<<static_cast<unsigned>((2 * a.cols + 255) / 256), 256, 0, stream>>>(
        a.partial, static_cast<int>(grid), a.cols, a.dweight, a.dshift);
    return cudaGetLastError();
}

}  // namespace

int64_t norm_partials(int64_t rows) { return rows < kNormPartials ? rows : kNormPartials; }

cudaError_t launch_layer_norm(const NormArgs& a, bool f32, bool params_f32, cudaStream_t stream) {
    if (f32) return params_f32 ? norm_launch<float, float>(a, stream) : norm_launch<float, bf16_bits>(a, stream);
    return params_f32 ? norm_launch<bf16_bits, float>(a, stream) : norm_launch<bf16_bits, bf16_bits>(a, stream);
}

cudaError_t launch_layer_norm_backward(const NormBackwardArgs& a, bool f32, bool params_f32, cudaStream_t stream) {
    if (f32)
        return params_f32 ? norm_backward_launch<float, float>(a, stream)
                          : norm_backward_launch<float, bf16_bits>(a, stream);
    return params_f32 ? norm_backward_launch<bf16_bits, float>(a, stream)
                      : norm_backward_launch<bf16_bits, bf16_bits>(a, stream);
}

}  // namespace mxq
