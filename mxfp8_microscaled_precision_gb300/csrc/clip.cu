// clip.cu -- the norm over all gradients of a step, and the gradients scaled so
// that it does not exceed max_norm:
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + eps)),
//   out = g c.
//
// The tensors' addresses and sizes travel in the kernel's parameters (kTable
// tensors a launch), so nothing is copied to the device and the launches can be
// captured.  The tensors are cut into chunks that the blocks of a fixed grid take in turn;
// each block writes one partial sum, and whoever needs the norm adds the
// partial sums in their order: the result does not depend on timing.

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 1024;          // tensors of one launch
constexpr int64_t kChunk = 32768;     // bytes of gradient that a block takes at a time

struct Table {
    const void* in[kTable];
    void* out[kTable];
    int64_t n[kTable];        // elements, negative for FP32
    int first[kTable];        // first chunk of the tensor
    int count;
    int chunks;
};
static_assert(sizeof(Table) <= 32000, "a launch's parameters hold 32764 bytes");

// The tensor of chunk c: the largest i with first[i] <= c (empty tensors have no chunk).
__device__ __forceinline__ int tensor_of(const Table& t, int c) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= c) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum_double(double v, double* sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (lane == 0) sh[warp] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) v += sh[w];
    __syncthreads();
    return v;
}

// Sum of the squares of elements [lo, hi) of a tensor, this thread's share.
// Vectors of 16 bytes from the first aligned element on, the ends one by one.
template <typename T>
__device__ __forceinline__ float squares(const T* p, int64_t lo, int64_t hi) {
    constexpr int V = kVec16<T>;
    p += lo;
    const int64_t n = hi - lo;
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
    if (head > n) head = n;
    const int64_t vectors = (n - head) / V;
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < vectors; i += kThreads) {
        float f[V];
        unpack<T>(*reinterpret_cast<const uint4*>(p + head + i * V), f);
#pragma unroll
        for (int c = 0; c < V; ++c) s = fmaf(f[c], f[c], s);
    }
    const int64_t tail = head + vectors * V;
    const int64_t i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;   // the ends: fewer than 2 V elements
    if (i < n) {
        const float f = to_float(p[i]);
        s = fmaf(f, f, s);
    }
    return s;
}

__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table t, double* partial) {
    __shared__ double sh[kThreads / 32];
    float s = 0.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const bool f32 = t.n[i] < 0;
        const int64_t n = f32 ? -t.n[i] : t.n[i], per = kChunk / (f32 ? 4 : 2);
        const int64_t lo = (c - t.first[i]) * per, hi = min(n, lo + per);
        s += f32 ? squares(static_cast<const float*>(t.in[i]), lo, hi)
                 : squares(static_cast<const bf16_bits*>(t.in[i]), lo, hi);
    }
    const double sum = block_sum_double(s, sh);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The norm from the partial sums, by every thread of the block.
__device__ __forceinline__ float norm_of(const double* partial, int parts, double* sh) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    return static_cast<float>(sqrt(block_sum_double(s, sh)));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* partial, int parts, float* norm) {
    __shared__ double sh[kThreads / 32];
    const float n = norm_of(partial, parts, sh);
    if (threadIdx.x == 0) *norm = n;
}

template <typename T>
__device__ __forceinline__ void scale(const T* in, T* out, int64_t lo, int64_t hi, float c) {
    constexpr int V = kVec16<T>;
    in += lo;
    out += lo;
    const int64_t n = hi - lo;
    if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
        for (int64_t i = threadIdx.x; i < n; i += kThreads) out[i] = from_float<T>(to_float(in[i]) * c);
        return;
    }
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15) / sizeof(T);
    if (head > n) head = n;
    const int64_t vectors = (n - head) / V;
    for (int64_t i = threadIdx.x; i < vectors; i += kThreads) {
        float f[V];
        unpack<T>(*reinterpret_cast<const uint4*>(in + head + i * V), f);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] *= c;
        *reinterpret_cast<uint4*>(out + head + i * V) = pack<T>(f);
    }
    const int64_t tail = head + vectors * V;
    const int64_t i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    if (i < n) out[i] = from_float<T>(to_float(in[i]) * c);
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table t, const double* partial, int parts,
                                                         float max_norm, float eps, float* norm) {
    __shared__ double sh[kThreads / 32];
    const float n = norm_of(partial, parts, sh);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    float c = max_norm / (n + eps);
    if (c > 1.0f) c = 1.0f;   // a NaN stays: it shows in every gradient
    for (int k = blockIdx.x; k < t.chunks; k += gridDim.x) {
        const int i = tensor_of(t, k);
        const bool f32 = t.n[i] < 0;
        const int64_t size = f32 ? -t.n[i] : t.n[i], per = kChunk / (f32 ? 4 : 2);
        const int64_t lo = (k - t.first[i]) * per, hi = min(size, lo + per);
        if (f32) scale(static_cast<const float*>(t.in[i]), static_cast<float*>(t.out[i]), lo, hi, c);
        else scale(static_cast<const bf16_bits*>(t.in[i]), static_cast<bf16_bits*>(t.out[i]), lo, hi, c);
    }
}

// Fills the table with the tensors from `at` on; the first one not taken.
int fill(Table* t, const ClipTensor* tensors, int count, int at) {
    t->count = 0;
    t->chunks = 0;
    for (; at < count && t->count < kTable; ++at) {
        const ClipTensor& g = tensors[at];
        if (g.n == 0) continue;
        const int64_t per = kChunk / (g.f32 ? 4 : 2);
        const int i = t->count++;
        t->in[i] = g.in;
        t->out[i] = g.out;
        t->n[i] = g.f32 ? -g.n : g.n;
        t->first[i] = t->chunks;
        t->chunks += static_cast<int>((g.n + per - 1) / per);
    }
    return at;
}

}  // namespace

int clip_partials(int count) {
    const int launches = count <= kTable ? 1 : (count + kTable - 1) / kTable;
    return launches * kClipBlocks;
}

cudaError_t launch_clip(const ClipTensor* tensors, int count, bool scale_too, float max_norm, float eps, float* norm,
                        double* partial, cudaStream_t stream) {
    Table t;
    int parts = 0;
    for (int at = 0; at < count || parts == 0;) {
        at = fill(&t, tensors, count, at);
        const int grid = kClipBlocks;
        squares_kernel<<<grid, kThreads, 0, stream>>>(t, partial + parts);
        parts += grid;
    }
    if (!scale_too) {
        norm_kernel<<<1, kThreads, 0, stream>>>(partial, parts, norm);
        return cudaGetLastError();
    }
    bool first = true;
    for (int at = 0; at < count || first; first = false) {
        at = fill(&t, tensors, count, at);
        scale_kernel<<<kClipBlocks, kThreads, 0, stream>>>(t, partial, parts, max_norm, eps, first ? norm : nullptr);
    }
    return cudaGetLastError();
}

}  // namespace mxq
