// clip.cu -- the norm over all gradients of a step, and the gradients scaled so
// that it does not exceed max_norm:
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + eps)),
//   out = g c.
//
// The tensors' addresses and sizes travel in the kernel's parameters, so nothing is copied
// to the device and the launches can be captured.  The tensors are cut into chunks that the
// blocks of a fixed grid take in turn; each block writes one partial sum, and whoever needs
// the norm adds the partial sums in their order: the result does not depend on
// timing.  (Sums in FP64 cost more than the whole rest of a small call: this GPU adds two doubles
// a clock and SM.)  The scaling blocks take the chunks backwards: what the other pass read last
// still lies in the L2.  Bound by memory: one read for the norm, one read and one write.
// Measured: 36 gradients of 671 MB: the norm 101 us (98% of a copy's 6787 GB/s), scaled too 323 us
// (3 x 671 MB: 92%); 300 ragged ones of 56 MB 16 us and 31 us; 6 of 2.6 MB 5.5 us and 8.2 us.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTable = 1024;   // tensors of one launch at most

// The tensors of one launch.  A launch copies its parameters (28 KB for 1024 tensors
// took 5 us of the host's time) and a block reads them through the constant cache, so there are
// tables of several sizes.
template <int kTable>
struct Table {
    int first[kTable];        // first chunk of the tensor
    const void* in[kTable];
    void* out[kTable];
    int64_t n[kTable];        // elements, negative for FP32
    int count, chunks;
    int chunk_bytes;
};
static_assert(sizeof(Table<kMaxTable>) <= 32000, "a launch's parameters hold 32764 bytes");

// The tensor of chunk c, the largest i with first[i] <= c (empty tensors are not in the table):
// 32 entries at a step, by a whole warp.
template <int kTable>
__device__ __forceinline__ int tensor_of(const Table<kTable>& t, int c) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    if (kTable > 32) {
        const int i = 32 * lane;
        const unsigned below = __ballot_sync(0xFFFFFFFFu, i < t.count && t.first[i < kTable ? i : 0] <= c);
        base = 32 * (31 - __clz(below));
    }
    const int i = base + lane;
    const unsigned below = __ballot_sync(0xFFFFFFFFu, i < t.count && t.first[i < kTable ? i : 0] <= c);
    return base + 31 - __clz(below);
}

__device__ __forceinline__ float block_sum(float v, float* sh) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[threadIdx.x & (kThreads / 32 - 1)];
#pragma unroll
    for (int d = kThreads / 64; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// This thread's share of `vectors` vectors, kBatch loads in flight at a time.
// (16 experts' gradients, 671 MB: 100 us for the norm with 2 and 1216 blocks, 104 with 4 or 8 and 608, 120
// with 608 and no batches.)
constexpr int kBatch = 2;
template <typename L, typename U>
__device__ __forceinline__ void in_batches(int64_t vectors, L load, U use) {
    int64_t i = threadIdx.x;
    for (; i + (kBatch - 1) * kThreads < vectors; i += kBatch * kThreads) {
        uint4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) v[b] = load(i + b * kThreads);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) use(i + b * kThreads, v[b]);
    }
    for (; i < vectors; i += kThreads) use(i, load(i));
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
    f32x2 sum = 0;
    in_batches(vectors, [&](int64_t i) { return reinterpret_cast<const uint4*>(p + head)[i]; },
               [&](int64_t, const uint4 v) {
                   f32x2 f[V / 2];
                   unpack2<T>(v, f);
#pragma unroll
                   for (int c = 0; c < V / 2; ++c) sum = fma2(f[c], f[c], sum);
               });
    float s = lo_of(sum) + hi_of(sum);
    const int64_t tail = head + vectors * V;
    const int64_t i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;   // the ends: fewer than 2 V elements
    if (i < n) {
        const float f = to_float(p[i]);
        s = fmaf(f, f, s);
    }
    return s;
}

template <int kTable>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<kTable> t, float* partial) {
    __shared__ float sh[kThreads / 32];
    float s = 0.0f;
    for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const int i = tensor_of(t, c);
        const bool f32 = t.n[i] < 0;
        const int64_t n = f32 ? -t.n[i] : t.n[i], per = t.chunk_bytes / (f32 ? 4 : 2);
        const int64_t lo = (c - t.first[i]) * per, hi = min(n, lo + per);
        s += f32 ? squares(static_cast<const float*>(t.in[i]), lo, hi)
                 : squares(static_cast<const bf16_bits*>(t.in[i]), lo, hi);
    }
    s = block_sum(s, sh);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the partial sums, by every thread of the block.
__device__ __forceinline__ float norm_of(const float* partial, int parts, float* sh) {
    float s = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    return sqrtf(block_sum(s, sh));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const float* partial, int parts, float* norm) {
    __shared__ float sh[kThreads / 32];
    wait_for_previous();
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
    in_batches(vectors, [&](int64_t i) { return reinterpret_cast<const uint4*>(in + head)[i]; },
               [&](int64_t i, const uint4 v) {
                   f32x2 f[V / 2];
                   unpack2<T>(v, f);
#pragma unroll
                   for (int k = 0; k < V / 2; ++k) f[k] = mul2(f[k], pair(c, c));
                   // not read again: leaves the L2 to the inputs
                   __stcs(reinterpret_cast<uint4*>(out + head) + i, pack2<T>(f));
               });
    const int64_t tail = head + vectors * V;
    const int64_t i = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    if (i < n) out[i] = from_float<T>(to_float(in[i]) * c);
}

template <int kTable>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<kTable> t, const float* partial,
                                                         int parts, float max_norm, float eps, float* norm) {
    __shared__ float sh[kThreads / 32];
    wait_for_previous();
    const float n = norm_of(partial, parts, sh);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    float c = max_norm / (n + eps);
    if (c > 1.0f) c = 1.0f;   // a NaN stays: it shows in every gradient
    // the block's chunks, the last one first
    for (int k = (t.chunks - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) * gridDim.x + blockIdx.x;
         k >= 0 && k < t.chunks; k -= gridDim.x) {
        const int i = tensor_of(t, k);
        const bool f32 = t.n[i] < 0;
        const int64_t size = f32 ? -t.n[i] : t.n[i], per = t.chunk_bytes / (f32 ? 4 : 2);
        const int64_t lo = (k - t.first[i]) * per, hi = min(size, lo + per);
        if (f32) scale(static_cast<const float*>(t.in[i]), static_cast<float*>(t.out[i]), lo, hi, c);
        else scale(static_cast<const bf16_bits*>(t.in[i]), static_cast<bf16_bits*>(t.out[i]), lo, hi, c);
    }
}

// Fills the table with the tensors from `at` on; the first one not taken.
template <int kTable>
int fill(Table<kTable>* t, const ClipTensor* tensors, int count, int at, int chunk_bytes) {
    t->count = 0;
    t->chunks = 0;
    t->chunk_bytes = chunk_bytes;
    for (; at < count && t->count < kTable; ++at) {
        const ClipTensor& g = tensors[at];
        if (g.n == 0) continue;
        const int64_t per = chunk_bytes / (g.f32 ? 4 : 2);
        const int i = t->count++;
        t->in[i] = g.in;
        t->out[i] = g.out;
        t->n[i] = g.f32 ? -g.n : g.n;
        t->first[i] = t->chunks;
        t->chunks += static_cast<int>((g.n + per - 1) / per);
    }
    return at;
}

template <int kTable>
cudaError_t clip_launch(const ClipTensor* tensors, int count, int chunk_bytes, bool scale_too, float max_norm, float eps,
                        float* norm, float* partial, cudaStream_t stream) {
    Table<kTable> t;
    int parts = 0;
    bool whole = false;   // one table held everything: the scaling launch takes the same
    for (int at = 0; at < count || parts == 0;) {
        whole = at == 0;
        at = fill(&t, tensors, count, at, chunk_bytes);
        squares_kernel<kTable><<<kClipBlocks, kThreads, 0, stream>>>(t, partial + parts);
        const cudaError_t e = cudaGetLastError();   // without its sums nothing may be scaled
        if (e != cudaSuccess) return e;
        parts += kClipBlocks;
    }
    if (!scale_too) {
        return launch_behind(norm_kernel, 1, kThreads, 0, stream, partial, parts, norm);
    }
    bool first = true;
    for (int at = 0; at < count || first; first = false) {
        at = whole ? count : fill(&t, tensors, count, at, chunk_bytes);
        const cudaError_t e = launch_behind(scale_kernel<kTable>, kClipBlocks, kThreads, 0, stream, t, partial, parts,
                                            max_norm, eps, first ? norm : nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int clip_partials(int count) {
    const int launches = count <= kMaxTable ? 1 : (count + kMaxTable - 1) / kMaxTable;
    return launches * kClipBlocks;
}

cudaError_t launch_clip(const ClipTensor* tensors, int count, bool scale_too, float max_norm, float eps, float* norm,
                        float* partial, cudaStream_t stream) {
    // Chunks of 4 to 32 KB: small enough that every block has one, large enough that a thread has
    // 8 vectors of 16 bytes of each.
    int64_t bytes = 0;
    for (int i = 0; i < count; ++i) bytes += tensors[i].n * (tensors[i].f32 ? 4 : 2);
    const int chunk = bytes >= 32768ll * kClipBlocks ? 32768 : bytes >= 16384ll * kClipBlocks ? 16384
                      : bytes >= 8192ll * kClipBlocks ? 8192 : 4096;
    auto go = [&](auto table) {
        return clip_launch<table.value>(tensors, count, chunk, scale_too, max_norm, eps, norm, partial, stream);
    };
    if (count <= 32) return go(std::integral_constant<int, 32>{});
    if (count <= 128) return go(std::integral_constant<int, 128>{});
    if (count <= 512) return go(std::integral_constant<int, 512>{});
    return go(std::integral_constant<int, kMaxTable>{});
}

}  // namespace mxq
