// norm.cu -- layer norm over the rows of a matrix and its backward pass.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r w + b
//   h = (x - mu) r, u = dy w:
//   dx = r (u - mean(u) - h mean(u h)),  dw = sum_rows dy h,  db = sum_rows dy
//
// Forward: a row is held in registers, so the mean and the variance are two
// passes without reading it again, and the variance is that of the centred values
// (no cancellation of mean(x^2) - mu^2).  Backward: a fixed number of blocks
// walks over the rows; a thread owns the same columns in every row and keeps its
// share of dw and db in FP32 registers, the shares meet in a workspace and are
// added in a fixed order.  Both are bound by memory.

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kSMs = 152;
constexpr int64_t kRingBytes = 200 * 1024;   // rows in flight of an SM's blocks (backward)

// ---- sums over the threads of a row ---------------------------------------------------
//
// A row belongs to tpr threads: a part of a warp (4 .. 32 lanes), or the whole
// block.  Sums are taken in the same order on every call and known to all of them.

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// sh: 32 floats per call site, not written again before every thread of the
// block has passed another barrier.
__device__ __forceinline__ float row_sum(float v, int tpr, float* sh) {
    if (tpr <= 32) return lanes_sum(v, tpr);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < (tpr >> 5); ++w) s += sh[w];
    return s;
}

// ---- forward ----------------------------------------------------------------------------

// Thread i of a row holds the vectors i, i + tpr, ... (kN of 16 bytes).
template <typename T, typename W, int kN, bool kAny>
__global__ void __launch_bounds__(kN == 8 ? 512 : 1024) norm_kernel(const NormArgs a, int tpr) {
    constexpr int V = kVec16<T>;
    __shared__ float sh[2][32];
    const int group = threadIdx.x / tpr, at = threadIdx.x % tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + group;
    const bool live = row < a.rows;
    const int64_t cols = live ? a.cols : 0;   // a row past the end loads and stores nothing
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
    T* y = static_cast<T*>(a.y) + (live ? row : 0) * a.ldy;
    const float inv = 1.0f / static_cast<float>(a.cols);
    uint4 q[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) q[n] = load16<sizeof(T), kAny>(x, (n * tpr + at) * V, cols);
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        float f[V];
        unpack<T>(q[n], f);
#pragma unroll
        for (int c = 0; c < V; ++c) sum += f[c];   // elements past the row are 0
    }
    const float mu = row_sum(sum, tpr, sh[0]) * inv;
    float sq = 0.0f;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        float f[V];
        unpack<T>(q[n], f);
        const int64_t i = (n * tpr + at) * V;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            const float d = f[c] - mu;
            if (kAny ? i + c < cols : i < cols) sq = fmaf(d, d, sq);
        }
    }
    const float r = 1.0f / sqrtf(row_sum(sq, tpr, sh[1]) * inv + a.eps);
    if (live && at == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.shift);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int64_t i = (n * tpr + at) * V;
        float f[V], fw[V], fb[V];
        unpack<T>(q[n], f);
        load_params<W, V, kAny>(w, i, cols, 1.0f, fw);
        load_params<W, V, kAny>(b, i, cols, 0.0f, fb);
#pragma unroll
        for (int c = 0; c < V; ++c) f[c] = fmaf((f[c] - mu) * r, fw[c], fb[c]);
        store16<sizeof(T), kAny>(y, i, cols, pack<T>(f), tpr < 32 ? tpr : 32);
    }
}

// Rows longer than the registers of a block hold (512 threads x 8 vectors):
// read again in each pass, one block per row.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    __shared__ float sh[2][32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.shift);
    const float inv = 1.0f / static_cast<float>(a.cols);
    float sum = 0.0f, sq = 0.0f;
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) sum += to_float(x[i]);
    const float mu = row_sum(sum, blockDim.x, sh[0]) * inv;
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
        const float d = to_float(x[i]) - mu;
        sq = fmaf(d, d, sq);
    }
    const float r = 1.0f / sqrtf(row_sum(sq, blockDim.x, sh[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
    for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x)
        y[i] = from_float<T>(fmaf((to_float(x[i]) - mu) * r, w ? to_float(w[i]) : 1.0f, b ? to_float(b[i]) : 0.0f));
}

// ---- backward ---------------------------------------------------------------------------

// One vector of x and dy: adds to the column sums, and to sum(u), sum(u h) of the row.
template <int V>
__device__ __forceinline__ void add_vector(const float (&fx)[V], const float (&g)[V], const float (&fw)[V], float mu,
                                           float r, float (&dw)[V], float (&db)[V], float2& sum) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
        const float h = (fx[c] - mu) * r;
        dw[c] = fmaf(g[c], h, dw[c]);
        db[c] += g[c];
        const float u = g[c] * fw[c];
        sum.x += u;
        sum.y = fmaf(u, h, sum.y);
    }
}

// dx of one vector; m1 = mean(u), m2 = mean(u h).
template <int V>
__device__ __forceinline__ void dx_vector(const float (&fx)[V], float (&g)[V], const float (&fw)[V], float mu, float r,
                                          float m1, float m2) {
#pragma unroll
    for (int c = 0; c < V; ++c) g[c] = r * (g[c] * fw[c] - m1 - (fx[c] - mu) * r * m2);
}

// Short rows (up to 512 elements): tpr = 4 .. 32 lanes a row, no barrier per row.
// The groups' column sums meet by shuffles within a warp and in shared memory over the warps.
constexpr int kShortThreads = 256;
template <typename T, typename W, int kN, bool kAny>
__global__ void __launch_bounds__(kShortThreads, 2) norm_backward_short_kernel(const NormBackwardArgs a, int tpr) {
    constexpr int V = kVec16<T>;
    extern __shared__ float cols_sh[];   // [2][cols]: column sums of the block
    const int per = kShortThreads / tpr;
    const int group = threadIdx.x / tpr, at = threadIdx.x % tpr, lane = threadIdx.x & 31;
    const W* w = static_cast<const W*>(a.weight);
    const float inv = 1.0f / static_cast<float>(a.cols);
    float dw[kN][V] = {}, db[kN][V] = {};
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * per; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        const bool live = row < a.rows;
        const int64_t cols = live ? a.cols : 0, at_row = live ? row : 0;
        const T* x = static_cast<const T*>(a.x) + at_row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + at_row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + at_row * a.lddx;
        uint4 qx[kN], qg[kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            qx[n] = load16<sizeof(T), kAny>(x, (n * tpr + at) * V, cols);
            qg[n] = load16<sizeof(T), kAny>(dy, (n * tpr + at) * V, cols);   // 0 past the row: adds nothing
        }
        // elements past the row, and rows past the end, add nothing: their dy is 0
        const float mu = live ? a.mean[at_row] : 0.0f, r = live ? a.rstd[at_row] : 0.0f;
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            float fx[V], g[V], fw[V];
            unpack<T>(qx[n], fx);
            unpack<T>(qg[n], g);
            load_params<W, V, kAny>(w, (n * tpr + at) * V, a.cols, 1.0f, fw);
            add_vector<V>(fx, g, fw, mu, r, dw[n], db[n], sum);
        }
        const float m1 = lanes_sum(sum.x, tpr) * inv, m2 = lanes_sum(sum.y, tpr) * inv;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            float fx[V], g[V], fw[V];
            unpack<T>(qx[n], fx);
            unpack<T>(qg[n], g);
            load_params<W, V, kAny>(w, (n * tpr + at) * V, a.cols, 1.0f, fw);
            dx_vector<V>(fx, g, fw, mu, r, m1, m2);
            store16<sizeof(T), kAny>(dx, (n * tpr + at) * V, cols, pack<T>(g), tpr);
        }
    }
    // groups of the warp, then the block's warps one after the other
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            for (int d = tpr; d < 32; d <<= 1) {
                dw[n][c] += __shfl_xor_sync(0xFFFFFFFFu, dw[n][c], d);
                db[n][c] += __shfl_xor_sync(0xFFFFFFFFu, db[n][c], d);
            }
        }
    }
    for (int warp = 0; warp < kShortThreads / 32; ++warp) {
        if ((threadIdx.x >> 5) == warp && lane < tpr) {
#pragma unroll
            for (int n = 0; n < kN; ++n) {
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int i = (n * tpr + at) * V + c;
                    if (i < a.cols) {
                        cols_sh[i] = (warp ? cols_sh[i] : 0.0f) + dw[n][c];
                        cols_sh[a.cols + i] = (warp ? cols_sh[a.cols + i] : 0.0f) + db[n][c];
                    }
                }
            }
        }
        __syncthreads();
    }
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    for (int i = threadIdx.x; i < 2 * a.cols; i += kShortThreads) part[i] = cols_sh[i];
}

// Rows of up to 512 threads x kN vectors.  With kRing the rows of x and dy come
// through a ring of `stages` bulk copies in shared memory, so that some 100 KB a
// SM are in flight while a row's sums are formed; without (rows off the 16-byte grid, or
// too long for two stages) they are read from memory.  dx reads a row a second time from there:
// registers hold the column sums.
template <typename T, typename W, int kN, bool kAny, bool kRing>
__global__ void __launch_bounds__(512, kN * kVec16<T> > 16 ? 1 : 2) norm_backward_kernel(const NormBackwardArgs a, int stages) {
    constexpr int V = kVec16<T>;
    extern __shared__ __align__(128) unsigned char ring[];   // [stages][x row, dy row]
    __shared__ float2 sh[2][16];
    __shared__ __align__(8) uint64_t bars[8];
    __shared__ int abort_flag;
    const int tpr = blockDim.x, warp = threadIdx.x >> 5, warps = tpr >> 5;
    const uint32_t bytes = static_cast<uint32_t>(a.cols * sizeof(T));
    const W* w = static_cast<const W*>(a.weight);
    const float inv = 1.0f / static_cast<float>(a.cols);
    const uint32_t bar0 = smem_u32(bars), ring0 = smem_u32(ring);
    const WaitGuard guard{&abort_flag, a.status, kDefaultWaitLimitNs};
    int64_t fetched = blockIdx.x;   // the next row to fetch (thread 0)
    int to = 0;                     // and its stage
    auto fetch = [&]() {
        if (fetched >= a.rows) return;
        const uint32_t bar = bar0 + 8 * to, dst = ring0 + 2 * to * bytes;
        mbar_arrive_expect_tx(bar, 2 * bytes);
        bulk_load(dst, static_cast<const T*>(a.x) + fetched * a.ldx, bytes, bar);
        bulk_load(dst + bytes, static_cast<const T*>(a.dy) + fetched * a.lddy, bytes, bar);
        fetched += gridDim.x;
        if (++to == stages) to = 0;
    };
    if (kRing) {
        if (threadIdx.x == 0) {
            abort_flag = 0;
            for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8 * s, 1);
            fence_mbar_init();
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int s = 0; s < stages; ++s) fetch();
    }
    float dw[kN][V] = {}, db[kN][V] = {};
    int stage = 0, phase = 0;
    bool odd = false;
    float mu = a.mean[blockIdx.x], r = a.rstd[blockIdx.x];
    int64_t row = blockIdx.x;
    for (; row < a.rows; row += gridDim.x) {
        const int64_t after = row + gridDim.x;
        float mu_next = 0.0f, r_next = 0.0f;
        if (after < a.rows) mu_next = a.mean[after], r_next = a.rstd[after];
        const void* x = static_cast<const T*>(a.x) + row * a.ldx;
        const void* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        if (kRing) {
            x = ring + 2 * stage * bytes;
            dy = ring + (2 * stage + 1) * bytes;
            mbar_wait(bar0 + 8 * stage, phase, guard);   // false: abort_flag is set, seen below
        }
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = (n * tpr + static_cast<int>(threadIdx.x)) * V;
            float fx[V], g[V], fw[V];
            unpack<T>(load16<sizeof(T), kAny>(x, i, a.cols), fx);
            unpack<T>(load16<sizeof(T), kAny>(dy, i, a.cols), g);
            load_params<W, V, kAny>(w, i, a.cols, 1.0f, fw);
            add_vector<V>(fx, g, fw, mu, r, dw[n], db[n], sum);
        }
        sum.x = warp_sum(sum.x);
        sum.y = warp_sum(sum.y);
        if ((threadIdx.x & 31) == 0) sh[odd][warp] = sum;
        __syncthreads();   // every thread is done with the row before this one: its stage is free
        if (kRing && abort_flag) break;
        if (kRing && threadIdx.x == 0 && row != blockIdx.x) fetch();
        float m1 = 0.0f, m2 = 0.0f;
        for (int i = 0; i < warps; ++i) {
            m1 += sh[odd][i].x;
            m2 += sh[odd][i].y;
        }
        m1 *= inv;
        m2 *= inv;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = (n * tpr + static_cast<int>(threadIdx.x)) * V;
            float fx[V], g[V], fw[V];
            unpack<T>(load16<sizeof(T), kAny>(x, i, a.cols), fx);
            unpack<T>(load16<sizeof(T), kAny>(dy, i, a.cols), g);
            load_params<W, V, kAny>(w, i, a.cols, 1.0f, fw);
            dx_vector<V>(fx, g, fw, mu, r, m1, m2);
            store16<sizeof(T), kAny>(dx, i, a.cols, pack<T>(g));
        }
        mu = mu_next, r = r_next;
        odd = !odd;
        if (++stage == stages) stage = 0, phase ^= 1;
    }
    if (kRing && abort_flag) {   // a copy did not arrive in time: wait for those in flight (bounded) and give up
        if (threadIdx.x == 0) {
            int again = 0;
            const WaitGuard last{&again, a.status, kDefaultWaitLimitNs};
            for (; row < fetched; row += gridDim.x) {
                mbar_wait(bar0 + 8 * stage, phase, last);
                if (++stage == stages) stage = 0, phase ^= 1;
            }
        }
        return;
    }
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = (n * tpr + static_cast<int>(threadIdx.x)) * V;
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (i + c < a.cols) {
                part[i + c] = dw[n][c];
                part[a.cols + i + c] = db[n][c];
            }
    }
}

// Longer rows: dw and db by columns, one thread each, over the block's rows (their
// shares in the workspace), then dx from two passes over each row.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormBackwardArgs a) {
    __shared__ float sh[2][32];
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
        __syncthreads();   // the sums of the row before, and (dx may be dy) the pass over columns
        const float m1 = row_sum(sum.x, blockDim.x, sh[0]) * inv, m2 = row_sum(sum.y, blockDim.x, sh[1]) * inv;
        for (int64_t i = threadIdx.x; i < a.cols; i += blockDim.x) {
            const float u = to_float(dy[i]) * (w ? to_float(w[i]) : 1.0f);
            dx[i] = from_float<T>(r * (u - m1 - (to_float(x[i]) - mu) * r * m2));
        }
    }
}

// Columns of dw (and of db): 32 columns a block, 8 threads a column that take
// the blocks' shares in turn; their 8 sums are added in order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* partial, int parts, int64_t cols, float* dw,
                                                          float* db) {
    __shared__ float sh[8][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (i < 2 * cols) {
#pragma unroll 8
        for (int p = y; p < parts; p += 8) s += partial[static_cast<int64_t>(p) * 2 * cols + i];
    }
    sh[y][lane] = s;
    __syncthreads();
    if (y == 0 && i < 2 * cols) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += sh[k][lane];
        float* out = i < cols ? dw : db;
        if (out != nullptr) out[i < cols ? i : i - cols] = t;
    }
}

// ---- launches ---------------------------------------------------------------------------

// Whether every row (and the parameters) lies on the 16-byte grid in whole vectors.
bool on_grid(int64_t cols, size_t size, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
    if (cols * size % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    for (int64_t ld : lds)
        if (ld * size % 16 != 0) return false;
    return true;
}

template <int kMost, typename F>
cudaError_t by_count(int64_t n, F f) {   // the smallest of 1, 2, 4, 8 (up to kMost) that is >= n, else kMost
    if (n <= 1) return f(std::integral_constant<int, 1>{});
    if (n <= 2 || kMost == 2) return f(std::integral_constant<int, 2>{});
    if (n <= 4 || kMost == 4) return f(std::integral_constant<int, kMost < 4 ? kMost : 4>{});
    return f(std::integral_constant<int, kMost>{});
}

int lanes_of(int64_t vectors) {   // 4 .. 32 lanes, a power of two
    int lanes = 4;
    while (lanes < 32 && lanes < vectors) lanes *= 2;
    return lanes;
}

template <typename T, typename W, bool kAny>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
    const int64_t vectors = (a.cols + kVec16<T> - 1) / kVec16<T>;
    // Few rows: as many threads to a row as it has vectors for (latency).  Many
    // rows: up to 8 vectors a thread, which keeps 128 bytes a thread in flight and needs few barriers.
    const int64_t most = a.rows <= 2 * kSMs ? 2 : 8;
    if (vectors > 8 * 512) {
        norm_long_kernel<T, W><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
        return cudaGetLastError();
    }
    int64_t n = (vectors + 31) / 32;   // vectors of a thread if a warp has the row
    if (n > most) n = most;
    if (vectors > n * 512) n = (vectors + 511) / 512;
    return by_count<8>(n, [&](auto count) {
        constexpr int kN = count.value;
        int tpr = lanes_of(vectors);
        if (vectors > 32 * kN) tpr = static_cast<int>((vectors + 32 * kN - 1) / (32 * kN)) * 32;
        const int threads = tpr <= 32 ? 128 : tpr;
        const int64_t per = threads / tpr;
        norm_kernel<T, W, kN, kAny><<<static_cast<unsigned>((a.rows + per - 1) / per), threads, 0, stream>>>(a, tpr);
        return cudaGetLastError();
    });
}

template <typename T, typename W, int kN, bool kAny>
cudaError_t backward_short(const NormBackwardArgs& a, int64_t vectors, unsigned grid, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(2 * a.cols) * sizeof(float);
    norm_backward_short_kernel<T, W, kN, kAny><<<grid, kShortThreads, smem, stream>>>(a, lanes_of(vectors));
    return cudaGetLastError();
}

template <typename T, typename W, int kN, bool kAny>
cudaError_t backward_block(const NormBackwardArgs& a, int64_t vectors, int64_t* grid, cudaStream_t stream) {
    const int threads = static_cast<int>((vectors + 32 * kN - 1) / (32 * kN)) * 32;
    const int64_t stage = 2 * a.cols * sizeof(T);
    int64_t blocks = (*grid + kSMs - 1) / kSMs;   // of an SM
    if (!kAny)   // fewer blocks where that makes room for two stages
        while (blocks > 1 && kRingBytes / blocks / stage < 2) --blocks;
    if (*grid > blocks * kSMs) *grid = blocks * kSMs;
    int64_t stages = kRingBytes / blocks / stage;
    if (stages > 8) stages = 8;
    if (!kAny && stages >= 2) {
        auto kernel = norm_backward_kernel<T, W, kN, false, true>;
        const int smem = static_cast<int>(stages * stage);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kernel<<<static_cast<unsigned>(*grid), threads, smem, stream>>>(a, static_cast<int>(stages));
    } else {
        norm_backward_kernel<T, W, kN, kAny, false><<<static_cast<unsigned>(*grid), threads, 0, stream>>>(a, 1);
    }
    return cudaGetLastError();
}

template <typename T, typename W, bool kAny>
cudaError_t norm_backward_launch(const NormBackwardArgs& a, cudaStream_t stream) {
    constexpr int V = kVec16<T>;
    const int64_t vectors = (a.cols + V - 1) / V;
    int64_t parts = norm_partials(a.rows, a.cols);
    cudaError_t e;
    if (a.cols <= 512) {
        constexpr int kMost = 16 / V;   // 16 elements a lane
        e = by_count<kMost>((vectors + 31) / 32, [&](auto count) {
            const int64_t per = kShortThreads / lanes_of(vectors);
            const int64_t cap = count.value * V > 8 ? 2 * kSMs : 3 * kSMs;   // what fits the SMs by registers
            if (parts > cap) parts = cap;
            if (parts > (a.rows + per - 1) / per) parts = (a.rows + per - 1) / per;
            return backward_short<T, W, count.value, kAny>(a, vectors, static_cast<unsigned>(parts), stream);
        });
    } else if (vectors <= 512 * (8 / V)) {   // 8 elements a thread
        e = backward_block<T, W, 8 / V, kAny>(a, vectors, &parts, stream);
    } else if (vectors <= 512 * (16 / V)) {
        e = backward_block<T, W, 16 / V, kAny>(a, vectors, &parts, stream);
    } else if (vectors <= 512 * (32 / V)) {
        e = backward_block<T, W, 32 / V, kAny>(a, vectors, &parts, stream);
    } else {
        norm_backward_long_kernel<T, W><<<static_cast<unsigned>(parts), 1024, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || (a.dweight == nullptr && a.dshift == nullptr)) return e;
    norm_reduce_kernel<<<static_cast<unsigned>((2 * a.cols + 31) / 32), 256, 0, stream>>>(
        a.partial, static_cast<int>(parts), a.cols, a.dweight, a.dshift);
    return cudaGetLastError();
}

// f(T, W) of the tensors' and the parameters' types.
template <typename F>
cudaError_t by_types(bool f32, bool params_f32, F f) {
    if (f32) return params_f32 ? f(float{}, float{}) : f(float{}, bf16_bits{});
    return params_f32 ? f(bf16_bits{}, float{}) : f(bf16_bits{}, bf16_bits{});
}

}  // namespace

// Blocks of the backward pass at most, each with 2 x cols column sums: what fits 1024
// threads of an SM, so that rows of few threads still fill it and the sums stay near
// 10 MB; one a SM for rows whose sums take the registers of 512 threads.
int64_t norm_partials(int64_t rows, int64_t cols) {
    const int64_t held = cols <= 4096 ? 8 : cols <= 8192 ? 16 : 32;   // elements of a row in a thread
    const int64_t threads = (cols + 32 * held - 1) / (32 * held) * 32;
    int64_t per = held == 32 ? 1 : 1024 / (threads < 32 ? 32 : threads);
    if (per > 8) per = 8;
    const int64_t most = per * kSMs;
    return rows < most ? rows : most;
}

cudaError_t launch_layer_norm(const NormArgs& a, bool f32, bool params_f32, cudaStream_t stream) {
    return by_types(f32, params_f32, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        return on_grid(a.cols, sizeof(T), {a.x, a.y, a.weight, a.shift}, {a.ldx, a.ldy})
                   ? norm_launch<T, W, false>(a, stream) : norm_launch<T, W, true>(a, stream);
    });
}

cudaError_t launch_layer_norm_backward(const NormBackwardArgs& a, bool f32, bool params_f32, cudaStream_t stream) {
    return by_types(f32, params_f32, [&](auto t, auto w) {
        using T = decltype(t);
        using W = decltype(w);
        return on_grid(a.cols, sizeof(T), {a.x, a.dy, a.dx, a.weight}, {a.ldx, a.lddy, a.lddx})
                   ? norm_backward_launch<T, W, false>(a, stream) : norm_backward_launch<T, W, true>(a, stream);
    });
}

}  // namespace mxq
