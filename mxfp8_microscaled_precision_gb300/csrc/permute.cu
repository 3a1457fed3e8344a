// permute.cu -- rows into expert order and back, around the grouped GEMMs:
// the plan (a stable counting sort of the routed slots by expert), dispatch
// (copies of the tokens' rows in expert order), combine (the weighted sum of a
// token's rows) and the gradients of combine.
//
// A slot (t, j) is the j-th expert of token t; rows[t, j] is its row in expert
// order.  A dropped slot (no expert) has a row too, behind all experts' rows:
// it is given as -1 - row, so that every row is written by exactly one slot and
// nothing needs clearing beforehand.  No floating-point atomics: results do not depend on
// the order in which blocks run.
//
// The row kernels are bound by memory, which they move once.  Measured, of the 6787 GB/s a
// copy reaches: 16384 tokens x 8 slots of 4096 BF16: dispatch 181 us (98%), combine 181 us
// (98%), its backward pass 331 us (the copy's rate); 8191 x 4 of 4097 BF16, off the 16-byte grid: 59 us
// (84%), 74 us (67%), 107 us (83%), where elements one by one took 148, 164 and 206 us.

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace cg = cooperative_groups;

namespace mxq {
namespace {

constexpr int64_t kPlanWords = 50 * 1024;   // of the plan's counts by warp, in words
// Shared memory of a block of the plan at most (1024 experts and the dropped slots).  It is what the kernel's limit
// is set to, whatever a call needs: the limit is the kernel's, and host threads with other shapes launch it too.
constexpr int kPlanBytes = 4 * (kPlanWords + 2 * 1025 + 32);

// ---- plan ------------------------------------------------------------------------

// One cluster counts and places all slots: warp w of the cluster's warps owns
// the slots [w * chunk, (w + 1) * chunk).  Bucket E takes the dropped slots.  Counting
// goes by integer atomics in shared memory; the places keep the slots' order by the set of a warp's
// lanes in each bucket, which the lanes write as bits into a word of the bucket.  Bound by
// the latency of shared memory and of the cluster's barriers: 16384 x 8 slots to 128 experts 9.7 us
// (37 us with a warp-wide match instruction and 8 blocks), 8 x 8 slots 3.3 us.
//
// Shared memory, B = E + 1 words each: hist[warps][B] slots of a warp in a bucket, then
// where its next one goes; lanes[warps][B], zero between steps; count[B] of the
// block; base[B]; 32 for the scan.
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* ids, int64_t slots, int E, int64_t chunk,
                                                    int64_t* offsets, int32_t* rows) {
    extern __shared__ int sh[];
    cg::cluster_group cluster = cg::this_cluster();
    const int B = E + 1;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* hist = sh;
    int* lanes = hist + warps * B;
    int* count = lanes + warps * B;
    int* base = count + B;
    int* scan = base + B;
    const unsigned rank = cluster.block_rank(), blocks = cluster.num_blocks();

    for (int i = threadIdx.x; i < 2 * warps * B; i += blockDim.x) sh[i] = 0;
    __syncthreads();
    const int64_t lo = (static_cast<int64_t>(rank) * warps + warp) * chunk;
    const int64_t hi = min(slots, lo + chunk);
    int* mine = hist + warp * B;
    int* bits = lanes + warp * B;
    auto bucket = [&](int64_t s) {
        const int e = ids[s];
        return e < 0 || e >= E ? E : e;
    };
#pragma unroll 4
    for (int64_t s = lo + lane; s < hi; s += 32) atomicAdd(mine + bucket(s), 1);
    __syncthreads();
    for (int e = threadIdx.x; e < B; e += blockDim.x) {   // exclusive over the block's warps
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) {
            const int n = hist[w * B + e];
            hist[w * B + e] = sum;
            sum += n;
        }
        count[e] = sum;
    }
    cluster.sync();
    // First row of each bucket (a scan over the buckets' totals) plus the slots of the
    // cluster's earlier blocks in it.
    int carry = 0;
    for (int e0 = 0; e0 < B; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int before = 0, total = 0;
        if (e < B) {
            for (unsigned b = 0; b < blocks; ++b) {
                const int n = cluster.map_shared_rank(count, b)[e];
                total += n;
                if (b < rank) before += n;
            }
        }
        int sum = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        int earlier = carry, all = carry;   // the warps before this one, and all
        for (int w = 0; w < warps; ++w) {
            all += scan[w];
            if (w < warp) earlier += scan[w];
        }
        __syncthreads();
        carry = all;
        if (e < B) {
            const int first = earlier + sum - total;
            base[e] = first + before;
            if (rank == 0) offsets[e] = first;   // bucket E starts where the experts' rows end
        }
    }
    cluster.sync();   // base is written, and nobody reads another block's count any more
    int next = lo + lane < hi ? bucket(lo + lane) : -1;
    for (int64_t s0 = lo; s0 < hi; s0 += 32) {
        const int64_t s = s0 + lane;
        const int e = next;
        next = s + 32 < hi ? bucket(s + 32) : -1;
        if (e >= 0) atomicOr(bits + e, 1 << lane);
        __syncwarp();
        unsigned peers = 0;
        int at = 0;
        if (e >= 0) {
            peers = static_cast<unsigned>(bits[e]);
            at = mine[e];
            const int row = base[e] + at + __popc(peers & ((1u << lane) - 1u));
            rows[s] = e == E ? -1 - row : row;
        }
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) {
            mine[e] = at + __popc(peers);
            bits[e] = 0;
        }
        __syncwarp();
    }
}

// ---- rows ------------------------------------------------------------------------

constexpr int kThreads = 256;
constexpr int kRowThreads = 320;   // of dispatch and combine at most

// Where a slot's entry of `rows` points: the row and whether the slot is kept.
// Entries that mxq_moe_plan does not give (a row that does not exist) point nowhere.
struct Place {
    int64_t row;
    bool kept, exists;
};
__device__ __forceinline__ Place place_of(int entry, int64_t slots) {
    const bool kept = entry >= 0;
    const int row = kept ? entry : -1 - entry;
    return {row, kept, row < slots};
}

// a[rows[t, j]] = x[t], zeros for a dropped slot.  Threads of one threadIdx.y have a token; 16 bytes of
// the row per thread, blockIdx.y over the row: x is read once, whatever k.  With kAny
// the vectors are those of the row that is written, shifted out of x's.
template <int kSize, bool kAny>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const unsigned char* x, int64_t ldx, unsigned char* a,
                                                            int64_t lda, int H, const int32_t* rows, int64_t tokens,
                                                            int k) {
    constexpr int V = 16 / kSize;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    const int at = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    const int32_t* r = rows + t * k;
    const int64_t slots = tokens * k;
    const unsigned char* from = x + t * ldx * kSize;
    if constexpr (!kAny) {
        if (at >= H) return;
        const uint4 v = load16<kSize, false>(from, at, H);
        for (int j = 0; j < k; ++j) {
            const Place p = place_of(r[j], slots);
            if (p.exists)
                store16<kSize, false>(a + p.row * lda * kSize, at, H, p.kept ? v : make_uint4(0u, 0u, 0u, 0u));
        }
    } else {
        if (at >= H + V) return;
        // The three blocks of x's row that the vectors of any lead lie in, loaded once (two for every row of a: 66 us
        // instead of 59); what is outside the row is never stored.
        const int lead = lead_of<kSize>(from);
        const bool between = is_between<kSize>(t, tokens, H);
        uint4 part[3];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            const int i = at - lead + (c - 1) * V;
            part[c] = make_uint4(0u, 0u, 0u, 0u);
            if (i < H && i + V > 0) part[c] = load16<kSize, true>(from, i, H, between);
        }
        for (int j = 0; j < k; ++j) {
            const Place p = place_of(r[j], slots);
            if (!p.exists) continue;
            unsigned char* to = a + p.row * lda * kSize;
            const int lead_to = lead_of<kSize>(to);
            const unsigned off = static_cast<unsigned>((V + lead - lead_to) * kSize);   // 1 to 2 V - 1 elements
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (p.kept) v = off < 16 ? shift16(part[0], part[1], off) : shift16(part[1], part[2], off - 16);
            store16<kSize, true>(to, at - lead_to, H, v);
        }
    }
}

// out[t] = sum_j w_j y[rows[t, j]] (w_j = 1 without weights), summed in FP32 in
// the order of j and rounded once.  With kAny the vectors are those of out's row.
template <typename T, bool kAny>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const T* y, int64_t ldy, const int32_t* rows,
                                                           const float* weights, int64_t tokens, int k, T* out,
                                                           int64_t ldo, int H) {
    constexpr int V = kVec16<T>, S = sizeof(T);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (t >= tokens) return;
    const int at = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    T* to = out + t * ldo;
    const int i = kAny ? at - lead_of<S>(to) : at;
    if (i >= H) return;
    const int32_t* r = rows + t * k;
    const int64_t slots = tokens * k;
    f32x2 acc[V / 2] = {};
    // kB rows' loads in flight at a time: 4 on the grid (16384 tokens x 8 rows of 4096 BF16: 180 us, one at a
    // time 203), one off it, where a load is two already (8191 x 4 rows of 4097: 74 us, with 2 82, with 4 124).
    auto add = [&](auto batch, auto load) {
        constexpr int kB = batch.value;
        for (int j0 = 0; j0 < k; j0 += kB) {
            uint4 v[kB];
            float w[kB];
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                // a dropped slot: neither its row of y nor its weight is read
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                w[j] = 0.0f;
                if (j0 + j >= k) continue;
                const Place p = place_of(r[j0 + j], slots);
                if (!p.kept || !p.exists) continue;
                w[j] = weights != nullptr ? weights[t * k + j0 + j] : 1.0f;
                v[j] = load(p.row);
            }
#pragma unroll
            for (int j = 0; j < kB; ++j) {
                f32x2 f[V / 2];
                unpack2<T>(v[j], f);
#pragma unroll
                for (int c = 0; c < V / 2; ++c) acc[c] = fma2(pair(w[j], w[j]), f[c], acc[c]);
            }
        }
    };
    using std::integral_constant;
    if constexpr (!kAny) add(integral_constant<int, 4>{}, [&](int64_t row) { return load16<S, false>(y + row * ldy, i, H); });
    else add(integral_constant<int, 1>{}, [&](int64_t row) {
        return load_shifted<S>(y + row * ldy, i, H, is_between<S>(row, slots, H));
    });
    store16<S, kAny>(to, i, H, pack2<T>(acc));
}

// dy[rows[t, j]] = w_j dout[t], dw_j = <dout[t], y[rows[t, j]]>: one warp per slot, or 1 << shift lanes of it
// for rows of up to 16 vectors (kShort; 16384 tokens x 7 rows of 120 BF16: 20 us, a warp each 28).
// With kAny the vectors are those of dy's row.
template <typename T, bool kAny, bool kShort>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const T* dout, int64_t ldd, const T* y, int64_t ldy,
                                                                    const int32_t* rows, const float* weights, int k,
                                                                    int64_t slots, int shift, T* dy, int64_t lddy,
                                                                    float* dweights, int H) {
    constexpr int V = kVec16<T>, S = sizeof(T);
    if (!kShort) shift = 5;
    const int64_t s = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> shift;
    const int lanes = 1 << shift, lane = threadIdx.x & (lanes - 1), step_by = lanes * V;
    const Place p = s < slots ? place_of(rows[s], slots) : Place{0, false, false};
    T* to = dy + (p.exists ? p.row : 0) * lddy;
    const int first = lane * V - (kAny ? lead_of<S>(to) : 0);
    f32x2 dot = 0;
    if (!p.kept || !p.exists) {
        for (int i = first; p.exists && i < H; i += step_by) store16<S, kAny>(to, i, H, make_uint4(0u, 0u, 0u, 0u));
    } else {
        const T* d = dout + (s / k) * ldd;
        const T* from = y + p.row * ldy;
        const float w = weights[s];
        const f32x2 ww = pair(w, w);
        auto step = [&](int i, const uint4 vg, const uint4 vf) {
            f32x2 g[V / 2], f[V / 2];
            unpack2<T>(vg, g);
            unpack2<T>(vf, f);
#pragma unroll
            for (int c = 0; c < V / 2; ++c) dot = fma2(g[c], f[c], dot);
#pragma unroll
            for (int c = 0; c < V / 2; ++c) g[c] = mul2(g[c], ww);
            store16<S, kAny>(to, i, H, pack2<T>(g));
        };
        // Rows of the same length in buffers of their own start alike: no shift of y's then (8191 x 4 rows of 4097: 107 us,
        // shifting both 122; two vectors in flight, as on the grid, 120).
        const bool alike = kAny && lead_of<S>(from) == lead_of<S>(to);
        int i = first;
        if constexpr (!kAny) {   // two vectors of each row in flight; more, as unrolled loops have them, are slower
                                 // (16384 tokens x 8 rows of 4096: 331 us, unrolled 361)
#pragma unroll 1
            for (; i + step_by < H; i += 2 * step_by) {
                const uint4 g0 = load16<S, false>(d, i, H), f0 = load16<S, false>(from, i, H);
                const uint4 g1 = load16<S, false>(d, i + step_by, H), f1 = load16<S, false>(from, i + step_by, H);
                step(i, g0, f0);
                step(i + step_by, g1, f1);
            }
        }
#pragma unroll 1
        for (; i < H; i += step_by) {
            if constexpr (!kAny) step(i, load16<S, false>(d, i, H), load16<S, false>(from, i, H));
            else if (is_inner<S>(i, H))
                step(i, load_inner<S>(d, i), alike ? *reinterpret_cast<const uint4*>(from + i) : load_inner<S>(from, i));
            else step(i, load_ends<S>(d, i, H), load_ends<S>(from, i, H));
        }
    }
    float total = lo_of(dot) + hi_of(dot);
    for (int half = lanes >> 1; half > 0; half >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, half);
    if (lane == 0 && s < slots) dweights[s] = total;   // 0 for a dropped slot
}

// Whether every row lies on the 16-byte grid in whole vectors.
bool on_grid(int64_t H, size_t size, std::initializer_list<const void*> ptrs,
             std::initializer_list<int64_t> lds) {
    if (H * size % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    for (int64_t ld : lds)
        if (ld * size % 16 != 0) return false;
    return true;
}

// One block per token and per part of its row of 256 vectors; a rest of less than 64
// vectors joins the parts before it (4097 BF16: two parts of 288 threads).  Rows of up to 32 vectors share a
// block of 256 threads, a power of two of them each (16384 tokens x 7 rows of 120 BF16 dispatched: 6.5 us, a warp
// and block each 10.1).  kAny: a row off the grid lies in one vector more.
struct RowGrid {
    dim3 grid, threads;
};
RowGrid row_grid(int64_t tokens, int64_t H, int64_t size, bool any) {
    const int64_t vectors = (H * size + 15) / 16 + (any ? 1 : 0);
    if (vectors <= 32) {
        unsigned threads = 1;
        while (threads < vectors) threads *= 2;
        const unsigned together = 256 / threads;
        return {dim3(static_cast<unsigned>((tokens + together - 1) / together)), dim3(threads, together)};
    }
    int64_t parts = (vectors + 191) / 256;
    if (parts < 1) parts = 1;
    int64_t threads = ((vectors + parts - 1) / parts + 31) / 32 * 32;
    if (parts > 1 && threads < 256) threads = 256;
    return {dim3(static_cast<unsigned>(tokens), static_cast<unsigned>((vectors + threads - 1) / threads)),
            dim3(static_cast<unsigned>(threads))};
}

template <int kSize, bool kAny>
cudaError_t dispatch_launch(const PermuteArgs& a, const void* x, void* out, cudaStream_t stream) {
    const RowGrid g = row_grid(a.tokens, a.H, kSize, kAny);
    dispatch_kernel<kSize, kAny><<<g.grid, g.threads, 0, stream>>>(
        static_cast<const unsigned char*>(x), a.ld_tokens, static_cast<unsigned char*>(out), a.ld_rows, static_cast<int>(a.H),
        a.rows, a.tokens, a.k);
    return cudaGetLastError();
}

template <typename T, bool kAny>
cudaError_t combine_launch(const PermuteArgs& a, const void* y, const float* weights, void* out, cudaStream_t stream) {
    const RowGrid g = row_grid(a.tokens, a.H, sizeof(T), kAny);
    combine_kernel<T, kAny><<<g.grid, g.threads, 0, stream>>>(
        static_cast<const T*>(y), a.ld_rows, a.rows, weights, a.tokens, a.k, static_cast<T*>(out), a.ld_tokens,
        static_cast<int>(a.H));
    return cudaGetLastError();
}

template <typename T, bool kAny>
cudaError_t combine_backward_launch(const PermuteArgs& a, const void* dout, const void* y, int64_t ldy,
                                    const float* weights, void* dy, float* dweights, cudaStream_t stream) {
    const int64_t slots = a.tokens * a.k;
    const int64_t vectors = (a.H * static_cast<int64_t>(sizeof(T)) + 15) / 16 + (kAny ? 1 : 0);
    int shift = 0;   // lanes of a slot: a power of two up to a warp
    while (shift < 5 && (1 << shift) < vectors) ++shift;
    const int64_t per = kThreads >> shift, blocks = (slots + per - 1) / per;
    auto kernel = shift < 5 ? combine_backward_kernel<T, kAny, true> : combine_backward_kernel<T, kAny, false>;
    kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(
        static_cast<const T*>(dout), a.ld_tokens, static_cast<const T*>(y), ldy, a.rows, weights, a.k, slots, shift,
        static_cast<T*>(dy), a.ld_rows, dweights, static_cast<int>(a.H));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_plan(const int32_t* ids, int64_t slots, int experts, int64_t* offsets, int32_t* rows,
                            cudaStream_t stream) {
    // A warp takes 32 slots at least; one block up to 1024 slots, else a cluster of up to 16 (the most
    // that an SM group of this GPU holds).
    const int64_t B = experts + 1;
    int64_t warps = 32, blocks = 16;
    if (warps > kPlanWords / (2 * B)) warps = kPlanWords / (2 * B);
    if (slots <= 32 * warps) {
        blocks = 1;
        warps = (slots + 31) / 32 > 8 ? (slots + 31) / 32 : 8;
    } else {
        while (blocks > 2 && slots <= blocks / 2 * warps * 32) blocks /= 2;
    }
    const int64_t all = blocks * warps;
    const int64_t chunk = ((slots + all - 1) / all + 31) / 32 * 32;
    const size_t smem = sizeof(int) * static_cast<size_t>(2 * warps * B + 2 * B + 32);
    if (smem > 48 * 1024) {   // more than a launch has unasked
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanBytes);
        if (e != cudaSuccess) return e;
    }
    if (blocks > 8) {
        const cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(blocks), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_kernel, ids, slots, experts, chunk, offsets, rows);
}

cudaError_t launch_moe_dispatch(const PermuteArgs& a, bool f32, const void* x, void* out, cudaStream_t stream) {
    const bool grid = on_grid(a.H, f32 ? 4 : 2, {x, out}, {a.ld_tokens, a.ld_rows});
    if (f32) return grid ? dispatch_launch<4, false>(a, x, out, stream) : dispatch_launch<4, true>(a, x, out, stream);
    return grid ? dispatch_launch<2, false>(a, x, out, stream) : dispatch_launch<2, true>(a, x, out, stream);
}

cudaError_t launch_moe_combine(const PermuteArgs& a, bool f32, const void* y, const float* weights, void* out,
                               cudaStream_t stream) {
    const bool grid = on_grid(a.H, f32 ? 4 : 2, {y, out}, {a.ld_tokens, a.ld_rows});
    if (f32) return grid ? combine_launch<float, false>(a, y, weights, out, stream)
                         : combine_launch<float, true>(a, y, weights, out, stream);
    return grid ? combine_launch<bf16_bits, false>(a, y, weights, out, stream)
                : combine_launch<bf16_bits, true>(a, y, weights, out, stream);
}

cudaError_t launch_moe_combine_backward(const PermuteArgs& a, bool f32, const void* dout, const void* y, int64_t ldy,
                                        const float* weights, void* dy, float* dweights, cudaStream_t stream) {
    const bool grid = on_grid(a.H, f32 ? 4 : 2, {dout, y, dy}, {a.ld_tokens, ldy, a.ld_rows});
    if (f32) return grid ? combine_backward_launch<float, false>(a, dout, y, ldy, weights, dy, dweights, stream)
                         : combine_backward_launch<float, true>(a, dout, y, ldy, weights, dy, dweights, stream);
    return grid ? combine_backward_launch<bf16_bits, false>(a, dout, y, ldy, weights, dy, dweights, stream)
                : combine_backward_launch<bf16_bits, true>(a, dout, y, ldy, weights, dy, dweights, stream);
}

}  // namespace mxq
