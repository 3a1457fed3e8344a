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
// added in a fixed order.
//
// Bound by memory for long rows and many.  Measured, of the 6787 GB/s a copy reaches:
// forward 16384 x 7168 BF16 79 us (87%), 16384 x 4096 45 us (87%), 32767 x 1000 FP32 41 us
// (94%), 8 x 4096 2.3 us; backward 132 us (79%), 71 us (83%), 73 us (80%).  Rows off the
// 16-byte grid: 8191 x 4097 BF16 forward 48 us (41%), backward 72 us (41%).
//
// kAny: rows that start at any element (mxq_elem.cuh), in vectors of x's rows.  dy and the
// result mostly start like x, as rows of the same length in buffers of their own do; where
// one does not, it goes element by element.  The sums are formed in the same order either way.

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kSMs = 152;
constexpr int kHeldGroups = 16;       // of more than a warp (forward, held parameters): named barriers
// Shared memory at most.  The limits of the kernels are set to these sizes whatever a call needs: a limit
// belongs to the kernel, and host threads with other shapes launch it too.
constexpr int kHeldBytes = 200 * 1024;
constexpr int kRingBytes = 204 * 1024;
constexpr int64_t kShortCols = 512;   // rows up to this long need no ring (backward)

// ---- sums over the threads of a row ---------------------------------------------------
//
// A row belongs to tpr threads: a part of a warp (4 .. 32 lanes), or several
// warps.  Sums are taken in the same order on every call and known to all of them.

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Rows of whole blocks.  sh: 32 floats per call site, not written again before every
// thread of the block has passed another barrier.
__device__ __forceinline__ float row_sum(float v, int tpr, float* sh) {
    if (tpr <= 32) return lanes_sum(v, tpr);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum((threadIdx.x & 31) < (tpr >> 5) ? sh[threadIdx.x & 31] : 0.0f);
}

__device__ __forceinline__ f32x2 warp_sum2(f32x2 v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = add2(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// 1 / sqrt(v): the approximation (2 ulp) and a step of Newton's method.
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v);
    const float better = r * fmaf(-0.5f * v * r, r, 1.5f);
    return v > 0.0f && v < INFINITY ? better : r;   // 0 and infinity: r is exact, the step would be NaN
}

// ---- forward ----------------------------------------------------------------------------

template <int H>
__device__ __forceinline__ f32x2 squares_of(const f32x2 (&f)[H]) {
    f32x2 s = 0;
#pragma unroll
    for (int c = 0; c < H; ++c) s = fma2(f[c], f[c], s);
    return s;
}

// Thread i of a row holds the vectors i, i + tpr, ... (kN of 16 bytes), packed as they
// came: unpacking them in each pass costs less than the registers of 32-bit copies (a ring of
// bulk copies, as in the backward pass, took 96 us where this takes 80).  A block has one row
// (or one for each group of lanes), and the parameters come from the L1.
template <typename T, typename W, int kN>
__global__ void __launch_bounds__(kN == 8 ? 512 : 1024) norm_kernel(const NormArgs a, int tpr) {
    constexpr int V = kVec16<T>, H = V / 2, S = sizeof(T);
    __shared__ float sh[2][32];
    // rows of lanes (a power of two of them) share a block, longer ones have it alone
    const int shift = tpr <= 32 ? 31 - __clz(tpr) : 31;
    const int group = threadIdx.x >> shift, at = threadIdx.x - (group << shift);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (tpr <= 32 ? blockDim.x >> shift : 1) + group;
    const bool live = row < a.rows;
    // Never so, with a block a row; but 8 vectors' loads come out better ordered behind it (3000 x 12288
    // FP32: 55 us, without 61; fewer vectors are 1.5% faster without).
    if (kN == 8 && row - group >= a.rows) return;
    const int first = at * V, cols = live ? static_cast<int>(a.cols) : 0;   // a row past the end loads and stores nothing
    const float inv = 1.0f / static_cast<float>(a.cols);
    const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
    T* y = static_cast<T*>(a.y) + (live ? row : 0) * a.ldy;
    uint4 q[kN];
#pragma unroll
    for (int n = 0; n < kN; ++n) q[n] = load16<S, false>(x, first + n * tpr * V, cols);
    f32x2 sum = 0;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        f32x2 f[H];
        unpack2<T>(q[n], f);
#pragma unroll
        for (int c = 0; c < H; ++c) sum = add2(sum, f[c]);   // elements outside the row are 0
    }
    const float mu = row_sum(lo_of(sum) + hi_of(sum), tpr, sh[0]) * inv;
    const f32x2 minus = pair(-mu, -mu);
    f32x2 sq = 0;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        if (first + n * tpr * V >= cols) continue;
        f32x2 f[H];
        unpack2<T>(q[n], f);
#pragma unroll
        for (int c = 0; c < H; ++c) f[c] = add2(f[c], minus);
        sq = add2(sq, squares_of<H>(f));
    }
    const float r = inverse_root(row_sum(lo_of(sq) + hi_of(sq), tpr, sh[1]) * inv + a.eps);
    if (live && at == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
    const f32x2 rr = pair(r, r);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = first + n * tpr * V;
        if (i >= cols) continue;
        f32x2 f[H], fw[H], fb[H];
        unpack2<T>(q[n], f);
        load_params2<W, V, false>(static_cast<const W*>(a.weight), i, cols, 1.0f, fw);
        load_params2<W, V, false>(static_cast<const W*>(a.shift), i, cols, 0.0f, fb);
#pragma unroll
        for (int c = 0; c < H; ++c) f[c] = fma2(mul2(add2(f[c], minus), rr), fw[c], fb[c]);
        store16<S, false>(y, i, cols, pack2<T>(f));
    }
}

// The same where the parameters cost more than the row: off the grid, where they would have to be
// shifted for every row, and in FP32 beside BF16 rows.  One block an SM keeps them in shared memory (in
// registers they left room for two vectors a thread: 8191 x 513 18.6 us, so 14.6) and walks over its
// rows blockIdx.x, + gridDim.x, ... with groups of tpr threads, a row each.  gridDim.x
// is a multiple of 8 (or a block has one row), so a block's rows all start alike.  FP32 parameters of
// 16384 x 7168 BF16: 150 us from the L1, so 105.  BF16 ones on the grid are faster from the L1 (81 us, so
// 88), where fewer registers and no loop leave the SM more rows.  Bound by instructions (issue slots 63%
// used at 4097 columns) and by the warps of a row that wait for those with its ends; the next row's loads
// before this row's sums change nothing.
template <typename T, typename W, int kN, bool kAny>
__global__ void __launch_bounds__(kN == 8 ? 512 : 1024) norm_held_kernel(const NormArgs a, int tpr) {
    constexpr int V = kVec16<T>, H = V / 2, S = sizeof(T);
    extern __shared__ __align__(16) unsigned char params[];
    __shared__ float sh[kHeldGroups][2][32];
    const int group = threadIdx.x / tpr, at = threadIdx.x - group * tpr, groups = blockDim.x / tpr;
    const int all = static_cast<int>(a.cols);
    const int first = at * V - (kAny ? lead_of<S>(static_cast<const T*>(a.x) + blockIdx.x * a.ldx) : 0);
    const float inv = 1.0f / static_cast<float>(all);
    const ParamSlots<W, V> w(params, at, tpr), b(params + ParamSlots<W, V>::bytes_of(kN, tpr), at, tpr);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int i = first + n * tpr * V;
        if (group != 0) break;
        Params<W, V> p;
        p.template load<kAny>(static_cast<const W*>(a.weight), i, all, 1.0f);
        w.put(n, p);
        p.template load<kAny>(static_cast<const W*>(a.shift), i, all, 0.0f);
        b.put(n, p);
    }
    __syncthreads();
    auto sum_of_row = [&](float v, int place) {   // as row_sum, over the group's threads
        if (tpr <= 32) return lanes_sum(v, tpr);
        v = warp_sum(v);
        float* s = sh[group][place];
        if ((at & 31) == 0) s[at >> 5] = v;
        named_bar_sync(group, tpr);
        return warp_sum((at & 31) < (tpr >> 5) ? s[at & 31] : 0.0f);
    };
    // The groups of a warp walk together: the last turn may find rows for some of them only.
    const int in_warp = tpr < 32 ? group & (32 / tpr - 1) : 0;
    for (int64_t row0 = blockIdx.x + static_cast<int64_t>(group - in_warp) * gridDim.x; row0 < a.rows;
         row0 += static_cast<int64_t>(groups) * gridDim.x) {
        const int64_t row = row0 + static_cast<int64_t>(in_warp) * gridDim.x;
        const bool live = row < a.rows;
        const int cols = live ? all : -V;   // a row past the end loads and stores nothing
        const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx;
        T* y = static_cast<T*>(a.y) + (live ? row : 0) * a.ldy;
        uint4 q[kN];
        const bool between = kAny && is_between<S>(row, a.rows, cols);
#pragma unroll
        for (int n = 0; n < kN; ++n) q[n] = load16<S, kAny>(x, first + n * tpr * V, cols, between);
        f32x2 sum = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            f32x2 f[H];
            unpack2<T>(q[n], f);
#pragma unroll
            for (int c = 0; c < H; ++c) sum = add2(sum, f[c]);   // elements outside the row are 0
        }
        const float mu = sum_of_row(lo_of(sum) + hi_of(sum), 0) * inv;
        const f32x2 minus = pair(-mu, -mu);
        f32x2 sq = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = first + n * tpr * V;
            if (i >= cols) continue;
            f32x2 f[H];
            unpack2<T>(q[n], f);
#pragma unroll
            for (int c = 0; c < H; ++c) f[c] = add2(f[c], minus);
            if (kAny && (i < 0 || i + V > cols)) {   // 0 outside the row
#pragma unroll
                for (int c = 0; c < H; ++c) {
                    const int e = i + 2 * c;
                    f[c] = pair(e >= 0 && e < cols ? lo_of(f[c]) : 0.0f,
                                e + 1 >= 0 && e + 1 < cols ? hi_of(f[c]) : 0.0f);
                }
            }
            sq = add2(sq, squares_of<H>(f));
        }
        const float r = inverse_root(sum_of_row(lo_of(sq) + hi_of(sq), 1) * inv + a.eps);
        if (live && at == 0) {
            a.mean[row] = mu;
            a.rstd[row] = r;
        }
        const f32x2 rr = pair(r, r);
        const bool alike = !kAny || lead_of<S>(y) == lead_of<S>(x);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int i = first + n * tpr * V;
            if (i >= cols) continue;
            f32x2 f[H], fw[H], fb[H];
            unpack2<T>(q[n], f);
            w.get(n, fw);
            b.get(n, fb);
#pragma unroll
            for (int c = 0; c < H; ++c) f[c] = fma2(mul2(add2(f[c], minus), rr), fw[c], fb[c]);
            store16<S, kAny>(y, i, cols, pack2<T>(f), alike);
        }
    }
}

// Rows longer than the registers of a block hold (over 32768 BF16 or 16384 FP32; off the grid also those whose FP32
// parameters beside BF16 rows do not fit the shared memory): element by element, read again in each pass, one block
// per row (2048 x 32767 FP32 212 us, 37% of a copy's rate; 2048 x 25999 BF16 with FP32 parameters 157 us, 20%).
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
    __shared__ float sh[2][32];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    T* y = static_cast<T*>(a.y) + row * a.ldy;
    const W* w = static_cast<const W*>(a.weight);
    const W* b = static_cast<const W*>(a.shift);
    const int cols = static_cast<int>(a.cols);
    const float inv = 1.0f / static_cast<float>(cols);
    float sum = 0.0f, sq = 0.0f;
#pragma unroll 4
    for (int i = threadIdx.x; i < cols; i += blockDim.x) sum += to_float(x[i]);
    const float mu = row_sum(sum, blockDim.x, sh[0]) * inv;
#pragma unroll 4
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
        const float d = to_float(x[i]) - mu;
        sq = fmaf(d, d, sq);
    }
    const float r = inverse_root(row_sum(sq, blockDim.x, sh[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
        a.mean[row] = mu;
        a.rstd[row] = r;
    }
    for (int i = threadIdx.x; i < cols; i += blockDim.x)
        y[i] = from_float<T>(fmaf((to_float(x[i]) - mu) * r, w ? to_float(w[i]) : 1.0f, b ? to_float(b[i]) : 0.0f));
}

// ---- backward ---------------------------------------------------------------------------

// One vector of x and dy: adds to the column sums, and to sum(u), sum(u h) of the row;
// leaves h = (x - mu) r in x and u in g.  rr = (r, r), minus = (-mu, -mu).  The difference comes first: in
// x r - mu r the rounding of mu r stays when the rest cancels (with a mean of 4096 spreads h was off by 1e-4; the
// instruction that it saved is 2% at 16384 x 7168, nothing at other sizes).  Elements outside the row are 0 in dy
// and add nothing.
template <int H>
__device__ __forceinline__ void add_vector(f32x2 (&x)[H], f32x2 (&g)[H], const f32x2 (&w)[H], f32x2 rr, f32x2 minus,
                                           f32x2 (&dw)[H], f32x2 (&db)[H], f32x2& s1, f32x2& s2) {
#pragma unroll
    for (int c = 0; c < H; ++c) {
        x[c] = mul2(add2(x[c], minus), rr);
        dw[c] = fma2(g[c], x[c], dw[c]);
        db[c] = add2(db[c], g[c]);
        g[c] = mul2(g[c], w[c]);
        s1 = add2(s1, g[c]);
        s2 = fma2(g[c], x[c], s2);
    }
}

// dx = u r + (-m1 r) + h (-m2 r) of one vector, in u; c1 = -m1 r, c2 = -m2 r.
template <int H>
__device__ __forceinline__ void dx_vector(const f32x2 (&h)[H], f32x2 (&u)[H], f32x2 rr, f32x2 c1, f32x2 c2) {
#pragma unroll
    for (int c = 0; c < H; ++c) u[c] = fma2(u[c], rr, fma2(h[c], c2, c1));
}

// The column sums of a block: each group of tpr threads leaves its own in shared memory
// ([group][dw, db][kN tpr V], where element e of a row lies at e + lead), and after a
// barrier the block's threads add up the groups' in their order and write them out side by side.  (One group
// after the other onto the same sums took a barrier and 32 dependent additions each: 8191 x 513 32 us, so 23;
// 32767 x 1000 FP32 80 us, so 73; straight to the workspace from one group 2047 x 16384 68 us, so 61.)
template <int kN, int H>
__device__ __forceinline__ void leave_columns(float* meet, int group, int tpr, int at, const f32x2 (&dw)[kN][H],
                                              const f32x2 (&db)[kN][H]) {
    const int all = kN * tpr * 2 * H;
    float* mine = meet + group * 2 * all;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
        for (int c = 0; c < H; c += 2) {
            const int place = (n * tpr + at) * 2 * H + 2 * c;
            *reinterpret_cast<ulonglong2*>(mine + place) = make_ulonglong2(dw[n][c], dw[n][c + 1]);
            *reinterpret_cast<ulonglong2*>(mine + all + place) = make_ulonglong2(db[n][c], db[n][c + 1]);
        }
    }
}

// lead(group): of the group's rows.
template <typename F>
__device__ __forceinline__ void add_columns(const float* meet, int groups, int all, int cols, float* part, F lead) {
    for (int i = threadIdx.x; i < 2 * cols; i += blockDim.x) {
        const bool second = i >= cols;
        const float* of = meet + (second ? all - cols : 0) + i;
        float s = 0.0f;
        for (int g = 0; g < groups; ++g) s += of[g * 2 * all + lead(g)];
        part[i] = s;
    }
}

// Short rows: tpr = 4 .. 32 lanes a row, no barrier per row.  A group's rows are gridDim.x x
// groups apart, a multiple of 8 rows, so they all start alike and the group's threads
// keep their columns.
constexpr int kShortThreads = 256;
template <typename T, typename W, int kN, bool kAny>
__global__ void __launch_bounds__(kShortThreads, 2) norm_backward_short_kernel(const NormBackwardArgs a, int tpr) {
    constexpr int V = kVec16<T>, H = V / 2, S = sizeof(T);
    extern __shared__ __align__(16) float cols_sh[];
    __shared__ int leads[kShortThreads / 4];   // of the groups' rows
    const int shift = 31 - __clz(tpr);   // tpr is a power of two
    const int groups = kShortThreads >> shift;
    const int group = threadIdx.x >> shift, at = threadIdx.x & (tpr - 1);
    const int64_t row_first = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int all = static_cast<int>(a.cols);
    const int first = at * V - (kAny ? lead_of<S>(static_cast<const T*>(a.x) + row_first * a.ldx) : 0);
    const float inv = 1.0f / static_cast<float>(all);
    f32x2 w[kN][H];
#pragma unroll
    for (int n = 0; n < kN; ++n)
        load_params2<W, V, kAny>(static_cast<const W*>(a.weight), first + n * tpr * V, all, 1.0f, w[n]);
    f32x2 dw[kN][H] = {}, db[kN][H] = {};
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups; row0 < a.rows; row0 += step) {
        const int64_t row = row0 + group;
        const bool live = row < a.rows;
        const int64_t at_row = live ? row : 0;
        const int cols = live ? all : -V;   // a row past the end loads and stores nothing
        const T* x = static_cast<const T*>(a.x) + at_row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + at_row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + at_row * a.lddx;
        const bool between = kAny && is_between<S>(row, a.rows, cols);
        uint4 qx[kN], qg[kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            qx[n] = load16<S, kAny>(x, first + n * tpr * V, cols, between);
            if (!kAny || lead_of<S>(dy) == lead_of<S>(x)) qg[n] = load16<S, kAny>(dy, first + n * tpr * V, cols, between);
            else qg[n] = load_ends<S>(dy, first + n * tpr * V, cols);
        }
        const float mu = live ? a.mean[at_row] : 0.0f, r = live ? a.rstd[at_row] : 0.0f;
        const f32x2 rr = pair(r, r), minus = pair(-mu, -mu);
        f32x2 h[kN][H], u[kN][H], s1 = 0, s2 = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            unpack2<T>(qx[n], h[n]);
            unpack2<T>(qg[n], u[n]);
            add_vector<H>(h[n], u[n], w[n], rr, minus, dw[n], db[n], s1, s2);
        }
        const float m1 = lanes_sum(lo_of(s1) + hi_of(s1), tpr) * inv;
        const float m2 = lanes_sum(lo_of(s2) + hi_of(s2), tpr) * inv;
        const f32x2 c1 = pair(-m1 * r, -m1 * r), c2 = pair(-m2 * r, -m2 * r);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            dx_vector<H>(h[n], u[n], rr, c1, c2);
            store16<S, kAny>(dx, first + n * tpr * V, cols, pack2<T>(u[n]), !kAny || lead_of<S>(dx) == lead_of<S>(x));
        }
    }
    leave_columns<kN, H>(cols_sh, group, tpr, at, dw, db);
    if (kAny && at == 0) leads[group] = -first;
    __syncthreads();
    add_columns(cols_sh, groups, kN * tpr * V, all, a.partial + static_cast<int64_t>(blockIdx.x) * 2 * all,
                [&](int g) { return kAny ? leads[g] : 0; });
}

// ---- a ring of rows in shared memory (longer rows) ---------------------------------------
//
// One block an SM reads its rows (row blockIdx.x, + gridDim.x, ...) of x and dy through a
// ring of bulk copies in shared memory, so that some 100 KB an SM are in flight while
// sums are formed.  The block's threads form groups of tpr; its row i belongs to group
// i % groups and lies in stage i % stages.  At the barrier that a group needs for a row's sums
// anyway all its threads have read the row, and one thread copies the row `stages`
// further into that stage.  stages is a multiple of groups: a stage belongs to one
// group, which takes its phases one after the other.  (A group that asked for a phase while the
// one before it, another group's row, was on its way would be answered by the
// parity of the phase before that.)
//
// With kAny a row's copy takes the whole 16-byte blocks that it lies in: inside the
// matrix, as rows lie before and after it; the first and the last row's ends go
// element by element.  The block's rows are gridDim.x apart, a multiple of 8 (or
// there is one row), so they all start alike.

constexpr int kMaxStages = 32;
constexpr int kMaxGroups = 14;               // named barriers: one each, and one for all
constexpr int kRingThreads = 512;
constexpr int kManyThreads = 640;

struct RingBars {
    uint64_t full[kMaxStages];
    int abort_flag;            // a wait ran out
    int stop[kMaxGroups][2];   // it as one thread of a group saw it before the barrier of a row (by parity):
                               // the whole group acts on that
};

// Place of a group in the ring and in the rows.
struct RingPlace {
    int64_t row;
    int stage, phase;
    __device__ __forceinline__ void move(int by, int stages) {   // to the block's row that many further
        row += static_cast<int64_t>(by) * gridDim.x;
        stage += by;
        while (stage >= stages) stage -= stages, phase ^= 1;
    }
};

template <typename T, bool kAny>
struct RowRing {
    const T* src[2];
    int64_t ld[2], rows;
    unsigned char* buf;    // [stages][2][row_bytes]
    RingBars* bars;
    uint32_t full;         // shared address of the mbarriers
    int cols, row_bytes, stages;

    static int64_t bytes_of(int64_t cols) {   // of one row in the ring: the blocks that it can lie in
        return (cols * static_cast<int64_t>(sizeof(T)) + 15) / 16 * 16 + (kAny ? 16 : 0);
    }

    // By all threads; a __syncthreads must follow.  Starts the first copies.
    __device__ __forceinline__ void init(const NormBackwardArgs& a, RingBars* all, unsigned char* memory,
                                         int stage_count) {
        src[0] = static_cast<const T*>(a.x);
        src[1] = static_cast<const T*>(a.dy);
        ld[0] = a.ldx;
        ld[1] = a.lddy;
        rows = a.rows;
        cols = static_cast<int>(a.cols);
        buf = memory;
        bars = all;
        full = smem_u32(bars->full);
        row_bytes = (cols * static_cast<int>(sizeof(T)) + 15) / 16 * 16 + (kAny ? 16 : 0);
        stages = stage_count;
        if (threadIdx.x == 0) bars->abort_flag = 0;
        if (threadIdx.x < stages) {   // stages <= 32: a lane of the first warp each
            mbar_init(full + 8 * threadIdx.x, 1);
            fence_mbar_init();
            const int64_t row = blockIdx.x + static_cast<int64_t>(threadIdx.x) * gridDim.x;
            if (row < rows) fetch(row, threadIdx.x);
        }
    }

    // Copies a row of x and of dy into a stage (one thread).
    __device__ __forceinline__ void fetch(int64_t at, int stage) {
        const bool ends = kAny && (at == 0 || at == rows - 1);
        unsigned char* dst = buf + 2 * stage * row_bytes;
        const unsigned char* from[2];
        uint32_t skip[2], bytes[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const T* row = src[k] + at * ld[k];
            const unsigned char* p = reinterpret_cast<const unsigned char*>(row);
            const uint32_t lead = kAny ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u) : 0u;
            const uint32_t size = static_cast<uint32_t>(cols * static_cast<int>(sizeof(T)));
            uint32_t lo = 0, hi = (lead + size + 15u) & ~15u;   // blocks, from the one that holds the first element
            if (ends) {
                if (lead != 0) lo = 16;
                hi = (lead + size) & ~15u;
                T* to_row = reinterpret_cast<T*>(dst + k * row_bytes + lead);
                const int head = static_cast<int>((lo - (lo ? lead : 0u)) / sizeof(T));
                for (int i = 0; i < head; ++i) to_row[i] = row[i];
                for (int i = static_cast<int>((hi - lead) / sizeof(T)); i < cols; ++i) to_row[i] = row[i];
            }
            from[k] = p - lead + lo;
            skip[k] = lo;
            bytes[k] = hi - lo;
        }
        const uint32_t bar = full + 8 * stage;
        mbar_arrive_expect_tx(bar, bytes[0] + bytes[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) bulk_load(smem_u32(dst + k * row_bytes + skip[k]), from[k], bytes[k], bar);
    }

    // All threads of its group have read a row (the values are in use): its stage takes the row
    // `stages` further.
    __device__ __forceinline__ void refill(int64_t row, int stage) {
        const int64_t next = row + static_cast<int64_t>(stages) * gridDim.x;
        if (next >= rows) return;
        fence_proxy_async_smem();   // the group's accesses to the stage before the copy's writes
        fetch(next, stage);
    }

    // After a wait that ran out, by the first thread of a group that gave up: waits (bounded) for
    // the copies in flight into the group's stages (from p on, every groups-th row; groups = stages: for
    // the row at p alone), as the block must not end before them.
    __device__ __noinline__ void drain(RingPlace p, int groups, const WaitGuard& guard) {
        int again = 0;
        const WaitGuard last{&again, guard.status, guard.limit_ns};
        for (int i = 0; i < stages / groups && p.row < rows; ++i, p.move(groups, stages))
            mbar_wait(full + 8 * p.stage, p.phase, last);
    }

    // False, with abort_flag set, if the row did not arrive in time.
    __device__ __forceinline__ bool wait(const RingPlace& p, const WaitGuard& guard) const {
        return mbar_try_wait(full + 8 * p.stage, p.phase) || mbar_wait(full + 8 * p.stage, p.phase, guard);
    }

    // Vector q of x's row (k = 0) in `stage`, elements [i, i + V), or the same elements of dy's,
    // which starts `lead` elements into its first block and alike or not: 0 outside the row.
    __device__ __forceinline__ uint4 read(int k, int stage, int q, int i, int lead = 0, bool alike = true) const {
        const unsigned char* row = buf + (2 * stage + k) * row_bytes;
        if (kAny && !alike) return load_ends<sizeof(T)>(row + lead * sizeof(T), i, cols);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < cols) v = *reinterpret_cast<const uint4*>(row + 16 * q);
        if (kAny && (i < 0 || i + kVec16<T> > cols)) v = inside<sizeof(T)>(v, i, cols);
        return v;
    }
};

__device__ __forceinline__ void group_barrier(int group, int tpr) {
    if (tpr == 32) __syncwarp();
    else named_bar_sync(1 + group, tpr);
}

// A thread of 16 elements a row (kKeep) keeps h and u of the row between the two passes; a
// longer row is read a second time from the ring: registers hold the column sums.  What
// bounds it: the chain of a row's sums (wait, shuffles, barrier, shuffles) and its arithmetic, some 2200
// clocks, of which 14 to 16 warps of 128 registers fill less than half (issue slots 44% used, DRAM 59%,
// at 8192 x 7168).  Tried at 16384 x 7168 on the form that took 138 us there (132 now): twice the threads with half the
// registers spill and are slower (211 us), as are 8 elements a thread (194 us) and the sums of the next row before the
// results of this one (170 us: two rows' values leave the scheduler no registers); a warp of its own for the
// copies changed nothing; without any loads and stores 118 us remained.  The weights wait in shared memory: in
// registers they took 146 us when that took 142, and from the L1, of which the ring leaves little, 206 us (FP32).
template <typename T, typename W, int kN, bool kAny, int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
norm_backward_kernel(const NormBackwardArgs a, int stages, int tpr) {
    constexpr int V = kVec16<T>, H = V / 2, S = sizeof(T);
    constexpr bool kKeep = kN * V <= 16;
    extern __shared__ __align__(128) unsigned char buf[];   // the weights, then the ring
    __shared__ f32x2 sums[kMaxGroups][2][16];    // [group][row parity][warp]: of u and of u h
    __shared__ float2 stats[kMaxGroups][2];      // mean and rstd of the group's row
    __shared__ __align__(8) RingBars bars;
    const int groups = blockDim.x / tpr, group = threadIdx.x / tpr, at = threadIdx.x - group * tpr;
    const int warp = at >> 5, lane = threadIdx.x & 31;
    RowRing<T, kAny> ring;
    ring.init(a, &bars, buf + ParamSlots<W, V>::bytes_of(kN, tpr), stages);
    for (int i = threadIdx.x; i < kMaxGroups * 2 * 16; i += blockDim.x)
        (&sums[0][0][0])[i] = 0;   // warps that a group does not have
    RingPlace place{blockIdx.x, 0, 0};
    place.move(group, stages);
    const int64_t stride = static_cast<int64_t>(groups) * gridDim.x;
    // A thread of the group's last warp, as the first one has the copies to start, loads mean
    // and rstd two rows ahead.
    const bool ahead = at == tpr - 32;
    auto statistics = [&](int64_t row) {
        return row < a.rows ? make_float2(a.mean[row], a.rstd[row]) : make_float2(0.0f, 0.0f);
    };
    float2 later = make_float2(0.0f, 0.0f);
    if (ahead) {
        stats[group][0] = statistics(place.row);
        later = statistics(place.row + stride);
    }
    const WaitGuard guard{&bars.abort_flag, a.status, kDefaultWaitLimitNs};
    const int cols = static_cast<int>(a.cols);
    const float inv = 1.0f / static_cast<float>(cols);
    const int lead_x = kAny ? lead_of<S>(static_cast<const T*>(a.x) + blockIdx.x * a.ldx) : 0;
    const int lead_g = kAny ? lead_of<S>(static_cast<const T*>(a.dy) + blockIdx.x * a.lddy) : 0;
    const int first = at * V - lead_x;
    const bool alike = lead_g == lead_x;
    const ParamSlots<W, V> w(buf, at, tpr);
#pragma unroll
    for (int n = 0; n < kN; ++n) {   // the same from every group: their rows start alike
        Params<W, V> p;
        p.template load<kAny>(static_cast<const W*>(a.weight), first + n * tpr * V, cols, 1.0f);
        w.put(n, p);
    }
    __syncthreads();
    f32x2 dw[kN][H] = {}, db[kN][H] = {};
    bool stop = false;
    int odd = 0;
    while (place.row < a.rows) {
        const float2 st = stats[group][odd];
        const f32x2 rr = pair(st.y, st.y), minus = pair(-st.x, -st.x);
        if (ahead) {
            bars.stop[group][odd] = *static_cast<volatile int*>(&bars.abort_flag);
            stats[group][odd ^ 1] = later;
            later = statistics(place.row + 2 * stride);
        }
        const bool arrived = ring.wait(place, guard);   // if not, abort_flag is set: the group stops at its next row
        f32x2 h[kKeep ? kN : 1][H], u[kKeep ? kN : 1][H];
        f32x2 s1 = 0, s2 = 0;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int q = n * tpr + at, i = first + n * tpr * V, m = kKeep ? n : 0;
            f32x2 fw[H];
            unpack2<T>(ring.read(0, place.stage, q, i), h[m]);
            unpack2<T>(ring.read(1, place.stage, q, i, lead_g, alike), u[m]);
            w.get(n, fw);
            add_vector<H>(h[m], u[m], fw, rr, minus, dw[n], db[n], s1, s2);
        }
        const f32x2 both = warp_sum2(pair(lo_of(s1) + hi_of(s1), lo_of(s2) + hi_of(s2)));
        if (lane == 0) sums[group][odd][warp] = both;
        group_barrier(group, tpr);
        stop = bars.stop[group][odd] != 0;   // the same for the whole group
        if (stop) break;
        if (kKeep && at == 0 && arrived) ring.refill(place.row, place.stage);   // never into a copy on its way
        f32x2 total = sums[group][odd][lane & 15];
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) total = add2(total, __shfl_xor_sync(0xFFFFFFFFu, total, d));
        const float m1 = -lo_of(total) * inv * st.y, m2 = -hi_of(total) * inv * st.y;
        const f32x2 c1 = pair(m1, m1), c2 = pair(m2, m2);
        T* dx = static_cast<T*>(a.dx) + place.row * a.lddx;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int q = n * tpr + at, i = first + n * tpr * V, m = kKeep ? n : 0;
            if constexpr (!kKeep) {
                f32x2 fw[H];
                unpack2<T>(ring.read(0, place.stage, q, i), h[m]);
                unpack2<T>(ring.read(1, place.stage, q, i, lead_g, alike), u[m]);
                w.get(n, fw);
#pragma unroll
                for (int c = 0; c < H; ++c) {
                    h[m][c] = mul2(add2(h[m][c], minus), rr);
                    u[m][c] = mul2(u[m][c], fw[c]);
                }
            }
            dx_vector<H>(h[m], u[m], rr, c1, c2);
            store16<S, kAny>(dx, i, cols, pack2<T>(u[m]), !kAny || lead_of<S>(dx) == lead_x);
        }
        if constexpr (!kKeep) {   // the row has been read a second time
            group_barrier(group, tpr);
            if (at == 0 && arrived) ring.refill(place.row, place.stage);
        }
        if (at == 0 && !arrived) ring.drain(place, stages, guard);
        place.move(groups, stages);
        odd ^= 1;
    }
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    named_bar_sync(15, groups * tpr);   // in the ring, when all rows have been read
    leave_columns<kN, H>(reinterpret_cast<float*>(buf), group, tpr, at, dw, db);
    named_bar_sync(15, groups * tpr);
    add_columns(reinterpret_cast<const float*>(buf), groups, kN * tpr * V, cols, part, [&](int) { return lead_x; });
    if (stop && at == 0) ring.drain(place, groups, guard);   // the group gave up
}

// The longest rows: element by element.  dw and db by columns, one thread each, over the
// block's rows (their shares in the workspace), then dx from two passes over each row.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormBackwardArgs a) {
    __shared__ float sh[2][32];
    const W* w = static_cast<const W*>(a.weight);
    const int cols = static_cast<int>(a.cols);
    const float inv = 1.0f / static_cast<float>(cols);
    float* part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    for (int i = threadIdx.x; i < cols; i += blockDim.x) {
        float dw = 0.0f, db = 0.0f;
#pragma unroll 4
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
            const float g = to_float(static_cast<const T*>(a.dy)[row * a.lddy + i]);
            dw = fmaf(g, (to_float(static_cast<const T*>(a.x)[row * a.ldx + i]) - a.mean[row]) * a.rstd[row], dw);
            db += g;
        }
        part[i] = dw;
        part[cols + i] = db;
    }
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
        const float mu = a.mean[row], r = a.rstd[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 4
        for (int i = threadIdx.x; i < cols; i += blockDim.x) {
            const float u = to_float(dy[i]) * (w ? to_float(w[i]) : 1.0f);
            s1 += u;
            s2 = fmaf(u, (to_float(x[i]) - mu) * r, s2);
        }
        __syncthreads();   // the sums of the row before, and (dx may be dy) the pass over columns
        const float m1 = row_sum(s1, blockDim.x, sh[0]) * inv, m2 = row_sum(s2, blockDim.x, sh[1]) * inv;
        for (int i = threadIdx.x; i < cols; i += blockDim.x) {
            const float u = to_float(dy[i]) * (w ? to_float(w[i]) : 1.0f);
            dx[i] = from_float<T>(r * (u - m1 - (to_float(x[i]) - mu) * r * m2));
        }
    }
}

// Columns of dw (and of db): 32 columns a block, 32 threads a column that take the
// blocks' shares in turn; a warp adds up the 32 sums of a column.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int parts, int cols, float* dw,
                                                           float* db) {
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    int i = blockIdx.x * 32 + lane;
    float s = 0.0f;
    wait_for_previous();
    if (i < 2 * cols) {
#pragma unroll 5
        for (int p = y; p < parts; p += 32) s += partial[static_cast<int64_t>(p) * 2 * cols + i];
    }
    sh[y][lane] = s;
    __syncthreads();
    s = warp_sum(sh[lane][y]);
    i = blockIdx.x * 32 + y;
    if (lane == 0 && i < 2 * cols) {
        float* out = i < cols ? dw : db;
        if (out != nullptr) out[i < cols ? i : i - cols] = s;
    }
}

// ---- launches ---------------------------------------------------------------------------

// Whether the rows of several tensors all lie on the 16-byte grid in whole vectors.
bool on_grid(int64_t cols, size_t size, std::initializer_list<const void*> ptrs,
             std::initializer_list<int64_t> lds) {
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

// Vectors that a row lies in: one more where x's rows start anywhere.
template <typename T>
int64_t vectors_of(const void* x, int64_t ldx, int64_t cols) {
    return (cols + kVec16<T> - 1) / kVec16<T> + (on_grid(cols, sizeof(T), {x}, {ldx}) ? 0 : 1);
}

template <typename T, typename W, bool kAny>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
    const int64_t vectors = vectors_of<T>(a.x, a.ldx, a.cols);
    constexpr int V = kVec16<T>;
    const bool few = a.rows <= 2 * kSMs;
    const bool hold = kAny || (sizeof(W) > sizeof(T) && !few);
    auto longest = [&] {
        norm_long_kernel<T, W><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
        return cudaGetLastError();
    };
    if (vectors > 8 * 512) return longest();
    // Few rows: 2 vectors a thread (latency).  Many: 4, and 8 for the longest rows, so that
    // several rows share an SM (16384 x 4096 BF16: 52 us with 4, 61 with 8, 72 with 2), but 2 off the grid where 4
    // leave a third more places empty (8191 x 1025: 21 us, with 4 23; 8191 x 4097: 48 with 4, 58 with 2).
    auto places = [&](int64_t k) { return (vectors + 32 * k - 1) / (32 * k) * 32 * k; };
    const int64_t most = few || (kAny && 3 * places(4) >= 4 * places(2)) ? 2 : 4;
    int64_t n = (vectors + 31) / 32;   // vectors of a thread if a warp has the row
    if (n > most) n = most;
    while (n < 8 && vectors > n * 512) n *= 2;
    return by_count<8>(n, [&](auto count) {
        constexpr int kN = count.value;
        int tpr = lanes_of(vectors);
        if (vectors > 32 * kN) tpr = static_cast<int>((vectors + 32 * kN - 1) / (32 * kN)) * 32;
        const int64_t held = 2 * ParamSlots<W, V>::bytes_of(kN, tpr);
        if constexpr (kAny || sizeof(W) > sizeof(T)) {
            if (hold && held <= kHeldBytes) {
                const int64_t grid = a.rows < kSMs ? a.rows : kSMs, rows = (a.rows + grid - 1) / grid;
                int64_t groups = (kN == 8 ? 512 : 1024) / tpr;
                if (tpr > 32 && groups > kHeldGroups) groups = kHeldGroups;
                if (groups > rows) groups = rows;
                const unsigned threads = static_cast<unsigned>((groups * tpr + 31) / 32 * 32);
                auto kernel = norm_held_kernel<T, W, kN, kAny>;
                if (held > 40 * 1024) {   // beside the kernel's own 4 KB more than a launch has unasked
                    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldBytes);
                    if (e != cudaSuccess) return e;
                }
                kernel<<<static_cast<unsigned>(grid), threads, held, stream>>>(a, tpr);
                return cudaGetLastError();
            }
        }
        if constexpr (kAny) {
            return longest();   // FP32 parameters of BF16 rows over 25000 columns
        } else {
            const int threads = tpr <= 32 ? 128 : tpr;
            const int64_t per = threads / tpr;
            norm_kernel<T, W, kN><<<static_cast<unsigned>((a.rows + per - 1) / per), threads, 0, stream>>>(a, tpr);
            return cudaGetLastError();
        }
    });
}

template <typename T, typename W, int kN, bool kAny>
cudaError_t backward_ring(const NormBackwardArgs& a, int64_t vectors, int64_t grid, cudaStream_t stream) {
    constexpr int V = kVec16<T>;
    const int64_t stage = 2 * RowRing<T, kAny>::bytes_of(a.cols);
    const int tpr = static_cast<int>((vectors + 32 * kN - 1) / (32 * kN)) * 32;
    const int64_t weights = ParamSlots<W, V>::bytes_of(kN, tpr);
    int64_t stages = (kRingBytes - weights) / stage;
    if (stages > kMaxStages) stages = kMaxStages;
    const int64_t rows = (a.rows + grid - 1) / grid;
    // as many groups as there are threads for, with two stages each, and none without a row
    auto go = [&](auto kernel, int64_t threads) {
        int64_t groups = threads / tpr;
        if (groups > kMaxGroups) groups = kMaxGroups;
        if (groups > stages / 2) groups = stages / 2;
        if (groups > rows) groups = rows;
        if (groups < 1) groups = 1;
        stages -= stages % groups;
        int64_t bytes = weights + stages * stage;
        const int64_t meet = groups * 2 * kN * tpr * V * static_cast<int64_t>(sizeof(float));   // at most 128 KB
        if (bytes < meet) bytes = meet;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (e != cudaSuccess) return e;
        kernel<<<static_cast<unsigned>(grid), static_cast<unsigned>(tpr * groups), bytes, stream>>>(
            a, static_cast<int>(stages), tpr);
        return cudaGetLastError();
    };
    if constexpr (kN * V <= 16) {
        // Rows that leave a block of 512 threads half empty: two groups of 320 threads, with 96 registers
        // (8192 x 5120 BF16: 51 us, one group of 128 registers 63 us; where 512 threads hold as many groups
        // more registers are faster: 16384 x 4096 71 us against 76).
        if (tpr > kRingThreads / 2 && tpr <= kManyThreads / 2)
            return go(norm_backward_kernel<T, W, kN, kAny, kManyThreads>, kManyThreads);
    }
    return go(norm_backward_kernel<T, W, kN, kAny, kRingThreads>, kRingThreads);
}

template <typename T, typename W, bool kAny>
cudaError_t norm_backward_launch(const NormBackwardArgs& a, cudaStream_t stream) {
    constexpr int V = kVec16<T>;
    const int64_t vectors = vectors_of<T>(a.x, a.ldx, a.cols);
    int64_t parts = norm_partials(a.rows, a.cols);
    cudaError_t e;
    if (a.cols <= kShortCols) {
        constexpr int kMost = 16 / V;   // 16 elements a lane, one vector more for a row off the grid
        const int64_t n = (vectors + 31) / 32;
        auto go = [&](auto count) {
            const int tpr = lanes_of(vectors);
            const int64_t per = kShortThreads / tpr;
            if (parts > (a.rows + per - 1) / per) parts = (a.rows + per - 1) / per;
            if (count.value * V > 8 && parts > 2 * kSMs) parts = 2 * kSMs;   // what the registers leave room for
            const int smem = 2 * count.value * kShortThreads * V * static_cast<int>(sizeof(float));   // at most 48 KB
            auto kernel = norm_backward_short_kernel<T, W, count.value, kAny>;
            if (smem > 40 * 1024) {
                const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
                if (err != cudaSuccess) return err;
            }
            kernel<<<static_cast<unsigned>(parts), kShortThreads, smem, stream>>>(a, tpr);
            return cudaGetLastError();
        };
        e = n <= 1 ? go(std::integral_constant<int, 1>{}) : n <= 2 ? go(std::integral_constant<int, 2>{})
            : n <= kMost ? go(std::integral_constant<int, kMost>{}) : go(std::integral_constant<int, kMost + 1>{});
    } else if (vectors <= kRingThreads * (16 / V)) {
        if (parts > kSMs) parts = kSMs;
        e = backward_ring<T, W, 16 / V, kAny>(a, vectors, parts, stream);
    } else if (vectors <= kRingThreads * (32 / V)) {   // 16384 columns: one stage at least beside the weights
        e = backward_ring<T, W, 32 / V, kAny>(a, vectors, parts, stream);
    } else {   // off the grid from 16384 less a vector's elements on, as such a row lies in one vector more
               // (2048 x 16373 BF16 73 us in the ring, 2048 x 16381 so 288 us, 2048 x 32768 600 us)
        norm_backward_long_kernel<T, W><<<static_cast<unsigned>(parts), 1024, 0, stream>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || (a.dweight == nullptr && a.dshift == nullptr)) return e;
    return launch_behind(norm_reduce_kernel, static_cast<unsigned>((2 * a.cols + 31) / 32), 1024, 0, stream, a.partial,
                         static_cast<int>(parts), static_cast<int>(a.cols), a.dweight, a.dshift);
}

// f(T, W) of the tensors' and the parameters' types.
template <typename F>
cudaError_t by_types(bool f32, bool params_f32, F f) {
    if (f32) return params_f32 ? f(float{}, float{}) : f(float{}, bf16_bits{});
    return params_f32 ? f(bf16_bits{}, float{}) : f(bf16_bits{}, bf16_bits{});
}

}  // namespace

// Blocks of the backward pass at most, each with 2 x cols column sums: one an SM, three for
// the short rows that need no ring, fewer where the sums would take more than 80 MB, but 8 at least
// (512 MB of sums at 2^23 columns).
int64_t norm_partials(int64_t rows, int64_t cols) {
    int64_t most = cols <= kShortCols ? 3 * kSMs : kSMs;
    if (cols > 65536) most = most * 65536 / cols;
    if (most < 8) most = 8;
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
