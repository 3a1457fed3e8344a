// fp4.cu -- MXFP4 quantization (E2M1 elements, one E8M0 scale per 32) along one or both axes of BF16
// or FP32 matrices, and the values that a microscaled payload stands for.
//
//   e = ceil(log2(amax / 6)) over 32 consecutive elements, -127 at least;  q = E2M1(x 2^-e)
//
// The amax exponent comes from FP32 bits (BF16 is its upper half), the scaling by a power of two is
// exact, one instruction rounds two values to nearest even.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "mxq_elem.cuh"
#include "mxq_internal.h"
#include "mxq_quant_math.cuh"

namespace mxq {
namespace {

constexpr int kTile = 128;
constexpr int kFewTiles = 2;   // on each SM
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight elements of a row, as they are stored.
template <typename T>
struct Eight {
    static constexpr int kWords = sizeof(T) / 2;
    uint4 w[kWords];
    // The elements [c, c + 8) of a row whose neighbourhood is all there.  kVec: rows start on 16 bytes.
    template <bool kVec>
    __device__ __forceinline__ void load_whole(const T* row, int c) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int at = c + i * kVec16<T>;
            w[i] = kVec ? *reinterpret_cast<const uint4*>(row + at) : load_inner<sizeof(T)>(row, at);
        }
    }
    __device__ __forceinline__ void from_shared(const T* p) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void to_shared(T* p) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            float s[kVec16<T>];
            unpack<T>(w[i], s);
#pragma unroll
            for (int j = 0; j < kVec16<T>; ++j) f[i * kVec16<T> + j] = s[j];
        }
    }
    // largest |x|, as FP32 bits
    __device__ __forceinline__ uint32_t amax() const {
        if constexpr (sizeof(T) == 2) {
            return amax8_bits(w[0]) << 16;
        } else {
            float f[8];
            floats(f);
            uint32_t m = abs_bits(f[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) m = max(m, abs_bits(f[i]));
            return m;
        }
    }
    // times 2^-e; the BF16 product is exact, or so small that it converts to a signed zero as the exact one does
    __device__ __forceinline__ void scaled(int e, float (&f)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t s = pow2_neg_bf16(e) * 0x10001u;
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = mul_bf16x2(u[i], s);
                f[2 * i] = bf16_lo(v);
                f[2 * i + 1] = bf16_hi(v);
            }
        } else {
            floats(f);
            const float s = pow2_neg(e);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= s;
        }
    }
};

// Codes of eight elements of a group with a NaN or an infinity: 7 with the sign.
__device__ __forceinline__ uint32_t bad_codes(const float (&f)[8]) {
    uint32_t r = 0x77777777u;
#pragma unroll
    for (int i = 0; i < 8; ++i) r |= (__float_as_uint(f[i]) >> 31) << (4 * i + 3);
    return r;
}

// Codes of a column's 32 rows f, of which the largest |x| has the bits m; *code: the scale.
__device__ __forceinline__ uint4 column_codes(const float (&f)[32], uint32_t m, uint32_t* code) {
    uint32_t o[4];
    if (m >= kInfBits) {
        *code = 0xFFu;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float part[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) part[n] = f[8 * i + n];
            o[i] = bad_codes(part);
        }
    } else {
        const int e = rceil_exponent_f32<kE2M1>(m);
        *code = static_cast<uint32_t>(e + 127);
        const float s = pow2_neg(e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float part[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) part[n] = f[8 * i + n] * s;
            o[i] = cvt_e2m1x8(part);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Shape {
    int tiles_c, per_batch;   // 128 x 128 tiles of a row of tiles and of a matrix
};

// Where 16-byte block `block` (32 rows) of a column of the tile waits to be stored: the blocks of a column take
// turns so that a warp's 32 column pairs do not meet in the same banks.
__device__ __forceinline__ int place_of(int column, int block) { return 4 * column + (block ^ ((column >> 1) & 3)); }

// The four codes of row r's groups g .. g + 3 in the scales of a matrix [rows, 32 groups].
__device__ __forceinline__ void store_codes(uint8_t* out, bool tiled, int64_t r, int64_t rows, int64_t g, int64_t groups,
                                            uint32_t codes) {
    if (tiled) {   // one word of the tile's 512-byte atom; padding is zero
        *reinterpret_cast<uint32_t*>(out + tiled_scale_offset(r, g, groups)) = codes;
    } else if (r < rows) {
        for (int i = 0; i < 4; ++i)
            if (g + i < groups) out[r * groups + g + i] = static_cast<uint8_t>(codes >> (8 * i));
    }
}

// kRows rows r, r + step, .. of `rows` rows of n elements: their elements [c, c + 8), 0 outside the matrix.  What a vector
// load may touch comes first, as many loads in flight as registers hold and nothing between them; then what lies outside
// is cut off; the ends that a vector may not touch (of a matrix's first and last row) come last, element by element.
template <typename T, bool kVec, int kRows>
__device__ __forceinline__ void load_rows(Eight<T> (&v)[kRows], const T* x, int64_t ld, int64_t r, int step, int64_t rows, int c, int n) {
    constexpr int kWords = Eight<T>::kWords, kAtOnce = 2;   // rows of which the loads are in flight
    static_assert(kRows % kAtOnce == 0 || kRows == 1, "rows in groups");
    uint32_t ends = 0;
#pragma unroll
    for (int j0 = 0; j0 < kRows; j0 += kAtOnce) {
        uint4 q[kAtOnce][kWords][2];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int64_t row = r + (j0 + j) * step;
                const int at = c + i * kVec16<T>;
                const bool in = j0 + j < kRows && row < rows && at < n;
                const bool whole = kVec ? at + kVec16<T> <= n : is_between<sizeof(T)>(row, rows, n) || is_inner<sizeof(T)>(at, n);
                const char* p = reinterpret_cast<const char*>(x + (j0 + j) * step * ld + at);
                const uint4* from = reinterpret_cast<const uint4*>(p - (kVec ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15u)));
                q[j][i][0] = q[j][i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (in && whole) q[j][i][0] = from[0];
                if (!kVec && in && whole) q[j][i][1] = from[1];
                if (in && !whole) ends |= 1u << ((j0 + j) * kWords + i);
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if (j0 + j >= kRows) continue;
                const int at = c + i * kVec16<T>;
                const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(x + (j0 + j) * step * ld + at) & 15u);
                v[j0 + j].w[i] = kVec ? q[j][i][0] : inside<sizeof(T)>(shift16(q[j][i][0], q[j][i][1], off), at, n);
            }
        }
    }
    if (ends == 0) return;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (ends >> (j * kWords + i) & 1) v[j].w[i] = load_ends<sizeof(T)>(x + j * step * ld, c + i * kVec16<T>, n);
    }
}

// Codes of a thread's eight elements and the scale code of their group, which four neighbouring threads hold.
template <typename T>
__device__ __forceinline__ uint32_t group_codes(const Eight<T>& v, uint32_t* code) {
    uint32_t m = v.amax();
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    float f[8];
    if (m >= kInfBits) {
        *code = 0xFFu;
        v.floats(f);
        return bad_codes(f);
    }
    const int e = rceil_exponent_f32<kE2M1>(m);
    *code = static_cast<uint32_t>(e + 127);
    v.scaled(e, f);
    return cvt_e2m1x8(f);
}

// Whether a tile's elements, and of rows that start anywhere the 16 bytes around each row's part, lie in the matrix.
template <bool kVec>
__device__ __forceinline__ bool is_whole(int64_t rows, int64_t cols, int64_t r0, int height, int64_t c0, int width) {
    return c0 + width <= cols && (kVec ? r0 + height <= rows : r0 > 0 && r0 + height < rows);
}

// Row copy alone: 64 rows (FP32: 32; few rows: 8) of 256 elements a block.  A warp has a row of it at a time, eight elements a lane, and
// stores its 128 bytes of payload together; all loads of a thread are issued before the first is used.
// Bound by memory: 131072 x 4096 BF16 210 us (95% of the copy rate), 16384 x 7168 FP32 77 us, 16381 x 7167 BF16 65 us (68%).
constexpr int kColTile = 256;
template <typename T>
constexpr int kRowTile = 128 / static_cast<int>(sizeof(T));
// Few rows: blocks of 8 rows, a row a warp, as long as one wave holds them (8 blocks on each SM, of which GB300 has 152).  Such calls are
// bound by latency, the fetching of instructions in it.  Measured, tall blocks / these (us, in a graph): 1 x 7168 BF16
// 2.4 / 1.4, 64 x 4096 2.5 / 1.5, 64 x 4099 5.1 / 1.8, 512 x 4096 3.8 / 2.9, 1024 x 4096 (two waves) 3.9 / 4.6.
constexpr int kFewRows = 8, kFewBlocks = 8;

template <typename T, bool kVec, int kHeight>
__global__ void __launch_bounds__(kThreads, 4) quant_rows_kernel(const Quant4Args a, const Shape s) {
    __shared__ uint32_t s_codes[kHeight][2];   // four scale codes of every row and 128 columns
    __shared__ int64_t s_at[kHeight];          // grouped: the row in the scales, -1: none
    let_next_start();
    wait_for_previous();
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int b = static_cast<int>(blockIdx.x) / s.per_batch, local = static_cast<int>(blockIdx.x) - b * s.per_batch;
    const int tr = local / s.tiles_c, tc = local - tr * s.tiles_c;
    const int64_t r0 = static_cast<int64_t>(tr) * kHeight, c0 = static_cast<int64_t>(tc) * kColTile;
    const int64_t groups = (a.cols + 31) >> 5;
    const T* x = static_cast<const T*>(a.x) + b * a.batch_stride + (r0 + w) * a.ld;
    constexpr int kPer = kHeight / 8;   // rows of a warp
    Eight<T> v[kPer];
    if (is_whole<kVec>(a.rows, a.cols, r0, kHeight, c0, kColTile)) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j].template load_whole<kVec>(x + 8 * j * a.ld, static_cast<int>(c0) + 8 * lane);
    } else {
        load_rows<T, kVec, kPer>(v, x, a.ld, r0 + w, 8, a.rows, static_cast<int>(c0) + 8 * lane, static_cast<int>(a.cols));
    }
    const int64_t live = a.offsets != nullptr ? min(a.rows, a.offsets[a.G]) : a.rows;   // rows that are written
    if (a.offsets != nullptr && t < kHeight) {   // tiled by expert: its first row starts a band
        const int64_t r = r0 + t;
        int lo = 0, hi = a.G;   // the last expert that starts at or before the row
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.offsets[mid] <= r) lo = mid; else hi = mid;
        }
        const int64_t first = a.offsets[lo], end = a.offsets[lo + 1], at = (first / kTile + lo) * kTile + (r - first);
        s_at[t] = r < a.rows && first >= 0 && r >= first && r < end && at < a.bands_cap * kTile ? at : -1;
    }
    const int64_t g = (c0 >> 5) + (lane >> 2);
    uint8_t* q = static_cast<uint8_t*>(a.q_row) + (b * a.rows + r0 + w) * groups * 16 + c0 / 2 + 4 * lane;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int64_t r = r0 + w + 8 * j;
        uint32_t code;
        const uint32_t o = group_codes(v[j], &code);
        const bool in = r < live && g < groups;
        if (in) *reinterpret_cast<uint32_t*>(q + 8 * j * groups * 16) = o;
        if ((lane & 3) == 0)
            reinterpret_cast<uint8_t*>(s_codes[w + 8 * j])[lane >> 2] = in ? static_cast<uint8_t>(code) : 0;
    }
    __syncthreads();
    const int row = t >> 1, part = t & 1;
    const int64_t first = (c0 >> 5) + 4 * part;   // of the four groups
    uint8_t* out = static_cast<uint8_t*>(a.s_row) + b * a.s_row_bytes;
    if (first >= groups) return;
    if (t < 2 * kHeight) {
        if (a.offsets == nullptr) store_codes(out, a.tiled, r0 + row, a.rows, first, groups, s_codes[row][part]);
        else if (s_at[row] >= 0) store_codes(out, true, s_at[row], 0, first, groups, s_codes[row][part]);
    } else if (kHeight == kFewRows && a.offsets == nullptr && a.tiled && r0 + kHeight >= a.rows) {
        // the last rows: no block of their own for the padding up to 128
        if (r0 + row < (a.rows + kTile - 1) / kTile * kTile) store_codes(out, true, r0 + row, 0, first, groups, 0u);
    }
}

// Column copy, alone or with the row copy: a 128 x 128 tile in shared memory, its loads in flight at once (rows that start
// on 16 bytes: without passing registers), several blocks on an SM.  Rows: a thread takes a group of 32 of a row (FP32:
// eight elements, four threads a group).  Columns: a thread takes 32 rows of a column (BF16: of two
// neighbouring ones, in packed operations), and the payload goes out through shared memory, 64 bytes of a
// column together.
// FP32: 512 threads where the tiles are few, since a tile is long work; of many tiles more fit an SM with 256.  Both copies
// with 256 / 512 threads (us, in a graph): 2048 x 2048 (256 tiles) 6.9 / 5.4, 777 x 2085 7.8 / 6.2, 4096 x 1280 (320 tiles)
// 6.9 / 7.7, 4096 x 4096 14.8 / 17.0.
// Rows that start anywhere: FP32 by asynchronous copies of single elements, which need no shift and no ends (4099 x 1111:
// 6.4 us, 8.5 us by shifted vectors); BF16 by vectors shifted in registers (6.5 us).
// Bound by memory, with both copies nearly by instructions too (73% of the issue slots): 16384 x 7168 BF16 63 us (84%
// of the copy rate), the column copy alone 47 us (93%); 131072 x 4096 272 us (89%) and 203 us (99%).
// kExperts (column copy alone): the rows of each expert as a slot of their own.
template <typename T, bool kRow, bool kVec, bool kExperts, int kNT>
__global__ void __launch_bounds__(kNT, sizeof(T) == 2 ? 4 : 2) quant_tile_kernel(const Quant4Args a, const Shape s) {
    constexpr int kStep = kNT / 16, kPasses = kTile / kStep;   // rows of 16 threads each at once
    extern __shared__ __align__(16) uint8_t s_memory[];
    T* tile = reinterpret_cast<T*>(s_memory);
    uint4* s_out = reinterpret_cast<uint4*>(s_memory + kTile * kTile * sizeof(T));
    __shared__ uint32_t s_row_codes[kTile], s_col_codes[kTile];   // four scale codes of every row and column
    let_next_start();
    wait_for_previous();
    const int t = threadIdx.x;
    const int b = static_cast<int>(blockIdx.x) / s.per_batch, local = static_cast<int>(blockIdx.x) - b * s.per_batch;
    const int tr = local / s.tiles_c, tc = local - tr * s.tiles_c;
    const int64_t c0 = static_cast<int64_t>(tc) * kTile;
    const int64_t row_groups = (a.cols + 31) >> 5;
    // rows [r0, rows) of the matrix, as the column copy's groups g0 .. of col_groups
    int64_t r0 = static_cast<int64_t>(tr) * kTile, rows = a.rows, g0 = r0 >> 5, col_groups = (a.rows + 31) >> 5;
    if constexpr (kExperts) {   // band tr of the experts: whose it is, all of them asked at once
        __shared__ int s_expert;
        if (threadIdx.x == 0) s_expert = -1;
        __syncthreads();
        for (int g = threadIdx.x; g < a.G; g += kNT) {
            const int64_t lo = a.offsets[g], hi = a.offsets[g + 1], band = lo / kTile + g;
            // lo < hi first: of offsets that break the rule the difference may not fit 64 bits
            if (lo >= 0 && lo < hi && hi <= a.rows && band <= tr && tr < band + (hi - lo + kTile - 1) / kTile) s_expert = g;
        }
        __syncthreads();
        if (s_expert < 0) return;
        const int64_t lo = a.offsets[s_expert];
        r0 = lo + (tr - (lo / kTile + s_expert)) * kTile;
        rows = a.offsets[s_expert + 1];
        g0 = 4 * static_cast<int64_t>(tr);
        col_groups = 4 * a.bands_cap;
    }
    const T* x = static_cast<const T*>(a.x) + b * a.batch_stride;
    const int chunk = t & 15;
    if (kVec) {   // 16 bytes a copy, neighbouring threads side by side; what lies outside is filled up with zeros
        constexpr int kPer = kTile / kVec16<T>;   // copies of a row
        const int at = t % kPer, rows_step = kNT / kPer;
        const int64_t c = c0 + at * kVec16<T>, left = (a.cols - c) * static_cast<int64_t>(sizeof(T));
        const uint32_t bytes = left >= 16 ? 16u : (left > 0 ? static_cast<uint32_t>(left) : 0u);
        const T* from = x + (r0 + t / kPer) * a.ld + c;
        const uint32_t to = smem_u32(tile + t / kPer * kTile + at * kVec16<T>);
        const int left_rows = static_cast<int>(min(rows - r0, static_cast<int64_t>(kTile))) - t / kPer;
#pragma unroll
        for (int i = 0; i < kTile / rows_step; ++i) {
            const bool in = rows_step * i < left_rows && bytes > 0;
            cp_async16(to + static_cast<uint32_t>(i * rows_step * kTile * sizeof(T)), in ? from : x, in ? bytes : 0u);
            from += rows_step * a.ld;
        }
        cp_async_wait_all();
    } else if constexpr (sizeof(T) == 4) {   // an element a copy, a warp's side by side
        const int lane = t & 31, warp = t >> 5;
        const int left_rows = static_cast<int>(min(rows - r0, static_cast<int64_t>(kTile))), left = static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kTile)));
        const T* from = x + (r0 + warp) * a.ld + c0 + lane;
        uint32_t to = smem_u32(tile + warp * kTile + lane);
#pragma unroll 4
        for (int row = warp; row < kTile; row += kNT / 32) {
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k) {
                const bool in = row < left_rows && lane + 32 * k < left;
                cp_async4(to + 128u * k, in ? from + 32 * k : x, in ? 4u : 0u);
            }
            from += kNT / 32 * a.ld;
            to += kNT / 32 * kTile * static_cast<uint32_t>(sizeof(T));
        }
        cp_async_wait_all();
    } else {
        Eight<T> v[kPasses];
        const T* p = x + (r0 + (t >> 4)) * a.ld;
        if (is_whole<kVec>(rows, a.cols, r0, kTile, c0, kTile)) {
#pragma unroll
            for (int j = 0; j < kPasses; ++j) v[j].template load_whole<kVec>(p + kStep * j * a.ld, static_cast<int>(c0) + 8 * chunk);
        } else {
            load_rows<T, kVec, kPasses>(v, p, a.ld, r0 + (t >> 4), kStep, rows, static_cast<int>(c0) + 8 * chunk, static_cast<int>(a.cols));
        }
#pragma unroll
        for (int j = 0; j < kPasses; ++j) v[j].to_shared(tile + ((t >> 4) + kStep * j) * kTile + 8 * chunk);
    }
    __syncthreads();
    if constexpr (kRow && sizeof(T) == 2) {
        // A thread takes the groups t % 4 of the rows t / 4 and t / 4 + 64, each as four 16-byte chunks in the order
        // i ^ rot, so that the eight lanes of a load (two rows, four groups) hit different banks.
        const int group = t & 3, rot = (group & 2) | ((t >> 2) & 1);
        const int64_t g = (c0 >> 5) + group;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int tile_row = (t >> 2) + 64 * j;
            const uint32_t from = smem_u32(tile + tile_row * kTile + 32 * group);
            uint4 v[4];   // v[i]: chunk i ^ rot
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lds128(from + 16u * static_cast<uint32_t>(i ^ rot));
            uint32_t m2 = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m2 = max_abs_bf16x2(m2, max_abs_bf16x2(max_abs_bf16x2(v[i].x, v[i].y), max_abs_bf16x2(v[i].z, v[i].w)));
            m2 &= 0x7FFF7FFFu;
            const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16) << 16;
            uint32_t o[4], code;
            if (m >= kInfBits) {
                code = 0xFFu;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[8];
                    unpack<T>(v[i], f);
                    o[i] = bad_codes(f);
                }
            } else {
                const int e = rceil_exponent_f32<kE2M1>(m);
                code = static_cast<uint32_t>(e + 127);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Eight<T> eight;
                    eight.w[0] = v[i];
                    float f[8];
                    eight.scaled(e, f);
                    o[i] = cvt_e2m1x8(f);
                }
            }
            if (rot & 1) {   // back into order, a bit of the XOR at a time
                uint32_t x = o[0]; o[0] = o[1]; o[1] = x;
                x = o[2]; o[2] = o[3]; o[3] = x;
            }
            if (rot & 2) {
                uint32_t x = o[0]; o[0] = o[2]; o[2] = x;
                x = o[1]; o[1] = o[3]; o[3] = x;
            }
            const bool in = r0 + tile_row < a.rows && g < row_groups;
            if (in)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.q_row) + ((b * a.rows + r0 + tile_row) * row_groups + g) * 16) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            reinterpret_cast<uint8_t*>(s_row_codes)[4 * tile_row + group] = in ? static_cast<uint8_t>(code) : 0;
        }
    } else if constexpr (kRow) {
        const int64_t g = (c0 >> 5) + (chunk >> 2);
        uint8_t* q = static_cast<uint8_t*>(a.q_row) + (b * a.rows + r0 + (t >> 4)) * row_groups * 16 + c0 / 2 + 4 * chunk;
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
            const int tile_row = (t >> 4) + kStep * j;
            Eight<T> v;
            v.from_shared(tile + tile_row * kTile + 8 * chunk);
            uint32_t code;
            const uint32_t o = group_codes(v, &code);
            const bool in = r0 + tile_row < a.rows && g < row_groups;
            if (in) *reinterpret_cast<uint32_t*>(q + kStep * j * row_groups * 16) = o;
            if ((chunk & 3) == 0)
                reinterpret_cast<uint8_t*>(s_row_codes)[4 * tile_row + (chunk >> 2)] = in ? static_cast<uint8_t>(code) : 0;
        }
    }
    {
        uint8_t* codes8 = reinterpret_cast<uint8_t*>(s_col_codes);
        if constexpr (sizeof(T) == 2) {
            const int pair = t & 63, block = t >> 6;
            const uint32_t* from = reinterpret_cast<const uint32_t*>(tile) + 32 * block * (kTile / 2) + pair;
            uint32_t w[32], m2 = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                w[i] = from[i * (kTile / 2)];
                m2 = max_abs_bf16x2(m2, w[i]);
            }
            m2 &= 0x7FFF7FFFu;
            const uint32_t m[2] = {m2 << 16, m2 & 0xFFFF0000u};
            uint32_t code[2];
            uint4 o[2];
            if (m[0] < kInfBits && m[1] < kInfBits) {
                const int e0 = rceil_exponent_f32<kE2M1>(m[0]), e1 = rceil_exponent_f32<kE2M1>(m[1]);
                const uint32_t s2 = pow2_neg_bf16(e0) | (pow2_neg_bf16(e1) << 16);
                code[0] = static_cast<uint32_t>(e0 + 127), code[1] = static_cast<uint32_t>(e1 + 127);
                uint32_t p[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo[8], hi[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const uint32_t u = mul_bf16x2(w[8 * i + n], s2);
                        lo[n] = bf16_lo(u);
                        hi[n] = bf16_hi(u);
                    }
                    p[0][i] = cvt_e2m1x8(lo);
                    p[1][i] = cvt_e2m1x8(hi);
                }
                o[0] = make_uint4(p[0][0], p[0][1], p[0][2], p[0][3]);
                o[1] = make_uint4(p[1][0], p[1][1], p[1][2], p[1][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = k == 0 ? bf16_lo(w[i]) : bf16_hi(w[i]);
                    o[k] = column_codes(f, m[k], &code[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int c = 2 * pair + k;
                s_out[place_of(c, block)] = o[k];
                codes8[4 * c + block] = c0 + c < a.cols && g0 + block < col_groups ? static_cast<uint8_t>(code[k]) : 0;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4 * kTile / kNT; ++k) {
                const int c = t & (kTile - 1), block = (t >> 7) + kNT / kTile * k;
                float f[32];
                uint32_t m = 0u, code;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    f[i] = tile[(32 * block + i) * kTile + c];
                    m = max(m, abs_bits(f[i]));
                }
                s_out[place_of(c, block)] = column_codes(f, m, &code);
                codes8[4 * c + block] = c0 + c < a.cols && g0 + block < col_groups ? static_cast<uint8_t>(code) : 0;
            }
        }
        __syncthreads();
        uint8_t* q = static_cast<uint8_t*>(a.q_col) + b * a.cols * col_groups * 16;
#pragma unroll
        for (int k = 0; k < 4 * kTile / kNT; ++k) {
            const int c = (t >> 2) + kNT / 4 * k, block = t & 3;
            const int64_t g = g0 + block;
            if (c0 + c < a.cols && g < col_groups)
                *reinterpret_cast<uint4*>(q + ((c0 + c) * col_groups + g) * 16) = s_out[place_of(c, block)];
        }
        if (t < kTile) {
            store_codes(static_cast<uint8_t*>(a.s_col) + b * a.s_col_bytes, a.tiled, c0 + t, a.cols, g0, col_groups,
                        s_col_codes[t]);
            if (kRow)
                store_codes(static_cast<uint8_t*>(a.s_row) + b * a.s_row_bytes, a.tiled, r0 + t, a.rows, c0 >> 5, row_groups,
                            s_row_codes[t]);
        }
    }
}

template <typename T, bool kVec>
cudaError_t launch_quant_t(const Quant4Args& a, cudaStream_t stream) {
    if (a.q_col == nullptr) {
        const int64_t tiles_c = (a.cols + kColTile - 1) / kColTile, few = (a.rows + kFewRows - 1) / kFewRows;
        // tiled scales: whole 512-byte atoms, with their padding
        const int64_t many = ((a.tiled ? (a.rows + kTile - 1) / kTile * kTile : a.rows) + kRowTile<T> - 1) / kRowTile<T>;
        const bool is_few = a.batch * few * tiles_c <= static_cast<int64_t>(kFewBlocks) * a.sms;
        const int64_t per_batch = tiles_c * (is_few ? few : many), blocks = a.batch * per_batch;
        if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
        const Shape s{static_cast<int>(tiles_c), static_cast<int>(per_batch)};
        const dim3 grid(static_cast<unsigned>(blocks));
        return is_few ? launch_behind(quant_rows_kernel<T, kVec, kFewRows>, grid, kThreads, 0, stream, a, s)
                      : launch_behind(quant_rows_kernel<T, kVec, kRowTile<T>>, grid, kThreads, 0, stream, a, s);
    }
    const int64_t tiles_c = (a.cols + kTile - 1) / kTile;
    const int64_t per_batch = tiles_c * (a.offsets != nullptr ? a.bands_cap : (a.rows + kTile - 1) / kTile);
    const int64_t blocks = a.batch * per_batch;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const Shape s{static_cast<int>(tiles_c), static_cast<int>(per_batch)};
    const dim3 grid(static_cast<unsigned>(blocks));
    constexpr unsigned kShared = kTile * kTile * sizeof(T) + 4 * kTile * sizeof(uint4);
    const auto go = [&](auto threads) {
        constexpr int kNT = decltype(threads)::value;
        if (a.offsets != nullptr) return launch_behind(quant_tile_kernel<T, false, kVec, true, kNT>, grid, kNT, kShared, stream, a, s);
        if (a.q_row == nullptr) return launch_behind(quant_tile_kernel<T, false, kVec, false, kNT>, grid, kNT, kShared, stream, a, s);
        return launch_behind(quant_tile_kernel<T, true, kVec, false, kNT>, grid, kNT, kShared, stream, a, s);
    };
    if constexpr (sizeof(T) == 4) {
        if (blocks <= static_cast<int64_t>(kFewTiles) * a.sms) return go(std::integral_constant<int, 512>{});
    }
    return go(std::integral_constant<int, 256>{});
}

// ---- values ----------------------------------------------------------------------------
//
// Bound by the values that are written.  Rows that hold whole vectors: 16 elements a thread, one 8- or 16-byte load and
// 32 or 64 bytes of values.  Any other rows: 16 elements a thread on the 16-byte grid of the values, the payload's words
// shifted to them; element by element at a row's ends only (16381 x 7167 74 us, 59% of the copy rate).

template <int kFormat>
__device__ __forceinline__ void values8(uint32_t lo, uint32_t hi, float s, float (&f)[8]) {
    uint32_t h[4];
    if constexpr (kFormat == kE2M1) {
        cvt_f16_e2m1x8(lo, h);
    } else {
        h[0] = cvt_f16_fp8x2<kFormat>(lo & 0xFFFFu), h[1] = cvt_f16_fp8x2<kFormat>(lo >> 16);
        h[2] = cvt_f16_fp8x2<kFormat>(hi & 0xFFFFu), h[3] = cvt_f16_fp8x2<kFormat>(hi >> 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = f16_lo(h[i]) * s;
        f[2 * i + 1] = f16_hi(h[i]) * s;
    }
}

// The scale codes of row r.
struct RowScales {
    const uint8_t* first;
    bool tiled;
    __device__ __forceinline__ RowScales(const Dequant4Args& a, int64_t r)
        : first(static_cast<const uint8_t*>(a.s) + (a.tiled ? tiled_scale_offset(r, 0, (a.cols + 31) >> 5) : r * a.lds)), tiled(a.tiled) {}
    __device__ __forceinline__ uint32_t operator[](int g) const { return first[tiled ? (g >> 2) * 512 + (g & 3) : g]; }
};

template <int kFormat, typename T>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const Dequant4Args a, int log_row) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads >> log_row) + (threadIdx.x >> log_row);
    const int c = static_cast<int>((blockIdx.y << log_row) + (threadIdx.x & ((1u << log_row) - 1u))) * 16;
    if (r >= a.rows || c >= a.cols) return;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + r * a.ldq + (kFormat == kE2M1 ? c / 2 : c);
    uint32_t w[4];
    if constexpr (kFormat == kE2M1) {
        const uint2 v = *reinterpret_cast<const uint2*>(q);
        w[0] = v.x, w[2] = v.y, w[1] = w[3] = 0u;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(q);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    const float s = scale_of(RowScales(a, r)[c >> 5]);
    T* out = static_cast<T*>(a.out) + r * a.ldo + c;
    float f[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) values8<kFormat>(w[2 * i], w[2 * i + 1], s, f[i]);
    // 32 bytes a store, a whole sector, and not a streaming one: what follows reads the values (E2M1 to BF16: 16384 x 7168
    // 49.4 us, 51.6 us with two streaming stores of 16 bytes; 8192 x 4096 12.8 us, 18.6 us)
    uint32_t o[8];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = cvt_bf16x2(f[i >> 2][2 * i & 7], f[i >> 2][(2 * i & 7) + 1]);
        stg256(out, o);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(f[k][i]);
            stg256(out + 8 * k, o);
        }
    }
}

template <int kFormat, typename T>
__global__ void __launch_bounds__(kThreads) dequant_any_kernel(const Dequant4Args a, int log_row) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kThreads >> log_row) + (threadIdx.x >> log_row);
    if (r >= a.rows) return;
    T* out = static_cast<T*>(a.out) + r * a.ldo;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + r * a.ldq;
    const int cols = static_cast<int>(a.cols), groups = (cols + 31) >> 5;   // at most 2^23
    const RowScales scales(a, r);
    // 16 elements from i on, which lies on the output's 16-byte grid
    const int i = static_cast<int>((blockIdx.y << log_row) + (threadIdx.x & ((1u << log_row) - 1u))) * 16 - lead_of<sizeof(T)>(out);
    if (i >= cols) return;
    const int g = i >> 5;
    const int in_first = 32 - (i & 31);   // elements that the first of at most two groups has here
    const uint32_t c0 = g >= 0 ? scales[g] : 0u;
    const float s0 = scale_of(c0), s1 = scale_of(in_first < 16 && g + 1 < groups ? scales[g + 1] : c0);
    uint32_t w[5];
    if constexpr (kFormat == kE2M1) {   // the payload's rows start on words: three of them, shifted by elements
        const uint32_t* words = reinterpret_cast<const uint32_t*>(q);
        const int first = i >> 3;   // -1: before the row
#pragma unroll
        for (int k = 0; k < 3; ++k) w[k] = first + k >= 0 && first + k < 4 * groups ? words[first + k] : 0u;
    } else {
        const uint8_t* p = q + i;
        const unsigned at = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 3u);
        if (i >= 4 && i + 20 <= cols) {   // whole words around it lie in the row
            const uint32_t* words = reinterpret_cast<const uint32_t*>(p - at);
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = words[k];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 8 * at);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = 0u;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (i + k >= 0 && i + k < cols) w[k >> 2] |= static_cast<uint32_t>(p[k]) << (8 * (k & 3));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];   // exact: the scale follows
        if constexpr (kFormat == kE2M1) values8<kFormat>(__funnelshift_r(w[h], w[h + 1], 4 * (i & 7)), 0u, 1.0f, f);
        else values8<kFormat>(w[2 * h], w[2 * h + 1], 1.0f, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= 8 * h + k < in_first ? s0 : s1;
        const int c = i + 8 * h;
        if (c >= 0 && c + 8 <= cols) {   // no end of the row, which it shares with its neighbours
#pragma unroll
            for (int k = 0; k < 8 / kVec16<T>; ++k) {
                float part[kVec16<T>];
#pragma unroll
                for (int j = 0; j < kVec16<T>; ++j) part[j] = f[k * kVec16<T> + j];
                reinterpret_cast<uint4*>(out + c)[k] = pack<T>(part);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k >= 0 && c + k < cols) out[c + k] = from_float<T>(f[k]);
        }
    }
}

// log2 of a block's threads along a row of `units`: the least power of two that holds it, at most 8; of a longer row than a
// warp the one of those down to a warp that leaves the fewest threads idle (4099 x 1111: 5.8 us to 5.0 us).
int threads_along_row(int64_t units) {
    int most = 0;
    while (most < 8 && (int64_t(1) << most) < units) ++most;
    const auto idle = [&](int l) { return ((units + (int64_t(1) << l) - 1) >> l << l) - units; };
    int best = most;
    for (int l = most - 1; l >= 5; --l)
        if (idle(l) < idle(best)) best = l;
    return best;
}

template <int kFormat, typename T>
cudaError_t launch_dequant_t(const Dequant4Args& a, cudaStream_t stream) {
    constexpr int64_t kLoad = kFormat == kE2M1 ? 8 : 16;
    const bool vec = a.cols % 16 == 0 && (reinterpret_cast<uintptr_t>(a.q) | static_cast<uintptr_t>(a.ldq)) % kLoad == 0 &&
                     (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 && a.ldo * static_cast<int64_t>(sizeof(T)) % 32 == 0;
    const int64_t units = vec ? a.cols / 16 : (a.cols + 7 + 15) / 16;   // a row that starts off the grid may have one more
    const int log_row = threads_along_row(units);
    const int64_t down = kThreads >> log_row, x = (a.rows + down - 1) / down, y = (units + (1 << log_row) - 1) >> log_row;
    if (x > 0x7FFFFFFF || y > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
    if (vec) dequant_kernel<kFormat, T><<<grid, kThreads, 0, stream>>>(a, log_row);
    else dequant_any_kernel<kFormat, T><<<grid, kThreads, 0, stream>>>(a, log_row);
    return cudaGetLastError();
}

template <int kFormat>
cudaError_t launch_dequant_of(const Dequant4Args& a, bool f32, cudaStream_t stream) {
    return f32 ? launch_dequant_t<kFormat, float>(a, stream) : launch_dequant_t<kFormat, bf16_bits>(a, stream);
}

}  // namespace

cudaError_t launch_quant_mxfp4(const Quant4Args& a, bool f32, cudaStream_t stream) {
    const int64_t size = f32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld * size % 16 == 0 && a.batch_stride * size % 16 == 0;
    if (f32) return vec ? launch_quant_t<float, true>(a, stream) : launch_quant_t<float, false>(a, stream);
    return vec ? launch_quant_t<bf16_bits, true>(a, stream) : launch_quant_t<bf16_bits, false>(a, stream);
}

cudaError_t launch_dequant(const Dequant4Args& a, int format, bool f32, cudaStream_t stream) {
    if (format == kE2M1) return launch_dequant_of<kE2M1>(a, f32, stream);
    if (format == kE5M2) return launch_dequant_of<kE5M2>(a, f32, stream);
    return launch_dequant_of<kE4M3>(a, f32, stream);
}

}  // namespace mxq
