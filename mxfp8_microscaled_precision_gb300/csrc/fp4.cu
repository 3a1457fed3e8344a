// fp4.cu -- MXFP4 quantization (E2M1 elements, one E8M0 scale per 32) along one or both axes of BF16
// or FP32 matrices, and the values that a microscaled payload stands for.
//
//   e = ceil(log2(amax / 6)) over 32 consecutive elements, -127 at least;  q = E2M1(x 2^-e)
//
// The amax exponent comes from FP32 bits (BF16 is its upper half), the scaling by a power of two is
// exact, one instruction rounds two values to nearest even.

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"
#include "mxq_quant_math.cuh"

namespace mxq {
namespace {

constexpr int kTile = 128;
constexpr int kThreads = 256;

// Eight elements of a row, as they are stored.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            float s[kVec16<T>];
            unpack<T>(w[i], s);
#pragma unroll
            for (int j = 0; j < kVec16<T>; ++j) f[i * kVec16<T> + j] = s[j];
        }
    }
    // The elements [c, c + 8) of a row of n, 0 behind it.  kVec: rows start on 16 bytes.
    template <bool kVec>
    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t n) {
        if (kVec && c + 8 <= n) {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(row + c)[i];
            return;
        }
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < n ? to_float(row[c + i]) : 0.0f;
        if constexpr (sizeof(T) == 2) {
            w[0] = pack<T>(f);   // exact
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                                  __float_as_uint(f[4 * i + 3]));
        }
    }
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Codes of eight elements of a group whose largest |x| has the bits `amax`; *code: its scale.
__device__ __forceinline__ uint32_t quant8_e2m1(const float (&f)[8], uint32_t amax, uint32_t* code) {
    if (amax >= kInfBits) {   // NaN or infinity in the group: 7 with the sign
        uint32_t r = 0x77777777u;
#pragma unroll
        for (int i = 0; i < 8; ++i) r |= (__float_as_uint(f[i]) >> 31) << (4 * i + 3);
        *code = 0xFFu;
        return r;
    }
    const int e = rceil_exponent_f32<kE2M1>(amax);
    *code = static_cast<uint32_t>(e + 127);
    float v[8];
    const float s = pow2_neg(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = f[i] * s;
    return cvt_e2m1x8(v);
}

struct Shape {
    int64_t tiles_c, per_batch;   // 128 x 128 tiles of a row of tiles and of a matrix
};

// One 128 x 128 tile.  Thread t holds the elements 8 (t % 16) .. of the tile's rows t / 16 + 16 j; the
// four threads of a group sit side by side.  The column copy reads the tile back from shared memory: a
// thread takes a column of 32 rows.
template <typename T, bool kRow, bool kCol, bool kVec>
__global__ void __launch_bounds__(kThreads) quant_mxfp4_kernel(const Quant4Args a, const Shape s) {
    __shared__ __align__(16) T tile[kCol ? kTile * kTile : 1];
    __shared__ uint32_t s_codes[kTile];   // four scale codes of every row (of every column)
    const int t = threadIdx.x;
    const int64_t b = blockIdx.x / s.per_batch, local = blockIdx.x - b * s.per_batch;
    const int64_t tr = local / s.tiles_c, tc = local - tr * s.tiles_c;
    const int64_t r0 = tr * kTile, c0 = tc * kTile;
    const int64_t row_groups = (a.cols + 31) >> 5, col_groups = (a.rows + 31) >> 5;
    const T* x = static_cast<const T*>(a.x) + b * a.batch_stride;
    const int chunk = t & 15;
    uint8_t* codes8 = reinterpret_cast<uint8_t*>(s_codes);
    Eight<T> v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t r = r0 + (t >> 4) + 16 * j;
        v[j].template load<kVec>(x + r * a.ld, c0 + 8 * chunk, r < a.rows ? a.cols : 0);
    }
    if constexpr (kCol) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                reinterpret_cast<uint4*>(tile + ((t >> 4) + 16 * j) * kTile + 8 * chunk)[i] = v[j].w[i];
    }
    if constexpr (kRow) {
        uint8_t* q = static_cast<uint8_t*>(a.q_row) + b * a.rows * row_groups * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int tile_row = (t >> 4) + 16 * j;
            const int64_t r = r0 + tile_row, g = (c0 >> 5) + (chunk >> 2);
            float f[8];
            v[j].floats(f);
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, abs_bits(f[i]));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            uint32_t code;
            const uint32_t o = quant8_e2m1(f, m, &code);
            const bool in = r < a.rows && g < row_groups;
            if (in) *reinterpret_cast<uint32_t*>(q + (r * row_groups + (c0 >> 5)) * 16 + 4 * chunk) = o;
            if ((chunk & 3) == 0) codes8[4 * tile_row + (chunk >> 2)] = in ? static_cast<uint8_t>(code) : 0;
        }
        __syncthreads();
        // the four codes of a row: one word of the tile's 512-byte atom, or bytes of a plain row
        if (t < kTile) {
            uint8_t* out = static_cast<uint8_t*>(a.s_row) + b * a.s_row_bytes;
            const int64_t r = r0 + t, g = c0 >> 5;
            if (a.offsets != nullptr) {   // tiled by expert: its first row starts a band
                int lo = 0, hi = a.G;   // the last expert that starts at or before the row
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.offsets[mid] <= r) lo = mid; else hi = mid;
                }
                const int64_t first = a.offsets[lo], end = a.offsets[lo + 1];
                const int64_t at = (first / kTile + lo) * kTile + (r - first);
                if (r < a.rows && first >= 0 && r >= first && r < end && at < a.bands_cap * kTile)
                    *reinterpret_cast<uint32_t*>(out + tiled_scale_offset(at, g, row_groups)) = s_codes[t];
            } else if (a.tiled) {
                *reinterpret_cast<uint32_t*>(out + tiled_scale_offset(r, g, row_groups)) = s_codes[t];
            } else if (r < a.rows) {
                for (int i = 0; i < 4; ++i)
                    if (g + i < row_groups) out[r * row_groups + g + i] = codes8[4 * t + i];
            }
        }
    }
    if constexpr (kCol) {
        __syncthreads();   // the tile is written, the rows' codes are read
        uint8_t* q = static_cast<uint8_t*>(a.q_col) + b * a.cols * col_groups * 16;
#pragma unroll 1
        for (int k = t; k < 4 * kTile; k += kThreads) {
            const int c = k & (kTile - 1), block = k >> 7;   // a column, 32 rows of it
            float f[32];
            uint32_t m = 0u;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                f[i] = to_float(tile[(32 * block + i) * kTile + c]);
                m = max(m, abs_bits(f[i]));
            }
            uint32_t o[4], code;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float part[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) part[n] = f[8 * i + n];
                o[i] = quant8_e2m1(part, m, &code);
            }
            const int64_t col = c0 + c, g = (r0 >> 5) + block;
            const bool in = col < a.cols && g < col_groups;
            if (in) *reinterpret_cast<uint4*>(q + (col * col_groups + g) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
            codes8[4 * c + block] = in ? static_cast<uint8_t>(code) : 0;
        }
        __syncthreads();
        if (t < kTile) {
            uint8_t* out = static_cast<uint8_t*>(a.s_col) + b * a.s_col_bytes;
            const int64_t c = c0 + t, g = r0 >> 5;
            if (a.tiled) {
                *reinterpret_cast<uint32_t*>(out + tiled_scale_offset(c, g, col_groups)) = s_codes[t];
            } else if (c < a.cols) {
                for (int i = 0; i < 4; ++i)
                    if (g + i < col_groups) out[c * col_groups + g + i] = codes8[4 * t + i];
            }
        }
    }
}

template <typename T, bool kVec>
cudaError_t launch_quant_t(const Quant4Args& a, cudaStream_t stream) {
    const Shape s{(a.cols + kTile - 1) / kTile, (a.cols + kTile - 1) / kTile * ((a.rows + kTile - 1) / kTile)};
    const int64_t blocks = a.batch * s.per_batch;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(blocks);
    if (a.q_col == nullptr) quant_mxfp4_kernel<T, true, false, kVec><<<grid, kThreads, 0, stream>>>(a, s);
    else if (a.q_row == nullptr) quant_mxfp4_kernel<T, false, true, kVec><<<grid, kThreads, 0, stream>>>(a, s);
    else quant_mxfp4_kernel<T, true, true, kVec><<<grid, kThreads, 0, stream>>>(a, s);
    return cudaGetLastError();
}

// ---- values ----------------------------------------------------------------------------

// Eight elements a thread.
template <int kFormat, typename T>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const Dequant4Args a, int64_t per_row) {
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t r = i / per_row, c = (i - r * per_row) * 8;
    if (r >= a.rows) return;
    const int64_t groups = (a.cols + 31) >> 5, g = c >> 5;
    const uint8_t* q = static_cast<const uint8_t*>(a.q) + r * a.ldq;
    const uint8_t* sc = static_cast<const uint8_t*>(a.s);
    const float s = scale_of(a.tiled ? sc[tiled_scale_offset(r, g, groups)] : sc[r * a.lds + g]);
    T* out = static_cast<T*>(a.out) + r * a.ldo;
    for (int k = 0; k < 8 && c + k < a.cols; k += 2) {
        uint32_t h;
        if constexpr (kFormat == kE2M1) {
            uint32_t all[4];
            cvt_f16_e2m1x8(q[(c + k) >> 1], all);
            h = all[0];
        } else {
            h = cvt_f16_fp8x2<kFormat>(q[c + k] | (c + k + 1 < a.cols ? q[c + k + 1] << 8 : 0));
        }
        out[c + k] = from_float<T>(f16_lo(h) * s);
        if (c + k + 1 < a.cols) out[c + k + 1] = from_float<T>(f16_hi(h) * s);
    }
}

template <int kFormat>
cudaError_t launch_dequant_t(const Dequant4Args& a, bool f32, cudaStream_t stream) {
    const int64_t per_row = (a.cols + 7) / 8, blocks = (a.rows * per_row + kThreads - 1) / kThreads;
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if (f32) dequant_kernel<kFormat, float><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, per_row);
    else dequant_kernel<kFormat, bf16_bits><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, per_row);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_mxfp4(const Quant4Args& a, bool f32, cudaStream_t stream) {
    const int64_t size = f32 ? 4 : 2;
    const bool vec = (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && a.ld * size % 16 == 0 && a.batch_stride * size % 16 == 0;
    if (f32) return vec ? launch_quant_t<float, true>(a, stream) : launch_quant_t<float, false>(a, stream);
    return vec ? launch_quant_t<bf16_bits, true>(a, stream) : launch_quant_t<bf16_bits, false>(a, stream);
}

cudaError_t launch_dequant(const Dequant4Args& a, int format, bool f32, cudaStream_t stream) {
    if (format == kE2M1) return launch_dequant_t<kE2M1>(a, f32, stream);
    if (format == kE5M2) return launch_dequant_t<kE5M2>(a, f32, stream);
    return launch_dequant_t<kE4M3>(a, f32, stream);
}

}  // namespace mxq
