// gemm_fp4.cu -- products of MXFP4 operands with BF16 output, dense and grouped by expert.
//
//   y[m, n] = sum_k (qa[m, k] 2^ea[m, k/32]) (qb[n, k] 2^eb[n, k/32])

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"
#include "mxq_quant_math.cuh"

namespace mxq {
namespace {

constexpr int kSide = 16;

// One output a thread, FP32 sums.
template <bool kGrouped>
__global__ void __launch_bounds__(kSide* kSide) gemm_mxfp4_kernel(const Gemm4Args a) {
    const int64_t m = blockIdx.y * static_cast<int64_t>(kSide) + threadIdx.y;
    const int64_t n = blockIdx.x * static_cast<int64_t>(kSide) + threadIdx.x;
    if (m >= a.M || n >= a.N) return;
    const int64_t groups = (a.K + 31) >> 5;
    int64_t a_row = m, b_row = n, b_scale = n;
    if constexpr (kGrouped) {
        int lo = 0, hi = a.G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.offsets[mid] <= m) lo = mid; else hi = mid;
        }
        const int64_t first = a.offsets[lo];
        if (first < 0 || m < first || m >= a.offsets[lo + 1]) return;
        a_row = (first / 128 + lo) * 128 + (m - first);
        if (a_row >= a.bands_cap * 128) return;
        b_row = lo * a.N + n;
        b_scale = lo * ((a.N + 127) / 128 * 128) + n;
    }
    const uint8_t* qa = static_cast<const uint8_t*>(a.a_q) + m * groups * 16;
    const uint8_t* qb = static_cast<const uint8_t*>(a.b_q) + b_row * groups * 16;
    const uint8_t* sa = static_cast<const uint8_t*>(a.a_s);
    const uint8_t* sb = static_cast<const uint8_t*>(a.b_s);
    float sum = 0.0f;
    for (int64_t g = 0; g < groups; ++g) {
        const uint4 va = reinterpret_cast<const uint4*>(qa)[g], vb = reinterpret_cast<const uint4*>(qb)[g];
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t ha[4], hb[4];
            cvt_f16_e2m1x8(wa[i], ha);
            cvt_f16_e2m1x8(wb[i], hb);
#pragma unroll
            for (int j = 0; j < 4; ++j) part += f16_lo(ha[j]) * f16_lo(hb[j]) + f16_hi(ha[j]) * f16_hi(hb[j]);
        }
        sum += part * scale_of(sa[tiled_scale_offset(a_row, g, groups)]) * scale_of(sb[tiled_scale_offset(b_scale, g, groups)]);
    }
    static_cast<bf16_bits*>(a.y)[m * a.ldy + n] = from_float<bf16_bits>(sum);
}

}  // namespace

cudaError_t launch_gemm_mxfp4(const DeviceInfo&, const Gemm4Args& a, cudaStream_t stream) {
    const int64_t by = (a.M + kSide - 1) / kSide;
    if (by > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((a.N + kSide - 1) / kSide), static_cast<unsigned>(by)), block(kSide, kSide);
    if (a.offsets != nullptr) gemm_mxfp4_kernel<true><<<grid, block, 0, stream>>>(a);
    else gemm_mxfp4_kernel<false><<<grid, block, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace mxq
