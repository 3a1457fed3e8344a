// api_fp4.cu -- the extern "C" entry points of MXFP4 quantization and products and of activations
// kept in 8 bits (declared in include/mxq.h).
//
// Each call validates its arguments on the host, checks that the current
// device is a GB300 (sm_103), and launches on the caller's stream.  Nothing is
// allocated on the device, nothing is kept from one call to the next.

#include <cuda_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "mxq.h"
#include "mxq_internal.h"

namespace {

using namespace mxq;   // api_util.h

constexpr int kMaxExperts = 1024;

inline int64_t groups_of(int64_t cols) { return (cols + 31) / 32; }
inline int64_t bands_of(int64_t rows) { return (rows + 127) / 128; }

mxq_status check_act(mxq_dtype dtype, int64_t rows, int64_t inter, mxq_act kind, int32_t gated) {
    if (bad_dtype(dtype) || rows < 0 || inter < 0 || (kind != MXQ_ACT_SILU && kind != MXQ_ACT_GELU) ||
        (gated != 0 && gated != 1))
        return MXQ_ERR_INVALID_ARG;
    if (rows > kMaxRows || inter > kMaxCols) return MXQ_ERR_UNSUPPORTED_SHAPE;
    return MXQ_OK;
}

// Operands of a product (a_q .. b_s: 16-byte aligned).
bool bad_operands(const void* a_q, const void* a_s, const void* b_q, const void* b_s) {
    return !a_q || !a_s || !b_q || !b_s || !aligned(a_q, 16) || !aligned(a_s, 16) || !aligned(b_q, 16) || !aligned(b_s, 16);
}

}  // namespace

extern "C" {

mxq_status mxq_quant_mxfp4(const void* x, mxq_dtype dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld,
                           int64_t batch_stride, void* q_row, void* s_row, void* q_col, void* s_col,
                           mxq_scale_layout layout, mxq_stream_t stream) {
    if (bad_dtype(dtype) || (layout != MXQ_SCALE_ROWMAJOR && layout != MXQ_SCALE_MMA_TILED)) return MXQ_ERR_INVALID_ARG;
    if (batch < 0 || rows < 0 || cols < 0 || ld < cols || batch_stride < 0) return MXQ_ERR_INVALID_ARG;
    if (batch > 65535 || rows > kMaxRows || cols > kMaxRows || bands_of(rows) * bands_of(cols) > 0x7FFFFFFF / (batch > 0 ? batch : 1))
        return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (batch == 0 || rows == 0 || cols == 0) return MXQ_OK;
    if (!x || (!q_row && !q_col) || !q_row != !s_row || !q_col != !s_col) return MXQ_ERR_INVALID_ARG;
    if (!aligned(x, size_of(dtype)) || !aligned(q_row, 16) || !aligned(s_row, 16) || !aligned(q_col, 16) || !aligned(s_col, 16))
        return MXQ_ERR_INVALID_ARG;
    int sms = 0;
    const mxq_status st = device_ok(&sms);
    if (st != MXQ_OK) return st;
    const Quant4Args a{x, batch, rows, cols, ld, batch > 1 ? batch_stride : 0, q_row, s_row, q_col, s_col,
                       static_cast<int64_t>(mxq_scale_bytes(rows, 32 * groups_of(cols), layout)),
                       static_cast<int64_t>(mxq_scale_bytes(cols, 32 * groups_of(rows), layout)),
                       layout == MXQ_SCALE_MMA_TILED, nullptr, 0, 0, sms};
    return from_cuda(launch_quant_mxfp4(a, dtype == MXQ_F32, cu(stream)));
}

mxq_status mxq_quant_mxfp4_grouped(const void* x, mxq_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                   const int64_t* group_offsets, int32_t G, int64_t bands_cap, void* q, void* s,
                                   mxq_stream_t stream) {
    if (bad_dtype(dtype) || rows < 0 || cols < 0 || ld < cols || G < 1) return MXQ_ERR_INVALID_ARG;
    if (G > kMaxExperts || rows > kMaxRows || cols > kMaxRows || bands_of(rows) * bands_of(cols) > 0x7FFFFFFF)
        return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (bands_cap < bands_of(rows) + G) return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MXQ_OK;
    if (!x || !group_offsets || !q || !s || !aligned(x, size_of(dtype)) || !aligned(group_offsets, 8) || !aligned(q, 16) ||
        !aligned(s, 16))
        return MXQ_ERR_INVALID_ARG;
    int sms = 0;
    const mxq_status st = device_ok(&sms);
    if (st != MXQ_OK) return st;
    const Quant4Args a{x, 1, rows, cols, ld, 0, q, s, nullptr, nullptr, 0, 0, true, group_offsets, G, bands_cap, sms};
    return from_cuda(launch_quant_mxfp4(a, dtype == MXQ_F32, cu(stream)));
}

mxq_status mxq_quant_mxfp4_cols_grouped(const void* x, mxq_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                        const int64_t* group_offsets, int32_t G, int64_t capacity, void* q, void* s,
                                        mxq_stream_t stream) {
    if (bad_dtype(dtype) || rows < 0 || cols < 0 || ld < cols || G < 1 || capacity < 0) return MXQ_ERR_INVALID_ARG;
    if (G > kMaxExperts || rows > kMaxRows || cols > kMaxRows || capacity > kMaxRows || capacity % 128 != 0 ||
        capacity / 128 * bands_of(cols) > 0x7FFFFFFF)
        return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (capacity / 128 < bands_of(rows) + G) return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return MXQ_OK;
    if (!x || !group_offsets || !q || !s || !aligned(x, size_of(dtype)) || !aligned(group_offsets, 8) || !aligned(q, 16) ||
        !aligned(s, 16))
        return MXQ_ERR_INVALID_ARG;
    int sms = 0;
    const mxq_status st = device_ok(&sms);
    if (st != MXQ_OK) return st;
    const Quant4Args a{x, 1, rows, cols, ld, 0, nullptr, nullptr, q, s, 0, 0, true, group_offsets, G, capacity / 128, sms};
    return from_cuda(launch_quant_mxfp4(a, dtype == MXQ_F32, cu(stream)));
}

mxq_status mxq_dequant_1x32(const void* q, const void* s, mxq_element element, int64_t rows, int64_t cols, int64_t ldq,
                            int64_t lds, mxq_scale_layout layout, void* out, mxq_dtype dtype, int64_t ldo,
                            mxq_stream_t stream) {
    if (bad_dtype(dtype) || (layout != MXQ_SCALE_ROWMAJOR && layout != MXQ_SCALE_MMA_TILED)) return MXQ_ERR_INVALID_ARG;
    if (element != MXQ_ELEM_E4M3 && element != MXQ_ELEM_E5M2 && element != MXQ_ELEM_E2M1) return MXQ_ERR_INVALID_ARG;
    if (rows < 0 || cols < 0 || ldo < cols) return MXQ_ERR_INVALID_ARG;
    const bool four = element == MXQ_ELEM_E2M1;
    if (ldq < (four ? 16 * groups_of(cols) : cols)) return MXQ_ERR_INVALID_ARG;
    if (layout == MXQ_SCALE_ROWMAJOR && lds < groups_of(cols)) return MXQ_ERR_INVALID_ARG;
    if (rows > kMaxRows || cols > kMaxCols) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0 || cols == 0) return MXQ_OK;
    if (!q || !s || !out || !aligned(out, size_of(dtype)) || (four && (!aligned(q, 4) || ldq % 4 != 0))) return MXQ_ERR_INVALID_ARG;
    const mxq_status st = device_ok();
    if (st != MXQ_OK) return st;
    const Dequant4Args a{q, s, rows, cols, ldq, lds, layout == MXQ_SCALE_MMA_TILED, out, ldo};
    return from_cuda(launch_dequant(a, static_cast<int>(element), dtype == MXQ_F32, cu(stream)));
}

mxq_status mxq_gemm_mxfp4(const void* a_q, const void* a_s, const void* b_q, const void* b_s, int64_t M, int64_t N,
                          int64_t K, void* y, int64_t ldy, mxq_stream_t stream) {
    if (M < 0 || N < 0 || K < 0 || ldy < N) return MXQ_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxRows) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return MXQ_OK;
    if (!y || !aligned(y, 2) || (K > 0 && bad_operands(a_q, a_s, b_q, b_s))) return MXQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    const mxq_status st = device_ok(&dev);
    if (st != MXQ_OK) return st;
    if (K == 0)   // sums of nothing
        return from_cuda(cudaMemset2DAsync(y, static_cast<size_t>(ldy) * 2, 0, static_cast<size_t>(N) * 2,
                                           static_cast<size_t>(M), cu(stream)));
    return from_cuda(launch_gemm_mxfp4(dev, {a_q, a_s, b_q, b_s, M, N, K, y, ldy, nullptr, 0, 0}, cu(stream)));
}

mxq_status mxq_grouped_gemm_mxfp4(const void* a_q, const void* a_s, int64_t a_bands_cap, const void* b_q,
                                  const void* b_s, const int64_t* group_offsets, int32_t G, int64_t M_total, int64_t N,
                                  int64_t K, void* y, int64_t ldy, mxq_stream_t stream) {
    if (G < 1 || M_total < 0 || N < 0 || K < 1 || ldy < N) return MXQ_ERR_INVALID_ARG;
    if (G > kMaxExperts || M_total > kMaxRows || K > kMaxRows || N > kMaxRows / G) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (a_bands_cap < bands_of(M_total) + G) return MXQ_ERR_INVALID_ARG;
    if (M_total == 0 || N == 0) return MXQ_OK;
    if (!y || !aligned(y, 2) || !group_offsets || !aligned(group_offsets, 8) || bad_operands(a_q, a_s, b_q, b_s))
        return MXQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    const mxq_status st = device_ok(&dev);
    if (st != MXQ_OK) return st;
    return from_cuda(launch_gemm_mxfp4(dev, {a_q, a_s, b_q, b_s, M_total, N, K, y, ldy, group_offsets, G, a_bands_cap},
                                       cu(stream)));
}

mxq_status mxq_grouped_gemm_mxfp4_wgrad(const void* a_q, const void* a_s, const void* b_q, const void* b_s,
                                        const int64_t* group_offsets, int32_t G, int64_t M_total, int64_t capacity,
                                        int64_t M, int64_t N, void* y, int64_t ldy, mxq_stream_t stream) {
    if (G < 1 || M_total < 0 || capacity < 0 || M < 0 || N < 0 || ldy < N) return MXQ_ERR_INVALID_ARG;
    if (G > kMaxExperts || M_total > kMaxRows || capacity > kMaxRows || capacity % 128 != 0 || N > kMaxRows || M > kMaxRows / G)
        return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (capacity / 128 < bands_of(M_total) + G) return MXQ_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MXQ_OK;
    if (!y || !aligned(y, 2) || !group_offsets || !aligned(group_offsets, 8) || bad_operands(a_q, a_s, b_q, b_s))
        return MXQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    const mxq_status st = device_ok(&dev);
    if (st != MXQ_OK) return st;
    return from_cuda(launch_grouped_wgrad_mxfp4(dev, {a_q, a_s, b_q, b_s, M, N, capacity, y, ldy, group_offsets, G, 0}, M_total,
                                                cu(stream)));
}

mxq_status mxq_activation(const void* z, mxq_dtype dtype, int64_t rows, int64_t inter, int64_t ldz, mxq_act kind,
                          int32_t gated, void* y, int64_t ldy, void* q, void* s, mxq_stream_t stream) {
    mxq_status st = check_act(dtype, rows, inter, kind, gated);
    if (st != MXQ_OK) return st;
    if (ldz < (gated ? 2 : 1) * inter || ldy < inter || !q != !s) return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || inter == 0) return MXQ_OK;
    if (!z || !y || !aligned(z, size_of(dtype)) || !aligned(y, size_of(dtype)) || !aligned(q, 16) || !aligned(s, 16))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(launch_activation({rows, inter, ldz, ldy, z, y, q, s}, dtype == MXQ_F32, static_cast<int>(kind),
                                       gated != 0, cu(stream)));
}

mxq_status mxq_activation_backward(const void* dy, mxq_dtype dtype, int64_t lddy, const void* q, const void* s,
                                   int64_t rows, int64_t inter, mxq_act kind, int32_t gated, void* dz, int64_t lddz,
                                   void* y, int64_t ldy, mxq_stream_t stream) {
    mxq_status st = check_act(dtype, rows, inter, kind, gated);
    if (st != MXQ_OK) return st;
    if (lddy < inter || lddz < (gated ? 2 : 1) * inter || (y && ldy < inter)) return MXQ_ERR_INVALID_ARG;
    if (rows == 0 || inter == 0) return MXQ_OK;
    if (!dy || !q || !s || !dz) return MXQ_ERR_INVALID_ARG;
    if (!aligned(dy, size_of(dtype)) || !aligned(dz, size_of(dtype)) || !aligned(y, size_of(dtype)) || !aligned(q, 16) ||
        !aligned(s, 16))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(launch_activation_backward({rows, inter, lddy, lddz, ldy, dy, q, s, dz, y}, dtype == MXQ_F32,
                                                static_cast<int>(kind), gated != 0, cu(stream)));
}

}  // extern "C"
