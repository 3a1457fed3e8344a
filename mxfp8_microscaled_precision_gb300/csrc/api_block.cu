// api_block.cu -- the extern "C" entry points of the operators around the GEMMs
// (declared in include/mxq.h): routing to experts, rows into expert order and
// back, layer norm, and clipping by the norm over all gradients.
//
// Each call validates its arguments on the host, checks that the current
// device is a GB300 (sm_103), and launches on the caller's stream.  Nothing is
// allocated on the device, nothing is kept from one call to the next.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "api_util.h"
#include "mxq.h"
#include "mxq_internal.h"

namespace {

using namespace mxq;   // api_util.h

// Shapes and the stride rule shared by the routing calls.
mxq_status check_route(mxq_dtype dtype, int64_t tokens, int32_t experts, int64_t ld, mxq_route_score score, int32_t topk,
                       float scale) {
    if (bad_dtype(dtype) || (score != MXQ_SCORE_SOFTMAX && score != MXQ_SCORE_SIGMOID)) return MXQ_ERR_INVALID_ARG;
    if (tokens < 0 || experts < 1 || topk < 1 || ld < experts || !std::isfinite(scale)) return MXQ_ERR_INVALID_ARG;
    if (topk > experts) return MXQ_ERR_INVALID_ARG;
    if (experts > MXQ_MAX_EXPERTS || topk > MXQ_MAX_TOPK || tokens > kMaxRows) return MXQ_ERR_UNSUPPORTED_SHAPE;
    return MXQ_OK;
}

mxq_status check_rows(mxq_dtype dtype, int64_t tokens, int32_t k, int64_t H) {
    if (bad_dtype(dtype) || tokens < 0 || k < 1 || H < 0) return MXQ_ERR_INVALID_ARG;
    if (tokens > kMaxRows / k || H > kMaxCols) return MXQ_ERR_UNSUPPORTED_SHAPE;
    return MXQ_OK;
}

mxq_status check_norm(mxq_dtype dtype, mxq_dtype param_dtype, int64_t rows, int64_t cols) {
    if (bad_dtype(dtype) || bad_dtype(param_dtype) || rows < 0 || cols < 0) return MXQ_ERR_INVALID_ARG;
    if (rows > kMaxRows || cols > kMaxCols) return MXQ_ERR_UNSUPPORTED_SHAPE;
    return MXQ_OK;
}

mxq_status clip(const mxq_grad_desc* grads, int32_t count, bool scale, float max_norm, float eps, float* norm,
                void* workspace, size_t workspace_bytes, mxq_stream_t stream) {
    if (count < 0 || (count > 0 && grads == nullptr) || norm == nullptr || workspace == nullptr)
        return MXQ_ERR_INVALID_ARG;
    if (!aligned(norm, 4) || !aligned(workspace, 16)) return MXQ_ERR_INVALID_ARG;
    if (count > MXQ_MAX_GRADS) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (workspace_bytes < mxq_grad_norm_workspace_size(count)) return MXQ_ERR_INVALID_ARG;
    if (scale && (!(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps))) return MXQ_ERR_INVALID_ARG;
    std::unique_ptr<mxq::ClipTensor[]> list(new (std::nothrow) mxq::ClipTensor[count > 0 ? count : 1]);
    if (!list) return MXQ_ERR_CUDA;
    for (int32_t i = 0; i < count; ++i) {
        const mxq_grad_desc& g = grads[i];
        if (bad_dtype(g.dtype) || g.numel < 0 || g.numel > (int64_t(1) << 40)) return MXQ_ERR_INVALID_ARG;
        if (g.numel > 0 && (!g.grad || !aligned(g.grad, size_of(g.dtype)))) return MXQ_ERR_INVALID_ARG;
        if (g.numel > 0 && scale && (!g.out || !aligned(g.out, size_of(g.dtype)))) return MXQ_ERR_INVALID_ARG;
        list[i] = {g.grad, g.out, g.numel, g.dtype == MXQ_F32};
    }
    const mxq_status st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(mxq::launch_clip(list.get(), count, scale, max_norm, eps, norm, static_cast<float*>(workspace),
                                      cu(stream)));
}

}  // namespace

extern "C" {

mxq_status mxq_route(const void* logits, mxq_dtype dtype, int64_t tokens, int32_t experts, int64_t ld,
                     const float* bias, const uint8_t* token_mask, mxq_route_score score, int32_t n_group,
                     int32_t topk_group, mxq_group_score group_score, int32_t topk, int32_t renorm, float scale,
                     int32_t* ids, float* weights, mxq_stream_t stream) {
    mxq_status st = check_route(dtype, tokens, experts, ld, score, topk, scale);
    if (st != MXQ_OK) return st;
    if (group_score != MXQ_GROUP_MAX && group_score != MXQ_GROUP_TOP2SUM) return MXQ_ERR_INVALID_ARG;
    if (n_group < 1 || topk_group < 1 || topk_group > n_group || (renorm != 0 && renorm != 1))
        return MXQ_ERR_INVALID_ARG;
    if (n_group > 32 || experts % n_group != 0) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (topk > experts / n_group * topk_group) return MXQ_ERR_INVALID_ARG;
    if (tokens == 0) return MXQ_OK;
    if (!logits || !ids || !weights) return MXQ_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(bias, 4))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    mxq::RouteArgs a{tokens, ld, experts, topk, n_group, topk_group, group_score == MXQ_GROUP_TOP2SUM ? 1 : 0,
                     renorm, scale, bias, token_mask, ids, weights};
    return from_cuda(mxq::launch_route(logits, dtype == MXQ_F32, a, score == MXQ_SCORE_SOFTMAX, cu(stream)));
}

mxq_status mxq_route_backward(const float* dweights, const int32_t* ids, const void* logits, mxq_dtype dtype,
                              int64_t tokens, int32_t experts, int64_t ld, mxq_route_score score, int32_t topk,
                              int32_t renorm, float scale, void* dlogits, int64_t ld_out, mxq_stream_t stream) {
    mxq_status st = check_route(dtype, tokens, experts, ld, score, topk, scale);
    if (st != MXQ_OK) return st;
    if (ld_out < experts || (renorm != 0 && renorm != 1)) return MXQ_ERR_INVALID_ARG;
    if (tokens == 0) return MXQ_OK;
    if (!dweights || !ids || !logits || !dlogits) return MXQ_ERR_INVALID_ARG;
    if (!aligned(logits, size_of(dtype)) || !aligned(dlogits, size_of(dtype)) || !aligned(ids, 4) ||
        !aligned(dweights, 4))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    mxq::RouteBackwardArgs a{tokens, ld, ld_out, experts, topk, renorm, scale, ids, dweights};
    return from_cuda(mxq::launch_route_backward(logits, dlogits, dtype == MXQ_F32, a, score == MXQ_SCORE_SOFTMAX,
                                                cu(stream)));
}

mxq_status mxq_moe_plan(const int32_t* ids, int64_t tokens, int32_t k, int32_t experts, int64_t* offsets, int32_t* rows,
                        mxq_stream_t stream) {
    if (tokens < 0 || k < 1 || experts < 1) return MXQ_ERR_INVALID_ARG;
    if (experts > MXQ_MAX_EXPERTS || tokens > kMaxRows / k) return MXQ_ERR_UNSUPPORTED_SHAPE;
    if (!offsets || !aligned(offsets, 8)) return MXQ_ERR_INVALID_ARG;
    if (tokens > 0 && (!ids || !rows || !aligned(ids, 4) || !aligned(rows, 4))) return MXQ_ERR_INVALID_ARG;
    const mxq_status st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(mxq::launch_moe_plan(ids, tokens * k, experts, offsets, rows, cu(stream)));
}

mxq_status mxq_moe_dispatch(const void* x, mxq_dtype dtype, int64_t tokens, int32_t k, int64_t H, int64_t ldx,
                            const int32_t* rows, void* a, int64_t lda, mxq_stream_t stream) {
    mxq_status st = check_rows(dtype, tokens, k, H);
    if (st != MXQ_OK) return st;
    if (ldx < H || lda < H) return MXQ_ERR_INVALID_ARG;
    if (tokens == 0 || H == 0) return MXQ_OK;
    if (!x || !rows || !a) return MXQ_ERR_INVALID_ARG;
    if (!aligned(x, size_of(dtype)) || !aligned(a, size_of(dtype)) || !aligned(rows, 4)) return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(mxq::launch_moe_dispatch({tokens, H, k, rows, ldx, lda}, dtype == MXQ_F32, x, a, cu(stream)));
}

mxq_status mxq_moe_combine(const void* y, mxq_dtype dtype, int64_t tokens, int32_t k, int64_t H, int64_t ldy,
                           const int32_t* rows, const float* weights, void* out, int64_t ldo, mxq_stream_t stream) {
    mxq_status st = check_rows(dtype, tokens, k, H);
    if (st != MXQ_OK) return st;
    if (ldy < H || ldo < H) return MXQ_ERR_INVALID_ARG;
    if (tokens == 0 || H == 0) return MXQ_OK;
    if (!y || !rows || !out) return MXQ_ERR_INVALID_ARG;
    if (!aligned(y, size_of(dtype)) || !aligned(out, size_of(dtype)) || !aligned(rows, 4) || !aligned(weights, 4))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(mxq::launch_moe_combine({tokens, H, k, rows, ldo, ldy}, dtype == MXQ_F32, y, weights, out,
                                             cu(stream)));
}

mxq_status mxq_moe_combine_backward(const void* dout, const void* y, mxq_dtype dtype, int64_t tokens, int32_t k,
                                    int64_t H, int64_t ldd, int64_t ldy, const int32_t* rows, const float* weights,
                                    void* dy, int64_t lddy, float* dweights, mxq_stream_t stream) {
    mxq_status st = check_rows(dtype, tokens, k, H);
    if (st != MXQ_OK) return st;
    if (ldd < H || ldy < H || lddy < H) return MXQ_ERR_INVALID_ARG;
    if (tokens == 0) return MXQ_OK;
    if (!rows || !weights || !dweights || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return MXQ_ERR_INVALID_ARG;
    if (H > 0 && (!dout || !y || !dy)) return MXQ_ERR_INVALID_ARG;
    if (!aligned(dout, size_of(dtype)) || !aligned(y, size_of(dtype)) || !aligned(dy, size_of(dtype)))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    return from_cuda(mxq::launch_moe_combine_backward({tokens, H, k, rows, ldd, lddy}, dtype == MXQ_F32, dout, y, ldy,
                                                      weights, dy, dweights, cu(stream)));
}

mxq_status mxq_layer_norm(const void* x, mxq_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, const void* weight,
                          const void* shift, mxq_dtype param_dtype, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, mxq_stream_t stream) {
    mxq_status st = check_norm(dtype, param_dtype, rows, cols);
    if (st != MXQ_OK) return st;
    if (ldx < cols || ldy < cols || !(eps >= 0.0f) || std::isinf(eps)) return MXQ_ERR_INVALID_ARG;
    if (rows == 0) return MXQ_OK;
    if (cols > 0 && (!x || !y || !mean || !rstd)) return MXQ_ERR_INVALID_ARG;
    const size_t s = size_of(dtype), p = size_of(param_dtype);
    if (!aligned(x, s) || !aligned(y, s) || !aligned(weight, p) || !aligned(shift, p) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MXQ_ERR_INVALID_ARG;
    st = device_ok();
    if (st != MXQ_OK) return st;
    if (cols == 0) {   // 0 / 0 in every row: all bits set are a NaN
        cudaError_t e = cudaSuccess;
        if (mean) e = cudaMemsetAsync(mean, 0xFF, static_cast<size_t>(rows) * 4, cu(stream));
        if (e == cudaSuccess && rstd) e = cudaMemsetAsync(rstd, 0xFF, static_cast<size_t>(rows) * 4, cu(stream));
        return from_cuda(e);
    }
    return from_cuda(mxq::launch_layer_norm({rows, cols, ldx, ldy, x, weight, shift, eps, y, mean, rstd},
                                            dtype == MXQ_F32, param_dtype == MXQ_F32, cu(stream)));
}

size_t mxq_layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxCols) return 0;
    return static_cast<size_t>(mxq::norm_partials(rows, cols) * 2 * cols) * sizeof(float);
}

mxq_status mxq_layer_norm_backward(const void* dy, const void* x, mxq_dtype dtype, int64_t rows, int64_t cols,
                                   int64_t lddy, int64_t ldx, const void* weight, mxq_dtype param_dtype,
                                   const float* mean, const float* rstd, void* dx, int64_t lddx, float* dweight,
                                   float* dshift, void* workspace, size_t workspace_bytes, mxq_stream_t stream) {
    mxq_status st = check_norm(dtype, param_dtype, rows, cols);
    if (st != MXQ_OK) return st;
    if (lddy < cols || ldx < cols || lddx < cols) return MXQ_ERR_INVALID_ARG;
    if (cols == 0) return MXQ_OK;
    if (!aligned(dweight, 4) || !aligned(dshift, 4)) return MXQ_ERR_INVALID_ARG;
    const size_t s = size_of(dtype);
    if (rows > 0) {
        if (!dy || !x || !mean || !rstd || !dx || !workspace) return MXQ_ERR_INVALID_ARG;
        if (!aligned(dy, s) || !aligned(x, s) || !aligned(dx, s) || !aligned(weight, size_of(param_dtype)) ||
            !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
            return MXQ_ERR_INVALID_ARG;
        if (workspace_bytes < mxq_layer_norm_backward_workspace_size(rows, cols)) return MXQ_ERR_INVALID_ARG;
    }
    DeviceInfo info;
    st = device_ok(&info);
    if (st != MXQ_OK) return st;
    if (rows == 0) {   // sums over no rows
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols) * 4, cu(stream));
        if (e == cudaSuccess && dshift) e = cudaMemsetAsync(dshift, 0, static_cast<size_t>(cols) * 4, cu(stream));
        return from_cuda(e);
    }
    return from_cuda(mxq::launch_layer_norm_backward({rows, cols, lddy, ldx, lddx, dy, x, weight, mean, rstd, dx,
                                                      dweight, dshift, static_cast<float*>(workspace),
                                                      info.status},
                                                     dtype == MXQ_F32, param_dtype == MXQ_F32, cu(stream)));
}

size_t mxq_grad_norm_workspace_size(int32_t count) {
    if (count < 0 || count > MXQ_MAX_GRADS) return 0;
    return static_cast<size_t>(mxq::clip_partials(count)) * sizeof(float);
}

mxq_status mxq_grad_norm(const mxq_grad_desc* grads, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                         mxq_stream_t stream) {
    return clip(grads, count, false, 0.0f, 0.0f, norm, workspace, workspace_bytes, stream);
}

mxq_status mxq_clip_grad_norm(const mxq_grad_desc* grads, int32_t count, float max_norm, float eps, float* norm,
                              void* workspace, size_t workspace_bytes, mxq_stream_t stream) {
    return clip(grads, count, true, max_norm, eps, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
