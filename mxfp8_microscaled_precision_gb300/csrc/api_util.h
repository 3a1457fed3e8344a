// api_util.h -- argument checks shared by the extern "C" entry points whose tensors may start at any
// element (api_block.cu, api_fp4.cu).  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq.h"
#include "mxq_internal.h"

namespace mxq {

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool bad_dtype(mxq_dtype d) { return d != MXQ_BF16 && d != MXQ_F32; }
inline size_t size_of(mxq_dtype d) { return d == MXQ_F32 ? 4 : 2; }

inline mxq_status device_ok(DeviceInfo* info) {
    if (current_device_info(info) != cudaSuccess) return MXQ_ERR_CUDA;
    return info->cc_major == 10 && info->cc_minor == 3 ? MXQ_OK : MXQ_ERR_UNSUPPORTED_DEVICE;
}

inline mxq_status device_ok() {
    bool yes = false;
    if (current_device_is_supported(&yes) != cudaSuccess) return MXQ_ERR_CUDA;
    return yes ? MXQ_OK : MXQ_ERR_UNSUPPORTED_DEVICE;
}

inline mxq_status device_ok(int* sms) {
    if (current_device_sms(sms) != cudaSuccess) return MXQ_ERR_CUDA;
    return *sms > 0 ? MXQ_OK : MXQ_ERR_UNSUPPORTED_DEVICE;
}

// The runtime keeps an error for the next cudaGetLastError: it is taken here, or it would be read as that
// of a later call's launch.
inline mxq_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return MXQ_OK;
    (void)cudaGetLastError();
    return MXQ_ERR_CUDA;
}

inline cudaStream_t cu(mxq_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 4096;   // rows of a launch: grids and int32 rows hold them
constexpr int64_t kMaxCols = int64_t(1) << 23;            // elements of a row: blocks along a row fit the grid's y

}  // namespace mxq
