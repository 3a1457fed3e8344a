// fp4_recorder.cpp -- the stand-in for the CUDA runtime of launch_recorder.cpp with the calls of MXFP4 quantization, of a
// payload's values and of the activation, on a device of as many SMs as the test says.

#include "launch_recorder.cpp"

namespace {
int sms = 152;
}

extern "C" {

cudaError_t cudaMemset2DAsync(void*, size_t, int, size_t, size_t, cudaStream_t) { return cudaSuccess; }

// Of api.cu, which is not linked: as documented.
size_t mxq_scale_bytes(int64_t rows, int64_t cols, mxq_scale_layout layout) {
    if (layout == MXQ_SCALE_ROWMAJOR) return static_cast<size_t>(rows * (cols / 32));
    return static_cast<size_t>((rows + 127) / 128 * ((cols / 32 + 3) / 4) * 512);
}

void rec_sms(int n) { sms = n; }

int rec_quant4(int dtype, int64_t batch, int64_t rows, int64_t cols, int copies) {
    return mxq_quant_mxfp4(place(0), static_cast<mxq_dtype>(dtype), batch, rows, cols, cols, rows * cols, copies & 1 ? place(1) : nullptr,
                           copies & 1 ? place(2) : nullptr, copies & 2 ? place(3) : nullptr, copies & 2 ? place(4) : nullptr,
                           MXQ_SCALE_MMA_TILED, nullptr);
}

int rec_quant4_grouped(int dtype, int64_t rows, int64_t cols, int G, int columns) {
    const int64_t bands = (rows + 127) / 128 + G;
    const int64_t* offsets = static_cast<const int64_t*>(place(1));
    return columns ? mxq_quant_mxfp4_cols_grouped(place(0), static_cast<mxq_dtype>(dtype), rows, cols, cols, offsets, G, 128 * bands,
                                                  place(2), place(3), nullptr)
                   : mxq_quant_mxfp4_grouped(place(0), static_cast<mxq_dtype>(dtype), rows, cols, cols, offsets, G, bands, place(2),
                                             place(3), nullptr);
}

int rec_values(int dtype, int element, int64_t rows, int64_t cols) {
    return mxq_dequant_1x32(place(0), place(1), static_cast<mxq_element>(element), rows, cols, (cols + 31) / 32 * 32, 0, MXQ_SCALE_MMA_TILED,
                            place(2), static_cast<mxq_dtype>(dtype), cols, nullptr);
}

int rec_act(int dtype, int64_t rows, int64_t inter, int backward) {
    const mxq_dtype t = static_cast<mxq_dtype>(dtype);
    return backward ? mxq_activation_backward(place(0), t, inter, place(1), place(2), rows, inter, MXQ_ACT_GELU, 1, place(3), 2 * inter,
                                              place(4), inter, nullptr)
                    : mxq_activation(place(0), t, rows, inter, 2 * inter, MXQ_ACT_SILU, 1, place(1), inter, place(2), place(3), nullptr);
}

}  // extern "C"

namespace mxq {
cudaError_t current_device_sms(int* n) {
    *n = sms;
    return cudaSuccess;
}
// The products, which are not linked.
cudaError_t launch_gemm_mxfp4(const DeviceInfo&, const Gemm4Args&, cudaStream_t) { return cudaErrorInvalidValue; }
cudaError_t launch_grouped_wgrad_mxfp4(const DeviceInfo&, const Gemm4Args&, int64_t, cudaStream_t) { return cudaErrorInvalidValue; }
}  // namespace mxq
