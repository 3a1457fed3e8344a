// mxq_internal.h -- host-side launchers shared between the C ABI (api.cu)
// and the kernel translation units.  Not part of the public interface.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mxq {

// Per-device facts the launchers need.
struct DeviceInfo {
    int device = -1;
    int sm_count = 0;
    int cc_major = 0, cc_minor = 0;
    size_t smem_optin = 0;            // max dynamic shared memory per block
    unsigned int* status = nullptr;   // device status word (timeouts)
};

// Returns cudaSuccess and fills `info` for the current device.
cudaError_t current_device_info(DeviceInfo* info);

// Whether the current device is an sm_103 (GB300): the one question of the calls that are
// made for single tokens, without the lookups of the above.
cudaError_t current_device_is_supported(bool* yes);
// The same with the device's SMs as the answer, 0 for another device.
cudaError_t current_device_sms(int* sms);

// Launches a kernel that begins with wait_for_previous(), so that its launch overlaps the end of the kernel
// before it on the stream (clipping 6 gradients 8.7 us to 8.2 us, 16384 x 64 layer norm backward 11.2 us to 10.6 us then).  Letting its
// blocks start before that end changes nothing more for these; the quantizers of MXFP4 do (let_next_start), for the products
// behind them.
template <typename... Params>
inline cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, unsigned block, unsigned shared,
                                 cudaStream_t stream, const std::remove_cv_t<Params>&... args) {
    if (shared > 48 * 1024) {   // a constant of the kernel at each call
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attribute{};
    attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attribute.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(block);
    config.dynamicSmemBytes = shared;
    config.stream = stream;
    config.attrs = &attribute;
    config.numAttrs = 1;
    void* addresses[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    return cudaLaunchKernelExC(&config, reinterpret_cast<const void*>(kernel), addresses);
}

// 2-D tensor map over a row-major matrix [outer, inner] of 1- or 2-byte
// elements with the given row stride, box [box_outer, box_inner].
bool encode_tensor_map_2d(CUtensorMap* map, const void* base, bool two_byte_elems, uint64_t inner,
                          uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner,
                          uint32_t box_outer, bool swizzle_128b);

// Bytes [rows, row_bytes] (row_bytes a multiple of 128) as [chunk][row][128 bytes], boxes of box_chunks x box_rows x
// 128 with the 128-byte swizzle.
bool encode_tensor_map_chunks(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows,
                              uint32_t box_chunks);

// 3-D tensor map [outer, mid, inner], box [1, box_mid, box_inner], no swizzle.
// BF16 [rows, cols] (row stride ld elements) for 32 x 32 tiled stores with the
// 64-byte swizzle.
bool encode_tensor_map_bf16_store(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                                  uint64_t ld);
// The same for 32 x 16 tiled stores with the 32-byte swizzle.
bool encode_tensor_map_bf16_store16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t ld);
// Bytes [rows, cols] (row stride ld bytes) for 32 x 32 tiled stores, no swizzle.
bool encode_tensor_map_u8_store(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t ld);
bool encode_tensor_map_3d(CUtensorMap* map, const void* base, bool two_byte_elems, uint64_t inner,
                          uint64_t mid, uint64_t outer, uint64_t mid_stride_bytes,
                          uint64_t outer_stride_bytes, uint32_t box_inner, uint32_t box_mid);

// 1x32 quantization of `batch` matrices [rows, cols] (row stride ld, matrix
// stride batch_stride elements); outputs of matrix b follow each other.
// fmt: 0 = E4M3, 1 = E5M2.
cudaError_t launch_quant_1x32(const DeviceInfo& dev, const void* x, int64_t batch, int64_t rows,
                              int64_t cols, int64_t ld, int64_t batch_stride, void* q_row,
                              void* s_row, void* q_col, void* s_col, bool tiled, int fmt,
                              cudaStream_t stream);

// Token-axis 1x32 quantization inside each expert (zero-padded, 128-aligned slots).
cudaError_t launch_quant_cols_grouped(const DeviceInfo& dev, const void* x, int64_t rows,
                                      int64_t cols, int64_t ld, const int64_t* offsets, int G,
                                      int64_t capacity, void* q_col, void* s_col, bool tiled, int fmt,
                                      cudaStream_t stream);

// 32x32 block quantization (fmt: 0 = E4M3, 1 = E5M2).
cudaError_t launch_quant_32x32(const DeviceInfo& dev, const void* w, int64_t n, int64_t k,
                               int64_t ld, void* q, void* s_fwd, void* s_bwd, bool tiled, int fmt,
                               cudaStream_t stream);

// One dense GEMM y = A B^T of a multi-GEMM launch (fields as in mxq_gemm_bf16out_fmt).
struct DenseGemm {
    const void* a_q;
    const void* a_s;
    const void* b_q;
    const void* b_s;
    int64_t M, N, K;
    void* y;
    int64_t ldy;
    int a_fmt, b_fmt;
};

// 1 to 4 dense GEMMs (all with B K-major, or all MN-major) in one persistent
// launch over their output tiles.  cudaErrorInvalidValue for a bad count or
// shapes whose tensor maps cannot be encoded.
cudaError_t launch_gemm_multi(const DeviceInfo& dev, const DenseGemm* gemms, int count, bool b_mn_major,
                              cudaStream_t stream);

// Dense block-scaled GEMM (see mxq_gemm_bf16out).  Returns cudaErrorInvalidValue
// when a tensor map cannot be encoded for the given shapes.
cudaError_t launch_gemm(const DeviceInfo& dev, const void* a_q, const void* a_s, const void* b_q,
                        const void* b_s, int64_t M, int64_t N, int64_t K, bool b_mn_major, void* y,
                        int64_t ldy, int a_fmt, int b_fmt, cudaStream_t stream);

// Dense GEMM whose epilogue also writes the 1x32 E4M3 quantization of the BF16
// output (y may be null: quantized output only).
cudaError_t launch_gemm_quant(const DeviceInfo& dev, const void* a_q, const void* a_s, const void* b_q,
                              const void* b_s, int64_t M, int64_t N, int64_t K, bool b_mn_major, void* y,
                              int64_t ldy, void* y_q, void* y_s, cudaStream_t stream);

// All-gather payload of a pre-quantized weight shard: tensor byte offsets in
// one rank's payload (offsets[2] = -1 for the 32x32 recipe) and its size.
// False when the shape is not supported (n % (128*world), k % 32).
bool fsdp_payload_layout(int recipe, int64_t n, int64_t k, int32_t world, int64_t offsets[4],
                         int64_t* payload_bytes);
cudaError_t launch_fsdp_unpack(const DeviceInfo& dev, int recipe, int64_t n, int64_t k, int32_t world,
                               const void* gathered, void* q_fwd, void* s_fwd, void* q_bwd, void* s_bwd,
                               cudaStream_t stream);

// a_bands_cap: 0 = A scales MMA-tiled over all rows; > 0 = group-tiled (see
// mxq_scale_regroup_rows) in a buffer of a_bands_cap bands.
cudaError_t launch_grouped_gemm(const DeviceInfo& dev, const void* a_q, const void* a_s,
                                const void* b_q, const void* b_s, const int64_t* offsets, int G,
                                int64_t M_total, int64_t N, int64_t K, int64_t a_bands_cap, void* y,
                                int64_t ldy, int a_fmt, int b_fmt, cudaStream_t stream);

// Group-tiled copy of the MMA-tiled scales of a row quantization (see
// mxq_scale_regroup_rows).
cudaError_t launch_scale_regroup_rows(const DeviceInfo& dev, const void* s_tiled, int64_t rows, int64_t cols,
                                      const int64_t* offsets, int G, int64_t bands_cap, void* s_out,
                                      cudaStream_t stream);

// Grouped contraction (MoE weight gradient): y[g] = A_g B_g^T where the K range
// of expert g is its 128-aligned token slot; A [M, capacity], B [N, capacity].
cudaError_t launch_grouped_gemm_wgrad(const DeviceInfo& dev, const void* a_q, const void* a_s,
                                      const void* b_q, const void* b_s, const int64_t* offsets, int G,
                                      int64_t M_total, int64_t capacity, int64_t M, int64_t N, void* y,
                                      int64_t ldy, int a_fmt, int b_fmt, cudaStream_t stream);

cudaError_t launch_wait_probe(const DeviceInfo& dev, uint64_t limit_ns, cudaStream_t stream);

// ---- the operators around the GEMMs (route.cu, permute.cu, norm.cu, clip.cu) ----

// Routing of tokens to experts (see mxq_route).  token_mask and bias may be null.
struct RouteArgs {
    int64_t tokens, ld;
    int experts, topk, n_group, topk_group, top2sum, renorm;
    float scale;
    const float* bias;
    const uint8_t* token_mask;
    int32_t* ids;
    float* weights;
};
cudaError_t launch_route(const void* logits, bool f32, const RouteArgs& a, bool softmax, cudaStream_t stream);

// Gradient of the routing weights by the logits (see mxq_route_backward).
struct RouteBackwardArgs {
    int64_t tokens, ld, ld_out;
    int experts, topk, renorm;
    float scale;
    const int32_t* ids;
    const float* dweights;
};
cudaError_t launch_route_backward(const void* logits, void* dlogits, bool f32, const RouteBackwardArgs& a,
                                  bool softmax, cudaStream_t stream);

// Expert order of the routed slots (see mxq_moe_plan).
cudaError_t launch_moe_plan(const int32_t* ids, int64_t slots, int experts, int64_t* offsets, int32_t* rows,
                            cudaStream_t stream);

// Rows of H elements of `tokens` tokens and of their tokens * k slots.
struct PermuteArgs {
    int64_t tokens, H;
    int k;
    const int32_t* rows;
    int64_t ld_tokens, ld_rows;   // row strides of the matrix by tokens and of the (written) matrix by rows
};
cudaError_t launch_moe_dispatch(const PermuteArgs& a, bool f32, const void* x, void* out, cudaStream_t stream);
cudaError_t launch_moe_combine(const PermuteArgs& a, bool f32, const void* y, const float* weights, void* out,
                               cudaStream_t stream);
cudaError_t launch_moe_combine_backward(const PermuteArgs& a, bool f32, const void* dout, const void* y, int64_t ldy,
                                        const float* weights, void* dy, float* dweights, cudaStream_t stream);

// Layer norm (see mxq_layer_norm).  weight and shift may be null.
struct NormArgs {
    int64_t rows, cols, ldx, ldy;
    const void *x, *weight, *shift;
    float eps;
    void* y;
    float *mean, *rstd;
};
cudaError_t launch_layer_norm(const NormArgs& a, bool f32, bool params_f32, cudaStream_t stream);

// Its backward pass: partial holds norm_partials(rows, cols) x 2 x cols floats.
int64_t norm_partials(int64_t rows, int64_t cols);
struct NormBackwardArgs {
    int64_t rows, cols, lddy, ldx, lddx;
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void* dx;
    float *dweight, *dshift, *partial;
    unsigned int* status;   // device status word
};
cudaError_t launch_layer_norm_backward(const NormBackwardArgs& a, bool f32, bool params_f32, cudaStream_t stream);

// Norm over all gradients and scaling to a largest norm (see mxq_clip_grad_norm).
struct ClipTensor {
    const void* in;
    void* out;
    int64_t n;
    bool f32;
};
constexpr int kClipBlocks = 1216;   // partial sums of one launch
int clip_partials(int count);
cudaError_t launch_clip(const ClipTensor* tensors, int count, bool scale_too, float max_norm, float eps, float* norm,
                        float* partial, cudaStream_t stream);

// ---- MXFP4, and activations kept in 8 bits (fp4.cu, gemm_fp4.cu, act.cu) ----

// MXFP4 quantization of `batch` matrices (see mxq_quant_mxfp4).  offsets, with one matrix and one copy: of the row copy the
// scales tiled by expert in bands_cap bands (see mxq_quant_mxfp4_grouped); the column copy inside each expert, in bands_cap
// slots of 128 rows (see mxq_quant_mxfp4_cols_grouped).
struct Quant4Args {
    const void* x;
    int64_t batch, rows, cols, ld, batch_stride;
    void *q_row, *s_row, *q_col, *s_col;      // either copy may be null
    int64_t s_row_bytes, s_col_bytes;         // of one matrix
    bool tiled;
    const int64_t* offsets;
    int G;
    int64_t bands_cap;
    int sms;                                  // of the device
};
cudaError_t launch_quant_mxfp4(const Quant4Args& a, bool f32, cudaStream_t stream);

// Values of a microscaled payload (see mxq_dequant_1x32); lds: row stride of plain scales.
struct Dequant4Args {
    const void *q, *s;
    int64_t rows, cols, ldq, lds;
    bool tiled;
    void* out;
    int64_t ldo;
};
cudaError_t launch_dequant(const Dequant4Args& a, int format, bool f32, cudaStream_t stream);

// Product of MXFP4 operands (see mxq_gemm_mxfp4, mxq_grouped_gemm_mxfp4); offsets null: dense.
struct Gemm4Args {
    const void *a_q, *a_s, *b_q, *b_s;
    int64_t M, N, K;
    void* y;
    int64_t ldy;
    const int64_t* offsets;
    int G;
    int64_t bands_cap;
};
cudaError_t launch_gemm_mxfp4(const DeviceInfo& dev, const Gemm4Args& a, cudaStream_t stream);
// Weight gradients of the experts (see mxq_grouped_gemm_mxfp4_wgrad): K is the capacity, y [G, M, N]; rows: of the
// token-sorted inputs.
cudaError_t launch_grouped_wgrad_mxfp4(const DeviceInfo& dev, const Gemm4Args& a, int64_t rows, cudaStream_t stream);

// The activation between two products (see mxq_activation); q and s null: nothing is kept.
struct ActArgs {
    int64_t rows, inter, ldz, ldy;
    const void* z;
    void *y, *q, *s;
};
cudaError_t launch_activation(const ActArgs& a, bool f32, int kind, bool gated, cudaStream_t stream);

// Its backward pass; y may be null.
struct ActBackwardArgs {
    int64_t rows, inter, lddy, lddz, ldy;
    const void *dy, *q, *s;
    void *dz, *y;
};
cudaError_t launch_activation_backward(const ActBackwardArgs& a, bool f32, int kind, bool gated, cudaStream_t stream);

}  // namespace mxq
