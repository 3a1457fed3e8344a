// launch_recorder.cpp -- a stand-in for the CUDA runtime that writes down what the library's calls
// ask of it (kernels, shapes, shared memory, attributes) and can refuse one launch.  Linked with the
// library's own objects of the operators around the GEMMs it runs without a GPU.

#include <cuda_runtime.h>

#include <cstdint>
#include <map>
#include <string>
#include <vector>

#include "mxq.h"
#include "mxq_internal.h"

namespace {

std::map<const void*, std::string> names;   // of the kernels by their host functions
std::string text;                           // one line per request
int launches = 0, refused = 0;              // the launch that is refused, from 1 on; 0: none
cudaError_t pending = cudaSuccess;          // what cudaGetLastError gives next

struct Config {
    dim3 grid, block;
    size_t shared;
    cudaStream_t stream;
};
std::vector<Config> configs;

cudaError_t launch(const void* f, dim3 grid, dim3 block, size_t shared) {
    if (++launches == refused) return pending = cudaErrorInvalidValue;
    text += "launch " + names[f] + " " + std::to_string(static_cast<uint64_t>(grid.x) * grid.y * grid.z) + " " +
            std::to_string(block.x * block.y * block.z) + " " + std::to_string(shared) + "\n";
    return cudaSuccess;
}

void* place(int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(i + 1) << 40); }   // never dereferenced

}  // namespace

extern "C" {

void** __cudaRegisterFatBinary(void*) {
    static void* handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
    names[host] = name;
}
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t shared, cudaStream_t stream) {
    configs.push_back({grid, block, shared, stream});
    return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, void* stream) {
    const Config c = configs.back();
    configs.pop_back();
    *grid = c.grid, *block = c.block, *shared = c.shared, *static_cast<cudaStream_t*>(stream) = c.stream;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* kernel, const void* f) {
    *kernel = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
    return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t kernel, dim3 grid, dim3 block, void**, size_t shared, cudaStream_t) {
    return launch(reinterpret_cast<const void*>(kernel), grid, block, shared);
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    return launch(f, c->gridDim, c->blockDim, c->dynamicSmemBytes);
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attribute, int value) {
    text += "attribute " + names[f] + " " + std::to_string(static_cast<int>(attribute)) + " " + std::to_string(value) + "\n";
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t bytes, cudaStream_t) {
    text += "memset - " + std::to_string(bytes) + "\n";
    return cudaSuccess;
}
cudaError_t cudaGetLastError() {
    const cudaError_t e = pending;
    pending = cudaSuccess;
    return e;
}

// ---- what the tests call ---------------------------------------------------------------

void rec_begin(int refuse, int forget) {
    text.clear();
    launches = 0;
    refused = refuse;
    if (forget) pending = cudaSuccess;
}
const char* rec_text() { return text.c_str(); }
int rec_launches() { return launches; }

int rec_route(int64_t tokens, int experts, int k) {
    return mxq_route(place(0), MXQ_F32, tokens, experts, experts, nullptr, nullptr, MXQ_SCORE_SOFTMAX, 1, 1, MXQ_GROUP_MAX,
                     k, 1, 1.0f, static_cast<int32_t*>(place(1)), static_cast<float*>(place(2)), nullptr);
}

int rec_plan(int64_t tokens, int k, int experts) {
    return mxq_moe_plan(static_cast<const int32_t*>(place(0)), tokens, k, experts, static_cast<int64_t*>(place(1)),
                        static_cast<int32_t*>(place(2)), nullptr);
}

int rec_norm(int dtype, int params, int64_t rows, int64_t cols) {
    return mxq_layer_norm(place(0), static_cast<mxq_dtype>(dtype), rows, cols, cols, place(1), place(2),
                          static_cast<mxq_dtype>(params), 1e-5f, place(3), cols, static_cast<float*>(place(4)),
                          static_cast<float*>(place(5)), nullptr);
}

int rec_norm_backward(int dtype, int params, int64_t rows, int64_t cols) {
    return mxq_layer_norm_backward(place(0), place(1), static_cast<mxq_dtype>(dtype), rows, cols, cols, cols, place(2),
                                   static_cast<mxq_dtype>(params), static_cast<const float*>(place(3)),
                                   static_cast<const float*>(place(4)), place(5), cols, static_cast<float*>(place(6)),
                                   static_cast<float*>(place(7)), place(8),
                                   mxq_layer_norm_backward_workspace_size(rows, cols), nullptr);
}

int rec_clip(int count, int64_t numel, int scale_too) {
    std::vector<mxq_grad_desc> list(static_cast<size_t>(count));
    for (int i = 0; i < count; ++i) list[i] = {place(0), place(1), numel, i % 2 != 0 ? MXQ_F32 : MXQ_BF16};
    float* norm = static_cast<float*>(place(2));
    const size_t bytes = mxq_grad_norm_workspace_size(count);
    return scale_too != 0 ? mxq_clip_grad_norm(list.data(), count, 1.0f, 1e-6f, norm, place(3), bytes, nullptr)
                          : mxq_grad_norm(list.data(), count, norm, place(3), bytes, nullptr);
}

}  // extern "C"

// The device: a GB300, as far as the calls ask.
namespace mxq {
cudaError_t current_device_info(DeviceInfo* info) {
    *info = DeviceInfo{};
    info->sm_count = 152;
    info->cc_major = 10;
    info->cc_minor = 3;
    info->status = static_cast<unsigned int*>(place(20));
    return cudaSuccess;
}
cudaError_t current_device_is_supported(bool* yes) {
    *yes = true;
    return cudaSuccess;
}
}  // namespace mxq
