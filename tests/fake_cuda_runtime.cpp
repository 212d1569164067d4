// fake_cuda_runtime.cpp -- what the channel operators' translation units call
// of the CUDA runtime and of the rest of the library, for tests of their host
// side without a GPU: launches are written down and can be made to fail.
#include <cuda.h>
#include <cuda_runtime_api.h>

#include <vector>

#include "channel.h"

namespace {
struct Launch {
    int64_t grid, block, smem, kernel, cluster;
};
std::vector<Launch> launches;
int fail_at = -1;                         // this launch fails
cudaError_t last_error = cudaSuccess;

cudaError_t launch(const void *kernel, dim3 grid, dim3 block, size_t smem, int cluster) {
    launches.push_back({(int64_t)grid.x * grid.y * grid.z, (int64_t)block.x * block.y * block.z, (int64_t)smem,
                        (int64_t)kernel, cluster});
    if ((int)launches.size() - 1 != fail_at) return cudaSuccess;
    return last_error = cudaErrorLaunchOutOfResources;
}

CUresult encode(...) { return CUDA_SUCCESS; }
int status_word;
}  // namespace

extern "C" {
// fail: number of the launch to fail (-1: none); stale: an error some earlier call left behind
void fake_reset(int fail, int stale) {
    launches.clear();
    fail_at = fail;
    last_error = stale ? cudaErrorInvalidValue : cudaSuccess;
}
int fake_launches(int64_t *out, int most) {
    for (int i = 0; i < (int)launches.size() && i < most; ++i) {
        out[5 * i] = launches[i].grid, out[5 * i + 1] = launches[i].block, out[5 * i + 2] = launches[i].smem;
        out[5 * i + 3] = launches[i].kernel, out[5 * i + 4] = launches[i].cluster;
    }
    return (int)launches.size();
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **) {
    int cluster = 0;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = (int)c->attrs[i].val.clusterDim.x;
    return launch(f, c->gridDim, c->blockDim, c->dynamicSmemBytes, cluster);
}
cudaError_t __cudaLaunchKernel(cudaKernel_t f, dim3 grid, dim3 block, void **, size_t smem, cudaStream_t) {
    return launch(f, grid, block, smem, 0);
}
cudaError_t cudaGetLastError(void) {
    const cudaError_t e = last_error;
    last_error = cudaSuccess;
    return e;
}
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaGetDevice(int *d) {
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
    *f = (void *)encode;
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) {
    *k = (cudaKernel_t)f;
    return cudaSuccess;
}
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
void **__cudaRegisterFatBinary(void *) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *, void *, int *) {}
}

namespace i8c {
conv_status check_device() { return CONV_OK; }
uint64_t wait_limit_ns() { return 1000000000; }
int device_sm_count() { return 152; }
int *device_status_word() { return &status_word; }
}  // namespace i8c
