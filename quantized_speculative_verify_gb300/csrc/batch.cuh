// batch.cuh -- launchers and helpers of the calls for a batch of requests.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hq_internal.cuh"

namespace hq {

__host__ __device__ inline int type_bytes(int type) { return type == HQ_F32 ? 4 : 2; }

// A launch with programmatic dependent launch where `pdl` is set.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t s,
                          A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct NormArgs {
    const void *x, *res;
    void *res_out, *h;
    const float *weight;
    const uint32_t *signs;
    int8_t *qx;
    int32_t *gsum;
    uint8_t *qop;
    float *sx;
    int64_t ldx, ldr, ldh;
    float eps;
    int x_type, r_type, h_type;
    int M, K, G;
    int rs, e4, sums;  // encoding of the operand (hq_internal.cuh)
};
cudaError_t launch_norm(const NormArgs &a, bool pdl, cudaStream_t s);

struct LoraArgs {
    const void *x, *A, *B;
    const int32_t *ids, *ranks;
    const float *scale, *base;
    float *Y, *t;  // t: [M][r_max], the products A x
    int64_t ldx, ldb, ldy;
    int x_type, M, K, N, n_adapters, r_max;
};
cudaError_t launch_lora(const LoraArgs &a, int w_type, bool pdl, cudaStream_t s);

}  // namespace hq
