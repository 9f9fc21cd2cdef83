// act_common.cuh -- device helpers of the kernels that rotate and quantize
// activations (k_act.cu, k_norm.cu): sign flips, butterfly stages, the e4m3
// digits of the GEMM's operand.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "hq_internal.cuh"

namespace hq {

__device__ __forceinline__ float flip(float x, uint32_t bit) {
    return __int_as_float(__float_as_int(x) ^ (int)(bit << 31));
}

// Stage h in {4, 8, 16}: lane partner = lane ^ (h / 4).  The lane holding the
// lower index keeps a + b, the other keeps a - b (a = lower, b = upper).
__device__ __forceinline__ float bfly_x(float v, int lane_bit, bool upper) {
    float p = __shfl_xor_sync(0xffffffffu, v, lane_bit);
    return upper ? __fsub_rn(p, v) : __fadd_rn(v, p);
}

// e4m3 byte of an integer v in [-8, 8] (exact): 1..8 are 2^e * (1 + m/8).
__device__ __forceinline__ uint32_t e4m3_small(int v) {
    const uint32_t a = (uint32_t)(v < 0 ? -v : v);
    if (a == 0) return 0u;
    const uint32_t e = 31u - __clz(a);          // 0..3
    const uint32_t m = ((a << 3) >> e) & 7u;    // mantissa bits
    return ((e + 7u) << 3) | m | (v < 0 ? 0x80u : 0u);
}
// Low and high e4m3 digits of four codes, one byte each.
__device__ __forceinline__ void digits4(int q0, int q1, int q2, int q3, uint32_t &lo, uint32_t &hi) {
    const int q[4] = {q0, q1, q2, q3};
    lo = hi = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int l = ((q[i] + 8) & 15) - 8;
        const int h = (q[i] - l) / 16;
        lo |= e4m3_small(l) << (8 * i);
        hi |= e4m3_small(h) << (8 * i);
    }
}

}  // namespace hq
