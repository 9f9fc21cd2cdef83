// k_norm.cu -- residual addition, RMS norm, rotation and int8 quantization of
// the rows that enter a quantized layer, in one pass.
//
//   s = x + r,  y = s * rstd * w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   z = the rotated w * s (32-blocks: sign flips, butterfly 1..16, 1/sqrt(32))
//   x' = rstd * z,  sx = rstd * max|z| / 127,  qx = rint(127 z / max|z|)
//
// rstd is one factor for the whole row, so the codes do not depend on it: the
// sum of squares and the largest |z| are reduced together, with one barrier,
// where norming first and rotating after needs two.
//
// One thread block per row at a time; a thread holds octets of 8 consecutive features
// (one 16-byte load of 16-bit values, two of fp32), so butterfly strides 1, 2
// and 4 stay inside the thread and strides 8 and 16 are two lane exchanges.
// With more rows than resident blocks a block takes several rows in turn: the
// next row's loads are issued before the reduction of the current one, and
// weight and signs stay in registers.  (One row per block left the memory idle
// during the reductions: 8190 rows of 8192, all bf16, 232 us = 2.6 TB/s; the
// loop: 154 us = 3.9 TB/s, then bound by issue slots.)
// Everything is fp32 until the outputs: residual_out, h and the codes are
// rounded once each.
#include "act_common.cuh"
#include "batch.cuh"

namespace hq {
namespace {

// 8 consecutive values of a row of type `type` (uniform over the block) as
// they lie in memory, and as floats.
struct Raw {
    uint4 u, v;  // v: fp32 only
};
__device__ __forceinline__ Raw load_raw(const void *row, int type, int octet) {
    Raw r;
    if (type == HQ_F32) {
        const uint4 *p = static_cast<const uint4 *>(row) + 2 * (size_t)octet;
        r.u = p[0];
        r.v = p[1];
    } else {
        r.u = static_cast<const uint4 *>(row)[octet];
        r.v = make_uint4(0, 0, 0, 0);
    }
    return r;
}
__device__ __forceinline__ void widen(const Raw &r, int type, float (&f)[8]) {
    const uint32_t w[8] = {r.u.x, r.u.y, r.u.z, r.u.w, r.v.x, r.v.y, r.v.z, r.v.w};
    if (type == HQ_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = type == HQ_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[i]))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
}

__device__ __forceinline__ void store8(void *row, int type, int octet, const float (&v)[8]) {
    if (type == HQ_F32) {
        float4 *p = static_cast<float4 *>(row) + 2 * (size_t)octet;
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (type == HQ_F16) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    static_cast<uint4 *>(row)[octet] = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ const void *row_of(const void *p, int type, int64_t ld, int row) {
    return static_cast<const uint8_t *>(p) + (size_t)row * (size_t)ld * type_bytes(type);
}

template <int V, int T>
__global__ void __launch_bounds__(T) k_add_norm_quant(const NormArgs a) {
    __shared__ float s_sum[2][T / 32], s_max[2][T / 32];  // by the parity of the row's turn
    __shared__ int s_gs[MAX_K / 16];  // group sums of this row
    int row = blockIdx.x;
    const int MT = gridDim.x, tid = threadIdx.x, lane = tid & 31;
    const int K = a.K, G = a.G, n8 = K >> 3;
    const bool quant = a.sx != nullptr;

    // the operand's layout (hq_internal.cuh): K tiles of code blocks, then group sums
    const int n8pad = act_blocks(K) * (ACT_BLOCK / 8);
    const int bpt = act_kt(G) / ACT_BLOCK, gpt = act_kt(G) / G, ngk = K / G, ngp = act_ktiles(K, G) * gpt;
    const int cb = MT * (a.rs ? ACT_RS_PITCH : 256);
    const size_t tb = (size_t)bpt * cb + (a.sums ? (size_t)gpt * MT * 4 : 0);
    auto put = [&](int idx, uint4 codes16, uint2 lo, uint2 hi) {  // 8 features from 8 idx on
        const int f = idx * 8, kb = f / ACT_BLOCK, fb = f % ACT_BLOCK;
        uint8_t *blk = a.qop + (size_t)(bpt == 1 ? kb : kb >> 1) * tb + (size_t)(bpt == 1 ? 0 : kb & 1) * cb;
        if (a.rs) {
            *reinterpret_cast<uint4 *>(blk + (size_t)row * ACT_RS_PITCH + (size_t)fb * 2) = codes16;
        } else if (a.e4) {
            uint8_t *d = blk + ((size_t)(fb / 16) * 2 * MT + row) * 16 + (size_t)(fb % 16);
            *reinterpret_cast<uint2 *>(d) = lo;
            *reinterpret_cast<uint2 *>(d + (size_t)MT * 16) = hi;
        } else {
            *reinterpret_cast<uint4 *>(blk + ((size_t)(fb / 8) * MT + row) * 16) = codes16;
        }
    };
    auto put_sum = [&](int g, float v) {
        reinterpret_cast<float *>(a.qop + (size_t)(g / gpt) * tb + (size_t)bpt * cb)[(size_t)(g % gpt) * MT + row] = v;
    };

    if (row >= a.M) {  // padding row of the operand
        pdl_wait();
        for (int idx = tid; idx < n8pad; idx += T) put(idx, make_uint4(0, 0, 0, 0), make_uint2(0, 0), make_uint2(0, 0));
        if (a.sums)
            for (int g = tid; g < ngp; g += T) put_sum(g, 0.0f);
        pdl_launch_dependents();
        return;
    }

    // weight and signs are not outputs of the kernel before this one
    float w[V][8];
    uint32_t sg[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int idx = tid + j * T;
        sg[j] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[j][i] = 0.0f;
        if (idx < n8) {
            widen(load_raw(a.weight, HQ_F32, idx), HQ_F32, w[j]);
            if (quant) sg[j] = (__ldg(a.signs + (idx >> 2)) >> ((idx & 3) * 8)) & 0xffu;
        }
    }
    pdl_wait();
    const bool need_gs = a.gsum != nullptr || (a.qop != nullptr && a.sums != 0);
    Raw xn[V], rn[V];  // the next row
    auto fetch = [&](int r) {
        const void *xr = row_of(a.x, a.x_type, a.ldx, r);
        const void *rr = a.res ? row_of(a.res, a.r_type, a.ldr, r) : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            xn[j].u = xn[j].v = rn[j].u = rn[j].v = make_uint4(0, 0, 0, 0);
            if (idx >= n8) continue;
            xn[j] = load_raw(xr, a.x_type, idx);
            if (rr) rn[j] = load_raw(rr, a.r_type, idx);
        }
    };
    constexpr bool AHEAD = V == 1;  // more octets a thread leave no registers for the next row
    for (int turn = 0; row < a.M; ++turn, row += MT) {
        if (need_gs) {
            if (turn) __syncthreads();  // the last row's sums have been read
            for (int g = tid; g < ngk; g += T) s_gs[g] = 0;
        }
        if (!AHEAD || turn == 0) fetch(row);
        void *ro = a.res_out ? const_cast<void *>(row_of(a.res_out, a.r_type, a.ldr, row)) : nullptr;
        float v[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float r[8];
            widen(xn[j], a.x_type, v[j]);
            widen(rn[j], a.r_type, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += r[i];
        }
        if (AHEAD && row + MT < a.M) fetch(row + MT);
        pdl_launch_dependents();
        float ss = 0.0f, amax = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            if (ro && idx < n8) store8(ro, a.r_type, idx, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(v[j][i], v[j][i], ss);
                v[j][i] *= w[j][i];
            }
        }
        // z: the rotated w * s
        float z[V][8];
        if (quant) {
            const float c = __int_as_float((int)HADAMARD_SCALE_BITS);
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[j][i] = flip(v[j][i], (sg[j] >> i) & 1u);
#pragma unroll
                for (int st = 1; st <= 4; st <<= 1)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if ((i & st) == 0) {
                            const float p = z[j][i], q = z[j][i + st];
                            z[j][i] = p + q;
                            z[j][i + st] = p - q;
                        }
#pragma unroll
                for (int lb = 1; lb <= 2; lb <<= 1) {
                    // lower lane a + b, upper lane a - b: one exact multiply-add
                    const float sign = (lane & lb) != 0 ? -1.0f : 1.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[j][i] = fmaf(sign, z[j][i], __shfl_xor_sync(0xffffffffu, z[j][i], lb));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[j][i] *= c;
                    amax = fmaxf(amax, fabsf(z[j][i]));
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        if (lane == 0) {
            s_sum[turn & 1][tid >> 5] = ss;
            s_max[turn & 1][tid >> 5] = amax;
        }
        __syncthreads();
        ss = lane < T / 32 ? s_sum[turn & 1][lane] : 0.0f;
        amax = lane < T / 32 ? s_max[turn & 1][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        // an all-zero row with eps = 0 gives zeros; NaN and infinities reach sx and h
        const float d = ss / (float)K + a.eps;
        const float rstd = d == 0.0f ? 0.0f : 1.0f / sqrtf(d);
        if (a.h) {
            void *hr = const_cast<void *>(row_of(a.h, a.h_type, a.ldh, row));
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int idx = tid + j * T;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = v[j][i] * rstd;
                if (idx < n8) store8(hr, a.h_type, idx, y);
            }
        }
        if (!quant) continue;
        if (tid == 0) a.sx[row] = rstd * (amax / 127.0f);
        const float inv = amax == 0.0f ? 0.0f : 127.0f / amax;

        int8_t *qr = a.qx ? a.qx + (size_t)row * K : nullptr;
        const int width = G / 8 < 32 ? G / 8 : 32;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            int q[8], gs = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // |z| <= amax: the product rounds to at most 127 (NaN to 0)
                q[i] = idx < n8 ? __float2int_rn(z[j][i] * inv) : 0;
                gs += q[i];
            }
            if (qr && idx < n8) {
                uint32_t lo = 0, hi = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo |= (uint32_t)(q[i] & 255) << (8 * i);
                    hi |= (uint32_t)(q[i + 4] & 255) << (8 * i);
                }
                reinterpret_cast<uint2 *>(qr)[idx] = make_uint2(lo, hi);
            }
            if (a.qop && idx < n8pad) {
                uint4 c16 = make_uint4(0, 0, 0, 0);
                uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
                if (a.e4) {
                    digits4(q[0], q[1], q[2], q[3], lo.x, hi.x);
                    digits4(q[4], q[5], q[6], q[7], lo.y, hi.y);
                } else {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2 p = __halves2half2(__int2half_rn(q[2 * i]), __int2half_rn(q[2 * i + 1]));
                        h[i] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                    c16 = make_uint4(h[0], h[1], h[2], h[3]);
                }
                put(idx, c16, lo, hi);
            }
            // a group's G / 8 threads are consecutive lanes (G = 16: two lanes)
            if (need_gs) {
                for (int o = width / 2; o > 0; o >>= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
                if (idx < n8 && (lane & (width - 1)) == 0) atomicAdd(&s_gs[(idx * 8) / G], gs);
            }
        }
        if (!need_gs) continue;
        __syncthreads();
        for (int g = tid; g < ngp; g += T) {
            const int v2 = g < ngk ? s_gs[g] : 0;
            if (a.gsum && g < ngk) a.gsum[(size_t)row * ngk + g] = v2;
            if (a.qop && a.sums) put_sum(g, (float)v2);
        }
    }
}

template <int V, int T>
cudaError_t launch_norm_t(const NormArgs &a, bool pdl, cudaStream_t s) {
    int grid = a.M;
    if (a.qop) {
        grid = act_rows(a.M);  // one block per row of the operand, padding included
    } else {
        const int sms = device_sm_count();
        if (sms <= 0) return cudaErrorNoDevice;
        int dev = 0, per_sm = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        static std::atomic<int> resident[CACHE_DEVICES];
        e = cached_per_device(resident, dev, &per_sm, [&](int *v) {
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, k_add_norm_quant<V, T>, T, 0);
        });
        if (e != cudaSuccess) return e;
        const int most = sms * (per_sm > 0 ? per_sm : 1);
        if (grid > most) grid = most;
    }
    return launch_kernel(k_add_norm_quant<V, T>, dim3((unsigned)grid), dim3(T), 0, pdl, s, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, bool pdl, cudaStream_t s) {
    const int n8 = a.K / 8;
    // As many threads as the row has octets, up to 1024: a row is one short
    // dependent chain.  Every V * T is a multiple of 16 octets, so the
    // operand's padding up to whole 128-feature blocks is covered too.
    if (n8 <= 128) return launch_norm_t<1, 128>(a, pdl, s);
    if (n8 <= 256) return launch_norm_t<1, 256>(a, pdl, s);
    if (n8 <= 512) return launch_norm_t<1, 512>(a, pdl, s);
    if (n8 <= 1024) return launch_norm_t<1, 1024>(a, pdl, s);
    if (n8 <= 2048) return launch_norm_t<2, 1024>(a, pdl, s);
    if (n8 <= 4096) return launch_norm_t<4, 1024>(a, pdl, s);
    if (n8 <= 8192) return launch_norm_t<8, 1024>(a, pdl, s);
    return cudaErrorInvalidValue;
}

}  // namespace hq
