// rows.cuh -- device helpers of the kernels that norm or gate rows and form their
// codes (k_norm.cu, k_gate.cu): octets of a row of any type, the rotation of a
// 32-block, codes and group sums where the GEMM wants them.
#pragma once

#include "act_common.cuh"
#include "batch.cuh"

namespace hq {

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

// `signs`: bit i set, value i is negated.
__device__ __forceinline__ void store8(void *row, int type, int octet, const float (&v)[8], uint32_t signs = 0) {
    if (type == HQ_F32) {
        float4 *p = static_cast<float4 *>(row) + 2 * (size_t)octet;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = flip(v[i], (signs >> i) & 1u);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
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
        // the pair's signs: its two bits, 15 apart after the product
        w[i] ^= (((signs >> (2 * i)) & 3u) * 0x40008000u) & 0x80008000u;
    }
    static_cast<uint4 *>(row)[octet] = make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger value, the largest of the warp's lanes; NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Four integers in [-128, 127] as bytes, x0 lowest.
__device__ __forceinline__ uint32_t pack_s8(int x0, int x1, int x2, int x3) {
    uint32_t hi, d;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(x3), "r"(x2));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(x1), "r"(x0), "r"(hi));
    return d;
}

// The rotation of a 32-block, without its factor: 8 consecutive values a lane,
// four lanes a block.
__device__ __forceinline__ void rotate8(float (&z)[8], int lane) {
#pragma unroll
    for (int st = 1; st <= 4; st <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i & st) == 0) {
                const float p = z[i], q = z[i + st];
                z[i] = p + q;
                z[i + st] = p - q;
            }
#pragma unroll
    for (int lb = 1; lb <= 2; lb <<= 1) {
        // lower lane a + b, upper lane a - b: one exact multiply-add
        const float sign = (lane & lb) != 0 ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = fmaf(sign, z[i], __shfl_xor_sync(0xffffffffu, z[i], lb));
    }
}

__device__ __forceinline__ const void *row_of(const void *p, int type, int64_t ld, int row) {
    return static_cast<const uint8_t *>(p) + (size_t)row * (size_t)ld * type_bytes(type);
}

// The range in which a head's sum of squares is taken as it is; head_norm forms
// others again in units of a power of two.
constexpr float HEAD_LEAST = 0x1p-80f, HEAD_EPS = 0x1p-60f;

// x / sqrt(mean(x^2) + eps) of a head whose octets lie in U consecutive lanes
// (8, 16 or 32); every lane of the warp calls.  rsqrtf is off by 2 units in the
// last place, far below the rounding of 16-bit outputs.  A head of zeros stays
// zeros, with eps = 0 too; one with an infinity gives zeros and NaN, as the
// formula does.
template <int U>
__device__ __forceinline__ void head_norm(float (&x)[8], float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = U / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    // squares below fp32's range count for nothing beside an eps above it
    const bool fine = ss < INFINITY && (ss >= HEAD_LEAST || eps >= HEAD_EPS);
    float r = rsqrtf(fmaf(ss, 1.0f / (8 * U), eps));
    if (__any_sync(0xffffffffu, !fine)) {
        float top = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(x[i]));
#pragma unroll
        for (int o = U / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        float down = 1.0f, rest = 1.0f;
        const bool scaled = top > 0.0f && top < INFINITY;
        if (scaled) {
            // 2^(e - 1) <= top < 2^e; 2^-e as two factors, each of them a float
            const bool small = top < 0x1p-60f;
            const int e = (__float_as_int(small ? top * 0x1p80f : top) >> 23) - (small ? 206 : 126), half = e / 2;
            down = __int_as_float((127 - half) << 23);
            rest = __int_as_float((127 - e + half) << 23);
        }
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = x[i] * down * rest;
            s2 = fmaf(u[i], u[i], s2);
        }
#pragma unroll
        for (int o = U / 2; o > 0; o >>= 1) s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        if (!fine) {
            const float root = sqrtf(eps), q = root * down * rest;  // sqrt(eps) in the same units
            if (!scaled) {
                r = top == INFINITY ? 0.0f : top;  // (0 for zeros)
            } else if (q < 0x1p60f) {
                r = rsqrtf(fmaf(s2, 1.0f / (8 * U), q * q));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = u[i];
            } else {
                r = 1.0f / root;  // eps is all that counts
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r;
}

// A row's codes and group sums, where they go (OPERAND: into the GEMM's operand
// too, whose layout hq_internal.cuh has: K tiles of code blocks, then group sums).
template <bool OPERAND>
struct Codes {
    const NormArgs &a;
    int *s_gs;  // group sums of the row, in shared memory
    int MT, n8, n8pad, bpt, gpt, ngk, ngp, cb;
    size_t tb;
    bool sums;
    __device__ __forceinline__ Codes(const NormArgs &a, int K, int G, int MT, int *s_gs) : a(a), s_gs(s_gs), MT(MT) {
        n8 = K >> 3;
        n8pad = act_blocks(K) * (ACT_BLOCK / 8);
        bpt = act_kt(G) / ACT_BLOCK, gpt = act_kt(G) / G, ngk = K / G, ngp = act_ktiles(K, G) * gpt;
        cb = MT * (a.rs ? ACT_RS_PITCH : 256);
        tb = (size_t)bpt * cb + (a.sums ? (size_t)gpt * MT * 4 : 0);
        sums = a.gsum != nullptr || (OPERAND && a.qop != nullptr && a.sums != 0);
    }
    // 8 features from 8 idx on
    __device__ __forceinline__ void put(int row, int idx, uint4 codes16, uint2 lo, uint2 hi) const {
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
    }
    __device__ __forceinline__ void put_sum(int row, int g, float v) const {
        reinterpret_cast<float *>(a.qop + (size_t)(g / gpt) * tb + (size_t)bpt * cb)[(size_t)(g % gpt) * MT + row] = v;
    }
    template <int T>
    __device__ __forceinline__ void pad(int row) const {  // a row past the last
        for (int idx = threadIdx.x; idx < n8pad; idx += T) put(row, idx, make_uint4(0, 0, 0, 0), make_uint2(0, 0), make_uint2(0, 0));
        if (a.sums)
            for (int g = threadIdx.x; g < ngp; g += T) put_sum(row, g, 0.0f);
    }
    template <int T>
    __device__ __forceinline__ void clear_sums() const {
        for (int g = threadIdx.x; g < ngk; g += T) s_gs[g] = 0;
    }
    // The codes of an octet of the rotated row; inv: 127 / max|z|.
    __device__ __forceinline__ void write(int row, int8_t *qr, int idx, const float (&z)[8], float inv) const {
        int q[8], gs = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // |z| <= amax, 127 / amax is finite: the product rounds to at most 127
            q[i] = idx < n8 ? __float2int_rn(z[i] * inv) : 0;
        }
        if (qr && idx < n8)
            reinterpret_cast<uint2 *>(qr)[idx] =
                make_uint2(pack_s8(q[0], q[1], q[2], q[3]), pack_s8(q[4], q[5], q[6], q[7]));
        if (OPERAND && a.qop && idx < n8pad) {
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
            put(row, idx, c16, lo, hi);
        }
        // a group's G / 8 threads are consecutive lanes (G = 16: two lanes)
        if (sums) {
#pragma unroll
            for (int i = 0; i < 8; ++i) gs += q[i];
            const int width = a.G / 8 < 32 ? a.G / 8 : 32;
            for (int o = width / 2; o > 0; o >>= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
            if (idx < n8 && (threadIdx.x & (width - 1)) == 0) atomicAdd(&s_gs[(idx * 8) / a.G], gs);
        }
    }
    template <int T>
    __device__ __forceinline__ void write_sums(int row) const {
        if (!sums) return;
        __syncthreads();
        for (int g = threadIdx.x; g < ngp; g += T) {
            const int v = g < ngk ? s_gs[g] : 0;
            if (a.gsum && g < ngk) a.gsum[(size_t)row * ngk + g] = v;
            if (OPERAND && a.qop && a.sums) put_sum(row, g, (float)v);
        }
    }
};

}  // namespace hq
