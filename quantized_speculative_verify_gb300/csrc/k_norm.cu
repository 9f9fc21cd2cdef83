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
// The 1/sqrt(32) enters sx alone: the codes are rint(127 z / max|z|) for any
// factor of z.  w holds the weight with the feature's sign, so the butterfly
// starts from the product, and h takes the sign back.
//
// One thread block per row at a time; a thread holds octets of 8 consecutive
// features (one 16-byte load of 16-bit values, two of fp32), so butterfly
// strides 1, 2 and 4 stay inside the thread and strides 8 and 16 are two lane
// exchanges.  What bounds it: few rows, the chain load - reduction - store (128
// rows of 8192: 6.8 us, 6.3 of which one row takes).  With more rows than
// resident blocks a block takes several in turn, weight and signs stay in
// registers and each thread copies its share of the next two rows into a ring
// in shared memory.  Then the instructions bound it, not the memory: 8190 rows
// of 8192, all bf16, 112 us = 5.4 TB/s at 400 instructions a warp and row, four
// fifths of the issue slots used.  On the way there: one row per block 232 us
// (the memory idle during reductions); a loop with the next row in registers
// 148; the ring 145; types known at compile time 115; the largest value by one
// instruction 111.  (At that step two octets a thread and half the threads took
// 106 in bf16, but 240 instead of 183 with x in fp32.)  The types are known where
// residual and h are of one 16-bit type and x of the same or fp32 (8192 rows of
// 8192, x in fp32, the others in bf16: 152 us); any others take the general code
// (all in fp32: 251 us).
// Everything is fp32 until the outputs: residual_out, h and the codes are
// rounded once each.
#include "rows.cuh"

namespace hq {
namespace {

// The range in which a row's sum of squares and largest |z| are taken as they
// are.  Below it squares, or quotients by it, leave fp32's range; a sum of squares
// that overflows is above it.  Rows outside are formed again (form_again) in units
// of 2^e, the power of two above their largest |s|: sums and codes of 2^-e s, with
// eps and 1/rms to match.
constexpr float SUM_LEAST = 0x1p-80f, MAX_LEAST = 0x1p-110f;
constexpr float MAX_CODED = 0x1p-120f;  // 127 / it is finite
// They need the row's inputs once more.  Without a ring, a 16-bit input that
// residual_out lies over is kept in shared memory (an fp32 residual_out is s itself).
enum { KEEP_NONE = 0, KEEP_X = 1, KEEP_R = 2 };

// 8 weights with the features' signs (sg: the signs).
__device__ __forceinline__ void load_weight(const NormArgs &a, int idx, float (&w)[8], uint32_t &sg) {
    sg = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
    if (idx < a.K >> 3) {
        widen(load_raw(a.weight, HQ_F32, idx), HQ_F32, w);
        if (a.sx) sg = (__ldg(a.signs + (idx >> 2)) >> ((idx & 3) * 8)) & 0xffu;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = flip(w[i], (sg >> i) & 1u);
}

// A whole row by the block in three passes over its inputs: rows that are not
// finite, and those described at SUM_LEAST (without codes, rows of zeros too).
// in: the row in the ring, xu and ru pieces an octet; without one (DIRECT), the
// input that residual_out lies over and has replaced.  s_far: 3 T / 32 floats.
//
// It must not take registers from the rows of the common kind: without a ring it
// is called (1 row of 4096: 3.5 us as before), in the loop over the ring a call
// costs every row 60 %, so it is inlined there, with the weights read again after
// it.  Without such rows' code and with it, 8192 rows: of 8192 in bf16 113 and 117
// us, with fp32 x 148 and 152; of 12288 197 and 217, with fp32 x 267 and 295.
template <int T, bool DIRECT>
__device__ __forceinline__ void form_again(const NormArgs &a, int row, int MT, const uint8_t *in, int xu, int ru, int *s_gs,
                                           float *s_far) {
    int tid = threadIdx.x, K = a.K, G = a.G;
    float eps = a.eps;
    asm volatile("" : "+r"(tid), "+r"(K), "+r"(G), "+f"(eps));  // nothing of this is worked out ahead, in registers of every row
    const int lane = tid & 31, n8 = K >> 3;
    const bool quant = a.sx != nullptr;
    const Codes<DIRECT> codes(a, K, G, MT, s_gs);
    const bool s_out = DIRECT && a.res_out && a.r_type == HQ_F32 && (a.res_out == a.res || a.res_out == a.x);
    auto load = [&](int j, float (&s)[8]) {  // s of octet j T + tid
        const int idx = j * T + tid;
        float r[8];
        Raw x = {}, y = {};
        if (idx < n8) {
            if (!DIRECT) {
                const uint4 *d = reinterpret_cast<const uint4 *>(in) + (size_t)j * (xu + ru) * T + tid;
                x.u = d[0];
                if (xu == 2) x.v = d[T];
                if (ru) y.u = d[xu * T];
                if (ru == 2) y.v = d[(xu + 1) * T];
            } else if (s_out) {
                x = load_raw(row_of(a.res_out, HQ_F32, a.ldr, row), HQ_F32, idx);
            } else {
                if (a.keep && a.x == a.res_out) x.u = reinterpret_cast<const uint4 *>(in)[idx];
                else x = load_raw(row_of(a.x, a.x_type, a.ldx, row), a.x_type, idx);
                if (a.keep && a.res == a.res_out) y.u = reinterpret_cast<const uint4 *>(in)[idx];
                else if (a.res) y = load_raw(row_of(a.res, a.r_type, a.ldr, row), a.r_type, idx);
            }
        }
        widen(x, s_out ? HQ_F32 : a.x_type, s);
        widen(y, a.r_type, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += r[i];
    };
    float s[8], u[8], ss = 0.0f, amax = 0.0f, top = 0.0f;
    uint32_t signs;
#pragma unroll 1
    for (int j = 0; j * T < n8; ++j) {
        load(j, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(s[i]));
    }
    top = warp_max(top);
    if (lane == 0) s_far[tid >> 5] = top;
    __syncthreads();
    top = warp_max(lane < T / 32 ? s_far[lane] : 0.0f);
    float down = 1.0f, rest = 1.0f, rstd = -1.0f;
    if (top > 0.0f && top < INFINITY) {
        // 2^(e - 1) <= top < 2^e; 2^-e as two factors, each of them a float
        const bool small = top < 0x1p-60f;
        const int e = (__float_as_int(small ? top * 0x1p80f : top) >> 23) - (small ? 206 : 126), half = e / 2;
        down = __int_as_float((127 - half) << 23);
        rest = __int_as_float((127 - e + half) << 23);
        // eps in the units of s^2; where it is all that counts, 1/rms itself
        const float root = sqrtf(eps), q = root * down * rest;
        if (q < 0x1p60f)
            eps = q * q;
        else
            rstd = 1.0f / root * __int_as_float((127 + half) << 23) * __int_as_float((127 + e - half) << 23);
    }
#pragma unroll 1
    for (int j = 0; j * T < n8; ++j) {
        load(j, s);
        load_weight(a, j * T + tid, u, signs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = s[i] * down * rest;
            ss = fmaf(s[i], s[i], ss);
            s[i] *= u[i];
        }
        if (quant) rotate8(s, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(s[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    amax = warp_max(amax);
    if (lane == 0) {
        s_far[T / 32 + (tid >> 5)] = ss;
        s_far[2 * (T / 32) + (tid >> 5)] = amax;
    }
    __syncthreads();
    ss = lane < T / 32 ? s_far[T / 32 + lane] : 0.0f;
    amax = warp_max(lane < T / 32 ? s_far[2 * (T / 32) + lane] : 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (rstd < 0.0f) {  // (an all-zero row with eps = 0 gives zeros)
        const float d = ss * (1.0f / (float)K) + eps;
        rstd = d == 0.0f ? 0.0f : 1.0f / sqrtf(d);
    }
    // A row with an infinity has sx = NaN, whatever the butterfly made of it
    // (infinities of both signs cancel to NaN, and 1/rms is 0).
    if (quant && tid == 0)
        a.sx[row] = isfinite(ss) ? rstd * (amax * __int_as_float((int)HADAMARD_SCALE_BITS) / 127.0f) : __int_as_float(0x7fffffff);
    // No codes for maxima that are 0 (the weight's doing, next to it too), NaN or
    // infinite: 0 * z, 0 * infinity and NaN round to 0.
    const float inv = amax >= MAX_CODED ? 127.0f / amax : 0.0f;
#pragma unroll 1
    for (int j = 0; j * T < codes.n8pad; ++j) {
        const int idx = j * T + tid;
        load(j, s);
        load_weight(a, idx, u, signs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = s[i] * down * rest * u[i];
            u[i] = s[i] * rstd;
        }
        if (idx < n8 && a.h) store8(const_cast<void *>(row_of(a.h, a.h_type, a.ldh, row)), a.h_type, idx, u, signs);
        if (!quant) continue;
        rotate8(s, lane);
        codes.write(row, a.qx ? a.qx + (size_t)row * K : nullptr, idx, s, inv);
    }
    codes.template write_sums<T>(row);
}

template <int T>
__device__ __noinline__ void form_again_call(const NormArgs &a, int row, int MT, const uint8_t *in, int *s_gs, float *s_far) {
    form_again<T, true>(a, row, MT, in, 0, 0, s_gs, s_far);
}

// Copies of 16 bytes into shared memory that the thread waits for by groups, in
// the order in which it committed them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Rows in the ring.  Two and three, 8192 rows, when they were compared: of 1024 in
// bf16 21.6 and 23.6 us, of 8192 in bf16 114 both, of 12288 in fp32 and bf16 321
// and (three do not fit) 400.  Now, with two: 16.7, 117 and 295.
constexpr int NSTAGES = 2;
constexpr int NORM_SMEM = 220 << 10;  // shared memory of an SM's blocks
constexpr int NORM_FIXED = 19 << 10;  // of which a block needs beside its ring, with the system's 1 KB

// RING: 0, or rows through the ring (no operand is written): of any types, or
// residual and h of one 16-bit type and x of the same or fp32 (a projection's
// output).
enum { DIRECT = 0, RING_ANY = 1, RING_F16 = 2, RING_BF16 = 3, RING_F32_F16 = 4, RING_F32_BF16 = 5 };
template <int V, int T, int RING>
__global__ void __launch_bounds__(T, 1024 / T) k_add_norm_quant(const NormArgs a) {
    extern __shared__ __align__(16) uint8_t s_ring[];  // [stage][16-byte piece of a thread's share][thread]
    __shared__ float s_sum[2][T / 32], s_max[2][T / 32];  // by the row's place in the ring
    __shared__ int s_gs[MAX_K / 16];  // group sums of this row
    __shared__ float s_far[3][T / 32];  // for form_again
    __shared__ NormArgs s_args;         // for form_again_call
    int row = blockIdx.x;
    const int MT = gridDim.x, tid = threadIdx.x, lane = tid & 31;
    const int K = a.K, n8 = K >> 3;
    const bool quant = a.sx != nullptr;
    const Codes<RING == DIRECT> codes(a, K, a.G, MT, s_gs);
    constexpr int ONE = RING == RING_F16 || RING == RING_F32_F16 ? HQ_F16 : RING == RING_BF16 || RING == RING_F32_BF16 ? HQ_BF16 : -1;
    const int x_type = RING >= RING_F32_F16 ? HQ_F32 : ONE >= 0 ? ONE : a.x_type;
    const int r_type = ONE >= 0 ? ONE : a.r_type, h_type = ONE >= 0 ? ONE : a.h_type;
    const float inv_k = 1.0f / (float)K;

    if (row >= a.M) {  // padding row of the operand
        pdl_wait();
        codes.template pad<T>(row);
        pdl_launch_dependents();
        return;
    }

    // weight and signs are not outputs of the kernel before this one.  w: the
    // weight with the feature's sign, sg: the signs
    float w[V][8];
    uint32_t sg[V];
#pragma unroll
    for (int j = 0; j < V; ++j) load_weight(a, tid + j * T, w[j], sg[j]);
    if (RING == DIRECT && tid == 0) s_args = a;
    pdl_wait();
    Raw xn[V], rn[V];
    auto fetch = [&](int r) {
        const void *xr = row_of(a.x, x_type, a.ldx, r);
        const void *rr = a.res ? row_of(a.res, r_type, a.ldr, r) : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            xn[j].u = xn[j].v = rn[j].u = rn[j].v = make_uint4(0, 0, 0, 0);
            if (idx >= n8) continue;
            xn[j] = load_raw(xr, x_type, idx);
            if (rr) rn[j] = load_raw(rr, r_type, idx);
        }
    };
    // The ring: each thread copies, waits for and reads its own octets only.
    const int xu = x_type == HQ_F32 ? 2 : 1, ru = ONE < 0 && !a.res ? 0 : r_type == HQ_F32 ? 2 : 1;
    const uint32_t stage_bytes = (uint32_t)(V * (xu + ru) * T * 16);
    auto issue = [&](int r, int st) {
        if (r < a.M) {
            const uint8_t *xr = static_cast<const uint8_t *>(row_of(a.x, x_type, a.ldx, r));
            const uint8_t *rr = ru ? static_cast<const uint8_t *>(row_of(a.res, r_type, a.ldr, r)) : nullptr;
            uint32_t d = smem_addr(s_ring) + (uint32_t)st * stage_bytes + (uint32_t)tid * 16;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int idx = tid + j * T;
                if (idx < n8) {
                    cp_async16(d, xr + (size_t)idx * xu * 16);
                    if (xu == 2) cp_async16(d + T * 16, xr + (size_t)idx * 32 + 16);
                    if (ru) cp_async16(d + xu * T * 16, rr + (size_t)idx * ru * 16);
                    if (ru == 2) cp_async16(d + (xu + 1) * T * 16, rr + (size_t)idx * 32 + 16);
                }
                d += (xu + ru) * T * 16;
            }
        }
        cp_async_commit();
    };
    auto take = [&](int st) {
        const uint8_t *d = s_ring + (size_t)st * stage_bytes + (size_t)tid * 16;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            xn[j].u = xn[j].v = rn[j].u = rn[j].v = make_uint4(0, 0, 0, 0);
            if (tid + j * T < n8) {
                xn[j].u = *reinterpret_cast<const uint4 *>(d);
                if (xu == 2) xn[j].v = *reinterpret_cast<const uint4 *>(d + T * 16);
                if (ru) rn[j].u = *reinterpret_cast<const uint4 *>(d + xu * T * 16);
                if (ru == 2) rn[j].v = *reinterpret_cast<const uint4 *>(d + (xu + 1) * T * 16);
            }
            d += (xu + ru) * T * 16;
        }
    };
    int stage = 0;
    if constexpr (RING != DIRECT)
        for (int i = 0; i < NSTAGES; ++i) issue(row + i * MT, i);
    static_assert(NSTAGES == 2, "a row's sums are read while the next one's are written");
    for (; row < a.M; row += MT) {
        if (codes.sums) {
            if (RING != DIRECT) __syncthreads();  // the last row's sums have been read
            codes.template clear_sums<T>();
        }
        if constexpr (RING != DIRECT) {
            asm volatile("cp.async.wait_group %0;" ::"n"(NSTAGES - 1) : "memory");
            take(stage);
        } else {
            fetch(row);
        }
        void *ro = a.res_out ? const_cast<void *>(row_of(a.res_out, r_type, a.ldr, row)) : nullptr;
        float v[V][8];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float r[8];
            widen(xn[j], x_type, v[j]);
            widen(rn[j], r_type, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] += r[i];
        }
        pdl_launch_dependents();
        float ss = 0.0f, amax = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            if (RING == DIRECT && a.keep) reinterpret_cast<uint4 *>(s_ring)[j * T + tid] = a.keep == KEEP_X ? xn[j].u : rn[j].u;
            if (ro && idx < n8) store8(ro, r_type, idx, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = fmaf(v[j][i], v[j][i], ss);
                v[j][i] *= w[j][i];
            }
        }
        // z: the rotated w * s
        float z[V][8];
        if (quant) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[j][i] = v[j][i];
                rotate8(z[j], lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(z[j][i]));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        amax = warp_max(amax);
        if (lane == 0) {
            s_sum[RING == DIRECT ? 0 : stage][tid >> 5] = ss;
            s_max[RING == DIRECT ? 0 : stage][tid >> 5] = amax;
        }
        __syncthreads();
        ss = lane < T / 32 ? s_sum[RING == DIRECT ? 0 : stage][lane] : 0.0f;
        amax = lane < T / 32 ? s_max[RING == DIRECT ? 0 : stage][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        amax = warp_max(amax);
        // (a row of zeros, padding of a batch, is of the common kind)
        if ((!(ss >= SUM_LEAST && ss < INFINITY) || (quant && !(amax >= MAX_LEAST && amax < INFINITY))) &&
            !(quant && ss == 0.0f && amax == 0.0f)) {
            if constexpr (RING == DIRECT) {
                form_again_call<T>(s_args, row, MT, s_ring, s_gs, &s_far[0][0]);
                return;
            }
            form_again<T, false>(a, row, MT, s_ring + (size_t)stage * stage_bytes, xu, ru, s_gs, &s_far[0][0]);
#pragma unroll
            for (int j = 0; j < V; ++j) load_weight(a, tid + j * T, w[j], sg[j]);  // (not held meanwhile)
            issue(row + NSTAGES * MT, stage);
            if (++stage == NSTAGES) stage = 0;
            continue;
        }
        if constexpr (RING != DIRECT) {  // what the thread took has been used
            issue(row + NSTAGES * MT, stage);
            if (++stage == NSTAGES) stage = 0;
        }
        const float rstd = 1.0f / sqrtf(fmaxf(ss * inv_k + a.eps, MAX_CODED));  // (finite for zeros)
        if (a.h) {
            void *hr = const_cast<void *>(row_of(a.h, h_type, a.ldh, row));
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int idx = tid + j * T;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = v[j][i] * rstd;
                if (idx < n8) store8(hr, h_type, idx, y, sg[j]);
            }
        }
        if (!quant) continue;
        if (tid == 0) a.sx[row] = rstd * (amax * __int_as_float((int)HADAMARD_SCALE_BITS) / 127.0f);
        const float inv = 127.0f / fmaxf(amax, MAX_CODED);
        int8_t *qr = a.qx ? a.qx + (size_t)row * K : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) codes.write(row, qr, tid + j * T, z[j], inv);
        codes.template write_sums<T>(row);
    }
}

template <int V, int T>
cudaError_t launch_norm_t(const NormArgs &a, bool pdl, cudaStream_t s) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    int dev = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> resident[CACHE_DEVICES];
    e = cached_per_device(resident, dev, &per_sm, [&](int *v) {
        for (auto f : {k_add_norm_quant<V, T, RING_ANY>, k_add_norm_quant<V, T, RING_F16>, k_add_norm_quant<V, T, RING_BF16>,
                       k_add_norm_quant<V, T, RING_F32_F16>, k_add_norm_quant<V, T, RING_F32_BF16>, k_add_norm_quant<V, T, DIRECT>}) {
            const cudaError_t r = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_SMEM - NORM_FIXED);
            if (r != cudaSuccess) return r;
        }
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, k_add_norm_quant<V, T, RING_ANY>, T, 0);
    });
    if (e != cudaSuccess) return e;
    if (per_sm < 1) per_sm = 1;
    const size_t kept = a.keep ? (size_t)V * T * 16 : 0;
    if (a.qop)  // one block per row of the operand, padding included
        return launch_kernel(k_add_norm_quant<V, T, DIRECT>, dim3((unsigned)act_rows(a.M)), dim3(T), kept, pdl, s, a);
    // the ring where blocks take several rows and its rows fit
    const int row_bytes = V * T * 8 * (type_bytes(a.x_type) + (a.res ? type_bytes(a.r_type) : 0));
    const int ring = NSTAGES * row_bytes;
    while (per_sm > 1 && ring > NORM_SMEM / per_sm - NORM_FIXED) --per_sm;
    const long long most = (long long)sms * per_sm;
    if (a.M <= most || ring > NORM_SMEM / per_sm - NORM_FIXED)
        return launch_kernel(k_add_norm_quant<V, T, DIRECT>, dim3((unsigned)a.M), dim3(T), kept, pdl, s, a);
    const bool one = a.res && a.r_type != HQ_F32 && (!a.h || a.h_type == a.r_type), wide = a.x_type == HQ_F32;
    auto f = k_add_norm_quant<V, T, RING_ANY>;
    if (one && a.r_type == HQ_F16 && (wide || a.x_type == HQ_F16))
        f = wide ? k_add_norm_quant<V, T, RING_F32_F16> : k_add_norm_quant<V, T, RING_F16>;
    else if (one && a.r_type == HQ_BF16 && (wide || a.x_type == HQ_BF16))
        f = wide ? k_add_norm_quant<V, T, RING_F32_BF16> : k_add_norm_quant<V, T, RING_BF16>;
    return launch_kernel(f, dim3((unsigned)most), dim3(T), (size_t)ring, pdl, s, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &args, bool pdl, cudaStream_t s) {
    NormArgs a = args;
    a.keep = !a.res_out || a.r_type == HQ_F32 ? KEEP_NONE : a.res_out == a.x ? KEEP_X : a.res_out == a.res ? KEEP_R : KEEP_NONE;
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
