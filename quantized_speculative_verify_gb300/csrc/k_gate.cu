// k_gate.cu -- the norm per head with its gate, and the codes of the result for
// the output projection, in one pass over the rows.
//
//   y = x * w / sqrt(mean_head(x^2) + eps) * act(gate)
//   z = the rotated y (32-blocks, without the factor 1/sqrt(32))
//   sx = max|z| / sqrt(32) / 127,  qx = rint(127 z / max|z|)
//
// A head is 8, 16 or 32 lanes of 8 features, so the norm is lane exchanges and
// needs no barrier; only the codes need the row's largest value.  So h alone is one
// long list of octets over resident blocks, bound by memory and, nearly, by
// instructions: 8190 rows of 8192, all bf16, with a silu gate 75 us = 5.4 TB/s.  On
// the way there: an exact division and expf per gate 112 us; the quotient by the
// approximate reciprocal and the types known at compile time 83.  One, two and four
// octets a thread on their way 76, 74 and 94 us (registers end the fourth block an
// SM); five blocks an SM 88.  With codes few rows are one chain of waits (128 rows of
// 8192 4.3 us, 3.1 of which one row of 4096 takes), many are bound by instructions:
// 8190 rows of 8192 in bf16 111 us = 4.2 TB/s.  On the way there: a block per row 213;
// resident blocks with the next row's loads ahead 138; weights and signs in registers
// 130; types known at compile time 111.
#include "rows.cuh"

namespace hq {
namespace {

constexpr float MAX_LEAST = 0x1p-110f;  // below it a row's largest |z| is formed again

// 1 / (1 + e^-g) in nine instructions, two of them of the special unit: expf and a
// division with their care for subnormal results take 25 and bound the kernel.  e^-g
// = 2^t (1 + d), t = -g log2(e) as it is rounded and d = -g - t ln 2 what that left
// out, of the constant's own rounding too: below 2^-17 where 2^t is neither 0 nor
// infinite.  Past that d is large, infinite or (infinite g) NaN; the factor's bounds
// leave the 0 or infinity in front of it what it is.  The power is off by 2^-22, d by t
// times 2^-29 (ln 2 rounded; 2^-22 at the most), the reciprocal by one unit in the last
// place, with three roundings 13 * 2^-24 together; a quotient below 2^-126 is 0.
__device__ __forceinline__ float sigmoid(float g) {
    constexpr float L = -1.4426950408889634f, LN2 = 0.6931471805599453f;
    const float t = g * L, d = fmaf(t, -LN2, -g);
    float p, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.0f + p * fminf(fmaxf(1.0f + d, 0.99f), 1.01f)));
    return q;
}
__device__ __forceinline__ float gated(float y, float g, int act) {
    return act == HQ_GATE_NONE ? y * g : act == HQ_GATE_SILU ? y * (g * sigmoid(g)) : y * sigmoid(g);
}

// 8 weights of a head, 1 each where there are none.
template <int U>
__device__ __forceinline__ void load_weight(const GateArgs &a, int idx, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (a.n.weight) widen(load_raw(a.n.weight, HQ_F32, idx % U), HQ_F32, w);
}

// 8 features of y: head normed, weighted (ALWAYS: where there is no norm too),
// gated.
template <int U, bool ALWAYS = false>
__device__ __forceinline__ void form(const GateArgs &a, const Raw &rx, int x_type, const Raw &rg, int g_type, const float (&w)[8],
                                     float (&y)[8]) {
    widen(rx, x_type, y);
    if (a.n.weight) head_norm<U>(y, a.n.eps);
    if (ALWAYS || a.n.weight) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= w[i];
    }
    if (a.gate) {
        float g[8];
        widen(rg, g_type, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = gated(y[i], g[i], a.act);
    }
}

// h alone: heads are independent, so the rows' octets are one long list.
constexpr int FT = 256;    // threads
constexpr int FLIGHT = 2;  // octets of a thread on their way together

// XT, GT: the types of x, and of gate and h, where they are known at compile time
// (else -1).
template <int U, int XT, int GT>
__global__ void __launch_bounds__(FT, 4) k_gate_heads(const GateArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int x_type = XT >= 0 ? XT : a.n.x_type, g_type = GT >= 0 ? GT : a.g_type, h_type = GT >= 0 ? GT : a.n.h_type;
    const int n8 = a.n.K / 8, step = gridDim.x * FT;
    const long long total = (long long)a.n.M * n8, start = (long long)blockIdx.x * FT + threadIdx.x;
    long long row = start / n8;
    int idx = (int)(start % n8);
    float w[8];  // (steps are whole heads: the thread's features keep their place)
    load_weight<U>(a, idx, w);
    const int rows_on = step / n8, idx_on = step % n8;
    // A warp's 32 octets start at a multiple of 32; n8 is a multiple of 8, so the
    // last warp may have heads that are not there.
    for (long long base = start - (threadIdx.x & 31); base < total; base += (long long)step * FLIGHT) {
        Raw x[FLIGHT], g[FLIGHT];
        int rows[FLIGHT], at[FLIGHT];
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            x[k] = g[k] = Raw{};
            rows[k] = row < a.n.M ? (int)row : -1;
            at[k] = idx;
            if (rows[k] >= 0) {
                x[k] = load_raw(row_of(a.n.x, x_type, a.n.ldx, rows[k]), x_type, idx);
                if (a.gate) g[k] = load_raw(row_of(a.gate, g_type, a.ldg, rows[k]), g_type, idx);
            }
            row += rows_on;
            idx += idx_on;
            if (idx >= n8) {
                idx -= n8;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) {
            float y[8];
            form<U>(a, x[k], x_type, g[k], g_type, w, y);
            if (rows[k] >= 0) store8(const_cast<void *>(row_of(a.n.h, h_type, a.n.ldh, rows[k])), h_type, at[k], y);
        }
    }
}

// The largest of the block's values; NaN if one is.  Every thread calls; s_max is
// not in use by another call before the next barrier.
template <int T>
__device__ __forceinline__ float block_max(float x, float *s_max) {
    x = warp_max(x);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = x;
    __syncthreads();
    return warp_max((threadIdx.x & 31) < T / 32 ? s_max[threadIdx.x & 31] : 0.0f);
}

// h and codes.  ROWS: resident blocks take rows in turn, the next one's loads on
// their way while this one is rotated, reduced and written (no operand); else a
// block per row of the operand or the codes.  XT, GT as above.
template <int U, int V, int T, bool ROWS, int XT = -1, int GT = -1>
__global__ void __launch_bounds__(T, 1024 / T) k_gate_row(const GateArgs a) {
    const int x_type = XT >= 0 ? XT : a.n.x_type, g_type = GT >= 0 ? GT : a.g_type, h_type = GT >= 0 ? GT : a.n.h_type;
    __shared__ float s_max[2][T / 32], s_far[2][T / 32];  // by the row's turn; for rows of unusual size
    __shared__ int s_gs[MAX_K / 16];  // group sums of this row
    pdl_launch_dependents();
    pdl_wait();
    const int MT = gridDim.x, tid = threadIdx.x, lane = tid & 31;
    int row = blockIdx.x, turn = 0;
    const int K = a.n.K, n8 = K / 8;
    const Codes<!ROWS> codes(a.n, K, a.n.G, MT, s_gs);
    if (!ROWS && row >= a.n.M) {  // padding row of the operand
        codes.template pad<T>(row);
        return;
    }
    Raw x[V], g[V];
    auto fetch = [&](int row) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            x[j] = g[j] = Raw{};
            if (idx < n8) {
                x[j] = load_raw(row_of(a.n.x, x_type, a.n.ldx, row), x_type, idx);
                if (a.gate) g[j] = load_raw(row_of(a.gate, g_type, a.ldg, row), g_type, idx);
            }
        }
    };
    fetch(row);
    // the weights with the features' signs: what leaves the gate is what is rotated,
    // and h takes the sign back
    float w[V][8];
    uint32_t sg[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int idx = tid + j * T;
        sg[j] = idx < n8 ? (__ldg(a.n.signs + (idx >> 2)) >> ((idx & 3) * 8)) & 0xffu : 0u;
        load_weight<U>(a, idx, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[j][i] = flip(w[j][i], (sg[j] >> i) & 1u);
    }
    for (; row < a.n.M; row += MT, turn ^= 1) {
        if (codes.sums) {
            if (ROWS) __syncthreads();  // the last row's sums have been read
            codes.template clear_sums<T>();
        }
        float y[V][8], z[V][8], amax = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            form<U, true>(a, x[j], x_type, g[j], g_type, w[j], y[j]);
        }
        if (ROWS && row + MT < a.n.M) fetch(row + MT);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int idx = tid + j * T;
            if (idx < n8 && a.n.h) store8(const_cast<void *>(row_of(a.n.h, h_type, a.n.ldh, row)), h_type, idx, y[j], sg[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] = y[j][i];
            rotate8(z[j], lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(z[j][i]));
        }
        amax = block_max<T>(amax, s_max[turn]);
        float up = 1.0f, more = 1.0f;
        if (!(amax >= MAX_LEAST && amax < INFINITY) && amax != 0.0f) {
            // sums of the rotation, or quotients by the largest, leave fp32's range: in
            // units of 2^e, the power of two above the row's largest |y|
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(y[j][i]));
            top = block_max<T>(top, s_far[0]);
            if (top > 0.0f && top < INFINITY) {
                const bool small = top < 0x1p-60f;
                const int e = (__float_as_int(small ? top * 0x1p80f : top) >> 23) - (small ? 206 : 126), half = e / 2;
                const float down = __int_as_float((127 - half) << 23), rest = __int_as_float((127 - e + half) << 23);
                up = __int_as_float((127 + half) << 23);
                more = __int_as_float((127 + e - half) << 23);
                amax = 0.0f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[j][i] = y[j][i] * down * rest;
                    rotate8(z[j], lane);
#pragma unroll
                    for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(z[j][i]));
                }
                amax = block_max<T>(amax, s_far[1]);
            }
        }
        if (tid == 0) a.n.sx[row] = amax * __int_as_float((int)HADAMARD_SCALE_BITS) / 127.0f * up * more;
        // no codes of zeros, and of rows with an infinity or NaN: 0 * infinity and NaN round to 0
        const float inv = amax > 0.0f ? 127.0f / amax : 0.0f;
        int8_t *qr = a.n.qx ? a.n.qx + (size_t)row * K : nullptr;
#pragma unroll
        for (int j = 0; j < V; ++j) codes.write(row, qr, tid + j * T, z[j], inv);
        codes.template write_sums<T>(row);
        if (!ROWS) break;
    }
}

template <int U, int V, int T>
cudaError_t launch_rows(const GateArgs &a, bool pdl, cudaStream_t s) {
    if (a.n.qop) return launch_kernel(k_gate_row<U, V, T, false>, dim3((unsigned)act_rows(a.n.M)), dim3(T), 0, pdl, s, a);
    if constexpr (V * T > 2048) {
        return launch_kernel(k_gate_row<U, V, T, false>, dim3((unsigned)a.n.M), dim3(T), 0, pdl, s, a);
    } else {
        const int sms = device_sm_count(), most = sms * (1024 / T);
        if (sms <= 0) return cudaErrorNoDevice;
        auto f = k_gate_row<U, V, T, true>;
        // Types known at compile time where a thread holds one octet (with two, registers
        // spill).  Without and with them, bf16: 8190 rows of 8192 130 and 111 us, 20000
        // of 2048 89 and 71, 30000 of 1024 69 and 56, one of 1024 2.65 and 2.55.
        if constexpr (V == 1) {
            const bool one = a.gate && a.g_type != HQ_F32 && (!a.n.h || a.g_type == a.n.h_type), wide = a.n.x_type == HQ_F32;
            if (one && a.g_type == HQ_F16 && (wide || a.n.x_type == HQ_F16))
                f = wide ? k_gate_row<U, V, T, true, HQ_F32, HQ_F16> : k_gate_row<U, V, T, true, HQ_F16, HQ_F16>;
            else if (one && a.g_type == HQ_BF16 && (wide || a.n.x_type == HQ_BF16))
                f = wide ? k_gate_row<U, V, T, true, HQ_F32, HQ_BF16> : k_gate_row<U, V, T, true, HQ_BF16, HQ_BF16>;
        }
        return launch_kernel(f, dim3((unsigned)(a.n.M < most ? a.n.M : most)), dim3(T), 0, pdl, s, a);
    }
}

template <int U>
cudaError_t launch_u(const GateArgs &a, bool pdl, cudaStream_t s) {
    const int n8 = a.n.K / 8;
    if (!a.n.sx) {
        const int sms = device_sm_count();
        if (sms <= 0) return cudaErrorNoDevice;
        const long long blocks = ((long long)a.n.M * n8 + FT * FLIGHT - 1) / (FT * FLIGHT), most = 8ll * sms;
        const bool one = a.gate && a.g_type == a.n.h_type && a.g_type != HQ_F32, wide = a.n.x_type == HQ_F32;
        auto f = k_gate_heads<U, -1, -1>;
        if (one && a.g_type == HQ_F16 && (wide || a.n.x_type == HQ_F16))
            f = wide ? k_gate_heads<U, HQ_F32, HQ_F16> : k_gate_heads<U, HQ_F16, HQ_F16>;
        else if (one && a.g_type == HQ_BF16 && (wide || a.n.x_type == HQ_BF16))
            f = wide ? k_gate_heads<U, HQ_F32, HQ_BF16> : k_gate_heads<U, HQ_BF16, HQ_BF16>;
        return launch_kernel(f, dim3((unsigned)(blocks < most ? blocks : most)), dim3(FT), 0, pdl, s, a);
    }
    // As many threads as a row has octets, up to 1024.  Every V * T is a multiple of
    // 16 octets, so the operand's padding up to whole 128-feature blocks is covered
    // too.
    if (n8 <= 128) return launch_rows<U, 1, 128>(a, pdl, s);
    if (n8 <= 256) return launch_rows<U, 1, 256>(a, pdl, s);
    if (n8 <= 512) return launch_rows<U, 1, 512>(a, pdl, s);
    if (n8 <= 1024) return launch_rows<U, 1, 1024>(a, pdl, s);
    if (n8 <= 2048) return launch_rows<U, 2, 1024>(a, pdl, s);
    if (n8 <= 4096) return launch_rows<U, 4, 1024>(a, pdl, s);
    return launch_rows<U, 8, 1024>(a, pdl, s);
}

}  // namespace

cudaError_t launch_gated_norm(const GateArgs &a, bool pdl, cudaStream_t s) {
    switch (a.D) {
        case 64: return launch_u<8>(a, pdl, s);
        case 128: return launch_u<16>(a, pdl, s);
        default: return launch_u<32>(a, pdl, s);
    }
}

}  // namespace hq
