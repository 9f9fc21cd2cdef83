// k_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   t[m] = A[a] x[m]  (a = ids[m], rank r),   Y[m] = base[m] + scale[a] * B[a] t[m]
//
// Two kernels.  The rows of one adapter form items of up to 16 rows (the MMA's
// M); every thread block finds the items itself from ids (128 compares a
// thread) and takes every gridDim.y-th, so no list is built on the host, ids
// may come in any order, and an item reads its adapter once.
//
// k_lora_shrink: a cluster of 8 thread blocks per item splits K; every warp
// forms 16 x 64 partial sums with m16n8k16 MMAs straight from global memory.
// The sum over k does not care in which order the k are taken as long as both
// operands agree, so a lane's 16-byte loads of 8 consecutive k serve two MMA
// steps as they are.  Warps add up in shared memory, the blocks through the
// cluster's distributed shared memory, in a fixed order.
// k_lora_expand: each warp forms 16 rows x 32 outputs with the same MMAs over
// the rank and adds base.
// Items of one or two rows (a token per request) use multiply-adds on the same
// loads instead: an MMA takes 16 rows' time whatever it is given, and the
// loads, not the products, should be what bounds them.
//
// Exactness: products of two 16-bit values are exact in fp32.  Where the
// operand's type is not the adapter's (fp32 activations, and t, which is kept
// in fp32), the value enters as three bf16 terms whose sum is the value
// (8 significant bits each), an fp16 weight as two.
#include <cooperative_groups.h>

#include "batch.cuh"

namespace cg = cooperative_groups;

namespace hq {
namespace {

constexpr int LR = 16;        // rows per item
constexpr int LG = 64;        // ranks per block of the shrink
constexpr int LCL = 8;        // thread blocks per cluster (parts of K)
constexpr int LWARPS = 8;
constexpr int LNT = 4;        // 8-column tiles per warp of the expand
constexpr int LCOLS = LWARPS * LNT * 8;

template <bool BF>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// x = t[0] + t[1] + t[2], each a bf16 (packed in pairs).  An infinity stays
// in the first term alone.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t (&t)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        t[i] = pack_bf16(x0, x1);
        const float h0 = __uint_as_float(t[i] << 16), h1 = __uint_as_float(t[i] & 0xffff0000u);
        x0 = isinf(h0) ? 0.0f : x0 - h0;
        x1 = isinf(h1) ? 0.0f : x1 - h1;
    }
}

// A pair of fp16 weights as two pairs of bf16 whose sum they are (11
// significant bits = 8 + 3).
__device__ __forceinline__ void split_half(uint32_t w, uint32_t (&t)[2]) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    t[0] = pack_bf16(f.x, f.y);
    const float h0 = __uint_as_float(t[0] << 16), h1 = __uint_as_float(t[0] & 0xffff0000u);
    t[1] = pack_bf16(isinf(h0) ? 0.0f : f.x - h0, isinf(h1) ? 0.0f : f.y - h1);
}

// The items of the batch.  All threads of the block call find(), then rows().
struct Items {
    int id[HQ_MAX_M];      // the row's adapter, -1 for none
    int number[HQ_MAX_M];  // its number among the rows of its adapter
    int lead[HQ_MAX_M];    // the first row of each item
    int row[LR];           // the rows of the current item
    int warp_count[HQ_MAX_M / 32];
    int n;
};

__device__ void find_items(Items &it, const int32_t *ids, int M, int n_adapters) {
    const int t = threadIdx.x;
    int id = -2;  // no row
    if (t < HQ_MAX_M) {
        if (t < M) {
            id = ids[t];
            if (id < 0 || id >= n_adapters) id = -1;
        }
        it.id[t] = id;
    }
    __syncthreads();
    bool lead = false;
    if (t < HQ_MAX_M) {
        int n = 0;
        const int4 *v = reinterpret_cast<const int4 *>(it.id);
#pragma unroll 8
        for (int j = 0; j < HQ_MAX_M / 4; ++j) {
            const int4 x = v[j];
            n += (x.x == id && 4 * j < t) + (x.y == id && 4 * j + 1 < t) + (x.z == id && 4 * j + 2 < t) +
                 (x.w == id && 4 * j + 3 < t);
        }
        it.number[t] = n;
        lead = t < M && n % LR == 0;
    }
    const uint32_t b = __ballot_sync(0xffffffffu, lead);
    if (t < HQ_MAX_M && (t & 31) == 0) it.warp_count[t >> 5] = __popc(b);
    __syncthreads();
    if (t < HQ_MAX_M) {
        int at = __popc(b & ((1u << (t & 31)) - 1u));
        for (int w = 0; w < (t >> 5); ++w) at += it.warp_count[w];
        if (lead) it.lead[at] = t;
    }
    if (t == 0) {
        int n = 0;
        for (int w = 0; w < HQ_MAX_M / 32; ++w) n += it.warp_count[w];
        it.n = n;
    }
    __syncthreads();
}

// The rows of item i into it.row; their number.  (The block has finished with
// the item before: the barrier comes first.)
__device__ int item_rows(Items &it, int i, int M) {
    const int t = threadIdx.x, lead = it.lead[i], id = it.id[lead], part = it.number[lead] / LR;
    const bool mine = t < M && t < HQ_MAX_M && it.id[t] == id && it.number[t] / LR == part;
    const int n = __syncthreads_count(mine);
    if (mine) it.row[it.number[t] % LR] = t;
    __syncthreads();
    return n;
}

__device__ __forceinline__ int rank_of(const LoraArgs &a, int id) {
    const int r = a.ranks ? a.ranks[id] : a.r_max;
    return r < 0 ? 0 : r > a.r_max ? a.r_max : r;
}

// 8 consecutive values of x as MMA words: one 16-byte load where the types
// agree, else three bf16 terms of each value.
template <bool SAME>
__device__ __forceinline__ void load_x(const LoraArgs &a, const uint8_t *row, int k, bool live,
                                       uint32_t (&w)[SAME ? 1 : 3][4]) {
    if constexpr (SAME) {
        const uint4 u = live ? *reinterpret_cast<const uint4 *>(row + (size_t)k * 2) : make_uint4(0, 0, 0, 0);
        w[0][0] = u.x, w[0][1] = u.y, w[0][2] = u.z, w[0][3] = u.w;
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
        if (live) {
            if (a.x_type == HQ_F32) {
                const float4 *p = reinterpret_cast<const float4 *>(row + (size_t)k * 4);
                const float4 u = p[0], v = p[1];
                f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
            } else {
                const uint4 u = *reinterpret_cast<const uint4 *>(row + (size_t)k * 2);
                const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = a.x_type == HQ_F16
                                         ? __half22float2(*reinterpret_cast<const __half2 *>(&p[i]))
                                         : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&p[i]));
                    f[2 * i] = v.x;
                    f[2 * i + 1] = v.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[3];
            split3(f[2 * i], f[2 * i + 1], t);
            w[0][i] = t[0];
            w[1][i] = t[1];
            w[2][i] = t[2];
        }
    }
}

// 8 consecutive values as floats: x of type `type`, weights.
__device__ __forceinline__ void wide8(const uint8_t *p, int type, float (&f)[8]) {
    if (type == HQ_F32) {
        const float4 u = reinterpret_cast<const float4 *>(p)[0], v = reinterpret_cast<const float4 *>(p)[1];
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
        return;
    }
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = type == HQ_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[i]))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}
template <bool BF>
__device__ __forceinline__ void wide_w(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = BF ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]))
                            : __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

template <bool WBF, bool SAME>
__global__ void __cluster_dims__(LCL, 1, 1) __launch_bounds__(LWARPS * 32) k_lora_shrink(const LoraArgs a) {
    __shared__ __align__(16) Items it;
    __shared__ float s_part[LWARPS][LR][LG + 4];
    cg::cluster_group cluster = cg::this_cluster();
    const int part = blockIdx.x, r0 = blockIdx.z * LG;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    find_items(it, a.ids, a.M, a.n_adapters);
    pdl_launch_dependents();
    const int xb = type_bytes(a.x_type);
    const int units = (a.K + 31) / 32;
    const int u0 = (int)((long long)units * part / LCL), u1 = (int)((long long)units * (part + 1) / LCL);
    bool waited = false;
    for (int i = blockIdx.y; i < it.n; i += gridDim.y) {  // the same for the whole cluster
        const int id = it.id[it.lead[i]];
        const int rank = id < 0 ? 0 : rank_of(a, id) - r0;
        if (rank <= 0) continue;
        const int nr = item_rows(it, i, a.M);
        const int nt = rank >= LG ? LG / 8 : (rank + 7) / 8;
        const uint8_t *Aw = static_cast<const uint8_t *>(a.A) + ((size_t)id * a.r_max + r0 + g) * (size_t)a.K * 2;
        const uint8_t *xA = static_cast<const uint8_t *>(a.x) + (size_t)it.row[g < nr ? g : 0] * (size_t)a.ldx * xb;
        const uint8_t *xB = static_cast<const uint8_t *>(a.x) + (size_t)it.row[g + 8 < nr ? g + 8 : 0] * (size_t)a.ldx * xb;
        float acc[LG / 8][4];
#pragma unroll
        for (int j = 0; j < LG / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
        if (nr <= 2) {
            // lane (g, t4): ranks 8 j + g, k = 8 t4 .. 8 t4 + 7 of each unit
            const uint8_t *x0 = static_cast<const uint8_t *>(a.x) + (size_t)it.row[0] * (size_t)a.ldx * xb;
            const uint8_t *x1 = static_cast<const uint8_t *>(a.x) + (size_t)it.row[nr - 1] * (size_t)a.ldx * xb;
            for (int u = u0 + warp; u < u1; u += LWARPS) {
                const int k = u * 32 + t4 * 8;
                const bool live = k < a.K;
                uint4 b[LG / 8];
#pragma unroll
                for (int j = 0; j < LG / 8; ++j)
                    b[j] = j < nt && live && j * 8 + g < rank
                               ? *reinterpret_cast<const uint4 *>(Aw + ((size_t)j * 8 * a.K + k) * 2)
                               : make_uint4(0, 0, 0, 0);
                if (!waited) {
                    pdl_wait();
                    waited = true;
                }
                float x[2][8] = {};
                if (live) {
                    wide8(x0 + (size_t)k * xb, a.x_type, x[0]);
                    if (nr == 2) wide8(x1 + (size_t)k * xb, a.x_type, x[1]);
                }
#pragma unroll
                for (int j = 0; j < LG / 8; ++j) {
                    if (j >= nt) break;
                    float w[8];
                    wide_w<WBF>(b[j], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[j][e & 1] = fmaf(w[e], x[0][e], acc[j][e & 1]);
                    if (nr == 2)
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[j][2 + (e & 1)] = fmaf(w[e], x[1][e], acc[j][2 + (e & 1)]);
                }
            }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
#pragma unroll
            for (int j = 0; j < LG / 8; ++j) {
                if (j >= nt) break;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float v = acc[j][2 * m] + acc[j][2 * m + 1];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (t4 == 0) s_part[warp][m][j * 8 + g] = v;
                }
            }
        } else {
            constexpr int NX = SAME ? 1 : 3;
            for (int u = u0 + warp; u < u1; u += LWARPS) {
                const int k = u * 32 + t4 * 8;
                const bool live = k < a.K;
                uint4 b[LG / 8];
#pragma unroll
                for (int j = 0; j < LG / 8; ++j)
                    b[j] = j < nt && live && j * 8 + g < rank
                               ? *reinterpret_cast<const uint4 *>(Aw + ((size_t)j * 8 * a.K + k) * 2)
                               : make_uint4(0, 0, 0, 0);
                if (!waited) {
                    pdl_wait();
                    waited = true;
                }
                uint32_t p[NX][4], q[NX][4];
                load_x<SAME>(a, xA, k, live && g < nr, p);
                load_x<SAME>(a, xB, k, live && g + 8 < nr, q);
#pragma unroll
                for (int j = 0; j < LG / 8; ++j) {
                    if (j >= nt) break;
                    const uint32_t w[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
                    for (int st = 0; st < 2; ++st)
#pragma unroll
                        for (int x = 0; x < NX; ++x) {
                            const uint32_t x4[4] = {p[x][2 * st], q[x][2 * st], p[x][2 * st + 1], q[x][2 * st + 1]};
                            if constexpr (SAME || WBF) {
                                mma16<WBF>(acc[j], x4, w[2 * st], w[2 * st + 1]);
                            } else {
                                uint32_t h0[2], h1[2];
                                split_half(w[2 * st], h0);
                                split_half(w[2 * st + 1], h1);
                                mma16<true>(acc[j], x4, h0[0], h1[0]);
                                mma16<true>(acc[j], x4, h0[1], h1[1]);
                            }
                        }
                }
            }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
#pragma unroll
            for (int j = 0; j < LG / 8; ++j) {
                if (j >= nt) break;
                float *d = &s_part[warp][g][j * 8 + 2 * t4];
                d[0] = acc[j][0];
                d[1] = acc[j][1];
                float *e = &s_part[warp][g + 8][j * 8 + 2 * t4];
                e[0] = acc[j][2];
                e[1] = acc[j][3];
            }
        }
        __syncthreads();
        const int cols = nt * 8, elems = nr * cols;
        for (int i2 = tid; i2 < elems; i2 += LWARPS * 32) {
            const int m = i2 / cols, c = i2 % cols;
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < LWARPS; ++w) v += s_part[w][m][c];
            s_part[0][m][c] = v;
        }
        cluster.sync();
        // each block of the cluster adds up its share of the item's elements
        for (int i2 = part + tid * LCL; i2 < elems; i2 += LCL * LWARPS * 32) {
            const int m = i2 / cols, c = i2 % cols;
            float v = 0.0f;
#pragma unroll
            for (int b = 0; b < LCL; ++b) v += *cluster.map_shared_rank(&s_part[0][m][c], b);
            a.t[(size_t)it.row[m] * a.r_max + r0 + c] = v;
        }
        cluster.sync();  // the others may still be reading this block's sums
    }
    if (!waited) pdl_wait();
}

template <bool WBF>
__global__ void __launch_bounds__(LWARPS * 32) k_lora_expand(const LoraArgs a) {
    __shared__ __align__(16) Items it;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    find_items(it, a.ids, a.M, a.n_adapters);
    pdl_launch_dependents();
    const long long n0 = (long long)blockIdx.x * LCOLS + warp * LNT * 8;
    // pairs of outputs where every row starts at an 8-byte boundary
    const bool pairs = (a.N & 1) == 0 && (a.ldy & 1) == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 7) == 0 &&
                       (!a.base || ((a.ldb & 1) == 0 && (reinterpret_cast<uintptr_t>(a.base) & 7) == 0));
    bool waited = false;
    for (int i = blockIdx.y; i < it.n; i += gridDim.y) {
        const int id = it.id[it.lead[i]];
        if (id < 0 && a.base == a.Y) continue;  // no adapter, in place: nothing to change
        const int nr = item_rows(it, i, a.M);
        const int rank = id < 0 ? 0 : rank_of(a, id);
        const uint8_t *Bw = static_cast<const uint8_t *>(a.B) + (size_t)(id < 0 ? 0 : id) * a.N * (size_t)a.r_max * 2;
        const float sc = id >= 0 && a.scale ? a.scale[id] : 1.0f;
        float acc[LNT][4];
#pragma unroll
        for (int j = 0; j < LNT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
        for (int k0 = 0; k0 < rank; k0 += 32) {
            const int k = k0 + t4 * 8, left = rank - k;  // ranks left from this lane's first on
            uint4 b[LNT];
#pragma unroll
            for (int j = 0; j < LNT; ++j) {
                const long long n = n0 + j * 8 + g;
                b[j] = left > 0 && n < a.N ? *reinterpret_cast<const uint4 *>(Bw + ((size_t)n * a.r_max + k) * 2)
                                           : make_uint4(0, 0, 0, 0);
                if (left > 0 && left < 8) {  // what lies past the rank is not used
                    uint32_t w[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = 2 * x + 1 < left ? w[x] : 2 * x < left ? w[x] & 0xffffu : 0u;
                    b[j] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (!waited) {
                pdl_wait();
                waited = true;
            }
            if (nr <= 2) {
                // lane (g, t4): outputs 8 j + g, ranks 8 t4 .. 8 t4 + 7 of the 32
                float t[2][8];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const float *tr = a.t + (size_t)it.row[m < nr ? m : 0] * a.r_max + k;
#pragma unroll
                    for (int e = 0; e < 8; ++e) t[m][e] = m < nr && e < left ? tr[e] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < LNT; ++j) {
                    float w[8];
                    wide_w<WBF>(b[j], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[j][0] = fmaf(w[e], t[0][e], acc[j][0]);
                        acc[j][1] = fmaf(w[e], t[1][e], acc[j][1]);
                    }
                }
                continue;
            }
            uint32_t p[3][4], q[3][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m = g + 8 * h;
                const float *tr = a.t + (size_t)it.row[m < nr ? m : 0] * a.r_max + k;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float f0 = m < nr && 2 * x < left ? tr[2 * x] : 0.0f;
                    const float f1 = m < nr && 2 * x + 1 < left ? tr[2 * x + 1] : 0.0f;
                    uint32_t s[3];
                    split3(f0, f1, s);
#pragma unroll
                    for (int y = 0; y < 3; ++y) (h ? q : p)[y][x] = s[y];
                }
            }
#pragma unroll
            for (int j = 0; j < LNT; ++j) {
                const uint32_t w[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    uint32_t h0[2] = {w[2 * st], 0}, h1[2] = {w[2 * st + 1], 0};
                    if constexpr (!WBF) {
                        split_half(w[2 * st], h0);
                        split_half(w[2 * st + 1], h1);
                    }
#pragma unroll
                    for (int x = 0; x < 3; ++x) {
                        const uint32_t x4[4] = {p[x][2 * st], q[x][2 * st], p[x][2 * st + 1], q[x][2 * st + 1]};
                        mma16<true>(acc[j], x4, h0[0], h1[0]);
                        if constexpr (!WBF) mma16<true>(acc[j], x4, h0[1], h1[1]);
                    }
                }
            }
        }
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        if (nr <= 2) {
            // the four lanes of an output add up; lane t4 writes output 8 t4 + g
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float mine = 0.0f;
#pragma unroll
                for (int j = 0; j < LNT; ++j) {
                    float v = acc[j][m];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    if (t4 == j) mine = v;
                }
                static_assert(LNT == 4, "one output a lane");
                const long long n = n0 + t4 * 8 + g;
                if (m >= nr || n >= a.N) continue;
                const size_t r = (size_t)it.row[m];
                const float base = a.base ? a.base[r * a.ldb + n] : 0.0f;
                a.Y[r * a.ldy + n] = rank > 0 ? base + sc * mine : base;
            }
            continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = g + 8 * h;
            if (m >= nr) continue;
            const size_t r = (size_t)it.row[m];
            float2 base[LNT];
#pragma unroll
            for (int j = 0; j < LNT; ++j) {
                const long long n = n0 + j * 8 + 2 * t4;
                base[j] = make_float2(0.0f, 0.0f);
                if (!a.base || n >= a.N) continue;
                const float *s = a.base + r * a.ldb + n;
                if (pairs) {
                    base[j] = *reinterpret_cast<const float2 *>(s);
                } else {
                    base[j].x = s[0];
                    if (n + 1 < a.N) base[j].y = s[1];
                }
            }
#pragma unroll
            for (int j = 0; j < LNT; ++j) {
                const long long n = n0 + j * 8 + 2 * t4;
                if (n >= a.N) continue;
                if (rank > 0) {
                    base[j].x += sc * acc[j][2 * h];
                    base[j].y += sc * acc[j][2 * h + 1];
                }
                float *d = a.Y + r * a.ldy + n;
                if (pairs) {
                    *reinterpret_cast<float2 *>(d) = base[j];
                } else {
                    d[0] = base[j].x;
                    if (n + 1 < a.N) d[1] = base[j].y;
                }
            }
        }
    }
    if (!waited) pdl_wait();
}

}  // namespace

cudaError_t launch_lora(const LoraArgs &a, int w_type, bool pdl, cudaStream_t s) {
    const bool bf = w_type == HQ_BF16, same = a.x_type == w_type;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    // items in turn: enough clusters for four blocks an SM, enough blocks for
    // eight (a block without an item costs a microsecond all the same)
    const int rg = (a.r_max + LG - 1) / LG, tiles = (int)(((long long)a.N + LCOLS - 1) / LCOLS);
    auto least = [&](long long want) { return (unsigned)(want < 1 ? 1 : want < a.M ? want : a.M); };
    const dim3 grid(LCL, least((4LL * sms / LCL + rg - 1) / rg), (unsigned)rg), block(LWARPS * 32);
    cudaError_t e;
    if (bf)
        e = same ? launch_kernel(k_lora_shrink<true, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<true, false>, grid, block, 0, pdl, s, a);
    else
        e = same ? launch_kernel(k_lora_shrink<false, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<false, false>, grid, block, 0, pdl, s, a);
    if (e != cudaSuccess) return e;
    const dim3 eg((unsigned)tiles, least((8LL * sms + tiles - 1) / tiles));
    // the expand always follows the shrink programmatically: it loads its
    // weights while the shrink runs
    return bf ? launch_kernel(k_lora_expand<true>, eg, block, 0, true, s, a)
              : launch_kernel(k_lora_expand<false>, eg, block, 0, true, s, a);
}

}  // namespace hq
