// k_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   t[m] = A[a] x[m]  (a = ids[m], rank r),   Y[m] = base[m] + scale[a] * B[a] t[m]
//
// Two kernels.  The rows of one adapter form items of up to 16 rows (the MMA's
// M); every thread block finds the items itself from ids (128 compares a
// thread) and takes every gridDim.y-th, so no list is built on the host, ids
// may come in any order, and an item reads its adapter once.
//
// k_lora_shrink, items of three rows and more: a cluster of 8 thread blocks
// splits K; every warp forms 16 x 64 partial sums with m16n8k16 MMAs straight
// from global memory.  The sum over k does not care in which order the k are
// taken as long as both operands agree, so a lane's 16-byte loads of 8
// consecutive k serve two MMA steps as they are.  Warps add up in shared
// memory, the blocks through the cluster's distributed shared memory, in a
// fixed order.  Items of one or two rows (a token per request): the cluster's
// blocks split the ranks instead, a warp takes one row of A over all of K with
// multiply-adds, eight 512-byte loads in flight, and nothing is left to add up
// but its lanes.  (With K split, the items of a row each waited for two cluster
// barriers: 97 rows of rank 16 to 64, K = 12288, took 45 us instead of 33 then;
// now 27.)
// k_lora_expand: each warp forms 16 rows x 32 outputs with the same MMAs over
// the rank, or with multiply-adds where the item has one or two rows, and adds
// base.  97 rows of 4096 outputs take 15 us, 128 rows of 24576 17.5.  (A thread per
// output column with t in shared memory, fp32 products and the next item's loads
// in flight took 28 and 34 us where this form took 21 and 21: its reads of t bound
// it.)
//
// Exactness: products of two 16-bit values are exact in fp32.  Where the
// MMAs' operand is not of the adapter's type (fp32 activations, and t, which
// is kept in fp32), the value enters as three bf16 terms whose sum is the value
// (8 significant bits each), an fp16 weight as two.  That holds for finite values
// up to bf16's largest; beyond it the first term is an infinity, which meets
// terms that are 0.  Such a sum comes out not finite, whatever the other operand,
// and is formed again from the values themselves (dot_again), so that a row's
// result does not depend on how many rows share its adapter.
#include <cooperative_groups.h>

#include "batch.cuh"

namespace cg = cooperative_groups;

namespace hq {
namespace {

constexpr int LR = 16;        // rows per item
constexpr int LG = 64;        // ranks per block of the shrink
constexpr int LCL = 8;        // thread blocks per cluster (parts of K)
constexpr int LWARPS = 8;
constexpr int LTAB = 2 * HQ_MAX_M;  // places of a hash table of a batch's adapters, at most half full
static_assert(LTAB == LWARPS * 32 && HQ_MAX_M == 128, "a thread a place, a row a bit");
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

// x = t[0] + t[1] + t[2], each a bf16 (packed in pairs); finite x up to bf16's
// largest value.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t (&t)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        t[i] = pack_bf16(x0, x1);
        const float h0 = __uint_as_float(t[i] << 16), h1 = __uint_as_float(t[i] & 0xffff0000u);
        x0 -= h0;
        x1 -= h1;
    }
}

// A pair of fp16 weights as two pairs of bf16 whose sum they are (11
// significant bits = 8 + 3).
__device__ __forceinline__ void split_half(uint32_t w, uint32_t (&t)[2]) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    t[0] = pack_bf16(f.x, f.y);
    const float h0 = __uint_as_float(t[0] << 16), h1 = __uint_as_float(t[0] & 0xffff0000u);
    t[1] = pack_bf16(f.x - h0, f.y - h1);
}

// The items of the batch, found by all threads of the block.
struct Items {
    int id[HQ_MAX_M];      // the row's adapter, -1 for none
    int rank[HQ_MAX_M];    // of the row's adapter
    int lead[HQ_MAX_M];    // the first row of each item
    int rows[HQ_MAX_M];    // rows of each item
    int mate[HQ_MAX_M];    // the second row of the item that a row leads
    int unit0[HQ_MAX_M + 1];  // k_lora_shrink: the few-row items' shares before each item
    uint8_t row[HQ_MAX_M][LR];  // the rows of each item
    int warp_count[HQ_MAX_M / 32];
    int n;
    // the batch's adapters, hashed: id, rows (a bit each), items
    int key[LTAB];
    uint4 mask[LTAB];
    uint8_t item[LTAB][HQ_MAX_M / LR];
};

// Sum over the first HQ_MAX_M threads before this one; `total` over all.
__device__ int sum_below(Items &it, int v, int &total) {
    const int t = threadIdx.x, lane = t & 31;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (t < HQ_MAX_M && lane == 31) it.warp_count[t >> 5] = x;
    __syncthreads();
    int below = x - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < HQ_MAX_M / 32; ++w) {
        if (w < (t >> 5)) below += it.warp_count[w];
        total += it.warp_count[w];
    }
    return below;
}

// A hash table finds the rows of each adapter (comparing every row with every
// other took 1 us longer, in each of the two kernels).
__device__ void find_items(Items &it, const LoraArgs &a) {
    const int M = a.M, t = threadIdx.x, w = t >> 5;
    const uint32_t below = (1u << (t & 31)) - 1;
    it.key[t] = -2;
    it.mask[t] = make_uint4(0, 0, 0, 0);
    int id = -2, rank = 0, place = 0;
    if (t < M) {
        id = a.ids[t];
        if (id < 0 || id >= a.n_adapters) id = -1;
    }
    __syncthreads();
    if (t < M) {
        rank = id < 0 ? 0 : a.ranks ? a.ranks[id] : a.r_max;  // on its way meanwhile
        place = (int)(((uint32_t)id * 2654435761u) >> 16) & (LTAB - 1);
        for (int probe = 0; probe < LTAB; ++probe) {
            const int old = atomicCAS(&it.key[place], -2, id);
            if (old == -2 || old == id) break;
            place = (place + 1) & (LTAB - 1);
        }
        atomicOr(reinterpret_cast<uint32_t *>(&it.mask[place]) + w, 1u << (t & 31));
    }
    __syncthreads();
    bool lead = false;
    int n = 0, size = 0;
    if (t < HQ_MAX_M) {
        if (t < M) {
            const uint4 m4 = it.mask[place];
            const uint32_t m[4] = {m4.x, m4.y, m4.z, m4.w};
            int last = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                size += __popc(m[i]);
                const uint32_t before = i < w ? m[i] : i == w ? m[i] & below : 0u;
                n += __popc(before);
                if (before) last = 32 * i + 31 - __clz(before);
            }
            lead = n % LR == 0;
            if (n % LR == 1) it.mate[last] = t;
            it.id[t] = id;
            it.rank[t] = rank < 0 ? 0 : rank > a.r_max ? a.r_max : rank;
        }
        const uint32_t leads = __ballot_sync(0xffffffffu, lead);
        if ((t & 31) == 0) it.warp_count[w] = (int)leads;
    }
    __syncthreads();
    int total = 0, at = 0;
#pragma unroll
    for (int i = 0; i < HQ_MAX_M / 32; ++i) {
        const uint32_t leads = (uint32_t)it.warp_count[i];
        at += i < w ? __popc(leads) : i == w ? __popc(leads & below) : 0;
        total += __popc(leads);
    }
    if (lead) {
        it.lead[at] = t;
        it.rows[at] = size - n < LR ? size - n : LR;
        it.item[place][n / LR] = (uint8_t)at;
    }
    if (t == 0) it.n = total;
    __syncthreads();
    if (t < M) it.row[it.item[place][n / LR]][n % LR] = (uint8_t)t;
    __syncthreads();
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

// The sum of n products of values of x (type x_type) and of weights as they are,
// by one thread, 8 at a time (both are allocated in eights): for sums of split
// terms that came out not finite.
template <bool WBF>
__device__ __noinline__ float dot_again(const uint8_t *x, int x_type, const uint8_t *w, int n) {
    float sum = 0.0f;
#pragma unroll 4
    for (int k = 0; k < n; k += 8) {
        float f[8], v[8];
        wide8(x + (size_t)k * type_bytes(x_type), x_type, f);
        wide_w<WBF>(*reinterpret_cast<const uint4 *>(w + (size_t)k * 2), v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < n) sum = fmaf(v[e], f[e], sum);
    }
    return sum;
}

// A row's n <= 8 neighbouring outputs, the sums formed as in dot_again.
template <bool WBF>
__device__ __noinline__ void outputs_again(const float *base, float *y, const float *t, const uint8_t *b, int r_max,
                                           int rank, float scale, int n) {
    for (int e = 0; e < n; ++e) {
        const float add = rank > 0 ? scale * dot_again<WBF>(reinterpret_cast<const uint8_t *>(t), HQ_F32, b, rank) : 0.0f;
        y[e] = (base ? base[e] : 0.0f) + add;
        b += (size_t)r_max * 2;
    }
}

// Of 8 values of 16 bits the first `left`, zeros behind them.
__device__ __forceinline__ uint4 below_rank(const uint4 &u, int left) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = 2 * x + 1 < left ? w[x] : 2 * x < left ? w[x] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Items of one or two rows: t[row] for the 8 ranks of this block's share, one a
// warp, over all of K, in chunks of 2048 k: x in shared memory as fp32 (the
// first and last four of each eight apart, which keeps its 16-byte reads free
// of bank conflicts), the next chunk's loads in flight during the products.
template <bool WBF>
__device__ __forceinline__ void shrink_few(const LoraArgs &a, int row0, int row1, int nr, int id, int rank, int r0,
                                           int part, float *s_x, bool &waited) {
    constexpr int NB = 8, CH = NB * 256;
    static_assert(CH == LWARPS * 32 * 8, "a thread brings 8 values of x a chunk");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j = part * (LG / LCL) + warp;  // this warp's rank of the group
    const bool live = j < rank;
    const int xb = type_bytes(a.x_type);
    const uint8_t *xr[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
        xr[m] = static_cast<const uint8_t *>(a.x) + (size_t)(m ? row1 : row0) * (size_t)a.ldx * xb;
    const uint8_t *Ar = static_cast<const uint8_t *>(a.A) + ((size_t)id * a.r_max + r0 + (live ? j : 0)) * (size_t)a.K * 2;
    uint4 b[NB];
    float x[2][8];
    auto load_b = [&](int k0) {
#pragma unroll
        for (int h = 0; h < NB; ++h) {
            const int k = k0 + h * 256 + lane * 8;
            b[h] = live && k < a.K ? *reinterpret_cast<const uint4 *>(Ar + (size_t)k * 2) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_x = [&](int k0) {
        const int k = k0 + tid * 8;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[m][e] = 0.0f;
            if (m < nr && k < a.K) wide8(xr[m] + (size_t)k * xb, a.x_type, x[m]);
        }
    };
    load_b(0);
    if (!waited) {
        pdl_wait();
        waited = true;
    }
    load_x(0);
    float sum[2][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += CH) {
        __syncthreads();  // the chunk before has been used
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float4 *>(s_x + (m * 2 + h) * (CH / 2) + tid * 4) =
                    make_float4(x[m][4 * h], x[m][4 * h + 1], x[m][4 * h + 2], x[m][4 * h + 3]);
        __syncthreads();
        uint4 c[NB];
#pragma unroll
        for (int h = 0; h < NB; ++h) c[h] = b[h];
        if (k0 + CH < a.K) {
            load_b(k0 + CH);
            load_x(k0 + CH);
        }
#pragma unroll
        for (int h = 0; h < NB; ++h) {
            float w[8];
            wide_w<WBF>(c[h], w);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (m == 1 && nr == 1) break;
                const float4 u = *reinterpret_cast<const float4 *>(s_x + m * CH + (h * 32 + lane) * 4);
                const float4 v = *reinterpret_cast<const float4 *>(s_x + m * CH + CH / 2 + (h * 32 + lane) * 4);
                sum[m][0] = fmaf(w[0], u.x, sum[m][0]);
                sum[m][1] = fmaf(w[1], u.y, sum[m][1]);
                sum[m][2] = fmaf(w[2], u.z, sum[m][2]);
                sum[m][3] = fmaf(w[3], u.w, sum[m][3]);
                sum[m][0] = fmaf(w[4], v.x, sum[m][0]);
                sum[m][1] = fmaf(w[5], v.y, sum[m][1]);
                sum[m][2] = fmaf(w[6], v.z, sum[m][2]);
                sum[m][3] = fmaf(w[7], v.w, sum[m][3]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        float v = (sum[m][0] + sum[m][1]) + (sum[m][2] + sum[m][3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0 && live && m < nr) a.t[(size_t)(m ? row1 : row0) * a.r_max + r0 + j] = v;
    }
}

template <bool WBF, bool SAME>
__global__ void __cluster_dims__(LCL, 1, 1) __launch_bounds__(LWARPS * 32, 2) k_lora_shrink(const LoraArgs a) {
    __shared__ __align__(16) Items it;
    __shared__ __align__(16) float s_part[LWARPS][LR][LG + 4];
    cg::cluster_group cluster = cg::this_cluster();
    const int part = blockIdx.x, r0 = blockIdx.z * LG;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    find_items(it, a);
    pdl_launch_dependents();
    const int xb = type_bytes(a.x_type);
    const int units = (a.K + 31) / 32;
    const int u0 = (int)((long long)units * part / LCL), u1 = (int)((long long)units * (part + 1) / LCL);
    bool waited = false;
    {
        // items of one or two rows: their shares of 8 ranks, over all blocks
        int share = 0, shares;
        if (tid < it.n && it.rows[tid] <= 2 && it.id[it.lead[tid]] >= 0) {
            const int rank = it.rank[it.lead[tid]] - r0;
            share = rank <= 0 ? 0 : rank >= LG ? LG / 8 : (rank + 7) / 8;
        }
        const int below = sum_below(it, share, shares);
        if (tid < HQ_MAX_M) it.unit0[tid] = below;
        if (tid == 0) it.unit0[HQ_MAX_M] = shares;
        __syncthreads();
        for (int u = part + LCL * (int)blockIdx.y; u < shares; u += LCL * gridDim.y) {
            int lo = 0, hi = HQ_MAX_M;  // the last item that starts at or before u
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (it.unit0[mid] <= u) lo = mid;
                else hi = mid;
            }
            const int lead = it.lead[lo], nr = it.rows[lo];
            shrink_few<WBF>(a, lead, nr == 2 ? it.mate[lead] : lead, nr, it.id[lead], it.rank[lead] - r0, r0,
                            u - it.unit0[lo], &s_part[0][0][0], waited);
        }
        __syncthreads();
    }
    for (int i = blockIdx.y; i < it.n; i += gridDim.y) {  // the same for the whole cluster
        const int id = it.id[it.lead[i]];
        const int rank = it.rank[it.lead[i]] - r0;
        if (rank <= 0 || it.rows[i] <= 2) continue;
        const int nr = it.rows[i];
        const uint8_t *rows = it.row[i];
        const int nt = rank >= LG ? LG / 8 : (rank + 7) / 8;
        const uint8_t *Aw = static_cast<const uint8_t *>(a.A) + ((size_t)id * a.r_max + r0 + g) * (size_t)a.K * 2;
        const uint8_t *xA = static_cast<const uint8_t *>(a.x) + (size_t)rows[g < nr ? g : 0] * (size_t)a.ldx * xb;
        const uint8_t *xB = static_cast<const uint8_t *>(a.x) + (size_t)rows[g + 8 < nr ? g + 8 : 0] * (size_t)a.ldx * xb;
        float acc[LG / 8][4];
#pragma unroll
        for (int j = 0; j < LG / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
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
            if (!SAME && !isfinite(v) && c < rank)
                v = dot_again<WBF>(static_cast<const uint8_t *>(a.x) + (size_t)rows[m] * (size_t)a.ldx * xb, a.x_type,
                                   static_cast<const uint8_t *>(a.A) + ((size_t)id * a.r_max + r0 + c) * (size_t)a.K * 2, a.K);
            a.t[(size_t)rows[m] * a.r_max + r0 + c] = v;
        }
        cluster.sync();  // the others may still be reading this block's sums
    }
    if (!waited) pdl_wait();
}

template <bool WBF>
__global__ void __launch_bounds__(LWARPS * 32, 3) k_lora_expand(const LoraArgs a) {
    __shared__ __align__(16) Items it;
    // t of an item, a step of 64 ranks, as three bf16 terms (16-byte pieces
    // swizzled by row: the lanes' reads are free of bank conflicts)
    __shared__ __align__(16) uint16_t s_t[3][LR][64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    find_items(it, a);
    pdl_launch_dependents();
    const long long n0 = (long long)blockIdx.x * LCOLS + warp * LNT * 8;
    // an adapter's factor, after the wait only: the kernel before may write it
    auto scale_of = [&](int id) { return id >= 0 && a.scale ? a.scale[id] : 1.0f; };
    // four outputs at a time where every row starts at a 16-byte boundary
    const bool quads = (a.N & 3) == 0 && (a.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 15) == 0 &&
                       (!a.base || ((a.ldb & 3) == 0 && (reinterpret_cast<uintptr_t>(a.base) & 15) == 0));
    // Items of one or two rows first, the warps on their own: lane (g, t4) has
    // the outputs 8 j + g and the ranks 8 t4 .. 8 t4 + 7 of each 32; the next
    // item's row pieces of B are on their way during this one's products.
    {
        auto next_few = [&](int i) {
            while (i < it.n && (it.rows[i] > 2 || (it.id[it.lead[i]] < 0 && a.base == a.Y))) i += gridDim.y;
            return i;
        };
        const long long nb = n0 + g;
        uint32_t cols = 0;  // bit j: this lane's output 8 j + g is there
#pragma unroll
        for (int j = 0; j < LNT; ++j) cols |= nb + j * 8 < a.N ? 1u << j : 0u;
        const size_t b_lane = ((size_t)nb * a.r_max + t4 * 8) * 2, b_adapter = (size_t)a.N * a.r_max * 2;
        auto load_b = [&](int i, int k0, uint4 (&b)[LNT]) {
            const int id = it.id[it.lead[i]], left = it.rank[it.lead[i]] - k0 - t4 * 8;
            const uint8_t *p = static_cast<const uint8_t *>(a.B) + (size_t)(id < 0 ? 0 : id) * b_adapter + b_lane + (size_t)k0 * 2;
#pragma unroll
            for (int j = 0; j < LNT; ++j) {
                b[j] = left > 0 && ((cols >> j) & 1u) ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
                p += 16 * a.r_max;
            }
        };
        int i = next_few(blockIdx.y);
        uint4 next[LNT];
        if (i < it.n) load_b(i, 0, next);
        pdl_wait();
        while (i < it.n) {
            uint4 b[LNT];
#pragma unroll
            for (int j = 0; j < LNT; ++j) b[j] = next[j];
            const int lead = it.lead[i], nr = it.rows[i], rank = it.rank[lead], cur = i;
            const int row[2] = {lead, nr == 2 ? it.mate[lead] : lead};
            const float sc = scale_of(it.id[lead]);
            i = next_few(i + gridDim.y);
            // what comes after the first 32 ranks: of this item, or the next item's
            if (rank > 32) load_b(cur, 32, next);
            else if (i < it.n) load_b(i, 0, next);
            const long long nw = n0 + t4 * 8 + g;  // the output this lane writes
            float base[2], acc[LNT][2] = {};
#pragma unroll
            for (int m = 0; m < 2; ++m)
                base[m] = a.base && m < nr && nw < a.N ? a.base[(size_t)row[m] * a.ldb + nw] : 0.0f;
            for (int k0 = 0; k0 < rank; k0 += 32) {
                const int k = k0 + t4 * 8, left = rank - k;
                if (k0 > 0) {
#pragma unroll
                    for (int j = 0; j < LNT; ++j) b[j] = next[j];
                    if (k0 + 32 < rank) load_b(cur, k0 + 32, next);
                    else if (i < it.n) load_b(i, 0, next);
                }
                float t[2][8];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float4 u = make_float4(0, 0, 0, 0), v = u;
                    if (m < nr && left > 0) {
                        const float4 *tr = reinterpret_cast<const float4 *>(a.t + (size_t)row[m] * a.r_max + k);
                        u = tr[0];
                        v = tr[1];
                    }
                    t[m][0] = u.x, t[m][1] = u.y, t[m][2] = u.z, t[m][3] = u.w;
                    t[m][4] = v.x, t[m][5] = v.y, t[m][6] = v.z, t[m][7] = v.w;
                }
                if (left < 8) {  // past the rank t is not written and B not used
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (e >= left) t[0][e] = t[1][e] = 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < LNT; ++j) b[j] = below_rank(b[j], left);
                }
#pragma unroll
                for (int j = 0; j < LNT; ++j) {
                    float w[8];
                    wide_w<WBF>(b[j], w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[j][0] = fmaf(w[e], t[0][e], acc[j][0]);
                    if (nr == 2)
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[j][1] = fmaf(w[e], t[1][e], acc[j][1]);
                }
            }
            // the four lanes of an output add up; lane t4 writes output 8 t4 + g
            static_assert(LNT == 4, "one output a lane");
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
                if (m < nr && nw < a.N) a.Y[(size_t)row[m] * a.ldy + nw] = rank > 0 ? base[m] + sc * mine : base[m];
            }
        }
    }
    // Items of three rows and more, in steps of 64 ranks: the block splits t
    // into its three terms once, in shared memory, and the next step's B and t
    // are on their way during the last additions of this one.
    auto next_many = [&](int i) {
        while (i < it.n && (it.rows[i] <= 2 || (it.id[it.lead[i]] < 0 && a.base == a.Y))) i += gridDim.y;
        return i;
    };
    // Column c of the MMAs' tile j is output 8 (c / 2) + 2 j + c % 2, so that a
    // lane's columns of the four tiles are 8 consecutive outputs.
    uint4 b[2][LNT];
    const long long ny = n0 + t4 * 8, nb = n0 + (g >> 1) * 8 + (g & 1);
    uint32_t cols = 0;  // bit j: this lane's row of B for tile j is there
#pragma unroll
    for (int j = 0; j < LNT; ++j) cols |= nb + j * 2 < a.N ? 1u << j : 0u;
    const bool y4[2] = {ny < a.N, ny + 4 < a.N};  // where quads
    const size_t b_lane = ((size_t)nb * a.r_max + t4 * 8) * 2, b_adapter = (size_t)a.N * a.r_max * 2;
    auto load_b = [&](int i, int k0) {
        const int id = it.id[it.lead[i]], left = it.rank[it.lead[i]] - k0 - t4 * 8;
        const uint8_t *p = static_cast<const uint8_t *>(a.B) + (size_t)(id < 0 ? 0 : id) * b_adapter + b_lane + (size_t)k0 * 2;
#pragma unroll
        for (int j = 0; j < LNT; ++j) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                b[c][j] = left > c * 32 && ((cols >> j) & 1u) ? *reinterpret_cast<const uint4 *>(p + c * 64)
                                                              : make_uint4(0, 0, 0, 0);
            p += 4 * a.r_max;
        }
    };
    const int tm = tid >> 4, tk = (tid & 15) * 4;  // the row and ranks of t that this thread brings
    auto load_t = [&](int i, int k0) {
        return tm < it.rows[i] && k0 + tk < it.rank[it.lead[i]]
                   ? *reinterpret_cast<const float4 *>(a.t + (size_t)it.row[i][tm] * a.r_max + k0 + tk)
                   : make_float4(0, 0, 0, 0);
    };
    const int sw = (tk >> 3 ^ tm & 7) * 8 + (tk & 4);  // where it lies in the row
    int i = next_many(blockIdx.y), k0 = 0;
    float4 tv = make_float4(0, 0, 0, 0);
    if (i < it.n) {
        load_b(i, 0);
        tv = load_t(i, 0);
    }
    // The item from which on this thread leaves its outputs to the loop at the end
    // (formed again in here, with what calls keep in registers, they cost every
    // call 2 us of 19).
    int again = HQ_MAX_M;
    float acc[LNT][4];
#pragma unroll
    for (int j = 0; j < LNT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    while (i < it.n) {
        const int nr = it.rows[i], rank = it.rank[it.lead[i]], cur = i;
        const float sc = scale_of(it.id[it.lead[i]]);
        const bool end = k0 + 64 >= rank;
        {
            const int left = rank - k0 - tk;  // past the rank nothing is used
            uint32_t u[3], v[3];
            split3(left > 0 ? tv.x : 0.0f, left > 1 ? tv.y : 0.0f, u);
            split3(left > 2 ? tv.z : 0.0f, left > 3 ? tv.w : 0.0f, v);
#pragma unroll
            for (int x = 0; x < 3; ++x)
                *reinterpret_cast<uint2 *>(&s_t[x][tm][sw]) = make_uint2(u[x], v[x]);
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int left = rank - k0 - c * 32 - t4 * 8;  // ranks left from this lane's first on
            if (k0 + c * 32 >= rank) break;
            if (left > 0 && left < 8)
#pragma unroll
                for (int j = 0; j < LNT; ++j) b[c][j] = below_rank(b[c][j], left);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                const uint4 p = *reinterpret_cast<const uint4 *>(&s_t[x][g][(c * 4 + t4 ^ g) * 8]);
                const uint4 q = *reinterpret_cast<const uint4 *>(&s_t[x][g + 8][(c * 4 + t4 ^ g) * 8]);
                const uint32_t xa[4] = {p.x, q.x, p.y, q.y}, xb[4] = {p.z, q.z, p.w, q.w};
#pragma unroll
                for (int j = 0; j < LNT; ++j) {
                    if constexpr (WBF) {
                        mma16<true>(acc[j], xa, b[c][j].x, b[c][j].y);
                        mma16<true>(acc[j], xb, b[c][j].z, b[c][j].w);
                    } else {
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            uint32_t h0[2], h1[2];
                            split_half(st ? b[c][j].z : b[c][j].x, h0);
                            split_half(st ? b[c][j].w : b[c][j].y, h1);
                            mma16<true>(acc[j], st ? xb : xa, h0[0], h1[0]);
                            mma16<true>(acc[j], st ? xb : xa, h0[1], h1[1]);
                        }
                    }
                }
            }
        }
        __syncthreads();  // the next step writes s_t
        k0 = end ? 0 : k0 + 64;
        if (end) i = next_many(i + gridDim.y);
        if (i < it.n) {
            load_b(i, k0);
            tv = load_t(i, k0);
        }
        if (!end) continue;
        float odd = 0.0f;  // NaN where a sum is not finite
#pragma unroll
        for (int j = 0; j < LNT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) odd = fmaf(acc[j][e], 0.0f, odd);
        if (odd != 0.0f && again > cur) again = cur;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = g + 8 * h;
            if (m >= nr || again <= cur) continue;
            const size_t r = it.row[cur][m];
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = 0.0f;
            if (a.base) {
                const float *s = a.base + r * a.ldb + ny;
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    if (quads) {
                        if (y4[e >> 2]) {
                            const float4 u = *reinterpret_cast<const float4 *>(s + e);
                            y[e] = u.x, y[e + 1] = u.y, y[e + 2] = u.z, y[e + 3] = u.w;
                        }
                    } else {
#pragma unroll
                        for (int f = e; f < e + 4; ++f)
                            if (ny + f < a.N) y[f] = s[f];
                    }
                }
            }
            if (rank > 0)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += sc * acc[e >> 1][2 * h + (e & 1)];
            float *d = a.Y + r * a.ldy + ny;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                if (quads) {
                    if (y4[e >> 2]) *reinterpret_cast<float4 *>(d + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else {
#pragma unroll
                    for (int f = e; f < e + 4; ++f)
                        if (ny + f < a.N) d[f] = y[f];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < LNT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    }
    // the first item with a sum that is not finite, and what comes after it
    for (i = again; i < it.n; i = next_many(i + gridDim.y))
        for (int h = 0; h < 2; ++h) {
            if (g + 8 * h >= it.rows[i] || ny >= a.N) continue;
            const size_t r = it.row[i][g + 8 * h];
            const int id = it.id[it.lead[i]];
            outputs_again<WBF>(a.base ? a.base + r * a.ldb + ny : nullptr, a.Y + r * a.ldy + ny, a.t + r * a.r_max,
                               static_cast<const uint8_t *>(a.B) + ((size_t)(id < 0 ? 0 : id) * a.N + ny) * (size_t)a.r_max * 2,
                               a.r_max, it.rank[it.lead[i]], scale_of(id), a.N - ny < 8 ? (int)(a.N - ny) : 8);
        }
}

}  // namespace

cudaError_t launch_lora(const LoraArgs &a, int w_type, bool pdl, cudaStream_t s) {
    const bool bf = w_type == HQ_BF16, same = a.x_type == w_type;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    // items in turn by as many blocks as are resident at once: two an SM of the
    // shrink, three of the expand (two, with registers for more loads ahead:
    // the whole call for 128 rows of 24576 outputs 39 us instead of 31 then; now 25)
    const int rg = (a.r_max + LG - 1) / LG, tiles = (int)(((long long)a.N + LCOLS - 1) / LCOLS);
    auto least = [&](long long want) { return (unsigned)(want < 1 ? 1 : want < a.M ? want : a.M); };
    const dim3 grid(LCL, least((2LL * sms / LCL + rg - 1) / rg), (unsigned)rg), block(LWARPS * 32);
    cudaError_t e;
    if (bf)
        e = same ? launch_kernel(k_lora_shrink<true, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<true, false>, grid, block, 0, pdl, s, a);
    else
        e = same ? launch_kernel(k_lora_shrink<false, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<false, false>, grid, block, 0, pdl, s, a);
    if (e != cudaSuccess) return e;
    const dim3 eg((unsigned)tiles, least(3LL * sms / tiles));
    // the expand always follows the shrink programmatically: it loads its
    // weights while the shrink runs
    return bf ? launch_kernel(k_lora_expand<true>, eg, block, 0, true, s, a)
              : launch_kernel(k_lora_expand<false>, eg, block, 0, true, s, a);
}

}  // namespace hq
