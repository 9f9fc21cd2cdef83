// k_lora.cu -- low-rank adapters of many requests beside a shared projection.
//
//   t[m] = A[a] x[m]  (a = ids[m], rank r),   Y[m] = base[m] + scale[a] * B[a] t[m]
//
// Two kernels.  The rows of one adapter form items of up to 16 rows (the MMA's
// M); an item is led by the row whose number among the rows of its adapter is
// a multiple of 16, so the grid has one slot per row and the blocks of the
// other rows leave at once: no list is built on the host, and ids may come in
// any order.  Each item reads its adapter once.
//
// k_lora_shrink: a cluster of 8 thread blocks per item splits K; every warp
// forms 16 x 64 partial sums with m16n8k16 MMAs straight from global memory.
// The sum over k does not care in which order the k are taken as long as both
// operands agree, so a lane's 16-byte loads of 8 consecutive k serve two MMA
// steps as they are.  Warps add up in shared memory, the blocks through the
// cluster's distributed shared memory, in a fixed order.
// k_lora_expand: each warp forms 16 rows x 32 outputs with the same MMAs over
// the rank and adds base.
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

// The item led by `row`: its rows in s_rows (their number returned, 0 if
// `row` leads none).  All threads of the block call it.
__device__ int item_rows(const int32_t *ids, int M, int n_adapters, int row, int id, int *s_rows, uint32_t *s_mask) {
    const int tid = threadIdx.x;
    if (tid < HQ_MAX_M) {
        const bool same = tid < M && ids[tid] == id;
        const uint32_t b = __ballot_sync(0xffffffffu, same);
        if ((tid & 31) == 0) s_mask[tid >> 5] = b;
    }
    __syncthreads();
    if (id < 0 || id >= n_adapters) return 0;
    auto before = [&](int r) {  // rows of this adapter below row r
        int n = __popc(s_mask[r >> 5] & ((1u << (r & 31)) - 1u));
        for (int w = 0; w < (r >> 5); ++w) n += __popc(s_mask[w]);
        return n;
    };
    const int first = before(row);
    if (first % LR != 0) return 0;
    int total = 0;
#pragma unroll
    for (int w = 0; w < HQ_MAX_M / 32; ++w) total += __popc(s_mask[w]);
    const int n = total - first < LR ? total - first : LR;
    if (tid < HQ_MAX_M && ((s_mask[tid >> 5] >> (tid & 31)) & 1u)) {
        const int k = before(tid) - first;
        if (k >= 0 && k < LR) s_rows[k] = tid;
    }
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

template <bool WBF, bool SAME>
__global__ void __cluster_dims__(LCL, 1, 1) __launch_bounds__(LWARPS * 32) k_lora_shrink(const LoraArgs a) {
    __shared__ int s_rows[LR];
    __shared__ uint32_t s_mask[HQ_MAX_M / 32];
    __shared__ float s_part[LWARPS][LR][LG + 4];
    cg::cluster_group cluster = cg::this_cluster();
    const int part = blockIdx.x, row0 = blockIdx.y, r0 = blockIdx.z * LG;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int id = a.ids[row0];
    const int nr = item_rows(a.ids, a.M, a.n_adapters, row0, id, s_rows, s_mask);
    const int rank = nr > 0 ? rank_of(a, id) - r0 : 0;
    pdl_launch_dependents();
    if (nr == 0 || rank <= 0) {  // the same for the whole cluster
        pdl_wait();
        return;
    }
    const int nt = rank >= LG ? LG / 8 : (rank + 7) / 8;

    constexpr int NX = SAME ? 1 : 3;
    const int units = (a.K + 31) / 32;
    const int u0 = (int)((long long)units * part / LCL), u1 = (int)((long long)units * (part + 1) / LCL);
    const uint8_t *Aw = static_cast<const uint8_t *>(a.A) + ((size_t)id * a.r_max + r0 + g) * (size_t)a.K * 2;
    float acc[LG / 8][4];
#pragma unroll
    for (int j = 0; j < LG / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    const int xb = type_bytes(a.x_type);
    const uint8_t *xA = static_cast<const uint8_t *>(a.x) + (size_t)s_rows[g < nr ? g : 0] * (size_t)a.ldx * xb;
    const uint8_t *xB = static_cast<const uint8_t *>(a.x) + (size_t)s_rows[g + 8 < nr ? g + 8 : 0] * (size_t)a.ldx * xb;
    bool waited = false;
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
                for (int i = 0; i < NX; ++i) {
                    const uint32_t x4[4] = {p[i][2 * st], q[i][2 * st], p[i][2 * st + 1], q[i][2 * st + 1]};
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
    if (!waited) pdl_wait();
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
    const int cols = nt * 8;
    for (int i = tid; i < LR * cols; i += LWARPS * 32) {
        const int m = i / cols, c = i % cols;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < LWARPS; ++w) v += s_part[w][m][c];
        s_part[0][m][c] = v;
    }
    cluster.sync();
    // each block of the cluster adds up its share of the item's elements
    for (int i = part * (LWARPS * 32) + tid; i < nr * cols; i += LCL * LWARPS * 32) {
        const int m = i / cols, c = i % cols;
        float v = 0.0f;
#pragma unroll
        for (int b = 0; b < LCL; ++b) v += *cluster.map_shared_rank(&s_part[0][m][c], b);
        a.t[(size_t)s_rows[m] * a.r_max + r0 + c] = v;
    }
    cluster.sync();  // the others may still be reading this block's sums
}

template <bool WBF>
__global__ void __launch_bounds__(LWARPS * 32) k_lora_expand(const LoraArgs a) {
    __shared__ int s_rows[LR];
    __shared__ uint32_t s_mask[HQ_MAX_M / 32];
    const int row0 = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int id = a.ids[row0];
    const int nr = item_rows(a.ids, a.M, a.n_adapters, row0, id, s_rows, s_mask);
    pdl_launch_dependents();
    if (nr == 0) {
        pdl_wait();
        if (id >= 0 && id < a.n_adapters) return;     // part of another row's item
        if (a.base == a.Y) return;                    // in place: nothing to change
        const long long c0 = (long long)blockIdx.x * LCOLS, c1 = c0 + LCOLS < a.N ? c0 + LCOLS : a.N;
        for (long long n = c0 + tid; n < c1; n += LWARPS * 32)
            a.Y[(size_t)row0 * a.ldy + n] = a.base ? a.base[(size_t)row0 * a.ldb + n] : 0.0f;
        return;
    }
    const int rank = rank_of(a, id);
    const long long n0 = (long long)blockIdx.x * LCOLS + warp * LNT * 8;
    const uint8_t *Bw = static_cast<const uint8_t *>(a.B) + (size_t)id * a.N * (size_t)a.r_max * 2;
    float acc[LNT][4];
#pragma unroll
    for (int j = 0; j < LNT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    bool waited = false;
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
                for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < left ? w[i] : 2 * i < left ? w[i] & 0xffffu : 0u;
                b[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (!waited) {
            pdl_wait();
            waited = true;
        }
        uint32_t p[3][4], q[3][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = g + 8 * h;
            const float *tr = a.t + (size_t)s_rows[m < nr ? m : 0] * a.r_max + k;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f0 = m < nr && 2 * i < left ? tr[2 * i] : 0.0f;
                const float f1 = m < nr && 2 * i + 1 < left ? tr[2 * i + 1] : 0.0f;
                uint32_t s[3];
                split3(f0, f1, s);
#pragma unroll
                for (int x = 0; x < 3; ++x) (h ? q : p)[x][i] = s[x];
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
    if (!waited) pdl_wait();
    const float sc = a.scale ? a.scale[id] : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = g + 8 * h;
        if (m >= nr) continue;
        const size_t r = (size_t)s_rows[m];
#pragma unroll
        for (int j = 0; j < LNT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const long long n = n0 + j * 8 + 2 * t4 + e;
                if (n >= a.N) continue;
                const float d = rank > 0 ? sc * acc[j][2 * h + e] : 0.0f;
                a.Y[r * a.ldy + n] = a.base ? a.base[r * a.ldb + n] + d : d;
            }
    }
}

}  // namespace

cudaError_t launch_lora(const LoraArgs &a, int w_type, bool pdl, cudaStream_t s) {
    const bool bf = w_type == HQ_BF16, same = a.x_type == w_type;
    const dim3 grid(LCL, (unsigned)a.M, (unsigned)((a.r_max + LG - 1) / LG)), block(LWARPS * 32);
    cudaError_t e;
    if (bf)
        e = same ? launch_kernel(k_lora_shrink<true, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<true, false>, grid, block, 0, pdl, s, a);
    else
        e = same ? launch_kernel(k_lora_shrink<false, true>, grid, block, 0, pdl, s, a)
                 : launch_kernel(k_lora_shrink<false, false>, grid, block, 0, pdl, s, a);
    if (e != cudaSuccess) return e;
    const dim3 eg((unsigned)(((long long)a.N + LCOLS - 1) / LCOLS), (unsigned)a.M);
    // the expand always follows the shrink programmatically: it loads its
    // weights while the shrink runs
    return bf ? launch_kernel(k_lora_expand<true>, eg, block, 0, true, s, a)
              : launch_kernel(k_lora_expand<false>, eg, block, 0, true, s, a);
}

}  // namespace hq
