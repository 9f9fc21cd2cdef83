// k_prefix.cu -- attention of a batch over a paged cache whose sequences share
// a long prefix, the shared keys and values read once for all rows.
//
//   out[i][h] = sum_p w_p V[p] / sum_p w_p,   w_p = exp(scale q[i][h] . K[p])
//
// over the positions row i sees.  A softmax over a union of positions is the
// merge of the softmaxes over its parts, each known by its running maximum m,
// its sum l = sum exp(x - m) and its unnormalized output: so the positions are
// cut into parts that different thread blocks take, and a second kernel merges
// them.  The parts of a row:
//   - the shared positions, in whole tiles of 64: all rows of the batch that
//     read one key/value head (rows * G of them) are one matrix, cut into
//     tiles of rows; long prefixes are split further;
//   - the sequence's own positions (with what the shared ones leave over of a
//     tile), for the sequence's own rows only.
// Shared tiles have no mask at all; the own positions end with the tree.
//
// Per block: one producer warp brings each 64-position tile of K and V with
// TMA tiled copies (a page, or 64 positions of it, per box, in 128-byte
// swizzle) into a ring of stages; the lanes look the pages up in parallel.
// Four consumer warps form S = Q K^T and O += P V on the tensor cores with fp32
// accumulation and an online softmax in base-2 units: KW of them share 16 rows
// and take every KW-th group of 16 positions of a tile (a single token's few
// rows do not fill more than one warp's MMA), 4 / KW row groups to a block; at
// the end the warps of a row group merge in shared memory.  What bounds it is
// memory where there are many blocks: 128 sequences' own positions, 270 MB in 50
// us = 5.4 TB/s (beside the shared parts: less, see launch_prefix_attention);
// the chain sequence - page - tile - merge where there are few: 4 rows, 1000
// shared and up to 200 own positions, 11 us for both kernels.
// Many rows go to the tensor-memory kernels of k_prefix_tc.cu.
#include "prefix_common.cuh"

namespace hq {
namespace {

constexpr int XKEYS = 64;     // positions per stage
constexpr int XSTAGES = 3;
constexpr int XCW = 4;        // consumer warps
constexpr int XTHREADS = (XCW + 1) * 32;
constexpr int TC_KEYS = 128;    // positions (and query rows) of a tile of the tensor-memory kernels
// Times below: whole calls replayed from a graph, cold L2 cache, 32 query and 8
// key/value heads of 128, bf16.
// From TC_ROWS rows a head on, and with at least one of its tiles, the shared
// parts go to the tensor-memory kernel.  With it and without: 32 rows on 4096
// shared positions 23.7 us both; 48 on 1000 24 and 27; 64 on 32768 50 and 79;
// 256 on 4096 46 and 79.
constexpr int TC_ROWS = 33;
// From TC_ROWS_OWN rows a head on so do a sequence's own parts.  16 sequences of
// 700 own positions behind 2048 shared: 16 rows 37 and 34 us; 20 rows 35 and 37;
// 32 rows 37 and 40; 48 rows 38 and 47.  A lone tree takes its prefix along: 32
// rows on 2048 + 700 positions 19 us, 22 with the prefix apart.
constexpr int TC_ROWS_OWN = 17;
// In the time of one tile of the shared parts' tensor-memory kernel (1.6 us) an
// SM takes about this many own positions of a head, in k_prefix_attn and in
// k_prefix_own.  (From two calls, 128 single tokens and 48 draft trees, with heads
// of 128 and G = 4; other shapes only take another number of blocks by it.)
constexpr int OWN_POS = 160, OWN_POS_TC = 35;
// Probabilities are formed relative to the running maximum less this many base-2
// units.  fp16's smallest normal value is 2^-14, its largest nearly 2^16: 2^15 at
// the maximum leaves 29 of its powers for the smaller ones (with 0, a flat tail
// 2^-26 below one key was lost altogether).  bf16 has fp32's range.
constexpr float P_SHIFT_F16 = 15.0f;
constexpr int MAX_PARTS = 64;   // shared_parts + own_parts, at most 32 each

template <int D>
struct Tile {
    static constexpr int BOX = XKEYS * 128;           // 64 positions x 64 dimensions
    static constexpr int BYTES = (D / 64) * BOX;      // K or V of a stage
    static constexpr int STAGE = 2 * BYTES;
    static constexpr size_t SMEM = 1024 + (size_t)XSTAGES * STAGE + 2 * XSTAGES * 8 + 64 * 16 + HQ_MAX_M * 4;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

template <bool BF>
__device__ __forceinline__ void mma_x(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Whether a pair holds an infinity or NaN (all exponent bits set).
template <bool BF>
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
    constexpr uint32_t e = BF ? 0x7f80u : 0x7c00u;
    return (w & e) == e || ((w >> 16) & e) == e;
}

template <int D, bool BF, int KW>
__global__ void __launch_bounds__(XTHREADS, 2)
    k_prefix_attn(const PrefixArgs a, const PrefixPlan pl, const __grid_constant__ CUtensorMap map) {
    using T = Tile<D>;
    constexpr int XROWS = 64 / KW;     // query rows of the block
    constexpr int NJ = XKEYS / 8 / KW; // this warp's groups of 8 positions in a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + (size_t)XSTAGES * T::STAGE);  // full[S], empty[S]
    uint32_t *s_anc = reinterpret_cast<uint32_t *>(bars + 2 * XSTAGES);                // [XROWS][4]
    int32_t *s_par = reinterpret_cast<int32_t *>(s_anc + XROWS * 4);                   // [HQ_MAX_M]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < XSTAGES; ++i) {
            mbar_init(smem_addr(&bars[i]), 1);
            mbar_init(smem_addr(&bars[XSTAGES + i]), XCW);
        }
        fence_mbar_init();
    }
    __syncthreads();
    // Behind the tensor-memory kernel nothing is waited for: each of its blocks
    // has itself waited for the call's inputs before this kernel may start, and
    // the SMs that it leaves idle, or is done with, begin here at once.  Only
    // this grid's end, which the merge waits for, must not come before its end.
    const bool last = pl.tc_shared && blockIdx.x == gridDim.x - 1;
    if (!pl.tc_shared) pdl_wait();
    pdl_launch_dependents();  // after the wait: the merge reads lengths before its own

    // which part this block is; nothing to do (ntiles 0) where no row uses it
    int unit = blockIdx.x;
    const int hk = unit % a.Hkv;
    unit /= a.Hkv;
    const int nshared = pl.tc_shared ? 0 : pl.np * pl.ptiles;
    int split, rt, first, nrows, k0, k1, slot, tree0 = 0x7fffffff, nodes = 0, ntiles = 0;
    int early = -1;  // the producer's table entries of the first tile
    if (unit < nshared) {
        split = unit / pl.ptiles;
        rt = unit % pl.ptiles;
        first = 0;
        nrows = a.rows * a.G;
        k0 = split * pl.pchunk;
        k1 = k0 + pl.pchunk < pl.s0 ? k0 + pl.pchunk : pl.s0;
        const Seq s = first_live(a);
        slot = s.slot;
        if (s.live) ntiles = (k1 - k0) / XKEYS;
    } else {
        unit -= nshared;
        const int b = unit / (pl.ns * pl.stiles);
        unit %= pl.ns * pl.stiles;
        split = unit / pl.stiles;
        rt = unit % pl.stiles;
        k0 = pl.s0 + split * pl.schunk;
        if (warp == XCW) early = early_entry<XKEYS>(a, b, k0);
        const Seq s = seq_of(a, b);
        first = s.first;
        nodes = s.m;
        nrows = s.m * a.G;
        k1 = s.len - k0 > pl.schunk ? k0 + pl.schunk : s.len;
        slot = s.slot;
        tree0 = s.len - s.m;
        split += pl.np;
        // (past the sequence's end the merge does not look)
        if (s.live && rt * XROWS < nrows && k0 < k1) ntiles = (k1 - k0 + XKEYS - 1) / XKEYS;
    }
    if (ntiles == 0) {
        if (last) pdl_wait();
        return;
    }

    if (warp == XCW) {
        // ------------------------------------------------------ producer ---
        const int32_t *row = a.table + (size_t)slot * a.max_pages;
        int i = 0;
        for (; i < ntiles; ++i) {
            const int st = i % XSTAGES, p = k0 + i * XKEYS;
            const int page = i == 0 && nodes > 0 ? checked_page<XKEYS>(a, early, p, k1) : lookup_page<XKEYS>(a, row, p, k1);
            if (i >= XSTAGES &&
                !mbar_wait_short(smem_addr(&bars[XSTAGES + st]), (uint32_t)((i / XSTAGES) & 1) ^ 1u, a.err))
                break;
            __syncwarp();
            const uint32_t bar = smem_addr(&bars[st]), kt = smem_addr(ring + (size_t)st * T::STAGE);
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)T::STAGE);
            __syncwarp();
            load_tile<XKEYS, D>(a, &map, kt, p, hk, a.k_plane, page, bar);
            load_tile<XKEYS, D>(a, &map, kt + T::BYTES, p, hk, a.v_plane, page, bar);
            __syncwarp();
        }
        // no copy may still be landing in shared memory when the block exits
        for (int j = i > XSTAGES ? i - XSTAGES : 0; j < i; ++j)
            mbar_wait_short(smem_addr(&bars[j % XSTAGES]), (uint32_t)((j / XSTAGES) & 1), a.err);
        if (last) pdl_wait();
        return;
    }

    // ---------------------------------------------------------- consumers ---
    const int g8 = lane >> 2, t4 = lane & 3;
    const int kw = warp % KW;                                        // this warp's share of the positions
    const int rA = rt * XROWS + (warp / KW) * 16 + g8, rB = rA + 8;  // this lane's two rows of the part
    uint32_t qa[D / 16][4];
    {
        const bool vA = rA < nrows, vB = rB < nrows;
        const int nA = vA ? rA : 0, nB = vB ? rB : 0;
        const uint32_t *qA = reinterpret_cast<const uint32_t *>(
            static_cast<const uint16_t *>(a.q) + (size_t)(first + nA / a.G) * a.ldq + (size_t)(hk * a.G + nA % a.G) * D);
        const uint32_t *qB = reinterpret_cast<const uint32_t *>(
            static_cast<const uint16_t *>(a.q) + (size_t)(first + nB / a.G) * a.ldq + (size_t)(hk * a.G + nB % a.G) * D);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const int c = ks * 8 + t4;  // 32-bit column: dims 2c, 2c + 1
            qa[ks][0] = vA ? qA[c] : 0u;
            qa[ks][1] = vB ? qB[c] : 0u;
            qa[ks][2] = vA ? qA[c + 4] : 0u;
            qa[ks][3] = vB ? qB[c + 4] : 0u;
        }
    }
    // Ancestor sets of this block's nodes where the part reaches the tree
    // (without `parent`: a chain, every earlier node).
    const int node0 = rt * XROWS / a.G;
    if (k1 > tree0) {
        if (a.parent)
            for (int i = threadIdx.x; i < nodes; i += XCW * 32) s_par[i] = a.parent[first + i];
        named_barrier(1, XCW * 32);
        if (threadIdx.x < XROWS) {
            const int node = node0 + threadIdx.x;
            uint32_t m4[4] = {0u, 0u, 0u, 0u};
            if (node < nodes) {
                m4[node >> 5] |= 1u << (node & 31);
                int cur = node;
                for (int step = 0; step < HQ_MAX_M && cur > 0; ++step) {
                    const int p = a.parent ? s_par[cur] : cur - 1;
                    if (p < 0 || p >= cur) break;
                    m4[p >> 5] |= 1u << (p & 31);
                    cur = p;
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) s_anc[threadIdx.x * 4 + w] = m4[w];
        }
        named_barrier(1, XCW * 32);
    }
    const uint32_t *ancA = s_anc + (rA / a.G - node0) * 4, *ancB = s_anc + (rB / a.G - node0) * 4;

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    float mrun[2] = {-INFINITY, -INFINITY}, lrun[2] = {0.0f, 0.0f};
    bool ok = true;
    const int k_row = (lane >> 4) * 8 + (lane & 7), k_half = (lane >> 3) & 1;
    const int v_row = ((lane >> 3) & 1) * 8 + (lane & 7), v_half = lane >> 4;

    for (int i = 0; i < ntiles; ++i) {
        const int st = i % XSTAGES;
        if (ok) ok = mbar_wait_short(smem_addr(&bars[st]), (uint32_t)((i / XSTAGES) & 1), a.err);
        __syncwarp();
        const uint32_t kt = smem_addr(ring + (size_t)st * T::STAGE), vt = kt + T::BYTES;
        const int p0 = k0 + i * XKEYS;

        // group n of this warp: the 16 positions kw + n * KW of the tile
        float s[NJ][4];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int n = 0; n < NJ / 2; ++n) {
                uint32_t b0, b1, b2, b3;
                ldsm4(kt + (uint32_t)((ks >> 2) * T::BOX) + swz128((kw + n * KW) * 16 + k_row, 2 * (ks & 3) + k_half),
                      b0, b1, b2, b3);
                mma_x<BF>(s[2 * n], qa[ks], b0, b1);
                mma_x<BF>(s[2 * n + 1], qa[ks], b2, b3);
            }

        // scale to base-2 units, mask, running maximum.  `sees`: which of the
        // tile's positions each of this lane's two rows sees (bit = position)
        const bool full = p0 + XKEYS <= tree0 && p0 + XKEYS <= k1;
        uint64_t sees[2] = {~0ull, ~0ull};
        if (!full) {
            const int n = k1 - p0, old = tree0 - p0;  // positions in the part; before the tree
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t *anc = h ? ancB : ancA;
                uint64_t v = old >= 64 ? ~0ull : old > 0 ? (1ull << old) - 1 : 0ull;
                if (old < 64) {
                    const uint64_t lo = anc[0] | (uint64_t)anc[1] << 32, hi = anc[2] | (uint64_t)anc[3] << 32;
                    if (old >= 0)
                        v |= lo << old;
                    else if (old > -64)
                        v |= lo >> -old | hi << (64 + old);
                    else
                        v |= hi >> (-64 - old);  // old > -128: the part ends with the tree
                }
                if (n < 64) v &= (1ull << n) - 1;
                sees[h] = v >> (kw * 16 + 2 * t4);
            }
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = (j >> 1) * KW * 16 + (j & 1) * 8 + (e & 1);  // the position, less kw * 16 + 2 * t4
                const float x = full || ((sees[e >> 1] >> at) & 1) ? s[j][e] * a.c_log2 : -INFINITY;
                s[j][e] = x;
                mx[e >> 1] = fmaxf(mx[e >> 1], x);
            }
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            if constexpr (!BF) mx[h] -= P_SHIFT_F16;  // mrun is the reference, not the maximum
            const float mnew = fmaxf(mrun[h], mx[h]);
            alpha[h] = mnew == -INFINITY ? 1.0f : ex2(mrun[h] - mnew);
            mx[h] = mnew == -INFINITY ? 0.0f : mnew;  // no visible position yet: probabilities 0
            mrun[h] = mnew;
        }
        float rs[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = ex2(s[j][e] - mx[e >> 1]);
                s[j][e] = p;
                rs[e >> 1] += p;
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) lrun[h] = lrun[h] * alpha[h] + rs[h];
        if (!__all_sync(0xffffffffu, alpha[0] == 1.0f && alpha[1] == 1.0f)) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
        }

        // O += P V: P rounded to the cache's type.  A masked position weighs 0,
        // and 0 times an infinity or NaN is NaN: in a masked group of 16
        // positions whose values are not all finite, each row adds the
        // positions it sees one by one.
#pragma unroll
        for (int kk = 0; kk < NJ / 2; ++kk) {
            uint32_t pa[4];
            pa[0] = pack2<BF>(s[2 * kk][0], s[2 * kk][1]);
            pa[1] = pack2<BF>(s[2 * kk][2], s[2 * kk][3]);
            pa[2] = pack2<BF>(s[2 * kk + 1][0], s[2 * kk + 1][1]);
            pa[3] = pack2<BF>(s[2 * kk + 1][2], s[2 * kk + 1][3]);
            uint32_t v[D / 16][4];
            const int r0 = (kw + kk * KW) * 16;  // the group's first row of the tile
            bool odd = false;
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp)
                ldsm4t(vt + (uint32_t)((dp >> 2) * T::BOX) + swz128(r0 + v_row, 2 * (dp & 3) + v_half), v[dp][0], v[dp][1],
                       v[dp][2], v[dp][3]);
            if (!full && (p0 + r0 + 16 > tree0 || p0 + r0 + 16 > k1)) {
#pragma unroll
                for (int dp = 0; dp < D / 16; ++dp)
#pragma unroll
                    for (int e = 0; e < 4; ++e) odd |= nonfinite2<BF>(v[dp][e]);
                odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
#pragma unroll
                for (int dp = 0; dp < D / 16; ++dp) {
                    mma_x<BF>(o[2 * dp], pa, v[dp][0], v[dp][1]);
                    mma_x<BF>(o[2 * dp + 1], pa, v[dp][2], v[dp][3]);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < 16; ++c) {
                    const int from = (lane & ~3) | ((c & 7) >> 1);
                    const float x = c & 8 ? (c & 1 ? s[2 * kk + 1][1] : s[2 * kk + 1][0]) : (c & 1 ? s[2 * kk][1] : s[2 * kk][0]);
                    const float y = c & 8 ? (c & 1 ? s[2 * kk + 1][3] : s[2 * kk + 1][2]) : (c & 1 ? s[2 * kk][3] : s[2 * kk][2]);
                    const float pA = __shfl_sync(0xffffffffu, x, from), pB = __shfl_sync(0xffffffffu, y, from);
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        uint32_t w;
                        asm volatile("ld.shared.b32 %0, [%1];"
                                     : "=r"(w)
                                     : "r"(vt + (uint32_t)((n >> 3) * T::BOX) + swz128(r0 + c, n & 7) + (uint32_t)t4 * 4));
                        const float2 f = unpack2<BF>(w);
                        if (pA != 0.0f) {
                            o[n][0] = fmaf(pA, f.x, o[n][0]);
                            o[n][1] = fmaf(pA, f.y, o[n][1]);
                        }
                        if (pB != 0.0f) {
                            o[n][2] = fmaf(pB, f.x, o[n][2]);
                            o[n][3] = fmaf(pB, f.y, o[n][3]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars[XSTAGES + st]));
    }

#pragma unroll
    for (int h = 0; h < 2; ++h) {
        lrun[h] += __shfl_xor_sync(0xffffffffu, lrun[h], 1);
        lrun[h] += __shfl_xor_sync(0xffffffffu, lrun[h], 2);
    }
    {
        // The warps of a row group merge through the ring, which nothing
        // writes any more: every tile has arrived and been read.
        float *box = reinterpret_cast<float *>(ring);  // [consumer warp][D / 8 * 4 + 4][32 lanes]
        constexpr int PER = (D / 8 * 4 + 4) * 32;
        named_barrier(1, XCW * 32);
        float *mine = box + warp * PER + lane;
        if (kw > 0) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) mine[(j * 4 + e) * 32] = o[j][e];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mine[(D / 2 + h) * 32] = mrun[h];
                mine[(D / 2 + 2 + h) * 32] = lrun[h];
            }
        }
        named_barrier(1, XCW * 32);
        if (kw > 0) return;
        float top[2] = {mrun[0], mrun[1]}, wt[2][KW];
#pragma unroll
        for (int k = 1; k < KW; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) top[h] = fmaxf(top[h], mine[k * PER + (D / 2 + h) * 32]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float t = top[h] == -INFINITY ? 0.0f : top[h];  // nothing seen by any: all weights 0
            wt[h][0] = exp2f(mrun[h] - t);
            lrun[h] *= wt[h][0];
#pragma unroll
            for (int k = 1; k < KW; ++k) {
                wt[h][k] = exp2f(mine[k * PER + (D / 2 + h) * 32] - t);
                lrun[h] += wt[h][k] * mine[k * PER + (D / 2 + 2 + h) * 32];
            }
            mrun[h] = top[h];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[j][e] *= wt[e >> 1][0];
#pragma unroll
                for (int k = 1; k < KW; ++k) o[j][e] += wt[e >> 1][k] * mine[k * PER + (j * 4 + e) * 32];
            }
    }
    // this part's unnormalized outputs, maxima and sums
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = h ? rB : rA;
        if (r >= nrows) continue;
        const size_t row = ((size_t)split * a.rows + first + r / a.G) * a.Hq + hk * a.G + r % a.G;
        float *dst = a.ws_o + row * D;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2 *>(dst + j * 8 + 2 * t4) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
        if (t4 == 0) *reinterpret_cast<float2 *>(a.ws_ml + row * 2) = make_float2(mrun[h], lrun[h]);
    }
}

// Merges the parts of `HG` query heads of one row: blockIdx = (row, group of
// heads).  First the weight of every part, exp2(m - top) over the sum of
// weight times l, into shared memory; then each thread adds up four dimensions
// of one head over every PG-th part (PG groups of threads where the heads
// alone do not fill the block), 8 loads in flight (4 where rows are many), and the groups add up in
// order.  What bounds it is the chain of dependent loads (row -> sequence ->
// maxima -> outputs): the sequence is found by all threads at once and before
// the wait for the parts.  551 rows of 32 heads in 3 parts, 27 MB: 11.5
// us (13.3 with 8 parts in flight for all; 13 with 16 heads a block).
template <int D, int HG>
__global__ void __launch_bounds__(256) k_prefix_merge(const PrefixArgs a, const PrefixPlan pl) {
    constexpr int COLS = HG * D / 4;            // float4 columns
    constexpr int PG = COLS >= 256 ? 1 : 256 / COLS, BATCH = HG == 8 ? 4 : 8;
    __shared__ float s_w[MAX_PARTS][HG];
    __shared__ float4 s_acc[PG > 1 ? 256 : 1];
    __shared__ int s_b;
    const int tid = threadIdx.x, row = blockIdx.x, h0 = blockIdx.y * HG;
    if (tid == 0) s_b = -1;
    __syncthreads();
    pdl_launch_dependents();
    // The inputs of the call are complete: the kernels before this one have
    // waited for them before they let it start.  Only their results are not.
    // The sequence whose rows hold this one (the last, should `starts` repeat it)
    if (a.starts) {
        int mine = -1;
        for (int b = tid; b < a.B; b += 256) {
            int first, m;
            batch_rows(a.starts, b, a.rows, a.max_rows, first, m);
            if (row >= first && row < first + m) mine = b;
        }
        if (mine >= 0) atomicMax(&s_b, mine);
    } else if (tid == 0 && row / a.max_rows < a.B) {
        s_b = row / a.max_rows;
    }
    __syncthreads();
    int parts = 0;
    if (s_b >= 0) {
        const Seq s = seq_of(a, s_b);
        // own parts that reach into the sequence
        if (s.live) parts = pl.np + (s.len - pl.s0 + pl.schunk - 1) / pl.schunk;
    }
    pdl_wait();
    // what went wrong in the parts reaches the cache's status word as well, for
    // callers that keep no workspace of their own
    const bool reports = tid == 0 && blockIdx.x == 0 && blockIdx.y == 0;
    const int wrong = reports ? *static_cast<volatile int *>(a.err) : 0;
    const size_t step = (size_t)a.rows * a.Hq, r0 = (size_t)row * a.Hq + h0;
    // weights: a warp per head, two parts a lane
    static_assert(MAX_PARTS <= 64, "two parts a lane");
    for (int h = tid >> 5; h < HG; h += 8) {
        const int lane = tid & 31;
        const bool in = h0 + h < a.Hq;
        float m2[2], l2[2], top = -INFINITY, den = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int p = lane + 32 * i;
            const float2 ml = in && p < parts ? *reinterpret_cast<const float2 *>(a.ws_ml + (r0 + h + p * step) * 2)
                                              : make_float2(-INFINITY, 0.0f);
            m2[i] = ml.x;
            l2[i] = ml.y;
            top = fmaxf(top, ml.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // a part in which the row saw nothing weighs 0 and is not read
            m2[i] = m2[i] == -INFINITY && l2[i] == 0.0f ? 0.0f : exp2f(m2[i] - top);
            den += m2[i] * l2[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < parts) s_w[lane + 32 * i][h] = m2[i] == 0.0f ? 0.0f : m2[i] / den;
    }
    __syncthreads();
    const int pg = PG > 1 ? tid / COLS : 0;
    for (int c = PG > 1 ? tid % COLS : tid; c < COLS; c += 256) {
        const int h = c / (D / 4), d = (c % (D / 4)) * 4;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float *src = a.ws_o + (r0 + h) * D + d;
        for (int p0 = pg; p0 < parts; p0 += PG * BATCH) {
            float4 v[BATCH];
            float w[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int p = p0 + i * PG;
                w[i] = p < parts && h0 + h < a.Hq ? s_w[p][h] : 0.0f;
                v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (w[i] != 0.0f) v[i] = *reinterpret_cast<const float4 *>(src + (size_t)p * step * D);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                acc.x += w[i] * v[i].x;
                acc.y += w[i] * v[i].y;
                acc.z += w[i] * v[i].z;
                acc.w += w[i] * v[i].w;
            }
        }
        if constexpr (PG > 1) {
            s_acc[tid] = acc;
            __syncthreads();
            if (pg > 0) return;
#pragma unroll
            for (int g = 1; g < PG; ++g) {
                const float4 v = s_acc[tid + g * COLS];
                acc.x += v.x;
                acc.y += v.y;
                acc.z += v.z;
                acc.w += v.w;
            }
        }
        if (h0 + h >= a.Hq) continue;
        const size_t at = (size_t)row * a.ldo + (size_t)(h0 + h) * D + d;
        if (a.out_type == HQ_F32)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = acc;
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                a.out_type == HQ_F16 ? make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w))
                                     : make_uint2(pack2<true>(acc.x, acc.y), pack2<true>(acc.z, acc.w));
    }
    if (reports && wrong != 0)
        atomicCAS(a.status, 0, wrong == DEV_ERR_TIMEOUT ? (int)HQ_ERR_TIMEOUT : (int)HQ_ERR_INVALID_ARG);
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<EncodeFn>(p);
            fn.store(f, std::memory_order_release);
        }
    }
    return f;
}

// Map of the pool (dimension, row in page, head, page, plane); boxes of 64
// dimensions x min(page_size, box_rows) rows, 128-byte swizzle.
cudaError_t pool_map(CUtensorMap *m, const hq_pages &c, int D, int type, int box_rows) {
    EncodeFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)c.row_bytes, page = row * c.page_size;
    const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)c.page_size, (cuuint64_t)c.heads, (cuuint64_t)c.n_pages,
                                (cuuint64_t)c.n_planes};
    const cuuint64_t strides[4] = {row, page, page * c.heads, (cuuint64_t)c.plane_bytes};
    const cuuint32_t box[5] = {64, (cuuint32_t)(c.page_size < box_rows ? c.page_size : box_rows), 1, 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(m, type == HQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                           c.pool, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Partial results (rows x heads x parts) the workspace holds, for a size that
// does not depend on the lengths or on B and grows with rows and max_rows: as
// many parts as it takes to give every SM a block, up to 32 of each kind.  A
// block of the shared parts has up to 256 rows of the n = rows * Hq; the own
// parts of B >= rows / max_rows sequences are wanted for 1280 blocks in all.
long long shared_slots(long long n) { return 32 * n < 40960 + 2 * n ? 32 * n : 40960 + 2 * n; }
long long own_slots(long long n, int max_rows, int G) {
    const long long want = 1280LL * max_rows * G + n;
    return 32 * n < want ? 32 * n : want;
}
int shared_parts(long long n) {
    const long long p = 40960 / n + 1;
    return p > 32 ? 32 : p < 2 ? 2 : (int)p;
}
int own_parts(long long n, int B, int max_rows, int Hkv, int G) {
    const long long p = 1280 / ((long long)B * Hkv) + 1, room = own_slots(n, max_rows, G) / n;
    return (int)(p < room ? p : room);
}

template <int D, bool BF, int KW>
cudaError_t launch_t(const PrefixArgs &a, const PrefixPlan &pl, const CUtensorMap &map, unsigned grid, bool pdl,
                     cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> configured[CACHE_DEVICES];
    int done = 0;
    e = cached_per_device(configured, dev, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(k_prefix_attn<D, BF, KW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tile<D>::SMEM);
    });
    if (e != cudaSuccess) return e;
    return launch_kernel(k_prefix_attn<D, BF, KW>, dim3(grid), dim3(XTHREADS), Tile<D>::SMEM, pdl, s, a, pl, map);
}

template <int D, bool BF>
cudaError_t launch_kw(int kw, const PrefixArgs &a, const PrefixPlan &pl, const CUtensorMap &map, unsigned grid, bool pdl,
                      cudaStream_t s) {
    return kw == 4 ? launch_t<D, BF, 4>(a, pl, map, grid, pdl, s) : launch_t<D, BF, 2>(a, pl, map, grid, pdl, s);
}

template <int D>
cudaError_t launch_merge(const PrefixArgs &a, const PrefixPlan &pl, int sms, cudaStream_t s) {
    // 8 heads a block where that gives every SM one, fewer heads and more
    // threads on the parts of each where rows are few.  Whole calls with 8, 2
    // and 1 heads: 64 rows 36, 38, 40 us; 4 rows 21.6, 16.5, 15.5 us.
    auto grid = [&](int hg) { return dim3((unsigned)a.rows, (unsigned)((a.Hq + hg - 1) / hg)); };
    auto enough = [&](int hg) { return (long long)a.rows * ((a.Hq + hg - 1) / hg) >= sms; };
    if (enough(8)) return launch_kernel(k_prefix_merge<D, 8>, grid(8), dim3(256), 0, true, s, a, pl);
    if (enough(2)) return launch_kernel(k_prefix_merge<D, 2>, grid(2), dim3(256), 0, true, s, a, pl);
    return launch_kernel(k_prefix_merge<D, 1>, grid(1), dim3(256), 0, true, s, a, pl);
}

}  // namespace

size_t prefix_workspace_bytes(int rows, int max_rows, int Hq, int Hkv, int D) {
    const long long n = (long long)rows * Hq;
    return 16 + (size_t)(shared_slots(n) + own_slots(n, max_rows, Hq / Hkv)) * (size_t)(D + 2) * 4;
}

cudaError_t launch_prefix_attention(const hq_pages &c, PrefixArgs a, int D, void *workspace, bool pdl, cudaStream_t s) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    const long long n = (long long)a.rows * a.Hq;
    const int pcap = shared_parts(n), scap = own_parts(n, a.B, a.max_rows, a.Hkv, a.G);
    const long long head_rows = (long long)a.rows * a.G, seq_rows = (long long)a.max_rows * a.G;
    // Which kernel takes which parts: see TC_ROWS.  A short prefix goes with the
    // own parts; so does the prefix of a lone draft tree.  (In the tensor-memory
    // kernels a scale below 0 would turn the maximum into a minimum, a scale of
    // 0 the masks into NaN.)
    PrefixPlan pl;
    pl.tc_shared = head_rows >= TC_ROWS && a.shared >= TC_KEYS && a.c_log2 > 0.0f;
    pl.tc_own = seq_rows >= TC_ROWS_OWN && (pl.tc_shared || a.shared < TC_KEYS || a.B == 1) && a.c_log2 > 0.0f;
    const bool split = pl.tc_shared || (!pl.tc_own && a.shared >= TC_KEYS), pair = head_rows > TC_KEYS;
    // Warps that share 16 rows, from the rows that a block of the other kernel
    // has.  64 sequences of 2000 positions: 16 rows each 108 us with four, 114
    // with two (one: 204); 32 rows each 128 and 120.
    const long long few = split && !pl.tc_shared ? head_rows : seq_rows;
    const int kw = few <= 16 ? 4 : 2, xrows = 64 / kw;
    const int pkey = pl.tc_shared ? TC_KEYS : XKEYS, skey = pl.tc_own ? TC_KEYS : XKEYS;
    const int prows = !pl.tc_shared ? xrows : pair ? 2 * TC_KEYS : TC_KEYS, srows = pl.tc_own ? TC_KEYS : xrows;
    pl.s0 = split ? a.shared / pkey * pkey : 0;
    pl.ptiles = (int)((head_rows + prows - 1) / prows);
    pl.stiles = (int)((seq_rows + srows - 1) / srows);
    // whole tiles, and no more parts than the workspace holds
    auto cut = [&](long long positions, long long want, int most, int tile, int &n, int &chunk) {
        if (want > most) want = most;
        if (want < 1) want = 1;
        long long len = (positions + want - 1) / want;
        len = (len + tile - 1) / tile * tile;
        if (len < tile) len = tile;
        chunk = (int)len;
        n = (int)((positions + len - 1) / len);
    };
    const long long pblocks = (long long)a.Hkv * pl.ptiles, sblocks = (long long)a.Hkv * a.B * pl.stiles;
    long long want = (2LL * sms + pblocks - 1) / pblocks;
    if (pl.tc_shared) {
        // At most one block of the tensor-memory kernel per SM.  The SMs that
        // are left over work on the own parts meanwhile, so fewer blocks than
        // SMs can end earlier: the count with the least estimated time, in units
        // of a block's tile.  All SMs together, bound by memory, take own parts
        // at two thirds of a single one's rate; sequences are taken to have half the
        // largest length (of equal lengths, that is half of what there is).  (128 rows, 32768 shared and up to 1024 own positions: 144
        // blocks 113 us, 112 106, 96 and 80 96, 64 112.)
        const long long tiles = pl.s0 / TC_KEYS, own = sblocks * (a.max_len - pl.s0) / (2 * (pl.tc_own ? OWN_POS_TC : OWN_POS));
        long long best = -1;
        for (long long np = 1; np <= pcap && (np == 1 || np * pblocks <= sms); ++np) {
            const long long t = (tiles + np - 1) / np, rest = own - (sms - pblocks * np) * t;
            const long long cost = 2 * sms * t + (rest > 0 ? 3 * rest : 0);
            if (best < 0 || cost < best) {
                best = cost;
                want = np;
            }
        }
    }
    cut(pl.s0, want, pcap, pkey, pl.np, pl.pchunk);
    cut((long long)a.max_len - pl.s0, ((pl.tc_own ? 2LL : 4LL) * sms + sblocks - 1) / sblocks, scap, skey, pl.ns, pl.schunk);

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.err = reinterpret_cast<int *>(ws);
    a.ws_o = reinterpret_cast<float *>(ws + 16);
    a.ws_ml = a.ws_o + (size_t)(pcap + scap) * n * D;
    a.pool = static_cast<const uint8_t *>(c.pool);
    a.plane_bytes = c.plane_bytes;
    const bool bf = a.type == HQ_BF16;
    CUtensorMap map;
    cudaError_t e;
    if (pl.tc_shared || pl.tc_own) {
        e = pool_map(&map, c, D, a.type, TC_KEYS);
        if (e != cudaSuccess) return e;
        e = launch_prefix_tc(a, pl, map, D, pdl, s);
        if (e != cudaSuccess) return e;
        pdl = true;
    }
    if (!pl.tc_own) {  // the own parts are always there
        e = pool_map(&map, c, D, a.type, XKEYS);
        if (e != cudaSuccess) return e;
        const long long grid = (pl.tc_shared ? 0 : pblocks * pl.np) + sblocks * pl.ns;
        if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        if (D == 128)
            e = bf ? launch_kw<128, true>(kw, a, pl, map, (unsigned)grid, pdl, s)
                   : launch_kw<128, false>(kw, a, pl, map, (unsigned)grid, pdl, s);
        else
            e = bf ? launch_kw<64, true>(kw, a, pl, map, (unsigned)grid, pdl, s)
                   : launch_kw<64, false>(kw, a, pl, map, (unsigned)grid, pdl, s);
        if (e != cudaSuccess) return e;
    }
    return D == 128 ? launch_merge<128>(a, pl, sms, s) : launch_merge<64>(a, pl, sms, s);
}

}  // namespace hq
