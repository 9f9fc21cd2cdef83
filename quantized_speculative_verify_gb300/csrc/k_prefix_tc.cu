// k_prefix_tc.cu -- the prefix attention on the fifth-generation tensor cores
// (tcgen05): the shared parts of batches with many rows (k_prefix_tc), and the
// own parts of sequences with many rows, draft trees (k_prefix_own).
//
// Over the shared positions the batch is one dense attention without a mask:
// all rows that read one key/value head (rows * G of them) against the prefix.
// With enough rows it is bound by the tensor cores, not by memory, and the
// warp-level MMAs of k_prefix.cu reach a tenth of their rate (170 TFLOP/s).
// k_prefix_tc: 512 rows a head (G = 4) on 32768 positions of 8 heads, 96 blocks
// in 72 us, 954 TFLOP/s or 77% of what 96 SMs can; 48 trees' 2204 rows a head on
// 12288 positions, 144 blocks in 80 us, 1.39 PFLOP/s or 75%.
//
// A thread block works on two streams at once, each with its own 128 columns
// of scores and its output accumulator in tensor memory (2 x (128 + 128)
// columns: all 512):
//   S = Q K^T        both operands in shared memory
//   P = exp2(c S - c m), in fp16 times 2^7, rounded to the cache's type, written
//   over S
//   O += P V         P from tensor memory, V from shared memory
// While one stream is in its softmax the tensor core works for the other.
// PAIR: the streams are two 128-row query tiles against the same positions.
// Otherwise (at most 128 rows) they are one query tile against
// alternating tiles of positions, added up at the end through shared memory.
//   warps 0-3, 4-7  softmax of stream 0, 1: a thread owns one row, so maximum
//                   and sum need no exchange between lanes
//   warp 8          K and V tiles by TMA into a ring of four slots
//   warp 9          issues the MMAs; warps 10, 11 only fill the warpgroup
//                   whose registers go to the softmax
// The reference maximum m of a row is raised only when a score exceeds it by
// 8 or more in base-2 units: then O is scaled by the softmax warps themselves,
// between two products; P stays below 2^8 (2^15 in fp16), and output and sum are
// relative to the same m.
//
// The wait for S(j + 1) also orders the scaling of O behind P V(j): MMAs of
// one thread complete in order, and P V(j) is issued before S(j + 1).
//
// Own parts end with the sequence's draft tree: a row's visible positions of a
// tile are 128 bits.  A masked position weighs 0, but 0 times an infinity or
// NaN is NaN: in a masked tile the softmax warps set the non-finite values of
// V from the tree on to 0 in shared memory before the product may read it, and
// the rows that see such a value add it at the end from the cache itself.
#include <type_traits>

#include "hq_tc.cuh"
#include "prefix_common.cuh"

namespace hq {
namespace {

constexpr int CR = 128;       // rows of a query tile, positions of a K/V tile
constexpr int CSLOTS = 4;     // ring slots, each one K or one V tile
constexpr int CTHREADS = 384;
// Registers: three warpgroups start with the 168 that 384 threads allow; the
// third gives up 96 a thread, the softmax warpgroups take 48 each (2 * 216 +
// 72 = 3 * 168): a row's 128 scores then stay in registers.
constexpr int CREG_SOFTMAX = 216, CREG_REST = 72;
constexpr float LAZY = 8.0f;  // base-2 units a score may exceed the reference maximum by
// P is 2^7 at the reference maximum in fp16, so that at most 2^15 may occur and the
// 21 powers below the maximum are normal values (k_prefix.cu: P_SHIFT_F16).
template <bool BF>
constexpr float P_SHIFT = BF ? 0.0f : 7.0f;

template <int D>
struct TcTile {
    static constexpr int BOX = CR * 128;          // 128 rows x 64 dimensions
    static constexpr int BYTES = (D / 64) * BOX;
    static constexpr size_t SMEM = 1024 + (size_t)(2 + CSLOTS) * BYTES + 256;
};

// D[128 x N] (+)= A[128 x 16] * B[16 x N], A and B in shared memory, fp32 D;
// issued by the lane with `leader` set, executed by the converged warp (the
// operands stay warp-uniform: one lane in a branch of its own took 3600 cycles
// for the 32 MMAs of two tiles that the tensor core needs 2048 for).
__device__ __forceinline__ void tc_mma_ss_if(uint32_t leader, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: 8 x 128-byte atoms,
// `sbo` bytes between the atoms of consecutive groups of 8 rows (K-major: rows
// of the operand; MN-major: steps along K), `lbo` between blocks of 64
// elements along MN (MN-major only).
__device__ __forceinline__ uint64_t desc_swz128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: 128 x N, fp32 D, A and B fp16 or bf16; B K-major
// (scores) or MN-major (V as it lies in the cache).
template <bool BF>
__host__ __device__ constexpr uint32_t idesc_of(int N, bool b_mn) {
    return (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((128u >> 4) << 24);
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
    return d;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The low n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Sets the infinities and NaN of a pair to 0; whether there was one.
template <bool BF>
__device__ __forceinline__ bool clear_nonfinite(uint32_t &x) {
    constexpr uint32_t e = BF ? 0x7f80u : 0x7c00u;
    const bool lo = (x & e) == e, hi = ((x >> 16) & e) == e;
    if (lo) x &= 0xffff0000u;
    if (hi) x &= 0x0000ffffu;
    return lo || hi;
}

template <int D, bool BF, bool PAIR>
__global__ void __launch_bounds__(CTHREADS, 1)
    k_prefix_tc(const PrefixArgs a, const PrefixPlan pl, const __grid_constant__ CUtensorMap map) {
    using T = TcTile<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *s_q = sm, *s_ring = sm + 2 * T::BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_ring + CSLOTS * T::BYTES);
    const uint32_t full = smem_addr(bars), empty = full + 8 * CSLOTS, sfull = empty + 8 * CSLOTS, phalf = sfull + 16,
                   pready = phalf + 16, ofull = pready + 16, qready = ofull + 16;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 2 * CSLOTS + 9);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < CSLOTS; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(sfull + 8 * w, 1);
            mbar_init(phalf + 8 * w, 4);
            mbar_init(pready + 8 * w, 4);
            mbar_init(ofull + 8 * w, 1);
        }
        mbar_init(qready, 8);
        fence_mbar_init();
    }
    pdl_wait();
    // (columns are taken after the wait: a kernel before this one may want them)
    if (warp == 9) tmem_alloc(smem_addr(s_tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_launch_dependents();

    // which part this block is
    int unit = blockIdx.x;
    const int hk = unit % a.Hkv;
    unit /= a.Hkv;
    constexpr bool pair = PAIR;
    const int part = unit / pl.ptiles, row0 = (unit % pl.ptiles) * (pair ? 2 * CR : CR), nrows = a.rows * a.G;
    const int k0 = part * pl.pchunk, k1 = k0 + pl.pchunk < pl.s0 ? k0 + pl.pchunk : pl.s0;
    const Seq seq = first_live(a);
    const int ntiles = seq.live ? (k1 - k0) / CR : 0;  // no live sequence: no row uses this part

    if (warp < 8) {
        // ------------------------------------------------------- softmax ---
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CREG_SOFTMAX));
        if (ntiles > 0) {
            const int w = warp >> 2, r = threadIdx.x & 127;  // stream, row of its tile
            const int row = row0 + (pair ? w * CR : 0) + r;  // row among the part's
            const size_t at = ((size_t)part * a.rows + row / a.G) * a.Hq + hk * a.G + row % a.G;
            const int n = pair ? ntiles : (ntiles - w + 1) / 2;
            bool ok = true;
            // the query rows, swizzled as the tensor core reads them
            if (pair || w == 0) {
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    static_cast<const uint16_t *>(a.q) +
                    (row < nrows ? (size_t)(row / a.G) * a.ldq + (size_t)(hk * a.G + row % a.G) * D : 0));
                uint8_t *dst = s_q + w * T::BYTES;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * T::BOX + swz128(r, c & 7)) =
                        row < nrows ? src[c] : make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(qready);
            const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 lanes
            const uint32_t tS = lane_base + w * 128, tO = lane_base + 256 + w * 128;
            const float c = a.c_log2;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                if (ok) ok = mbar_wait_short(sfull + 8 * w, (uint32_t)(j & 1), a.err);
                __syncwarp();
                tc_fence_after();
                float s[128];
                // each quarter's maximum is taken while the next one is on its way
                tmem_ld32(tS, s);
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_wait_ld();
                    if (q < 3) tmem_ld32(tS + 32 * (q + 1), s + 32 * (q + 1));
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        mx[0] = max3(mx[0], s[32 * q + i], s[32 * q + i + 1]);
                        mx[1] = max3(mx[1], s[32 * q + i + 2], s[32 * q + i + 3]);
                    }
                }
                const float top = fmaxf(mx[0], mx[1]);
                if (j == 0) {
                    m = top;
                } else {
                    const bool raise = (top - m) * c > LAZY;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = raise ? top : m;
                        const float al = raise ? ex2((m - mn) * c) : 1.0f;
                        m = mn;
                        l *= al;
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            float o[32];
                            uint32_t u[32];
                            tmem_ld32(tO + 32 * i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * al);
                            tmem_st32(tO + 32 * i, u);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.0f : m * c - P_SHIFT<BF>;
                const f2 cc = f2_make(c, c), mm = f2_make(-mc, -mc);
                f2 sum[2] = {f2_make(0.0f, 0.0f), f2_make(0.0f, 0.0f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float x, y;
                        f2_split(f2_fma(f2_make(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]), cc, mm), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sum[i & 1] = f2_add(sum[i & 1], f2_make(x, y));
                        p[i] = pack16<BF>(x, y);
                    }
                    tmem_st32(tS + 32 * h, p);
                    if (h == 0) {  // the product may start on the first half
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(phalf + 8 * w);
                    }
                }
                float x0, x1, x2, x3;
                f2_split(sum[0], x0, x1);
                f2_split(sum[1], x2, x3);
                l += (x0 + x1) + (x2 + x3);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready + 8 * w);
            }
            // a stream's O is complete with its last product; both streams' where
            // they are added up, through the ring that nothing reads any more
            for (int x = 0; x < 2; ++x)
                if (pair ? x == w : x < ntiles) {
                    if (ok) ok = mbar_wait_short(ofull + 8 * x, 0u, a.err);
                    __syncwarp();
                }
            tc_fence_after();
            if (l == 0.0f) m = -INFINITY;  // no tile, or no finite score: adds nothing
            float mb = m == -INFINITY ? -INFINITY : m * c - P_SHIFT<BF>;  // in base-2 units
            float scale = 1.0f, other = 0.0f;
            float *box = reinterpret_cast<float *>(s_ring);  // [D][128 rows], then m, l
            // O of this thread's row, dimensions 32 i .. 32 i + 31
            auto load_o = [&](int i, float (&o)[32]) {
                if (n > 0) {
                    tmem_ld32(tO + 32 * i, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                }
            };
            if (!pair) {
                if (w == 1) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float o[32];
                        load_o(i, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) box[(32 * i + e) * CR + r] = o[e];
                    }
                    box[D * CR + r] = mb;
                    box[(D + 1) * CR + r] = l;
                }
                named_barrier(1, 256);
                if (w == 0) {
                    const float mo = box[D * CR + r], lo = box[(D + 1) * CR + r];
                    const float top = fmaxf(mb, mo), t = top == -INFINITY ? 0.0f : top;
                    scale = ex2(mb - t);
                    other = ex2(mo - t);
                    l = scale * l + other * lo;
                    mb = top;
                }
            }
            if (pair || w == 0) {
                float4 *dst = reinterpret_cast<float4 *>(a.ws_o + at * D);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float o[32];
                    load_o(i, o);
                    if (row < nrows) {
                        if (!pair)
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = scale * o[e] + other * box[(32 * i + e) * CR + r];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[8 * i + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                    __syncwarp();
                }
                if (row < nrows) *reinterpret_cast<float2 *>(a.ws_ml + at * 2) = make_float2(mb, l);
            }
            tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CREG_REST));
    }
    if (warp == 8) {
        // ---------------------------------------------------------- K, V ---
        // the order in which the MMAs use them: pair K0 V0 K1 V1 ...; else
        // K0 K1 V0 K2 V1 K3 ...
        const int32_t *row = a.table + (size_t)(ntiles > 0 ? seq.slot : 0) * a.max_pages;
        int i = 0;
        bool ok = true;
        auto put = [&](int tile, int plane) {
            const int p = k0 + tile * CR, st = i % CSLOTS;
            const int page = lookup_page<CR>(a, row, p, k1);
            if (ok && i >= CSLOTS)
                ok = mbar_wait_short(empty + 8 * st, (uint32_t)((i / CSLOTS) & 1) ^ 1u, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            if (lane == 0) mbar_arrive_expect_tx(full + 8 * st, (uint32_t)T::BYTES);
            __syncwarp();
            load_tile<CR, D>(a, &map, smem_addr(s_ring + st * T::BYTES), p, hk, plane, page, full + 8 * st);
            __syncwarp();
            ++i;
        };
        if constexpr (pair) {
            for (int t = 0; t < ntiles; ++t) {
                put(t, a.k_plane);
                put(t, a.v_plane);
            }
        } else if (ntiles > 0) {
            put(0, a.k_plane);
            if (ntiles > 1) put(1, a.k_plane);
            for (int t = 0; t < ntiles; ++t) {
                put(t, a.v_plane);
                if (t + 2 < ntiles) put(t + 2, a.k_plane);
            }
        }
        // no copy may still be landing in shared memory when the block exits
        for (int j = i > CSLOTS ? i - CSLOTS : 0; j < i; ++j)
            mbar_wait_short(full + 8 * (j % CSLOTS), (uint32_t)((j / CSLOTS) & 1), a.err);
    } else if (warp == 9 && ntiles > 0) {
        // ---------------------------------------------------------- MMAs ---
        const uint32_t leader = elect_one() ? 1u : 0u;
        const uint64_t dq = desc_swz128(smem_addr(s_q), 16, 1024), dk = desc_swz128(smem_addr(s_ring), 16, 1024);
        const uint64_t dv = desc_swz128(smem_addr(s_ring), T::BOX, 1024);  // addresses count in 16 bytes, below bit 14
        constexpr uint32_t id_s = idesc_of<BF>(CR, false), id_o = idesc_of<BF>(D, true);
        bool ok = mbar_wait_short(qready, 0u, a.err);
        int use = 0;  // ring uses so far
        auto next = [&]() -> int {  // the slot of the next K or V tile, arrived
            const int st = use % CSLOTS;
            if (ok) ok = mbar_wait_short(full + 8 * st, (uint32_t)((use / CSLOTS) & 1), a.err);
            __syncwarp();
            ++use;
            return st;
        };
        auto scores = [&](int w, int st) {  // S_w = Q K^T
            const uint64_t q = dq + (uint64_t)((pair ? w : 0) * (T::BYTES / 16)), k = dk + (uint64_t)(st * (T::BYTES / 16));
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t o = (uint64_t)((ks >> 2) * (T::BOX / 16) + (ks & 3) * 2);
                tc_mma_ss_if(leader, tmem + w * 128, q + o, k + o, id_s, ks > 0);
            }
            tc_commit_if(leader, sfull + 8 * w);
        };
        auto product = [&](int w, int st, int j) {  // O_w += P_w V
            const uint64_t v = dv + (uint64_t)(st * (T::BYTES / 16));
#pragma unroll
            for (int ks = 0; ks < CR / 16; ++ks) {
                if (ks == 0 || ks == CR / 32) {
                    if (ok) ok = mbar_wait_short((ks ? pready : phalf) + 8 * w, (uint32_t)(j & 1), a.err);
                    __syncwarp();
                    tc_fence_after();
                }
                tc_mma_f16_ts_if(leader, tmem + 256 + w * 128, tmem + w * 128 + ks * 8, v + (uint64_t)(ks * 128), id_o,
                                 j > 0 || ks > 0);
            }
        };
        if constexpr (pair) {
            int kst = next();
            scores(0, kst);
            scores(1, kst);
            tc_commit_if(leader, empty + 8 * kst);
            for (int j = 0; j < ntiles; ++j) {
                const bool more = j + 1 < ntiles;
                const int vst = next();
                product(0, vst, j);
                if (more) {
                    kst = next();
                    scores(0, kst);
                } else {
                    tc_commit_if(leader, ofull);
                }
                product(1, vst, j);
                tc_commit_if(leader, empty + 8 * vst);
                if (more) {
                    scores(1, kst);
                    tc_commit_if(leader, empty + 8 * kst);
                } else {
                    tc_commit_if(leader, ofull + 8);
                }
            }
        } else {
            for (int w = 0; w < 2 && w < ntiles; ++w) {
                const int st = next();
                scores(w, st);
                tc_commit_if(leader, empty + 8 * st);
            }
            for (int t = 0; t < ntiles; ++t) {
                const int w = t & 1, vst = next();
                product(w, vst, t >> 1);
                tc_commit_if(leader, empty + 8 * vst);
                if (t + 2 < ntiles) {
                    const int st = next();
                    scores(w, st);
                    tc_commit_if(leader, empty + 8 * st);
                } else {
                    tc_commit_if(leader, ofull + 8 * w);
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// The own parts of draft trees: one query tile (at most 128 rows of a sequence)
// against its own positions, few tiles of them, so what counts is how fast a
// part starts and ends.  Two thread blocks an SM (half the tensor memory, a K
// and a V tile, 192 threads each) hide that in one another; there is one stream
// of tiles, whose scores are read twice from tensor memory instead of being
// held in registers, and warps whose 32 rows are all past the tile's end leave
// out the softmax.  48 trees of 64 rows a head on up to 700 + 16 positions: 32
// us alone (the kernel above with one tile against alternating positions, one
// block an SM: 41; the warp-level MMAs 7 more), about 20 of them beside and behind
// the shared parts.  Shorter parts, two or three a sequence, cost more in
// partial results than they gain: 119 us instead of 113 for the whole call.
//   warps 0-3 softmax, warp 4 K and V tiles, warp 5 the MMAs
constexpr int OTHREADS = 192;
constexpr size_t OSMEM = 1024 + 3 * (size_t)TcTile<128>::BYTES + 128 + HQ_MAX_M * 4;  // D = 64: as much, two blocks an SM

template <int D, bool BF>
__global__ void __launch_bounds__(OTHREADS, 2)
    k_prefix_own(const PrefixArgs a, const PrefixPlan pl, const __grid_constant__ CUtensorMap map) {
    using T = TcTile<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *s_q = sm, *s_k = sm + T::BYTES, *s_v = sm + 2 * T::BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + 3 * T::BYTES);
    const uint32_t kfull = smem_addr(bars), kempty = kfull + 8, vfull = kfull + 16, vempty = kfull + 24, sfull = kfull + 32,
                   phalf = kfull + 40, pready = kfull + 48, ofull = kfull + 56, qready = kfull + 64;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(bars + 9);
    volatile int *s_odd = reinterpret_cast<int *>(s_tmem + 1);  // values of V have been set to 0
    int32_t *s_par = reinterpret_cast<int32_t *>(s_tmem + 2);   // [HQ_MAX_M]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 9; ++i) mbar_init(kfull + 8 * i, i == 5 || i == 6 || i == 8 ? 4 : 1);
        *s_odd = 0;
        fence_mbar_init();
    }
    // Behind shared parts nothing is waited for: each of their blocks has itself
    // waited for the call's inputs, and taken its tensor memory, before these
    // may start, and the SMs that they leave idle, or are done with, begin here
    // at once.  Only this grid's end, which the merge waits for, must not come
    // before theirs (see the end).
    const bool behind = pl.tc_shared;
    if (!behind) pdl_wait();
    if (warp == 5) tmem_alloc(smem_addr(s_tmem), 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;  // 128 columns of scores, then O
    pdl_launch_dependents();

    // which part this block is; nothing to do (ntiles 0) where no row uses it
    int unit = blockIdx.x;
    const int hk = unit % a.Hkv;
    unit /= a.Hkv;
    const int b = unit / (pl.ns * pl.stiles);
    unit %= pl.ns * pl.stiles;
    const int part = unit / pl.stiles, row0 = (unit % pl.stiles) * CR;
    const int k0 = pl.s0 + part * pl.schunk;
    int early = -1;  // the table entries of the first tile
    if (warp == 4) early = early_entry<CR>(a, b, k0);
    const Seq seq = seq_of(a, b);
    const int first = seq.first, nodes = seq.m, nrows = seq.m * a.G, slot = seq.slot, tree0 = seq.len - seq.m;
    const int k1 = seq.len - k0 > pl.schunk ? k0 + pl.schunk : seq.len;
    const int ntiles = seq.live && row0 < nrows && k0 < k1 ? (k1 - k0 + CR - 1) / CR : 0;

    if (warp < 4 && ntiles > 0) {
        // ------------------------------------------------------- softmax ---
        const int r = threadIdx.x, row = row0 + r;  // row of the tile, among the sequence's
        const bool idle = row0 + warp * 32 >= nrows;
        bool ok = true;
        {
            // the query rows, swizzled as the tensor core reads them
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(a.q) +
                (row < nrows ? (size_t)(first + row / a.G) * a.ldq + (size_t)(hk * a.G + row % a.G) * D : 0));
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<uint4 *>(s_q + (c >> 3) * T::BOX + swz128(r, c & 7)) =
                    row < nrows ? src[c] : make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(qready);
        // the tree nodes this row sees (without `parent`: a chain)
        uint32_t anc[4] = {0u, 0u, 0u, 0u};
        if (k1 > tree0) {
            if (a.parent) {
                for (int i = r; i < nodes; i += 128) s_par[i] = a.parent[first + i];
                named_barrier(1, 128);
            }
            if (row < nrows) {
                int cur = row / a.G;
                for (int step = 0; step < HQ_MAX_M; ++step) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (cur >> 5 == i) anc[i] |= 1u << (cur & 31);
                    const int p = cur == 0 ? -1 : a.parent ? s_par[cur] : cur - 1;
                    if (p < 0 || p >= cur) break;
                    cur = p;
                }
            }
            __syncwarp();
        }
        const uint32_t tS = tmem + ((uint32_t)warp << 21), tO = tS + 128;  // this warp's 32 lanes
        const float c = a.c_log2;
        float m = -INFINITY, l = 0.0f;
        // masked tiles are a code of their own: the masks slow the common one down
        auto step = [&](auto masked, int j) {
            constexpr bool MASKED = decltype(masked)::value;
            const int p0 = k0 + j * CR;
            if (ok) ok = mbar_wait_short(sfull, (uint32_t)(j & 1), a.err);
            __syncwarp();
            tc_fence_after();
            uint32_t sees[4];
            if constexpr (MASKED) {
                // bit i: position p0 + i is before the tree, or a node this row
                // sees; and inside the part
                const int old = tree0 - p0, in = k1 - p0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v = bits_below(old - 32 * i);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {  // word x of the nodes starts at bit old + 32 x
                        const int sh = old + 32 * (x - i);
                        if (sh >= 0 && sh < 32) v |= anc[x] << sh;
                        if (sh < 0 && sh > -32) v |= anc[x] >> -sh;
                    }
                    sees[i] = v & bits_below(in - 32 * i);
                }
            }
            auto scores = [&](int q, float (&s)[32]) {
                tmem_ld32(tS + 32 * q, s);
                tmem_wait_ld();
                if constexpr (MASKED)
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[i] = (sees[q] >> i) & 1u ? s[i] : -INFINITY;
            };
            if (!idle) {
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float s[32];
                    scores(q, s);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        mx[0] = max3(mx[0], s[i], s[i + 1]);
                        mx[1] = max3(mx[1], s[i + 2], s[i + 3]);
                    }
                }
                const float top = fmaxf(mx[0], mx[1]);
                if (j == 0) {
                    m = top;
                } else {
                    const bool raise = (top - m) * c > LAZY;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float mn = raise ? top : m;
                        const float al = raise ? ex2((m - mn) * c) : 1.0f;
                        m = mn;
                        l *= al;
#pragma unroll
                        for (int i = 0; i < D / 32; ++i) {
                            float o[32];
                            uint32_t u[32];
                            tmem_ld32(tO + 32 * i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * al);
                            tmem_st32(tO + 32 * i, u);
                        }
                    }
                }
            }
            if constexpr (MASKED) {
                // V from the tree on: finite, or set to 0 (see above)
                if (ok) ok = mbar_wait_short(vfull, (uint32_t)(j & 1), a.err);
                __syncwarp();
                const int lo = tree0 > p0 ? tree0 - p0 : 0;
                bool odd = false;
                for (int i = lo * (D / 8) + r; i < CR * (D / 8); i += CR) {
                    const int vr = i / (D / 8), ch = i % (D / 8);
                    uint4 *x = reinterpret_cast<uint4 *>(s_v + (ch >> 3) * T::BOX + swz128(vr, ch & 7));
                    uint4 u = *x;
                    if (clear_nonfinite<BF>(u.x) | clear_nonfinite<BF>(u.y) | clear_nonfinite<BF>(u.z) |
                        clear_nonfinite<BF>(u.w)) {
                        *x = u;
                        odd = true;
                    }
                }
                if (odd) {
                    *s_odd = 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
            }
            const float mc = m == -INFINITY ? 0.0f : m * c - P_SHIFT<BF>;
            const f2 cc = f2_make(c, c), mm = f2_make(-mc, -mc);
            f2 sum[2] = {f2_make(0.0f, 0.0f), f2_make(0.0f, 0.0f)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!idle) {
                    uint32_t p[32];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float s[32];
                        scores(2 * h + q, s);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x, y;
                            f2_split(f2_fma(f2_make(s[2 * i], s[2 * i + 1]), cc, mm), x, y);
                            x = ex2(x);
                            y = ex2(y);
                            sum[i & 1] = f2_add(sum[i & 1], f2_make(x, y));
                            p[16 * q + i] = pack16<BF>(x, y);
                        }
                    }
                    tmem_st32(tS + 32 * h, p);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(h ? pready : phalf);  // the product may start on the first half
            }
            float x0, x1, x2, x3;
            f2_split(sum[0], x0, x1);
            f2_split(sum[1], x2, x3);
            l += (x0 + x1) + (x2 + x3);
        };
        for (int j = 0; j < ntiles; ++j) {
            const int p0 = k0 + j * CR;
            if (p0 + CR <= tree0 && p0 + CR <= k1)
                step(std::false_type{}, j);
            else
                step(std::true_type{}, j);
        }
        if (ok) ok = mbar_wait_short(ofull, 0u, a.err);
        __syncwarp();
        tc_fence_after();
        if (k1 > tree0) named_barrier(1, 128);
        const bool odd = k1 > tree0 && *s_odd != 0;
        if (l == 0.0f) m = -INFINITY;  // no finite score: adds nothing
        if (!idle) {
            const size_t at = ((size_t)(pl.np + part) * a.rows + first + row / a.G) * a.Hq + hk * a.G + row % a.G;
            float4 *dst = reinterpret_cast<float4 *>(a.ws_o + at * D);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                float o[32];
                tmem_ld32(tO + 32 * i, o);
                tmem_wait_ld();
                if (odd) {  // what the masked tiles' non-finite values add to the rows that see them
                    for (int t = 0; t < nodes; ++t) {
                        const int p = tree0 + t;
                        uint32_t word = 0;
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (t >> 5 == x) word = anc[x];
                        if (!((word >> (t & 31)) & 1u) || p < k0 || p >= k1) continue;
                        const int page = a.table[(size_t)slot * a.max_pages + (p >> a.page_shift)];
                        if (page < 0 || page >= a.n_pages) continue;
                        const int ps = 1 << a.page_shift;
                        const uint16_t *v = reinterpret_cast<const uint16_t *>(
                                                a.pool + (size_t)a.v_plane * (size_t)a.plane_bytes +
                                                (((size_t)page * a.Hkv + hk) * ps + (p & (ps - 1))) * (size_t)(2 * D)) +
                                            32 * i;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            uint32_t one = v[e];
                            const float f = BF ? __uint_as_float(one << 16) : __half2float(__ushort_as_half((unsigned short)one));
                            if (clear_nonfinite<BF>(one)) o[e] += f;
                        }
                    }
                    __syncwarp();
                }
                if (row < nrows)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[8 * i + e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                __syncwarp();
            }
            if (row < nrows)
                *reinterpret_cast<float2 *>(a.ws_ml + at * 2) = make_float2(m == -INFINITY ? -INFINITY : m * c - P_SHIFT<BF>, l);
        }
        tc_fence_before();
    } else if (warp == 4) {
        // ---------------------------------------------------------- K, V ---
        const int32_t *row = a.table + (size_t)(ntiles > 0 ? slot : 0) * a.max_pages;
        bool ok = true;
        int nk = 0, nv = 0;
        auto put = [&](int tile, int plane, uint8_t *dst, uint32_t fb, uint32_t eb, int &n) {
            const int p = k0 + tile * CR;
            const int page = tile == 0 ? checked_page<CR>(a, early, p, k1) : lookup_page<CR>(a, row, p, k1);
            if (ok && tile > 0) ok = mbar_wait_short(eb, (uint32_t)(tile & 1) ^ 1u, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)T::BYTES);
            __syncwarp();
            load_tile<CR, D>(a, &map, smem_addr(dst), p, hk, plane, page, fb);
            __syncwarp();
            ++n;
        };
        for (int t = 0; t < ntiles; ++t) {
            put(t, a.k_plane, s_k, kfull, kempty, nk);
            put(t, a.v_plane, s_v, vfull, vempty, nv);
        }
        // no copy may still be landing in shared memory when the block exits
        if (nk > 0) mbar_wait_short(kfull, (uint32_t)((nk - 1) & 1), a.err);
        if (nv > 0) mbar_wait_short(vfull, (uint32_t)((nv - 1) & 1), a.err);
    } else if (warp == 5 && ntiles > 0) {
        // ---------------------------------------------------------- MMAs ---
        const uint32_t leader = elect_one() ? 1u : 0u;
        const uint64_t dq = desc_swz128(smem_addr(s_q), 16, 1024), dk = desc_swz128(smem_addr(s_k), 16, 1024);
        const uint64_t dv = desc_swz128(smem_addr(s_v), T::BOX, 1024);
        constexpr uint32_t id_s = idesc_of<BF>(CR, false), id_o = idesc_of<BF>(D, true);
        bool ok = mbar_wait_short(qready, 0u, a.err);
        for (int j = 0; j < ntiles; ++j) {
            // S = Q K^T.  (The products of the tile before, which read P where S
            // goes, were issued first and complete first.)
            if (ok) ok = mbar_wait_short(kfull, (uint32_t)(j & 1), a.err);
            __syncwarp();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint64_t o = (uint64_t)((ks >> 2) * (T::BOX / 16) + (ks & 3) * 2);
                tc_mma_ss_if(leader, tmem, dq + o, dk + o, id_s, ks > 0);
            }
            tc_commit_if(leader, sfull);
            tc_commit_if(leader, kempty);
            // O += P V
            if (ok) ok = mbar_wait_short(vfull, (uint32_t)(j & 1), a.err);
#pragma unroll
            for (int ks = 0; ks < CR / 16; ++ks) {
                if (ks == 0 || ks == CR / 32) {
                    if (ok) ok = mbar_wait_short(ks ? pready : phalf, (uint32_t)(j & 1), a.err);
                    __syncwarp();
                    tc_fence_after();
                }
                tc_mma_f16_ts_if(leader, tmem + 128, tmem + ks * 8, dv + (uint64_t)(ks * 128), id_o, j > 0 || ks > 0);
            }
            tc_commit_if(leader, vempty);
        }
        tc_commit_if(leader, ofull);
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, 256);
    if (behind && blockIdx.x == gridDim.x - 1) pdl_wait();
}

template <class F>
cudaError_t launch_part(F f, std::atomic<int> (&configured)[CACHE_DEVICES], long long grid, int threads, size_t smem, const PrefixArgs &a,
                        const PrefixPlan &pl, const CUtensorMap &map, bool pdl, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int done = 0;
    e = cached_per_device(configured, dev, &done, [&](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_kernel(f, dim3((unsigned)grid), dim3(threads), smem, pdl, s, a, pl, map);
}

template <int D, bool BF>
cudaError_t launch_parts(const PrefixArgs &a, const PrefixPlan &pl, const CUtensorMap &map, bool pdl, cudaStream_t s) {
    static std::atomic<int> pair[CACHE_DEVICES], single[CACHE_DEVICES], own[CACHE_DEVICES];
    if (pl.tc_shared) {
        const long long grid = (long long)a.Hkv * pl.np * pl.ptiles;
        const cudaError_t e =
            (long long)a.rows * a.G > CR
                ? launch_part(k_prefix_tc<D, BF, true>, pair, grid, CTHREADS, TcTile<D>::SMEM, a, pl, map, pdl, s)
                : launch_part(k_prefix_tc<D, BF, false>, single, grid, CTHREADS, TcTile<D>::SMEM, a, pl, map, pdl, s);
        if (e != cudaSuccess) return e;
        pdl = true;
    }
    if (!pl.tc_own) return cudaSuccess;
    return launch_part(k_prefix_own<D, BF>, own, (long long)a.Hkv * a.B * pl.ns * pl.stiles, OTHREADS, OSMEM, a, pl, map, pdl, s);
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixArgs &a, const PrefixPlan &pl, const CUtensorMap &map, int D, bool pdl,
                             cudaStream_t s) {
    const bool bf = a.type == HQ_BF16;
    if (D == 128) return bf ? launch_parts<128, true>(a, pl, map, pdl, s) : launch_parts<128, false>(a, pl, map, pdl, s);
    return bf ? launch_parts<64, true>(a, pl, map, pdl, s) : launch_parts<64, false>(a, pl, map, pdl, s);
}

}  // namespace hq
