// prefix_common.cuh -- what the kernels of the shared-prefix attention share:
// how a call is cut into parts, the sequences of a batch, TMA copies of pages.
#pragma once

#include <cuda.h>

#include "batch.cuh"

namespace hq {

constexpr int DEV_ERR_ARG = 2;  // error word: a bad table entry or length

struct PrefixPlan {
    int s0;             // shared positions taken by the shared parts (a multiple of the tile)
    int np, pchunk;     // shared parts of a row, positions each
    int ns, schunk;     // own parts of a row, positions each
    int ptiles, stiles; // row tiles: all rows, one sequence's rows
    int tc_shared, tc_own;  // which kind the tensor-memory kernel takes
};

// Tiled copy (dimension, row in page, head, page, plane) into shared memory.
// x is 0 or 64 elements of 2 bytes: a multiple of 16 bytes.
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, int x, int y, int head, int page,
                                         int plane, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(head), "r"(page), "r"(plane), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t swz128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// 2^x by the hardware's unit (2 ulp; results below the normal range are 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sequence of the batch: its slot, rows, length; `live` false where it is
// empty or its length contradicts the call.
struct Seq {
    int slot, first, m, len;
    bool live;
};
__device__ __forceinline__ Seq seq_of(const PrefixArgs &a, int b) {
    Seq s;
    batch_rows(a.starts, b, a.rows, a.max_rows, s.first, s.m);
    s.slot = a.seqs ? a.seqs[b] : b;
    s.len = s.slot >= 0 && s.slot < a.n_seqs ? a.len[s.slot] : -1;
    s.live = s.m > 0 && s.len <= a.max_len && s.len - s.m >= a.shared;
    if (!s.live && s.m > 0 && s.len != 0) atomicExch(a.err, DEV_ERR_ARG);
    return s;
}

// The first live sequence of the batch, through which the shared positions
// are read; live == false if there is none.
__device__ __forceinline__ Seq first_live(const PrefixArgs &a) {
    Seq s = seq_of(a, 0);
    for (int b = 1; !s.live && b < a.B; ++b) s = seq_of(a, b);
    return s;
}

// A warp loads one tile of TILE positions from p0 on of K or V (`plane`) of
// head hk into `dst` (boxes of 64 dimensions, TILE * 128 bytes each): lane j
// looks up and loads the j-th run of positions that lie in one page.  `row` is
// the sequence's table; runs that start at or past `end` and bad pages arrive
// as zeros.  `page` is the lane's page as lookup_page returned it.
template <int TILE>
__device__ __forceinline__ int page_entry(const PrefixArgs &a, const int32_t *row, int p0, int end) {
    const int lane = threadIdx.x & 31;
    constexpr int SHIFT = TILE == 128 ? 7 : 6;
    const int sh = a.page_shift < SHIFT ? a.page_shift : SHIFT;
    const int p = p0 + (lane << sh);
    return lane < (TILE >> sh) && p < end ? row[p >> a.page_shift] : a.n_pages;
}
template <int TILE>
__device__ __forceinline__ int checked_page(const PrefixArgs &a, int page, int p0, int end) {
    const int lane = threadIdx.x & 31;
    constexpr int SHIFT = TILE == 128 ? 7 : 6;
    const int sh = a.page_shift < SHIFT ? a.page_shift : SHIFT;
    if (lane >= (TILE >> sh) || p0 + (lane << sh) >= end) return a.n_pages;  // outside the map: zeros
    if (page < 0 || page >= a.n_pages) {
        atomicExch(a.err, DEV_ERR_ARG);
        return a.n_pages;
    }
    return page;
}
template <int TILE>
__device__ __forceinline__ int lookup_page(const PrefixArgs &a, const int32_t *row, int p0, int end) {
    return checked_page<TILE>(a, page_entry<TILE>(a, row, p0, end), p0, end);
}
// The table entries of the first tile of a sequence's part, on their way beside
// its length (which tells where they end) instead of after it.
template <int TILE>
__device__ __forceinline__ int early_entry(const PrefixArgs &a, int b, int p0) {
    const int slot = a.seqs ? a.seqs[b] : b;
    if (slot < 0 || slot >= a.n_seqs) return a.n_pages;
    return page_entry<TILE>(a, a.table + (size_t)slot * a.max_pages, p0, a.max_pages << a.page_shift);
}
template <int TILE, int D>
__device__ __forceinline__ void load_tile(const PrefixArgs &a, const CUtensorMap *map, uint32_t dst, int p0, int hk,
                                          int plane, int page, uint32_t bar) {
    const int lane = threadIdx.x & 31;
    constexpr int SHIFT = TILE == 128 ? 7 : 6;
    const int sh = a.page_shift < SHIFT ? a.page_shift : SHIFT;
    if (lane >= (TILE >> sh)) return;
    const int y = (p0 + (lane << sh)) & ((1 << a.page_shift) - 1);
    const uint32_t at = dst + (uint32_t)(lane << sh) * 128u;
#pragma unroll
    for (int bx = 0; bx < D / 64; ++bx) tma_page(at + bx * TILE * 128, map, bx * 64, y, hk, page, plane, bar);
}

// mbar_wait_bounded for waits that are short and frequent: the clock is read
// only after the hardware's own waiting (up to a millisecond each) gave up.
__device__ __forceinline__ bool mbar_wait_short(uint32_t bar, uint32_t parity, int *err) {
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_bounded(bar, parity, err);
}

// The parts that the plan gives to the tensor-memory kernel (k_prefix_tc.cu).
cudaError_t launch_prefix_tc(const PrefixArgs &a, const PrefixPlan &pl, const CUtensorMap &map, int D, bool pdl,
                             cudaStream_t s);

}  // namespace hq
