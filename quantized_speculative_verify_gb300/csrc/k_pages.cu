// k_pages.cu -- the page table of a paged key/value cache: fork, extend with
// copy on write, free, compaction, copies, and the write of new rows.
//
// The table operations check their lists completely before they change
// anything, so a call that fails leaves the cache as it was.  Fork, free and
// compact run in one cluster of 8 thread blocks, whose barrier separates the
// check from the change: fork and free spread the table entries over the
// cluster, compact the kept positions.  Extend and compact hand out pages,
// which is a scan over the counts (the lowest free pages, in the lists'
// order): one block does it and writes a job list, and a second kernel,
// launched programmatically, moves the rows of all planes.
//
// What bounds them: the table operations, chains of dependent loads and
// barriers (4 requests of 57 pages / 96 branches of 126: free 4.8 / 7.2 us, fork
// 4.5 / 5.9, extend 6.4 / 7.0, compact 8.8 / 9.7; 6 sequences of 500 pages cut to
// half: compact 25); the write of 4 / 96 sequences' 16 rows takes 4.5 / 6.5 us.
// The move is bound by memory: 6 x 8000 rows of 16 planes and 8 heads of 128,
// 2.4 GB read and written in 377 us = 6.4 TB/s (427 us with every thread looking
// its places up by itself).
#include <cooperative_groups.h>

#include "batch.cuh"

namespace cg = cooperative_groups;

namespace hq {
namespace {

constexpr int PCL = 8;         // thread blocks of the clustered table kernels
constexpr int PT = 1024;       // threads of each
constexpr int PMAX = 1024;     // entries of a list
constexpr int PSEQ = 8192;     // sequences of a cache (bits of the duplicate check)
constexpr int MOVE_BATCH = 8;  // rows a thread has in flight
constexpr int MOVE_RUN = 128;
constexpr size_t NOWHERE = ~(size_t)0;
static_assert(MOVE_RUN % MOVE_BATCH == 0 && MOVE_RUN <= 256, "whole batches, a thread a position");

// One sequence whose rows move: positions [p0, end); position p comes from p
// itself where p < from, else from base + keep[p - base - 1].  Old pages are
// in the job's row of the scratch table, new ones in the cache's table.
struct Job {
    int seq, p0, end, from, base, old_len;
    int whole;  // every destination page is fresh: rows may move in any order
    int item;   // row of the keep lists
};

// Scratch: [0, 16) number of jobs (int) and padding; jobs; the list of pages
// handed out; old tables [list][max_pages].
__host__ __device__ inline size_t scratch_jobs() { return 16; }
__host__ __device__ inline size_t scratch_pages() { return scratch_jobs() + (size_t)PMAX * sizeof(Job); }
__host__ __device__ inline size_t scratch_tables(int n_pages) {
    return (scratch_pages() + (size_t)n_pages * 4 + 15) / 16 * 16;
}
__device__ __forceinline__ int *jobs_count(const hq_pages &c) { return static_cast<int *>(c.scratch); }
__device__ __forceinline__ Job *jobs_of(const hq_pages &c) {
    return reinterpret_cast<Job *>(static_cast<uint8_t *>(c.scratch) + scratch_jobs());
}
__device__ __forceinline__ int32_t *list_of(const hq_pages &c) {
    return reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c.scratch) + scratch_pages());
}
__device__ __forceinline__ int32_t *old_table(const hq_pages &c, int job) {
    return reinterpret_cast<int32_t *>(static_cast<uint8_t *>(c.scratch) + scratch_tables(c.n_pages)) +
           (size_t)job * c.max_pages;
}

__device__ __forceinline__ int pages_of(int len, int ps) { return len / ps + (len % ps != 0); }

// Sum of `v` over the block; `below`: over the threads before this one.
__device__ int block_scan(int v, int *s_warp, int &below) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    below = x - v + (warp ? s_warp[warp - 1] : 0);
    return s_warp[31];
}

// Whether seq is a sequence not seen before in this list (a bit per sequence).
__device__ __forceinline__ bool first_use(const hq_pages &c, int seq, uint32_t *s_bits) {
    if (seq < 0 || seq >= c.n_seqs) return false;
    const uint32_t bit = 1u << (seq & 31);
    return (atomicOr(&s_bits[seq >> 5], bit) & bit) == 0;
}

__global__ void __cluster_dims__(PCL, 1, 1) __launch_bounds__(PT)
    k_pages_fork(const hq_pages c, const int32_t *src, const int32_t *dst, int n) {
    __shared__ uint32_t s_bits[PSEQ / 32];
    __shared__ int s_src[PMAX], s_dst[PMAX], s_len[PMAX];
    const int tid = threadIdx.x;
    for (int i = tid; i < PSEQ / 32; i += PT) s_bits[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    bool bad = false;
    int s = -1;
    if (tid < n) {
        s = src[tid];
        const int d = dst[tid];
        s_src[tid] = s;
        s_dst[tid] = d;
        bad = !first_use(c, d, s_bits) || s < 0 || s >= c.n_seqs;
        if (!bad) {
            const int len = c.len[s];
            s_len[tid] = len;
            bad = c.len[d] != 0 || !len_ok(c, len);
        }
    }
    __syncthreads();
    if (tid < n && !bad) bad = (s_bits[s >> 5] >> (s & 31)) & 1u;  // a source that is also a destination
    bad = __syncthreads_or(bad);
    cg::this_cluster().sync();  // every block has read the lengths
    if (bad) {                  // the same in every block
        if (blockIdx.x == 0 && tid == 0) set_status(c, HQ_ERR_INVALID_ARG);
        return;
    }
    // one warp per (sequence, 32 pages)
    const int warp = (int)(blockIdx.x * PT + tid) >> 5, lane = tid & 31, warps = PCL * PT / 32;
    const int chunks = (c.max_pages + 31) / 32;
    for (int w = warp; w < n * chunks; w += warps) {
        const int i = w / chunks, p = (w % chunks) * 32 + lane;
        if (p >= pages_of(s_len[i], c.page_size)) continue;
        const int page = c.table[(size_t)s_src[i] * c.max_pages + p];
        c.table[(size_t)s_dst[i] * c.max_pages + p] = page;
        if (page_ok(c, page)) atomicAdd(&c.ref[page], 1);
    }
    if (blockIdx.x == 0 && tid < n) c.len[s_dst[tid]] = s_len[tid];
}

__global__ void __cluster_dims__(PCL, 1, 1) __launch_bounds__(PT)
    k_pages_free(const hq_pages c, const int32_t *seqs, int n) {
    __shared__ uint32_t s_bits[PSEQ / 32];
    __shared__ int s_seq[PMAX], s_len[PMAX];
    const int tid = threadIdx.x;
    for (int i = tid; i < PSEQ / 32; i += PT) s_bits[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    bool bad = false;
    if (tid < n) {
        const int s = seqs[tid];
        s_seq[tid] = s;
        bad = !first_use(c, s, s_bits);
        if (!bad) {
            s_len[tid] = c.len[s];
            bad = !len_ok(c, s_len[tid]);
        }
    }
    bad = __syncthreads_or(bad);
    cg::this_cluster().sync();
    if (bad) {
        if (blockIdx.x == 0 && tid == 0) set_status(c, HQ_ERR_INVALID_ARG);
        return;
    }
    const int warp = (int)(blockIdx.x * PT + tid) >> 5, lane = tid & 31, warps = PCL * PT / 32;
    const int chunks = (c.max_pages + 31) / 32;
    for (int w = warp; w < n * chunks; w += warps) {
        const int i = w / chunks, p = (w % chunks) * 32 + lane;
        if (p >= pages_of(s_len[i], c.page_size)) continue;
        int32_t *e = &c.table[(size_t)s_seq[i] * c.max_pages + p];
        const int page = *e;
        *e = -1;
        if (page_ok(c, page)) atomicSub(&c.ref[page], 1);
    }
    if (blockIdx.x == 0 && tid < n) c.len[s_seq[tid]] = 0;
}

// The `want` lowest free pages, ascending, into list[]; whether there are that
// many.  All threads of the block call it; list is visible to them after it.
__device__ bool find_free(const hq_pages &c, int want, int32_t *list, int *s_warp) {
    int got = 0;
    for (int p0 = 0; p0 < c.n_pages && got < want; p0 += PT * 4) {
        const int p = p0 + (int)threadIdx.x * 4;
        int free4 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (p + i < c.n_pages && c.ref[p + i] == 0) free4 |= 1 << i;
        int below;
        const int sum = block_scan(__popc(free4), s_warp, below);
        int k = got + below;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((free4 >> i) & 1) {
                if (k < want) list[k] = p + i;
                ++k;
            }
        got += sum;
    }
    __syncthreads();
    return got >= want;
}

__global__ void __launch_bounds__(PT) k_pages_extend(const hq_pages c, const int32_t *seqs, const int32_t *add, int n) {
    __shared__ uint32_t s_bits[PSEQ / 32];
    __shared__ int s_warp[32];
    __shared__ int s_first[PMAX], s_n[PMAX], s_at[PMAX], s_seq[PMAX];
    const int tid = threadIdx.x, ps = c.page_size;
    int32_t *list = list_of(c);
    for (int i = tid; i < PSEQ / 32; i += PT) s_bits[i] = 0;
    pdl_wait();
    __syncthreads();
    bool bad = false, cow = false;
    int seq = -1, len = 0, grow = 0, more = 0, part = -1;
    if (tid < n) {
        seq = seqs[tid];
        grow = add[tid];
        bad = !first_use(c, seq, s_bits) || grow < 0;
        if (!bad) {
            len = c.len[seq];
            bad = !len_ok(c, len) || grow > c.max_pages * ps - len;
        }
        if (!bad && grow > 0) {
            more = pages_of(len + grow, ps) - pages_of(len, ps);
            if (len % ps) {
                part = c.table[(size_t)seq * c.max_pages + len / ps];
                cow = page_ok(c, part) && c.ref[part] > 1;
            }
        }
    }
    bad = __syncthreads_or(bad);
    int first, job;
    const int want = block_scan(bad ? 0 : more + (cow ? 1 : 0), s_warp, first);
    const int njobs = block_scan(cow ? 1 : 0, s_warp, job);
    const bool enough = !bad && find_free(c, want, list, s_warp);
    if (tid == 0) {
        *jobs_count(c) = enough ? njobs : 0;
        if (!enough) set_status(c, bad ? HQ_ERR_INVALID_ARG : HQ_ERR_NO_PAGES);
    }
    if (!enough) {
        pdl_launch_dependents();
        return;
    }
    if (tid < n) {
        if (cow) {
            const int page = list[first];
            c.table[(size_t)seq * c.max_pages + len / ps] = page;
            c.ref[page] = 1;
            atomicSub(&c.ref[part], 1);
            jobs_of(c)[job] = Job{seq, len / ps * ps, len, len, len, len, 1, 0};
            old_table(c, job)[len / ps] = part;
        }
        s_first[tid] = first + (cow ? 1 : 0);
        s_n[tid] = more;
        s_at[tid] = pages_of(len, ps);
        s_seq[tid] = seq;
        if (grow > 0) c.len[seq] = len + grow;
    }
    __syncthreads();
    // one warp per sequence: its new pages
    const int lane = tid & 31;
    for (int i = tid >> 5; i < n; i += PT / 32)
        for (int k = lane; k < s_n[i]; k += 32) {
            const int page = list[s_first[i] + k];
            c.table[(size_t)s_seq[i] * c.max_pages + s_at[i] + k] = page;
            c.ref[page] = 1;
        }
    pdl_launch_dependents();
}

// What k_pages_compact knows of its sequences, in shared memory.
struct Compact {
    int seq[PMAX], len[PMAX], base[PMAX], nk[PMAX], d0[PMAX], fresh[PMAX], first[PMAX], job[PMAX];
    int warp[32];
    int bad, most;
};

// The page passes of the compaction, G lanes a sequence (8 where every sequence
// changes few pages, else 32).
template <int G>
struct PagePasses {
    // lane of the group, its bits in the warp, sequences side by side
    int lane, sub;
    uint32_t mask;
    __device__ PagePasses() {
        const int l = threadIdx.x & 31;
        lane = l & (G - 1);
        sub = threadIdx.x / G;
        mask = G == 32 ? ~0u : ((1u << (G & 31)) - 1u) << (l & ~(G - 1));
    }
    __device__ static bool moves(const Compact &s, int i) { return s.nk[i] >= 0 && s.d0[i] < s.nk[i]; }

    // fresh pages of each sequence: those of its changed pages that are shared
    __device__ void count(const hq_pages &c, Compact &s, int n, bool bad) const {
        const int ps = c.page_size;
        for (int i = sub; i < n; i += PT / G) {
            int k = 0;
            if (!bad && moves(s, i)) {
                const int p1 = pages_of(s.base[i] + 1 + s.nk[i], ps);
                const int32_t *row = c.table + (size_t)s.seq[i] * c.max_pages;
                for (int p = (s.base[i] + 1 + s.d0[i]) / ps + lane; p < p1; p += G) {
                    const int page = row[p];
                    k += page_ok(c, page) && c.ref[page] > 1;
                }
            }
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) k += __shfl_xor_sync(mask, k, o);
            if (lane == 0) s.fresh[i] = k;
        }
    }
    // Notes the old pages and the new ones.  Which pages are shared is decided
    // for all before any count changes: a page held by two listed sequences is
    // shared for both.
    __device__ void note(const hq_pages &c, const Compact &s, int n) const {
        const int ps = c.page_size;
        const int32_t *list = list_of(c);
        for (int i = sub; i < n; i += PT / G) {
            if (s.nk[i] < 0) continue;
            int32_t *row = c.table + (size_t)s.seq[i] * c.max_pages;
            const int p1 = pages_of(s.base[i] + 1 + s.nk[i], ps), q1 = pages_of(s.len[i], ps);
            const bool mv = s.job[i] >= 0;
            const int lo = mv ? (s.base[i] + 1 + s.d0[i]) / ps : p1;
            int32_t *o = mv ? old_table(c, s.job[i]) : nullptr;
            int k = s.first[i];
            for (int p0 = lo; p0 < q1; p0 += G) {
                const int p = p0 + lane;
                int page = -1;
                if (p < q1) {
                    page = row[p];
                    if (!page_ok(c, page)) row[p] = page = -1;  // below -1 only -2 - (a page) from here on
                    if (mv) o[p] = page;
                }
                const bool fresh = mv && p < p1 && page >= 0 && c.ref[page] > 1;
                const uint32_t m = __ballot_sync(mask, fresh) & mask;
                if (fresh) row[p] = -2 - list[k + __popc(m & ((1u << (threadIdx.x & 31)) - 1u))];
                if (fresh && p == lo) jobs_of(c)[s.job[i]].p0 = lo * ps;
                k += __popc(m);
            }
        }
    }
    __device__ void apply(const hq_pages &c, const Compact &s, int n) const {
        const int ps = c.page_size;
        for (int i = sub; i < n; i += PT / G) {
            if (s.nk[i] < 0) continue;
            int32_t *row = c.table + (size_t)s.seq[i] * c.max_pages;
            const int end = s.base[i] + 1 + s.nk[i], p1 = pages_of(end, ps), q1 = pages_of(s.len[i], ps);
            const bool mv = s.job[i] >= 0;
            const int lo = mv ? (s.base[i] + 1 + s.d0[i]) / ps : p1;
            const int32_t *o = mv ? old_table(c, s.job[i]) : row;
            for (int p = lo + lane; p < q1; p += G) {
                const int now = row[p];
                int gone = -1;  // the page this sequence gives up here
                if (now <= -2) {
                    gone = o[p];
                    row[p] = -2 - now;
                    c.ref[-2 - now] = 1;
                } else if (p >= p1) {
                    gone = now;
                    row[p] = -1;
                }
                if (gone >= 0) atomicSub(&c.ref[gone], 1);
            }
            if (lane == 0) c.len[s.seq[i]] = end;
        }
    }
};

__global__ void __cluster_dims__(PCL, 1, 1) __launch_bounds__(PT)
    k_pages_compact(const hq_pages c, const int32_t *seqs, const int32_t *base, const int32_t *keep, int ldkeep,
                    int max_keep, const int32_t *n_keep, int n) {
    __shared__ uint32_t s_bits[PSEQ / 32];
    __shared__ Compact s;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, ps = c.page_size;
    for (int i = tid; i < PSEQ / 32; i += PT) s_bits[i] = 0;
    if (tid == 0) s.bad = s.most = 0;
    pdl_wait();
    __syncthreads();
    int span = 0;
    if (tid < n) {
        const int q = seqs[tid], b = base[tid], k = n_keep[tid];
        int len = 0;
        bool bad = !first_use(c, q, s_bits);
        if (!bad && k >= 0) {
            len = c.len[q];
            bad = !len_ok(c, len) || b < -1 || b >= len || k > max_keep || k > len - 1 - b;
        }
        if (bad) s.bad = 1;
        s.seq[tid] = q;
        s.base[tid] = b;
        s.nk[tid] = bad ? -1 : k;
        s.len[tid] = len;
        s.d0[tid] = k < 0 ? 0 : k;
        if (!bad && k >= 0) {
            atomicMax(&s.most, k);
            span = pages_of(len, ps) - (b + 1) / ps;  // pages it may look at
        }
    }
    const bool few = !__syncthreads_or(span > 16);
    // Every kept position: ascending, inside the sequence; d0 = the first that
    // moves.  The cluster's warps share the lists in runs of 32.
    const int warp = (int)(blockIdx.x * PT + tid) >> 5, warps = PCL * PT / 32, runs = (s.most + 31) / 32;
    for (int w = warp; w < n * runs; w += warps) {
        const int i = w / runs, d = (w % runs) * 32 + lane;
        if (d >= s.nk[i]) continue;
        const int32_t *kp = keep + (size_t)i * ldkeep;
        const int k = kp[d], before = d ? kp[d - 1] : 0;
        if (k <= before || k > s.len[i] - 1 - s.base[i]) s.bad = 1;
        if (k != d + 1) atomicMin(&s.d0[i], d);
    }
    cluster.sync();
    if (blockIdx.x != 0) {
        cluster.sync();  // block 0 has read this block's findings
        pdl_launch_dependents();
        return;
    }
    bool bad = false;
    if (tid < PCL) bad = *cluster.map_shared_rank(&s.bad, tid) != 0;
    if (tid < n) {
        int d0 = s.d0[tid];
#pragma unroll
        for (int r = 1; r < PCL; ++r) {
            const int v = cluster.map_shared_rank(s.d0, r)[tid];
            d0 = v < d0 ? v : d0;
        }
        s.d0[tid] = d0;
    }
    bad = __syncthreads_or(bad);
    cluster.sync();

    const PagePasses<8> narrow;
    const PagePasses<32> wide;
    if (few)
        narrow.count(c, s, n, bad);
    else
        wide.count(c, s, n, bad);
    __syncthreads();
    int first, job;
    const int want = block_scan(tid < n ? s.fresh[tid] : 0, s.warp, first);
    const bool moves = !bad && tid < n && PagePasses<32>::moves(s, tid);
    const int njobs = block_scan(moves ? 1 : 0, s.warp, job);
    const bool enough = !bad && find_free(c, want, list_of(c), s.warp);
    if (tid == 0) {
        *jobs_count(c) = enough ? njobs : 0;
        if (!enough) set_status(c, bad ? HQ_ERR_INVALID_ARG : HQ_ERR_NO_PAGES);
    }
    if (!enough) {
        pdl_launch_dependents();
        return;
    }
    if (tid < n) {
        s.first[tid] = first;
        s.job[tid] = moves ? job : -1;
        if (moves) {
            const int from = s.base[tid] + 1 + s.d0[tid], end = s.base[tid] + 1 + s.nk[tid];
            jobs_of(c)[job] = Job{s.seq[tid], from, end, from, s.base[tid], s.len[tid],
                                  s.fresh[tid] == pages_of(end, ps) - from / ps, tid};
        }
    }
    __syncthreads();
    if (few)
        narrow.note(c, s, n);
    else
        wide.note(c, s, n);
    __syncthreads();
    if (few)
        narrow.apply(c, s, n);
    else
        wide.apply(c, s, n);
    pdl_launch_dependents();
}

// Moves the rows of the jobs: blockIdx = (column block, job, run of positions).
// The block looks up where the positions lie, MOVE_RUN at a time; a thread owns
// one 16-byte column of one head and plane and takes positions in ascending
// order, MOVE_BATCH loads in flight.  Rows only move down, and a
// page that is both read and written belongs to this sequence alone, so within
// a column no row is overwritten before it has been read; where every
// destination page is fresh the positions are also split over blockIdx.z.
__global__ void __launch_bounds__(256) k_pages_move(const hq_pages c, const int32_t *keep, int ldkeep, int runs) {
    __shared__ size_t s_from[MOVE_RUN], s_to[MOVE_RUN];
    pdl_launch_dependents();
    pdl_wait();
    if ((int)blockIdx.y >= *jobs_count(c)) return;
    const Job j = jobs_of(c)[blockIdx.y];
    const int32_t *old = old_table(c, blockIdx.y);
    const int32_t *now = c.table + (size_t)j.seq * c.max_pages;
    const int32_t *kp = keep ? keep + (size_t)j.item * ldkeep : nullptr;  // extend moves nothing past `from`
    const int units = c.row_bytes / 16, columns = c.n_planes * c.heads * units;
    const int col = blockIdx.x * 256 + threadIdx.x;
    int p0 = j.p0, p1 = j.end;
    if (j.whole) {
        const int per = ((p1 - p0 + runs - 1) / runs + MOVE_BATCH - 1) / MOVE_BATCH * MOVE_BATCH;
        p0 += per * (int)blockIdx.z;
        if (p1 - p0 > per) p1 = p0 + per;
    } else if (blockIdx.z != 0) {
        return;
    }
    const int plane = col / (c.heads * units), head = col / units % c.heads, unit = col % units;
    const size_t page_bytes = (size_t)c.heads * c.page_size * c.row_bytes;
    uint8_t *at = static_cast<uint8_t *>(c.pool) + (size_t)plane * c.plane_bytes +
                  (size_t)head * c.page_size * c.row_bytes + (size_t)unit * 16;
    for (int p = p0; p < p1; p += MOVE_RUN) {
        const int n = p1 - p < MOVE_RUN ? p1 - p : MOVE_RUN;
        __syncthreads();  // the places of the run before have been used
        if ((int)threadIdx.x < MOVE_RUN) {
            const int q = p + threadIdx.x;
            size_t from = 0, to = NOWHERE;
            if (q < p1) {
                const int src = q < j.from ? q : j.base + kp[q - j.base - 1];
                if (src >= q && src < j.old_len) {  // always: the lists were checked
                    const int x = old[src / c.page_size], z = now[q / c.page_size];
                    if (page_ok(c, x) && page_ok(c, z)) {
                        from = (size_t)x * page_bytes + (size_t)(src % c.page_size) * c.row_bytes;
                        to = (size_t)z * page_bytes + (size_t)(q % c.page_size) * c.row_bytes;
                    }
                }
            }
            s_from[threadIdx.x] = from;
            s_to[threadIdx.x] = to;
        }
        __syncthreads();
        if (col >= columns) continue;
        for (int i = 0; i < n; i += MOVE_BATCH) {
            uint4 v[MOVE_BATCH];
#pragma unroll
            for (int b = 0; b < MOVE_BATCH; ++b)  // (past the run: s_to says nowhere)
                if (s_to[i + b] != NOWHERE) v[b] = *reinterpret_cast<const uint4 *>(at + s_from[i + b]);
#pragma unroll
            for (int b = 0; b < MOVE_BATCH; ++b)
                if (s_to[i + b] != NOWHERE) *reinterpret_cast<uint4 *>(at + s_to[i + b]) = v[b];
        }
    }
}

// One block per (pair, plane).
__global__ void __launch_bounds__(256) k_pages_copy(const hq_pages c, const int32_t *src, const int32_t *dst) {
    pdl_launch_dependents();
    pdl_wait();
    const int s = src[blockIdx.x], d = dst[blockIdx.x];
    if (!page_ok(c, s) || !page_ok(c, d)) {
        if (threadIdx.x == 0 && blockIdx.y == 0) set_status(c, HQ_ERR_INVALID_ARG);
        return;
    }
    const size_t bytes = (size_t)c.heads * c.page_size * c.row_bytes, n = bytes / 16;
    uint8_t *plane = static_cast<uint8_t *>(c.pool) + (size_t)blockIdx.y * c.plane_bytes;
    const uint4 *a = reinterpret_cast<const uint4 *>(plane + (size_t)s * bytes);
    uint4 *b = reinterpret_cast<uint4 *>(plane + (size_t)d * bytes);
    for (size_t i = threadIdx.x; i < n; i += 256 * 4) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * 256 < n) v[k] = a[i + k * 256];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k * 256 < n) b[i + k * 256] = v[k];
    }
}

// One thread block per row, its K and its V: blockIdx = (row of a sequence,
// sequence).  The row is on its way while its place is looked up.
__global__ void __launch_bounds__(128) k_pages_write(const hq_pages c, const WriteArgs w) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.y, i = blockIdx.x;
    int first, m;
    batch_rows(w.starts, b, w.rows, w.max_rows, first, m);
    if (i >= m) return;
    const int units = c.row_bytes / 16, n = c.heads * units;
    const uint8_t *src[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
        src[x] = static_cast<const uint8_t *>(x ? w.v : w.k) +
                 (size_t)(first + i) * (size_t)(x ? w.ldv : w.ldk) * type_bytes(w.in_type);
    auto load = [&](int u, uint4 (&o)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (w.in_type != HQ_F32) {
                o[x] = reinterpret_cast<const uint4 *>(src[x])[u];
                continue;
            }
            const float4 y = reinterpret_cast<const float4 *>(src[x])[2 * u], z = reinterpret_cast<const float4 *>(src[x])[2 * u + 1];
            const float f[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (w.type == HQ_F16) {
                    const __half2 t = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
                    h[e] = *reinterpret_cast<const uint32_t *>(&t);
                } else {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                    h[e] = *reinterpret_cast<const uint32_t *>(&t);
                }
            }
            o[x] = make_uint4(h[0], h[1], h[2], h[3]);
        }
    };
    uint4 o[2];
    int u = threadIdx.x;
    if (u < n) load(u, o);
    const int seq = w.seqs ? w.seqs[b] : b;
    int page = -1, p = 0;
    if (seq >= 0 && seq < c.n_seqs) {
        const int len = c.len[seq];
        p = len - m + i;
        if (len_ok(c, len) && p >= 0) page = c.table[(size_t)seq * c.max_pages + p / c.page_size];
    }
    if (!page_ok(c, page)) {
        if (threadIdx.x == 0) set_status(c, HQ_ERR_INVALID_ARG);
        return;
    }
    uint8_t *dst = static_cast<uint8_t *>(c.pool) + (size_t)page * c.heads * c.page_size * c.row_bytes +
                   (size_t)(p % c.page_size) * c.row_bytes;
    while (u < n) {
        const size_t at = (size_t)(u / units) * c.page_size * c.row_bytes + (size_t)(u % units) * 16;
        *reinterpret_cast<uint4 *>(dst + (size_t)w.k_plane * c.plane_bytes + at) = o[0];
        *reinterpret_cast<uint4 *>(dst + (size_t)w.v_plane * c.plane_bytes + at) = o[1];
        u += 128;
        if (u < n) load(u, o);
    }
}

cudaError_t launch_move(const hq_pages &c, const int32_t *keep, int ldkeep, int n, long long most, cudaStream_t s) {
    const int columns = c.n_planes * c.heads * (c.row_bytes / 16), cb = (columns + 255) / 256;
    // positions split so that there are some blocks for every SM, with at
    // least 64 positions each
    const int sms = device_sm_count();
    long long runs = (4LL * (sms > 0 ? sms : 1) + (long long)cb * n - 1) / ((long long)cb * n);
    if (runs > (most + 63) / 64) runs = (most + 63) / 64;
    if (runs < 1) runs = 1;
    return launch_kernel(k_pages_move, dim3((unsigned)cb, (unsigned)n, (unsigned)runs), dim3(256), 0, true, s, c, keep,
                         ldkeep, (int)runs);
}

}  // namespace

size_t pages_scratch_bytes(const hq_pages &c) {
    const size_t rows = c.n_seqs < PMAX ? c.n_seqs : PMAX;
    return (scratch_tables(c.n_pages) + rows * (size_t)c.max_pages * 4 + 15) / 16 * 16;
}

cudaError_t launch_pages_fork(const hq_pages &c, const int32_t *src, const int32_t *dst, int n, bool pdl, cudaStream_t s) {
    return launch_kernel(k_pages_fork, dim3(PCL), dim3(PT), 0, pdl, s, c, src, dst, n);
}

cudaError_t launch_pages_free(const hq_pages &c, const int32_t *seqs, int n, bool pdl, cudaStream_t s) {
    return launch_kernel(k_pages_free, dim3(PCL), dim3(PT), 0, pdl, s, c, seqs, n);
}

cudaError_t launch_pages_extend(const hq_pages &c, const int32_t *seqs, const int32_t *add, int n, bool pdl, cudaStream_t s) {
    cudaError_t e = launch_kernel(k_pages_extend, dim3(1), dim3(PT), 0, pdl, s, c, seqs, add, n);
    if (e != cudaSuccess) return e;
    return launch_move(c, nullptr, 0, n, c.page_size, s);
}

cudaError_t launch_pages_compact(const hq_pages &c, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                                 int ldkeep, int max_keep, const int32_t *n_keep, int n, bool pdl,
                                 cudaStream_t s) {
    cudaError_t e = launch_kernel(k_pages_compact, dim3(PCL), dim3(PT), 0, pdl, s, c, seqs, base, keep, ldkeep, max_keep,
                                  n_keep, n);
    if (e != cudaSuccess) return e;
    return launch_move(c, keep, ldkeep, n, (long long)max_keep + c.page_size, s);
}

cudaError_t launch_pages_copy(const hq_pages &c, const int32_t *src, const int32_t *dst, int n, bool pdl, cudaStream_t s) {
    return launch_kernel(k_pages_copy, dim3((unsigned)n, (unsigned)c.n_planes), dim3(256), 0, pdl, s, c, src, dst);
}

cudaError_t launch_pages_write(const hq_pages &c, const WriteArgs &w, bool pdl, cudaStream_t s) {
    return launch_kernel(k_pages_write, dim3((unsigned)w.max_rows, (unsigned)w.B), dim3(128), 0, pdl, s, c, w);
}

}  // namespace hq
