// k_accept_batch.cu -- acceptance of a batch of draft trees, and the growth of
// the requests' histories by what was accepted.
//
// Node i > 0 agrees when its token is the model's greedy token after its parent,
// and is valid when it and all of its ancestors agree; the deepest valid node is
// accepted, the lowest index among equally deep ones.  "All ancestors" and depths
// are found by doubling: after k rounds a node knows its 2^k-th ancestor, the
// depth it has passed and whether all of those agree, so a tree of 128 nodes
// takes 7 rounds instead of 127 dependent steps.  The same table of ancestors
// gives every entry of the accepted path at once: the entry at depth d is the
// accepted node's ancestor (depth - d) levels up, a sum of powers of two.
//
// One thread block per sequence, a thread per node.  It is one chain of loads,
// rounds and stores: one tree of 16 nodes and 512 of 128 take 3.8 and 4.0 us with
// the copy in front that puts the lengths back.
#include "batch.cuh"

namespace hq {
namespace {

constexpr int AT = HQ_MAX_M;      // threads
constexpr int LEVELS = 7;         // 2^7 = HQ_MAX_M
static_assert(1 << LEVELS == HQ_MAX_M, "a level for each doubling");

// A node's 2^k-th ancestor, the levels up to it, and whether all on the way agree.
__device__ __forceinline__ uint32_t packed(uint32_t up, uint32_t levels, uint32_t agree) { return up | levels << 8 | agree << 16; }

__global__ void __launch_bounds__(AT) k_accept_batch(const AcceptBatchArgs a) {
    __shared__ int32_t s_g[AT], s_tok[AT];
    __shared__ uint32_t s_up[LEVELS + 1][AT];
    __shared__ int s_best[AT / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x, t = threadIdx.x;
    int first, m;
    batch_rows(a.starts, b, a.rows, a.max_rows, first, m);
    int32_t *path = a.path + (size_t)b * a.ldpath;
    int parent = 0, token = 0;
    if (t < m) {
        parent = t == 0 ? 0 : a.parent ? a.parent[first + t] : t - 1;
        token = a.tokens[first + t];
        s_g[t] = a.greedy[first + t];
        s_tok[t] = token;
    }
    const bool bad = t > 0 && t < m && (parent < 0 || parent >= t);
    if (__syncthreads_or(bad || m == 0)) {
        if (t < a.max_rows) path[t] = -1;
        if (t == 0) a.n_accept[b] = a.bonus[b] = -1;
        return;
    }
    // the root and the threads past the last node stand on the root
    const bool node = t > 0 && t < m;
    uint32_t w = node ? packed(parent, 1, s_g[parent] >= 0 && s_g[parent] == token) : packed(0, 0, 1);
    s_up[0][t] = w;
#pragma unroll
    for (int k = 0; k < LEVELS; ++k) {
        __syncthreads();
        const uint32_t v = s_up[k][w & 0xff];
        w = packed(v & 0xff, (w >> 8 & 0xff) + (v >> 8 & 0xff), (w >> 16) & (v >> 16));
        s_up[k + 1][t] = w;
    }
    // the deepest valid node, the lowest index among equally deep ones
    int key = t < m && (w >> 16) != 0 ? (int)(w >> 8 & 0xff) << 8 | (AT - 1 - t) : -1;
    key = __reduce_max_sync(0xffffffffu, key);
    if ((t & 31) == 0) s_best[t >> 5] = key;
    // what the history has, and whether this sequence may write there
    int seq = -1, len = -1;
    bool dup = false;
    if (a.history.tokens) {
        seq = a.seqs ? a.seqs[b] : b;
        if (seq >= 0 && seq < a.history.n_slots) len = a.history.len[seq];
        if (a.seqs)
            for (int i = t; i < b; i += AT) dup = dup || a.seqs[i] == seq;
    }
    dup = __syncthreads_or(dup);
    key = s_best[0];
#pragma unroll
    for (int i = 1; i < AT / 32; ++i) key = s_best[i] > key ? s_best[i] : key;
    const int n = key >> 8, best = AT - 1 - (key & 0xff), bonus = s_g[best];
    int at = -1;
    if (t < n) {
        at = best;
        const int up = n - 1 - t;
#pragma unroll
        for (int k = 0; k < LEVELS; ++k)
            if (up >> k & 1) at = (int)(s_up[k][at] & 0xff);
    }
    if (t < a.max_rows) path[t] = at;
    if (t == 0) {
        a.n_accept[b] = n;
        a.bonus[b] = bonus;
    }
    if (!a.history.tokens) return;
    const int more = n + (bonus >= 0 ? 1 : 0);
    if (dup || len < 0 || len > a.history.cap - more) {
        if (t == 0) atomicCAS(a.history.status, 0, (int)HQ_ERR_INVALID_ARG);
        return;
    }
    if (t < more) a.history.tokens[(size_t)seq * a.history.cap + len + t] = t < n ? s_tok[at] : bonus;
    if (t == 0) a.history.len[seq] = len + more;
}

}  // namespace

cudaError_t launch_accept_batch(const AcceptBatchArgs &a, bool pdl, cudaStream_t s) {
    return launch_kernel(k_accept_batch, dim3((unsigned)a.B), dim3(AT), 0, pdl, s, a);
}

}  // namespace hq
