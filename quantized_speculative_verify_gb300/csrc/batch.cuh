// batch.cuh -- launchers and helpers of the calls for a batch of requests.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hq_internal.cuh"

namespace hq {

__host__ __device__ inline int type_bytes(int type) { return type == HQ_F32 ? 4 : 2; }

// A launch with programmatic dependent launch where `pdl` is set.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t s,
                          A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct NormArgs {
    const void *x, *res;
    void *res_out, *h;
    const float *weight;
    const uint32_t *signs;
    int8_t *qx;
    int32_t *gsum;
    uint8_t *qop;
    float *sx;
    int64_t ldx, ldr, ldh;
    float eps;
    int x_type, r_type, h_type;
    int M, K, G;
    int rs, e4, sums;  // encoding of the operand (hq_internal.cuh)
    int keep;          // set by launch_norm
};
cudaError_t launch_norm(const NormArgs &a, bool pdl, cudaStream_t s);

struct LoraArgs {
    const void *x, *A, *B;
    const int32_t *ids, *ranks;
    const float *scale, *base;
    float *Y, *t;  // t: [M][r_max], the products A x
    int64_t ldx, ldb, ldy;
    int x_type, M, K, N, n_adapters, r_max;
};
cudaError_t launch_lora(const LoraArgs &a, int w_type, bool pdl, cudaStream_t s);

// Page operations (k_pages.cu).
size_t pages_scratch_bytes(const hq_pages &c);
cudaError_t launch_pages_fork(const hq_pages &c, const int32_t *src, const int32_t *dst, int n, bool pdl, cudaStream_t s);
cudaError_t launch_pages_extend(const hq_pages &c, const int32_t *seqs, const int32_t *add, int n, bool pdl, cudaStream_t s);
cudaError_t launch_pages_free(const hq_pages &c, const int32_t *seqs, int n, bool pdl, cudaStream_t s);
cudaError_t launch_pages_compact(const hq_pages &c, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                                 int ldkeep, int max_keep, const int32_t *n_keep, int n, bool pdl,
                                 cudaStream_t s);
cudaError_t launch_pages_copy(const hq_pages &c, const int32_t *src, const int32_t *dst, int n, bool pdl, cudaStream_t s);

struct WriteArgs {
    const void *k, *v;
    int64_t ldk, ldv;
    const int32_t *seqs, *starts;
    int k_plane, v_plane, in_type, type, B, rows, max_rows;
};
cudaError_t launch_pages_write(const hq_pages &c, const WriteArgs &w, bool pdl, cudaStream_t s);

// Attention of a batch over a paged cache (k_prefix.cu).
struct PrefixArgs {
    const void *q;
    void *out;
    const int32_t *seqs, *starts, *parent, *table, *len;
    const uint8_t *pool;
    int64_t plane_bytes;
    int *err, *status;  // the workspace's error word, the cache's status word
    float *ws_o, *ws_ml;  // [part][row][Hq][D], [part][row][Hq][2]: running maximum (base-2 units), sum
    int64_t ldq, ldo;
    int B, rows, max_rows, Hq, Hkv, G, n_seqs, max_pages, page_shift, n_pages, k_plane, v_plane;
    int shared, max_len, type, out_type;
    float c_log2;  // scale * log2(e)
};
size_t prefix_workspace_bytes(int rows, int max_rows, int Hq, int Hkv, int D);
cudaError_t launch_prefix_attention(const hq_pages &c, PrefixArgs a, int D, void *workspace, bool pdl, cudaStream_t s);

// Rotary positions on the way into the cache (k_rope.cu).
struct RopeArgs {
    const void *q, *k, *v;
    void *q_out;
    const float *qw, *kw;
    const uint64_t *turns;
    const int32_t *seqs, *starts, *parent, *positions;
    int64_t ldq, ldk, ldv, ldo;
    float eps, gain;
    int in_type, type, layout, rot, Hq, B, rows, max_rows, k_plane, v_plane;
};
cudaError_t launch_rope_write(const hq_pages &c, const RopeArgs &a, bool pdl, cudaStream_t s);

// The norm per head with its gate (k_gate.cu).  n: the rows, h and the codes as
// in the norm of whole rows; its residual is not used and its weight is [D].
struct GateArgs {
    NormArgs n;
    const void *gate;
    int64_t ldg;
    int g_type, act, D;
};
cudaError_t launch_gated_norm(const GateArgs &a, bool pdl, cudaStream_t s);

// Rules on the logits and greedy tokens (k_greedy.cu), acceptance (k_accept_batch.cu).
struct GreedyArgs {
    const void *logits;
    void *out;
    const int32_t *mask_ids, *seqs, *starts, *parent, *tokens;
    int32_t *greedy;
    uint8_t *workspace;
    hq_history history;  // tokens NULL: none
    hq_logit_rules rules;
    int64_t ldl, ldo;
    int type, out_type, V, B, rows, max_rows;
};
size_t greedy_workspace_bytes(int rows);
cudaError_t launch_greedy_tokens(const GreedyArgs &a, bool pdl, cudaStream_t s);

struct AcceptBatchArgs {
    const int32_t *greedy, *parent, *tokens, *seqs, *starts;
    int32_t *path, *n_accept, *bonus;
    hq_history history;  // tokens NULL: none
    int ldpath, B, rows, max_rows;
};
cudaError_t launch_accept_batch(const AcceptBatchArgs &a, bool pdl, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ void set_status(const hq_pages &c, int err) { atomicCAS(c.status, 0, err); }
__device__ __forceinline__ bool page_ok(const hq_pages &c, int page) { return page >= 0 && page < c.n_pages; }
// max_pages * page_size is below 2^31 (checked by the host)
__device__ __forceinline__ bool len_ok(const hq_pages &c, int len) { return len >= 0 && len <= c.max_pages * c.page_size; }

// Rows of sequence b of a batch: the first row and their number, always
// within [0, rows) and at most max_rows, whatever `starts` holds.
__device__ __forceinline__ void batch_rows(const int32_t *starts, int b, int rows, int max_rows, int &first, int &m) {
    int lo, hi;
    if (starts) {
        lo = starts[b];
        hi = starts[b + 1];
    } else {  // B * max_rows is at most rows (checked by the host)
        lo = b * max_rows;
        hi = lo + max_rows;
    }
    if (lo < 0 || lo > rows || hi < lo) {
        first = 0;
        m = 0;
        return;
    }
    if (hi > rows) hi = rows;
    first = lo;
    m = hi - lo < max_rows ? hi - lo : max_rows;
}

// The sequence that claims a row, by one warp: how many of starts[1..B] are at
// most `row` (32 probes a round).  Whatever starts holds, the answer is within
// [0, B]; batch_rows says whether the row is that sequence's.
__device__ __forceinline__ int row_sequence(const int32_t *starts, int B, int max_rows, int row) {
    if (!starts) {
        const int b = row / max_rows;
        return b < B ? b : B;
    }
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (n > 0) {
        const int step = (n + 31) / 32;
        const long long at = (lane + 1ll) * step;
        const bool below = at <= n && starts[lo + (int)at] <= row;
        const int k = __popc(__ballot_sync(0xffffffffu, below)) * step;
        lo += k;
        n = n - k < step - 1 ? n - k : step - 1;
    }
    return lo;
}
#endif

}  // namespace hq
