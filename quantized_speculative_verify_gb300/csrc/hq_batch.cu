// hq_batch.cu -- the C ABI of the calls for a batch of requests: argument
// validation (before anything is launched) and dispatch.
#include <cfloat>
#include <climits>
#include <cmath>

#include "batch.cuh"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA; }
bool type_ok(int t) { return t == HQ_F32 || t == HQ_F16 || t == HQ_BF16; }
bool type16(int t) { return t == HQ_F16 || t == HQ_BF16; }
cudaStream_t stream_of(void *s) { return static_cast<cudaStream_t>(s); }
bool pdl_of(uint32_t flags) { return (flags & HQ_LAUNCH_PDL) != 0; }

// Rows of `cols` elements, `ld` apart, every row 16-byte aligned.
bool rows_ok(const void *p, int type, int64_t ld, int64_t cols) {
    return aligned(p, 16) && ld >= cols && ld <= (1ll << 40) && (ld * hq::type_bytes(type)) % 16 == 0;
}

bool cache_ok(const hq_pages *c) {
    if (!c || !c->pool || !c->ref || !c->table || !c->len || !c->status || !c->scratch) return false;
    if (!aligned(c->pool, 16) || !aligned(c->scratch, 16) || !aligned(c->ref, 4) || !aligned(c->table, 4) ||
        !aligned(c->len, 4) || !aligned(c->status, 4))
        return false;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return false;
    if (c->row_bytes <= 0 || c->row_bytes > 4096 || c->row_bytes % 16 != 0) return false;
    if (c->n_planes <= 0 || c->n_planes > 65535 || c->heads <= 0 || c->heads > 65535) return false;
    if (c->n_pages <= 0 || c->n_pages > (1 << 24) || c->n_seqs <= 0 || c->n_seqs > 8192) return false;
    if (c->max_pages <= 0 || c->max_pages > (1 << 20)) return false;
    if ((long long)c->n_pages * c->page_size > INT_MAX || (long long)c->max_pages * c->page_size > INT_MAX) return false;
    const long long page = (long long)c->heads * c->page_size * c->row_bytes;  // below 2^36
    if (c->plane_bytes % 16 != 0 || c->plane_bytes / page < c->n_pages) return false;
    // a thread's column number stays an int
    return (long long)c->n_planes * c->heads * (c->row_bytes / 16) <= INT_MAX - 256;
}

bool history_ok(const hq_history *h) {
    return h->tokens && h->len && h->status && aligned(h->tokens, 4) && aligned(h->len, 4) && aligned(h->prompt, 4) &&
           aligned(h->status, 4) && h->n_slots >= 1 && h->n_slots <= 65536 && h->cap >= 1 && h->cap <= 1 << 24;
}

// Synchronizes, reads a status word and clears it.
int take_status(int32_t *status, void *stream) {
    if (cudaStreamSynchronize(stream_of(stream)) != cudaSuccess) return HQ_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, status, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return HQ_ERR_CUDA;
    if (v == 0) return HQ_OK;
    const int zero = 0;
    if (cudaMemcpy(status, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return HQ_ERR_CUDA;
    return v;
}

// A list of a page operation: n entries; a sequence stands in it once.
bool list_ok(const hq_pages *c, int32_t n) { return n >= 0 && n <= 1024 && n <= c->n_seqs; }

}  // namespace

extern "C" {

int hq_add_norm_quant(const hq_layer_desc *desc, const void *x, int32_t x_type, int64_t ldx, const void *residual,
                      void *residual_out, int32_t r_type, int64_t ldr, const float *weight, float eps, int32_t M,
                      const uint32_t *signs, void *h, int32_t h_type, int64_t ldh, int8_t *qx, int32_t *gsum,
                      void *qop, float *sx, uint32_t flags, void *stream) {
    if (!hq::desc_ok(desc) || M < 0 || M > (qop ? HQ_MAX_M : 1 << 20)) return HQ_ERR_INVALID_ARG;
    if ((flags & ~HQ_LAUNCH_PDL) != 0 || !(eps >= 0.0f) || eps > 3.0e38f) return HQ_ERR_INVALID_ARG;
    if (!type_ok(x_type) || !type_ok(r_type) || !type_ok(h_type)) return HQ_ERR_INVALID_ARG;
    if (M == 0) return HQ_OK;
    const int K = desc->K;
    const bool quant = qx || gsum || qop;
    if (!x || !weight || (!quant && !h && !residual_out)) return HQ_ERR_INVALID_ARG;
    if (quant && (!signs || !sx || !aligned(signs, 4) || !aligned(sx, 4))) return HQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_type, ldx, K) || !aligned(weight, 16)) return HQ_ERR_INVALID_ARG;
    if ((residual || residual_out) && (!rows_ok(residual, r_type, ldr, K) || !rows_ok(residual_out, r_type, ldr, K)))
        return HQ_ERR_INVALID_ARG;
    if (h && !rows_ok(h, h_type, ldh, K)) return HQ_ERR_INVALID_ARG;
    if ((qx && !aligned(qx, 8)) || (gsum && !aligned(gsum, 4)) || (qop && !aligned(qop, 16))) return HQ_ERR_INVALID_ARG;
    hq::NormArgs a;
    a.x = x;
    a.res = residual;
    a.res_out = residual_out;
    a.h = h;
    a.weight = weight;
    a.signs = signs;
    a.qx = qx;
    a.gsum = gsum;
    a.qop = static_cast<uint8_t *>(qop);
    a.sx = quant ? sx : nullptr;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.eps = eps;
    a.x_type = x_type;
    a.r_type = r_type;
    a.h_type = h_type;
    a.M = M;
    a.K = K;
    a.G = desc->group;
    a.rs = qop && hq::act_rs(desc->format, M);
    a.e4 = qop && hq::act_e4(desc->format, M, desc->group);
    a.sums = qop && hq::act_sums(desc->format, M);
    return cuda_status(hq::launch_norm(a, pdl_of(flags), stream_of(stream)));
}

size_t hq_lora_workspace_bytes(int32_t M, int32_t r_max) {
    if (M <= 0 || M > HQ_MAX_M || r_max <= 0 || r_max > 256 || r_max % 8 != 0) return 0;
    return (size_t)M * r_max * 4;
}

int hq_lora_apply(const void *x, int32_t x_type, int64_t ldx, int32_t M, int32_t K, int32_t N, const void *A,
                  const void *B, int32_t w_type, int32_t n_adapters, int32_t r_max, const int32_t *ids,
                  const int32_t *ranks, const float *scale, const float *base, int64_t ldb, float *Y, int64_t ldy,
                  void *workspace, uint32_t flags, void *stream) {
    if (M < 0 || M > HQ_MAX_M || K <= 0 || K > hq::MAX_K || K % 8 != 0 || N <= 0) return HQ_ERR_INVALID_ARG;
    if (r_max <= 0 || r_max > 256 || r_max % 8 != 0 || n_adapters <= 0 || n_adapters > (1 << 24)) return HQ_ERR_INVALID_ARG;
    if ((flags & ~HQ_LAUNCH_PDL) != 0 || !type_ok(x_type) || !type16(w_type)) return HQ_ERR_INVALID_ARG;
    if (M == 0) return HQ_OK;
    if (!x || !A || !B || !ids || !Y || !workspace) return HQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_type, ldx, K) || !aligned(A, 16) || !aligned(B, 16) || !aligned(workspace, 16))
        return HQ_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(ranks, 4) || !aligned(scale, 4) || !aligned(base, 4) || !aligned(Y, 4))
        return HQ_ERR_INVALID_ARG;
    if (ldy < N || ldy > (1ll << 40) || (base && (ldb < N || ldb > (1ll << 40)))) return HQ_ERR_INVALID_ARG;
    if (base == Y && ldb != ldy) return HQ_ERR_INVALID_ARG;
    hq::LoraArgs a;
    a.x = x;
    a.A = A;
    a.B = B;
    a.ids = ids;
    a.ranks = ranks;
    a.scale = scale;
    a.base = base;
    a.Y = Y;
    a.t = static_cast<float *>(workspace);
    a.ldx = ldx;
    a.ldb = ldb;
    a.ldy = ldy;
    a.x_type = x_type;
    a.M = M;
    a.K = K;
    a.N = N;
    a.n_adapters = n_adapters;
    a.r_max = r_max;
    return cuda_status(hq::launch_lora(a, w_type, pdl_of(flags), stream_of(stream)));
}

size_t hq_pages_scratch_bytes(const hq_pages *cache) {
    if (!cache) return 0;
    hq_pages c = *cache;  // sized before it is allocated: the pointers do not count
    alignas(16) static int32_t any[4];
    c.pool = c.scratch = any;
    c.ref = c.table = c.len = c.status = any;
    return cache_ok(&c) ? hq::pages_scratch_bytes(c) : 0;
}

int hq_pages_fork(const hq_pages *cache, const int32_t *src, const int32_t *dst, int32_t n, uint32_t flags,
                  void *stream) {
    if (!cache_ok(cache) || !list_ok(cache, n) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (n == 0) return HQ_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return HQ_ERR_INVALID_ARG;
    return cuda_status(hq::launch_pages_fork(*cache, src, dst, n, pdl_of(flags), stream_of(stream)));
}

int hq_pages_extend(const hq_pages *cache, const int32_t *seqs, const int32_t *add, int32_t n, uint32_t flags,
                    void *stream) {
    if (!cache_ok(cache) || !list_ok(cache, n) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (n == 0) return HQ_OK;
    if (!seqs || !add || !aligned(seqs, 4) || !aligned(add, 4)) return HQ_ERR_INVALID_ARG;
    return cuda_status(hq::launch_pages_extend(*cache, seqs, add, n, pdl_of(flags), stream_of(stream)));
}

int hq_pages_free(const hq_pages *cache, const int32_t *seqs, int32_t n, uint32_t flags, void *stream) {
    if (!cache_ok(cache) || !list_ok(cache, n) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (n == 0) return HQ_OK;
    if (!seqs || !aligned(seqs, 4)) return HQ_ERR_INVALID_ARG;
    return cuda_status(hq::launch_pages_free(*cache, seqs, n, pdl_of(flags), stream_of(stream)));
}

int hq_pages_compact(const hq_pages *cache, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                     int32_t ldkeep, int32_t max_keep, const int32_t *n_keep, int32_t n, uint32_t flags,
                     void *stream) {
    if (!cache_ok(cache) || !list_ok(cache, n) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (max_keep < 0 || ldkeep < max_keep || ldkeep > 1 << 20) return HQ_ERR_INVALID_ARG;
    if (n == 0) return HQ_OK;
    if (!seqs || !base || !keep || !n_keep || !aligned(seqs, 4) || !aligned(base, 4) || !aligned(keep, 4) ||
        !aligned(n_keep, 4))
        return HQ_ERR_INVALID_ARG;
    return cuda_status(
        hq::launch_pages_compact(*cache, seqs, base, keep, ldkeep, max_keep, n_keep, n, pdl_of(flags), stream_of(stream)));
}

int hq_pages_copy(const hq_pages *cache, const int32_t *src, const int32_t *dst, int32_t n, uint32_t flags,
                  void *stream) {
    if (!cache_ok(cache) || n < 0 || n > 65535 || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (n == 0) return HQ_OK;
    if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return HQ_ERR_INVALID_ARG;
    return cuda_status(hq::launch_pages_copy(*cache, src, dst, n, pdl_of(flags), stream_of(stream)));
}

int hq_pages_write(const hq_pages *cache, int32_t k_plane, int32_t v_plane, const void *k, const void *v,
                   int32_t in_type, int64_t ldk, int64_t ldv, int32_t type, const int32_t *seqs,
                   const int32_t *starts, int32_t B, int32_t rows, int32_t max_rows, uint32_t flags, void *stream) {
    if (!cache_ok(cache) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (k_plane < 0 || k_plane >= cache->n_planes || v_plane < 0 || v_plane >= cache->n_planes) return HQ_ERR_INVALID_ARG;
    if (!type16(type) || (in_type != HQ_F32 && in_type != type)) return HQ_ERR_INVALID_ARG;
    if (B < 0 || B > 65535 || rows < 0 || max_rows < 1) return HQ_ERR_INVALID_ARG;
    if (!starts && (long long)B * max_rows > rows) return HQ_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return HQ_OK;
    const int64_t cols = (int64_t)cache->heads * (cache->row_bytes / 2);
    if (!k || !v || !rows_ok(k, in_type, ldk, cols) || !rows_ok(v, in_type, ldv, cols)) return HQ_ERR_INVALID_ARG;
    if (!aligned(seqs, 4) || !aligned(starts, 4)) return HQ_ERR_INVALID_ARG;
    hq::WriteArgs w;
    w.k = k;
    w.v = v;
    w.ldk = ldk;
    w.ldv = ldv;
    w.seqs = seqs;
    w.starts = starts;
    w.k_plane = k_plane;
    w.v_plane = v_plane;
    w.in_type = in_type;
    w.type = type;
    w.B = B;
    w.rows = rows;
    w.max_rows = max_rows < rows ? max_rows : rows;
    return cuda_status(hq::launch_pages_write(*cache, w, pdl_of(flags), stream_of(stream)));
}

int hq_pages_status(const hq_pages *cache, void *stream) {
    if (!cache_ok(cache)) return HQ_ERR_INVALID_ARG;
    return take_status(cache->status, stream);
}

size_t hq_prefix_attention_workspace_bytes(int32_t B, int32_t rows, int32_t max_rows, int32_t Hq, int32_t Hkv,
                                           int32_t D) {
    if (B <= 0 || B > 65535 || rows <= 0 || max_rows <= 0 || max_rows > HQ_MAX_M || Hkv <= 0 || Hq <= 0 || Hq % Hkv != 0)
        return 0;
    if ((D != 64 && D != 128) || (long long)rows * Hq > (1 << 28)) return 0;
    return hq::prefix_workspace_bytes(rows, max_rows, Hq, Hkv, D);
}

int hq_prefix_attention(const hq_pages *cache, int32_t k_plane, int32_t v_plane, int32_t type, const void *q,
                        int64_t ldq, const int32_t *seqs, const int32_t *starts, int32_t B, int32_t rows,
                        int32_t max_rows, const int32_t *parent, int32_t Hq, int32_t shared, int32_t max_len,
                        float scale, void *out, int32_t out_type, int64_t ldo, void *workspace, uint32_t flags,
                        void *stream) {
    if (!cache_ok(cache) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (k_plane < 0 || k_plane >= cache->n_planes || v_plane < 0 || v_plane >= cache->n_planes) return HQ_ERR_INVALID_ARG;
    if (!type16(type) || (out_type != HQ_F32 && out_type != type)) return HQ_ERR_INVALID_ARG;
    if (B < 0 || B > 65535 || rows < 0 || max_rows < 1 || max_rows > HQ_MAX_M) return HQ_ERR_INVALID_ARG;
    if (!starts && (long long)B * max_rows > rows) return HQ_ERR_INVALID_ARG;
    if (Hq <= 0 || Hq > 65535 || Hq % cache->heads != 0 || (long long)rows * Hq > (1 << 28)) return HQ_ERR_INVALID_ARG;
    const float c_log2 = scale * 1.4426950408889634f;
    if (!(c_log2 <= FLT_MAX && c_log2 >= -FLT_MAX)) return HQ_ERR_INVALID_ARG;
    if (shared < 0 || max_len < 1 || max_len > 1 << 30 || shared >= max_len ||
        max_len > (long long)cache->max_pages * cache->page_size)
        return HQ_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return HQ_OK;
    const int D = cache->row_bytes / 2;
    if (!q || !out || !workspace || !rows_ok(q, type, ldq, (int64_t)Hq * D) ||
        !rows_ok(out, out_type, ldo, (int64_t)Hq * D))
        return HQ_ERR_INVALID_ARG;
    if (!aligned(workspace, 16) || !aligned(seqs, 4) || !aligned(starts, 4) || !aligned(parent, 4))
        return HQ_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return HQ_ERR_UNSUPPORTED;
    if (cache->plane_bytes >= (1ll << 40)) return HQ_ERR_UNSUPPORTED;  // the tensor map's largest stride
    hq::PrefixArgs a = {};
    a.q = q;
    a.out = out;
    a.seqs = seqs;
    a.starts = starts;
    a.parent = parent;
    a.table = cache->table;
    a.len = cache->len;
    a.status = cache->status;
    a.ldq = ldq;
    a.ldo = ldo;
    a.B = B;
    a.rows = rows;
    a.max_rows = max_rows;
    a.Hq = Hq;
    a.Hkv = cache->heads;
    a.G = Hq / cache->heads;
    a.n_seqs = cache->n_seqs;
    a.max_pages = cache->max_pages;
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.n_pages = cache->n_pages;
    a.k_plane = k_plane;
    a.v_plane = v_plane;
    a.shared = shared;
    a.max_len = max_len;
    a.type = type;
    a.out_type = out_type;
    a.c_log2 = c_log2;
    return cuda_status(hq::launch_prefix_attention(*cache, a, D, workspace, pdl_of(flags), stream_of(stream)));
}

int hq_rope_freqs(int32_t rot, double base, int32_t kind, double factor, double original, double low, double high,
                  double *freqs_host) {
    if (rot < 2 || rot > 65536 || rot % 2 != 0 || !(base > 1.0) || base > DBL_MAX || !freqs_host) return HQ_ERR_INVALID_ARG;
    if (kind < HQ_ROPE_PLAIN || kind > HQ_ROPE_BANDS) return HQ_ERR_INVALID_ARG;
    if (kind != HQ_ROPE_PLAIN && !(factor >= 1.0 && factor <= 1e9)) return HQ_ERR_INVALID_ARG;
    if (kind == HQ_ROPE_NTK && rot < 4) return HQ_ERR_INVALID_ARG;
    const bool mixed = kind == HQ_ROPE_YARN || kind == HQ_ROPE_BANDS;
    if (mixed && !(original > 0.0 && original <= 1e18 && low > 0.0 && high > low && high <= 1e18)) return HQ_ERR_INVALID_ARG;
    const double pi2 = 6.283185307179586476925286766559;
    if (kind == HQ_ROPE_NTK) base *= std::pow(factor, (double)rot / (rot - 2));
    double lo = 0.0, hi = 0.0;
    if (kind == HQ_ROPE_YARN) {
        lo = std::fmax(std::floor(rot * std::log(original / (high * pi2)) / (2.0 * std::log(base))), 0.0);
        hi = std::fmin(std::ceil(rot * std::log(original / (low * pi2)) / (2.0 * std::log(base))), rot - 1.0);
    }
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        double keep = 1.0;  // share of f itself, the rest of f / factor
        if (kind == HQ_ROPE_LINEAR) keep = 0.0;
        if (kind == HQ_ROPE_YARN) keep = 1.0 - std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
        if (kind == HQ_ROPE_BANDS) keep = std::fmin(std::fmax((original * f / pi2 - low) / (high - low), 0.0), 1.0);
        freqs_host[i] = keep == 1.0 || kind == HQ_ROPE_PLAIN ? f : f / factor + (f - f / factor) * keep;
    }
    return HQ_OK;
}

int hq_rope_turns(const double *freqs_host, int32_t n, uint64_t *turns_host) {
    if (!freqs_host || !turns_host || n < 1 || n > 32768) return HQ_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!(freqs_host[i] >= 0.0 && freqs_host[i] <= 3.141592653589793116)) return HQ_ERR_INVALID_ARG;
    // 1 / (2 pi) in units of 2^-128
    const uint64_t hi = 0x28BE60DB9391054Aull, lo = 0x7F09D5F47D4D3770ull;
    for (int i = 0; i < n; ++i) {
        int e = 0;
        const uint64_t m = (uint64_t)std::ldexp(std::frexp(freqs_host[i], &e), 53);  // f = m 2^(e - 53)
        // m / (2 pi) in units of 2^-64, below 2^118; f in turns is that, times 2^(e - 53)
        const unsigned __int128 p = (unsigned __int128)m * hi + (((unsigned __int128)m * lo) >> 64);
        const int shift = 53 - e;  // at least 51
        turns_host[i] = shift > 120 ? 0 : (uint64_t)((p + ((unsigned __int128)1 << (shift - 1))) >> shift);
    }
    return HQ_OK;
}

int hq_rope_write(const hq_pages *cache, int32_t k_plane, int32_t v_plane, int32_t type, const void *q, const void *k,
                  const void *v, int32_t in_type, int64_t ldq, int64_t ldk, int64_t ldv, int32_t Hq,
                  const float *q_weight, const float *k_weight, float eps, const uint64_t *turns, int32_t rot,
                  int32_t layout, float gain, const int32_t *seqs, const int32_t *starts, int32_t B, int32_t rows,
                  int32_t max_rows, const int32_t *parent, const int32_t *positions, void *q_out, int64_t ldo,
                  uint32_t flags, void *stream) {
    if (!cache_ok(cache) || (flags & ~HQ_LAUNCH_PDL) != 0) return HQ_ERR_INVALID_ARG;
    if (k_plane < 0 || k_plane >= cache->n_planes || v_plane < 0 || v_plane >= cache->n_planes) return HQ_ERR_INVALID_ARG;
    if (k_plane == v_plane) return HQ_ERR_INVALID_ARG;  // they are written side by side
    if (!type16(type) || (in_type != HQ_F32 && in_type != type)) return HQ_ERR_INVALID_ARG;
    if (Hq <= 0 || Hq > 65535 || (layout != HQ_ROPE_HALF && layout != HQ_ROPE_INTERLEAVED)) return HQ_ERR_INVALID_ARG;
    if (!(eps >= 0.0f && eps <= FLT_MAX) || !(gain <= FLT_MAX && gain >= -FLT_MAX)) return HQ_ERR_INVALID_ARG;
    const int D = cache->row_bytes / 2;
    if (rot < 16 || rot % 16 != 0 || rot > D) return HQ_ERR_INVALID_ARG;
    if (B < 0 || B > 65535 || rows < 0 || max_rows < 1 || (parent && max_rows > HQ_MAX_M)) return HQ_ERR_INVALID_ARG;
    if (!starts && (long long)B * max_rows > rows) return HQ_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return HQ_OK;
    if (!q || !k || !v || !q_out || !turns) return HQ_ERR_INVALID_ARG;
    if (!rows_ok(q, in_type, ldq, (int64_t)Hq * D) || !rows_ok(q_out, type, ldo, (int64_t)Hq * D) ||
        !rows_ok(k, in_type, ldk, (int64_t)cache->heads * D) || !rows_ok(v, in_type, ldv, (int64_t)cache->heads * D))
        return HQ_ERR_INVALID_ARG;
    if (q_out == q && (in_type != type || ldo != ldq)) return HQ_ERR_INVALID_ARG;
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(turns, 8) || !aligned(seqs, 4) || !aligned(starts, 4) ||
        !aligned(parent, 4) || !aligned(positions, 4))
        return HQ_ERR_INVALID_ARG;
    if (D != 64 && D != 128 && D != 256) return HQ_ERR_UNSUPPORTED;
    hq::RopeArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.qw = q_weight;
    a.kw = k_weight;
    a.turns = turns;
    a.seqs = seqs;
    a.starts = starts;
    a.parent = parent;
    a.positions = positions;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldo = ldo;
    a.eps = eps;
    a.gain = gain;
    a.in_type = in_type;
    a.type = type;
    a.layout = layout;
    a.rot = rot;
    a.Hq = Hq;
    a.B = B;
    a.rows = rows;
    a.max_rows = max_rows < rows ? max_rows : rows;
    a.k_plane = k_plane;
    a.v_plane = v_plane;
    return cuda_status(hq::launch_rope_write(*cache, a, pdl_of(flags), stream_of(stream)));
}

int hq_gated_norm_quant(const hq_layer_desc *desc, const void *x, int32_t x_type, int64_t ldx, const void *gate,
                        int32_t g_type, int64_t ldg, int32_t act, const float *weight, int32_t D, float eps, int32_t M,
                        const uint32_t *signs, void *h, int32_t h_type, int64_t ldh, int8_t *qx, int32_t *gsum,
                        void *qop, float *sx, uint32_t flags, void *stream) {
    if (!hq::desc_ok(desc) || M < 0 || M > (qop ? HQ_MAX_M : 1 << 20)) return HQ_ERR_INVALID_ARG;
    if ((flags & ~HQ_LAUNCH_PDL) != 0 || !(eps >= 0.0f && eps <= FLT_MAX)) return HQ_ERR_INVALID_ARG;
    if (!type_ok(x_type) || !type_ok(g_type) || !type_ok(h_type)) return HQ_ERR_INVALID_ARG;
    if (act < HQ_GATE_NONE || act > HQ_GATE_SILU || (D != 64 && D != 128 && D != 256)) return HQ_ERR_INVALID_ARG;
    const int K = desc->K;
    if (K % D != 0) return HQ_ERR_INVALID_ARG;
    if (M == 0) return HQ_OK;
    const bool quant = qx || gsum || qop;
    if (!x || (!quant && !h)) return HQ_ERR_INVALID_ARG;
    if (quant && (!signs || !sx || !aligned(signs, 4) || !aligned(sx, 4))) return HQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_type, ldx, K) || !aligned(weight, 16)) return HQ_ERR_INVALID_ARG;
    if ((gate && !rows_ok(gate, g_type, ldg, K)) || (h && !rows_ok(h, h_type, ldh, K))) return HQ_ERR_INVALID_ARG;
    if (h && ((h == x && (h_type != x_type || ldh != ldx)) || (h == gate && (h_type != g_type || ldh != ldg))))
        return HQ_ERR_INVALID_ARG;
    if ((qx && !aligned(qx, 8)) || (gsum && !aligned(gsum, 4)) || (qop && !aligned(qop, 16))) return HQ_ERR_INVALID_ARG;
    hq::GateArgs a = {};
    a.n.x = x;
    a.n.h = h;
    a.n.weight = weight;
    a.n.signs = signs;
    a.n.qx = qx;
    a.n.gsum = gsum;
    a.n.qop = static_cast<uint8_t *>(qop);
    a.n.sx = quant ? sx : nullptr;
    a.n.ldx = ldx;
    a.n.ldh = ldh;
    a.n.eps = eps;
    a.n.x_type = x_type;
    a.n.h_type = h_type;
    a.n.M = M;
    a.n.K = K;
    a.n.G = desc->group;
    a.n.rs = qop && hq::act_rs(desc->format, M);
    a.n.e4 = qop && hq::act_e4(desc->format, M, desc->group);
    a.n.sums = qop && hq::act_sums(desc->format, M);
    a.gate = gate;
    a.ldg = ldg;
    a.g_type = g_type;
    a.act = act;
    a.D = D;
    return cuda_status(hq::launch_gated_norm(a, pdl_of(flags), stream_of(stream)));
}

size_t hq_greedy_tokens_workspace_bytes(int32_t rows) {
    return rows > 0 && rows <= 1 << 26 ? hq::greedy_workspace_bytes(rows) : 0;
}

int hq_greedy_tokens(const void *logits, int32_t type, int64_t ldl, int32_t V, const hq_history *history,
                     const hq_logit_rules *rules, const int32_t *mask_ids, const int32_t *seqs, const int32_t *starts,
                     int32_t B, int32_t rows, int32_t max_rows, const int32_t *parent, const int32_t *tokens, void *out,
                     int32_t out_type, int64_t ldo, int32_t *greedy, void *workspace, uint32_t flags, void *stream) {
    if ((flags & ~HQ_LAUNCH_PDL) != 0 || !type_ok(type) || (out_type != type && out_type != HQ_F32)) return HQ_ERR_INVALID_ARG;
    if (V < 1 || V > 1 << 24) return HQ_ERR_INVALID_ARG;
    if (history && !history_ok(history)) return HQ_ERR_INVALID_ARG;
    if (rules) {
        const hq_logit_rules &r = *rules;
        if (r.n_slots < 0 || r.n_slots > 65536 || r.n_bias < 0 || r.n_masks < 0) return HQ_ERR_INVALID_ARG;
        if (!aligned(r.repetition, 4) || !aligned(r.presence, 4) || !aligned(r.frequency, 4) || !aligned(r.bias_starts, 4) ||
            !aligned(r.bias_tokens, 4) || !aligned(r.bias_values, 4) || !aligned(r.masks, 4))
            return HQ_ERR_INVALID_ARG;
        if (r.bias_starts && r.n_bias > 0 && (!r.bias_tokens || !r.bias_values)) return HQ_ERR_INVALID_ARG;
        if (r.masks && (r.ldmask < (V + 31) / 32 || r.ldmask > 1ll << 40)) return HQ_ERR_INVALID_ARG;
    }
    if (B < 0 || B > 65535 || rows < 0 || rows > 1 << 26 || max_rows < 1 || max_rows > HQ_MAX_M) return HQ_ERR_INVALID_ARG;
    if (!starts && (long long)B * max_rows > rows) return HQ_ERR_INVALID_ARG;
    if (B == 0 || rows == 0) return HQ_OK;
    if (!logits || !greedy || !workspace || !aligned(workspace, 16) || !aligned(greedy, 4)) return HQ_ERR_INVALID_ARG;
    if (!aligned(logits, hq::type_bytes(type)) || ldl < V || ldl > 1ll << 40) return HQ_ERR_INVALID_ARG;
    if (out && (!aligned(out, hq::type_bytes(out_type)) || ldo < V || ldo > 1ll << 40)) return HQ_ERR_INVALID_ARG;
    if (out == logits && (out_type != type || ldo != ldl)) return HQ_ERR_INVALID_ARG;
    if (!aligned(mask_ids, 4) || !aligned(seqs, 4) || !aligned(starts, 4) || !aligned(parent, 4) || !aligned(tokens, 4))
        return HQ_ERR_INVALID_ARG;
    hq::GreedyArgs a = {};
    a.logits = logits;
    a.out = out;
    a.mask_ids = mask_ids;
    a.seqs = seqs;
    a.starts = starts;
    a.parent = parent;
    a.tokens = tokens;
    a.greedy = greedy;
    a.workspace = static_cast<uint8_t *>(workspace);
    if (history) a.history = *history;
    if (rules) a.rules = *rules;
    a.ldl = ldl;
    a.ldo = ldo;
    a.type = type;
    a.out_type = out_type;
    a.V = V;
    a.B = B;
    a.rows = rows;
    a.max_rows = max_rows < rows ? max_rows : rows;
    return cuda_status(hq::launch_greedy_tokens(a, pdl_of(flags), stream_of(stream)));
}

int hq_tree_accept_batch(const int32_t *greedy, const int32_t *parent, const int32_t *tokens, const int32_t *seqs,
                         const int32_t *starts, int32_t B, int32_t rows, int32_t max_rows, const hq_history *history,
                         int32_t *path, int32_t ldpath, int32_t *n_accept, int32_t *bonus, uint32_t flags,
                         void *stream) {
    if ((flags & ~HQ_LAUNCH_PDL) != 0 || (history && !history_ok(history))) return HQ_ERR_INVALID_ARG;
    if (B < 0 || B > 65535 || rows < 0 || max_rows < 1 || max_rows > HQ_MAX_M || ldpath < max_rows) return HQ_ERR_INVALID_ARG;
    if (!starts && (long long)B * max_rows > rows) return HQ_ERR_INVALID_ARG;
    if (B == 0) return HQ_OK;
    if (!path || !n_accept || !bonus || (rows > 0 && (!greedy || !tokens))) return HQ_ERR_INVALID_ARG;
    if (!aligned(greedy, 4) || !aligned(parent, 4) || !aligned(tokens, 4) || !aligned(seqs, 4) || !aligned(starts, 4) ||
        !aligned(path, 4) || !aligned(n_accept, 4) || !aligned(bonus, 4))
        return HQ_ERR_INVALID_ARG;
    hq::AcceptBatchArgs a = {};
    a.greedy = greedy;
    a.parent = parent;
    a.tokens = tokens;
    a.seqs = seqs;
    a.starts = starts;
    a.path = path;
    a.n_accept = n_accept;
    a.bonus = bonus;
    if (history) a.history = *history;
    a.ldpath = ldpath;
    a.B = B;
    a.rows = rows;
    a.max_rows = max_rows;
    return cuda_status(hq::launch_accept_batch(a, pdl_of(flags), stream_of(stream)));
}

int hq_history_status(const hq_history *history, void *stream) {
    if (!history || !history_ok(history)) return HQ_ERR_INVALID_ARG;
    return take_status(history->status, stream);
}

}  // extern "C"
