// hq_batch.cu -- the C ABI of the calls for a batch of requests: argument
// validation (before anything is launched) and dispatch.
#include <climits>

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

}  // extern "C"
