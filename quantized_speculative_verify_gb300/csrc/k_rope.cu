// k_rope.cu -- rotary positions of the newest rows, their q rotated for the
// attention, their k rotated and written into the paged cache together with v.
//
//   (u, v) -> (u c - v s, v c + u s),  c, s = gain cos, gain sin of p f_i
//
// A pair's angle is p f_i.  In fp32 that product loses the angle at far
// positions; here a frequency is a fraction of a turn in 64-bit fixed point, the
// product with the position wraps modulo a turn by itself, and its upper 32 bits
// are the angle in (-1/2, 1/2] turns: one integer multiplication, exact at any
// position, and sincospif sees a small argument.
//
// One thread block per row.  A thread holds octets of 8 consecutive elements of
// a head (one 16-byte load of 16-bit values, two of fp32); a head is D / 8
// consecutive lanes, so its norm and the partners half a rotated width away are
// lane exchanges, and since the block is a multiple of a head the thread's
// cosines are the same for all of its heads.  The first octets are on their way
// while one warp looks up the row's sequence, depth and page.
//
// Four tokens 3.7 us, 100 rows of trees with normed heads 5.0 (one row's chain:
// sequence, length, page, cosines, stores); 10000 prompt rows 43.5 us = 5.6 TB/s,
// 84 % of the copy rate.
#include "rows.cuh"

namespace hq {
namespace {

// RT: threads.  HALF: the layout.  WIDE: fp32 inputs.  NORM: heads are normed first.
template <int RT, int U, bool HALF, bool WIDE, bool NORM>
__global__ void __launch_bounds__(RT, (NORM ? 768 : 1024) / RT) k_rope_write(const hq_pages c, const RopeArgs a) {
    constexpr int AHEAD = WIDE ? 2 : 4;  // octets of a thread that are loaded before they are used
    const int in_type = WIDE ? HQ_F32 : a.type;
    __shared__ float2 s_turn[4 * U];  // cosine and sine of each pair
    __shared__ int s_place, s_page, s_pos;
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int nq = a.Hq * U, nk = c.heads * U, n = nq + 2 * nk;
    Raw raw[AHEAD];
    auto fetch = [&](int u0) {
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int u = u0 + tid + j * RT;
            if (u < nq) raw[j] = load_raw(row_of(a.q, in_type, a.ldq, row), in_type, u);
            else if (u < nq + nk) raw[j] = load_raw(row_of(a.k, in_type, a.ldk, row), in_type, u - nq);
            else if (u < n) raw[j] = load_raw(row_of(a.v, in_type, a.ldv, row), in_type, u - nq - nk);
            else raw[j].u = raw[j].v = make_uint4(0, 0, 0, 0);
        }
    };
    fetch(0);
    if (tid < 32) {
        int place = -1, page = -1, pos = 0;
        const int b = row_sequence(a.starts, a.B, a.max_rows, row);
        int first = 0, m = 0;
        if (b < a.B) batch_rows(a.starts, b, a.rows, a.max_rows, first, m);
        const int i = row - first;
        if (i >= 0 && i < m) {
            const int seq = a.seqs ? a.seqs[b] : b;
            const int len = seq >= 0 && seq < c.n_seqs ? c.len[seq] : -1;
            int depth = i;
            if (a.parent) {  // at most HQ_MAX_M nodes, four a lane
                int p[HQ_MAX_M / 32];
#pragma unroll
                for (int t = 0; t < HQ_MAX_M / 32; ++t) p[t] = lane + 32 * t <= i ? a.parent[first + lane + 32 * t] : -1;
                depth = 0;
                for (int node = i;;) {
                    int up = p[0];
#pragma unroll
                    for (int t = 1; t < HQ_MAX_M / 32; ++t) up = (node >> 5) == t ? p[t] : up;
                    up = __shfl_sync(0xffffffffu, up, node & 31);
                    if (up < 0 || up >= node) break;
                    node = up;
                    ++depth;
                }
            }
            if (len_ok(c, len) && len - m + i >= 0) {
                place = len - m + i;
                page = c.table[(size_t)seq * c.max_pages + place / c.page_size];
                pos = a.positions ? a.positions[row] : len - m + depth;
            }
            if (!page_ok(c, page)) {
                page = -1;
                if (lane == 0) set_status(c, HQ_ERR_INVALID_ARG);
            }
        }
        if (lane == 0) {
            s_place = place;
            s_page = page;
            s_pos = pos;
        }
    }
    __syncthreads();
    const int place = s_place, page = s_page;
    if (place < 0) return;
    for (int i = tid; i < a.rot / 2; i += RT) {
        const uint64_t angle = (uint64_t)(int64_t)s_pos * a.turns[i];
        float2 t;
        sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &t.y, &t.x);
        s_turn[i] = make_float2(t.x * a.gain, t.y * a.gain);
    }
    __syncthreads();
    const int o = tid % U, half = a.rot / 16;  // octets of half the rotated width
    const bool turned = o < 2 * half;
    const int partner = (lane - o % 32) + (HALF && turned ? (o < half ? o + half : o - half) : o);
    float co[8], si[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float2 t = make_float2(1.0f, 0.0f);
        if (turned) t = s_turn[HALF ? (o < half ? o : o - half) * 8 + e : o * 4 + e / 2];
        co[e] = t.x;
        si[e] = (HALF ? o < half : (e & 1) == 0) ? -t.y : t.y;
    }
    uint8_t *kv = static_cast<uint8_t *>(c.pool) + (size_t)(page < 0 ? 0 : page) * c.heads * c.page_size * c.row_bytes +
                  (size_t)(place % c.page_size) * c.row_bytes;
    for (int u0 = 0; u0 < n; u0 += AHEAD * RT) {
        if (u0) fetch(u0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (u0 + j * RT >= n) break;
            const int u = u0 + tid + j * RT;
            const bool is_q = u < nq, is_v = u >= nq + nk;
            float x[8], y[8];
            widen(raw[j], in_type, x);
            if (NORM) {
                const float *w = is_q ? a.qw : is_v ? nullptr : a.kw;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e];
                head_norm<U>(y, a.eps);
                if (w) {
                    const float4 lo = reinterpret_cast<const float4 *>(w)[2 * o], hi = reinterpret_cast<const float4 *>(w)[2 * o + 1];
                    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = y[e] * f[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = HALF ? __shfl_sync(0xffffffffu, x[e], partner) : x[e ^ 1];
                y[e] = turned && !is_v ? fmaf(x[e], co[e], p * si[e]) : x[e];
            }
            if (is_q) {
                store8(const_cast<void *>(row_of(a.q_out, a.type, a.ldo, row)), a.type, u, y);
            } else if (u < n && page >= 0) {
                const int head = (u - nq - (is_v ? nk : 0)) / U;
                store8(kv + (size_t)(is_v ? a.v_plane : a.k_plane) * c.plane_bytes + (size_t)head * c.page_size * c.row_bytes,
                       a.type, o, y);
            }
        }
    }
}

template <int RT, int U, bool HALF>
cudaError_t launch_layout(const hq_pages &c, const RopeArgs &a, bool pdl, cudaStream_t s) {
    const bool wide = a.in_type == HQ_F32, norm = a.qw || a.kw;
    const auto f = wide ? (norm ? k_rope_write<RT, U, HALF, true, true> : k_rope_write<RT, U, HALF, true, false>)
                        : (norm ? k_rope_write<RT, U, HALF, false, true> : k_rope_write<RT, U, HALF, false, false>);
    return launch_kernel(f, dim3((unsigned)a.rows), dim3(RT), 0, pdl, s, c, a);
}

template <int U>
cudaError_t launch_u(const hq_pages &c, const RopeArgs &a, bool pdl, cudaStream_t s) {
    // A row is a chain of waits and then a stream: few rows take many threads each,
    // many rows many blocks an SM (16 rows an SM and more).  10000 prompt rows of 48
    // heads in bf16: 256 threads 58 us, 128 47, 64 43.5; 100 rows of trees: 5.0, 5.7
    // and 8.0 us.
    const bool many = a.rows >= 16 * device_sm_count();
    if (a.layout == HQ_ROPE_HALF)
        return many ? launch_layout<64, U, true>(c, a, pdl, s) : launch_layout<256, U, true>(c, a, pdl, s);
    return many ? launch_layout<64, U, false>(c, a, pdl, s) : launch_layout<256, U, false>(c, a, pdl, s);
}

}  // namespace

cudaError_t launch_rope_write(const hq_pages &c, const RopeArgs &a, bool pdl, cudaStream_t s) {
    switch (c.row_bytes / 16) {
        case 8: return launch_u<8>(c, a, pdl, s);
        case 16: return launch_u<16>(c, a, pdl, s);
        default: return launch_u<32>(c, a, pdl, s);
    }
}

}  // namespace hq
