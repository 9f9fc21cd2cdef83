// k_greedy.cu -- penalties, biases and grammar masks on the logits of a batch's
// trees, and the greedy token of every row, in one pass over the logits.
//
//   seen:   l = l > 0 ? l / repetition : l * repetition
//   n > 0:  l = l - frequency n;  l = l - presence
//   biased: l = l + bias;   masked: l = -infinity
//   greedy = the lowest token of the largest l that is not masked
//
// Rows hold 100 thousand logits, a history a few thousand tokens: most logits
// meet no rule but the mask.  A thread block takes a chunk of the vocabulary for
// some rows of one sequence.  It counts the history's tokens of its chunk in
// shared memory (a word a token: seen, biased, drafted, and how often behind the
// prompt), once for its rows; what a row's own path adds to that is the drafted
// tokens of its ancestors, at most 127 and found only at the few tokens that are
// marked as drafted.  Then the rows stream through: four logits a load, four
// words of shared memory, and code for the rules only where a word is not zero.
//
// A block's largest value and its token make one 64-bit key (a larger key is a
// larger value, or the same value at a lower token); chunks meet by the maximum
// of their keys, which does not depend on the order, and the last one writes the
// token and leaves the workspace as it found it.
#include <type_traits>

#include "batch.cuh"

namespace hq {
namespace {

constexpr int GT = 256;          // threads
constexpr int GROUP = 4;         // rows of a sequence that share one count of its history
constexpr int MOST = 16384, LEAST = 1024;  // tokens of a chunk
constexpr uint32_t SEEN = 1u << 31, BIASED = 1u << 30, DRAFTED = 1u << 29, TIMES = DRAFTED - 1;

// The larger value, the largest; NaN if one is.
__device__ __forceinline__ float max_nan2(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ unsigned long long key_of(float v, int token) {
    if (token < 0) return 0ull;  // below every real key
    uint32_t u = __float_as_uint(v);
    if (v != v) u = 0x7FC00000u;  // every NaN ranks above +inf
    if (v == 0.0f) u = 0u;        // -0 and +0 are equal
    u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((unsigned long long)u << 32) | (0xFFFFFFFFu - (uint32_t)token);
}
__device__ __forceinline__ int token_of(unsigned long long key) {
    return key == 0ull ? -1 : (int)(0xFFFFFFFFu - (uint32_t)key);
}

template <class T>
__device__ __forceinline__ float to_f32(T x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}
template <class T>
__device__ __forceinline__ T from_f32(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

template <class T>
struct alignas(4 * sizeof(T)) Quad {
    T x[4];
};

struct Shared {
    unsigned long long key[GROUP][GT / 32];
    uint32_t above[GROUP][HQ_MAX_M / 32];  // the nodes on each row's path, without the root
    int32_t node[HQ_MAX_M], token[HQ_MAX_M];  // drafted tokens of this chunk
    int n;
};

// RULES: penalties or biases, which need the words in shared memory.
template <class T, class O, bool RULES>
__global__ void __launch_bounds__(GT) k_greedy(const GreedyArgs a, const int chunk, const int group) {
    extern __shared__ __align__(16) uint32_t s_word[];  // [chunk], then the place of a token's bias, plus one [chunk]
    __shared__ Shared s;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.z;
    int first, m;
    batch_rows(a.starts, b, a.rows, a.max_rows, first, m);
    const int r0 = blockIdx.y * group, r1 = r0 + group < m ? r0 + group : m;
    if (r0 >= m) return;
    const int lo = blockIdx.x * chunk, n = a.V - lo < chunk ? a.V - lo : chunk;
    const int slot = a.seqs ? a.seqs[b] : b;
    uint32_t *s_bias = s_word + chunk;
    float rep = 1.0f, pres = 0.0f, freq = 0.0f;
    bool use_rep = false, use_times = false;
    const float *bias = nullptr;
    if (RULES) {
        for (int i = tid; i < (n + 3) / 4; i += GT) reinterpret_cast<uint4 *>(s_word)[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) s.n = 0;
        const bool ruled = slot >= 0 && slot < a.rules.n_slots;
        use_rep = ruled && a.rules.repetition;
        use_times = ruled && (a.rules.presence || a.rules.frequency);
        if (use_rep) rep = a.rules.repetition[slot];
        if (ruled && a.rules.presence) pres = a.rules.presence[slot];
        if (ruled && a.rules.frequency) freq = a.rules.frequency[slot];
        int j0 = 0, j1 = 0;  // the slot's biases
        if (ruled && a.rules.bias_starts) {
            j0 = a.rules.bias_starts[slot];
            j1 = a.rules.bias_starts[slot + 1];
            if (j0 < 0 || j1 > a.rules.n_bias || j1 < j0) j0 = j1 = 0;
            bias = a.rules.bias_values + j0;
        }
        __syncthreads();
        if (use_rep || use_times) {
            if (a.history.tokens && slot < a.history.n_slots) {
                int len = a.history.len[slot];
                len = len < 0 ? 0 : len > a.history.cap ? a.history.cap : len;
                const int prompt = a.history.prompt ? a.history.prompt[slot] : 0;
                const int32_t *text = a.history.tokens + (size_t)slot * a.history.cap;
                auto count = [&](int32_t t, int p) {
                    const uint32_t d = (uint32_t)t - (uint32_t)lo;
                    if (d < (uint32_t)n) {
                        if (p >= prompt) atomicAdd(&s_word[d], 1u);
                        else atomicOr(&s_word[d], SEEN);
                    }
                };
                int p = 0;
                if ((reinterpret_cast<uintptr_t>(text) & 15) == 0) {
                    const int4 *q = reinterpret_cast<const int4 *>(text);
#pragma unroll 4
                    for (int i = tid; i < len / 4; i += GT) {
                        const int4 t = q[i];
                        count(t.x, 4 * i);
                        count(t.y, 4 * i + 1);
                        count(t.z, 4 * i + 2);
                        count(t.w, 4 * i + 3);
                    }
                    p = len / 4 * 4;
                }
#pragma unroll 4
                for (int i = p + tid; i < len; i += GT) count(text[i], i);
            }
            if (a.tokens) {
                for (int i = 1 + tid; i < m; i += GT) {
                    const int32_t t = a.tokens[first + i];
                    const uint32_t d = (uint32_t)t - (uint32_t)lo;
                    if (d < (uint32_t)n) {
                        const int at = atomicAdd(&s.n, 1);  // (any order: the entries are counted)
                        s.node[at] = i;
                        s.token[at] = t;
                        atomicOr(&s_word[d], DRAFTED);
                    }
                }
                for (int r = r0 + warp; r < r1; r += GT / 32) {
                    int up[HQ_MAX_M / 32];
                    uint32_t on[HQ_MAX_M / 32];
#pragma unroll
                    for (int k = 0; k < HQ_MAX_M / 32; ++k) {
                        const int i = lane + 32 * k;
                        up[k] = i > r ? -1 : a.parent ? a.parent[first + i] : i - 1;
                        on[k] = 0;
                    }
                    for (int node = r; node > 0;) {
                        int p = up[0];
#pragma unroll
                        for (int k = 0; k < HQ_MAX_M / 32; ++k) {
                            if ((node >> 5) == k) {
                                p = up[k];
                                on[k] |= 1u << (node & 31);
                            }
                        }
                        p = __shfl_sync(0xffffffffu, p, node & 31);
                        if (p < 0 || p >= node) break;
                        node = p;
                    }
                    if (lane == 0) {
#pragma unroll
                        for (int k = 0; k < HQ_MAX_M / 32; ++k) s.above[r - r0][k] = on[k];
                    }
                }
            }
        }
        for (int j = j0 + tid; j < j1; j += GT) {
            const uint32_t d = (uint32_t)a.rules.bias_tokens[j] - (uint32_t)lo;
            if (d < (uint32_t)n) s_bias[d] = 0;
        }
        __syncthreads();
        for (int j = j0 + tid; j < j1; j += GT) {
            const uint32_t d = (uint32_t)a.rules.bias_tokens[j] - (uint32_t)lo;
            if (d < (uint32_t)n) {
                atomicMax(&s_bias[d], (uint32_t)(j - j0 + 1));  // of a token listed twice the last one
                atomicOr(&s_word[d], BIASED);
            }
        }
        __syncthreads();
    }

    // a logit that a rule reaches
    auto adjust = [&](float l, uint32_t word, int d, int r) {
        int times = (int)(word & TIMES);
        if (word & DRAFTED)
            for (int i = 0; i < s.n; ++i)
                if (s.token[i] == lo + d && (s.above[r - r0][s.node[i] >> 5] >> (s.node[i] & 31) & 1u)) ++times;
        if (use_rep && (times > 0 || (word & SEEN))) l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
        if (use_times && times > 0) {
            if (a.rules.frequency) l = __fsub_rn(l, __fmul_rn(freq, (float)times));
            if (a.rules.presence) l = __fsub_rn(l, pres);
        }
        if (word & BIASED) l = __fadd_rn(l, bias[s_bias[d] - 1]);
        return l;
    };

    for (int r = r0; r < r1; ++r) {
        const int row = first + r;
        const T *x = static_cast<const T *>(a.logits) + (size_t)row * (size_t)a.ldl + lo;
        O *out = a.out ? static_cast<O *>(a.out) + (size_t)row * (size_t)a.ldo + lo : nullptr;
        const uint32_t *mask = nullptr;
        if (a.rules.masks) {
            const int id = a.mask_ids ? a.mask_ids[row] : row;
            if (id >= 0 && id < a.rules.n_masks) mask = a.rules.masks + (size_t)id * (size_t)a.rules.ldmask + (lo >> 5);
        }
        float best = -INFINITY;
        int token = -1;
        auto take = [&](float l, int d) {  // d grows
            if (token < 0 || l > best || (l != l && best == best)) {
                best = l;
                token = lo + d;
            }
        };
        auto one = [&](int d) {
            float l = to_f32(x[d]);
            if (RULES && s_word[d]) l = adjust(l, s_word[d], d, r);
            const bool allowed = !mask || (mask[d >> 5] >> (d & 31) & 1u);
            if (!allowed) l = -INFINITY;
            if (out) out[d] = from_f32<O>(l);
            if (allowed) take(l, d);
        };
        if ((reinterpret_cast<uintptr_t>(x) & (4 * sizeof(T) - 1)) == 0) {
            const bool whole = out && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(O) - 1)) == 0;
            for (int q0 = tid; q0 < n / 4; q0 += 4 * GT) {
                Quad<T> v[4];
                uint32_t bits[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int q = q0 + k * GT;
                    bits[k] = 0xffffffffu;
                    if (q < n / 4) {
                        v[k] = reinterpret_cast<const Quad<T> *>(x)[q];
                        if (mask) bits[k] = mask[q >> 3] >> (4 * (q & 7));
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int q = q0 + k * GT, d = 4 * q;
                    if (q >= n / 4) break;
                    float l[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) l[e] = to_f32(v[k].x[e]);
                    if (RULES) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(s_word + d);
                        if (w.x | w.y | w.z | w.w) {
                            const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (word[e]) l[e] = adjust(l[e], word[e], d + e, r);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(bits[k] >> e & 1u)) l[e] = -INFINITY;
                    if (out) {
                        Quad<O> o;
#pragma unroll
                        for (int e = 0; e < 4; ++e) o.x[e] = from_f32<O>(l[e]);
                        if (whole) {
                            reinterpret_cast<Quad<O> *>(out)[q] = o;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) out[d + e] = o.x[e];
                        }
                    }
                    const float top = max_nan2(max_nan2(l[0], l[1]), max_nan2(l[2], l[3]));
                    if (token < 0 || !(top <= best)) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (bits[k] >> e & 1u) take(l[e], d + e);
                    }
                }
            }
            for (int d = n / 4 * 4 + tid; d < n; d += GT) one(d);
        } else {
#pragma unroll 4
            for (int d = tid; d < n; d += GT) one(d);
        }
        unsigned long long key = key_of(best, token);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
            key = other > key ? other : key;
        }
        if (lane == 0) s.key[r - r0][warp] = key;
    }
    __syncthreads();
    if (tid < r1 - r0) {
        const int row = first + r0 + tid;
        unsigned long long key = s.key[tid][0];
#pragma unroll
        for (int i = 1; i < GT / 32; ++i) key = s.key[tid][i] > key ? s.key[tid][i] : key;
        if (gridDim.x > 1) {
            atomicMax(&a.best[row], key);
            __threadfence();
            if (atomicInc(&a.done[row], gridDim.x - 1) != gridDim.x - 1) return;  // (the last one sets it to 0)
            __threadfence();
            key = atomicExch(&a.best[row], 0ull);
        }
        a.greedy[row] = token_of(key);
    }
}

template <class T, class O>
cudaError_t launch_t(const GreedyArgs &a, bool pdl, cudaStream_t s) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    int dev = 0, ready = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<int> set[CACHE_DEVICES];
    e = cached_per_device(set, dev, &ready, [&](int *v) {
        *v = 0;
        return cudaFuncSetAttribute(k_greedy<T, O, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST * 4);
    });
    if (e != cudaSuccess) return e;
    const bool biased = a.rules.n_slots > 0 && a.rules.bias_starts && a.rules.n_bias > 0;
    const bool penalties = a.rules.n_slots > 0 && (a.rules.repetition || a.rules.presence || a.rules.frequency) &&
                           (a.history.tokens || a.tokens);
    const int group = a.max_rows < GROUP ? a.max_rows : GROUP, groups = (a.max_rows + group - 1) / group;
    int chunk = biased ? MOST / 2 : MOST;
    while (chunk > LEAST && (long long)a.B * groups * ((a.V + chunk - 1) / chunk) < 4ll * sms) chunk /= 2;
    const dim3 grid((unsigned)((a.V + chunk - 1) / chunk), (unsigned)groups, (unsigned)a.B);
    if (biased || penalties)
        return launch_kernel(k_greedy<T, O, true>, grid, dim3(GT), (size_t)chunk * (biased ? 8 : 4), pdl, s, a, chunk, group);
    return launch_kernel(k_greedy<T, O, false>, grid, dim3(GT), 0, pdl, s, a, chunk, group);
}

}  // namespace

cudaError_t launch_greedy_tokens(const GreedyArgs &a, bool pdl, cudaStream_t s) {
    if (a.type == HQ_F32) return launch_t<float, float>(a, pdl, s);
    if (a.type == HQ_F16)
        return a.out && a.out_type == HQ_F32 ? launch_t<__half, float>(a, pdl, s) : launch_t<__half, __half>(a, pdl, s);
    return a.out && a.out_type == HQ_F32 ? launch_t<__nv_bfloat16, float>(a, pdl, s)
                                         : launch_t<__nv_bfloat16, __nv_bfloat16>(a, pdl, s);
}

}  // namespace hq
