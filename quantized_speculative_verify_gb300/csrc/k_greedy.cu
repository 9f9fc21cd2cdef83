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
// some rows of one sequence.  In shared memory it makes a table of the tokens of
// its chunk that a rule reaches, once for its rows: a word a token (seen, biased,
// drafted, how often behind the prompt), a bit a token, and a list of them in
// order.  Meanwhile the logits are on their way into the threads' registers, eight
// a load, asked for before anything else (the next row's before this one is looked
// at); the list's take no part in their maximum, by their bits.  All the code for
// the rules is in a pass over the list after that.  What a row's own path adds to
// the table is the drafted tokens of its ancestors, at most 127 and looked for only
// at tokens that are marked as drafted.
//
// A block is a chain of waits (its sequence, the history's length, the history, the
// list's logits, the ticket at the end), 6 us of them for 16 KB of logits, so the
// chunks are small enough for six blocks an SM.  Frequent tokens have low
// numbers: the first chunks' lists are far longer than the others', and their
// blocks come first in the grid.
//
// V = 151552, fp32: one row 7.1 us (a chain; the rules at each logit, without a table,
// took 6.0 for it), eight trees of up to 16 nodes with masks and biases 30 us (57 MB),
// 128 rows with histories of 16000 tokens, adjusted logits kept, 61 us (162 MB, 2.7
// TB/s).  Histories are sorted first in the last two.  What bounds them is instructions
// and waits about alike (41 and 46 % of the issue slots; 1300 and 1600 instructions a
// warp, 200 of them for its logits).  Without rules the trees take 14 us, with masks
// alone 21.  On the way there (trees, 128 rows): the rules at each logit 80 and 115 us; the table and its list 30 and 73, with chunks of 8192 and each
// block reading the whole history; logits in a ring in shared memory 38 and 124 (it
// leaves room for two blocks an SM); a table by rank for 1024 tokens at a time 33 and
// 118 (the first chunk's block takes 70); this, with the histories sorted, 30 and 67;
// the stream before the list and a sort that stores in rows, 30 and 61.
//
// Every chunk's block would read the whole history of its sequence.  Where that
// adds up, a kernel in front sorts the histories by chunk into the workspace.
//
// Of a slot's biases a block keeps those of its chunk, up to 128; where there are
// more, another pass over the slot's list finds each token's last one.  So a block's
// work grows with the list and not with its square: one row of 151552 with 300 biases
// next to one another 8.3 us (a walk through the list for each: 33), with 5000
// anywhere 16.5, with one for every token 0.34 ms (70).
//
// The order of values is that of a signed integer (a float's bits, the lower 31
// inverted where it is negative; NaN above all), so the largest of a warp is one
// instruction.  A thread keeps its largest value and where the eight logits with
// it lie; which of them it was is looked up once a row and block.  Chunks meet by
// the maximum of 64-bit keys (value, then the lowest token), which does not depend
// on the order; the last one writes the token and leaves its words as it found
// them.
#include <climits>
#include <type_traits>

#include "batch.cuh"

namespace hq {
namespace {

constexpr int GT = 128;          // threads
constexpr int GROUP = 4;         // rows of a sequence that share one table
constexpr int MOST = 4096, LEAST_SHIFT = 10;  // tokens of a chunk, a power of two: at most 4096, at least 2^10
constexpr int EIGHTS = MOST / 8 / GT;     // loads of a thread for a row
constexpr int FLIGHT = 4;        // loads of the history of a thread on their way together
constexpr int BIASES = 128;      // biases of a chunk that are kept; with more, a place for each of
constexpr int LASTS = MOST / 2;  // so many tokens at a time
constexpr uint32_t SEEN = 1u << 31, BIASED = 1u << 30, DRAFTED = 1u << 29, TIMES = DRAFTED - 1;

// The largest value; NaN (one pattern of it) if one is.
__device__ __forceinline__ float max_nan2(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}
__device__ __forceinline__ float max_nan3(float x, float y, float w) {
    float z;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(z) : "f"(x), "f"(y), "f"(w));
    return z;
}
// The order of values, NONE below all; NaN as max_nan2 gives it.
constexpr int NONE = INT_MIN;
__device__ __forceinline__ int order_of(float x) {
    const int i = __float_as_int(x + 0.0f);  // (-0 is 0)
    return i ^ ((i >> 31) & 0x7fffffff);
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

// Eight values, 16 bytes at a time.
template <class T>
struct alignas(16) Oct {
    T x[8];
};
template <class T>
__device__ __forceinline__ void load(const T *p, Oct<T> &v) {
#pragma unroll
    for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i) reinterpret_cast<uint4 *>(&v)[i] = reinterpret_cast<const uint4 *>(p)[i];
}
template <class T>
__device__ __forceinline__ void store(T *p, const Oct<T> &v) {
#pragma unroll
    for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(&v)[i];
}

// The workspace: a record for each row (its largest key so far, how many chunks are
// in it) and, in the first SORT_MOST records, a sequence's sorted history.  A
// record's place depends on its number alone, so calls of different sizes share a
// workspace without meeting one another's leavings.
constexpr int SORTED = 16384, CHUNKS = 64;
constexpr int SORT_MOST = 256;  // sequences
constexpr size_t RECORD = 16 + (SORTED + CHUNKS) * 4;
__host__ __device__ inline size_t record_at(int i) {
    return i < SORT_MOST ? i * RECORD : SORT_MOST * RECORD + (size_t)(i - SORT_MOST) * 16;
}

struct Shared {
    uint32_t word[MOST];            // what reaches each token
    uint32_t bits[MOST / 32 + 4];   // (one more for reads across the last one's end)
    union {
        uint16_t list[MOST];
        int32_t last[LASTS];        // with more than BIASES biases: each token's last one
    };
    int32_t bias_at[BIASES];        // biases of this chunk: their number in the slot's list, their token
    uint16_t bias_of[BIASES];
    int order[GROUP][GT / 32], at[GROUP][GT / 32];  // of each warp, of the logits that stream
    int list_order[GROUP][GT / 32], list_at[GROUP][GT / 32];  // and of the list
    int mask_id[GROUP];
    uint32_t above[GROUP][HQ_MAX_M / 32];  // the nodes on each row's path, without the root
    int32_t node[HQ_MAX_M], token[HQ_MAX_M];  // drafted tokens of this chunk
    int n_drafted, n_biased, counts[GT / 32];
};

// Bits d .. d + 7 of a bit field; s = d % 8, the same for all of a row's loads.
__device__ __forceinline__ uint32_t eight_bits(const uint32_t *words, int d, int s) {
    const uint8_t *p = reinterpret_cast<const uint8_t *>(words) + (d >> 3);
    uint32_t w = p[0];
    if (s != 0) w = ((w | (uint32_t)p[1] << 8) >> s) & 0xffu;
    return w;
}

// Histories sorted by chunk.  Of each sequence the first SORTED tokens: which chunk
// they are of, counted by each lane for itself (64 counters a chunk next to one
// another: a third of a text lies in one chunk, and no two lanes of a warp meet at a
// counter or a bank), then each token's place.  A token
// of the prompt has its top bit set.
//
// Worth it where all blocks together would otherwise read more than SORT_FROM bytes
// of what it sorts; the host knows the histories' room, not their lengths, and goes by
// that.  Without and with it, full rooms, V = 151552: 128 rows with 16000 tokens each,
// kept (289 MB), 102 and 56 us, with 500 (9 MB) 52 and 48; 64 with 4000 (36 MB) 31.6 and
// 26.0; eight trees with all rules and 2000 (18 MB) 30.6 and 30.5.  V = 32000: 128 with 4000
// (16 MB) 20.0 and 18.0, with 2000 (8 MB) 16.6 and 17.3; 32 with 4000 (16 MB) 17.5 and
// 15.1; 8 with 16000 (16 MB) 18.5 and 19.0; one with 16000 (2 MB) 18.5 and 19.8.  In rooms
// of 131072, V = 32000, a tree of 16 nodes with 500 tokens 9.25 and 9.8, with 16000 20.7
// and 19.6 (by the room 32 MB: sorted); one row with 500 7.3 and 9.3 (2 MB: not).
//
// It has its limits: 256 sequences; 63 chunks, so no vocabulary from 258049 tokens on
// (128 rows of 262144 76 us with 500 tokens each, 153 with 16000) and, as few rows have
// smaller chunks, with V = 151552 no call of 16 rows or fewer (a tree of 16 nodes with
// 16000 tokens 35 us); and of a longer text every block reads the tokens past the
// first SORTED (16 rows of 32000 with 60000 tokens 49 us).
constexpr int ST = 1024;
constexpr long long SORT_FROM = 12ll << 20;
__global__ void __launch_bounds__(ST) k_sort_history(const GreedyArgs a, const int shift, const int chunks) {
    extern __shared__ __align__(16) int32_t s_sorted[];  // [SORTED]
    __shared__ int s_count[CHUNKS][64];
    __shared__ int s_start[CHUNKS + 1];
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, mine = tid & 63;
    const int slot = a.seqs ? a.seqs[b] : b;
    int len = 0, prompt = 0;
    if (slot >= 0 && slot < a.history.n_slots) {
        len = a.history.len[slot];
        if (a.history.prompt) prompt = a.history.prompt[slot];
    }
    len = len < 0 ? 0 : len > a.history.cap ? a.history.cap : len;
    if (len > SORTED) len = SORTED;
    const int32_t *text = a.history.tokens + (size_t)(len > 0 ? slot : 0) * a.history.cap;
    int32_t t[SORTED / ST];
    int place[SORTED / ST];
#pragma unroll
    for (int k = 0; k < SORTED / ST; ++k) t[k] = k * ST + tid < len ? text[k * ST + tid] : -1;
    for (int i = tid; i < CHUNKS * 64; i += ST) (&s_count[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SORTED / ST; ++k)
        if (t[k] >= 0 && t[k] < a.V) place[k] = atomicAdd(&s_count[t[k] >> shift][mine], 1);
    __syncthreads();
    for (int c = warp; c < chunks; c += ST / 32) {  // each counter's first place in its chunk, from the chunk's start
        const int x = s_count[c][2 * lane], y = s_count[c][2 * lane + 1];
        int n = x + y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += z;
        }
        s_count[c][2 * lane] = n - x - y;
        s_count[c][2 * lane + 1] = n - y;
        if (lane == 31) s_start[c + 1] = n;
    }
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        if (tid == 0) s_start[0] = 0;
        for (int i = tid; i - tid < chunks; i += 32) {
            int x = i < chunks ? s_start[i + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += y;
            }
            if (i < chunks) s_start[i + 1] = x + carry;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    int32_t *sorted = reinterpret_cast<int32_t *>(a.workspace + record_at(b) + 16);
    if (tid <= chunks && tid < CHUNKS) sorted[SORTED + tid] = s_start[tid];
#pragma unroll
    for (int k = 0; k < SORTED / ST; ++k)
        if (t[k] >= 0 && t[k] < a.V)
            s_sorted[s_start[t[k] >> shift] + s_count[t[k] >> shift][mine] + place[k]] =
                t[k] | (k * ST + tid < prompt ? (int32_t)0x80000000 : 0);
    // (stored from there in rows: 16000 stores to places of their own take 8 us)
    __syncthreads();
    for (int i = tid; i < s_start[chunks]; i += ST) sorted[i] = s_sorted[i];
}

// RULES: penalties or biases, which need the table.  MANY: a slot may have more than
// BIASES of them (else their code is left out: the chain of one row waits for its
// instructions too, 7.1 us without it and 7.35 with it).  sorted: the histories are.
template <class T, class O, bool RULES, bool MANY = false>
__global__ void __launch_bounds__(GT, 6) k_greedy(const GreedyArgs a, const int chunk, const int group, const bool sorted) {
    __shared__ __align__(16) Shared s;
    pdl_launch_dependents();
    // The sorting kernel starts this one after its own wait, so that all but its
    // result is there already.
    if (!sorted) pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int groups = (a.max_rows + group - 1) / group, b = blockIdx.x / groups;
    int first, m;
    batch_rows(a.starts, b, a.rows, a.max_rows, first, m);
    const int slot = a.seqs ? a.seqs[b] : b;
    const int r0 = blockIdx.x % groups * group, r1 = r0 + group < m ? r0 + group : m;
    if (r0 >= m) {
        if (sorted) pdl_wait();
        return;
    }
    const int lo = blockIdx.y * chunk, n = a.V - lo < chunk ? a.V - lo : chunk;
    auto logits_of = [&](int row) { return static_cast<const T *>(a.logits) + (size_t)row * (size_t)a.ldl + lo; };
    // A row's logits up to the first aligned eight, the eights, the rest.
    auto head_of = [&](const T *x) {
        const int off = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (16 / (int)sizeof(T) - 1);
        const int head = off == 0 ? 0 : 16 / (int)sizeof(T) - off;
        return head < n ? head : n;
    };
    Oct<T> v[EIGHTS];
    auto fetch = [&](int r) {
        const T *x = logits_of(first + r);
        const int head = head_of(x), eights = (n - head) / 8;
#pragma unroll
        for (int k = 0; k < EIGHTS; ++k)
            if (tid + k * GT < eights) load(x + head + 8 * (tid + k * GT), v[k]);
    };
    fetch(r0);
    if (a.rules.masks && tid < r1 - r0) s.mask_id[tid] = a.mask_ids ? a.mask_ids[first + r0 + tid] : first + r0 + tid;
    auto out_of = [&](int row) { return a.out ? static_cast<O *>(a.out) + (size_t)row * (size_t)a.ldo + lo : nullptr; };
    auto mask_of = [&](int r) -> const uint32_t * {
        if (!a.rules.masks) return nullptr;
        const int id = s.mask_id[r - r0];
        return id >= 0 && id < a.rules.n_masks ? a.rules.masks + (size_t)id * (size_t)a.rules.ldmask + (lo >> 5) : nullptr;
    };
    float rep = 1.0f, pres = 0.0f, freq = 0.0f;
    bool use_rep = false, use_times = false;
    int listed_tokens = 0, first_bias = 0, last_bias = 0;
    bool many_biases = false;
    // The tokens of the list from i0 to i1, for all rows: the block's warps take the
    // rows in turn.  by_token: the tokens themselves, those of the bit field, with
    // their last biases in s.last.
    auto for_list = [&](auto by_token, int i0, int i1) {
        const int share = GT / 32 / (r1 - r0), r = r0 + warp / share;
        if (r >= r1) return;
        const T *x = logits_of(first + r);
        O *out = out_of(first + r);
        const uint32_t *mask = mask_of(r);
        int best = NONE, at = INT_MAX;
        for (int i = i0 + warp % share * 32 + lane; i < i1; i += 32 * share) {
            const int d = by_token ? i : s.list[i];
            if (by_token && !(s.bits[d >> 5] >> (d & 31) & 1u)) continue;
            const uint32_t word = s.word[d];
            const bool allowed = !mask || (mask[d >> 5] >> (d & 31) & 1u);
            float l = to_f32(x[d]);
            int times = (int)(word & TIMES);
            if (word & DRAFTED) {
                for (int t = 0; t < s.n_drafted; ++t)
                    if (s.token[t] == lo + d && (s.above[r - r0][s.node[t] >> 5] >> (s.node[t] & 31) & 1u)) ++times;
            }
            if (use_rep && (times > 0 || (word & SEEN))) l = l > 0.0f ? __fdiv_rn(l, rep) : __fmul_rn(l, rep);
            if (use_times && times > 0) {
                if (a.rules.frequency) l = __fsub_rn(l, __fmul_rn(freq, (float)times));
                if (a.rules.presence) l = __fsub_rn(l, pres);
            }
            if (word & BIASED) {  // of a token listed twice the last one
                int j = by_token ? s.last[i - i0] : 0;
                if (!by_token) {
                    for (int t = 0; t < s.n_biased; ++t)
                        if (s.bias_of[t] == d && s.bias_at[t] > j) j = s.bias_at[t];
                }
                l = __fadd_rn(l, a.rules.bias_values[j]);
            }
            if (!allowed) l = -INFINITY;
            if (out) out[d] = from_f32<O>(l);
            const int o = order_of(max_nan2(l, l));
            if (allowed && o > best) {  // (d grows)
                best = o;
                at = d;
            }
        }
        const int most = __reduce_max_sync(0xffffffffu, best);
        at = __reduce_min_sync(0xffffffffu, best == most ? at : INT_MAX);
        if (lane == 0 && (!by_token || most > s.list_order[r - r0][warp])) {
            s.list_order[r - r0][warp] = most;
            s.list_at[r - r0][warp] = at;
        }
    };
    // The same where a chunk has many biases, LASTS tokens at a time: the last bias of
    // each by another pass over the slot's (j0 .. j1).  Every thread calls.
    auto for_tokens = [&](int j0, int j1) {
        for (int from = 0; from < n; from += LASTS) {
            const int to = from + LASTS < n ? from + LASTS : n;
            for (int i = tid; i < to - from; i += GT) s.last[i] = 0;
            __syncthreads();
            for (int j = j0 + tid; j < j1; j += GT) {
                const int32_t t = a.rules.bias_tokens[j];
                if (t >= lo + from && t < lo + to) atomicMax(&s.last[t - lo - from], j);
            }
            __syncthreads();
            for_list(std::true_type{}, from, to);
            __syncthreads();
        }
    };
    if (RULES) {
        const bool ruled = slot >= 0 && slot < a.rules.n_slots;
        use_rep = ruled && a.rules.repetition;
        use_times = ruled && (a.rules.presence || a.rules.frequency);
        const bool told = (use_rep || use_times) && a.history.tokens && slot < a.history.n_slots;
        const bool drafts = (use_rep || use_times) && a.tokens;
        int len = 0, prompt = 0, j0 = 0, j1 = 0;  // j0 .. j1: the slot's biases
        if (told) {
            len = a.history.len[slot];
            if (a.history.prompt) prompt = a.history.prompt[slot];
        }
        if (ruled && a.rules.bias_starts) {
            j0 = a.rules.bias_starts[slot];
            j1 = a.rules.bias_starts[slot + 1];
        }
        if (use_rep) rep = a.rules.repetition[slot];
        if (ruled && a.rules.presence) pres = a.rules.presence[slot];
        if (ruled && a.rules.frequency) freq = a.rules.frequency[slot];
        static_assert(GT >= HQ_MAX_M && GT / 32 >= GROUP, "a thread per node, a warp per row");
        const int32_t draft = drafts && tid > 0 && tid < m ? a.tokens[first + tid] : -1;
        int up[HQ_MAX_M / 32];  // of the nodes up to this warp's row, four a lane
        if (drafts && r0 + warp < r1) {
#pragma unroll
            for (int k = 0; k < HQ_MAX_M / 32; ++k) {
                const int i = lane + 32 * k;
                up[k] = i > r0 + warp ? -1 : a.parent ? a.parent[first + i] : i - 1;
            }
        }
        for (int i = tid; i < (n + 3) / 4; i += GT) reinterpret_cast<uint4 *>(s.word)[i] = make_uint4(0, 0, 0, 0);
        for (int i = tid; i < (n + 31) / 32 + 1; i += GT) s.bits[i] = 0;
        if (tid == 0) s.n_drafted = s.n_biased = 0;
        if (tid < GROUP * (GT / 32)) (&s.list_order[0][0])[tid] = NONE;
        len = len < 0 ? 0 : len > a.history.cap ? a.history.cap : len;
        if (j0 < 0 || j1 > a.rules.n_bias || j1 < j0) j0 = j1 = 0;
        const int32_t *text = a.history.tokens + (size_t)(told ? slot : 0) * a.history.cap;
        const int4 *text4 = reinterpret_cast<const int4 *>(text);
        const int from = sorted ? SORTED : 0;  // where the tokens that are read from there begin
        const int fours = told && !sorted && (reinterpret_cast<uintptr_t>(text) & 15) == 0 ? len / 4 : 0;
        const int4 none = make_int4(-1, -1, -1, -1);
        int4 t4[FLIGHT];
#pragma unroll
        for (int k = 0; k < FLIGHT; ++k) t4[k] = tid + k * GT < fours ? text4[tid + k * GT] : none;
        const int32_t biased = j0 + tid < j1 ? a.rules.bias_tokens[j0 + tid] : -1;
        if (drafts && r0 + warp < r1) {
            uint32_t on[HQ_MAX_M / 32] = {};
            for (int node = r0 + warp; node > 0;) {
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
                for (int k = 0; k < HQ_MAX_M / 32; ++k) s.above[warp][k] = on[k];
            }
        }
        __syncthreads();
        if (sorted) pdl_wait();
        const int32_t *mine = reinterpret_cast<const int32_t *>(a.workspace + record_at(b) + 16);
        const int mine0 = sorted && told ? mine[SORTED + blockIdx.y] : 0, mine1 = sorted && told ? mine[SORTED + blockIdx.y + 1] : 0;
        const uint32_t bits = smem_addr(s.bits), word = smem_addr(s.word);
        // A rule reaches a token: `how` is set; or it is in the history, and SEEN is set or
        // one time more is counted.  Without branches: in most warps some lane's token is
        // in the chunk.
        auto mark = [bits, word, lo, n](int32_t t, uint32_t how) {
            const uint32_t d = (uint32_t)t - (uint32_t)lo;
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\t@p red.shared.or.b32 [%2], %3;\n\t@p red.shared.or.b32 [%4], %5;\n\t}" ::"r"(d),
                "r"(n), "r"(word + 4 * d), "r"(how), "r"(bits + (d >> 3 & ~3u)), "r"(1u << (d & 31))
                : "memory");
        };
        auto told_of = [bits, word, lo, n](int32_t t, bool prompts) {
            const uint32_t d = (uint32_t)t - (uint32_t)lo;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.lt.u32 p, %0, %1;\n\tsetp.ne.and.u32 q, %6, 0, p;\n\t@q red.shared.or.b32 [%2], %3;\n\t"
                "setp.eq.and.u32 q, %6, 0, p;\n\t@q red.shared.add.u32 [%2], 1;\n\t@p red.shared.or.b32 [%4], %5;\n\t}" ::"r"(d),
                "r"(n), "r"(word + 4 * d), "r"(SEEN), "r"(bits + (d >> 3 & ~3u)), "r"(1u << (d & 31)), "r"((uint32_t)prompts)
                : "memory");
        };
        for (int i0 = tid; fours > 0;) {
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int at = 4 * (i0 + k * GT);
                told_of(t4[k].x, at < prompt);
                told_of(t4[k].y, at + 1 < prompt);
                told_of(t4[k].z, at + 2 < prompt);
                told_of(t4[k].w, at + 3 < prompt);
            }
            i0 += FLIGHT * GT;
            if (i0 >= fours) break;
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) t4[k] = i0 + k * GT < fours ? text4[i0 + k * GT] : none;
        }
        for (int i0 = from + 4 * fours + tid; i0 < len; i0 += 2 * FLIGHT * GT) {
            int32_t t[2 * FLIGHT];
#pragma unroll
            for (int k = 0; k < 2 * FLIGHT; ++k) t[k] = i0 + k * GT < len ? text[i0 + k * GT] : -1;
#pragma unroll
            for (int k = 0; k < 2 * FLIGHT; ++k) told_of(t[k], i0 + k * GT < prompt);
        }
        for (int i0 = mine0 + tid; i0 < mine1; i0 += FLIGHT * GT) {
            int32_t t[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) t[k] = i0 + k * GT < mine1 ? mine[i0 + k * GT] : 0x7fffffff;
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) told_of(t[k] & 0x7fffffff, t[k] < 0);
        }
        mark(draft, DRAFTED);
        if (draft >= lo && draft < lo + n) {
            const int at = atomicAdd(&s.n_drafted, 1);  // (any order: the entries are counted)
            s.node[at] = tid;
            s.token[at] = draft;
        }
        for (int j = j0 + tid; j < j1; j += GT) {
            const int32_t t = j == j0 + tid ? biased : a.rules.bias_tokens[j];
            mark(t, BIASED);
            if (t >= lo && t < lo + n) {
                const int at = atomicAdd(&s.n_biased, 1);
                if (at < BIASES) {
                    s.bias_at[at] = j;
                    s.bias_of[at] = (uint16_t)(t - lo);
                }
            }
        }
        __syncthreads();
        // the list: a word of bits a thread
        static_assert(MOST / 32 <= GT, "a word of bits a thread");
        uint32_t field = tid < (n + 31) / 32 ? s.bits[tid] : 0u;
        int before = __popc(field);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31) s.counts[warp] = before;
        before -= __popc(field);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < GT / 32; ++i) {
            if (i < warp) before += s.counts[i];
            listed_tokens += s.counts[i];
        }
        for (; field != 0; field &= field - 1) s.list[before++] = (uint16_t)(32 * tid + __ffs(field) - 1);
        many_biases = MANY && s.n_biased > BIASES;
        first_bias = j0;
        last_bias = j1;
        __syncthreads();  // the list is whole
    } else {
        __syncthreads();
    }
    // The logits that stream.
    auto stream = [&]() {
        for (int r = r0; r < r1; ++r) {
            const T *x = logits_of(first + r);
            O *out = out_of(first + r);
            const uint32_t *mask = mask_of(r);
            int best = NONE, at = INT_MAX;  // at: the first of the eight
            auto one = [&](int d) {         // a logit outside the aligned eights
                const bool listed = RULES && (s.bits[d >> 5] >> (d & 31) & 1u);
                const float l = to_f32(x[d]);
                const bool allowed = !mask || (mask[d >> 5] >> (d & 31) & 1u);
                if (out) out[d] = from_f32<O>(allowed ? l : -INFINITY);
                const int o = order_of(max_nan2(l, l));
                if (allowed && !listed && o > best) {
                    best = o;
                    at = d;
                }
            };
            const int head = head_of(x), eights = (n - head) / 8;
            const bool whole = out && (reinterpret_cast<uintptr_t>(out + head) & 15) == 0;
            uint32_t bits[EIGHTS];
#pragma unroll
            for (int k = 0; k < EIGHTS; ++k) {
                bits[k] = 0xffu;
                if (mask && tid + k * GT < eights) bits[k] = eight_bits(mask, head + 8 * (tid + k * GT), head & 7);
            }
            if (tid < head) one(tid);
#pragma unroll
            for (int k = 0; k < EIGHTS; ++k) {
                const int d = head + 8 * (tid + k * GT);
                if (tid + k * GT >= eights) break;
                const uint32_t listed = RULES ? eight_bits(s.bits, d, head & 7) : 0u;
                float l[8];
                if (out) {
                    Oct<O> o;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o.x[e] = from_f32<O>((bits[k] >> e & 1u) ? to_f32(v[k].x[e]) : -INFINITY);
                    if (whole) {
                        store(out + d, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) out[d + e] = o.x[e];
                    }
                }
                const uint32_t use = bits[k] & ~listed;
#pragma unroll
                for (int e = 0; e < 8; ++e) l[e] = (use >> e & 1u) ? to_f32(v[k].x[e]) : -INFINITY;
                const int o = order_of(max_nan3(max_nan3(l[0], l[1], l[2]), max_nan3(l[3], l[4], l[5]), max_nan2(l[6], l[7])));
                if (use != 0 && o > best) {
                    best = o;
                    at = d;
                }
            }
            if (r + 1 < r1) fetch(r + 1);
            const int d = head + 8 * eights + tid;
            if (d < n) one(d);
            const int most = __reduce_max_sync(0xffffffffu, best);
            at = __reduce_min_sync(0xffffffffu, best == most ? at : INT_MAX);
            if (lane == 0) {
                s.order[r - r0][warp] = most;
                s.at[r - r0][warp] = at;
            }
        }
    };
    // Where the logits are kept the stream comes first, with what the list is of, and
    // the list is written over it: one store of eight instead of one for each logit in
    // between (128 rows 64 us, else 67).  Where they are not, the list's loads come
    // first (eight trees 30 us, else 32).
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {
        if ((phase == 0) == (a.out != nullptr)) stream();
        else if (MANY && many_biases) for_tokens(first_bias, last_bias);
        else if (RULES && listed_tokens > 0) for_list(std::false_type{}, 0, listed_tokens);
        __syncthreads();
    }
    if (tid >= r1 - r0) return;
    const int row = first + r0 + tid;
    int best = NONE, at = INT_MAX;
#pragma unroll
    for (int i = 0; i < GT / 32; ++i) {
        const int o = s.order[tid][i], d = s.at[tid][i];
        if (o > best || (o == best && d < at)) {
            best = o;
            at = d;
        }
    }
    if (best != NONE) {  // which of the eight (a logit that was taken by itself is the first)
        const T *x = logits_of(row);
        const uint32_t *mask = mask_of(r0 + tid);
        float l[8];
        uint32_t use[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = at + e < n ? at + e : at;
            l[e] = to_f32(x[d]);
            use[e] = mask ? mask[d >> 5] >> (d & 31) & 1u : 1u;
            if (RULES) use[e] &= ~(s.bits[d >> 5] >> (d & 31));
        }
        int e = 0;
#pragma unroll
        for (int k = 7; k >= 0; --k)
            if ((use[k] & 1u) && order_of(max_nan2(l[k], l[k])) == best) e = k;
        at += e;
    }
    if (RULES && listed_tokens > 0) {
#pragma unroll
        for (int i = 0; i < GT / 32; ++i) {
            const int o = s.list_order[tid][i], d = s.list_at[tid][i];
            if (o > best || (o == best && d < at)) {
                best = o;
                at = d;
            }
        }
    }
    unsigned long long key = 0;  // below those of tokens
    if (best != NONE)
        key = ((unsigned long long)((uint32_t)best ^ 0x80000000u) << 32) | (0xFFFFFFFFu - (uint32_t)(lo + at));
    if (gridDim.y > 1) {
        // released by the ticket, which the last chunk acquires and sets to 0
        unsigned long long *most = reinterpret_cast<unsigned long long *>(a.workspace + record_at(row));
        unsigned before;
        asm volatile("red.relaxed.gpu.global.max.u64 [%0], %1;" ::"l"(most), "l"(key) : "memory");
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(before) : "l"(most + 1), "r"(gridDim.y - 1) : "memory");
        if (before != gridDim.y - 1) return;
        key = atomicExch(most, 0ull);
    }
    a.greedy[row] = key == 0ull ? -1 : (int)(0xFFFFFFFFu - (uint32_t)key);
}

template <class T, class O>
cudaError_t launch_t(const GreedyArgs &a, bool pdl, cudaStream_t s) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    const bool biased = a.rules.n_slots > 0 && a.rules.bias_starts && a.rules.n_bias > 0;
    const bool penalties = a.rules.n_slots > 0 && (a.rules.repetition || a.rules.presence || a.rules.frequency) &&
                           (a.history.tokens || a.tokens);
    // Chunks as large as leaves four blocks an SM, each row by itself (a token's row
    // of 151552 in chunks of 1024 7.2 us); then two or four rows of a sequence to a
    // block where there are more than 16 blocks an SM (eight trees of 16 nodes, V =
    // 151552, chunks of 4096: one row a block 42 us, two 29.5, four 31.6; five
    // sequences of 7 rows, V = 32003, chunks of 1024: 10.4, 12.0 and 14.7).
    int shift = LEAST_SHIFT;
    while ((1 << shift) < MOST && (long long)a.B * a.max_rows * ((a.V + (2 << shift) - 1) >> (shift + 1)) >= 4ll * sms) ++shift;
    const int chunk = 1 << shift, chunks = (a.V + chunk - 1) >> shift;
    int group = 1;
    while (group < GROUP && group < a.max_rows && (long long)a.B * ((a.max_rows + group - 1) / group) * chunks > 16ll * sms) group *= 2;
    const int groups = (a.max_rows + group - 1) / group;
    const dim3 grid((unsigned)(a.B * groups), (unsigned)chunks);
    if (!biased && !penalties)
        return launch_kernel(k_greedy<T, O, false>, grid, dim3(GT), 0, pdl, s, a, chunk, group, false);
    const bool sorted = penalties && a.history.tokens && a.B <= SORT_MOST && a.B <= a.rows && chunks < CHUNKS &&
                        4ll * (a.history.cap < SORTED ? a.history.cap : SORTED) * a.B * groups * chunks > SORT_FROM;
    if (sorted) {
        int dev = 0, ready = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        static std::atomic<int> set[CACHE_DEVICES];
        e = cached_per_device(set, dev, &ready, [](int *v) {
            *v = 0;
            return cudaFuncSetAttribute(k_sort_history, cudaFuncAttributeMaxDynamicSharedMemorySize, SORTED * 4);
        });
        if (e != cudaSuccess) return e;
        e = launch_kernel(k_sort_history, dim3((unsigned)a.B), dim3(ST), SORTED * 4, pdl, s, a, shift, chunks);
        if (e != cudaSuccess) return e;
    }
    const bool many = biased && a.rules.n_bias > BIASES;
    return launch_kernel(many ? k_greedy<T, O, true, true> : k_greedy<T, O, true>, grid, dim3(GT), 0, pdl || sorted, s, a, chunk, group,
                         sorted);
}

}  // namespace

size_t greedy_workspace_bytes(int rows) { return record_at(rows); }

cudaError_t launch_greedy_tokens(const GreedyArgs &a, bool pdl, cudaStream_t s) {
    if (a.type == HQ_F32) return launch_t<float, float>(a, pdl, s);
    if (a.type == HQ_F16)
        return a.out && a.out_type == HQ_F32 ? launch_t<__half, float>(a, pdl, s) : launch_t<__half, __half>(a, pdl, s);
    return a.out && a.out_type == HQ_F32 ? launch_t<__nv_bfloat16, float>(a, pdl, s)
                                         : launch_t<__nv_bfloat16, __nv_bfloat16>(a, pdl, s);
}

}  // namespace hq
