/*
 * hq.h -- C ABI of the quantized speculative-verify linear layer for GB300
 * (sm_103a).
 *
 * The layer is the target model's linear layer in the verification pass of
 * speculative decoding: M drafted tree tokens (M = 1..128 rows) go through
 *   1. a block-diagonal randomized Hadamard rotation (blocks of 32, seeded
 *      +-1 sign flips, one overall scale 1/sqrt(32)) and per-row int8
 *      quantization of the activations, computed on the fly;
 *   2. an integer GEMM against weights that were rotated with the same
 *      transform and quantized offline, either to 4-bit asymmetric grouped
 *      integers ("Medium") or to 8-bit symmetric grouped integers ("Large");
 *   3. a per-group fp32 dequantization epilogue.
 * Source: page "Karpathy's Trick for Faster Local LLMs Finally Has Proper
 * Tooling" (blog.dailydoseofds.com): section "How Uzu optimizes bytes and
 * tokens per pass" (the two weight formats, 8-bit activations on the fly,
 * int8 matrix path, 32-block randomized Hadamard transform, transform block
 * independent of the quantization group) and section "Producing several
 * tokens from one model pass" (the verify batch is the 16-32 token draft
 * tree, "16 rows of work instead of 1").
 *
 * After the verify pass, the same library accepts the draft tree
 * (hq_tree_accept) and runs the two stateful layer kinds of the verified model
 * over the tree without changing their committed state, then commits the
 * accepted path: tree-masked attention over a KV cache (hq_tree_attention,
 * hq_tree_commit_kv) and the gated delta-rule DeltaNet layer (hq_delta_tree,
 * hq_delta_commit).  Source: the same page, section "Verifying a draft tree
 * without restoring model state".
 *
 * For a batch of requests there are the residual addition and norm in front of
 * a layer (hq_add_norm_quant), low-rank adapters beside it (hq_lora_apply), a
 * paged key/value cache (hq_pages_*), rotary positions on the way into it
 * (hq_rope_write), attention over it that reads a shared prefix once
 * (hq_prefix_attention), the gated norm behind a layer's core
 * (hq_gated_norm_quant), rules on the logits (hq_greedy_tokens) and the
 * acceptance of all trees at once (hq_tree_accept_batch).
 *
 * Conventions
 *   - Row-major everywhere.  X is [M][K], W is [N][K], Y = X W^T is [M][N].
 *   - Pointers are DEVICE pointers unless their name ends in _host.  The
 *     caller owns and allocates every buffer; the library allocates no
 *     memory and keeps no per-call state.
 *   - Every call that takes a `stream` (a cudaStream_t, NULL = legacy default
 *     stream) only enqueues work and returns without synchronizing.
 *   - Arguments are validated before anything is launched.  A call that
 *     returns an error launched nothing, except HQ_ERR_CUDA, which reports
 *     that the launch itself failed.  Faults of kernels that did launch show
 *     up, as always with CUDA, at the caller's next synchronization.
 *   - Calls are reentrant.  Two calls that share a workspace must not run
 *     concurrently (use one workspace per stream).
 */
#ifndef HQ_H
#define HQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    HQ_OK = 0,
    HQ_ERR_INVALID_ARG = 1, /* NULL pointer, bad size, misaligned pointer   */
    HQ_ERR_UNSUPPORTED = 2, /* valid request the library does not implement */
    HQ_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed          */
    HQ_ERR_TIMEOUT = 4,     /* a bounded device-side wait gave up            */
    HQ_ERR_NO_PAGES = 5     /* a page operation found too few free pages     */
} hq_status;

typedef enum {
    HQ_W4_ASYM = 0, /* "Medium": uint4 codes, fp32 scale + uint4 zero point per group */
    HQ_W8_SYM = 1   /* "Large":  int8 codes, fp32 scale per group                     */
} hq_format;

/* One linear layer.  K = input features (multiple of 32 and of `group`, at
 * most 65536), N = output features (>= 1), group = quantization group along
 * K, one of 16, 32, 64, 128, 256 (independent of the 32-element transform
 * block), format = hq_format.  The layer may have at most 2^30 weight tiles
 * of 128 output features x max(128, group) input features (a blob far larger
 * than any GPU memory); a descriptor beyond that is invalid. */
typedef struct {
    int32_t K;
    int32_t N;
    int32_t group;
    int32_t format;
} hq_layer_desc;

/* Launch flags. */
#define HQ_LAUNCH_DEFAULT 0u
/* Launch with programmatic dependent launch: the kernel may start while the
 * previous kernel of the stream is still running and waits for it (and for
 * its memory) before reading anything that kernel could have produced.
 * Some inputs are read before that wait, so with this flag they must not be
 * written by the operation launched immediately before in the same stream, nor,
 * where that one has the flag too, by the one before it, and so on back to the
 * last operation launched without it (an operation may let the next one start
 * before its own wait is over): the blob (hq_verify_gemm streams the packed weights early), the committed
 * cache positions [0, L) (hq_tree_attention), the committed state
 * (hq_delta_tree), weight and signs (hq_add_norm_quant), and ids, ranks, A and
 * B (hq_lora_apply). */
#define HQ_LAUNCH_PDL 1u
/* hq_verify_gemm only: combine the thread blocks that share an output in a
 * fixed order, so that results repeat bit for bit from run to run (the blocks
 * wait for one another before that sum; slower).  Without it, their fp32
 * partial sums are added into Y atomically as each block finishes, and the
 * last bits of such outputs may differ between runs. */
#define HQ_LAUNCH_DETERMINISTIC 2u
/* hq_verify_gemm only: no output's K range is split between thread blocks:
 * each thread block takes whole blocks of 128 output channels, so every
 * output is summed over its groups in ascending order by one thread block,
 * each product scale * P rounded and then added (the definition's
 * arithmetic), and is bit-identical to the sequential fp32 sum of the
 * definition (see hq_verify_gemm).  Without this flag (and without check-mode
 * partials) a group is folded with one fused multiply-add, one rounding
 * fewer per group.  Slower on layers with few 128-channel blocks (fewer
 * thread blocks than SMs); implies HQ_LAUNCH_DETERMINISTIC. */
#define HQ_LAUNCH_EXACT_ORDER 4u

/* Maximum number of token rows per call. */
#define HQ_MAX_M 128

/* Human-readable name of a status code (static string, never NULL). */
const char *hq_status_string(int status);

/* ABI version of this library: (major << 16) | minor. */
int32_t hq_version(void);

/* Size in bytes of the packed weight blob of `desc` (0 if desc is invalid).
 * The blob layout is private to the library; hq_unpack_codes gives the
 * canonical view. */
size_t hq_packed_bytes(const hq_layer_desc *desc);

/* Size in bytes of the workspace hq_verify_gemm needs for `desc` and M rows
 * (0 if the arguments are invalid).  The workspace holds the device error
 * word, the split-K partial sums (two slots of 128 channels x 128 rows per
 * thread block, up to 480 blocks: 60 MiB) and two counters per 128 output
 * channels, at offsets
 * that depend on neither the layer nor M: one workspace of the largest size
 * serves calls of every layer and M in turn (calls that may overlap on the
 * GPU need workspaces of their own).  It must be zero-filled once after
 * allocation; every call leaves the error word and the counters at zero
 * again (except after a time-out, see hq_workspace_status); the partial sums
 * need no clearing. */
size_t hq_workspace_bytes(const hq_layer_desc *desc, int32_t M);

/* Sign vector of the randomized Hadamard transform ("random sign flips
 * applied before the mixing", section "How Uzu optimizes bytes and tokens
 * per pass").  Host-only.  Feature k is negated when the top bit of the k-th
 * output of SplitMix64 (Steele, Lea & Flood 2014) seeded with `seed` is set;
 * the result is bit-packed: bit (k % 32) of signs_host[k / 32].
 * K must be a positive multiple of 32; signs_host has K/32 words.  The same
 * vector must be used for the weights and for the activations of a layer. */
int hq_make_signs(uint64_t seed, int32_t K, uint32_t *signs_host);

/* Offline: rotate, quantize and pack the weights of one layer (section "How
 * Uzu optimizes bytes and tokens per pass": Medium = 4-bit asymmetric,
 * Large = 8-bit symmetric, transform before quantization).
 *   W      fp32 [N][K], 16-byte aligned
 *   signs  uint32 [K/32] (device copy of hq_make_signs' output)
 *   blob   hq_packed_bytes(desc) bytes, 16-byte aligned, written in full
 * Per (output channel n, group g): Medium: lo = min(0, min w), hi = max(0,
 * max w), scale = (hi - lo) / 15, zero = rint(-lo / scale), code =
 * clamp(rint(w / scale) + zero, 0, 15); Large: scale = max|w| / 127, code =
 * clamp(rint(w / scale), -127, 127); an all-zero group has scale 0 and
 * codes 0.  rint rounds half to even; divisions are IEEE. */
int hq_pack_weights(const hq_layer_desc *desc, const float *W, const uint32_t *signs, void *blob,
                    void *stream);

/* Offline, fused layers: pack `rows` rows of weights (fp32 [rows][K]) as the
 * output channels n0 .. n0 + rows - 1 of the layer `desc`, writing only the
 * blob's tiles of those channels.  Layers that read the same activations
 * (the q, k and v projections, or the gate and up projections) are packed
 * part by part into one blob of N = the sum of their widths and run as one
 * hq_verify_gemm; Y's columns n0 .. n0 + rows - 1 are that part's outputs,
 * identical to what the part alone would give (per output, the same
 * arithmetic).  n0 must be a multiple of 128, and the rows of the last part
 * may end anywhere before N; channels of the blob that no call packs are
 * left as they were.  Signs, formats and errors as in hq_pack_weights. */
int hq_pack_weights_at(const hq_layer_desc *desc, int32_t n0, int32_t rows, const float *W, const uint32_t *signs,
                       void *blob, void *stream);

/* Size in bytes of the GEMM's activation operand for M rows of the
 * activations of layers like `desc` (its K, group and format; N is not used),
 * 0 if the arguments are invalid or M = 0.  The operand is an opaque buffer
 * written by hq_rotate_quant_act and read by hq_verify_gemm of layers with the
 * same K, group and format; its layout is private to this version of the
 * library (it depends on the format and on M). */
size_t hq_act_operand_bytes(const hq_layer_desc *desc, int32_t M);

/* Verify pass, step 1: rotate and quantize the activations of M rows
 * (section "How Uzu optimizes bytes and tokens per pass": activations
 * quantized to 8 bits on the fly, after the same randomized Hadamard
 * transform as the weights).
 *   desc  the layers that read these activations: K (a multiple of 32, at
 *         most 65536), group (16, 32, 64, 128 or 256, dividing K) and format
 *         choose the operand's encoding; N is not used
 *   X     fp32 [M][K], 16-byte aligned, 0 <= M <= HQ_MAX_M (M = 0: no-op)
 *   signs uint32 [K/32]
 *   qx    int8 [M][K] (4-byte aligned) or NULL: clamp(rint(x' / sx), -127, 127)
 *   gsum  int32 [M][K/group] (4-byte aligned) or NULL: the sum of the codes
 *         qx over each group (the correction term of the Medium format:
 *         sum qx (q - z) = sum qx q - z * gsum)
 *   qop   the GEMM's activation operand (hq_act_operand_bytes(desc, M)
 *         bytes, 16-byte aligned, opaque) or NULL
 *   sx    fp32 [M]:  max_k |x'[m][k]| / 127  (0 for an all-zero row)
 * At least one of qx, gsum, qop must be given.  x' is the rotated row: per
 * 32-block, sign flip, unnormalized Walsh-Hadamard butterfly at strides 1, 2,
 * 4, 8, 16 in fp32 without fused multiply-add, then multiplication by
 * fp32(1/sqrt(32)).  flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL. */
int hq_rotate_quant_act(const hq_layer_desc *desc, const float *X, int32_t M, const uint32_t *signs, int8_t *qx,
                        int32_t *gsum, void *qop, float *sx, uint32_t flags, void *stream);

/* Verify pass, step 2: integer GEMM of the quantized activations against the
 * packed weights with the per-group dequantization epilogue (section "How
 * Uzu optimizes bytes and tokens per pass": both matmul operands integers).
 *   blob      packed by hq_pack_weights for the same desc (16-byte aligned)
 *   qop, sx   from hq_rotate_quant_act with the same M, a descriptor of the
 *             same K, group and format, and the same signs
 *   M         0..HQ_MAX_M (0: no-op); one launch for every M
 *   Y         fp32 [M][N]:
 *               Y[m][n] = sx[m] * sum_g ( scale[n][g] * P[m][n][g] )
 *             with P[m][n][g] = sum_{k in g} qx[m][k] * (code[n][k] - zero[n][g])
 *             (zero = 0 for Large), the sum over g in fp32.
 *   partials  check mode: NULL, or int32 [M][N][K/group] that receives P
 *             exactly (slower; for verification)
 *   workspace hq_workspace_bytes(desc, M) bytes, 16-byte aligned, zero-filled
 *             before its first use
 * The integer sums P are exact: the codes are multiplied on the tensor cores
 * with fp32 accumulation, exact for these ranges (up to 32 rows: warp-level
 * fp16 MMAs on the weight codes widened in registers, 4-bit codes to
 * q - z; above: tcgen05 MMAs with e4m3 or fp16 operands, the Medium zero
 * point entering through the group sums).  The fp32 sum over groups is taken in ascending
 * group order.  An output whose K range is
 * split across thread blocks is the sum of the blocks' partial sums: by
 * default each block adds sx[m] * (its partial sum) into Y with an fp32
 * atomic add when it finishes (Y is zeroed first by the kernel itself), so
 * the order of those adds, and the last bits of such outputs, may change from
 * run to run; with HQ_LAUNCH_DETERMINISTIC the blocks wait for one another
 * and sum the partial sums in ascending K order, then multiply by sx[m].
 * Outputs computed by one block are the same in both modes.  Every wait is
 * bounded; the grid never exceeds the blocks resident at once, but a kernel
 * running concurrently on another stream that holds SMs for longer than the
 * bound makes the call time out (HQ_ERR_TIMEOUT from hq_workspace_status;
 * zero the workspace again before reusing it after a time-out).  flags: any
 * of HQ_LAUNCH_PDL, HQ_LAUNCH_DETERMINISTIC, HQ_LAUNCH_EXACT_ORDER (see
 * above); with HQ_LAUNCH_PDL,
 * Y is written only after the wait for the previous kernel. */
int hq_verify_gemm(const hq_layer_desc *desc, const void *blob, const void *qop, const float *sx, int32_t M, float *Y,
                   int32_t *partials, void *workspace, uint32_t flags, void *stream);

/* The verify GEMM on int8 activation codes, the boundary's form with qx, sx
 * and the group sums (page "Karpathy's Trick for Faster Local LLMs Finally
 * Has Proper Tooling", section "How Uzu optimizes bytes and tokens per pass":
 * both matmul operands are integers).  The result is that of
 * hq_verify_gemm on the operand hq_rotate_quant_act would write for these
 * codes (same Y, same modes and flags, same errors).
 *   qx        int8 [M][K] (4-byte aligned): clamp(rint(x' / sx), -127, 127)
 *             from hq_rotate_quant_act or any other producer of the codes
 *   sx        fp32 [M]
 *   gsum      int32 [M][K/group] or NULL: not read (the group sums the
 *             Medium zero point needs are formed from qx, exactly)
 *   workspace hq_workspace_q8_bytes(desc, M) bytes, 16-byte aligned: the
 *             hq_workspace_bytes(desc, M) bytes of hq_verify_gemm (zero-filled
 *             before first use, as there), then room for the operand
 * One launch converts qx into the operand inside the workspace, the GEMM
 * follows on the same stream (with programmatic dependent launch: its weight
 * stream starts while the conversion runs). */
size_t hq_workspace_q8_bytes(const hq_layer_desc *desc, int32_t M);
int hq_verify_gemm_q8(const hq_layer_desc *desc, const void *blob, const int8_t *qx, const float *sx,
                      const int32_t *gsum, int32_t M, float *Y, int32_t *partials, void *workspace, uint32_t flags,
                      void *stream);

/* Canonical view of a blob (for verification and for saving in a portable
 * form): codes uint8 [N][K] (Medium: 0..15; Large: the int8 code's byte),
 * scales fp32 [N][K/group], zeros uint8 [N][K/group] (Medium only; may be
 * NULL for Large). */
int hq_unpack_codes(const hq_layer_desc *desc, const void *blob, uint8_t *codes, float *scales, uint8_t *zeros,
                    void *stream);

/* Synchronizes `stream`, then reads and clears the error word of a
 * workspace (of hq_verify_gemm, hq_tree_attention or hq_prefix_attention).
 * Returns HQ_ERR_TIMEOUT if a bounded wait inside a call that used the
 * workspace gave up since the word was last cleared (the outputs of that call
 * are then incomplete), HQ_ERR_INVALID_ARG if an hq_prefix_attention call met
 * a bad page table entry or length (see there), HQ_OK otherwise. */
int hq_workspace_status(void *workspace, void *stream);

/* hq_verify_gemm without a caller-supplied workspace, for callers that
 * cannot allocate device memory at the point of the call: code that runs
 * under an allocator that forbids new allocations (for example inside a
 * memory-capped serving process, or a plugin whose host owns all device
 * memory), or code that must not call cudaMalloc because it would
 * synchronize the device.  The pages have no counterpart of this call.
 *
 * The scratch lives in one file-scope device array of
 * HQ_NOALLOC_SCRATCH_BYTES (60 MiB + 128 KiB) that every GPU which loads the
 * library holds until the process exits.  A call is accepted when
 * hq_workspace_bytes(desc, M) fits in it (any M, for N up to about two
 * million outputs); larger calls return HQ_ERR_UNSUPPORTED and launch
 * nothing.  The call allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library routine.  The first call on a device looks up the
 * array's device address (cudaGetSymbolAddress) with that device current
 * and zero-fills the array once (a synchronous cudaMemset); make that first
 * call before any stream capture.  Later calls only launch the GEMM: the
 * kernels leave the array's error word and counters at zero after every
 * call whose waits all succeed.  A bounded wait that gives up (see
 * hq_verify_gemm) leaves the outputs of that call incomplete and records
 * the time-out in the array; hq_noalloc_status reports it and cleans the
 * array up.  All calls on a device share the one array, so calls that may
 * overlap on the GPU (different streams, or graphs replayed concurrently)
 * race and must be serialized by the caller.  Arguments, outputs and flags
 * are those of hq_verify_gemm; HQ_LAUNCH_PDL works as there (nothing runs
 * between the previous kernel and the GEMM). */
#define HQ_NOALLOC_SCRATCH_BYTES (60u * 1024u * 1024u + 128u * 1024u)
int hq_verify_gemm_noalloc(const hq_layer_desc *desc, const void *blob, const void *qop, const float *sx,
                           int32_t M, float *Y, int32_t *partials, uint32_t flags, void *stream);

/* Status of the allocation-free calls on the current device: synchronizes
 * `stream`, then returns HQ_ERR_TIMEOUT if a bounded wait inside an
 * hq_verify_gemm_noalloc call gave up since the last status call (the
 * outputs of that call are incomplete; the array's error word and counters
 * are reset to zero before returning), HQ_OK otherwise (also when no such
 * call has run on the device).  Allocates nothing. */
int hq_noalloc_status(void *stream);

/* Draft-tree acceptance, after the verify pass (sections "Producing several
 * tokens from one model pass": the main model checks the drafted positions
 * together, accepts the valid prefix and adds its own token at the first
 * position it does not confirm; and "Verifying a draft tree without restoring
 * model state": on a tree, the longest valid path is accepted).
 *   logits    fp32 [M][V], row i = the main model's output after tree node i
 *   M         1..HQ_MAX_M tree nodes; node 0 is the root (the last committed
 *             token)
 *   parent    int32 [M], parent[0] ignored, 0 <= parent[i] < i otherwise
 *   tokens    int32 [M], the drafted token of each node (tokens[0] ignored)
 *   greedy    int32 [M] out: argmax of each row (lowest index among equal
 *             maxima; a NaN ranks above every number, the first NaN wins)
 *   path      int32 [M] out: the accepted drafted nodes from the root's child
 *             down, n_accept of them; the other entries -1
 *   n_accept  int32 out: accepted drafted tokens (the sequence advances by
 *             n_accept + 1); -1 (and bonus -1) if parent is not a tree listed
 *             parents-first
 *   bonus     int32 out: greedy[accepted node], the main model's own token
 *   workspace hq_tree_accept_workspace_bytes(M, V) bytes, 16-byte aligned
 * A node i > 0 is valid when its parent is and tokens[i] == greedy[parent[i]];
 * the deepest valid node is accepted, the lowest index among equally deep
 * ones.  All pointers are device memory.  flags: HQ_LAUNCH_DEFAULT or
 * HQ_LAUNCH_PDL. */
size_t hq_tree_accept_workspace_bytes(int32_t M, int32_t V);
int hq_tree_accept(const float *logits, int32_t M, int32_t V, const int32_t *parent, const int32_t *tokens,
                   int32_t *greedy, int32_t *path, int32_t *n_accept, int32_t *bonus, void *workspace, uint32_t flags,
                   void *stream);

/* Tree-masked verify attention (section "Verifying a draft tree without
 * restoring model state": an attention layer keeps a cache of every past
 * token, and the main model checks every branch of the draft tree in one pass
 * without changing its committed state).  The page gives no mask; node i
 * attends to the L committed positions, to its ancestors and to itself (the
 * prefix its branch would have had if decoded alone).  The ancestor walk
 * follows parent[] while the parent lies in [0, node); a parent outside that
 * range ends it.  Textbook softmax attention with grouped heads: query head h
 * reads key/value head h / (Hq / Hkv).
 *   q        fp16 [M][Hq][D], the tree nodes' queries
 *   k_cache  fp16 [Hkv][cap][D]: positions [0, L) committed, position L + j
 *   v_cache  = tree node j (written by this pass's key/value projection)
 *   cap      positions per head in the cache, >= L + M
 *   M        1..HQ_MAX_M tree nodes (node 0 the root); L >= 0
 *   Hq, Hkv  Hq a multiple of Hkv; 64 a multiple of Hq / Hkv
 *   D        HQ_ATTN_HEAD_DIM
 *   parent   int32 [M] (device)
 *   scale    softmax scale (typically 1/sqrt(D)), finite
 *   out      fp32 [M][Hq][D]
 *   workspace hq_tree_attention_workspace_bytes(Hkv) bytes, 16-byte aligned;
 *            its first word is the error word read by hq_workspace_status
 * The probabilities are rounded to fp16 for the product with V (fp32
 * accumulation everywhere): |out - exact| <= 2^-11 * max|v| + fp32 rounding.
 * All pointers are device memory, 16-byte aligned.  flags: HQ_LAUNCH_DEFAULT
 * or HQ_LAUNCH_PDL.  With HQ_LAUNCH_PDL the committed positions [0, L) are
 * read before waiting for the previous kernel of the stream, so that kernel
 * must not write them (the tree rows, q and parent may be its outputs).
 * Launches two kernels (chunks of key positions, then their merge). */
#define HQ_ATTN_HEAD_DIM 128
size_t hq_tree_attention_workspace_bytes(int32_t Hkv);
int hq_tree_attention(const void *q, const void *k_cache, const void *v_cache, int32_t cap, int32_t L, int32_t M,
                      int32_t Hq, int32_t Hkv, int32_t D, const int32_t *parent, float scale, float *out,
                      void *workspace, uint32_t flags, void *stream);

/* Commit of the accepted path into the attention cache (same section: state
 * is committed only along the chosen path).  The root stays at position L;
 * accepted node path[d] (depth d + 1) moves to position L + 1 + d for
 * d < *n_accept, in k_cache and v_cache (layout as in hq_tree_attention);
 * nothing moves when *n_accept <= 0 (no drafted token accepted, or the -1 of
 * a malformed tree) or when L + 1 + *n_accept > cap.  path and n_accept are
 * hq_tree_accept's outputs in device memory, so no host round trip is
 * needed; path entries outside [1, M) are skipped.  The next committed length
 * is L + 1 + *n_accept. */
int hq_tree_commit_kv(void *k_cache, void *v_cache, int32_t cap, int32_t L, int32_t M, int32_t Hkv, int32_t D,
                      const int32_t *path, const int32_t *n_accept, uint32_t flags, void *stream);

/* Rollback-free DeltaNet tree pass (section "Verifying a draft tree without
 * restoring model state": a Gated DeltaNet layer keeps a fixed-size state that
 * every accepted token changes; the verify pass computes every branch's
 * outputs without changing it, and the state is updated only along the
 * accepted path).  The page gives no equations; the recurrence is the
 * published gated delta rule, per head with a D x D state S (rows: value
 * dimensions, columns: key dimensions):
 *     S_i = alpha_i S_p (I - beta_i k_i k_i^T) + beta_i v_i k_i^T,  o_i = S_i q_i
 * with p the parent of tree node i, or the committed state for the root and
 * for a node whose parent lies outside [0, i).
 *   state  fp32 [H][D][D], the committed state; only read
 *   q, k, v  fp32 [M][H][D] (q, k as they enter the recurrence: any
 *          normalization is applied before); alpha, beta fp32 [M][H]
 *   parent int32 [M]; M 1..HQ_MAX_M; D = HQ_DELTA_HEAD_DIM
 *   out    fp32 [M][H][D]
 * Computed without forming any node's state: o_i = S w_i + sum_j c_j v_j over
 * node i's root path (w_i, c_j from D-vector steps), fp32 arithmetic.  With
 * HQ_LAUNCH_PDL the state is read before waiting for the previous kernel of
 * the stream, which therefore must not write it.  All pointers are device
 * memory, 16-byte aligned. */
#define HQ_DELTA_HEAD_DIM 128
int hq_delta_tree(const float *state, const float *q, const float *k, const float *v, const float *alpha,
                  const float *beta, const int32_t *parent, int32_t M, int32_t H, int32_t D, float *out,
                  uint32_t flags, void *stream);

/* Commit of the accepted path into the DeltaNet state (same section): in
 * place, one step for the root and one for each accepted node path[d],
 * d < *n_accept, in order (the new state is the accepted node's state).
 * path and n_accept are hq_tree_accept's outputs in device memory; path
 * entries outside [1, M) are skipped; nothing changes when *n_accept < 0.
 * Arguments as in hq_delta_tree. */
int hq_delta_commit(float *state, const float *k, const float *v, const float *alpha, const float *beta,
                    const int32_t *path, const int32_t *n_accept, int32_t M, int32_t H, int32_t D, uint32_t flags,
                    void *stream);

/* ------------------------------------------------------------------------
 * A batch of requests.  The calls below run the verify pass for several
 * sequences at once: sequences that share a long prefix, hold their keys and
 * values in pages of one cache, and use low-rank adapters of their own beside
 * the shared quantized projections.  The pages this library follows describe
 * one sequence; these calls have no counterpart there.
 * ------------------------------------------------------------------------ */

/* Element types of activations, residuals, adapters and caches. */
typedef enum { HQ_F32 = 0, HQ_F16 = 1, HQ_BF16 = 2 } hq_type;

/* Residual addition, RMS norm and the quantization of the result for the
 * layers like `desc`, in one pass over the rows:
 *     s  = x + residual                        (fp32)
 *     y  = s / sqrt(mean(s^2) + eps) * weight
 *     residual_out = round(s), h = round(y)
 *     x' = the rotated y (hq_rotate_quant_act), sx = max|x'| / 127,
 *     qx = clamp(rint(x' / sx), -127, 127)
 * The norm is taken of s before it is rounded into residual_out.  The codes
 * are formed from weight * s, without the factor 1 / sqrt(mean + eps): it is
 * the same for the whole row, so it cancels in x' / sx and enters sx alone,
 * and one reduction per row gives both the norm and the largest value.
 *   x         x_type [M][K], rows ldx elements apart
 *   residual  r_type [M][K], rows ldr elements apart, or NULL: s = x
 *   residual_out  r_type [M][K], rows ldr elements apart, or NULL; may be
 *             `residual` itself (or x, where types and strides agree)
 *   weight    fp32 [K];  eps >= 0, finite
 *   h         h_type [M][K], rows ldh elements apart, or NULL: the normed row
 *             without rotation (for adapters, routers, ...); must not overlap
 *             the inputs, except that it may be x with the same type and stride
 *   signs, qx, gsum, qop, sx  as in hq_rotate_quant_act (qx 8-byte aligned);
 *             all of qx, gsum and qop may be NULL when h or residual_out is
 *             given (then signs and sx may be NULL too: the norm alone)
 *   M         0..HQ_MAX_M with qop, else 0..2^20 (the codes of a longer batch
 *             feed hq_verify_gemm_q8 in slices)
 * x, residual, residual_out, weight and h are 16-byte aligned and their rows
 * too (ldx, ldr, ldh at least K and a multiple of 16 bytes).  An all-zero row
 * has sx = 0 and codes 0.  A row whose sums hold a NaN or an infinity, and a
 * row whose product with the weight does, has a NaN or infinite sx and codes
 * 0, so that a GEMM of it gives NaN.  Other rows may be of any size: sums and
 * codes of very large or small ones are formed in units of a power of two.
 * flags:
 * HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL (weight and signs are then read before
 * the wait for the previous kernel). */
int hq_add_norm_quant(const hq_layer_desc *desc, const void *x, int32_t x_type, int64_t ldx, const void *residual,
                      void *residual_out, int32_t r_type, int64_t ldr, const float *weight, float eps, int32_t M,
                      const uint32_t *signs, void *h, int32_t h_type, int64_t ldh, int8_t *qx, int32_t *gsum,
                      void *qop, float *sx, uint32_t flags, void *stream);

/* Low-rank adapters of many requests beside a shared projection: for each row
 * m with adapter a = ids[m],
 *     Y[m] = base[m] + scale[a] * B[a] (A[a] x[m])
 * over the first ranks[a] rows of A[a] and columns of B[a]; a row whose id is
 * outside [0, n_adapters) has no adapter: Y[m] = base[m].
 *   x      x_type [M][K], rows ldx elements apart, 16-byte aligned rows
 *   A      w_type (HQ_F16 or HQ_BF16) [n_adapters][r_max][K], 16-byte aligned
 *   B      w_type [n_adapters][N][r_max], 16-byte aligned
 *   ids    int32 [M] (device), in any order; rows of equal id share the reads
 *          of their adapter, 16 rows at a time
 *   ranks  int32 [n_adapters] (device) or NULL (r_max each); clamped to
 *          [0, r_max]; rank 0: no change
 *   scale  fp32 [n_adapters] (device) or NULL (1 each)
 *   base   fp32 [M][N], rows ldb elements apart, or NULL (zeros); base may be
 *          Y itself with ldb = ldy (in place, beside hq_verify_gemm's output)
 *   Y      fp32 [M][N], rows ldy elements apart (any 4-byte alignment: a part
 *          of a fused layer's columns); otherwise no overlap with the inputs
 *   K      a multiple of 8 up to 65536; r_max a multiple of 8 up to 256;
 *          N >= 1; 0 <= M <= HQ_MAX_M (M = 0: no-op)
 *   workspace hq_lora_workspace_bytes(M, r_max) bytes, 16-byte aligned
 * Products of 16-bit values are exact and sums are fp32; fp32 activations (and
 * the products A x, which stay fp32) enter the tensor cores as three bf16
 * terms that together hold them.  Sums are taken in a fixed order: results
 * repeat bit for bit.  Infinities and NaN give what the formula gives in fp32,
 * however many rows share an adapter.  Elements of A and B past a rank are not
 * used in any sum.  flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL (ids, ranks, A and B are
 * then read before the wait for the previous kernel, which must not write
 * them; scale, like x and base, is read after it).  Launches two kernels. */
size_t hq_lora_workspace_bytes(int32_t M, int32_t r_max);
int hq_lora_apply(const void *x, int32_t x_type, int64_t ldx, int32_t M, int32_t K, int32_t N, const void *A,
                  const void *B, int32_t w_type, int32_t n_adapters, int32_t r_max, const int32_t *ids,
                  const int32_t *ranks, const float *scale, const float *base, int64_t ldb, float *Y, int64_t ldy,
                  void *workspace, uint32_t flags, void *stream);

/* A paged key/value cache.  All arrays are the caller's device memory; this
 * struct is host memory, read during the call only.
 *   pool    [n_planes][n_pages][heads][page_size] rows of row_bytes bytes
 *           (a plane: the keys or the values of one layer), planes plane_bytes
 *           apart, 16-byte aligned
 *   ref     int32 [n_pages]: how many sequences hold the page; 0 = free
 *   table   int32 [n_seqs][max_pages]: position p of sequence s lies in row
 *           p % page_size of page table[s][p / page_size]; unused entries -1
 *   len     int32 [n_seqs]: positions held (0 = an empty slot)
 *   status  int32, zeroed once: the first error of a page operation or of
 *           hq_prefix_attention since it was last read (hq_pages_status)
 *   scratch hq_pages_scratch_bytes(&cache) bytes, 16-byte aligned: one call at
 *           a time
 * page_size is 16, 32, 64, 128 or 256; row_bytes a multiple of 16 up to 4096;
 * at most 2^24 pages, 8192 sequences, 2^20 pages a sequence, 65535 heads and
 * planes; n_pages * page_size and max_pages * page_size below 2^31. */
typedef struct {
    void *pool;
    int32_t *ref;
    int32_t *table;
    int32_t *len;
    int32_t *status;
    void *scratch;
    int64_t plane_bytes;
    int32_t n_planes;
    int32_t n_pages;
    int32_t n_seqs;
    int32_t max_pages;
    int32_t page_size;
    int32_t heads;
    int32_t row_bytes;
} hq_pages;

/* Page operations.  Each takes lists in device memory of n entries, n between
 * 0 and the smaller of 1024 and n_seqs (0: no-op); a sequence may stand in a
 * list once.  Pages are handed out deterministically: the free pages of lowest
 * index, to the listed sequences in order, each sequence's positions
 * ascending.  A call changes everything it was asked to, or nothing: a bad
 * entry (a sequence outside [0, n_seqs), listed twice, a length that does not
 * fit, a list that is not ascending) sets the status word to
 * HQ_ERR_INVALID_ARG, too few free pages to HQ_ERR_NO_PAGES, and nothing is
 * changed.  A page given up by a call is free for the next call, not for the
 * same one.  Table entries outside [0, n_pages) inside a sequence's length are
 * skipped.
 *
 * Sequences that share a page never see one another's later writes: a page
 * held more than once at the time of the call is copied before it is written
 * (the rows in use, every plane).  flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL.
 *
 * hq_pages_fork: dst[i], an empty slot, takes the pages and length of src[i]
 *   (src may repeat, and is not changed); no data moves.
 * hq_pages_extend: seqs[i] grows by add[i] >= 0 positions; where its last
 *   page has free rows and is shared, the page is replaced by a copy.
 * hq_pages_free: gives up every page of seqs[i]; its slot becomes empty (an
 *   empty slot stays as it is).
 * hq_pages_compact: drops positions of seqs[i].  base[i] (>= -1, below the
 *   length) is the last position that stays where it is; the kept ones after
 *   it are base[i] + keep[i][d], d < n_keep[i], keep strictly ascending from
 *   at least 1 (rows of `keep` hold max_keep entries, ldkeep apart, 0 <=
 *   max_keep <= ldkeep <= 2^20, and n_keep[i] is at most max_keep);
 *   they move to base[i] + 1 + d, the length becomes base[i] + 1 + n_keep[i]
 *   and the pages past it are given up.  Pages from the first position that
 *   moves on are replaced where they are shared.  A sequence with n_keep[i] <
 *   0 is left as it is.  After a tree of m nodes at positions len - m .. len -
 *   1, base = len - m, keep = hq_tree_accept's path and n_keep = its n_accept
 *   commit the accepted path.
 * hq_pages_copy: page dst[i] of every plane becomes a copy of page src[i]
 *   (counts and tables are not changed).  No page may stand in both lists or
 *   twice in dst; a pair with an index outside [0, n_pages) is skipped and
 *   sets the status word to HQ_ERR_INVALID_ARG.  n up to 65535. */
size_t hq_pages_scratch_bytes(const hq_pages *cache);
int hq_pages_fork(const hq_pages *cache, const int32_t *src, const int32_t *dst, int32_t n, uint32_t flags,
                  void *stream);
int hq_pages_extend(const hq_pages *cache, const int32_t *seqs, const int32_t *add, int32_t n, uint32_t flags,
                    void *stream);
int hq_pages_free(const hq_pages *cache, const int32_t *seqs, int32_t n, uint32_t flags, void *stream);
int hq_pages_compact(const hq_pages *cache, const int32_t *seqs, const int32_t *base, const int32_t *keep,
                     int32_t ldkeep, int32_t max_keep, const int32_t *n_keep, int32_t n, uint32_t flags,
                     void *stream);
int hq_pages_copy(const hq_pages *cache, const int32_t *src, const int32_t *dst, int32_t n, uint32_t flags,
                  void *stream);

/* Writes the newest rows of B sequences into two planes of the cache: row i
 * of sequence seqs[b] (seqs NULL: b), i < m_b = starts[b + 1] - starts[b]
 * (starts NULL: max_rows rows each), goes to position len - m_b + i.
 *   k, v      in_type [rows][heads][D], rows ldk and ldv elements apart,
 *             16-byte aligned rows; D = row_bytes / 2
 *   type      the cache's element type, HQ_F16 or HQ_BF16 (in_type F32 or
 *             `type`; fp32 is rounded to nearest)
 *   starts    int32 [B + 1] (device), ascending, within [0, rows]; B <= 65535
 *   max_rows  the most rows of a sequence, at least 1
 * Rows whose position or page does not exist are skipped and set the status
 * word to HQ_ERR_INVALID_ARG.  Pages are written as they are: after a fork,
 * hq_pages_extend first gives the sequence pages of its own. */
int hq_pages_write(const hq_pages *cache, int32_t k_plane, int32_t v_plane, const void *k, const void *v,
                   int32_t in_type, int64_t ldk, int64_t ldv, int32_t type, const int32_t *seqs,
                   const int32_t *starts, int32_t B, int32_t rows, int32_t max_rows, uint32_t flags, void *stream);

/* Synchronizes `stream`, then reads and clears the cache's status word:
 * HQ_OK, HQ_ERR_INVALID_ARG, HQ_ERR_NO_PAGES or (hq_prefix_attention)
 * HQ_ERR_TIMEOUT. */
int hq_pages_status(const hq_pages *cache, void *stream);

/* Attention of a batch over a paged cache whose sequences share their first
 * `shared` positions: the shared keys and values are read once for all rows,
 * each sequence's own positions by its own rows.  Row i of sequence b (its
 * m_b newest positions, as in hq_pages_write; draft-tree node i) attends to
 * the positions [0, len_b - m_b), to its ancestors in the tree and to itself;
 * parent as in hq_tree_attention (numbered within the sequence), or NULL: a
 * chain (node i - 1 is the parent of node i: the newest tokens of a prompt or
 * a single token).  Query head h reads key/value head h / (Hq / heads).
 *   Hq        a multiple of heads, at most 65535
 *   cache     row_bytes = 2 D, D = 64 or 128; type HQ_F16 or HQ_BF16;
 *             plane_bytes below 2^40
 *   q         type [rows][Hq][D], rows ldq elements apart, 16-byte aligned rows
 *   seqs, starts, B, rows, max_rows  as in hq_pages_write; max_rows <= HQ_MAX_M
 *   parent    int32 [rows] (device) or NULL
 *   shared    positions that all active sequences hold alike (0: none), at
 *             most len_b - m_b of each; they are read through the table of the
 *             first active sequence
 *   max_len   at least every sequence's length (it sizes the launch), above
 *             `shared`, at most max_pages * page_size and 2^30
 *   scale     softmax scale, finite also in base-2 units (scale * log2(e))
 *   out       out_type [rows][Hq][D], rows ldo elements apart, 16-byte aligned
 *             rows; out_type is `type` or HQ_F32
 *   workspace hq_prefix_attention_workspace_bytes(B, rows, max_rows, Hq,
 *             heads, D) bytes, 16-byte aligned, its first 16 bytes zeroed
 *             once; the size grows with rows and max_rows and does not depend
 *             on B or the lengths, so one workspace of the largest rows and
 *             max_rows serves every call of these heads in turn
 * B = 0 or rows = 0: no-op (out is not written).  A row of an empty sequence
 * (len 0), and a row that no sequence claims, is zero.  A length that contradicts shared, m_b or max_len makes the
 * sequence's rows zero, a table entry outside [0, n_pages) makes its
 * positions read as zeros; both set the error word (hq_workspace_status:
 * HQ_ERR_INVALID_ARG).  A call that ends with the error word set, by itself or
 * by an earlier call, enters it in the cache's status word too
 * (hq_pages_status).  Rows past a sequence's length, other branches of the
 * tree and other sequences' pages do not influence a row, whatever they hold
 * (infinities and NaN included).  Scores, softmax statistics and outputs are
 * accumulated in fp32; the probabilities are rounded to `type` for the
 * product with V, whatever out_type is: at most eps / 2 of `type` relative
 * each, but with HQ_F16 a probability below 2^-21 of the largest of its part of
 * the positions by at most 2^-32 of that largest.  Sums are taken in a fixed
 * order: results repeat bit for bit. */
size_t hq_prefix_attention_workspace_bytes(int32_t B, int32_t rows, int32_t max_rows, int32_t Hq, int32_t Hkv,
                                           int32_t D);
int hq_prefix_attention(const hq_pages *cache, int32_t k_plane, int32_t v_plane, int32_t type, const void *q,
                        int64_t ldq, const int32_t *seqs, const int32_t *starts, int32_t B, int32_t rows,
                        int32_t max_rows, const int32_t *parent, int32_t Hq, int32_t shared, int32_t max_len,
                        float scale, void *out, int32_t out_type, int64_t ldo, void *workspace, uint32_t flags,
                        void *stream);

/* Rotary positions.  Pair i of a head's first `rot` elements turns by freqs[i]
 * radians a position; the other elements stay as they are.  Host-only.
 *
 * hq_rope_freqs: the frequencies of a head with rot rotated elements (even, 2
 * to 65536), rot / 2 doubles, f_i = base^(-2i / rot) with base > 1, and, for
 * contexts `factor` >= 1 times as long as the model's own of `original`
 * positions:
 *   HQ_ROPE_PLAIN   f_i (factor, original, low and high are not used)
 *   HQ_ROPE_LINEAR  f_i / factor
 *   HQ_ROPE_NTK     f_i of the base times factor^(rot / (rot - 2)); rot >= 4
 *   HQ_ROPE_YARN    f_i where a pair's number is at most lo, f_i / factor from
 *                   hi on, a ramp t = (i - lo) / (hi - lo) between: f_i (1 - t)
 *                   + f_i / factor t.  lo and hi are where pairs turn `high` and
 *                   `low` times over `original` positions (rounded down and up,
 *                   within 0 and rot - 1): rot ln(original / (2 pi turns)) /
 *                   (2 ln base).  Usually high = 32, low = 1, and the gain of
 *                   hq_rope_write 0.1 ln(factor) + 1
 *   HQ_ROPE_BANDS   the same mix by the turns themselves: 1 - t = (original f_i
 *                   / (2 pi) - low) / (high - low) within 0 and 1; usually low =
 *                   1, high = 4
 * high > low > 0 and original > 0 for the last two.
 *
 * hq_rope_turns: n frequencies (0 <= f <= pi) as hq_rope_write reads them:
 * turns a position, f / (2 pi), in units of 2^-64, rounded to nearest.  The
 * product with a position is then exact modulo a turn, at any position, in one
 * integer multiplication. */
typedef enum { HQ_ROPE_PLAIN = 0, HQ_ROPE_LINEAR = 1, HQ_ROPE_NTK = 2, HQ_ROPE_YARN = 3, HQ_ROPE_BANDS = 4 } hq_rope_kind;
int hq_rope_freqs(int32_t rot, double base, int32_t kind, double factor, double original, double low, double high,
                  double *freqs_host);
int hq_rope_turns(const double *freqs_host, int32_t n, uint64_t *turns_host);

/* Between the projection and hq_prefix_attention: rotates the newest rows' q
 * and k by their positions and writes k and v into the cache (hq_pages_write
 * with the rotation), in one launch.  Row i of sequence seqs[b], its rows and
 * their places in the cache as in hq_pages_write (k_plane and v_plane differ, and
 * a sequence stands in seqs once).  A row's rotary position is
 * positions[row] or, where positions is NULL, len - m_b + d: d is its depth in
 * the tree of `parent` (numbered within the sequence as in hq_tree_attention;
 * the walk ends at a parent outside [0, node)), or i where parent is NULL.
 * Nodes of one depth share a position, so the accepted path's keys hold the
 * positions that it has after hq_pages_compact.
 *   q, k, v   in_type (HQ_F32 or `type`) [rows][Hq][D] and [rows][heads][D],
 *             rows ldq, ldk, ldv elements apart, 16-byte aligned rows; D =
 *             row_bytes / 2 = 64, 128 or 256; Hq 1..65535
 *   q_weight, k_weight  fp32 [D] or NULL: the head is normed first, x *
 *             weight / sqrt(mean(x^2) + eps); eps >= 0, finite
 *   turns     uint64 [rot / 2] (device), from hq_rope_turns
 *   rot       a multiple of 16 from 16 to D
 *   layout    HQ_ROPE_HALF: element i < rot / 2 pairs with i + rot / 2;
 *             HQ_ROPE_INTERLEAVED: element 2i with 2i + 1
 *   gain      factor of the rotated elements (1: none), finite
 *   q_out     type [rows][Hq][D], rows ldo elements apart, 16-byte aligned
 *             rows; may be q itself where types and strides agree, otherwise no
 *             overlap with the inputs
 *   parent    int32 [rows] (device) or NULL; with it max_rows <= HQ_MAX_M
 *   positions int32 [rows] (device) or NULL; any value
 * Arithmetic is fp32 with one rounding to `type` per element; the angle is off
 * by at most 2^-23, a normed head by 2^-20 of each element.  v is rounded or copied.  Rows that no sequence claims
 * are left as they were, in q_out too.  A row whose sequence, length or place does not
 * exist is not written, k and v of a row whose page does not exist are not
 * written (its q is); both set the cache's status word to HQ_ERR_INVALID_ARG.
 * flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL (nothing is read before the wait). */
typedef enum { HQ_ROPE_HALF = 0, HQ_ROPE_INTERLEAVED = 1 } hq_rope_layout;
int hq_rope_write(const hq_pages *cache, int32_t k_plane, int32_t v_plane, int32_t type, const void *q, const void *k,
                  const void *v, int32_t in_type, int64_t ldq, int64_t ldk, int64_t ldv, int32_t Hq,
                  const float *q_weight, const float *k_weight, float eps, const uint64_t *turns, int32_t rot,
                  int32_t layout, float gain, const int32_t *seqs, const int32_t *starts, int32_t B, int32_t rows,
                  int32_t max_rows, const int32_t *parent, const int32_t *positions, void *q_out, int64_t ldo,
                  uint32_t flags, void *stream);

/* A norm per head with a gate, and its quantization for the output projection
 * `desc` (behind hq_delta_tree or hq_prefix_attention, in front of
 * hq_verify_gemm), in one pass over the rows.  For each head of D features:
 *     y = x * weight / sqrt(mean(x^2) + eps) * act(gate)
 *     h = round(y);  x', sx, qx, gsum, qop of y as in hq_add_norm_quant
 *   x      x_type [M][K], rows ldx elements apart
 *   gate   g_type [M][K], rows ldg elements apart, or NULL: 1
 *   act    HQ_GATE_NONE: the gate itself; HQ_GATE_SIGMOID: 1 / (1 + e^-gate);
 *          HQ_GATE_SILU: gate / (1 + e^-gate); a quotient 1 / (1 + e^-gate) below
 *          2^-126 is 0
 *   weight fp32 [D], the same for every head, or NULL: no norm, y = x *
 *          act(gate)
 *   D      64, 128 or 256, dividing K = desc->K
 *   eps    >= 0, finite
 *   h      h_type [M][K], rows ldh elements apart, or NULL; must not overlap the
 *          inputs, except that it may be x or gate with the same type and stride
 *   signs, qx, gsum, qop, sx and their rules as in hq_add_norm_quant; all of
 *          qx, gsum and qop may be NULL when h is given
 *   M      0..HQ_MAX_M with qop, else 0..2^20
 * x, gate, h and weight are 16-byte aligned, rows too.  Heads of any size are
 * normed as the formula says (their squares are taken in units of a power of
 * two where fp32's range would end).  Arithmetic is fp32: the quotient 1 / (1 +
 * e^-gate) is within 2^-20 of its value, y within 2^-19 (relative to it; a
 * normed head's sum, root and products 14 * 2^-24 of that), and h has its own
 * rounding.  A row of y with a NaN or an infinity has a NaN or infinite sx and
 * codes 0.  flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL
 * (nothing is read before the wait). */
typedef enum { HQ_GATE_NONE = 0, HQ_GATE_SIGMOID = 1, HQ_GATE_SILU = 2 } hq_gate_act;
int hq_gated_norm_quant(const hq_layer_desc *desc, const void *x, int32_t x_type, int64_t ldx, const void *gate,
                        int32_t g_type, int64_t ldg, int32_t act, const float *weight, int32_t D, float eps, int32_t M,
                        const uint32_t *signs, void *h, int32_t h_type, int64_t ldh, int8_t *qx, int32_t *gsum,
                        void *qop, float *sx, uint32_t flags, void *stream);

/* What requests have said so far.  All arrays are the caller's device memory;
 * this struct is host memory, read during the call only.
 *   tokens  int32 [n_slots][cap]: a slot's prompt, then what was generated, the
 *           root of its next draft tree (its newest token) last
 *   len     int32 [n_slots]: tokens held; values outside [0, cap] count as the
 *           nearer end when read
 *   prompt  int32 [n_slots] or NULL (0): how many of them are the prompt's
 *   status  int32, zeroed once: the first error of hq_tree_accept_batch since it
 *           was last read (hq_history_status)
 * 1 to 65536 slots, cap from 1 to 2^24. */
typedef struct {
    int32_t *tokens;
    int32_t *len;
    const int32_t *prompt;
    int32_t *status;
    int32_t n_slots;
    int32_t cap;
} hq_history;

/* Rules on the logits.  Device arrays, each may be NULL (the rule is not
 * applied); host struct, read during the call only.
 *   repetition, presence, frequency  fp32 [n_slots]
 *   bias_starts  int32 [n_slots + 1], ascending, within [0, n_bias]: slot s has the
 *           biases bias_values[j] of tokens bias_tokens[j] (int32, fp32 [n_bias]),
 *           bias_starts[s] <= j < bias_starts[s + 1]; of a token listed twice the
 *           last one counts.  Each part of the vocabulary (1024 to 4096 tokens)
 *           reads its slot's list once or twice: thousands of entries cost
 *           microseconds, one for each of 151552 tokens a third of a millisecond
 *   masks   uint32 [n_masks][ldmask], ldmask at least ceil(V / 32): token t is
 *           allowed where bit t % 32 of word t / 32 is set
 * n_slots from 0 to 65536 (0: no rule but the masks); 0 <= n_bias, n_masks < 2^31. */
typedef struct {
    const float *repetition;
    const float *presence;
    const float *frequency;
    const int32_t *bias_starts;
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *masks;
    int64_t ldmask;
    int32_t n_slots;
    int32_t n_bias;
    int32_t n_masks;
} hq_logit_rules;

/* Penalties, biases and grammar masks on the logits of a batch's trees, and the
 * greedy token of every row, in one pass.  For row i of the b-th sequence (rows
 * as in hq_pages_write; slot s = seqs[b], or b) and every token t, in fp32, each
 * operation rounded once:
 *     l = logits[row][t]
 *     t is in the history or drafted on the row's path:
 *         l = l > 0 ? l / repetition[s] : l * repetition[s]
 *     it is there n > 0 times behind the prompt:
 *         l = l - frequency[s] * n;  l = l - presence[s]
 *     t has a bias:  l = l + bias
 *     t is masked:   l = -infinity
 *     greedy[row] = the token of the largest l among those that are not masked,
 *         the lowest one among equals; a NaN ranks above every number, the first
 *         NaN wins; -1 if every token is masked
 *     out[row][t] = l, rounded to out_type
 * The row's path is that of hq_tree_accept: `tokens` of node i and of its
 * ancestors but the root (node 0, whose token is the history's last).
 *   logits  type [rows][V], rows ldl elements apart, any alignment of its
 *           elements; V from 1 to 2^24
 *   history, rules  or NULL: none.  A slot outside [0, n_slots) has none
 *   seqs, starts, B, rows, max_rows  as in hq_pages_write; max_rows <= HQ_MAX_M
 *   parent  int32 [rows] (device) or NULL: a chain; as in hq_tree_attention
 *   tokens  int32 [rows] (device) or NULL: nothing drafted
 *   mask_ids  int32 [rows] (device) or NULL (row r has mask r): the row's mask;
 *           a row whose id is outside [0, n_masks) has none
 *   out     out_type (type or HQ_F32) [rows][V], rows ldo elements apart, or
 *           NULL; may be logits itself with the same type and stride, otherwise
 *           no overlap
 *   greedy  int32 [rows]
 *   workspace hq_greedy_tokens_workspace_bytes(rows) bytes, 16-byte aligned,
 *           zeroed once: counters, and room for long histories sorted by token
 *           (64 KB a row, for 256 rows at most).  One workspace of the most rows
 *           serves every call in turn
 * Long histories of many rows are sorted by token in front, by another kernel:
 * where cap (at most 16384 of it) and the rows are so large that it pays for
 * histories that fill it.  Up to 256 sequences and vocabularies below 258049 do
 * that, with more rows than 16 at 151552 tokens; other calls read a history once
 * for each 1024 to 4096 tokens of the vocabulary, and so do all what lies past a
 * history's first 16384.
 * Tokens outside [0, V), in any of the lists, are passed over.  Rows that no
 * sequence claims are left as they were, in out and greedy.  Results repeat bit
 * for bit.  flags: HQ_LAUNCH_DEFAULT or HQ_LAUNCH_PDL (nothing is read before
 * the wait). */
size_t hq_greedy_tokens_workspace_bytes(int32_t rows);
int hq_greedy_tokens(const void *logits, int32_t type, int64_t ldl, int32_t V, const hq_history *history,
                     const hq_logit_rules *rules, const int32_t *mask_ids, const int32_t *seqs, const int32_t *starts,
                     int32_t B, int32_t rows, int32_t max_rows, const int32_t *parent, const int32_t *tokens, void *out,
                     int32_t out_type, int64_t ldo, int32_t *greedy, void *workspace, uint32_t flags, void *stream);

/* Acceptance of a batch of draft trees (hq_tree_accept for each sequence, from
 * greedy tokens that are there already), which also grows the histories, so
 * that the next step's penalties follow without the host.
 *   greedy, parent, tokens  int32 [rows] (device); parent NULL: chains
 *   seqs, starts, B, rows, max_rows  as in hq_pages_write; max_rows <= HQ_MAX_M
 *   history   or NULL.  Slot seqs[b] (or b) grows by the accepted drafts and the
 *             bonus token (if it is not negative).  A slot outside [0, n_slots),
 *             a length that is outside [0, cap] or would pass cap, and a slot
 *             listed before leave the history as it was and set its status word to
 *             HQ_ERR_INVALID_ARG
 *   path      int32 [B][ldpath], ldpath >= max_rows: the accepted drafted nodes of
 *             sequence b from the root's child down, then -1 up to max_rows
 *   n_accept, bonus  int32 [B]; both -1 (and the history as it was) for a
 *             sequence without rows and for one whose parents are not a tree
 *             listed parents-first
 * A negative greedy token accepts nothing.  path and n_accept are what
 * hq_pages_compact takes as keep and n_keep.  flags: HQ_LAUNCH_DEFAULT or
 * HQ_LAUNCH_PDL (nothing is read before the wait). */
int hq_tree_accept_batch(const int32_t *greedy, const int32_t *parent, const int32_t *tokens, const int32_t *seqs,
                         const int32_t *starts, int32_t B, int32_t rows, int32_t max_rows, const hq_history *history,
                         int32_t *path, int32_t ldpath, int32_t *n_accept, int32_t *bonus, uint32_t flags,
                         void *stream);

/* Synchronizes `stream`, then reads and clears the history's status word. */
int hq_history_status(const hq_history *history, void *stream);

/* Self-test of the bounded-wait path: launches one block that waits on a
 * shared-memory barrier nothing will ever complete, giving up after
 * `limit_ns` nanoseconds (1000..100000000) and setting the error word of
 * `workspace` (>= 16 bytes, zero-filled).  hq_workspace_status then
 * returns HQ_ERR_TIMEOUT.  No fault and no hang: the kernel returns. */
int hq_selftest_wait_timeout(void *workspace, int64_t limit_ns, void *stream);

/* Self-test of the GEMM's bounded waits between thread blocks: runs
 * hq_verify_gemm (arguments as there, HQ_LAUNCH_DETERMINISTIC) with every
 * wait for the other contributors of a split output asking for one arrival
 * more than there are and giving up after `limit_ns` nanoseconds
 * (1000..100000000).  On a layer with split outputs (K of several 128-feature
 * tiles and more tiles than SMs) the waits run out: hq_workspace_status then
 * returns HQ_ERR_TIMEOUT; Y is unspecified.  No fault and no hang: the kernel
 * returns.  Zero the workspace before reusing it. */
int hq_selftest_gemm_wait_timeout(const hq_layer_desc *desc, const void *blob, const void *qop, const float *sx,
                                  int32_t M, float *Y, void *workspace, int64_t limit_ns, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* HQ_H */
