/*
 * spec_verify.h -- C ABI of the GB300 (sm_103a) speculative-decoding
 * verification step.
 *
 * The operation (one verification round, after the target model's single
 * forward over the drafted tokens) is the modified rejection sampler that all
 * of these pages state:
 *   [P1] "Speculative Decoding" (atonlee.tistory.com/330), ch.2 (one round:
 *        accept in order, cut at the first rejection, k accepted + 1 token)
 *        and ch.3 (accept test r < min(1, p(x)/q(x)), residual
 *        norm(max(0, p - q)), greedy rule at temperature 0);
 *   [P2] "Speculative Decoding으로 LLM 추론 속도 높이기" (donmain.dev), section
 *        "품질은 rejection sampling이 지킨다";
 *   [P3] "Fast Inference from Transformers via Speculative Decoding" notes
 *        (obsidian-dorae222.pages.dev), method details, steps 2-3 (gamma+1
 *        target distributions from one forward, accept probability, residual
 *        sample, bonus token from p at row gamma when every draft passes);
 *   [P4] "투기적 디코딩 — 초안 모델을 무엇으로 세울 것인가" (ailab.paldyn.com),
 *        section on why the output does not change (greedy: draft == argmax).
 *
 * For each sequence b with g = num_draft[b] drafts and temperature T = temperature[b]:
 *   T > 0:  p_i = softmax(target_logits[b, i, :] / T) for i <= g,
 *           q_i = softmax(draft_logits[b, i, :] / T) for i < g.
 *           Position i < g accepts draft x_i = draft_tokens[b, i] iff
 *           uniforms[b, i] * q_i(x_i) < p_i(x_i); n = first rejected i, or g.
 *           One more token y is drawn by inverse CDF with u = uniforms[b, gamma_max]
 *           from max(0, p_n - q_n) (n < g) or from p_g (n == g): y is the
 *           smallest id j with u * S < C_j, C_j the running sum of the weights
 *           in id order and S their total.  The weights are integers on a
 *           2^-60 grid, each within about 2^-36 of its exact value where it
 *           matters (ids whose weight is within a factor 2^15 of the row's
 *           largest; float32, to about 2^-22, for the rest), so every sum is
 *           exact and y differs from the float64 definition only when u lies
 *           within ~1e-9 of a boundary C_j / S (rows whose
 *           |logit| * log2(e) / T passes 2^21 keep float32 weights throughout).
 *   T == 0: greedy; a_i = argmax of the raw target logits of row i (lowest id
 *           on ties); position i accepts iff x_i == a_i; y = a_n.  No draft row
 *           and no uniform is read.
 *   Output: out_tokens[b, 0..n-1] = x_0..x_{n-1}, out_tokens[b, n] = y,
 *           out_tokens[b, n+1..gamma_max] = -1, out_num_accepted[b] = n.
 * Point-mass proposals (draft_logits == NULL; a deterministic proposer such as
 * prompt lookup, "Speculative Decoding" ch.5): q_i is 1 at x_i, so position i
 * accepts iff uniforms[b, i] < p_i(x_i) and a rejection samples p_n with x_n
 * removed (max(0, p - q) for that q).  No draft row is read.
 * The full sweep (options.kernel 2) also reads the rows after the cut; the
 * early exit (kernel 3, the automatic choice for large batches and tiny rows)
 * reads none.  Rows i > g (target) and i >= g (draft), and every draft row of
 * a greedy sequence, are never read.
 *
 * Layout.  All arrays are dense, row-major, and readable by the device of the
 * calling thread's current CUDA context:
 *   target_logits  [B, gamma_max + 1, V]   dtype (SPEC_F32 or SPEC_BF16)
 *   draft_logits   [B, gamma_max, V]       dtype, or NULL for point-mass proposals
 *   draft_tokens   [B, gamma_max]          int32
 *   num_draft      [B]                     int32
 *   uniforms       [B, gamma_max + 1]      float32 in [0, 1)
 *   temperature    [B]                     float32
 *   out_tokens     [B, gamma_max + 1]      int32 (written)
 *   out_num_accepted [B]                   int32 (written)
 * Logit pointers must be aligned to their element size; the fast path is
 * taken when both are 16-byte aligned and V * element size is a multiple of
 * 16 bytes, a scalar-load path otherwise.  int32/float32 arrays must be
 * 4-byte aligned.  Outputs must not overlap inputs.
 * Where the inputs live.  Arrays the kernels only read (logits, tokens,
 * num_draft, uniforms, temperature) may be device memory or page-locked host
 * memory mapped into the device's address space (cudaHostAlloc, or
 * cudaHostRegister with cudaHostRegisterMapped); pass the address that
 * spec_device_pointer returns for it.  The kernels then read those bytes over
 * the host link while they run ("zero copy"): no staging copy is made, and the
 * early-exit kernel (options.kernel 3) moves only the rows it needs across
 * the link, each once where two row slices fit in shared memory (it keeps the
 * decided rows there for the final sample; host memory is not cached in L2).
 * The kernels read such memory after the call has returned, so the caller
 * keeps it allocated and unchanged until the stream has passed the call (for
 * example until an event recorded after the call completes).  Everything the
 * kernels write (outputs, status, counters, diagnostics) must be device
 * memory.
 *
 * Ownership and execution.  The caller owns every buffer.  The call enqueues
 * one kernel on 'stream' (a cudaStream_t; NULL = legacy default stream) and
 * returns without synchronising; it allocates no memory.  It is reentrant:
 * the only process-wide state is a per-device cache of kernel attributes.
 *
 * Errors.  Argument problems found on the host return an error code before
 * anything is enqueued.  Problems in the data never trap: a sequence with
 * num_draft outside [0, gamma_max], a temperature that is negative, NaN,
 * infinite or positive but below FLT_MIN, a drafted id outside [0, V) at a
 * position it uses, or a sampled row it uses whose logits have no finite
 * softmax normaliser (all -inf, any +inf or NaN) gets out_tokens[b, :] = -1
 * and out_num_accepted[b] = 0, and its SPEC_STATUS_* bit is OR-ed into
 * *status when status is not NULL (the caller zeroes it).  The kernels wait only
 * at hardware barriers that every thread of the CTA or cluster reaches.  NaN
 * logits in greedy rows give unspecified (in-range) tokens.
 *
 * Limits: 0 <= B <= SPEC_MAX_BATCH (B == 0 is a no-op), 0 <= gamma_max <=
 * SPEC_MAX_GAMMA, 1 <= V <= SPEC_MAX_VOCAB.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_MAX_GAMMA 16
#define SPEC_MAX_VOCAB (1 << 24)
#define SPEC_MAX_BATCH (1 << 26)
#define SPEC_MAX_TREE_NODES 256

typedef enum {
    SPEC_OK = 0,
    SPEC_ERR_INVALID_ARG = 1, /* null pointer, size out of range, misaligned pointer */
    SPEC_ERR_UNSUPPORTED = 2, /* unknown dtype, or no usable launch shape on this device */
    SPEC_ERR_CUDA = 3         /* a CUDA runtime call or the launch failed */
} spec_status;

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype;

/* Per-sequence data problems (bits OR-ed into *status). */
#define SPEC_STATUS_BAD_TOKEN 1u
#define SPEC_STATUS_BAD_TEMPERATURE 2u
#define SPEC_STATUS_BAD_NUM_DRAFT 4u
#define SPEC_STATUS_BAD_LOGITS 8u
/* spec_tree_verify: a node's parent is not an earlier node. */
#define SPEC_STATUS_BAD_TREE 32u
/* spec_cache_*: a length or a number of new tokens out of range; a page id out of range. */
#define SPEC_STATUS_BAD_LENGTH 64u
#define SPEC_STATUS_BAD_PAGE 128u
/* spec_cache_*: a bounded wait inside a kernel ran out; the call's outputs are not valid. */
#define SPEC_STATUS_INTERNAL 256u

/* One verification round for B independent sequences (see the top of this
 * file for the operation, layout, ownership and errors).
 * status: optional device word (may be NULL) receiving SPEC_STATUS_* bits. */
spec_status spec_verify(const void *target_logits, const void *draft_logits, const int32_t *draft_tokens,
                        const int32_t *num_draft, const float *uniforms, const float *temperature,
                        int32_t *out_tokens, int32_t *out_num_accepted, int B, int gamma_max, int V,
                        spec_dtype dtype, uint32_t *status, void *stream);

/* Launch options (tuning, A/B measurement and the early-exit variant).  They
 * change no decision except one that lies very close to its boundary: the
 * normalisers are merged from per-CTA partials, so the split of a row (the
 * cluster size) and the kernel variant move p-hat and q-hat by about 1e-7
 * relative, and an accept test that close to its threshold (or a final draw
 * within ~1e-9 of a CDF boundary) may come out differently.  Greedy (T == 0)
 * results never change. */
typedef struct spec_verify_options {
    int cluster_size; /* CTAs sharing one sequence's rows: 0 = automatic, else 1 to 16 */
    int kernel;       /* 0 = automatic: the early exit (3) when the full sweep's grid would
                             fill more than half of the device's resident CTA slots or the
                             rows are tiny (V * element size <= 8 KB), else the full sweep (2);
                         1 = not a kernel (SPEC_ERR_INVALID_ARG);
                         2 = full sweep, register loads;
                         3 = row-ordered early exit: position i's rows are read, reduced
                             and tested before position i+1's, and no row after the first
                             rejection is read (n+1 target and min(n+1, g) draft rows per
                             sequence; the method needs nothing after the cut, "Speculative
                             Decoding" ch.2).  Diagnostics then cover the rows read only. */
    uint64_t *counters; /* optional device array [3] (8-byte aligned), accumulated with atomics:
                           += drafted ids, += accepted ids, += verified sequences (valid ones).
                           Their ratio is the acceptance rate; accepted / sequences + 1 the mean
                           tokens per round (the counts a serving engine exports, per
                           "Speculative Decoding으로 LLM 추론 속도 높이기", vLLM section).  NULL: none. */
    uint64_t *accept_hist; /* optional device array [SPEC_MAX_GAMMA + 1] (8-byte aligned): += 1 at
                              index n (accepted count; min(n, SPEC_MAX_GAMMA) for trees) for each
                              verified sequence, the distribution behind the mean.  NULL: none. */
} spec_verify_options;

/* Same round, plus optional float32 diagnostics for tests (any may be NULL):
 *   p_hat [B, gamma_max]     p_i(x_i) for i < g of sampled sequences, NaN elsewhere
 *   q_hat [B, gamma_max]     q_i(x_i), same positions
 *   logz_t [B, gamma_max+1]  natural-log normaliser log sum_j exp(l_j / T) of
 *                            target rows i <= g of sampled sequences, NaN elsewhere
 *   logz_d [B, gamma_max]    same for draft rows i < g
 *   resid_mass [B]           total weight S of the decided row of a sampled
 *                            sequence (residual mass, or ~1 for a bonus row)
 *   seq_status [B]           SPEC_STATUS_* bits of each sequence (0 = valid)
 * The diagnostic rows are computed for every i <= g, also after the cut (with
 * the full-sweep kernels; options.kernel 0 takes the full sweep here).  A sequence with a data problem (seq_status != 0)
 * may carry partial diagnostics: the rows swept before the problem was found.
 * options: as for spec_verify_ex (NULL = automatic). */
spec_status spec_verify_debug(const void *target_logits, const void *draft_logits, const int32_t *draft_tokens,
                              const int32_t *num_draft, const float *uniforms, const float *temperature,
                              int32_t *out_tokens, int32_t *out_num_accepted, int B, int gamma_max, int V,
                              spec_dtype dtype, uint32_t *status, void *stream, float *p_hat, float *q_hat,
                              float *logz_t, float *logz_d, float *resid_mass, int32_t *seq_status,
                              const spec_verify_options *options);

/* spec_verify with explicit launch options (NULL = automatic).  Returns
 * SPEC_ERR_UNSUPPORTED if the device cannot co-schedule the requested shape. */
spec_status spec_verify_ex(const void *target_logits, const void *draft_logits, const int32_t *draft_tokens,
                           const int32_t *num_draft, const float *uniforms, const float *temperature,
                           int32_t *out_tokens, int32_t *out_num_accepted, int B, int gamma_max, int V,
                           spec_dtype dtype, uint32_t *status, void *stream, const spec_verify_options *options);

/* Sampling from one distribution per sequence: y_b ~ softmax(logits[b, :] / T_b)
 * by inverse CDF with u = uniforms[b] (the smallest id j with u * S < C_j), or
 * y_b = argmax logits[b, :] (lowest id on ties) when T_b == 0.  This is the
 * verification round with no drafts: the draft-side sampling of a proposer
 * ("Fast Inference from Transformers via Speculative Decoding" notes, method
 * details step 1: x ~ q) and target-only decoding, with the same kernels.
 *   logits [B, V] dtype; uniforms [B] float32 in [0, 1); temperature [B];
 *   out_tokens [B] int32 (-1 for a sequence with an invalid temperature or a
 *   sampled row without a finite normaliser; its bit goes to *status).
 * options: as for spec_verify_ex.
 * Same ownership, stream and error rules as spec_verify. */
spec_status spec_sample(const void *logits, const float *uniforms, const float *temperature, int32_t *out_tokens,
                        int B, int V, spec_dtype dtype, uint32_t *status, void *stream,
                        const spec_verify_options *options);

/* Prompt-lookup (n-gram) proposer: drafts without a model.  "Speculative
 * Decoding" (atonlee.tistory.com/330) ch.5: find the current suffix earlier in
 * the context and propose the tokens that followed it; the vLLM section of
 * "Speculative Decoding으로 LLM 추론 속도 높이기" sets the n-gram lengths with
 * prompt_lookup_min / prompt_lookup_max.  For each sequence b, with
 * L = context_len[b] tokens in context[b * context_stride, +L): the longest
 * n in [min_n, max_n] whose last-n-token suffix also occurs at an earlier start
 * j < L - n wins, and among its occurrences the most recent one; the proposal
 * is the min(gamma_max, L - (j + n)) tokens after it.  No occurrence: no
 * drafts.
 *   context        int32, row b starts at b * context_stride (device memory,
 *                  or mapped host memory as for spec_verify)
 *   context_len    [B] int32, clamped to [0, context_stride]
 *   draft_tokens   [B, gamma_max] int32 (written; -1 after the proposal)
 *   num_draft      [B] int32 (written)
 * Limits: 1 <= min_n <= max_n <= 64, 0 <= gamma_max <= SPEC_MAX_GAMMA.  One
 * kernel on 'stream'; allocates nothing.  The proposals feed spec_verify with
 * draft_logits == NULL (point-mass proposals). */
spec_status spec_ngram_propose(const int32_t *context, int64_t context_stride, const int32_t *context_len, int B,
                               int min_n, int max_n, int gamma_max, int32_t *draft_tokens, int32_t *num_draft,
                               void *stream);

/* Candidate-tree verification: one round in which the target checked a tree
 * of candidates in one forward ("Speculative Decoding" (atonlee.tistory.com/
 * 330) ch.5: Medusa heads propose their top few tokens per position, the
 * combinations form a tree checked through a tree attention mask; the EAGLE
 * paragraph of "Speculative Decoding으로 LLM 추론 속도 높이기": EAGLE-2 drafts
 * a tree).  For each sequence b with nn = num_nodes[b] nodes:
 *   node 0 is the root (the last emitted token); node k in [1, nn) carries the
 *   candidate id tokens[b, k] and hangs under parent[b, k] in [0, k);
 *   target_logits[b, k, :] is the target's next-token logits after the path
 *   root..k (row 0: after the root).
 * The candidates are deterministic (a proposer's top tokens), i.e. point
 * masses.  Walking from the root, the children of the current node are tried
 * in index order with the single-candidate rule ("Speculative Decoding"
 * ch.3) applied to p without the ids already rejected there (R): child c is
 * accepted iff uniforms[b, c] * (1 - p(R)) < p(tokens[b, c]), p = softmax(row /
 * T_b); the first accepted child becomes the current node.  When none is (or
 * the node is a leaf), one token is sampled from p without R, renormalised,
 * by inverse CDF with uniforms[b, 0] (smallest j with u*S < C_j on the exact
 * fixed-point grid), which keeps the target's law at every step; with one
 * child per node this is spec_verify with point-mass drafts.  T_b == 0: the
 * accepted child is the first whose id is the argmax of the node's raw
 * logits (lowest id on ties), and the walk ends by emitting that argmax.
 * Only the rows on the accepted path are read.
 *   target_logits  [B, max_nodes, V] dtype; rows of nodes >= nn are never read
 *   parent, tokens [B, max_nodes] int32 (entries 0 and >= nn ignored)
 *   num_nodes      [B] int32 in [1, max_nodes]
 *   uniforms       [B, max_nodes] float32 in [0, 1): column c tests node c,
 *                  column 0 drives the final sample
 *   temperature    [B] float32 (0: greedy)
 *   out_tokens     [B, max_nodes] int32: the n accepted ids, then the sampled
 *                  (or argmax) id, then -1
 *   out_num_accepted [B] int32: n, the accepted path length
 *   out_path       [B, max_nodes] int32 or NULL: the accepted node indices,
 *                  then -1 (for keeping their cache entries)
 * Invalid data (num_nodes outside [1, max_nodes], a parent outside [0, k), a
 * candidate id outside [0, V), a bad temperature, a sampled row on the path
 * without a finite normaliser) gives -1 tokens, n = 0 and a status bit
 * (SPEC_STATUS_BAD_NUM_DRAFT for num_nodes, SPEC_STATUS_BAD_TREE, ...).
 * options: cluster_size and counters as for spec_verify_ex (counters add
 * nn - 1 candidates, n accepted, 1 sequence); kernel must be 0.  Limits:
 * 1 <= max_nodes <= SPEC_MAX_TREE_NODES, 1 <= V <= SPEC_MAX_VOCAB.  Same
 * ownership, stream and error rules as spec_verify; allocates nothing. */
spec_status spec_tree_verify(const void *target_logits, const int32_t *parent, const int32_t *tokens,
                             const int32_t *num_nodes, const float *uniforms, const float *temperature,
                             int32_t *out_tokens, int32_t *out_num_accepted, int32_t *out_path, int B,
                             int max_nodes, int V, spec_dtype dtype, uint32_t *status, void *stream,
                             const spec_verify_options *options);

/* Launch shape spec_verify would use on the current device for these sizes
 * (device-memory rows): cluster size (CTAs per sequence), total CTAs, threads
 * per CTA and the kernel the automatic choice takes (2 = full sweep, 3 = early
 * exit; see spec_verify_options.kernel).  Any output pointer may be NULL.
 * Touches the device (attribute queries) but enqueues nothing. */
spec_status spec_verify_launch_shape(int B, int gamma_max, int V, spec_dtype dtype, int *cluster_size,
                                     int *num_ctas, int *threads_per_cta, int *kernel);

/* The address the kernels use for ptr: ptr itself for this device's memory,
 * the device alias for page-locked host memory mapped into the device's
 * address space (with unified addressing, the same value).  Returns
 * SPEC_ERR_INVALID_ARG (and leaves *device_ptr unchanged) for pageable or
 * unregistered host memory, another device's memory or a NULL argument, and
 * SPEC_ERR_CUDA if the runtime query fails.  Enqueues nothing. */
spec_status spec_device_pointer(const void *ptr, const void **device_ptr);

/* ---------------------------------------------------------------------------
 * The target's key/value cache, held in 8 bits.
 *
 * Tokens live in blocks ("pages") of `block` tokens.  Per block and key/value
 * head there is one scale for the keys and one for the values: token value =
 * code * scale, the code an 8-bit float (e4m3: largest 448, or e5m2: largest
 * 57344).  Sequence b's token j is row j % block of page
 * block_table[b * table_stride + j / block].
 * Rejected drafts of a chain leave the cache by length alone: the next append
 * writes over them.  The accepted path of a candidate tree lies scattered among
 * its nodes: append its keys and values once more at the length before the tree
 * (node 0, then spec_tree_verify's out_path), and count those.
 *   k, v            codes; element (page, head, row, d) at
 *                   page * stride[0] + head * stride[1] + row * stride[2] + d bytes;
 *                   16-byte aligned, strides positive multiples of 16
 *   k_scale, v_scale [num_pages, kv_heads] float32, dense
 *   positions       [num_pages, kv_heads, block] int32, dense, or NULL: the
 *                   position of each cached token in its text, which the bias by
 *                   distance uses (NULL: the token's index j).  16-byte aligned.
 *   block_table     [batch, >= max_blocks] int32
 * A length is valid in [0, max_blocks * block], which is SPEC_MAX_CACHED at most.  Data problems never trap: a
 * sequence with a length (or number of new tokens) out of range is skipped, its
 * outputs zero (lse -inf, lengths 0), and a token on a page outside
 * [0, num_pages) counts as not cached; SPEC_STATUS_BAD_LENGTH and
 * SPEC_STATUS_BAD_PAGE are OR-ed into *status when status is not NULL.  Scales
 * that a call reads are positive and finite (attention is made for those that
 * spec_cache_append chooses, 2^-100 to 2^120; smaller ones may count as 0).
 * Ownership, stream and error rules as for spec_verify, but that a call may
 * enqueue up to three kernels; every array is device memory.  Nothing is
 * allocated. */
#define SPEC_MAX_CACHED (1 << 30) /* tokens of a sequence: loops over them count in 32 bits */

typedef enum { SPEC_E4M3 = 0, SPEC_E5M2 = 1 } spec_code;

typedef struct spec_cache {
    void *k, *v;
    float *k_scale, *v_scale;
    int32_t *positions;
    const int32_t *block_table;
    int64_t k_stride[3], v_stride[3];
    int64_t table_stride;
    int32_t batch, max_blocks, num_pages, kv_heads, block, dim; /* block 16, 32, 64 or 128; dim 64 or 128 */
    int32_t code;                                               /* spec_code */
} spec_cache;

/* Writes new tokens: token i < num_new[b] of k, v [batch, n, kv_heads, dim]
 * (float32 or bf16, element strides of the first three dimensions in k_stride
 * and v_stride, the last one dense) becomes cached token lengths[b] + i, in
 * 8 bits.  For each block that is written, with s_old its scale if it already
 * holds tokens of this sequence (index < lengths[b]) and nothing else:
 *   s = max(s_old, 2^e), 2^e the smallest power of two with |x| <= 2^e * top
 *       for every finite new x of the block and head (2^-100 at least);
 *   new codes round(x / s) to nearest even; the older codes become
 *   round(code * s_old / s) where s differs from s_old.
 * A power of two costs a floating-point code no precision, and moving a code to
 * a larger power of two is exact down to the subnormal codes.  Infinities and
 * NaN are stored as NaN and do not enter s.  lengths is not changed (the caller
 * adds num_new, or, after a verification round, the accepted part of it).  A
 * block that a call writes belongs to one sequence; full blocks may be shared.
 *   num_new    [batch] int32 in [0, n], or NULL: n for every sequence
 *   positions  [batch, n] int32 or NULL (lengths[b] + i), written to
 *              cache.positions where that is present */
spec_status spec_cache_append(const spec_cache *cache, const int32_t *lengths, const void *k, const void *v,
                              const int64_t k_stride[3], const int64_t v_stride[3], int n, spec_dtype dtype,
                              const int32_t *num_new, const int32_t *positions, uint32_t *status, void *stream);

/* How queries see the cache.  Query i < m (m = num_new[b], or n) of sequence b
 * is the token at index a_i = lengths[b] - m + i: the newest m cached tokens
 * ask.  It sees token j < lengths[b] when
 *   parent == NULL: j <= a_i; else j < lengths[b] - m, or token j is node i or
 *     an ancestor of it in the candidate tree (node k is token lengths[b] - m + k,
 *     parent[b, k] in [0, k) for k >= 1, as in spec_tree_verify); n <= 256;
 *   and, with window > 0, j > a_i - window;
 *   or j < prefix[b] (a prefix that every query sees, also outside the window).
 * Its score is x = scale * q.k, then softcap * tanh(x / softcap) where softcap
 * > 0, then - slopes[head] * |position(a_i) - position(j)| where slopes is given.
 * A row that sees nothing gets zeros and lse = -inf.  Scores past 2^29 in magnitude
 * count as infinite: a row that sees a positive one becomes NaN, one that sees none
 * but negative ones is as if it saw nothing.  A parent outside [0, k)
 * counts as no parent and sets SPEC_STATUS_BAD_TREE.  What a query does not see
 * changes nothing in its row, NaN included; a NaN key that it sees makes its row
 * NaN, a NaN value that dimension of its row or all of it. */
typedef struct spec_cache_form {
    float scale, softcap;
    int32_t window;
    const float *slopes;    /* [heads] or NULL */
    const int32_t *prefix;  /* [batch] or NULL */
    const int32_t *parent;  /* [batch, n] or NULL */
    const int32_t *num_new; /* [batch] in [0, n] or NULL (n) */
} spec_cache_form;

/* Attention: out[b, i, h, :] = sum_j softmax_j(x) v_j, lse[b, i, h] the natural
 * logarithm of the sum of exp(x).  Query head h reads key/value head
 * h / (heads / kv_heads).  Rows i >= num_new[b] are zeros with lse = -inf.
 *   q    [batch, n, heads, dim] bf16, element strides q_stride (multiples of 8),
 *        16-byte aligned, the last dimension dense
 *   out  [batch, n, heads, dim] bf16, 16-byte aligned; lse [batch, n, heads] float32
 *   workspace  spec_cache_attend_workspace bytes, 16-byte aligned; its contents
 *              do not matter and concurrent calls need one each
 * Precision.  Scores, the softmax's sums and lse are 32-bit; out is rounded to
 * bf16 once.  The products take 8-bit operands, so what multiplies the codes is
 * held as two or three of them:
 *   a query's elements are exact down to 2^-14 of the largest of their row, and
 *     off by at most 2^-21 of that one below;
 *   a token's softmax weight is off by at most r of itself or, where that is more,
 *     by s of the largest weight times the largest value scale of the 128 tokens
 *     (counted from the sequence's first) that it lies among, divided by its own
 *     value scale: r = 2^-10 and s = 2^-21 with up to 32 rows (queries times query
 *     heads) a key head, as in a round of drafts; r = 2^-8, as in bf16, and s =
 *     2^-17 with more, as in a prompt.
 * The second part matters only in dimensions that the tokens of most weight leave
 * near 0; there, weights of less than s / 2 of the largest one count as 0. */
spec_status spec_cache_attend(const spec_cache *cache, const int32_t *lengths, const void *q,
                              const int64_t q_stride[3], int n, int heads, const spec_cache_form *form, void *out,
                              float *lse, void *workspace, int64_t workspace_bytes, uint32_t *status, void *stream);
spec_status spec_cache_attend_workspace(const spec_cache *cache, int n, int heads, int64_t *bytes);

/* How many clocks of an SM a wait inside spec_cache_attend's and spec_cache_weigh's
 * kernels may take (2^31 - 1, about a second, if this is never called).  A kernel
 * whose wait ran out ends all the same and sets SPEC_STATUS_INTERNAL: give those
 * calls a status to learn of it.  The limit holds for the calls that this process
 * makes from now on; a captured call keeps the one it was captured with. */
spec_status spec_cache_set_wait_limit(int clocks);

/* Attention weight received: weights[page, kv head, row] += sum over the m
 * queries and the head's query heads of exp(x - lse), for every cached token of
 * every sequence (lse as spec_cache_attend gave it; rows whose lse is -inf add
 * nothing).  weights [num_pages, kv_heads, block] float32, dense.  Each sum has
 * a fixed order.  Nothing else adds to weights or clears them (spec_cache_append
 * leaves them as they are): a slot must hold 0 when a token is written to it.  In
 * a speculative round, call this after the accept test with the accepted tokens
 * only (their number as num_new, lengths to match, the same q and lse); then the
 * slots of rejected tokens stay at 0 and what those looked at does not count.
 * A query's elements are exact down to 2^-10 of the largest of their row and off
 * by at most 2^-17 of it below; all else is 32-bit.  workspace: as for spec_cache_attend.  Pages that several sequences share must not be weighed in one
 * call: their sums would race. */
spec_status spec_cache_weigh(const spec_cache *cache, const int32_t *lengths, const void *q,
                             const int64_t q_stride[3], int n, int heads, const spec_cache_form *form,
                             const float *lse, float *weights, void *workspace, int64_t workspace_bytes,
                             uint32_t *status, void *stream);

/* Eviction: of each sequence and key/value head, the `recent` newest tokens and,
 * of the others, the keep - recent with the largest weights (the lower index on
 * ties, NaN below every number), or all tokens when there are no more than
 * `keep`.  They are moved, in their order, with their weights and positions, to
 * the pages of out_table[b * out_stride + ...], ceil(keep / block) each, which
 * must be in no sequence's block_table.  A new block's scale is the largest of
 * its tokens' scales, the codes as for spec_cache_append.  A kept token on a page
 * out of range becomes one of zeros with weight and position 0 (a block of
 * nothing else gets the scale 2^-100).
 *   out_lengths [batch] int32: min(lengths[b], keep); may be lengths itself
 *   out_index   [batch, kv_heads, keep] int32: the kept indices, then -1
 * Limits: 1 <= keep, 0 <= recent <= keep. */
spec_status spec_cache_evict(const spec_cache *cache, const int32_t *lengths, float *weights, int keep, int recent,
                             const int32_t *out_table, int64_t out_stride, int32_t *out_lengths, int32_t *out_index,
                             uint32_t *status, void *stream);

/* Static description of a status code. */
const char *spec_status_string(spec_status s);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
