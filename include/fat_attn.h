/*
 * fat_attn.h -- C ABI of the GB300 (sm_103a) fused attention library with an in-kernel
 * relative-position bias (T5 log-bucket table and/or ALiBi), padding-free varlen packing,
 * forward and backward.
 *
 * What is computed. FAT5 report, "Noyau CUDA" section (second kernel version, "Flash Attention
 * RPE"): per document and head, S = Q K^T, S' = S + B, P = softmax(S'), O = P V, where B is not
 * passed in but built inside the kernel from the relative position of each (query, key) pair, so
 * that memory stays linear in the sequence length. Readings of points the pages leave open:
 *   - scale: S' = softmax_scale * (Q K^T) + B (the scale does not multiply the bias);
 *   - relative position: delta = key_position - query_position, positions local to each
 *     document (they restart at 0 at every cu_seqlens boundary: padding-free packing page);
 *   - T5 bias: B = bias_table[bucket(delta), head] with the T5 paper's log-bucket function
 *     (exact real floor; bidirectional: negative deltas use buckets [0, nb/2), positive ones
 *     [nb/2, nb); causal/unidirectional: only delta <= 0 is distinguished);
 *   - ALiBi bias: B = -alibi_slopes[head] * |delta|; T5 and ALiBi may be combined (they add);
 *   - causal: keys with delta > 0 are masked (top-left aligned, self-attention per document);
 *   - backward: gradients of sum(out * dout) with the standard softmax-attention calculus
 *     (the pages benchmark the backward, "Benchmark / TFLOPS" section, but give no derivation);
 *     the bias-table gradient sums dS over all (query, key) pairs that share a bucket.
 *
 * Layout (all row-major, contiguous, device memory unless stated):
 *   q, k, v, out, dout, dq, dk, dv : bf16 [total_tokens, num_heads, head_dim]
 *   lse                            : fp32 [num_heads, total_tokens], natural-log logsumexp of S'
 *   cu_seqlens                     : int32 [num_seqs + 1], cu[0] = 0, non-decreasing,
 *                                    cu[num_seqs] = total_tokens (read on the device only)
 *   bias_table, dbias_table        : fp32 [num_buckets, num_heads]
 *   alibi_slopes                   : fp32 [num_heads]
 * Every pointer must be 16-byte aligned. head_dim must be 64 or 128.
 *
 * Ownership and execution. The caller allocates every buffer, including the backward
 * workspace; no call allocates device memory. Calls are asynchronous on shape->stream (a
 * cudaStream_t; NULL = legacy default stream) and return after enqueueing. Global state: a
 * device error word per GPU (see fat_attn_get_device_error) and the scratch array of
 * fat_attn_bwd_noalloc (FAT_NOALLOC_SCRATCH_BYTES per GPU), both file-scope device variables
 * that every GPU on which the library's module is loaded holds until the process exits, whether
 * or not those calls are made; and a host-side cache of encoded TMA tensor maps, keyed by every
 * field they encode (address, sizes, tile box, element type), so that a cached map is identical
 * to a fresh one.
 *
 * Errors. Every call returns 0 on success or a negative FAT_E* code; nothing throws, exits or
 * traps. Argument errors are detected on the host before anything is enqueued. Device-side
 * problems (a pipeline wait that exceeded its time limit, a cu_seqlens entry outside
 * [0, total_tokens]) make the kernel skip the remaining work of that block and set a bit in the
 * device error word, which fat_attn_get_device_error reports.
 */
#ifndef FAT_ATTN_H
#define FAT_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define FAT_OK 0
#define FAT_EINVAL_NULL (-1)    /* a required pointer is NULL */
#define FAT_EINVAL_SHAPE (-2)   /* bad size, head_dim not 64/128, misaligned pointer */
#define FAT_EINVAL_BUCKETS (-3) /* bad num_buckets / max_distance / bidirectional */
#define FAT_ECUDA (-4)          /* a CUDA runtime/driver call failed (launch, tensor map, ...) */
#define FAT_EUNSUPPORTED (-5)   /* valid but unsupported combination (see each call) */
#define FAT_EDEVICE (-6)        /* the device error word was set (see below) */

/* bits of the device error word */
#define FAT_DEVERR_TIMEOUT_FWD 1 /* a forward pipeline wait exceeded its time limit */
#define FAT_DEVERR_TIMEOUT_BWD 2 /* a backward pipeline wait exceeded its time limit */
#define FAT_DEVERR_INDEX 8       /* a target beyond the vocabulary, a slot beyond the cache, a tree's bad
                                    parent or position */
#define FAT_DEVERR_SEQLENS 4     /* cu_seqlens had an entry outside [0, total_tokens] or out of
                                    order, or a document longer than max_seqlen (its rows beyond
                                    the grid were not computed) */
#define FAT_DEVERR_PAGES 16      /* paged cache: the free pages or a table row do not hold a request,
                                    or a page index lies outside the cache */

typedef struct {
  int32_t total_tokens; /* T: sum of document lengths (rows of q, k, v) */
  int32_t num_seqs;     /* n: number of documents; cu_seqlens has n + 1 entries */
  int32_t max_seqlen;   /* upper bound on every document length (sizes the grid; must not be
                           smaller than the longest document: the host cannot check it, the
                           kernels report a longer one as FAT_DEVERR_SEQLENS) */
  int32_t num_heads;    /* H (q, k and v share the head count) */
  int32_t head_dim;     /* d: 64 or 128 */
  void *stream;         /* cudaStream_t the work is enqueued on */
} fat_shape_t;

/*
 * Forward. out = softmax(softmax_scale * Q K^T + B) V per document and head; lse = logsumexp
 * of the same logits (natural log). The bias B is the sum of the T5 term (when bias_table is
 * not NULL: num_buckets, max_distance, bidirectional describe the bucket function; bidirectional
 * needs an even num_buckets; the buckets per direction nbh must satisfy 2 <= nbh <= 128 and
 * max_distance > nbh/2) and the ALiBi term (when alibi_slopes is not NULL). Both NULL gives
 * plain attention. lse may be NULL if the caller does not need it (the backward needs it).
 * FAT_EUNSUPPORTED: the bucket layout needs a larger in-kernel lookup table than shared memory
 * holds. The table has sat_pos + sat_neg + 507 entries (sat_neg = the saturation distance of
 * fat_attn_bucket_thresholds, sat_pos = the same when bidirectional, else 0); the forward takes
 * up to 24687 entries at head_dim 64 and 8303 at head_dim 128 (32 buckets, bidirectional:
 * max_distance up to 34404 / 9436).
 */
int fat_attn_fwd(const fat_shape_t *shape, const void *q, const void *k, const void *v,
                 const float *bias_table, int num_buckets, int max_distance, int bidirectional,
                 const float *alibi_slopes, const int32_t *cu_seqlens, int causal,
                 float softmax_scale, void *out, float *lse);

/*
 * fat_attn_fwd with a caller-owned device workspace (may be NULL). When every document has
 * length max_seqlen (total_tokens = num_seqs * max_seqlen), there is no causal mask, and the
 * forward grid (one CTA per 256 query rows x head x document, one per SM) ends in a partial
 * wave, a workspace of at least fat_attn_fwd_workspace_size(shape) bytes (256-byte aligned;
 * contents need not be initialised) lets the library split that wave's CTAs along the keys
 * and merge their partial rows in a second pass, so the last wave no longer leaves most SMs
 * idle. A smaller workspace (or NULL) gives the fat_attn_fwd schedule; results agree up to the
 * rounding of the merge. Errors as fat_attn_fwd; a misaligned workspace: FAT_EINVAL_SHAPE.
 */
int fat_attn_fwd_ws(const fat_shape_t *shape, const void *q, const void *k, const void *v,
                    const float *bias_table, int num_buckets, int max_distance, int bidirectional,
                    const float *alibi_slopes, const int32_t *cu_seqlens, int causal,
                    float softmax_scale, void *out, float *lse, void *workspace,
                    size_t workspace_bytes);
/* Bytes fat_attn_fwd_ws uses for this shape on the current device (its SM count sets the
   waves): 0 when the shape has no split last wave. */
size_t fat_attn_fwd_workspace_size(const fat_shape_t *shape);

/* Bytes of device workspace for fat_attn_bwd at its fastest. The layout starts with an fp32 dQ
   accumulator [T, H, d] and the fp32 row statistics D = rowsum(dout * out) [H, T], each
   256-byte aligned: that prefix is the minimum every backward call accepts. Shapes whose
   documents all have length max_seqlen (total_tokens = num_seqs * max_seqlen) and whose
   one-CTA-per-key-tile backward grid ends in a partial wave (head_dim 128, or more than 8192
   keys at head_dim 64) add fp32 dK/dV rows for splitting that wave along the queries, which
   fat_attn_bwd uses without the causal mask when the workspace holds them (the dK/dV of those
   rows are then summed with fp32 atomics: order-dependent rounding). The size depends on the
   current device's SM count. */
size_t fat_attn_bwd_workspace_size(const fat_shape_t *shape);

/*
 * Backward of sum(out * dout) for the forward above (same bias, mask and scale arguments).
 * Inputs: q, k, v, out and lse from the forward, dout. Outputs dq, dk, dv (bf16) and, when
 * dbias_table is not NULL (requires bias_table), the T5 table gradient, which is OVERWRITTEN
 * (zeroed by the library, then accumulated with fp32 atomics: bit-exact bucket assignment,
 * order-dependent rounding). ALiBi slopes receive no gradient. workspace must hold
 * fat_attn_bwd_workspace_size(shape) bytes; its contents need not be initialised.
 * It enqueues the three stages below; the second and third are launched as programmatic
 * dependents of the grid before them (each is scheduled while that grid drains and waits for
 * its outputs inside the kernel), which the stage-by-stage calls do not do.
 * FAT_EUNSUPPORTED: the lookup table (entries as for the forward), with its per-delta gradient
 * sums, does not fit next to the backward's tiles: up to 3083 entries at head_dim 64 and 6951
 * at head_dim 128 (32 buckets, bidirectional: max_distance up to 2661 / 7590).
 */
int fat_attn_bwd(const fat_shape_t *shape, const void *q, const void *k, const void *v,
                 const float *bias_table, int num_buckets, int max_distance, int bidirectional,
                 const float *alibi_slopes, const int32_t *cu_seqlens, int causal,
                 float softmax_scale, const void *out, const float *lse, const void *dout,
                 void *workspace, size_t workspace_bytes, void *dq, void *dk, void *dv,
                 float *dbias_table);

/*
 * The three stages fat_attn_bwd runs, in order, on the same stream and workspace (exposed so
 * that callers can schedule or time them separately):
 *   preprocess: D = rowsum(dout * out) (fp32, into the workspace), zero the fp32 dQ
 *               accumulator, zero dbias_table when given (num_buckets rows);
 *   main:       dK, dV (written), dQ (accumulated into the workspace) and the table gradient
 *               (accumulated into dbias_table), one CTA per (document, head, 128-key tile);
 *   finalize:   dq = bf16(softmax_scale * dQ accumulator).
 * Arguments mean what they mean for fat_attn_bwd; the same errors apply.
 */
int fat_attn_bwd_preprocess(const fat_shape_t *shape, const void *out, const void *dout,
                            void *workspace, size_t workspace_bytes, float *dbias_table,
                            int num_buckets);
int fat_attn_bwd_main(const fat_shape_t *shape, const void *q, const void *k, const void *v,
                      const float *bias_table, int num_buckets, int max_distance,
                      int bidirectional, const float *alibi_slopes, const int32_t *cu_seqlens,
                      int causal, float softmax_scale, const float *lse, const void *dout,
                      void *workspace, size_t workspace_bytes, void *dk, void *dv,
                      float *dbias_table);
int fat_attn_bwd_finalize(const fat_shape_t *shape, const void *workspace,
                          size_t workspace_bytes, float softmax_scale, void *dq);

/*
 * Backward for callers that cannot allocate device memory (no counterpart in the paper; an
 * addition of this library). Examples: an application that owns every allocation on the GPU and
 * hands libraries only fixed, caller-owned buffers, or a plug-in inside a framework whose
 * allocator must not be bypassed and which offers no way to request scratch space. Such a caller
 * cannot provide the workspace fat_attn_bwd needs, so this entry point uses a scratch array of
 * FAT_NOALLOC_SCRATCH_BYTES that the library keeps in device memory: every GPU that loads the
 * library holds it until the process exits. Otherwise it is fat_attn_bwd (same arguments minus
 * the workspace, same results, same errors); it allocates nothing and calls nothing that does.
 *   - Limit: problems whose fat_attn_bwd_workspace_size() exceeds FAT_NOALLOC_SCRATCH_BYTES are
 *     rejected with FAT_EUNSUPPORTED before any work is enqueued (fat_attn_last_error_message
 *     says why); e.g. T * H * (d + 1) * 4 bytes must fit, about 8 M elements of q at d = 64.
 *   - The first call on a device looks up the array's device address with that device current;
 *     make that first call before any stream capture. Make the device of shape->stream current
 *     for every call (as for any kernel launch); resetting a device after its first call is not
 *     supported (the looked-up address is kept for the life of the process).
 *   - Argument errors are reported exactly as fat_attn_bwd reports them, before the size test.
 *   - All calls on a device share the one array, which keeps whatever the last call left there
 *     (each call zeroes the part that must start at zero). Calls whose work overlaps on the GPU
 *     (other streams, other host threads) race on it and must be serialised by the caller.
 */
#define FAT_NOALLOC_SCRATCH_BYTES (32u << 20)
int fat_attn_bwd_noalloc(const fat_shape_t *shape, const void *q, const void *k, const void *v,
                         const float *bias_table, int num_buckets, int max_distance,
                         int bidirectional, const float *alibi_slopes, const int32_t *cu_seqlens,
                         int causal, float softmax_scale, const void *out, const float *lse,
                         const void *dout, void *dq, void *dk, void *dv, float *dbias_table);

/*
 * Cross-attention, grouped-query heads and decode (own query and key lengths per document).
 *
 * What is computed. The FAT5 report keeps T5's encoder-decoder architecture ("Motivation"
 * section): the decoder attends over the encoder's output (cross-attention, query and key
 * sequences of different lengths; T5 puts no positional bias there) and, when generating, over
 * a key/value cache longer than the new queries; the report's plans for linear-cost inference
 * ("La suite" section) rest on that decode step. The pages give no formulas for these; the
 * readings, which reduce exactly to the self-attention calls above when every document has
 * Lq = Lk and num_heads_kv = num_heads_q:
 *   - per document, query p sits at key position p + (Lk - Lq): the last query lines up with
 *     the last key (bottom-right alignment); the relative position of the bias is
 *     delta = key_position - (p + Lk - Lq), and causal masks delta > 0;
 *   - query head h reads key/value head h / (num_heads_q / num_heads_kv) (grouped-query heads);
 *     the bias table and slopes are indexed by the query head;
 *   - a query row that sees no key (causal with Lk < Lq, or Lk = 0) has out = 0, lse = -inf and
 *     contributes no gradient;
 *   - the backward sums dK, dV of a key/value head over the query heads that read it.
 * Layout: q, out, dout, dq bf16 [total_q, num_heads_q, head_dim]; k, v, dk, dv bf16
 * [total_k, num_heads_kv, head_dim]; lse fp32 [num_heads_q, total_q]; cu_seqlens_q and
 * cu_seqlens_k int32 [num_seqs + 1] (device); bias_table / dbias_table fp32
 * [num_buckets, num_heads_q]; alibi_slopes fp32 [num_heads_q]. Ownership, alignment, errors and
 * streams as above; num_heads_q must be a multiple of num_heads_kv.
 */
typedef struct {
  int32_t total_q;      /* rows of q, out, dout, dq */
  int32_t total_k;      /* rows of k, v, dk, dv */
  int32_t num_seqs;     /* documents; both cu_seqlens arrays have num_seqs + 1 entries */
  int32_t max_seqlen_q; /* bound on every document's query count (a longer one is reported as
                           FAT_DEVERR_SEQLENS) */
  int32_t max_seqlen_k; /* bound on every document's key count (likewise) */
  int32_t num_heads_q;
  int32_t num_heads_kv; /* divides num_heads_q */
  int32_t head_dim;     /* 64 or 128 */
  void *stream;         /* cudaStream_t */
} fat_xshape_t;

/* Forward of the generalised problem (arguments as fat_attn_fwd, with both cu_seqlens). */
int fat_xattn_fwd(const fat_xshape_t *shape, const void *q, const void *k, const void *v,
                  const float *bias_table, int num_buckets, int max_distance, int bidirectional,
                  const float *alibi_slopes, const int32_t *cu_seqlens_q,
                  const int32_t *cu_seqlens_k, int causal, float softmax_scale, void *out,
                  float *lse);

/*
 * The same forward with the keys of every document split into num_splits ranges, each range
 * computed by blocks of its own, and the partial results merged by a second grid
 * (out = sum_s exp(lse_s - lse) out_s, lse = log sum_s exp(lse_s)). For decode steps and other
 * problems with few query rows and long key sequences, where whole rows alone would occupy only
 * a few SMs. num_splits in [1, 64] (1 = fat_xattn_fwd); fat_xattn_splitkv_num_splits suggests
 * one (about two blocks per SM). The workspace (256-byte aligned, contents need not be
 * initialised) holds the partial outputs: fat_xattn_splitkv_workspace_size bytes (0 for one
 * split). num_seqs * num_splits must not exceed 65535 (FAT_EUNSUPPORTED).
 */
int fat_xattn_splitkv_num_splits(const fat_xshape_t *shape);
size_t fat_xattn_splitkv_workspace_size(const fat_xshape_t *shape, int num_splits);
int fat_xattn_fwd_splitkv(const fat_xshape_t *shape, const void *q, const void *k, const void *v,
                          const float *bias_table, int num_buckets, int max_distance,
                          int bidirectional, const float *alibi_slopes,
                          const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int causal,
                          float softmax_scale, int num_splits, void *workspace,
                          size_t workspace_bytes, void *out, float *lse);

/* Backward workspace of the generalised problem: the fp32 dQ accumulator [total_q, Hq, d];
   when num_heads_kv < num_heads_q also fp32 dK and dV accumulators [total_k, Hkv, d]; then D
   [Hq, total_q]; each 256-byte aligned (the minimum a call accepts); then, as for
   fat_attn_bwd_workspace_size, the rows of a split last wave when the shape has one (own
   key/value heads; with grouped heads the split wave adds into the dK/dV accumulators). */
size_t fat_xattn_bwd_workspace_size(const fat_xshape_t *shape);

/* Backward of the generalised problem (arguments as fat_attn_bwd, with both cu_seqlens). */
int fat_xattn_bwd(const fat_xshape_t *shape, const void *q, const void *k, const void *v,
                  const float *bias_table, int num_buckets, int max_distance, int bidirectional,
                  const float *alibi_slopes, const int32_t *cu_seqlens_q,
                  const int32_t *cu_seqlens_k, int causal, float softmax_scale, const void *out,
                  const float *lse, const void *dout, void *workspace, size_t workspace_bytes,
                  void *dq, void *dk, void *dv, float *dbias_table);

/*
 * Rotary position embedding (RoPE). The FAT5 report lists RoFormer's rotary embedding among the
 * positional encodings its attention kernels take ("Noyau CUDA" section); it prints no formula,
 * and the plainest reading is RoFormer's: channel pair (2i, 2i + 1) of a row at position m turns
 * by the angle m * base^(-2i/d) (base 10000 in RoFormer), positions local to each document
 * (restarting at every cu_seqlens boundary). Unlike the T5 and ALiBi biases it acts on Q and K
 * rather than on the logits: rotate q and k with this call, run fat_attn_fwd / fat_attn_bwd on
 * the rotated tensors (no bias), and turn dq and dk back with inverse = 1 (the rotation is
 * orthogonal, so the gradient of the unrotated input is the transposed rotation of the
 * rotated one's).
 *   x, y: bf16 [total_tokens, num_heads, head_dim] (y may equal x: in place); head_dim 64/128;
 *   cu_seqlens as for the attention calls; base > 1; inverse: 0 rotates, 1 turns back.
 * Angles are reduced exactly modulo one turn (64-bit fixed-point turns per position), so cosine
 * and sine carry fp32 accuracy at any position; the result is rounded to bf16.
 * A document longer than max_seqlen, or a corrupt cu_seqlens entry, sets FAT_DEVERR_SEQLENS.
 */
int fat_rope_apply(const fat_shape_t *shape, const void *x, void *y, const int32_t *cu_seqlens,
                   double base, int inverse);

/*
 * The FAT5 report's two other fused kernels ("Noyau Triton" section; their speed and memory are
 * compared with PyTorch in "Torch vs Triton"). The pages print no formulas; the readings:
 *
 * RMSNorm, the T5 layer norm (no mean subtraction, no bias):
 *   rstd = 1 / sqrt(mean_j x_j^2 + eps),  y = weight * x * rstd.
 * fat_rmsnorm_fwd: x, y bf16 [rows, dim]; weight fp32 [dim]; rstd fp32 [rows] (may be NULL; the
 *   backward needs it). dim a multiple of 256, at most 2048.
 * fat_rmsnorm_bwd: gradients of sum(y * dy): dx bf16 [rows, dim] and dweight fp32 [dim], which is
 *   OVERWRITTEN (zeroed by the call, then accumulated with fp32 atomics: order-dependent
 *   rounding). x, weight and rstd as given to / returned by the forward.
 *
 * Cross-entropy with a z-loss term (the auxiliary loss that keeps the log-partition near 0):
 *   lse = log sum_v exp(z_v),  loss = lse - z_target + z_loss * lse^2;
 *   rows with a negative target are ignored (loss 0, gradient 0).
 * fat_cross_entropy: logits bf16 [rows, vocab] (vocab a multiple of 8, at most 65536); target
 *   int32 [rows]; loss and lse fp32 [rows] (either may be NULL). When dlogits (bf16
 *   [rows, vocab]) is not NULL, the gradient of grad_scale * sum(loss) is written there in the
 *   same pass (grad_scale = 1 / number of counted rows gives the mean's gradient):
 *   dz_v = grad_scale * (softmax_v * (1 + 2 z_loss lse) - [v == target]).
 *   A target at or beyond vocab sets FAT_DEVERR_INDEX (that row: loss 0, gradient 0).
 * All three are asynchronous on `stream` (a cudaStream_t), allocate nothing and return FAT_*.
 */
int fat_rmsnorm_fwd(long long rows, int dim, const void *x, const float *weight, float eps,
                    void *y, float *rstd, void *stream);
int fat_rmsnorm_bwd(long long rows, int dim, const void *x, const float *weight,
                    const float *rstd, const void *dy, void *dx, float *dweight, void *stream);
int fat_cross_entropy(long long rows, int vocab, const void *logits, const int32_t *target,
                      float z_loss, float grad_scale, float *loss, float *lse, void *dlogits,
                      void *stream);

/*
 * Cross-entropy of hidden rows over a vocabulary, the output layer's product and fat_cross_entropy's
 * loss in one, without the logits in memory (an addition of this library):
 *   z_rv = logit_scale * (hidden_r . weight_v),  lse_r = log sum_v exp(z_rv),
 *   loss_r = lse_r - z_r,target + z_loss * lse_r^2;
 *   rows with a negative target are ignored (loss 0, gradient 0; lse is theirs all the same).
 * With few rows: minus the loss is the log-probability of a drafted token.
 *   hidden: bf16 [rows, dim], weight: bf16 [vocab, dim], rows hidden_stride and weight_stride elements
 *   apart; target int32 [rows]; loss, lse fp32 [rows] (either may be NULL).
 * fat_linear_cross_entropy_bwd: gradients of grad_scale * sum_r dloss_r loss_r (dloss fp32 [rows]; NULL:
 *   ones), with lse as the forward gives it: dhidden bf16 [rows, dim] and dweight bf16 [vocab, dim], both
 *   contiguous and OVERWRITTEN, either NULL if it is not wanted. dz, the gradient of the logits, is
 *   rounded to bf16 (without grad_scale and logit_scale) as the operand of the two products; sums are
 *   fp32, without atomics whose order matters: a call's result does not depend on timing. Hidden rows
 *   that are ignored may hold anything (NaN, infinities); the others and the weights are finite.
 *   A target at or beyond vocab sets FAT_DEVERR_INDEX (that row: loss 0, gradient 0).
 * dim a multiple of 8, up to 65536; strides multiples of 8; any vocab and rows up to 2^28 each
 * (FAT_EUNSUPPORTED beyond, and for more than 2^30 tiles of 256 rows x 16 entries); logit_scale > 0,
 * z_loss >= 0. Index and statistics arrays need 4-byte alignment, the others 16. Results and workspace
 * lie over no other array of the call.
 * workspace: fat_linear_cross_entropy_workspace_size bytes (256-byte aligned, contents need not be
 * initialised), for one call at a time: captured graphs that may overlap take one each. One for a
 * number of rows does for fewer of the same vocab and dim. Its size depends on the current device's
 * SMs. The forward's holds 8 bytes for up to 128 logits of a row, and for calls of at least 1536 rows
 * whose dim is an odd multiple of 8 a copy of the hidden rows and weights with longer rows (odd
 * numbers of 16 bytes load at half the rate). The backward's holds a copy of the hidden rows; dz in
 * bf16, all of it (up to 128 MB) or two pieces of the vocabulary (256 MB); partial sums of dhidden in
 * fp32, dim * 1 KB for each 256 rows of up to 16384 and for up to three more for each pair of SMs and
 * 256 channels; and beyond 16384 rows dweight in fp32 as well, vocab * dim * 4 bytes.
 */
typedef struct {
  int32_t rows, vocab, dim;
  int64_t hidden_stride, weight_stride; /* elements from row to row */
  float logit_scale, z_loss;
  void *stream;
} fat_linear_ce_shape_t;
size_t fat_linear_cross_entropy_workspace_size(const fat_linear_ce_shape_t *shape, int backward);
int fat_linear_cross_entropy_fwd(const fat_linear_ce_shape_t *shape, const void *hidden,
                                 const void *weight, const int32_t *target, void *workspace,
                                 size_t workspace_bytes, float *loss, float *lse);
int fat_linear_cross_entropy_bwd(const fat_linear_ce_shape_t *shape, const void *hidden,
                                 const void *weight, const int32_t *target, const float *lse,
                                 const float *dloss, float grad_scale, void *workspace,
                                 size_t workspace_bytes, void *dhidden, void *dweight);

/*
 * Paged key/value cache: the operators of a serving step. (No counterpart in the FAT5 report beyond
 * its plans for inference, "La suite" section; an addition of this library.) A decoder that serves
 * many requests keeps their keys and values in pages of page_size tokens; a block table lists each
 * request's pages in order. One step brings some new tokens of some requests:
 *   fat_paged_plan    the step's maps on the GPU: pages taken from a free list, slots, positions;
 *   fat_paged_append  the new keys and values into their slots (rotary embedding on the way);
 *   fat_paged_attn    attention of the new tokens over their requests' pages.
 * Nothing here reads a length on the host, so a step can be captured in a CUDA graph and replayed
 * with other lengths. Index arrays (int32) need 4-byte alignment, everything else 16 bytes.
 */
typedef struct {
  void *k, *v;        /* bf16, read by fat_paged_attn, written by fat_paged_append */
  int32_t num_pages;
  int32_t page_size;  /* tokens per page: a power of two, 16 .. 65536; num_pages * page_size < 2^31 */
  int32_t num_heads;  /* key/value heads */
  int32_t head_dim;   /* a multiple of 8 (fat_paged_attn: 64 or 128) */
  /* strides of k and of v in elements, multiples of 8; a row of head_dim elements is contiguous.
     [num_pages, page_size, num_heads, head_dim] in memory order gives (page_size * num_heads *
     head_dim, num_heads * head_dim, head_dim); pages with the heads outside, or the pages of
     several layers in one block, give others. No two rows overlap. */
  int64_t stride_page, stride_token, stride_head;
} fat_paged_cache_t;

/*
 * The step's maps. Request i holds ctx_lens[i] cached tokens in the first ceil(ctx / page_size)
 * entries of its table row and brings new_lens[i] tokens. The pages it lacks are the next ones of
 * free_pages, request by request:
 *   block_table  [num_seqs, table_width]: the new pages' entries are written, the others stay;
 *   cu_seqlens_q [num_seqs + 1]: running sums of new_lens;  seqlens_k [num_seqs]: ctx + new;
 *   positions, slots [max_tokens]: of token cu_seqlens_q[i] + j, ctx_lens[i] + j and
 *     page * page_size + offset; tokens behind the last request get position 0 and slot -1 (a
 *     padded batch);
 *   counts [2]: pages needed (the caller drops that many entries of free_pages), tokens.
 * FAT_DEVERR_PAGES: the free list is too short (missing pages are written as -1), a request longer
 * than table_width pages (it takes none), or a page index outside [0, num_pages); the tokens
 * concerned get slot -1. FAT_DEVERR_SEQLENS: a negative length (taken as 0 and 0), or more tokens
 * than max_tokens (cu_seqlens_q stops there). table_width = 0 is a table without entries.
 * No result may lie over another array of the call (FAT_EINVAL_SHAPE): the lengths and the free list
 * are read until the end. A program that keeps its lengths in place copies seqlens_k over ctx_lens
 * behind the call.
 */
typedef struct {
  int32_t num_seqs, page_size, num_pages;
  int32_t table_width; /* entries of a block_table row */
  int32_t num_free;    /* entries of free_pages */
  int32_t max_tokens;  /* entries of positions and of slots */
  void *stream;
} fat_plan_shape_t;
int fat_paged_plan(const fat_plan_shape_t *shape, const int32_t *ctx_lens, const int32_t *new_lens,
                   const int32_t *free_pages, int32_t *block_table, int32_t *cu_seqlens_q,
                   int32_t *seqlens_k, int32_t *positions, int32_t *slots, int32_t *counts);

/*
 * Rotary embedding at explicit positions. The first rotary_dim channels of a head turn, the others
 * are copied: pair i by the angle position * theta'_i, theta_i = base^(-2 i / rotary_dim). Pairs
 * are the channels (2i, 2i + 1) when interleaved, else (i, i + rotary_dim / 2). For contexts longer
 * than a model was trained on:
 *   original_length = 0: theta'_i = theta_i / factor (factor = 1: as it is);
 *   original_length > 0: with t_i = original_length * theta_i / (2 pi) turns over that length and
 *     keep_i = clamp((t_i - low_turns) / (high_turns - low_turns), 0, 1):
 *     theta'_i = theta_i * (keep_i + (1 - keep_i) / factor);
 *   amplitude multiplies the turned channels.
 * fat_rope_init (host only) fills the record, which a program keeps for all its calls; its fields
 * are the library's own. rotary_dim: a multiple of 16, 16 .. 256; base > 1; factor, amplitude > 0
 * (amplitude as fp32, and no factor so small that a frequency overflows).
 */
#define FAT_ROPE_MAX_PAIRS 128
typedef struct {
  int32_t rotary_dim, interleaved;
  float amplitude;
  int32_t reserved;
  uint64_t rate[FAT_ROPE_MAX_PAIRS]; /* turns per position of each pair, 2^-64 units */
} fat_rope_t;
int fat_rope_init(fat_rope_t *rope, int rotary_dim, int interleaved, double base, double factor,
                  double low_turns, double high_turns, double original_length, double amplitude);

/*
 * y = the rotation of x (bf16 rows of head_dim channels) at positions[token] (int32, any value);
 * inverse = 1: its transpose, which turns the gradient of y into the gradient of x. y may be x
 * itself (equal strides) but not otherwise overlap it. Strides in elements, multiples of 8; rows of
 * x may repeat (stride 0), those of y lie apart. head_dim a multiple of 8, at least rotary_dim.
 * Angles are exact modulo one turn at any position, as in fat_rope_apply.
 */
typedef struct {
  int32_t tokens, num_heads, head_dim;
  int64_t x_stride_token, x_stride_head, y_stride_token, y_stride_head;
  void *stream;
} fat_rope_shape_t;
int fat_rope_embed(const fat_rope_shape_t *shape, const fat_rope_t *rope, const void *x, void *y,
                   const int32_t *positions, int inverse);

/*
 * New rows into the cache: token t's key and value rows [num_heads, head_dim] go to slot
 * slots[t] = page * page_size + offset; a negative slot drops them (padding), one at or beyond
 * num_pages * page_size drops them and sets FAT_DEVERR_INDEX. Slots of one call are distinct (if
 * one is named twice, each 16 bytes there come from either row). With `rope` the keys are turned at
 * positions[t] on the way (NULL: copied), and with q the queries are too, into q_out (bf16
 * [tokens, num_heads_q, head_dim] contiguous, of every token, padding included; q itself is
 * allowed when it is contiguous). q, k and v may be views of one packed projection: strides in
 * elements, multiples of 8. q and q_out are both given or both NULL; positions may be NULL without
 * rope. Neither the caches nor q_out (q aside) lie over the call's other arrays, nor over one another.
 */
typedef struct {
  int32_t tokens, num_heads_q;
  int64_t q_stride_token, q_stride_head, k_stride_token, k_stride_head, v_stride_token,
      v_stride_head;
  void *stream;
} fat_append_shape_t;
int fat_paged_append(const fat_append_shape_t *shape, const fat_paged_cache_t *cache,
                     const fat_rope_t *rope, const void *q, const void *k, const void *v,
                     const int32_t *positions, const int32_t *slots, void *q_out);

/*
 * Attention of new tokens over a paged cache: fat_xattn_fwd with request i's seqlens_k[i] keys in
 * the pages block_table[i][0 .. ceil(seqlens_k[i] / page_size)) instead of a packed array. Queries
 * q [total_q, num_heads_q, head_dim] are packed by cu_seqlens_q; the last query lines up with the
 * last key (append first); bias, causal mask, grouped heads, out and lse as there. Rows behind
 * cu_seqlens_q[num_seqs] are left as they were.
 *   - What lies in a page behind a request's last key is never used, whatever it holds (NaN and
 *     infinities included). Keys and values below seqlens_k are finite: a value that the causal
 *     mask hides from an earlier query of the same step still enters that query's product with
 *     weight 0, and an infinite one makes the output NaN. A NaN in a query, or in a key it sees, makes
 *     its output and lse NaN.
 *   - A bias of -infinity (or below -2e38: logits are formed times log2 e) masks its keys; a row
 *     that is left with none gets 0 and lse -infinity. Keys with large finite biases (-1e9) get the
 *     weight that fp32 can tell: none beside other keys; among themselves their logits are lost.
 *   - Requests may name the same pages (a common prefix).
 *   - A page index outside [0, num_pages) sets FAT_DEVERR_PAGES; its keys and values count as 0.
 *   - A request whose query count exceeds max_seqlen_q or whose seqlens_k is negative, exceeds
 *     max_seqlen_k or its table row (table_width pages) sets FAT_DEVERR_SEQLENS, as does a corrupt
 *     cu_seqlens_q; its rows are left as they were.
 *   - workspace: fat_paged_attn_workspace_size bytes (256-byte aligned, contents need not be
 *     initialised), for this call alone until it has finished: calls that may overlap, and captured
 *     graphs that do, take one each. The size never falls as total_q, num_seqs, max_seqlen_q or
 *     max_seqlen_k grows: one buffer for the largest bounds serves every smaller step too.
 *   - Logits, statistics and sums are fp32. Weights are rounded as operands of their product with the
 *     values: to 16 bits where max_seqlen_q * num_heads_q / num_heads is at most 16 (in a step of mixed
 *     lengths for the requests whose own queries make no more), else to bf16.
 * head_dim 64 or 128, num_heads_q / num_heads at most 128, max_seqlen_k at most 2^30.
 * A call whose total_q is exactly num_seqs * max_seqlen_q (beyond 16 rows a request, queries x
 * group) is taken as a batch of equal chunks; a step whose rows are padded to that total runs faster
 * with a row more.
 * FAT_EUNSUPPORTED: more query heads per key/value head, longer bounds, saturation distances of more
 * than 8192 keys in all (their buckets are looked up in shared memory), bias tables of more than 4096
 * entries a key/value head (num_buckets * num_heads_q / num_heads: a limit of what is tested), or cache
 * strides of which, in rising order, one is no multiple of the one before.
 */
typedef struct {
  int32_t total_q;      /* rows of q and out */
  int32_t num_seqs;
  int32_t max_seqlen_q; /* bounds on the requests' query and key counts */
  int32_t max_seqlen_k;
  int32_t num_heads_q;
  int32_t table_width;  /* entries of a block_table row */
  void *stream;
} fat_paged_shape_t;
size_t fat_paged_attn_workspace_size(const fat_paged_shape_t *shape,
                                     const fat_paged_cache_t *cache);
int fat_paged_attn(const fat_paged_shape_t *shape, const fat_paged_cache_t *cache, const void *q,
                   const int32_t *block_table, const int32_t *cu_seqlens_q,
                   const int32_t *seqlens_k, const float *bias_table, int num_buckets,
                   int max_distance, int bidirectional, const float *alibi_slopes, int causal,
                   float softmax_scale, void *workspace, size_t workspace_bytes, void *out,
                   float *lse);

/*
 * Trees of drafted tokens over a paged cache (verification of a tree in one step). Request i's new tokens are
 * the nodes of a tree (or of several): their keys and values are appended behind the cached context in
 * the nodes' order (fat_paged_plan's slots), but a node sees, besides the context, only its own path.
 *
 * fat_paged_tree_plan: parents [total_q], of each node the index, within its request, of the node that it
 * follows (an earlier one), or -1 where it follows the context. Results, of all total_q rows:
 *   positions [total_q]: seqlens_k - nodes + depth, what the node's rotary angles and biases go by;
 *   tree_mask [total_q, mask_words]: bit b of word w is node 32 w + b of the same request, set for the node
 *     itself and its ancestors.
 * Rows behind cu_seqlens_q[num_seqs], and of requests of more than max_seqlen_q nodes or whose
 * seqlens_k is smaller than their nodes (FAT_DEVERR_SEQLENS), get 0 and no bits; a parent that is no
 * earlier node counts as -1 (FAT_DEVERR_INDEX). With a corrupt cu_seqlens_q (FAT_DEVERR_SEQLENS) a
 * request whose bounds lie outside [0, total_q] or out of order writes no rows; where other bounds make
 * requests claim each other's rows, such a row holds what one of them, or the rows behind the last
 * one, gives it. mask_words at least ceil(max_seqlen_q / 32); max_seqlen_q at most 4096
 * (FAT_EUNSUPPORTED; a request has one warp, which drafted trees of up to some hundred nodes suit, and
 * larger ones are right but slow). The results lie over no other array of the call.
 */
typedef struct {
  int32_t total_q;      /* rows of parents, positions and tree_mask */
  int32_t num_seqs;
  int32_t max_seqlen_q; /* bound on the requests' node counts */
  int32_t mask_words;
  void *stream;
} fat_tree_shape_t;
int fat_paged_tree_plan(const fat_tree_shape_t *shape, const int32_t *parents,
                        const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int32_t *positions,
                        int32_t *tree_mask);

/*
 * fat_paged_attn for such trees: query j of a request sees the keys before the request's first query's
 * (index below seqlens_k - queries), and of its own queries' keys those whose bit is set in row j of
 * tree_mask (any pattern, not only paths; bits at or beyond the query count are not read as keys). A row that
 * sees nothing has out 0, lse -infinity. The bias's delta is key position - positions[j]; a key of the
 * context lies at its index, that of query k at positions[k]. A position outside [seqlens_k - queries,
 * seqlens_k) sets FAT_DEVERR_INDEX and is taken as the nearest end. All else, the workspace's size
 * too, as fat_paged_attn without its causal mask; a request with fewer keys than queries sets
 * FAT_DEVERR_SEQLENS and is left out. Keys and values that a node does not see are finite as well: they
 * enter its product with weight 0. Weights are rounded to 16 bits where max_seqlen_q * num_heads_q /
 * num_heads is at most 16, else to bf16, for every request of the call.
 */
int fat_paged_tree_attn(const fat_paged_shape_t *shape, const fat_paged_cache_t *cache, const void *q,
                        const int32_t *block_table, const int32_t *cu_seqlens_q,
                        const int32_t *seqlens_k, const int32_t *positions,
                        const int32_t *tree_mask, int mask_words, const float *bias_table,
                        int num_buckets, int max_distance, int bidirectional,
                        const float *alibi_slopes, float softmax_scale, void *workspace,
                        size_t workspace_bytes, void *out, float *lse);

/* Synchronises `stream`, reads the current GPU's device error word, clears it, and returns
   FAT_OK if it was zero, else FAT_EDEVICE with the word's bits stored in *bits (if not NULL). */
int fat_attn_get_device_error(void *stream, int *bits);

/* Static English description of a FAT_* return code. */
const char *fat_attn_strerror(int code);

/* Description of the last CUDA call that failed in this thread (which call, its error code and
   text); empty if none has. The string stays valid until the next failing call of the thread. */
const char *fat_attn_last_error_message(void);

/*
 * Host-only helper (no GPU needed): the integer thresholds the kernels compare distances with.
 * For t = 1 .. E-1 (E = nbh - nbh/2 log buckets per direction), thresholds[t-1] is the smallest
 * distance n with bucket_offset(n) >= nbh/2 + t. *count receives E - 1 and *saturation the
 * distance from which the bucket no longer changes. `thresholds` needs room for 63 entries.
 */
int fat_attn_bucket_thresholds(int num_buckets, int max_distance, int bidirectional,
                               int32_t *thresholds, int *count, int *saturation);

#ifdef __cplusplus
}
#endif
#endif /* FAT_ATTN_H */
