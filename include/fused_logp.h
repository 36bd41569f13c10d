/*
 * fused_logp.h: C ABI of the GB300 selected-token log-probability library
 * (libfused_logp.so, sm_103a).
 *
 * The operation (RL-Kernel issue #241 "TP-aware deterministic logprob",
 * Background and Goal): for BF16 logits x[N, V] and int64 targets y[N],
 *     LSE_t  = log sum_v exp(x[t, v])           (FP32 accumulation)
 *     logp_t = x[t, y_t] - LSE_t
 * and its gradient (RL-Kernel PR #495 "zero-workspace fused backward",
 * Summary item 2) for an upstream gradient g[N]:
 *     dlogits[t, v] = g_t * (onehot(y_t)[v] - exp(x[t, v] - LSE_t))
 * written straight to BF16 with no FP32 [N, V] workspace.
 *
 * A row is ACTIVE when 0 <= y_t < V and y_t != ignore_index.  Inactive rows
 * get logp = 0 and an all-zero gradient row (PR #495, Behavior changes:
 * out-of-range targets); their LSE is still computed.
 *
 * Vocabulary tiles.  Each row is cut into FLP_NUM_TILES = 16 fixed tiles of
 * width W = flp_tile_width(V) = 8 * ceil(V / 128) columns (the last ones
 * clipped or empty).  Every tile is reduced by the same fixed tree whatever N,
 * the row's position in the batch, or the shard that holds it; the 16 tile
 * partials are then merged in tile-index order.  This is the tile-level merge
 * of RL-Kernel PR #314 ("Deterministic config option", the tensor-parallel
 * section: fixed tiles reduced as the same shape on any rank, then one fixed
 * merge order), which makes results bitwise independent of N, of the row's
 * position and of the shard split.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers of one CUDA device, owned and allocated by
 *     the caller.  The library allocates nothing (no workspace, PR #495
 *     Summary item 2).  BF16 buffers are passed as void pointers to
 *     IEEE bfloat16 data.  Row-major with a row stride (ld) in elements.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream)
 *     and run on the device that holds `logits` (or the first device pointer);
 *     the caller's current device is restored before returning (the device
 *     guard of PR #495's review thread).
 *   - All extents and index arithmetic are int64 (PR #495 review: the
 *     int32 loop overflow near INT_MAX).
 *   - n == 0 returns FLP_OK without touching the device (PR #495 Tests:
 *     empty input).
 *   - Errors are reported by the return code, before any launch, with a
 *     thread-local message from flp_last_error().  Nothing traps on the GPU.
 *   - Results are deterministic: repeated calls give identical bits.
 */
#ifndef FUSED_LOGP_H
#define FUSED_LOGP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum flp_status {
    FLP_OK = 0,
    FLP_EINVAL = 1,        /* null pointer, bad extent or stride, host pointer,
                              pointers on different devices, bad overlap */
    FLP_EUNSUPPORTED = 2,  /* shard bounds off the tile grid */
    FLP_ECUDA = 3          /* a CUDA runtime call or the launch failed */
} flp_status;

/* Same type as cudaStream_t, declared without CUDA headers. */
typedef struct CUstream_st* flp_stream_t;

#define FLP_NUM_TILES 16

/* Logit dtypes of the _ex entry points (the gradient is written in the same
 * dtype).  PR #495 Tests name FP32/BF16/FP16 logits. */
#define FLP_DTYPE_BF16 0
#define FLP_DTYPE_F16 1
#define FLP_DTYPE_F32 2

/* Message of the last failing call on this thread ("" after success). */
const char* flp_last_error(void);

/* Library version string. */
const char* flp_version(void);

/* Tile width W for a vocabulary of v columns: 8 * ceil(v / 128); 0 if v < 1. */
int64_t flp_tile_width(int64_t v);

/*
 * Forward.  For t in [0, n):
 *   lse[t]  = M + log S, with (M, S) the index-order merge of the 16 tile
 *             partials (m_k, s_k), m_k = max over tile k, s_k = sum over tile
 *             k of exp(x - m_k), all FP32; the final log and add are carried
 *             in FP64 and rounded once to FP32.
 *   logp[t] = x[t, y_t] - lse (rounded once from FP64) if the row is active,
 *             else 0.
 *   logits   [n, ld] BF16, ld >= v >= 1 (columns >= v are never read)
 *   targets  [n] int64
 *   logp     [n] FP32 out
 *   lse      [n] FP32 out (keep it for the backward)
 *   lse_lo   [n] FP32 out, or NULL: the FP32 rounding residual of the LSE
 *            (LSE - lse, |lse_lo| <= half an ulp of lse).  Passing it to the
 *            backward removes the FP32 quantisation of the LSE from the
 *            gradient (an addition of this library; the pages store FP32 only).
 *            Both together hold LSE to 2^-48 |LSE|, and where M times the inverse
 *            temperature is a binary32 number (temperature 1) log S to 2^-24
 *            whatever M is.
 * Any alignment and any ld are accepted.  16-byte aligned rows with ld % 8 == 0
 * (and v < 2^31) stream through per-warp bulk-copy (TMA) rings in shared
 * memory; other layouts take a scalar-load path with the same arithmetic
 * (same bits).
 * Errors: FLP_EINVAL for n < 0, v < 1, ld < v, a null or host pointer.
 */
flp_status fused_logp_forward(const void* logits, int64_t n, int64_t v, int64_t ld,
                              const int64_t* targets, int64_t ignore_index,
                              float* logp, float* lse, float* lse_lo, flp_stream_t stream);

/*
 * Backward.  dlogits[t, c] for c in [0, v):
 *   active row:   g_t * (onehot(y_t)[c] - exp(x[t, c] - lse[t])), rounded
 *                 to nearest-even BF16 once, from an FP32 computation whose
 *                 exponent argument is carried with its rounding error;
 *   inactive row: +0.
 *   logits   [n, ld] BF16
 *   targets  [n] int64, lse [n] FP32 (from fused_logp_forward), grad [n] FP32
 *   lse_lo   [n] FP32 from fused_logp_forward, or NULL (then taken as 0)
 *   dlogits  [n, ld_out] BF16 out, ld_out >= v; columns >= v are untouched.
 * Gradient values below 2^-126 in magnitude flush to zero.
 * dlogits may alias logits exactly (same pointer and ld == ld_out: the
 * gradient then overwrites the logits in place); any other overlap is
 * FLP_EINVAL.  Elementwise, so batch-invariant by construction.
 */
flp_status fused_logp_backward(const void* logits, int64_t n, int64_t v, int64_t ld,
                               const int64_t* targets, int64_t ignore_index,
                               const float* lse, const float* lse_lo, const float* grad,
                               void* dlogits, int64_t ld_out, flp_stream_t stream);

/*
 * Vocab-shard partials (issue #241 PR 3 and PR 6 bullets; PR #314
 * ReductionSpec).  A shard holds global columns [vocab_start, vocab_start +
 * real_width) of a v_total-column vocabulary in its own buffer
 * shard_logits[n, ld_shard] (ld_shard >= real_width; columns >= real_width
 * are padding, masked to -inf, never read).  For each global tile k the shard
 * covers, writes part_max[t, k] and part_sum[t, k] (FP32, [n, 16] row-major),
 * bitwise equal to the forward's own tile partials.  For each row whose
 * target falls inside the shard, writes sel[t] = x[t, y_t] (the single-owner
 * copy of the selected logit); other rows' sel is left untouched.
 * The shard bounds must lie on the tile grid: vocab_start % W == 0, and
 * real_width % W == 0 unless the shard ends at v_total; otherwise
 * FLP_EUNSUPPORTED (the capability gate of issue #241 PR 6).
 * Columns of part_max/part_sum for tiles outside the shard are untouched.
 */
flp_status logp_shard_partials(const void* shard_logits, int64_t n, int64_t ld_shard,
                               int64_t vocab_start, int64_t real_width, int64_t v_total,
                               const int64_t* targets, float* part_max, float* part_sum,
                               float* sel, flp_stream_t stream);

/*
 * Merge (issue #241 PR 3 bullets: M = max m_l, S = sum s_l exp(m_l - M),
 * LSE = M + log S in fixed index order).  Folds the tile partials [n, 16]
 * of tiles 0 .. ceil(v_total / W) - 1 in index order with the same arithmetic
 * as the forward, then writes lse[t] and logp[t] = sel[t] - lse (active rows)
 * or 0.  Together with logp_shard_partials over shards that cover
 * [0, v_total), the results are bitwise equal to fused_logp_forward.
 * sel is read only for active rows.  lse_lo (nullable) as in the forward.
 */
flp_status logp_merge_partials(const float* part_max, const float* part_sum,
                               const float* sel, const int64_t* targets,
                               int64_t ignore_index, int64_t n, int64_t v_total,
                               float* logp, float* lse, float* lse_lo, flp_stream_t stream);

/*
 * Generalised forms (the calls above are these with FLP_DTYPE_BF16, no mask
 * and inv_temperature = 1).
 *   dtype           FLP_DTYPE_BF16 / FLP_DTYPE_F16 / FLP_DTYPE_F32: the dtype of
 *                   logits, shard_logits and dlogits.
 *   active_mask     [n] uint8 or NULL: a row is active only if its byte is
 *                   nonzero (and its target is in [0, v) and not ignore_index)
 *                   (PR #314, MaskMode explicit_active_mask).
 *   inv_temperature s = 1/T > 0, finite: the logits are scaled by s before the
 *                   log-softmax, as in rollout logprobs at a temperature (PR
 *                   #495, provider experiment at T = 1.0 and 0.7):
 *                   LSE = log sum exp(s x), logp = s x_y - LSE, and the
 *                   gradient with respect to the unscaled logits is
 *                   s g (onehot - exp(s x - LSE)).
 * Shard partials hold m = max x (unscaled) and sum exp(s (x - m)); a merge
 * must use the same inv_temperature as the partials.  Any other value of
 * dtype or inv_temperature is FLP_EINVAL.
 */
flp_status fused_logp_forward_ex(const void* logits, int dtype, int64_t n, int64_t v, int64_t ld,
                                 const int64_t* targets, int64_t ignore_index,
                                 const uint8_t* active_mask, float inv_temperature, float* logp,
                                 float* lse, float* lse_lo, flp_stream_t stream);
flp_status fused_logp_backward_ex(const void* logits, int dtype, int64_t n, int64_t v, int64_t ld,
                                  const int64_t* targets, int64_t ignore_index,
                                  const uint8_t* active_mask, float inv_temperature,
                                  const float* lse, const float* lse_lo, const float* grad,
                                  void* dlogits, int64_t ld_out, flp_stream_t stream);
flp_status logp_shard_partials_ex(const void* shard_logits, int dtype, int64_t n, int64_t ld_shard,
                                  int64_t vocab_start, int64_t real_width, int64_t v_total,
                                  float inv_temperature, const int64_t* targets, float* part_max,
                                  float* part_sum, float* sel, flp_stream_t stream);
flp_status logp_merge_partials_ex(const float* part_max, const float* part_sum, const float* sel,
                                  const int64_t* targets, int64_t ignore_index,
                                  const uint8_t* active_mask, int64_t n, int64_t v_total,
                                  float inv_temperature, float* logp, float* lse, float* lse_lo,
                                  flp_stream_t stream);

/*
 * Backward of one vocabulary shard (PR #314 "Deterministic config option":
 * the vocab-parallel logprob op is an autograd function over the local shard,
 * whose backward each rank runs on its own columns with the merged LSE; the
 * method's backward, PR #495 Summary item 2).  The shard holds global columns
 * [vocab_start, vocab_start + real_width) of a v_total-column vocabulary in
 * shard_logits[n, ld_shard].  For c in [0, real_width):
 *   dshard[t, c] = s g_t (onehot(y_t)[vocab_start + c] - exp(s x[t, c] - LSE_t))
 * with lse (+ lse_lo) the merged, global values.  A row is active by its
 * global target (0 <= y_t < v_total, not ignore_index, mask byte nonzero);
 * the one-hot term appears only in the shard that holds y_t.  Inactive rows
 * get +0.  Elementwise, with the unsharded backward's arithmetic: the shards'
 * outputs side by side are bitwise the unsharded dlogits, for any split (the
 * bounds need not lie on the tile grid).  dshard may alias shard_logits
 * exactly (in place); other overlap is FLP_EINVAL.  Other arguments and
 * errors as for fused_logp_backward_ex; FLP_EINVAL if the shard is not inside
 * [0, v_total).
 */
flp_status logp_shard_backward(const void* shard_logits, int64_t n, int64_t ld_shard, int64_t vocab_start,
                               int64_t real_width, int64_t v_total, const int64_t* targets,
                               int64_t ignore_index, const float* lse, const float* lse_lo,
                               const float* grad, void* dshard, int64_t ld_out, flp_stream_t stream);
flp_status logp_shard_backward_ex(const void* shard_logits, int dtype, int64_t n, int64_t ld_shard,
                                  int64_t vocab_start, int64_t real_width, int64_t v_total,
                                  const int64_t* targets, int64_t ignore_index, const uint8_t* active_mask,
                                  float inv_temperature, const float* lse, const float* lse_lo,
                                  const float* grad, void* dshard, int64_t ld_out, flp_stream_t stream);

/*
 * Merge of partials gathered from the ranks of a vocabulary-parallel group
 * (issue #241 PR 3 bullets: per-shard (max, sumexp) partials, the collective
 * only transports them, one merge in fixed index order; PR 6: each rank emits
 * (max, sumexp, selected_logit); PR #314 Tensor Parallel section: the tile
 * partials are all-gathered and every rank runs the same merge).
 *   gathered     device FP32; rank r's block starts at gathered + r *
 *                rank_stride and holds, in this order, its tile maxima
 *                [n, 16], tile sums [n, 16] and selected logits [n] (33 n
 *                floats), as logp_shard_partials_ex writes them into
 *                part_max = block, part_sum = block + 16 n, sel = block + 32 n.
 *                An all-gather of each rank's block is the whole exchange.
 *   rank_stride  floats between consecutive ranks' blocks (>= 33 n when
 *                world > 1; ignored when world == 1)
 *   world        ranks, 1 ..16
 *   vocab_starts, real_widths  HOST arrays [world]: rank r's shard is
 *                [vocab_starts[r], vocab_starts[r] + real_widths[r]); each on
 *                the tile grid (as logp_shard_partials requires), together
 *                covering every tile of [0, v_total) exactly once, else
 *                FLP_EUNSUPPORTED (off the grid) or FLP_EINVAL (gap, overlap).
 * Tile k's partial is read from the rank holding it; row t's selected logit
 * from the rank holding column y_t.  Other bytes of the blocks are never
 * read.  Then as logp_merge_partials_ex: the result is bitwise equal to
 * fused_logp_forward_ex on the unsharded logits, for any world and split.
 */
flp_status logp_merge_gathered_partials_ex(const float* gathered, int64_t rank_stride, int64_t world,
                                           const int64_t* vocab_starts, const int64_t* real_widths,
                                           const int64_t* targets, int64_t ignore_index,
                                           const uint8_t* active_mask, int64_t n, int64_t v_total,
                                           float inv_temperature, float* logp, float* lse, float* lse_lo,
                                           flp_stream_t stream);

/*
 * Fused LM head + logp (linear_logp, named in RL-Kernel PR #495 Summary; the
 * pages give no formula or design).  The logits z = H W^T of BF16 hidden
 * states and BF16 LM-head weight rows are formed on the tensor cores and
 * reduced where they are formed; they never reach memory.  Then, as for
 * fused_logp_forward_ex on logits s z:
 *   lse[t]  = log sum_j exp(s z[t, j]),  logp[t] = s z[t, y_t] - lse[t]
 * (0 for inactive rows), lse_lo[t] the FP32 rounding residual of the LSE.
 *   hidden    [n, ld_h] BF16 device, row-major; the first d columns are used
 *   weight    [v, ld_w] BF16 device, row-major (one row per vocabulary entry)
 *   targets   [n] int64; ignore_index and active_mask as for the forward
 *   inv_temperature  s = 1/T (> 0, finite)
 *   workspace device scratch of at least fused_linear_logp_workspace_size
 *             bytes (16-byte aligned), owned by the caller; contents on
 *             return are unspecified.  Layout: FP32 tile maxima [n,
 *             ceil(v/256)], tile sums [n, ceil(v/256)], selected logits [n].
 *   logp, lse [n] FP32 out; lse_lo [n] FP32 out or NULL
 * Accumulation: FP32 on the tensor cores (BF16 products exact), 128 x 256
 * tiles, K in increasing order; each row's result is independent of n, of
 * its position in the batch and of the grid (deterministic, batch-invariant).
 * Requirements: hidden and weight 16-byte aligned, ld_h and ld_w multiples
 * of 8 (16-byte row strides for the tensor-map copies), n, v, d < 2^31;
 * otherwise FLP_EUNSUPPORTED.  FLP_EINVAL for negative sizes, ld < d, a null
 * or small workspace, pointers on different devices.  n == 0 is a no-op.
 * Asynchronous on `stream`; the library allocates nothing.
 */
flp_status fused_linear_logp_workspace_size(int64_t n, int64_t v, int64_t* bytes);
flp_status fused_linear_logp_forward(const void* hidden, int64_t n, int64_t d, int64_t ld_h,
                                     const void* weight, int64_t v, int64_t ld_w, const int64_t* targets,
                                     int64_t ignore_index, const uint8_t* active_mask, float inv_temperature,
                                     void* workspace, int64_t workspace_bytes, float* logp, float* lse,
                                     float* lse_lo, flp_stream_t stream);

/*
 * Vocabulary-sharded fused LM head on one GPU (issue #241 PR 3 and PR 6: a
 * shard emits (max, sumexp) partials of the tiles it holds plus the selected
 * logit it owns; one fixed-order merge; PR #314 Tensor Parallel section: the
 * tile grid makes every shard count give the same bits).  The weight rows of
 * a vocabulary-parallel LM head are split into shards; shard l holds global
 * columns [vocab_start, vocab_start + real_width) as its own [real_width,
 * ld_w] BF16 buffer.
 *   fused_linear_logp_shard_partials writes that shard's tile partials into
 *     `workspace` (the layout of fused_linear_logp_forward's workspace for n
 *     rows and v_total columns: FP32 [n, ceil(v_total/256)] maxima and sums,
 *     [n] selected logits) and the selected logit of every row whose target
 *     is in the shard.  vocab_start must be a multiple of 256 (the tile
 *     grid), else FLP_EUNSUPPORTED; [vocab_start, vocab_start + real_width)
 *     must lie in [0, v_total).
 *   fused_linear_logp_merge merges, in tile order, the partials of all tiles
 *     of [0, v_total) into logp, lse (and lse_lo), as the forward does.
 * The shards must together cover [0, v_total) (the merge reads every tile's
 * partial).  With that, the result is bitwise equal to
 * fused_linear_logp_forward on the unsharded weight, for any shard count.
 * All calls asynchronous on `stream`; the library allocates nothing.
 */
flp_status fused_linear_logp_shard_partials(const void* hidden, int64_t n, int64_t d, int64_t ld_h,
                                            const void* weight_shard, int64_t real_width, int64_t ld_w,
                                            int64_t vocab_start, int64_t v_total, const int64_t* targets,
                                            float inv_temperature, void* workspace, int64_t workspace_bytes,
                                            flp_stream_t stream);
flp_status fused_linear_logp_merge(const void* workspace, int64_t workspace_bytes, int64_t n, int64_t v_total,
                                   const int64_t* targets, int64_t ignore_index, const uint8_t* active_mask,
                                   float inv_temperature, float* logp, float* lse, float* lse_lo,
                                   flp_stream_t stream);

/*
 * Backward of the fused LM head (no counterpart in the pages beyond the name
 * linear_logp; the method's backward, PR #495 Summary item 2, taken through
 * the contraction): for the loss sum_t grad[t] logp[t],
 *   dZ[t, j] = s grad[t] (onehot(y_t)[j] - exp(s z[t, j] - LSE_t)),
 *   dhidden = dZ W   [n, d],   dweight = dZ^T H   [v, d],
 * with dZ recomputed on the tensor cores from hidden and weight and the
 * forward's lse (+ lse_lo) and written in BF16 (as the method writes dlogits)
 * one chunk of 4096 rows at a time into the workspace, never as an [n, v]
 * tensor.  The two products run on this library's own tensor-core kernels,
 * reading dZ, W and H where they lie (FP32 accumulation): dhidden in
 * S = ceil(ceil(v / 64) / 512) fixed splits of the vocabulary added in split
 * order, dweight added chunk after chunk in row order.  No atomics:
 * deterministic.
 *   hidden, weight, targets, ignore_index, active_mask, inv_temperature: as
 *             for fused_linear_logp_forward (the same call's arguments)
 *   lse       [n] FP32, lse_lo [n] FP32 or NULL: the forward's outputs
 *   grad      [n] FP32 d loss / d logp (0 for inactive rows by definition)
 *   workspace device scratch of fused_linear_logp_backward_workspace_size
 *             bytes (256-byte aligned), caller-owned: dZ [4096, ceil(v/8)*8]
 *             BF16 and, when S > 1, the splits' partial dhidden
 *             [S, 4096, d] FP32
 *   dhidden   [n, ld_dh] FP32 out
 *   dweight   [v, ld_dw] FP32: overwritten with dZ^T H when
 *             accumulate_dweight == 0 (all zero when n == 0), or with
 *             dweight + dZ^T H when it is nonzero (gradient accumulation over
 *             micro-batches; unchanged when n == 0).  With n == 0 only dweight
 *             is touched and the workspace may be NULL.
 * Each element of dhidden is a tensor-core dot product over the vocabulary
 * with split points fixed by v, whatever else the chunk holds, so a row's
 * dhidden does not depend on n or on its position.
 * Requirements and errors as for the forward, plus ld_dh, ld_dw >= d.
 * Asynchronous on `stream`; the library allocates nothing.
 */
flp_status fused_linear_logp_backward_workspace_size(int64_t d, int64_t v, int64_t* bytes);
flp_status fused_linear_logp_backward(const void* hidden, int64_t n, int64_t d, int64_t ld_h, const void* weight,
                                      int64_t v, int64_t ld_w, const int64_t* targets, int64_t ignore_index,
                                      const uint8_t* active_mask, float inv_temperature, const float* lse,
                                      const float* lse_lo, const float* grad, void* workspace,
                                      int64_t workspace_bytes, float* dhidden, int64_t ld_dh, float* dweight,
                                      int64_t ld_dw, int accumulate_dweight, flp_stream_t stream);

/*
 * Backward of one vocabulary shard of the fused LM head (the shard layout of
 * fused_linear_logp_shard_partials; lse and lse_lo are the merged, global
 * values): dZ for the shard's columns, its rows of dweight, and its term of
 * dhidden = sum over shards of dZ_shard W_shard.
 *   dhidden           [n, ld_dh] FP32: overwritten with this shard's term,
 *                     or added to when accumulate_dhidden is nonzero (call
 *                     the shards in a fixed order, the first without it)
 *   dweight_shard     [real_width, ld_dw] FP32 (overwritten, or added to with
 *                     accumulate_dweight)
 *   workspace         fused_linear_logp_backward_workspace_size(d, real_width)
 * vocab_start must be a multiple of 256, else FLP_EUNSUPPORTED.  The
 * summed dhidden is deterministic for a fixed shard layout; it is not bitwise
 * equal to the unsharded backward's (the sum over the vocabulary is split).
 * Other arguments and errors as for fused_linear_logp_backward.
 */
flp_status fused_linear_logp_shard_backward(const void* hidden, int64_t n, int64_t d, int64_t ld_h,
                                            const void* weight_shard, int64_t real_width, int64_t ld_w,
                                            int64_t vocab_start, int64_t v_total, const int64_t* targets,
                                            int64_t ignore_index, const uint8_t* active_mask, float inv_temperature,
                                            const float* lse, const float* lse_lo, const float* grad,
                                            void* workspace, int64_t workspace_bytes, float* dhidden,
                                            int64_t ld_dh, int accumulate_dhidden, float* dweight_shard,
                                            int64_t ld_dw, int accumulate_dweight, flp_stream_t stream);

/*
 * Fused LM head + logp with no allocation and no workspace argument.  The
 * pages have no counterpart: this is a convenience of this library.
 *
 * Some callers cannot allocate device memory at all: a plugin that a host
 * application hands only its input and output buffers, code running under an
 * application-wide memory pool that owns all device memory and forbids direct
 * cudaMalloc calls, or a tight loop where a cudaMalloc/cudaFree pair would
 * synchronise the device.  For them this entry point computes exactly what
 * fused_linear_logp_forward computes (same arguments minus the workspace;
 * identical bits) and takes its scratch from a fixed 16 MiB array in the
 * library's static device memory.  It calls no allocator.
 *   Limit: the scratch needed, fused_linear_logp_workspace_size(n, v), must
 *   be at most 16 MiB (16777216 bytes): up to 3527 rows per call at
 *   v = 151936.  Larger calls return FLP_EUNSUPPORTED with a message naming
 *   the sizes; split the rows, or use fused_linear_logp_forward.
 *   Memory: every GPU that loads the library holds the 16 MiB until the
 *   process exits.
 *   First call per device: looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current) and caches it; make
 *   that first call before any stream capture.  The cached address belongs
 *   to the device's context: after cudaDeviceReset it is stale, so do not
 *   call this entry point again in a process that has reset the device.
 *   Sharing: all calls in the process use the same array.  Calls whose work
 *   can overlap on a GPU (different streams, or different host threads
 *   without ordering) race on it and give wrong results; order them, e.g. on
 *   one stream.  The array keeps the previous call's contents, and nothing in
 *   it needs to start at zero: every element a call reads was written
 *   earlier in that same call.
 * Errors: as fused_linear_logp_forward, plus FLP_EUNSUPPORTED above the limit.
 */
flp_status fused_linear_logp_forward_noalloc(const void* hidden, int64_t n, int64_t d, int64_t ld_h,
                                             const void* weight, int64_t v, int64_t ld_w,
                                             const int64_t* targets, int64_t ignore_index,
                                             const uint8_t* active_mask, float inv_temperature, float* logp,
                                             float* lse, float* lse_lo, flp_stream_t stream);

/*
 * The fused LM head across several processes, one vocabulary slice of the
 * weight per rank (the tensor-parallel output layer; the exchange is the
 * tile-partial all-gather of issue #241 PR 3 / PR #314 Tensor Parallel,
 * transport only, then the same fixed-order merge on every rank).
 *
 * fused_linear_logp_merge_gathered: every rank ran
 * fused_linear_logp_shard_partials on its slice into its own workspace (the
 * slices on the 256-column tile grid, covering every tile once); `gathered`
 * holds the world workspaces one after another, rank r's at gathered +
 * r * rank_stride (floats; rank_stride >= (2 ceil(v_total / 256) + 1) n, e.g.
 * the workspace's size / 4).  vocab_starts / real_widths are host arrays of
 * world entries (at most 16).  Tile k is read from the rank that holds it
 * and row t's selected logit from the rank that holds its target's tile:
 * logp, lse (and lse_lo) are those of fused_linear_logp_merge over one
 * workspace that all slices wrote, bit for bit.
 * Errors: FLP_EINVAL for bad extents, a stride below one block, a slice
 * outside the vocabulary, a tile held by no rank or by two;
 * FLP_EUNSUPPORTED for a slice off the tile grid.
 *
 * flp_sum_blocks: out[r, c] = ((b_0 + b_1) + b_2) + ... over world FP32
 * blocks [rows, cols] (row pitch cols) at blocks + k * block_stride, one
 * rounding per addition in block order -- the sum that the one-GPU sharded
 * LM-head backward forms when each later shard adds its term of dhidden, so
 * the ranks' all-gathered terms summed here give its dhidden bit for bit.
 * out has row pitch ld_out and must not overlap the blocks.
 */
flp_status fused_linear_logp_merge_gathered(const float* gathered, int64_t rank_stride, int world,
                                            const int64_t* vocab_starts, const int64_t* real_widths, int64_t n,
                                            int64_t v_total, const int64_t* targets, int64_t ignore_index,
                                            const uint8_t* active_mask, float inv_temperature, float* logp,
                                            float* lse, float* lse_lo, flp_stream_t stream);
flp_status flp_sum_blocks(const float* blocks, int64_t block_stride, int world, int64_t rows, int64_t cols,
                          float* out, int64_t ld_out, flp_stream_t stream);

/*
 * GRPO loss on the logp path (issue #241 PR 5: ratio, clip, KL, advantage,
 * a declared normaliser and a fixed summation order; the pages name these
 * terms, the formulas below are the standard clipped-surrogate form).
 * Per active token t (active_mask byte nonzero, or all when NULL):
 *   r = exp(logp - old_logp),
 *   pg = max(-A r, -A clip(r, 1 - eps_lo, 1 + eps_hi)),
 *   kl = exp(ref - logp) - (ref - logp) - 1 (only if ref_logp != NULL),
 *   l = pg + beta kl.
 * mode FLP_GRPO_TOKEN_MEAN:          loss = sum_t l / D (D = active tokens)
 *      FLP_GRPO_SEQ_MEAN_TOKEN_MEAN: loss = mean over non-empty sequences of
 *                                    the sequence's mean l
 *      FLP_GRPO_SEQ_MEAN_TOKEN_SUM:  loss = mean over non-empty sequences of
 *                                    the sequence's summed l
 * Sequences are [cu_seqlens[s], cu_seqlens[s+1]) for s < num_seqs (int64 on
 * the device; bounds are clamped to [0, n]); with cu_seqlens == NULL the whole
 * batch is one sequence.  normalizer > 0 replaces D (token mean) or the
 * sequence count, e.g. by a count global to all micro-batches.
 *   loss       [1] FP32 out
 *   grad       [n] FP32 out: d loss / d logp (the unclipped term's -A r when
 *              it is the max, ties included, else 0; plus beta (1 - e^(ref -
 *              logp)); times the token's normaliser weight; 0 when inactive)
 *              -- the upstream gradient for fused_logp_backward.
 *   token_loss [n] FP32 out or NULL: l per token (0 when inactive).
 *   workspace  device scratch of logp_grpo_loss_workspace_size(n, num_seqs)
 *              bytes (16-byte aligned), caller-owned, no initial contents
 *              needed: 32 bytes for a count and the fold's ticket, 9.5 KB
 *              for the token pass's per-CTA sums, 16 KB of counts, and with
 *              sequences 8 bytes per sequence and 4 per 16 tokens; rounded
 *              up to 256 bytes.  One workspace serves one call at a time.
 * Tokens outside every sequence (before cu_seqlens[0] or from
 * cu_seqlens[num_seqs] on) are inactive: l = 0, grad 0.  cu_seqlens must be
 * non-decreasing; for one that is not, the result is unspecified, but every
 * access stays inside the arrays.
 * Kernels: when a weight depends on the mask (any normaliser but the
 * caller's uniform one), a count of the mask's active tokens per 16-token
 * word and per range, then per sequence its active count, the number of
 * non-empty sequences and the active tokens; then one token pass that
 * writes each final gradient once and folds the loss.  Integer counts are
 * exact.  Deterministic: the batch is cut into fixed 256-token chunks (one
 * warp each) whatever the sequence lengths; sums are plain FP32 within a
 * chunk and compensated two-float sums in FP32 from there on, folded per
 * warp over its contiguous chunks, per CTA in warp order and over the CTAs
 * in order, a shape fixed by n; the result does not depend on timing.  A
 * gradient is dl/dlogp times its weight, rounded once: 1 / den, or for the
 * sequence mean of token means the product of the correctly rounded 1 / den
 * and 1 / n_s.  With logp == old_logp the ratio is exactly 1 and grad = -A
 * times the weight (the KL = 0 identity of PR 5).
 * Errors: FLP_EINVAL for a bad mode, eps_lo outside [0, 1), a negative or
 * non-finite eps_hi, beta or normalizer, a sequence mode without sequences,
 * or num_seqs >= 2^31 - 1.
 */
#define FLP_GRPO_TOKEN_MEAN 0
#define FLP_GRPO_SEQ_MEAN_TOKEN_MEAN 1
#define FLP_GRPO_SEQ_MEAN_TOKEN_SUM 2
flp_status logp_grpo_loss_workspace_size(int64_t n, int64_t num_seqs, int64_t* bytes);
flp_status logp_grpo_loss(const float* logp, const float* old_logp, const float* ref_logp,
                          const float* advantages, const uint8_t* active_mask,
                          const int64_t* cu_seqlens, int64_t num_seqs, int64_t n, int mode,
                          float eps_lo, float eps_hi, float beta, float normalizer, void* workspace,
                          int64_t workspace_bytes, float* loss, float* grad, float* token_loss,
                          flp_stream_t stream);

/*
 * The GRPO loss in two parts, for a batch whose layout (active_mask,
 * cu_seqlens, n, num_seqs, mode, normalizer) is known before its logp: the
 * normaliser weights depend on the layout only (issue #241 PR 5's declared
 * normaliser), so they can be counted once, e.g. on a second stream while
 * the logp forward runs, or once for several optimisation epochs over the
 * same batch.
 *
 * logp_grpo_loss_counts runs the counting kernels of logp_grpo_loss (the
 * mask's counts, each sequence's active count, the number of non-empty
 * sequences) into `workspace` and records a tag of the layout: the mask and
 * cu_seqlens pointers, n, num_seqs, mode and normalizer.  Arguments as for
 * logp_grpo_loss; nothing else is read or written.
 *
 * logp_grpo_loss_counted is logp_grpo_loss with the counting left out: it
 * runs the token pass on counts that an earlier logp_grpo_loss_counts (or
 * logp_grpo_loss) call left in the same workspace, which must have completed
 * on the device first (same stream, or an event).  Results are bitwise those
 * of logp_grpo_loss.  The layout arguments must be the ones the counts were
 * taken for and the mask and cu_seqlens contents unchanged since: the token
 * pass compares the recorded tag with the call's, and on a mismatch writes
 * NaN for the loss and for the gradient of every token inside a sequence (the
 * contents themselves are not compared).  Calls may repeat on the same
 * counts.  When the weight is the caller's (a normalizer with the token mean
 * or the sequence mean of token sums) nothing is counted and the call is
 * logp_grpo_loss, which replaces the counts and the tag in the workspace
 * (a later counted call for the earlier layout then gets NaN: count again).
 * Errors: as logp_grpo_loss.
 */
flp_status logp_grpo_loss_counts(const uint8_t* active_mask, const int64_t* cu_seqlens, int64_t num_seqs,
                                 int64_t n, int mode, float normalizer, void* workspace, int64_t workspace_bytes,
                                 flp_stream_t stream);
flp_status logp_grpo_loss_counted(const float* logp, const float* old_logp, const float* ref_logp,
                                  const float* advantages, const uint8_t* active_mask,
                                  const int64_t* cu_seqlens, int64_t num_seqs, int64_t n, int mode,
                                  float eps_lo, float eps_hi, float beta, float normalizer, void* workspace,
                                  int64_t workspace_bytes, float* loss, float* grad, float* token_loss,
                                  flp_stream_t stream);

/*
 * Selected-token log-probability with the row's entropy and its k best
 * alternatives, and the gradient of all three (no counterpart in the pages).
 * With z = inv_temperature * logits, p = softmax(z), for each active row:
 *   logp      z[y] - LSE (given targets only)
 *   entropy   H = -sum p log p
 *   top_ids, top_logp  the k largest logits in falling order, of equal ones the
 *             lowest column first, and their z - LSE
 * Forward:
 *   logits    `dtype` [n, ld], any alignment; targets int64 [n], or NULL (then
 *             logp is NULL too and every row that the mask allows is active)
 *   active_mask  byte per row, or NULL.  Rows that are masked out or whose
 *             target is ignore_index or outside [0, v) are not read: their
 *             logp, lse, entropy and top_logp are 0, their top_ids -1
 *   k         0 .. min(64, v); with 0 top_ids and top_logp may be NULL
 *   lse, lse_lo  as of fused_logp_forward_ex (lse_lo nullable), for the backward
 *   workspace fused_logp_topk_workspace_size(n, v, dtype, k) bytes, 16-byte
 *             aligned, caller-owned, no initial contents needed; one workspace
 *             serves one call at a time
 * logp and lse agree with fused_logp_forward_ex's within a few FP32 roundings (a
 * term's exponent is formed in another way).  A -inf logit has probability 0 and adds nothing to the entropy; among the
 * alternatives it comes last (top_logp -inf).  A NaN logit makes logp, lse and the
 * entropy NaN and counts as the largest value among the alternatives; a +inf logit,
 * or a row of -inf alone, leaves no distribution: logp, the entropy and top_logp are
 * NaN and the alternatives are by value.
 * Backward, with lp = z - LSE and G = g + sum_j gt_j:
 *   dlogits = inv_temperature (g 1_y + sum_j gt_j 1_idj - p (G + gh (lp + H)))
 *   grad_logp (g), grad_entropy (gh) FP32 [n], grad_top (gt) FP32 [n, k]; each may
 *             be NULL (zeros)
 *   lse, lse_lo, entropy, top_ids  the forward's (entropy is not read without
 *             grad_entropy, top_ids not without grad_top); columns in top_ids
 *             that are outside [0, v) count nowhere, the same column twice counts
 *             with the sum of both gradients.  Where |lse| is 2^18 or more, lse and
 *             lse_lo do not hold log S well enough: the row's maximum and sum are
 *             taken from its logits again
 *   dlogits   `dtype` [n, ld_out], may be logits itself (ld_out == ld); inactive
 *             rows are zeros
 * Deterministic, and a row's results depend on that row only.
 * Errors: FLP_EINVAL for a bad dtype, extent, stride, k, temperature, workspace or
 * overlap, or targets without logp; FLP_EUNSUPPORTED for v >= 2^31.
 */
flp_status fused_logp_topk_workspace_size(int64_t n, int64_t v, int dtype, int64_t k, int64_t* bytes);
flp_status fused_logp_topk_forward(const void* logits, int dtype, int64_t n, int64_t v, int64_t ld,
                                   const int64_t* targets, int64_t ignore_index, const uint8_t* active_mask,
                                   float inv_temperature, int64_t k, void* workspace, int64_t workspace_bytes,
                                   float* logp, float* lse, float* lse_lo, float* entropy, int64_t* top_ids,
                                   float* top_logp, flp_stream_t stream);
flp_status fused_logp_topk_backward(const void* logits, int dtype, int64_t n, int64_t v, int64_t ld,
                                    const int64_t* targets, int64_t ignore_index, const uint8_t* active_mask,
                                    float inv_temperature, const float* lse, const float* lse_lo,
                                    const float* entropy, const int64_t* top_ids, int64_t k, const float* grad_logp,
                                    const float* grad_entropy, const float* grad_top, void* dlogits, int64_t ld_out,
                                    flp_stream_t stream);

/*
 * The norm in front of the LM head: layer norm, or RMS norm when center == 0.
 * For each row x of width d (sums in FP32, one rounding to x's dtype):
 *   mu = mean(x) (0 when center == 0), var = mean((x - mu)^2),
 *   rstd = (var + eps)^(-1/2), xh = (x - mu) rstd, y = xh weight + bias.
 * Forward:
 *   x      [n, ld_x] of `dtype`, y [n, ld_y] of the same dtype (y may be x
 *          itself with ld_y == ld_x; any other overlap is FLP_EINVAL)
 *   weight, bias  [d] of weight_dtype (x's dtype or FP32), or NULL (1 and 0)
 *   mean, rstd    [n] FP32 out for the backward, or NULL (mean is not written
 *          when center == 0)
 * Backward, with g = dy weight:
 *   dx = rstd (g - mean(g) - xh mean(g xh))  (no mean(g) when center == 0)
 *   dweight = sum over rows of dy xh, dbias = sum over rows of dy
 *   dy     [n, ld_dy] of dy_dtype: x's dtype or FP32 (the dhidden of
 *          fused_linear_logp_backward is FP32)
 *   mean (NULL allowed when center == 0), rstd  from the forward
 *   dx     [n, ld_dx] of x's dtype, not overlapping x or dy
 *   dweight, dbias  [d] FP32 out, or NULL when not wanted; with `accumulate`
 *          they are added to (gradient accumulation over micro-batches)
 *   workspace  fused_layer_norm_backward_rows_workspace_size(n, d) bytes, or
 *          fused_layer_norm_backward_workspace_size(d) whatever n is; 16-byte
 *          aligned, caller-owned, no initial contents needed (the partial
 *          sums of dweight and dbias); may be NULL without both
 * A row's y, mean, rstd and dx depend on that row (and the vectors) only;
 * dweight and dbias are summed in an order fixed by n, d and the layout, so
 * repeated calls give identical bits.  Rows may have any alignment and any
 * stride >= d.  n == 0 writes empty sums (zeros, unless accumulating).
 * Errors: FLP_EINVAL for a bad dtype, extent, stride, eps or overlap;
 * FLP_EUNSUPPORTED for d >= 2^31.
 */
flp_status fused_layer_norm_forward(const void* x, int dtype, int64_t n, int64_t d, int64_t ld_x,
                                    const void* weight, const void* bias, int weight_dtype, float eps, int center,
                                    void* y, int64_t ld_y, float* mean, float* rstd, flp_stream_t stream);
flp_status fused_layer_norm_backward_workspace_size(int64_t d, int64_t* bytes);
flp_status fused_layer_norm_backward_rows_workspace_size(int64_t n, int64_t d, int64_t* bytes);
flp_status fused_layer_norm_backward(const void* dy, int dy_dtype, int64_t ld_dy, const void* x, int dtype, int64_t n,
                                     int64_t d, int64_t ld_x, const void* weight, int weight_dtype, const float* mean,
                                     const float* rstd, int center, void* workspace, int64_t workspace_bytes, void* dx,
                                     int64_t ld_dx, float* dweight, float* dbias, int accumulate,
                                     flp_stream_t stream);

/*
 * RMS norm behind the residual's addition, with an output in x's type or in 8
 * bits with scales (an operand of flp_fp8_matmul).  For each row of width d,
 * sums in FP32:
 *   h = x + residual, rounded to x's dtype (h = x without a residual)
 *   rstd = (mean(h^2) + eps)^(-1/2), y = h rstd weight
 * Forward:
 *   x, residual  [n, ld] of `dtype`; residual may be NULL
 *   weight  [d] of weight_dtype (x's dtype or FP32), or NULL (1)
 *   h       [n, ld_h] of `dtype` out, NULL without a residual; may be x or
 *           residual itself (same stride)
 *   y       [n, ld_y] of `dtype` out, one rounding; may be x or residual itself
 *           (same stride), not h.  Or y NULL and
 *   q, scale  e4m3 [n, ld_q] and FP32 [ceil(d / 128), ld_scale >= n]: for each
 *           128 columns of a row scale = max(amax |y| / 448, 2^-126) and q =
 *           e4m3(y (1 / scale)), the reciprocal and product rounded to FP32;
 *           entry [b, r] is the scale of row r's block b.  What lies behind
 *           column d of q and behind column n of scale is left as it is.
 *   rstd    [n] FP32 out for the backward, or NULL
 * Backward, with g = dy weight and xh = h rstd:
 *   dx = rstd (g - xh mean(g xh)) + dh   (the gradient of x and of residual)
 *   dweight = sum over rows of dy xh
 *   dy      [n, ld_dy] of dy_dtype (`dtype` or FP32): the gradient of y, or of
 *           the values that q and scale stand for
 *   dh      [n, ld_dh] of `dtype`: the gradient of h from elsewhere, or NULL
 *   dx      [n, ld_dx] of `dtype`; may be dh itself (same stride), not h or dy
 *   dweight [d] FP32 out or NULL; added to with `accumulate`
 *   workspace  fused_layer_norm_backward_rows_workspace_size(n, d) bytes,
 *           16-byte aligned, caller-owned; may be NULL without dweight
 * A row's results depend on that row and the weight only, dweight is summed in
 * an order fixed by n, d and the layout.  A NaN or infinity in a block of y
 * makes that block's scale NaN or infinite, other blocks are as without it
 * (as far as rstd is finite).  Rows may have any alignment and stride >= d.
 * Errors: FLP_EINVAL for a bad dtype, extent, stride, eps, overlap or
 * workspace, or not exactly one of y and (q, scale); FLP_EUNSUPPORTED for d >=
 * 2^31.
 */
flp_status fused_add_rms_norm_forward(const void* x, int dtype, int64_t n, int64_t d, int64_t ld_x,
                                      const void* residual, int64_t ld_residual, const void* weight, int weight_dtype,
                                      float eps, void* h, int64_t ld_h, void* y, int64_t ld_y, void* q, int64_t ld_q,
                                      float* scale, int64_t ld_scale, float* rstd, flp_stream_t stream);
flp_status fused_add_rms_norm_backward(const void* dy, int dy_dtype, int64_t ld_dy, const void* dh, int64_t ld_dh,
                                       const void* h, int dtype, int64_t n, int64_t d, int64_t ld_h,
                                       const void* weight, int weight_dtype, const float* rstd, void* workspace,
                                       int64_t workspace_bytes, void* dx, int64_t ld_dx, float* dweight,
                                       int accumulate, flp_stream_t stream);

/*
 * A matrix x [rows, cols] (`dtype`, row stride ld_x, any alignment) as e4m3 values
 * with FP32 scales, the operands of flp_fp8_matmul: for each block
 *   scale = max(amax |x| / 448, 2^-126), q = e4m3(x (1 / scale))
 * (nearest even; the reciprocal and the product rounded to FP32).  Blocks are
 * 128 columns of a row, or with `square` 128 x 128; cut at the ends.
 *   q, scale      bytes [rows, ld_q]; entry [c, r] of scale [ceil(cols / 128),
 *                 ld_scale] is that of row r's (or 128-row block r's) column
 *                 block c; both may be NULL
 *   qt, scale_t   the same of x's transpose: bytes [cols, ld_qt], blocks of 128
 *                 rows of x, scale_t [ceil(rows / 128), ld_scale_t]; both may
 *                 be NULL
 * What lies behind the columns of q and qt and of the scales is left as it is.
 * A block of zeros has zeros under 2^-126; a NaN or infinity makes its block's
 * scale NaN or infinite, other blocks are as without it.
 * Errors: FLP_EINVAL for a bad dtype, extent, stride or overlap or a missing
 * output; FLP_EUNSUPPORTED for a side of 2^31 - 1024 or more.
 */
flp_status flp_quantize_fp8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, int square, void* q,
                            int64_t ld_q, float* scale, int64_t ld_scale, void* qt, int64_t ld_qt, float* scale_t,
                            int64_t ld_scale_t, flp_stream_t stream);

/*
 * Product of e4m3 matrices with a scale for each block of 128:
 *   c[i, j] = sum over b of a_scale[b, i] b_scale[b, j]
 *             sum over k in [128 b, 128 b + 128) of a[i, k] b[j, k]
 *   a  bytes [m, ld_a >= k], a_scale FP32 [ceil(k / 128), ld_a_scale >= m]
 *   b  bytes [n, ld_b >= k], b_scale FP32 [ceil(k / 128), ld_b_scale], one a row
 *      of b, or with b_square one for each 128 rows (b_scale[b, j / 128])
 *   c  [m, ld_c >= n] of out_dtype (BF16, FP16 or FP32), one rounding
 * Rows of a and b start on 16-byte boundaries (base, ld_a and ld_b multiples of
 * 16); bytes between k and ld are not used.  The products and the sums within a
 * block run on the tensor cores, a block's sum is scaled and added in FP32.
 * Products of two scales should be normal FP32 numbers: below 2^-126 their
 * digits, above 2^128 all is lost.  Equal calls give equal bits; the order of
 * the blocks' sums depends on m, n and k.  k >= 1.
 * Errors: FLP_EINVAL for a bad dtype, extent, stride, alignment or overlap;
 * FLP_EUNSUPPORTED for a side of 2^31 - 1024 or more.
 */
flp_status flp_fp8_matmul(const void* a, int64_t m, int64_t k, int64_t ld_a, const float* a_scale, int64_t ld_a_scale,
                          const void* b, int64_t n, int64_t ld_b, const float* b_scale, int64_t ld_b_scale,
                          int b_square, void* c, int out_dtype, int64_t ld_c, flp_stream_t stream);

/*
 * Preference loss of pairs of packed sequences on the logp path.  Sequence s
 * is tokens [cu_seqlens[s], cu_seqlens[s + 1]) (int64 on the device, num_seqs
 * + 1 of them, num_seqs = 2 P even); pair p is (chosen, rejected) =
 * (2 p, 2 p + 1) with FLP_PREF_INTERLEAVED, (p, p + P) with FLP_PREF_HALVES.
 * Over the active tokens (active_mask byte nonzero, or all when NULL) of s,
 *   r_s = sum of logp - ref_logp (ref_logp NULL: of logp), divided by their
 *         number n_s with `average`;
 *   h = r_chosen - r_rejected, u = beta h - margin, and the pair's loss
 * kind FLP_PREF_SIGMOID: -(1 - e) log sigma(u) - e log sigma(-u), e =
 *                        label_smoothing
 *      FLP_PREF_HINGE:   max(0, 1 - u)
 *      FLP_PREF_IPO:     (h - 1 / (2 beta))^2 (no margin)
 * A pair is live when both its sequences have an active token; other pairs
 * (padding) count nowhere.  D = the number of live pairs, or normalizer when
 * that is > 0 (e.g. a count global to all micro-batches).
 *   loss     [1] FP32 out: the live pairs' sum / D (0 without live pairs)
 *   grad     [n] FP32 out: d loss / d logp, the upstream gradient for the
 *            logp backward (+-(dl/dh) / D, / n_s with `average`); 0 for
 *            tokens that are inactive, outside every sequence or in a pair
 *            that is not live
 *   rewards  [P, 2] FP32 out: beta r_chosen, beta r_rejected (0 for a
 *            sequence without active tokens)
 *   workspace  logp_preference_loss_workspace_size(n, num_seqs) bytes,
 *            16-byte aligned, caller-owned, no initial contents needed; one
 *            workspace serves one call at a time.
 * logp and ref_logp are never used where the mask is 0 (they may hold NaN or
 * infinities there).  Sums are FP32 within 512-token chunks and two-float
 * sums over them, in an order fixed by the layout: repeated calls give
 * identical bits.
 * Bounds in cu_seqlens are clamped to [0, n]; when they decrease, the result
 * is unspecified, but every access stays inside the arrays.
 * Errors: FLP_EINVAL for an odd or too large num_seqs, a bad kind or layout,
 * beta not finite and positive, label_smoothing outside [0, 1] or nonzero
 * without the sigmoid, a margin not finite or nonzero with ipo, or a bad
 * normalizer or workspace.
 */
#define FLP_PREF_SIGMOID 0
#define FLP_PREF_HINGE 1
#define FLP_PREF_IPO 2
#define FLP_PREF_INTERLEAVED 0
#define FLP_PREF_HALVES 1
flp_status logp_preference_loss_workspace_size(int64_t n, int64_t num_seqs, int64_t* bytes);
flp_status logp_preference_loss(const float* logp, const float* ref_logp, const uint8_t* active_mask,
                                const int64_t* cu_seqlens, int64_t num_seqs, int64_t n, int kind, int layout,
                                int average, float beta, float label_smoothing, float margin, float normalizer,
                                void* workspace, int64_t workspace_bytes, float* loss, float* grad, float* rewards,
                                flp_stream_t stream);

/*
 * Orthogonalised update: Newton-Schulz products on the tensor cores.  For each
 * matrix G [rows, cols] of a batch (e.g. the momentum of a weight, or of a
 * stack of equal weights),
 *   X = G / (|G|_F + eps);  `steps` times, with the step's (a, b, c):
 *   A = X X^T,  X <- a X + (b A + c A^2) X      (A on the smaller side)
 *   out = scale X
 * which brings every singular value of G near 1 (with the usual quintic
 * coefficients (3.4445, -4.7750, 2.0315) and 5 steps into about 0.7 .. 1.2)
 * and keeps its singular vectors.
 *   x        `dtype` (BF16, FP16 or FP32) [batch] matrices stride_x elements
 *            apart, rows ld_x elements apart (stride_x is not read for one
 *            matrix)
 *   coefficients  HOST pointer to steps x 3 floats; they should keep singular
 *            values in [0, 1] below 2 (FP16 overflows where an entry of X,
 *            X X^T or b A + c A^2 passes 255)
 *   out      out_dtype BF16 or FP32, ld_out, stride_out; may be x itself (same
 *            layout and element size), any other overlap is FLP_EINVAL
 *   workspace  flp_orthogonalize_workspace_size(batch, rows, cols) bytes,
 *            128-byte aligned, caller-owned, no initial contents needed
 * The products run on FP16 operands with FP32 accumulators; X is carried as
 * two FP16 numbers (22 bits) and the diagonals of A and b A + c A^2 in FP32.
 * With the usual coefficients and 5 steps out is within 3e-4 to 2e-3 (of its
 * norm, before the rounding to out_dtype) of the result in 64 bits, 4e-3 at
 * most, for spectra from alike singular values to rank 1 over any floor (where
 * a side is below 8, a handful of roundings do not average: 1e-2, and 3e-2
 * after 8 steps).  More
 * steps multiply, by a each, what rounding puts beside singular values near
 * zero: 6 steps are within 4.5e-3, 8 within 1.5e-2, 10 within 8e-2 (in plain
 * FP32 up to 4e-2 there); where no singular value is near zero, 10 steps are
 * within 4e-3.  Coefficients that settle at 1 (such as (1.5, -0.5, 0)) multiply
 * nothing.  The squares are
 * scaled where FP32 would not hold their sum, so that every finite G counts.  A zero
 * matrix gives zeros (with eps == 0 too); an infinity or NaN makes its matrix NaN.  Deterministic:
 * equal calls give equal bits (the order of the sums over K depends on the
 * sizes and the batch).
 * Errors: FLP_EINVAL for a bad dtype, extent, stride, steps, coefficient, eps,
 * scale or workspace; FLP_EUNSUPPORTED for a smaller side above 65536 or sizes
 * beyond the 32-bit coordinates of the tensor maps.
 */
flp_status flp_orthogonalize_workspace_size(int64_t batch, int64_t rows, int64_t cols, int64_t* bytes);
flp_status flp_orthogonalize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld_x,
                             int64_t stride_x, int steps, const float* coefficients, float eps, float scale,
                             void* workspace, int64_t workspace_bytes, void* out, int out_dtype, int64_t ld_out,
                             int64_t stride_out, flp_stream_t stream);

/*
 * Health of the device side (no counterpart in the pages: a guard of this
 * library's own waits).  The bulk-copy forward waits on its own copies with a
 * bounded wait (about 2 s); if one runs out, the kernel records it in a
 * sticky device word, stops issuing copies, drains the ones in flight and
 * returns, so the context stays usable.  flp_device_error synchronises with
 * `device`, returns that word in *code (0 = no wait ran out) and clears it.
 */
flp_status flp_device_error(int device, int* code);

/*
 * Self-test of the bounded wait: launches one thread on `device` that waits on
 * a barrier nothing arrives on, with a limit of limit_cycles SM cycles
 * (at most 1e8), synchronises, and sets *timed_out = 1 if the wait gave up
 * (it must).  Also sets the sticky word read by flp_device_error.
 */
flp_status flp_selftest_wait_timeout(int device, int64_t limit_cycles, int* timed_out);

/*
 * Self-test of the exp2 bias correction (no counterpart in the pages).  The
 * forward sums terms 2^a from the special-function unit's ex2.approx, whose
 * results are low by a nearly constant ~5e-8 relative; each tile sum is
 * scaled by (1 + c) to remove it.  This measures the mean relative error of
 * ex2.approx over 2^20 arguments in [-24, 0) on `device` (synchronising) and
 * returns it with the compiled-in c, so a test can check that c still
 * matches the hardware (mean_rel_err ~ -c).
 */
flp_status flp_selftest_ex2_bias(int device, double* mean_rel_err, double* compensation);

/*
 * Self-test of the orthogonalised update's choice of kernels, on the host: *form is the
 * form of a product of `batch` matrices with a side above 128 on `sms` SMs that hold
 * `pairs` CTA pairs: 0 = a cluster a tile, 1 = persistent CTAs on 128 x 128 tiles, 2 =
 * persistent pairs on 256 x 256 tiles.  product 0: the symmetric ones (X X^T, A^2),
 * 1: those with X.
 */
flp_status flp_selftest_orthogonalize_form(int product, int64_t batch, int64_t rows, int64_t cols, int sms, int pairs,
                                           int* form);

/*
 * Self-test of the 8-bit product's choice of kernels, on the host: *bn = 0: CTA pairs on
 * 256 x 256 tiles, else 128 rows of b by *bn rows of a a tile, *split CTAs each.
 */
flp_status flp_selftest_fp8_form(int64_t m, int64_t n, int64_t k, int b_square, int sms, int* bn, int* split);

/*
 * Self-test of the bounded waits of flp_fp8_matmul: one warp waits on a signal
 * that nothing gives.  With `aborted` its CTA's abort flag is set from the start
 * and every wait has to see it at once; without, the epilogue's wait has to run
 * out (within about 2 s) and sets the device error word.  *gave_up is 1 when they
 * did.
 */
flp_status flp_selftest_fp8_wait(int device, int aborted, int* gave_up);

/*
 * Self-test of the norm's backward where the rows' CTAs are fewer than those that
 * can be resident (as on a part with more SMs than the rows' grid is sized for, 152):
 * fused_layer_norm_backward with that grid sized for `sms` (1 to 152) of them.
 */
flp_status flp_selftest_norm_backward(int sms, const void* dy, int dy_dtype, int64_t ld_dy, const void* x, int dtype,
                                      int64_t n, int64_t d, int64_t ld_x, const void* weight, int weight_dtype,
                                      const float* mean, const float* rstd, int center, void* workspace,
                                      int64_t workspace_bytes, void* dx, int64_t ld_dx, float* dweight, float* dbias,
                                      int accumulate, flp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FUSED_LOGP_H */
