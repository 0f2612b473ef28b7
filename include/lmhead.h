/*
 * lmhead.h -- C ABI of liblmhead.so: the LM output layer with FP32 logits and
 * a fused FP32 vocabulary cross-entropy, hand-written HIP for gfx950 (MI355X).
 *
 * Sources the operations follow (cited by page title and section):
 *  [MIXED] Megatron-LM pull request "Add mixed-precision (FP32) LM output
 *          logits": section "What does this PR do?" (the output-layer GEMM
 *          keeps its FP32 accumulator as FP32 logits instead of rounding each
 *          logit to BF16; the backward casts the logits gradient to BF16 for
 *          the GEMMs that follow) and section "Tests" (the logit dtype option
 *          accepts bf16 and fp32 and rejects fp16).
 *  [XENT]  Transformer Engine issue "[Pytorch] change fused cross entropy
 *          backward grad to fp32 and reduce one read/...": sections
 *          "Description" and "Changes" (the backward gradient is computed in
 *          FP32; one logits read is removed) and the discussion (the forward
 *          keeps the input, an n_rows x 1 target and an n_rows x 4 m_d_X_y
 *          record; the original kernel wrote the gradient over its input).
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers on the current HIP device.  The
 *    caller owns every buffer; the library allocates nothing and keeps no
 *    state between calls.  Calls are thread-safe.
 *  - Matrices are row-major with a leading dimension `ld*` in ELEMENTS
 *    (row r starts at base + r * ld).  BF16 tensors are raw 16-bit words
 *    (the top half of an IEEE binary32).
 *  - Every call validates its arguments on the host first and returns a
 *    non-zero LMH_ERR_* code WITHOUT touching the GPU when they are invalid.
 *    Otherwise it enqueues its kernels on `stream` (a hipStream_t passed as
 *    void*, NULL = the default stream) and returns at once; LMH_ERR_LAUNCH
 *    reports a failed launch.  Results are ready when the stream reaches
 *    that point.
 *  - Alignment: every pointer 16-byte aligned; `ld` a multiple of 8 for BF16
 *    and of 4 for FP32 (LMH_ERR_ALIGN).  ld must be >= the row length, and
 *    a matrix may span at most 2^44 elements ((rows - 1) * ld + row length;
 *    the same for a stride between blocks of records) (LMH_ERR_SHAPE).  Sizes
 *    are >= 0; a zero-size output is a no-op.
 *    The GEMMs run fastest with 128-byte aligned rows (BF16 ld a multiple
 *    of 64); rows only 16-byte aligned are accepted but measured up to a
 *    third slower.
 *  - Padding between a row's end and the next row (ld > row length) is never
 *    written.
 *  - Results are bitwise deterministic run to run; no kernel uses floating
 *    point atomics.
 *  - No entry point allocates device memory, waits on the stream or the
 *    device, or enqueues a memset: calls made under stream capture record
 *    kernel launches only.
 *  - Launch limits: one kernel launch holds at most 2^31 work-items.  The
 *    cross-entropy calls that would need more (e.g. 2^25 rows, or 64-column
 *    blocks of 8192 x 131072 logits) run as several launches over row ranges,
 *    with the same results.  A GEMM call whose R x C output (logits: V x M,
 *    dgrad: K x M, wgrad: K x V) has ceil(R / 128) * ceil(C / 32) > 2^23
 *    (with a split V sum also 16 ceil(R / 256) ceil(C / 128) > 2^22 or
 *    C ceil(R / 4) > 2^31) returns LMH_ERR_SHAPE before anything is enqueued;
 *    such outputs are larger than a GPU's memory.
 */
#ifndef LMHEAD_H
#define LMHEAD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  LMH_FP16 exists only so that it can be rejected ([MIXED],
 * "Tests": the logit dtype accepts bf16 and fp32 and rejects fp16). */
enum lmh_dtype { LMH_BF16 = 0, LMH_FP32 = 1, LMH_FP16 = 2 };

enum lmh_status {
    LMH_OK = 0,
    LMH_ERR_DTYPE = 1,  /* unsupported element type (fp16 or unknown)        */
    LMH_ERR_SHAPE = 2,  /* negative size, ld too small, bad stride or limit  */
    LMH_ERR_NULL = 3,   /* required pointer is NULL                          */
    LMH_ERR_ALIGN = 4,  /* pointer not 16-B aligned or ld not a multiple     */
    LMH_ERR_ALIAS = 5,  /* an output overlaps an input in an unsupported way */
    LMH_ERR_LAUNCH = 6, /* the HIP launch failed (see hipGetLastError)       */
    LMH_ERR_SCRATCH = 7 /* needs more than the fixed scratch array holds     */
};

/* Human-readable name of a status code (static string, never NULL). */
const char *lmhead_status_str(int32_t status);

/* Library ABI version (major * 100 + minor). */
int32_t lmhead_version(void);

/*
 * lmhead_logits -- logits[M x V] = x[M x K] . W[V x K]^T        ([MIXED])
 *
 *  x    BF16 activations, row-major [M x K], leading dimension ldx >= K.
 *  W    BF16 vocabulary weights, row-major [V x K] (K contiguous), ldw >= K.
 *  out  logits, row-major [M x V], ldo >= V, element type out_dtype:
 *         LMH_FP32 -- the FP32 MFMA accumulator stored as is (the new path);
 *         LMH_BF16 -- the same accumulator rounded to BF16, nearest-even (the
 *                     legacy path kept for comparison);
 *         LMH_FP16 or anything else -- LMH_ERR_DTYPE.
 *  Products of BF16 values are exact in FP32 and every sum is FP32; with
 *  integer operands whose partial sums stay below 2^24 the FP32 result is
 *  exact, independent of summation order.  K == 0 writes zeros.
 *  `out` must not overlap x or W (LMH_ERR_ALIAS).
 */
int32_t lmhead_logits(const void *x, int64_t ldx, const void *W, int64_t ldw,
                      void *out, int64_t ldo, int32_t out_dtype,
                      int64_t M, int64_t K, int64_t V, void *stream);

/*
 * lmhead_logits_xent -- FP32 logits plus their cross-entropy block records
 *
 *  The FP32 logits of lmhead_logits (out_dtype LMH_FP32) and, from the same
 *  FP32 accumulators, the records lmhead_xent_partial would write for those
 *  logits with block_cols = 256 and col0 = 0: for each 256-column block b of
 *  the vocabulary and each token i, part[b * part_stride + 4 i + {0..3}] =
 *  {m_b, d_b, X_b, own_b}.  lmhead_xent_merge (n_parts = ceil(V / 256),
 *  vocab = V) then gives the forward's stats without reading the logits:
 *  [XENT]'s point of removing a logits read ("Description"), carried into
 *  the GEMM's epilogue -- an extension the pages do not describe.  For
 *  shapes whose GEMM kernel lacks this epilogue (M <= 256, or operands too
 *  large for 32-bit tile offsets) the records are computed from the stored
 *  logits by a second kernel (one extra read), with the same meaning.
 *
 *  x, W, out as lmhead_logits (out FP32, ldo a multiple of 4).  target int32
 *  [M], global vocabulary indices; ignore_index as in the forward.
 *  part_stride >= 4 M and a multiple of 4; part 16-byte aligned.  out, part
 *  and target must not overlap each other or the operands.
 */
int32_t lmhead_logits_xent(const void *x, int64_t ldx, const void *W, int64_t ldw,
                           float *out, int64_t ldo, int64_t M, int64_t K, int64_t V,
                           const int32_t *target, int32_t ignore_index,
                           float *part, int64_t part_stride, void *stream);

/*
 * lmhead_xent_fwd -- fused cross-entropy forward over FP32 logits  ([XENT])
 *
 *  logits  FP32 [n_rows x n_cols], leading dimension ld >= n_cols; read once.
 *  target  int32 [n_rows]; a row whose target equals ignore_index is ignored.
 *  loss    FP32 [n_rows] per-row loss, or NULL to skip it.
 *  stats   FP32 [n_rows x 4], one 16-byte record per row:
 *            stats[i] = { m_i   = max_j z_ij,
 *                         d_i   = sum_j exp(z_ij - m_i),
 *                         X_i   = z_i,target_i,
 *                         loss_i = (m_i - X_i) + log d_i }.
 *          An ignored row stores {m_i, d_i, 0, 0} and loss 0.  A target that is
 *          neither ignore_index nor in [0, n_cols) cannot be reported from the
 *          kernel: that row stores X = NaN and loss = NaN.
 *  n_cols >= 1 when n_rows > 0.  stats and loss must not overlap the logits.
 */
int32_t lmhead_xent_fwd(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                        const int32_t *target, int32_t ignore_index,
                        float *loss, float *stats, void *stream);

/*
 * lmhead_xent_partial -- split-vocabulary CE forward, step 1        ([XENT])
 *
 *  The per-shard half of vocabulary-parallel cross entropy ([XENT],
 *  "Description", names Megatron's vocabulary-parallel CE as the FP32
 *  reference): the statistics of a slice of each logits row, per column
 *  block, to be combined by lmhead_xent_merge.  The same call serves a vocab
 *  shard of a larger model (col0 = the shard's first global column) and a
 *  single GPU that splits long rows into blocks so that few rows still fill
 *  the chip.
 *
 *  logits  FP32 [n_rows x n_cols], leading dimension ld; the slice holds the
 *          global columns [col0, col0 + n_cols).  Read once.
 *  block_cols  columns per block, a positive multiple of 4, at most
 *          INT32_MAX; the slice is cut into n_blocks = ceil(n_cols /
 *          block_cols) blocks (the last one may be shorter).  n_blocks * n_rows must not exceed INT32_MAX
 *          (LMH_ERR_SHAPE).
 *  target  int32 [n_rows], GLOBAL column indices; ignore_index as in the
 *          forward.
 *  part    FP32 output, n_blocks arrays of n_rows 16-byte records:
 *          part[b * part_stride + 4 i + {0,1,2,3}] =
 *            { m_b   = max of the row's block,
 *              d_b   = sum over the block of exp(z - m_b),
 *              X_b   = the target logit if col0 <= target_i - b block_cols
 *                      < col0 + (width of block b), else 0,
 *              own_b = 1 in that case, else 0 }   (ignored rows: X = own = 0).
 *          part_stride (elements) >= 4 n_rows and a multiple of 4.  part must
 *          not overlap the logits or the target.
 */
int32_t lmhead_xent_partial(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                            int64_t col0, int64_t block_cols, const int32_t *target,
                            int32_t ignore_index, float *part, int64_t part_stride,
                            void *stream);

/*
 * lmhead_xent_merge -- split-vocabulary CE forward, step 2          ([XENT])
 *
 *  Combines n_parts partial records per row (from one or more
 *  lmhead_xent_partial calls, at part + p * part_stride + 4 i for part p) in
 *  a fixed order (64 interleaved running pairs, then a butterfly), so the
 *  result is deterministic:  m = max m_p,  d = sum_p d_p exp(m_p - m),  X_y
 *  from the one part that owns the target,  loss = (m - X_y) + log d.
 *  Writes the same stats record and loss as lmhead_xent_fwd, so that
 *  lmhead_xent_bwd can run on the merged statistics.
 *
 *  vocab   total number of columns; a target outside [0, vocab) that is not
 *          ignore_index, or one owned by no part or by several, gives
 *          X = loss = NaN (m and d are still merged).  Ignored rows: X = loss = 0.
 *  loss    FP32 [n_rows] or NULL;  stats FP32 [n_rows x 4].
 *  n_parts >= 1, vocab >= 1, part_stride >= 4 n_rows and a multiple of 4.
 *  stats and loss must not overlap the parts or the target.
 */
int32_t lmhead_xent_merge(const float *part, int64_t n_parts, int64_t part_stride,
                          int64_t n_rows, const int32_t *target, int32_t ignore_index,
                          int64_t vocab, float *loss, float *stats, void *stream);

/*
 * lmhead_xent_mean -- mean reduction of the per-row loss
 *
 *  Not an operation the pages describe: they state no reduction.  The
 *  workloads this library is measured on take the mean loss over the rows
 *  whose target is not ignore_index (-100 there), the usual language-model
 *  training loss, and its 1 / n_valid is the upstream gradient of every row.
 *
 *  loss     FP32 [n_rows]; target int32 [n_rows] (rows equal to ignore_index
 *           are excluded).  loss may be NULL when mean_out is NULL: 1 / n_valid
 *           depends on the targets only, so it can be had before the forward
 *           (for lmhead_xent_fused).
 *  mean_out FP32 scalar: sum of valid losses / n_valid (0 if n_valid == 0),
 *           or NULL.
 *  inv_nvalid_out FP32 scalar: 1 / n_valid (0 if n_valid == 0), or NULL; it is
 *           the upstream gradient of every row of a mean loss and can be passed
 *           to lmhead_xent_bwd as `dloss` with dloss_stride 0.
 *  One workgroup sums in a fixed order (FP64), so the result is
 *  deterministic.  Both outputs NULL is a no-op.
 */
int32_t lmhead_xent_mean(const float *loss, const int32_t *target, int32_t ignore_index,
                         int64_t n_rows, float *mean_out, float *inv_nvalid_out,
                         void *stream);

/*
 * lmhead_xent_bwd -- fused cross-entropy backward in FP32          ([XENT])
 *
 *  dlogits_ij = dloss_i * (exp(z_ij - m_i) / d_i - [j == target_i]),
 *  computed in FP32 from the logits (read once more) and the stats record of
 *  lmhead_xent_fwd; rows whose target is ignore_index get zeros.
 *
 *  logits   FP32 [n_rows x n_cols], leading dimension ld.
 *  stats    FP32 [n_rows x 4] from lmhead_xent_fwd (m and d are used).
 *  target   int32 [n_rows]; ignore_index as in the forward.
 *  dloss    FP32 device pointer: dloss_i = dloss[dloss_stride * i] with
 *           dloss_stride 0 (one scalar for every row, e.g. the inv_nvalid
 *           output of lmhead_xent_mean) or 1 (one value per row).
 *  dlogits  [n_rows x n_cols], leading dimension ldg, type grad_dtype:
 *             LMH_FP32 -- FP32 gradient;
 *             LMH_BF16 -- the same FP32 value rounded to BF16 (nearest-even),
 *                         the cast the backward applies before the GEMMs
 *                         ([MIXED]);
 *           In place: dlogits == logits with ldg == ld and LMH_FP32 writes the
 *           gradient over the logits (each element is read, then overwritten
 *           by the same thread).  Any other overlap with logits, stats, target
 *           or dloss, or BF16 in place, is LMH_ERR_ALIAS.
 *  A target outside [0, n_cols) that is not ignore_index yields a NaN row.
 */
int32_t lmhead_xent_bwd(const float *logits, int64_t ld, const float *stats,
                        const int32_t *target, int32_t ignore_index,
                        const float *dloss, int64_t dloss_stride,
                        void *dlogits, int64_t ldg, int32_t grad_dtype,
                        int64_t n_rows, int64_t n_cols, void *stream);

/*
 * lmhead_xent_fused -- forward and backward in one read of the logits ([XENT])
 *
 *  For an upstream gradient known before the forward (a mean loss: dloss =
 *  1 / n_valid, which lmhead_xent_mean gives from the targets alone): writes
 *  the forward's loss and stats record (as lmhead_xent_fwd) and the
 *  backward's dlogits (as lmhead_xent_bwd) while reading the logits once.
 *  [XENT]'s discussion: the original fused kernel wrote the gradient over its
 *  input during the forward; the FP32 backward of [XENT] "Changes" is kept.
 *  Rows of up to 65536 columns are held in registers by one workgroup per
 *  row (8 bytes of traffic per element with FP32 gradients instead of 12);
 *  longer rows run the forward and then the backward (two reads).
 *
 *  Arguments as lmhead_xent_fwd (logits, ld, n_rows, n_cols, target,
 *  ignore_index, loss (may be NULL), stats) and lmhead_xent_bwd (dloss,
 *  dloss_stride, dlogits, ldg, grad_dtype, in place when dlogits == logits
 *  with ldg == ld and LMH_FP32).  The stats, loss and dlogits outputs must not
 *  overlap each other, the target or dloss; stats and loss must not overlap
 *  the logits.  Results agree with lmhead_xent_fwd + lmhead_xent_bwd to
 *  rounding (the row reduction runs over a different thread layout).
 */
int32_t lmhead_xent_fused(const float *logits, int64_t ld, int64_t n_rows, int64_t n_cols,
                          const int32_t *target, int32_t ignore_index,
                          const float *dloss, int64_t dloss_stride,
                          float *loss, float *stats,
                          void *dlogits, int64_t ldg, int32_t grad_dtype, void *stream);

/*
 * lmhead_dgrad -- input gradient dX[M x K] = dlogits[M x V] . W[V x K]
 *
 *  The GEMM that consumes the BF16 logits gradient ([MIXED]: the backward
 *  casts the gradient to BF16 for the following GEMMs).
 *  dlogits BF16 [M x V], ldd >= V;  W BF16 [V x K], ldw >= K;
 *  dX [M x K], ldx >= K, dx_dtype LMH_BF16 (nearest-even) or LMH_FP32.
 *  FP32 accumulation; V == 0 writes zeros.  dX must not overlap the inputs.
 */
int32_t lmhead_dgrad(const void *dlogits, int64_t ldd, const void *W, int64_t ldw,
                     void *dX, int64_t ldx, int32_t dx_dtype,
                     int64_t M, int64_t K, int64_t V, void *stream);

/*
 * lmhead_dgrad_workspace_bytes / lmhead_dgrad_ws -- lmhead_dgrad with the sum
 * over V split in parts ([MIXED] "What does this PR do?", the GEMMs after the
 * BF16 cast: the same product dX = dlogits . W).
 *
 *  When M x K has too few 256 x 256 output tiles to fill the chip (fewer than
 *  256, e.g. M = 1024, K = 8192, or few tokens), the V sum is split `splits`
 *  ways; every part writes an FP32 partial dX into `workspace`, and a second
 *  kernel adds the partials in split order and stores dX (FP32, or BF16
 *  rounded to nearest-even once, from the FP32 sum).  splits == 0 picks the
 *  shape's default (1 - 16 parts, for ~256 workgroups); 1 <= splits <= 16
 *  asks for that many parts of whole 64-deep stages (fewer when V is small).
 *  The result is deterministic run to run; its summation order differs from
 *  lmhead_dgrad's, so the two agree within the FP32 tolerance, and bitwise on
 *  integer inputs.
 *
 *  lmhead_dgrad_workspace_bytes returns the workspace bytes that
 *  lmhead_dgrad_ws needs for (M, K, V, splits): parts x M x K4 x 4 with K4 =
 *  K rounded up to a multiple of 4, or 0 when the shape runs unsplit; a
 *  negative LMH_ERR_SHAPE for negative sizes, splits outside [0, 16], or a dX
 *  of more than 2^44 elements.
 *
 *  lmhead_dgrad_ws takes lmhead_dgrad's arguments plus splits and the
 *  caller's device workspace (16-byte aligned, workspace_bytes >= the size
 *  above, else LMH_ERR_ALIGN / LMH_ERR_SHAPE; NULL -> LMH_ERR_NULL).  The
 *  workspace must not overlap dlogits, W or dX (LMH_ERR_ALIAS); its contents
 *  on entry do not matter and are garbage afterwards.  When the size above is
 *  0 the call is lmhead_dgrad and the workspace is not touched.  Two calls that
 *  share a workspace must be ordered on one stream.
 */
int64_t lmhead_dgrad_workspace_bytes(int64_t M, int64_t K, int64_t V, int32_t splits);
int32_t lmhead_dgrad_ws(const void *dlogits, int64_t ldd, const void *W, int64_t ldw,
                        void *dX, int64_t ldx, int32_t dx_dtype,
                        int64_t M, int64_t K, int64_t V, int32_t splits,
                        void *workspace, int64_t workspace_bytes, void *stream);

/*
 * lmhead_dgrad_noalloc -- lmhead_dgrad_ws with no workspace argument and no
 * allocation, for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).
 *
 *  Same arguments, split choice, kernels and results as lmhead_dgrad_ws
 *  (bitwise, for the same splits); the FP32 partial sums go to a fixed device
 *  array of LMH_DGRAD_NOALLOC_MAX_BYTES (64 MiB) that the library holds on
 *  each GPU it runs on until the process ends.  Shapes whose split needs more
 *  than that (lmhead_dgrad_workspace_bytes(M, K, V, splits) >
 *  LMH_DGRAD_NOALLOC_MAX_BYTES) return LMH_ERR_SCRATCH before anything is
 *  enqueued; shapes that run unsplit are lmhead_dgrad.  The first call on a
 *  device looks up the array's device address (with that device current); the
 *  call never allocates, frees or clears memory.  Every call on one GPU
 *  shares that GPU's array: calls that may overlap on one GPU (different
 *  streams, or host threads without ordering) race and must be serialised
 *  by the caller.  Nothing needs the array zeroed: every partial is written
 *  before it is read.
 */
#define LMH_DGRAD_NOALLOC_MAX_BYTES (((int64_t)64) << 20)
int32_t lmhead_dgrad_noalloc(const void *dlogits, int64_t ldd, const void *W, int64_t ldw,
                             void *dX, int64_t ldx, int32_t dx_dtype,
                             int64_t M, int64_t K, int64_t V, int32_t splits, void *stream);

/*
 * lmhead_wgrad -- weight gradient dW[V x K] (+)= dlogits[M x V]^T . x[M x K]
 *
 *  The other GEMM that consumes the BF16 logits gradient ([MIXED] "What does
 *  this PR do?": the backward casts the gradient to BF16 for the GEMMs that
 *  follow).  The pages say nothing of dW's type; it is kept in FP32 (the
 *  GEMM's accumulator), so that it can be accumulated over micro-batches.
 *
 *  dlogits BF16 [M x V], ldd >= V;  x BF16 [M x K], ldx >= K;
 *  dW FP32 [V x K], ldw >= K.  accumulate == 0 overwrites dW; accumulate != 0
 *  adds the product to the FP32 values already in dW.  FP32 accumulation over
 *  M; M == 0 writes zeros (or leaves dW unchanged when accumulating).
 *  dW must not overlap the inputs.
 */
int32_t lmhead_wgrad(const void *dlogits, int64_t ldd, const void *x, int64_t ldx,
                     float *dW, int64_t ldw, int32_t accumulate,
                     int64_t M, int64_t K, int64_t V, void *stream);

/*
 * lmhead_logits_lora -- logits of a batch whose tokens use different low-rank
 * adapters beside the shared vocabulary weight
 *
 *  z[m][v] = sum_k x[m][k] W[v][k] + s_a sum_j (sum_k x[m][k] A_a[j][k]) B_a[v][j],
 *  a = adapter[m].  An extension the pages do not describe: lmhead_logits for
 *  a batch that mixes requests of several fine-tuned variants.
 *
 *  x, W, out, out_dtype as lmhead_logits (FP32 keeps the FP32 sum, BF16 rounds
 *  it once).
 *  A        BF16 [n_adapters][rank][K], row pitch lda >= K, pitch stride_a
 *           between adapters (both multiples of 8; stride_a at least one
 *           adapter's span).
 *  B        BF16 [n_adapters][V][rank], row pitch ldb >= rank, pitch stride_b
 *           (the same).
 *  adapter  int32 [M], the token's adapter in any order; a negative value:
 *           none (the row equals lmhead_logits' up to rounding).  A value >=
 *           n_adapters cannot be reported from the kernel: that row is NaN.
 *  scale    FP32 [n_adapters] or NULL (1).
 *  rank     1 .. 128, n_adapters >= 0 (at most 2^23 - 2), M <= 2^22.
 *  One token's result depends on its own x and adapter only: a NaN or infinity
 *  in another token or another adapter of the batch does not reach it.
 *  A x is an FP32 sum and enters the second product unrounded (in three BF16
 *  pieces of 8 bits, some of them zero: an infinity in a token's own row of B
 *  gives an infinity or NaN).
 *  workspace: device memory of at least lmhead_logits_lora_workspace_bytes(M,
 *  K, V, rank, out_dtype) bytes (negative LMH_ERR_* for bad sizes), 16-byte
 *  aligned; its contents do not matter on entry.  Two calls that share one
 *  must be ordered on one stream.  out and workspace must not overlap each
 *  other or an input.
 */
int64_t lmhead_logits_lora_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t rank,
                                           int32_t out_dtype);
int32_t lmhead_logits_lora(const void *x, int64_t ldx, const void *W, int64_t ldw, const void *A,
                           int64_t lda, int64_t stride_a, const void *B, int64_t ldb,
                           int64_t stride_b, const int32_t *adapter, const float *scale,
                           int64_t n_adapters, int64_t rank, void *out, int64_t ldo,
                           int32_t out_dtype, int64_t M, int64_t K, int64_t V, void *workspace,
                           int64_t workspace_bytes, void *stream);

/*
 * lmhead_lora_bwd -- gradients of the adapters' part of lmhead_logits_lora
 *
 *  With u[m] = s_a A_a x[m] and t[m] = s_a B_a^T g[m] (g = dlogits, a =
 *  adapter[m]):
 *    dX[m]  = A_a^T t[m]          (the adapters' part only: lmhead_dgrad with
 *                                  FP32 dX gives the shared part, and
 *                                  accumulate adds this one to it)
 *    dA_a   = sum over a's tokens of t[m] x[m]^T
 *    dB_a   = sum over a's tokens of g[m] u[m]^T
 *  dlogits BF16 [M x V], ldd >= V; x BF16 [M x K]; A, B, adapter, scale, rank
 *  and n_adapters as lmhead_logits_lora.
 *  dX FP32 [M x K], dA FP32 [n_adapters][rank][K], dB FP32
 *  [n_adapters][V][rank], pitches multiples of 4; each may be NULL (not
 *  computed).  accumulate == 0 overwrites them (an adapter without tokens and
 *  a token without an adapter get zeros), accumulate != 0 adds to them.  A
 *  token whose id is >= n_adapters gets a NaN row in dX and enters no other
 *  gradient.  u and t are FP32 sums, not rounded before the second product (an
 *  infinity that meets them gives an infinity or NaN, as in the forward).
 *  Results are deterministic.
 *  workspace as lmhead_logits_lora, of lmhead_lora_bwd_workspace_bytes(M, K,
 *  V, rank, n_adapters) bytes.  Limits (LMH_ERR_SHAPE): M <= 2^22,
 *  ceil(V / 256) n_adapters and ceil(K / 256) (2 n_adapters + M / 64 + 2) <=
 *  2^23, ceil(M / 256) (n_adapters + 2) <= 2^31.
 */
int64_t lmhead_lora_bwd_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t rank,
                                        int64_t n_adapters);
int32_t lmhead_lora_bwd(const void *dlogits, int64_t ldd, const void *x, int64_t ldx, const void *A,
                        int64_t lda, int64_t stride_a, const void *B, int64_t ldb, int64_t stride_b,
                        const int32_t *adapter, const float *scale, int64_t n_adapters, int64_t rank,
                        float *dX, int64_t lddx, float *dA, int64_t ldda, int64_t stride_da,
                        float *dB, int64_t lddb, int64_t stride_db, int32_t accumulate, int64_t M,
                        int64_t K, int64_t V, void *workspace, int64_t workspace_bytes,
                        void *stream);

/*
 * lmhead_beam_select -- the next beams of a beam search from its logits
 *
 *  Request b holds beams w < n_beams; row b n_beams + w of the logits and
 *  scores[b][w] (the beam's summed log-probability) belong to beam w.  Every
 *  (w, v) is a candidate with
 *    c = scores[b][w] + ((z[v] - max z) - log sum_v exp(z[v] - max z)),
 *  except that a finished beam has c = scores[b][w] at v = eos and -inf
 *  elsewhere.  A NaN c counts as -inf, as does every candidate of a beam whose
 *  score is NaN or +inf.  The n_out largest are returned in descending order,
 *  equal ones by ascending w, then descending logit, then ascending v:
 *    out_scores[b][i] = c (computed in FP64; the terms of the sum below the
 *    largest, which is exactly 1, have a relative error below 4e-9; rounded
 *    once to FP32: a candidate below its range, such as a beam at -FLT_MAX
 *    over a logit masked with it, comes after those in it and before those at
 *    -inf, and is returned as -inf),
 *    out_parent[b][i] = w, out_token[b][i] = v,
 *    out_finished[b][i] = 1 if beam w was finished or v == eos, else 0.
 *  No c is above its beam's score; a row with one finite logit has c equal to
 *  it; rows that differ by a constant (each z - max z exact) have equal c.  A
 *  row whose largest logit lies below -2^126 holds only masks of the type's
 *  lowest value: it is not normalised, the logarithm counting as 0 (it would
 *  be lost beside max z in 64 bits).
 *  The logits are read once; rows of finished beams and of beams whose score
 *  is -inf, NaN or +inf are not read (but for at most 2 n_out values where
 *  fewer than n_out candidates lie above -inf).
 *
 *  logits   [n_requests n_beams x n_cols], leading dimension ld, FP32 or BF16
 *           (logits_dtype), as lmhead_logits writes them.
 *  scores   FP32 [n_requests x n_beams]; finished uint8 of that shape or NULL
 *           (none).  eos: any value; outside [0, n_cols) no token ends a beam.
 *  Limits: 1 <= n_beams, n_out <= 64; n_out <= n_beams n_cols < 2^31;
 *  n_requests <= 2^23 and n_requests n_beams ceil(n_cols / 2048) <= 2^25.
 *  out_scores may be `scores` and out_finished may be `finished` when n_out ==
 *  n_beams; no other overlap.
 *  workspace as lmhead_logits_lora, of lmhead_beam_select_workspace_bytes(
 *  n_requests, n_beams, n_cols, n_out) bytes.
 */
int64_t lmhead_beam_select_workspace_bytes(int64_t n_requests, int64_t n_beams, int64_t n_cols,
                                           int64_t n_out);
int32_t lmhead_beam_select(const void *logits, int64_t ld, int32_t logits_dtype, int64_t n_requests,
                           int64_t n_beams, int64_t n_cols, const float *scores,
                           const uint8_t *finished, int32_t eos, int64_t n_out, float *out_scores,
                           int32_t *out_parent, int32_t *out_token, uint8_t *out_finished,
                           void *workspace, int64_t workspace_bytes, void *stream);

/*
 * lmhead_beam_reorder -- per-beam states after a selection
 *
 *  A state is n_outer x (n_requests beams) x n_heads runs of n_positions
 *  positions of position_bytes contiguous bytes (a key or value cache of
 *  [layer][beam][head][position][dim], token histories [beam][position], ...),
 *  of any element type; src_outer / src_row / src_head are its strides in
 *  BYTES, and any alignment will do.
 *    dst run (o, b beams_out + i, h) = src run (o, b beams_in + parent[b][i], h)
 *  for the first lengths[b] positions (int32 [n_requests], clamped to [0,
 *  n_positions]; NULL: all).  Positions from there on, and rows whose parent
 *  lies outside [0, beams_in), are left as they were.
 *  parent int32 [n_requests x beams_out], as lmhead_beam_select writes it.
 *  In place: dst == src with equal strides and beams_out == beams_in; any
 *  parent map, rows that stay are not touched.  Any other overlap of dst with
 *  src, parent or lengths is LMH_ERR_ALIAS.  The runs of dst must be disjoint
 *  (LMH_ERR_SHAPE).  Limits: beams <= 64; every count below 2^31; n_requests
 *  n_heads (n_positions position_bytes / 1024 + 2) <= 2^23; spans up to 2^44
 *  bytes (a run of one position may be as long as these allow, 8 GiB).
 */
int32_t lmhead_beam_reorder(const void *src, int64_t src_outer, int64_t src_row, int64_t src_head,
                            void *dst, int64_t dst_outer, int64_t dst_row, int64_t dst_head,
                            const int32_t *parent, const int32_t *lengths, int64_t n_outer,
                            int64_t n_requests, int64_t beams_in, int64_t beams_out,
                            int64_t n_heads, int64_t n_positions, int64_t position_bytes,
                            void *stream);

/*
 * lmhead_logprobs -- log-probabilities of given tokens, with the rows' entropies,
 * the tokens' ranks and the most likely alternatives
 *
 *  With x = (z - max z) / T and p = softmax(z / T), row i of the logits gives
 *    logprob[i] = log p[token[i]]; 0 for token[i] == ignore_index, NaN for any
 *                 other token outside [0, n_cols),
 *    entropy[i] = - sum_j p_j log p_j,
 *    rank[i]    = the number of columns before the token in descending order of
 *                 the logits, equal ones by ascending column (0: the likeliest);
 *                 -1 where the log-probability is 0 by ignore_index or NaN,
 *    top_logprob[i][l], top_token[i][l] = log p and column of the n_top first
 *                 columns in that order; columns at -inf are not listed, what
 *                 they leave free holds -inf and -1,
 *    stats[i]   = {m = max z, d = sum exp(x), entropy, logprob}: what
 *                 lmhead_logprobs_bwd needs.
 *  The logits are read once.  A wave's sums are FP32 and joined in FP64; ranks and
 *  alternatives come from the logits, not from rounded probabilities.  A row that
 *  holds NaN or +inf, one of -inf only, and one whose temperature is none, is NaN
 *  (tokens -1).
 *
 *  logits   [n_rows x n_cols], leading dimension ld, FP32 or BF16 (logits_dtype),
 *           as lmhead_logits writes them.
 *  token    int32 [n_rows], or NULL: then logprob and rank must be NULL too, and
 *           stats holds 0 in logprob's place.
 *  temperature  FP32, stride 0 (one value) or 1 (one per row), or NULL (1).  One
 *           that is not positive and finite is none, and neither is one so small
 *           (below 4.3e-39) that log2(e) / T is beyond FP32.
 *  logprob, entropy, rank  [n_rows] or NULL (not wanted).
 *  top_logprob FP32, top_token int32 [n_rows x n_top], contiguous; not used when
 *           n_top == 0.
 *  Limits: 1 <= n_cols <= 2^30, n_top <= min(64, n_cols).
 *  workspace as lmhead_logits_lora, of lmhead_logprobs_workspace_bytes(n_rows,
 *  n_cols, n_top) bytes (may be NULL where that is 0).  Outputs overlap neither
 *  inputs nor each other.
 */
int64_t lmhead_logprobs_workspace_bytes(int64_t n_rows, int64_t n_cols, int64_t n_top);
int32_t lmhead_logprobs(const void *logits, int64_t ld, int32_t logits_dtype, int64_t n_rows,
                        int64_t n_cols, const int32_t *token, int32_t ignore_index,
                        const float *temperature, int64_t temperature_stride, int64_t n_top,
                        float *logprob, float *entropy, int32_t *rank, float *top_logprob,
                        int32_t *top_token, float *stats, void *workspace, int64_t workspace_bytes,
                        void *stream);

/*
 * lmhead_logprobs_bwd -- gradient of lmhead_logprobs with respect to the logits
 *
 *    dlogits[i][j] = (1 / T) [ g_i ([j == token[i]] - p_j) - h_i p_j (log p_j + H_i) ],
 *  g = dlogprob, h = dentropy (FP32, stride 0 or 1; NULL: 0), H the entropy.
 *  stats as the forward wrote it for the same logits and temperature.  g counts
 *  as 0 in rows of ignore_index (token NULL: in all rows).  A row whose token is
 *  neither ignore_index nor a column gets NaN, whatever its g and h; any other
 *  whose g and h are 0 gets zeros, whatever its logits and its temperature.
 *  dlogits [n_rows x n_cols], leading dimension ldg, FP32 or BF16 (grad_dtype:
 *  the FP32 value rounded once); it may be the logits themselves when types and
 *  leading dimensions agree, and otherwise overlaps no input.
 */
int32_t lmhead_logprobs_bwd(const void *logits, int64_t ld, int32_t logits_dtype,
                            const float *stats, const int32_t *token, int32_t ignore_index,
                            const float *temperature, int64_t temperature_stride,
                            const float *dlogprob, int64_t dlogprob_stride,
                            const float *dentropy, int64_t dentropy_stride, void *dlogits,
                            int64_t ldg, int32_t grad_dtype, int64_t n_rows, int64_t n_cols,
                            void *stream);

/*
 * lmhead_distill_fwd -- cross-entropy against a teacher known by its top tokens
 *
 *  Row i has a list of n_list tokens c_l = teacher_token[i][l] with values v_l =
 *  teacher_value[i][l]; an entry of a negative token or of value -inf is absent
 *  (so that lists may be shorter, and lmhead_logprobs' alternatives fit).  With
 *  p = softmax(z / T):
 *    tail == 0: the values are logits; q = softmax(v / T) over the list,
 *      loss[i] = sum_l q_l (log q_l - log p_{c_l}).
 *    tail != 0: the values are log-probabilities (of the teacher at temperature
 *      T; used as they are), q_l = exp(v_l), and all other columns are one class
 *      with q_r = max(0, 1 - sum q) and p_r the sum of their p:
 *      loss[i] = sum_l q_l (log q_l - log p_{c_l}) + q_r (log q_r - log p_r).
 *      Where every other column is at -inf that class is left out.
 *  Both are Kullback-Leibler divergences (multiply the upstream gradient by T^2
 *  to scale them as is common).  A token that is listed twice counts twice in q
 *  and once in p.  A row whose list is empty has loss 0 and gradient 0.  A row
 *  with a token >= n_cols, a value of NaN or +inf, a logit of NaN or +inf, no
 *  logit above -inf or a temperature that is none (see lmhead_logprobs) is NaN.
 *  A listed column at -inf with q > 0 makes the loss +inf.
 *    stats[i] = 8 floats: {max z, sum exp((z - max z) / T), loss, sum of q (with
 *      q_r), o, w, t, u}: off the list the gradient per unit of dloss / T is
 *      exp((z - o) / T) w, and q_l = exp((v_l - t) / T) / u (tail != 0: t = 0,
 *      u = 1, without T); all 0 where the list is empty.
 *  logits, logits_dtype, temperature as lmhead_logprobs.  teacher_token int32 and
 *  teacher_value FP32 or BF16 (teacher_dtype), [n_rows x n_list], row pitches
 *  ldt, ldv >= n_list, aligned to their elements.
 *  loss [n_rows] or NULL.  Limits: 1 <= n_cols <= 2^30, 0 <= n_list <= 256.
 *  workspace as lmhead_logits_lora, of lmhead_distill_workspace_bytes(n_rows,
 *  n_cols) bytes (may be NULL where that is 0).  Outputs overlap neither inputs
 *  nor each other.
 */
int64_t lmhead_distill_workspace_bytes(int64_t n_rows, int64_t n_cols);
int32_t lmhead_distill_fwd(const void *logits, int64_t ld, int32_t logits_dtype, int64_t n_rows,
                           int64_t n_cols, const int32_t *teacher_token, int64_t ldt,
                           const void *teacher_value, int64_t ldv, int32_t teacher_dtype,
                           int64_t n_list, int32_t tail, const float *temperature,
                           int64_t temperature_stride, float *loss, float *stats, void *workspace,
                           int64_t workspace_bytes, void *stream);

/*
 * lmhead_distill_bwd -- its gradient with respect to the logits
 *
 *  With q = 0 off the list, and Q = sum q (+ q_r):
 *    tail == 0: dlogits[i][j] = (dloss_i / T) (p_j - q_j)
 *    tail != 0: dlogits[i][j] = (dloss_i / T) (Q p_j - q_j) on the list,
 *               dlogits[i][j] = (dloss_i / T) p_j (Q - q_r / p_r) off it.
 *  stats as lmhead_distill_fwd wrote it for the same logits, lists, tail and
 *  temperature.  dloss FP32, stride 0 or 1; a row whose dloss is 0 gets zeros,
 *  whatever its logits, its list and its temperature (the forward's loss of such
 *  a row is NaN all the same where one of them is bad).  dlogits as
 *  lmhead_logprobs_bwd.
 */
int32_t lmhead_distill_bwd(const void *logits, int64_t ld, int32_t logits_dtype,
                           const float *stats, const int32_t *teacher_token, int64_t ldt,
                           const void *teacher_value, int64_t ldv, int32_t teacher_dtype,
                           int64_t n_list, int32_t tail, const float *temperature,
                           int64_t temperature_stride, const float *dloss, int64_t dloss_stride,
                           void *dlogits, int64_t ldg, int32_t grad_dtype, int64_t n_rows,
                           int64_t n_cols, void *stream);

/*
 * lmhead_distill_fused -- lmhead_distill_fwd and lmhead_distill_bwd in one call,
 * for an upstream gradient known before the forward
 *
 *  Rows of up to 65536 columns are read once, longer ones twice; a row whose
 *  list is empty is not read, or (beyond 65536 columns) as far as its parts' first
 *  segments by the forward.  Its results agree with the two calls' up to rounding.
 */
int32_t lmhead_distill_fused(const void *logits, int64_t ld, int32_t logits_dtype, int64_t n_rows,
                             int64_t n_cols, const int32_t *teacher_token, int64_t ldt,
                             const void *teacher_value, int64_t ldv, int32_t teacher_dtype,
                             int64_t n_list, int32_t tail, const float *temperature,
                             int64_t temperature_stride, const float *dloss, int64_t dloss_stride,
                             float *loss, float *stats, void *dlogits, int64_t ldg,
                             int32_t grad_dtype, void *workspace, int64_t workspace_bytes,
                             void *stream);

/*
 * lmhead_diag_mfma_loop -- diagnostic: the sustained BF16 matrix-core rate.
 *
 *  Not a step of the method: a register-only loop that the benchmark runs
 *  beside the GEMMs so their throughput can be compared with what the chip
 *  sustains under full matrix load at its power limit (the datasheet peak
 *  assumes 2.4 GHz).  n_workgroups workgroups of 256 threads (4 waves) each
 *  run 8 independent chains of `iters` 32x32x16 BF16 MFMAs:
 *  2 * 32 * 32 * 16 * 8 * iters FLOP per wave, 4 waves per workgroup.
 *  operands selects the data, which sets how much the multipliers switch and
 *  so the power drawn:
 *    0  every operand 1.0.  sink FP32 [n_workgroups * 256] receives, per
 *       thread, 128 * iters exactly (the sum of element 0 of its 8
 *       accumulators), which checks that every MFMA ran.
 *    1  pseudo-random BF16 operands (random sign and 7 mantissa bits, |v| in
 *       [1, 2), a different set per lane) cycling through (A1, B1), (A2, B2),
 *       (A1, -B1), (A2, -B2), so every accumulator returns to exactly 0 each
 *       fourth MFMA of its chain (all partial sums are exact in FP32).  sink
 *       receives, per thread, element 0 of its 8 accumulators weighted
 *       1 ... 8: 0 when iters % 4 == 0, and for other iters a value that
 *       depends only on iters % 4.
 *  Limits: operands in {0, 1}, 0 <= iters, 128 * iters < 2^24 and
 *  0 <= n_workgroups <= 65536, else LMH_ERR_SHAPE; n_workgroups == 0 is a
 *  no-op.  sink must not be NULL (LMH_ERR_NULL) and 16-byte aligned.
 */
int32_t lmhead_diag_mfma_loop(int64_t iters, int64_t n_workgroups, int32_t operands,
                              float *sink, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LMHEAD_H */
