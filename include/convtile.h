/*
 * convtile -- NCHW 2-D convolution (implicit GEMM on CDNA4 matrix cores) and
 * per-channel broadcast for AMD Instinct MI355X (gfx950).  C ABI.
 *
 * The operation (TVM tutorial "Tuning High Performance Convolution on NVIDIA
 * GPUs", Step 1, the conv2d_nchw compute of the template):
 *
 *   y[n][f][oy][ox] = sum_{c<CI} sum_{ky<KH} sum_{kx<KW}
 *                     xp[n][c][oy*stride+ky][ox*stride+kx] * w[f][c][ky][kx]
 *
 *   xp = x zero-padded by `pad` on every side (never materialised: padding is
 *   applied inline while gathering), dilation 1, no kernel flip, and
 *   OH = (H + 2 pad - KH) / stride + 1, OW likewise (integer division).
 *   Output is always fp32 (the template's out_dtype='float32'), also for fp16 /
 *   bf16 inputs, which are multiplied exactly and accumulated in fp32.
 *
 * Optional per-channel epilogue (Paddle PR "[CINN] Add the TileBroadcastTactic
 * for NCHW broadcast", Performance Impact: per-channel div/exp/rsqrt chains,
 * with the channel bound to a grid axis so its value is computed once per
 * workgroup):
 *   CT_EPI_NONE            out = y
 *   CT_EPI_BIAS            out = y + bias[f]
 *   CT_EPI_EXP_BIAS_RSQRT  out = exp(y + bias[f]) * rsqrt(var[f] + eps)
 *
 * Layouts (all contiguous, row-major, device memory owned by the caller):
 *   x    [N][CI][H][W]      dtype CT_F32 (float), CT_F16 (IEEE half), CT_BF16
 *   w    [CO][CI][KH][KW]   same dtype as x
 *   y    [N][CO][OH][OW]    float; must not alias x, w, bias or var
 *   bias [CO], var [CO]     float (NULL when the epilogue does not read them)
 *
 * Conventions
 *   - Every entry point returns a status (CT_OK = 0, negative on error) and
 *     never throws across the ABI.  ct_last_error() gives a message for the
 *     last failure on the calling thread.
 *   - Argument errors are reported with CT_ERR_INVALID_ARG before any HIP call.
 *   - `stream` is a hipStream_t (NULL = the default stream).  Launch calls are
 *     asynchronous on that stream.  Once a device is set up (ct_init, or the
 *     first launch on it) and a stream's workspace has grown to what a shape
 *     needs (the first split-reduction launch of that size on the stream),
 *     a launch neither synchronises nor allocates, so it may be captured into
 *     a HIP graph.  A launch that would need either step while its stream is
 *     capturing returns CT_ERR_UNSUPPORTED and captures nothing.
 *   - The library owns: the compiled kernels, a process-wide tile-config cache
 *     (mutex-protected), a launch plan per (device, shape) derived from it,
 *     and per-(device, stream) split-reduction workspaces.  A workspace grows
 *     by allocating a larger buffer; the buffer it replaces stays allocated
 *     until ct_release(), because a graph captured earlier on that stream may
 *     still use it.  Two launches that use split reduction on the same stream
 *     are ordered by the stream; launches on different streams get different
 *     workspaces.  A captured launch keeps the workspace of the stream it was
 *     captured on: replays of such graphs must not overlap one another or
 *     other launches on that stream.
 */
#ifndef CONVTILE_H
#define CONVTILE_H

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---------------------------------------------------- */
#define CT_OK 0
#define CT_ERR_INVALID_ARG (-1)  /* bad shape, NULL pointer, unknown enum      */
#define CT_ERR_UNSUPPORTED (-2)  /* legal arguments no kernel here can run    */
#define CT_ERR_HIP (-3)          /* a HIP runtime call failed                 */
#define CT_ERR_NO_MEMORY (-4)    /* workspace / scratch allocation failed     */
#define CT_ERR_IO (-5)           /* cache file could not be read or written   */
#define CT_ERR_TUNE_FAILED (-6)  /* no candidate of the search ran correctly  */

/* ---- enums ------------------------------------------------------------ */
enum ct_dtype {
    CT_F32 = 0,
    CT_F16 = 1,
    CT_BF16 = 2,
    CT_E4M3 = 3  /* OCP 8-bit float; transformer blocks only (below)          */
};
enum ct_epilogue { CT_EPI_NONE = 0, CT_EPI_BIAS = 1, CT_EPI_EXP_BIAS_RSQRT = 2 };
enum ct_bcast_op { CT_BC_EXP = 0 };
enum ct_bcast_mode {
    CT_BC_AUTO = 0,    /* channel-bound when it applies, else flat            */
    CT_BC_CHANNEL = 1, /* channel index on a grid axis; value computed once   */
    CT_BC_FLAT = 2     /* all axes fused; value loaded and computed per element */
};

/* Measurement outcome codes of a tuning trial (the meanings of the autotvm
 * MeasureResult error_no values printed in the tutorial's tuning log). */
enum ct_trial_error {
    CT_TRIAL_OK = 0,
    CT_TRIAL_ILLEGAL = 1,  /* rejected by the legality check, never launched */
    CT_TRIAL_RUNTIME = 4,  /* HIP error, or output differs from the reference */
    CT_TRIAL_TIMEOUT = 6   /* exceeded the per-trial time limit               */
};

/* One point of a shape's tile-config space. */
typedef struct ct_tile_config {
    int variant;     /* kernel variant id (see ct_variant_info)               */
    int split_k;     /* S: workgroups that share one output tile's reduction  */
    int stages;      /* LDS stages each workgroup runs                        */
    int kc;          /* input channels per LDS stage                          */
    long long index; /* flat index in the shape's space; -1 = not from space  */
    float us;        /* mean microseconds per launch when measured, else 0    */
    int error_no;    /* ct_trial_error of the measurement, 0 if never timed   */
} ct_tile_config;

/* A compiled kernel variant (one instantiation of the tiled template). */
typedef struct ct_variant_desc {
    char name[48];
    int dtype;        /* ct_dtype it accepts                                   */
    int kind;         /* 0 = direct (one lane per output), 1 = implicit GEMM   */
    int mfma_m, mfma_n, mfma_k; /* matrix-core instruction shape (0 for direct) */
    int waves_m, waves_n, waves_k; /* waves per workgroup along CO, P, K       */
    int reps_m, reps_n;  /* MFMA tiles per wave along CO and P                 */
    int tile_m, tile_n;  /* workgroup output tile: CO x P                      */
    int kc_max;          /* most input channels one LDS stage holds            */
    int threads;         /* workgroup size                                     */
} ct_variant_desc;

/* One timed candidate of ct_conv2d_tune (autotvm MeasureResult analogue). */
typedef struct ct_tune_record {
    ct_tile_config cfg;
    float costs_us[3];   /* mean us per launch of each repeat                  */
    int n_costs;
    int error_no;        /* ct_trial_error                                     */
    double all_cost_s;   /* wall seconds spent on this trial                   */
    double timestamp;    /* seconds since the epoch when the trial ended       */
} ct_tune_record;

/* ---- convolution ----------------------------------------------------- */

/* Forward convolution with the cached tile config for this shape (or the
 * built-in default when none is cached; with the environment variable
 * CT_TUNE=1, a shape with no cached config is first searched with
 * ct_conv2d_tune on `stream`, once per process -- CT_TUNE_TRIALS bounds the
 * trials, CT_TUNE_MS sets min_repeat_ms (default 20) -- unless the stream is
 * capturing).  Shapes/layouts as above; `eps` is
 * used only by CT_EPI_EXP_BIAS_RSQRT.  Errors: CT_ERR_INVALID_ARG for any
 * dimension <= 0, stride <= 0, pad < 0, OH or OW <= 0, NULL x/w/y, unknown
 * dtype/epilogue, or bias/var missing when the epilogue reads them;
 * CT_ERR_UNSUPPORTED when the device is not set up or the stream's workspace
 * must grow while the stream is capturing (see Conventions);
 * CT_ERR_NO_MEMORY if the split workspace cannot grow; CT_ERR_HIP on a launch
 * failure. */
int ct_conv2d_nchw_fwd(const void* x, const void* w, float* y,
                       int N, int CI, int H, int W, int CO, int KH, int KW,
                       int stride, int pad, int dtype, int epilogue,
                       const float* bias, const float* var, float eps,
                       void* stream);

/* Half-precision filters in the layout the kernels stage from.  The
 * half-precision kernels read the filter as 16-byte records of 8 input
 * channels at one tap:
 *
 *   wp[co][g][t][j] = w[co][8g + j][t]   (t = ky*KW + kx; 0 when 8g + j >= CI)
 *
 * wp is [CO][CI64/8][KH*KW][8] halves with CI64 = CI rounded up to a multiple
 * of 64 (every stage of the kernels' reduction then lies inside a row),
 * ct_conv2d_filter_prepared_bytes bytes.  ct_conv2d_nchw_fwd reorders the caller's filter into its scratch
 * on every call (one small kernel before the convolution); a caller whose
 * filter does not change between calls (inference) prepares it once with
 * ct_conv2d_prepare_filter (asynchronous on `stream`, wp caller-owned device
 * memory, 16-byte aligned) and calls ct_conv2d_nchw_fwd_prepared, which
 * takes the same arguments as ct_conv2d_nchw_fwd with wp in place of w and
 * gives the same bits, without the reorder.  The prepared entry point uses
 * the cached tile config when its variant reads a prepared filter, else the
 * best such default.  Errors: CT_ERR_INVALID_ARG for dtype CT_F32 (fp32
 * kernels read the caller's layout directly) or a NULL pointer, and those of
 * ct_conv2d_nchw_fwd; CT_ERR_UNSUPPORTED when no tile config of the shape
 * reads a prepared filter. */
long long ct_conv2d_filter_prepared_bytes(int CO, int CI, int KH, int KW, int dtype);
int ct_conv2d_prepare_filter(const void* w, void* wp, int CO, int CI, int KH, int KW, int dtype,
                             void* stream);
int ct_conv2d_nchw_fwd_prepared(const void* x, const void* wp, float* y,
                                int N, int CI, int H, int W, int CO, int KH, int KW,
                                int stride, int pad, int dtype, int epilogue,
                                const float* bias, const float* var, float eps,
                                void* stream);

/* For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The same
 * convolution as ct_conv2d_nchw_fwd (same arguments, config, kernel and
 * bits), but a launch's scratch -- the split partials, their arrival
 * counters and the half-precision kernels' reordered filter -- lives in a
 * fixed array inside the library instead of a per-stream workspace:
 * CT_NOALLOC_SCRATCH_BYTES for partials plus filter and 16384 counters (at
 * most 512 split tiles), held by every device the library runs on until the
 * process ends.  Never calls hipMalloc or hipFree.  Errors: those of
 * ct_conv2d_nchw_fwd, and CT_ERR_UNSUPPORTED when the config needs more
 * scratch than that (the message says how much).  Every call on a device
 * shares that device's array, which keeps the last call's contents: calls
 * that overlap in time on one device (launches on different streams, or
 * concurrent graph replays) race and give wrong results. */
#define CT_NOALLOC_SCRATCH_BYTES (16LL << 20)
int ct_conv2d_nchw_fwd_noalloc(const void* x, const void* w, float* y,
                               int N, int CI, int H, int W, int CO, int KH, int KW,
                               int stride, int pad, int dtype, int epilogue,
                               const float* bias, const float* var, float eps,
                               void* stream);

/* The same with an explicit tile config (cfg->variant, split_k, stages, kc);
 * cfg->index is ignored.  Returns CT_ERR_UNSUPPORTED when the config is not
 * legal for the shape (the check of ct_conv2d_space_entity). */
int ct_conv2d_nchw_fwd_config(const void* x, const void* w, float* y,
                              int N, int CI, int H, int W, int CO, int KH, int KW,
                              int stride, int pad, int dtype, int epilogue,
                              const float* bias, const float* var, float eps,
                              const ct_tile_config* cfg, void* stream);

/* Reference kernel: one lane per output, fp32 fused multiply-add over the
 * taps in definition order.  Slow; used as the on-device check of every
 * tuning candidate.  Same arguments and errors as ct_conv2d_nchw_fwd. */
int ct_conv2d_nchw_direct(const void* x, const void* w, float* y,
                          int N, int CI, int H, int W, int CO, int KH, int KW,
                          int stride, int pad, int dtype, int epilogue,
                          const float* bias, const float* var, float eps,
                          void* stream);

/* ---- matrix product (the 1x1-convolution view) -----------------------
 * The TVM tutorial notes, in its opening, that the same tiled template also
 * serves a matrix product.  Here that is literal:
 *
 *   C[m][n] = sum_{k<K} A[m][k] * B[k][n]      (row-major, all contiguous)
 *
 * is the batch-1 convolution with a 1x1 filter, CO = M, CI = K and H*W = N:
 * w = A as [M][K][1][1], x = B as [1][K][H][W], y = C as [1][M][H][W] (a 1x1
 * filter sees pixels only as a flat index, so every split of N has the same
 * layout; W is the largest divisor of N not above 256).  A and B
 * have dtype `dtype` (CT_F32 / CT_F16 / CT_BF16), C is float.  The epilogue is
 * per row m (bias[m], var[m]).  Tuned configs are cached under that
 * convolution's shape, so ct_conv2d_tune and ct_gemm_tune share records.
 * Errors: CT_ERR_INVALID_ARG for M, N or K <= 0; otherwise those of
 * ct_conv2d_nchw_fwd / ct_conv2d_tune / ct_conv2d_query. */
int ct_gemm_fwd(const void* A, const void* B, float* C, int M, int N, int K,
                int dtype, int epilogue, const float* bias, const float* var,
                float eps, void* stream);
int ct_gemm_tune(int M, int N, int K, int dtype, int epilogue,
                 int max_trials, float min_repeat_ms, void* stream,
                 ct_tile_config* best_out,
                 ct_tune_record* records, int max_records, int* n_records);
int ct_gemm_query(int M, int N, int K, int dtype, int epilogue,
                  ct_tile_config* cfg_out, int* from_cache);

/* ---- general per-channel broadcast -----------------------------------
 * The Paddle PR's Introduction generalises its tactic, by axis fusion, to
 * [1,P,1] => [B,P,B] with the last axis a broadcast axis, and its
 * Performance Impact section names div / exp / rsqrt chains as the work the
 * tactic saves.  Here: out is [outer][P][inner] (inner contiguous) and a
 * program of three chains, each at most CT_CHAIN_MAX_OPS steps applied in
 * order to a value that starts at 0, is evaluated in fp32 per element:
 *
 *   chain 0 -> c0   operands: immediates, arrays a0..a3 at [p]
 *   chain 1 -> c1   operands: the same, and c0
 *   chain 2 -> v    operands: the same, c0, c1, and x[o][p][i]
 *   out[o][p][i] = v, or c0 when chain 2 is empty
 *
 * A step is (op, src, imm): CT_OP_SET v = a; ADD v + a; SUB v - a; MUL v * a;
 * DIV v / a; RSUB a - v; RDIV a / v; EXP exp(v); RSQRT 1/sqrt(v); SQRT
 * sqrt(v) (the unary steps ignore their operand); a is imm, x, c0, c1 or
 * a_k[p] by `src`.  exp and rsqrt run on the hardware units (about 1 ulp
 * each), division and sqrt are correctly rounded, nothing is contracted into
 * a fused multiply-add, and fp16 output is rounded to nearest even. */
#define CT_CHAIN_MAX_OPS 8
#define CT_OP_SET 0
#define CT_OP_ADD 1
#define CT_OP_SUB 2
#define CT_OP_MUL 3
#define CT_OP_DIV 4
#define CT_OP_RSUB 5
#define CT_OP_RDIV 6
#define CT_OP_EXP 7
#define CT_OP_RSQRT 8
#define CT_OP_SQRT 9
#define CT_SRC_IMM 0
#define CT_SRC_X 1
#define CT_SRC_C0 2
#define CT_SRC_C1 3
#define CT_SRC_A0 4  /* CT_SRC_A0 + k for array a_k, k < 4 */

typedef struct ct_chain_op {
    int op;      /* CT_OP_* */
    int src;     /* CT_SRC_* */
    float imm;   /* the operand when src == CT_SRC_IMM */
} ct_chain_op;

typedef struct ct_bcast_program {
    int n_ops[3];                             /* steps in chains 0, 1, 2 */
    ct_chain_op ops[3][CT_CHAIN_MAX_OPS];
} ct_bcast_program;

/* Evaluate `prog` into out ([outer][P][inner], out_dtype CT_F32 or CT_F16).
 * a0..a3: per-channel fp32 arrays of P floats on the device (NULL when no
 * step reads them); x: the producer's fp32 output, same [outer][P][inner]
 * layout (NULL when no step reads it; x == out is allowed for fp32 output,
 * any other overlap is not).  mode: CT_BC_CHANNEL (channel-bound: c0 and c1
 * once per block), CT_BC_FLAT (everything per element) or CT_BC_AUTO, which
 * takes the channel-bound form when inner >= 32, each row is a whole number
 * of 16-byte vectors of out (and x), both are 16-byte aligned and the grid
 * fits, and the flat form otherwise.  Both forms give identical bits.
 * Errors: CT_ERR_INVALID_ARG for a NULL prog or out, outer, P or inner < 1,
 * more than 2^46 elements, a step count outside [0, CT_CHAIN_MAX_OPS], an
 * unknown op or source, a source a chain may not read, a NULL array or x
 * that a step reads, an unknown dtype or mode, or x == out with fp16 output;
 * CT_ERR_UNSUPPORTED for CT_BC_CHANNEL when the channel-bound conditions
 * fail; CT_ERR_HIP on a launch failure.  Asynchronous on `stream`. */
int ct_broadcast_chain(const ct_bcast_program* prog, const float* a0, const float* a1,
                       const float* a2, const float* a3, const float* x, void* out,
                       int out_dtype, long long outer, int P, long long inner, int mode,
                       void* stream);

/* ---- depthwise convolution -------------------------------------------
 * The TVM tutorial names, in its opening, depthwise convolution as another
 * operator its template covers.  Each channel is convolved with its own
 * filter:
 *
 *   y[n][c][oy][ox] = sum_{ky<KH} sum_{kx<KW} xp[n][c][oy*s+ky][ox*s+kx] * w[c][0][ky][kx]
 *
 * x [N][C][H][W] and w [C][1][KH][KW] (contiguous, dtype `dtype`), y
 * [N][C][OH][OW] float with OH, OW as for ct_conv2d_nchw_fwd, xp x padded with
 * `pad` zeros, fp32 accumulation, and the per-channel epilogue (bias[c],
 * var[c]).  No channel reduction, so no tile config: one LDS-tiled kernel.
 * Errors: those of ct_conv2d_nchw_fwd for the arguments, and
 * CT_ERR_UNSUPPORTED for more than 256 taps (KH*KW), N*C or H*W above 2^31 - 1, or
 * an output row too wide for one workgroup's LDS window (about
 * ((3*stride + KH) * ((OW-1)*stride + KW)) > 40960); CT_ERR_HIP on a launch
 * failure.  Asynchronous on `stream`. */
int ct_conv2d_nchw_depthwise(const void* x, const void* w, float* y,
                             int N, int C, int H, int W, int KH, int KW,
                             int stride, int pad, int dtype, int epilogue,
                             const float* bias, const float* var, float eps,
                             void* stream);

/* ---- transformer-block rows ------------------------------------------
 * The dense path of a transformer block when serving: rows are normalised,
 * brought to 8 bits, and multiplied with weights.
 *
 * Rows.  Every matrix here is a run of rows with contiguous elements; ld* is
 * the distance between rows in elements (>= the row's length, at most 8 MiB
 * where a product reads more than one row).  Pointers are aligned to their
 * element; rows that are not multiples of 16 bytes, or start off them, are read
 * at full width all the same, but the loads that write LDS directly need that
 * alignment: products of more than 32 such rows may take up to twice as long.
 * M = 0 rows (an empty batch) is a legal call that does nothing.
 *
 * 8-bit rows are e4m3 (OCP: largest value 448, NaN, no infinity) with one
 * fp32 scale a row: the row stands for scale * q.  From a row of values v:
 *   a = max(max_k |v[k]|, 2^-100),  scale = a / 448,  q[k] = rne_e4m3(v[k] / scale)
 * with scale and the quotient in fp32, each rounded to nearest, so that q is
 * the same bit for bit on any machine that follows the formula.
 * A row of zeros has scale 2^-100 / 448 and q = 0; a row with a NaN a NaN
 * scale; a row with an infinity (and no NaN) an infinite scale and q = 0 at
 * its finite places, NaN at the others.
 *
 * None of these calls allocates, synchronises or needs the device to have
 * been set up: all may be captured as a stream's first work.  They take no
 * workspace from the library. */

/* h = x + residual (fp32), y = h * rsqrt(mean_k h^2 + eps) * gain.
 * x, residual and h are [M][D] of `dtype` (CT_F32, CT_F16 or CT_BF16); gain
 * is float [D] (NULL: ones).  residual may be NULL; then h is not written and
 * must be NULL too.  With a residual, h (the new residual stream, rounded to
 * dtype) may be NULL if it is not wanted; y is made from the unrounded sum.
 * y [M][D] is of out_dtype: CT_F32, CT_F16 or CT_BF16 (scale is NULL), or
 * CT_E4M3 with scale float [M]: the 8-bit rows of y's fp32 values.  Sums are
 * fp32; a row of zeros with eps = 0 is NaN, and one whose squares pass the
 * range of fp32 zeros, as the formula says in fp32.  h and y may each be
 * exactly x or residual (same pointer, stride and type), not the same one; no
 * other overlap.  Errors: CT_ERR_INVALID_ARG for M < 0, D < 1, a NULL or misaligned pointer,
 * a stride below D, an unknown dtype, h without residual, scale missing (or
 * given without CT_E4M3), h or y at the address of an input with another
 * stride or type, or eps negative or not finite; CT_ERR_HIP on a launch
 * failure.  Asynchronous on `stream`. */
int ct_rmsnorm_fwd(const void* x, long long ldx, const void* residual, long long ldr,
                   const float* gain, void* h, long long ldh, void* y, long long ldy,
                   float* scale, int M, int D, int dtype, int out_dtype, float eps,
                   void* stream);

/* Rows x [M][D] (CT_F32, CT_F16 or CT_BF16) to e4m3 q [M][D] with scale [M],
 * as above: a layer's weights once, and activations that no norm produces.
 * q must not overlap x.  Errors as for ct_rmsnorm_fwd. */
int ct_quantize_rows(const void* x, long long ldx, void* q, long long ldq, float* scale,
                     int M, int D, int dtype, void* stream);

/* Each in fp32 to a few units in the last place of its value, the negative
 * tails included (relative errors grow as z^2 2^-23 with gelu and |u| 2^-21 with
 * gelu_tanh, u its exponent); 16-bit results to 2^-17 before their rounding. */
enum ct_activation {
    CT_ACT_NONE = 0,
    CT_ACT_RELU = 1,
    CT_ACT_GELU = 2,       /* z (1 + erf(z / sqrt 2)) / 2                     */
    CT_ACT_GELU_TANH = 3,  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    CT_ACT_SILU = 4        /* z / (1 + exp(-z))                               */
};

/* What a product does with its sums z, in this order:
 *   y = act(z + bias[n]) * gate[m][n] + residual[m][n]
 * gate and residual are [M][N] of y's type; NULL members are left out.  y may
 * be exactly gate or residual (same pointer and stride); no other overlap.
 * All of it is fp32, with one rounding, to y's type. */
typedef struct ct_linear_epilogue {
    int act;              /* ct_activation */
    const float* bias;    /* [N] */
    const void* gate;
    long long ldg;
    const void* residual;
    long long ldr;
} ct_linear_epilogue;

/* Linear layer y = epilogue(x w^T):
 *   z[m][n] = sum_{k<K} x[m][k] * w[n][k]
 * x [M][K] and w [N][K] of `dtype` (CT_F32, CT_F16 or CT_BF16), y [M][N] of
 * out_dtype (the same three), sums in fp32.  epi may be NULL (y = z).
 * Results that do not fill the device may have their sum split over k: the
 * parts are fp32 and joined in order, so a result depends on the sizes and
 * the dtypes alone (with rows that are not 16-byte aligned, on that too), and
 * repeats bit for bit.  Products of rows whose length is no multiple of 16
 * bytes may work on a copy of x and w.  Either needs `workspace`, of at least
 * ct_linear_workspace_bytes bytes (often 0; then it may be NULL), 16-byte
 * aligned, written by the call and free again when its work on the stream is
 * done: calls that may overlap, and graphs that may be replayed at the same
 * time, need one each.
 * Errors: CT_ERR_INVALID_ARG for M < 0, N or K < 1, a NULL or misaligned
 * pointer, a stride below the row's length, an unknown dtype or activation,
 * y equal to x or w, or to gate or residual with another stride, or a
 * workspace that is too small; CT_ERR_UNSUPPORTED for
 * M, N or a row's bytes above 2^30, x or w rows more than 8 MiB apart, or
 * results that one launch cannot cover (2^23 tiles of 64 x 64 to 256 x 256,
 * chosen by the sizes); CT_ERR_HIP on a launch failure.  Asynchronous on `stream`. */
int ct_linear_fwd(const void* x, long long ldx, const void* w, long long ldw,
                  void* y, long long ldy, int M, int N, int K, int dtype, int out_dtype,
                  const ct_linear_epilogue* epi, void* workspace, long long workspace_bytes,
                  void* stream);

/* The same on 8-bit rows: x [M][K] and w [N][K] are CT_E4M3 with row scales
 * xs [M] and ws [N]:
 *   z[m][n] = xs[m] * ws[n] * sum_{k<K} x[m][k] * w[n][k]
 * With CT_F32 output, and for up to 32 rows of x, the operands are widened to
 * fp16, exactly, and the sums are fp32.  Otherwise (16-bit results of more
 * rows) the 8-bit matrix instruction is used, which aligns each 8 neighbouring
 * products to the largest of them and cuts what lies 2^-13 below it: about
 * 1.5e-5 of a sum's size on normally distributed rows, 1/130 of the
 * rounding to bf16 and 1/16 of that to fp16. */
int ct_linear_q8_fwd(const void* x, long long ldx, const float* xs,
                     const void* w, long long ldw, const float* ws,
                     void* y, long long ldy, int M, int N, int K, int out_dtype,
                     const ct_linear_epilogue* epi, void* workspace, long long workspace_bytes,
                     void* stream);

/* Bytes of workspace a product of these sizes needs (dtype: that of x and w,
 * CT_E4M3 for ct_linear_q8_fwd); < 0 (a status) for sizes or a dtype the
 * product refuses.  Host only. */
long long ct_linear_workspace_bytes(int M, int N, int K, int dtype);

/* ---- key-value cache and attention -----------------------------------
 * What a transformer block does between its projections when serving: new
 * tokens' keys and values go into a cache, and the tokens attend over it.
 *
 * The cache is a pool of pages, each with `page` places for rows of `dim`
 * elements in every head.  A sequence's place i lies at place i % page of the page
 * that its row of `table` names for i / page; without a table, sequence b has
 * page b and no other.  Any order of the axes will do: ld_* are the distances,
 * in elements, between pages, heads and places (the same in k and v), lds_* those
 * of the scales.  Rows are contiguous, 16-byte aligned, of a whole multiple
 * of 16 elements up to 256.  CT_F16 and CT_BF16 caches hold values; CT_E4M3 ones
 * codes with a scale a place and head, made from a row of values v by
 *   a = max(largest finite |v|, 2^-100)
 *   s = the least power of two with a <= 448 s,  code = rne_e4m3(v / s)
 * and standing for s * code.  What is not finite becomes the NaN code. */
typedef struct ct_kv_cache {
    void* k;         /* [pages][heads][page][dim] of dtype */
    void* v;
    float* k_scale;  /* [pages][heads][page], CT_E4M3 only (NULL otherwise); */
    float* v_scale;  /* attention takes their sign and fraction for 0        */
    int dtype, pages, heads, page, dim;
    long long ld_page, ld_head, ld_token;
    long long lds_page, lds_head, lds_token;
} ct_kv_cache;

/* The tokens of a call: rows starts[b] to starts[b + 1] - 1 are the new tokens of
 * sequence b; without starts every sequence has tokens / sequences of them.
 * lens[b] counts the places in use WITH the new tokens, which are the last:
 * token i of n has place lens[b] - n + i.  lens, starts and table are read on the
 * device when the call runs, so a captured graph follows them.  Tokens before
 * starts[0] and from starts[sequences] on belong to nobody: their rows are
 * not used and not written.  Contents that do not fit are the caller's fault, but
 * lead nowhere else: lens are taken as 0 to 2^30, starts as 0 to tokens (an end
 * before its start as no tokens; what rows of two sequences become is not said),
 * places past the table's columns as not there; what a page number outside of
 * the pool does is said at each call. */
typedef struct ct_kv_batch {
    int tokens, sequences;
    const int* lens;    /* [sequences] */
    const int* starts;  /* [sequences + 1], or NULL */
    const int* table;   /* [sequences][width], rows ldt apart, or NULL */
    long long ldt;
    int width;
} ct_kv_batch;

/* New tokens' k and v, [tokens][heads][dim] of `dtype` (CT_F32, CT_F16 or
 * CT_BF16), into their places: rounded to a 16-bit cache's type, or to e4m3 as
 * above.  *_token and *_head are distances in elements (slices of a fused
 * projection's rows will do).  A token whose place or page does not exist is
 * left out.  Two tokens of a call must not have one place, unless their rows are
 * equal: no page may be two sequences' where they write other rows.  Neither k nor v
 * may overlap the cache.
 * tokens = 0 is a legal call that does nothing.  None of the calls of this section
 * allocates, synchronises or needs the device to have been set up: all may be
 * captured as a stream's first work.
 * Errors: CT_ERR_INVALID_ARG for NULL or misaligned pointers, counts that are not
 * positive, strides that are negative or let rows of the cache (or of k and v, when
 * they are written) overlap, an unknown dtype, scales missing (or given without
 * CT_E4M3), more sequences than pages without a table, tokens that the
 * sequences do not divide without starts, or one place for the cache's k and v or
 * for their scales; CT_ERR_UNSUPPORTED for a dim that is no multiple of 16 or above
 * 256, 2^26 rows (tokens x heads) or more, or more than 2^30 places a sequence,
 * 2^24 sequences (2^16 with starts) or 2^16 heads; CT_ERR_HIP on a launch failure.
 * Asynchronous on `stream`. */
int ct_kv_write(const ct_kv_cache* cache, const ct_kv_batch* batch, const void* k,
                long long k_token, long long k_head, const void* v, long long v_token,
                long long v_head, int dtype, void* stream);

/* The last tokens of every sequence back out of the cache, as values rounded
 * to `dtype`: what ct_kv_write would take.  A token whose place or page does not
 * exist gives zeros.  Errors as for ct_kv_write. */
int ct_kv_read(const ct_kv_cache* cache, const ct_kv_batch* batch, void* k, long long k_token,
               long long k_head, void* v, long long v_token, long long v_head, int dtype,
               void* stream);

/* Which places a token sees.  Without a tree, those up to its own, of which with
 * a window only the last `window` (its own among them) and the first `sinks`.
 * With a tree the new tokens of a sequence are drafted nodes: node i sees the
 * context (the places before the new tokens) and node j if bit j % 64 of word
 * j / 64 of its row is set, its own bit among them if it is to see itself; bits past
 * the sequence's nodes and nodes past the words count as not set.  For window
 * and sinks, the nodes that i sees are taken in order to lie behind the context, one
 * place each, and i's place is the last of them. */
typedef struct ct_kv_mask {
    int window;             /* 0: none */
    int sinks;              /* with a window only */
    const long long* tree;  /* [tokens][words], or NULL */
    int words;              /* 0 without a tree */
} ct_kv_mask;

/* Attention of the new tokens over the cache, which holds them already:
 *   y = sum_j exp(scale q . k_j) v_j / sum_j exp(scale q . k_j)
 * over the places j that a token sees; zeros where it sees none, NaN where all that
 * it sees have a score of -infinity (0 / 0).  q and y are
 * [tokens][heads][dim] of `dtype` (CT_F16 or CT_BF16, that of a 16-bit cache);
 * `heads` is a multiple of the cache's, whose head h the heads h * heads / cache
 * heads and following share.  mask may be NULL (causal).  max_len: the longest
 * of lens if the caller knows (0 otherwise); it only guides how the work is divided.
 * Sums, maximum and weights are fp32; the weights are rounded to `dtype` for the
 * product with v.  With CT_F16, 8-bit rows must stay within the range of fp16;
 * what passes it counts as infinite.  What lies in places that a token does not see has no part in its
 * result, whatever it is; NaN and infinities that it sees do, those of v (in 16 bits)
 * whatever their weight.  A page number outside of the pool is read as page 0.
 * Few tokens have their keys split over workgroups, whose sums are joined in
 * order: a result depends on the sizes and the batch's contents and repeats
 * bit for bit.  That needs `workspace`, of at least
 * ct_kv_attention_workspace_bytes bytes for the same sizes (often 0; then it may
 * be NULL), 16-byte aligned and free again when the call's work on the stream is
 * done: calls that may overlap, and graphs that may be replayed at the same time,
 * need one each.  y must not overlap q or the cache.
 * Errors: those of ct_kv_write, and CT_ERR_INVALID_ARG for a scale that is not
 * positive and finite, heads that are no multiple of the cache's, a negative
 * window, sinks without a window, words without a tree (or the reverse), another
 * type than that of a 16-bit cache, or a workspace that is too small;
 * CT_ERR_UNSUPPORTED for 2^26 rows of q (tokens x heads) or more, or more than
 * 2^23 workgroups.  Asynchronous on `stream`. */
int ct_kv_attention_fwd(const ct_kv_cache* cache, const ct_kv_batch* batch, const ct_kv_mask* mask,
                        const void* q, long long q_token, long long q_head, void* y,
                        long long y_token, long long y_head, int heads, int dtype, float scale,
                        long long max_len, void* workspace, long long workspace_bytes,
                        void* stream);

/* Bytes of workspace that a call of these sizes over a cache of cache_dtype
 * needs (window 0: none); < 0 (a status) for what it refuses.  Host only. */
long long ct_kv_attention_workspace_bytes(int tokens, int sequences, int heads, int kv_heads,
                                          int dim, long long max_len, int window, int sinks,
                                          int cache_dtype);

/* ---- tile-config search ----------------------------------------------
 * The space of a shape follows the TVM tutorial's template (Step 1): ordered
 * knobs, each a split (all ordered factorizations of an extent, the
 * "policy=all" of the gist's ConfigSpace dump) or an option list, and a flat
 * index that is mixed radix over the knobs with the first knob least
 * significant.  Knobs here, in order:
 *   tile_ci = split(CI, 3) -> [split_k, stages, kc]
 *   variant = option(ids of the compiled variants for the dtype)
 */

/* Number of points in the space of this shape (legal or not); < 0 on error. */
long long ct_conv2d_space_size(int N, int CI, int H, int W, int CO, int KH, int KW,
                               int stride, int pad, int dtype, int epilogue);

/* Decode flat `index` into *cfg_out and report in *legal (1/0) whether the
 * point passes the legality check (LDS bytes within 160 KiB, workgroup size
 * within 1024, channels per stage within the variant's limit, ...).  The
 * check never launches anything.  CT_ERR_INVALID_ARG for an index outside
 * [0, size). */
int ct_conv2d_space_entity(int N, int CI, int H, int W, int CO, int KH, int KW,
                           int stride, int pad, int dtype, int epilogue,
                           long long index, ct_tile_config* cfg_out, int* legal);

/* Enumerate the legal points, time up to `max_trials` of them on `stream`
 * (0 = all legal points), keep the fastest whose output matches the direct
 * reference kernel, store it in the cache and in *best_out.  Timing follows
 * the TVM tutorial's runner (Step 2): a warm-up, then `repeat` (3)
 * measurements each of at least `min_repeat_ms` milliseconds of back-to-back
 * launches, and a per-trial limit of 4 s (CT_TUNE_TIMEOUT_S overrides it),
 * checked while the launches run: a trial past it records error 6 and issues
 * no more launches.  Scratch inputs are allocated and filled on the device
 * by the library.  `records` (may be NULL) receives up to `max_records` trial
 * records and *n_records their count.
 * Tuning log (the tutorial's log_to_file): when the environment variable
 * CT_CACHE_PATH names a file, every trial record is appended to it as one
 * JSON line when the trial ends (error_no 1/4/6 included), and a search of a
 * shape first reads the file: points already logged for the shape are not
 * measured again (resume), and their logged results take part in choosing
 * the winner; `records` lists only the trials measured by this call.
 * Synchronises the stream; may take seconds.  Returns CT_ERR_TUNE_FAILED if
 * no candidate ran correctly, CT_ERR_IO if the log cannot be appended. */
int ct_conv2d_tune(int N, int CI, int H, int W, int CO, int KH, int KW,
                   int stride, int pad, int dtype, int epilogue,
                   int max_trials, float min_repeat_ms, void* stream,
                   ct_tile_config* best_out,
                   ct_tune_record* records, int max_records, int* n_records);

/* The flat indices ct_conv2d_tune would time for this shape, in order (legal
 * points by the analytic time estimate, then the illegal ones), leaving out
 * the points already recorded in the CT_CACHE_PATH log (resume), at most
 * `max_trials` (0 = all).  Writes up to `max_out` of them to order_out and
 * their full count to *n_out.  Host-only: launches nothing. */
int ct_conv2d_tune_order(int N, int CI, int H, int W, int CO, int KH, int KW,
                         int stride, int pad, int dtype, int epilogue, int max_trials,
                         long long* order_out, int max_out, int* n_out);

/* Guided search for spaces too large to time exhaustively (the role of the
 * TVM tutorial's cost-model tuner, XGBTuner, in Step 2).  Times at most
 * `max_trials` legal configs (0 = all), `batch` at a time: the first batch
 * drawn uniformly (SplitMix64 on `seed`), each later one the lowest
 * predictions of a ridge regression of log(time) on 11 features of a config
 * (ct_ridge_fit, lambda 1e-3, refitted after every batch) plus max(1,
 * batch/4) uniform draws among the untimed configs.  Trials, records, the
 * cache entry and errors as ct_conv2d_tune; CT_ERR_INVALID_ARG also for
 * batch < 1.  The CT_CACHE_PATH log is written and resumed from as for
 * ct_conv2d_tune. */
int ct_conv2d_tune_guided(int N, int CI, int H, int W, int CO, int KH, int KW,
                          int stride, int pad, int dtype, int epilogue,
                          int max_trials, int batch, unsigned long long seed,
                          float min_repeat_ms, void* stream,
                          ct_tile_config* best_out,
                          ct_tune_record* records, int max_records, int* n_records);

/* The guided search's parts on host data (no device): ct_ridge_fit solves
 * min |X w - y|^2 + lambda |w|^2 (X row-major n x d, 1 <= d <= 64) by a
 * Cholesky factorisation, CT_ERR_INVALID_ARG when X^T X + lambda I is
 * singular; ct_guided_search_table runs the search of ct_conv2d_tune_guided
 * over n points with features feats (n x d) whose costs are given (cost <= 0
 * or not finite = a failed trial, left out of the fit), with n_explore
 * draws a batch after the first, and writes the order in which it would time
 * them (at most max_trials) to order_out, their count to *n_order. */
int ct_ridge_fit(const double* X, const double* y, int n, int d, double lambda, double* w);
int ct_guided_search_table(const double* feats, const double* costs, int n, int d,
                           int max_trials, int batch, int n_explore,
                           unsigned long long seed, double lambda,
                           int* order_out, int* n_order);

/* The config ct_conv2d_nchw_fwd would use for this shape; *from_cache = 1
 * when it came from a tuning record, 0 when it is the built-in default.  The
 * TVM tutorial's closing step looks the tuned config of a workload up in its
 * log this way (apply_history_best, then query of the best record) before it
 * builds the kernel.  Errors: those of ct_conv2d_space_size, CT_ERR_INVALID_ARG
 * for a NULL cfg_out. */
int ct_conv2d_query(int N, int CI, int H, int W, int CO, int KH, int KW,
                    int stride, int pad, int dtype, int epilogue,
                    ct_tile_config* cfg_out, int* from_cache);

/* Compiled variants. */
int ct_variant_count(void);
int ct_variant_info(int variant, ct_variant_desc* out);

/* Ordered factorizations of n into k factors ("policy=all" split): count, and
 * the i-th one written to out[0..k-1] in the space's order (ascending by
 * (x_k, ..., x_2)).  Count < 0 for n <= 0 or k outside [1, 8]. */
long long ct_split_count(long long n, int k);
int ct_split_entity(long long n, int k, long long i, long long* out);

/* ---- the tutorial template's own space ---------------------------------
 * The conv2d_nchw schedule of the TVM tutorial "Tuning High Performance
 * Convolution on NVIDIA GPUs" (Step 1) has eight knobs, in declaration order:
 *   tile_f = split(CO, 4), tile_y = split(OH, 4), tile_x = split(OW, 4),
 *   tile_rc = split(CI, 3), tile_ry = split(KH, 3), tile_rx = split(KW, 3)
 *   (each in ct_split_entity's order), auto_unroll_max_step in {0, 512,
 *   1500}, unroll_explicit in {0, 1};
 * the flat index is mixed radix over them, tile_f least significant: the
 * space the gist's run prints for the last ResNet layer (10,454,400 points)
 * and the index beside each record of its tuning log.  This library does not
 * build that schedule (its kernels are the MFMA variants above); the space
 * and the check below reproduce which of the tutorial's candidates its run
 * rejected before timing them (error_no 1, "invalid gpu kernel"). */
typedef struct {
    int tile_f[4], tile_y[4], tile_x[4];
    int tile_rc[3], tile_ry[3], tile_rx[3];
    int auto_unroll_max_step;
    int unroll_explicit;
} ct_tvm_config;

/* Points of the template's space for this shape; < 0 on a bad shape. */
long long ct_tvm_space_size(int N, int CI, int H, int W, int CO, int KH, int KW,
                            int stride, int pad);
/* Decode flat `index` into *out.  CT_ERR_INVALID_ARG for a bad shape, a NULL
 * out or an index outside [0, size). */
int ct_tvm_space_entity(int N, int CI, int H, int W, int CO, int KH, int KW,
                        int stride, int pad, long long index, ct_tvm_config* out);
/* The flat index of *cfg in the space (the inverse of ct_tvm_space_entity);
 * CT_ERR_INVALID_ARG for a bad shape or a NULL cfg, -1 (with no error
 * recorded) when *cfg is not a point of the space. */
long long ct_tvm_space_index(int N, int CI, int H, int W, int CO, int KH, int KW,
                             int stride, int pad, const ct_tvm_config* cfg);

#define CT_TVM_LIMITS_PAGE 0    /* the tutorial run's GPU: 48 KiB shared memory, 1024 threads per block */
#define CT_TVM_LIMITS_GFX950 1  /* this device: 160 KiB LDS, 1024 threads per workgroup */

/* The tutorial schedule's block resources under *cfg, without building it.
 * The schedule stages the padded input (AA) and the filter (WW) in shared
 * memory at the outer rx loop, inside the outer rc, ry and rx loops, so each
 * holds one block's output tile against the middle x inner reduction
 * extents, in fp32:
 *   AA = RC_s * ((Y_b - 1) * stride + RY_s) * ((X_b - 1) * stride + RX_s)
 *   WW = F_b * RC_s * RY_s * RX_s
 * with F_b = tile_f[1] * tile_f[2] * tile_f[3] (vthread, thread and inner
 * factors; Y_b and X_b alike), RC_s = tile_rc[1] * tile_rc[2] and, as the
 * schedule is printed, the ry axis split by tile_rx's factors and rx by
 * tile_ry's: RY_s = tile_rx[1] * tile_rx[2], RX_s = tile_ry[1] * tile_ry[2].
 * Threads per block = tile_f[2] * tile_y[2] * tile_x[2].  Writes
 * *shared_bytes = 4 * (AA + WW) and *threads (either may be NULL); returns
 * 1 when both fit the limits of `mode`, 0 when not, CT_ERR_INVALID_ARG for a
 * NULL cfg, a factor < 1, stride < 1 or an unknown mode. */
int ct_tvm_config_check(const ct_tvm_config* cfg, int stride, int mode,
                        long long* shared_bytes, int* threads);

/* ---- per-channel broadcast --------------------------------------------
 * out[n][c][h][w] = exp(var[c])  (Paddle PR, Introduction and Example:
 * [1,C,1,1] => [N,C,H,W]).  var: C floats on the device; out: N*C*H*W
 * elements of out_dtype (CT_F32 or CT_F16, rounded to nearest even).  The
 * channel-bound form needs H*W % 32 == 0 and a 16-byte aligned `out`;
 * CT_BC_AUTO falls back to the flat form otherwise, CT_BC_CHANNEL returns
 * CT_ERR_UNSUPPORTED.  Results are identical in every mode. */
int ct_broadcast_nchw(const float* var, void* out, int N, int C, int H, int W,
                      int out_dtype, int op, int mode, void* stream);

/* ---- cache, lifetime, errors ----------------------------------------- */

/* Append-only JSON-lines tuning log: the TVM tutorial's Step 2 writes every
 * measure record to a log file (log_to_file), and its closing step picks the
 * best record per workload from that log (apply_history_best).  Here a record
 * is one line with the shape key, the config, its costs, error_no and a
 * timestamp.  load merges the file into memory, keeping per shape the fastest
 * successful record (lines that do not parse, name an unknown variant or are
 * not legal for their shape are skipped); save appends every in-memory
 * winner to the file.  CT_ERR_INVALID_ARG for a NULL path, CT_ERR_IO when the
 * file cannot be opened or written.  clear empties the in-memory cache; size
 * is its number of shapes. */
int ct_cache_load(const char* path);
int ct_cache_save(const char* path);
int ct_cache_clear(void);
int ct_cache_size(void);

/* Free the library's device workspaces, and every buffer a workspace
 * outgrew (all devices, all streams).  Synchronises each stream that owns a
 * workspace first.  No graph that captured a launch may be replayed after
 * this. */
int ct_release(void);

/* Set up `device` for launches: the zero page's device address and the
 * workgroup-placement probe of the XCD-local variants (which launches and
 * synchronises a private stream).  Idempotent.  Call it before capturing
 * the first launch on a device into a HIP graph.  CT_ERR_INVALID_ARG for a
 * device that does not exist, CT_ERR_HIP when a HIP call fails. */
int ct_init(int device);

/* How many times ct_conv2d_nchw_fwd resolved a launch plan (a first call for
 * a (device, shape), or the first after the config cache changed); every
 * other call reused a plan.  For tests and diagnostics. */
long long ct_plan_misses(void);

const char* ct_status_string(int status);
const char* ct_last_error(void);
const char* ct_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CONVTILE_H */
