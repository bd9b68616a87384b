/*
 * gemm_epilog.h - C ABI of the fused GEMM + epilogue library for AMD Instinct MI355X (gfx950).
 *
 * One call computes D = epilogue(A . B) in a single HIP kernel: the bias add, the
 * activation, the ReLU mask or the masked bias gradient are applied to the fp32
 * accumulators before the only store of D.
 *
 * Sources (web pages describing the method):
 *  [P1] "Fusing bias addition via the nvmath-python epilog mechanism: parameter
 *       configuration and engineering practice guide" (blog.hotdry.top).
 *  [P2] "nvmath-python wraps cuBLASLt: low-overhead matmul and bias-fusion primitives
 *       for PyTorch" (blog.hotdry.top).
 *  [P3] "Fusing epilogs with matrix multiplication using nvmath-python" (itzkxy.com).
 *  [P4] "Dissecting nvmath-python: a seamless bridge between NumPy and cuBLASLt"
 *       (blog.hotdry.top).
 *  [P5] "Operator fusion in AI inference compilers: implementation and trade-offs"
 *       (mqxn.cn).
 *
 * Lifecycle ([P4] paragraph on the plan-execute-free lifecycle; [P2] body, plan and
 * execute steps; [P1] paragraph 4, second item): gemm_epilog_plan validates the
 * problem, picks a kernel configuration and allocates the plan's workspace once;
 * gemm_epilog_execute only enqueues work and may be called any number of times;
 * gemm_epilog_free releases the plan.
 *
 * Layouts. Every matrix is dense row-major with no leading-dimension padding:
 *   A (m, k), B (k, n), D (m, n). bias and bgrad hold m values, one per row of D:
 *   the bias has shape (m,) or (m, 1) and is added to every column ([P1] paragraph 2;
 *   [P2] body, initialisation example).
 *   The ReLU mask (aux) is uint32 words [ceil(m/32)][n], row-major: bit (i % 32) of
 *   word (i / 32, j) is 1 exactly when the pre-activation at (i, j) is > 0; bits of
 *   rows i >= m are 0. The pages keep this mask opaque ([P1] paragraph 3, [P3]
 *   section on the fused forward epilogs); this layout is the library's own.
 *
 * Arithmetic. Products are accumulated in fp32 whatever the storage type ([P2] body,
 * plan step: FP32 accumulator with FP16 inputs/outputs; [P5] section 4.3). Every
 * narrowing conversion rounds to nearest even. The order of the k reduction is the
 * kernel's own; results agree with a plain ascending-k fp32 sum to rounding.
 *
 * Ownership and threading. The caller owns every tensor pointer and the stream; the
 * plan owns only its workspace. A plan may be used from one stream at a time (its
 * workspace is shared between executes). All pointers passed to execute are device
 * pointers of the device that was current at plan time.
 *
 * Errors. Every argument check runs on the host before any HIP call, so invalid
 * arguments never launch a kernel. Faults inside a kernel surface at the caller's
 * next synchronisation, as for any asynchronous HIP work ([P1] paragraph 4, third
 * item: execute is asynchronous and the caller synchronises the stream).
 */
#ifndef GEMM_EPILOG_H_
#define GEMM_EPILOG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ge_plan* ge_handle_t; /* opaque; owned by the library */

/* Storage types. */
typedef enum { GE_F32 = 0, GE_F16 = 1, GE_BF16 = 2 } ge_dtype_t;

/* ab: type of A and B; d: type of D (must equal ab); vec: type of bias / bgrad
 * (equal to d, or GE_F32) - [P1] paragraph 4, first item: with fp16 A and B the
 * bias is fp16 or fp32. Accumulation is always fp32. */
typedef struct {
  ge_dtype_t ab;
  ge_dtype_t d;
  ge_dtype_t vec;
} ge_dtypes_t;

typedef enum {
  /* D = A.B (no epilogue); also the first kernel of the unfused chain. */
  GE_EPILOG_NONE = 0,
  /* D = max(A.B + bias, 0)  ([P2] body, plan step; [P3] section on the fused forward epilogs). */
  GE_EPILOG_RELU_BIAS = 1,
  /* D = gelu(A.B + bias), tanh form 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3)))
   * ([P1] final paragraph and [P2] "other epilogs" paragraph name GELU_BIAS). */
  GE_EPILOG_GELU_BIAS = 2,
  /* RELU_BIAS that also writes the packed ReLU mask to aux ([P1] paragraph 3; [P3]
   * section on the fused forward epilogs). */
  GE_EPILOG_RELU_AUX_BIAS = 3,
  /* Backward: D = mask ? A.B : 0 using the mask in aux, and bgrad[i] = sum over j of
   * that masked fp32 product, before D's rounding ([P3] section "The DRELU_BGRAD path
   * in the backward pass"). No bias input. */
  GE_EPILOG_DRELU_BGRAD = 4,
  /* D = A.B + bias ([P1] paragraph 2). */
  GE_EPILOG_BIAS = 5,
  /* Measurement baseline: three kernels GEMM -> T1, T1 + bias -> T2, max(T2, 0) -> D,
   * with T1 and T2 in D's type held in the plan's workspace ([P5] section 2.2 diagram
   * of the chain before fusion). */
  GE_EPILOG_RELU_BIAS_UNFUSED = 100,
  /* Measurement baseline of the backward: the three steps DRELU_BGRAD does in one call
   * ([P3] section "The DRELU_BGRAD path in the backward pass"), each as its own kernel
   * as in [P5] section 2.2: GEMM -> T1 in D's type (held in the plan's workspace);
   * D = T1 where the forward activation in aux is > 0, else +0; bgrad[i] = the sum of
   * row i of the stored D. The unfused forward writes no bit mask, so aux holds its ReLU
   * output. No bias input. */
  GE_EPILOG_DRELU_BGRAD_UNFUSED = 101
} ge_epilog_t;

typedef enum {
  GE_OK = 0,
  GE_ERR_INVALID_VALUE = 1, /* m, n or k out of range; unknown enum value */
  GE_ERR_NOT_SUPPORTED = 2, /* dtype combination or shape outside the supported set */
  GE_ERR_NULL_POINTER = 3,  /* a pointer the epilogue needs is NULL */
  GE_ERR_MISALIGNED = 4,    /* a pointer violates its alignment rule */
  GE_ERR_ALLOC = 5,         /* host or device allocation failed in plan */
  GE_ERR_HIP = 6,           /* a HIP runtime call failed (launch, device query) */
  GE_ERR_SCRATCH = 7        /* gemm_epilog_execute_noalloc: the problem needs more workspace
                               than the static scratch holds */
} ge_status_t;

/*
 * gemm_epilog_plan - validate a problem and build its plan.
 *   m, n, k : problem sizes, 1 <= m <= 2^31 - 1, 1 <= n, k <= 2^20.
 *             n and k must be multiples of 8 for fp16/bf16 and of 4 for fp32
 *             (16-byte rows); otherwise GE_ERR_NOT_SUPPORTED. m is arbitrary.
 *   dt      : storage types (see ge_dtypes_t).
 *   ep      : epilogue.
 *   out     : receives the handle; untouched on error.
 * Allocates the workspace on the current device: the per-tile bias-gradient
 * partial sums for DRELU_BGRAD, T1 and T2 for RELU_BIAS_UNFUSED, T1 for
 * DRELU_BGRAD_UNFUSED, nothing otherwise.
 * Environment (tuning experiments): GE_TILE=S|M|L|LH|LM|LM4|LMD|L3|LW forces a tile configuration;
 * GE_GROUP_M=g (1..1024) sets how many m-tiles share one group of the tile order;
 * GE_STREAMK=0 keeps a sparse last round of tiles whole instead of splitting its k loop;
 * GE_SK_RUN=r sets the k-tiles per split run (at least one run per compute unit);
 * GE_PERSIST=0 launches one workgroup per tile instead of the persistent kernel;
 * GE_LOG=1 prints each plan's configuration and workspace size to stderr.
 */
ge_status_t gemm_epilog_plan(int64_t m, int64_t n, int64_t k, ge_dtypes_t dt, ge_epilog_t ep,
                             ge_handle_t* out);

/* Storage order of an operand ([P3] section "The DRELU_BGRAD path in the backward
 * pass", second paragraph: the backward's weight transpose and gradient layout must
 * match the matmul call; its FAQ: the rest of the backward pass, such as the weight
 * gradient, is outside DRELU_BGRAD). The product always uses A as (m, k) and B as
 * (k, n); GE_OP_T says the operand is passed as its transpose:
 *   op_a = GE_OP_T: the A pointer holds a row-major (k, m) matrix At, A[i][kk] = At[kk][i]
 *                   (e.g. dX = W^T . dY with W passed as stored);
 *   op_b = GE_OP_T: the B pointer holds a row-major (n, k) matrix Bt, B[kk][j] = Bt[j][kk]
 *                   (e.g. dW = dZ . X^T with X passed as stored). */
typedef enum { GE_OP_N = 0, GE_OP_T = 1 } ge_op_t;

/*
 * gemm_epilog_plan_ex - gemm_epilog_plan with the storage order of A and B.
 *   op_a, op_b : GE_OP_N or GE_OP_T (anything else: GE_ERR_INVALID_VALUE).
 * GE_OP_T needs fp16 or bf16 operands (fp32: GE_ERR_NOT_SUPPORTED). With op_a =
 * GE_OP_T, m follows the rules of n: a multiple of 8 and at most 2^20, else
 * GE_ERR_NOT_SUPPORTED. Every other argument, rule and error is that of
 * gemm_epilog_plan, which equals gemm_epilog_plan_ex(..., GE_OP_N, GE_OP_N, out).
 * Plans with a transposed operand run the 256 x 256 tile (the persistent kernel
 * included) and the 128 x 128 tiles with eight waves (LM, and LMD for a small grid
 * with 24 or more k-tiles), but never split their k loop; the 192 x 256, 128 x 256
 * and four-wave 128 x 128 tiles take untransposed operands only. GE_TILE may pick
 * L, LH, LM or LMD.
 */
ge_status_t gemm_epilog_plan_ex(int64_t m, int64_t n, int64_t k, ge_dtypes_t dt, ge_epilog_t ep, ge_op_t op_a,
                                ge_op_t op_b, ge_handle_t* out);

/*
 * gemm_epilog_execute - enqueue the planned computation on `stream` and return.
 *   A, B   : device inputs (m,k) and (k,n), type dt.ab, 16-byte aligned; (k,m) for A
 *            and (n,k) for B when the plan was made with op_a / op_b = GE_OP_T.
 *   bias   : device, m values of type dt.vec, aligned to its element size.
 *            Read by BIAS, RELU_BIAS, GELU_BIAS, RELU_AUX_BIAS, RELU_BIAS_UNFUSED;
 *            ignored (may be NULL) otherwise.
 *   D      : device output (m,n), type dt.d, 16-byte aligned.
 *   aux    : device mask words, gemm_epilog_aux_bytes(m,n) bytes, 16-byte aligned.
 *            Written by RELU_AUX_BIAS, read by DRELU_BGRAD, ignored otherwise.
 *            For DRELU_BGRAD_UNFUSED instead the forward activation, (m,n) of type
 *            dt.d, 16-byte aligned, read.
 *   bgrad  : device output, m values of type dt.vec, aligned to its element size.
 *            Written by DRELU_BGRAD and DRELU_BGRAD_UNFUSED, ignored otherwise.
 *   stream : a hipStream_t; NULL means the null stream.
 * Every output element in range is written; nothing outside the stated extents is.
 * Returns GE_ERR_HIP if a launch fails.
 * An execute enqueues kernel launches only (no memset, no host synchronisation), so it
 * may be captured into a HIP graph and replayed; replays of one plan must not overlap,
 * as for any two executes of a plan.
 */
ge_status_t gemm_epilog_execute(ge_handle_t h, const void* A, const void* B, const void* bias, void* D,
                                void* aux, void* bgrad, void* stream);

/*
 * gemm_epilog_autotune - time the kernel configurations that can run this plan on the
 * caller's own operands and keep the fastest in the plan. The plan's configuration
 * comes from a fixed per-shape table; this is the measured search that [P1] (final
 * paragraph: hand tuning through the algorithm heuristic) and [P2] (body, plan step:
 * the plan picks the best algorithm for the problem) describe. It runs on the real
 * data because the matrix cores' clock under the power limit depends on the values.
 *   h, A, B, bias, D, aux, bgrad, stream : as for gemm_epilog_execute (same rules and
 *            errors, checked first). D, aux and bgrad are written: on return they hold
 *            what one execute of the chosen configuration writes.
 *   repeats : timed executes per candidate, 1..1000 (else GE_ERR_INVALID_VALUE), each
 *            candidate after one untimed execute.
 *   best_ms : optional (may be NULL): receives the chosen configuration's mean time per
 *            execute in milliseconds, from HIP events on `stream`.
 * Candidates: for fp32 the 64x64 and 128x128 tiles; for fp16/bf16 with transposed
 * operands the 256x256 and 128x128 lockstep tiles (the latter with a 2- and a 3-stage
 * ring); otherwise the 256x256 tile (persistent, and one workgroup per tile with the
 * fragment reads interleaved into the MFMAs or issued in blocks), the 192x256 and 128x256
 * tiles (persistent) and the 128x128 tile with eight waves (2- or 3-stage ring) or four,
 * each with and without the split tail where it applies. A candidate whose
 * workspace cannot be allocated is skipped. The call synchronises `stream`, must
 * not overlap another execute of this plan, and runs on the device current at plan
 * time. On an error the plan keeps its configuration (GE_ERR_HIP if a launch or an
 * event call failed).
 */
ge_status_t gemm_epilog_autotune(ge_handle_t h, const void* A, const void* B, const void* bias, void* D, void* aux,
                                 void* bgrad, void* stream, int repeats, float* best_ms);

/* What a plan decides, as reported by gemm_epilog_plan_info. */
typedef struct {
  int tile_m, tile_n, tile_k;  /* workgroup tile and k-tile (tile_k 0: register-staged kernel) */
  int waves;                   /* waves per workgroup */
  int64_t tiles;               /* output tiles */
  int persistent_workgroups;   /* > 0: that many workgroups walk the tiles; 0: one per tile */
  int whole_tiles;             /* tiles computed whole (== tiles unless the last round is split) */
  int split_workgroups;        /* workgroups sharing the k loops of the remaining tiles */
  int split_run_ktiles;        /* k-tiles per split workgroup */
  int group_m;                 /* m-tiles per group of the tile order */
  size_t workspace_bytes;      /* device workspace the plan allocates */
  int stages;                  /* LDS stages of the operand ring (0: register-staged kernel) */
} ge_plan_info_t;

/*
 * gemm_epilog_plan_info - the configuration gemm_epilog_plan_ex would choose for this
 * problem on a gfx950 device with `compute_units` compute units, computed on the host
 * with no HIP call and no allocation (no device needed). The plan step of [P2] (body:
 * the costly choices are made once, when planning), exposed for inspection.
 *   m .. op_b      : as for gemm_epilog_plan_ex, same rules and errors.
 *   compute_units  : 1 .. 4096 (else GE_ERR_INVALID_VALUE); 256 on MI355X.
 *   info           : receives the decisions (GE_ERR_NULL_POINTER if NULL).
 * Honours the same environment switches as gemm_epilog_plan.
 */
ge_status_t gemm_epilog_plan_info(int64_t m, int64_t n, int64_t k, ge_dtypes_t dt, ge_epilog_t ep, ge_op_t op_a,
                                  ge_op_t op_b, int compute_units, ge_plan_info_t* info);

/*
 * gemm_epilog_lost_waits - how many split-tail waits of this plan's executes ran out
 * since the plan was made or since the last call, and reset the count.
 * A plan whose last round of tiles is split hands parts of a tile's k loop to other
 * workgroups; the workgroup that finishes the tile waits, bounded (about a second),
 * for their partial sums. A wait that runs out gives that tile NaN in D instead of
 * hanging the device, and leaves the plan's flags clean for later executes. The waits
 * end once the workgroups they wait for are scheduled, which a split plan's grid alone
 * always allows (its split workgroups fit the device at once); kernels of other streams
 * that keep compute units busy for longer than the bound (a second split plan's waiting
 * workgroups among them) can make a wait run out, so callers that run split plans
 * concurrently should check this count. This call
 * synchronises `stream` (hipStream_t, NULL = null stream), reads the count from the
 * plan's workspace and clears it; a plan without a split tail reports 0 at once.
 *   h     : the plan (GE_ERR_NULL_POINTER if NULL).
 *   count : receives the count (GE_ERR_NULL_POINTER if NULL).
 * GE_ERR_HIP if a copy or the synchronisation fails. Must not overlap an execute of h.
 */
ge_status_t gemm_epilog_lost_waits(ge_handle_t h, void* stream, uint32_t* count);

/* Bytes of the static device scratch that gemm_epilog_execute_noalloc works in. */
#define GEMM_EPILOG_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * gemm_epilog_execute_noalloc - gemm_epilog_plan_ex and gemm_epilog_execute in one call
 * that allocates nothing: for callers that cannot allocate device memory, such as code
 * under HIP graph capture, tight serving loops and harnesses that forbid hipMalloc.
 * The plan's decisions are made on the host (as gemm_epilog_plan_info reports them) and
 * the kernels of gemm_epilog_execute run with their workspace (bias-gradient partial
 * sums, the unfused chains' T1 and T2, the split tail's partials and flags) in a static
 * device array of GEMM_EPILOG_NOALLOC_SCRATCH_BYTES (64 MiB) per device, which each GPU
 * the library runs on holds until the process ends. No hipMalloc, hipFree or other
 * allocating call is made; the first call on a device takes the array's address once
 * (hipGetSymbolAddress) and clears its flag words with a kernel on `stream`.
 *   m .. op_b : as for gemm_epilog_plan_ex, same rules and errors.
 *   A .. stream : as for gemm_epilog_execute, same rules and errors.
 * Returns GE_ERR_SCRATCH when the workspace does not fit the scratch even without the
 * split tail (e.g. DRELU_BGRAD with ceil(n/64) * m * 4 bytes of partial sums above
 * 64 MiB, the unfused chain with 2 m n element bytes above it, or the unfused backward
 * with m n element bytes above it); nothing is launched
 * then. A split tail that does not fit is left out (the tiles run whole).
 * Every call on a device shares that device's array, and the array keeps the last
 * call's contents: calls that overlap on one device (two streams, two threads) race and
 * give wrong results; calls on one stream are ordered and safe. A split-tail wait that
 * runs out gives its tile NaN in D, as for gemm_epilog_execute.
 */
ge_status_t gemm_epilog_execute_noalloc(int64_t m, int64_t n, int64_t k, ge_dtypes_t dt, ge_epilog_t ep,
                                        ge_op_t op_a, ge_op_t op_b, const void* A, const void* B, const void* bias,
                                        void* D, void* aux, void* bgrad, void* stream);

/* gemm_epilog_free - release a plan and its workspace. NULL is accepted (GE_OK).
 * Must not be called while an execute on this plan may still be running. */
ge_status_t gemm_epilog_free(ge_handle_t h);

/* Bytes of the ReLU mask for an (m, n) output: 4 * ceil(m/32) * n (0 if m or n < 1). */
size_t gemm_epilog_aux_bytes(int64_t m, int64_t n);

/* Bytes of device workspace held by a plan (0 for NULL). */
size_t gemm_epilog_workspace_bytes(ge_handle_t h);

/* Human-readable name of the kernel configuration a plan chose, e.g.
 * "f16 RELU_BIAS tile 256x256 waves 2x2". Valid while the plan lives; "" for NULL. */
const char* gemm_epilog_describe(ge_handle_t h);

/* Static string for a status code. */
const char* gemm_epilog_status_string(ge_status_t s);

/* ---- Microscaled feed-forward operators ---------------------------------------------
 * The serving form of a feed-forward block: the residual addition and root-mean-square
 * norm in front of it, its operands in 8 and 4 bits with a shared scale per 32 values,
 * and its products, dense or by expert, with the epilogues above. The tokens lie along
 * the rows here (X (m, k), W (n, k), D = act(X . W^T + bias) of (m, n), one bias per
 * column), as a serving stack holds them.
 *
 * Microscaled values. Each 32 consecutive k values of a row share the scale 2^(s - 127)
 * of one byte s; s = 255 stands for NaN. With a the block's largest magnitude,
 * s = floor(log2 a) - emax + 127 held to 0 .. 254 (emax 2 for MXFP4, 8 for MXFP8; 0 for
 * a = 0), and 255 if the block holds an infinity or a NaN. The elements are the values over
 * the scale rounded to nearest even, saturating at the largest element.
 * Layout (the order the matrix instructions read; k is padded to a multiple of 256 with
 * zeros, rows to a multiple of 32, C = padded k / V, KT = padded k / 256):
 *   code byte of (r, k):  ((r/32) C + k/V) 512 + (r%32) 16 + b, with V = 32 and
 *     b = (k%32)/2, even k in the low nibble (MXFP4), or V = 16 and b = k%16 (MXFP8);
 *   scale byte of (r, k): ((r/32) KT + k/256) 256 + (k/32%2) 128 + (r%32) 4 + k/64%4.
 * gemm_epilog_mx_code_bytes / _scale_bytes give the buffers' sizes; both buffers are
 * 16-byte aligned. The contents of padding rows do not matter to any reader.
 *
 * Threading and errors as above: checks on the host first, work enqueued on `stream`,
 * kernel launches only (an execute may be captured into a HIP graph).
 */
typedef enum {
  GE_MXFP4 = 0, /* 4-bit elements e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives */
  GE_MXFP8 = 1  /* 8-bit elements e4m3: up to 448, no infinity */
} ge_mx_format_t;

/* Bytes of the codes / scales of a (rows, k) operand; 0 for sizes outside the supported
 * set (0 <= rows <= 2^31 - 1, 1 <= k <= 2^20, at most 2^24 - 1 tiles of 32 x 256). */
size_t gemm_epilog_mx_code_bytes(ge_mx_format_t fmt, int64_t rows, int64_t k);
size_t gemm_epilog_mx_scale_bytes(int64_t rows, int64_t k);

/*
 * gemm_epilog_mx_quantize - (rows, k) values of type dt to microscaled form.
 *   src  : device; element (r, k) at src[r row_stride + k col_stride] (strides in
 *          elements, not negative). Rows contiguous along k (col_stride 1), the columns of
 *          a features-by-batch matrix (row_stride 1), or any other strides.
 *   codes, scales : device, written whole, padding included.
 * rows = 0 does nothing. The blocks run along k in both orders.
 */
ge_status_t gemm_epilog_mx_quantize(int64_t rows, int64_t k, ge_dtype_t dt, const void* src, int64_t row_stride,
                                    int64_t col_stride, ge_mx_format_t fmt, void* codes, void* scales, void* stream);

/* gemm_epilog_mx_dequantize - the values (element times scale, rounded to dt) of a
 * microscaled operand, to dst[r row_stride + k], row_stride >= k. */
ge_status_t gemm_epilog_mx_dequantize(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* codes,
                                      const void* scales, ge_dtype_t dt, void* dst, int64_t row_stride, void* stream);

/* gemm_epilog_mx_pack - row-major codes ((rows, ceil(k/2)) bytes for MXFP4, (rows, k) for
 * MXFP8) and row-major scales ((rows, ceil(k/32)) bytes), as checkpoints hold them, into
 * the layout above. Once per weight. */
ge_status_t gemm_epilog_mx_pack(int64_t rows, int64_t k, ge_mx_format_t fmt, const void* src_codes,
                                const void* src_scales, void* codes, void* scales, void* stream);

/* Type of a product's D: 32 or 16 bits, row-major (m, n), or MXFP8 in the layout above
 * (rows m, k = n), ready to be the next product's X. */
typedef enum { GE_MX_D_F32 = 0, GE_MX_D_F16 = 1, GE_MX_D_BF16 = 2, GE_MX_D_MXFP8 = 3 } ge_mx_out_t;

/* x: format of X (W is MXFP4); d: type of D; vec: type of bias (fp32, or D's type; any
 * type with an MXFP8 D).
 * Accumulators are always fp32. The matrix unit adds eight neighbouring products at a time,
 * aligned to the largest of them, and drops what lies more than 13 bits below it. MXFP4 by
 * MXFP4 fits in that whole. An MXFP8 X does not: for an fp32 or MXFP8 D, and for any D where
 * the rows are few (plan_info gives stages 0), X is multiplied in two parts that do, and the
 * sums are fp32's (2.5e-8 of the result's norm at k = 4096). A 16-bit D of more rows takes one
 * part, 1.3e-5 of the norm of the sums (its own rounding is 2e-4 of it in fp16, 1.7e-3 in bf16):
 * a value far below the others, its terms or its sum and bias having cancelled, can be off by
 * more than its own rounding. */
typedef struct {
  ge_mx_format_t x;
  ge_mx_out_t d;
  ge_dtype_t vec;
} ge_mx_types_t;

typedef struct ge_mx_plan* ge_mx_handle_t; /* opaque; owned by the library */

/*
 * gemm_epilog_mx_plan - plan D = act(X . W^T + bias) for one (n, k) and any m.
 *   n, k    : 1 .. 2^20.
 *   experts : 0 for one product; 1 .. 4096 for products by expert, where the rows of X
 *             are sorted by expert and each expert has its own W and bias.
 *   ep      : NONE, BIAS, RELU_BIAS or GELU_BIAS (other epilogues: GE_ERR_NOT_SUPPORTED).
 *             As above, the ReLU keeps a value only where it is > 0: of NaN it gives 0.
 * Allocates the workspace (sums of a product whose k loop is split over workgroups). A
 * plan may be used from one stream at a time; any number of weights may share it. Its
 * executes run on the device that was current when it was made, which has to be current
 * again, with that device's pointers.
 */
ge_status_t gemm_epilog_mx_plan(int64_t n, int64_t k, int64_t experts, ge_mx_types_t types, ge_epilog_t ep,
                                ge_mx_handle_t* out);

/* What an execute of m rows would launch. */
typedef struct {
  int tile_m, tile_n;      /* rows of X and of W per workgroup */
  int waves;               /* waves per workgroup */
  int stages;              /* LDS stages of the operand ring (0: W goes straight to registers) */
  int splits;              /* workgroups that share a tile's k loop */
  int64_t tiles;           /* by expert: the most there can be */
  int64_t workgroups;      /* fewer than tiles times splits where they walk the tiles (a second
                              launch, not counted here, may take a short last round of them) */
  size_t workspace_bytes;  /* device workspace of the plan (independent of m) */
} ge_mx_plan_info_t;

/* gemm_epilog_mx_plan_info - computed on the host with no HIP call, for a gfx950 device
 * with `compute_units` compute units (1 .. 4096). */
ge_status_t gemm_epilog_mx_plan_info(int64_t n, int64_t k, int64_t experts, ge_mx_types_t types, ge_epilog_t ep,
                                     int64_t m, int compute_units, ge_mx_plan_info_t* info);

/*
 * gemm_epilog_mx_execute - enqueue the product for m rows (0 <= m <= 2^31 - 1; 0 does
 * nothing).
 *   x_codes, x_scales : X (m, k).
 *   w_codes, w_scales : W (n, k), MXFP4; by expert: the experts' buffers one after the
 *             other, each of the size of an (n, k) operand.
 *   bias    : n values of type vec, (experts, n) by expert; ignored (may be NULL) for NONE.
 *   offsets : by expert: device, experts + 1 int32; expert e has rows offsets[e] ..
 *             offsets[e+1] - 1 of X and D. Read when the kernel runs, so they may come from
 *             a kernel before it. Values outside 0 .. m or that run backwards are held to
 *             valid or empty ranges, and each range to the rows past the furthest end of
 *             those before it, so that a row has one expert at most; rows that no expert has
 *             are not written. NULL otherwise.
 *   D       : (m, n) of type d, aligned to its element; or MXFP8 codes, 16-byte aligned
 *             (written with the padding along n, without padding rows).
 *   d_scales: MXFP8 D: its scales; ignored otherwise.
 */
ge_status_t gemm_epilog_mx_execute(ge_mx_handle_t h, int64_t m, const void* x_codes, const void* x_scales,
                                   const void* w_codes, const void* w_scales, const void* bias, const void* offsets,
                                   void* D, void* d_scales, void* stream);

/* gemm_epilog_mx_free - release a plan and its workspace. NULL is accepted (GE_OK). */
ge_status_t gemm_epilog_mx_free(ge_mx_handle_t h);

/*
 * gemm_epilog_rms_norm - s = x + residual rounded to dt (s = x without a residual) and
 * y = s / sqrt(mean(s^2) + eps) * weight, over rows of d values; sums in fp32.
 *   rows, d  : 0 <= rows <= 2^31 - 1 (0 does nothing), 1 <= d <= 32768 (above:
 *              GE_ERR_NOT_SUPPORTED).
 *   x, residual : (rows, d) of type dt, row strides ldx, ldr in elements (0 repeats a
 *              row). residual may be NULL.
 *   weight   : d values of type wdt (dt or fp32).
 *   eps      : >= 0 and finite.
 *   sum      : receives s, row stride lds; needed with a residual, optional without. May be
 *              x or residual itself.
 *   y        : receives y as dt, row stride ldy; NULL if not wanted.
 *   codes, scales : receive y as MXFP8, with zeros in the padding along d (NaN in a row that
 *              is NaN; padding rows are not written); both NULL if not wanted. At least one
 *              form of y is needed. Their size limits rows and d as for an operand (above:
 *              GE_ERR_NOT_SUPPORTED).
 * Pointers are aligned to their elements (codes and scales to 16 bytes); 16-byte aligned
 * rows with d a multiple of 8 run fastest, by far so where d is over 8192.
 */
ge_status_t gemm_epilog_rms_norm(int64_t rows, int64_t d, ge_dtype_t dt, const void* x, int64_t ldx,
                                 const void* residual, int64_t ldr, const void* weight, ge_dtype_t wdt, float eps,
                                 void* sum, int64_t lds, void* y, int64_t ldy, void* codes, void* scales,
                                 void* stream);

/* Bytes of the workspace of gemm_epilog_rms_norm_backward (0 for rows = 0). */
size_t gemm_epilog_rms_norm_workspace_bytes(int64_t rows, int64_t d);

/*
 * gemm_epilog_rms_norm_backward - gradients of the norm from the stored s:
 * dx = r (g - h mean(g h)) + dresidual with r = 1 / sqrt(mean(s^2) + eps), g = dy weight,
 * h = s r; dweight = sum over rows of dy h, in fp32 and in a fixed order. dx is the gradient
 * of x and of residual alike.
 *   dy, s, dresidual : (rows, d) of type dt with their row strides; dresidual (the gradient
 *              that reaches s past the norm) may be NULL.
 *   dx       : (rows, d) of type dt; may be dy or dresidual itself.
 *   dweight  : d values of type wdt (zeros for rows = 0).
 *   workspace: device, workspace_bytes >= gemm_epilog_rms_norm_workspace_bytes(rows, d)
 *              (else GE_ERR_SCRATCH), 16-byte aligned, used until the work is done.
 */
ge_status_t gemm_epilog_rms_norm_backward(int64_t rows, int64_t d, ge_dtype_t dt, const void* dy, int64_t lddy,
                                          const void* s, int64_t lds, const void* weight, ge_dtype_t wdt, float eps,
                                          const void* dresidual, int64_t lddr, void* dx, int64_t lddx, void* dweight,
                                          void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_EPILOG_H_ */
