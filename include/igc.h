/*
 * igc.h -- C ABI of libigc: a software-pipelined bf16/fp16 GEMM with fp32
 * accumulation, and the same mainloop run as implicit-GEMM (im2col) NHWC
 * convolutions (forward, data gradient, filter gradient), for AMD Instinct
 * MI355X (gfx950); products and forward convolutions with bias, activation and
 * residual in their epilogue, the epilogue's gradient, and group norm with an
 * activation, forward and backward; products of 8-bit integers with a scale for
 * each row and column, and the row operators that feed them: the root-mean-square
 * norm (to 16 or 8 bits, and its gradient) and activations rounded to 8 bits.
 *
 * What is computed follows the "B200 TMA Pipeline Designer" page (section
 * "E -- Executable steps": a tiled matrix product fed by a ring of PIPE_DEPTH
 * shared-memory stages under ready/free synchronisation, with a prologue /
 * steady-state / epilogue timeline) and the "two free pipeline stages" note
 * (section "The atom changes the fragment": the same pipelined mainloop
 * driving an implicit-GEMM convolution with IM2COL operand loads).  The pages'
 * NVIDIA mechanisms (TMA descriptors, mbarriers, elected issuer lanes, 2-SM
 * atoms) are not used; the library uses gfx950 direct-to-LDS buffer loads,
 * s_waitcnt / s_barrier (or LDS counters) and MFMA.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers owned by the caller.  The library
 *   never frees or retains them; calls are thread-safe.
 * - Each call only validates its arguments and enqueues work on `stream` (a
 *   hipStream_t; NULL = the default stream), which must belong to the current
 *   device.  It returns before the GPU finishes; synchronise the stream to
 *   observe the result.
 * - Workspace.  A call whose schedule splits K (k_splits > 1, or stream-K)
 *   needs an fp32 workspace of igc_workspace_bytes(...) bytes.  The `_ex`
 *   entry points take it from the caller (`workspace`, 256-byte aligned,
 *   `workspace_bytes` at least that size); the call then allocates nothing.
 *   With workspace == NULL (and always for the entry points without `_ex`)
 *   the library takes it stream-ordered on `stream` from a memory pool it
 *   creates on the current device at the first such call, and releases it
 *   with hipFreeAsync on the same stream; the pool keeps up to 256 MiB of freed
 *   workspace mapped until the process ends (the device's default pool is not
 *   changed).  A schedule that does not split K needs and takes nothing.
 *   Calls that share one workspace must be ordered (one stream).  On a stream
 *   that is being captured into a graph, a call whose schedule needs a
 *   workspace must be given one (or use gemm_bf16_noalloc): the library does
 *   not take one from its pool during capture (IGC_ERR_UNSUPPORTED).
 * - Leading dimensions are in ELEMENTS, not bytes.
 * - Alignment: every tensor base pointer must be 16-byte aligned and every
 *   leading dimension times the element size a multiple of 16 bytes (8
 *   elements for 16-bit types, 4 for fp32, 16 for 8-bit integers).  Otherwise IGC_ERR_MISALIGNED.
 *   A matrix's rows may be read to the end of the 16-byte piece that holds their
 *   last value, the last row's too (what lies there does not matter and is never
 *   written).  Vectors (bias, gamma, beta, scales, rstd) have no leading dimension:
 *   their values lie together, and nothing beside them is read.
 * - Arguments are checked before anything is launched; on any error nothing
 *   is enqueued and the output is untouched.  No exception crosses the ABI.
 * - Outputs must not alias inputs except where an operation says so (not
 *   checked; the result is undefined).
 * - Results are deterministic: the same inputs and tune give the same bits on
 *   every call (no atomics; a fixed summation order per output element).
 * - Device errors: a stream-K owner waits for the partials of the workgroups
 *   sharing its tile with a bounded poll.  If a wait ever gives up (which a
 *   correct schedule with every workgroup resident never does) the owner
 *   writes its tile as NaN and sets the device's error word, which
 *   igc_take_device_error reads.
 */
#ifndef IGC_H
#define IGC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t *igc_stream_t; /* the same type as hipStream_t */

typedef enum {
    IGC_OK = 0,
    IGC_ERR_INVALID_VALUE = 1, /* negative size, leading dimension too small, bad enum, NULL pointer, short workspace */
    IGC_ERR_MISALIGNED = 2,    /* pointer or leading dimension breaks the 16-byte rule; conv channels % 8 != 0 */
    IGC_ERR_UNSUPPORTED = 3,   /* tuning choice not compiled in, or an operand span / index >= 2^31 */
    IGC_ERR_HIP = 4            /* the HIP runtime reported an error when allocating or launching */
} igc_status_t;

typedef enum { IGC_ROW_MAJOR = 0, IGC_COL_MAJOR = 1 } igc_layout_t;

typedef enum { IGC_OUT_F32 = 0, IGC_OUT_BF16 = 1, IGC_OUT_F16 = 2 } igc_out_t;

/* The operation whose GEMM view a workspace or default-tile query is about. */
typedef enum { IGC_OP_GEMM = 0, IGC_OP_CONV_FPROP = 1, IGC_OP_CONV_DGRAD = 2, IGC_OP_CONV_WGRAD = 3 } igc_op_t;

/* Optional tuning.
 *   bm, bn, bk    output tile BM x BN and K tile BK;
 *   pipe_depth    number of LDS stages in the ring ("PIPE_DEPTH" of the B200
 *                 TMA Pipeline Designer page, Executable steps 6 and 7);
 *   waves         wave64s per workgroup (4: one per SIMD; 8: two per SIMD);
 *   mfma          MFMA block edge (32: v_mfma_f32_32x32x16, 16:
 *                 v_mfma_f32_16x16x32; 0 means 32);
 *   half_stage    1: the ring holds one more operand tile (A or B) than
 *                 pipe_depth whole stages (2*pipe_depth + 1 operand slots);
 *   loader_waves  how many waves issue the global->LDS loads (0 or `waves`:
 *                 every wave; 4 of 8: one per SIMD);
 *   k_splits      <= 1: none; S > 1: split K into up to S ranges computed by
 *                 separate workgroups whose fp32 partial tiles a second kernel
 *                 sums in split order;
 *   stream_k      0: none; G > 0: a persistent grid of G workgroups takes
 *                 equal runs of the tiles' K ranges, in units of one ring
 *                 period; a tile shared by several runs is finished by the
 *                 workgroup that computes its last K unit, which adds the fp32
 *                 partials of the others in a fixed order (deterministic).
 *                 Assumes the G workgroups are resident together (G at most
 *                 the CU count, nothing else occupying the device);
 *   ring_sync     0: one workgroup barrier per K tile is both the "ready" and
 *                 the "free" signal; 1: per-slot LDS ready/free counters
 *                 (Executable step 4: every stage has its own ready and free
 *                 signal with one producer side and one consumer side);
 *   sk_hybrid     with stream_k: 1 runs whole tiles in data-parallel rounds
 *                 first and splits only the last, partial round's tiles into
 *                 K runs; 0 splits every tile.
 * k_splits > 1 together with stream_k > 0, stream_k < 0, or sk_hybrid without
 * stream_k is IGC_ERR_INVALID_VALUE.  Only compiled (bm, bn, bk, pipe_depth,
 * waves, mfma, half_stage, loader_waves, ring_sync) combinations are accepted
 * (igc_tune_count / igc_tune_get list them, igc_tune_scope says what each
 * is built for); NULL selects the built-in choice for the shape
 * (igc_default_tune). */
typedef struct {
    int bm, bn, bk, pipe_depth, waves, mfma, half_stage, loader_waves, k_splits, stream_k, ring_sync, sk_hybrid;
} igc_tune_t;

/*
 * GEMM: C = A * B with bf16 inputs, fp32 accumulation, output type `c_type`.
 * The tiled, software-pipelined product of the "B200 TMA Pipeline Designer"
 * page (section "E -- Executable steps", steps 6-8).
 *   A is M x K: IGC_ROW_MAJOR -> A[i*lda + k] (lda >= K);
 *               IGC_COL_MAJOR -> A[k*lda + i] (lda >= M).
 *   B is K x N: IGC_ROW_MAJOR -> B[k*ldb + j] (ldb >= N);
 *               IGC_COL_MAJOR -> B[j*ldb + k] (ldb >= K).
 *   C is M x N row-major: C[i*ldc + j] (ldc >= N), element type per c_type;
 *     fp32 -> bf16/fp16 rounds to nearest-even.
 * K == 0 writes zeros; M == 0 or N == 0 is a no-op returning IGC_OK.
 * Errors: IGC_ERR_INVALID_VALUE for negative sizes, bad enums, NULL pointers or
 * leading dimensions below the minimum; IGC_ERR_MISALIGNED; IGC_ERR_UNSUPPORTED
 * when one tile's rows span 2^31 bytes or more; IGC_ERR_HIP.
 */
igc_status_t gemm_bf16(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                       const void *B, int64_t ldb, igc_layout_t lb, void *C, int64_t ldc, igc_out_t c_type,
                       igc_stream_t stream);

/* The same contract with IEEE binary16 (fp16) inputs. */
igc_status_t gemm_fp16(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                       const void *B, int64_t ldb, igc_layout_t lb, void *C, int64_t ldc, igc_out_t c_type,
                       igc_stream_t stream);

/* gemm_bf16 / gemm_fp16 with an explicit tile, pipeline depth and schedule
 * (tune == NULL: the built-in choice) and a caller-owned workspace (see the
 * conventions above; NULL: the library's pool).  A non-NULL workspace shorter
 * than igc_workspace_bytes(IGC_OP_GEMM, M, N, K, tune) or not 256-byte
 * aligned is IGC_ERR_INVALID_VALUE. */
igc_status_t gemm_bf16_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                          const void *B, int64_t ldb, igc_layout_t lb, void *C, int64_t ldc, igc_out_t c_type,
                          const igc_tune_t *tune, void *workspace, int64_t workspace_bytes, igc_stream_t stream);
igc_status_t gemm_fp16_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                          const void *B, int64_t ldb, igc_layout_t lb, void *C, int64_t ldc, igc_out_t c_type,
                          const igc_tune_t *tune, void *workspace, int64_t workspace_bytes, igc_stream_t stream);

/*
 * Convolutions.  Shared geometry: N images of H x W pixels with C channels,
 * K filters of R x S taps, strides (stride_h, stride_w) >= 1, zero padding
 * (pad_h, pad_w) >= 0, dilations (dil_h, dil_w) >= 1, and the output size
 *   P = (H + 2*pad_h - dil_h*(R-1) - 1)/stride_h + 1,
 *   Q = (W + 2*pad_w - dil_w*(S-1) - 1)/stride_w + 1   (both must be >= 1).
 * Layouts: x NHWC (N*H*W*C elements), w KRSC (K*R*S*C), y NPQK (N*P*Q*K), all
 * dense.  Requirements: H, W, C, R, S >= 1 and N, K >= 0, else
 * IGC_ERR_INVALID_VALUE (an empty output is a no-op; an empty sum -- the data
 * gradient with K = 0, the filter gradient with N = 0 -- writes zeros); C % 8 == 0 (and K % 8 == 0 for the gradients),
 * else IGC_ERR_MISALIGNED; every tensor spanning < 2^31 bytes and every GEMM
 * dimension and index below 2^31, else IGC_ERR_UNSUPPORTED.
 */

/*
 * Forward convolution (cross-correlation) as an implicit GEMM, bf16 inputs,
 * fp32 accumulation: the convolution that the "two free pipeline stages" note
 * runs through the pipelined mainloop with IM2COL operand loads (section "The
 * atom changes the fragment"):
 *   y[n][p][q][k] = sum_{r<R, s<S, c<C} x[n][p*sh - ph + r*dh][q*sw - pw + s*dw][c] * w[k][r][s][c]
 * with taps outside the H x W image contributing nothing.  y has type y_type.
 * GEMM view (for igc_workspace_bytes / igc_default_tune): M = N*P*Q,
 * N_gemm = K, K_gemm = R*S*C.
 */
igc_status_t conv2d_nhwc_implicit_gemm(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                       int stride_w, int pad_h, int pad_w, int dil_h, int dil_w, const void *x,
                                       const void *w, void *y, igc_out_t y_type, igc_stream_t stream);
/* The same contract with IEEE binary16 (fp16) x and w. */
igc_status_t conv2d_nhwc_implicit_gemm_fp16(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                            int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                            const void *x, const void *w, void *y, igc_out_t y_type,
                                            igc_stream_t stream);
/* With an explicit tune and a caller-owned workspace (as gemm_bf16_ex). */
igc_status_t conv2d_nhwc_implicit_gemm_ex(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                          int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                          const void *x, const void *w, void *y, igc_out_t y_type,
                                          const igc_tune_t *tune, void *workspace, int64_t workspace_bytes,
                                          igc_stream_t stream);
igc_status_t conv2d_nhwc_implicit_gemm_fp16_ex(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                               int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                               const void *x, const void *w, void *y, igc_out_t y_type,
                                               const igc_tune_t *tune, void *workspace, int64_t workspace_bytes,
                                               igc_stream_t stream);

/*
 * Data gradient of the forward convolution above, as an implicit GEMM on the
 * same mainloop: with dy (NPQK, the gradient of y) and w (KRSC),
 *   dx[n][h][w][c] = sum over (r, s, k) of dy[n][p][q][k] * w[k][r][s][c]
 * over the filter taps whose forward read lands on (h, w), i.e.
 * p*sh - ph + r*dh = h and q*sw - pw + s*dw = w for integers 0 <= p < P,
 * 0 <= q < Q.  dx (NHWC) has type dx_type and is fully written (pixels no tap
 * reaches get 0).  The pages run only the forward pass through the mainloop;
 * this is its adjoint in x, the other operand iterator the same mainloop
 * serves.  GEMM view: M = N*H*W, N_gemm = C, K_gemm = R*S*K.  A unit stride
 * and R, S <= 16 use per-pixel tap masks; other strides test each tap's
 * landing position for divisibility by the stride.
 */
igc_status_t conv2d_nhwc_dgrad_implicit_gemm(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                             int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                             const void *dy, const void *w, void *dx, igc_out_t dx_type,
                                             igc_stream_t stream);
igc_status_t conv2d_nhwc_dgrad_implicit_gemm_fp16(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                  int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                  const void *dy, const void *w, void *dx, igc_out_t dx_type,
                                                  igc_stream_t stream);
igc_status_t conv2d_nhwc_dgrad_implicit_gemm_ex(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                const void *dy, const void *w, void *dx, igc_out_t dx_type,
                                                const igc_tune_t *tune, void *workspace, int64_t workspace_bytes,
                                                igc_stream_t stream);
igc_status_t conv2d_nhwc_dgrad_implicit_gemm_fp16_ex(int N, int H, int W, int C, int K, int R, int S,
                                                     int stride_h, int stride_w, int pad_h, int pad_w, int dil_h,
                                                     int dil_w, const void *dy, const void *w, void *dx,
                                                     igc_out_t dx_type, const igc_tune_t *tune, void *workspace,
                                                     int64_t workspace_bytes, igc_stream_t stream);

/*
 * Filter gradient of the forward convolution above, as an implicit GEMM on
 * the same mainloop: with x (NHWC) and dy (NPQK),
 *   dw[k][r][s][c] = sum over (n, p, q) of dy[n][p][q][k] * x[n][p*sh - ph + r*dh][q*sw - pw + s*dw][c]
 * with taps outside the image contributing nothing; dw (KRSC) has type
 * dw_type.  The adjoint of the forward convolution in w.  GEMM view:
 * M = K, N_gemm = R*S*C, K_gemm = N*P*Q (deep: the default schedule splits
 * it over the CUs).
 */
igc_status_t conv2d_nhwc_wgrad_implicit_gemm(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                             int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                             const void *x, const void *dy, void *dw, igc_out_t dw_type,
                                             igc_stream_t stream);
igc_status_t conv2d_nhwc_wgrad_implicit_gemm_fp16(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                  int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                  const void *x, const void *dy, void *dw, igc_out_t dw_type,
                                                  igc_stream_t stream);
igc_status_t conv2d_nhwc_wgrad_implicit_gemm_ex(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                const void *x, const void *dy, void *dw, igc_out_t dw_type,
                                                const igc_tune_t *tune, void *workspace, int64_t workspace_bytes,
                                                igc_stream_t stream);
igc_status_t conv2d_nhwc_wgrad_implicit_gemm_fp16_ex(int N, int H, int W, int C, int K, int R, int S,
                                                     int stride_h, int stride_w, int pad_h, int pad_w, int dil_h,
                                                     int dil_w, const void *x, const void *dy, void *dw,
                                                     igc_out_t dw_type, const igc_tune_t *tune, void *workspace,
                                                     int64_t workspace_bytes, igc_stream_t stream);

/* gemm_bf16 for callers that cannot allocate (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): the built-in
 * schedule, with its workspace (K-split or stream-K partial tiles and flags)
 * in a library-owned device array of 16 MiB + 4 KiB that each GPU holds until
 * the process ends.  The call allocates nothing.  When the built-in schedule's
 * workspace fits the array it runs that schedule and gives the same bits as
 * gemm_bf16; otherwise (a K split of 256 x 128 tiles, e.g. 1024 x 1024 x 65536)
 * it runs 128 x 128 stream-K over 256 workgroups, whose workspace always fits,
 * with a different summation order.  Calls that overlap on one GPU share the
 * array and race: order them (one stream).  IGC_ERR_HIP if the array cannot
 * be located on the current device; otherwise as gemm_bf16. */
igc_status_t gemm_bf16_noalloc(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                               const void *B, int64_t ldb, igc_layout_t lb, void *C, int64_t ldc, igc_out_t c_type,
                               igc_stream_t stream);

/*
 * Fused epilogues.  What a layer does to a product before it is rounded, in
 * fp32 and with one rounding:
 *   backward 0:  z = (A*B)[m][n] + bias[n];  pre[m][n] = z (rounded, if pre is given);
 *                D[m][n] = act(z) + residual[m][n]
 *   backward 1:  D[m][n] = ((A*B)[m][n] + bias[n]) * act'(pre[m][n]) + residual[m][n]
 * the second being the gradient that reaches z of the layer below when A*B is
 * the product of dy with the upper layer's weights.
 *   act            IGC_ACT_NONE: z; RELU: max(z, 0), derivative 0 at 0; GELU:
 *                  z Phi(z); GELU_TANH: z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)));
 *                  SILU: z / (1 + exp(-z)).  A NaN stays a NaN.
 *   bias           N values of bias_type, aligned to their size; NULL: none
 *   residual       M x N of residual_type, row-major, ldr >= N; NULL: none
 *   pre            M x N of pre_type, row-major, ldp >= N: written (backward 0)
 *                  or read (backward 1); NULL: not kept, allowed with backward 1
 *                  only for IGC_ACT_NONE
 * residual and pre keep the alignment rule of every tensor.  Either may be D
 * itself (same pointer, leading dimension and type) when it is read: each
 * element is read before it is written.  Otherwise nothing may alias.
 */
typedef enum {
    IGC_ACT_NONE = 0,
    IGC_ACT_RELU = 1,
    IGC_ACT_GELU = 2,
    IGC_ACT_GELU_TANH = 3,
    IGC_ACT_SILU = 4
} igc_act_t;

typedef struct {
    igc_act_t act;
    int backward;
    const void *bias;
    igc_out_t bias_type;
    const void *residual;
    int64_t ldr;
    igc_out_t residual_type;
    void *pre;
    int64_t ldp;
    igc_out_t pre_type;
} igc_epilogue_t;

/* GEMM with a fused epilogue: operands, layouts, sizes, alignment and errors
 * as gemm_bf16 / gemm_fp16, D in the place of C; epilogue must not be NULL.
 * K == 0 leaves z = bias.  The built-in choice has tiles down to 64 x 64 and
 * never stream-K; a product of at most 32 rows of a row-major A runs on a kernel
 * that streams B once where that is faster.  With an explicit tune, tiles and
 * schedules as gemm_bf16_ex, except that stream-K, and without a K split a
 * configuration without IGC_SCOPE_EPILOGUE, are IGC_ERR_UNSUPPORTED; so is a D,
 * residual or pre of which the rows of one tile span 2^31 bytes or more.
 * An epilogue of nothing (IGC_ACT_NONE, every pointer NULL) gives the plain product
 * on these schedules, which is the faster call where gemm_bf16 / gemm_fp16 take
 * 128 x 128 tiles for a small output (1024 x 1024 x 1024 6.1 us against 9.5) or
 * 256 x 256 tiles with a column-major A, such as a wide layer's weight gradient
 * (4096 x 4096 x 8192 219 us against 548).
 * Workspace: igc_epilogue_workspace_bytes. */
igc_status_t gemm_bf16_epilogue(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                                const void *B, int64_t ldb, igc_layout_t lb, void *D, int64_t ldd, igc_out_t d_type,
                                const igc_epilogue_t *epilogue, igc_stream_t stream);
igc_status_t gemm_fp16_epilogue(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                                const void *B, int64_t ldb, igc_layout_t lb, void *D, int64_t ldd, igc_out_t d_type,
                                const igc_epilogue_t *epilogue, igc_stream_t stream);
igc_status_t gemm_bf16_epilogue_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                                   const void *B, int64_t ldb, igc_layout_t lb, void *D, int64_t ldd,
                                   igc_out_t d_type, const igc_epilogue_t *epilogue, const igc_tune_t *tune,
                                   void *workspace, int64_t workspace_bytes, igc_stream_t stream);
igc_status_t gemm_fp16_epilogue_ex(int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, igc_layout_t la,
                                   const void *B, int64_t ldb, igc_layout_t lb, void *D, int64_t ldd,
                                   igc_out_t d_type, const igc_epilogue_t *epilogue, const igc_tune_t *tune,
                                   void *workspace, int64_t workspace_bytes, igc_stream_t stream);

/* Forward convolution with a fused epilogue: arguments and errors as
 * conv2d_nhwc_implicit_gemm; bias has one value per filter, residual and pre
 * are dense NPQK like y (ldr and ldp are not looked at).  backward 1 is
 * IGC_ERR_UNSUPPORTED. */
igc_status_t conv2d_nhwc_implicit_gemm_epilogue(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                const void *x, const void *w, void *y, igc_out_t y_type,
                                                const igc_epilogue_t *epilogue, igc_stream_t stream);
igc_status_t conv2d_nhwc_implicit_gemm_epilogue_fp16(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                     int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                     const void *x, const void *w, void *y, igc_out_t y_type,
                                                     const igc_epilogue_t *epilogue, igc_stream_t stream);
igc_status_t conv2d_nhwc_implicit_gemm_epilogue_ex(int N, int H, int W, int C, int K, int R, int S, int stride_h,
                                                   int stride_w, int pad_h, int pad_w, int dil_h, int dil_w,
                                                   const void *x, const void *w, void *y, igc_out_t y_type,
                                                   const igc_epilogue_t *epilogue, const igc_tune_t *tune,
                                                   void *workspace, int64_t workspace_bytes, igc_stream_t stream);
igc_status_t conv2d_nhwc_implicit_gemm_epilogue_fp16_ex(int N, int H, int W, int C, int K, int R, int S,
                                                        int stride_h, int stride_w, int pad_h, int pad_w, int dil_h,
                                                        int dil_w, const void *x, const void *w, void *y,
                                                        igc_out_t y_type, const igc_epilogue_t *epilogue,
                                                        const igc_tune_t *tune, void *workspace,
                                                        int64_t workspace_bytes, igc_stream_t stream);

/* Workspace bytes of a call with an epilogue (op IGC_OP_GEMM or
 * IGC_OP_CONV_FPROP; GEMM view M x N x K; enough for every operand layout): the
 * fp32 parts of a K split, or the fp32 product of a convolution whose filter
 * count is not a multiple of 8; otherwise 0; -1 for bad arguments. */
int64_t igc_epilogue_workspace_bytes(igc_op_t op, int64_t M, int64_t N, int64_t K, const igc_tune_t *tune);

/* The built-in choice of a call with an epilogue (op IGC_OP_GEMM with operand
 * layouts la and lb, or IGC_OP_CONV_FPROP, which does not look at them) into
 * *out; returns 1, or 0 for bad arguments or a choice that is not compiled for
 * both input types.  Where a product of dense operands runs on the kernel of few
 * rows, which has no tile: bm = 0, bn the columns of a workgroup, k_splits the
 * parts along K, and 0 elsewhere. */
int igc_epilogue_default_tune(igc_op_t op, int64_t M, int64_t N, int64_t K, igc_layout_t la, igc_layout_t lb,
                              igc_tune_t *out);

/*
 * Gradient of the epilogue in one pass, for a dD and a pre of the input type
 * (bf16 or fp16), M x N row-major (a convolution's dense y: M = N*P*Q, N = K):
 *   dz[m][n] = dD[m][n] * act'(pre[m][n])      (rounded once)
 *   dbias[n] = sum over m of dD[m][n] * act'(pre[m][n])      (summed in fp32 before any rounding)
 * The gradient of the residual is dD itself.  dz NULL: only dbias (of
 * dbias_type, aligned to its size); dbias NULL: only dz; both NULL is
 * IGC_ERR_INVALID_VALUE.  pre is read only when act is not IGC_ACT_NONE.  dz
 * may be dD or pre (same leading dimension).  M == 0 writes dbias = 0.
 * N >= 2^31 or M >= 2^40 is IGC_ERR_UNSUPPORTED.  Workspace when dbias is
 * given: igc_epilogue_backward_workspace_bytes (-1 for sizes that the call refuses).
 */
igc_status_t epilogue_backward_bf16(int64_t M, int64_t N, igc_act_t act, const void *dD, int64_t ldd, const void *pre,
                                    int64_t ldp, void *dz, int64_t ldz, void *dbias, igc_out_t dbias_type,
                                    igc_stream_t stream);
igc_status_t epilogue_backward_fp16(int64_t M, int64_t N, igc_act_t act, const void *dD, int64_t ldd, const void *pre,
                                    int64_t ldp, void *dz, int64_t ldz, void *dbias, igc_out_t dbias_type,
                                    igc_stream_t stream);
igc_status_t epilogue_backward_bf16_ex(int64_t M, int64_t N, igc_act_t act, const void *dD, int64_t ldd,
                                       const void *pre, int64_t ldp, void *dz, int64_t ldz, void *dbias,
                                       igc_out_t dbias_type, void *workspace, int64_t workspace_bytes,
                                       igc_stream_t stream);
igc_status_t epilogue_backward_fp16_ex(int64_t M, int64_t N, igc_act_t act, const void *dD, int64_t ldd,
                                       const void *pre, int64_t ldp, void *dz, int64_t ldz, void *dbias,
                                       igc_out_t dbias_type, void *workspace, int64_t workspace_bytes,
                                       igc_stream_t stream);
int64_t igc_epilogue_backward_workspace_bytes(int64_t M, int64_t N);

/*
 * Group norm with an activation over channels-last images (bf16 or fp16 x and
 * y, fp32 inside): N images of H x W pixels whose C channels lie together,
 * pixels ldx (ldy) elements apart, images H*W*ldx apart, so that a slice of a
 * wider tensor's channels can be read or written in place.  The C channels
 * form G groups of C/G neighbours; mean and variance (of the values, not of a
 * sample) are taken over a group's H*W*(C/G) values of one image:
 *   y = act((x - mean) / sqrt(var + eps) * gamma[c] + beta[c])
 * gamma, beta: C values of param_type, aligned to their size; NULL: 1 and 0.
 * mean, rstd: N*G fp32 values each, written when not NULL (the backward pass
 * takes them).  y may be x (ldy == ldx).
 * Requirements: H, W, C, G >= 1, N >= 0 (N == 0 is a no-op), C % G == 0, ldx,
 * ldy >= C, eps >= 0, else IGC_ERR_INVALID_VALUE; C % 8 == 0 and the alignment
 * rule, else IGC_ERR_MISALIGNED; H*W < 2^31 and N*C < 2^30, else
 * IGC_ERR_UNSUPPORTED, which is also what a call whose launch would need 2^32
 * threads returns: none with N < 2^25, N*H*W*C < 2^35 and, with dgamma or dbeta,
 * C <= 2^28 - 32.  Workspace: igc_group_norm_workspace_bytes.
 */
igc_status_t group_norm_nhwc_bf16(int N, int H, int W, int C, int G, const void *x, int64_t ldx, const void *gamma,
                                  const void *beta, igc_out_t param_type, float eps, igc_act_t act, void *y,
                                  int64_t ldy, float *mean, float *rstd, igc_stream_t stream);
igc_status_t group_norm_nhwc_fp16(int N, int H, int W, int C, int G, const void *x, int64_t ldx, const void *gamma,
                                  const void *beta, igc_out_t param_type, float eps, igc_act_t act, void *y,
                                  int64_t ldy, float *mean, float *rstd, igc_stream_t stream);
igc_status_t group_norm_nhwc_bf16_ex(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                     const void *gamma, const void *beta, igc_out_t param_type, float eps,
                                     igc_act_t act, void *y, int64_t ldy, float *mean, float *rstd, void *workspace,
                                     int64_t workspace_bytes, igc_stream_t stream);
igc_status_t group_norm_nhwc_fp16_ex(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                     const void *gamma, const void *beta, igc_out_t param_type, float eps,
                                     igc_act_t act, void *y, int64_t ldy, float *mean, float *rstd, void *workspace,
                                     int64_t workspace_bytes, igc_stream_t stream);

/*
 * Gradient of the group norm above, from its x, gamma, beta, act and the mean
 * and rstd that it wrote: with xh = (x - mean) rstd and dz = dy * act'(gamma xh + beta),
 *   dx = rstd (gamma dz - mean(gamma dz) - xh mean(gamma dz xh))     (means over the group)
 *   dgamma[c] = sum dz xh,  dbeta[c] = sum dz      (over every image's pixels; of param_type; either may be NULL)
 * dx may be dy or x (same pixel distance).  N == 0 writes zero dgamma and
 * dbeta.  Requirements and workspace as the forward pass.
 */
igc_status_t group_norm_nhwc_backward_bf16(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                           const void *gamma, const void *beta, igc_out_t param_type,
                                           const float *mean, const float *rstd, igc_act_t act, const void *dy,
                                           int64_t lddy, void *dx, int64_t lddx, void *dgamma, void *dbeta,
                                           igc_stream_t stream);
igc_status_t group_norm_nhwc_backward_fp16(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                           const void *gamma, const void *beta, igc_out_t param_type,
                                           const float *mean, const float *rstd, igc_act_t act, const void *dy,
                                           int64_t lddy, void *dx, int64_t lddx, void *dgamma, void *dbeta,
                                           igc_stream_t stream);
igc_status_t group_norm_nhwc_backward_bf16_ex(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                              const void *gamma, const void *beta, igc_out_t param_type,
                                              const float *mean, const float *rstd, igc_act_t act, const void *dy,
                                              int64_t lddy, void *dx, int64_t lddx, void *dgamma, void *dbeta,
                                              void *workspace, int64_t workspace_bytes, igc_stream_t stream);
igc_status_t group_norm_nhwc_backward_fp16_ex(int N, int H, int W, int C, int G, const void *x, int64_t ldx,
                                              const void *gamma, const void *beta, igc_out_t param_type,
                                              const float *mean, const float *rstd, igc_act_t act, const void *dy,
                                              int64_t lddy, void *dx, int64_t lddx, void *dgamma, void *dbeta,
                                              void *workspace, int64_t workspace_bytes, igc_stream_t stream);

/* Workspace bytes of either direction of the group norm; -1 for bad arguments. */
int64_t igc_group_norm_workspace_bytes(int N, int H, int W, int C, int G);

/*
 * Product of 8-bit integers with scales, and an epilogue:
 *   z[m][n] = scale_a[m] * scale_b[n] * sum_k A[m*lda + k] * B[n*ldb + k] + bias[n]
 *   pre = z (rounded), D = act(z) + residual
 * A is M x K and B N x K, K together in both (row-major A, column-major B of
 * the 16-bit products; the layout of a layer's weights): a row of either stands
 * for its integers times its scale.  scale_a: M, scale_b: N fp32 values,
 * 4-byte aligned; NULL: 1.  The sum is exact whatever the schedule; it is
 * rounded to fp32 once, and once for each scale.  D, the epilogue's tensors and
 * aliasing are as in gemm_bf16_epilogue; epilogue may be NULL (D = z), and
 * backward 1 is IGC_ERR_UNSUPPORTED.  K == 0 leaves z = bias, as 0 * scale does;
 * M == 0 or N == 0 is a no-op.
 * Requirements: lda, ldb >= K and multiples of 16 (the 16-byte rule), sizes,
 * pointers and types as everywhere; K < 2^17 (a longer sum may not fit 32 bits),
 * M and N < 2^31 and a grid of fewer than 2^32 threads, leading dimensions and
 * the rows of one tile spanning less than 2^31 bytes, else IGC_ERR_UNSUPPORTED.
 * Tunes are those of the 16-bit products with IGC_SCOPE_ALL and
 * IGC_SCOPE_EPILOGUE, and two more tiles: 64 x 64 x 64 of depth 5 (8 waves, 4 of
 * them loading) and 32 x 64 x 64 of depth 5 (4 waves); a K tile of bk holds 2*bk
 * values; stream-K is
 * IGC_ERR_UNSUPPORTED.  The parts of a K split are int32 in the workspace, of
 * igc_gemm_int8_workspace_bytes (-1 for sizes or a tune that the call refuses).
 * igc_gemm_int8_default_tune tells the built-in choice as
 * igc_epilogue_default_tune does (bm = 0: the kernel of few rows), k_splits the
 * parts that run, as whole ring periods may make them fewer than a tune asks for.
 */
igc_status_t gemm_int8(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a,
                       const int8_t *B, int64_t ldb, const float *scale_b, void *D, int64_t ldd, igc_out_t d_type,
                       const igc_epilogue_t *epilogue, igc_stream_t stream);
igc_status_t gemm_int8_ex(int64_t M, int64_t N, int64_t K, const int8_t *A, int64_t lda, const float *scale_a,
                          const int8_t *B, int64_t ldb, const float *scale_b, void *D, int64_t ldd, igc_out_t d_type,
                          const igc_epilogue_t *epilogue, const igc_tune_t *tune, void *workspace,
                          int64_t workspace_bytes, igc_stream_t stream);
int64_t igc_gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K, const igc_tune_t *tune);
int igc_gemm_int8_default_tune(int64_t M, int64_t N, int64_t K, igc_tune_t *out);

/*
 * Root-mean-square norm of M rows of C values (bf16 or fp16), with the
 * addition of a residual before it:
 *   h = x + residual, rounded to their type;  rstd[m] = 1 / sqrt(mean_c h^2 + eps)
 *   y = h * rstd[m] * gamma[c]     (rounded once)
 * h is what is normed, so a later call, or the gradient, from the stored h sees
 * the same numbers.  residual NULL: h = x.  h (the residual stream's new value)
 * is written when not NULL; rstd likewise (M fp32 values, which the gradient
 * takes).  gamma: C values of param_type, aligned to their size; NULL: 1.
 *   rms_norm_int8_*: y goes to 8 bits instead, for gemm_int8's A:
 *   scale[m] = max_c |y| / 127,  q = y / scale to the nearest integer, ties to
 *   even, so that q * scale stands for y (rstd cancels in q: it is taken of
 *   h * gamma in fp32, rounded to fp32 once before it is to an integer).  A row of zeros has scale 0 and zeros;
 *   a row with an infinity or a NaN, its own or of h * gamma, has scale NaN and
 *   zeros, and so gives NaN in the product: h * gamma has to fit fp32, and loses
 *   bits below 2^-126, as scales do.
 * h may be x or residual, and y may be x or residual if h is not the same one
 * (same leading dimension): a row's values are read before they are written.
 * A row's mean square need not fit fp32 (bf16's squares do not from 2^64 on, or
 * below 2^-63), only rstd: beyond 2^126 a root mean square leaves rstd few bits,
 * and with eps 0 one below 2^-128 makes it infinite.  With eps 0 a row of zeros
 * has rstd infinite and gives NaN (y, and the scale with zeros), as the formula does.
 * Requirements: M >= 0 (0 is a no-op), C >= 1, leading dimensions >= C, eps >= 0,
 * else IGC_ERR_INVALID_VALUE; the alignment rule (q: ldq a multiple of 16), any C;
 * M and C < 2^30, leading dimensions < 2^32 and fewer than 2^32 threads (M < 2^22
 * holds for every C), else IGC_ERR_UNSUPPORTED.  No workspace.
 */
igc_status_t rms_norm_bf16(int64_t M, int64_t C, const void *x, int64_t ldx, const void *residual, int64_t ldr, void *h,
                           int64_t ldh, const void *gamma, igc_out_t param_type, float eps, void *y, int64_t ldy,
                           float *rstd, igc_stream_t stream);
igc_status_t rms_norm_fp16(int64_t M, int64_t C, const void *x, int64_t ldx, const void *residual, int64_t ldr, void *h,
                           int64_t ldh, const void *gamma, igc_out_t param_type, float eps, void *y, int64_t ldy,
                           float *rstd, igc_stream_t stream);
igc_status_t rms_norm_int8_bf16(int64_t M, int64_t C, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                void *h, int64_t ldh, const void *gamma, igc_out_t param_type, float eps, int8_t *q,
                                int64_t ldq, float *scale, igc_stream_t stream);
igc_status_t rms_norm_int8_fp16(int64_t M, int64_t C, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                                void *h, int64_t ldh, const void *gamma, igc_out_t param_type, float eps, int8_t *q,
                                int64_t ldq, float *scale, igc_stream_t stream);

/*
 * Gradient of the norm above, from its h (x where there was no residual),
 * gamma and rstd.  With g = dy * gamma and xh = h * rstd[m]:
 *   dx = rstd[m] * (g - xh * mean_c(g * xh)) + dh     (rounded once)
 *   dgamma[c] = sum_m dy * xh     (summed in fp32, rounded once to param_type)
 * dh is the gradient that reaches h itself, past the norm (NULL: none).  dx is
 * the gradient of x and of residual alike.  dgamma NULL: not computed.  dx may be
 * dy, dh or h (same leading dimension).  M == 0 writes dgamma = 0.  The mean is of
 * dy * gamma * h, which has to fit fp32, its sum over a row too, and loses bits below 2^-126.
 * Requirements as the norm's, but that the grid is small for every M, and
 * dgamma takes C < 2^27.  Workspace when dgamma is given:
 * igc_rms_norm_backward_workspace_bytes (-1 for bad or refused sizes).
 */
igc_status_t rms_norm_backward_bf16(int64_t M, int64_t C, const void *h, int64_t ldh, const void *gamma,
                                    igc_out_t param_type, const float *rstd, const void *dy, int64_t lddy,
                                    const void *dh, int64_t lddh, void *dx, int64_t lddx, void *dgamma,
                                    igc_stream_t stream);
igc_status_t rms_norm_backward_fp16(int64_t M, int64_t C, const void *h, int64_t ldh, const void *gamma,
                                    igc_out_t param_type, const float *rstd, const void *dy, int64_t lddy,
                                    const void *dh, int64_t lddh, void *dx, int64_t lddx, void *dgamma,
                                    igc_stream_t stream);
igc_status_t rms_norm_backward_bf16_ex(int64_t M, int64_t C, const void *h, int64_t ldh, const void *gamma,
                                       igc_out_t param_type, const float *rstd, const void *dy, int64_t lddy,
                                       const void *dh, int64_t lddh, void *dx, int64_t lddx, void *dgamma,
                                       void *workspace, int64_t workspace_bytes, igc_stream_t stream);
igc_status_t rms_norm_backward_fp16_ex(int64_t M, int64_t C, const void *h, int64_t ldh, const void *gamma,
                                       igc_out_t param_type, const float *rstd, const void *dy, int64_t lddy,
                                       const void *dh, int64_t lddh, void *dx, int64_t lddx, void *dgamma,
                                       void *workspace, int64_t workspace_bytes, igc_stream_t stream);
int64_t igc_rms_norm_backward_workspace_bytes(int64_t M, int64_t C);

/*
 * Rows of an activation to 8 bits, the A of a following gemm_int8: with
 * v = act(x) * gate (gate NULL: act(x)), M rows of C values,
 *   scale[m] = max_c |v| / 127,  q = v / scale to the nearest integer, ties to even.
 * v is taken in fp32.  Rows of zeros, infinities, NaN and tiny values as in
 * rms_norm_int8_*, but that the scale of a row with an infinity (and no NaN) is
 * infinite.  x and gate of one type; a gate beside x in the same rows (x's columns
 * C and up) begins at a 16-byte multiple.  Requirements as the norm's.
 */
igc_status_t quantize_rows_int8_bf16(int64_t M, int64_t C, igc_act_t act, const void *x, int64_t ldx, const void *gate,
                                     int64_t ldg, int8_t *q, int64_t ldq, float *scale, igc_stream_t stream);
igc_status_t quantize_rows_int8_fp16(int64_t M, int64_t C, igc_act_t act, const void *x, int64_t ldx, const void *gate,
                                     int64_t ldg, int8_t *q, int64_t ldq, float *scale, igc_stream_t stream);

/* Workspace bytes a call needs for operation `op` with GEMM view M x N x K
 * (see each operation above) under `tune` (NULL: the built-in choice): 0 when
 * the schedule does not split K.  Returns -1 for negative sizes, a bad op or
 * an invalid tune. */
int64_t igc_workspace_bytes(igc_op_t op, int64_t M, int64_t N, int64_t K, const igc_tune_t *tune);

/* 1 if (bm, bn, bk, pipe_depth, waves, mfma, half_stage, loader_waves, ring_sync) is a compiled
 * configuration (for the bf16 GEMM with row-major A at least), else 0. */
int igc_tune_supported(const igc_tune_t *tune);

/* The configuration the library picks for operation `op` with GEMM view
 * M x N x K when no tune is given; 1 on success. */
int igc_default_tune(igc_op_t op, int64_t M, int64_t N, int64_t K, igc_tune_t *out);

/* Number of compiled configurations; igc_tune_get(i, &t) fills t for i in [0, count).
 * igc_tune_scope(i) is a bit mask of what configuration i is built for: IGC_SCOPE_ALL (every input type,
 * operand layout, operation and loop variant; without it only the bf16 and fp16 GEMM with row-major A and
 * K % 8 == 0, and the bf16 forward convolution with whole filter taps per K tile and filters of at most
 * 16 x 16 -- other calls are IGC_ERR_UNSUPPORTED), IGC_SCOPE_STREAM_K (stream-K schedules; without it
 * a tune with stream_k > 0 is IGC_ERR_UNSUPPORTED) and IGC_SCOPE_CONV_FPROP (the bf16 and fp16 forward
 * convolution with every loop variant, besides the GEMMs with row-major A) and IGC_SCOPE_EPILOGUE (the fused
 * epilogue of the forward convolution, and with IGC_SCOPE_ALL of the GEMMs); 0 for an index out of range. */
enum { IGC_SCOPE_ALL = 1, IGC_SCOPE_STREAM_K = 2, IGC_SCOPE_CONV_FPROP = 4, IGC_SCOPE_EPILOGUE = 8 };
int igc_tune_count(void);
int igc_tune_get(int i, igc_tune_t *out);
int igc_tune_scope(int i);

/* LDS bytes one workgroup of the given configuration uses (0 if not compiled). */
int64_t igc_tune_lds_bytes(const igc_tune_t *tune);

/* Static text for a status code (never NULL). */
const char *igc_status_string(igc_status_t status);

/* Reads the current device's error word into *word (0: no stream-K wait has
 * given up since the last call) and clears it.  Synchronous: it waits for the
 * device's outstanding work.  IGC_ERR_INVALID_VALUE for NULL, IGC_ERR_HIP if
 * the copy fails. */
igc_status_t igc_take_device_error(int *word);

/* Test hook: for later stream-K launches in this process, poll a partial's
 * flag at most `spin_limit` times (<= 0: the built-in bound, about a second of
 * polling) and never raise the flag of workgroup `drop_workgroup` (-1: raise
 * all).  Lets a test make the bounded wait give up while every kernel still
 * exits normally. */
void igc_debug_stream_k(int spin_limit, int drop_workgroup);

/* Number of workspaces the library has taken from its own pool in this
 * process (a call given a workspace, or needing none, adds nothing). */
int64_t igc_pool_allocations(void);

/*
 * Ring schedule of the mainloop, for inspection and testing on the host.
 * The LDS ring holds U = 2*pipe_depth + half_stage operand slots; the K loop
 * consumes units, unit 2t being the A tile and unit 2t+1 the B tile of K tile
 * t, and unit s always lives in slot s % U.  For a K loop of `k_tiles` tiles,
 * writes up to `cap` events into `events` as int quadruples
 * (kind, tile, operand, x):
 *   kind 0 = issue the loads of operand `operand` (0: A, 1: B) of `tile` into
 *            slot x,
 *   kind 1 = wait until both operands of `tile` have landed (each wave waits
 *            on its own loads, then the workgroup barrier runs); x is how many
 *            newer units the wave's s_waitcnt vmcnt lets stay in flight
 *            (operand is -1),
 *   kind 2 = read operand `operand` of `tile` from slot x (fragment loads,
 *            then MFMAs),
 *   kind 3 = workgroup barrier only (pipe_depth 1 frees its single stage with
 *            it; every schedule ends with one once nothing is left in flight).
 * Rings of up to four slots pad the K loop to a whole number of ring periods
 * (U/2 tiles; no padding for pipe_depth 1) with tiles whose loads are all out
 * of range: they land as zeros and add nothing, so tiles up to that padded
 * count appear.  Rings of five or more slots run exactly k_tiles tiles: they
 * issue units 0..U-3 up front and, during each tile t, units 2t+U-2 and
 * 2t+U-1 (interleaved with t's MFMAs) into the two slots the last barrier
 * freed; units past k_tiles are issued out of range and never read.  Two-stage rings issue tile
 * t+2 right after the barrier that frees tile t.  Each wave drains its own
 * LDS reads before every barrier, so a barrier after a unit's reads frees its
 * slot.  (With ring_sync 1 the barrier of a wait event is replaced by the
 * slot's ready counter, and a slot is refilled once its free counter shows
 * every wave done with it; the order of issues, waits and reads is the same.)
 * Returns the number of events (which may exceed cap), or -1 on bad input
 * (pipe_depth outside 1..8, half_stage not 0/1 or with pipe_depth 1, negative
 * k_tiles or cap).  The kernels' loops are written to follow this sequence;
 * the GPU tests' K-chain tags check that they do.
 */
int igc_ring_schedule(int pipe_depth, int half_stage, int k_tiles, int *events, int cap);

/*
 * LDS swizzle of the operand tiles, for inspection and testing on the host.
 * Operand tiles live in LDS as rows of 16-byte chunks; the chunk holding
 * logical chunk `logical_chunk` of row `row` is stored at the returned
 * physical chunk of the same row.  k_contiguous = 1: rows of the K tile
 * (chunks_per_row = BK/8, 8 or 4); 0: rows of BM or BN elements read with the
 * transposing LDS load (chunks_per_row 8 or a multiple of 16).  Returns -1 for an
 * unsupported geometry.  These are the maps the kernels use.
 */
int igc_lds_chunk(int k_contiguous, int chunks_per_row, int row, int logical_chunk);

/*
 * LDS swizzle of the output epilogue's staged rows, for inspection and
 * testing on the host.  A wave stages its 16-bit output sub-tile in LDS as
 * rows of slots_per_row 8-byte slots (16: 128-byte rows, 32: 256-byte rows);
 * logical slot `slot` of row `row` is stored at the returned physical slot of
 * the same row.  Returns -1 for a negative row, a slot outside the row or
 * another row width.  This is the map the kernels use.
 */
int igc_stage_slot(int row, int slot, int slots_per_row);

#ifdef __cplusplus
}
#endif

#endif /* IGC_H */
