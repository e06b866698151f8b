/*
 * conv_fwd.h -- C ABI of libconvfwd.so, a convolution forward engine for one
 * AMD Instinct MI355X (gfx950).
 *
 * What it computes.  For a 2D convolution with one square kernel size K, one
 * stride s and one symmetric zero pad p (page "Hand-writing Conv2D", 1.1-1.2):
 *
 *     y[n][oc][oh][ow] = bias[oc] + sum_{ic, kh, kw}
 *                        x[n][ic][oh*s + kh - p][ow*s + kw - p] * w[oc][ic][kh][kw]
 *
 * where a tap whose input coordinate falls outside the input contributes 0
 * (zero padding by bounds checks, no padded copy).  The output size per
 * spatial dimension is  out = floor((in + 2p - K)/s) + 1  (same section).
 * The engine evaluates it as the product  W_row (C_out x C_in*K*K) @ X_col
 * (C_in*K*K x N*H_out*W_out)  of the page "Why use matrix multiplication for
 * convolution", 2.2-2.3, either with X_col materialised in device memory
 * (the *_explicit and *_im2col entry points) or gathered tile by tile inside
 * the GEMM kernel and never stored (implicit GEMM, same page, 4.3).  The 3D
 * form adds a depth dimension with the same K, s, p (page "PyTorch tensor
 * products and conv2d/conv3d dimension semantics", 5.1-5.2).
 *
 * Conventions for every entry point below:
 *   Layout     x is dense NCHW (2D) or NCDHW (3D); w is dense OIHW / OIDHW,
 *              i.e. (C_out, C_in, K, K[, K]); bias is (C_out); y is dense
 *              N C_out H_out W_out (or N C_out D_out H_out W_out).  Strided
 *              views are not accepted: pass contiguous buffers.
 *   Types      "bf16" pointers hold raw bfloat16 bit patterns (uint16_t).
 *              The output is always fp32; accumulation is fp32; bias is fp32.
 *   Memory     every tensor pointer is a DEVICE pointer owned by the caller.
 *              The library allocates nothing, frees nothing and keeps no
 *              pointer after the call returns (conv2d_fwd_bf16_noalloc uses
 *              a fixed array of its own instead of a workspace; see there).
 *   Streams    `stream` is a hipStream_t (NULL = the null stream).  Work is
 *              enqueued on it and the call returns before the work finishes;
 *              the caller synchronises.  Calls on one stream run in order.
 *   Errors     arguments are validated on the host BEFORE any HIP call; on a
 *              validation error nothing is launched and y is not written.  A
 *              status other than CONV_OK is returned, never an exit or abort.
 *              CONV_ERR_HIP reports a failed launch (the HIP error is then
 *              also left in the runtime's last-error slot).
 *   Limits     each tensor (x, w, y, X_col) must hold fewer than 2^31
 *              elements; N, C_in, C_out, spatial sizes and K >= 1; stride >= 1;
 *              pad >= 0; every padded input extent must be >= K.
 *   Aliasing   y must not overlap x, w, bias (or the workspace).
 */
#ifndef CONV_FWD_H
#define CONV_FWD_H

#include <stddef.h>
#include <stdint.h>

/* Only the functions below are exported from the shared library. */
#define CONV_API __attribute__((visibility("default")))

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CONV_OK = 0,
    CONV_ERR_NULL = 1,       /* a required pointer (x, w, y, workspace) is NULL            */
    CONV_ERR_PARAM = 2,      /* a size < 1, K < 1, stride < 1, pad < 0 (or, for the general
                                entry points, dilation < 1 or groups not dividing C_in, C_out) */
    CONV_ERR_SHAPE = 3,      /* in + 2*pad < K in some spatial dimension (no output)        */
    CONV_ERR_OVERFLOW = 4,   /* a tensor would hold 2^31 or more elements                   */
    CONV_ERR_ALIAS = 5,      /* y overlaps x, w, bias or the workspace                      */
    CONV_ERR_WORKSPACE = 6,  /* workspace smaller than conv*_im2col_bytes() requires        */
    CONV_ERR_ALGO = 7,       /* the requested algorithm does not exist for this dtype/shape */
    CONV_ERR_HIP = 8,        /* a HIP launch failed                                         */
    CONV_ERR_SCRATCH = 9     /* conv2d_fwd_bf16_noalloc: the problem needs more than
                                CONV_STATIC_SCRATCH_BYTES of scratch                        */
} conv_status_t;

/* Kernel route.  AUTO picks by shape, for bf16: first the matrix cores'
 * short-reduction kernel when C_in/groups*K^dims <= 128 and one output row's
 * input patch fits its LDS tile (this takes the thin stem layer, 3 channels x
 * 3x3, and the 3-channel 3D layer); else one input channel per group in 2D
 * (depthwise) -> the VALU depthwise kernel; else a reduction of at most 32
 * (C_in/groups*K^dims) -> the VALU direct kernel; else the MFMA implicit
 * GEMM.  fp32 -> VALU.  MFMA is bf16-only (CONV_ERR_ALGO for fp32).
 * CONV_ALGO_VALU forces the direct FMA route for any bf16 shape. */
typedef enum {
    CONV_ALGO_AUTO = 0,
    CONV_ALGO_MFMA = 1,      /* implicit GEMM on bf16 matrix cores, fp32 accumulate */
    CONV_ALGO_VALU = 2,      /* direct convolution, fp32 FMA on the vector ALUs       */
    CONV_ALGO_WINOGRAD = 3   /* Winograd F(2x2,3x3) ("Why use matrix multiplication for
                                convolution", 5.1): conv_fwd_ex_bf16 only, with a
                                workspace; 3x3, stride 1, dilation 1, groups 1, NCHW,
                                C_in % 16 == 0.  Never chosen by AUTO.  The transformed
                                operands are fp16: x and w are first scaled by powers of
                                two chosen from max|x| and max|w| (one pass over both), so
                                any finite bf16 data fits; elements more than ~2^27 below
                                their tensor's largest magnitude lose precision (fp16
                                subnormals), which the 1e-3 * sum|x w| bound absorbs. */
} conv_algo_t;

/* floor((in + 2*pad - K)/stride) + 1, or -1 if in < 1, K < 1, stride < 1,
 * pad < 0 or in + 2*pad < K ("Hand-writing Conv2D", 1.1; the explicit reject
 * of a negative numerator follows "Conv2d from the official docs", 3.2, which
 * warns that C division truncates rather than floors for negatives). */
CONV_API int64_t conv_out_dim(int64_t in, int64_t K, int64_t stride, int64_t pad);

/* Static, NUL-terminated text for a status code; never NULL. */
CONV_API const char *conv_status_str(int status);

/* Library version as major*10000 + minor*100 + patch. */
CONV_API int conv_version(void);

/* ---- direct entry points: y = conv(x, w) + bias ------------------------- */

/* 2D, bf16 inputs and weights, fp32 bias (NULL = no bias) and output.
 * Shapes: x (N, C_in, H, W), w (C_out, C_in, K, K), y (N, C_out, H_out, W_out). */
CONV_API conv_status_t conv2d_fwd_bf16(const uint16_t *x, const uint16_t *w, const float *bias, float *y,
                              int N, int C_in, int H, int W, int C_out,
                              int K, int stride, int pad, int algo, void *stream);

/* 2D, fp32 everywhere (VALU route only).  Same shapes. */
CONV_API conv_status_t conv2d_fwd_f32(const float *x, const float *w, const float *bias, float *y,
                             int N, int C_in, int H, int W, int C_out,
                             int K, int stride, int pad, int algo, void *stream);

/* 3D, bf16 inputs: x (N, C_in, D, H, W), w (C_out, C_in, K, K, K),
 * y (N, C_out, D_out, H_out, W_out). */
CONV_API conv_status_t conv3d_fwd_bf16(const uint16_t *x, const uint16_t *w, const float *bias, float *y,
                              int N, int C_in, int D, int H, int W, int C_out,
                              int K, int stride, int pad, int algo, void *stream);

/* 3D, fp32 everywhere (VALU route only). */
CONV_API conv_status_t conv3d_fwd_f32(const float *x, const float *w, const float *bias, float *y,
                             int N, int C_in, int D, int H, int W, int C_out,
                             int K, int stride, int pad, int algo, void *stream);

/* ---- with a workspace --------------------------------------------------- */

/* Bytes of device workspace conv2d_fwd_bf16_ws can use for these arguments:
 * the 3x3 stride-1 pad-1 MFMA kernels (C_in % 16 == 0, C_out % 128 == 0,
 * W % 8 == 0, and 32 <= W <= 64, or C_in >= 32 and 8 <= W <= 64) repack the
 * weights once per call into C_out*C_in*9*2 bytes laid out as per-stage LDS
 * images, so that they stream them with coalesced direct-to-LDS loads
 * instead of transposing OIHW in every workgroup.  0 when no route uses a
 * workspace. */
CONV_API size_t conv2d_fwd_workspace_bytes(int N, int C_in, int H, int W, int C_out,
                                           int K, int stride, int pad, int algo);

/* conv2d_fwd_bf16 plus a caller-owned device workspace (16-byte aligned, at
 * least conv2d_fwd_workspace_bytes() bytes; may be NULL when that is 0).  The
 * workspace is overwritten; the result equals conv2d_fwd_bf16's.  Returns
 * CONV_ERR_WORKSPACE if it is needed and missing, too small or misaligned,
 * CONV_ERR_ALIAS if it overlaps x, w or y.  Two calls in flight at once must
 * not share a workspace. */
CONV_API conv_status_t conv2d_fwd_bf16_ws(const uint16_t *x, const uint16_t *w, const float *bias,
                                          float *y, void *workspace, size_t workspace_bytes,
                                          int N, int C_in, int H, int W, int C_out,
                                          int K, int stride, int pad, int algo, void *stream);

/* The two halves of conv2d_fwd_bf16_ws, for callers whose weights do not
 * change between calls (the weight view W_row of "Why use matrix
 * multiplication for convolution", 2.2, prepared once): */

/* Writes the packed weights for these arguments into the workspace (16-byte
 * aligned, >= conv2d_fwd_workspace_bytes() bytes) on `stream`.  w: OIHW bf16,
 * 16-byte aligned.  Returns CONV_ERR_ALGO when no route of these arguments
 * uses packed weights (conv2d_fwd_workspace_bytes() == 0) or w is not 16-byte
 * aligned, CONV_ERR_WORKSPACE if the workspace is too small or misaligned,
 * CONV_ERR_ALIAS if it overlaps w. */
CONV_API conv_status_t conv2d_pack_weights_bf16(const uint16_t *w, void *workspace, size_t workspace_bytes,
                                                int N, int C_in, int H, int W, int C_out,
                                                int K, int stride, int pad, int algo, void *stream);

/* conv2d_fwd_bf16 with the weights taken from a workspace that
 * conv2d_pack_weights_bf16 filled for the same sizes and algo (the weight
 * tensor itself is not read).  Same result as conv2d_fwd_bf16_ws.  The
 * workspace is only read, so concurrent calls may share it.  Errors as
 * conv2d_fwd_bf16_ws, plus CONV_ERR_ALGO when these arguments have no
 * packed-weight route. */
CONV_API conv_status_t conv2d_fwd_bf16_prepacked(const uint16_t *x, const void *workspace,
                                                 size_t workspace_bytes, const float *bias, float *y,
                                                 int N, int C_in, int H, int W, int C_out,
                                                 int K, int stride, int pad, int algo, void *stream);

/* ---- without allocation ------------------------------------------------- */

/* Size of the library's own device scratch array (one per GPU, kept until
 * the process ends), used by conv2d_fwd_bf16_noalloc. */
#define CONV_STATIC_SCRATCH_BYTES ((size_t)8 << 20)

/* For callers that cannot allocate device memory (code under stream or graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * computation and result as conv2d_fwd_bf16_ws, with the workspace taken from
 * a file-scope device array of CONV_STATIC_SCRATCH_BYTES inside the library
 * instead of from the caller.  No hipMalloc, hipFree or other allocating call
 * is made.  The array's address on the current device is looked up on the
 * first call on that device.  Arguments, layouts, ownership and errors as
 * conv2d_fwd_bf16_ws (minus the workspace pair), plus CONV_ERR_SCRATCH, before
 * any launch, when conv2d_fwd_workspace_bytes() of these arguments exceeds
 * CONV_STATIC_SCRATCH_BYTES (3x3 layers with C_out*C_in*9*2 > 8 MiB, e.g.
 * C_in = C_out = 1024), and CONV_ERR_HIP if the address lookup fails.  All
 * calls on one GPU share its one array and every call overwrites it (nothing
 * in it needs to start at zero): two calls that can run at the same time on
 * one GPU (different streams, or different host threads) race and may give
 * wrong results; serialise them, e.g. on one stream. */
CONV_API conv_status_t conv2d_fwd_bf16_noalloc(const uint16_t *x, const uint16_t *w, const float *bias,
                                               float *y, int N, int C_in, int H, int W, int C_out,
                                               int K, int stride, int pad, int algo, void *stream);

/* ---- explicit im2col path ("Why use matrix multiplication for convolution",
 *      2.2 and 3.1): X_col is materialised in caller-owned device memory. ---- */

/* Bytes of the bf16 X_col matrix, (C_in*K*K) x (N*H_out*W_out) elements, for
 * these arguments; 0 if the arguments are invalid or X_col would hold 2^31 or
 * more elements.  D = 1 and the 2D formula apply when ndim == 2. */
CONV_API size_t conv_im2col_bytes(int ndim, int N, int C_in, int D, int H, int W,
                         int K, int stride, int pad);

/* X_col[r][j] = x[n][ic][oh*s+kh-p][ow*s+kw-p] (0 outside the input), with
 * row r = (ic*K + kh)*K + kw and column j = (n*H_out + oh)*W_out + ow, stored
 * row-major as bf16 into xcol (which must hold conv_im2col_bytes() bytes).
 * The copy is exact (bit for bit). */
CONV_API conv_status_t conv2d_im2col_bf16(const uint16_t *x, uint16_t *xcol,
                                 int N, int C_in, int H, int W,
                                 int K, int stride, int pad, void *stream);

/* 3D twin: row r = ((ic*K + kd)*K + kh)*K + kw, column
 * j = ((n*D_out + od)*H_out + oh)*W_out + ow. */
CONV_API conv_status_t conv3d_im2col_bf16(const uint16_t *x, uint16_t *xcol,
                                 int N, int C_in, int D, int H, int W,
                                 int K, int stride, int pad, void *stream);

/* im2col into `workspace`, then one MFMA GEMM  W_row @ X_col  whose epilogue
 * adds bias and writes y directly in N C_out H_out W_out order (the reshape and
 * axis swap of "Why use matrix multiplication for convolution", 3.2, fused
 * into the store).  workspace: device memory of at least
 * conv_im2col_bytes(2, ...) bytes, owned by the caller, clobbered. */
CONV_API conv_status_t conv2d_fwd_bf16_explicit(const uint16_t *x, const uint16_t *w, const float *bias,
                                       float *y, void *workspace, size_t workspace_bytes,
                                       int N, int C_in, int H, int W, int C_out,
                                       int K, int stride, int pad, void *stream);

/* 3D twin of conv2d_fwd_bf16_explicit; workspace of conv_im2col_bytes(3, ...). */
CONV_API conv_status_t conv3d_fwd_bf16_explicit(const uint16_t *x, const uint16_t *w, const float *bias,
                                       float *y, void *workspace, size_t workspace_bytes,
                                       int N, int C_in, int D, int H, int W, int C_out,
                                       int K, int stride, int pad, void *stream);

/* ---- general problems: dilation and groups -------------------------------
 *
 * Dilation d places the K taps of a window d inputs apart, so a window spans
 * d(K-1)+1 inputs and  out = floor((in + 2*pad - d(K-1) - 1)/stride) + 1
 * ("PyTorch tensor products and conv2d/conv3d dimension semantics", 4.2;
 * "Conv2d from the official docs", 3.2-3.3).  Groups G cut C_in and C_out into
 * G equal consecutive blocks; output block g reads input block g only, and the
 * weight holds C_in/G input channels per filter (same pages, 4.3 and 3.4).
 * G == C_in is the depthwise layer.  With g = oc / (C_out/G):
 *
 *     y[n][oc][oh][ow] = bias[oc] + sum_{j < C_in/G, kh, kw}
 *         x[n][g*C_in/G + j][oh*s + kh*d - p][ow*s + kw*d - p] * w[oc][j][kh][kw]
 *
 * (3D adds od*s + kd*d - p on the depth axis).  Taps outside the input add 0.
 * Layouts as above, except w is (C_out, C_in/G, K, K[, K]).  With d = 1 and
 * G = 1 every entry point below computes exactly what its conv2d_/conv3d_
 * counterpart computes.  Extra errors: CONV_ERR_PARAM when dilation < 1,
 * groups < 1, groups does not divide C_in and C_out, or ndim is not 2 or 3;
 * CONV_ERR_NULL when the parameter block is NULL. */
typedef struct {
    int ndim;        /* 2 or 3                                                  */
    int N, C_in;
    int D;           /* input depth; ignored (taken as 1) when ndim == 2         */
    int H, W;
    int C_out;
    int K;           /* kernel extent, the same in every spatial dimension       */
    int stride, pad; /* the same in every spatial dimension                      */
    int dilation;    /* >= 1                                                     */
    int groups;      /* >= 1, divides C_in and C_out                             */
} conv_params_t;

/* floor((in + 2*pad - dilation*(K-1) - 1)/stride) + 1, or -1 on a bad
 * parameter or when the dilated window does not fit in the padded input. */
CONV_API int64_t conv_out_dim_dilated(int64_t in, int64_t K, int64_t stride, int64_t pad, int64_t dilation);

/* y = conv(x, w) + bias for a general problem, bf16 x and w, fp32 bias (NULL =
 * none) and y.  AUTO: one input channel per group (C_in/G == 1, 2D) -> the
 * depthwise VALU kernel, which reads each input once and writes each output
 * once; a per-group reduction (C_in/G * K^ndim) <= 32 -> the direct VALU
 * kernel; otherwise the MFMA implicit GEMM, one GEMM of C_out/G x
 * (C_in/G * K^ndim) per group.  It takes no workspace: the 3x3 kernels that
 * read packed weights (dilation 1 or 2 with pad = dilation, or groups of 32
 * output channels) are reached through conv_fwd_ex_bf16 with a workspace. */
CONV_API conv_status_t conv_fwd_bf16(const conv_params_t *params, const uint16_t *x, const uint16_t *w,
                                     const float *bias, float *y, int algo, void *stream);

/* fp32 twin (VALU route only). */
CONV_API conv_status_t conv_fwd_f32(const conv_params_t *params, const float *x, const float *w,
                                    const float *bias, float *y, int algo, void *stream);

/* Bytes of the bf16 X_col of a general problem: C_in*K^ndim rows (groups do
 * not change X_col; group g uses rows [g, g+1) * C_in/G * K^ndim) by
 * N * (output positions) columns; 0 on invalid parameters or when X_col would
 * hold 2^31 or more elements. */
CONV_API size_t conv_xcol_bytes(const conv_params_t *params);

/* X_col of a general problem: row ((ic*K + kd)*K + kh)*K + kw (kd absent in
 * 2D), column in output order, entry x at the dilated tap coordinate, 0
 * outside.  xcol must hold conv_xcol_bytes() bytes.  Exact copy. */
CONV_API conv_status_t conv_im2col_bf16(const conv_params_t *params, const uint16_t *x, uint16_t *xcol,
                                        void *stream);

/* conv_im2col_bf16 into the workspace (>= conv_xcol_bytes() bytes), then per
 * group g the GEMM W_row[g] (C_out/G x C_in/G*K^ndim) @ X_col[rows of g] with
 * bias, stored into y in N C_out (D) H W order. */
CONV_API conv_status_t conv_fwd_explicit_bf16(const conv_params_t *params, const uint16_t *x,
                                              const uint16_t *w, const float *bias, float *y,
                                              void *workspace, size_t workspace_bytes, void *stream);

/* ---- options: channels-last layout, ReLU, bf16 output ---------------------
 *
 * layout CONV_LAYOUT_NHWC: x is (N, [D,] H, W, C_in) and y is (N, [D_out,]
 * H_out, W_out, C_out), the channel index fastest (channels_last, "PyTorch
 * tensor products and conv2d/conv3d dimension semantics", 6.3); w stays
 * (C_out, C_in/G, K, K[, K]).  relu = 1: y = max(y, 0) after the bias (the
 * activation that follows the convolution in the same page, 6.2).
 * out_dtype CONV_OUT_BF16: y holds bf16 bits, the fp32 result rounded to the
 * nearest bf16, ties to even; accumulation stays fp32.  A NULL options
 * pointer means NCHW, fp32, no ReLU. */
typedef enum { CONV_LAYOUT_NCHW = 0, CONV_LAYOUT_NHWC = 1 } conv_layout_t;
typedef enum { CONV_OUT_F32 = 0, CONV_OUT_BF16 = 1 } conv_out_t;
typedef struct {
    int layout;      /* conv_layout_t, for x and y                  */
    int out_dtype;   /* conv_out_t                                   */
    int relu;        /* 0 or 1                                       */
} conv_options_t;

/* Workspace conv_fwd_ex_bf16 can use (C_out x C_in/G x 9 bf16: the packed
 * weights of the 3x3 column-group kernels, for 3x3 stride-1 layers with
 * dilation 1 or 2 and pad = dilation, or with groups of 32 output channels
 * (NCHW, dilation 1); any epilogue, and channels-last for groups 1) or, with
 * algo CONV_ALGO_WINOGRAD, needs
 * (the fp16 transformed weights, 16 x C_out x C_in, and transformed input
 * blocks, 16 x N*ceil(H_out/2)*ceil(W_out/2) x C_in rounded up to a multiple
 * of 32); 0 when none, or on
 * invalid arguments or a shape Winograd does not take. */
CONV_API size_t conv_fwd_ex_workspace_bytes(const conv_params_t *params, const conv_options_t *opts, int algo);

/* conv_fwd_bf16 with options.  y is float* (fp32) or uint16_t* (bf16 bits)
 * as out_dtype says.  workspace: NULL, or 16-byte aligned (256-byte aligned
 * with Winograd) device memory of at least conv_fwd_ex_workspace_bytes()
 * bytes (overwritten).  Kernels that
 * do not take an option step aside for the general ones: channels-last runs
 * on the 3x3 column-group kernel (groups 1), a channels-last pointwise
 * kernel, and otherwise the general implicit GEMM and the direct VALU kernel;
 * the 3x3, pointwise and depthwise kernels apply ReLU and bf16 output in
 * their own epilogue.
 * algo CONV_ALGO_WINOGRAD computes U = G g G^T and V = B^T d B in fp16, the
 * 16 transform-point GEMMs on the matrix cores with fp32 accumulation, and
 * A^T M A per 2x2 block; its error scale is the transform-domain magnitude
 * sum, up to ~4x the direct one on N(0,1) data (the page's low-precision
 * caveat).  Extra errors: CONV_ERR_PARAM for an unknown layout, out_dtype or
 * relu value; CONV_ERR_WORKSPACE as for conv2d_fwd_bf16_ws (required with
 * Winograd); CONV_ERR_ALGO when Winograd does not take the shape. */
CONV_API conv_status_t conv_fwd_ex_bf16(const conv_params_t *params, const conv_options_t *opts, const uint16_t *x,
                                        const uint16_t *w, const float *bias, void *y, void *workspace,
                                        size_t workspace_bytes, int algo, void *stream);

/* fp32 twin (VALU route). */
CONV_API conv_status_t conv_fwd_ex_f32(const conv_params_t *params, const conv_options_t *opts, const float *x,
                                       const float *w, const float *bias, void *y, int algo, void *stream);

/* ---- backward: gradients of y = conv(x, w) + b ----------------------------
 *
 * With upstream gradient dout (the shape of y) ("Hand-writing Conv2D", 5.1;
 * "Why use matrix multiplication for convolution", 3.3):
 *     db[oc]             = sum over n and output positions of dout[n][oc]
 *     dw[oc][j][taps]    = sum over n, output positions of dout[n][oc][o] *
 *                          x[n][g*C_in/G + j][o*s + k*d - p]   (dW_row = dout_col @ X_col^T)
 *     dx[n][ic][i]       = sum over the (oc, o, k) whose tap k of output o read
 *                          input i of w[oc][j][k] * dout[n][oc][o]  (col2im(W_row^T @ dout_col))
 * for the general problem of conv_params_t (dilation, groups, 2D/3D).  x, w and
 * dout are bf16 bits; dx, dw, db are fp32; accumulation is fp32.  Results are
 * bitwise reproducible (fixed summation order, no atomics).  Errors as for
 * conv_fwd_bf16, plus CONV_ERR_WORKSPACE when the workspace is missing, too
 * small or not 16-byte aligned, and CONV_ERR_ALIAS when an output overlaps an
 * input or the workspace. */

/* Device workspace for conv_bwd_data_bf16: the flipped weights (and, for 3x3
 * stride-1 layers, their per-stage packing); 0 on invalid parameters. */
CONV_API size_t conv_bwd_data_workspace_bytes(const conv_params_t *params);

/* dx (N, C_in, [D,] H, W) from dout and w.  The data gradient is computed as
 * a forward convolution of dout with w transposed per group (C_in x C_out/G)
 * and every tap reversed, pad d(K-1) - p, on the forward kernels; a strided
 * layer reads dout through zero insertion (the transposed convolution) on the
 * general implicit-GEMM kernel.  The workspace is overwritten. */
CONV_API conv_status_t conv_bwd_data_bf16(const conv_params_t *params, const uint16_t *dout, const uint16_t *w,
                                          float *dx, void *workspace, size_t workspace_bytes, void *stream);

/* Device workspace for conv_bwd_weight_bf16: fp32 partial sums of dw (and
 * of db) over ranges of output positions; 0 on invalid parameters. */
CONV_API size_t conv_bwd_weight_workspace_bytes(const conv_params_t *params);

/* dw (C_out, C_in/G, K, K[, K]) and, when db is not NULL, db (C_out) from x
 * and dout.  dw is reduced over output positions in ranges on the matrix
 * cores, then the ranges are added in a fixed order.  The workspace is
 * overwritten. */
CONV_API conv_status_t conv_bwd_weight_bf16(const conv_params_t *params, const uint16_t *x, const uint16_t *dout,
                                            float *dw, float *db, void *workspace, size_t workspace_bytes,
                                            void *stream);

/* ---- sequences of tokens ---------------------------------------------------
 *
 * The operators below run along a sequence: row t holds the C channels of
 * token t, the channel index fastest (the channels-last order of
 * CONV_LAYOUT_NHWC with H = 1, so a pointwise convolution over tokens produces
 * and consumes these rows).  Sequence b of a batch is rows [b*T, (b+1)*T), or,
 * with `offsets`, rows [offsets[b], offsets[b+1]) of one packed tensor: odd,
 * single-token and empty sequences in any mixture.  A sequence's results (not
 * the sums over all of them) have the same bits in any batch.
 *
 * Strides.  Unlike the tensors above, rows may be strided: `ld*` is the number
 * of elements from one row to the next, >= C (C when dense), so that a slice
 * of a fused projection is read, or written, in place.  Channels of a row are
 * adjacent.  Row offsets are 64-bit: a tensor may hold more than 2^31 elements
 * (rows stay below 2^30).  All other arrays are dense.
 *
 * Types.  x, gates, y, their gradients and the convolution's weights and state
 * are `dtype` (CONV_OUT_BF16: raw bf16 bits; CONV_OUT_F32); bias, decay, the
 * recurrent state and the gradients of parameters are fp32.  Arithmetic, sums
 * and the recurrence are fp32; bf16 results are rounded once, to nearest even.
 * Infinities and NaN follow IEEE rules within their own sequence and channel.
 *
 * Memory, streams and errors are as above: CONV_ERR_NULL for a NULL required
 * pointer (tensors of zero rows may be NULL), CONV_ERR_PARAM for B < 1, T < 0,
 * C < 1, an unknown dtype, ld < C, a pointer not aligned to its element or a
 * bad option, CONV_ERR_OVERFLOW for 2^30 or more rows, more than 2^20 channels,
 * B*C of 2^31 or more, or rows/64 + 2 B or (rows/64 + B) * (C/64) above 2^23
 * (for the recurrence the latter of 2^23 or more, or 2^23 - 1 with CONV_SEQ_FILL),
 * CONV_ERR_WORKSPACE for a workspace that is needed and missing, too small or
 * not 16-byte aligned,
 * CONV_ERR_ALIAS when an output overlaps an input, another output or the
 * workspace (interleaved column slices of one buffer do not overlap).
 * `offsets` are read on the device only: values outside [0, tokens] are clamped,
 * rows of a sequence past T tokens are ignored, and where values descend,
 * which rows are computed is unspecified (never any outside the tensors).
 * Rows that no sequence holds (in front of offsets[0], behind offsets[B], past T
 * tokens) are left as they are in every output of rows, or, with CONV_SEQ_FILL, set to zero.
 * Results are bitwise reproducible. */
#define CONV_SEQ_FILL 256    /* added to dtype: rows of outputs that no sequence holds are set to zero */

typedef struct {
    int dtype;               /* CONV_OUT_F32 or CONV_OUT_BF16, and CONV_SEQ_FILL or not     */
    int B;                   /* sequences                                                   */
    int T;                   /* tokens in each; with offsets, in the longest (0 is allowed)  */
    int C;                   /* channels                                                    */
    const int32_t *offsets;  /* NULL, or B+1 first rows, ascending, on the device           */
    int64_t tokens;          /* rows of a packed tensor; ignored when offsets is NULL       */
} conv_seq_t;

/* Causal depthwise convolution over the tokens of each sequence, 1 <= K <= 8:
 *
 *     p[t][c] = bias[c] + sum_{j<K} w[c][j] * X[t-K+1+j][c]
 *     y = p, or p * sigmoid(p) with silu = 1
 *
 * X is x preceded by the carried rows: X[-i] = state[b][K-1-i], i = 1..K-1
 * (zeros when state is NULL).  w is (C, K), tap K-1 on the token itself; bias
 * (C) may be NULL; state and state_out are (B, K-1, C), oldest row first.
 * state_out (NULL: not wanted) receives the last K-1 rows of X, the state
 * with which the next tokens continue.  (It is a copy: a gradient of state_out
 * is to be added to the gradients of the rows it holds.) */
CONV_API conv_status_t conv_causal_fwd(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx,
                                       const void *w, const float *bias, const void *state, void *y, int64_t ldy,
                                       void *state_out, void *stream);

/* Device workspace of conv_causal_bwd (partial sums of dw and db over ranges
 * of tokens); 0 on invalid arguments. */
CONV_API size_t conv_causal_bwd_workspace_bytes(const conv_seq_t *seq, int K);

/* Gradients for upstream dy (of y): dx, dw (C, K) and db (C) in fp32, and
 * dstate (B, K-1, C) of the carried rows.  db and dstate may be NULL.  The
 * pre-activation p is recomputed from x.  With dp = dy * dy/dp:
 *     dX[t] = sum_j w[j] dp[t+K-1-j],  dw[j] = sum_t dp[t] X[t-K+1+j],  db = sum_t dp[t] */
CONV_API conv_status_t conv_causal_bwd(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx,
                                       const void *w, const float *bias, const void *state, const void *dy,
                                       int64_t lddy, void *dx, int64_t lddx, float *dw, float *db, void *dstate,
                                       void *workspace, size_t workspace_bytes, void *stream);

/* One new token for each of B sequences: x and y are (B, C) rows, and state
 * (B, K-1, C) is read, shifted by one row and extended by x in place.
 * seq->T, offsets and tokens are not read. */
CONV_API conv_status_t conv_causal_step(const conv_seq_t *seq, int K, int silu, const void *x, int64_t ldx,
                                        const void *w, const float *bias, void *state, void *y, int64_t ldy,
                                        void *stream);

/* Gated linear recurrence.  Per token and channel, with the gates' inputs
 * gate and inp and the parameter decay (C):
 *
 *     r = sigmoid(gate),  s = sigmoid(inp),  k = scale * log(1 + exp(decay))
 *     a = exp(-k r),      h[t] = a h[t-1] + sqrt(1 - a^2) s x,      y = h
 *
 * A sigmoid below 2^-126, the smallest normal fp32 (an argument under about
 * -87.3), counts as 0: a gate that far down is shut.  So does a factor a below 2^-126
 * (k r above about 87.3): nothing of the state before it is left, and an infinite one
 * becomes NaN there.
 * h before a sequence's first token is h0 (B, C), or 0 when NULL; hT (B, C),
 * when not NULL, receives h after its last token (h0 for an empty one).
 * states, when not NULL, receives what conv_scan_bwd starts from: h before
 * tokens 0, 64, 128, ... of each sequence, (B, ceil(T/64), C) fp32; entries
 * past a sequence's end are not written.  scale: finite, >= 0. */
#define CONV_SCAN_BLOCK 64

/* Device workspace of conv_scan_fwd; 0 when none is needed, or on invalid
 * arguments.  Overwritten by each call; two calls in flight must not share it. */
CONV_API size_t conv_scan_fwd_workspace_bytes(const conv_seq_t *seq);

CONV_API conv_status_t conv_scan_fwd(const conv_seq_t *seq, float scale, const void *x, int64_t ldx,
                                     const void *gate, int64_t ldg, const void *inp, int64_t ldi,
                                     const float *decay, const float *h0, void *y, int64_t ldy, float *hT,
                                     float *states, void *workspace, size_t workspace_bytes, void *stream);

/* Device workspace of conv_scan_bwd; 0 on invalid arguments. */
CONV_API size_t conv_scan_bwd_workspace_bytes(const conv_seq_t *seq);

/* Gradients for upstream dy (of y) and dhT (of hT; NULL: zero): dx, dgate,
 * dinp; ddecay (C) fp32; dh0 (B, C) fp32, or NULL.  h is recomputed in fp32 from
 * states, as conv_scan_fwd saved them for the same inputs.  With dh the total
 * gradient of h and la = log a:
 *     dh[t] = dy[t] + a[t+1] dh[t+1]           (dhT instead of the last term at the end)
 *     dx = dh sqrt(1-a^2) s,   dinp = dh sqrt(1-a^2) x s (1-s)
 *     dla = dh (a h[t-1] - s x a^2 / sqrt(1-a^2)),   dgate = -k dla r (1-r)
 *     ddecay = -scale sigmoid(decay) sum_t r dla,    dh0 = a[0] dh[0] */
CONV_API conv_status_t conv_scan_bwd(const conv_seq_t *seq, float scale, const void *x, int64_t ldx,
                                     const void *gate, int64_t ldg, const void *inp, int64_t ldi,
                                     const float *decay, const float *states, const void *dy, int64_t lddy,
                                     const float *dhT, void *dx, int64_t lddx, void *dgate, int64_t lddg,
                                     void *dinp, int64_t lddi, float *ddecay, float *dh0, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* One new token for each of B sequences: x, gate, inp and y are (B, C) rows;
 * h (B, C) is updated in place.  seq->T, offsets and tokens are not read. */
CONV_API conv_status_t conv_scan_step(const conv_seq_t *seq, float scale, const void *x, int64_t ldx,
                                      const void *gate, int64_t ldg, const void *inp, int64_t ldi,
                                      const float *decay, float *h, void *y, int64_t ldy, void *stream);

/* ---- gated delta rule -------------------------------------------------------
 *
 * A recurrence whose state is a matrix: a memory that is read at a key, corrected
 * towards a value there, and read at a query.  Each of heads_v value heads has a
 * state S (dim_k x dim_v).  Per token, with the head's query and key q, k (dim_k),
 * value v (dim_v), log decay g and strength beta:
 *
 *     e = v - exp(g) S^T k,    S = exp(g) S + beta k e^T,    y = scale S^T q
 *
 * heads query and key heads; heads divides heads_v, and value head h uses query
 * and key head h / (heads_v/heads).  unit = 1: q and k of each head are brought to unit
 * length first, q / sqrt(sum q^2 + eps); with unit = 0 they are used as they are
 * (k with beta |k|^2 < 2, or the state grows without bound).
 *
 * Sequences, rows, strides, packing and errors are those of the operators over
 * sequences; seq->C is heads_v*dim_v, the channels of v, y, dy and dv, head after
 * head.  Rows of q, k, dq and dk hold heads*dim_k channels.  gate (the log decays g)
 * and beta, and their gradients, are fp32 rows of heads_v.  States are fp32,
 * (B, heads_v, dim_k, dim_v) with dim_v fastest.
 *
 * 1 <= dim_k, dim_v <= 128, heads, heads_v >= 1.  CONV_ERR_PARAM otherwise, and where
 * heads does not divide heads_v, seq->C is not heads_v*dim_v, scale is not finite, or
 * eps is negative or not finite; CONV_ERR_OVERFLOW where B*heads_v*dim_k*dim_v is 2^31 or
 * more, the sequences' 64-token blocks (rows/64 + B of them) times heads_v 2^21 or more, or a
 * row stride 2^22 elements or more.
 *
 * Whole sequences are computed in blocks of 64 tokens by matrix products whose
 * operands are sums of two fp16 numbers under a power of two, accumulated in fp32; decays
 * are added up in fp64.  The power of two is that of the largest value in a row or column: in a
 * column of values or of upstream gradients, of the largest of tokens 0..31, or 32..63, of a block;
 * in the gradients of q and k, of the largest in a head's state.  A value has 22 bits down to 2^-16
 * of that largest, and an error of up to 2^-38 of it below.  Rows and columns whose largest value is below
 * 2^-90 (of q and k with unit = 0) have fewer bits; values and states beyond 2^100 may end as infinities.
 * A log decay below -10000 counts as -10000: nothing of the state is left.
 *
 * Infinities and NaN: results that depend on one are not finite, in its own sequence and head
 * only.  Nor need those be of tokens in front of it among the same 32, or gradients of its
 * 64-token block; what is finite is right.
 *
 * Long sequences are cut into segments that run at once and are joined where a batch has few of them: results then
 * differ by roundings from those of the same sequence in another batch.  They have the same bits in any batch with T of at
 * most 448, and in batches of the same T, B and rows; a step always has. */
typedef struct {
    int heads, heads_v;      /* of queries and keys; of values                  */
    int dim_k, dim_v;        /* of each head                                    */
    int unit;                /* 0 or 1                                          */
    float scale, eps;        /* of the output; of the unit length               */
} conv_delta_t;

/* Device workspace of conv_delta_fwd: what each block needs before its state is
 * known; 0 where none is needed, or on invalid arguments.  Overwritten by each
 * call; two calls in flight must not share it. */
CONV_API size_t conv_delta_fwd_workspace_bytes(const conv_seq_t *seq, const conv_delta_t *par);

/* S before a sequence's first token is s0, or 0 when NULL; sT, when not NULL,
 * receives S after its last token (s0 for an empty one).  states, when not NULL,
 * receives what conv_delta_bwd starts from: S before tokens 0, 64, 128, ... of
 * each sequence, (B, ceil(T/64), heads_v, dim_k, dim_v) fp32; entries past a
 * sequence's end are not written. */
CONV_API conv_status_t conv_delta_fwd(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq,
                                      const void *k, int64_t ldk, const void *v, int64_t ldv, const float *gate,
                                      int64_t ldg, const float *beta, int64_t ldb, const float *s0, void *y, int64_t ldy,
                                      float *sT, float *states, void *workspace, size_t workspace_bytes, void *stream);

/* Device workspace of conv_delta_bwd; 0 where none is needed, or on invalid
 * arguments. */
CONV_API size_t conv_delta_bwd_workspace_bytes(const conv_seq_t *seq, const conv_delta_t *par);

/* Gradients for upstream dy (of y) and dsT (of sT; NULL: zero): dq, dk, dv, dgate,
 * dbeta, and ds0 (B, heads_v, dim_k, dim_v), or NULL.  states: as conv_delta_fwd saved
 * them for the same inputs.  dq and dk are sums over the value heads that share a
 * head, and with unit = 1 lead through the unit length.  With dS the total gradient of S, u = beta e and
 * S' = exp(g) S[t-1], per token from the last to the first:
 *     dS[t] += scale q dy^T,  dq = scale S[t] dy,  z = dS[t]^T k,  dbeta = z.e,  dv = beta z,
 *     dk = dS[t] u - beta S' z,  dS' = dS[t] - beta k z^T,  dgate = <dS', S'>,  dS[t-1] = exp(g) dS' */
CONV_API conv_status_t conv_delta_bwd(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq,
                                      const void *k, int64_t ldk, const void *v, int64_t ldv, const float *gate,
                                      int64_t ldg, const float *beta, int64_t ldb, const float *states, const void *dy,
                                      int64_t lddy, const float *dsT, void *dq, int64_t lddq, void *dk, int64_t lddk,
                                      void *dv, int64_t lddv, float *dgate, int64_t lddg, float *dbeta, int64_t lddb,
                                      float *ds0, void *workspace, size_t workspace_bytes, void *stream);

/* One new token for each of B sequences: q, k, v, gate, beta and y are one row
 * for each; S (B, heads_v, dim_k, dim_v) is updated in place.  seq->T, offsets and
 * tokens are not read. */
CONV_API conv_status_t conv_delta_step(const conv_seq_t *seq, const conv_delta_t *par, const void *q, int64_t ldq,
                                       const void *k, int64_t ldk, const void *v, int64_t ldv, const float *gate,
                                       int64_t ldg, const float *beta, int64_t ldb, float *S, void *y, int64_t ldy,
                                       void *stream);

/* ---- layer norm ------------------------------------------------------------
 *
 * Over the C channels of each of `rows` rows (those of any sequences, packed or
 * not, or one row for each head), in the layouts, types and strides of the
 * operators over sequences; dtype is CONV_OUT_F32 or CONV_OUT_BF16, for x, y, dy
 * and dx.  weight, bias (C; NULL: ones, zeros), mean, rstd (rows) and the gradients of
 * parameters are fp32:
 *
 *     mean = sum x / C,   rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),   y = (x - mean) rstd weight + bias
 *
 * Arithmetic is fp32 (squares beyond its range, of values beyond 10^19, make rstd 0), y is rounded once.  mean and rstd, where not NULL, receive
 * what conv_norm_bwd starts from.  eps: finite, >= 0.  A row's results have the
 * same bits among any other rows (dweight and dbias are sums over all).  Errors
 * are those of the operators over sequences: rows < 0, C < 1, ld < C and
 * alignment CONV_ERR_PARAM, 2^30 or more rows or more than 2^20 channels
 * CONV_ERR_OVERFLOW.  No rows: nothing is done, and sums are zeros. */
CONV_API conv_status_t conv_norm_fwd(int dtype, int64_t rows, int C, float eps, const void *x, int64_t ldx,
                                     const float *weight, const float *bias, void *y, int64_t ldy, float *mean,
                                     float *rstd, void *stream);

/* Device workspace of conv_norm_bwd: sums of dweight and dbias over ranges of
 * rows; 0 on invalid arguments, and where there are no rows. */
CONV_API size_t conv_norm_bwd_workspace_bytes(int dtype, int64_t rows, int C);

/* Gradients for upstream dy, with mean and rstd as the forward pass gave them and xh = (x - mean) rstd:
 *     dx = rstd (weight dy - sum(weight dy) / C - xh sum(weight dy xh) / C)
 *     dweight = sum over rows of dy xh,   dbias = sum over rows of dy
 * dweight and dbias (C) may be NULL; with both NULL no workspace is needed. */
CONV_API conv_status_t conv_norm_bwd(int dtype, int64_t rows, int C, const void *x, int64_t ldx, const float *weight,
                                     const float *mean, const float *rstd, const void *dy, int64_t lddy, void *dx,
                                     int64_t lddx, float *dweight, float *dbias, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* ---- the optimiser step --------------------------------------------------
 *
 * AdamW over `count` tensors at once, from the fp32 (or bf16) gradients that
 * conv_bwd_weight_bf16, conv_causal_bwd, conv_scan_bwd and conv_norm_bwd write to the bf16
 * weights that the next forward pass reads.  With c1 = 1 - beta1^step and
 * c2 = 1 - beta2^step (step: this one's number, from 1):
 *
 *     g = grad * *grad_scale                   (grad_scale: device scalar, NULL = 1)
 *     m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay) - (lr/c1) m / (sqrt(v)/sqrt(c2) + eps)
 *     copy = bf16(p)                           (copy: NULL = none)
 *
 * bits = 32: m and v are fp32.  bits = 8: m is int8 and v uint8 codes q in
 * blocks of 256 elements (counted from the tensor's first), each block with an
 * fp32 scale, its largest |m| (largest v):
 *     m = scale * sign(q) (q/127)^2,   v = scale * (q/255)^4
 * m_scale and v_scale hold ceil(n/256) floats; all-zero codes and scales are
 * the zero state.  A new value lies between two codes and takes the upper one
 * with the probability with which that makes it right on average: rounding to
 * the nearest would leave v where it is, as one step changes it by less than a
 * code.  The random bits depend on seed, step, the tensor's place in the list
 * and the element only, so a step is reproducible.  v > 0 never takes code 0.
 * A block whose largest value is below 2^-126 is stored as zeros.  A
 * non-finite gradient, or a square beyond fp32, makes its element (bits = 8: its
 * block's scales) non-finite.
 *
 * The numbers in `opt` are taken when the call is made.  A call captured in a
 * graph therefore takes the same step again at every replay: the step's number in
 * c1 and c2, the rates, and with bits = 8 the same random bits for every element,
 * whose rounding is then no longer right on average.  Only the gradients' scale is read
 * on the device.  Capture the passes, and call the step beside the graph.
 *
 * `tensors` is a HOST array, read before the call returns (its pointers are
 * device pointers).  No two of them may share memory that is written (not
 * checked).  Every tensor: n >= 0; n = 0 is skipped.  Errors:
 * CONV_ERR_NULL for a NULL array, p, g, m or v (bits = 8: scale), CONV_ERR_PARAM for
 * count < 0, n < 0, step < 1, betas outside [0, 1), lr, eps or weight_decay
 * negative or not finite, bits other than 32 or 8, an unknown grad_dtype, or a
 * pointer not aligned to its element; CONV_ERR_OVERFLOW for n >= 2^31;
 * CONV_ERR_ALIAS when what is written overlaps anything else of its tensor. */
typedef struct {
    int64_t n;            /* elements                                     */
    float *p;             /* parameters, fp32, updated                    */
    const void *g;        /* gradient, grad_dtype                         */
    void *m, *v;          /* moments: fp32, or int8 / uint8 codes, updated */
    float *m_scale;       /* bits = 8: scales of m and v, updated         */
    float *v_scale;
    uint16_t *copy;       /* bf16 copy of p, written, or NULL             */
    float weight_decay;
} conv_adamw_tensor_t;

typedef struct {
    double lr, beta1, beta2, eps;
    int64_t step;             /* number of this step, from 1             */
    int bits;                 /* 32 or 8                                 */
    int grad_dtype;           /* CONV_OUT_F32 or CONV_OUT_BF16            */
    uint32_t seed;            /* bits = 8: of the random rounding         */
    const float *grad_scale;  /* device scalar, or NULL                  */
} conv_adamw_t;

CONV_API conv_status_t conv_adamw_step(const conv_adamw_t *opt, const conv_adamw_tensor_t *tensors, int count,
                                       void *stream);

/* The values that 8-bit moments stand for, fp32: m_out[i] and v_out[i] (HOST
 * arrays of device pointers, n of tensors[i] elements each) receive tensor i's.
 * Reads n, m, v and the scales of `tensors` only. */
CONV_API conv_status_t conv_adamw_state_values(const conv_adamw_tensor_t *tensors, int count, float *const *m_out,
                                               float *const *v_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_FWD_H */
