/*
 * b200norm.h -- C ABI of the fused residual-add + normalization kernels for
 * NVIDIA GB300 (sm_103a).
 *
 * Operators (ONNX Runtime contrib operators, as described by the README pages
 * of the webgpu-kernels packages):
 *   b200norm_skip_rms    com.microsoft.SkipSimplifiedLayerNormalization
 *   b200norm_gated_rms   com.microsoft.GatedRMSNorm
 *   b200norm_skip_group  com.microsoft.SkipGroupNorm
 * and the operators that stand beside them on a residual stream, in serving
 * and in training:
 *   b200norm_skip_layer, b200norm_skip_layer_grad
 *                        layer normalization (with the residual add fused in),
 *                        and its gradients
 *   b200norm_linear, b200norm_linear_grad
 *                        y = act(x W^T + b) + residual, and its gradients
 *   b200norm_gated_linear, b200norm_gated_linear_grad
 *                        h = act(x Wg^T + bg) * (x Wu^T + bu), and its gradients
 *   b200norm_rotary, b200norm_head_rms_rotary, b200norm_head_rms_rotary_grad
 *                        position rotation of query and key heads, with or
 *                        without an RMS norm of each head, and its gradients
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is a DEVICE pointer to a dense, contiguous,
 *     row-major tensor owned by the caller (heads have strides of their own).
 *     The library never allocates, frees or synchronises; it only enqueues
 *     kernels on `stream`.
 *   - Pointers need only be aligned to their element size.  16-byte aligned
 *     pointers (with spans that are whole 16-byte vectors) take the vector
 *     path; anything else takes a scalar path with identical results.
 *   - Element types: B200NORM_F32 (IEEE binary32), B200NORM_F16 (IEEE
 *     binary16) and B200NORM_BF16 (bfloat16: the upper half of a binary32).
 *     The pages' type constraints list float32 and float16 only, and the
 *     GatedRMSNorm README, Description, says bfloat16 is not implemented
 *     there; this library adds it as a storage type with the same arithmetic
 *     (binary32 compute, one rounding to nearest-even at each store).  For
 *     SkipGroupNorm the gamma/beta type M is B200NORM_F32 or T itself, and
 *     also B200NORM_F16 when T is B200NORM_F32; other pairs return
 *     B200NORM_ERR_UNSUPPORTED.
 *   - Rounding: the residual sum S is formed in binary32 as
 *     (x + skip) + bias -- no add at all when bias is NULL -- and rounded once
 *     to nearest-even at the tensor type; statistics are taken over that
 *     rounded S (SkipGroupNorm README, Description).  Every later
 *     intermediate is binary32; only the final store narrows to T.
 *   - Outputs must not overlap any input or each other
 *     (B200NORM_ERR_INVALID_ARGUMENT).
 *   - Argument errors are reported before anything is enqueued.  Launch
 *     failures return B200NORM_ERR_CUDA.  A call on empty tensors returns
 *     B200NORM_OK and enqueues nothing.
 *   - b200norm_last_error() returns a thread-local, human-readable reason for
 *     the last non-OK status returned on the calling thread.
 *   - Calls are stateless apart from the caller-provided workspaces, and may
 *     be issued from several host threads at once.
 *   - Kernels are launched with programmatic dependent launch allowed: one
 *     may be scheduled while the previous kernel on the stream drains, but it
 *     waits for that kernel to complete (and its writes to be visible) before
 *     touching memory, so stream order is kept.
 */
#ifndef B200NORM_H
#define B200NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define B200NORM_API __attribute__((visibility("default")))
#else
#define B200NORM_API
#endif

/* Same object as cudaStream_t (declared here so that this header does not
 * need the CUDA headers).  NULL is the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st* b200norm_stream_t;

typedef enum {
    B200NORM_F32 = 0,
    B200NORM_F16 = 1,
    B200NORM_BF16 = 2
} b200norm_dtype;

typedef enum {
    B200NORM_OK = 0,
    B200NORM_ERR_INVALID_ARGUMENT = 1, /* bad pointer, shape, attribute or overlap   */
    B200NORM_ERR_UNSUPPORTED = 2,      /* element type or shape the library refuses   */
    B200NORM_ERR_CUDA = 3,             /* a CUDA runtime call or launch failed        */
    B200NORM_ERR_WORKSPACE = 4,        /* workspace missing, too small or misaligned  */
    B200NORM_ERR_DEVICE_TIMEOUT = 5    /* a device-side wait gave up (see below)      */
} b200norm_status;

/* Contract version of this ABI (1). */
B200NORM_API int b200norm_version(void);

/* Static string naming a status code. */
B200NORM_API const char* b200norm_status_string(b200norm_status status);

/* Reason for the last non-OK status returned on the calling thread ("" if
 * none).  The pointer stays valid until the next call on this thread. */
B200NORM_API const char* b200norm_last_error(void);

/*
 * SkipSimplifiedLayerNormalization
 * (com.microsoft.SkipSimplifiedLayerNormalization README: Description,
 * Inputs, Outputs, Attributes):
 *
 *   S[r, j]      = round_T((input[r, j] + skip[r, j]) + bias[j])
 *   output[r, j] = round_T(S[r, j] * (1 / sqrt(mean_j(S[r, :]^2) + epsilon)) * gamma[j])
 *
 *   input, skip          T, (rows, hidden), row-major.  rows is the product of
 *                        the leading axes: (token_count) or (batch * sequence).
 *   gamma                T, (hidden).
 *   bias                 T, (hidden), or NULL when absent.
 *   output               T, (rows, hidden).
 *   input_skip_bias_sum  T, (rows, hidden): receives S; NULL when not requested.
 *   epsilon              >= 0 and not NaN; the operator default is
 *                        9.999999960041972e-13 (float32 of 1e-12).
 *
 * rows == 0 is a no-op.  hidden must be > 0.
 */
B200NORM_API b200norm_status b200norm_skip_rms(const void* input, const void* skip,
                                               const void* gamma, const void* bias, void* output,
                                               void* input_skip_bias_sum, int64_t rows,
                                               int64_t hidden, b200norm_dtype T, float epsilon,
                                               b200norm_stream_t stream);

/*
 * Same as b200norm_skip_rms, and also writes the per-row statistics outputs
 * that the operator schema lists (SkipSimplifiedLayerNormalization README,
 * Outputs: mean, inv_std_var, element type U = float32, shape of the input
 * with the last axis replaced by 1):
 *   mean[r]        = 0 (the simplified form does not centre the row)
 *   inv_std_var[r] = 1 / sqrt(mean_j(S[r, :]^2) + epsilon)
 * Either pointer may be NULL.  Both are float32 device arrays of `rows`.
 */
B200NORM_API b200norm_status b200norm_skip_rms_stats(const void* input, const void* skip,
                                                     const void* gamma, const void* bias,
                                                     void* output, void* input_skip_bias_sum,
                                                     float* mean, float* inv_std_var,
                                                     int64_t rows, int64_t hidden,
                                                     b200norm_dtype T, float epsilon,
                                                     b200norm_stream_t stream);

/*
 * GatedRMSNorm (com.microsoft.GatedRMSNorm README: Description, Inputs,
 * Attributes):
 *
 *   for each contiguous span r of C elements (rows = numel / C):
 *   y[r, j] = round_T(x[r, j] * (1 / sqrt(mean_j(x[r, :]^2) + epsilon))
 *                     * scale[j] * SiLU(gate[r, j])),   SiLU(g) = g / (1 + e^-g)
 *
 *   x, gate, y   T, numel elements (any rank >= 1, folded to (numel / C, C)).
 *   scale        T, C elements: (C), (1, C) and (C, 1) are the same vector.
 *   numel        must be a multiple of C; numel == 0 is a no-op.
 *   C            > 0.
 *   epsilon      >= 0 and not NaN; operator default 1e-5.
 *
 * Every intermediate, SiLU included, is binary32.
 */
B200NORM_API b200norm_status b200norm_gated_rms(const void* x, const void* gate,
                                                const void* scale, void* y, int64_t numel,
                                                int64_t C, b200norm_dtype T, float epsilon,
                                                b200norm_stream_t stream);

/* Synchronise `stream`, then read the device-side record of the pipelined row
 * schedule on the current device.  SkipSimplifiedLayerNormalization and
 * GatedRMSNorm calls with short rows (at most 32 16-byte vectors), and
 * b200norm_skip_layer_grad calls, may run a kernel that streams its inputs
 * through shared memory; its waits on copy
 * completion are bounded (about one second), and one that gives up records
 * B200NORM_ERR_DEVICE_TIMEOUT in a per-device word and returns early (that
 * call's outputs are then undefined).  Returns B200NORM_OK, or
 * B200NORM_ERR_DEVICE_TIMEOUT (and clears the record) if any such launch on
 * the device gave up since the last call; B200NORM_ERR_CUDA if the read
 * failed.  No correct launch records anything. */
B200NORM_API b200norm_status b200norm_rows_status(b200norm_stream_t stream);

/*
 * SkipGroupNorm (com.microsoft.SkipGroupNorm README: Description, Inputs,
 * Outputs, Attributes, Type constraints):
 *
 *   S = round_T((X + skip) + bias)                          (bias may be NULL)
 *   Y = round_T(act((S - mean) * rstd * gamma[c] + beta[c])), evaluated in
 *       binary32, rstd = 1 / sqrt(var + epsilon), act = SiLU (z / (1 + e^-z))
 *       when activation == 1, identity when 0.
 *   mean and var (population) are taken per batch item n and group g over the
 *   C / groups channels of g and every spatial position.
 *
 *   x, y, s   T.  Physical layout (N, H, W, C) when channels_last != 0, else
 *             (N, C, H, W).  N, C, H, W below are the LOGICAL sizes.
 *   skip      T.  skip_rank / skip_dims give its shape:
 *               - exactly x's physical shape                     full skip;
 *               - (N, C) or (N, 1, 1, C)       one value per (n, c), at
 *                                              offset n * C + c, both layouts.
 *             A (N, 1, 1, C) skip when H == W == 1 is an exact match and takes
 *             the full route (same offsets, same results).
 *   bias      T, (C), or NULL.
 *   gamma, beta  M, (C).  M is B200NORM_F32 or T, or B200NORM_F16 when T is
 *             B200NORM_F32.
 *   s         receives S when not NULL.
 *   groups    > 0 and must divide C.
 *   activation  0 (none) or 1 (SiLU); required.
 *   epsilon   >= 0 and not NaN; operator default 1e-5.
 *   workspace device memory of at least
 *             b200norm_skip_group_workspace_size(...) bytes, 256-byte aligned,
 *             ZERO-FILLED before its first use (b200norm_workspace_init does
 *             that).  A call that completes normally leaves it ready for the
 *             next call.  Calls that share a workspace must not overlap on the
 *             device (enqueue them on one stream).
 *
 * Device-side waits inside the kernels (on other CTAs at a grid barrier, or
 * on a bulk copy into shared memory) are bounded: a wait that does not
 * complete within about one second makes the kernel record
 * B200NORM_ERR_DEVICE_TIMEOUT in the workspace and return early (outputs are
 * then undefined).  b200norm_workspace_status() reads that record.
 */
B200NORM_API size_t b200norm_skip_group_workspace_size(int64_t N, int64_t C, int64_t H,
                                                       int64_t W, int groups, b200norm_dtype T,
                                                       int channels_last);

B200NORM_API b200norm_status b200norm_skip_group(
    const void* x, const void* skip, int skip_rank, const int64_t* skip_dims, const void* bias,
    const void* gamma, const void* beta, void* y, void* s, int64_t N, int64_t C, int64_t H,
    int64_t W, b200norm_dtype T, b200norm_dtype M, int groups, float epsilon, int activation,
    int channels_last, void* workspace, size_t workspace_bytes, b200norm_stream_t stream);

/*
 * SkipGroupNorm without a workspace, for callers that cannot allocate device
 * memory: for example a plugin whose host passes it only its input and output
 * buffers and provides no allocator, or a service that reserved its device
 * memory up front and must not allocate (and possibly fail or synchronise)
 * while serving a request.  The operator pages have no counterpart of this
 * entry point; it exists only because of that constraint.
 *
 * Arguments and results are those of b200norm_skip_group without
 * `workspace` / `workspace_bytes`.  Instead the library uses a fixed scratch
 * array of 256 + 2 MiB bytes in device memory, which every GPU that loads
 * the library holds until the process exits.  A call fits exactly when
 * b200norm_skip_group_workspace_size() of its shape is at most that size;
 * with L = C / groups * H * W, NHWC shapes with at most 32 groups and
 * N * ceil(L / 4096) <= 4,096 fit, and NCHW shapes fit when
 * N * groups * ceil(L / 4096) <= 131,072.  A larger shape returns
 * B200NORM_ERR_UNSUPPORTED (see b200norm_last_error); use
 * b200norm_skip_group with a workspace for it.  Every argument is checked
 * before anything is enqueued, as for b200norm_skip_group: a call that
 * returns an error has enqueued nothing.  No call allocates or frees memory.
 *
 *   - The first call on a device looks up the scratch array's device address
 *     (cudaGetSymbolAddress) with that device current, and keeps it for the
 *     life of the process: make that first call before any stream capture
 *     begins, and do not use the library across a cudaDeviceReset().
 *   - Each call clears the scratch's barrier counters on `stream` before its
 *     kernels; the slots keep the previous call's contents and are always
 *     written before they are read.
 *   - A bounded device-side wait that gives up (see b200norm_skip_group)
 *     records B200NORM_ERR_DEVICE_TIMEOUT in the scratch, where it stays,
 *     through later calls, until b200norm_skip_group_noalloc_status() reads
 *     and clears it.
 *   - All calls on a device share the one array: calls whose work overlaps on
 *     the GPU (different streams without ordering between them) race and give
 *     undefined results.  Order them, e.g. issue them on one stream.
 */
B200NORM_API b200norm_status b200norm_skip_group_noalloc(
    const void* x, const void* skip, int skip_rank, const int64_t* skip_dims, const void* bias,
    const void* gamma, const void* beta, void* y, void* s, int64_t N, int64_t C, int64_t H,
    int64_t W, b200norm_dtype T, b200norm_dtype M, int groups, float epsilon, int activation,
    int channels_last, b200norm_stream_t stream);

/* Synchronise `stream`, then read and clear the device-side error record of
 * b200norm_skip_group_noalloc's scratch on the current device: B200NORM_OK,
 * or B200NORM_ERR_DEVICE_TIMEOUT if a bounded wait of an earlier call gave up
 * (that call's outputs are undefined).  B200NORM_ERR_CUDA if the copy failed.
 * Allocates nothing. */
B200NORM_API b200norm_status b200norm_skip_group_noalloc_status(b200norm_stream_t stream);

/* Zero-fill a SkipGroupNorm workspace (cudaMemsetAsync on `stream`). */
B200NORM_API b200norm_status b200norm_workspace_init(void* workspace, size_t workspace_bytes,
                                                     b200norm_stream_t stream);

/* Synchronise `stream`, then read the workspace's device-side error record:
 * B200NORM_OK, or B200NORM_ERR_DEVICE_TIMEOUT if a bounded wait gave up (the
 * workspace must then be re-initialised).  B200NORM_ERR_CUDA if the copy
 * failed. */
B200NORM_API b200norm_status b200norm_workspace_status(const void* workspace,
                                                       b200norm_stream_t stream);

/*
 * Layer normalization over the last axis, with the residual add fused in:
 *
 *   S[r, j]      = round_T((input[r, j] + skip[r, j]) + bias[j])
 *   mu[r]        = mean_j(S[r, :]),  var[r] = mean_j((S[r, :] - mu[r])^2)
 *   output[r, j] = round_T((S[r, j] - mu[r]) * (1 / sqrt(var[r] + epsilon)) * gamma[j]
 *                          + beta[j])
 *
 *   input, skip          T, (rows, hidden).  skip may be NULL: S is then the
 *                        input, and bias and input_skip_bias_sum must be NULL.
 *   gamma, beta          M, (hidden); M is T or B200NORM_F32.  beta may be NULL.
 *   bias                 T, (hidden), or NULL.
 *   output               T, (rows, hidden).
 *   input_skip_bias_sum  T, (rows, hidden): receives S; NULL when not requested.
 *   mean, inv_std_var    float32, (rows): mu and 1 / sqrt(var + epsilon); either
 *                        may be NULL.  b200norm_skip_layer_grad needs both.
 *   epsilon              >= 0 and not NaN.
 *
 * rows == 0 is a no-op.  hidden must be > 0.
 */
B200NORM_API b200norm_status b200norm_skip_layer(
    const void* input, const void* skip, const void* gamma, const void* beta, const void* bias,
    void* output, void* input_skip_bias_sum, float* mean, float* inv_std_var, int64_t rows,
    int64_t hidden, b200norm_dtype T, b200norm_dtype M, float epsilon, b200norm_stream_t stream);

/*
 * Gradients of b200norm_skip_layer.  With u = (S - mean) * inv_std_var and
 * g = dy * gamma:
 *
 *   dx[r, j]  = round_T(inv_std_var[r] * (g - mean_j(g) - u * mean_j(g * u)) + ds[r, j])
 *   dgamma[j] = round_M(sum_r dy * u)
 *   dbeta[j]  = round_M(sum_r dy)
 *   dbias[j]  = round_T(sum_r of dx before its rounding)
 *
 *   dy           T, (rows, hidden): gradient of output.
 *   s            T, (rows, hidden): input_skip_bias_sum of the forward call, or
 *                its input where it had no skip.
 *   mean, inv_std_var  float32, (rows): of the forward call.
 *   gamma        M, (hidden); M is T or B200NORM_F32.
 *   ds           T, (rows, hidden): the gradient that reaches S by other paths
 *                (the residual stream's own), or NULL.
 *   dx           T: the gradient of S, which is that of input and of skip.
 *   dgamma, dbeta  M, (hidden).   dbias  T, (hidden).
 *   Any of dx, dgamma, dbeta and dbias may be NULL when not wanted.
 *   workspace    at least b200norm_skip_layer_grad_workspace_size() bytes,
 *                256-byte aligned; its contents before the call do not matter.
 *                Calls that share one must not overlap on the device.
 *
 * Sums over rows are binary32, in a fixed order (equal calls give equal bits).
 * rows == 0 stores zeros in dgamma, dbeta and dbias.  The first call on a device
 * looks up a device address: make it before any stream capture begins.
 */
B200NORM_API size_t b200norm_skip_layer_grad_workspace_size(int64_t rows, int64_t hidden);

B200NORM_API b200norm_status b200norm_skip_layer_grad(
    const void* dy, const void* s, const float* mean, const float* inv_std_var, const void* gamma,
    const void* ds, void* dx, void* dgamma, void* dbeta, void* dbias, int64_t rows,
    int64_t hidden, b200norm_dtype T, b200norm_dtype M, void* workspace, size_t workspace_bytes,
    b200norm_stream_t stream);

/*
 * The linear operator:
 *
 *   z[r, o] = sum_i x[r, i] * weight[o, i] + bias[o]
 *   y[r, o] = round_T(act(z[r, o]) + residual[r, o])
 *
 *   x          T, (rows, in_features).
 *   weight     T, (out_features, in_features).
 *   bias       T, (out_features), or NULL.
 *   residual   T, (rows, out_features), or NULL.
 *   y          T, (rows, out_features).
 *   z          T, (rows, out_features): receives round_T(z) for
 *              b200norm_linear_grad; NULL when not requested.  y is formed from
 *              the unrounded z, so requesting z does not change it.
 *   activation 0 none, 1 SiLU (z / (1 + e^-z)), 2 GELU (z times the normal
 *              distribution function), 3 GELU in its tanh form
 *              (z / 2 * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3)))),
 *              4 ReLU.
 *   workspace  at least b200norm_linear_workspace_size() bytes, 256-byte
 *              aligned (NULL where that is 0); its contents before the call do
 *              not matter.  Calls that share one must not overlap on the device.
 *
 * Sums are binary32, in a fixed order.  rows == 0 is a no-op; rows may be 2^30
 * at most, in_features and out_features must be in [1, 2^20].  The first call on
 * a device looks up a device address: make it before any stream capture begins.
 */
B200NORM_API size_t b200norm_linear_workspace_size(int64_t rows, int64_t in_features,
                                                   int64_t out_features, b200norm_dtype T,
                                                   int aligned16);

B200NORM_API b200norm_status b200norm_linear(
    const void* x, const void* weight, const void* bias, const void* residual, void* y, void* z,
    int64_t rows, int64_t in_features, int64_t out_features, b200norm_dtype T, int activation,
    void* workspace, size_t workspace_bytes, b200norm_stream_t stream);

/*
 * Gradients of b200norm_linear (that of residual is dy itself):
 *
 *   dz[r, o] = dy[r, o] * act'(z[r, o])
 *   dx[r, i] = round_T(sum_o round_T(dz[r, o]) * weight[o, i])
 *   dw[o, i] = round_T(sum_r round_T(dz[r, o]) * x[r, i])
 *   db[o]    = round_T(sum_r dz[r, o])
 *
 *   dy, z      T, (rows, out_features); z of the forward call, NULL (and not
 *              read) when activation is 0.  The derivative of ReLU at 0 is 0.
 *   x, weight  as in the forward call; x may be NULL without dw, weight
 *              without dx.
 *   dx, dw, db T, of x's, weight's and bias's shapes; any may be NULL when not
 *              wanted.
 *   workspace  at least b200norm_linear_grad_workspace_size() bytes, as above.
 *
 * Sums are binary32, in a fixed order.  rows == 0 stores zeros in dw and db.
 */
B200NORM_API size_t b200norm_linear_grad_workspace_size(int64_t rows, int64_t in_features,
                                                        int64_t out_features, b200norm_dtype T,
                                                        int activation, int aligned16);

B200NORM_API b200norm_status b200norm_linear_grad(
    const void* dy, const void* x, const void* weight, const void* z, void* dx, void* dw, void* db,
    int64_t rows, int64_t in_features, int64_t out_features, b200norm_dtype T, int activation,
    void* workspace, size_t workspace_bytes, b200norm_stream_t stream);

/*
 * The gated linear operator: two products of the same rows, one of them the other's gate.
 * With out_features = F:
 *
 *   z[r, o] = sum_i x[r, i] * weight[o, i] + bias[o],  o < 2 F
 *   h[r, o] = round_T(act(z[r, o]) * z[r, F + o]),     o < F
 *
 *   x          T, (rows, in_features).
 *   weight     T, (2 F, in_features): the gate's rows, then those of what it gates.
 *   bias       T, (2 F), in the same order, or NULL.
 *   h          T, (rows, F).
 *   z          T, (rows, 2 F): receives round_T(z) for b200norm_gated_linear_grad; NULL
 *              when not requested.  h is formed from the unrounded z.
 *   activation, workspace  as in b200norm_linear (of its own _workspace_size()).
 *
 * Limits as in b200norm_linear, with F in [1, 2^19]; rows == 0 is a no-op.  Sums are
 * binary32, in a fixed order.  Large float32 calls (from 9 rows, or 5 of in_features
 * that 4 does not divide, and 2^26 products of rows, in_features and F; gradients from 64
 * rows and 2^24, or 9 and 2^27) run on the tensor cores: every value is split into three
 * bfloat16 numbers that add up to it (24 bits; below 2^-110 of magnitude some of the last
 * are lost), and six of their nine products are summed, which leaves errors of about
 * 2^-24 of a product (an operand below 2^-126 counts as that).  A sum that is not finite
 * so is made again from the values: infinities, NaN and overflows are those of binary32
 * sums.  The workspace holds the pieces.
 */
B200NORM_API size_t b200norm_gated_linear_workspace_size(int64_t rows, int64_t in_features,
                                                         int64_t out_features, b200norm_dtype T,
                                                         int aligned16);

B200NORM_API b200norm_status b200norm_gated_linear(
    const void* x, const void* weight, const void* bias, void* h, void* z, int64_t rows,
    int64_t in_features, int64_t out_features, b200norm_dtype T, int activation, void* workspace,
    size_t workspace_bytes, b200norm_stream_t stream);

/*
 * Gradients of b200norm_gated_linear:
 *
 *   dz[r, o]     = dh[r, o] * z[r, F + o] * act'(z[r, o])
 *   dz[r, F + o] = dh[r, o] * act(z[r, o])
 *   dx[r, i] = round_T(sum_o round_T(dz[r, o]) * weight[o, i])
 *   dw[o, i] = round_T(sum_r round_T(dz[r, o]) * x[r, i])
 *   db[o]    = round_T(sum_r dz[r, o])
 *
 * (dz is not rounded where the weight and its gradient are passed in one launch: up to four
 * rows, and up to eight of rows * in_features * F <= 2^25).
 *
 *   dh         T, (rows, F): gradient of h.   z   of the forward call.
 *   x, weight  as in the forward call; x may be NULL without dw, weight without dx.
 *   dx, dw, db T, of x's, weight's and bias's shapes; any may be NULL when not wanted.
 *   workspace  at least b200norm_gated_linear_grad_workspace_size() bytes, as above;
 *              aligned16: x and weight start on 16-byte boundaries.
 *
 * Sums are binary32, in a fixed order; large float32 calls as in b200norm_gated_linear (and
 * dz in pieces too).  In 16-bit types the rounded dz has the type's range: in float16 a
 * product dh * z above 65,504 in magnitude may become an infinity.  rows == 0 stores zeros
 * in dw and db.
 */
B200NORM_API size_t b200norm_gated_linear_grad_workspace_size(int64_t rows, int64_t in_features,
                                                              int64_t out_features,
                                                              b200norm_dtype T, int aligned16);

B200NORM_API b200norm_status b200norm_gated_linear_grad(
    const void* dh, const void* x, const void* weight, const void* z, void* dx, void* dw, void* db,
    int64_t rows, int64_t in_features, int64_t out_features, b200norm_dtype T, int activation,
    void* workspace, size_t workspace_bytes, b200norm_stream_t stream);

/* Synchronise `stream`, then read the device-side record of the linear
 * operator's kernels (the gated ones as well) on the current device.  On the
 * tensor cores (16-bit types, large gated float32 calls) their roles wait on
 * one another through shared memory; the waits are bounded (a second and
 * more for long sums), and one that gives up records
 * B200NORM_ERR_DEVICE_TIMEOUT in a per-device word, with the kind of the first
 * such wait, and ends early (that call's outputs are then undefined).  Returns B200NORM_OK, or
 * B200NORM_ERR_DEVICE_TIMEOUT (and clears the record) if any such launch on the
 * device gave up since the last call; B200NORM_ERR_CUDA if the read failed.  No
 * correct launch records anything. */
B200NORM_API b200norm_status b200norm_linear_status(b200norm_stream_t stream);

/*
 * Query and key heads on the way to attention.
 *
 * Rotation: the pair (a, b) of a head with frequency f, of a token at position p,
 * becomes (a c - b s, b c + a s) with c = scale * cos(p f), s = scale * sin(p f);
 * the inverse has -s, and is the rotation's gradient.  With R = rotary_size, pair i
 * (i < R / 2) is elements (i, i + R / 2) of the head, or (2 i, 2 i + 1) when
 * interleaved; elements from R on stay as they are.  Angles are exact to about
 * 2^-25 of a radian, 2^-53 of p f and 2^-64 p of a turn, at any position.  A frequency
 * that is not finite makes its pair NaN.
 *
 * RMS norm of a head, before its rotation: u = x / sqrt(mean(x^2) + epsilon) * gamma,
 * with binary32 sums of squares.
 */
typedef struct b200norm_rotation {
  const void* positions;   /* int32 or int64: of token t of sequence b at
                              [b * batch_stride + t * token_stride]; any sign */
  int position_bytes;      /* 4 or 8 */
  int64_t batch_stride, token_stride; /* >= 0, in elements */
  const double* inv_freq;  /* device, rotary_size / 2 frequencies in radians per position
                              (b200norm_rotary_frequencies makes them) */
  int64_t rotary_size;     /* R: even, in [0, head_size]; 0: no rotation, and positions
                              and inv_freq are not read */
  int interleaved;         /* 0: pairs (i, i + R / 2); 1: pairs (2 i, 2 i + 1) */
  float scale;             /* 1, or what a scaled context wants; finite */
} b200norm_rotation;

/* Queries, or keys: element d of head h of token t of sequence b of a tensor is at
 * [b * strides[0] + t * strides[1] + h * strides[2] + d], strides >= 0 in elements.  So
 * heads may lie inside a product's rows, next to others, or be permuted. */
typedef struct b200norm_heads {
  const void* x;
  void* y;                 /* the result: x itself with x's strides (in place), or no
                              element of any input */
  const void* gamma;       /* M, (head_size), or NULL (ones); NULL for b200norm_rotary */
  int64_t heads;           /* 0: none (the pointers are not used) */
  int64_t x_strides[3], y_strides[3];
} b200norm_heads;

/*
 * y = round_T(rotation(x)), or round_T(rotation(u)), of queries and of keys, in one
 * launch.  Either tensor may be NULL.
 *
 *   batch, seq   tokens are (batch, seq); their product may be 2^31 - 1 at most,
 *                times the heads 2^40.
 *   head_size    elements of a head, in [1, 1024]; heads: at most 2^16.
 *   T, M         element types of heads and gamma; M is T or B200NORM_F32.
 *   epsilon      >= 0 and not NaN.
 *
 * The outputs may interleave (heads next to one another in one row), but no element
 * may be written twice.  batch * seq == 0 is a no-op.
 */
B200NORM_API b200norm_status b200norm_rotary(const b200norm_heads* queries,
                                             const b200norm_heads* keys,
                                             const b200norm_rotation* rotation, int64_t batch,
                                             int64_t seq, int64_t head_size, b200norm_dtype T,
                                             int inverse, b200norm_stream_t stream);

B200NORM_API b200norm_status b200norm_head_rms_rotary(
    const b200norm_heads* queries, const b200norm_heads* keys, const b200norm_rotation* rotation,
    int64_t batch, int64_t seq, int64_t head_size, b200norm_dtype T, b200norm_dtype M,
    float epsilon, b200norm_stream_t stream);

/* The same of the gradient. */
typedef struct b200norm_heads_grad {
  const void* dy;          /* T: gradient of y */
  const void* x;           /* T: the forward call's input */
  const void* gamma;       /* M, or NULL (ones) */
  void* dx;                /* T, or NULL when not wanted */
  void* dgamma;            /* M, (head_size), or NULL when not wanted */
  int64_t heads;           /* 0: none (the pointers are not used: dgamma keeps what it has) */
  int64_t dy_strides[3], x_strides[3], dx_strides[3];
} b200norm_heads_grad;

/*
 * Gradients of b200norm_head_rms_rotary.  With da the inverse rotation of dy, r =
 * 1 / sqrt(mean(x^2) + epsilon), v = x r and g = da * gamma, over each head:
 *
 *   dx     = round_T(r * (g - v * mean(g * v)))
 *   dgamma = round_M(sum over tokens and heads of da * v)
 *
 *   workspace  at least b200norm_head_rms_rotary_grad_workspace_size() bytes, 256-byte
 *              aligned; its contents before the call do not matter.  Calls that share
 *              one must not overlap on the device.
 *
 * Outputs overlap nothing (dx of queries and of keys may interleave).  Sums are
 * binary32, in a fixed order (equal calls give equal bits).  batch * seq == 0 stores
 * zeros in dgamma.
 */
B200NORM_API size_t b200norm_head_rms_rotary_grad_workspace_size(int64_t batch, int64_t seq,
                                                                 int64_t query_heads,
                                                                 int64_t key_heads,
                                                                 int64_t head_size);

B200NORM_API b200norm_status b200norm_head_rms_rotary_grad(
    const b200norm_heads_grad* queries, const b200norm_heads_grad* keys,
    const b200norm_rotation* rotation, int64_t batch, int64_t seq, int64_t head_size,
    b200norm_dtype T, b200norm_dtype M, float epsilon, void* workspace, size_t workspace_bytes,
    b200norm_stream_t stream);

/*
 * Frequencies of rotary positions: f_i = base^(-2 i / rotary_size), i < rotary_size / 2,
 * scaled for a context longer than the one the model was trained on:
 *
 *   scaling 0  as they are (factor, original_length, low and high are not used)
 *           1  positions interpolated: f_i / factor
 *           2  another base: base * factor^(R / (R - 2)), which divides the lowest
 *              frequency by factor and keeps the highest (R > 2)
 *           3  by the turns t_i = original_length * f_i / (2 pi) that a pair makes over
 *              the original length: kept for t_i >= high, divided by factor for
 *              t_i <= low, and a mixture in proportion between them
 *
 * inv_freq is a HOST array of rotary_size / 2.  rotary_size is even, in [2, 1024];
 * base > 0; factor > 0; original_length > 0; 0 <= low < high; all finite.  Touches no
 * GPU.  (Scaled contexts often want a `scale` of 0.1 ln(factor) + 1 in the rotation.)
 */
B200NORM_API b200norm_status b200norm_rotary_frequencies(double* inv_freq, int64_t rotary_size,
                                                         double base, int scaling, double factor,
                                                         double original_length, double low,
                                                         double high);

#ifdef __cplusplus
}
#endif

#endif /* B200NORM_H */
