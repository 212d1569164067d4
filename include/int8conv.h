/*
 * int8conv.h -- C ABI of the GB300 (sm_103a) INT8 2-D convolution forward
 * propagation library, libint8conv.so.
 *
 * The operation is conv_fprop as defined in the cuDNN documentation page
 * "Convolutions", section "Convolution Fprop" (response = image * filter),
 * with the arguments of its "Python API" list: image, weight, pre_padding,
 * post_padding, stride, dilation, convolution_mode, compute_data_type; the
 * "symmetric-padding overload" (padding in place of pre/post) is
 * conv_params_set_symmetric_padding below.  Tensors are described as in the
 * forum thread "INT8 convolution using cuDNN Python Frontend": logical dims
 * plus one element stride per logical dim.
 *
 * Semantics (integer arithmetic throughout, exact):
 *   Y[n,k,p,q] = sum_{c,r,s} X[n,c,h,w] * W[k,c,r',s']   (+ bias[k]) (ReLU)
 *     h = p*stride[0] - pre_padding[0] + r*dilation[0]
 *     w = q*stride[1] - pre_padding[1] + s*dilation[1]
 *     taps outside the image contribute 0 (zero padding)
 *     (r',s') = (r,s) for CONV_CROSS_CORRELATION,
 *               (R-1-r, S-1-s) for CONV_CONVOLUTION (the filter flipped in
 *               both spatial axes; channels are not flipped)
 *     P = floor((H + pre[0] + post[0] - dilation[0]*(R-1) - 1) / stride[0]) + 1
 *     Q likewise with index 1.
 *   The accumulator is exact: the validator rejects shapes for which
 *   C*R*S*2^14 could exceed 2^31-1.  The bias is added with two's-complement
 *   int32 wrap-around, then ReLU is max(0, .).
 *
 * Ownership: the caller owns every buffer and the stream.  conv_fprop never
 * allocates and never synchronises; all work is queued on `stream`.  The
 * library keeps one small device status word per device (see
 * conv_device_status) and, in static host memory, the plan caches described
 * at conv_shutdown.
 *
 * Errors: every entry point returns a conv_status; nothing is thrown across
 * the ABI.  Descriptors are validated before anything is launched (a call
 * whose descriptors and parameters equal those of an earlier, validated call
 * reuses that validation from the plan cache).  Kernel launch failures give
 * CONV_ERR_CUDA.  A kernel whose internal wait runs out of time records
 * CONV_ERR_DEVICE_TIMEOUT in the
 * device status word and returns early; conv_device_status reports it.
 *
 * Thread safety: all entry points are reentrant; concurrent calls on
 * different streams are independent (they share only the status word).
 */
#ifndef INT8CONV_H
#define INT8CONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CONV_OK = 0,
    CONV_ERR_NULL_PTR = 1,            /* a required pointer is NULL */
    CONV_ERR_RANK = 2,                /* a descriptor's rank is not 4 */
    CONV_ERR_DTYPE = 3,               /* image/filter not INT8; output not INT32 (INT8 with CONV_EPILOGUE_INT8_OUT);
                                         a channel operator's matrix of another type than it takes */
    CONV_ERR_SHAPE_MISMATCH = 4,      /* C, K, N or the output dims disagree */
    CONV_ERR_BAD_STRIDES = 5,         /* non-positive stride of a dim > 1, or elements alias */
    CONV_ERR_BUFFER_TOO_SMALL = 6,    /* descriptor's capacity_bytes below its extent */
    CONV_ERR_BAD_PARAM = 7,           /* stride/dilation < 1, padding < 0, empty output, bad mode */
    CONV_ERR_OVERFLOW_RISK = 8,       /* C*R*S*2^14 > 2^31-1: int32 could overflow */
    CONV_ERR_UNSUPPORTED_COMPUTE = 9, /* compute_dtype other than CONV_INT32 */
    CONV_ERR_ALIGNMENT = 10,          /* a forced algorithm cannot take these pointers/strides; an address that
                                         is no multiple of its element's size (channel operators) */
    CONV_ERR_CUDA = 11,               /* a CUDA runtime call failed */
    CONV_ERR_DEVICE_TIMEOUT = 12,     /* a kernel gave up waiting (see conv_device_status) */
    CONV_ERR_WORKSPACE = 13,          /* workspace NULL or smaller than conv_fprop_workspace_size */
    CONV_ERR_UNSUPPORTED_DEVICE = 14, /* the current device is not sm_103 */
    CONV_ERR_OVERLAP = 15,            /* output bytes overlap an input or the workspace */
    CONV_ERR_TOO_LARGE = 16,          /* an extent or offset exceeds the library's index range */
    CONV_ERR_STATIC_WORKSPACE_LIMIT = 17 /* call needs more scratch than CONV_STATIC_WORKSPACE_BYTES */
} conv_status;

/* The convolution entry points take CONV_INT8 and CONV_INT32; the float types
 * belong to the channel operators (conv_linear, conv_layer_norm and what
 * follows them below).  The 8-bit floats are the ones with 4 exponent and 3
 * mantissa bits (largest 448, no infinity) and with 5 and 2 (largest 57344). */
typedef enum {
    CONV_INT8 = 1,
    CONV_INT32 = 2,
    CONV_FLOAT32 = 3,
    CONV_FLOAT16 = 4,
    CONV_BFLOAT16 = 5,
    CONV_FLOAT8_E4M3 = 6,
    CONV_FLOAT8_E5M2 = 7
} conv_dtype;

typedef enum { CONV_CROSS_CORRELATION = 0, CONV_CONVOLUTION = 1 } conv_mode;

/* Algorithm selection; CONV_ALGO_AUTO lets the planner choose. */
typedef enum {
    CONV_ALGO_AUTO = 0,
    CONV_ALGO_IMPLICIT_GEMM = 1, /* tcgen05 tensor-core implicit GEMM */
    CONV_ALGO_DIRECT_DP4A = 2,   /* CUDA-core direct kernel, 4-way int8 dot products */
    CONV_ALGO_DIRECT_GENERIC = 3, /* CUDA-core direct kernel, any strides */
    /* the tensor-core kernel with the image gathered by per-thread global
       loads instead of TMA im2col tiles (what CONV_ALGO_IMPLICIT_GEMM falls
       back to when a TMA im2col map cannot express the call: stride > 8,
       padding or reach beyond the map's corner range) */
    CONV_ALGO_IMPLICIT_GEMM_GLOBAL_LOADS = 4
} conv_algo;

/* Epilogue flags (bit set). */
#define CONV_EPILOGUE_BIAS 1u /* add int32 bias[k] */
#define CONV_EPILOGUE_RELU 2u /* max(0, .) after the bias */
/* int8 output: after bias and ReLU, v -> floor((v + 2^(s-1)) / 2^s) for
 * s = out_shift > 0 (a rounding right shift; s = 0 leaves v), then clamped to
 * [-128, 127].  The output descriptor must then be CONV_INT8 (and must be
 * CONV_INT32 without this flag: an output type is never inferred). */
#define CONV_EPILOGUE_INT8_OUT 4u

/*
 * Tensor descriptor.  dims and strides are in LOGICAL order: [N,C,H,W] for
 * the image and output ([N,K,P,Q]), [K,C,R,S] for the filter.  strides are in
 * elements (not bytes), one per logical dim, as in the forum thread's
 * graph.tensor(dim=..., stride=...).  The stride of a dim of extent 1 is
 * never multiplied by a non-zero index and is ignored.  capacity_bytes is the
 * size of the buffer behind the pointer; the largest addressed element must
 * lie inside it.
 */
typedef struct {
    int32_t dtype;          /* conv_dtype */
    int32_t rank;           /* must be 4 */
    int64_t dims[4];
    int64_t strides[4];
    uint64_t capacity_bytes;
} conv_tensor_desc;

/* conv_fprop attributes (cuDNN "Convolutions": Conv_fprop_attributes setters
 * and the Python argument list).  Index 0 is the H axis, index 1 the W axis. */
typedef struct {
    int64_t pre_padding[2];
    int64_t post_padding[2];
    int64_t stride[2];
    int64_t dilation[2];
    int32_t mode;          /* conv_mode */
    int32_t compute_dtype; /* must be CONV_INT32 */
    uint32_t epilogue;     /* CONV_EPILOGUE_* bits */
    int32_t algo;          /* conv_algo */
    int32_t out_shift;     /* 0..31, with CONV_EPILOGUE_INT8_OUT only (else 0) */
    int32_t reserved;      /* must be 0 */
} conv_fprop_params;

/* Fill *p with: no padding, stride 1, dilation 1, cross-correlation,
 * compute INT32, no epilogue, automatic algorithm, shift 0. */
void conv_params_init(conv_fprop_params *p);

/* The symmetric-padding overload: pre_padding = post_padding = pad. */
void conv_params_set_symmetric_padding(conv_fprop_params *p, const int64_t pad[2]);

/* Stride calculator: fill d for a packed tensor.  layout is one of "NCHW",
 * "NHWC" (image/output) or "KCRS", "KRSC" (filter); dims are logical.
 * capacity_bytes is set to the packed size.  Returns CONV_ERR_BAD_PARAM for
 * an unknown layout or a non-positive dim. */
conv_status conv_tensor_desc_packed(conv_tensor_desc *d, int32_t dtype, const int64_t dims[4],
                                    const char *layout);

/* Output dims [N,K,P,Q] for image x, filter w and params p. */
conv_status conv_fprop_output_dims(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                   const conv_fprop_params *p, int64_t out_dims[4]);

/* Full host-side validation of a call (no device work).  bias_elems is the
 * number of int32 elements behind the bias pointer (ignored unless the bias
 * flag is set; must be >= K when it is). */
conv_status conv_fprop_validate(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                const conv_tensor_desc *y, const conv_fprop_params *p,
                                int64_t bias_elems);

/* Algorithm the planner would run for this call (after validation). */
conv_status conv_fprop_plan(const conv_tensor_desc *x, const conv_tensor_desc *w,
                            const conv_tensor_desc *y, const conv_fprop_params *p,
                            int32_t *algo_out);

/* Bytes of device workspace conv_fprop needs for this call (0 for the direct
 * kernels; for the implicit GEMM the repacked half-precision filter, plus
 * the int32 partial sums of tiles whose reduction is cut over several SMs
 * (calls with fewer tiles than SMs and long reductions, or a short partial
 * last round of tiles), plus a channels-last copy of the image when its
 * strides allow neither direct channels-last loads nor whole-row loads: an
 * NCHW-like image, each channel's rows contiguous, is read in place when its
 * rows are at most 192 bytes (a multiple of 16), the stride along W is 1 and
 * Q, the pre-padding along W and every tap offset s*dilation_w are multiples
 * of 4, for K <= 192).  The caller allocates it, 256-byte
 * aligned.  The size assumes a
 * 16-byte-aligned image pointer (as every cudaMalloc or PyTorch allocation
 * is); with a misaligned one the image needs the copy too, and conv_fprop
 * returns CONV_ERR_WORKSPACE if the workspace cannot hold it. */
conv_status conv_fprop_workspace_size(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                      const conv_tensor_desc *y, const conv_fprop_params *p,
                                      size_t *bytes);

/* Number of kernels conv_fprop launches for this call, under the same
 * assumption of 16-byte aligned image and filter pointers: 0 for an empty
 * output, 1 for the direct kernels; for the implicit GEMM the filter repack
 * (none when the 128- or 192-column kernel converts the filter itself: K <=
 * 192, a channels-last (or copied) image, a filter with contiguous channels
 * and 16-byte aligned strides), the channels-last image copy when needed,
 * the convolution, and the reduction of cut tiles when the call cuts them.
 * (conv_fprop_pack_filter launches the repack, conv_fprop_prepacked the
 * others, the convolution then reading the repacked filter.)
 * Errors as conv_fprop_validate; CONV_ERR_NULL_PTR if count is NULL. */
conv_status conv_fprop_kernel_count(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                    const conv_tensor_desc *y, const conv_fprop_params *p, int32_t *count);

/* Tile shape of the implicit-GEMM convolution for this call, under the same
 * alignment assumption: shape[0] output pixels per tile (128), shape[1]
 * output channels per tile (128, 192 or 256: the smallest that covers K),
 * shape[2] the number of tiles, shape[3] the number of work units (whole
 * tiles, plus the runs of the tiles cut along the reduction: calls with
 * fewer tiles than SMs and long reductions, or a short partial last round,
 * on the current device).  All four are 0 for the direct kernels and for
 * an empty output.  Errors as conv_fprop_validate; CONV_ERR_NULL_PTR if
 * shape is NULL.  Host-only; no device work. */
conv_status conv_fprop_tile_shape(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                  const conv_tensor_desc *y, const conv_fprop_params *p, int64_t shape[4]);

/*
 * Y = conv_fprop(X, W) on `stream` (a cudaStream_t; NULL = legacy default).
 * x_dev, w_dev, y_dev, bias_dev and workspace are device pointers on the
 * current device.  bias_dev holds K int32 values and is read only when
 * p->epilogue has CONV_EPILOGUE_BIAS.  y_dev holds int32 elements, or int8
 * elements with CONV_EPILOGUE_INT8_OUT (as its descriptor says).  The output
 * must not overlap the inputs or the workspace.  Asynchronous: returns after
 * queuing the kernels.
 */
conv_status conv_fprop(const conv_tensor_desc *x, const int8_t *x_dev,
                       const conv_tensor_desc *w, const int8_t *w_dev,
                       const conv_tensor_desc *y, void *y_dev,
                       const int32_t *bias_dev, const conv_fprop_params *p,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * conv_fprop in two halves, for callers that reuse one filter across many
 * images (the filter repack then runs once):
 *   conv_fprop_pack_filter writes the repacked filter into the workspace
 *   (nothing to do for the direct kernels);
 *   conv_fprop_prepacked runs the convolution from that workspace.
 * Both take the same descriptors and params as conv_fprop and validate them
 * the same way; conv_fprop_prepacked still needs w_dev (the direct kernels
 * read the filter itself), and its tensor-core kernels always read the
 * repacked filter, also where conv_fprop would have them convert the filter
 * themselves.  The workspace contents must come from a
 * conv_fprop_pack_filter call with the same filter, descriptors and params;
 * the library cannot check that.  Calling the two in order on one stream is
 * conv_fprop.
 */
conv_status conv_fprop_pack_filter(const conv_tensor_desc *x, const conv_tensor_desc *w, const int8_t *w_dev,
                                   const conv_tensor_desc *y, const conv_fprop_params *p, void *workspace,
                                   size_t workspace_bytes, void *stream);

conv_status conv_fprop_prepacked(const conv_tensor_desc *x, const int8_t *x_dev,
                                 const conv_tensor_desc *w, const int8_t *w_dev,
                                 const conv_tensor_desc *y, void *y_dev,
                                 const int32_t *bias_dev, const conv_fprop_params *p,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * conv_fprop with the image, filter, bias and output in HOST memory (same
 * descriptors and semantics as conv_fprop; x_host, w_host, y_host and
 * bias_host are host pointers, page-locked for the copies to overlap).
 *
 * The filter and bias are copied once; the batch is then processed in a
 * short lead chunk (a quarter of a chunk, so that the copy back to the host
 * starts early) and up to four chunks of whole images on three
 * library-owned streams, so that the
 * copy of chunk c to the device, the convolution of chunk c-1 and the copy
 * of chunk c-2 back to the host run at the same time.  Chunking needs every
 * image in its own byte range of the buffers (batch outermost in memory, as
 * in NCHW or NHWC); otherwise the whole batch is one chunk.
 *
 * device_buffer (device memory, 256-byte aligned, at least
 * conv_fprop_host_buffer_size bytes, owned by the caller) holds the filter,
 * bias, workspace and double-buffered image and output chunks.  The call is
 * asynchronous: it returns after queueing the work, and `stream` (the
 * caller's) is made to wait for its completion, so synchronising `stream`
 * means y_host holds the result.  The streams and events it uses are created
 * on the first call on each device and live until the process exits; calls
 * on one device are queued one after the other.
 */
conv_status conv_fprop_host_buffer_size(const conv_tensor_desc *x, const conv_tensor_desc *w,
                                        const conv_tensor_desc *y, const conv_fprop_params *p,
                                        size_t *bytes);

conv_status conv_fprop_host(const conv_tensor_desc *x, const int8_t *x_host,
                            const conv_tensor_desc *w, const int8_t *w_host,
                            const conv_tensor_desc *y, void *y_host,
                            const int32_t *bias_host, const conv_fprop_params *p,
                            void *device_buffer, size_t device_buffer_bytes, void *stream);

/*
 * conv_fprop without a caller-provided workspace.  (The pages have no
 * counterpart to this entry point; it exists for callers that cannot
 * allocate device memory: a plugin whose host framework owns all device
 * allocations and hands none to it, or a latency-critical loop that must not
 * call cudaMalloc, which may synchronise the device.)
 *
 * Same arguments and results as conv_fprop, minus the workspace: the scratch
 * (the repacked filter; the int32 partial sums of the tiles whose reduction
 * a call cuts into runs for different SMs, which on a 32 x 256 x 56 x 56
 * 3x3 call are 18.9 MB of the 20.1 MB it needs; and, when the image strides
 * need it, a channels-last image copy) lives in a device array of
 * CONV_STATIC_WORKSPACE_BYTES that is part of the library, so every GPU that
 * loads the library holds that much memory until the process exits.  Calls needing more scratch than that
 * return CONV_ERR_STATIC_WORKSPACE_LIMIT and launch nothing
 * (conv_fprop_workspace_size tells the need in advance).  It allocates
 * nothing: no cudaMalloc, cudaFree or allocating library routine.
 *
 * The first call on a device looks up that device's copy of the array (one
 * cudaGetSymbolAddress with the device current), so make that first call
 * before any stream capture.  The address is kept per device ordinal for
 * the life of the device's primary context (the runtime's context): after
 * cudaDeviceReset, or with another context made current on that ordinal, it
 * is stale; use conv_fprop with a workspace there.  Every call shares the one array and the
 * kernels overwrite all scratch they read, so nothing needs clearing between
 * calls; but calls whose work overlaps on the GPU (different streams, or
 * different host threads) race on the array: order them on one stream.
 */
#define CONV_STATIC_WORKSPACE_BYTES (32u << 20)

conv_status conv_fprop_static_workspace(const conv_tensor_desc *x, const int8_t *x_dev,
                                        const conv_tensor_desc *w, const int8_t *w_dev,
                                        const conv_tensor_desc *y, void *y_dev,
                                        const int32_t *bias_dev, const conv_fprop_params *p,
                                        void *stream);

/*
 * Gradients of the same convolution (cuDNN "Convolutions", sections
 * "Convolution Dgrad" and "Convolution Wgrad": the data and weight gradients
 * during backpropagation).  The pages name the operations and their
 * arguments but print no formula; they are computed as the transposes of
 * the forward sum:
 *
 *   dX[n,c,h,w]   = sum over k, r, s of dY[n,k,p,q] * W[k,c,r',s'],
 *                   p = (h + pre_h - r*dil_h) / stride_h when that division
 *                   is exact and 0 <= p < P (q likewise),
 *   dW[k,c,r',s'] = sum over n, p, q of dY[n,k,p,q] * X[n,c,h,w],
 *                   h = p*stride_h - pre_h + r*dil_h (w likewise), zero
 *                   outside the image,
 *
 * with (r', s') = (r, s) in CROSS_CORRELATION and (R-1-r, S-1-s) in
 * CONVOLUTION, exactly as conv_fprop pairs image and filter elements.
 *
 * Descriptors: dy is the loss gradient, int8 [N,K,P,Q]; w and x as in
 * conv_fprop (int8); dx is int32 [N,C,H,W] and dw int32 [K,C,R,S], any
 * strides.  H, W (dgrad) and R, S (wgrad) come from the output descriptor;
 * P, Q must be the forward output size for them.  p is the forward call's
 * parameters with no epilogue (epilogue and out_shift 0) and algo AUTO,
 * IMPLICIT_GEMM or DIRECT_GENERIC.  Results are exact: dgrad needs
 * K*R*S*2^14 <= 2^31-1 and wgrad N*P*Q*2^14 <= 2^31-1, else
 * CONV_ERR_OVERFLOW_RISK.
 *
 * conv_dgrad runs on the tensor cores as stride_h*stride_w forward
 * convolutions of dY, one per residue class (h mod stride_h, w mod
 * stride_w) of dX's pixels, each by the filter taps that reach that class
 * (taken backwards, K and C exchanged) with stride 1, each in its own part of
 * the workspace; the filters of all classes are repacked by one launch on
 * `stream`, a dY that is neither channels-last nor read in place by rows
 * (as for conv_fprop's image) is copied once for all classes,
 * and the classes run as one kernel launch on `stream` (each on its share
 * of the SMs) when they use the same kernel variant and cut no tiles;
 * otherwise side by side on up to four library-owned streams forked from
 * `stream` and joined back to it (events; streams and events are created on
 * the first such call on a device, so make that call outside a stream
 * capture; one such call at a time per device forks and joins, the others
 * wait on a host mutex); a class no tap reaches is written with zeros.
 * More than 64 classes take the CUDA-core kernel.  conv_wgrad runs on the
 * tensor cores as a forward convolution of the image (batch and channel
 * dims exchanged) by dY (its batch as channels, its pixels as taps) when the
 * tensor-core kernel can express it; with a batch of at most 32 it folds T
 * = min(64 / N, Q, 8) columns of dY into the channels, reading a copy of
 * the image T times its size.  Those routes need the workspace the
 * *_workspace_size call reports (256-byte aligned, caller-owned; for dgrad
 * it holds every class's filter repacked to f16 blocks, for wgrad dY
 * repacked to f16 blocks, about 2*K*P*ceil(Q/T)*64 bytes (T = 1 unfolded,
 * times ceil(N/64)), plus the int32 partial sums of the reduction split over
 * the SMs, plus the folded image copy, C*H*U*ceil(T*N/16)*16 bytes with U
 * about T*stride_w*ceil(Q/T) + dilation_w*(S-1)).  Other calls, and algo
 * DIRECT_GENERIC, run CUDA-core kernels and need none; IMPLICIT_GEMM on a
 * call that cannot take the tensor cores returns CONV_ERR_ALIGNMENT.
 * Pointers are device pointers on the current device, outputs must not
 * overlap inputs or the workspace; the calls are asynchronous on `stream`
 * and allocate nothing.  An empty dX (N, C, H or W zero) is a no-op; an
 * empty batch in conv_wgrad writes an all-zero dW and reads neither input,
 * so x_dev and dy_dev may then be null.
 */
conv_status conv_dgrad_workspace_size(const conv_tensor_desc *dy, const conv_tensor_desc *w,
                                      const conv_tensor_desc *dx, const conv_fprop_params *p, size_t *bytes);
conv_status conv_dgrad(const conv_tensor_desc *dy, const int8_t *dy_dev, const conv_tensor_desc *w,
                       const int8_t *w_dev, const conv_tensor_desc *dx, int32_t *dx_dev,
                       const conv_fprop_params *p, void *workspace, size_t workspace_bytes, void *stream);
conv_status conv_wgrad_workspace_size(const conv_tensor_desc *x, const conv_tensor_desc *dy,
                                      const conv_tensor_desc *dw, const conv_fprop_params *p, size_t *bytes);
conv_status conv_wgrad(const conv_tensor_desc *x, const int8_t *x_dev, const conv_tensor_desc *dy,
                       const int8_t *dy_dev, const conv_tensor_desc *dw, int32_t *dw_dev,
                       const conv_fprop_params *p, void *workspace, size_t workspace_bytes, void *stream);

/* Synchronise `stream`, then read and clear the current device's status
 * word: CONV_OK, or CONV_ERR_DEVICE_TIMEOUT if a kernel gave up waiting
 * since the last call. */
conv_status conv_device_status(void *stream);

/* Self-test of the timeout path: launches one kernel that waits on a barrier
 * nobody signals, with a limit of `limit_us` microseconds, so that it records
 * CONV_ERR_DEVICE_TIMEOUT and exits.  Returns the launch status. */
conv_status conv_selftest_wait_timeout(uint32_t limit_us, void *stream);

/*
 * Peak microbenchmark: the measured rates of the instruction routes an exact
 * int8 product can take on the current device, and its copy bandwidth.  The
 * pages quote no peak; the benchmark divides by these (or by the driver's
 * measured bf16 rate and copy bandwidth) instead of a datasheet figure.
 * sm_103a has no integer kind of tcgen05.mma, so the routes are:
 *   tcgen05_f16_tflops   tcgen05.mma.cta_group::1.kind::f16, M=128 N=256
 *                        K=16, f32 accumulators in tensor memory, one CTA
 *                        per SM issuing back to back (the route the
 *                        convolution kernel takes, exact by grouping);
 *   mma_sync_s8_tops     warp-level mma.sync m16n8k32 s8 x s8 -> s32;
 *   mma_sync_f16_tflops  warp-level mma.sync m16n8k16 f16 x f16 -> f32;
 *   dp4a_tops            the CUDA cores' dp4a (4 products + 4 adds);
 *   hbm_copy_gbs         read + write bytes per second of a 16-byte copy
 *                        kernel over the two halves of `scratch` (0 when
 *                        scratch_bytes is below 512 MiB + 4 KiB);
 *   sm_mhz               SM clock during the tcgen05 run (clock64 cycles per
 *                        global-timer nanosecond).
 * Rates count 2 operations per multiply-add, dense.  Each kernel runs about
 * a millisecond (best of three launches timed with events on `stream`).
 * `scratch`: caller-owned device buffer, 256-byte aligned, at least 1 MiB
 * (timing records; the copy uses the rest).  Synchronises `stream`; not
 * for use inside a stream capture.  Errors: CONV_ERR_NULL_PTR,
 * CONV_ERR_WORKSPACE (scratch too small or misaligned), CONV_ERR_CUDA,
 * CONV_ERR_DEVICE_TIMEOUT (an MMA completion wait ran out).
 */
typedef struct {
    double tcgen05_f16_tflops;
    double mma_sync_s8_tops;
    double mma_sync_f16_tflops;
    double dp4a_tops;
    double hbm_copy_gbs;
    double sm_mhz;
} conv_peak_rates;

conv_status conv_measure_peak_rates(void *scratch, size_t scratch_bytes, conv_peak_rates *out, void *stream);

/*
 * Plan caches (the cuDNN-frontend tutorial's kernel/plan cache, for repeated
 * calls of one shape): conv_fprop, its two halves, the static-workspace and
 * host-buffer variants and the gradients' forward convolutions keep
 *   - the validated geometry, algorithm and tensor-core plan of a call,
 *     keyed by the three descriptors, the parameters, the device and whether
 *     the image pointer is 16-byte aligned (64 entries), and
 *   - the tensor-core kernel's launch arguments with their encoded TMA
 *     tensor maps, keyed by that plan and the 16-byte alignment of the image
 *     and output pointers (32 entries); a call with other buffers re-targets
 *     the cached maps to its addresses (cuTensorMapReplaceAddress) instead of
 *     encoding them again;
 *   - for conv_dgrad, the residue classes with their tensor-core plans,
 *     keyed like the first cache on dY, W, dX and the parameters (16
 *     entries).
 * A call whose key is cached skips validation, planning and map encoding;
 * its pointer checks (null, overlap, workspace) still run.  The caches are
 * library-owned host memory, shared by all threads (a mutex guards them),
 * least recently used entries giving way.  Cache lookups make no CUDA calls,
 * so cached calls stay capturable in CUDA graphs.
 *
 * conv_shutdown empties the three caches (their memory is static; nothing is
 * freed or allocated; the data gradient's side streams and events stay).  Call it when no other thread is inside a library
 * call.  conv_plan_cache_stats reads the hit and miss counts since the
 * library was loaded.
 */
void conv_shutdown(void);
conv_status conv_plan_cache_stats(uint64_t *plan_hits, uint64_t *plan_misses, uint64_t *launch_hits,
                                  uint64_t *launch_misses);

/*
 * Channel operators: what a network does between and after its convolutions
 * on matrices whose rows are pixels or tokens and whose columns are channels
 * (a channels-last image [N,H,W,C] is the matrix [N*H*W, C]).
 *
 * Matrix descriptor: rows x cols with one element stride each, like the
 * tensor descriptors above.  Strides are positive and no two elements may
 * share an address (a broadcast stride of 0 is refused); the stride of a dim
 * of extent 1 is ignored.  Both orders and any padding are taken, rows or
 * columns may be the contiguous dim.
 */
typedef struct {
    int32_t dtype;     /* conv_dtype */
    int32_t reserved;  /* must be 0 */
    int64_t rows;
    int64_t cols;
    int64_t row_stride; /* elements from one row to the next */
    int64_t col_stride; /* elements from one column to the next */
    uint64_t capacity_bytes;
} conv_matrix_desc;

/* Activations of conv_linear:
 *   CONV_ACT_RELU       max(0, z)
 *   CONV_ACT_GELU       z * Phi(z), Phi the standard normal distribution
 *                       (0 at minus infinity, its limit); Phi is off by 3e-7
 *                       at most, which is an absolute error: the value is off
 *                       by 0.24 % of itself at z = -4, 2.1 % at -5
 *   CONV_ACT_GELU_TANH  z/2 * (1 + tanh(sqrt(2/pi) * (z + 0.044715 z^3)))
 *   CONV_ACT_SILU       z / (1 + exp(-z)) */
typedef enum {
    CONV_ACT_NONE = 0,
    CONV_ACT_RELU = 1,
    CONV_ACT_GELU = 2,
    CONV_ACT_GELU_TANH = 3,
    CONV_ACT_SILU = 4
} conv_activation;

typedef struct {
    int32_t activation;  /* conv_activation */
    int32_t bias_dtype;  /* type of the bias (of its gradient, in conv_linear_grad): CONV_FLOAT32 or x's type;
                            ignored without one */
    int32_t reserved[2]; /* must be 0 */
} conv_linear_params;

/*
 * Matrix product with bias, activation and residual:
 *   z[m,n] = sum_k x[m,k] * w[n,k] + bias[n]
 *   y[m,n] = act(z[m,n]) + residual[m,n],   preact[m,n] = z[m,n]
 * x [M,K] and w [N,K] are both CONV_FLOAT16 or both CONV_BFLOAT16; y [M,N]
 * is of x's type or CONV_FLOAT32, residual [M,N] of y's type, preact [M,N]
 * of x's type.  Products are exact and summed in 32 bits; bias, activation
 * and residual are applied to the 32-bit sum, and y and preact are each
 * rounded once (to nearest even; f16 overflows to infinity).
 * bias_dev, residual (with residual_dev) and preact (with preact_dev) may be
 * NULL: none.  residual may be the same matrix as y (same address and
 * strides, then y is updated in place); any other overlap of an output with
 * an input, the other output or the workspace is refused.
 * M = 0 or N = 0 does nothing; K = 0 gives act(bias) + residual.
 *
 * Workspace: conv_linear_workspace_size bytes, 256-byte aligned (may be NULL
 * when that is 0).  It holds a packed copy of each of x and w that the
 * tensor-memory accelerator cannot read in place: unless one of the
 * strides is 1, the other one a multiple of 8 elements and the address
 * 16-byte aligned; and the partial sums of products whose reduction is cut
 * into runs (long reductions with few output tiles, or a short last round of
 * tiles).  x_dev and w_dev of the size query are the addresses the
 * call will use (read only for their alignment; NULL counts as aligned).
 * Asynchronous on `stream`; nothing is allocated and nothing synchronises.
 * Results are the same from run to run: no sum's order depends on timing.
 *
 * Errors: CONV_ERR_NULL_PTR; CONV_ERR_DTYPE; CONV_ERR_BAD_PARAM (negative
 * extent, unknown activation, reserved fields not 0); CONV_ERR_SHAPE_MISMATCH;
 * CONV_ERR_BAD_STRIDES; CONV_ERR_BUFFER_TOO_SMALL; CONV_ERR_ALIGNMENT (an
 * address that is not a multiple of its element's size); CONV_ERR_TOO_LARGE
 * (an extent of 2^31 - 256 or more); CONV_ERR_OVERLAP; CONV_ERR_WORKSPACE;
 * CONV_ERR_CUDA; CONV_ERR_UNSUPPORTED_DEVICE.  A refused call launches
 * nothing.
 */
conv_status conv_linear_workspace_size(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                       const void *w_dev, size_t *bytes);

conv_status conv_linear(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w, const void *w_dev,
                        const void *bias_dev, const conv_matrix_desc *residual, const void *residual_dev,
                        const conv_matrix_desc *preact, void *preact_dev, const conv_matrix_desc *y, void *y_dev,
                        const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gradients of conv_linear for the loss gradient dy [M,N] (of x's type):
 *   dz = dy * act'(preact)     (dz = dy for CONV_ACT_NONE)
 *   dx = dz w,  dw = dz^T x,  dbias = sum over the rows of dz
 * preact [M,N] is the pre-activation conv_linear wrote; it is required with
 * an activation and not read without one.  The residual's gradient is dy
 * itself.  dx [M,K] and dw [N,K] are of x's type or CONV_FLOAT32, dbias [N]
 * of p->bias_dtype.  Each of dx (with dx_dev), dw (with dw_dev) and
 * dbias_dev may be NULL: not computed; at least one is wanted.  With an
 * activation dz is rounded once to x's type before the products (as a
 * stored gradient would be); dbias sums it unrounded, in 32 bits.
 * ReLU's slope at 0 is 0, and so it is at a NaN; the other slopes of a NaN are
 * NaN.  At an infinite pre-activation (a 16-bit one may have overflowed) every
 * slope is its limit, 1 or 0.  M = 0 gives dw = 0 and dbias = 0; N = 0 gives
 * dx = 0.
 *
 * The workspace (conv_linear_grad_workspace_size bytes, 256-byte aligned)
 * holds dz where it is not dy itself, the partial sums of dbias, and packed
 * copies and partial sums as for conv_linear; the size query takes the same descriptors and
 * addresses as the call.  Errors, asynchrony and repeatability as for
 * conv_linear.
 */
conv_status conv_linear_grad_workspace_size(const conv_matrix_desc *dy, const void *dy_dev,
                                            const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                            const void *w_dev, const conv_linear_params *p, size_t *bytes);

conv_status conv_linear_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *x,
                             const void *x_dev, const conv_matrix_desc *w, const void *w_dev,
                             const conv_matrix_desc *preact, const void *preact_dev, const conv_matrix_desc *dx,
                             void *dx_dev, const conv_matrix_desc *dw, void *dw_dev, void *dbias_dev,
                             const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream);

typedef struct {
    float eps;           /* > 0, finite: added to the variance */
    float scale;         /* finite, not 0: x is taken as scale * x (1 for float inputs as they are) */
    int32_t param_dtype; /* type of gain and shift (and of their gradients): CONV_FLOAT32, or y's type (dx's) */
    int32_t reserved;    /* must be 0 */
} conv_layer_norm_params;

/*
 * Layer norm of every row of x [M,C]: with v = scale * x,
 *   mean = sum v / C,  var = sum (v - mean)^2 / C,  rstd = 1 / sqrt(var + eps)
 *   y = (v - mean) * rstd * gain + shift
 * x is CONV_FLOAT32, CONV_FLOAT16, CONV_BFLOAT16 or CONV_INT32: conv_fprop's
 * channels-last accumulators are normalised as they are, `scale` being the
 * step of the quantised product (integers above 2^24 are rounded to 32-bit
 * floats).  y [M,C] is CONV_FLOAT32, CONV_FLOAT16 or CONV_BFLOAT16.
 * gain_dev and shift_dev hold C values of param_dtype and may be NULL (1 and
 * 0); mean_dev and rstd_dev receive M 32-bit floats and may be NULL.
 * All arithmetic is in 32 bits, the variance from the differences to the
 * mean; y is rounded once.  y may be the same matrix as x when the types
 * have one size (same address and strides).  No workspace.  M = 0 does
 * nothing; C must be at least 1.  A row with an infinity or a NaN gives NaN
 * in that row alone.
 * Errors as for conv_linear (CONV_ERR_BAD_PARAM also for eps and scale).
 */
conv_status conv_layer_norm(const conv_matrix_desc *x, const void *x_dev, const void *gain_dev,
                            const void *shift_dev, const conv_matrix_desc *y, void *y_dev, float *mean_dev,
                            float *rstd_dev, const conv_layer_norm_params *p, void *stream);

/*
 * Gradients of conv_layer_norm (float x, scale 1) for the loss gradient
 * dy [M,C] (of x's type), with the mean and rstd that the forward call wrote:
 *   n = (x - mean) * rstd,  t = dy * gain
 *   dx = rstd * (t - sum t / C - n * sum (t n) / C) + residual_grad
 *   dgain = sum over the rows of dy * n,  dshift = sum over the rows of dy
 * residual_grad [M,C] (of x's type; NULL: none) is the gradient that reaches
 * x past the norm, through a residual connection.  dx [M,C] is of x's type.
 * dx (with dx_dev), dgain_dev and dshift_dev may each be NULL: not computed;
 * at least one is wanted.  dx may be the same matrix as residual_grad.
 * Sums run in 32 bits in an order that does not depend on timing.  M = 0
 * gives dgain = dshift = 0.  The workspace
 * (conv_layer_norm_grad_workspace_size bytes, 256-byte aligned) holds
 * partial sums of dgain and dshift.  Errors as for conv_layer_norm;
 * CONV_ERR_DTYPE for an integer x.
 */
conv_status conv_layer_norm_grad_workspace_size(const conv_matrix_desc *x, size_t *bytes);

conv_status conv_layer_norm_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *x,
                                 const void *x_dev, const void *gain_dev, const float *mean_dev,
                                 const float *rstd_dev, const conv_matrix_desc *residual_grad,
                                 const void *residual_grad_dev, const conv_matrix_desc *dx, void *dx_dev,
                                 void *dgain_dev, void *dshift_dev, const conv_layer_norm_params *p, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * 8-bit operands: blocks of 128 elements with a 32-bit scale each.
 *
 * Quantisation of x [M,C] (CONV_FLOAT32, CONV_FLOAT16 or CONV_BFLOAT16): with
 * v = x, or v = x * act'(preact) where an activation is given (the loss
 * gradient before an activation, unrounded; preact [M,C] of CONV_FLOAT16 or
 * CONV_BFLOAT16, or x's type; slopes as in conv_linear_grad),
 *   scale = max(a / L, 2^-126),  q = v / scale rounded to nearest even
 * where a is the largest magnitude of the block and L the largest value of
 * q's type.  (The quotient, by the scale before that is rounded, is exact
 * where 32 bits hold it and within 2^-23 of itself elsewhere: a value of 16
 * bits goes to the nearest 8-bit one, or of two equally near ones to the even.)
 * Blocks are 128 elements of a row (tile 1) or squares of 128 x 128 (tile 128),
 * counted from the first row and column; the last ones may be short.  A block
 * that holds an infinity or a NaN has it as its scale, and everything made of
 * the block is NaN.
 *   q   [M,C], scale  [ceil(M / tile), ceil(C / 128)]   (rows)
 *   qt  [C,M], scale_t [ceil(C / tile), ceil(M / 128)]  (columns: the same of
 *              x transposed, which is what a product over the rows wants)
 * Either pair, or both from one reading of x; at least one is wanted.  q and
 * qt are of one type, CONV_FLOAT8_E4M3 or CONV_FLOAT8_E5M2; the scales are
 * CONV_FLOAT32.  Any strides.  (For tile 128 scale_t is scale transposed.)
 * No workspace.  M = 0 or C = 0 does nothing.
 *
 * Errors: CONV_ERR_NULL_PTR (also a pair half given, and an activation
 * without preact); CONV_ERR_DTYPE; CONV_ERR_BAD_PARAM (tile, activation,
 * reserved fields); CONV_ERR_SHAPE_MISMATCH; CONV_ERR_BAD_STRIDES;
 * CONV_ERR_BUFFER_TOO_SMALL; CONV_ERR_ALIGNMENT; CONV_ERR_TOO_LARGE;
 * CONV_ERR_OVERLAP (an output shares bytes with anything else of the call);
 * CONV_ERR_CUDA; CONV_ERR_UNSUPPORTED_DEVICE.
 */
typedef struct {
    int32_t tile;        /* rows that share a scale: 1 or 128 */
    int32_t activation;  /* conv_activation */
    int32_t reserved[2]; /* must be 0 */
} conv_quantize_params;

conv_status conv_quantize(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *preact,
                          const void *preact_dev, const conv_matrix_desc *q, void *q_dev,
                          const conv_matrix_desc *scale, void *scale_dev, const conv_matrix_desc *qt, void *qt_dev,
                          const conv_matrix_desc *scale_t, void *scale_t_dev, const conv_quantize_params *p,
                          void *stream);

/*
 * conv_linear of 8-bit operands with block scales: with sx and sw the scales
 * of row m's and row n's blocks (b counts 128 elements of K),
 *   z[m,n] = sum_b sx[m,b] * sw[n,b] * (sum over block b of x[m,k] * w[n,k])
 *            + bias[n]
 *   y[m,n] = act(z[m,n]) + residual[m,n],   preact[m,n] = z[m,n]
 * x [M,K] and w [N,K] are CONV_FLOAT8_E4M3 or CONV_FLOAT8_E5M2, each its own,
 * with adjacent columns (any row stride).  x_scale is CONV_FLOAT32 of
 * [M, ceil(K / 128)] (a scale for each row) or [ceil(M / 128), ceil(K / 128)]
 * (for each square), w_scale likewise with N; any strides.  y [M,N] is
 * CONV_FLOAT32, CONV_FLOAT16 or CONV_BFLOAT16, residual [M,N] of y's type,
 * preact [M,N] CONV_FLOAT16 or CONV_BFLOAT16; the bias holds
 * p->bias_dtype, CONV_FLOAT32 or y's type.
 * Products are exact, the sums of a block and over the blocks are in 32 bits,
 * and y and preact are each rounded once.  The two scales of a block are
 * multiplied with each other first, in 32 bits: scales whose product is beyond
 * them are of no use.
 *
 * The gradients are products of the same kind: with w quantised in columns
 * (wt) and the loss gradient dz quantised both ways (dz, dzt),
 *   dx = dz wt^T (M x K over N),  dw = dzt xt^T (N x K over M).
 *
 * M = 0 or N = 0 does nothing; K = 0 gives act(bias) + residual.  residual may
 * be the same matrix as y.  The workspace holds packed copies of x and w
 * unless their rows are 16-byte aligned, and partial sums of products cut
 * into runs.  Workspace rules, asynchrony, repeatability and errors as for
 * conv_linear (CONV_ERR_BAD_STRIDES also for columns of x or w that are not
 * adjacent).
 */
conv_status conv_linear_fp8_workspace_size(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *w,
                                           const void *w_dev, size_t *bytes);

conv_status conv_linear_fp8(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *x_scale,
                            const void *x_scale_dev, const conv_matrix_desc *w, const void *w_dev,
                            const conv_matrix_desc *w_scale, const void *w_scale_dev, const void *bias_dev,
                            const conv_matrix_desc *residual, const void *residual_dev,
                            const conv_matrix_desc *preact, void *preact_dev, const conv_matrix_desc *y, void *y_dev,
                            const conv_linear_params *p, void *workspace, size_t workspace_bytes, void *stream);

/*
 * A residual block's end and the next one's beginning: the norm behind the
 * block, its gate, the residual sum and the norm before the next block.  For
 * a block's output x [M,C] and the stream skip [M,C] that went around it:
 *   n   = x * rx * post_gain, rx = 1 / sqrt(sum x^2 / C + eps)  (post_norm;
 *         otherwise n = x)
 *   sum = skip_scale * skip + branch_scale * gate * n
 *   y   = sum * rs * gain,    rs = 1 / sqrt(sum of sum^2 / C + eps)
 * Every part may be left out: skip (with skip_dev) NULL is none; gate NULL is
 * 1; post_gain_dev and gain_dev NULL are 1; sum NULL is not written, y NULL
 * not computed (at least one of the two is wanted).  With x and y alone this
 * is the root-mean-square norm of x.
 * x is CONV_FLOAT32, CONV_FLOAT16 or CONV_BFLOAT16; skip and sum are of one
 * type, x's or CONV_FLOAT32; y is of x's type or, with y_scale [M,
 * ceil(C / 128)] of CONV_FLOAT32, CONV_FLOAT8_E4M3: quantised as by
 * conv_quantize with tile 1.  gate is [G,C] of CONV_FLOAT32 or x's type, M a
 * multiple of G: row g of it serves rows g M/G up to (g + 1) M/G.  Gains hold
 * C values of param_dtype; post_rstd_dev (rx) and rstd_dev (rs) receive M
 * 32-bit floats and may be NULL.
 * Everything between reading and the rounding of sum and y (each once; y is
 * made of the unrounded sum) is in 32 bits.  sum may be the same matrix as
 * skip, and y or sum the same as x where the types are the same.  C is 1 to
 * 49152.  M = 0 does nothing.  No workspace.  A row with an infinity or a NaN
 * gives NaN in that row alone, and so does one whose sum of squares is beyond
 * 32-bit floats (values of some 2^60 or more).
 * Speed: rows with adjacent columns, x's and skip's starting equally far past a
 * multiple of 8 elements (with an 8-bit y at one), are held in registers where
 * two of each and the parameters fit shared memory: up to 8192 columns of 16
 * bits (not those of 7674 to 8040), fewer of 32.  Others go an element at a
 * time, several times slower.
 * Errors as for conv_layer_norm (CONV_ERR_SHAPE_MISMATCH also where G does
 * not divide M, CONV_ERR_TOO_LARGE also for C).
 */
typedef struct {
    float eps;           /* > 0, finite */
    float skip_scale;    /* finite */
    float branch_scale;  /* finite */
    int32_t post_norm;   /* 0 or 1 */
    int32_t param_dtype; /* type of the gains (and of their gradients): CONV_FLOAT32 or x's type */
    int32_t reserved[3]; /* must be 0 */
} conv_block_norm_params;

conv_status conv_block_norm(const conv_matrix_desc *x, const void *x_dev, const conv_matrix_desc *skip,
                            const void *skip_dev, const conv_matrix_desc *gate, const void *gate_dev,
                            const void *post_gain_dev, const void *gain_dev, const conv_matrix_desc *sum,
                            void *sum_dev, const conv_matrix_desc *y, void *y_dev, const conv_matrix_desc *y_scale,
                            void *y_scale_dev, float *post_rstd_dev, float *rstd_dev,
                            const conv_block_norm_params *p, void *stream);

/*
 * Gradients of conv_block_norm for the loss gradients dy [M,C] of y (of x's
 * type) and dsum [M,C] of sum (what reaches the stream from later blocks; of
 * the stream's type), either of which may be NULL (0), not both; with
 * h = sum as the forward call wrote it and the statistics rx and rs:
 *   t  = dy * gain,  u = h * rs,  dh = dsum + rs * (t - u * sum (t u) / C)
 *   dskip = skip_scale * dh,  db = branch_scale * gate * dh
 *   v  = x * rx (post_norm; else x),  dn = db * post_gain
 *   dx = rx * (dn - v * sum (dn v) / C)  (post_norm; else dx = db)
 *   dgate[g] = branch_scale * post_gain * sum over g's rows of dh * v
 *   dgain = sum over the rows of dy * u,  dpost_gain = sum over the rows of db * v
 * h (sum) and rstd_dev are wanted with dy, x with a post norm or dgate, and
 * post_rstd_dev with a post norm.  Each of dx (of x's type), dskip (of the
 * stream's type: h's and dsum's), dgate ([G,C] of CONV_FLOAT32 or x's type;
 * without a gate G is its number of rows), dgain_dev and dpost_gain_dev (C
 * values of param_dtype; dpost_gain only with a post norm, dgain only with
 * dy) may be NULL: not computed; at least one is wanted.  dskip may be the
 * same matrix as dsum, and dx the same as dy.  Sums are in 32 bits, in an
 * order that does not depend on timing.  M = 0 gives zero for the sums over
 * rows.  C is 1 to 24576.  Speed: as for conv_block_norm, with rows of 16 bits
 * held in registers up to 6649 columns (not those of 4593 to 4608 and 5441 to
 * 5632; with several gates aligned ones only), fewer of 32.
 *
 * The workspace (conv_block_norm_grad_workspace_size bytes, 256-byte aligned)
 * holds partial sums (five lines of C for each of up to 608 blocks, or 2432
 * where C is 512 at most, whatever is wanted); groups is G of gate and dgate (1
 * without them).
 * Errors as for conv_block_norm.
 */
conv_status conv_block_norm_grad_workspace_size(const conv_matrix_desc *x, int64_t groups, size_t *bytes);

conv_status conv_block_norm_grad(const conv_matrix_desc *dy, const void *dy_dev, const conv_matrix_desc *dsum,
                                 const void *dsum_dev, const conv_matrix_desc *x, const void *x_dev,
                                 const conv_matrix_desc *sum, const void *sum_dev, const conv_matrix_desc *gate,
                                 const void *gate_dev, const void *post_gain_dev, const void *gain_dev,
                                 const float *post_rstd_dev, const float *rstd_dev, const conv_matrix_desc *dx,
                                 void *dx_dev, const conv_matrix_desc *dskip, void *dskip_dev,
                                 const conv_matrix_desc *dgate, void *dgate_dev, void *dpost_gain_dev,
                                 void *dgain_dev, const conv_block_norm_params *p, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * Global norm of many gradient tensors, and clipping by it:
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   out  = g * min(1, max_norm / (norm + eps)), rounded once
 * Each tensor is `count` adjacent elements of CONV_FLOAT32, CONV_FLOAT16 or
 * CONV_BFLOAT16; out is of the same type, and NULL for clipping in place
 * (where a factor of 1 writes nothing).  norm_dev receives one 32-bit float.
 * max_norm infinite only takes the norm (out is not written).  The squares are
 * summed in 32 bits over 32 elements and in 64 beyond, with 64-bit squares
 * where 32 bits would overflow or underflow, in an order that depends on
 * neither timing nor addresses.  As the formulas have it, an infinite norm
 * gives a factor of 0 and a NaN one of NaN.
 * Tensors that share bytes (also one that is given twice) are refused, as is
 * an out that shares bytes with any tensor or out but its own.  The table of
 * tensors is read before the call returns.
 * Workspace: conv_clip_grads_workspace_size bytes, 256-byte aligned (partial
 * sums).  Errors: CONV_ERR_NULL_PTR; CONV_ERR_DTYPE; CONV_ERR_BAD_PARAM
 * (n or count negative, max_norm or eps negative or NaN, eps infinite,
 * reserved not 0); CONV_ERR_ALIGNMENT; CONV_ERR_TOO_LARGE (2^45 elements or
 * more in one tensor, 2^31 chunks of 16384 elements in all);
 * CONV_ERR_OVERLAP; CONV_ERR_WORKSPACE; CONV_ERR_CUDA;
 * CONV_ERR_UNSUPPORTED_DEVICE.
 */
typedef struct {
    const void *grad;
    void *out;
    int64_t count;
    int32_t dtype;
    int32_t reserved; /* must be 0 */
} conv_grad_tensor;

conv_status conv_clip_grads_workspace_size(const conv_grad_tensor *tensors, int64_t n, size_t *bytes);

conv_status conv_clip_grads(const conv_grad_tensor *tensors, int64_t n, float max_norm, float eps, float *norm_dev,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Human-readable name of a status. */
const char *conv_status_string(conv_status s);

/* Library version, major*10000 + minor*100 + patch. */
int32_t conv_library_version(void);

#ifdef __cplusplus
}
#endif

#endif /* INT8CONV_H */
