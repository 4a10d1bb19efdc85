/*
 * awq4.h -- C ABI of the MI355X (gfx950) 4-bit-weight GEMM library.
 *
 * The library computes the group-quantised 4-bit-weight linear layer
 *     Y = X . dequant(Wq),   w[k,n] = (q[k,n] - z[k/G,n]) * s[k/G,n]
 * in the first-generation AWQ GEMM weight format, in a decode regime (GEMV,
 * M <= 8) and a prefill regime (GEMM, any M), plus the QQQ-style W4A8 variant
 * (per-token int8 activations x symmetric int4 weights, exact int32
 * accumulation, per-token and per-channel (optionally per-group) scales).
 * Around those layers it has RMS norm with the residual's addition and an
 * 8-bit output, and attention over a paged key/value cache in 4 bits; for
 * mixtures of experts the routing and the same products grouped by expert; and
 * products of E4M3 activations and weights with a scale for each block of 128.
 *
 * Sources (web pages, cited by title and passage):
 *  [P1] vLLM pull request "Speed up AWQ 2.5x with updated kernel": the list of
 *       differences between the old and new AWQ packings (old GEMM order map
 *       [0,2,4,6,1,3,5,7]), and the dispatch snippet (M > 8 -> GEMM, else GEMV;
 *       kernels take inputs, qweight, scales, qzeros, group_size, and the GEMM
 *       a split_k_iters count).
 *  [P2] AutoAWQ pull request "Marlin symmetric quantization and inference":
 *       the symmetric variant without zero points; one workspace per device
 *       rather than per layer.
 *  [P5] vLLM pull request "Support W4A8 quantization for vllm" (QQQ): dynamic
 *       per-token activation quantisation; int4 -> int8 by placing the nibble
 *       in the upper four bits; int32 global reduce through a temporary
 *       buffer; s1 (per token) and s2 (per channel) applied to the output,
 *       with per-group scales in addition for grouped weights; the GEMM
 *       signature (a, b_q_weight, s1, s2, s3, workspace, size_m, size_n,
 *       size_k) with const operands; a missing clamp in packing as a real bug.
 *
 * Conventions for every entry point:
 *  - All tensors are dense, row-major and contiguous, in device memory owned
 *    by the caller (awq_kv4_append takes token strides).  Device pointers must
 *    be 16-byte aligned (AWQ_EALIGN), those of the kv4 calls' index arrays
 *    and awq_moe_*'s index arrays and weights aligned to their type.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *    Work is enqueued on it; no entry point synchronises or allocates device
 *    memory, so all of them are asynchronous and safe to call from several
 *    host threads on different streams.  Faults inside a kernel surface at
 *    the caller's next synchronisation, as for any HIP launch.
 *  - Arguments are validated before anything is enqueued; a call that
 *    returns an error has written nothing.  Validation needs no GPU.
 *  - Return value: AWQ_OK or a negative AWQ_E* status.
 *  - Results are deterministic: the same inputs give the same bits on every
 *    run (split-K partials are summed in a fixed order).
 */
#ifndef AWQ4_H
#define AWQ4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define AWQ_OK 0
#define AWQ_EINVAL (-1)       /* bad shape, null pointer, unknown enum value */
#define AWQ_EUNSUPPORTED (-2) /* valid request this library does not implement (e.g. GEMV with M > 8) */
#define AWQ_EWORKSPACE (-3)   /* workspace missing or smaller than awq_workspace_bytes() */
#define AWQ_EALIGN (-4)       /* a device pointer is not 16-byte aligned */
#define AWQ_EHIP (-5)         /* the HIP runtime reported an error when launching */

/* Activation / scale / output dtypes. */
#define AWQ_DTYPE_F16 0
#define AWQ_DTYPE_BF16 1
#define AWQ_DTYPE_F32 2 /* logits of awq_moe_route only */

/* Packed layouts for awq_pack / awq_unpack. */
#define AWQ_LAYOUT_N8 0  /* AWQ: uint8 vals [rows, cols] in 0..15 -> int32 [rows, cols/8];
                            nibble i of word [r][j] holds column 8j + {0,2,4,6,1,3,5,7}[i] ([P1]) */
#define W4A8_LAYOUT_K8 1 /* W4A8: int8 vals [K=rows, N=cols] in -8..7 -> int32 [K/8, N];
                            nibble i of word [kb][n] holds k = 8kb + {0,4,1,5,2,6,3,7}[i],
                            two's complement (this library's own layout) */

#define AWQ_LAYOUT_V2 2   /* the newer AWQ packing ([P1], list of differences; this library's reading):
                            uint8 vals [rows, cols] in 0..15 -> int32 [rows, ceil(cols/8)];
                            nibble i of word [r][j] holds column 8j + i (identity order map),
                            nibbles past the last column are left 0 (skipped); any cols */

/* Operation ids for awq_workspace_bytes. */
#define AWQ_OP_GEMM_W4A16 0
#define AWQ_OP_GEMV_W4A16 1
#define AWQ_OP_W4A8_GEMM 2
#define AWQ_OP_W4A8_FP8_GEMM 3
/* Of awq_grouped_plan_info only. */
#define AWQ_OP_MOE_GEMM_W4A16 4
#define AWQ_OP_FP8_BLOCK_GEMM 5

/* Human-readable name of a status code (static string, never NULL). */
const char *awq_status_str(int status);

/* Library ABI version (major * 100 + minor). */
int awq_version(void);

/*
 * awq_pack -- pack 4-bit values into 32-bit words ([P1] order map for
 * AWQ_LAYOUT_N8; K-packed two's complement for W4A8_LAYOUT_K8).  Used for
 * qweight and qzeros alike.
 *   vals:        device, uint8 [rows, cols] (N8) or int8 [rows, cols] (K8).
 *   packed:      device, int32 [rows, cols/8] (N8) or [rows/8, cols] (K8).
 *   clamp_count: device int32 or NULL.  Values outside 0..15 (N8) / -8..7 (K8)
 *                are clamped into range (the lesson of the missing clamp in
 *                [P5]) and their number is atomically added to *clamp_count,
 *                which the caller zeroes beforehand.
 * rows == 0 or cols == 0 is a no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL if a pointer is NULL, rows/cols < 0, cols % 8 (N8) or
 * rows % 8 (K8) is non-zero, or the layout is unknown.  AWQ_LAYOUT_V2 takes
 * any cols.
 */
int awq_pack(const void *vals, int32_t *packed, int64_t rows, int64_t cols, int layout,
             int32_t *clamp_count, void *stream);

/*
 * awq_unpack -- inverse of awq_pack: words -> uint8 (N8, 0..15) or int8
 * (K8, -8..7) values [rows, cols].  Same shape rules and errors as awq_pack.
 */
int awq_unpack(const int32_t *packed, void *vals, int64_t rows, int64_t cols, int layout,
               void *stream);

/*
 * awq_repack_v2 -- weights in the newer AWQ packing ([P1]: identity order
 * map, zero points packed per output channel along the groups with unused
 * nibbles skipped, a zeros width of ceil(groups / 8) words) rewritten into
 * the first-generation format that the GEMM and GEMV calls take, bit for bit
 * the same logical values.  A checkpoint in the newer format is repacked
 * once at load; the scales are the same [K/G, N] tensor in both.
 *   qweight_v2: device int32 [K, N/8], AWQ_LAYOUT_V2 along each row.
 *   qzeros_v2:  device int32 [N, ceil((K/G)/8)], AWQ_LAYOUT_V2 along each
 *               output channel's groups; NULL = symmetric (then qzeros is
 *               not written).
 *   qweight:    device int32 [K, N/8], AWQ_LAYOUT_N8 (written).
 *   qzeros:     device int32 [K/G, N/8], AWQ_LAYOUT_N8 (written).
 * Errors: AWQ_EINVAL (shapes, G, NULL qzeros with non-NULL qzeros_v2),
 * AWQ_EALIGN, AWQ_EHIP.
 */
int awq_repack_v2(const int32_t *qweight_v2, const int32_t *qzeros_v2, int32_t *qweight, int32_t *qzeros,
                  int64_t N, int64_t K, int group_size, void *stream);

/*
 * awq_workspace_bytes -- bytes of device workspace the given call needs
 * (0 if none) on the current device.  split_k as passed to the call
 * (0 = automatic).  For W4A8, group_size is the one passed to w4a8_gemm.
 * Workspace rules ([P2]: one workspace per device, reused by every layer):
 *  - it is caller-owned, 16-byte aligned, and may be shared by any number of
 *    calls that are ordered on one stream;
 *  - a split-K fp16 decode GEMV, or a split-K W4A8 call on the skinny
 *    kernel (M <= 32), uses one 64-bit counting accumulator per output
 *    element (M x N); the last contribution to an element writes the output
 *    and clears it (the size returned for the W4A16 calls covers both
 *    activation dtypes);
 *  - a split-K bf16 decode GEMV and the GEMM kernels (M > 8 for W4A16,
 *    M > 32 for W4A8) use one 32-bit
 *    arrival counter per output tile (padded to 256 bytes) followed by S
 *    partial [M, N] results of 4 bytes each (fp32 for W4A16, int32 for
 *    W4A8); the last workgroup of a tile to arrive adds the S partials in
 *    split order, writes the output, clears them and re-arms the counter --
 *    or, where the partials are large (always for the W4A8 GEMMs), a second
 *    kernel enqueued right after the first on the same stream adds them in
 *    split order, writes the output and clears them (counters untouched);
 *  - either way the workspace is zero again after every call;
 *  - it must be zero-filled once when allocated; no per-call clearing is
 *    needed;
 *  - calls that overlap in time (different streams) need separate workspaces;
 *  - a captured graph holds its calls' workspace: it has to live as long as the
 *    graph, and a zero-fill that is only recorded has not happened before the
 *    graph's first replay.
 * Returns 0 for invalid arguments.
 */
size_t awq_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int group_size, int split_k);

/*
 * awq_stream_capture_id -- for callers that keep workspaces: *id is the number
 * of the graph capture that `stream` is recording, different for every
 * capture, or 0 if it records none.  Errors: AWQ_EINVAL (id NULL), AWQ_EHIP.
 */
int awq_stream_capture_id(void *stream, uint64_t *id);

/*
 * awq_plan_info -- how a call would be launched, without launching it: the
 * kernel, grid and workspace the library's planner picks for the given shape
 * on a device with `cu_count` compute units (0 = the current device, queried
 * once per device and cached; a whole MI355X, 256, when no device is
 * visible).  The planners size their grids from this count, so a partitioned
 * or smaller part gets grids of its own size.  Needs no GPU when cu_count > 0.
 *   op: AWQ_OP_*; other arguments as for the call (group_size -1 = W4A8
 *   per-channel).
 *   out: host pointer, written on success.
 * Errors: the validation status the call itself would return for the shape
 * (AWQ_EINVAL, AWQ_EUNSUPPORTED), or AWQ_EINVAL for a NULL out or a negative
 * cu_count.
 */
typedef struct {
    int kernel;    /* W4A16: 0 decode GEMV, 1 register-tiled GEMM, 3 LDS-pipelined GEMM;
                      W4A8: 0 skinny split-K, 1 register-tiled, 2 LDS-pipelined */
    int tiles_n;   /* workgroup tiles along N */
    int tiles_m;   /* workgroup tiles along M */
    int splits;    /* workgroups along K (1 = no split) */
    int row_tiles; /* 16-row matrix-core tiles per wave or workgroup column */
    int ksplit;    /* wave groups splitting K inside one workgroup (1 or 2) */
    int cu_count;  /* the compute-unit count the plan was made for */
    int64_t workspace_bytes;
    int tile_cols; /* LDS-pipelined GEMMs: output columns per workgroup tile (128 or 256);
                      0 for the other kernels */
} awq_plan_t;
int awq_plan_info(int op, int64_t M, int64_t N, int64_t K, int group_size, int split_k, int cu_count,
                  awq_plan_t *out);

/*
 * awq_gemm_w4a16 -- Y = X . dequant(qweight, qzeros, scales) for any M >= 1
 * (the prefill path of the [P1] dispatch; also correct for small M).
 *   x:       device, [M, K] fp16 or bf16 (dtype).
 *   qweight: device, int32 [K, N/8], AWQ_LAYOUT_N8.
 *   scales:  device, [K/G, N] in the activation dtype.
 *   qzeros:  device, int32 [K/G, N/8], AWQ_LAYOUT_N8; NULL = symmetric
 *            weights with z = 8 ([P2]).
 *   y:       device, [M, N] in the activation dtype (written, not accumulated).
 *   group_size G in {32, 64, 128}; K % G == 0; N % 8 == 0; M, N, K >= 1.
 *   split_k: number of K slices reduced through the workspace (0 = chosen by
 *            the library, 1 = none, at most min(K/32, 255)).  For M <= 8
 *            the library's decode kernel fixes the K split itself and
 *            ignores split_k.
 * Numerics: M <= 32, and bf16 up to M = 64 -- the exact (q - z) products
 * are summed in fp32 on the matrix cores and scaled by s in fp32 once per
 * chunk (32 to 128 consecutive k inside one group); fp16 at 32 < M <= 64
 * and M > 64 -- each weight is dequantised exactly to (q - z) and multiplied
 * by s with one rounding to the activation dtype, products accumulating in
 * fp32.  The
 * output is rounded to nearest even.
 * Errors: AWQ_EINVAL (shapes, pointers, dtype, G), AWQ_EALIGN, AWQ_EWORKSPACE,
 * AWQ_EHIP.
 */
int awq_gemm_w4a16(const void *x, const int32_t *qweight, const void *scales,
                   const int32_t *qzeros, void *y, int64_t M, int64_t N, int64_t K,
                   int group_size, int dtype, int split_k, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * awq_gemv_w4a16 -- the decode path of the [P1] dispatch: same tensors,
 * formats, numerics and errors as awq_gemm_w4a16, for 1 <= M <= 8
 * (AWQ_EUNSUPPORTED otherwise).  The weight stream is split over K across
 * the whole GPU and reduced through the workspace.
 */
int awq_gemv_w4a16(const void *x, const int32_t *qweight, const void *scales,
                   const int32_t *qzeros, void *y, int64_t M, int64_t N, int64_t K,
                   int group_size, int dtype, int split_k, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * awq_dequant_w4a16 -- the dense weight matrix W[k,n] = (q - z) * s rounded
 * once (to nearest even) to the activation dtype, [K, N] row-major: the
 * operand a dense vendor GEMM needs for the "dequantise, then call the dense
 * BLAS GEMM for long sequences" route of the [P1] TODO list.  Not used by the
 * 4-bit GEMM calls; provided for comparison and export.
 *   qweight, scales, qzeros, group_size, dtype: as awq_gemm_w4a16 (qzeros
 *   NULL = symmetric, z = 8).
 *   w: device, [K, N] fp16 or bf16, written.
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EHIP.
 */
int awq_dequant_w4a16(const int32_t *qweight, const void *scales, const int32_t *qzeros, void *w,
                      int64_t N, int64_t K, int group_size, int dtype, void *stream);

/*
 * awq_gemv_w4a16_static -- awq_gemv_w4a16 for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): the same kernels, results and argument rules,
 * without a workspace argument.  The split-K reduction runs in a static
 * scratch array of 16 MiB (AWQ_STATIC_SCRATCH_BYTES) that each device holds
 * from the library's load until the process ends; the call itself allocates
 * and frees nothing.
 *   Its first call on a device looks up that device's copy of the array and
 *   enqueues a clear of it on `stream` ahead of the GEMV (again on each later
 *   call until one runs outside graph capture, since a clear recorded into a
 *   graph runs only with the graph).
 *   Every call on one device shares that device's array, which the kernels
 *   leave zero after each call: calls that overlap in time on one device
 *   (different streams, or a graph replayed beside an eager call) race and
 *   must be ordered by the caller.
 * Errors: as awq_gemv_w4a16 (AWQ_EUNSUPPORTED for M > 8), plus
 * AWQ_EWORKSPACE when the call's split-K reduction needs more than
 * AWQ_STATIC_SCRATCH_BYTES (awq_plan_info reports the need), and AWQ_EHIP if
 * the device or its copy of the array cannot be found.
 */
#define AWQ_STATIC_SCRATCH_BYTES (16u << 20)
int awq_gemv_w4a16_static(const void *x, const int32_t *qweight, const void *scales,
                          const int32_t *qzeros, void *y, int64_t M, int64_t N, int64_t K,
                          int group_size, int dtype, void *stream);

/*
 * w4a8_quant_act -- dynamic per-token int8 quantisation of activations
 * ([P5], the dynamic_quant helper):
 *   s1[m]   = float( act( max_k |x[m,k]| / 127 ) )
 *   a8[m,k] = clamp( round_half_even( float(x[m,k]) / s1[m] ), -128, 127 )
 * with a correctly rounded fp32 divide; act() rounds to the activation type
 * (nearest even); a row whose s1 is 0 gives a8 = 0.  [P5] defines the fp16
 * form and lists bf16 as not yet supported; for bf16 this library takes the
 * same recipe with the quotient rounded to bf16.
 *   x: device fp16 or bf16 [M, K] (dtype AWQ_DTYPE_F16 / AWQ_DTYPE_BF16);
 *   a8: device int8 [M, K]; s1: device fp32 [M].
 * Errors: AWQ_EINVAL (M, K < 1, pointers, dtype), AWQ_EALIGN, AWQ_EHIP.
 */
int w4a8_quant_act(const void *x, int8_t *a8, float *s1, int64_t M, int64_t K, int dtype, void *stream);

/*
 * w4a8_gemm -- QQQ-style W4A8 GEMM ([P5]):
 *   acc[m,n] = sum_k a8[m,k] * w8[k,n]   (exact, int32)
 *   y[m,n]   = act( acc[m,n] * s1[m] * s2[n] )   (fp32 arithmetic, RNE)
 * with w8 = q for per-channel weights (s3 == NULL, group_size == -1) and
 * w8 = q * s3[k/G, n] for per-group weights, where s3 holds small integers
 * 1..16 so that w8 stays an int8.  s2, s3 and y are in the activation type
 * `dtype` (AWQ_DTYPE_F16 or AWQ_DTYPE_BF16; acc does not depend on it).
 *   a8:       device int8 [M, K] (from w4a8_quant_act).
 *   b_packed: device int32 [K/8, N], W4A8_LAYOUT_K8 (q in -8..7).
 *   s1:       device fp32 [M];  s2: device [N];  s3: device [K/G, N] or NULL.
 *   y:        device [M, N].
 *   acc_out:  device int32 [M, N] or NULL: if given, the exact accumulators
 *             are written too (for checking).
 *   K % 64 == 0 and K <= 131008 (so that the int32 accumulator, which
 *   holds up to 2^14 * K, cannot wrap); N % 8 == 0; group_size -1
 *   (per-channel) or one of 32, 64, 128.
 * Errors: AWQ_EINVAL (also an unknown dtype), AWQ_EALIGN, AWQ_EWORKSPACE,
 * AWQ_EUNSUPPORTED (K % 64 != 0 or K > 131008), AWQ_EHIP.
 */
int w4a8_gemm(const int8_t *a8, const int32_t *b_packed, const float *s1, const void *s2,
              const void *s3, void *y, int32_t *acc_out, int64_t M, int64_t N,
              int64_t K, int group_size, int dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * w4a8_linear -- the whole W4A8 layer in one call: w4a8_quant_act of x
 * followed by w4a8_gemm, with identical results (y, s1 and acc_out bit for
 * bit).  The pages note that quantising activations in a separate kernel
 * costs performance ([P5]); for a single token (M == 1, K <= 32768, fp16 or
 * bf16) the quantisation runs inside the GEMM kernel: every workgroup reads
 * the activation row, derives s1 and quantises its own K range into LDS, so
 * the int8 activations never travel through device memory and there is one
 * launch.  Otherwise the two steps run back to back.
 *   x:   device fp16 or bf16 [M, K] (dtype).
 *   a8:  device int8 [M, K], scratch: holds the quantised activations when
 *        the two-step path runs, left untouched by the fused path.
 *   s1:  device fp32 [M], written (the per-token scales).
 *   other arguments, layouts, workspace and errors: as w4a8_gemm.
 */
int w4a8_linear(const void *x, int8_t *a8, float *s1, const int32_t *b_packed,
                const void *s2, const void *s3, void *y, int32_t *acc_out,
                int64_t M, int64_t N, int64_t K, int group_size, int dtype, void *workspace,
                size_t workspace_bytes, void *stream);

/*
 * INT4-FP8 W4A8.  [P5] names "INT4-FP8 QQQ (W4A8)" as its authors' next step
 * and gives nothing more; this library takes the int8 recipe above with OCP
 * FP8 E4M3 activation codes (sign, 4 exponent bits biased by 7, 3 mantissa
 * bits; largest finite value 448; 0x7f and 0xff are NaN and never produced)
 * and 448 in place of the int8 codes and 127, per-channel scales only.
 *
 * w4a8_fp8_quant_act -- per-token E4M3 quantisation:
 *   s1[m]   = float( act( max_k |x[m,k]| / 448 ) )   (correctly rounded fp32
 *             divide, then rounded to the activation type)
 *   a[m,k]  = e4m3( clamp( float(x[m,k]) / s1[m], -448, 448 ) )  (fp32
 *             divide, round to nearest even); a row whose s1 is 0 gives codes 0
 *   asum[m] = float( sum_k value(a[m,k]) )  (the exact sum, rounded once; the
 *             GEMM needs it)
 *   x: device fp16/bf16 [M, K] (dtype); a: device uint8 [M, K];
 *   s1, asum: device fp32 [M].
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EHIP.
 */
int w4a8_fp8_quant_act(const void *x, uint8_t *a, float *s1, float *asum, int64_t M, int64_t K, int dtype,
                       void *stream);

/*
 * w4a8_fp8_gemm -- y[m,n] = act( acc[m,n] * s1[m] * s2[n] ) with
 * acc[m,n] = sum_k value(a[m,k]) * q[k,n], accumulated in fp32 on the fp8
 * matrix cores (not exact: compare within a tolerance).
 *   a, s1, asum: from w4a8_fp8_quant_act; b_packed: int32 [K/8, N],
 *   W4A8_LAYOUT_K8 (q in -8..7); s2: device [N] and y: device [M, N] in the
 *   activation type `dtype`; acc_out: device fp32 [M, N] or NULL (the fp32
 *   sums, for checking).
 *   K % 128 == 0 and K <= 131008; N % 8 == 0.  Workspace as for w4a8_gemm
 *   (op AWQ_OP_W4A8_FP8_GEMM in awq_workspace_bytes).
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EWORKSPACE, AWQ_EUNSUPPORTED (K), AWQ_EHIP.
 */
int w4a8_fp8_gemm(const uint8_t *a, const int32_t *b_packed, const float *s1, const float *asum,
                  const void *s2, void *y, float *acc_out, int64_t M, int64_t N, int64_t K, int dtype,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * w4a8_fp8_linear -- the whole INT4-FP8 layer in one call:
 * w4a8_fp8_quant_act of x followed by w4a8_fp8_gemm.  As for w4a8_linear
 * ([P5]: quantising in a separate kernel costs performance), a single token
 * (M == 1) runs as one kernel: every workgroup reads the activation row,
 * derives s1 and quantises its own K range into LDS, and the GEMM's epilogue
 * takes each range's own sum of the codes' values, so no workgroup needs the
 * whole row's.  s1 and every code are those of w4a8_fp8_quant_act; the output
 * forms acc = 512 t - 8 asum once from the exact split-K sum, where the
 * two-launch path first rounds t to fp32 (at most one fp32 rounding of acc
 * apart; y then at most one rounding of the activation type).  Otherwise the
 * two steps run back to back.
 *   x: device fp16/bf16 [M, K] (dtype).
 *   a, asum: device uint8 [M, K] and fp32 [M], scratch: the codes and row
 *            sums when the two-step path runs, untouched by the fused path.
 *   s1: device fp32 [M], written.
 *   other arguments, layouts, workspace (op AWQ_OP_W4A8_FP8_GEMM) and errors:
 *   as w4a8_fp8_gemm.
 */
int w4a8_fp8_linear(const void *x, uint8_t *a, float *s1, float *asum, const int32_t *b_packed,
                    const void *s2, void *y, float *acc_out, int64_t M, int64_t N, int64_t K, int dtype,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * The operators around the linear layers: RMS norm with an 8-bit output, and
 * the attention block's cache in 4 bits.  fl32(v) is v rounded to binary32
 * and act(v) v rounded to the activation type, both to nearest even; every
 * rounding written below is part of the definition, so codes, scales and
 * packed words are the same bits on every run, launch and machine.
 *
 * w4a8_rmsnorm_quant -- residual addition, root-mean-square norm and per-token
 * int8 quantisation in one pass, the input of w4a8_gemm:
 *   h[m,k]  = act( fl32( x + residual ) )            (no residual: h = x)
 *   v[m]    = fl32( sum_k h^2 / K + eps )            (sum, in an order that K fixes, and
 *                                                         quotient in binary64)
 *   q[m]    = fl32( 1 / fl32( sqrt(v) ) )
 *   y[m,k]  = act( fl32( fl32( h q ) weight[k] ) )
 *   s1, a8  = w4a8_quant_act of y
 *   x, residual: device fp16/bf16 [M, K] (dtype); residual NULL = none.
 *   weight:      device [K], same type.
 *   residual_out: device [M, K], h (written); NULL iff residual is.  May be
 *                residual itself, or x.
 *   y:           device [M, K], the norm in the activation type, or NULL.
 *                May be x (where residual_out is not).
 *   a8, s1:      device int8 [M, K] and fp32 [M]; both NULL for the norm alone
 *                (then y must be given), the input of a W4A16 layer.
 *   No other tensors may overlap.  A row whose h holds a NaN or an infinity,
 *   or whose norm overflows the activation type, has an s1 that is not
 *   finite; its codes mean nothing.  eps >= 0 and finite.
 * Errors: AWQ_EINVAL (M, K < 1, K > 2^20, pointers, y at residual_out, dtype,
 * eps), AWQ_EALIGN,
 * AWQ_EHIP.
 */
int w4a8_rmsnorm_quant(const void *x, const void *residual, const void *weight, void *residual_out, void *y,
                       int8_t *a8, float *s1, int64_t M, int64_t K, float eps, int dtype, void *stream);

/*
 * w4a8_fp8_rmsnorm_quant -- the same with E4M3 codes, the input of
 * w4a8_fp8_gemm: s1, a, asum = w4a8_fp8_quant_act of y.  a, s1 and asum must
 * be given.
 */
int w4a8_fp8_rmsnorm_quant(const void *x, const void *residual, const void *weight, void *residual_out, void *y,
                           uint8_t *a, float *s1, float *asum, int64_t M, int64_t K, float eps, int dtype,
                           void *stream);

/*
 * The paged key/value cache in 4 bits: int32 [num_pages, Hkv, W] with
 * W = awq_kv4_head_words(head_dim, page_size) = page_size (head_dim / 4 + 2).
 * The words of one page and key/value head:
 *   K words  [page_size][head_dim/8]       AWQ_LAYOUT_N8 along the dimensions
 *   V words  [page_size/4][head_dim/8][4]  the same words, those of four
 *                                          consecutive tokens side by side
 *   K meta   [page_size], V meta [page_size]
 *            bits 15..0 the scale s in the activation type, 31..16 the zero
 *            point z (0..15), one pair per token and head
 * and value = (code - z) s, as for the weights.  head_dim 64 or 128;
 * page_size a power of two, 16..1024.  A page belongs to the sequences whose
 * block tables name it; the library keeps no other state, and no word that is
 * not read below need be initialised.
 *
 * awq_kv4_head_words -- W, or 0 for sizes the library does not take.
 */
int64_t awq_kv4_head_words(int64_t head_dim, int64_t page_size);

/*
 * awq_kv4_append -- rotary positions on the queries and keys of T tokens, and
 * their keys and values quantised into the cache.
 * Rotation of the pair (x1, x2) with the cosine c and sine s of its angle:
 *   act( fl32( fl32(x1 c) - fl32(x2 s) ) ),  act( fl32( fl32(x2 c) + fl32(x1 s) ) )
 * over the first `rot` dimensions of each head, pairs (i, i + rot/2), or
 * (2i, 2i + 1) if interleaved; angle i of position p is row p of the table.
 * Quantisation of one token and head x (keys after the rotation):
 *   lo = min(0, min x), hi = max(0, max x), s = act( fl32( fl32(hi - lo) / 15 ) )
 *   z = min( rint( fl32(-lo / s) ), 15 ),  code = clamp( rint( fl32(x / s) ) + z, 0, 15 )
 * with rint to nearest even; s = 0 gives z = code = 0.  A head that holds a
 * NaN or an infinity is stored as s = NaN, z = code = 0.
 *   q, k, v:   device [T, Hq or Hkv, head_dim] (dtype), the heads of a token
 *              dense, q_stride / k_stride / v_stride elements from one token
 *              to the next (multiples of 8), so that a fused QKV product's
 *              output serves as all three.  q NULL iff Hq == 0.
 *   rope:      device fp32 [max_pos, rot]: rot/2 cosines, then rot/2 sines.
 *              rot a multiple of 16, 0..head_dim; 0 = no rotation (rope and
 *              positions may be NULL).
 *   positions: device int32 [T].  A token whose position is outside
 *              0..max_pos-1 is not stored and its rotated query dimensions
 *              are NaN.
 *   slots:     device int64 [T], page * page_size + place in the page; a slot
 *              outside the cache (-1, say) stores nothing.  Two tokens with
 *              one slot leave either's words.
 *   q_out:     device [T, Hq, head_dim], dense; may be q where q is dense.
 * T == 0 is a no-op that returns AWQ_OK.  Index arrays need the alignment of
 * their type only.
 * Errors: AWQ_EINVAL, AWQ_EUNSUPPORTED (head_dim, page_size), AWQ_EALIGN
 * (strides too), AWQ_EHIP.
 */
int awq_kv4_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                   const float *rope, const int32_t *positions, const int64_t *slots, void *q_out, int32_t *cache,
                   int64_t T, int64_t Hq, int64_t Hkv, int64_t head_dim, int64_t page_size, int64_t num_pages,
                   int64_t rot, int64_t max_pos, int interleaved, int dtype, void *stream);

/*
 * awq_kv4_attention -- causal attention of B sequences' new tokens over the
 * cache (which holds the new tokens' keys and values too: append first).
 * Sequence b has n = cu_q[b+1] - cu_q[b] new tokens, rows cu_q[b].. of q, and
 * L = lens[b] tokens in all; its new token i stands at p = L - n + i and sees
 * the tokens j <= p, with a window w > 0 only j > p - w:
 *   out = sum_j softmax_j( scale q . k_j ) v_j
 * over the keys and values that the cache's words stand for.  Query head e
 * reads key/value head e / (Hq / Hkv).  A row that sees nothing (p < 0,
 * L = 0) is 0.
 *   q, out:  device [total_q, Hq, head_dim], dense; out may be q.
 *   tables:  device int32 [B, table_stride]: entry t / page_size names the
 *            page of token t.  An entry that names no page of the cache (-1)
 *            hides its tokens.
 *   lens:    device int32 [B]; taken as 0 below 0 and as table_stride *
 *            page_size above it.
 *   cu_q:    device int32 [B + 1], rising from 0 to total_q; NULL = one new
 *            token per sequence (total_q == B, max_q == 1).
 *   max_q:   the most new tokens of a sequence (the rows of a sequence past
 *            its first max_q are not written).
 *   max_kv:  the longest sequence, or an upper bound: it sizes the launch and
 *            the workspace, results depend on it by their rounding only.  Few
 *            sequences under a loose bound are shared among too few workgroups
 *            (four of 8192 to 16384 tokens under 131072: 58 us, under 16384 20),
 *            and so are few sequences with a window far below max_kv.
 * One kernel takes the whole call, by max_q and the other bounds: prompts and
 * single tokens go faster in calls of their own (a prompt of 1024 tokens at the
 * end of 8192, and 63 single ones over 4096 to 8192, 32 heads over 8: 960 us in
 * one call, 163 + 90 in two).
 * Numerics: the codes enter the matrix cores exactly; scores, running maxima,
 * sums and outputs are fp32; the softmax numerators times the values' scales
 * are rounded once to 11 bits for the second product (those below 2^-19 of a
 * row's largest to 2^-30 of it); out is rounded to nearest even.  (Down to
 * value scales of 2^-79 in magnitude; smaller ones keep fewer bits.)  A NaN or
 * infinity in q, or a NaN scale in a token that a row sees, makes that row NaN;
 * nothing that a row does not see changes it by more than its rounding.
 * Scores of 2^24 and more in magnitude have binary32's steps of two and more
 * (times log2(e)), the softmax with them; a row whose largest is past 2.3 10^7
 * (2^25 / log2(e)), or below minus that, is NaN.
 * Workspace: as for the GEMMs (shared, zero before and after each call).
 * B == 0 or total_q == 0 is a no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL (also scale <= 0), AWQ_EUNSUPPORTED (head_dim,
 * page_size, more tiles of query rows than a launch holds), AWQ_EALIGN, AWQ_EWORKSPACE,
 * AWQ_EHIP.
 */
int awq_kv4_attention(const void *q, const int32_t *cache, const int32_t *tables, const int32_t *lens,
                      const int32_t *cu_q, void *out, int64_t B, int64_t total_q, int64_t max_q, int64_t max_kv,
                      int64_t Hq, int64_t Hkv, int64_t head_dim, int64_t page_size, int64_t num_pages,
                      int64_t table_stride, float scale, int64_t window, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Bytes of workspace that awq_kv4_attention needs on the current device (0 if
 * none, or for invalid arguments). */
size_t awq_kv4_attention_workspace_bytes(int64_t B, int64_t max_q, int64_t Hq, int64_t Hkv, int64_t head_dim,
                                         int64_t max_kv);

/*
 * Mixture of experts: routing, products grouped by expert, and their weighted
 * sum.  A token t takes part in k products; slot t k + j is its j-th.  The products'
 * rows lie in the order of their experts: expert e has rows offsets[e] ..
 * offsets[e+1] - 1, which the device alone knows, so no call waits for them.
 *
 * awq_moe_route -- each token's k experts, their weights, and the plan.
 * Of the logits l[t, .] the k largest, larger ones first, equal ones by expert (-0 is
 * 0; +infinity counts as the largest finite binary32 number; -infinity and NaN
 * are never chosen).  With m the largest,
 *   weight = exp(l - m) / sum_e exp(l_e - m)
 * over all experts that could be chosen, or over the chosen ones (renormalize);
 * fp32.  A token with fewer than k such experts has expert -1 and weight 0 in
 * the places left, and no rows for them.
 *   logits:  device [T, E] in dtype (AWQ_DTYPE_F32 too).
 *   weights: device fp32 [T, k];  experts: device int32 [T, k].
 *   offsets: device int32 [E + 1]: the rows of each expert.
 *   rows:    device int32 [T k]: the slot of each row -- by expert, then by slot;
 *            -1 behind the last.
 *   places:  device int32 [T k]: the row of each slot, or -1.
 *   1 <= k <= min(E, 32), E <= 1024, T <= 2^20, T k <= 2^24.  T == 0 writes offsets.
 *   Workspace: awq_moe_route_workspace_bytes of any contents, not left zero:
 *   not the one that the products share.
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EWORKSPACE, AWQ_EHIP.
 */
int awq_moe_route(const void *logits, float *weights, int32_t *experts, int32_t *offsets, int32_t *rows,
                  int32_t *places, int64_t T, int64_t E, int64_t k, int renormalize, int dtype, void *workspace,
                  size_t workspace_bytes, void *stream);
size_t awq_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k);

/*
 * awq_moe_gemm_w4a16 -- y[r] = x[row of r] . dequant(weights of r's expert), the
 * layer of awq_gemm_w4a16 with a matrix per expert.
 *   x:       device [x_rows, K] (dtype).
 *   qweight: device int32 [E, K, N/8], scales [E, K/G, N], qzeros int32
 *            [E, K/G, N/8] or NULL, each expert's as for awq_gemm_w4a16.
 *   offsets: device int32 [E + 1], not falling, in 0 .. R: a plan's, or for some
 *            consecutive experts' matrices its part from the first of them on.
 *            (Whatever they hold, nothing outside the tensors is read or written.)
 *   rows:    device int32 [R]: row r reads x[rows[r] / top_k] (the plan's rows:
 *            the first product of a layer, x one row a token); or NULL: it reads
 *            x[r] (x_rows == R; the second one, on rows in the plan's order).  An entry
 *            that names no row of x reads row 0.
 *   y:       device [R, N]; rows before offsets[0] and from offsets[E] on are not
 *            written.
 *   G, K, N as for awq_gemm_w4a16; E <= 1024, R <= 2^24, 1 <= top_k <= 32.  With
 *   rows, x is under 2^31 bytes, and an expert's words are in any case (else
 *   AWQ_EUNSUPPORTED).  One kernel takes the whole call, chosen by R over the
 *   experts that R rows reach on average, as if all had alike.
 * Numerics: up to 24 such rows an expert, and where K % 64 or N % 32 is not 0,
 *   y = act( sum over runs of min(G, 64) k of s ( sum x q' - z' sum x ) )
 * with q' = q and z' = z (fp16), or both 128 more (bf16): exact operands of the fp32
 * matrix cores, weights that are not rounded, runs added by fp32 FMAs.  Where these
 * are not finite, the sums are made again from the exact q - z, so that an
 * infinity in x gives what it gives in the definition (bf16: |x| under 2^118).
 * Else as awq_gemm_w4a16 for M > 64: weights rounded once to the activation type.
 * Workspace: as for the GEMMs (shared, zero before and after each call).  R == 0
 * is a no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL, AWQ_EUNSUPPORTED, AWQ_EALIGN, AWQ_EWORKSPACE, AWQ_EHIP.
 */
int awq_moe_gemm_w4a16(const void *x, const int32_t *qweight, const void *scales, const int32_t *qzeros,
                       const int32_t *offsets, const int32_t *rows, void *y, int64_t R, int64_t x_rows, int64_t top_k,
                       int64_t E, int64_t N, int64_t K, int group_size, int dtype, void *workspace,
                       size_t workspace_bytes, void *stream);
size_t awq_moe_gemm_w4a16_workspace_bytes(int64_t R, int64_t E, int64_t N, int64_t K, int group_size);

/*
 * awq_moe_combine -- out[t] = act( sum_j weights[t,j] y[places[t k + j]] ), summed
 * by fp32 FMAs in the order of j; a place outside 0 .. R - 1 (-1: no expert)
 * adds nothing.
 *   y: device [R, N];  weights: device fp32 [T, k];  places: device int32 [T k];
 *   out: device [T, N], not overlapping y.  N % 8 == 0, k <= 32.
 * T == 0 is a no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EHIP.
 */
int awq_moe_combine(const void *y, const float *weights, const int32_t *places, void *out, int64_t T, int64_t R,
                    int64_t N, int64_t k, int dtype, void *stream);

/*
 * E4M3 (as for INT4-FP8 above) with one scale for each block of 128 along K.
 *
 * awq_fp8_block_quant_act -- activations, one scale for each run of 128 values
 * of a row (the last run of a row may be shorter):
 *   s[m,b] = fl32( max |x| / 448 ),  a = e4m3( clamp( fl32(x / s), -448, 448 ) )
 * A run whose s is 0 has codes 0; one that holds a NaN or an infinity has an s
 * that is not finite and codes 0, which makes its row of a product NaN.
 *   x: device fp16/bf16 [M, K] (dtype); a: device uint8 [M, K]; s: device fp32
 *   [M, ceil(K/128)].  K % 16 == 0.  M == 0 is a no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EHIP.
 */
int awq_fp8_block_quant_act(const void *x, uint8_t *a, float *s, int64_t M, int64_t K, int dtype, void *stream);

/*
 * awq_fp8_block_gemm -- y[m,n] = act( sum_b sa[m,b] sw[n/128,b]
 *                                     sum_{k in b} value(a[m,k]) value(w[n,k]) )
 *   a, sa: from awq_fp8_block_quant_act.
 *   w:     device uint8 [N, K]: E4M3 codes, a row per output (finite ones).
 *   sw:    device fp32 [ceil(N/128), ceil(K/128)].
 *   y:     device [M, N] fp16/bf16 (dtype).
 *   K % 16 == 0, N % 8 == 0, N K under 2^31 (AWQ_EUNSUPPORTED), M <= 2^24.
 * Numerics: a block's sum of 128 products comes from the fp8 matrix cores in
 * fp32; the blocks are added by fp32 FMAs, times fl32(sa sw).  Not exact: the
 * matrix cores line up the products of four consecutive k with the one of the largest
 * exponent, and drop what lies below 2^-13 of it.  (On random data that is 6 10^-5
 * of the result's norm, a third of fp16's own rounding.)
 * Workspace: as for the GEMMs (E = 0 in awq_fp8_block_gemm_workspace_bytes).  M == 0 is a
 * no-op that returns AWQ_OK.
 * Errors: AWQ_EINVAL, AWQ_EUNSUPPORTED, AWQ_EALIGN, AWQ_EWORKSPACE, AWQ_EHIP.
 *
 * awq_moe_fp8_block_gemm -- the same with a matrix per expert: w [E, N, K], sw
 * [E, ceil(N/128), ceil(K/128)]; offsets, rows, R, x_rows, top_k and y as for
 * awq_moe_gemm_w4a16, the gathered rows' scales with them.  With rows, a is under 2^31
 * bytes (AWQ_EUNSUPPORTED).
 */
int awq_fp8_block_gemm(const uint8_t *a, const uint8_t *w, const float *sa, const float *sw, void *y, int64_t M,
                       int64_t N, int64_t K, int dtype, void *workspace, size_t workspace_bytes, void *stream);
int awq_moe_fp8_block_gemm(const uint8_t *a, const uint8_t *w, const float *sa, const float *sw,
                           const int32_t *offsets, const int32_t *rows, void *y, int64_t R, int64_t x_rows,
                           int64_t top_k, int64_t E, int64_t N, int64_t K, int dtype, void *workspace,
                           size_t workspace_bytes, void *stream);
size_t awq_fp8_block_gemm_workspace_bytes(int64_t M, int64_t E, int64_t N, int64_t K);

/*
 * awq_grouped_plan_info -- as awq_plan_info, for the products above.
 *   op: AWQ_OP_MOE_GEMM_W4A16 (awq_moe_gemm_w4a16), or AWQ_OP_FP8_BLOCK_GEMM
 *   (awq_moe_fp8_block_gemm, or awq_fp8_block_gemm: E = 0; group_size is not
 *   looked at).  R >= 1 rows.
 *   out: kernel 5 is a streaming kernel, 3 one through LDS; row_tiles and
 *   tile_cols are those of a workgroup's tile, tiles_m the row tiles that any
 *   offsets can need.
 * Errors: as awq_plan_info.
 */
int awq_grouped_plan_info(int op, int64_t R, int64_t E, int64_t N, int64_t K, int group_size, int cu_count,
                          awq_plan_t *out);

/*
 * awq_stream_read -- measurement helper, not a step of the method: reads
 * `bytes` bytes at `src` once (16-byte loads spread over up to 2048
 * workgroups) and writes an XOR checksum per wave to `sink`, so that the
 * achievable device-memory read rate at the size of a layer's weights can be
 * timed beside the GEMV that streams them.
 *   src:   device, 16-byte aligned, bytes > 0 and bytes % 16 == 0.
 *   sink:  device uint32 [AWQ_STREAM_SINK_WORDS], overwritten (contents are
 *          meaningless beyond keeping the loads alive).
 * Errors: AWQ_EINVAL, AWQ_EALIGN, AWQ_EHIP.
 */
#define AWQ_STREAM_SINK_WORDS 8192
int awq_stream_read(const void *src, int64_t bytes, uint32_t *sink, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ4_H */
