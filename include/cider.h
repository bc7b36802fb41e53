/*
 * cider.h -- C ABI of the fused quantized linear layer for AMD Instinct MI355X
 * (gfx950): online per-token INT8 activation quantization, INT8 x INT8 -> INT32
 * matrix product on the matrix cores, and a fused dequantization to fp16.
 *
 * The operation (Cider README, ossradar.top repo page):
 *   - "Modes" table: W8A8 = INT8 symmetric weights x INT8 per-token
 *     activations; W4A8 = INT4 weights packed in uint8 x INT8 per-token
 *     activations.
 *   - "W8A8 Quantization Granularity" table: weights per output channel, or
 *     per group of 64 / 128 input elements.  The pages give W4A8 per column
 *     only; this library also offers W4A8 per group of 64 / 128, the same
 *     groups with int4 codes (one int4 scale per group).
 *   - "Quantization" table: symmetric INT8 activations per token, INT32
 *     accumulation, output C_fp16 = C_int32 * s_act * s_weight per element;
 *     W4A8 weights symmetric INT4 with zero-point 8.
 *   - "Metal Kernel Pipeline": prefill quantizes FP16 activations to INT8 plus
 *     per-token scales, then runs INT8 x INT8 -> INT32 -> FP16 with the scales
 *     applied in the same kernel; a one-token call goes to a matrix-vector
 *     kernel.
 *   - "Low-Level API" / "Layer-level API": quantize_weight_int8(W) -> (w_int8,
 *     scale), pack_weight_int4(W) -> (packed, scale), perchannel_linear(x, w,
 *     scale), w4a8_linear(x, packed, scale); group_size = 0 means per channel.
 *
 * Definitions used by every call (the pages give the granularity, not the
 * arithmetic; these are the readings this library implements):
 *   scale      s = absmax / 127 (int8) or absmax / 7 (int4), fp32, correctly
 *              rounded division; s = 0 for an all-zero row / group.
 *   code       q = clamp(rint(x / s), -127, 127) (int8) or clamp(.., -8, 7)
 *              (int4), x / s a correctly rounded fp32 division, rint rounding
 *              half to even; q = 0 when s = 0.
 *   int4 pack  nibble u = q + 8; byte j of a row holds k = 2j in bits 0..3
 *              and k = 2j + 1 in bits 4..7.
 *   product    acc[m, n] = sum_k xq[m, k] * q_w[n, k] in int32 (exact; needs
 *              K * 127^2 < 2^31, i.e. K <= 133144).  Per group g of gs
 *              elements: acc_g[m, n] = the same sum over k in [g*gs, (g+1)*gs).
 *   output     per channel: y = fp16(acc * s_tok[m] * s_w[n]);
 *              per group:   y = fp16(s_tok[m] * sum_g s_w[n, g] * acc_g),
 *              evaluated in fp32 and rounded to nearest even.
 *
 * Layouts (all row-major, element strides in elements):
 *   x      fp16 [M, K], row stride ldx >= K        (activations, tokens x in)
 *   xq     int8 [M, K], row stride K               (quantized activations)
 *   s_tok  fp32 [M]                                 (per-token scales)
 *   w      fp16 [N, K]                              (nn.Linear weight, out x in)
 *   wq     int8 [N, K]  (bits 8)  or  uint8 [N, K/2] packed (bits 4)
 *   s_w    fp32 [N] (group_size 0) or [N, K/group_size] (group_size 64/128)
 *   y      fp16 [M, N]
 *
 * Ownership and threading: every pointer is device memory owned by the
 * caller; the library allocates, frees and synchronizes nothing.  Work is
 * enqueued asynchronously on `stream` (a hipStream_t passed as void*; NULL is
 * the default stream).  The library keeps no state between calls except the
 * cached device check and the path override below; calls are thread-safe.
 *
 * Errors: every call checks its arguments on the host before touching the
 * HIP runtime and returns a cider_status.  Nothing is launched when the
 * status is not CIDER_OK, except CIDER_ERR_HIP (a launch failed).  Inputs
 * are assumed finite; NaN or Inf inputs give unspecified codes.
 *
 * Envelope: M >= 0 (M = 0 is a no-op), N >= 0 with N % 64 == 0, K > 0 with
 * K % 64 == 0 and K <= 133144, (M + 256) * K < 2^31 and (N + 256) * K < 2^31
 * for the products, group_size in {0, 64, 128} for W8A8 and W4A8;
 * device pointers 16-byte aligned; ldx % 8 == 0.
 */
#ifndef CIDER_H
#define CIDER_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CIDER_OK = 0,
    CIDER_ERR_INVALID_ARG = 1,       /* null pointer, negative size, ldx < K, bits or group_size not allowed */
    CIDER_ERR_UNSUPPORTED_SHAPE = 2, /* outside the envelope: K % 64, N % 64, K % group_size, K too large */
    CIDER_ERR_MISALIGNED = 3,        /* a pointer not 16-byte aligned, or ldx % 8 != 0 */
    CIDER_ERR_NO_DEVICE = 4,         /* no usable gfx950 device (or CIDER_FORCE_UNAVAILABLE=1) */
    CIDER_ERR_HIP = 5,               /* the HIP runtime reported an error at launch */
    CIDER_ERR_WORKSPACE = 6,         /* workspace missing or smaller than cider_linear_workspace_bytes */
    CIDER_ERR_SCRATCH_LIMIT = 7      /* cider_linear_ex_noalloc: the call needs more than
                                        CIDER_NOALLOC_SCRATCH_BYTES of workspace */
} cider_status;

/* Element type of 16-bit activations, weights and outputs (Cider README
   feature list: automatic dtype handling, float16 / bfloat16).  Values of
   either type are widened exactly to fp32; outputs are rounded once from the
   fp32 result to nearest even. */
typedef enum {
    CIDER_DTYPE_F16 = 0,
    CIDER_DTYPE_BF16 = 1
} cider_dtype;

/* 1 if the current HIP device is a gfx950 GPU that the library can use, else 0.
   Never crashes: returns 0 when the runtime finds no device.  The environment
   variable CIDER_FORCE_UNAVAILABLE=1 makes it return 0 (a test hook for the
   degrade-gracefully behaviour of Cider README "Conditional Compilation"). */
int cider_is_available(void);

/* Static English text for a status code (never NULL). */
const char *cider_status_str(int status);

/* Weight quantization (Cider README "Low-Level API": quantize_weight_int8,
   pack_weight_int4; "Quantization" table).
   w: fp16 [N, K].  bits 8: wq int8 [N, K]; bits 4: wq uint8 [N, K/2] packed.
   group_size 0: s_w fp32 [N]; 64 or 128: s_w fp32 [N, K/gs] (for bits 4 each
   group's scale is its absmax / 7 and its codes are packed like a row's). */
cider_status cider_quantize_weight(const void *w_f16, int64_t N, int64_t K, int bits,
                                   int group_size, void *wq, float *s_w, void *stream);

/* Weight quantization with percentile clipping (Cider README, "LLM
   Quantization: Precision vs. Speed" note: a percentile method besides plain
   min-max, clip_percentile=99.9).  As cider_quantize_weight, except that each
   row's (group's) range -- the absmax in s = range / 127 or / 7 -- is the
   clip_percentile-th percentile of its |w|: linear interpolation between the
   order statistics around the fractional rank (n - 1) * p / 100, numpy's
   default method, evaluated in fp64 and rounded to fp32.  Values beyond the
   range saturate at the end codes (+-127; int4: 7 and -8).
   0 < clip_percentile <= 100 (else CIDER_ERR_INVALID_ARG); 100 gives exactly
   cider_quantize_weight's result. */
cider_status cider_quantize_weight_clipped(const void *w_f16, int64_t N, int64_t K, int bits,
                                           int group_size, double clip_percentile, void *wq,
                                           float *s_w, void *stream);

/* Weight quantization for either 16-bit type, with optional percentile
   clipping: cider_quantize_weight / cider_quantize_weight_clipped for a w of
   type w_dtype (bf16 magnitudes order like fp16 ones, so clipping finds the
   same order statistics).  clip_percentile = 100 is plain absmax. */
cider_status cider_quantize_weight_ex(const void *w, int w_dtype, int64_t N, int64_t K, int bits,
                                      int group_size, double clip_percentile, void *wq, float *s_w,
                                      void *stream);

/* SmoothQuant's weight fold (Cider README: SmoothQuant named among the
   preprocessing methods for quantization-friendly models).  With smoothing
   factors s [K] (fp32, positive, 16-byte aligned) the activations are
   divided by s inside cider_quantize_act_ex / cider_linear_ex and the weights
   absorb it offline: w_out[n, k] = w[n, k] * s[k], the exact product rounded
   once to nearest even in w's own type.  w, w_out [N, K] of type w_dtype,
   16-byte aligned; K % 8 == 0; w_out may equal w. */
cider_status cider_smooth_fold_weight(const void *w, int w_dtype, int64_t N, int64_t K,
                                      const float *smooth, void *w_out, void *stream);

/* Per-token activation quantization of fp16 or bf16 activations, with an
   optional SmoothQuant smoothing vector smooth [K] (fp32, 16-byte aligned,
   NULL for none): x'[m, k] = fp32(x[m, k] / smooth[k]) (correctly rounded)
   before the absmax, and the codes are those of x'.  Otherwise as
   cider_quantize_act. */
cider_status cider_quantize_act_ex(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                   const float *smooth, int8_t *xq, float *s_tok, void *stream);

/* Per-token activation quantization (Cider README "Metal Kernel Pipeline",
   step quantize_per_token; "Quantization" table, Activations row).
   x: fp16 [M, K] with row stride ldx.  xq: int8 [M, K]; s_tok: fp32 [M]. */
cider_status cider_quantize_act(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                                int8_t *xq, float *s_tok, void *stream);

/* W8A8 product with fused dequantization (Cider README "Metal Kernel
   Pipeline", step matmul_fused_dequant; "TensorOps matmul2d"; "W8A8
   Quantization Granularity").  group_size 0: per-channel s_w [N];
   64 / 128: per-group s_w [N, K/gs].  y: fp16 [M, N].
   Under the automatic path setting the matrix-vector kernel takes
   M * K <= 65536 with M <= 3 per channel or M <= 2 per group where the
   few-token matrix-core kernel applies (K a multiple of 128 int8 / 256 int4
   values), else M <= 8 (M <= 4 for int4 weights); everything else runs the
   matrix-core kernels. */
cider_status cider_w8a8_gemm(const int8_t *xq, const float *s_tok, const int8_t *wq,
                             const float *s_w, int64_t M, int64_t N, int64_t K,
                             int group_size, void *y_f16, void *stream);

/* W4A8 product (Cider README "Modes": Unpack -> TensorOps; "Metal Kernel
   Pipeline": INT4 -> INT8 unpacking before the INT8 product).
   wq4: uint8 [N, K/2] packed nibbles.  group_size 0: s_w fp32 [N];
   64 / 128: per-group s_w fp32 [N, K/gs] (the per-group output formula). */
cider_status cider_w4a8_gemm(const int8_t *xq, const float *s_tok, const uint8_t *wq4,
                             const float *s_w, int64_t M, int64_t N, int64_t K,
                             int group_size, void *y_f16, void *stream);

/* Either product (bits 8: wq int8 [N, K]; bits 4: packed uint8 [N, K/2]) with
   the output rounded to y_dtype (fp16 or bf16): y [M, N]. */
cider_status cider_gemm_ex(const int8_t *xq, const float *s_tok, const void *wq, const float *s_w,
                           int64_t M, int64_t N, int64_t K, int bits, int group_size, int y_dtype,
                           void *y, void *stream);

/* Test hooks: the same kernels with the dequant epilogue replaced by a raw
   store of the int32 accumulators ("Quantization" table, Accumulation INT32):
   acc int32 [M, N] (group_size 0) or [M, N, K/gs] (one sum per group). */
cider_status cider_w8a8_gemm_i32(const int8_t *xq, const int8_t *wq, int64_t M, int64_t N,
                                 int64_t K, int group_size, int32_t *acc, void *stream);
cider_status cider_w4a8_gemm_i32(const int8_t *xq, const uint8_t *wq4, int64_t M, int64_t N,
                                 int64_t K, int group_size, int32_t *acc, void *stream);

/* Bytes of device workspace cider_w8a8_linear / cider_w4a8_linear need for M
   tokens of K features (the int8 activations and their scales). */
size_t cider_linear_workspace_bytes(int64_t M, int64_t K);

/* Bytes of workspace that also let a linear call of this shape split K over
   several workgroups per output tile (2 to 8 splits on the matrix-core path,
   where that is faster: per group up to 256 tokens; per channel never): the
   int8 activations and scales as above, then the partial sums of the split
   product (4 bytes per output of each 64 x 32, 64 or 128 tile and split) and
   one counter per tile. Equal to cider_linear_workspace_bytes(M, K) when the
   shape is not split, shapes the matrix-vector kernel serves under the
   current path setting included. The split count follows the current
   device's compute-unit count. A linear call given at least this many bytes
   splits; given fewer (but at least cider_linear_workspace_bytes(M, K)) it
   runs unsplit. The fp32 partial sums of the splits are added in split order
   (deterministic; a different rounding order from the unsplit group-by-group
   sum, within the same tolerance of the exact result). */
size_t cider_linear_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int bits,
                                       int group_size);

/* The whole layer on fp16 activations, mirroring perchannel_linear(x, w, s)
   and w4a8_linear(x, packed, s) of Cider README "Low-Level API":
   quantize_act into `workspace`, then the product.  On the matrix-vector path
   the quantization is fused into the matrix-vector kernel and the workspace
   is not touched (it may be null).  Under the automatic path setting that
   path takes M * K <= 65536 with M <= 3 per channel or M <= 2 per group
   where the few-token matrix-core kernel applies (K a multiple of 128 for
   int8 weights, 256 for int4), else M <= 8 (M <= 4 for int4 weights); calls
   within M <= 8 (int4: 4) and M * K <= 65536 given no workspace, or less
   than cider_linear_workspace_bytes(M, K), also take it.  x: fp16 [M, K]
   row stride ldx; y: fp16 [M, N]. */
cider_status cider_w8a8_linear(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                               const int8_t *wq, const float *s_w, int64_t N, int group_size,
                               void *workspace, size_t workspace_bytes, void *y_f16,
                               void *stream);
cider_status cider_w4a8_linear(const void *x_f16, int64_t M, int64_t K, int64_t ldx,
                               const uint8_t *wq4, const float *s_w, int64_t N, int group_size,
                               void *workspace, size_t workspace_bytes, void *y_f16,
                               void *stream);

/* The whole layer for any input / output type, with optional smoothing:
   cider_quantize_act_ex into `workspace`, then cider_gemm_ex.  fp16 tokens
   without smoothing on the matrix-vector path (see cider_w8a8_linear) are
   quantized inside the matrix-vector kernel and need no workspace; every
   other call needs cider_linear_workspace_bytes(M, K) bytes of it, or cider_linear_workspace_bytes_ex(...) bytes to split K.
   Calls that share a workspace must be ordered (one stream). */
cider_status cider_linear_ex(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                             const float *smooth, const void *wq, const float *s_w, int64_t N,
                             int bits, int group_size, int y_dtype, void *workspace,
                             size_t workspace_bytes, void *y, void *stream);

/* Size of the static device array that serves as cider_linear_ex_noalloc's
   workspace on each GPU (64 MiB). */
#define CIDER_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* For callers that cannot allocate device memory (code under HIP graph
   capture, tight serving loops, harnesses that forbid hipMalloc): the same
   layer as cider_linear_ex, with the workspace taken from a file-scope device
   array of CIDER_NOALLOC_SCRATCH_BYTES per GPU that the library holds until
   the process ends.  No allocation of any kind happens in the call; the
   first call on a device looks up that device's array address once.  The
   call splits K exactly when cider_linear_ex given
   cider_linear_workspace_bytes_ex(...) bytes would, as long as those bytes fit
   in the array, so its results equal that call's bit for bit; shapes whose
   split workspace does not fit run unsplit (equal to cider_linear_ex given
   cider_linear_workspace_bytes(M, K) bytes).  Calls whose
   cider_linear_workspace_bytes(M, K) exceeds the array (M * K above about
   64 Mi) return CIDER_ERR_SCRATCH_LIMIT before any launch; fused one-token
   calls use no workspace.  Every call on one GPU shares that GPU's array and
   leaves its contents behind (the quantize launch clears the split counters
   each call), so calls must be ordered on one stream: calls that overlap on
   one GPU (concurrent streams, several host threads) race on the array and
   give undefined results.  Arguments and other statuses as cider_linear_ex. */
cider_status cider_linear_ex_noalloc(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                     const float *smooth, const void *wq, const float *s_w,
                                     int64_t N, int bits, int group_size, int y_dtype, void *y,
                                     void *stream);

/* The pages' decode kernel (Cider README, "Metal Kernel Pipeline", Decode
   (M = 1): a direct matrix-vector product with on-the-fly weight
   dequantization and no activation quantization):
     y[n] = sum_g s_w[n, g] * sum_{k in g} x[k] * q[n, k]
   (per channel: one group of K), accumulated in fp32 and rounded once to
   y_dtype.  x fp16 [K]; wq / s_w as for the products (bits 8 or 4, group_size
   0 / 64 / 128); y [N].  K % 64 == 0 and K <= 32768; any N >= 0.  Unlike the W8A8 one-token path, the result is not
   that of the quantized-activation formula: it is the dequantized-weight
   product, the other reading of the pages' decode step. */
cider_status cider_decode_linear(const void *x_f16, int64_t K, const void *wq, const float *s_w,
                                 int64_t N, int bits, int group_size, int y_dtype, void *y,
                                 void *stream);

/* ---- Low-rank adapters -------------------------------------------------------
 *
 * Beside a product whose weights many requests share, each request's own
 * correction of them: rows seg_start[i] .. seg_start[i + 1] - 1 of a call are
 * segment i, with the adapter in slot[i],
 *   t[r, j] = sum_k A[slot, j, k] * x[r, k]               j < slices * rank
 *   y[r, n] = y_in[r, n] + scale[slot] * sum_j B[slot, n, j] * t[r, s(n) * rank + j]
 * with s(n) the slice of output n: a fused product (QKV, gate and up) has an A of
 * rank rows for each of its parts.  t and all sums are fp32, y is rounded once.  t
 * enters the second product off by 2^-17 of itself at most in bf16, in fp16 by 2^-22
 * or by 2^-38 of the token's largest |t| in the slice, whichever is more; it meets the
 * scale on the way there, and scale * t past fp32's end is infinite.  A slot outside
 * [0, slots) is no adapter: y = y_in.  Adapters of a smaller rank have zeros in
 * the rest of A or B.  Where x, A or t is infinite or NaN, y is what the formula
 * gives, row by row; where B is, outputs of that row of B are no finite numbers.
 *
 * A segment whose rows are not inside [0, rows], or are more than max_rows, is
 * left out, and its rows, like rows of no segment, stay as they are.  max_rows
 * sizes the launches, so calls captured into a graph replay with any segments and
 * slots within the bounds.  No row is in two segments.
 *
 * Envelope: rank a multiple of 8 up to 128, in_features a multiple of 64, 1 to 8
 * slices whose ends are multiples of 64 and rise, in_features and outputs below
 * 2^24, rows, max_rows <= 2^30, slots < 2^31, segments times the 16-row tiles of
 * max_rows times (outputs / 64 + slices * rank) < 2^31; device pointers 16-byte
 * aligned (int32 and scale arrays: 4), row strides multiples of 8.  segments, rows or
 * max_rows 0 is a no-op. */
#define CIDER_LORA_MAX_SLICES 8
typedef struct {
    const void *a;        /* device, [slots][slices * rank][in_features], of the call's dtype */
    const void *b;        /* device, [slots][slice_end[slices - 1]][rank] */
    const float *scale;   /* device, [slots], or null: 1 */
    int64_t slots, rank, in_features, slices;
    int64_t slice_end[CIDER_LORA_MAX_SLICES]; /* outputs of slice i end there */
} cider_lora;

/* Bytes of workspace with which the call uses as much of the GPU as it measured
   faster (0 outside the envelope).  Needed at the least, else
   CIDER_ERR_WORKSPACE: 4 * rows * slices * rank. */
size_t cider_lora_workspace_bytes(const cider_lora *lora, int64_t segments, int64_t rows,
                                  int64_t max_rows);

/* Adds segments' adapters to a product's output.  x [rows][in_features], y_in, y
   [rows][outputs] of type dtype with row strides ldx, ldy_in, ldy; y may be y_in
   with the same stride (added in place), else it overlaps nothing.  Results do
   not depend on timing; another workspace size may group the fp32 sums of t
   otherwise.  Calls that share a workspace must be ordered (one stream). */
cider_status cider_lora_add(const cider_lora *lora, const int32_t *seg_start, const int32_t *slot,
                            int64_t segments, int64_t rows, int64_t max_rows, const void *x,
                            int dtype, int64_t ldx, const void *y_in, int64_t ldy_in,
                            void *workspace, size_t workspace_bytes, void *y, int64_t ldy,
                            void *stream);

/* ---- 4-bit key/value cache --------------------------------------------------
 *
 * What stands between the QKV product and the O product when a decoder serves:
 * keys and values quantized as they enter a paged cache, and attention that
 * reads the cache.  Codes and scales are the int4 ones of the definitions
 * above, one scale per group_size consecutive elements of a head:
 *   s = absmax / 7 (fp32, correctly rounded), q = clamp(rint(x / s), -8, 7),
 *   stored nibble u = q + 8; the value a code stands for is s * (u - 8).
 *
 * A batch holds `batch` sequences.  Sequence b brings the rows
 * row_start[b] .. row_start[b + 1] - 1 (n_b of them) to the call and holds
 * kv_len[b] tokens in the cache once they are in it, so its row i is the token
 * at position p = kv_len[b] - n_b + i.  A row at p < 0 is not there: append
 * skips it, read and attention write zeros (a slot a program pads its batch
 * with: one row, kv_len 0).
 *
 * Pages: a page holds 64 consecutive tokens of one sequence; token t of
 * sequence b is in page pages[b][t / 64] at t % 64.  The cache is
 * uint8 [num_pages][kv_heads][block], a block being one head of one page,
 * 64 * D + 512 * (D / group_size) bytes (D = head_dim):
 *   K codes   dword (t, j, m), t < 64, j < 4, m < D/32, row-major:
 *             nibble e is element d = 32 m + 8 j + e of token t;
 *   V codes   dword (B, g, j, c, x), B < 2, g < D/64, j < 4, c < 16, x < 4,
 *             row-major: nibble 4 b + i is token 32 B + 16 b + 4 j + i,
 *             element d = 64 g + 16 x + c;
 *   K scales  fp32 [D / group_size][64],  V scales  fp32 [D / group_size][64].
 * Memory of a page may hold anything before its tokens are written.
 *
 * The device arrays are read by the kernels only, with these bounds: kv_len
 * outside [0, max_kv_len] is taken as the nearer end; a sequence whose row
 * range is not inside [0, rows] or longer than max_rows is left out (its rows
 * are not written); a page number outside [0, num_pages) is never followed
 * (append skips its tokens, read writes zeros for them, attention does not
 * see them).  max_kv_len and max_rows also size the launches, so calls
 * captured into a graph replay with any lengths up to them.  Two sequences
 * may share pages (a common prefix) as long as no call appends to them.
 *
 * Envelope: head_dim 64 or 128, group_size 64 or 128 dividing it,
 * batch, rows, max_rows >= 0, 0 <= max_kv_len <= 64 * max_pages <= 2^30,
 * 1 <= num_pages < 2^31, 1 <= kv_heads <= 65536, q_heads a multiple of
 * kv_heads up to 65536, rows * q_heads <= 2^30, batch * kv_heads times the
 * 32-token spans of max_rows (attention: batch * q_heads * max_rows) < 2^31;
 * pointers 16-byte aligned (int32 arrays: 4), row strides in elements, multiples of 8, at
 * least the row's heads * head_dim.  batch, rows or max_rows 0 is a no-op. */
typedef struct {
    void *cache;              /* uint8 [num_pages][kv_heads][block] */
    const int32_t *pages;     /* [batch][max_pages] */
    const int32_t *row_start; /* [batch + 1], ascending */
    const int32_t *kv_len;    /* [batch] tokens cached, this call's rows among them */
    int64_t batch, rows;      /* sequences; rows of all of them in this call */
    int64_t max_rows;         /* bound on the rows of one sequence */
    int64_t max_kv_len;       /* bound on kv_len */
    int64_t max_pages;        /* row length of `pages` */
    int64_t num_pages, kv_heads, head_dim;
    int group_size;
} cider_kv4_batch;

/* Bytes of a cache of this geometry; 0 outside the envelope. */
size_t cider_kv4_cache_bytes(int64_t num_pages, int64_t kv_heads, int64_t head_dim, int group_size);

/* Quantizes the batch's rows into the cache.  k, v: [rows][kv_heads][head_dim]
   of type dtype with row strides ldk, ldv (the columns of a fused QKV
   product's output are read in place).  Tokens already in a page stay as they
   are; a token that is appended again is overwritten.  No two sequences of the
   call may append to the same page. */
cider_status cider_kv4_append(const cider_kv4_batch *b, const void *k, const void *v, int dtype,
                              int64_t ldk, int64_t ldv, void *stream);

/* Norm and rotation of a batch's queries and keys, on the keys' way into the
   cache.  For a head x of a row, r = 1 / sqrt(mean_d x_d^2 + eps):
     n_d = x_d * r * weight_d            (weight null: n = x)
   the first rot_dim elements of n form pairs (a, b), pair i being elements
   (i, i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved; each turns by the
   table's (c, s) = cos_sin[position][i]:
     a' = a * c - b * s,   b' = b * c + a * s
   and the elements past rot_dim stay.  What a model does to its angles
   (stretching, frequencies, a factor on both) is in the table, and what it adds
   to its weights in the weights.  position is the row's p, or positions[0][row];
   with several axes (time, height and width of images and video) pair i takes
   positions[pair_axis[i]][row].  A position outside the table is taken as the
   nearer end. */
typedef struct {
    const float *cos_sin;       /* device, [table_len][rot_dim / 2][2]; not read if rot_dim is 0 */
    const int32_t *positions;   /* device, [axes][rows], or null if axes is 1 */
    const float *q_weight;      /* device, [head_dim], or null: no norm of q */
    const float *k_weight;      /* the same of k */
    const uint8_t *pair_axis;   /* host, [rot_dim / 2], each below axes; not read if axes is 1 */
    int64_t table_len, rot_dim; /* rot_dim a multiple of 16 up to head_dim */
    int64_t axes;               /* 1 to 4 */
    int interleaved;
    float eps;                  /* positive; not looked at without weights */
} cider_rotation;

/* cider_kv4_append with norm and rotation in the same pass: q' rounded once to
   dtype into q_out, k' (evaluated in 64 bits and rounded once to fp32, so that
   its codes do not depend on the order of operations) and v quantized into the
   cache as cider_kv4_append does.  q, q_out: [rows][q_heads][head_dim] with row
   strides ldq, ldq_out; q_out may be q itself with the same stride (a fused QKV
   product's columns turned in place), else it overlaps nothing.  q_heads is a
   multiple of kv_heads; 0: only keys and values.  q_out is written with zeros
   for rows that are not there, and a row whose page is not in the cache has its
   q' all the same.  Row ranges, lengths and pages are bounded as above. */
cider_status cider_kv4_append_rotated(const cider_kv4_batch *b, const cider_rotation *rotation,
                                      const void *q, const void *k, const void *v, int dtype,
                                      int64_t ldq, int64_t ldk, int64_t ldv, int64_t q_heads,
                                      void *q_out, int64_t ldq_out, void *stream);

/* Reads the cached values of the batch's rows back: the fp32 product s * (u - 8) rounded
   to dtype (n_b = kv_len[b] reads a whole sequence).  k, v:
   [rows][kv_heads][head_dim] with row strides ldk, ldv. */
cider_status cider_kv4_read(const cider_kv4_batch *b, void *k, void *v, int dtype, int64_t ldk,
                            int64_t ldv, void *stream);

/* Causal attention of the batch's rows over the cache (grouped query heads:
   query head h reads kv head h / (q_heads / kv_heads)):
     t visible from p:  t <= p, and t > p - window or t < sinks (window > 0;
                        window 0: every t <= p)
     S[t] = scale * sum_d q[d] * K[t, d],  P[t] = exp(S[t] - max S)
     y[d] = sum_t P[t] * V[t, d] / sum_t P[t];  no visible t: y = 0
   with K, V the values the codes stand for; scores, softmax and sums in fp32
   (scale * |K| and scale * |q| * |K| of the largest elements are to stay
   below 2^118; a row that meets NaN or infinity where it may look, a scale of
   the cache among them, gives NaN, of an infinite value NaN or infinity in the
   group's elements, and what it may not see never reaches it). For the two
   products q, times a power of two of its row or of rows of about one size,
   and P times V's scales, times a power of two of the row, are fp16: elements
   of q down to 2^-17 of their row's largest lose nothing, smaller ones 2^-28
   of that at most; the weights keep 11 significant bits, 22 for few rows with
   fp16 outputs, as long as P times V's scale, P being up to 1, is above 2^-21
   of the largest of V's scales that the row sees. Few rows sum codes as 0 to 15
   and take the offset off, which costs about 2^-17 of the weighted mean of V's
   scales (over 1131 tokens). Against 64 bits (norm of the difference over norm
   of y) fp16 outputs are 2.0e-4 to 2.7e-4 off for few rows and 2.9e-4 for many,
   where y's own rounding is 2.0e-4, bf16 ones 1.7e-3, where it is 1.66e-3.
   Where rows that stand within 256 (row, head) pairs see values more than
   2^130 apart, the smaller ones lose bits, and so do a token's keys whose two
   groups have scales more than 2^120 apart. The rows' own tokens must have been appended before. q, y:
   [rows][q_heads][head_dim] of types q_dtype, y_dtype, row strides ldq, ldy.
   scale finite and positive; window, sinks >= 0 (the first `sinks` tokens stay
   visible behind a window).  One row per sequence is a decoding step, a few
   are drafted tokens, many a prompt or a chunk of one.  The kernel and the
   splitting are chosen by the bounds, max_rows among them, for all sequences:
   decoding steps in one call with a prompt's chunk are right but slow (63 steps
   over 8192 tokens and a chunk of 2048 rows: 758 us in one call, 119 + 351 in
   two).
   workspace: device scratch of any size, or null; given
   cider_kv4_attention_workspace_bytes(...) bytes, long caches with few rows
   are split over more workgroups (fp32 partial results, added in order:
   results do not depend on timing); given fewer the call splits less or not
   at all.  Calls that share a workspace must be ordered (one stream). */
cider_status cider_kv4_attention(const cider_kv4_batch *b, const void *q, int q_dtype, int64_t ldq,
                                 int64_t q_heads, float scale, int64_t window, int64_t sinks,
                                 void *workspace, size_t workspace_bytes, void *y, int y_dtype,
                                 int64_t ldy, void *stream);

/* Bytes of workspace with which the attention call splits as far as it
   measured faster (0 for shapes that are never split, and outside the
   envelope).  Reads only the sizes of *b, no device memory. */
size_t cider_kv4_attention_workspace_bytes(const cider_kv4_batch *b, int64_t q_heads,
                                           int64_t window, int64_t sinks);

/* Runs of sequences that hold the same first pages (conversations behind one
   system prompt, samples of one question, questions about one document): run g
   is the sequences group_start[g] .. group_start[g + 1] - 1, whose rows of
   `pages` name the same pages for the first shared_len[g] tokens.  Sequences in
   front of the first run and behind the last are in none. */
typedef struct {
    const int32_t *group_start; /* device, [groups + 1], ascending */
    const int32_t *shared_len;  /* device, [groups] */
    int64_t groups;
    int64_t max_rows;           /* bound on the rows of all sequences of a run */
    int64_t max_shared_len;     /* bound on shared_len, up to 64 * max_pages */
} cider_kv4_runs;

/* cider_kv4_attention (window 0) that reads the pages a run shares once for all
   rows of the run, with the same result but for the order of fp32 sums: a part
   over the shared pages, the rows of the run taken together, and one over each
   sequence's own pages are joined by their maxima and sums, all fp32.  Only whole pages count as shared
   (shared_len rounded down to 64).  Bounded on the device as the batch is:
   shared_len outside [0, max_shared_len] is taken as the nearer end; a run that
   is not inside the batch, or has more than max_rows rows, shares nothing, and
   neither does a sequence whose rows do not all stand behind the shared pages
   (a padded slot, one without rows): those attend to their own page table alone,
   which need not name the run's pages.  What the others name for them is read from
   the table of the first of those.
   Ranges and precision are those of cider_kv4_attention.  What sequences have
   behind their shared pages is dealt out for max_kv_len - max_shared_len tokens;
   more (of a sequence in no run, or behind a prefix far shorter than the bound)
   is right but one workgroup's (64 single rows behind 65536 tokens, bf16, 8 kv
   heads of 128: 129 us; with one of them in no run 406, where 63 in this call and
   that one in cider_kv4_attention take 122 + 22).  So max_shared_len is to be as
   tight as lengths allow, and long sequences of no run belong in a call apart.
   workspace: device scratch of cider_kv4_attention_shared_workspace_bytes(...)
   bytes at the least (else CIDER_ERR_WORKSPACE); calls that share one must be
   ordered.  groups, max_rows or max_shared_len / 64 of 0 make it
   cider_kv4_attention. */
cider_status cider_kv4_attention_shared(const cider_kv4_batch *b, const cider_kv4_runs *runs,
                                        const void *q, int q_dtype, int64_t ldq, int64_t q_heads,
                                        float scale, void *workspace, size_t workspace_bytes,
                                        void *y, int y_dtype, int64_t ldy, void *stream);

/* Bytes of workspace that the call needs (0 outside the envelope).  Reads only
   the sizes of *b and *runs, no device memory. */
size_t cider_kv4_attention_shared_workspace_bytes(const cider_kv4_batch *b,
                                                  const cider_kv4_runs *runs, int64_t q_heads);

/* Test hook: force the attentions' column tiles for subsequent calls in this
   process.  0 = automatic (by sizes), 16 = the few-row kernel, 128 or 256 = the
   many-row kernel with that many (row, query head) pairs a tile; every setting
   takes every shape.  Returns the previous setting, or -1 for an invalid value. */
int cider_kv4_set_tiles(int columns);

/* Test hook: force the product path for subsequent calls in this process.
   0 = automatic (M * K <= 65536 and M <= 8, or M <= 4 for int4 weights ->
   matrix-vector, else matrix cores),
   1 = always the matrix-vector kernel (calls with M > 8 or M * K > 65536 then
   return CIDER_ERR_UNSUPPORTED_SHAPE), 2 = always the matrix-core kernel.
   Returns the previous setting, or -1 for an invalid value. */
int cider_set_path(int path);

#ifdef __cplusplus
}
#endif

#endif /* CIDER_H */
