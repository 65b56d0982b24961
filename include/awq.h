/*
 * awq.h -- C ABI of libawq.so: the AWQ per-layer activation-aware scale
 * search and final group quantization on AMD Instinct MI355X (gfx950).
 *
 * The method (sources cited by page title and section):
 *   "AWQ (activation-aware weight quantization)" (pigeon guide), sections
 *   "How it works" and "The code, line by line": measure each input channel's
 *   mean activation magnitude s_X; for each alpha on an even grid over [0, 1]
 *   scale the weight columns by s = s_X^alpha (centred by sqrt(max s * min s)),
 *   round the scaled weights group-wise, undo the scaling, and measure the mean
 *   squared layer output error on the calibration inputs; keep the alpha with
 *   the smallest error. "AWQ vs GPTQ Quantization Architectures Compared",
 *   "What lands on disk": the deployable result is integer codes plus one scale
 *   and one zero point per group and output row.
 *
 * Conventions for every call:
 *   - Pointers are device pointers on the current HIP device unless stated;
 *     tensors are contiguous and row-major. W is (out, in), X is (tokens, in)
 *     (y = W x per token). W and X share one element type (awq_dtype).
 *   - The caller owns every buffer (inputs, outputs and workspace). The library
 *     keeps no state between calls and allocates no device memory.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream) and
 *     the call returns before it runs: outputs are valid once the caller has
 *     synchronised with the stream.
 *   - Every argument is checked on the host before anything is enqueued. A
 *     failed check returns a negative status and writes nothing. A failed
 *     kernel launch returns AWQ_ERR_HIP. No C++ exception crosses the ABI.
 */
#ifndef AWQ_H
#define AWQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { AWQ_F32 = 0, AWQ_F16 = 1, AWQ_BF16 = 2 } awq_dtype;
typedef enum { AWQ_SYM = 0, AWQ_ASYM = 1 } awq_qmode;

enum {
    AWQ_OK = 0,
    AWQ_ERR_INVALID_ARG = -1, /* null pointer, size < 1, in % group != 0, bits outside [2, 8], grid < 1, bad enum */
    AWQ_ERR_WORKSPACE = -2,   /* ws_bytes below the matching *_workspace_size() (or ws == NULL with a nonzero size) */
    AWQ_ERR_HIP = -3,         /* a HIP runtime call or kernel launch failed */
    AWQ_ERR_NONFINITE = -4,   /* reserved, never returned by a GPU entry point: a search whose
                               * candidate errors are all non-finite reports best = -1 in
                               * device memory, and that flag is the only authoritative
                               * report (the call returns before the kernels finish) */
    AWQ_ERR_UNSUPPORTED = -5  /* valid arguments outside what the GPU kernels implement (see each call) */
};

/* Largest grid accepted by awq_search / awq_s_table (grid + 1 candidates). */
#define AWQ_MAX_GRID 1024

/* Step 1, activation statistics ("AWQ (activation-aware weight quantization)",
 * "How it works" step 1 and the first line explained in "The code, line by line"):
 *   xmag[j] = fp32( mean_t |X[t, j]| + 1e-8 )
 * summed in fp64 in a fixed order: sequentially within consecutive 64-token
 * chunks, then the chunk sums in ascending chunk order; bitwise reproducible.
 *   X:    device, (tokens, in) of `dtype`.
 *   xmag: device, fp32[in] (output).
 *   ws:   device scratch of awq_act_stats_workspace_size(tokens, in) bytes; the
 *         current kernel keeps its partial sums on chip, the size is 0 and ws
 *         may be NULL (the argument stays for kernels that need scratch).
 */
int awq_act_stats(const void *X, int dtype, int64_t tokens, int64_t in, float *xmag,
                  void *ws, size_t ws_bytes, void *stream);
size_t awq_act_stats_workspace_size(int64_t tokens, int64_t in);

/* Step 2 alone, the candidate scales ("The code, line by line": grid + 1 evenly
 * spaced alpha in [0, 1] including 0; s = xmag^alpha divided by
 * sqrt(max s * min s)). alpha_k = k / grid in fp64, the power and centring in
 * fp64, one rounding to fp32:
 *   s_table[k][j] = fp32( xmag[j]^alpha_k / sqrt(max_j xmag^alpha_k * min_j xmag^alpha_k) )
 *   xmag:    device fp32[in];  s_table: device fp32[(grid + 1) * in] (output).
 * awq_search computes the same table internally; this call exposes it. */
int awq_s_table(const float *xmag, int64_t in, int grid, float *s_table, void *stream);

/* Steps 2-4, the search ("Source code", awq() listing of the pigeon guide;
 * "AWQ: move the error away from what matters", awq_scales()). For every
 * candidate k = 0..grid, with s = s_table[k]:
 *   Wq  = Q(W diag(s)) diag(s)^-1        (group round-to-nearest, see quantize_pack)
 *   mse[k] = mean over tokens*out of (X Wq^T - X W^T)^2
 * and best = the smallest k whose mse is strictly below every earlier one
 * (so the lowest alpha wins ties and a NaN error is never chosen).
 *   W, X:    device, (out, in) and (tokens, in) of `dtype`.
 *   xmag:    device fp32[in], as written by awq_act_stats (any positive values work).
 *   bits:    2..8;  group: divides in;  grid: 1..AWQ_MAX_GRID;  mode: awq_qmode.
 *   mse:     device fp64[grid + 1] (output).
 *   best:    device int32[1] (output); -1 when no candidate error is finite.
 *   s_best:  device fp32[in] (output): s_table[best], or all ones when best = -1.
 *            Deploy by multiplying W's columns by it and dividing the layer's
 *            input by it upstream.
 *   ws:      device scratch of at least awq_search_workspace_size(...) bytes:
 *            the s-table and its reciprocals, one fp64 partial per (candidate,
 *            block), and a 16-bit copy of X in matrix-fragment order padded to
 *            whole 256-token blocks (used by the 16-bit path).
 * The GPU kernels evaluate the error as X (Wq - W)^T (equal to the difference
 * of the two products by linearity), accumulating in fp32 and summing squares
 * in fp64; mse is accurate to about 1e-5 relative, not bitwise. Operands are
 * 16-bit (the input type) for fp16/bf16 layers with at least 256 rows and 16
 * tokens, and exact fp32 otherwise (fp32 inputs, or layers too small for the
 * unbiased 16-bit rounding of Wq - W to average out below 1e-3).
 * AWQ_ERR_UNSUPPORTED: group not in {32, 64, 128}; W, X or ws not 16-byte
 * aligned (any allocation is; an offset view need not be). */
int awq_search(const void *W, const void *X, int dtype, int64_t out, int64_t in,
               int64_t tokens, const float *xmag, int bits, int group, int grid, int mode,
               double *mse, int32_t *best, float *s_best, void *ws, size_t ws_bytes,
               void *stream);
size_t awq_search_workspace_size(int64_t out, int64_t in, int64_t tokens, int grid);

/* awq_search without a workspace argument, for callers that cannot allocate
 * device memory (code under stream capture, tight serving loops, harnesses
 * that forbid allocation). Arguments, outputs and results are those of
 * awq_search; the scratch is a fixed static device array of
 * AWQ_SEARCH_NOALLOC_MAX_BYTES per GPU, held until the process ends.
 *   - The scratch of the current device (hipGetDevice) is used: `stream` must
 *     belong to that device. The first call on a device looks its address up
 *     (no allocation); make that first call outside stream capture.
 *   - AWQ_ERR_WORKSPACE when awq_search_workspace_size(out, in, tokens, grid)
 *     exceeds AWQ_SEARCH_NOALLOC_MAX_BYTES (24 MiB: e.g. 4096 x 4096 with up to
 *     2048 tokens, 12288 x 4096 with 2048 tokens); nothing is launched then.
 *   - Every call on one GPU shares that GPU's scratch: calls that overlap in
 *     time on one GPU (two streams, two host threads) race and must be
 *     serialised by the caller. Nothing in the scratch has to start at zero:
 *     each call writes every scratch byte it later reads. */
#define AWQ_SEARCH_NOALLOC_MAX_BYTES ((size_t)24 << 20)
int awq_search_noalloc(const void *W, const void *X, int dtype, int64_t out, int64_t in,
                       int64_t tokens, const float *xmag, int bits, int group, int grid, int mode,
                       double *mse, int32_t *best, float *s_best, void *stream);

/* awq_search in its three stages, in this order on one stream with one
 * workspace. They let a caller time or profile the error kernel alone, and
 * they are where a search sharded over devices would combine its partial
 * sums. Arguments mean what they mean for awq_search; each stage validates
 * its own arguments the same way.
 *   awq_search_prepare:    the s-table and its reciprocals into ws (step 2),
 *                          and, for layers that take the 16-bit search, a
 *                          copy of X in matrix-fragment order (one launch).
 *   awq_search_candidates: the fused quantize-dequantize-error kernel; leaves
 *                          one fp64 partial sum of squares per (candidate,
 *                          block of 16 rows x 256 tokens) in ws. Needs the
 *                          ws that awq_search_prepare filled from the same X.
 *   awq_search_finish:     fixed-order reduction of the partials into mse,
 *                          argmin into best, s_best. Needs the candidates' ws.
 * awq_search is exactly the three stages. */
int awq_search_prepare(const void *X, int dtype, const float *xmag, int64_t out, int64_t in,
                       int64_t tokens, int grid, void *ws, size_t ws_bytes, void *stream);
int awq_search_candidates(const void *W, const void *X, int dtype, int64_t out, int64_t in,
                          int64_t tokens, int bits, int group, int grid, int mode, void *ws,
                          size_t ws_bytes, void *stream);
int awq_search_finish(int64_t out, int64_t in, int64_t tokens, int grid, double *mse,
                      int32_t *best, float *s_best, void *ws, size_t ws_bytes, void *stream);

/* Step 5, final quantization and packing of W diag(s). Per output row o and
 * group of `group` consecutive columns, with v = fp32(W[o, j] * s[j]):
 *   symmetric ("GPTQ and AWQ weight quantisation", "Per-group symmetric int4
 *   (RTN)" and the n-bit form in "Output MSE vs bit width"): L = 2^(bits-1) - 1,
 *     scale = max(max|v| / L, 1e-8), q = clamp(rne(v / scale), -L-1, L),
 *     code = q + 2^(bits-1), zero = 2^(bits-1);
 *   asymmetric ("AWQ vs GPTQ Quantization Architectures Compared", group_params
 *   and rtn in "GPTQ: compensate the error you just made"): maxq = 2^bits - 1,
 *     lo = min(min v, 0), hi = max(max v, 0), scale = max((hi - lo) / maxq, 1e-8),
 *     zero = rne(-lo / scale), code = clamp(rne(v / scale) + zero, 0, maxq).
 * All in fp32 with IEEE division and round-half-to-even, in exactly this order:
 * the outputs are bit-exact. Dequantize as scale * (code - zero).
 * Non-finite W or s: the scales, zeros and codes of the groups they touch are
 * unspecified (no error is reported); all other groups are unaffected.
 *   W:       device (out, in) of `dtype`;  s: device fp32[in] (e.g. s_best).
 *   qweight: device uint32[out][in * bits / 32 rounded up] (output): code i of a
 *            row at bits [i*bits, (i+1)*bits) of the row's little-endian stream
 *            of 32-bit words; every row starts on a word boundary.
 *   scales:  device fp32[out][in / group] (output).
 *   zeros:   device uint8[out][in / group] (output).
 * AWQ_ERR_UNSUPPORTED: group not in {32, 64, 128, 256, 512, 1024, 2048}; W or s
 * not 16-byte aligned. */
int awq_quantize_pack(const void *W, int dtype, int64_t out, int64_t in, const float *s,
                      int bits, int group, int mode, uint32_t *qweight, float *scales,
                      uint8_t *zeros, void *stream);

/* Largest n_clip accepted by awq_clip_search. */
#define AWQ_MAX_CLIP 64

/* Clipping-range search, run after the alpha search on W diag(s_best)
 * ("AWQ (activation-aware weight quantization)", "Simplifications": a
 * per-group clipping threshold that shrinks the range to cut rounding error;
 * "AWQ vs GPTQ Quantization Architectures Compared", "AWQ: move the error away
 * from what matters": a second, smaller search after the scale search that
 * shrinks each group's clipping range when that lowers the output error). The
 * pages fix no numbers; this library's reading: for ratio
 *   r_i = fp32(1 - i * max_shrink / n_clip)   (fp64 arithmetic), i = 0..n_clip-1,
 * each group's quantizer range (see awq_quantize_pack) is scaled by r_i --
 * symmetric [-r A, r A] with A = max|v|, asymmetric [r lo, r hi] -- the scaled
 * weights v = fp32(W[o, j] s[j]) are clamped into it and quantized with that
 * range's scale (and zero), Wq = dequantized value / s, and
 *   sse[o][g][i] = sum over tokens t of ( sum_{j in group g} X[t, j] (Wq[o, j] - W[o, j]) )^2
 * is the group's own squared output error. clip[o][g] = r_i of the first i
 * whose sse is strictly below every earlier one (r_0 = 1, no clipping, wins
 * ties; a NaN never wins).
 *   W, X:       device, (out, in) and (tokens, in) of `dtype`.
 *   s:          device fp32[in], positive (e.g. s_best of awq_search).
 *   bits, group, mode: as for awq_quantize_pack; group in {32, 64, 128}.
 *   n_clip:     1..AWQ_MAX_CLIP;  max_shrink: in [0, 1) (defaults in the
 *               Python binding: 20 and 0.5).
 *   clip:       device fp32[out][in / group] (output): the chosen ratios.
 *   sse:        device fp64[out][in / group][n_clip] (output), or NULL.
 * The kernel forms Wq - W in fp32 from the same quantizer as awq_quantize_pack
 * and multiplies it with X on the matrix cores, accumulating in fp32 over a
 * group: for fp16 X with Wq - W (scaled by a power of two per row) split into
 * two fp16 parts (22 significant bits), for bf16 X split exactly into three
 * bf16 parts, for fp32 X in fp32. The squares are summed over tokens in fp32
 * per 4 tokens, then in fp64, in a fixed order: bitwise reproducible, each
 * sse within a few group-length multiples of fp32 rounding of the exact
 * value; where two ratios' errors lie that close the choice between them may
 * differ from an exact evaluation.
 * AWQ_ERR_UNSUPPORTED: group not in {32, 64, 128}, more than 65535 groups, or
 * W or X not 16-byte aligned. */
int awq_clip_search(const void *W, const void *X, int dtype, int64_t out, int64_t in,
                    int64_t tokens, const float *s, int bits, int group, int mode, int n_clip,
                    float max_shrink, float *clip, double *sse, void *stream);

/* awq_quantize_pack with one clipping ratio per output row and group:
 *   clip: device fp32[out][in / group], each in (0, 1] (as written by
 *         awq_clip_search). Before quantization the group's range is scaled
 *         by its ratio (symmetric [-r max|v|, r max|v|], asymmetric [r lo, r hi]),
 *         v is clamped into that range, and scale and zero are those of the
 *         scaled range, in fp32 in that order: bit-exact. A ratio of 1 gives
 *         exactly awq_quantize_pack's outputs.
 * All other arguments and errors as awq_quantize_pack. */
int awq_quantize_pack_clip(const void *W, int dtype, int64_t out, int64_t in, const float *s,
                           const float *clip, int bits, int group, int mode, uint32_t *qweight,
                           float *scales, uint8_t *zeros, void *stream);

/* Folding the scales into the model ("AWQ (activation-aware weight
 * quantization)", "How it works" step 5 and the transformer paragraph after it;
 * "AWQ vs GPTQ Quantization Architectures Compared", "AWQ: move the error away
 * from what matters"). With W x = (W diag(s)) (diag(s)^-1 x), the searched
 * layer's weight is multiplied by s and whatever produces its input is
 * divided by s: the LayerNorm/RMSNorm weight (and bias) before q/k/v or
 * gate/up, or the output rows of the previous linear layer (up_proj for
 * down_proj; v_proj for o_proj only when its output width equals o_proj's
 * input width -- with grouped-query attention it usually does not).
 * One fp32 operation per element (IEEE), then one round-half-to-even
 * conversion to `dtype`: bit-exact.
 *   awq_fold_rows:  out[r][c] = A[r][c] / s[r]; A (rows, cols) is the producer
 *                   (rows = the searched layer's input width; cols = 1 for a
 *                   norm weight or bias vector).
 *   awq_scale_cols: out[o][j] = W[o][j] * s[j]; W (rows, cols) is the searched
 *                   layer (cols = its input width). awq_quantize_pack takes W
 *                   and s directly; this call writes the scaled weights
 *                   themselves (for export, or for another quantizer).
 *   A / W, out: device, (rows, cols) of `dtype`; out may equal the input (in
 *               place), otherwise the two must not overlap.
 *   s:          device fp32, length rows (fold) or cols (scale).
 * Non-finite or zero s gives the IEEE results (inf, NaN) in the affected
 * elements; no error is reported. */
int awq_fold_rows(const void *A, int dtype, int64_t rows, int64_t cols, const float *s, void *out,
                  void *stream);
int awq_scale_cols(const void *W, int dtype, int64_t rows, int64_t cols, const float *s, void *out,
                   void *stream);

/* The deployment product over the packed layout ("AWQ vs GPTQ Quantization
 * Architectures Compared", "What lands on disk": codes plus one scale and one
 * zero per group and output row; "From checkpoint to kernel": the serving
 * kernel multiplies activations by them, memory-bound at decode):
 *   Y[m][n] = sum_k X[m][k] * scale[n][k/group] * (code[n][k] - zero[n][k/group])
 * X is the layer's input with 1/s already folded into its producer (see
 * awq_fold_rows), so Y approximates the original layer's output.
 *   X:        device (M, in) of x_dtype (AWQ_F16 or AWQ_BF16); 16-byte aligned.
 *   qweight, scales, zeros: device, as written by awq_quantize_pack for an
 *             (out, in) layer with these bits and group; qweight 16-byte aligned.
 *   Y:        device (M, out) of y_dtype: AWQ_F32, or x_dtype (rounded to
 *             nearest even from the fp32 result).
 * Arithmetic: code - zero is exact in the 16-bit operand type; each group's
 * products are summed in fp32 by the matrix cores and multiplied once by the
 * group's scale into an fp32 total (fixed order, bitwise reproducible). Each
 * output is within (group + ngroups + 8) * 2^-24 * sum_k |X[m][k] * Wd[n][k]| of
 * the exact value (plus the final 16-bit rounding when y_dtype is 16-bit).
 * AWQ_ERR_UNSUPPORTED: x_dtype AWQ_F32, bits not in {4, 8}, group not in
 * {32, 64, 128}, a misaligned X or qweight, or M above 2 097 120. */
int awq_qgemm(const void *X, int x_dtype, int64_t M, int64_t in, const uint32_t *qweight,
              const float *scales, const uint8_t *zeros, int64_t out, int bits, int group,
              void *Y, int y_dtype, void *stream);

/* GPTQ on the same layer inputs, a second quantizer producing the same packed
 * outputs ("AWQ vs GPTQ Quantization Architectures Compared", "GPTQ:
 * compensate the error you just made"; "Advanced Quantization Algorithms: AWQ
 * and GPTQ Explained", section 3). In fp64:
 *   H = 2 X^T X;  H[i][i] += damp * mean(diag H);  U = upper Cholesky factor of H^-1;
 *   for each column i in order (all rows at once): at a group start fit the
 *   group's scale (and zero) on the current, already corrected weights of its
 *   columns; round column i; err = (w_i - dequantized) / U[i][i]; subtract
 *   err * U[i][j] from every later column j.
 * The quantizer is awq_quantize_pack's (symmetric or asymmetric), with the
 * range and scale in fp64 and the scale rounded once to fp32 and used as
 * stored; divisions and rounding (half to even) in fp64. Columns are processed
 * in their natural order (no act-order: the packed format has no group index).
 *   awq_gptq_hessian:  H (device fp64, in x in) = 2 X^T X, damped (damp >= 0, e.g. 0.01).
 *   awq_gptq_factor:   U (device fp64, in x in, upper; the strict lower part is 0)
 *                      from H (left unchanged). ws: awq_gptq_factor_workspace_size(in) bytes.
 *   awq_gptq_quantize: the column loop on W with U; writes qweight, scales and
 *                      zeros in awq_quantize_pack's layout. ws:
 *                      awq_gptq_quantize_workspace_size(out, in) bytes.
 *   awq_gptq:          the three in order with one workspace of
 *                      awq_gptq_workspace_size(out, in) bytes.
 * W, X: device (out, in) and (tokens, in) of `dtype`. in must be a multiple of
 * 128 (the column block); group in {32, 64, 128}; bits 2..8. H is positive
 * definite for damp > 0 unless a column of X is entirely zero and damp is 0;
 * otherwise the factor and all outputs are NaN (no error is reported).
 * The GPU accumulates in a different order from a sequential evaluation, so a
 * code can differ where a weight lies within about 1e-12 of a rounding
 * boundary (and the rest of that row may then follow a different path).
 * AWQ_ERR_UNSUPPORTED: in not a multiple of 128, group not in {32, 64, 128},
 * out above 4 194 240. */
int awq_gptq_hessian(const void *X, int dtype, int64_t tokens, int64_t in, double damp, double *H,
                     void *stream);
int awq_gptq_factor(const double *H, int64_t in, double *U, void *ws, size_t ws_bytes, void *stream);
int awq_gptq_quantize(const void *W, int dtype, int64_t out, int64_t in, const double *U, int bits,
                      int group, int mode, uint32_t *qweight, float *scales, uint8_t *zeros, void *ws,
                      size_t ws_bytes, void *stream);
int awq_gptq(const void *W, const void *X, int dtype, int64_t out, int64_t in, int64_t tokens, int bits,
             int group, int mode, double damp, uint32_t *qweight, float *scales, uint8_t *zeros,
             void *ws, size_t ws_bytes, void *stream);
size_t awq_gptq_factor_workspace_size(int64_t in);
size_t awq_gptq_quantize_workspace_size(int64_t out, int64_t in);
size_t awq_gptq_workspace_size(int64_t out, int64_t in);

/* Microscaled 4-bit floating point (MXFP4): every block of AWQ_MX4_BLOCK = 32
 * consecutive columns of a row shares a power of two, and a value is one of
 * +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it. The form that gfx950's scaled matrix
 * instructions take directly, for weights and for activations.
 *   codes:  device uint8 (rows, in / 2): column 2i in the low half of byte i of
 *           the row, column 2i + 1 in the high half; a code's bit 3 is the sign,
 *           bits 0-2 index the magnitudes above.
 *   scales: device uint8 (rows, in / 32): byte b stands for 2^(b - 127), 255 for
 *           NaN (every value of its block is NaN, whatever the codes).
 * `in` must be a multiple of 32. 4.25 bits per value.
 *
 * awq_mx4_quantize: with v = fp32(W[r, j] * s[j]) (s NULL: v = fp32(W[r, j]))
 * and A the largest |v| of a block, e = clamp(floor(log2 A) - 2, -127, 127) (A = 0:
 * -127), byte = e + 127; a code has v's sign and |v| * 2^-e rounded to the
 * nearest magnitude, ties to the even code, 6 above 6. Bit-exact. A block with
 * an infinity or a NaN gets byte 255 and codes 0.
 *   W: device (rows, in) of `dtype`, 16-byte aligned; e.g. a layer's weights,
 *      several layers' or experts' stacked, or activations.
 *   s: device fp32[in], 16-byte aligned, or NULL; e.g. a row of awq_s_table. Choose
 *      it by this format's error: s_best of awq_search makes the error of integer
 *      groups least and may do worse here than no s (the headline recipe at
 *      512x1024: output error 0.00850 with s_best, 0.00825 without, 0.00819 at
 *      the best row of the same table).
 * awq_mx4_dequantize: out (rows, in) of `dtype` = the values, rounded to nearest
 * even where `dtype` does not hold them (bf16 and fp32 hold all below 2^128).
 * Outputs must not overlap inputs, here and in the calls below.
 * AWQ_ERR_UNSUPPORTED: W, s, codes or out not 16-byte aligned, 2^37 values or
 * more, or `in` above 2^23. */
#define AWQ_MX4_BLOCK 32
int awq_mx4_quantize(const void *W, int dtype, int64_t rows, int64_t in, const float *s, uint8_t *codes,
                     uint8_t *scales, void *stream);
int awq_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t in, void *out,
                       int dtype, void *stream);

/* The deployment products over MXFP4 weights W (out, in):
 *   awq_mx4_gemm:    Y[m][n] = sum_k X[m][k] * W[n][k], X (M, in) of x_dtype
 *                    (AWQ_F16 or AWQ_BF16); Y of y_dtype: AWQ_F32 or x_dtype.
 *   awq_mx4_gemm_a4: the same with X MXFP4 too (as awq_mx4_quantize writes it);
 *                    Y of y_dtype, any.
 * Operands enter the matrix cores without rounding and are summed in fp32 in a
 * fixed order (bitwise reproducible): with S = sum_k |X[m][k] W[n][k]| below 2^127
 * each output is within (in + 16) * (2^-24 * S + 2^-149) of the exact value (the
 * second term is fp32's smallest step: products and sums may be subnormal), plus
 * the rounding to a 16-bit Y. In S an operand that is subnormal in its 16-bit type
 * (X below 2^-14 in fp16, X or W below 2^-126 in bf16) counts as the smallest
 * normal number: the matrix cores align its products as if it were that large.
 * A row of X or W that holds a NaN makes its own outputs NaN and no others.
 * awq_mx4_gemm takes values below 2^128: scale byte 253 stands under magnitudes up
 * to 3 and byte 254 under magnitudes up to 1.5 (awq_mx4_quantize writes neither
 * byte). A larger value, which no 16-bit or fp32 number holds, makes the outputs
 * of its row of W infinite or NaN, and no others. awq_mx4_gemm_a4 takes them all.
 * AWQ_ERR_UNSUPPORTED: x_dtype AWQ_F32, X or codes (xcodes) not 16-byte aligned,
 * M above 2 097 120, out above 2^28, `in` above 2^23, or M * out of 2^38 or more. */
int awq_mx4_gemm(const void *X, int x_dtype, int64_t M, int64_t in, const uint8_t *codes,
                 const uint8_t *scales, int64_t out, void *Y, int y_dtype, void *stream);
int awq_mx4_gemm_a4(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t in,
                    const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y, int y_dtype,
                    void *stream);

/* A mixture-of-experts layer for a few tokens (decoding), experts in MXFP4. For
 * each token x (a row of X):
 *   l = router x (fp32); the top_k experts with the largest l (equal ones: the
 *   lowest index; a NaN ranks lowest); p = softmax(l) over all experts at those,
 *   divided by their sum if renorm is not 0 (without it a NaN among l makes p NaN);
 *   h_e = silu(Wgate_e x) * (Wup_e x);  y = sum_e p_e Wdown_e h_e.
 * Everything is fp32 up to Y (the products with the experts as above) but p_e h_e,
 * which keeps 16 significant bits (and fp32's range).
 *   X:      device (M, hidden) of `dtype` (AWQ_F16 or AWQ_BF16), M <= AWQ_MX4_MOE_MAX_TOKENS.
 *   router: device (experts, hidden) of `dtype`.
 *   gu_codes, gu_scales: device, the MXFP4 matrix (experts * 2 * inter, hidden): of each
 *           expert the inter gate rows, then the inter up rows.
 *   dn_codes, dn_scales: device, the MXFP4 matrix (experts * hidden, inter).
 *   Y:      device (M, hidden) of `dtype` (output); must not overlap an input.
 *   ws:     device scratch of awq_mx4_moe_workspace_size(M, hidden, inter, top_k) bytes
 *           (0 for sizes that the call refuses). Calls that overlap in time need
 *           a workspace each.
 * hidden and inter must be multiples of 32, 1 <= top_k <= experts.
 * An expert's NaN values, and those of 2^128 or more (see above), reach only the
 * tokens routed to it.
 * AWQ_ERR_UNSUPPORTED: dtype AWQ_F32, M > AWQ_MX4_MOE_MAX_TOKENS, top_k >
 * AWQ_MX4_MOE_MAX_TOPK, experts > AWQ_MX4_MOE_MAX_EXPERTS, hidden or inter above
 * 2^20, X, router, codes or ws not 16-byte aligned. */
#define AWQ_MX4_MOE_MAX_TOKENS 64
#define AWQ_MX4_MOE_MAX_TOPK 16
#define AWQ_MX4_MOE_MAX_EXPERTS 256
int awq_mx4_moe(const void *X, int dtype, int64_t M, int64_t hidden, int64_t inter, int experts, int top_k,
                int renorm, const void *router, const uint8_t *gu_codes, const uint8_t *gu_scales,
                const uint8_t *dn_codes, const uint8_t *dn_scales, void *Y, void *ws, size_t ws_bytes,
                void *stream);
size_t awq_mx4_moe_workspace_size(int64_t M, int64_t hidden, int64_t inter, int top_k);

/* Microscaled 8-bit floating point (MXFP8): blocks of AWQ_MX4_BLOCK columns under a
 * power of two as in MXFP4, a value being an e4m3 number (sign, 4 exponent bits of
 * bias 7, 3 fraction bits; 0 to 448, steps of 2^-9 below 2^-6) times it: the form of
 * activations between 16 and 4 bits, which the scaled matrix instructions take
 * beside MXFP4 weights. 8.25 bits a value.
 *   codes:  device uint8 (rows, in): the e4m3 bits (0x7F and 0xFF are NaN).
 *   scales: device uint8 (rows, in / 32): as in MXFP4.
 * `in` must be a multiple of 32.
 *
 * awq_mx8_quantize: A the largest |v| of a block, v = fp32(X[r, j]); E the least whole
 * number with A * 2^-E <= 448, clamped to [-127, 127] (A = 0: -127); byte = E + 127,
 * code = v * 2^-E rounded to the nearest e4m3 number, ties to even (none is cut off).
 * Bit-exact. A block with an infinity or a NaN gets byte 255 and codes 0.
 *   X: device (rows, in) of `dtype`, 16-byte aligned.
 * awq_mx8_dequantize: out (rows, in) of `dtype` = the values, rounded to nearest even
 * where `dtype` does not hold them (bf16 and fp32 hold all below 2^128).
 * Outputs must not overlap inputs unless a call says so, here and below.
 * AWQ_ERR_UNSUPPORTED: X, codes or out not 16-byte aligned, 2^37 values or more, or
 * `in` above 2^23. */
int awq_mx8_quantize(const void *X, int dtype, int64_t rows, int64_t in, uint8_t *codes, uint8_t *scales,
                     void *stream);
int awq_mx8_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t in, void *out,
                       int dtype, void *stream);

/* Root-mean-square norm of the rows of a residual stream, to MXFP8:
 *   h = X + R, rounded to `dtype` (R NULL: h = X);
 *   v = fp32(h * weight / sqrt(mean over the row of h^2 + eps)), in 64 bits up to that
 *   rounding;  codes, scales = v as awq_mx8_quantize writes it;  Y = v rounded to `dtype`.
 * The codes are the formula's unless v lies within some 2^-50 of a rounding border. A
 * NaN or an infinity in a row of h makes v NaN, or 0 beside an infinity, in that row
 * and no other. A row of zeros under eps = 0 gives NaN.
 *   X, R:   device (rows, in) of `dtype` (AWQ_F16 or AWQ_BF16); R may be NULL.
 *   weight: device `dtype`[in], e.g. as awq_fold_rows leaves it.
 *   H:      device (rows, in) of `dtype` (output, h); with R only, and may be R or X itself.
 *   Y:      device (rows, in) of `dtype` (output), or NULL; e.g. for router logits.
 * AWQ_ERR_UNSUPPORTED: dtype AWQ_F32, a pointer other than scales not 16-byte aligned,
 * 2^22 rows or more, 2^37 values or more, or `in` above 2^23. */
int awq_mx8_rmsnorm(const void *X, const void *R, int dtype, int64_t rows, int64_t in, const void *weight,
                    double eps, void *H, void *Y, uint8_t *codes, uint8_t *scales, void *stream);

/* The product of MXFP8 activations X (M, in) and MXFP4 weights W (out, in):
 *   Y[m][n] = sum_k X[m][k] * W[n][k], Y of y_dtype, any.
 * Sums, NaN and limits as in awq_mx4_gemm_a4, with an fp32 Y the error too. With a 16-bit Y
 * there is one thing more: the matrix cores align the products of eight neighbouring
 * columns (8 i ... 8 i + 7) to the largest of them before they add them in fp32, and
 * cut off what lies below 2^-13 of it (of the power of two that its operands' exponents
 * make; an operand that is subnormal in its type, |code| < 2^-6 in X and < 1 in W, counts
 * as the smallest normal one). That is at most 2^-10 times the sum over the eights of the
 * largest |X| times the largest |W| of each, and in practice some 2^-15 of Y: far below
 * the rounding of X to e4m3, and of Y to 16 bits. For an fp32 Y, where it would show, the
 * products are made in two parts of X that lose nothing (many tokens take some 1.8 times
 * as long). */
int awq_mx4_gemm_a8(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t in,
                    const uint8_t *codes, const uint8_t *scales, int64_t out, void *Y, int y_dtype,
                    void *stream);

/* The choice of experts for every token from its router logits l:
 *   s_e = softmax(l)_e (AWQ_SOFTMAX) or 1 / (1 + exp(-l_e)) (AWQ_SIGMOID);
 *   r_e = s_e + bias_e, or without a bias l_e, which has the same order as s_e;
 *   the experts form `groups` equal groups of neighbours; the top_groups groups stay whose
 *   group_best (1 or 2) largest s_e + bias_e have the largest sum;
 *   ids = the top_k experts with the largest r_e there, in that order;
 *   weights = s_e of these, divided by their sum if renorm is not 0, times scale.
 * Equal ones: the lowest index first, groups and experts alike. Everything is 64 bits
 * wide up to the weights' rounding to fp32.
 * An expert with the logit -infinity (or the bias -infinity) is masked: never chosen,
 * and no part of a group's sum. Where fewer than top_k others are left, the places
 * behind them hold id -1 and weight 0. A NaN logit ranks below all numbers, counts
 * nothing in the softmax's sum, and makes the weights of its row NaN. Chosen scores
 * whose sum is 0 are not divided.
 *   logits:  device (M, experts) of `dtype`.
 *   bias:    device fp32[experts], or NULL.
 *   ids:     device int32 (M, top_k) (output); weights: device fp32 (M, top_k) (output).
 * groups divides experts; top_k <= top_groups * experts / groups; scale is finite.
 * AWQ_ERR_UNSUPPORTED: experts > AWQ_ROUTE_MAX_EXPERTS, top_k > AWQ_ROUTE_MAX_TOPK,
 * groups > AWQ_ROUTE_MAX_GROUPS, M above 2^25, logits not aligned to their type. */
typedef enum { AWQ_SOFTMAX = 0, AWQ_SIGMOID = 1 } awq_score;
#define AWQ_ROUTE_MAX_EXPERTS 512
#define AWQ_ROUTE_MAX_TOPK 32
#define AWQ_ROUTE_MAX_GROUPS 64
int awq_moe_route(const void *logits, int dtype, int64_t M, int experts, const float *bias, int score,
                  int groups, int top_groups, int group_best, int top_k, int renorm, float scale,
                  int32_t *ids, float *weights, void *stream);

/* SwiGLU experts in MXFP4 on MXFP8 activations, for a given routing and any number
 * of tokens. For each token x (a row of X) with its choices e_j and weights w_j:
 *   h_j = silu(Wgate_e x) * (Wup_e x), e = e_j, rounded as awq_mx8_quantize does;
 *   y = sum_j w_j (Wdown_e h_j), in the order of j.
 * Sums are fp32. Those of gate and up take their products whole, whatever M and y_dtype
 * are (the order of the sums goes with M, and with it an h at a border of its 8 bits);
 * those of down are as in awq_mx4_gemm_a8, whole for an fp32 Y. h as above and Y are the only roundings to
 * fewer bits. Choices outside [0, experts) are left out (a token without
 * any others gets zeros); an expert that a token names twice counts twice.
 *   xcodes, xscales: device, the MXFP8 matrix (M, hidden).
 *   ids, weights:    device int32 and fp32 (M, top_k), e.g. of awq_moe_route.
 *   gu_*, dn_*:      the experts as in awq_mx4_moe.
 *   Y:               device (M, hidden) of y_dtype, any (output).
 *   ws:              device scratch of awq_mx4_experts_workspace_size(M, hidden, inter, experts,
 *                    top_k) bytes (0 for sizes that the call refuses). Calls that overlap in
 *                    time need a workspace each.
 * hidden and inter must be multiples of 32. NaN values and weights reach only the
 * tokens routed to them. Results repeat bitwise.
 * AWQ_ERR_UNSUPPORTED: experts > AWQ_MX4_EXPERTS_MAX_EXPERTS, top_k > AWQ_MX4_EXPERTS_MAX_TOPK,
 * M * top_k > AWQ_MX4_EXPERTS_MAX_PAIRS, hidden or inter above 65536, M * hidden of 2^32 or
 * more, xcodes, gu_codes, dn_codes, Y or ws not 16-byte aligned. */
#define AWQ_MX4_EXPERTS_MAX_EXPERTS 512
#define AWQ_MX4_EXPERTS_MAX_TOPK 32
#define AWQ_MX4_EXPERTS_MAX_PAIRS 1048576
int awq_mx4_experts(const uint8_t *xcodes, const uint8_t *xscales, int64_t M, int64_t hidden, int64_t inter,
                    int experts, int top_k, const int32_t *ids, const float *weights, const uint8_t *gu_codes,
                    const uint8_t *gu_scales, const uint8_t *dn_codes, const uint8_t *dn_scales, void *Y,
                    int y_dtype, void *ws, size_t ws_bytes, void *stream);
size_t awq_mx4_experts_workspace_size(int64_t M, int64_t hidden, int64_t inter, int experts, int top_k);

/* Human-readable name of a status code (static string, never NULL). */
const char *awq_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif
