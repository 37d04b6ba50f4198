/*
 * aq.h -- C ABI of libaq: group-wise affine weight-only quantization and the
 * matmuls that consume the packed form, for AMD Instinct MI355X (gfx950).
 *
 * The format ("Quantization", metalworking MLX notes, opening paragraph and
 * "Mechanics"; "Quantizing a Model for MLX", "What MLX quantization stores"):
 * a weight matrix W [N, K] (N = out_features, K = in_features) is cut along
 * each row into groups of G = 32, 64 or 128 consecutive weights.  Each group
 * stores one fp16 scale s, one fp16 bias b and G codes q of `bits` = 2..8
 * bits, and w ~= q*s + b.  Layouts (all row-major, contiguous):
 *
 *   codes   uint32 [N, K*bits/32]  one least-significant-bit-first bitstream
 *                                  per row: code k sits at bits
 *                                  [k*bits, k*bits+bits) of the row, bit i
 *                                  of the stream being bit i%32 of word i/32
 *                                  ("Tutorial 10: Quantization", s.3, shift
 *                                  and mask extraction; for bits=3 eight
 *                                  codes fill three bytes)
 *   scales  uint16 [N, K/G]        fp16 bit patterns
 *   biases  uint16 [N, K/G]        fp16 bit patterns ("Tutorial 10", s.4
 *                                  container shapes [out, in/group_size])
 *
 * Conventions shared by every entry point:
 *  - Pointers named as device pointers must point to device memory
 *    (hipMalloc'd or torch CUDA tensors) and be 16-byte aligned, else
 *    AQ_ERR_ALIGNMENT.  The caller allocates and owns every buffer; the
 *    library only borrows them for the asynchronous operation and allocates
 *    nothing.
 *  - `stream` is a hipStream_t (NULL = the legacy default stream).  Work is
 *    enqueued asynchronously; results are visible after the stream syncs.
 *  - Arguments are checked on the host before anything is enqueued; a bad
 *    argument returns an error and enqueues nothing.  Launch failures return
 *    AQ_ERR_HIP.  Nothing aborts and no exception crosses the ABI.
 *  - Biases are optional for every consumer (dequantize, embedding and the
 *    matmuls): a NULL biases pointer means every bias is +0, i.e. w = q*s
 *    ("Tutorial 10: Quantization", s.4: biases "Optional ... or None").
 *    The results are then bit for bit those of an all-zero bias array, and
 *    no bias bytes are read.  The quantizers always write biases.
 *  - group_size in {32, 64, 128}; bits in [2, 8]; K % group_size == 0
 *    (a layer whose width is not a multiple of the group size is left
 *    unquantized: "Quantizing a Model for MLX", "What MLX quantization
 *    stores"); N, K >= 1.  No defaults: both are always explicit.
 *  - The entry points are stateless and re-entrant; calls on different
 *    streams may run concurrently.
 */
#ifndef AQ_H_
#define AQ_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum aq_status {
  AQ_OK = 0,
  AQ_ERR_INVALID_ARG = -1, /* shape, size, null pointer, dtype or enum out of range */
  AQ_ERR_UNSUPPORTED = -2, /* valid request this build does not implement */
  AQ_ERR_ALIGNMENT = -3,   /* a pointer is not 16-byte aligned */
  AQ_ERR_HIP = -4,         /* the HIP runtime reported an error at launch */
  AQ_ERR_RANGE = -5,       /* reserved: value out of the representable range */
  AQ_ERR_INDEX = -6,       /* reserved: index out of range */
  /* range markers, never returned: they make every 32-bit integer a value of
   * the type, so any int a caller passes is well defined in C and C++ */
  AQ_STATUS_RANGE_MIN_ = -0x7FFFFFFF - 1,
  AQ_STATUS_RANGE_MAX_ = 0x7FFFFFFF
} aq_status;

typedef enum aq_dtype {
  AQ_F32 = 0,  /* IEEE binary32 */
  AQ_F16 = 1,  /* IEEE binary16 */
  AQ_BF16 = 2, /* bfloat16 */
  /* range markers, never valid arguments (AQ_ERR_INVALID_ARG): every 32-bit
   * integer is a value of the type, so validating one is well defined */
  AQ_DTYPE_RANGE_MIN_ = -0x7FFFFFFF - 1,
  AQ_DTYPE_RANGE_MAX_ = 0x7FFFFFFF
} aq_dtype;

/* ---- host helpers (no GPU involved) ------------------------------------ */

/* Human-readable name of a status code (static string, never NULL). */
const char *aq_status_string(aq_status status);

/* Library version string. */
const char *aq_version(void);

/* uint32 words per packed row: K*bits/32 (one least-significant-bit-first
 * bitstream per row, several codes to a 32-bit word: "Quantizing a Model for
 * MLX", "What MLX quantization stores"; "Tutorial 10: Quantization", s.3 and
 * s.4, packed weight shape [out, in*bits/32]).  -1 if K*bits is not a
 * multiple of 32 or an argument is out of range. */
int64_t aq_codes_words(int64_t K, int bits);

/* Bytes of one quantized matrix: N*K*bits/8 codes + 2 bytes of scale and
 * 2 bytes of bias per group ("Quantizing a Model for MLX", "What MLX
 * quantization stores": 4.5 bits per weight at G=64, bits=4).  -1 on bad
 * arguments. */
int64_t aq_qweight_bytes(int64_t N, int64_t K, int group_size, int bits);

/* ---- device operations -------------------------------------------------- */

/* Quantize W [N, K] (device; w_dtype AQ_F32, AQ_F16 or AQ_BF16, the latter
 * two widened exactly to binary32) into codes/scales/biases (device,
 * layouts above).  Per group, following "mlx-gptq", "How it works" (the
 * grid spans the group's min-max range) and "Quantizing a Model for MLX"
 * (scale and offset chosen per group):
 *   b = the group minimum rounded down to fp16 (so b <= every member);
 *   s = the smallest fp16 >= 0 with b + (2^bits-1)*s >= the group maximum;
 *   q = the index of the grid point b + q*s nearest to w, ties to even q
 *       (q = 0 when s = 0);
 * hence |w - (q*s + b)| <= s/2 for every weight.
 * Precondition (not checked on the device): weights finite, group minima
 * >= -65504 and the needed scale <= 65504; otherwise the outputs for that
 * group are unspecified. */
aq_status aq_quantize(const void *w, aq_dtype w_dtype, int64_t N, int64_t K, int group_size,
                      int bits, uint32_t *codes, uint16_t *scales, uint16_t *biases,
                      void *stream);

/* Range-search quantize ("mlx-gptq", "How it works", the --mse option: a
 * group may be quantized over a range narrower than its min-max span,
 * trading error on its outermost members for a finer step on the others).
 * Same arguments, outputs, format and preconditions as aq_quantize, plus
 * steps in [1, 50]: candidate i < steps moves both ends of the group's range
 * inwards by d = (max - min) * (i / 200) (binary64, left to right), i.e.
 * keeps the centred fraction (100 - i)/100 of the width, so every candidate
 * lies inside [min, max]; it takes bias, scale and codes from that range by
 * the rules of aq_quantize (members outside it clip to code 0 or 2^bits-1)
 * and scores sum (w - (q*s + b))^2 in binary64; the least score wins, an
 * equal score keeping the wider candidate.  steps = 1 gives
 * exactly aq_quantize.  (The pages fix neither the grid nor the measure;
 * these are this library's choices.)  Scores that differ only in the last
 * bits of their binary64 sums may pick either candidate.
 * AQ_ERR_INVALID_ARG for steps outside [1, 50]. */
aq_status aq_quantize_mse(const void *w, aq_dtype w_dtype, int64_t N, int64_t K, int group_size,
                          int bits, int steps, uint32_t *codes, uint16_t *scales, uint16_t *biases,
                          void *stream);

/* Quantize with integer zero points ("mlx-gptq", "On NVIDIA: the same recipe
 * in AWQ format", --zero-point int: every group's offset is a whole number of
 * steps, so the result converts without loss to a layout that stores an
 * integer zero point z per group and decodes (q - z)*s).  Same arguments,
 * outputs, format and preconditions as aq_quantize, plus zeros: device uint8
 * [N, K/G] receiving each group's z, or NULL.  Per group:
 *   z is an integer in [0, 2^bits - 1], so the grid -z*s + q*s contains 0;
 *   s = the smallest fp16 >= 0 for which some such z has -z*s <= the group
 *       minimum, (2^bits-1-z)*s >= the group maximum and -z*s exactly an
 *       fp16 value; z = the smallest such integer for that s;
 *   b = -z*s (exact; +0 when z = 0), q as in aq_quantize;
 * hence q*s + b = (q - z)*s exactly and |w - (q*s + b)| <= s/2.  The output
 * is an ordinary (codes, scales, biases) container: every consumer below
 * takes it unchanged. */
aq_status aq_quantize_zp(const void *w, aq_dtype w_dtype, int64_t N, int64_t K, int group_size,
                         int bits, uint32_t *codes, uint16_t *scales, uint16_t *biases,
                         uint8_t *zeros, void *stream);

/* Dequantize ("Tutorial 10: Quantization", s.3 and s.7): out[n, k] =
 * q*s + b evaluated in binary32 (q*s is exact, the add rounds to nearest
 * even), then rounded to nearest even into out_dtype (AQ_F32, AQ_F16 or
 * AQ_BF16).  out is device memory [N, K]. */
aq_status aq_dequantize(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases,
                        int64_t N, int64_t K, int group_size, int bits, void *out,
                        aq_dtype out_dtype, void *stream);

/* Quantized embedding lookup ("Tutorial 10: Quantization", s.6 "Quantized
 * Embeddings"): the packed rows, scales and biases of the token ids are
 * selected and dequantized exactly as aq_dequantize does:
 *   out[t, :] = dequantize(row ids[t] of the V x K table), 0 <= t < T.
 * codes/scales/biases: the table (device, layouts above, V rows).  ids:
 * device int32 [T], T >= 1.  out: device [T, K] in out_dtype (AQ_F32, AQ_F16
 * or AQ_BF16).  An id outside [0, V) reads nothing and gives a zero row. */
aq_status aq_embedding(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases,
                       int64_t V, int64_t K, int group_size, int bits, const int32_t *ids,
                       int64_t T, void *out, aq_dtype out_dtype, void *stream);

/* Quantized matrix-vector product for decode, y = x @ W^T with W given in
 * packed form and dequantized in registers on every use ("Quantization",
 * metalworking, QMV bullet; "Tutorial 10", s.5 Approach 2 with
 * transpose=True).  x: device [M, K] in x_dtype (AQ_F16 or AQ_BF16), 1 <= M
 * <= 8.  y: device [M, N] in x_dtype.  Accumulation in binary32; y is
 * rounded to nearest even.  The kernel variant is chosen per shape (M, K,
 * bits, dtype). */
aq_status aq_qmv(const void *x, aq_dtype x_dtype, int64_t M, const uint32_t *codes,
                 const uint16_t *scales, const uint16_t *biases, int64_t N, int64_t K,
                 int group_size, int bits, void *y, void *stream);

/* Which kernel aq_qmv (and aq_quantized_matmul for M <= 8) launches for this
 * shape, as text: the kernel name and its compile-time shape (for reports and
 * profiles), written to buf (host memory, len bytes, always NUL-terminated).
 * Returns the length of the full text as snprintf does, or -1 for arguments
 * aq_qmv would reject.  For 2 <= M <= 8 it may query the current device's
 * compute-unit count. */
int aq_qmv_describe(int64_t M, int64_t N, int64_t K, int group_size, int bits, aq_dtype x_dtype,
                    char *buf, int len);

/* Quantized matrix-matrix product for prefill ("Quantization", metalworking,
 * QMM bullet): same operation and layouts as aq_qmv for any M >= 1.  Weight
 * tiles are dequantized to x_dtype (rounded to nearest even, the value
 * aq_dequantize returns for that type) and multiplied on the matrix cores
 * with binary32 accumulation.  AQ_ERR_UNSUPPORTED for K > 4194303 (a
 * 256-row tile of x is addressed with 32-bit byte offsets) or M > 8388352
 * (the launch grid holds at most 65535 row tiles of 128). */
aq_status aq_qmm(const void *x, aq_dtype x_dtype, int64_t M, const uint32_t *codes,
                 const uint16_t *scales, const uint16_t *biases, int64_t N, int64_t K,
                 int group_size, int bits, void *y, void *stream);

/* Shape dispatch for y = x @ W^T ("Quantization", metalworking: host-side
 * dispatch picks the kernel per shape): M <= 8 goes to the matrix-vector
 * kernels of aq_qmv.  For 9 <= M <= 256 with 4-bit or 8-bit codes, while
 * aq_qmm's 256 x 256 output tiles would be mostly empty or too few for the
 * chip (M <= 64, or fewer tiles than an eighth of the compute units), the
 * few-row matrix-core kernel of aq_qmv runs on slices of 16 or 32 rows of x
 * (binary32 accumulation, the same bound).  Otherwise aq_qmm.  Same arguments as aq_qmv
 * with any M >= 1; may query the current device's compute-unit count. */
aq_status aq_quantized_matmul(const void *x, aq_dtype x_dtype, int64_t M, const uint32_t *codes,
                              const uint16_t *scales, const uint16_t *biases, int64_t N,
                              int64_t K, int group_size, int bits, void *y, void *stream);

/* Gather variant for mixture-of-experts layers ("Quantization", metalworking:
 * gather variants for MoE experts): for every token t and slot j,
 *   y[t, j, :] = x[t, :] @ W_e^T   with e = ids[t, j].
 * x: device [T, K] (AQ_F16 or AQ_BF16); codes: device [E, N, K*bits/32];
 * scales, biases: device [E, N, K/G]; ids: device int32 [T, topk];
 * y: device [T, topk, N] in x_dtype.  No routing weights are applied.  The
 * routing is resolved on the device: each expert's weights are read once
 * for every batch of up to 16 (token, slot) pairs routed to it (8 on the
 * vector path for 2-, 3-, 5-, 6- and 7-bit codes), and experts no token
 * chose are never read.  An id outside [0, E) is not read from; its output
 * row is set to zero. */
aq_status aq_gather_qmv(const void *x, aq_dtype x_dtype, int64_t T, const uint32_t *codes,
                        const uint16_t *scales, const uint16_t *biases, int64_t E, int64_t N,
                        int64_t K, const int32_t *ids, int topk, int group_size, int bits,
                        void *y, void *stream);

/* The gather product at prefill size, on the matrix cores (the QMM engine
 * of aq_qmm): same operation, arguments and layouts as aq_gather_qmv, for
 * many tokens per expert.  The routing is resolved on the device: one
 * workgroup per (256 columns, expert) lists the (token, slot) pairs routed
 * to its expert and runs 256-row tiles of them, so each expert's weights are
 * read once per 256 routed rows.  Weight tiles are rounded to x_dtype as in
 * aq_qmm.  AQ_ERR_UNSUPPORTED if T*K*2 > 2^31-1 (x addressed with 32-bit
 * byte offsets), E > 65535 or T*topk > 2^31-1. */
aq_status aq_gather_qmm(const void *x, aq_dtype x_dtype, int64_t T, const uint32_t *codes,
                        const uint16_t *scales, const uint16_t *biases, int64_t E, int64_t N,
                        int64_t K, const int32_t *ids, int topk, int group_size, int bits,
                        void *y, void *stream);

/* Shape dispatch for the gather product: aq_gather_qmm when the routed rows
 * average at least 32 per expert (T*topk >= 32*E), else aq_gather_qmv. */
aq_status aq_gather_quantized_matmul(const void *x, aq_dtype x_dtype, int64_t T,
                                     const uint32_t *codes, const uint16_t *scales,
                                     const uint16_t *biases, int64_t E, int64_t N, int64_t K,
                                     const int32_t *ids, int topk, int group_size, int bits,
                                     void *y, void *stream);

/* ---- block-scaled float modes ------------------------------------------- */

/* The block-scaled float modes ("Quantization", metalworking MLX notes, the
 * paragraph on the newer modes; "Quantizing a Model for MLX", "Modes, bits
 * and mixed recipes": mxfp4, nvfp4 and mxfp8 with groups of 32, 16 and 32
 * weights and 4, 4 and 8-bit codes, a per-group scale in place of a scale
 * and a bias; ExecuTorch "Quantization": nvfp4 is NVIDIA's FP4 weight-only
 * format at group size 16).  The pages give no bit layout; this library
 * takes the definitions of those names (microscaling for mxfp4 and mxfp8,
 * NVFP4 for nvfp4):
 *
 *   E2M1 code (4 bits): bit 3 sign, bits 2..1 exponent e (bias 1), bit 0
 *     mantissa m; (1 + m/2)*2^(e-1), or m/2 for e = 0 (magnitudes 0, 0.5,
 *     1, 1.5, 2, 3, 4, 6).
 *   E4M3 code (8 bits): bit 7 sign, bits 6..3 exponent e (bias 7), bits
 *     2..0 mantissa m; (1 + m/8)*2^(e-7), or (m/8)*2^-6 for e = 0;
 *     magnitude pattern 0x7F is NaN; largest finite magnitude 448.
 *
 *   mode      group  codes                         scales
 *   AQ_MXFP4   32    uint32 [N, K/8]  E2M1         uint8 [N, K/32]  X + 127 for 2^X
 *   AQ_NVFP4   16    uint32 [N, K/8]  E2M1         uint8 [N, K/16]  E4M3 value s
 *   AQ_MXFP8   32    uint32 [N, K/4]  E4M3         uint8 [N, K/32]  X + 127 for 2^X
 *
 * Codes are packed least significant first into the row's words (code k of
 * a row at bits [b*k, b*k + b) of its bitstream, as above).  A weight's
 * value is code * 2^X (mx modes) or code * s * 2^T (nvfp4, where the whole
 * matrix shares the tensor scale 2^T, the argument tensor_exp = T in
 * [-100, 100]; 0 means no tensor scale; for the mx modes tensor_exp must
 * be 0).  N >= 1, K >= the group size and a multiple of it.  The
 * conventions above (device pointers 16-byte aligned, caller-owned buffers,
 * host-side checks, asynchronous on `stream`) hold. */
typedef enum aq_fp_mode {
  AQ_MXFP4 = 0,
  AQ_NVFP4 = 1,
  AQ_MXFP8 = 2,
  /* range markers, never valid arguments (AQ_ERR_INVALID_ARG) */
  AQ_FP_MODE_RANGE_MIN_ = -0x7FFFFFFF - 1,
  AQ_FP_MODE_RANGE_MAX_ = 0x7FFFFFFF
} aq_fp_mode;

/* Quantize W [N, K] (device; AQ_F32, AQ_F16 or AQ_BF16, widened exactly to
 * binary32) into codes and scales (device) of the given mode.  Per group:
 *   mxfp4, mxfp8: X = floor(log2 max|w|) - E, E the exponent of the
 *     largest code value (2 for E2M1's 6, 8 for E4M3's 448), clamped to
 *     [-127, 127]; -127 for a group of zeros.  The step is 2^X.
 *   nvfp4: s = the E4M3 value nearest to max|w| / (6 * 2^T), ties to the
 *     even code, 448 above it.  The step is s * 2^T.
 *   each weight's code is its own sign bit (so -0 keeps it) with the
 *   magnitude code nearest to |w| / step, ties to the even code, the
 *   largest finite magnitude above it; magnitude 0 when s = 0.
 * A tensor exponent that puts the largest group scale near the top of
 * E4M3's range is T = ceil(log2(max|W| / 2688)) (2688 = 6 * 448).
 * Precondition (not checked on the device): weights finite; otherwise the
 * outputs for that group are unspecified. */
aq_status aq_quantize_fp(const void *w, aq_dtype w_dtype, int64_t N, int64_t K, aq_fp_mode mode,
                         int tensor_exp, uint32_t *codes, uint8_t *scales, void *stream);

/* Dequantize: out[n, k] = the exact value code * step (NaN for NaN code or
 * scale patterns; steps from any scale byte, not only those the quantizer
 * writes), rounded to nearest even into out_dtype (AQ_F32, AQ_F16 or
 * AQ_BF16), +-inf past its range.  out is device memory [N, K]. */
aq_status aq_dequantize_fp(const uint32_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                           aq_fp_mode mode, int tensor_exp, void *out, aq_dtype out_dtype,
                           void *stream);

/* Decode matrix-vector product ("Quantization", metalworking, QMV bullet:
 * the weights are dequantized in registers on every use): y[n] =
 * sum_k x[k] * w^[n, k] for one row x.  x: device [K] in x_dtype (AQ_F16 or
 * AQ_BF16); y: device [N] in x_dtype.  Products are summed in binary32 per
 * group and scaled once per group; y is rounded to nearest even.
 * AQ_ERR_UNSUPPORTED for K not a multiple of 32 (nvfp4) or K > 49152 (x is
 * held on chip). */
aq_status aq_qmv_fp(const void *x, aq_dtype x_dtype, const uint32_t *codes,
                    const uint8_t *scales, int64_t N, int64_t K, aq_fp_mode mode, int tensor_exp,
                    void *y, void *stream);

/* The product for M rows of x ("Quantization", metalworking, QMV bullet and
 * its dispatch section on several rows of x per pass over W, as in
 * speculative decoding): y[m, n] = sum_k x[m, k] * w^[n, k].  x: device
 * [M, K] row-major in x_dtype (AQ_F16 or AQ_BF16); y: device [M, N] in
 * x_dtype.  M = 1 is aq_qmv_fp.  M >= 2 runs on the matrix cores in slices
 * of 16 rows of x, each slice one pass over W: per 32-code chunk the exact
 * code values times x, summed in binary32 per group and scaled once per
 * group (nvfp4: 2^T applied to the sums); y is rounded to nearest even.
 * Arguments as aq_qmv_fp (the same K limits; AQ_ERR_INVALID_ARG for
 * M < 1, AQ_ERR_UNSUPPORTED past M = 16 * 65535 or past 2^31 - 16 scale
 * bytes). */
aq_status aq_matmul_fp(const void *x, aq_dtype x_dtype, int64_t M, const uint32_t *codes,
                       const uint8_t *scales, int64_t N, int64_t K, aq_fp_mode mode,
                       int tensor_exp, void *y, void *stream);

/* Mixture-of-experts gather of the block-scaled product ("Quantization",
 * metalworking: gather variants of the kernels for MoE experts):
 * y[t, j, :] = x[t] @ W_{ids[t, j]}^T for every token t < T and slot
 * j < topk, one output row per (token, slot), no routing weights.  x: device
 * [T, K] in x_dtype (AQ_F16 or AQ_BF16); codes and scales: device, E
 * experts' arrays of aq_quantize_fp back to back ([E, N, ...]); ids: device
 * int32 [T, topk]; y: device [T, topk, N] in x_dtype.  An id outside
 * [0, E) gives a zero row and reads no weights; experts no pair chose are
 * never read.  Each expert's rows are read once per batch of 16 (token,
 * slot) pairs routed to it, on the matrix cores as in aq_matmul_fp (the
 * same sums, the same rounding).  AQ_ERR_INVALID_ARG for T, E or topk
 * below 1 or a bad mode, tensor exponent or pointer; AQ_ERR_UNSUPPORTED for
 * K not a multiple of 32 or past 49152, E > 65535, or x or the scale array
 * past 2^31 bytes. */
aq_status aq_gather_matmul_fp(const void *x, aq_dtype x_dtype, int64_t T, const uint32_t *codes,
                              const uint8_t *scales, int64_t E, int64_t N, int64_t K,
                              const int32_t *ids, int topk, aq_fp_mode mode, int tensor_exp,
                              void *y, void *stream);

/* Which kernel aq_qmv_fp launches for this shape and mode, as text (as
 * aq_qmv_describe does); -1 for arguments aq_qmv_fp would reject. */
int aq_qmv_fp_describe(int64_t N, int64_t K, aq_fp_mode mode, aq_dtype x_dtype, char *buf,
                       int len);

/* ---- key-value cache and attention ---------------------------------------
 *
 * A paged cache of attention keys and values in the format above, one packed
 * row per token and head: the head_dim values of a token's key (or value) in
 * one head are cut into groups of group_size along head_dim, each group
 * stored as `bits`-bit codes, one fp16 scale and one fp16 bias, w = q*s + b.
 * Page p holds page_size consecutive tokens of one sequence, all heads:
 *
 *   codes   uint32 [num_pages, kv_heads, page_size, head_dim*bits/32]
 *   scales  uint16 [num_pages, kv_heads, page_size, head_dim/group_size]
 *   biases  uint16, the same shape
 *
 * for K and for V.  With bits = 16 the code arrays hold the values themselves,
 * [num_pages, kv_heads, page_size, head_dim] in `dtype` (AQ_F16 or AQ_BF16);
 * scales and biases are then not looked at (may be NULL) and neither is
 * group_size.  A token's slot is page * page_size + its place in the page.
 *
 * Supported: bits 4, 8, 16; head_dim 64, 128, 256; group_size 32, 64, 128
 * dividing head_dim; page_size a multiple of 16; kv_heads * page_size *
 * head_dim <= 2^28 (a page is addressed with 32-bit offsets); the cache
 * itself may be of any size.  AQ_ERR_INVALID_ARG / AQ_ERR_UNSUPPORTED
 * otherwise.  All arrays are device memory, 16-byte aligned. */
typedef struct aq_kv_cache {
  void *k_codes;
  uint16_t *k_scales;
  uint16_t *k_biases;
  void *v_codes;
  uint16_t *v_scales;
  uint16_t *v_biases;
  int64_t num_pages;
  int32_t page_size;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t group_size;
  int32_t bits;
  int32_t dtype; /* aq_dtype of the pages when bits = 16, not looked at otherwise */
} aq_kv_cache;

/* Quantize keys and values into the cache as they are written: token t's rows
 * k[t, h, :] and v[t, h, :] go to slots[t], each group by the rule of
 * aq_quantize (the codes, scales and biases are those aq_quantize gives for
 * the row).  k, v: device, x_dtype AQ_F16 or AQ_BF16, heads and head_dim
 * contiguous, tokens k_stride and v_stride elements apart (multiples of 8, at
 * least kv_heads * head_dim), so both may be parts of one projection's rows.
 * slots: device int64 [T]; a slot outside [0, num_pages * page_size) writes
 * nothing; the slots of one call are to differ (equal ones leave a mixture of
 * their tokens' rows).  Values are clamped to fp16's finite range first; a group that holds
 * a NaN gets scale 0, bias NaN and codes 0, so all of it reads back as NaN.
 * bits = 16: x_dtype must be the cache's dtype, rows are copied as they are.
 * T = 0 does nothing.  Scales and biases are required unless bits = 16. */
aq_status aq_kv_append(const void *k, const void *v, aq_dtype x_dtype, int64_t T, int64_t k_stride,
                       int64_t v_stride, const int64_t *slots, const aq_kv_cache *cache,
                       void *stream);

/* Read rows of the cache back: k[t, h, :] and v[t, h, :] = the rows of
 * slots[t], q*s + b as aq_dequantize rounds it into out_dtype (AQ_F32, AQ_F16
 * or AQ_BF16).  k, v: device [T, kv_heads, head_dim].  A slot outside the
 * cache reads nothing and gives zero rows.  NULL bias arrays: every bias +0.
 * T = 0 does nothing. */
aq_status aq_kv_read(const int64_t *slots, int64_t T, const aq_kv_cache *cache, void *k, void *v,
                     aq_dtype out_dtype, void *stream);

/* Attention of the newest tokens of each sequence over the paged cache.  For
 * sequence b of B, its last L (1..8) tokens, query head h and j = h / (q_heads
 * / kv_heads):
 *
 *   out[b, i, h, :] = sum_t p_t v[t, j, :],   p = softmax_t(scale * q[b, i, h, :] . k[t, j, :])
 *
 * over the cached tokens t <= len - L + i, len = lengths[b] clamped to
 * [0, max_pages * page_size], which counts the L tokens themselves (append
 * them first).  Token t of the sequence is at place t % page_size of page
 * page_table[b, t / page_size]; the tokens of a page id outside
 * [0, num_pages) are left out, and nothing past len is looked at, whatever
 * it holds.  A row that sees no token is zero.
 *
 * q: device, x_dtype AQ_F16 or AQ_BF16 (bits = 16: the cache's dtype), rows
 * [q_heads, head_dim] contiguous, token b*L + i at q + (b*L + i) * q_stride
 * elements (a multiple of 8, at least q_heads * head_dim).  out: device [B, L,
 * q_heads, head_dim] in x_dtype, no part of q's memory.  page_table: device
 * int32 [B, max_pages].  lengths: device int32 [B].  q_heads a multiple of
 * kv_heads.  Scores and softmax statistics are held in binary32.  NULL bias
 * arrays: every bias +0.  Scales may be any finite fp16; one that is infinite
 * counts as NaN, and so may an infinite bias (aq_kv_append writes neither).
 * A value of a 16-bit page that is infinite or NaN is what the formula makes
 * of it in the rows that see its token, and nothing to the others.
 *
 * workspace: device memory of aq_paged_attention_workspace bytes, 16-byte
 * aligned, zeroed once before its first use; every call leaves it fit for the
 * next one, of any shape it is large enough for.  Calls that may run at the
 * same time need workspaces of their own.  The launches do not depend on the
 * lengths, so a captured graph follows them as they grow; results are the
 * same bits every time.
 * AQ_ERR_INVALID_ARG when workspace_bytes is too small, B < 1, L outside
 * 1..8; AQ_ERR_UNSUPPORTED for max_pages * page_size > 2^31 - 256 or B * L *
 * q_heads >= 2^24. */
aq_status aq_paged_attention(const void *q, aq_dtype x_dtype, int64_t B, int L, int q_heads,
                             int64_t q_stride, const aq_kv_cache *cache, const int32_t *page_table,
                             int64_t max_pages, const int32_t *lengths, float scale, void *out,
                             void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace aq_paged_attention needs for this shape (at most 64 MiB);
 * -1 on bad arguments.  May query the current device's compute-unit count. */
int64_t aq_paged_attention_workspace(int64_t B, int L, int q_heads, int kv_heads, int head_dim);

/* ---- attention with capped, biased and masked scores ----------------------
 *
 * How scores become weights, for the calls below.  The score of a row (one
 * query head of one token at position `pos` of its sequence) and the token at
 * position t is, in this order,
 *
 *   s = scale * q . k[t]
 *   s = softcap * tanh(s / softcap)     unless softcap is 0
 *   s = s - slopes[head] * |pos - t|    unless slopes is NULL
 *
 * and the row sees the token t when all of these hold:
 *
 *   t < the sequence's length
 *   t <= pos, or t < prefix[sequence]   (prefix NULL: t <= pos)
 *   pos - t < window                    (window 0: any)
 *   t >= first[...]                     (first NULL: any; the document that
 *                                        the row belongs to begins there)
 *
 * What a row does not see has no part in it, whatever it holds (infinite and
 * NaN values too).  A row that sees no token is zero.  lse, where it is given,
 * gets log(sum_t exp(s_t)) of each row, -inf for a row that sees no token.  A
 * row that sees a score of +inf or NaN is NaN, and so is its lse.
 *
 * softcap: 0, or from 1e-30 to 1e30.  window >= 0.  slopes: device float
 * [q_heads].  All pointers are device memory, 16-byte aligned. */
typedef struct aq_attention_scores {
  float softcap;
  int32_t window;
  const float *slopes;
  const int32_t *first;
  const int32_t *prefix;
  float *lse;
} aq_attention_scores;

/* aq_paged_attention with such scores: the newest L (1..8) tokens of each
 * sequence over the paged cache, token i of sequence b at position
 * lengths[b] - L + i.  first: device int32 [B], one per sequence; prefix: NULL
 * (AQ_ERR_INVALID_ARG otherwise: new tokens come after any prefix); lse: float
 * [B, L, q_heads] or NULL.  Tokens ahead of what any of a sequence's rows sees
 * are not read.  Everything else, the workspace too, as in aq_paged_attention;
 * with all of `scores` zero the results are its own. */
aq_status aq_paged_attention_masked(const void *q, aq_dtype x_dtype, int64_t B, int L, int q_heads,
                                    int64_t q_stride, const aq_kv_cache *cache,
                                    const int32_t *page_table, int64_t max_pages,
                                    const int32_t *lengths, float scale,
                                    const aq_attention_scores *scores, void *out, void *workspace,
                                    int64_t workspace_bytes, void *stream);

/* Attention of whole prompts, or of any number of new tokens, over keys and
 * values that are rows of 16 bits (a projection's, or a cache's read back):
 * sequence b's queries are the rows q_starts[b] .. q_starts[b + 1] - 1 of q,
 * its keys and values the rows k_starts[b] .. k_starts[b + 1] - 1 of k and v,
 * the queries' own among them as the last: query i of n is at position
 * (keys - n) + i.  first: device int32 [Tq], one per row of q; prefix: device
 * int32 [B]; lse: float [Tq, q_heads] or NULL.
 *
 * q [Tq, q_heads, head_dim], k and v [Tk, kv_heads, head_dim]: device, x_dtype
 * AQ_F16 or AQ_BF16, heads and head_dim contiguous, tokens the strides apart
 * in elements (multiples of 8, at least heads * head_dim).  q_starts, k_starts:
 * device int32 [B + 1], ascending, from 0 to at most Tq and Tk (they are
 * clamped to that); rows of q behind the last sequence are left as they are in
 * out and lse.  out: device [Tq, q_heads, head_dim], no part of q, k or v.
 * q_heads a multiple of kv_heads; head_dim 64, 128 or 256.  A weight is rounded
 * to x_dtype once before it meets the values; scores, statistics and sums are
 * binary32.  Results are the same bits every time.
 *
 * workspace: device memory of aq_prompt_attention_workspace bytes, 16-byte
 * aligned, no initial content needed; calls that may run at the same time need
 * workspaces of their own.  Tq = 0 does nothing.  AQ_ERR_UNSUPPORTED for Tq *
 * q_heads, Tk * kv_heads or B * kv_heads >= 2^24, and for tokens of k or v more
 * than 2^23 elements apart. */
aq_status aq_prompt_attention(const void *q, aq_dtype x_dtype, int64_t Tq, int q_heads,
                              int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, int64_t Tk, int kv_heads, int head_dim, int64_t B,
                              const int32_t *q_starts, const int32_t *k_starts, float scale,
                              const aq_attention_scores *scores, void *out, void *workspace,
                              int64_t workspace_bytes, void *stream);

/* Bytes of workspace aq_prompt_attention needs for this shape (at most 64 MiB);
 * -1 on bad arguments.  May query the current device's compute-unit count. */
int64_t aq_prompt_attention_workspace(int64_t Tq, int64_t Tk, int64_t B, int q_heads, int kv_heads,
                                      int head_dim);

/* ---- rotary positions ------------------------------------------------------
 *
 * The first `rotary` values of a head are rotary / 2 pairs; the pair i of a
 * token at position p is turned by the angle p * freqs[i]:
 *
 *   (x, y) -> (x c - y s, y c + x s),  c = cos(angle) * factor, s = sin(angle) * factor
 *
 * interleaved 0: pair i is the values i and rotary / 2 + i; 1: the values 2 i
 * and 2 i + 1.  The values from `rotary` on stay as they are.  The angle, its
 * sine and cosine and their product with the factor are binary64 and rounded
 * to binary32 once; each product and sum of the turn is rounded to binary32,
 * the result to the 16-bit type.  Any int32 position, far and negative ones
 * too; frequencies up to 2^20.  rotary: a multiple of 16, from 16 to head_dim; head_dim 64, 128 or 256
 * (AQ_ERR_UNSUPPORTED otherwise); factor finite. */
typedef struct aq_rotation {
  const int32_t *positions; /* device [T] */
  const float *freqs;       /* device [rotary / 2] */
  int32_t rotary;
  int32_t interleaved;
  double factor;
} aq_rotation;

/* Turn the rows of q [T, q_heads, head_dim] into q_out and those of k [T,
 * kv_heads, head_dim] into k_out.  Rows are 16-bit (AQ_F16 or AQ_BF16), heads
 * and head_dim contiguous, tokens the strides apart in elements (multiples of
 * 8, at least heads * head_dim).  q_out may be q itself (with its stride) and
 * k_out k; other overlaps are the caller's mistake.  q_heads = 0 or kv_heads =
 * 0 leaves that side out (its pointers may be NULL).  T = 0 does nothing;
 * AQ_ERR_UNSUPPORTED for T > 2^28 - 16. */
aq_status aq_rope(const void *q, int64_t q_stride, int q_heads, const void *k, int64_t k_stride,
                  int kv_heads, aq_dtype x_dtype, int64_t T, int head_dim,
                  const aq_rotation *rotation, void *q_out, int64_t q_out_stride, void *k_out,
                  int64_t k_out_stride, void *stream);

/* aq_rope and aq_kv_append in one launch: q turned into q_out, k turned,
 * rounded to x_dtype and written with v into the cache at slots.  The cache
 * gets bit for bit what aq_rope and then aq_kv_append would write.  k_out, if
 * not NULL, gets the turned keys as well (for attention over the rows
 * themselves).  q_heads = 0 leaves the queries out.  Arguments as in those. */
aq_status aq_rope_append(const void *q, int64_t q_stride, int q_heads, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, aq_dtype x_dtype,
                         int64_t T, const aq_rotation *rotation, const int64_t *slots,
                         const aq_kv_cache *cache, void *q_out, int64_t q_out_stride, void *k_out,
                         int64_t k_out_stride, void *stream);

/* How frequencies are changed for contexts longer than a model was trained on
 * (s = stretch, ctx = the trained context, f = base^(-2 i / rotary)):
 *   AQ_ROPE_PLAIN      f
 *   AQ_ROPE_LINEAR     f / s (positions interpolated)
 *   AQ_ROPE_BASE       f with base * s^(rotary / (rotary - 2))
 *   AQ_ROPE_BY_INDEX   f / s for pairs that turn less than `low` times in ctx,
 *                      f for those that turn more than `high` times, between
 *                      them a blend that is linear in the pair's index: with
 *                      d(r) = rotary ln(ctx / (2 pi r)) / (2 ln base), a =
 *                      max(floor d(high), 0), b = min(ceil d(low), rotary - 1),
 *                      the part g = clamp((i - a) / max(b - a, 0.001), 0, 1) of
 *                      f / s and 1 - g of f; factor 0.1 ln s + 1 for s > 1
 *   AQ_ROPE_BY_TURNS   the same, linear in the turns r = ctx f / (2 pi): g =
 *                      1 - clamp((r - low) / (high - low), 0, 1); factor 1 */
typedef enum aq_rope_stretch {
  AQ_ROPE_PLAIN = 0,
  AQ_ROPE_LINEAR = 1,
  AQ_ROPE_BASE = 2,
  AQ_ROPE_BY_INDEX = 3,
  AQ_ROPE_BY_TURNS = 4
} aq_rope_stretch;

/* Fills freqs, HOST memory of rotary / 2 floats, and *factor (may be NULL) by
 * that table, computed in binary64.  rotary even and >= 4, base > 1, stretch
 * >= 1 (not looked at for AQ_ROPE_PLAIN); ctx >= 1 and 0 < low < high for the
 * last two, AQ_ERR_INVALID_ARG otherwise. */
aq_status aq_rope_frequencies(int rotary, double base, aq_rope_stretch kind, double stretch,
                              double ctx, double low, double high, float *freqs, float *factor);

/* ---- keeping a cache within a budget ---------------------------------------
 *
 * What each cached token gathers of the attention of new tokens, added to what
 * it gathered before:
 *
 *   weights[b, t] += sum over rows i, h of exp(s - lse[b, i, h])
 *
 * for the tokens t < min(length, weights_stride) of sequence b, s and what a row sees as
 * in aq_paged_attention_masked (softcap, window, slopes, first; prefix NULL).
 * scores->lse, float [B, L, q_heads], is what that call gave for the same
 * queries, and is required; a row whose lse is -inf adds nothing.  weights:
 * device float, sequence b's at weights + b * weights_stride, weights_stride a
 * multiple of 4.  Only the keys of the cache are read.  The sums are binary32,
 * in an order that does not depend on timing.  AQ_ERR_UNSUPPORTED for B *
 * max_pages * page_size / 128 >= 2^31, beside what aq_paged_attention refuses. */
aq_status aq_kv_weigh(const void *q, aq_dtype x_dtype, int64_t B, int L, int q_heads,
                      int64_t q_stride, const aq_kv_cache *cache, const int32_t *page_table,
                      int64_t max_pages, const int32_t *lengths, float scale,
                      const aq_attention_scores *scores, float *weights, int64_t weights_stride,
                      void *stream);

/* Evict what gathered least.  Sequence b (length n = lengths[b], clamped to
 * [0, min(max_pages * page_size, weights_stride)]) keeps all its tokens if n <=
 * keep; otherwise the first `sinks`, the last `recent` and, of those between,
 * the keep - sinks - recent with the largest weights: the lowest positions of
 * equal ones, NaN below everything.  The kept tokens, in their order, become
 * the tokens 0, 1, ... of the pages of new_table [B, new_max_pages]; their rows
 * are copied there as they are.  Outputs: kept int32 [B, keep], the positions
 * they had, -1 behind the last; new_weights float [B, keep], their weights, 0
 * behind the last; new_lengths int32 [B].
 *
 * A kept token is from then on the token of its new place: `first`, windows and
 * slopes of aq_paged_attention_masked and aq_kv_weigh count places, so distances
 * shrink by what was evicted between, and a caller's `first` has to be moved by
 * `kept`.  Rotary positions are in the keys and stay.  A model whose slopes or
 * windows are to mean the conversation's distances is not served by eviction.
 * new_weights has rows of `keep`; aq_kv_weigh goes on in rows that have room for
 * the tokens to come (weights past a row's end are not gathered, and tokens past
 * it are not kept by the next eviction).
 *
 * The pages of new_table are to be other pages than those of page_table, since
 * a page may be shared by sequences and tokens move at once; the caller frees
 * the old ones afterwards.  Rows of a page id outside the cache read as zeros
 * (codes, scales and biases 0); rows that would go to one are not written.
 * keep >= 1, sinks and recent >= 0, sinks + recent <= keep <= new_max_pages *
 * page_size; AQ_ERR_INVALID_ARG otherwise.  lengths and new_lengths may be one
 * array; no other output is part of an input.  AQ_ERR_UNSUPPORTED for B >=
 * 2^22, B * keep >= 2^31, B * ceil(keep / 64) * kv_heads >= 2^24, keep or
 * weights_stride > 2^30, or tables of more than 2^31 - 256 tokens. */
aq_status aq_kv_evict(const float *weights, int64_t weights_stride, const int32_t *lengths,
                      int64_t B, const int32_t *page_table, int64_t max_pages,
                      const int32_t *new_table, int64_t new_max_pages, const aq_kv_cache *cache,
                      int64_t keep, int64_t sinks, int64_t recent, int32_t *kept,
                      float *new_weights, int32_t *new_lengths, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* AQ_H_ */
