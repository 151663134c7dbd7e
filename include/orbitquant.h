/*
 * orbitquant.h -- C ABI of liborbitquant.so, the MI355X (gfx950) library for
 * OrbitQuant's online quantized-linear path.
 *
 * The method (sources: the paper's abstract as reprinted on hotpaper.ai and
 * pith.science; paper.gecl.asia close-reading notes, section Method;
 * llmdb.app summary, section Mathematical Formulation; pith.science
 * Figure 2 caption and Supplementary A setup):
 *   - every activation token x (length d) keeps its L2 norm s = ||x|| apart
 *     and only its direction u = x / s is quantized;
 *   - u is rotated by RPBH: a seeded random permutation Pi, Rademacher signs
 *     D, then an orthonormal Walsh-Hadamard transform on each of the
 *     k = d / h blocks, h = the largest power of two dividing d;
 *   - each rotated coordinate is replaced by the nearest level of the
 *     Lloyd-Max codebook C_{d,b} for N(0, 1/d) (b = 2..4 bits, or 8: the
 *     pages' bit range runs from W2A4 up to W8A8, llmdb.app summary);
 *   - weights are prepared offline as the rows of W Pi^T, i.e. each row w_i
 *     goes through the same rotation and quantizer, with row norm r_i;
 *   - the linear is y[m][n] = s_m r_n sum_k C_{K,bw}[p_nk] C_{K,ba}[q_mk]
 *     (no bias; the rotation cancels inside the product).
 *
 * Conventions shared by every entry point
 *   - Return value: OQ_OK (0) or a negative OQ_E* status; oq_strerror()
 *     describes it.  Nothing throws across this boundary.
 *   - Arguments are validated on the host before any HIP call is made; a
 *     rejected call has no side effect.
 *   - Device pointers are caller-owned device memory (e.g. from PyTorch).
 *     The library never frees them.  Work is enqueued on `stream` (a
 *     hipStream_t passed as void*; NULL = the null stream) and is
 *     asynchronous: results are valid once the stream has reached them.
 *   - The library owns only its rotation-plan tables (a few tens of KB per
 *     (device, d, seed)) and codebook tables (decision grid, levels and
 *     thresholds: about 1 KB per (device, bits, family), 11 KB at 8 bits,
 *     per d for the sphere family); they live until oq_release_plans() or
 *     unload.
 *   - The rotation seed and flags of a layer's weights and of its
 *     activations must be the same; the library cannot check this.
 *   - Code layout ("storage order"): inside each whole group of 128
 *     consecutive rotated coordinates, coordinate 32c + p (c < 4, p < 32)
 *     is stored at slot 8 (p mod 16) + 4 (p div 16) + c; the coordinates
 *     of a last, partial group (d mod 128 = 32, 64 or 96 of them) are
 *     stored at their own index; slot t of a row holds the code
 *     in bits [b t, b t + b) of the row's bytes, little-endian bit order.
 *     A row of d codes therefore takes d*b/8 bytes.  Codes are level
 *     indices 0..2^b-1 in ascending level order.
 *     At 8 bits this is plain byte addressing: byte slot(i) holds code i.
 *   - Limits: d a multiple of 32, 32 <= d <= 16384 (so h = d & -d >= 32);
 *     the linear's K a multiple of 64 (whole 64-slot K steps); bits in
 *     {2, 3, 4, 8} (1..8 for oq_codebook; the exact-sphere family 1..4 and 8).
 *     Zero rows are valid (a zero token gets norm 0 and every code
 *     2^(b-1)).  NaN/Inf inputs give unspecified codes and no error.
 */
#ifndef ORBITQUANT_H
#define ORBITQUANT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define OQ_OK 0
#define OQ_EINVAL (-1)        /* bad argument (null/misaligned pointer, negative size, ...) */
#define OQ_EUNSUPPORTED (-2)  /* valid but not supported (d, bits, bit pair) */
#define OQ_ENOMEM (-3)        /* the library could not allocate its plan tables */
#define OQ_EDEVICE (-4)       /* a HIP call or kernel launch failed */

/* input element types */
#define OQ_F32 0   /* IEEE fp32 */
#define OQ_BF16 1  /* bfloat16, 16-bit patterns */

/* flags */
#define OQ_ROT_NO_SIGNS (1u << 0)     /* rotation without the Rademacher signs D (Pi then H only) */
#define OQ_OUT_F32_ROTATED (1u << 1)  /* oq_rotate_quantize writes the rotated unit vector z
                                         (fp32 [n_tok][d], coordinate order) instead of codes */
#define OQ_OUT_BF16_DEQUANT (1u << 2) /* oq_rotate_quantize writes the dequantized rotated token
                                         s * c_{code_i} (bf16 [n_tok][d], coordinate order, round
                                         to nearest even) instead of codes: fake quantization */
#define OQ_CODEBOOK_SPHERE (1u << 4)  /* Lloyd-Max for the exact marginal of one coordinate of
                                         a uniform point on S^{d-1} instead of its Gaussian limit
                                         N(0, 1/d); activations, weights and oq_linear_ex must
                                         all use the same family */
#define OQ_ROT_INPUT_PERMUTED (1u << 3) /* the input rows are already in rotation order,
                                           x'_i = x_{pi(i)} (see oq_permute_rows); only D and
                                           H are applied.  Same outputs as the unpermuted rows
                                           without this flag */

/* microscaled element formats (the value is the element's bits) */
#define OQ_MX_FP4 4 /* e2m1: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} */
#define OQ_MX_FP8 8 /* e4m3: largest 448, one NaN pattern per sign, no infinity */

/* rotary embedding flags */
#define OQ_ROPE_HALF (1u << 0)    /* pair j is elements (j, j + R/2) of the R turned ones instead
                                     of (2j, 2j + 1) */
#define OQ_ROPE_INVERSE (1u << 1) /* turn by the opposite angle: undoes the embedding, and is the
                                     gradient of it (the turn is orthogonal) */

/* attention flags */
#define OQ_ATTN_CAUSAL (1u << 0) /* a query sees no token behind its own position */

/* Text for a status code.  Never NULL; the string is static. */
const char *oq_strerror(int status);

/* Library ABI version (major * 100 + minor). */
int oq_version(void);

/* Lloyd-Max codebook C_{d,bits} for the dimension marginal N(0, 1/d)
 * (paper.gecl.asia notes, Core Idea and Method item 3; pith.science
 * Figure 2 caption).  Host only, synchronous.
 *   levels:     caller buffer of 2^bits floats, ascending, sigma = 1/sqrt(d)
 *   thresholds: caller buffer of 2^bits - 1 floats, the midpoints of
 *               adjacent levels (decision boundaries)
 * bits in 1..8, d >= 1.  Errors: OQ_EINVAL (null buffer, d < 1),
 * OQ_EUNSUPPORTED (bits).  The solver is Max's shooting method; at 8 bits
 * its levels lie within about 1e-9 (unit scale) of the fixed point. */
int oq_codebook(int d, int bits, float *levels, float *thresholds);

/* oq_codebook with a codebook family (flags 0 or OQ_CODEBOOK_SPHERE).  The
 * sphere family is the Lloyd-Max quantizer of the density
 * c_d (1 - t^2)^((d-3)/2) of one coordinate of a uniform point on S^{d-1}
 * (pith.science: the referee's minor comment 1 asks for this closed-form
 * marginal), defined for the dimensions the kernels take (d % 32 == 0,
 * d <= 16384) and bits 1..4 and 8 (else OQ_EUNSUPPORTED).  It differs from
 * the Gaussian one by 0.8% of a level at d = 256 and 0.015% at d = 13824
 * (4 bits).  Up to 4 bits the solver is Max's shooting method; at 8 bits
 * Newton's method on the Lloyd-Max conditions from the Gaussian codebook
 * (the conditions fix the 8-bit levels to about 1e-7 of the unit scale in
 * double precision). */
int oq_codebook_ex(int d, int bits, uint32_t flags, float *levels, float *thresholds);

/* Bytes of a packed code matrix: rows * d * bits / 8 (-1 on bad input). */
int64_t oq_codes_bytes(int64_t rows, int d, int bits);

/* Online activation path (paper.gecl.asia notes, Method items 1 and 4;
 * pith.science Supplementary A setup; llmdb.app Implementation Details):
 * for each of the n_tok rows of x, s = ||x||_2, z = RPBH(x / s), and each
 * coordinate of z is quantized to the nearest level of C_{d,bits} (ties to
 * the upper level).
 *   x:      device, [n_tok][d] row-major, dtype OQ_F32 or OQ_BF16, 16-byte
 *           aligned
 *   seed:   rotation seed (selects Pi and D)
 *   flags:  OQ_ROT_NO_SIGNS, OQ_ROT_INPUT_PERMUTED, OQ_CODEBOOK_SPHERE, and at
 *           most one of OQ_OUT_F32_ROTATED, OQ_OUT_BF16_DEQUANT
 *   out:    device; packed codes uint8 [n_tok][d*bits/8] (storage order,
 *           16-byte aligned), or with OQ_OUT_F32_ROTATED fp32 [n_tok][d], or
 *           with OQ_OUT_BF16_DEQUANT bf16 [n_tok][d]: coordinate i holds
 *           s * C_{d,bits}[code_i], the token's reconstruction in the rotated
 *           basis.  A bf16 GEMM of two such matrices (activations and weight
 *           rows, same seed) is the fake-quantized product the pages evaluate
 *           (paper.gecl.asia notes, Dataset/Evaluation; llmdb.app
 *           Implementation Details), equal to oq_linear up to operand rounding
 *   norms:  device fp32 [n_tok], receives s (4-byte aligned)
 * n_tok = 0 is a no-op that succeeds (the pointers may then be NULL).
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_ENOMEM, OQ_EDEVICE. */
int oq_rotate_quantize(const void *x, int dtype, int64_t n_tok, int d, uint64_t seed,
                       uint32_t flags, int bits, void *out, float *norms, void *stream);

/* Offline weight preparation (hotpaper.ai abstract: the same quantizer on
 * the weight rows, rotation absorbed into the weights; paper.gecl.asia
 * notes, Method item 2: W Pi^T): row i of W [n_out][d_in] becomes the
 * packed codes of RPBH(w_i / r_i) under C_{d_in,bits} plus r_i = ||w_i||.
 * Same layout, limits and errors as oq_rotate_quantize (w_codes
 * [n_out][d_in*bits/8], row_norms [n_out]); OQ_OUT_F32_ROTATED and
 * OQ_OUT_BF16_DEQUANT are rejected here (oq_rotate_quantize on the weight
 * rows gives the same outputs). */
int oq_prepare_weights(const void *W, int dtype, int64_t n_out, int d_in, uint64_t seed,
                       uint32_t flags, int bits, uint8_t *w_codes, float *row_norms,
                       void *stream);

/* Low-bit linear (llmdb.app Mathematical Formulation, y = Q_w(W R^-1)
 * Q_a(R x), no bias):
 *   y[m][n] = bf16( s_m r_n sum_k C_{K,w_bits}[p_nk] C_{K,a_bits}[q_mk] )
 * with both code matrices in storage order (the sum runs over the same
 * permuted coordinates on both sides).  Accumulation is fp32 over fp16
 * copies of the unit-variance levels; the output is rounded once to bf16
 * (round to nearest even).
 *   a_codes [M][K*a_bits/8], a_norms [M], w_codes [N][K*w_bits/8],
 *   w_norms [N]: device, as produced by oq_rotate_quantize /
 *   oq_prepare_weights with the same seed, flags and K
 *   y: device bf16 bit patterns, [M][N] row-major, 2-byte aligned; a y
 *      that shares a byte with any of the four inputs is rejected
 *      (OQ_EINVAL).  Until the call completes on the stream, y
 *      may hold intermediate values (a sparse last round of output tiles
 *      parks fp32 partial sums in y's first rows, which are then
 *      overwritten), so nothing may read it concurrently.
 * a_bits, w_bits in {2, 3, 4}, any pair, or both 8 (W8A8: the codes are
 * decoded through an fp16 table of the 256 levels; a pair with only one
 * side at 8 bits is OQ_EUNSUPPORTED).  K % 64 == 0, K <= 16384 (a K with a
 * last partial group of 32 or 96 coordinates is OQ_EUNSUPPORTED here, though
 * such rows can be rotated and prepared).  M and N up to 2^30
 * (OQ_EUNSUPPORTED beyond).  M = 0 or N = 0 is a no-op that succeeds (the pointers may then
 * be NULL).  Errors:
 * OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_linear(const uint8_t *a_codes, const float *a_norms, int a_bits,
              const uint8_t *w_codes, const float *w_norms, int w_bits,
              int64_t M, int64_t N, int K, uint16_t *y, void *stream);

/* oq_linear with a codebook family for both operands (flags 0 or
 * OQ_CODEBOOK_SPHERE; the codes must come from rotate/prepare calls with
 * the same family).  Same layout, limits and errors; flags outside the
 * family bit give OQ_EINVAL.  W8A8 takes either family. */
int oq_linear_ex(const uint8_t *a_codes, const float *a_norms, int a_bits,
                 const uint8_t *w_codes, const float *w_norms, int w_bits,
                 int64_t M, int64_t N, int K, uint32_t flags, uint16_t *y, void *stream);

/* Free every cached rotation plan and codebook table on every device (the
 * caller must ensure that no enqueued work still uses them, e.g. by
 * synchronising first, and that no other thread is inside a library call
 * meanwhile).  Handles from oq_plan_create stay valid to destroy
 * but name no tables any more. */
int oq_release_plans(void);

/* INT4 weight-only round-to-nearest for the AdaLN modulation projections
 * (paper.gecl.asia notes, Method item 5: a rotation cannot be folded into a
 * dynamic modulation, so those weights get INT4 RTN and the activations
 * stay unquantized; researchpod.app transcript).  Per output row n:
 * amax = max_k |W_nk|, scale_n = amax / 7, q_nk = rint(W_nk * (7 / amax)) in
 * [-7, 7], the decisions taken in fp32 (IEEE division and product, ties to
 * even); a zero row gives q = 0, scale 0.
 *   W:      device, fp32 or bf16 [n_out][d_in] (4-byte aligned)
 *   q4:     device uint8 [n_out][d_in/2] (16-byte aligned): nibble q + 8,
 *           coordinate 2i in the low nibble of byte i
 *   scales: device fp32 [n_out]
 *   d_in % 32 == 0, d_in <= 16384 (else OQ_EUNSUPPORTED); n_out = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_rtn4_prepare_weights(const void *W, int dtype, int64_t n_out, int d_in, uint8_t *q4,
                            float *scales, void *stream);

/* The AdaLN projection with those weights:
 *   y[m][n] = bf16( scale_n sum_k x_mk q_nk )
 * fp32 accumulation (exact products), one bf16 rounding (nearest even), no
 * bias.  x: device fp32 or bf16 [M][K] (16-byte aligned); y: bf16 [M][N].
 * Sized for modulation inputs (one row per sample): weights are read once
 * per block of 8 rows.  K % 32 == 0, K <= 16384; M = 0 or N = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_rtn4_linear(const void *x, int dtype, int64_t M, const uint8_t *q4, const float *scales,
                   int64_t N, int K, uint16_t *y, void *stream);

/* Permute rows by the rotation permutation pi of (d = rows, seed):
 * dst row i = src row pi(i), rows of row_bytes bytes each (any dtype).
 * Folds pi into a producer: permuting the output rows of the layer that
 * feeds the activations (and its bias), with an elementwise function such
 * as GELU between, makes the activations arrive in rotation order, and
 * oq_rotate_quantize with OQ_ROT_INPUT_PERMUTED then skips the permutation
 * (paper.gecl.asia notes, Limitations: rotation and norm cost at run time).
 * The signs D cannot be folded through a nonlinearity and stay in the call.
 *   src, dst: device, caller-owned, distinct (no in-place), [rows][row_bytes]
 *   rows:     the permutation length d: 32 <= d <= 16384, d % 32 == 0
 *   row_bytes >= 1
 * rows = 0 is rejected (there is no plan of length 0).
 * Errors: OQ_EINVAL (null or equal pointers, row_bytes < 1), OQ_EUNSUPPORTED
 * (rows), OQ_ENOMEM, OQ_EDEVICE. */
int oq_permute_rows(const void *src, void *dst, int64_t rows, int64_t row_bytes, uint64_t seed,
                    void *stream);

/* Optional explicit plan ownership.  The compute calls build the rotation
 * plan of (current device, d, seed) -- the permutation Pi and the signs D
 * (pith.science Supplementary A setup) as device tables -- on first use and
 * cache it.  oq_plan_create builds it now (no first-call latency) and pins
 * it; oq_plan_destroy drops the pin and frees the tables when no other
 * handle pins them (the caller must ensure that no enqueued work still
 * uses them and that no other thread's call on the same (d, seed) is in
 * progress).  A later compute call with the same (d, seed) rebuilds the plan.
 *   d:     32 <= d <= 16384, d % 32 == 0   (else OQ_EUNSUPPORTED)
 *   flags: 0 or OQ_ROT_NO_SIGNS (one plan serves both sign modes)
 *   plan:  receives an opaque handle (NULL on error)
 * Errors: OQ_EINVAL (null out pointer, bad flags, d <= 0, or a handle not
 * made by oq_plan_create), OQ_EUNSUPPORTED, OQ_ENOMEM, OQ_EDEVICE. */
int oq_plan_create(int d, uint64_t seed, uint32_t flags, void **plan);
int oq_plan_destroy(void *plan);

/* ---- the microscaled path: norm -> codes -> projection -> embedding ----
 *
 * What a diffusion transformer's block needs around a projection in
 * microscaled (MX) floating point (the OCP Microscaling formats, e2m1 and
 * e4m3 elements in blocks of 32 with an e8m0 scale): the calls below take and
 * give the same rows as the rest of the library and follow its conventions.
 * None of them keeps anything between calls or needs a workspace; each is one
 * or two kernels on `stream` and can be captured into a graph.
 *
 * MX rows: a row of d elements is d * format / 8 code bytes (e2m1: two codes a
 * byte, the even element in the low half; sign, two exponent bits, one mantissa
 * bit from the top; e4m3: one byte) and d / 32 scale bytes, both in coordinate
 * order.  Scale byte s of a block stands for 2^(s - 127); with m = max |x|
 * over the block, s = max(127 + floor(log2 m) - e_max, 0), e_max = 2 (e2m1)
 * or 8 (e4m3); an element is x / 2^(s - 127) rounded to the nearest value of
 * its type, ties to even, at most the largest.  A block of zeros has s = 0.
 * A block with a NaN or an infinity gets s = 255 and codes 0 and reads back
 * as NaN; in a product it makes the row's outputs NaN.
 * d (K): a multiple of 32, 32 <= d <= 16384; rows up to 2^30. */

/* Quantize rows to MX codes.
 *   x: device fp32 or bf16 [rows][d], 16-byte aligned
 *   codes: device [rows][d * format / 8], 16-byte aligned; scales: device
 *   [rows][d / 32].  No two of the arrays may share a byte.
 * rows = 0 is a no-op that succeeds.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_mx_quantize(const void *x, int dtype, int64_t rows, int d, int format, uint8_t *codes,
                   uint8_t *scales, void *stream);

/* Read MX codes back: out[i] = element * 2^(s - 127), in dtype (exact, but for
 * values of 2^128 and more, which are infinite, and in bf16 for e4m3 values
 * below 2^-126, which round).
 *   out: device fp32 or bf16 [rows][d], 16-byte aligned, apart from the inputs
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int format, int64_t rows, int d,
                     int dtype, void *out, void *stream);

/* Linear on MX codes:
 *   y[m][n] = bf16( sum_b 2^(sa_mb + sw_nb - 254) sum_{k in block b} a_mk w_nk )
 * fp32 accumulation on the matrix cores, one bf16 rounding, no bias; any
 * pair of formats.  Where a side is e4m3 the matrix cores line up the products
 * of 64 (up to 32 rows, or few outputs: 128) consecutive k to the largest of
 * them before they add: measured, off by at most 2^-11.3 of it.
 * A call gives the same bits every time; the order of a row's sums is chosen by
 * M, N and the formats, so a row may have other bits in another batch.
 *   a_codes [M][K * a_format / 8], a_scales [M][K / 32], w_codes
 *   [N][K * w_format / 8], w_scales [N][K / 32]: device, codes 16-byte aligned
 *   y: device bf16 [M][N], apart from every input
 * M = 0 or N = 0 is a no-op that succeeds.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_mx_linear(const uint8_t *a_codes, const uint8_t *a_scales, int a_format,
                 const uint8_t *w_codes, const uint8_t *w_scales, int w_format, int64_t M,
                 int64_t N, int K, uint16_t *y, void *stream);

/* Gated residual sum and modulated RMS norm of every row:
 *   h = residual + gate_g * x
 *   y = h / sqrt(mean(h^2) + eps) * weight * (1 + scale_g) + shift_g
 * with g = row / rows_per_mod; residual, gate, weight, scale and shift may
 * each be NULL (then 0, 1, 1, 0, 0).  fp32 arithmetic; the norm runs over h
 * before it is rounded to the stream's type.
 *   x, residual: device, dtype [rows][d]
 *   weight: device, param_dtype [d]; gate, scale, shift: device, param_dtype,
 *     row g at g * mod_stride elements (mod_stride >= d, a multiple of 16
 *     bytes, where there is more than one group: the slices of one modulation
 *     projection [groups][6 d] are passed as they lie)
 *   eps: finite, at least the smallest normal fp32 number
 *   sum: device, dtype [rows][d], receives h; may be NULL
 *   y_format 0: y is dtype [rows][d] and y_scales is NULL; OQ_MX_FP4 or
 *     OQ_MX_FP8: y are MX codes and y_scales their scale bytes, as
 *     oq_mx_quantize makes them of the fp32 values
 * Every pointer but y_scales 16-byte aligned.  sum, and a y in dtype, may be x
 * or the residual themselves (in place); otherwise an output may not share a
 * byte with an input or with another output.
 * d a multiple of 32, 32 <= d <= 16384; rows up to 2^30; rows = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_add_rms_norm(const void *x, const void *residual, int dtype, int64_t rows, int d, float eps,
                    const void *weight, const void *gate, const void *scale, const void *shift,
                    int param_dtype, int64_t rows_per_mod, int64_t mod_stride, void *sum,
                    int y_format, void *y, uint8_t *y_scales, void *stream);

/* Rotary embedding with several axes (time, height, width of a latent video).
 * The first R = sum(axis_dims) elements of each head are R/2 pairs, numbered
 * axis after axis; pair i of axis a turns by pos_a * theta^(-2 i / axis_dims[a]):
 *   (u, v) -> (u cos - v sin, u sin + v cos)
 * and the other head_dim - R elements are copied.  Angles are exact to 2^-30
 * of a turn at every int32 position.
 *   x, y: device, dtype; element e of head h of token t at t * token stride +
 *     h * head stride + e (strides in elements, multiples of 16 bytes, >= 0), so
 *     the queries and keys inside a fused projection's output are read in
 *     place; 16-byte aligned.  y is x with the same strides (in place), or
 *     its span may not meet x's; y's elements have addresses of their own
 *     (each head whole, heads inside tokens or tokens inside heads)
 *   pos: device int32 [tokens][axes]
 *   axes 1..4; axis_dims: host, even, >= 0, sum R <= head_dim
 *   head_dim % 8 == 0, <= 512; with OQ_ROPE_HALF R % 16 == 0; theta >= 1
 *   flags: OQ_ROPE_HALF, OQ_ROPE_INVERSE
 * tokens = 0 or heads = 0 is a no-op that succeeds; tokens up to 2^30.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_rope(const void *x, int dtype, int64_t tokens, int heads, int head_dim, int64_t x_token,
            int64_t x_head, const int32_t *pos, int axes, const int *axis_dims, double theta,
            uint32_t flags, void *y, int64_t y_token, int64_t y_head, void *stream);

/* ---- the cached-attention path: projection -> heads -> cache -> attention ----
 *
 * What a block with a key/value cache runs for its new tokens (one token a
 * step, a chunk of a streamed video, a prompt that every denoising step reads
 * again): the projection of few rows by 4-bit weights with group scales, the
 * norm and embedding of the query and key heads, the new keys and values into a
 * 4-bit cache, and attention over it.  Conventions as above.
 *
 * The cache: `pages` pages of `page_size` tokens, for keys and for values
 *   codes  [pages][kv_heads][page_size][head_dim / 2]
 *   scales [pages][kv_heads][page_size][head_dim / 32]
 * a head's row as an OQ_MX_FP4 row (so oq_mx_dequantize reads a cache back).  A
 * token's slot is page * page_size + its offset in the page.
 * head_dim: a multiple of 32, 32 <= head_dim <= 256; kv_heads up to 65535;
 * page_size >= 1; codes and scales 16-byte aligned. */

/* INT4 weights with a scale for every `group` consecutive coordinates of a row:
 *   zeros NULL: scale = max |w| / 7, nibble = rint(w / scale) + 8
 *   zeros:      scale = hi / 15 - lo / 15 with hi = max(w, 0), lo = min(w, 0),
 *               zero = rint(-lo / scale), nibble = rint(w / scale) + zero in [0, 15]
 * in fp32 (IEEE division, ties to even), with the scale already rounded to
 * scale_dtype; nibbles past 0 or 15 (by the scale's rounding) are 0 or 15; a scale
 * of 0 gives the nibble that stands for 0 (8, or zero = 0).  A NaN or an infinity
 * gives its group unspecified nibbles, scale and zero, and no error.
 *   W: device, fp32 or bf16 [n_out][d_in] (4-byte aligned)
 *   q4: device [n_out][d_in / 2] (16-byte aligned), the even coordinate in the
 *       low nibble; scales, zeros: device, scale_dtype [n_out][d_in / group]
 *       (4-byte aligned)
 * group a multiple of 32 that divides d_in; d_in <= 16384 (else
 * OQ_EUNSUPPORTED).  No two arrays may share a byte.  n_out = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_rtn4_group_prepare_weights(const void *W, int dtype, int64_t n_out, int d_in, int group,
                                  uint8_t *q4, void *scales, void *zeros, int scale_dtype,
                                  void *stream);

/* The projection with those weights (any nibbles, scales and zeros):
 *   y[m][n] = bf16( sum_g scale_ng sum_{k in g} x_mk (nibble_nk - zero_ng) )
 * zero = 8 where zeros is NULL; fp32 accumulation, one bf16 rounding, no bias.
 *   x: device fp32 or bf16 [M][K] (16-byte aligned); y: bf16 [M][N], apart from
 *   the inputs
 * Sized for few rows.  Sums hold x_mk (16 + nibble): a row whose |x| sum to 2^122
 * or more over a group may come out infinite or NaN, as one with an infinity or a
 * NaN does; no other row is touched by it.  N up to 2^27, M up to
 * 2^30.  M = 0 or N = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_rtn4_group_linear(const void *x, int dtype, int64_t M, const uint8_t *q4,
                         const void *scales, const void *zeros, int scale_dtype, int group,
                         int64_t N, int K, uint16_t *y, void *stream);

/* RMS norm of every query and key head with the rotary embedding (as oq_rope,
 * its axes, angles and pairs) in the same pass:
 *   n = x / sqrt(mean(x^2) + eps) * weight, over the head's elements
 *   (u, v) -> (u cos - v sin, u sin + v cos) for the turned pairs of n
 * fp32 arithmetic, one rounding to dtype.
 *   q, k, q_out, k_out: device, dtype, strided as oq_rope's x and y: each may
 *     be its own input (in place), no output may otherwise meet an input or the
 *     other output.  k and k_out NULL with k_heads 0: queries alone
 *   q_weight, k_weight: device, param_dtype [head_dim], 16-byte aligned, or NULL
 *   eps: finite, at least the smallest normal fp32 number
 *   pos: device int32 [tokens][axes]; flags: OQ_ROPE_HALF
 * Limits as oq_rope's; heads up to 2^24 together.  tokens = 0 is a no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_qk_norm_rope(const void *q, int q_heads, int64_t q_token, int64_t q_head, const void *k,
                    int k_heads, int64_t k_token, int64_t k_head, int dtype, int64_t tokens,
                    int head_dim, const void *q_weight, const void *k_weight, int param_dtype,
                    float eps, const int32_t *pos, int axes, const int *axis_dims, double theta,
                    uint32_t flags, void *q_out, int64_t q_out_token, int64_t q_out_head,
                    void *k_out, int64_t k_out_token, int64_t k_out_head, void *stream);

/* Write the keys and values of tokens into the cache, quantized as
 * oq_mx_quantize does.
 *   k, v: device, dtype [tokens][kv_heads][head_dim], any strides that are
 *     multiples of 16 bytes and >= 0, 16-byte aligned
 *   slots: device int64 [tokens]; a token whose slot is negative or past the
 *     cache is not written.  Two tokens may not share a slot (its contents are
 *     then unspecified)
 * The other slots keep their bytes.  tokens up to 2^30; tokens = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_mx_kv_write(const void *k, const void *v, int dtype, int64_t tokens, int64_t k_token,
                   int64_t k_head, int64_t v_token, int64_t v_head, const int64_t *slots,
                   uint8_t *k_codes, uint8_t *k_scales, uint8_t *v_codes, uint8_t *v_scales,
                   int64_t pages, int kv_heads, int page_size, int head_dim, void *stream);

/* Bytes of workspace that oq_mx_kv_attention takes for these sizes (0: none; -1: a
 * size that the call refuses). */
int64_t oq_mx_kv_attention_workspace(int64_t q_tokens, int q_heads, int kv_heads, int head_dim,
                                     int64_t batch, int page_size, int64_t table_pages);

/* Attention of new queries over the cached keys and values of their sequences:
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q k_j)
 * over the tokens j that the query sees; query head h reads key head
 * h / (q_heads / kv_heads).
 *   q, out: device, dtype [q_tokens][q_heads][head_dim], strided as oq_rope's x
 *     and y, apart from each other
 *   batch sequences; q_starts: device int32 [batch + 1], sequence b's queries
 *     are the tokens [q_starts[b], q_starts[b + 1]); the outputs of tokens behind
 *     the last sequence are left as they were.  Starts ascend and are clamped to
 *     [0, q_tokens]; where they descend, the outputs are unspecified (nothing else
 *     is touched).  NULL: the tokens are split
 *     evenly (q_tokens a multiple of batch)
 *   lengths: device int32 [batch], tokens in the cache (counting the new ones);
 *     taken as 0 below 0 and as table_pages * page_size above that
 *   table: device int32 [batch][table_pages], the pages of each sequence; a
 *     token whose page number is not in [0, pages) reads as NaN.  NULL: sequence
 *     b's tokens are page b alone (table_pages = 1, pages >= batch)
 *   With n queries and length L, query i stands at position L - n + i.  It sees
 *     every token, with OQ_ATTN_CAUSAL those up to its position, and with
 *     window > 0 (which needs OQ_ATTN_CAUSAL) of these the last `window`.  A
 *     query that sees none gets zeros (and lse -infinity)
 *   lse: device fp32 [q_tokens][q_heads], ln sum_j p_j; may be NULL
 *   scale: |scale| <= 2^127
 *   workspace: device, 16-byte aligned, at least oq_mx_kv_attention_workspace
 *     bytes, not shared with other work in flight; its contents before and after
 *     do not matter
 * fp32 statistics and sums.  bf16 queries: the products' operands are the bf16
 * values (the cache's are exact in bf16) and weights p rounded to bf16 (by 2^-8 of
 * each at most; their sum is of the fp32 ones); fp32 queries keep fp32 accuracy.
 * Scores q k_j, the sums that make them and scale q k_j log2 e must be finite in
 * fp32, and so must the sums of p_j |v_j|, in which p_j may be up to 2^8: values
 * below 2^119 / (tokens that a row sees) always are.  A row with a NaN in its query
 * or in a key that it sees is NaN, its lse too.  A block of 32 values with a NaN
 * makes these 32 elements NaN in the rows that see its token; their lse stays as it
 * is.  Tokens that a row does not see do not reach it.  Scale bytes 253 to 255 read
 * as NaN here (the writer makes none but 255), and values below 2^-126 may count as
 * 0.
 * A call gives the same bits every time; the order of a row's sums is chosen by
 * the sizes, as is the kernel that takes the call: by a sequence's rows on average
 * (queries times heads of a key head), so that single tokens beside a long prompt
 * are faster in a call of their own.  q_tokens * q_heads / kv_heads up to 2^27, batch up to 2^20,
 * table_pages * page_size up to 2^30.  q_tokens = 0 or batch = 0 no-op.
 * Errors: OQ_EINVAL, OQ_EUNSUPPORTED, OQ_EDEVICE. */
int oq_mx_kv_attention(const void *q, int dtype, int64_t q_tokens, int q_heads, int64_t q_token,
                       int64_t q_head, const uint8_t *k_codes, const uint8_t *k_scales,
                       const uint8_t *v_codes, const uint8_t *v_scales, int64_t pages,
                       int kv_heads, int page_size, int head_dim, int64_t batch,
                       const int32_t *lengths, const int32_t *q_starts, const int32_t *table,
                       int64_t table_pages, float scale, uint32_t flags, int window, void *out,
                       int64_t out_token, int64_t out_head, float *lse, void *workspace,
                       int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* ORBITQUANT_H */
