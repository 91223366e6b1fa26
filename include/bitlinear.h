/*
 * bitlinear.h -- C ABI of the MI355X (gfx950) BitLinear W1.58A8 library.
 *
 * The layer is the BitNet b1.58 BitLinear: weights are absmean-ternarized to
 * {-1, 0, +1} and stored packed at 2 bits each; activations are quantized per
 * token to int8 by absmax; the product is accumulated in int32 and rescaled to
 * bf16.  Sources, on the BitNet b1.58 pages:
 *   [P1] bako.co, "BitNet b1.58 and the 1-Bit AI Architecture Revolution",
 *        section "The BitLinear Layer and AbsMean Quantization": gamma is the
 *        mean absolute value of the entire weight matrix; each weight is
 *        divided by (gamma + 1e-5), rounded to the nearest integer and clamped
 *        to [-1, 1]; with ternary weights the matrix product reduces to
 *        integer additions and subtractions.
 *   [P2] deepmox.com chapter 8, "A low-bit model is a whole-stack design":
 *        weights take the three values -1, 0, +1; activations use a separate
 *        per-token 8-bit path (W1.58A8); the GPU path packs four ternary values
 *        per 8-bit storage unit, moves packed weights from HBM on chip,
 *        unpacks them and computes with the 8-bit activations.
 *   [P3] onilabs.co, "A Two-Billion Ternary Bet": activations are quantized
 *        dynamically; scale factors are staged for mixed-precision compute;
 *        the 2B4T model uses squared ReLU in its feed-forward block (as does
 *        [P2], same section).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees or synchronizes; it only enqueues work
 *     on `stream` (a hipStream_t; NULL means the null stream) and returns.
 *   - Tensors are dense and row-major.  W is [n][k] (n output features,
 *     k input features), activations are [m][k] (m tokens), outputs [m][n].
 *   - k must be a positive multiple of 64 and at most BL_MAX_K (2^22);
 *     m <= BL_MAX_M (2^23) and n <= BL_MAX_N (2^26); m and n may be 0
 *     (nothing is enqueued) except where stated; n * k, m * k and m * n must
 *     stay below 2^40.  A shape inside these limits whose launch grid would
 *     still exceed the device's 2^32 work-items (a very large m * n product)
 *     returns BL_ERR_SHAPE as well, before anything is enqueued.
 *   - Pointers that are read or written with 128-bit accesses (w, packed, x,
 *     xq, workspace) must be 16-byte aligned; alpha, gamma and acc 4-byte,
 *     y 2-byte aligned.
 *   - Validation happens on the host before anything is enqueued; a failing
 *     check returns its code and enqueues nothing.  Shapes are checked first;
 *     an empty problem (m or n = 0) then returns BL_OK at once, so empty
 *     tensors may pass NULL pointers.  A failed kernel launch
 *     returns BL_ERR_HIP.  Faults inside kernels surface at the caller's next
 *     synchronization.  Entry points are thread-safe; the only global
 *     mutable state is the device array of bl_ternarize_pack_noalloc (see
 *     there).  Calls on one stream execute in order.
 *   - Inputs must be finite (no Inf or NaN).
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define BL_MAX_K (1 << 22)
#define BL_MAX_M (1 << 23)
#define BL_MAX_N (1 << 26)
#define BL_MAX_BACKWARD_N (1 << 24)

/* Status codes.  bl_status is a plain int, so that any value a caller
 * passes back (bl_status_string) is well defined in C and C++ alike. */
typedef int bl_status;
enum {
    BL_OK = 0,
    BL_ERR_NULL = 1,      /* a required pointer is NULL                          */
    BL_ERR_SHAPE = 2,     /* m, n or k outside the supported range               */
    BL_ERR_ALIGN = 3,     /* a pointer is not aligned as required                */
    BL_ERR_WORKSPACE = 4, /* workspace smaller than bl_ternarize_pack_workspace_bytes */
    BL_ERR_HIP = 5        /* the HIP runtime rejected a launch                   */
};

/* Size in bytes of the packed ternary buffer for an [n][k] weight matrix:
 * ceil(n/16)*16 * k/4 (four trits per byte [P2]; rows padded to 16).
 * Returns 0 for an invalid shape. */
size_t bl_packed_bytes(int64_t n, int64_t k);

/* Device workspace needed by bl_ternarize_pack: a fixed 2 KiB (256 exponent
 * bins of 64-bit integers, into which the absmean pass adds).  Returns 0 for
 * an invalid shape. */
size_t bl_ternarize_pack_workspace_bytes(int64_t n, int64_t k);

/* Weight preparation [P1]: gamma = mean |w| over all n*k weights, computed
 * exactly and rounded once to fp32 (nearest, ties to even); then every weight
 * becomes q = clamp(round_half_even(w / fl32(gamma + 1e-5f)), -1, 1), the
 * division in correctly rounded fp32; q is stored packed.
 *   w         [n][k] fp32, read only.
 *   packed    out, bl_packed_bytes(n, k) bytes.  Layout: 2-bit code q + 1
 *             (0, 1, 2; 3 never occurs).  The matrix is cut into tiles of 16
 *             rows x 64 columns; tile (i, j) starts at byte
 *             256 * (i * (k/64) + j); inside it, row r owns bytes 16r..16r+15,
 *             and column 64j + t of that row sits in byte 16r + (t % 16) at
 *             bits 2*(t/16)..2*(t/16)+1.  Rows n..ceil(n/16)*16-1 hold code 1.
 *   gamma     out, one fp32 on the device (gamma, without eps).
 *   workspace device scratch of workspace_bytes >= the size above; its
 *             contents on entry do not matter and are clobbered.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (n < 1, bad k, or n*k > 2^35: 34 G
 *         weights, 137 GB of fp32 input), BL_ERR_ALIGN, BL_ERR_WORKSPACE,
 *         BL_ERR_HIP. */
bl_status bl_ternarize_pack(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma,
                            void* workspace, size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): exactly
 * bl_ternarize_pack (same gamma, same packed bytes), without a workspace
 * argument.  The 2 KiB of exponent bins live in a static device array of the
 * library, one per GPU, held until the process ends; it covers every shape
 * bl_ternarize_pack takes (n*k <= 2^35), and larger shapes are rejected with
 * BL_ERR_SHAPE.  The first call on a device looks the array's address up
 * (hipGetSymbolAddress, with that device current); later calls allocate and
 * free nothing.  Each call clears the bins on `stream` (with a kernel) before
 * using them, so leftovers of an earlier call do not matter, but two calls
 * that overlap on one GPU (on different streams, or from different host
 * threads) share the array and race: serialize them.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP (also when the
 *         array's address cannot be obtained). */
bl_status bl_ternarize_pack_noalloc(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma,
                                    void* stream);

/* Per-token absmax int8 activation quantization [P2, P3]: for each row i,
 * a = max_j |x[i][j]|, s = fl32(127 / max(a, 1e-5f)),
 * xq[i][j] = clamp(round_half_even(fl32(x[i][j] * s)), -128, 127), alpha[i] = a.
 *   x      [m][k] bf16 (raw 16-bit patterns), read only.
 *   xq     out [m][k] int8.
 *   alpha  out [m] fp32 (the per-token absmax, exactly a bf16 value).
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_quant_act(const uint16_t* x, int64_t m, int64_t k, int8_t* xq, float* alpha, void* stream);

/* Ternary x int8 product with rescale [P1, P3]:
 *   acc[i][j] = sum_t xq[i][t] * q[j][t]          (exact, int32)
 *   y[i][j]   = bf16(acc[i][j] * gamma * alpha[i] / 127)   (fp32 evaluation,
 *               within one bf16 ulp of the exactly rounded value; acc = 0
 *               gives +0)
 *   packed/gamma as written by bl_ternarize_pack for an [n][k] matrix;
 *   xq/alpha as written by bl_quant_act for [m][k] activations.
 *   acc    out [m][n] int32, or NULL to skip it.
 *   y      out [m][n] bf16 bit patterns, or NULL to skip it (not both NULL).
 * The kernel is chosen from m, n and k: decode kernels that stream the
 * weights once per block of 16 (or 64) tokens for up to 64 tokens, the tiled
 * int8 matrix-core GEMM beyond; results do not depend on the choice.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_linear(const uint8_t* packed, const float* gamma, const int8_t* xq, const float* alpha,
                    int64_t m, int64_t n, int64_t k, int32_t* acc, uint16_t* y, void* stream);

/* The whole layer in one call [P1, P2, P3]: per-token absmax int8
 * quantization of x followed by the ternary product and rescale, with exactly
 * the results of bl_quant_act followed by bl_linear.  For one token, and for
 * up to 16 tokens while m * k is at most 65536 (rows up to 8192; 32767
 * beyond) and the activations quantized over all workgroups stay below 2^24
 * (2^23 for rows of 8192 and more), a single kernel does both steps (each
 * workgroup quantizes the tokens it multiplies); otherwise the two kernels
 * run back to back on `stream`.  Results do not depend on the choice.
 *   x      [m][k] bf16 (raw 16-bit patterns), read only.
 *   xq     out [m][k] int8 (the quantized activations; also used as staging).
 *   alpha  out [m] fp32 (per-token absmax).
 *   acc, y as in bl_linear (either may be NULL, not both).
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_bitlinear(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t n, int64_t k,
                       int8_t* xq, float* alpha, int32_t* acc, uint16_t* y, void* stream);

/* ---- Five trits per byte ----
 * The denser weight code: [P4] bako.co, "BitNet b1.58 and the 1-Bit AI
 * Architecture Revolution", section "The Information Theory of 1.58 Bits" (a
 * three-state weight carries log2(3), about 1.58, bits) and [P5] deepmox.com
 * chapter 1, "Why Smaller Weights Are Not the Whole Story", section "A
 * different place to make efficiency decisions" (the 2B4T model keeps its
 * non-embedding weights below two bits per weight).  3^5 = 243 <= 256, so
 * five trits share one byte: 1.6 bits per weight, 20% fewer bytes to move
 * per decoded token than the 2-bit code, for the same gamma, trits and
 * results. */

#define BL_B3_MAX_K 64000
#define BL_B3_MAX_M 64

/* Size in bytes of the five-trits-per-byte buffer for an [n][k] matrix:
 * ceil(n/16)*16 rows of ceil(k/320)*64 bytes.  Returns 0 for an invalid shape. */
size_t bl_packed_bytes_b3(int64_t n, int64_t k);

/* Weight preparation in the five-trits-per-byte code [P1, P4, P5]: the same
 * gamma and trits as bl_ternarize_pack, stored as follows.  Five trits t_0..t_4
 * with codes c_d = t_d + 1 form v = sum_d c_d * 3^(4-d); the byte is
 * ceil(256 * v / 243) (so v = floor(243 * b / 256), and digit d is also
 * floor(3 * ((b * 3^d) mod 256) / 256)).  The matrix is cut into super-tiles
 * of 16 rows x 320 columns, 1024 bytes each, column super-tile fastest
 * (super-tile (i, s) at byte 1024 * (i * ceil(k/320) + s)); inside one,
 * column 80 g + 16 d + j (g < 4, d < 5, j < 16) of row r sits in byte
 * 256 g + 16 r + j as digit d.  Columns past k and rows past n hold trit 0.
 *   w, gamma, workspace as for bl_ternarize_pack; packed has
 *   bl_packed_bytes_b3(n, k) bytes.
 * Errors: as bl_ternarize_pack. */
bl_status bl_ternarize_pack_b3(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma,
                               void* workspace, size_t workspace_bytes, void* stream);

/* The whole layer from five-trits-per-byte weights, for decoding [P1, P2, P3,
 * P4]: per-token absmax int8 quantization of x (xq, alpha written exactly as
 * bl_quant_act would) and the ternary product with the bf16 rescale, with
 * exactly the results of bl_quant_act followed by bl_linear on the 2-bit
 * packing of the same trits.  One kernel per call; every token is its own
 * pass over the weights, so the call is meant for few tokens (m up to
 * BL_B3_MAX_M) and rows up to BL_B3_MAX_K columns (a row's activations are
 * held on chip).
 *   packed/gamma from bl_ternarize_pack_b3 for an [n][k] matrix;
 *   x [m][k] bf16; xq out [m][k] int8; alpha out [m] fp32;
 *   acc, y as in bl_linear (either may be NULL, not both).
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (m > BL_B3_MAX_M, k > BL_B3_MAX_K, or
 *         as bl_bitlinear), BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_bitlinear_b3(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t n,
                          int64_t k, int8_t* xq, float* alpha, int32_t* acc, uint16_t* y, void* stream);

/* ---- Gated feed-forward front half: gate+up BitLinear + squared ReLU ----
 * A feed-forward block with f hidden units has one gate+up BitLinear of 2f
 * output rows (rows 0..f-1 the gate, rows f..2f-1 the up projection; one
 * gamma for the whole matrix) followed by squared-ReLU gating [P2, P3]:
 *   h[i][j] = bf16(relu(g)^2 * u),  g = acc[i][j] * s,  u = acc[i][f + j] * s,
 *   s = gamma * alpha[i] / 127,
 * with acc the exact int32 products as in bl_linear.  g and u are not rounded
 * to bf16 first; h is evaluated in fp32 (within one bf16 ulp of the exactly
 * rounded value) and relu(g) = 0 gives +0 * u (so -0 for negative u).
 * f must be a positive multiple of 16. */

/* Weight preparation for a gate+up matrix: exactly bl_ternarize_pack of the
 * [2f][k] matrix w (gamma of all 2f*k weights), except that the packed row
 * tiles alternate: packed row tile 2t holds gate rows 16t..16t+15 and packed
 * row tile 2t+1 holds up rows 16t..16t+15 (rows f+16t.. of w), so that both
 * halves of 16 outputs sit next to each other.  packed has
 * bl_packed_bytes(2f, k) bytes; bl_unpack_ternary(packed, 2f, k) returns the
 * rows in that packed order.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (f not a positive multiple of 16, bad k,
 *         2f*k > 2^35), BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_ternarize_pack_glu(const float* w, int64_t f, int64_t k, uint8_t* packed, float* gamma,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Gated product from quantized activations: packed/gamma from
 * bl_ternarize_pack_glu, xq/alpha from bl_quant_act ([m][k]).
 *   h      out [m][f] bf16 bit patterns.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_linear_glu(const uint8_t* packed, const float* gamma, const int8_t* xq, const float* alpha,
                        int64_t m, int64_t f, int64_t k, uint16_t* h, void* stream);

/* The gated front half in one call: per-token quantization of x (xq and
 * alpha written exactly as bl_quant_act would) and the gated product, with
 * exactly the results of bl_quant_act followed by bl_linear_glu.  The token
 * counts that bl_bitlinear serves with a single kernel take one here too.
 *   x      [m][k] bf16; xq out [m][k] int8; alpha out [m] fp32;
 *   h      out [m][f] bf16 bit patterns.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_bitlinear_glu(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t f,
                           int64_t k, int8_t* xq, float* alpha, uint16_t* h, void* stream);

/* ---- Straight-through backward ----
 * [P1], section "Training Dynamics: The Straight-Through Estimator": the
 * backward pass treats the rounding step as the identity, so gradients pass
 * through the quantized weights to full-precision shadow weights, which are
 * ternarized again at the next forward pass (bl_ternarize_pack).  Both
 * quantizers are the identity in the backward pass and gamma, alpha are
 * constants; with the dequantized forward y = xhat What^T (xhat = alpha / 127
 * * xq, What = gamma * q):
 *   dx[i][t] = gamma * sum_j dy[i][j] * q[j][t]
 *   dw[j][t] = sum_i dy[i][j] * alpha[i] * xq[i][t] / 127
 * dy is bf16 [m][n]; dx and dw are fp32, accumulated in fp32 in any order
 * (within (n + 2) * 2^-24 * sum |terms| of the exact value for dx). */

/* The packed form of q^T ([k][n], the layout of bl_ternarize_pack with rows t
 * and columns j) from the packed form of q ([n][k]): the operand of
 * bl_bitlinear_backward_x, which contracts over the rows of q.  n must be a
 * positive multiple of 64; packed_t has bl_packed_bytes(k, n) bytes.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_pack_transposed(const uint8_t* packed, int64_t n, int64_t k, uint8_t* packed_t, void* stream);

/* Input gradient dx = gamma * dy q.
 *   packed_t  from bl_pack_transposed of the layer's packed weights; gamma
 *             the layer's gamma (device).
 *   dy        [m][n] bf16 bit patterns (16-byte aligned).
 *   dx        out [m][k] fp32.
 * n must be a multiple of 64 and at most BL_MAX_BACKWARD_N (2^24).
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_bitlinear_backward_x(const uint8_t* packed_t, const float* gamma, const uint16_t* dy, int64_t m,
                                  int64_t n, int64_t k, float* dx, void* stream);

/* Device workspace of bl_bitlinear_backward_w: 2 * (2n + k) * ceil(m/64)*64
 * bytes (the gradient, scaled by alpha and split into two bf16 parts, and the
 * int8 activations as bf16, both stored token-contiguous).  Returns 0 for an
 * invalid shape. */
size_t bl_backward_w_workspace_bytes(int64_t m, int64_t n, int64_t k);

/* Weight gradient for the shadow weights: dw[j][t] = sum_i dy[i][j] *
 * alpha[i] * xq[i][t] / 127.  alpha[i] * dy[i][j] (two bf16 values) is split
 * exactly into two bf16 parts, so every product is exact; the sums are fp32.
 * An alpha with more bits than bf16's (bl_rmsnorm_quant writes such) is taken
 * too: the two parts then hold each product to 2^-17 of it.
 *   dy         [m][n] bf16 bit patterns; xq [m][k] int8 and alpha [m] fp32 as
 *              written by bl_quant_act / bl_bitlinear for the layer's input.
 *   dw         out [n][k] fp32 (overwritten; zero for m = 0).
 *   workspace  device scratch of workspace_bytes >= bl_backward_w_workspace_bytes;
 *              contents on entry do not matter and are clobbered.
 * n must be a multiple of 64 and at most BL_MAX_BACKWARD_N.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_bitlinear_backward_w(const uint16_t* dy, const int8_t* xq, const float* alpha, int64_t m, int64_t n,
                                  int64_t k, float* dw, void* workspace, size_t workspace_bytes, void* stream);

/* Unpack a packed buffer back to trits (test and inspection helper [P2]):
 * q[j][t] in {-1, 0, 1} for the n real rows.  A code 3 (never produced by
 * bl_ternarize_pack) decodes as 0.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_unpack_ternary(const uint8_t* packed, int64_t n, int64_t k, int8_t* q, void* stream);

/* ---- Around the BitLinear layers of a transformer block ----
 * [P2, P3]: the 2B4T block keeps norms, rotary positions and attention around
 * its ternary layers.  The calls below take and give what those layers give
 * and take: bf16 activations, int8 rows with their absmax, fp32 gradients. */

/* Root-mean-square norm of each row, with the residual's addition before it
 * and the int8 quantization that bl_linear expects after it:
 *   h = x + residual (fp32; h = x without one),   r = bf16(h),
 *   n = (h * w) * c,  c = 1 / sqrt(mean_j h_j^2 + eps)       (fp32),
 *   alpha = max_j |n_j|,  s = fl32(127 / max(alpha, 1e-5f)),
 *   xq = round_half_even(fl32(n * s)),
 *   y = bf16(n),   xhat = bf16(xq * fl32(alpha / 127)).
 * The norm and its codes are those of the fp32 sum, not of the rounded r;
 * alpha is the fp32 maximum (bl_quant_act's is a bf16 value, as its input is).
 *   x, residual  [m][k] bf16; residual may be NULL.
 *   weight       [k] fp32.   eps finite, >= 0.  Where mean h^2 + eps is 0 (a row
 *                of zeros without an eps) c is 0, here and in the gradients.
 *   r, y, xhat   out [m][k] bf16, each NULL to skip it; r may be x or residual.
 *   xq, alpha    out [m][k] int8 and [m] fp32, both or neither NULL.
 * At least one output is required.  k is a multiple of 64, at most
 * BL_MAX_NORM_K (a row stays in registers); |h| below 2^56, so that the sum of
 * squares is finite, and, where eps is 0, mean h^2 no fp32 denormal.  x,
 * residual, weight and the [m][k] outputs are 16-byte aligned.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also a bad eps), BL_ERR_ALIGN, BL_ERR_HIP. */
#define BL_MAX_NORM_K 32768
bl_status bl_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const float* weight, int64_t m, int64_t k,
                           float eps, uint16_t* r, uint16_t* y, uint16_t* xhat, int8_t* xq, float* alpha,
                           void* stream);

/* Device workspace of bl_rmsnorm_backward: partial sums of dw.  Returns 0 for
 * an invalid shape. */
size_t bl_rmsnorm_backward_workspace_bytes(int64_t m, int64_t k);

/* Gradients of the norm (the quantizer is the identity in the backward pass,
 * as for bl_bitlinear_backward_x, whose fp32 dx is the dn here):
 *   c = 1 / sqrt(mean_j r_j^2 + eps),
 *   dx = bf16(c * (dn * w - r * c^2 * mean_j(dn_j w_j r_j)) + dr),
 *   dw = sum_i dn_i * r_i * c_i                               (fp32 sums).
 *   dn      [m][k] fp32; r [m][k] bf16, the norm's input as stored (r of the
 *           forward call, or x without a residual).
 *   dr      [m][k] bf16, the gradient that reaches r past the norm, or NULL.
 *   dx      out [m][k] bf16: the gradient of x and of the residual alike; may be dr.
 *   dw      out [k] fp32, 16-byte aligned (overwritten; zero for m = 0).
 * The order of the sums is fixed: equal inputs give equal bits.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_rmsnorm_backward(const float* dn, const uint16_t* r, const float* weight, const uint16_t* dr, int64_t m,
                              int64_t k, float eps, uint16_t* dx, float* dw, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Rotary positions.  Pair i of a head (i < rot / 2) turns by the angle
 * position * f_i:
 *   (a, b) -> magnitude * (a cos - b sin, a sin + b cos),
 * a and b being elements i and i + rot/2 (interleaved = 0) or 2i and 2i + 1
 * (interleaved = 1); elements from rot on pass unchanged.  f_i is held as
 * turns per position in two fp32 numbers (value and remainder), with which the
 * fraction of a turn is right to about 2^-23 for positions below 2^24: cos and
 * sin to 4e-7 in bf16 outputs, to 2^-23 in keys that bl_kv_append quantizes. */
typedef struct bl_rope_table {
    const float* turns; /* device, [rot / 2][2] fp32, as bl_rope_frequencies fills it */
    int64_t rot;        /* even, 0 < rot <= head dimension                           */
    int32_t interleaved;
    float magnitude; /* multiplies both outputs (1 unless a long-context scaling asks for more) */
} bl_rope_table;

/* Table of frequencies (host memory, evaluated in 64 bits):
 *   f_i = base^(-2i / rot), then
 *   BL_ROPE_PLAIN   as it is;
 *   BL_ROPE_LINEAR  f_i / factor (positions interpolated);
 *   BL_ROPE_BASE    base * factor^(rot / (rot - 2)) in base's place (the slowest
 *                   pair is slowed by factor, the fastest not at all; rot > 2);
 *   BL_ROPE_BLEND   with t = original * f_i / 2 pi turns over the original
 *                   length: f_i where t >= fast, f_i / factor where t <= slow,
 *                   and in between the two weighted linearly in t.
 * turns: [rot / 2][2] floats.  Errors: BL_ERR_NULL, BL_ERR_SHAPE (rot odd or
 * not in 2..BL_MAX_HEAD_DIM, a value that is not positive and finite, slow >= fast). */
enum { BL_ROPE_PLAIN = 0, BL_ROPE_LINEAR = 1, BL_ROPE_BASE = 2, BL_ROPE_BLEND = 3 };
#define BL_MAX_HEAD_DIM 256
bl_status bl_rope_frequencies(int64_t rot, double base, int scaling, double factor, double original, double fast,
                              double slow, float* turns);

/* Rotates the heads of every token.
 *   x, y       [tokens][heads][dim] bf16 with strides in elements (multiples of
 *              8; the dim elements of a head are adjacent); y may be x.
 *   position   [tokens] int32 (device).
 *   inverse    non-zero: the transposed rotation, the gradient of the forward
 *              one (the same magnitude).
 * dim: a multiple of 8, at most BL_MAX_HEAD_DIM.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN (also strides), BL_ERR_HIP. */
bl_status bl_rope(const uint16_t* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* position,
                  const bl_rope_table* rope, int64_t tokens, int64_t heads, int64_t dim, int inverse, uint16_t* y,
                  int64_t y_token_stride, int64_t y_head_stride, void* stream);

/* A key/value cache in 8 bits.  A page holds page_tokens consecutive tokens of
 * one sequence; k and v are int8 [pages][heads][page_tokens][dim], k_absmax
 * and v_absmax fp32 [pages][heads]: a code q of a page and head stands for
 * q * absmax / 127.  page_tokens: 16, 32, 64, 128 or 256; dim: a multiple of
 * 16, at most BL_MAX_HEAD_DIM; k and v are 16-byte aligned.  Positions may
 * address more than 2^32 bytes. */
typedef struct bl_kv_cache {
    int8_t* k;
    int8_t* v;
    float* k_absmax;
    float* v_absmax;
    int64_t pages;
    int32_t heads;
    int32_t page_tokens;
    int32_t dim;
} bl_kv_cache;

/* The tokens of one step: tokens offsets[s] .. offsets[s + 1] - 1 belong to
 * sequence s and stand at positions start[s], start[s] + 1, ...; position p of
 * sequence s is token p % page_tokens of page page_table[s][p / page_tokens].
 * max_new and max_len bound offsets[s + 1] - offsets[s] and start[s] +
 * offsets[s + 1] - offsets[s]; max_len <= table_stride * page_tokens.  A page
 * number outside 0 .. pages - 1 marks a page that is not there: nothing is
 * written to it, reading it gives zeros, attention skips it.
 * The host cannot see start and offsets.  Values of them that break these
 * bounds give no error and no access outside a buffer: start is taken as at
 * least 0, a sequence's tokens as at most max_new inside 0 .. tokens - 1,
 * positions past the table as pages that are not there, and attention sees no
 * position from max_len on. */
typedef struct bl_kv_batch {
    const int32_t* page_table; /* device [seqs][table_stride] */
    const int32_t* start;      /* device [seqs], >= 0         */
    const int32_t* offsets;    /* device [seqs + 1], ascending from 0 to tokens */
    int64_t seqs;
    int64_t table_stride;
    int64_t tokens;
    int64_t max_new;
    int64_t max_len;
} bl_kv_batch;

/* Writes the step's keys and values into the cache, quantized on the way.
 * For each page and head that new tokens enter, with a_old its absmax if it
 * holds earlier tokens of the sequence (else 0):
 *   a = max(a_old, max |new values|),  codes of new values
 *   round_half_even(fl32(value * fl32(127 / a))), and, where a > a_old, those
 *   already there become round_half_even(fl32(q * fl32(a_old / a)));
 * pages whose values all stay below 2^-64 are written as zeros with absmax 0.
 * A NaN or an infinity becomes the absmax of its page and head, which then
 * stands for NaN.
 * Writing the same tokens again gives the same cache.  A page that is written
 * must belong to one sequence of the batch only.
 *   k, v   bf16 [tokens][heads][dim], strides in elements (multiples of 8).
 *   rope   NULL, or the rotation that keys take at their positions before they
 *          are quantized (in fp32, without a rounding to bf16 in between).
 *   q      with rope: bf16 [tokens][q_heads][dim], rotated alike into q_out
 *          [tokens][q_heads][dim] bf16 (contiguous; q_out may be q if q is
 *          contiguous too); or NULL.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_append(const bl_kv_cache* cache, const bl_kv_batch* batch, const uint16_t* k, int64_t k_token_stride,
                       int64_t k_head_stride, const uint16_t* v, int64_t v_token_stride, int64_t v_head_stride,
                       const bl_rope_table* rope, const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                       int64_t q_heads, uint16_t* q_out, void* stream);

/* Reads the batch's tokens back: bf16(q * fl32(absmax / 127)), zeros where the
 * page is not there.   k, v  out bf16 [tokens][heads][dim], contiguous.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_read(const bl_kv_cache* cache, const bl_kv_batch* batch, uint16_t* k, uint16_t* v, void* stream);

/* Device workspace of bl_attention (0: none is needed, or an argument is invalid). */
size_t bl_attention_workspace_bytes(const bl_kv_cache* cache, const bl_kv_batch* batch, int64_t q_heads);

/* Attention of the step's queries over the cache, which already holds the
 * step's own tokens (bl_kv_append):
 *   out = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
 * over the positions j <= p of its sequence, p being the query's own; with
 * window > 0 only those with p - j < window or j < sinks.  Query head h reads
 * cache head h / (q_heads / heads).  A query that sees nothing (its pages are
 * not there) gives zeros; one that holds a NaN or an infinity, or sees a page
 * with such an absmax, gives NaN.
 *   q      bf16 [tokens][q_heads][dim], strides in elements (multiples of 8).
 *   out    bf16 [tokens][q_heads][dim], contiguous.
 *   lse    NULL, or out fp32 [tokens][q_heads]: log sum_j exp(scale * q . k_j)
 *          (-inf for a query that sees nothing).
 * Keys are read as stored; a query row enters the products as 16-bit integers
 * relative to its absmax; softmax statistics and sums are fp32; the weights
 * enter the product with v in fp16, scaled so that none above 2^-28 of the
 * row's largest contribution (weight times absmax of its page) loses precision.
 * An absmax of v below 2^-64, such as a page of zeros has, counts as 2^-64.
 * The result does not depend on the order in which workgroups run.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also q_heads no multiple of heads, sinks
 * without a window, scale not finite), BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_attention(const bl_kv_cache* cache, const bl_kv_batch* batch, const uint16_t* q, int64_t q_token_stride,
                       int64_t q_head_stride, int64_t q_heads, float scale, int64_t window, int64_t sinks,
                       uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Many answers to one prompt: pages of the cache ----
 * refs[p] counts the entries of page tables that hold page p; 0: the page is
 * free.  Sequences that begin alike may hold the same pages there (bl_kv_fork);
 * a page that is written (bl_kv_append) belongs to one sequence.  A new pool is all zeros.
 * One pool serves the caches of all blocks, which use the same page numbers.
 * A page number outside 0 .. pages - 1 in a table marks an entry without a
 * page (the calls below write -1).
 * Pages are handed out lowest number first, to requests in the order of
 * sequences and, within one, of positions: equal inputs give equal results.
 * shortage: NULL, or a device integer to which the number of requests that
 * found no free page is added (their entries stay, or become, -1, but for
 * those of shared pages in bl_kv_grow); the host clears it.  Counts that do not agree with the tables give no access outside
 * a buffer; no count goes below 0. */
#define BL_MAX_POOL_PAGES (1 << 24)
#define BL_MAX_FORK_SEQS 8192
typedef struct bl_kv_pool {
    int32_t* refs;       /* device [pages], 16-byte aligned    */
    int64_t pages;       /* 1 .. BL_MAX_POOL_PAGES             */
    int32_t page_tokens; /* tokens per page, as in the caches  */
} bl_kv_pool;

/* Gives pages to the entries without one in which the batch's new tokens
 * stand (positions start[s] .. start[s] + offsets[s + 1] - offsets[s] - 1):
 * call it before bl_kv_append.  page_table is written; entries past
 * table_stride get none and are not counted as a shortage.
 *   copies  NULL, or out device [seqs][3] for bl_kv_copy: a part-filled page in
 *           which a sequence goes on writing (position start[s]) and that others
 *           hold too is copied onto a fresh one, {source, target, tokens},
 *           {-1, -1, 0} elsewhere; of sequences of the batch that write in it, the
 *           last one keeps it if nobody else holds it then.  Such pages come from
 *           cutting back (bl_kv_free with keep) into pages that a fork shares.
 *           Where no page was free for a copy the entry stays as it is, shared,
 *           and copies has {source, -1, 0}, which bl_kv_copy passes over: such a
 *           sequence must not be written.  That is so for the last one too if one
 *           before it got no copy.  Each of them is counted in shortage; once pages
 *           are free again, the same call goes on from there.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also when sequences times the pages that
 * max_new tokens may enter pass 2^24, or seqs passes BL_MAX_FORK_SEQS with
 * copies), BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_grow(const bl_kv_pool* pool, const bl_kv_batch* batch, int32_t* copies, int32_t* shortage, void* stream);

/* Forks sequences: child c continues parent p = parent[c], which holds
 * length[p] tokens (taken as 0 .. table_stride * page_tokens).  The child
 * shares the parent's full pages; the last, part-filled one is copied onto a
 * fresh page: copies[c] = {source, target, tokens} for bl_kv_copy, {-1, -1, 0}
 * where nothing is to be copied.  Entries past length[p] are -1.  A parent[c]
 * outside 0 .. seqs - 1 makes an empty child: no page, length 0.
 *   keep_parents  non-zero: the parents keep their rows and pages.  0: they are
 *                 given up (beams): the first child of a parent takes its
 *                 part-filled page over as it is, and pages that no child holds
 *                 become free once the call is done (it hands out none of them
 *                 itself).  `table` is not changed, its rows mean nothing then.
 *   table         device [seqs][table_stride]; length device [seqs].
 *   parent        device [children].
 *   table_out     out device [children][table_stride].
 *   length_out    out device [children]: the parents' lengths.
 *   copies        out device [children][3].
 * seqs and children are at most BL_MAX_FORK_SEQS.  The outputs share no element
 * with each other or with what else the call reads or writes.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also outputs that share elements),
 * BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_fork(const bl_kv_pool* pool, const int32_t* table, int64_t table_stride, const int32_t* length,
                     int64_t seqs, const int32_t* parent, int64_t children, int keep_parents, int32_t* table_out,
                     int32_t* length_out, int32_t* copies, int32_t* shortage, void* stream);

/* Gives pages back: row s of table keeps those of its first keep[s] tokens
 * (none if keep is NULL or keep[s] < 1), the entries past them become -1 and
 * their pages lose a holder.
 *   table  device [seqs][table_stride]; keep device [seqs] or NULL.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_free(const bl_kv_pool* pool, int32_t* table, int64_t table_stride, int64_t seqs, const int32_t* keep,
                     void* stream);

/* Device workspace of bl_kv_compact (0: an argument is invalid). */
size_t bl_kv_compact_workspace_bytes(const bl_kv_pool* pool, int64_t moves);

/* Moves used pages to the front: with n pages in use, the highest used page
 * goes to the lowest free one below n, the second highest to the second lowest
 * and so on, at most `moves` of them (0 .. pages); then refs and the entries of table are
 * changed accordingly.  After as many moves as there are, pages 0 .. n - 1
 * are in use and the rest is free.  The codes are moved by bl_kv_copy with
 * copies and moved, before the next call that writes a cache.
 *   table   device [seqs][table_stride]: every row that holds pages of the pool.
 *   copies  out device [moves][3]: {source, target, page_tokens}, then {-1, -1, 0}.
 *   moved   out device [1]: how many there are.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE, BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_kv_compact(const bl_kv_pool* pool, int32_t* table, int64_t table_stride, int64_t seqs, int64_t moves,
                        int32_t* copies, int32_t* moved, void* workspace, size_t workspace_bytes, void* stream);

/* Copies pages inside each of `count` caches (one per block of a model, all of
 * one shape): for every {source, target, tokens} of copies the codes of the
 * first `tokens` tokens of all heads (at most page_tokens) and the scales; the
 * target's other tokens stay as they are and mean nothing.  Entries whose
 * pages are not there, or that have no tokens, are skipped.  The copies are
 * made at once: no target is a source or another target.
 *   caches  host array; copies device [n][3];
 *   valid   NULL, or a device integer: only that many entries are looked at.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also caches of different shapes), BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_kv_copy(const bl_kv_cache* caches, int64_t count, const int32_t* copies, int64_t n, const int32_t* valid,
                     void* stream);

/* Sequences that begin alike: sequences group[g] .. group[g + 1] - 1 share
 * their first prefix[g] tokens, which the pages of the first of them hold (the
 * others' entries for them need not name the same pages, if theirs hold the
 * same tokens).  No prefix[g] passes the start of one of its sequences.
 * max_group bounds group[g + 1] - group[g], max_prefix the prefixes.  Values
 * that break these bounds, or those of bl_kv_batch, give no error and no access
 * outside a buffer; the outputs of their group mean nothing then, nor do those
 * of sequences in no group. */
typedef struct bl_kv_shared {
    const int32_t* group;  /* device [groups + 1], ascending from 0 to seqs */
    const int32_t* prefix; /* device [groups]                               */
    int64_t groups;
    int64_t max_group;
    int64_t max_prefix;
} bl_kv_shared;

/* Device workspace of bl_attention_shared (0: none is needed, or an argument is invalid). */
size_t bl_attention_shared_workspace_bytes(const bl_kv_cache* cache, const bl_kv_batch* batch,
                                           const bl_kv_shared* shared, int64_t q_heads);

/* bl_attention without a window for such a batch: the keys and values of a
 * prefix are read for all queries of its group together, where the bounds
 * make that worth its while (short prefixes, and prompts whose rows fill tiles
 * of their own, are taken as bl_attention takes them).  The results are those
 * of bl_attention but for the order of the sums.  (A window leaves little of a
 * long prefix to see: bl_attention reads no more than that.)
 *   q, out, lse  as for bl_attention.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also groups * max_group below seqs, a
 * max_prefix past max_len), BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_attention_shared(const bl_kv_cache* cache, const bl_kv_batch* batch, const bl_kv_shared* shared,
                              const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                              float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ---- Log probabilities ----
 * Of the rows of logits x [m][n], with z_j = scale * x_j:
 *   lse = log sum_j exp z_j,   logprob = z_t - lse  for the given token t,
 *   entropy = -sum_j p_j log p_j,  p_j = exp(z_j - lse),
 *   top_id, top_logprob: the `top` largest logits and their log
 *   probabilities, in descending order, equal ones by ascending index.
 * A logit of -infinity is a token that cannot occur: its p is 0, it is no
 * alternative.  Where fewer than `top` tokens can occur, the rest of the row
 * is -1 and -infinity.  Where none can, lse and logprob are -infinity and the
 * entropy is 0.  A target outside 0 .. n - 1 has logprob 0 and no gradient.  A
 * row that holds a NaN or +infinity gives NaN, NaNs are no alternatives.
 * Statistics and sums are fp32; products scale * x must be finite where x is. */
#define BL_MAX_VOCABULARY (1 << 20)
#define BL_MAX_TOP 64
enum { BL_BF16 = 0, BL_FP32 = 1 };

/* Device workspace of bl_logprobs (0: none is needed, or an argument is invalid). */
size_t bl_logprobs_workspace_bytes(int64_t m, int64_t n, int type, int64_t top);

/*   x        [m][n] bf16 or fp32 (type), rows row_stride elements apart (>= n); aligned to its elements only.
 *   scale    > 0, at most 2^127: 1 / temperature.
 *   target   [m] int32, needed for logprob only.
 *   logprob, lse, entropy  out fp32 [m], each NULL to skip it.
 *   top      0 .. BL_MAX_TOP; top_id out int32 [m][top], top_logprob out fp32 [m][top].
 * At least one output is required; n is at most BL_MAX_VOCABULARY.
 * Results do not depend on the order in which workgroups run.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also a bad type or scale), BL_ERR_ALIGN, BL_ERR_WORKSPACE, BL_ERR_HIP. */
bl_status bl_logprobs(const void* x, int type, int64_t m, int64_t n, int64_t row_stride, float scale,
                      const int32_t* target, int64_t top, float* logprob, float* lse, float* entropy, int32_t* top_id,
                      float* top_logprob, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of sum_i (dlogprob_i logprob_i + dentropy_i entropy_i + dlse_i lse_i):
 *   dx_j = scale * (dlogprob ([j = t] - p_j) + dlse p_j - dentropy p_j (log p_j + entropy)),
 * from the logits and the lse and entropy that bl_logprobs gave for them.  Where
 * |lse| is 64 or more (fp32; 512 for bf16) its rounding would show in every p: the
 * row's sum is taken again then, by one workgroup per row.
 *   dlogprob (with target), dentropy (with entropy), dlse  fp32 [m], each NULL
 *            for zeros, not all.  A row whose gradients are all zero (or where
 *            no token can occur) gets zeros whatever its logits are.
 *   dx       out [m][n] of x's type, rows dx_stride elements apart; may be x
 *            (with dx_stride = row_stride), and has no element of x otherwise.
 *            Between rows nothing is written.
 * Errors: BL_ERR_NULL, BL_ERR_SHAPE (also rows of dx that begin inside those of
 * x, of the same stride), BL_ERR_ALIGN, BL_ERR_HIP. */
bl_status bl_logprobs_backward(const void* x, int type, int64_t m, int64_t n, int64_t row_stride, float scale,
                               const int32_t* target, const float* lse, const float* entropy, const float* dlogprob,
                               const float* dentropy, const float* dlse, void* dx, int64_t dx_stride, void* stream);

/* Static, human-readable name of a status code. */
const char* bl_status_string(bl_status s);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_H */
