// C ABI of the BitLinear W1.58A8 library: argument validation and dispatch.
// Declarations, argument meaning, layouts and error behaviour: include/bitlinear.h.
#include "../../include/bitlinear.h"
#include "internal.h"

#include <math.h>

namespace {

constexpr int64_t kLimit40 = (int64_t)1 << 40;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool valid_k(int64_t k) { return k >= 64 && k <= BL_MAX_K && k % 64 == 0; }

bool product_ok(int64_t a, int64_t b) { return a == 0 || b < kLimit40 / a; }

// A launch grid beyond the device's work-item limit is a shape error (the
// launchers detect it before any HIP call); any other failure is the runtime's.
bl_status from_hip(hipError_t e) {
  return e == hipSuccess ? BL_OK : e == bl::kErrGridTooLarge ? BL_ERR_SHAPE : BL_ERR_HIP;
}

// Largest weight count the packer takes: its grid covers n * k / 16 work-items.
constexpr int64_t kMaxPackWeights = (int64_t)1 << 35;

}  // namespace

extern "C" {

size_t bl_packed_bytes(int64_t n, int64_t k) {
  if (n < 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k)) return 0;
  return (size_t)((n + 15) / 16 * 16) * (size_t)(k / 4);
}

size_t bl_ternarize_pack_workspace_bytes(int64_t n, int64_t k) {
  if (n < 1 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k)) return 0;
  return bl::kPackWorkspaceBytes;
}

bl_status bl_ternarize_pack(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!w || !packed || !gamma || !workspace) return BL_ERR_NULL;
  if (n < 1 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k) || n * k > kMaxPackWeights) return BL_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(gamma, 4) || !aligned(workspace, 16)) return BL_ERR_ALIGN;
  if (workspace_bytes < bl_ternarize_pack_workspace_bytes(n, k)) return BL_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  unsigned long long* bins = (unsigned long long*)workspace;
  hipError_t e = bl::launch_absmean_bins(w, n * k, bins, s);
  if (e == hipSuccess) e = bl::launch_gamma_fold(bins, n * k, gamma, s);
  if (e == hipSuccess) e = bl::launch_ternarize_pack(w, n, k, gamma, packed, s);
  return from_hip(e);
}

bl_status bl_ternarize_pack_noalloc(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma,
                                    void* stream) {
  if (!w || !packed || !gamma) return BL_ERR_NULL;
  if (n < 1 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k) || n * k > kMaxPackWeights) return BL_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(gamma, 4)) return BL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  unsigned long long* bins = nullptr;  // the static array's device address, never its host-side name
  hipError_t e = bl::static_pack_bins(s, &bins);
  if (e == hipSuccess) e = bl::launch_absmean_bins(w, n * k, bins, s);
  if (e == hipSuccess) e = bl::launch_gamma_fold(bins, n * k, gamma, s);
  if (e == hipSuccess) e = bl::launch_ternarize_pack(w, n, k, gamma, packed, s);
  return from_hip(e);
}

size_t bl_packed_bytes_b3(int64_t n, int64_t k) {
  if (n < 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k)) return 0;
  return bl::packed_bytes_b3(n, k);
}

bl_status bl_ternarize_pack_b3(const float* w, int64_t n, int64_t k, uint8_t* packed, float* gamma, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (!w || !packed || !gamma || !workspace) return BL_ERR_NULL;
  if (n < 1 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k) || n * k > kMaxPackWeights) return BL_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(gamma, 4) || !aligned(workspace, 16)) return BL_ERR_ALIGN;
  if (workspace_bytes < bl_ternarize_pack_workspace_bytes(n, k)) return BL_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  unsigned long long* bins = (unsigned long long*)workspace;
  hipError_t e = bl::launch_absmean_bins(w, n * k, bins, s);
  if (e == hipSuccess) e = bl::launch_gamma_fold(bins, n * k, gamma, s);
  if (e == hipSuccess) e = bl::launch_ternarize_pack_b3(w, n, k, gamma, packed, s);
  return from_hip(e);
}

bl_status bl_bitlinear_b3(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t n,
                          int64_t k, int8_t* xq, float* alpha, int32_t* acc, uint16_t* y, void* stream) {
  if (m < 0 || m > BL_B3_MAX_M || n < 0 || n > BL_MAX_N || !valid_k(k) || k > BL_B3_MAX_K || !product_ok(n + 16, k))
    return BL_ERR_SHAPE;
  if (m == 0 || n == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!packed || !gamma || !x || !xq || !alpha || (!acc && !y)) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(xq, 16) || !aligned(gamma, 4) || !aligned(alpha, 4) ||
      (acc && !aligned(acc, 4)) || (y && !aligned(y, 2)))
    return BL_ERR_ALIGN;
  return from_hip(bl::launch_bitlinear_b3(packed, gamma, x, m, n, k, xq, alpha, acc, y, (hipStream_t)stream));
}

bl_status bl_quant_act(const uint16_t* x, int64_t m, int64_t k, int8_t* xq, float* alpha, void* stream) {
  if (m < 0 || m > BL_MAX_M || !valid_k(k) || !product_ok(m, k)) return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || !xq || !alpha) return BL_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(alpha, 4)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_quant_act(x, m, k, xq, alpha, (hipStream_t)stream));
}

bl_status bl_linear(const uint8_t* packed, const float* gamma, const int8_t* xq, const float* alpha, int64_t m,
                    int64_t n, int64_t k, int32_t* acc, uint16_t* y, void* stream) {
  if (m < 0 || m > BL_MAX_M || n < 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(m, k) || !product_ok(n + 16, k) ||
      !product_ok(m, n))
    return BL_ERR_SHAPE;
  if (m == 0 || n == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!packed || !gamma || !xq || !alpha || (!acc && !y)) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(xq, 16) || !aligned(gamma, 4) || !aligned(alpha, 4) ||
      (acc && !aligned(acc, 4)) || (y && !aligned(y, 2)))
    return BL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  if (bl::gemv_serves(m, n)) return from_hip(bl::launch_gemv(packed, gamma, xq, alpha, m, n, k, acc, y, s));
  return from_hip(bl::launch_gemm(packed, gamma, xq, alpha, m, n, k, acc, y, s));
}

bl_status bl_bitlinear(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t n, int64_t k,
                       int8_t* xq, float* alpha, int32_t* acc, uint16_t* y, void* stream) {
  if (m < 0 || m > BL_MAX_M || n < 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(m, k) || !product_ok(n + 16, k) ||
      !product_ok(m, n))
    return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || !xq || !alpha || (n > 0 && (!packed || !gamma || (!acc && !y)))) return BL_ERR_NULL;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(alpha, 4) || (n > 0 && (!aligned(packed, 16) ||
      !aligned(gamma, 4) || (acc && !aligned(acc, 4)) || (y && !aligned(y, 2)))))
    return BL_ERR_ALIGN;
  if (n > 0 && !bl::gemv_serves(m, n) && !bl::gemm_fits(m, n)) return BL_ERR_SHAPE;  // before the quantizer runs
  hipStream_t s = (hipStream_t)stream;
  if (n > 0 && bl::gemv_fused_applies(m, n, k))
    return from_hip(bl::launch_gemv_fused(packed, gamma, x, m, n, k, xq, alpha, acc, y, s));
  hipError_t e = bl::launch_quant_act(x, m, k, xq, alpha, s);
  if (e != hipSuccess || n == 0) return from_hip(e);
  if (bl::gemv_serves(m, n)) return from_hip(bl::launch_gemv(packed, gamma, xq, alpha, m, n, k, acc, y, s));
  return from_hip(bl::launch_gemm(packed, gamma, xq, alpha, m, n, k, acc, y, s));
}

bl_status bl_ternarize_pack_glu(const float* w, int64_t f, int64_t k, uint8_t* packed, float* gamma, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!w || !packed || !gamma || !workspace) return BL_ERR_NULL;
  if (f < 16 || f % 16 != 0 || 2 * f > BL_MAX_N || !valid_k(k) || !product_ok(2 * f + 16, k) ||
      2 * f * k > kMaxPackWeights)
    return BL_ERR_SHAPE;
  if (!aligned(w, 16) || !aligned(packed, 16) || !aligned(gamma, 4) || !aligned(workspace, 16)) return BL_ERR_ALIGN;
  if (workspace_bytes < bl_ternarize_pack_workspace_bytes(2 * f, k)) return BL_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  unsigned long long* bins = (unsigned long long*)workspace;
  hipError_t e = bl::launch_absmean_bins(w, 2 * f * k, bins, s);
  if (e == hipSuccess) e = bl::launch_gamma_fold(bins, 2 * f * k, gamma, s);
  if (e == hipSuccess) e = bl::launch_ternarize_pack(w, 2 * f, k, gamma, packed, s, f);
  return from_hip(e);
}

namespace {

bl_status check_glu_product(int64_t m, int64_t f, int64_t k) {
  if (m < 0 || m > BL_MAX_M || f < 16 || f % 16 != 0 || 2 * f > BL_MAX_N || !valid_k(k) || !product_ok(m, k) ||
      !product_ok(2 * f + 16, k) || !product_ok(m, 2 * f))
    return BL_ERR_SHAPE;
  return BL_OK;
}

}  // namespace

bl_status bl_linear_glu(const uint8_t* packed, const float* gamma, const int8_t* xq, const float* alpha, int64_t m,
                        int64_t f, int64_t k, uint16_t* h, void* stream) {
  if (bl_status st = check_glu_product(m, f, k)) return st;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!packed || !gamma || !xq || !alpha || !h) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(xq, 16) || !aligned(gamma, 4) || !aligned(alpha, 4) || !aligned(h, 2))
    return BL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  if (bl::gemv_serves(m, 2 * f)) return from_hip(bl::launch_gemv_glu(packed, gamma, xq, alpha, m, f, k, h, s));
  return from_hip(bl::launch_gemm_glu(packed, gamma, xq, alpha, m, f, k, h, s));
}

bl_status bl_bitlinear_glu(const uint8_t* packed, const float* gamma, const uint16_t* x, int64_t m, int64_t f,
                           int64_t k, int8_t* xq, float* alpha, uint16_t* h, void* stream) {
  if (bl_status st = check_glu_product(m, f, k)) return st;
  if (m == 0) return BL_OK;
  if (!packed || !gamma || !x || !xq || !alpha || !h) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(xq, 16) || !aligned(gamma, 4) || !aligned(alpha, 4) ||
      !aligned(h, 2))
    return BL_ERR_ALIGN;
  if (!bl::gemv_serves(m, 2 * f) && !bl::gemm_fits(m, 2 * f)) return BL_ERR_SHAPE;  // before the quantizer runs
  hipStream_t s = (hipStream_t)stream;
  if (bl::gemv_fused_glu_applies(m, f, k))
    return from_hip(bl::launch_gemv_fused_glu(packed, gamma, x, m, f, k, xq, alpha, h, s));
  hipError_t e = bl::launch_quant_act(x, m, k, xq, alpha, s);
  if (e != hipSuccess) return from_hip(e);
  if (bl::gemv_serves(m, 2 * f)) return from_hip(bl::launch_gemv_glu(packed, gamma, xq, alpha, m, f, k, h, s));
  return from_hip(bl::launch_gemm_glu(packed, gamma, xq, alpha, m, f, k, h, s));
}

bl_status bl_pack_transposed(const uint8_t* packed, int64_t n, int64_t k, uint8_t* packed_t, void* stream) {
  if (n < 64 || n % 64 != 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k)) return BL_ERR_SHAPE;
  if (!packed || !packed_t) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(packed_t, 16)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_pack_transposed(packed, n, k, packed_t, (hipStream_t)stream));
}

bl_status bl_bitlinear_backward_x(const uint8_t* packed_t, const float* gamma, const uint16_t* dy, int64_t m,
                                  int64_t n, int64_t k, float* dx, void* stream) {
  if (m < 0 || m > BL_MAX_M || n < 64 || n % 64 != 0 || n > BL_MAX_BACKWARD_N || !valid_k(k) || !product_ok(m, n) ||
      !product_ok(m, k) || !product_ok(n + 16, k))
    return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;
  if (!packed_t || !gamma || !dy || !dx) return BL_ERR_NULL;
  if (!aligned(packed_t, 16) || !aligned(gamma, 4) || !aligned(dy, 16) || !aligned(dx, 4)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_backward_x(packed_t, gamma, dy, m, n, k, dx, (hipStream_t)stream));
}

size_t bl_backward_w_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 1 || m > BL_MAX_M || n < 64 || n % 64 != 0 || n > BL_MAX_BACKWARD_N || !valid_k(k) || !product_ok(m + 64, n) ||
      !product_ok(m + 64, k))
    return 0;
  return bl::backward_w_workspace_bytes(m, n, k);
}

bl_status bl_bitlinear_backward_w(const uint16_t* dy, const int8_t* xq, const float* alpha, int64_t m, int64_t n,
                                  int64_t k, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
  if (m < 0 || m > BL_MAX_M || n < 64 || n % 64 != 0 || n > BL_MAX_BACKWARD_N || !valid_k(k) || !product_ok(m + 64, n) ||
      !product_ok(m + 64, k) || !product_ok(n, k))
    return BL_ERR_SHAPE;
  if (!dy && m > 0) return BL_ERR_NULL;
  if (!dw || (m > 0 && (!xq || !alpha || !workspace))) return BL_ERR_NULL;
  if (!aligned(dy, 2) || !aligned(alpha, 4) || !aligned(dw, 4) || !aligned(workspace, 16)) return BL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  if (m == 0) return from_hip(bl::launch_fill_zero(dw, n * k, s));  // empty sum
  if (workspace_bytes < bl::backward_w_workspace_bytes(m, n, k)) return BL_ERR_WORKSPACE;
  return from_hip(bl::launch_backward_w(dy, xq, alpha, m, n, k, dw, workspace, s));
}

bl_status bl_unpack_ternary(const uint8_t* packed, int64_t n, int64_t k, int8_t* q, void* stream) {
  if (n < 0 || n > BL_MAX_N || !valid_k(k) || !product_ok(n + 16, k)) return BL_ERR_SHAPE;
  if (n == 0) return BL_OK;
  if (!packed || !q) return BL_ERR_NULL;
  if (!aligned(packed, 16) || !aligned(q, 16)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_unpack(packed, n, k, q, (hipStream_t)stream));
}

bl_status bl_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const float* weight, int64_t m, int64_t k,
                           float eps, uint16_t* r, uint16_t* y, uint16_t* xhat, int8_t* xq, float* alpha,
                           void* stream) {
  if (m < 0 || m > BL_MAX_M || !valid_k(k) || k > BL_MAX_NORM_K || !(eps >= 0.0f && eps < INFINITY)) return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || !weight || (!r && !y && !xhat && !xq) || (!xq != !alpha)) return BL_ERR_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(r, 16) || !aligned(y, 16) ||
      !aligned(xhat, 16) || !aligned(xq, 16) || !aligned(alpha, 4))
    return BL_ERR_ALIGN;
  return from_hip(bl::launch_rmsnorm_quant(x, residual, weight, m, k, eps, r, y, xhat, xq, alpha, (hipStream_t)stream));
}

size_t bl_rmsnorm_backward_workspace_bytes(int64_t m, int64_t k) {
  if (m < 1 || m > BL_MAX_M || !valid_k(k) || k > BL_MAX_NORM_K) return 0;
  return bl::rmsnorm_backward_workspace_bytes(m, k);
}

bl_status bl_rmsnorm_backward(const float* dn, const uint16_t* r, const float* weight, const uint16_t* dr, int64_t m,
                              int64_t k, float eps, uint16_t* dx, float* dw, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (m < 0 || m > BL_MAX_M || !valid_k(k) || k > BL_MAX_NORM_K || !(eps >= 0.0f && eps < INFINITY)) return BL_ERR_SHAPE;
  if (!dw || (m > 0 && (!dn || !r || !weight || !dx || !workspace))) return BL_ERR_NULL;
  if (!aligned(dn, 16) || !aligned(r, 16) || !aligned(weight, 16) || !aligned(dr, 16) || !aligned(dx, 16) ||
      !aligned(dw, 16) || !aligned(workspace, 16))
    return BL_ERR_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  if (m == 0) return from_hip(bl::launch_fill_zero(dw, k, s));  // empty sum
  if (workspace_bytes < bl::rmsnorm_backward_workspace_bytes(m, k)) return BL_ERR_WORKSPACE;
  return from_hip(bl::launch_rmsnorm_backward(dn, r, weight, dr, m, k, eps, dx, dw, workspace, s));
}

bl_status bl_rope_frequencies(int64_t rot, double base, int scaling, double factor, double original, double fast,
                              double slow, float* turns) {
  auto good = [](double v) { return v > 0.0 && v < INFINITY; };
  if (rot < 2 || rot % 2 != 0 || rot > BL_MAX_HEAD_DIM || !good(base) || scaling < BL_ROPE_PLAIN ||
      scaling > BL_ROPE_BLEND || (scaling != BL_ROPE_PLAIN && !good(factor)) || (scaling == BL_ROPE_BASE && rot == 2) ||
      (scaling == BL_ROPE_BLEND && (!good(original) || !good(fast) || !good(slow) || slow >= fast)))
    return BL_ERR_SHAPE;
  if (!turns) return BL_ERR_NULL;
  const double two_pi = 6.283185307179586476925;
  if (scaling == BL_ROPE_BASE) base *= pow(factor, (double)rot / (double)(rot - 2));
  for (int64_t i = 0; i < rot / 2; ++i) {
    double t = pow(base, -2.0 * (double)i / (double)rot) / two_pi;  // turns per position
    if (scaling == BL_ROPE_LINEAR) t /= factor;
    if (scaling == BL_ROPE_BLEND) {
      const double keep = (original * t - slow) / (fast - slow);
      t *= keep >= 1.0 ? 1.0 : keep <= 0.0 ? 1.0 / factor : keep + (1.0 - keep) / factor;
    }
    turns[2 * i] = (float)t;
    turns[2 * i + 1] = (float)(t - (double)turns[2 * i]);
  }
  return BL_OK;
}

namespace {

bl_status check_rope(const bl_rope_table* rope, int64_t dim) {
  if (rope->rot < 2 || rope->rot % 2 != 0 || rope->rot > dim || !(fabsf(rope->magnitude) < INFINITY)) return BL_ERR_SHAPE;
  return BL_OK;
}

bool strides_ok(int64_t token, int64_t head) { return token % 8 == 0 && head % 8 == 0; }

// The kernels count tokens, positions and heads in 32 bits.
constexpr int64_t kMaxPositions = (int64_t)1 << 29;

bool page_tokens_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

bl_status check_cache(const bl_kv_cache* c) {
  if (c->heads < 1 || c->heads > 65536 || !page_tokens_ok(c->page_tokens) || c->dim < 16 || c->dim > BL_MAX_HEAD_DIM ||
      c->dim % 16 != 0 || c->pages < 1 || c->pages > 0x7FFFFFFF ||
      !product_ok(c->pages, (int64_t)c->heads * c->page_tokens * c->dim))
    return BL_ERR_SHAPE;
  return BL_OK;
}

bl_status check_cache_pointers(const bl_kv_cache* c) {
  if (!c->k || !c->v || !c->k_absmax || !c->v_absmax) return BL_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_absmax, 4) || !aligned(c->v_absmax, 4)) return BL_ERR_ALIGN;
  return BL_OK;
}

bl_status check_kv(const bl_kv_cache* c, const bl_kv_batch* b) {
  if (!c || !b) return BL_ERR_NULL;
  const int p = c->page_tokens;
  if (bl_status st = check_cache(c)) return st;
  if (b->seqs < 0 || b->seqs > 65535 || b->tokens < 0 || b->tokens > kMaxPositions || b->max_new < 0 ||
      b->max_new > b->tokens || b->max_len < b->max_new || b->max_len > kMaxPositions || b->table_stride < 0 ||
      b->table_stride > 0x7FFFFFFF || b->max_len > b->table_stride * p)
    return BL_ERR_SHAPE;
  if (b->seqs == 0 || b->tokens == 0 || b->max_new == 0) return BL_OK;
  if (!b->page_table || !b->start || !b->offsets) return BL_ERR_NULL;
  if (bl_status st = check_cache_pointers(c)) return st;
  if (!aligned(b->page_table, 4) || !aligned(b->start, 4) || !aligned(b->offsets, 4)) return BL_ERR_ALIGN;
  return BL_OK;
}

bool nothing_new(const bl_kv_batch* b) { return b->seqs == 0 || b->tokens == 0 || b->max_new == 0; }

bool q_heads_ok(int64_t q_heads) { return q_heads >= 1 && q_heads <= 65536; }

bl::KvView view(const bl_kv_cache* c) {
  bl::KvView kv;
  kv.k = c->k;
  kv.v = c->v;
  kv.k_absmax = c->k_absmax;
  kv.v_absmax = c->v_absmax;
  kv.pages = c->pages;
  kv.heads = c->heads;
  kv.page_tokens = c->page_tokens;
  kv.dim = c->dim;
  return kv;
}

bl::KvStep step_of(const bl_kv_batch* b) {
  bl::KvStep st;
  st.page_table = b->page_table;
  st.start = b->start;
  st.offsets = b->offsets;
  st.table_stride = b->table_stride;
  st.tokens = (int)b->tokens;
  st.max_new = (int)b->max_new;
  return st;
}

}  // namespace

bl_status bl_rope(const uint16_t* x, int64_t x_token_stride, int64_t x_head_stride, const int32_t* position,
                  const bl_rope_table* rope, int64_t tokens, int64_t heads, int64_t dim, int inverse, uint16_t* y,
                  int64_t y_token_stride, int64_t y_head_stride, void* stream) {
  if (!rope) return BL_ERR_NULL;
  if (tokens < 0 || tokens > kMaxPositions || heads < 0 || heads > 65536 || dim < 8 || dim > BL_MAX_HEAD_DIM || dim % 8 != 0)
    return BL_ERR_SHAPE;
  if (bl_status st = check_rope(rope, dim)) return st;
  if (tokens == 0 || heads == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || !position || !rope->turns || !y) return BL_ERR_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(position, 4) || !aligned(rope->turns, 16) ||
      !strides_ok(x_token_stride, x_head_stride) || !strides_ok(y_token_stride, y_head_stride))
    return BL_ERR_ALIGN;
  return from_hip(bl::launch_rope(x, x_token_stride, x_head_stride, position, rope->turns, (int)rope->rot,
                                  rope->interleaved != 0, rope->magnitude, tokens, (int)heads, (int)dim, inverse != 0, y,
                                  y_token_stride, y_head_stride, (hipStream_t)stream));
}

bl_status bl_kv_append(const bl_kv_cache* cache, const bl_kv_batch* batch, const uint16_t* k, int64_t k_token_stride,
                       int64_t k_head_stride, const uint16_t* v, int64_t v_token_stride, int64_t v_head_stride,
                       const bl_rope_table* rope, const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                       int64_t q_heads, uint16_t* q_out, void* stream) {
  if (bl_status st = check_kv(cache, batch)) return st;
  if (rope) {
    if (bl_status st = check_rope(rope, cache->dim)) return st;
  }
  if (q && !q_heads_ok(q_heads)) return BL_ERR_SHAPE;
  if (nothing_new(batch)) return BL_OK;  // empty tensors may carry NULL pointers
  if (!k || !v || (rope && !rope->turns) || (q && (!rope || !q_out))) return BL_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_token_stride, k_head_stride) ||
      !strides_ok(v_token_stride, v_head_stride) || (rope && !aligned(rope->turns, 16)) ||
      (q && (!aligned(q, 16) || !aligned(q_out, 16) || !strides_ok(q_token_stride, q_head_stride))))
    return BL_ERR_ALIGN;
  return from_hip(bl::launch_kv_append(view(cache), step_of(batch), batch->seqs, batch->max_new, k, k_token_stride,
                                       k_head_stride, v, v_token_stride, v_head_stride, rope ? rope->turns : nullptr,
                                       rope ? (int)rope->rot : 0, rope && rope->interleaved != 0,
                                       rope ? rope->magnitude : 1.0f, q, q_token_stride, q_head_stride, (int)q_heads,
                                       q_out, (hipStream_t)stream));
}

bl_status bl_kv_read(const bl_kv_cache* cache, const bl_kv_batch* batch, uint16_t* k, uint16_t* v, void* stream) {
  if (bl_status st = check_kv(cache, batch)) return st;
  if (nothing_new(batch)) return BL_OK;
  if (!k || !v) return BL_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_kv_read(view(cache), step_of(batch), batch->seqs, batch->max_new, k, v, (hipStream_t)stream));
}

size_t bl_attention_workspace_bytes(const bl_kv_cache* cache, const bl_kv_batch* batch, int64_t q_heads) {
  if (check_kv(cache, batch) != BL_OK || nothing_new(batch) || !q_heads_ok(q_heads) || q_heads % cache->heads != 0) return 0;
  return bl::attention_workspace_bytes(view(cache), batch->seqs, batch->tokens, batch->max_new, batch->max_len, q_heads);
}

bl_status bl_attention(const bl_kv_cache* cache, const bl_kv_batch* batch, const uint16_t* q, int64_t q_token_stride,
                       int64_t q_head_stride, int64_t q_heads, float scale, int64_t window, int64_t sinks,
                       uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (bl_status st = check_kv(cache, batch)) return st;
  if (!q_heads_ok(q_heads) || q_heads % cache->heads != 0 || !(fabsf(scale) < INFINITY) || window < 0 || sinks < 0 ||
      (sinks > 0 && window == 0) || batch->max_new * (q_heads / cache->heads) > kMaxPositions)
    return BL_ERR_SHAPE;
  if (nothing_new(batch)) return BL_OK;  // empty tensors may carry NULL pointers
  if (!q || !out) return BL_ERR_NULL;
  if (!aligned(q, 16) || !strides_ok(q_token_stride, q_head_stride) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 16))
    return BL_ERR_ALIGN;
  const bl::KvView kv = view(cache);
  const size_t need = bl::attention_workspace_bytes(kv, batch->seqs, batch->tokens, batch->max_new, batch->max_len, q_heads);
  if (need > 0 && !workspace) return BL_ERR_NULL;
  if (need > workspace_bytes) return BL_ERR_WORKSPACE;
  // no position passes max_len: longer windows hold everything, longer sinks too
  if (window > kMaxPositions) window = kMaxPositions;
  if (sinks > kMaxPositions) sinks = kMaxPositions;
  return from_hip(bl::launch_attention(kv, step_of(batch), batch->seqs, batch->tokens, batch->max_new, batch->max_len, q,
                                       q_token_stride, q_head_stride, (int)q_heads, scale, window, sinks, out, lse,
                                       workspace, (hipStream_t)stream));
}

namespace {

// Groups cover the sequences, as far as the host can see.
bl_status check_shared(const bl_kv_cache* cache, const bl_kv_batch* batch, const bl_kv_shared* shared, int64_t q_heads) {
  if (bl_status st = check_kv(cache, batch)) return st;
  if (!shared) return BL_ERR_NULL;
  if (shared->groups < 0 || shared->groups > 65535 || shared->max_group < 0 || shared->max_group > 65535 ||
      shared->max_prefix < 0 || shared->max_prefix > batch->max_len || shared->groups * shared->max_group < batch->seqs ||
      !q_heads_ok(q_heads) || q_heads % cache->heads != 0 ||
      shared->groups * shared->max_group > kMaxPositions / cache->heads ||
      batch->tokens * (q_heads / cache->heads) > kMaxPositions || !product_ok(batch->tokens, q_heads * cache->dim))
    return BL_ERR_SHAPE;
  return BL_OK;
}

bl::KvGroups groups_of(const bl_kv_shared* s) { return {s->group, s->prefix, s->groups, s->max_group, s->max_prefix}; }

}  // namespace

size_t bl_attention_shared_workspace_bytes(const bl_kv_cache* cache, const bl_kv_batch* batch, const bl_kv_shared* shared,
                                           int64_t q_heads) {
  if (check_shared(cache, batch, shared, q_heads) != BL_OK || nothing_new(batch)) return 0;
  return bl::attention_shared_workspace_bytes(view(cache), batch->seqs, batch->tokens, batch->max_new, batch->max_len,
                                              q_heads, groups_of(shared));
}

bl_status bl_attention_shared(const bl_kv_cache* cache, const bl_kv_batch* batch, const bl_kv_shared* shared,
                              const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                              float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (bl_status st = check_shared(cache, batch, shared, q_heads)) return st;
  if (!(fabsf(scale) < INFINITY)) return BL_ERR_SHAPE;
  if (nothing_new(batch)) return BL_OK;  // empty tensors may carry NULL pointers
  if (!q || !out || !shared->group || !shared->prefix) return BL_ERR_NULL;
  if (!aligned(q, 16) || !strides_ok(q_token_stride, q_head_stride) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(workspace, 16) || !aligned(shared->group, 4) || !aligned(shared->prefix, 4))
    return BL_ERR_ALIGN;
  const bl::KvView kv = view(cache);
  const bl::KvGroups groups = groups_of(shared);
  const size_t need = bl::attention_shared_workspace_bytes(kv, batch->seqs, batch->tokens, batch->max_new, batch->max_len,
                                                           q_heads, groups);
  if (need > 0 && !workspace) return BL_ERR_NULL;
  if (need > workspace_bytes) return BL_ERR_WORKSPACE;
  return from_hip(bl::launch_attention_shared(kv, step_of(batch), groups, batch->seqs, batch->tokens, batch->max_new,
                                              batch->max_len, q, q_token_stride, q_head_stride, (int)q_heads, scale, out, lse,
                                              workspace, (hipStream_t)stream));
}

namespace {

// Whether n elements from a on and m from b on have one in common.
bool share_elements(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return n > 0 && m > 0 && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}

// A pool, and a table of `seqs` rows that goes with it.
bl_status check_pool(const bl_kv_pool* pool, int64_t seqs, int64_t stride) {
  if (!pool) return BL_ERR_NULL;
  if (pool->pages < 1 || pool->pages > BL_MAX_POOL_PAGES || !page_tokens_ok(pool->page_tokens) || seqs < 0 || seqs > 65535 ||
      stride < 0 || stride > kMaxPositions / pool->page_tokens)
    return BL_ERR_SHAPE;
  return BL_OK;
}

}  // namespace

bl_status bl_kv_grow(const bl_kv_pool* pool, const bl_kv_batch* batch, int32_t* copies, int32_t* shortage, void* stream) {
  if (!pool || !batch) return BL_ERR_NULL;
  if (bl_status st = check_pool(pool, batch->seqs, batch->table_stride)) return st;
  if (batch->tokens < 0 || batch->tokens > kMaxPositions || batch->max_new < 0 || batch->max_new > batch->tokens ||
      batch->max_len < batch->max_new || batch->max_len > batch->table_stride * pool->page_tokens ||
      batch->seqs * ((batch->max_new + pool->page_tokens - 2) / pool->page_tokens + 1) > bl::kMaxGrowItems ||
      (copies && batch->seqs > BL_MAX_FORK_SEQS))
    return BL_ERR_SHAPE;
  if (nothing_new(batch)) return BL_OK;  // empty tensors may carry NULL pointers
  if (!pool->refs || !batch->page_table || !batch->start || !batch->offsets) return BL_ERR_NULL;
  if (!aligned(pool->refs, 16) || !aligned(batch->page_table, 4) || !aligned(batch->start, 4) ||
      !aligned(batch->offsets, 4) || !aligned(copies, 4) || !aligned(shortage, 4))
    return BL_ERR_ALIGN;
  return from_hip(bl::launch_kv_grow(pool->refs, pool->pages, pool->page_tokens, step_of(batch), batch->seqs, batch->max_new,
                                     const_cast<int32_t*>(batch->page_table), copies, shortage, (hipStream_t)stream));
}

bl_status bl_kv_fork(const bl_kv_pool* pool, const int32_t* table, int64_t table_stride, const int32_t* length,
                     int64_t seqs, const int32_t* parent, int64_t children, int keep_parents, int32_t* table_out,
                     int32_t* length_out, int32_t* copies, int32_t* shortage, void* stream) {
  if (bl_status st = check_pool(pool, seqs, table_stride)) return st;
  if (seqs > BL_MAX_FORK_SEQS || children < 0 || children > BL_MAX_FORK_SEQS || (table && table_out == table) ||
      (length && length_out == length))
    return BL_ERR_SHAPE;
  if ((children == 0 && (keep_parents || seqs == 0)) || (seqs > 0 && table_stride == 0 && children == 0)) return BL_OK;
  if (!pool->refs || (seqs > 0 && (!length || (table_stride > 0 && !table))) ||
      (children > 0 && (!parent || !length_out || !copies || (table_stride > 0 && !table_out))))
    return BL_ERR_NULL;
  if (!aligned(pool->refs, 16) || !aligned(table, 4) || !aligned(length, 4) || !aligned(parent, 4) ||
      !aligned(table_out, 4) || !aligned(length_out, 4) || !aligned(copies, 4) || !aligned(shortage, 4))
    return BL_ERR_ALIGN;
  // workgroups that run at once write the outputs and read the rest
  const struct { const int32_t* at; int64_t n; } parts[] = {
      {table_out, children * table_stride}, {length_out, children}, {copies, 3 * children}, {table, seqs * table_stride},
      {length, seqs}, {parent, children}, {pool->refs, pool->pages}, {shortage, shortage ? 1 : 0}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 8; ++j)
      if (share_elements(parts[i].at, parts[i].n, parts[j].at, parts[j].n)) return BL_ERR_SHAPE;
  return from_hip(bl::launch_kv_fork(pool->refs, pool->pages, pool->page_tokens, table, table_stride, length, seqs, parent,
                                     children, keep_parents != 0, table_out, length_out, copies, shortage,
                                     (hipStream_t)stream));
}

bl_status bl_kv_free(const bl_kv_pool* pool, int32_t* table, int64_t table_stride, int64_t seqs, const int32_t* keep,
                     void* stream) {
  if (bl_status st = check_pool(pool, seqs, table_stride)) return st;
  if (seqs == 0 || table_stride == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!pool->refs || !table) return BL_ERR_NULL;
  if (!aligned(pool->refs, 16) || !aligned(table, 4) || !aligned(keep, 4)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_kv_free(pool->refs, pool->pages, pool->page_tokens, table, table_stride, seqs, keep,
                                     (hipStream_t)stream));
}

size_t bl_kv_compact_workspace_bytes(const bl_kv_pool* pool, int64_t moves) {
  if (check_pool(pool, 0, 0) != BL_OK || moves < 0 || moves > pool->pages) return 0;
  return bl::kv_compact_workspace_bytes(pool->pages, moves);
}

bl_status bl_kv_compact(const bl_kv_pool* pool, int32_t* table, int64_t table_stride, int64_t seqs, int64_t moves,
                        int32_t* copies, int32_t* moved, void* workspace, size_t workspace_bytes, void* stream) {
  if (bl_status st = check_pool(pool, seqs, table_stride)) return st;
  if (moves < 0 || moves > pool->pages) return BL_ERR_SHAPE;
  if (!pool->refs || !moved || !workspace || (moves > 0 && !copies) || (seqs * table_stride > 0 && !table)) return BL_ERR_NULL;
  if (!aligned(pool->refs, 16) || !aligned(table, 4) || !aligned(copies, 4) || !aligned(moved, 4) || !aligned(workspace, 16))
    return BL_ERR_ALIGN;
  if (workspace_bytes < bl::kv_compact_workspace_bytes(pool->pages, moves)) return BL_ERR_WORKSPACE;
  return from_hip(bl::launch_kv_compact(pool->refs, pool->pages, pool->page_tokens, table, table_stride, seqs, moves, copies,
                                        moved, workspace, (hipStream_t)stream));
}

bl_status bl_kv_copy(const bl_kv_cache* caches, int64_t count, const int32_t* copies, int64_t n, const int32_t* valid,
                     void* stream) {
  if (count < 0 || count > bl::kMaxCaches || n < 0 || n > BL_MAX_POOL_PAGES) return BL_ERR_SHAPE;
  if (count > 0 && !caches) return BL_ERR_NULL;
  bl::KvView views[bl::kMaxCaches];
  for (int64_t i = 0; i < count; ++i) {
    if (bl_status st = check_cache(caches + i)) return st;
    if (caches[i].pages != caches[0].pages || caches[i].heads != caches[0].heads ||
        caches[i].page_tokens != caches[0].page_tokens || caches[i].dim != caches[0].dim)
      return BL_ERR_SHAPE;
    views[i] = view(caches + i);
  }
  if (count == 0 || n == 0) return BL_OK;  // empty tensors may carry NULL pointers
  for (int64_t i = 0; i < count; ++i)
    if (bl_status st = check_cache_pointers(caches + i)) return st;
  if (!copies) return BL_ERR_NULL;
  if (!aligned(copies, 4) || !aligned(valid, 4)) return BL_ERR_ALIGN;
  return from_hip(bl::launch_kv_copy(views, count, copies, n, valid, (hipStream_t)stream));
}

namespace {

bl_status check_logits(int type, int64_t m, int64_t n, int64_t stride, float scale) {
  if ((type != BL_BF16 && type != BL_FP32) || m < 0 || m > BL_MAX_M || n < 1 || n > BL_MAX_VOCABULARY || stride < n ||
      !product_ok(m, stride) || !(scale > 0.0f && scale <= 0x1p127f))  // times log2 e, still finite
    return BL_ERR_SHAPE;
  return BL_OK;
}

// Whether rows of n elements, `stride` apart, at two places have elements in
// common without being the same rows.
bool rows_cross(const void* a, const void* b, int64_t m, int64_t n, int64_t stride, int64_t size) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  const uint64_t apart = x < y ? y - x : x - y, row = (uint64_t)(m > 1 ? stride : n) * size, length = (uint64_t)n * size;
  const uint64_t rows = apart / row, rest = apart % row;
  return apart > 0 && ((rows < (uint64_t)m && rest < length) || (rows + 1 < (uint64_t)m && row - rest < length));
}

}  // namespace

size_t bl_logprobs_workspace_bytes(int64_t m, int64_t n, int type, int64_t top) {
  if (check_logits(type, m, n, n, 1.0f) != BL_OK || m == 0 || top < 0 || top > BL_MAX_TOP) return 0;
  return bl::logprobs_workspace_bytes(m, n, type == BL_BF16, top);
}

bl_status bl_logprobs(const void* x, int type, int64_t m, int64_t n, int64_t row_stride, float scale,
                      const int32_t* target, int64_t top, float* logprob, float* lse, float* entropy, int32_t* top_id,
                      float* top_logprob, void* workspace, size_t workspace_bytes, void* stream) {
  if (bl_status st = check_logits(type, m, n, row_stride, scale)) return st;
  if (top < 0 || top > BL_MAX_TOP) return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || (logprob && !target) || (top > 0 && (!top_id || !top_logprob)) || (!logprob && !lse && !entropy && top == 0))
    return BL_ERR_NULL;
  if (!aligned(x, type == BL_BF16 ? 2 : 4) || !aligned(target, 4) || !aligned(logprob, 4) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(top_id, 4) || !aligned(top_logprob, 4) || !aligned(workspace, 16))
    return BL_ERR_ALIGN;
  const size_t need = bl::logprobs_workspace_bytes(m, n, type == BL_BF16, top);
  if (need > 0 && !workspace) return BL_ERR_NULL;
  if (need > workspace_bytes) return BL_ERR_WORKSPACE;
  return from_hip(bl::launch_logprobs(x, type == BL_BF16, m, n, row_stride, scale, target, top, logprob, lse, entropy, top_id,
                                      top_logprob, workspace, (hipStream_t)stream));
}

bl_status bl_logprobs_backward(const void* x, int type, int64_t m, int64_t n, int64_t row_stride, float scale,
                               const int32_t* target, const float* lse, const float* entropy, const float* dlogprob,
                               const float* dentropy, const float* dlse, void* dx, int64_t dx_stride, void* stream) {
  if (bl_status st = check_logits(type, m, n, row_stride, scale)) return st;
  if (dx_stride < n || !product_ok(m, dx_stride) || (x && dx == x && dx_stride != row_stride && m > 1)) return BL_ERR_SHAPE;
  if (m == 0) return BL_OK;  // empty tensors may carry NULL pointers
  if (!x || !lse || !dx || (!dlogprob && !dentropy && !dlse) || (dlogprob && !target) || (dentropy && !entropy))
    return BL_ERR_NULL;
  const uintptr_t size = type == BL_BF16 ? 2 : 4;
  if (!aligned(x, size) || !aligned(dx, size) || !aligned(target, 4) || !aligned(lse, 4) || !aligned(entropy, 4) ||
      !aligned(dlogprob, 4) || !aligned(dentropy, 4) || !aligned(dlse, 4))
    return BL_ERR_ALIGN;
  if ((m == 1 || dx_stride == row_stride) && rows_cross(x, dx, m, n, row_stride, (int64_t)size)) return BL_ERR_SHAPE;
  return from_hip(bl::launch_logprobs_backward(x, type == BL_BF16, m, n, row_stride, scale, target, lse, entropy, dlogprob,
                                               dentropy, dlse, dx, dx_stride, (hipStream_t)stream));
}

const char* bl_status_string(bl_status s) {
  switch (s) {
    case BL_OK: return "BL_OK";
    case BL_ERR_NULL: return "BL_ERR_NULL: a required pointer is NULL";
    case BL_ERR_SHAPE: return "BL_ERR_SHAPE: m, n or k outside the supported range";
    case BL_ERR_ALIGN: return "BL_ERR_ALIGN: a pointer is not aligned as required";
    case BL_ERR_WORKSPACE: return "BL_ERR_WORKSPACE: workspace too small";
    case BL_ERR_HIP: return "BL_ERR_HIP: the HIP runtime rejected a launch";
  }
  return "unknown bl_status";
}

}  // extern "C"
