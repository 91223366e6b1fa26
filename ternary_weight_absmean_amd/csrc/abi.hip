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

bl_status check_kv(const bl_kv_cache* c, const bl_kv_batch* b) {
  if (!c || !b) return BL_ERR_NULL;
  const int p = c->page_tokens;
  if (c->heads < 1 || c->heads > 65536 || (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) || c->dim < 16 ||
      c->dim > BL_MAX_HEAD_DIM || c->dim % 16 != 0 || c->pages < 1 || c->pages > 0x7FFFFFFF ||
      !product_ok(c->pages, (int64_t)c->heads * p * c->dim))
    return BL_ERR_SHAPE;
  if (b->seqs < 0 || b->seqs > 65535 || b->tokens < 0 || b->tokens > kMaxPositions || b->max_new < 0 ||
      b->max_new > b->tokens || b->max_len < b->max_new || b->max_len > kMaxPositions || b->table_stride < 0 ||
      b->table_stride > 0x7FFFFFFF || b->max_len > b->table_stride * p)
    return BL_ERR_SHAPE;
  if (b->seqs == 0 || b->tokens == 0 || b->max_new == 0) return BL_OK;
  if (!c->k || !c->v || !c->k_absmax || !c->v_absmax || !b->page_table || !b->start || !b->offsets) return BL_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_absmax, 4) || !aligned(c->v_absmax, 4) ||
      !aligned(b->page_table, 4) || !aligned(b->start, 4) || !aligned(b->offsets, 4))
    return BL_ERR_ALIGN;
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
