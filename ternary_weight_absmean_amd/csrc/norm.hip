// Root-mean-square norm with the residual's addition and int8 output, and its
// gradients (bl_rmsnorm_quant, bl_rmsnorm_backward).
//
// Forward, per row: h = x + residual, c = 1 / sqrt(mean h^2 + eps),
// n = (h * w) * c, alpha = max |n|, xq = round(n * 127 / max(alpha, 1e-5)).
// Multiplying by c last makes max |n| = fl(max |h * w| * c) (rounding keeps
// order), so the sum of squares and the maximum come out of ONE reduction and
// the row is read once and stays in registers: 2 bytes in per element (4 with
// a residual), 1 to 5 out.  HBM-bound for many rows, a launch and two memory
// round trips for one.
#include "device_util.h"
#include "internal.h"

namespace bl {
namespace {

// A 16-byte chunk of eight bf16 as fp32.
__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(d[i] << 16);
    f[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                    f32x2_to_bf16x2(f[6], f[7]));
}

// 1 / sqrt(v), correctly rounded division and root; 0 for v = 0, which a row of
// zeros has without an eps: its norm is zeros and it adds nothing to a gradient.
__device__ __forceinline__ float rsqrt_or_zero(float v) { return v == 0.0f ? 0.0f : 1.0f / sqrtf(v); }

// A store that leaves the caches to others.  2048 x 8192 with residual and three
// sets of inputs in turn: 23 us against 31, because those stay in the Infinity
// Cache; a block of the decoder example takes the same 504 us per prompt pass
// either way.  The sum and xhat are read only after other kernels have passed.
// Where y is the only output the next kernel does read it, and loses nothing by
// it (norm and a reader: 4 x 2560 4.1 us either way, 2048 x 2560 8.5 against 8.9,
// 2048 x 8192 20.5 both).
__device__ __forceinline__ void store_past_caches(uint4* p, const uint4& v) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  __builtin_nontemporal_store((v4u){v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(p));
}

// Sum over the wave in a fixed order, the same value in every lane: lane moves
// within rows of 16 (DPP), then the four row sums as scalars.
__device__ __forceinline__ float wave_sum(float v) {
  auto move = [](float x, auto ctrl) {
    const int i = __float_as_int(x);
    return __int_as_float(__builtin_amdgcn_update_dpp(i, i, decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += move(v, std::integral_constant<int, 0xB1>{});
  v += move(v, std::integral_constant<int, 0x4E>{});
  v += move(v, std::integral_constant<int, 0x141>{});
  v += move(v, std::integral_constant<int, 0x140>{});
  const int i = __float_as_int(v);
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(i, 0)), r1 = __int_as_float(__builtin_amdgcn_readlane(i, 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(i, 32)), r3 = __int_as_float(__builtin_amdgcn_readlane(i, 48));
  return (r0 + r1) + (r2 + r3);
}

// One workgroup of T threads per row, kC chunks of eight columns per thread
// (chunk c of thread t covers columns 8 * (t + c * T)).  Loads go through
// buffer resources over the row, so chunks past k read as zero and add nothing.
// 2048 x 8192 with residual, sum and xhat (151 MB): 22.7 us; 1 x 2560: 2.2 us,
// a launch and its round trips.
template <int T, int kC>
__global__ __launch_bounds__(T) void k_rmsnorm_quant(const uint4* x, const uint4* residual, const uint4* __restrict__ w,
                                                     int k8, float eps, uint4* r, uint4* y, uint4* xhat, uint2* xq,
                                                     float* alpha) {
  __shared__ float wave_part[2][T / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(x + row * k8, (uint32_t)(k8 * 16));
  const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(residual ? residual + row * k8 : x, residual ? (uint32_t)(k8 * 16) : 0u);
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(w, (uint32_t)(k8 * 32));
  uint4 vx[kC], vr[kC], vw[2 * kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const uint32_t off = (uint32_t)((tid + c * T) * 16);
    vx[c] = buffer_load16(xr, off);
    vr[c] = buffer_load16(rr, off);  // zeros without a residual
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const uint32_t off = (uint32_t)((tid + c * T) * 32);
    vw[2 * c] = buffer_load16(wr, off);
    vw[2 * c + 1] = buffer_load16(wr, off + 16);
  }
  float h[kC][8], sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    float res[8];
    unpack_bf16x8(vx[c], h[c]);
    unpack_bf16x8(vr[c], res);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[c][i] += res[i];
      sum = __builtin_fmaf(h[c][i], h[c][i], sum);
    }
  }
  if (r) {
#pragma unroll
    for (int c = 0; c < kC; ++c)
      if (tid + c * T < k8) store_past_caches(&r[row * k8 + tid + c * T], pack_bf16x8(h[c]));
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const float wv[8] = {__uint_as_float(vw[2 * c].x),     __uint_as_float(vw[2 * c].y),
                         __uint_as_float(vw[2 * c].z),     __uint_as_float(vw[2 * c].w),
                         __uint_as_float(vw[2 * c + 1].x), __uint_as_float(vw[2 * c + 1].y),
                         __uint_as_float(vw[2 * c + 1].z), __uint_as_float(vw[2 * c + 1].w)};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[c][i] *= wv[i];
      top = fmaxf(top, fabsf(h[c][i]));
    }
  }
  sum = wave_sum(sum);
  top = __int_as_float(wave_reduce<true>(__float_as_int(top)));  // magnitudes order like their bits
  if (T > 64) {
    if ((tid & 63) == 0) {
      wave_part[0][tid >> 6] = sum;
      wave_part[1][tid >> 6] = top;
    }
    __syncthreads();
    sum = wave_part[0][0];
    top = wave_part[1][0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) {
      sum += wave_part[0][i];
      top = fmaxf(top, wave_part[1][i]);
    }
  }
  const float c = rsqrt_or_zero(sum / (float)(k8 * 8) + eps);
  const float a = top * c;
  const float s = 127.0f / fmaxf(a, 1e-5f);
  const float step = a / 127.0f;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int at = tid + i * T;
    if (at >= k8) break;
    float n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = h[i][j] * c;
    if (y) store_past_caches(&y[row * k8 + at], pack_bf16x8(n));
    if (!xq && !xhat) continue;
    // round half to even into the low byte of the sum (|n * s| is at most
    // 127 * (1 + 2^-22): no code leaves [-127, 127])
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = n[j] * s + 12582912.0f;
    if (xq) {
      auto four = [](float f0, float f1, float f2, float f3) {
        const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(f1), __float_as_uint(f0), 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(f3), __float_as_uint(f2), 0x0c0c0400u);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      };
      xq[row * k8 + at] = make_uint2(four(m[0], m[1], m[2], m[3]), four(m[4], m[5], m[6], m[7]));
    }
    if (xhat) {
#pragma unroll
      for (int j = 0; j < 8; ++j) m[j] = (m[j] - 12582912.0f) * step;
      store_past_caches(&xhat[row * k8 + at], pack_bf16x8(m));
    }
  }
  if (alpha && tid == 0) alpha[row] = a;
}

// ---- backward ----
// dx_j = c * (dn_j w_j - r_j c^2 mean(dn w r)) + dr_j and dw_j = sum_i dn r c.
// A workgroup walks over rows (row b, b + grid, ...) and keeps its columns' dw
// sums in registers; per row one reduction (sum r^2 and sum dn w r).  The
// workgroups' sums go to the workspace and a second kernel adds them in a
// fixed order, so no atomics and the same bits every time.  HBM-bound: 4096 x
// 8192 with dr (336 MB, and 8 MB of partial sums written and read again) 65 us,
// 5.2 TB/s; 333 x 6912 11 us (8.4 + 3.3): 77 of 256 workgroups take a second row,
// with its own round trip and reduction, and each writes 28 KB of partial sums.
template <int T, int kC>
__global__ __launch_bounds__(T) void k_rmsnorm_backward(const uint4* __restrict__ dn, const uint4* __restrict__ r,
                                                        const uint4* __restrict__ w, const uint4* dr, int64_t m, int k8,
                                                        float eps, uint4* dx, float* __restrict__ part) {
  __shared__ float wave_part[2][2][T / 64];
  const int tid = threadIdx.x;
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(w, (uint32_t)(k8 * 32));
  float acc[kC][8];
#pragma unroll
  for (int c = 0; c < kC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.0f;
  // the weights stay in registers (8192 x 640 16 us against 19 with two reads of
  // them per row, 4096 x 2560 24 against 27, 4096 x 8192 70 against 72); the longest
  // rows leave none for that (scratch: 1000 x 32768 144 against 91)
  constexpr bool kHold = kC < 8;
  uint4 vw[kHold ? 2 * kC : 1];
  if (kHold) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      vw[2 * c] = buffer_load16(wr, (uint32_t)(tid + c * T) * 32);
      vw[2 * c + 1] = buffer_load16(wr, (uint32_t)(tid + c * T) * 32 + 16);
    }
  }
  auto weight = [&](int c, int i) {
    return kHold ? vw[kHold ? 2 * c + i : 0] : buffer_load16(wr, (uint32_t)(tid + c * T) * 32 + 16 * i);
  };
  int turn = 0;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x, turn ^= 1) {
    const __amdgpu_buffer_rsrc_t nr = buffer_rsrc(dn + row * k8 * 2, (uint32_t)(k8 * 32));
    const __amdgpu_buffer_rsrc_t rr = buffer_rsrc(r + row * k8, (uint32_t)(k8 * 16));
    const __amdgpu_buffer_rsrc_t gr = buffer_rsrc(dr ? dr + row * k8 : r, dr ? (uint32_t)(k8 * 16) : 0u);
    uint4 vn[2 * kC], vr[kC], vg[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const uint32_t at = (uint32_t)(tid + c * T);
      vn[2 * c] = buffer_load16(nr, at * 32);
      vn[2 * c + 1] = buffer_load16(nr, at * 32 + 16);
      vr[c] = buffer_load16(rr, at * 16);
      if (kC < 8) vg[c] = buffer_load16(gr, at * 16);  // the longest rows have no registers left for it
    }
    float square = 0.0f, inner = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      float rv[8];
      unpack_bf16x8(vr[c], rv);
      const uint4 w0 = weight(c, 0), w1 = weight(c, 1);
      const uint32_t wb[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const uint32_t nb[8] = {vn[2 * c].x,     vn[2 * c].y,     vn[2 * c].z,     vn[2 * c].w,
                              vn[2 * c + 1].x, vn[2 * c + 1].y, vn[2 * c + 1].z, vn[2 * c + 1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        square = __builtin_fmaf(rv[j], rv[j], square);
        inner = __builtin_fmaf(__uint_as_float(nb[j]) * __uint_as_float(wb[j]), rv[j], inner);
      }
    }
    square = wave_sum(square);
    inner = wave_sum(inner);
    if ((tid & 63) == 0) {
      wave_part[turn][0][tid >> 6] = square;  // two buffers by turns: one barrier per row is enough
      wave_part[turn][1][tid >> 6] = inner;
    }
    __syncthreads();
    square = wave_part[turn][0][0];
    inner = wave_part[turn][1][0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) {
      square += wave_part[turn][0][i];
      inner += wave_part[turn][1][i];
    }
    const float inv = 1.0f / (float)(k8 * 8);
    const float c = rsqrt_or_zero(square * inv + eps);
    const float back = inner * inv * c * c;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int at = tid + i * T;
      if (at >= k8) break;
      float rv[8], g[8];
      unpack_bf16x8(vr[i], rv);
      if (kC == 8) vg[i] = buffer_load16(gr, (uint32_t)at * 16);
      unpack_bf16x8(vg[i], g);
      const uint4 w0 = weight(i, 0), w1 = weight(i, 1);
      const uint32_t wb[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      const uint32_t nb[8] = {vn[2 * i].x,     vn[2 * i].y,     vn[2 * i].z,     vn[2 * i].w,
                              vn[2 * i + 1].x, vn[2 * i + 1].y, vn[2 * i + 1].z, vn[2 * i + 1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = __uint_as_float(nb[j]);
        acc[i][j] = __builtin_fmaf(d * c, rv[j], acc[i][j]);
        g[j] += c * (d * __uint_as_float(wb[j]) - rv[j] * back);
      }
      dx[row * k8 + at] = pack_bf16x8(g);
    }
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int at = tid + c * T;
    if (at >= k8) break;
    float4* out = reinterpret_cast<float4*>(part + ((int64_t)blockIdx.x * k8 + at) * 8);
    out[0] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
    out[1] = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
  }
}

// dw = the workgroups' partial sums, added in a fixed order: 32 columns per
// workgroup (128-byte pieces of a row of partials, four columns per thread) and
// 32 rows at a time, eight loads of a thread in flight.
constexpr int kDwCols = 32, kDwSlots = 32;

__global__ __launch_bounds__(kDwCols / 4 * kDwSlots) void k_rmsnorm_dw(const float* __restrict__ part, int blocks,
                                                                       int64_t k, float* __restrict__ dw) {
  typedef float v4f __attribute__((ext_vector_type(4)));
  __shared__ v4f sums[kDwSlots][kDwCols / 4];
  const int quad = threadIdx.x % (kDwCols / 4), slot = threadIdx.x / (kDwCols / 4);
  const int64_t j = (int64_t)blockIdx.x * kDwCols + quad * 4;  // k is a multiple of 64
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int b = slot; b < blocks; b += kDwSlots) s += *reinterpret_cast<const v4f*>(part + b * k + j);
  sums[slot][quad] = s;
  __syncthreads();
  if (slot == 0) {
#pragma unroll
    for (int i = 1; i < kDwSlots; ++i) s += sums[i][quad];
    *reinterpret_cast<v4f*>(dw + j) = s;
  }
}

// Workgroups of the backward kernel: about as many as run at once, since each
// writes a row of partial sums.  4096 x 8192: 65 us with 256, 70 with 512; 4096 x
// 2560: 24 with 512, 30 with 256, 27 with 1024; 8192 x 2048: 35 with 512, 39 with
// 1024; 8192 x 1024: 19.5 with 1024, 22.5 with 512; 8192 x 640: 16 with 1024, 21
// with 512; 1000 x 28672: 81 us with 256, 93 with 512.
int back_blocks(int64_t m, int64_t k) {
  const int64_t most = k <= 1024 ? 1024 : k <= 4096 ? 512 : 256;
  return (int)(m < most ? m : most);
}

}  // namespace

hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* residual, const float* w, int64_t m, int64_t k,
                                float eps, uint16_t* r, uint16_t* y, uint16_t* xhat, int8_t* xq, float* alpha,
                                hipStream_t s) {
  const int k8 = (int)(k / 8);
  auto go = [&](auto t, auto c) {
    constexpr int T = decltype(t)::value, kC = decltype(c)::value;
    if (!grid_fits(m, T)) return kErrGridTooLarge;
    hipLaunchKernelGGL((k_rmsnorm_quant<T, kC>), dim3((unsigned)m), dim3(T), 0, s, (const uint4*)x,
                       (const uint4*)residual, (const uint4*)w, k8, eps, (uint4*)r, (uint4*)y, (uint4*)xhat, (uint2*)xq,
                       alpha);
    return hipGetLastError();
  };
  using std::integral_constant;
  // a wave per row for the shortest; more than four chunks per thread for none
  if (k8 <= 64) return go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (k8 <= 128) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (k8 <= 256) return go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (k8 <= 512) return go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (k8 <= 1024) return go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  if (k8 <= 2048) return go(integral_constant<int, 512>{}, integral_constant<int, 4>{});
  return go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

size_t rmsnorm_backward_workspace_bytes(int64_t m, int64_t k) { return (size_t)back_blocks(m, k) * (size_t)k * 4; }

hipError_t launch_rmsnorm_backward(const float* dn, const uint16_t* r, const float* w, const uint16_t* dr, int64_t m,
                                   int64_t k, float eps, uint16_t* dx, float* dw, void* workspace, hipStream_t s) {
  const int k8 = (int)(k / 8), blocks = back_blocks(m, k);
  float* part = (float*)workspace;
  auto go = [&](auto t, auto c) {
    constexpr int T = decltype(t)::value, kC = decltype(c)::value;
    hipLaunchKernelGGL((k_rmsnorm_backward<T, kC>), dim3((unsigned)blocks), dim3(T), 0, s, (const uint4*)dn,
                       (const uint4*)r, (const uint4*)w, (const uint4*)dr, m, k8, eps, (uint4*)dx, part);
  };
  using std::integral_constant;
  if (k8 <= 64)
    go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (k8 <= 128)
    go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (k8 <= 256)
    go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (k8 <= 512)
    go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (k8 <= 1024)
    go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (k8 <= 2048)  // 2000 x 16384 72 us against 91 with eight chunks per thread, 1500 x 12288 42 against 58
    go(integral_constant<int, 512>{}, integral_constant<int, 4>{});
  else
    go(integral_constant<int, 512>{}, integral_constant<int, 8>{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_rmsnorm_dw, dim3((unsigned)(k / kDwCols)), dim3(kDwCols / 4 * kDwSlots), 0, s, part, blocks, k, dw);
  return hipGetLastError();
}

}  // namespace bl
