// Rotary positions and the 8-bit key/value cache (bl_rope, bl_kv_append,
// bl_kv_read).
//
// A rotation by position * f is a rotation by the fraction of position * f / 2pi
// turns.  The table holds f / 2pi as two fp32 (value and remainder): with
// p = fl(pos * hi), e = fma(pos, hi, -p) is the product's exact error, so
// the turn's fraction is p - round(p) plus e + pos * lo at every position below
// 2^24, where a product of fp32 radians is off by pos * 2^-25.
//
// v_cos_f32 and v_sin_f32 of the turn are off by up to 2.7e-7 (4e-7 at the
// farthest positions): nothing beside a rounding to bf16, which queries and
// bl_rope's outputs take.  Keys are quantized from fp32, where such an error
// turns codes beside a rounding boundary and moves a page's scale; theirs are
// right to 2^-23 (unit_angles).
//
// All three calls move bytes: 2 in and 2 out per rotated element; 2 in and 1
// out per appended element, 1 in and 2 out per element read back.  HBM-bound
// for prompts, a launch and its dependent loads for a decoded token.
#include "device_util.h"
#include "internal.h"

namespace bl {
namespace {

// One thread's unit of a head: 16 elements as two runs of eight.  Units
// 0 .. R-1 (R = ceil(rot / 16)) hold eight pairs each, the rest copy.  Where
// runs are whole 16-byte pieces (kVec), neighbouring units' runs lie side by
// side, so that a wave's loads and stores cover whole lines:
//   turned: runs at 8u and rot/2 + 8u; pairs are (run 0 [j], run 1 [j]) or, for
//           neighbouring elements (kInter), those inside a run;
//   copied: runs at rot + 8(u - R) and as many units further.
// Otherwise the runs of a turned unit are at 8u and rot/2 + 8u, or 16u and
// 16u + 8, and those of a copied one at rot + 16(u - R) and 8 further, element
// by element (4099 tokens of 72 heads of 128: 132 us with 40 elements turned, 117
// with 72, 25 with 128).  A thread owns its unit's elements, so a rotation in
// place is safe.
struct Head {
  int dim, rot, half, turning, units;  // turning = R
};

__host__ __device__ inline Head make_head(int dim, int rot) {
  Head h;
  h.dim = dim;
  h.rot = rot;
  h.half = rot / 2;
  h.turning = (rot + 15) / 16;
  h.units = h.turning + (dim - rot + 15) / 16;
  return h;
}

// Runs are whole, 8-element-aligned 16-byte pieces (a copied unit may lack its second).
inline bool vector_runs(int dim, int rot) { return rot % 16 == 0 && dim % 8 == 0; }

// First element of run `run` of unit u, and one past the last the unit may touch there.
template <bool kVec, bool kInter>
__device__ __forceinline__ int run_start(const Head& h, int u, int run) {
  if (u >= h.turning)
    return kVec ? h.rot + 8 * (u - h.turning + run * (h.units - h.turning)) : h.rot + 16 * (u - h.turning) + 8 * run;
  return !kVec && kInter ? 16 * u + 8 * run : 8 * u + (run ? h.half : 0);
}
template <bool kVec, bool kInter>
__device__ __forceinline__ int run_limit(const Head& h, int u, int run) {
  if (u >= h.turning) return h.dim;
  return (!kVec && kInter) || run ? h.rot : h.half;
}

template <bool kVec, bool kInter>
__device__ __forceinline__ void load_unit(const Head& h, int u, const uint16_t* row, float (&v)[16]) {
#pragma unroll
  for (int run = 0; run < 2; ++run) {
    const int at = run_start<kVec, kInter>(h, u, run), limit = run_limit<kVec, kInter>(h, u, run);
    if (kVec) {
      uint4 d = make_uint4(0, 0, 0, 0);
      if (at < limit) d = *reinterpret_cast<const uint4*>(row + at);
      const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * run + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * run + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[8 * run + j] = at + j < limit ? __uint_as_float((uint32_t)row[at + j] << 16) : 0.0f;
    }
  }
}

// kPast: past the caches (k_rope says why).
template <bool kVec, bool kInter, bool kPast>
__device__ __forceinline__ void store_unit(const Head& h, int u, uint16_t* row, const float (&v)[16]) {
#pragma unroll
  for (int run = 0; run < 2; ++run) {
    const int at = run_start<kVec, kInter>(h, u, run), limit = run_limit<kVec, kInter>(h, u, run);
    if (kVec) {
      typedef unsigned v4u __attribute__((ext_vector_type(4)));
      const v4u w = {f32x2_to_bf16x2(v[8 * run], v[8 * run + 1]), f32x2_to_bf16x2(v[8 * run + 2], v[8 * run + 3]),
                     f32x2_to_bf16x2(v[8 * run + 4], v[8 * run + 5]), f32x2_to_bf16x2(v[8 * run + 6], v[8 * run + 7])};
      if (at >= limit) continue;
      if (kPast)
        __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(row + at));
      else
        *reinterpret_cast<v4u*>(row + at) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < limit) row[at + j] = f32_to_bf16_rne(v[8 * run + j]);
    }
  }
}

// Codes of 16 values: round half to even into the low byte of value * s + 1.5 * 2^23.
template <bool kVec, bool kInter>
__device__ __forceinline__ void store_codes(const Head& h, int u, int8_t* row, const float (&v)[16], float s) {
#pragma unroll
  for (int run = 0; run < 2; ++run) {
    const int at = run_start<kVec, kInter>(h, u, run), limit = run_limit<kVec, kInter>(h, u, run);
    uint32_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = __float_as_uint(v[8 * run + j] * s + 12582912.0f);
    if (kVec) {
      auto four = [](uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
        const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x0c0c0400u);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      };
      if (at < limit)
        *reinterpret_cast<uint2*>(row + at) = make_uint2(four(c[0], c[1], c[2], c[3]), four(c[4], c[5], c[6], c[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < limit) row[at + j] = (int8_t)c[j];
    }
  }
}

// cos and sin (times the magnitude; sin negated for the inverse) of the eight
// pairs of unit u at position pos.
// kFine: with q = round(4 t) for the turn t, x = t - q / 4 lies within an eighth
// of a turn, where polynomials in x^2 (interpolated at Chebyshev nodes, off by
// 3e-9 and 1e-10) give both; q's low bits exchange and negate them.  t is not
// rounded on the way to x, so both are right to 2^-23 (1.2e-7 at most over 4
// million angles).  For all rotations the prompts' rotation would take 31 us
// instead of 28 and the prompts' cache 63 instead of 59; for the keys alone it is 61.
template <bool kVec, bool kInter, bool kFine>
__device__ __forceinline__ void unit_angles(const Head& h, int u, const float* turns, float pos, float magnitude,
                                            float sign, float (&cs)[8], float (&sn)[8]) {
  float f[16];
  if (kVec) {
    // two pairs per 16 bytes: eight pairs from 8u on, or four from 4u and four from rot/4 + 4u
    const float4* t = reinterpret_cast<const float4*>(turns) + (kInter ? 2 : 4) * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = t[kInter && i >= 2 ? h.half / 4 + i - 2 : i];
      f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = 8 * u + j < h.half ? 8 * u + j : 0;
      f[2 * j] = turns[2 * i], f[2 * j + 1] = turns[2 * i + 1];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float p = pos * f[2 * j];
    const float rest = __builtin_fmaf(pos, f[2 * j + 1], __builtin_fmaf(pos, f[2 * j], -p));
    if (kFine) {
      const float near = p - rintf(p);
      const float q = rintf((near + rest) * 4.0f);
      const float x = __builtin_fmaf(q, -0.25f, near) + rest, u = x * x;
      float s = __builtin_fmaf(-75.401611328125f, u, 81.59254455566406f);
      s = __builtin_fmaf(s, u, -41.3416633605957f);
      s = __builtin_fmaf(s, u, 6.2831854820251465f) * x;
      float c = __builtin_fmaf(59.42410659790039f, u, -85.44882202148438f);
      c = __builtin_fmaf(c, u, 64.93936920166016f);
      c = __builtin_fmaf(c, u, -19.739208221435547f);
      c = __builtin_fmaf(c, u, 1.0f);
      const uint32_t quarter = (uint32_t)(int)q;
      const uint32_t flip_s = quarter << 30 & 0x80000000u, flip_c = (quarter + 1) << 30 & 0x80000000u;
      cs[j] = __uint_as_float(__float_as_uint(quarter & 1 ? s : c) ^ flip_c) * magnitude;
      sn[j] = __uint_as_float(__float_as_uint(quarter & 1 ? c : s) ^ flip_s) * (magnitude * sign);
    } else {
      const float turn = __builtin_amdgcn_fractf(p) + rest;
      cs[j] = __builtin_amdgcn_cosf(turn) * magnitude;
      sn[j] = __builtin_amdgcn_sinf(turn) * (magnitude * sign);
    }
  }
}

template <bool kInter>
__device__ __forceinline__ void turn_unit(float (&v)[16], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (kInter) {
      const float a = v[2 * j], b = v[2 * j + 1];
      v[2 * j] = __builtin_fmaf(a, cs[j], -(b * sn[j]));
      v[2 * j + 1] = __builtin_fmaf(a, sn[j], b * cs[j]);
    } else {
      const float a = v[j], b = v[8 + j];
      v[j] = __builtin_fmaf(a, cs[j], -(b * sn[j]));
      v[8 + j] = __builtin_fmaf(a, sn[j], b * cs[j]);
    }
  }
}

// ---- bl_rope ----
// One thread per unit of a head (unit fastest, then head, then token).  Several
// heads per thread would share the angles, but take registers from the waves
// that hide the loads: 4099 tokens of 72 heads of 128 (151 MB) took 31 us with
// one head per thread, 34 with two, 37 with four.  Stores go past the caches,
// which then keep the inputs of kernels before instead: 27 us against 32 for that
// size, three quarters of each head turned, three sets of inputs in turn.  The
// other side is a next kernel that reads the result at once (52 us for both
// against 47; 2048 tokens of 25 heads 12 either way).
constexpr int kRopeThreads = 256;

template <bool kVec, bool kInter>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const uint16_t* x, int64_t xt, int64_t xh,
                                                       const int32_t* __restrict__ position,
                                                       const float* __restrict__ turns, float magnitude, float sign,
                                                       Head h, uint32_t items, uint32_t heads, uint16_t* y, int64_t yt,
                                                       int64_t yh) {
  const uint32_t item = blockIdx.x * kRopeThreads + threadIdx.x;
  if (item >= items) return;
  const uint32_t rest = item / (uint32_t)h.units;
  const int u = (int)(item - rest * (uint32_t)h.units);
  const uint32_t token = rest / heads;
  const int64_t head = rest - token * heads;
  float v[16];
  load_unit<kVec, kInter>(h, u, x + (int64_t)token * xt + head * xh, v);
  if (u < h.turning) {
    float cs[8], sn[8];
    unit_angles<kVec, kInter, false>(h, u, turns, (float)position[token], magnitude, sign, cs, sn);
    turn_unit<kInter>(v, cs, sn);
  }
  store_unit<kVec, kInter, true>(h, u, y + (int64_t)token * yt + head * yh, v);
}

// ---- bl_kv_append ----
// Grid: y = sequence; x = (touched page, head, k or v), then blocks that
// rotate q.  A workgroup owns one page of one head: absmax of the new values
// (rotated in fp32), then codes.  A thread's first unit stays in registers
// between the two steps, further ones are read again (from L2), which costs
// less than the registers: 5 prompts of up to 1777 tokens (64 + 2 x 8 heads of
// 128, 227 MB) take 51 us (4.5 TB/s) with one unit held, 53 with two; the
// queries' rotation, most of their bytes, hides the pages' loads and is no
// faster in a launch of its own (40 + 16 us).  64 sequences' single tokens of
// 20 + 2 x 5 heads take 4 us, a launch and its dependent loads (page number,
// absmax).  A prompt's queries are stored past the caches like k_rope's outputs
// (58 us against 60 with the read back; with the attention over the same prompts
// next 244 against 240; the decoder example's pass is the same), a decoded token's
// are left in them for the attention.
struct Rows {
  const uint16_t* p;
  int64_t token, head;
};

// Magnitudes as bits, which order like the values, a NaN above them all: it
// becomes the page's absmax instead of vanishing in a code.
__device__ __forceinline__ int block_max(int v, int* part, int threads) {
  v = wave_reduce<true>(v);
  if (threads > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < threads / 64; ++i) v = max(v, part[i]);
  }
  return v;
}

template <bool kVec, bool kInter, int T>
__global__ __launch_bounds__(T) void k_kv_append(KvView kv, KvStep st, Rows k, Rows v, Head kh, Head vh,
                                                 const float* __restrict__ turns, float magnitude, int page_blocks,
                                                 Rows q, int q_heads, uint16_t* q_out) {
  __shared__ int part[T / 64];
  constexpr int kHold = 1;
  const int s = blockIdx.y, tid = threadIdx.x;
  const int begin = st.begin(s), count = st.count(s, begin), start = st.start_of(s);
  int b = blockIdx.x;
  if (b >= page_blocks) {  // rotate q: units of this sequence's tokens and heads
    const uint32_t item = (uint32_t)(b - page_blocks) * T + tid;
    const uint32_t rest = item / (uint32_t)kh.units;
    const int u = (int)(item - rest * (uint32_t)kh.units);
    const uint32_t i = rest / (uint32_t)q_heads, head = rest - i * (uint32_t)q_heads;
    if ((int64_t)i >= count) return;
    const int64_t token = begin + (int64_t)i;
    float x[16];
    load_unit<kVec, kInter>(kh, u, q.p + token * q.token + head * q.head, x);
    if (u < kh.turning) {
      float cs[8], sn[8];
      unit_angles<kVec, kInter, false>(kh, u, turns, (float)((int64_t)start + i), magnitude, 1.0f, cs, sn);
      turn_unit<kInter>(x, cs, sn);
    }
    store_unit<kVec, kInter, T != 64>(kh, u, q_out + (token * q_heads + head) * kh.dim, x);
    return;
  }
  const bool is_v = b & 1;
  b >>= 1;
  const int head = b % kv.heads;
  const int64_t index = start / kv.page_tokens + b / kv.heads;  // page of the sequence
  const int64_t first = index * kv.page_tokens;                 // its first position
  if (count == 0 || first >= (int64_t)start + count || index >= st.table_stride) return;
  const int64_t page = st.page(s, index);
  if (page < 0 || page >= kv.pages) return;
  const int keep = start > first ? (int)(start - first) : 0;
  const int64_t last = (int64_t)start + count - first;
  const int rows = (int)(last < kv.page_tokens ? last : kv.page_tokens) - keep;
  const int64_t source = begin + (first + keep - start);  // token of the page's first new row
  const Head h = is_v ? vh : kh;
  const Rows in = is_v ? v : k;
  float* absmax = (is_v ? kv.v_absmax : kv.k_absmax) + page * kv.heads + head;
  int8_t* codes = (is_v ? kv.v : kv.k) + (page * kv.heads + head) * (int64_t)(kv.page_tokens * kv.dim);
  const float a_old = keep > 0 ? *absmax : 0.0f;

  const int lanes = h.units <= 1 ? 0 : 32 - __clz(h.units - 1);  // log2 of the lanes per row
  const int items = rows << lanes;
  auto fetch = [&](int item, float(&x)[16]) {
    const int row = item >> lanes, u = item & ((1 << lanes) - 1);
    const bool real = item < items && u < h.units;
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.0f;
    if (!real) return;
    const uint16_t* from = in.p + (source + row) * in.token + head * in.head;
    if (is_v) {  // nothing turns: its runs are whole
      load_unit<true, false>(h, u, from, x);
      return;
    }
    load_unit<kVec, kInter>(h, u, from, x);
    if (u < h.turning) {
      float cs[8], sn[8];
      unit_angles<kVec, kInter, true>(h, u, turns, (float)(first + keep + row), magnitude, 1.0f, cs, sn);
      turn_unit<kInter>(x, cs, sn);
    }
  };
  auto top_of = [](const float(&x)[16], int top) {
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_int(fabsf(x[j])));
    return top;
  };
  float held[kHold][16];
  int top = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    fetch(tid + i * T, held[i]);
    top = top_of(held[i], top);
  }
  for (int item = tid + kHold * T; item < items; item += T) {
    float x[16];
    fetch(item, x);
    top = top_of(x, top);
  }
  float a = __int_as_float(max(__float_as_int(a_old), block_max(top, part, T)));
  if (a < 0x1p-64f) a = 0.0f;
  const float scale = a > 0.0f ? 127.0f / a : 0.0f;
  auto put = [&](int item, const float(&x)[16]) {
    const int row = item >> lanes, u = item & ((1 << lanes) - 1);
    if (item >= items || u >= h.units) return;
    int8_t* to = codes + (int64_t)(keep + row) * kv.dim;
    if (is_v)
      store_codes<true, false>(h, u, to, x, scale);
    else
      store_codes<kVec, kInter>(h, u, to, x, scale);
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) put(tid + i * T, held[i]);
  for (int item = tid + kHold * T; item < items; item += T) {
    float x[16];
    fetch(item, x);
    put(item, x);
  }
  if (keep > 0 && a > a_old) {  // the page's scale grew: its earlier rows (adjacent bytes) take the new one
    const float ratio = a_old / a;
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int i = tid; i < keep * kv.dim / 16; i += T) {
      const uint4 w = old[i];
      auto four = [&](uint32_t d) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = __float_as_uint((float)((int)(d << (24 - 8 * j)) >> 24) * ratio + 12582912.0f);
        const uint32_t lo = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u);
        return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      };
      old[i] = make_uint4(four(w.x), four(w.y), four(w.z), four(w.w));
    }
  }
  if (T > 64) __syncthreads();  // every wave has its a_old
  if (tid == 0) *absmax = a;
}

// ---- bl_kv_read ----
// One thread per 16 codes of a token's head (chunk fastest); y = sequence, z = k
// or v.  36 MB (a third in, two thirds out) in 10 us: three dependent loads
// (lengths, page number, codes and scale) for one 16-byte piece of a thread.
constexpr int kReadThreads = 256;

__global__ __launch_bounds__(kReadThreads) void k_kv_read(KvView kv, KvStep st, uint16_t* __restrict__ k,
                                                          uint16_t* __restrict__ v) {
  const int s = blockIdx.y;
  const bool is_v = blockIdx.z;
  const int begin = st.begin(s), count = st.count(s, begin);
  const uint32_t chunks = (uint32_t)kv.dim / 16;
  const uint32_t item = blockIdx.x * kReadThreads + threadIdx.x;
  const uint32_t rest = item / chunks, c = item - rest * chunks;
  const uint32_t i = rest / (uint32_t)kv.heads, head = rest - i * (uint32_t)kv.heads;
  if ((int64_t)i >= count) return;
  const int64_t pos = (int64_t)st.start_of(s) + i, index = pos / kv.page_tokens;
  const int64_t page = index < st.table_stride ? st.page(s, index) : -1;
  uint4 w = make_uint4(0, 0, 0, 0);
  float step = 0.0f;
  if (page >= 0 && page < kv.pages) {
    const int64_t block = page * kv.heads + head;
    const int slot = (int)(pos - index * kv.page_tokens);
    w = *reinterpret_cast<const uint4*>((is_v ? kv.v : kv.k) + (block * kv.page_tokens + slot) * kv.dim + c * 16);
    step = (is_v ? kv.v_absmax : kv.k_absmax)[block] / 127.0f;
  }
  uint4 out[2];
  auto two = [&](uint32_t d, int j) {
    return f32x2_to_bf16x2((float)((int)(d << (24 - 8 * j)) >> 24) * step, (float)((int)(d << (16 - 8 * j)) >> 24) * step);
  };
  out[0] = make_uint4(two(w.x, 0), two(w.x, 2), two(w.y, 0), two(w.y, 2));
  out[1] = make_uint4(two(w.z, 0), two(w.z, 2), two(w.w, 0), two(w.w, 2));
  uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (((int64_t)begin + i) * kv.heads + head) * kv.dim + c * 16);
  dst[0] = out[0];
  dst[1] = out[1];
}

}  // namespace

hipError_t launch_rope(const uint16_t* x, int64_t xt, int64_t xh, const int32_t* position, const float* turns, int rot,
                       bool interleaved, float magnitude, int64_t tokens, int heads, int dim, bool inverse, uint16_t* y,
                       int64_t yt, int64_t yh, hipStream_t s) {
  const Head h = make_head(dim, rot);
  const float sign = inverse ? -1.0f : 1.0f;
  const int64_t items = tokens * heads * h.units, blocks = (items + kRopeThreads - 1) / kRopeThreads;
  if (!grid_fits(blocks, kRopeThreads)) return kErrGridTooLarge;
  auto go = [&](auto vec, auto inter) {
    hipLaunchKernelGGL((k_rope<decltype(vec)::value, decltype(inter)::value>), dim3((unsigned)blocks), dim3(kRopeThreads),
                       0, s, x, xt, xh, position, turns, magnitude, sign, h, (uint32_t)items, (uint32_t)heads, y, yt, yh);
    return hipGetLastError();
  };
  using std::bool_constant;
  auto by_layout = [&](auto vec) {
    return interleaved ? go(vec, bool_constant<true>{}) : go(vec, bool_constant<false>{});
  };
  return vector_runs(dim, rot) ? by_layout(bool_constant<true>{}) : by_layout(bool_constant<false>{});
}

hipError_t launch_kv_append(const KvView& kv, const KvStep& st, int64_t seqs, int64_t max_new, const uint16_t* k,
                            int64_t kt, int64_t kh, const uint16_t* v, int64_t vt, int64_t vh, const float* turns,
                            int rot, bool interleaved, float magnitude, const uint16_t* q, int64_t qt, int64_t qh,
                            int q_heads, uint16_t* q_out, hipStream_t s) {
  const Head hk = make_head(kv.dim, rot), hv = make_head(kv.dim, 0);
  const int64_t touched = (max_new + kv.page_tokens - 2) / kv.page_tokens + 1;
  const int64_t page_blocks = touched * kv.heads * 2;
  auto go = [&](auto vec, auto inter, auto t) {
    constexpr bool kVec = decltype(vec)::value, kInter = decltype(inter)::value;
    constexpr int T = decltype(t)::value;
    const int64_t q_items = q ? max_new * q_heads * hk.units : 0;
    const int64_t blocks = page_blocks + (q_items + T - 1) / T;
    if (q_items >= (int64_t)1 << 32 || !grid_fits(blocks, T) || !grid_fits(blocks * seqs, T)) return kErrGridTooLarge;
    hipLaunchKernelGGL((k_kv_append<kVec, kInter, T>), dim3((unsigned)blocks, (unsigned)seqs), dim3(T), 0, s, kv, st,
                       (Rows{k, kt, kh}), (Rows{v, vt, vh}), hk, hv, turns, magnitude, (int)page_blocks,
                       (Rows{q, qt, qh}), q_heads, q_out);
    return hipGetLastError();
  };
  using std::bool_constant;
  using std::integral_constant;
  auto pick = [&](auto inter, auto t) {
    return vector_runs(kv.dim, rot) ? go(bool_constant<true>{}, inter, t) : go(bool_constant<false>{}, inter, t);
  };
  auto by_layout = [&](auto t) {
    return interleaved ? pick(bool_constant<true>{}, t) : pick(bool_constant<false>{}, t);
  };
  // a page's new rows are few: one wave, no barrier
  if (max_new <= 8) return by_layout(integral_constant<int, 64>{});
  return by_layout(integral_constant<int, 256>{});
}

hipError_t launch_kv_read(const KvView& kv, const KvStep& st, int64_t seqs, int64_t max_new, uint16_t* k, uint16_t* v,
                          hipStream_t s) {
  const int64_t items = max_new * kv.heads * (kv.dim / 16), blocks = (items + kReadThreads - 1) / kReadThreads;
  if (items >= (int64_t)1 << 32 || !grid_fits(blocks, kReadThreads) || !grid_fits(blocks * seqs * 2, kReadThreads))
    return kErrGridTooLarge;
  hipLaunchKernelGGL(k_kv_read, dim3((unsigned)blocks, (unsigned)seqs, 2), dim3(kReadThreads), 0, s, kv, st, k, v);
  return hipGetLastError();
}

}  // namespace bl
