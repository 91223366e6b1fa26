// Log probabilities of given tokens, entropy and the most likely alternatives
// (bl_logprobs), and their gradient (bl_logprobs_backward).
//
// With c = scale * log2 e, M = max x, B = fl(M c) and d_j = fma(x_j, c, -B):
//   S = sum 2^d_j,  W = sum 2^d_j d_j,
//   entropy = (log2 S - W / S) ln 2.
// B's rounding is the same in every d, and known: delta = fma(M, c, -B).  With
// log_s = (log2 S - delta) ln 2,
//   lse = scale M + log_s,  logprob_j = scale (x_j - M) - log_s.
// From |M c| = 2^30 on (up to rows of the type's lowest value, where M c may
// overflow), fp32 numbers next to M are at least 2^6 away in d, so that only
// elements equal to M count: c is a power of two near scale log2 e then, for which
// M c and d are exact.  Below, delta is at most 32, which W / S is rounded at; it
// would leave the exponents' range from 2^31 on.  All sums are fp32.
//
// A row is cut into chunks that one workgroup each holds in registers: one
// reading of the logits gives the chunk's maximum, then (from the registers) S, W and
// the candidates for the alternatives.  A second kernel joins the chunks of a
// row.  4096 x 128256 bf16: 167 us, 6.3 TB/s with the vector pipe full, so bound by
// both; few rows: a chain of load, maximum and sums.
//
// Alternatives.  Wave w's r-th largest of its lanes' maxima, r = ceil(top /
// waves), has r elements of that wave at or above it, so at least top elements
// of the chunk are at or above the smallest of these over the waves: those are
// collected in LDS (a few times top of them, as a rule) and ranked by counting.
// Where they are too many (equal logits, logits in ascending order) the top-th
// largest is found by bisection first, which reads the chunk 64 times, from the
// caches (64 x 128256 bf16 with 20 alternatives: 286 and 276 us, 10 otherwise).
#include "device_util.h"
#include "internal.h"

namespace bl {
namespace {

typedef unsigned v4u __attribute__((ext_vector_type(4)));

constexpr int kCandidates = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -0x1.fffffep127f;

struct LogArgs {
  const char* x;
  int64_t stride;  // bytes
  int n, chunks, top;
  float scale, c;  // c = scale * log2 e
  const int32_t* target;
  float *logprob, *lse, *entropy;
  int32_t* top_id;
  float* top_logprob;
  float* stats;  // [row][chunk][4]: max, S, W, candidates
  uint2* best;   // [row][chunk][top]: value, index
};

// Elements of a row by 16-byte pieces: up to 16 / size - 1 before the first
// aligned address, whole pieces, the rest.
template <bool kBf16>
struct Pieces {
  static constexpr int kSize = kBf16 ? 2 : 4, kPer = 16 / kSize;
  const char* row;
  int head, vecs, tail;
  __device__ Pieces(const char* x, int64_t stride, int64_t r, int n) : row(x + r * stride) {
    head = min((int)(-(intptr_t)row & 15) / kSize, n);
    vecs = (n - head) / kPer;
    tail = n - head - vecs * kPer;
  }
  __device__ const v4u* vec(int i) const { return reinterpret_cast<const v4u*>(row + head * kSize) + i; }
  __device__ float at(int j) const {
    if (kBf16) return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(row)[j] << 16);
    return reinterpret_cast<const float*>(row)[j];
  }
  // the t-th element outside whole pieces
  __device__ int edge(int t) const { return t < head ? t : vecs * kPer + t; }
  __device__ int edges() const { return head + tail; }
};

template <bool kBf16>
__device__ __forceinline__ float element(const v4u& v, int j) {
  if (kBf16) return __uint_as_float(j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16);
  return __uint_as_float(v[j]);
}

// Integers that order like the values, -0 like +0.
__device__ __forceinline__ int order_of(float f) {
  const int b = __float_as_int(f + 0.0f);
  return b ^ (b >> 31 & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int order) { return __int_as_float(order ^ (order >> 31 & 0x7FFFFFFF)); }

// Larger values first, then lower indices: one number for both, no two alike.
__device__ __forceinline__ uint64_t place_of(float value, uint32_t index) {
  return (uint64_t)((uint32_t)order_of(value) ^ 0x80000000u) << 32 | (0xFFFFFFFFu - index);
}

// Sum over a wave, the same in every lane: lane moves inside rows of 16 (as in
// lane_group_reduce), then the rows' sums.
__device__ __forceinline__ float wave_sum(float v) {
  auto moved = [&](auto control) {
    const int b = __float_as_int(v);
    v += __int_as_float(__builtin_amdgcn_update_dpp(b, b, decltype(control)::value, 0xF, 0xF, false));
  };
  moved(std::integral_constant<int, 0xB1>{});
  moved(std::integral_constant<int, 0x4E>{});
  moved(std::integral_constant<int, 0x141>{});
  moved(std::integral_constant<int, 0x140>{});
  auto row = [&](int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// The r-th largest of the lanes' values (as order_of), the largest being top;
// INT_MIN if there is none.
__device__ __forceinline__ int wave_rth(int v, int top, int r) {
  for (int i = 1; i < r; ++i) {
    const uint64_t at = __ballot(v == top);
    if ((int)(threadIdx.x & 63) == __ffsll((unsigned long long)at) - 1) v = INT_MIN;
    top = wave_reduce<true>(v);
  }
  return top;
}

// What is taken off the exponents of a row or chunk whose maximum is top: b, or
// where that is far, top * c itself.
struct Shift {
  float b;
  bool far;
  __device__ Shift(float top, float c) : b(top == -INFINITY ? 0.0f : top * c), far(!(fabsf(b) < 0x1p30f)) {}
  // top * c - b, exactly; 0 where top * c may be infinite
  __device__ float rest(float top, float c) const {
    return fabsf(b) < 0x1p126f && top != -INFINITY ? __builtin_fmaf(top, c, -b) : 0.0f;
  }
};

// The exponents d = x * c - b of such a row or chunk, for its sums.
struct Exponents {
  float c, b;
  __device__ Exponents(const Shift& shift, float top, float c_) : c(c_), b(shift.b) {
    if (!shift.far) return;
    // more than c, so that nothing next to top counts, or less, so that nothing overflows
    const float power = __int_as_float(__float_as_int(c_) & 0x7F800000);
    c = fabsf(b) < 0x1p100f ? fminf(power, 0x1p125f) * 4.0f : power * 0.5f;
    b = top * c;
  }
  __device__ float operator()(float x) const { return __builtin_fmaf(x, c, -b); }
};

struct Final {
  float top, scale, log_s, entropy, lse;
  // max, S and W of a whole row; S is 0 where nothing is possible
  __device__ Final(const LogArgs& a, float most, float s, float w) : top(most), scale(a.scale) {
    const Shift shift(most, a.c);
    const float log2_s = __log2f(s), delta = shift.far ? 0.0f : shift.rest(most, a.c);
    log_s = (log2_s - delta) * kLn2;
    entropy = s == 0.0f ? 0.0f : (log2_s - w / s) * kLn2;
    lse = s == 0.0f ? -INFINITY : __builtin_fmaf(top, scale, log_s);
  }
  __device__ float logprob(float x) const {
    if (x == -INFINITY && log_s == log_s) return -INFINITY;
    const float d = x - top;
    if (d == -INFINITY) return __builtin_fmaf(x, scale, -(top * scale)) - log_s;  // scale d may be finite all the same
    return __builtin_fmaf(d, scale, -log_s);
  }
};

template <bool kBf16>
__device__ __forceinline__ void store_row(const LogArgs& a, int64_t row, const Final& f) {
  if (a.lse) a.lse[row] = f.lse;
  if (a.entropy) a.entropy[row] = f.entropy;
  if (a.logprob) {
    const int t = a.target[row];
    float v = 0.0f;
    if ((uint32_t)t < (uint32_t)a.n) v = f.logprob(Pieces<kBf16>(a.x, a.stride, row, a.n).at(t));
    a.logprob[row] = v;
  }
}

// Puts the `top` best of `count` candidates into out(rank, place), in order.
template <int kBlock, typename Out>
__device__ __forceinline__ void rank_candidates(const uint64_t* place, int count, int top, Out out) {
  for (int i = threadIdx.x; i < count; i += kBlock) {
    const uint64_t mine = place[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += place[j] > mine;
    if (rank < top) out(rank, mine);
  }
}

template <bool kBf16, int E, bool kTop, int kThreads>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogArgs a) {
  constexpr int kWaves = kThreads / 64;
  constexpr int kPer = Pieces<kBf16>::kPer;
  __shared__ float wave_top[kWaves], wave_s[kWaves], wave_w[kWaves];
  __shared__ int wave_limit[kWaves], counter[2];
  __shared__ uint64_t place[kTop ? kCandidates : 1];
  const int64_t row = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x - row * a.chunks);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Pieces<kBf16> p(a.x, a.stride, row, a.n);
  const int per = (p.vecs + a.chunks - 1) / a.chunks, v0 = min(chunk * per, p.vecs), v1 = min(v0 + per, p.vecs);
  if (kTop && tid == 0) counter[0] = 0;

  const uint32_t none = kBf16 ? 0xFF80FF80u : 0xFF800000u;  // -infinity, which counts for nothing
  v4u data[E];
  if (v0 < v1) {
#pragma unroll
    for (int i = 0; i < E; ++i) data[i] = *p.vec(min(v0 + i * kThreads + tid, v1 - 1));
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (v0 + i * kThreads + tid >= v1) data[i] = (v4u){none, none, none, none};
  float edge = -INFINITY;
  if (chunk == 0 && tid < p.edges()) edge = p.at(p.edge(tid));

  float most[E], top = edge == edge ? edge : -INFINITY;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    most[i] = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) most[i] = fmaxf(most[i], element<kBf16>(data[i], j));
    top = fmaxf(top, most[i]);
  }
  const int key = order_of(top);
  const int wave_key = wave_reduce<true>(key);
  if (lane == 0) wave_top[wave] = value_of(wave_key);
  const int full = max(min((v1 - v0) / 64, kWaves), 1);  // waves with an element in every lane
  if (kTop) {
    const int limit = wave_rth(key, wave_key, (a.top + full - 1) / full);
    if (lane == 0) wave_limit[wave] = limit;
  }
  __syncthreads();
  top = wave_top[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, wave_top[w]);
  float limit = INFINITY;
  if (kTop) {
    int least = wave_limit[0];
    for (int w = 1; w < full; ++w) least = min(least, wave_limit[w]);
    limit = fmaxf(value_of(max(least, order_of(-INFINITY))), kLowest);  // -infinity is no candidate
  }

  const Exponents exponent(Shift(top, a.c), top, a.c);
  float s = 0.0f, w = 0.0f;
  auto add = [&](float x) {
    const float d = exponent(x), e = __builtin_amdgcn_exp2f(d);
    s += e;
    w = __builtin_fmaf(e, fmaxf(d, -300.0f), w);  // 0 * -infinity is 0 here
  };
  // This thread's elements, each with its index, read again: the rare passes
  // over them take no registers from the first.
  auto each = [&](auto f) {
    if (chunk == 0 && tid < p.edges()) f(edge, (uint32_t)p.edge(tid));
#pragma clang loop unroll(disable)
    for (int v = v0 + tid; v < v1; v += kThreads) {
      const v4u d = *p.vec(v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) f(element<kBf16>(d, j), (uint32_t)(p.head + v * kPer + j));
    }
  };
  auto collect = [&](float x, uint32_t index) {
    const int at = atomicAdd(&counter[0], 1);
    if (at < kCandidates) place[at] = place_of(x, index);
  };
  add(edge);
  int hits = 0;  // pieces with candidates
#pragma unroll
  for (int i = 0; i < E; ++i) {
    asm("" : "+v"(data[i]));  // taken apart anew: elements kept from above would take twice the registers
#pragma unroll
    for (int j = 0; j < kPer; ++j) add(element<kBf16>(data[i], j));
    if (kTop) hits |= (most[i] >= limit) << i;
  }
  if (kTop) {
    // Few lanes have one, and one as a rule: loops, since code that is not in the
    // instruction cache costs more (unrolled, one row of 128256 bf16 took 1 us more).
    if (edge >= limit) collect(edge, (uint32_t)p.edge(tid));
    while (hits) {
      const int i = __ffs(hits) - 1;
      hits &= hits - 1;
      v4u d = data[0];
#pragma unroll
      for (int k = 1; k < E; ++k)
        if (k == i) d = data[k];
      int bits = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) bits |= (element<kBf16>(d, j) >= limit) << j;
      while (bits) {
        const int j = __ffs(bits) - 1, word = kBf16 ? j >> 1 : j;
        bits &= bits - 1;
        const uint32_t w = word & 2 ? (word & 1 ? d[3] : d[2]) : (word & 1 ? d[1] : d[0]);
        const float x = __uint_as_float(!kBf16 ? w : j & 1 ? w & 0xFFFF0000u : w << 16);
        collect(x, (uint32_t)(p.head + (v0 + i * kThreads + tid) * kPer + j));
      }
    }
  }
  asm("" : "+v"(s), "+v"(w));  // summed here, not behind the branch with all terms kept until there
  s = wave_sum(s);
  w = wave_sum(w);
  if (lane == 0) {
    wave_s[wave] = s;
    wave_w[wave] = w;
  }
  __syncthreads();
  int count = kTop ? counter[0] : 0;
  if (kTop && count > kCandidates) {
    // the largest place that `top` elements reach, bit by bit
    uint64_t reach = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const uint64_t tried = reach | (uint64_t)1 << bit;
      int here = 0;
      each([&](float x, uint32_t index) { here += x > -INFINITY && place_of(x, index) >= tried; });
      here = wave_reduce<false>(here);
      __syncthreads();
      if (lane == 0) wave_limit[wave] = here;
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) all += wave_limit[i];
      if (all >= a.top) reach = tried;
    }
    if (tid == 0) counter[0] = 0;
    __syncthreads();
    each([&](float x, uint32_t index) {
      if (x > -INFINITY && place_of(x, index) >= reach) collect(x, index);
    });
    __syncthreads();
    count = counter[0];
  }
  s = w = 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    s += wave_s[i];
    w += wave_w[i];
  }
  if (a.chunks == 1) {
    const Final f(a, top, s, w);
    if (tid == 0) store_row<kBf16>(a, row, f);
    if (kTop) {
      int32_t* ids = a.top_id + row * a.top;
      float* values = a.top_logprob + row * a.top;
      rank_candidates<kThreads>(place, count, a.top, [&](int rank, uint64_t q) {
        ids[rank] = (int32_t)(0xFFFFFFFFu - (uint32_t)q);
        values[rank] = f.logprob(value_of((int)((uint32_t)(q >> 32) ^ 0x80000000u)));
      });
      for (int i = count + tid; i < a.top; i += kThreads) {
        ids[i] = -1;
        values[i] = -INFINITY;
      }
    }
    return;
  }
  const int64_t slot = row * a.chunks + chunk;
  if (tid == 0) *reinterpret_cast<float4*>(a.stats + 4 * slot) = make_float4(top, s, w, __int_as_float(min(count, a.top)));
  if (kTop)
    rank_candidates<kThreads>(place, count, a.top, [&](int rank, uint64_t q) {
      a.best[slot * a.top + rank] = make_uint2((uint32_t)q, (uint32_t)(q >> 32));
    });
}

// One workgroup per row joins its chunks.
constexpr int kJoinThreads = 256;
template <bool kBf16, bool kTop>
__global__ __launch_bounds__(kJoinThreads) void k_logprobs_join(LogArgs a) {
  __shared__ uint64_t place[kTop ? kMaxLogChunks * kMaxTop : 1];
  __shared__ int counter;
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63;
  if (kTop && tid == 0) counter = 0;
  // what is read goes out at once: the chunks' numbers, their alternatives (as
  // many as four per thread), and in another wave the token's logit
  const int held_best = kTop ? a.chunks * a.top : 0;
  const int of_chunks = min(a.chunks, 8), r = (a.top + of_chunks - 1) / of_chunks;
  const uint2* best = a.best + row * a.chunks * a.top;
  uint2 ahead[kTop ? 4 : 1];
  uint32_t rth = 0;
  if (kTop) {
#pragma unroll
    for (int i = 0; i < 4; ++i) ahead[i] = best[min(tid + i * kJoinThreads, held_best - 1)];
    rth = best[min(lane, a.chunks - 1) * a.top + r - 1].y;
  }
  float4 part = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
  if (lane < a.chunks) part = *reinterpret_cast<const float4*>(a.stats + 4 * (row * a.chunks + lane));
  const float top = value_of(wave_reduce<true>(order_of(part.x)));  // every wave has the row's
  // S and W relative to the row's maximum: from what was taken off in the chunk to
  // what is in the row, which may be far where the other is not
  const Shift whole(top, a.c), own(part.x, a.c);
  float shift = own.b - whole.b;
  if (own.far && whole.far)
    shift = (part.x - top) * a.c;
  else if (own.far || whole.far)
    shift += own.far ? own.rest(part.x, a.c) : -whole.rest(top, a.c);
  if (part.x == -INFINITY) shift = 0.0f;
  const float e = __builtin_amdgcn_exp2f(shift);
  const float s = wave_sum(part.y * e), w = wave_sum(e * __builtin_fmaf(part.y, fmaxf(shift, -300.0f), part.z));
  const Final f(a, top, s, w);
  if (tid == kJoinThreads - 1) store_row<kBf16>(a, row, f);
  if (!kTop) return;
  // at least `top` are at or above the eighth largest (the least, of fewer) of the
  // chunks' r-th best
  const int held = __float_as_int(part.w);
  int limit = lane < a.chunks && held >= r ? (int)(rth ^ 0x80000000u) : INT_MIN;
  limit = wave_rth(limit, wave_reduce<true>(limit), of_chunks);
  __syncthreads();
  for (int base = 0; base < held_best; base += 4 * kJoinThreads) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = base + tid + i * kJoinThreads, chunk = min(k, held_best - 1) / a.top;
      const int there = __shfl(held, chunk, 64);
      if (k < held_best && k - chunk * a.top < there && (int)(ahead[i].y ^ 0x80000000u) >= limit)
        place[atomicAdd(&counter, 1)] = (uint64_t)ahead[i].y << 32 | ahead[i].x;
    }
    if (base + 4 * kJoinThreads < held_best) {
#pragma unroll
      for (int i = 0; i < 4; ++i) ahead[i] = best[min(base + 4 * kJoinThreads + tid + i * kJoinThreads, held_best - 1)];
    }
  }
  __syncthreads();
  const int count = counter;
  int32_t* ids = a.top_id + row * a.top;
  float* values = a.top_logprob + row * a.top;
  rank_candidates<kJoinThreads>(place, count, a.top, [&](int rank, uint64_t q) {
    ids[rank] = (int32_t)(0xFFFFFFFFu - (uint32_t)q);
    values[rank] = f.logprob(value_of((int)((uint32_t)(q >> 32) ^ 0x80000000u)));
  });
  for (int i = count + tid; i < a.top; i += kJoinThreads) {
    ids[i] = -1;
    values[i] = -INFINITY;
  }
}

// ---- gradient ----
//   dx_j = scale * (g [j = t] + p_j (gz - g - gh (log p_j + H)))
// with p_j = 2^d, d = fma(x_j, scale, -lse) log2 e.  Rows whose gradients are all
// zero, and rows where nothing is possible, get zeros without being read.  The
// last rows come first: the forward call has left them in the Infinity Cache;
// stores (and loads, which are the last of a row) go past the caches.  4096 x 128256
// bf16, forward and this: 550 us, 605 in ascending order through the caches.
//
// lse is one fp32 number, so every p of a row is off by up to half its unit: 2^-19
// at 64, a factor n for a row of the type's lowest value, where log n is lost.
// From kFarLse on a row's sum of exponentials is taken again, by one of its
// workgroups, which then does the whole row (it may be overwritten in place): p_j =
// 2^(d_j - log2 S) with d_j from any one shift near the maximum.  Row r's is that of
// chunk r % chunks: the first ones may all lie on one XCD (4096 x 128256 bf16 at
// logits around 1000: 653 us, 4032 with them, 394 of a batch around 0).
// Below, the unit is within the exponent's own roundings (fp32) or under a
// sixtieth of the output's (bf16).
struct GradArgs {
  const char* x;
  int64_t x_stride;
  char* dx;
  int64_t dx_stride;
  int n, chunks;
  float scale;
  const int32_t* target;
  const float *lse, *entropy, *g, *gh, *gz;
};

template <bool kBf16>
constexpr float kFarLse = kBf16 ? 512.0f : 64.0f;
// From here on half a unit of lse is no small exponent: the maximum is looked for.
constexpr float kLostLse = 0x1p24f;

constexpr int kGradThreads = 256;
template <bool kBf16, int E, bool kAligned>
__global__ __launch_bounds__(kGradThreads) void k_logprobs_backward(GradArgs a) {
  typedef Pieces<kBf16> P;
  constexpr int kPer = P::kPer, kWaves = kGradThreads / 64;
  __shared__ float part[kWaves];
  const uint32_t block = gridDim.x - 1 - blockIdx.x;
  const int64_t row = block / a.chunks;
  const int chunk = (int)(block - row * a.chunks), tid = threadIdx.x;
  const P p(a.x, a.x_stride, row, a.n);
  const int per = (p.vecs + a.chunks - 1) / a.chunks, v0 = min(chunk * per, p.vecs), v1 = min(v0 + per, p.vecs);
  const int t = a.target ? a.target[row] : -1;
  const float lse = a.lse[row];
  const float g = a.g && (uint32_t)t < (uint32_t)a.n ? a.g[row] : 0.0f;
  const float gh = a.gh ? a.gh[row] : 0.0f, gz = a.gz ? a.gz[row] : 0.0f;
  const bool zero = lse == -INFINITY || (g == 0.0f && gh == 0.0f && gz == 0.0f);
  const float plain = a.scale * (gz - g - (gh != 0.0f ? gh * a.entropy[row] : 0.0f)), slope = -a.scale * gh * kLn2;
  const float hit = zero ? 0.0f : a.scale * g;
  char* out = a.dx + row * a.dx_stride;
  auto weigh = [&](float d) { return __builtin_amdgcn_exp2f(d) * __builtin_fmaf(slope, fmaxf(d, -300.0f), plain); };
  auto store = [&](int j, float v) {
    if (kBf16)
      reinterpret_cast<uint16_t*>(out)[j] = f32_to_bf16_rne(v);
    else
      reinterpret_cast<float*>(out)[j] = v;
  };
  auto store_piece = [&](int v, const v4u& data, auto value) {
    const int first = p.head + v * kPer;
    float y[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) y[j] = value(element<kBf16>(data, j));
    if ((uint32_t)(t - first) < (uint32_t)kPer) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) y[j] += first + j == t ? hit : 0.0f;
    }
    if (kAligned) {
      v4u w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = kBf16 ? f32x2_to_bf16x2(y[2 * j % kPer], y[(2 * j + 1) % kPer]) : __float_as_uint(y[j]);
      __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(out + (int64_t)first * P::kSize));
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) store(first + j, y[j]);
    }
  };
  const bool alone = !zero && fabsf(lse) >= kFarLse<kBf16>;
  const int leader = alone ? (int)(row % a.chunks) : 0;
  const bool has_edge = chunk == leader && tid < p.edges();
  const int edge = has_edge ? p.edge(tid) : 0;

  if (alone) {
    if (chunk != leader) return;
    const float at_edge = has_edge ? p.at(edge) : -INFINITY;
    auto pieces = [&](auto f) {  // E at a time
#pragma clang loop unroll(disable)
      for (int base = tid; base < p.vecs; base += E * kGradThreads) {
        v4u d[E];
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = *p.vec(min(base + i * kGradThreads, p.vecs - 1));
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (base + i * kGradThreads < p.vecs) f(base + i * kGradThreads, d[i]);
      }
    };
    const float c = a.scale * kLog2e;
    float top = at_edge, b = lse * kLog2e;
    bool far = false;
    if (fabsf(lse) >= kLostLse) {
      pieces([&](int, const v4u& d) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) top = fmaxf(top, element<kBf16>(d, j));
      });
      top = value_of(wave_reduce<true>(order_of(top)));
      if ((tid & 63) == 0) part[tid >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, part[w]);
      __syncthreads();  // part is written again
      const Shift shift(top, c);
      b = shift.b;
      far = shift.far;
    }
    // every weight's own here, however small
    auto exponent = [&](float x) { return far ? (x - top) * c : __builtin_fmaf(x, c, -b); };
    double all = __builtin_amdgcn_exp2f(exponent(at_edge));  // a thread's sum is a long one
    pieces([&](int, const v4u& d) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) s += __builtin_amdgcn_exp2f(exponent(element<kBf16>(d, j)));
      all += s;
    });
    const float s = wave_sum((float)all);
    if ((tid & 63) == 0) part[tid >> 6] = s;
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[w];
    const float log2_s = __log2f(sum);
    auto value = [&](float x) { return weigh(exponent(x) - log2_s); };
    if (has_edge) store(edge, value(at_edge) + (edge == t ? hit : 0.0f));
    pieces([&](int v, const v4u& d) { store_piece(v, d, value); });
    return;
  }

  auto value = [&](float x) { return zero ? 0.0f : weigh(__builtin_fmaf(x, a.scale, -lse) * kLog2e); };
  if (has_edge) store(edge, (zero ? 0.0f : value(p.at(edge))) + (edge == t ? hit : 0.0f));
  v4u data[E];
  if (!zero && v0 < v1) {
#pragma unroll
    for (int i = 0; i < E; ++i) data[i] = __builtin_nontemporal_load(p.vec(min(v0 + i * kGradThreads + tid, v1 - 1)));
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int v = v0 + i * kGradThreads + tid;
    if (v < v1) store_piece(v, data[i], value);
  }
}

// One workgroup holds a row, in one launch, where the row has up to 4096 pieces
// of 16 bytes (32768 bf16): 512 threads if rows are many, 1024 if few; for few
// rows up to 8192 (37 x 32003 fp32 6.6 us, 9.5 in chunks and a join; 2000 x 60000
// bf16 51 against 43; with alternatives 1 x 65000 9.1 against 10.1, but 333 x 30000
// fp32 15.7 against 14.6).  Longer rows are cut into chunks of eight pieces per
// thread while these still make a workgroup per CU, of fewer for few rows (64 x
// 128256 bf16 with 20 alternatives: 12.7 us at 256 workgroups, 13.4 at 512, 14.6 at
// 1024, 19 at 2048); never into more than the joining workgroup holds.
struct LogPlan {
  int threads, e;
  int64_t chunks;
};
LogPlan log_plan(int64_t m, int64_t n, bool bf16, bool top) {
  const int64_t vecs = bf16 ? (n + 7) / 8 : (n + 3) / 4;
  if (vecs <= 4096 || (vecs <= 8192 && m < (top ? 32 : 512))) {
    const int threads = vecs <= 512 || (m >= 512 && vecs <= 4096) ? 512 : 1024;
    int e = 1;
    while (e * threads < vecs) e <<= 1;
    return {threads, e, 1};
  }
  auto chunks = [&](int e) { return (vecs + e * 512 - 1) / (e * 512); };
  int e = 8;
  while (e > 1 && m * chunks(e) < 256 && chunks(e / 2) <= kMaxLogChunks) e >>= 1;
  return {512, e, chunks(e)};
}

}  // namespace

size_t logprobs_workspace_bytes(int64_t m, int64_t n, bool bf16, int64_t top) {
  const LogPlan p = log_plan(m, n, bf16, top > 0);
  return p.chunks == 1 ? 0 : (size_t)(m * p.chunks) * (16 + 8 * (size_t)top);
}

hipError_t launch_logprobs(const void* x, bool bf16, int64_t m, int64_t n, int64_t stride, float scale,
                           const int32_t* target, int64_t top, float* logprob, float* lse, float* entropy, int32_t* top_id,
                           float* top_logprob, void* workspace, hipStream_t s) {
  const LogPlan p = log_plan(m, n, bf16, top > 0);
  if (!grid_fits(m * p.chunks, p.threads)) return kErrGridTooLarge;
  LogArgs a = {(const char*)x, stride * (bf16 ? 2 : 4), (int)n,      (int)p.chunks, (int)top, scale, scale * kLog2e,
               target,         logprob,                 lse,     entropy,       top_id,   top_logprob};
  a.stats = (float*)workspace;
  a.best = (uint2*)(a.stats + 4 * m * p.chunks);
  const dim3 grid((unsigned)(m * p.chunks));
  auto go = [&](auto b, auto with_top, auto e) {
    constexpr bool kBf16 = decltype(b)::value, kTop = decltype(with_top)::value;
    constexpr int E = decltype(e)::value;
    if (p.threads == 1024)
      hipLaunchKernelGGL((k_logprobs<kBf16, E, kTop, 1024>), grid, dim3(1024), 0, s, a);
    else
      hipLaunchKernelGGL((k_logprobs<kBf16, E, kTop, 512>), grid, dim3(512), 0, s, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || p.chunks == 1) return err;
    hipLaunchKernelGGL((k_logprobs_join<kBf16, kTop>), dim3((unsigned)m), dim3(kJoinThreads), 0, s, a);
    return hipGetLastError();
  };
  using std::bool_constant;
  using std::integral_constant;
  auto by_e = [&](auto b, auto with_top) {
    switch (p.e) {
      case 1: return go(b, with_top, integral_constant<int, 1>{});
      case 2: return go(b, with_top, integral_constant<int, 2>{});
      case 4: return go(b, with_top, integral_constant<int, 4>{});
      default: return go(b, with_top, integral_constant<int, 8>{});
    }
  };
  auto by_top = [&](auto b) { return top > 0 ? by_e(b, bool_constant<true>{}) : by_e(b, bool_constant<false>{}); };
  return bf16 ? by_top(bool_constant<true>{}) : by_top(bool_constant<false>{});
}

hipError_t launch_logprobs_backward(const void* x, bool bf16, int64_t m, int64_t n, int64_t stride, float scale,
                                    const int32_t* target, const float* lse, const float* entropy, const float* g,
                                    const float* gh, const float* gz, void* dx, int64_t dx_stride, hipStream_t s) {
  constexpr int E = 4;
  const int size = bf16 ? 2 : 4, per = 16 / size;
  const int64_t vecs = (n + per - 1) / per, chunks = (vecs + E * kGradThreads - 1) / (E * kGradThreads);
  if (!grid_fits(m * chunks, kGradThreads)) return kErrGridTooLarge;
  const GradArgs a = {(const char*)x, stride * size, (char*)dx, dx_stride * size, (int)n, (int)chunks, scale,
                      target,         lse,           entropy,   g,                gh,     gz};
  // rows of both begin alike within 16 bytes: whole pieces of one are whole pieces of the other
  const bool aligned = ((intptr_t)x - (intptr_t)dx) % 16 == 0 && (m == 1 || (stride - dx_stride) * size % 16 == 0);
  const dim3 grid((unsigned)(m * chunks)), block(kGradThreads);
  if (bf16) {
    if (aligned)
      hipLaunchKernelGGL((k_logprobs_backward<true, E, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_logprobs_backward<true, E, false>), grid, block, 0, s, a);
  } else {
    if (aligned)
      hipLaunchKernelGGL((k_logprobs_backward<false, E, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((k_logprobs_backward<false, E, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace bl
