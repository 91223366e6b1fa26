// Attention over the 8-bit key/value cache (bl_attention).
//
// out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale * q_r . k_j), one pass
// over the keys with a running maximum and sum per row.  In base 2 and with
// the absmax values of the page of j (ka, va) taken out of the products:
//   t_rj = (q_r . K_j) * c_r * ka + log2(va),  P = 2^(t - m + 14),
//   O += P * V_j (codes),  l += P / va,  out = O / l / 127,
// m being the running maximum of t.  Taking va into the exponent keeps every P
// at or below 2^14 whatever the pages' scales, so P fits fp16 with 11 bits of
// precision for every term above 2^-28 of the row's largest contribution; l is
// summed in fp32 from the unrounded P.  A page of zeros has an absmax of 0: it
// counts as 2^-64, below which bl_kv_append keeps none, so that its weights
// reach l (at most 2^29 keys of 2^15.5 * 2^64) and do not push the others'
// below fp16's range.
//
// Products.  Keys stay int8: a query row becomes 16-bit integers (absmax /
// 32512 per step), split into signed high and low bytes, and two int8 MFMAs
// give the exact integer dot product (256 * high + low, below 2^31 for
// dim <= 256) at the cost of one bf16 MFMA and no conversion of K.  Values
// become fp16 on the way to the fp16 MFMA: v_perm_b32 picks a byte of two
// tokens into two halves, where the offset code u = q + 128 is the denormal
// u * 2^-24, and one packed fma gives (u - 128) * 2^-9 exactly: about 1.25
// instructions per element.
//
// Layouts.  S^T = K Q^T leaves tokens 4g + i (g = lane / 16) of a 16-token
// tile with query lane % 16; the k-slots of O^T = V^T P^T are numbered so that
// the same lane feeds them (slot 8g + j: token 4g + j of the first tile for
// j < 4, 4g + j - 4 of the second), so P never leaves its lane.  V's row slot
// m of MFMA tile t is element 4 DC m + t, so a lane reads 4 DC adjacent bytes
// of a token and ends with 16 DC adjacent outputs of its query.
#include "device_util.h"
#include "internal.h"

namespace bl {
namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 64;       // keys per step of a wave
constexpr float kLeastAbsmax = 0x1p-64f;
// A running maximum that nothing has raised: below every score (those that
// overflow are not seen), finite so that differences of two are 0.
constexpr float kNone = -0x1.fffffep127f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Attn {
  KvView kv;
  KvStep st;
  const uint16_t* q;
  int64_t qt, qh;
  int q_heads, group, page_shift;
  int max_len;
  int window, sinks;
  float scale;       // of q . k, in base 2
  int tile_rows;     // rows of a tile (16 or kPromptRows)
  int row_tiles;     // tiles per sequence and head
  int tiles;
  int splits, per;   // workgroups along the keys, steps of each
  uint16_t* out;
  float* lse;
  float* part_o;   // [token][q_head][split][dim]
  float* part_ml;  // [token][q_head][split][2]
};

// Wave-uniform values that nothing writes while the kernel runs (page numbers,
// page scales), through scalar loads: a vector load of one would be waited for
// together with all key and value loads in flight.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) T*>(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ int64_t page_number(const KvStep& st, int seq, int64_t index) {
  return uniform_load(st.page_table + seq * st.table_stride + index);
}

// The steps of keys that rows at positions first_pos .. last_pos take.  The
// lengths that the host planned for end at max_len, wherever the device's
// positions lead: keys from there on are not seen, so that no tile has more
// steps than the plan and its workspace hold.  There is one step at least (all
// masked, if nothing is visible), so every row is written.
struct Span {
  int keys;  // keys 0 .. keys-1 may be visible
  int sink_steps, base, steps;
  __host__ __device__ int key0(int step) const { return (step < sink_steps ? step : base + step - sink_steps) * kStep; }
};

__host__ __device__ inline Span span_of(int first_pos, int last_pos, int max_len, int window, int sinks) {
  Span s;
  s.keys = last_pos < max_len ? last_pos + 1 : max_len;
  const int last = (s.keys + kStep - 1) / kStep, from = first_pos - window + 1;
  s.base = window > 0 && from > 0 ? from / kStep : 0;
  if (s.base > last - 1) s.base = last - 1;
  s.sink_steps = (sinks + kStep - 1) / kStep;
  if (s.sink_steps > s.base) s.sink_steps = s.base;
  s.steps = s.sink_steps + last - s.base;
  return s;
}

// The rows and steps of one tile.
struct Tile : Span {
  int seq, head, begin, rows, row0, start;
  int first_pos, last_pos;  // positions of its first and last row
};

// Workgroups are dealt to the eight XCDs in turn: eight tiles are taken
// together, split by split, so that all splits of a tile run on one XCD and
// every XCD gets tiles of all lengths.
__device__ __forceinline__ bool tile_and_split(const Attn& a, int& index, int& split) {
  if (a.tiles < 64) {  // too few to spread by eights
    index = blockIdx.x / a.splits;
    split = blockIdx.x - index * a.splits;
    return index < a.tiles;
  }
  const int eight = blockIdx.x / (8 * a.splits), rest = blockIdx.x - eight * 8 * a.splits;
  split = rest >> 3;
  index = eight * 8 + (rest & 7);
  return index < a.tiles;
}

__device__ __forceinline__ bool find_tile(const Attn& a, int index, Tile& t) {
  const int rest = index / a.row_tiles;
  const int rt = index - rest * a.row_tiles;
  t.seq = rest / a.kv.heads;
  t.head = rest - t.seq * a.kv.heads;
  const KvStep& st = a.st;  // the three integers in one round trip
  const int from = uniform_load(st.offsets + t.seq), to = uniform_load(st.offsets + t.seq + 1);
  const int start = uniform_load(st.start + t.seq);
  t.begin = st.begin_of(from);
  const int count = st.count_of(t.begin, to);
  t.rows = count * a.group;
  t.row0 = rt * a.tile_rows;
  if (t.row0 >= t.rows) return false;
  t.start = st.start_from(start);
  t.first_pos = t.start + t.row0 / a.group;
  t.last_pos = t.start + (min(t.row0 + a.tile_rows, t.rows) - 1) / a.group;
  static_cast<Span&>(t) = span_of(t.first_pos, t.last_pos, a.max_len, a.window, a.sinks);
  return true;
}

// Largest value over lanes l and l ^ 32: v_permlane32_swap of a register with
// a copy leaves the low half in both halves of one and the high half in both of
// the other.
__device__ __forceinline__ float halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The same over the four rows of 16 lanes (l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float rows_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

// A query row (zeros past dim) as high and low bytes, in kChunks chunks of
// kWidth elements; lane group g of the kWidth / 16 that share a row holds
// elements kWidth c + 16 g .. +15.  Returns absmax / 32512.
template <int kWidth, int kChunks>
__device__ __forceinline__ float split_query(const uint16_t* row, bool valid, int dim, int g, v4i (&hi)[kChunks],
                                             v4i (&lo)[kChunks]) {
  uint4 d[kChunks][2];
  u16x2 most = {0, 0};
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    d[c][0] = d[c][1] = make_uint4(0, 0, 0, 0);
    if (valid && kWidth * c + 16 * g < dim) {
      const uint4* p = reinterpret_cast<const uint4*>(row + kWidth * c + 16 * g);
      d[c][0] = p[0];
      d[c][1] = p[1];
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) most = absmax_step(absmax_step(most, d[c][0]), d[c][1]);
  // as bits, which order like the values and hold a NaN (then every score is one)
  int top_bits = (int)max(most.x, most.y) << 16;
  if (kWidth == 64) top_bits = max(top_bits, __shfl_xor(top_bits, 16, 64));
  top_bits = max(top_bits, __shfl_xor(top_bits, 32, 64));
  const float top = __int_as_float(top_bits);
  const float s = top > 0x1p-100f ? 32512.0f / top : 0.0f;
  // x * s + 1.5 * 2^23 has the code (at most 32512 in magnitude) in its low
  // bytes; 128 more carries the low byte's sign into the high one
  auto pack = [](const uint32_t(&u)[4], uint32_t two) {  // one byte of each of four words
    const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], two), b = __builtin_amdgcn_perm(u[3], u[2], two);
    return (int)__builtin_amdgcn_perm(b, a, 0x05040100u);
  };
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint32_t w[8] = {d[c][0].x, d[c][0].y, d[c][0].z, d[c][0].w, d[c][1].x, d[c][1].y, d[c][1].z, d[c][1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t half = w[2 * i + (j >> 1)];
        u[j] = __float_as_uint(__builtin_fmaf(__uint_as_float(j & 1 ? half & 0xFFFF0000u : half << 16), s, 12582912.0f));
      }
      lo[c][i] = pack(u, 0x0c0c0400u);
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] += 128;
      hi[c][i] = pack(u, 0x0c0c0501u);
    }
  }
  return top * (1.0f / 32512.0f);
}

// Bytes b of two tokens' dwords (offset codes) as fp16 (u - 128) * 2^-9.
__device__ __forceinline__ uint32_t halves_of(uint32_t w0, uint32_t w1, int b) {
  const uint32_t sel = 0x0c000c04u + 0x00010001u * (uint32_t)b;  // [w0.b, 0, w1.b, 0]: bytes 0-3 are w1's, 4-7 w0's
  const uint32_t u = __builtin_amdgcn_perm(w0, w1, sel);
  const v2h scaled = __builtin_elementwise_fma(__builtin_bit_cast(v2h, u), (v2h){(_Float16)32768.0f, (_Float16)32768.0f},
                                               (v2h){(_Float16)-0.25f, (_Float16)-0.25f});
  return __builtin_bit_cast(uint32_t, scaled);
}

// The 4 DC adjacent bytes of a token that a lane of k_attn reads, by words.
template <int DC>
struct VBytes;
template <>
struct VBytes<1> {
  typedef uint32_t type;
  static __device__ uint32_t word(type v, int) { return v; }
};
template <>
struct VBytes<2> {
  typedef uint32_t type __attribute__((ext_vector_type(2)));
  static __device__ uint32_t word(type v, int c) { return v[c]; }
};
template <>
struct VBytes<4> {
  typedef uint32_t type __attribute__((ext_vector_type(4)));
  static __device__ uint32_t word(type v, int c) { return v[c]; }
};

// The running maximum m is raised only when a score passes it by more than
// this: P is then at most 2^(14 + kSlack) < 65504, and almost every step keeps
// its O and l as they are.
constexpr float kSlack = 1.5f;

// One workgroup: 16 query rows of one sequence and cache head, the steps of
// one split; wave w takes steps w, w + 4, ... with its own running state, and
// the waves' states are joined in LDS at the end.  A step's keys and values go
// straight into registers; the next step's keys are asked for as soon as the
// products have read this step's, its values as soon as those are converted, so
// that loads are in flight nearly all the time without a second set of
// registers (three waves per SIMD, 16 KB in flight each).  HBM-bound: 24
// sequences of up to 32768 tokens, 64/8 heads of 128 (883 MB): 160 us, 5.5 TB/s,
// and 9 us for the join; one token over 1500 (20/5 heads): 7.3 + 4.4 us, the
// chain of page number, keys, products, meeting of the waves, join.
// kPages: pages that 64 tokens lie in (1, or 4 for pages of 16 and
// 32 tokens, looked up for each 16 tokens).
template <int DC, int kPages>
__global__ __launch_bounds__(kThreads, DC == 1 ? 4 : DC == 2 ? (kPages == 1 ? 3 : 2) : 1) void k_attn(Attn a) {
  typedef typename VBytes<DC>::type vbytes;
  __shared__ float lds_o[kWaves][16][64 * DC + 4];  // rows four banks apart
  __shared__ float lds_ml[kWaves][16][2];
  int index, split;
  if (!tile_and_split(a, index, split)) return;
  Tile t;
  if (!find_tile(a, index, t)) return;
  const int s0 = split * a.per, s1 = min(t.steps, s0 + a.per);
  if (s0 >= s1) return;
  const bool whole = t.steps <= a.per;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int dim = a.kv.dim, row = t.row0 + col;
  const bool valid = row < t.rows;
  const int token = valid ? row / a.group : 0;
  const int q_head = t.head * a.group + (valid ? row - token * a.group : 0);
  const int pos = t.start + token, low = a.window > 0 ? pos - a.window + 1 : 0;

  // byte offsets inside a 16-token tile; elements past dim read element 0
  // instead (their query bytes are zero, their outputs are not stored)
  uint32_t koff[DC], voff;
#pragma unroll
  for (int c = 0; c < DC; ++c) koff[c] = (uint32_t)(col * dim + (64 * c + 16 * g < dim ? 64 * c + 16 * g : 0));
  voff = (uint32_t)(4 * g * dim + (4 * DC * col < dim ? 4 * DC * col : 0));

  struct Place {  // of a step's keys and values
    int64_t at[kPages];
    float ka[kPages], va[kPages];
    bool there[kPages];
  };
  auto look_up = [&](int step, int64_t(&page)[kPages]) {
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int key = step < s1 ? t.key0(step) + kStep / kPages * i : t.keys;
      page[i] = key < t.keys ? page_number(a.st, t.seq, key >> a.page_shift) : -1;
    }
  };
  auto place = [&](int step, const int64_t(&page)[kPages], Place& p) {
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      const int key = t.key0(step) + kStep / kPages * i;
      p.there[i] = page[i] >= 0 && page[i] < a.kv.pages;
      const int64_t block = p.there[i] ? page[i] * a.kv.heads + t.head : 0;
      p.at[i] = (block * a.kv.page_tokens + (p.there[i] ? key & (a.kv.page_tokens - 1) : 0)) * dim;
      p.ka[i] = uniform_load(a.kv.k_absmax + block);
      p.va[i] = uniform_load(a.kv.v_absmax + block);
    }
  };
  v4i k[4][DC];
  vbytes v[4][4];
  // a page of 16 or 32 tokens that is not there is read from the first page's
  // start; with one page per step its 64 tokens are there too
  auto load_k = [&](const Place& p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int8_t* from = a.kv.k + p.at[i * kPages / 4] + (kPages == 1 ? i * 16 * dim : 0);
#pragma unroll
      for (int c = 0; c < DC; ++c) k[i][c] = __builtin_nontemporal_load(reinterpret_cast<const v4i*>(from + koff[c]));
    }
  };
  auto load_v = [&](const Place& p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int8_t* from = a.kv.v + p.at[i * kPages / 4] + (kPages == 1 ? i * 16 * dim : 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = __builtin_nontemporal_load(reinterpret_cast<const vbytes*>(from + voff + j * dim));
    }
  };

  int step = s0 + wave;
  int64_t page[kPages];
  Place now, then;
  look_up(step, page);
  if (step < s1) {
    place(step, page, now);
    load_k(now);
    load_v(now);
  }
  look_up(step + kWaves, page);
  v4i qhi[DC], qlo[DC];
  const float row_scale =
      split_query<64, DC>(a.q + (int64_t)(t.begin + token) * a.qt + (int64_t)q_head * a.qh, valid, dim, g, qhi, qlo) *
      a.scale * (1.0f / 127.0f);

  v4f o[4 * DC];
#pragma unroll
  for (int i = 0; i < 4 * DC; ++i) o[i] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  float m = 0.0f, l = 0.0f;
  bool started = false;  // m means something: the row has seen a key

  for (; step < s1; step += kWaves) {
    const int j0 = t.key0(step);
    const bool more = step + kWaves < s1;
    float x[4][4], va[kPages];
    bool all = j0 + kStep <= min(t.first_pos + 1, t.keys) &&
               (a.window == 0 || j0 > t.last_pos - a.window || j0 + kStep <= a.sinks);
#pragma unroll
    for (int i = 0; i < kPages; ++i) {
      all = all && now.there[i];
      va[i] = now.va[i] < kLeastAbsmax ? kLeastAbsmax : now.va[i];
    }
    v4i high[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      high[i] = lo[i] = (v4i){0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        high[i] = mfma_16x16x64(k[i][c], qhi[c], high[i]);
        lo[i] = mfma_16x16x64(k[i][c], qlo[c], lo[i]);
      }
    }
    if (more) {
      place(step + kWaves, page, then);
      load_k(then);
    }
    float top = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float mul = row_scale * now.ka[i * kPages / 4], add = __builtin_amdgcn_logf(va[i * kPages / 4]) + (14.0f - m);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = __builtin_fmaf((float)(high[i][j] * 256 + lo[i][j]), mul, add);
    }
    if (!all) {
      asm volatile("; masked keys");  // stays a branch: most steps need none of this
      const int at = j0 + 4 * g, past = min(pos, t.keys - 1) - at, before = low - at, first = a.sinks - at;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = 16 * i + j;
          const bool seen = key <= past && (key >= before || key < first) && now.there[i * kPages / 4];
          x[i][j] = seen ? x[i][j] : -INFINITY;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, x[i][j]);
    top = rows_max(top);
    if (__any(top > 14.0f + kSlack || (!started && top > kNone))) {
      // lanes whose maximum grew (or that see their first key) take it
      asm volatile("; raised maximum");
      const bool grows = started ? top > 14.0f : top > kNone;
      const float delta = grows ? top - 14.0f : 0.0f;
      const float shrink = started ? __builtin_amdgcn_exp2f(-delta) : 0.0f;
      m += delta;
      started |= grows;
      l *= shrink;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] -= delta;
#pragma unroll
      for (int i = 0; i < 4 * DC; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= shrink;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = __builtin_amdgcn_exp2f(x[i][j]);
        sum += x[i][j];
      }
      // a NaN among the absmax is in the scores of the keys that see it, and only theirs
      l = __builtin_fmaf(sum, __builtin_amdgcn_rcpf(fmaxf(va[i * kPages / 4], kLeastAbsmax)), l);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v8h pf;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pf[j] = (_Float16)x[2 * h][j];
        pf[4 + j] = (_Float16)x[2 * h + 1][j];
      }
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = VBytes<DC>::word(v[2 * h + (j >> 2)][j & 3], c) ^ 0x80808080u;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint4 f = make_uint4(halves_of(w[0], w[1], b), halves_of(w[2], w[3], b), halves_of(w[4], w[5], b),
                                     halves_of(w[6], w[7], b));
          o[4 * c + b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, f), pf, o[4 * c + b], 0, 0, 0);
        }
      }
    }
    if (more) {
      load_v(then);
      now = then;
      look_up(step + 2 * kWaves, page);
    }
  }

  // join the waves: o[i][j] of the lane is element 16 DC g + 4 DC j + i of its row
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  m = started ? m : kNone;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4 * DC; ++i) lds_o[wave][col][16 * DC * g + 4 * DC * j + i] = o[i][j];
  if (g == 0) {
    lds_ml[wave][col][0] = m;
    lds_ml[wave][col][1] = l;
  }
  __syncthreads();
  const int r = tid >> 4, seg = (tid & 15) * 4 * DC;  // thread: 4 DC elements of row r
  if (t.row0 + r >= t.rows) return;
  const int tok = (t.row0 + r) / a.group;
  const int64_t out_row = (int64_t)(t.begin + tok) * a.q_heads + t.head * a.group + (t.row0 + r - tok * a.group);
  float top = kNone, sum = 0.0f, weight[kWaves], x[4 * DC];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lds_ml[w][r][0]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    weight[w] = __builtin_amdgcn_exp2f(lds_ml[w][r][0] - top);
    sum = __builtin_fmaf(weight[w], lds_ml[w][r][1], sum);
  }
#pragma unroll
  for (int i = 0; i < 4 * DC; ++i) {
    x[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x[i] = __builtin_fmaf(weight[w], lds_o[w][r][seg + i], x[i]);
  }
  if (whole) {
    const float mul = sum != 0.0f ? (512.0f / 127.0f) / sum : 0.0f;
    if (seg < dim) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + out_row * dim + seg);
#pragma unroll
      for (int i = 0; i < 2 * DC; ++i) dst[i] = f32x2_to_bf16x2(x[2 * i] * mul, x[2 * i + 1] * mul);
    }
    if (a.lse && (tid & 15) == 0) a.lse[out_row] = sum != 0.0f ? (__log2f(sum) + top - 14.0f) * kLn2 : -INFINITY;
    return;
  }
  const int64_t slot = out_row * a.splits + split;
  if (seg < dim) {
    float4* dst = reinterpret_cast<float4*>(a.part_o + slot * dim + seg);
#pragma unroll
    for (int i = 0; i < DC; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
  if ((tid & 15) == 0) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(top, sum);
}

// ---- many rows ----
// One workgroup: 128 query rows (tokens times the heads of a group) of one
// sequence and cache head, 32 rows per wave, over the steps of one split.  Keys
// and values of a step (64 tokens) go through LDS, in three buffers: wave w
// stages tokens 16w .. 16w + 15 while it computes on the step before, K as it
// is and V already as fp16, so each value is converted once per 128 rows.
// Bound by instruction issue: per 32 keys a wave issues about 145 vector
// instructions, 16 of which (the exponentials) take two turns, against 16 MFMAs
// of 32 cycles, and each MFMA takes two to three turns of issue itself.
// 24000 tokens of 20/5 heads of 128: 920 TFLOP/s (a bf16 library product of 8192
// cubed reaches 1217); 6000 tokens: 221 us, 833 TFLOP/s, where the longest tiles
// (94 steps) set the end.  Figures with steady clocks: the first calls after a
// pause, some 30 ms of them, take up to a quarter longer.
// One team of four waves takes all steps, two workgroups to a CU; or two teams
// take them in turn, each with its own running state and buffers, one workgroup
// to a CU, and are joined in LDS at the end (see make_plan for which).
//   K in LDS: rows of 64 DC bytes, 16-byte chunk c of token m at c ^ key(m), so
//     that 32 tokens' chunks are read without bank conflicts;
//   V in LDS: per 16 tokens and MFMA tile t the 64 lanes' operands side by
//     side; row slot m of tile t is element 2 DC m + t, k-slot 8g + j token
//     8 (j / 4) + 4g + j % 4, which is how S^T = K Q^T leaves P (g = lane / 32).
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kPromptRows = 128;
constexpr int kRing = 3;

template <int DC>
__device__ __forceinline__ int k_key(int m) {
  return DC == 1 ? (m >> 2) & 3 : DC == 2 ? (m >> 1) & 7 : m & 15;
}

template <int DC>
struct VPiece;
template <>
struct VPiece<1> {
  typedef uint16_t type;
  static __device__ type load(__amdgpu_buffer_rsrc_t r, uint32_t lane, int row) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, lane, row, 0);
  }
  static __device__ uint32_t word(type v, int) { return v; }
};
template <>
struct VPiece<2> {
  typedef uint32_t type;
  static __device__ type load(__amdgpu_buffer_rsrc_t r, uint32_t lane, int row) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, lane, row, 0);
  }
  static __device__ uint32_t word(type v, int) { return v; }
};
template <>
struct VPiece<4> {
  typedef uint32_t type __attribute__((ext_vector_type(2)));
  static __device__ type load(__amdgpu_buffer_rsrc_t r, uint32_t lane, int row) {
    return __builtin_bit_cast(type, __builtin_amdgcn_raw_buffer_load_b64(r, lane, row, 0));
  }
  static __device__ uint32_t word(type v, int c) { return v[c]; }
};

template <int DC, int kTeams>
__global__ __launch_bounds__(kThreads * kTeams, DC <= 2 ? 2 : 1) void k_attn_prompt(Attn a) {
  typedef typename VPiece<DC>::type vpiece;
  constexpr int kTiles = 2 * DC;  // 32-element tiles of the head
  struct Ring {
    uint4 v[kRing][4 * kTiles * 64];  // [16 tokens][tile][lane]
    v4i k[kRing][kStep * 4 * DC];     // [token][chunk]
    float4 scale[kRing][4];           // per 16 tokens: ka, log2 va, 1 / va, there
  };
  __shared__ Ring rings[kTeams];
  int index, split;
  if (!tile_and_split(a, index, split)) return;
  Tile t;
  {  // the longest (last) tiles of all heads first: they end about together
    const int lists = a.tiles / a.row_tiles, back = index / lists;
    index = (index - back * lists) * a.row_tiles + (a.row_tiles - 1 - back);
  }
  if (!find_tile(a, index, t)) return;
  const int s0 = split * a.per, s1 = min(t.steps, s0 + a.per);
  if (s0 >= s1) return;
  const bool whole = t.steps <= a.per;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5, col = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane((tid >> 6) & 3), team = __builtin_amdgcn_readfirstlane(tid >> 8);
  const int dim = a.kv.dim, wave_row = t.row0 + 32 * wave, row = wave_row + col;
  const bool busy = wave_row < t.rows, valid = row < t.rows;
  const int token = valid ? row / a.group : 0;
  const int q_head = t.head * a.group + (valid ? row - token * a.group : 0);
  const int pos = t.start + token, low = a.window > 0 ? pos - a.window + 1 : 0;
  const int first_pos = __builtin_amdgcn_readfirstlane(t.start + wave_row / a.group);
  const int last_pos = __builtin_amdgcn_readfirstlane(t.start + (min(wave_row + 32, t.rows) - 1) / a.group);
  v16f o[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.0f;
  float m = 0.0f, l = 0.0f;
  float limit = kNone;  // scores past it raise m; kNone until the row has seen a key

  // staging of this wave's 16 tokens of a step
  Ring& ring = rings[team];
  v4i k_raw[DC];
  vpiece v_raw[8];
  float ka_raw = 0.0f, va_raw = 0.0f;
  bool there = false;
  uint32_t koff[DC];  // lane offsets beside wave-uniform addresses
#pragma unroll
  for (int i = 0; i < DC; ++i) {
    const int unit = lane + 64 * i, tok = unit / (4 * DC), c = unit % (4 * DC);
    koff[i] = (uint32_t)(tok * dim + (16 * c < dim ? 16 * c : 0));
  }
  const uint32_t voff = (uint32_t)(4 * g * dim + (2 * DC * col < dim ? 2 * DC * col : 0));
  // Addresses stay in scalar registers: buffer loads take a base, a lane offset
  // and a row's offset.  Page numbers (a step ahead) and scales are vector loads
  // (none is a zero that the compiler does not know): the barrier below waits for
  // scalar ones, and by their use the rows before them are waited for anyway.
  uint32_t none;
  asm("v_mov_b32 %0, 0" : "=v"(none));
  auto word_at = [&](const auto* p) {
    return *reinterpret_cast<decltype(p)>(reinterpret_cast<const char*>(p) + none);
  };
  const int32_t* pages_of = a.st.page_table + t.seq * a.st.table_stride;
  const uint32_t pages = (uint32_t)min(a.kv.pages, (int64_t)0x7FFFFFFF);
  const int64_t head_bytes = (int64_t)a.kv.page_tokens * dim, page_bytes = head_bytes * a.kv.heads;
  const int8_t *k_head = a.kv.k + t.head * head_bytes, *v_head = a.kv.v + t.head * head_bytes;
  auto page_of = [&](int step) -> int {
    return word_at(pages_of + (min(t.key0(min(step, s1 - 1)) + 16 * wave, t.keys - 1) >> a.page_shift));
  };
  auto load = [&](int step, int raw) {
    const int number = __builtin_amdgcn_readfirstlane(raw);
    const int key = t.key0(step) + 16 * wave;
    there = key < t.keys && (uint32_t)number < pages;
    const int64_t page = there ? number : 0;
    const int64_t at = page * page_bytes + (key & (a.kv.page_tokens - 1)) * dim;
    ka_raw = word_at(a.kv.k_absmax + page * a.kv.heads + t.head);
    va_raw = word_at(a.kv.v_absmax + page * a.kv.heads + t.head);
    constexpr int kRaw = 0x00027000;  // a plain buffer of 32-bit words
    const auto k_rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(k_head + at), 0, 16 * dim, kRaw);
    const auto v_rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(v_head + at), 0, 16 * dim, kRaw);
#pragma unroll
    for (int i = 0; i < DC; ++i) k_raw[i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(k_rows, koff[i], 0, 0));
#pragma unroll
    for (int j = 0; j < 8; ++j) v_raw[j] = VPiece<DC>::load(v_rows, voff, (8 * (j >> 2) + (j & 3)) * dim);
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < DC; ++i) {
      const int unit = lane + 64 * i, tok = 16 * wave + unit / (4 * DC), c = unit % (4 * DC);
      ring.k[buf][tok * 4 * DC + (c ^ k_key<DC>(tok))] = k_raw[i];
    }
    uint32_t w[8][(DC + 1) / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int c = 0; c < (DC + 1) / 2; ++c) w[j][c] = VPiece<DC>::word(v_raw[j], c) ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      ring.v[buf][(wave * kTiles + i) * 64 + lane] =
          make_uint4(halves_of(w[0][i >> 2], w[1][i >> 2], i & 3), halves_of(w[2][i >> 2], w[3][i >> 2], i & 3),
                     halves_of(w[4][i >> 2], w[5][i >> 2], i & 3), halves_of(w[6][i >> 2], w[7][i >> 2], i & 3));
    }
    if (lane == 0) {
      // a NaN among the absmax is in the scores of the keys that see it, and only theirs
      const float va = fmaxf(va_raw, kLeastAbsmax);
      ring.scale[buf][wave] = make_float4(ka_raw, __builtin_fmaf(va_raw, 0.0f, __builtin_amdgcn_logf(va)),
                                          __builtin_amdgcn_rcpf(va), there ? 1.0f : 0.0f);
    }
  };

  // the first step's keys and values travel while the queries are split
  constexpr int kStride = kTeams;
  int step = s0 + team, buf = 0;
  int next_page = page_of(step);
  if (step < s1) {
    load(step, next_page);
    next_page = page_of(step + kStride);
  }
  v4i qhi[kTiles], qlo[kTiles];
  const float row_scale = split_query<32, kTiles>(a.q + (int64_t)(t.begin + token) * a.qt + (int64_t)q_head * a.qh, valid,
                                                  dim, g, qhi, qlo) *
                          a.scale * (1.0f / 127.0f);

  // Half h (32 keys) of the step in buffer buf: its softmax, with the value
  // products of the half before and the key products of the half after it (half
  // nh of buffer nbuf) independent of it and so among its instructions: of two
  // waves alone on a SIMD the one hides the other's products only in part (16
  // products and their softmax in turn 883 cycles, mixed 693).  Wave priorities:
  // staging, which other waves wait for, before the values' products before the
  // rest (6000 tokens, 20/5 heads: 223 us against 245 without; 6 x 509 under a
  // window of 1024 52.7 against 55.8).
  v16i high, lo;   // the next half's scores
  v8h pf[2];       // the half before: its probabilities,
  uint4 vf[2][kTiles];  // and its values
  v4i kf[kTiles];
  uint32_t kslot[kTiles];
#pragma unroll
  for (int c = 0; c < kTiles; ++c) kslot[c] = 16 * (col * 4 * DC + ((2 * c + g) ^ k_key<DC>(col)));
  auto read_k = [&](int buf, int h) {  // the key of token 32 + col is that of col
    const char* from = reinterpret_cast<const char*>(&ring.k[buf][32 * h * 4 * DC]);
#pragma unroll
    for (int c = 0; c < kTiles; ++c) kf[c] = *reinterpret_cast<const v4i*>(from + kslot[c]);
  };
  auto read_v = [&](int buf, int h) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kTiles; ++i) vf[b][i] = ring.v[buf][((2 * h + b) * kTiles + i) * 64 + lane];
  };
  auto key_products = [&]() {
#pragma unroll
    for (int j = 0; j < 16; ++j) high[j] = lo[j] = 0;
#pragma unroll
    for (int c = 0; c < kTiles; ++c) {
      high = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf[c], qhi[c], high, 0, 0, 0);
      lo = __builtin_amdgcn_mfma_i32_32x32x32_i8(kf[c], qlo[c], lo, 0, 0, 0);
    }
  };
  auto value_products = [&]() {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, vf[b][i]), pf[b], o[i], 0, 0, 0);
  };
  auto half = [&](int step, int buf, int h, int nbuf, int nh) {
    const int j0 = t.key0(step);
    const float4 sc[2] = {ring.scale[buf][2 * h], ring.scale[buf][2 * h + 1]};
    // wave-uniform: whether all of its rows see all of the half
    const bool all = j0 + 32 * h + 32 <= min(first_pos + 1, t.keys) &&
                     (a.window == 0 || j0 + 32 * h > last_pos - a.window || j0 + 32 * h + 32 <= a.sinks) &&
                     __builtin_amdgcn_readfirstlane(__float_as_int(sc[0].w) & __float_as_int(sc[1].w)) != 0;
    read_k(nbuf, nh);
    __builtin_amdgcn_s_setprio(1);
    value_products();
    float x[16], top = kNone;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float mul = row_scale * sc[b].x, add = sc[b].y + (14.0f - m);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[8 * b + j] = __builtin_fmaf((float)(high[8 * b + j] * 256 + lo[8 * b + j]), mul, add);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, x[j]);
    if (!all) {
      asm volatile("; masked keys");  // stays a branch: most steps need none of this
      const int at = j0 + 32 * h + 4 * g, past = min(pos, t.keys - 1) - at, before = low - at, first = a.sinks - at;
      top = kNone;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int key = 8 * (j >> 2) + (j & 3);
        const bool seen = key <= past && (key >= before || key < first) && sc[j >> 3].w != 0.0f;
        x[j] = seen ? x[j] : -INFINITY;
        top = fmaxf(top, x[j]);
      }
    }
    top = halves_max(top);
    if (__any(top > limit)) {
      // lanes whose maximum grew (or that see their first key) take it
      asm volatile("; raised maximum");
      const bool grows = top > fminf(limit, 14.0f);
      const float delta = grows ? top - 14.0f : 0.0f;
      const float shrink = limit == kNone ? 0.0f : __builtin_amdgcn_exp2f(-delta);
      m += delta;
      limit = grows ? 14.0f + kSlack : limit;
      l *= shrink;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] -= delta;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= shrink;
    }
    __builtin_amdgcn_s_setprio(0);
    key_products();
    read_v(buf, h);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = __builtin_amdgcn_exp2f(x[8 * b + j]);
        sum += p;
        pf[b][j] = (_Float16)p;
      }
      l = __builtin_fmaf(sum, sc[b].z, l);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // A team's step n + 1 is staged while step n is worked on, behind one barrier
  // between the halves of n: the buffer it takes was last read (values of the
  // second half of n - 2) before the barrier of n - 1.
  const int rounds = (s1 - s0 + kStride - 1) / kStride;
  if (step < s1) store(0);
  if (step + kStride < s1) {
    load(step + kStride, next_page);
    next_page = page_of(step + 2 * kStride);
  }
  __syncthreads();
  if (busy && step < s1) {
    read_k(0, 0);
    key_products();
    read_v(0, 0);  // anything finite: the first half has none before it
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) pf[b][j] = (_Float16)0.0f;
  }
  for (int round = 0; round < rounds; ++round, step += kStride) {
    const bool mine = busy && step < s1;
    const int next = buf == kRing - 1 ? 0 : buf + 1;
    if (mine) half(step, buf, 0, buf, 1);
    __builtin_amdgcn_s_setprio(3);
    if (step + kStride < s1) store(next);
    if (step + 2 * kStride < s1) {
      load(step + 2 * kStride, next_page);
      next_page = page_of(step + 3 * kStride);
    }
    __syncthreads();
    if (mine) half(step, buf, 1, next, 0);
    buf = next;
  }
  if (busy && s0 + team < s1) value_products();
  if (kTeams == 2) __syncthreads();  // before the teams meet in the buffers
  bool started = limit != kNone;

  l += __shfl_xor(l, 32, 64);
  if (kTeams == 2) {
    // the second team's rows meet the first's, lane by lane
    struct Meeting {  // over both teams' buffers, which nobody reads any more
      float4 o[4][4 * kTiles][64];
      float2 ml[4][64];
    };
    static_assert(kTeams == 1 || sizeof(Meeting) <= sizeof(rings), "the teams meet in their buffers");
    Meeting& meeting = *reinterpret_cast<Meeting*>(&rings);
    float4* out = &meeting.o[wave][0][lane];
    float2* out_ml = &meeting.ml[wave][lane];
    if (team == 1) {
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          out[(4 * i + b) * 64] = make_float4(o[i][4 * b], o[i][4 * b + 1], o[i][4 * b + 2], o[i][4 * b + 3]);
      *out_ml = make_float2(started ? m : kNone, l);
    }
    __syncthreads();
    if (team == 1) return;
    const float2 ml = *out_ml;
    const float mine = started ? m : kNone, top = fmaxf(mine, ml.x);
    const float w0 = __builtin_amdgcn_exp2f(mine - top), w1 = __builtin_amdgcn_exp2f(ml.x - top);
    l = l * w0 + ml.y * w1;
    m = top;
    started = top > kNone;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float4 f = out[(4 * i + b) * 64];
        o[i][4 * b] = o[i][4 * b] * w0 + f.x * w1;
        o[i][4 * b + 1] = o[i][4 * b + 1] * w0 + f.y * w1;
        o[i][4 * b + 2] = o[i][4 * b + 2] * w0 + f.z * w1;
        o[i][4 * b + 3] = o[i][4 * b + 3] * w0 + f.w * w1;
      }
  }
  if (!valid) return;
  const int64_t out_row = (int64_t)(t.begin + token) * a.q_heads + q_head;
  const float mul = l != 0.0f ? (512.0f / 127.0f) / l : 0.0f;
  const int64_t slot = out_row * a.splits + split;
  // o[i][4b + j] is element 2 DC (8b + 4g + j) + i: 8 DC adjacent ones per b
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int at = 2 * DC * (8 * b + 4 * g);
    if (at >= dim) break;
    float y[8 * DC];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kTiles; ++i) y[kTiles * j + i] = o[i][4 * b + j];
    if (whole) {
      uint4* dst = reinterpret_cast<uint4*>(a.out + out_row * dim + at);
#pragma unroll
      for (int i = 0; i < DC && at + 8 * i < dim; ++i)  // dim is a multiple of 16
        dst[i] = make_uint4(f32x2_to_bf16x2(y[8 * i] * mul, y[8 * i + 1] * mul),
                            f32x2_to_bf16x2(y[8 * i + 2] * mul, y[8 * i + 3] * mul),
                            f32x2_to_bf16x2(y[8 * i + 4] * mul, y[8 * i + 5] * mul),
                            f32x2_to_bf16x2(y[8 * i + 6] * mul, y[8 * i + 7] * mul));
    } else {
      float4* dst = reinterpret_cast<float4*>(a.part_o + slot * dim + at);
#pragma unroll
      for (int i = 0; i < 2 * DC && at + 4 * i < dim; ++i)
        dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
    }
  }
  if (g == 0) {
    if (!whole)
      *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(started ? m : kNone, l);
    else if (a.lse)
      a.lse[out_row] = l != 0.0f ? (__log2f(l) + m - 14.0f) * kLn2 : -INFINITY;
  }
}

// Joins the splits of a row (rows of one split are already done): kRowWaves
// waves per row, whose lanes take four elements each and, 16 DC lanes apart,
// different splits.  One wave per row for up to eight splits; four for more,
// where a row's partial sums are a serial chain of loads otherwise.
template <int DC, int kRowWaves>
__global__ __launch_bounds__(kThreads) void k_attn_join(Attn a) {
  constexpr int kRows = kWaves / kRowWaves, kLanes = 16 * DC, kGroups = 64 / kLanes;
  __shared__ v4f lds_x[kWaves][kLanes];
  __shared__ float lds_sum[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, dim = a.kv.dim;
  const int pieces = a.tile_rows / kRows, tile = blockIdx.x / pieces;
  const int r = (blockIdx.x - tile * pieces) * kRows + wave / kRowWaves;
  Tile t;
  if (!find_tile(a, tile, t) || t.steps <= a.per) return;
  const int splits = (t.steps + a.per - 1) / a.per, row = t.row0 + r;
  const bool valid = row < t.rows;
  const int tok = valid ? row / a.group : 0;
  const int64_t out_row = (int64_t)(t.begin + tok) * a.q_heads + t.head * a.group + (valid ? row - tok * a.group : 0);
  const float* ml = a.part_ml + out_row * a.splits * 2;
  float top = kNone;
  for (int i = lane; valid && i < splits; i += 64) top = fmaxf(top, ml[2 * i]);
  top = rows_max(top);
  for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const int at = (lane & (kLanes - 1)) * 4;
  float sum = 0.0f;
  v4f x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = (wave % kRowWaves) * kGroups + lane / kLanes; i < splits; i += kRowWaves * kGroups) {
    if (!valid) break;
    const float weight = __builtin_amdgcn_exp2f(ml[2 * i] - top);
    const v4f f = *reinterpret_cast<const v4f*>(a.part_o + (out_row * a.splits + i) * dim + (at < dim ? at : 0));
    sum = __builtin_fmaf(weight, ml[2 * i + 1], sum);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __builtin_fmaf(weight, f[j], x[j]);
  }
#pragma unroll
  for (int d = kLanes; d < 64; d <<= 1) {
    sum += __shfl_xor(sum, d, 64);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] += __shfl_xor(x[j], d, 64);
  }
  if (kRowWaves > 1) {
    if (lane < kLanes) lds_x[wave][lane] = x;
    if (lane == 0) lds_sum[wave] = sum;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      sum += lds_sum[w];
      x += lds_x[w][lane & (kLanes - 1)];
    }
  }
  if (!valid) return;
  const float mul = sum != 0.0f ? (512.0f / 127.0f) / sum : 0.0f;
  if (lane < kLanes && at < dim)
    *reinterpret_cast<uint2*>(a.out + out_row * dim + at) =
        make_uint2(f32x2_to_bf16x2(x[0] * mul, x[1] * mul), f32x2_to_bf16x2(x[2] * mul, x[3] * mul));
  if (a.lse && lane == 0) a.lse[out_row] = sum != 0.0f ? (__log2f(sum) + top - 14.0f) * kLn2 : -INFINITY;
}

// Workgroups along the keys: enough to fill the chip, none with less than a
// step per wave.  The split is a number of steps, the same for every sequence
// of the batch, so a short sequence takes fewer workgroups and not shorter ones.
constexpr int64_t kTargetBlocks = 4096, kTargetPromptBlocks = 512, kUnsplit = 16;

struct Plan {
  int tile_rows;
  int64_t row_tiles, tiles;
  int splits, per;
  int teams;  // of a workgroup of 128 rows
};

// Workgroups of 16 rows (k_attn) or of 128 (k_attn_prompt).  The former read
// and convert the keys and values once per 16 rows, but their four waves share
// a tile's steps, so that few rows, and many over few keys, are done sooner:
// 5 x 2800 rows of 128 over up to 700 keys 20 us against 22, 15 x 400 over 900 16
// against 23; but 28 x 2644 over 721 56 against 31, and 64 tokens of 20 heads over
// 4064 keys 30 against 24.  Between 16000 and 25000 tile steps either may win: 25
// x 1200 rows of 64 over 600 keys (16900) 15 us against 14, 40 x 512 of 128 over
// 600 (23000) 26 against 20.
bool few_rows(int64_t rows, int64_t lists, int64_t steps, int dim) {
  const int64_t tiles = lists * ((rows + 15) / 16), chunks = (dim + 63) / 64;
  return rows < 64 || (steps <= 32 && tiles * steps * chunks < 25000);
}

// Two teams (one workgroup of eight waves to a CU) while the tiles fill the
// 256 CUs less than twice and have many steps: a tile then takes half the
// time (470 tiles of up to 47 steps: 73 us against 91 with one team, 256 of 47: 61
// against 78, 235 of 24: 37 against 49).  One team (two independent workgroups to
// a CU) where there are tiles enough (940 of up to 94: 223 us against 240) or,
// past one per CU, few steps (480 of 20: 53 against 61).
bool two_teams(int dim, int64_t tiles, int64_t steps) {
  return dim <= 128 && ((tiles < 256 && steps > 6) || (tiles < 512 && steps > 24));
}

Plan make_plan(const KvView& kv, int64_t seqs, int64_t max_new, int64_t max_len, int64_t q_heads, int64_t window,
               int64_t sinks) {
  Plan p;
  const int64_t rows = max_new * (q_heads / kv.heads), lists = seqs * kv.heads;
  auto steps_of = [&](int64_t tile_rows) {
    const int64_t all = (max_len + kStep - 1) / kStep;
    if (window <= 0) return all;
    const int64_t tokens = tile_rows * kv.heads / q_heads + 2;  // that a tile spans
    const int64_t most = (window + tokens) / kStep + 2 + (sinks + kStep - 1) / kStep;
    return most < all ? most : all;
  };
  p.tile_rows = few_rows(rows, lists, steps_of(kPromptRows), kv.dim) ? 16 : kPromptRows;
  const int64_t steps = steps_of(p.tile_rows);
  p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  p.tiles = lists * p.row_tiles;
  p.teams = p.tile_rows != 16 && two_teams(kv.dim, p.tiles, steps) ? 2 : 1;
  auto pick = [&](int64_t blocks, int64_t least) {
    const int64_t wanted = p.tiles < blocks ? blocks / p.tiles : 1, most = (steps + least - 1) / least;
    return wanted < most ? wanted : most;
  };
  // Up to this many steps a split gives less than the join and its launch take
  // (steps of 128 elements, one workgroup against splits: 12 steps 9.0 us against
  // 10.2, 16 10.6 against 10.0, 24 14.0 against 10.7; 320 tiles of 16 18.7 against
  // 21.6).  Longer heads' steps take longer, which a few tiles' own time shows
  // (256 elements, 5 tiles of 16 steps 19.9 against 12.9, 80 of 11 16.8 against
  // 15.0; but 320 of 10 27 against 37).
  const int64_t unsplit = p.tile_rows == 16 && kv.dim > 128 && p.tiles < 160 ? kUnsplit / 2 : kUnsplit;
  int64_t splits = 1;
  if (steps <= unsplit) {
    // one workgroup
  } else if (p.tile_rows == 16) {
    const int64_t full = pick(kTargetBlocks, 4 * kWaves), few = pick(1024, kWaves);
    splits = full > few ? full : few;
  } else {
    splits = pick(kTargetPromptBlocks / p.teams, kWaves);
  }
  p.per = (int)((steps + splits - 1) / splits);
  p.splits = (int)((steps + p.per - 1) / p.per);
  return p;
}

// The most splits that any window of these sizes takes: with fewer steps the
// tiles may be of 16 rows instead of 128, and of either there are never more
// splits than these.
int64_t most_splits(const KvView& kv, int64_t seqs, int64_t max_new, int64_t max_len, int64_t q_heads) {
  const int64_t rows = max_new * (q_heads / kv.heads), steps = (max_len + kStep - 1) / kStep;
  auto most = [&](int64_t tile_rows, int64_t target) {
    const int64_t tiles = seqs * kv.heads * ((rows + tile_rows - 1) / tile_rows);
    const int64_t wanted = tiles < target ? target / tiles : 1, limit = (steps + kWaves - 1) / kWaves;
    return wanted < limit ? wanted : limit;
  };
  const int64_t a = most(16, kTargetBlocks), b = rows < 64 ? 1 : most(kPromptRows, kTargetPromptBlocks);
  return a > b ? a : b;
}

}  // namespace

size_t attention_workspace_bytes(const KvView& kv, int64_t seqs, int64_t tokens, int64_t max_new, int64_t max_len,
                                 int64_t q_heads) {
  const int64_t splits = most_splits(kv, seqs, max_new, max_len, q_heads);
  return splits <= 1 ? 0 : (size_t)tokens * (size_t)q_heads * (size_t)splits * (size_t)(kv.dim + 2) * 4;
}

hipError_t launch_attention(const KvView& kv, const KvStep& st, int64_t seqs, int64_t tokens, int64_t max_new,
                            int64_t max_len, const uint16_t* q, int64_t qt, int64_t qh, int q_heads, float scale,
                            int64_t window, int64_t sinks, uint16_t* out, float* lse, void* workspace, hipStream_t s) {
  const Plan p = make_plan(kv, seqs, max_new, max_len, q_heads, window, sinks);
  const int64_t blocks = (p.tiles + 7) / 8 * 8 * p.splits;
  if (!grid_fits(blocks, 2 * kThreads) || (p.splits > 1 && !grid_fits(p.tiles * p.tile_rows, kThreads))) return kErrGridTooLarge;
  Attn a;
  a.kv = kv;
  a.st = st;
  a.q = q;
  a.qt = qt;
  a.qh = qh;
  a.q_heads = q_heads;
  a.group = q_heads / kv.heads;
  a.page_shift = __builtin_ctz((unsigned)kv.page_tokens);
  a.max_len = (int)max_len;
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.scale = scale * kLog2e;
  a.tile_rows = p.tile_rows;
  a.row_tiles = (int)p.row_tiles;
  a.tiles = (int)p.tiles;
  a.splits = p.splits;
  a.per = p.per;
  a.out = out;
  a.lse = lse;
  a.part_o = (float*)workspace;
  a.part_ml = a.part_o + tokens * q_heads * p.splits * kv.dim;
  auto go = [&](auto dc) {
    constexpr int DC = decltype(dc)::value;
    auto prompt = [&](int teams) {
      if constexpr (DC <= 2) {
        if (teams == 2) {
          hipLaunchKernelGGL((k_attn_prompt<DC, 2>), dim3((unsigned)blocks), dim3(2 * kThreads), 0, s, a);
          return;
        }
      }
      hipLaunchKernelGGL((k_attn_prompt<DC, 1>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    };
    const dim3 grid((unsigned)blocks);
    if (p.tile_rows == 16) {
      if (kv.page_tokens >= kStep)
        hipLaunchKernelGGL((k_attn<DC, 1>), grid, dim3(kThreads), 0, s, a);
      else
        hipLaunchKernelGGL((k_attn<DC, 4>), grid, dim3(kThreads), 0, s, a);
    } else {
      prompt(p.teams);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits <= 1) return e;
    if (p.splits <= 8)
      hipLaunchKernelGGL((k_attn_join<DC, 1>), dim3((unsigned)(p.tiles * (p.tile_rows / kWaves))), dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_attn_join<DC, kWaves>), dim3((unsigned)(p.tiles * p.tile_rows)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  };
  if (kv.dim <= 64) return go(std::integral_constant<int, 1>{});
  if (kv.dim <= 128) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 4>{});
}

}  // namespace bl
