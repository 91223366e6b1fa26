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
// summed in fp32 from the unrounded P.
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
constexpr float kNone = -1e30f;  // a running maximum that nothing has raised
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Attn {
  KvView kv;
  KvStep st;
  const uint16_t* q;
  int64_t qt, qh;
  int q_heads, group, page_shift;
  int window, sinks;
  float scale;       // of q . k, in base 2
  int row_tiles;     // 16-row tiles per sequence and head
  int splits, per;   // workgroups along the keys, steps of each
  uint16_t* out;
  float* lse;
  float* part_o;   // [token][q_head][split][dim]
  float* part_ml;  // [token][q_head][split][2]
};

// The rows and steps of one 16-row tile.
struct Tile {
  int seq, head, begin, rows, row0, start;
  int first_pos, last_pos;  // positions of its first and last row
  int keys;                 // keys 0 .. keys-1 may be visible
  int sink_steps, base, steps;
  __device__ int key0(int step) const { return (step < sink_steps ? step : base + step - sink_steps) * kStep; }
};

__device__ __forceinline__ bool find_tile(const Attn& a, int index, Tile& t) {
  const int rest = index / a.row_tiles;
  const int rt = index - rest * a.row_tiles;
  t.seq = rest / a.kv.heads;
  t.head = rest - t.seq * a.kv.heads;
  t.begin = a.st.begin(t.seq);
  const int count = a.st.count(t.seq, t.begin);
  t.rows = count * a.group;
  t.row0 = rt * 16;
  if (t.row0 >= t.rows) return false;
  t.start = a.st.start_of(t.seq);
  t.first_pos = t.start + t.row0 / a.group;
  t.last_pos = t.start + (min(t.row0 + 16, t.rows) - 1) / a.group;
  const int64_t room = a.st.table_stride << a.page_shift;
  t.keys = (int)min((int64_t)t.last_pos + 1, room);
  const int last = (t.keys + kStep - 1) / kStep;
  t.base = a.window > 0 ? min(max(0, t.first_pos - a.window + 1) / kStep, last) : 0;
  t.sink_steps = min((a.sinks + kStep - 1) / kStep, t.base);
  t.steps = t.sink_steps + last - t.base;
  return true;
}

// reductions over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float groups_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float groups_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// A query row of 64 * DC elements (zeros past dim) as high and low bytes; the
// lane holds elements 64c + 16g .. +15 of row lane % 16.  Returns absmax / 32512.
template <int DC>
__device__ __forceinline__ float split_query(const uint16_t* row, bool valid, int dim, int g, v4i (&hi)[DC], v4i (&lo)[DC]) {
  float x[DC][16], top = 0.0f;
#pragma unroll
  for (int c = 0; c < DC; ++c) {
    uint4 d[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (valid && 64 * c + 16 * g < dim) {
      const uint4* p = reinterpret_cast<const uint4*>(row + 64 * c + 16 * g);
      d[0] = p[0];
      d[1] = p[1];
    }
    const uint32_t w[8] = {d[0].x, d[0].y, d[0].z, d[0].w, d[1].x, d[1].y, d[1].z, d[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[c][2 * i] = __uint_as_float(w[i] << 16);
      x[c][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      top = fmaxf(top, fmaxf(fabsf(x[c][2 * i]), fabsf(x[c][2 * i + 1])));
    }
  }
  top = groups_max(top);
  const float s = top > 0x1p-100f ? 32512.0f / top : 0.0f;
#pragma unroll
  for (int c = 0; c < DC; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h = 0, l = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int code = (int)rintf(x[c][4 * i + j] * s);  // |code| <= 32512
        h |= ((uint32_t)((code + 128) >> 8) & 255u) << (8 * j);
        l |= ((uint32_t)code & 255u) << (8 * j);
      }
      hi[c][i] = (int)h;
      lo[c][i] = (int)l;
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

template <int DC>
struct VBytes;
template <>
struct VBytes<1> { typedef uint32_t type; };
template <>
struct VBytes<2> { typedef uint2 type; };
template <>
struct VBytes<4> { typedef uint4 type; };

// One workgroup: 16 query rows of one sequence and cache head, the steps of
// one split; wave w takes steps w, w + 4, ... with its own running state, and
// the waves' states are joined in LDS at the end.
template <int DC>
__global__ __launch_bounds__(kThreads) void k_attn(Attn a) {
  typedef typename VBytes<DC>::type vbytes;
  __shared__ float lds_o[kWaves][16][64 * DC];
  __shared__ float lds_ml[kWaves][16][2];
  const int split = blockIdx.x % a.splits;
  Tile t;
  if (!find_tile(a, blockIdx.x / a.splits, t)) return;
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
  v4i qhi[DC], qlo[DC];
  const float row_scale =
      split_query<DC>(a.q + (int64_t)(t.begin + token) * a.qt + (int64_t)q_head * a.qh, valid, dim, g, qhi, qlo) *
      a.scale * (1.0f / 127.0f);

  // byte offsets inside a 16-token tile; elements past dim read element 0
  // instead (their query bytes are zero, their outputs are not stored)
  uint32_t koff[DC], voff;
#pragma unroll
  for (int c = 0; c < DC; ++c) koff[c] = (uint32_t)(col * dim + (64 * c + 16 * g < dim ? 64 * c + 16 * g : 0));
  voff = (uint32_t)(4 * g * dim + (4 * DC * col < dim ? 4 * DC * col : 0));

  v4f o[4 * DC];
#pragma unroll
  for (int i = 0; i < 4 * DC; ++i) o[i] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNone, l = 0.0f;

  for (int step = s0 + wave; step < s1; step += kWaves) {
    const int j0 = t.key0(step);
    const int8_t *kp[4], *vp[4];
    float ka[4], va[4];
    bool dead[4], any_dead = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = j0 + 16 * i;
      int64_t page = -1;
      if (key < t.keys) page = a.st.page(t.seq, key >> a.page_shift);
      dead[i] = page < 0 || page >= a.kv.pages;
      any_dead |= dead[i];
      const int64_t block = dead[i] ? 0 : page * a.kv.heads + t.head;
      const int64_t at = (block * a.kv.page_tokens + (dead[i] ? 0 : key & (a.kv.page_tokens - 1))) * dim;
      kp[i] = a.kv.k + at;
      vp[i] = a.kv.v + at;
      ka[i] = dead[i] ? 0.0f : a.kv.k_absmax[block];
      const float top = dead[i] ? 0.0f : a.kv.v_absmax[block];
      va[i] = top > 0.0f ? top : 1.0f;
    }
    v4i k[4][DC];
    vbytes v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < DC; ++c) k[i][c] = *reinterpret_cast<const v4i*>(kp[i] + koff[c]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = *reinterpret_cast<const vbytes*>(vp[i] + voff + j * dim);

    float p[4][4], top = kNone;
    const bool all = !any_dead && j0 + kStep <= t.first_pos + 1 && j0 + kStep <= t.keys &&
                     (a.window == 0 || j0 > t.last_pos - a.window || j0 + kStep <= a.sinks);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v4i high = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        high = mfma_16x16x64(k[i][c], qhi[c], high);
        lo = mfma_16x16x64(k[i][c], qlo[c], lo);
      }
      const float mul = row_scale * ka[i], add = __builtin_amdgcn_logf(va[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j] = __builtin_fmaf((float)(high[j] * 256 + lo[j]), mul, add);
      if (!all) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = j0 + 16 * i + 4 * g + j;
          const bool seen = !dead[i] && key <= pos && key < t.keys && (key >= low || key < a.sinks);
          p[i][j] = seen ? p[i][j] : -INFINITY;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, p[i][j]);
    }
    const float m_new = fmaxf(m, groups_max(top));
    const float shrink = __builtin_amdgcn_exp2f(m - m_new);
    m = m_new;
    l *= shrink;
#pragma unroll
    for (int i = 0; i < 4 * DC; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] *= shrink;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = __builtin_amdgcn_exp2f(p[i][j] - m + 14.0f);
        sum += p[i][j];
      }
      l = __builtin_fmaf(sum, __builtin_amdgcn_rcpf(va[i]), l);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v8h pf;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        pf[j] = (_Float16)p[2 * h][j];
        pf[4 + j] = (_Float16)p[2 * h + 1][j];
      }
      uint32_t w[8][DC];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const vbytes raw = v[2 * h + (j >> 2)][j & 3];
        __builtin_memcpy(w[j], &raw, sizeof(raw));
#pragma unroll
        for (int c = 0; c < DC; ++c) w[j][c] ^= 0x80808080u;
      }
#pragma unroll
      for (int i = 0; i < 4 * DC; ++i) {
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = halves_of(w[2 * j][i >> 2], w[2 * j + 1][i >> 2], i & 3);
        v8h vf;
        __builtin_memcpy(&vf, f, 16);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf, o[i], 0, 0, 0);
      }
    }
  }

  // join the waves: o[i][j] of the lane is element 16 DC g + 4 DC j + i of its row
  l = groups_sum(l);
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
    const float mul = sum > 0.0f ? (512.0f / 127.0f) / sum : 0.0f;
    if (seg < dim) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + out_row * dim + seg);
#pragma unroll
      for (int i = 0; i < 2 * DC; ++i) dst[i] = f32x2_to_bf16x2(x[2 * i] * mul, x[2 * i + 1] * mul);
    }
    if (a.lse && (tid & 15) == 0) a.lse[out_row] = sum > 0.0f ? (__log2f(sum) + top - 14.0f) * kLn2 : -INFINITY;
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

// Joins the splits of a 16-row tile (tiles of one split are already done).
template <int DC>
__global__ __launch_bounds__(kThreads) void k_attn_join(Attn a) {
  Tile t;
  if (!find_tile(a, blockIdx.x, t) || t.steps <= a.per) return;
  const int splits = (t.steps + a.per - 1) / a.per;
  const int tid = threadIdx.x, r = tid >> 4, seg = (tid & 15) * 4 * DC, dim = a.kv.dim;
  if (t.row0 + r >= t.rows) return;
  const int tok = (t.row0 + r) / a.group;
  const int64_t out_row = (int64_t)(t.begin + tok) * a.q_heads + t.head * a.group + (t.row0 + r - tok * a.group);
  const float* ml = a.part_ml + out_row * a.splits * 2;
  float top = kNone;
  for (int i = 0; i < splits; ++i) top = fmaxf(top, ml[2 * i]);
  float sum = 0.0f, x[4 * DC];
#pragma unroll
  for (int i = 0; i < 4 * DC; ++i) x[i] = 0.0f;
  for (int i = 0; i < splits; ++i) {
    const float weight = __builtin_amdgcn_exp2f(ml[2 * i] - top);
    sum = __builtin_fmaf(weight, ml[2 * i + 1], sum);
    if (seg < dim) {
      const float4* src = reinterpret_cast<const float4*>(a.part_o + (out_row * a.splits + i) * dim + seg);
#pragma unroll
      for (int j = 0; j < DC; ++j) {
        const float4 f = src[j];
        x[4 * j] = __builtin_fmaf(weight, f.x, x[4 * j]);
        x[4 * j + 1] = __builtin_fmaf(weight, f.y, x[4 * j + 1]);
        x[4 * j + 2] = __builtin_fmaf(weight, f.z, x[4 * j + 2]);
        x[4 * j + 3] = __builtin_fmaf(weight, f.w, x[4 * j + 3]);
      }
    }
  }
  const float mul = sum > 0.0f ? (512.0f / 127.0f) / sum : 0.0f;
  if (seg < dim) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + out_row * dim + seg);
#pragma unroll
    for (int i = 0; i < 2 * DC; ++i) dst[i] = f32x2_to_bf16x2(x[2 * i] * mul, x[2 * i + 1] * mul);
  }
  if (a.lse && (tid & 15) == 0) a.lse[out_row] = sum > 0.0f ? (__log2f(sum) + top - 14.0f) * kLn2 : -INFINITY;
}

// Workgroups along the keys: enough to fill the chip, none with less than a
// step per wave.  The split is a number of steps, the same for every sequence
// of the batch, so a short sequence takes fewer workgroups and not shorter ones.
constexpr int64_t kTargetBlocks = 2048;

struct Plan {
  int64_t row_tiles, tiles;
  int splits, per;
};

Plan make_plan(const KvView& kv, int64_t seqs, int64_t max_new, int64_t max_len, int64_t q_heads, int64_t window,
               int64_t sinks) {
  Plan p;
  p.row_tiles = (max_new * (q_heads / kv.heads) + 15) / 16;
  p.tiles = seqs * kv.heads * p.row_tiles;
  int64_t steps = (max_len + kStep - 1) / kStep;
  if (window > 0) {
    const int64_t most = (window + 16 + kStep) / kStep + 1 + (sinks + kStep - 1) / kStep;
    if (most < steps) steps = most;
  }
  int64_t splits = (kTargetBlocks + p.tiles - 1) / p.tiles;
  const int64_t most = (steps + kWaves - 1) / kWaves;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  p.per = (int)((steps + splits - 1) / splits);
  p.splits = (int)((steps + p.per - 1) / p.per);
  return p;
}

}  // namespace

size_t attention_workspace_bytes(const KvView& kv, int64_t seqs, int64_t tokens, int64_t max_new, int64_t max_len,
                                 int64_t q_heads) {
  // without a window there are the most splits
  const Plan p = make_plan(kv, seqs, max_new, max_len, q_heads, 0, 0);
  return p.splits <= 1 ? 0 : (size_t)tokens * (size_t)q_heads * (size_t)p.splits * (size_t)(kv.dim + 2) * 4;
}

hipError_t launch_attention(const KvView& kv, const KvStep& st, int64_t seqs, int64_t tokens, int64_t max_new,
                            int64_t max_len, const uint16_t* q, int64_t qt, int64_t qh, int q_heads, float scale,
                            int64_t window, int64_t sinks, uint16_t* out, float* lse, void* workspace, hipStream_t s) {
  const Plan p = make_plan(kv, seqs, max_new, max_len, q_heads, window, sinks);
  if (!grid_fits(p.tiles * p.splits, kThreads)) return kErrGridTooLarge;
  Attn a;
  a.kv = kv;
  a.st = st;
  a.q = q;
  a.qt = qt;
  a.qh = qh;
  a.q_heads = q_heads;
  a.group = q_heads / kv.heads;
  a.page_shift = __builtin_ctz((unsigned)kv.page_tokens);
  a.window = (int)window;
  a.sinks = (int)sinks;
  a.scale = scale * kLog2e;
  a.row_tiles = (int)p.row_tiles;
  a.splits = p.splits;
  a.per = p.per;
  a.out = out;
  a.lse = lse;
  a.part_o = (float*)workspace;
  a.part_ml = a.part_o + tokens * q_heads * p.splits * kv.dim;
  auto go = [&](auto dc) {
    constexpr int DC = decltype(dc)::value;
    hipLaunchKernelGGL(k_attn<DC>, dim3((unsigned)(p.tiles * p.splits)), dim3(kThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits <= 1) return e;
    hipLaunchKernelGGL(k_attn_join<DC>, dim3((unsigned)p.tiles), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  };
  if (kv.dim <= 64) return go(std::integral_constant<int, 1>{});
  if (kv.dim <= 128) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 4>{});
}

}  // namespace bl
