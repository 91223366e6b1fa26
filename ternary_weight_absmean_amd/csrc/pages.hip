// Pages of the 8-bit key/value cache: handing out (bl_kv_grow), forking
// sequences (bl_kv_fork), giving back (bl_kv_free), moving used pages to the
// front (bl_kv_compact), and the copies that go with them (bl_kv_copy).
//
// refs[p] counts the entries of page tables that hold page p.  Requests are
// taken in order and get the lowest free pages, so equal inputs give equal
// tables whatever the order in which workgroups run: ranks come from prefix
// sums, atomics only add to counts that nobody reads meanwhile.
#include "device_util.h"
#include "internal.h"

namespace bl {
namespace {

constexpr int kThreads = 1024;
constexpr int kPagesPerThread = 8;
constexpr int kScan = kThreads * kPagesPerThread;  // pages looked at together
constexpr int kQueue = 2 * kScan;                  // free pages found and not yet given
constexpr int kSkip = 4;                           // times kScan pages: looked through for any free one

// Sum of v over the threads before this one, and over all, in a workgroup of
// kThreads; part holds one number per wave.
__device__ __forceinline__ int block_prefix(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(sum, d, 64);
    if (lane >= d) sum += other;
  }
  if (lane == 63) part[wave] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    const int n = part[w];
    before += w < wave ? n : 0;
    all += n;
  }
  __syncthreads();  // part may be written again
  total = all;
  return before + sum - v;
}

// The requests i < items for which need(i) is true, in order, get the lowest
// free pages: give(i, page), page -1 where none is left.  Returns how many got
// none (in every thread).  One workgroup; refs is read from the front only as far as
// the requests need.  What give writes lies behind what has been read.
template <typename Need, typename Give>
__device__ __forceinline__ int hand_out(const int32_t* refs, int pages, int64_t items, int* queue, int* part, Need need,
                                        Give give) {
  const int tid = threadIdx.x;
  int head = 0, held = 0, at = 0, lacking = 0;  // the same in every thread
  int ahead[kPagesPerThread];                   // counts of the pages looked at next
  auto look = [&]() {
#pragma unroll
    for (int j = 0; j < kPagesPerThread; ++j) ahead[j] = refs[min(at + tid * kPagesPerThread + j, pages - 1)];
  };
  // On to the next kScan pages with a free one among them: pages in use stand
  // in front (the lowest are handed out first), and most calls pass over them.
  // 64 pages behind 120000 used ones: 18 us, 51 through the queue alone.
  auto skip = [&]() {
    while (at + kScan <= pages) {
      int4 r[kSkip][2];
#pragma unroll
      for (int c = 0; c < kSkip; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          r[c][j] = *reinterpret_cast<const int4*>(refs + min(at + c * kScan + tid * kPagesPerThread + 4 * j, (pages - 4) & ~3));
      int any = (1 << min((pages - at) / kScan, kSkip)) & ((1 << kSkip) - 1);  // the end is looked at in any case
#pragma unroll
      for (int c = 0; c < kSkip; ++c) {
        bool zero = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) zero |= r[c][j].x == 0 || r[c][j].y == 0 || r[c][j].z == 0 || r[c][j].w == 0;
        any |= (__ballot(zero) != 0) << c;
      }
      if ((tid & 63) == 0) part[tid >> 6] = any;
      __syncthreads();
      any = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) any |= part[w];
      __syncthreads();
      if (any) {
        at += (__ffs(any) - 1) * kScan;
        return;
      }
      at += kSkip * kScan;
    }
  };
  look();
  for (int64_t base = 0; base < items; base += kThreads) {
    const int64_t i = base + tid;
    const bool mine = i < items && need(i);
    int wanted;
    const int rank = block_prefix(mine, part, wanted);
    while (held < wanted && at < pages) {
      int free_bits = 0;
      const int first = at + tid * kPagesPerThread;
#pragma unroll
      for (int j = 0; j < kPagesPerThread; ++j) free_bits |= (ahead[j] == 0 && first + j < pages) << j;
      at += kScan;
      look();
      int found;
      int to = head + held + block_prefix(__popc(free_bits), part, found);
      while (free_bits) {
        const int j = __ffs(free_bits) - 1;
        free_bits &= free_bits - 1;
        queue[to++ & (kQueue - 1)] = first + j;
      }
      held += found;
      if (found == 0) {
        skip();
        look();
      }
      __syncthreads();
    }
    if (mine) give(i, rank < held ? queue[(head + rank) & (kQueue - 1)] : -1);
    const int given = min(wanted, held);
    lacking += wanted - given;
    head = (head + given) & (kQueue - 1);
    held -= given;
    __syncthreads();  // the queue may be written again
  }
  return lacking;
}

// Takes a page's count down by one, unless it is at 0.
__device__ __forceinline__ void release(int32_t* refs, int pages, int page) {
  if ((uint32_t)page < (uint32_t)pages && atomicAdd(refs + page, -1) <= 0) atomicAdd(refs + page, 1);
}

// ---- bl_kv_grow ----
// Item i is page i % touched of those that sequence i / touched may enter.  A
// page that the new tokens share with earlier ones and that others hold too is
// left for a copy; the sources lose their holders at the end, so that counts
// above 0 stay as they are while requests are looked at.
//
// Who leaves: all that would write in a shared page, but for the last of them if
// nobody else holds it.  Their pages go into a table in LDS, which takes the
// last writer of each by a maximum and then their number by a sum: a step per
// sequence at worst, all in one page (192 of them: 11 us, 3.7 where none shares
// one; 8192: 167, their atomics meeting in one word, and 23).
struct Grow {
  int32_t* refs;
  int pages, page_tokens;
  KvStep st;
  int64_t seqs;
  int touched;
  int32_t *table, *copies, *shortage;
  // first page that sequence s enters and the positions of its new tokens; false: none
  __device__ bool span(int s, int64_t& first, int64_t& start, int64_t& end) const {
    const int begin = st.begin(s), count = st.count(s, begin);
    start = st.start_of(s);
    end = start + count;
    first = start / page_tokens;
    return count > 0;
  }
  // the page that sequence s would go on writing in, -1 if it begins a new one
  __device__ int part_filled(int s) const {
    int64_t first, start, end;
    if (!span(s, first, start, end) || start % page_tokens == 0 || first >= st.table_stride) return -1;
    const int32_t e = table[s * st.table_stride + first];
    return (uint32_t)e < (uint32_t)pages ? e : -1;
  }
};

constexpr int kSlots = kMaxForkSeqs;  // of the table: never full of other pages than its own
static_assert(2 * kSlots <= kQueue && (kSlots & (kSlots - 1)) == 0 && kMaxForkSeqs <= 1 << 15, "");

// Sets the bits of the sequences that leave their page; false: none does.  words
// holds 2 kSlots of them and is free again afterwards.
__device__ __forceinline__ bool find_leavers(const Grow& g, int* words, uint64_t* leaves) {
  constexpr int kRounds = kMaxForkSeqs / kThreads;
  const int tid = threadIdx.x;
  int *key = words, *word = words + kSlots;
  int page[kRounds];
  bool any = false;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int s = r * kThreads + tid;
    page[r] = s < g.seqs ? g.part_filled(s) : -1;
    if (page[r] >= 0 && g.refs[page[r]] <= 1) page[r] = -1;
    any |= page[r] >= 0;
  }
  if (!__syncthreads_or(any)) return false;
  for (int i = tid; i < kSlots; i += kThreads) {
    key[i] = -1;
    word[i] = 0;
  }
  __syncthreads();
  int slot[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    slot[r] = 0;
    if (page[r] < 0) continue;
    int at = (uint32_t)page[r] * 2654435761u >> 16 & (kSlots - 1);
    for (;;) {  // as many slots as sequences: one is free or the page's own
      const int held = atomicCAS(key + at, -1, page[r]);
      if (held == -1 || held == page[r]) break;
      at = (at + 1) & (kSlots - 1);
    }
    slot[r] = at;
    atomicMax(word + at, r * kThreads + tid);
  }
  __syncthreads();
  for (int i = tid; i < kSlots; i += kThreads) word[i] <<= 16;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (page[r] >= 0) atomicAdd(word + slot[r], 1);
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int s = r * kThreads + tid, w = word[slot[r]];
    const bool leave = page[r] >= 0 && (w >> 16 != s || g.refs[page[r]] > (w & 0xFFFF));
    const uint64_t bits = __ballot(leave);
    if ((tid & 63) == 0) leaves[s >> 6] = bits;
  }
  __syncthreads();
  return true;
}

__global__ __launch_bounds__(kThreads) void k_kv_grow(Grow g) {
  __shared__ int queue[kQueue];
  __shared__ int part[kThreads / 64];
  __shared__ uint64_t leaves[kMaxForkSeqs / 64];
  const bool leaving = g.copies && find_leavers(g, queue, leaves);  // never without copies
  auto need = [&](int64_t i) {
    const int s = (int)(i / g.touched);
    const int64_t at = i - (int64_t)s * g.touched;
    int64_t first, start, end;
    const bool some = g.span(s, first, start, end);
    if (g.copies && at == 0) {
      g.copies[3 * s] = g.copies[3 * s + 1] = -1;
      g.copies[3 * s + 2] = 0;
    }
    const int64_t index = first + at;
    if (!some || index * g.page_tokens >= end || index >= g.st.table_stride) return false;
    const int32_t e = g.table[s * g.st.table_stride + index];
    if ((uint32_t)e >= (uint32_t)g.pages) return true;
    return leaving && at == 0 && (leaves[s >> 6] >> (s & 63) & 1);
  };
  auto give = [&](int64_t i, int page) {
    const int s = (int)(i / g.touched);
    int64_t first, start, end;
    g.span(s, first, start, end);
    int32_t* entry = g.table + s * g.st.table_stride + first + (i - (int64_t)s * g.touched);
    if ((uint32_t)*entry < (uint32_t)g.pages) {
      g.copies[3 * s] = *entry;  // without a target where no page is left
      g.copies[3 * s + 1] = page;
      g.copies[3 * s + 2] = page < 0 ? 0 : (int)(start % g.page_tokens);
    } else if (page >= 0) {
      *entry = page;
    }
    if (page >= 0) g.refs[page] = 1;
  };
  int lacking = hand_out(g.refs, g.pages, g.seqs * g.touched, queue, part, need, give);
  if (leaving) {
    for (int s = threadIdx.x; s < g.seqs; s += kThreads) {
      const int from = g.copies[3 * s], to = g.copies[3 * s + 1];
      if (to < 0) continue;
      int64_t first, start, end;
      g.span(s, first, start, end);
      g.table[s * g.st.table_stride + first] = to;
      release(g.refs, g.pages, from);
    }
    if (lacking > 0) {
      // A last writer that was to keep its page shares it still, if one before it
      // did not get its copy.
      __syncthreads();
      int kept = 0;
      for (int base = 0; base < g.seqs; base += kThreads) {
        const int s = base + (int)threadIdx.x;
        const int e = s < g.seqs && g.copies[3 * s] < 0 ? g.part_filled(s) : -1;
        const bool shares = e >= 0 && __hip_atomic_load(g.refs + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 1;
        if (shares) g.copies[3 * s] = e;
        kept += __syncthreads_count(shares);
      }
      lacking += kept;
    }
  }
  if (threadIdx.x == 0 && g.shortage && lacking > 0) *g.shortage += lacking;
}

// ---- bl_kv_fork ----
constexpr int64_t kReleaseHere = 32768;

struct Fork {
  int32_t* refs;
  int pages, page_tokens;
  const int32_t *table, *length, *parent;
  int64_t stride;
  int seqs, children, keep_parents;
  bool release_here;  // workgroup 0 also gives back what no child holds
  int32_t *table_out, *length_out, *copies, *shortage;
  __device__ bool parent_of(int c, int& p) const {
    p = parent[c];
    return (uint32_t)p < (uint32_t)seqs;
  }
  __device__ int64_t held(int p) const {
    const int64_t n = length[p] < 0 ? 0 : length[p], most = stride * page_tokens;
    return n < most ? n : most;
  }
};

// Workgroup 0 hands out the pages that part-filled ones are copied to, the
// others write one child's row each.  Counts that the latter raise are above 0
// already, so what workgroup 0 sees as free does not depend on them.
__global__ __launch_bounds__(kThreads) void k_kv_fork(Fork f) {
  __shared__ int queue[kQueue];
  __shared__ int part[kThreads / 64];
  __shared__ int first[kMaxForkSeqs];
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const int c = (int)blockIdx.x - 1;
    int p;
    const bool real = f.parent_of(c, p);
    bool elder = f.keep_parents;  // whether another holds the parent's pages: its counts go up
    if (!elder && real)
      for (int i = tid; i < c; i += kThreads) elder |= f.parent[i] == p;
    elder = __syncthreads_or(elder);
    const int64_t length = real ? f.held(p) : 0, full = length / f.page_tokens;
    const bool rest = length % f.page_tokens != 0;
    for (int64_t i = tid; i < f.stride; i += kThreads) {
      if (rest && i == full) continue;  // workgroup 0's
      const int32_t e = i < full ? f.table[p * f.stride + i] : -1;
      f.table_out[c * f.stride + i] = e;
      if (elder && (uint32_t)e < (uint32_t)f.pages) atomicAdd(f.refs + e, 1);
    }
    return;
  }
  if (!f.keep_parents) {
    for (int p = tid; p < f.seqs; p += kThreads) first[p] = f.children;
    __syncthreads();
    for (int c = tid; c < f.children; c += kThreads) {
      int p;
      if (f.parent_of(c, p)) atomicMin(&first[p], c);
    }
    __syncthreads();
  }
  // the part-filled page of child c's parent: its entry and tokens (0: there is none)
  auto last = [&](int c, int& tokens, int64_t& index) -> int32_t {
    int p;
    tokens = 0;
    index = 0;
    if (!f.parent_of(c, p)) return -1;
    const int64_t length = f.held(p);
    tokens = (int)(length % f.page_tokens);
    index = length / f.page_tokens;
    return tokens ? f.table[p * f.stride + index] : -1;
  };
  auto stays = [&](int c) { return !f.keep_parents && first[f.parent[c]] == c; };
  auto need = [&](int64_t i) {
    const int c = (int)i;
    int tokens, p;
    int64_t index;
    const int32_t e = last(c, tokens, index);
    f.length_out[c] = f.parent_of(c, p) ? (int32_t)f.held(p) : 0;
    f.copies[3 * c] = f.copies[3 * c + 1] = -1;
    f.copies[3 * c + 2] = 0;
    if (!tokens) return false;
    const bool there = (uint32_t)e < (uint32_t)f.pages, own = there && stays(c);
    f.table_out[c * f.stride + index] = own ? e : -1;
    return there && !own;
  };
  auto give = [&](int64_t i, int page) {
    const int c = (int)i;
    int tokens;
    int64_t index;
    const int32_t e = last(c, tokens, index);
    if (page < 0) return;
    f.refs[page] = 1;
    f.table_out[c * f.stride + index] = page;
    f.copies[3 * c] = e;
    f.copies[3 * c + 1] = page;
    f.copies[3 * c + 2] = tokens;
  };
  const int lacking = hand_out(f.refs, f.pages, f.children, queue, part, need, give);
  if (tid == 0 && f.shortage && lacking > 0) *f.shortage += lacking;
  if (!f.release_here) return;
  for (int i = tid; i < f.seqs * (int)f.stride; i += kThreads) {
    const int p = i / (int)f.stride, at = i - p * (int)f.stride;
    const int64_t from = first[p] < f.children ? (f.held(p) + f.page_tokens - 1) / f.page_tokens : 0;
    if (at >= from) release(f.refs, f.pages, f.table[i]);
  }
}

// The pages of consumed parents that no child took over: all of a parent without
// children, those past the length of the others.  Each is one of the parent's own
// holds, so no count falls to 0 while another row's workgroup raises it.  In a
// launch of its own where the rows are long (kReleaseHere entries and more).
__global__ __launch_bounds__(256) void k_kv_fork_release(Fork f) {
  const int p = (int)blockIdx.x, tid = threadIdx.x;
  bool has = false;
  for (int c = tid; c < f.children; c += 256) has |= f.parent[c] == p;
  has = __syncthreads_or(has);
  const int64_t from = has ? (f.held(p) + f.page_tokens - 1) / f.page_tokens : 0;
  for (int64_t i = from + tid; i < f.stride; i += 256) release(f.refs, f.pages, f.table[p * f.stride + i]);
}

// ---- bl_kv_free ----
__global__ __launch_bounds__(256) void k_kv_free(int32_t* refs, int pages, int page_tokens, int32_t* table, int64_t stride,
                                                 const int32_t* keep) {
  const int64_t s = blockIdx.x;
  const int64_t n = keep ? max(keep[s], 0) : 0;
  for (int64_t i = (n + page_tokens - 1) / page_tokens + threadIdx.x; i < stride; i += 256) {
    const int32_t e = table[s * stride + i];
    release(refs, pages, e);
    if (e != -1) table[s * stride + i] = -1;
  }
}

// ---- bl_kv_compact ----
// n pages are used.  The used pages from n on move, the highest to the lowest
// free page below n and so on: with u(p) used pages before page p, the free
// page p < n is the (p - u(p))-th target, the used page p >= n the (n - 1 -
// u(p))-th source.  Three launches: used pages per block; ranks, from the sums
// over the blocks before, taken by every block itself; lists, counts, tables.
constexpr int kCountThreads = 256;
constexpr int kBlockPages = 4096;
constexpr int kOnePages = 16 * kThreads;  // pool of k_kv_compact
constexpr int64_t kOneEntries = 32768;    // and its tables' entries

struct Compact {
  int32_t* refs;
  int pages, page_tokens;
  int32_t* table;
  int64_t entries;
  int moves, asked;  // asked: entries of copies
  int32_t *copies, *moved;
  int32_t *counts, *above, *source, *target, *rank;  // workspace: per block, one, per move (two), per page
};

__device__ __forceinline__ int used_bits(const int32_t* refs, int first, int pages) {
  int bits = 0;
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    if (first + j + 4 <= pages) {
      const int4 r = *reinterpret_cast<const int4*>(refs + first + j);
      bits |= ((r.x != 0) | (r.y != 0) << 1 | (r.z != 0) << 2 | (r.w != 0) << 3) << j;
    } else {
      for (int k = 0; k < 4; ++k)
        if (first + j + k < pages && refs[first + j + k] != 0) bits |= 1 << (j + k);
    }
  }
  return bits;
}

__global__ __launch_bounds__(kCountThreads) void k_kv_count(Compact c) {
  __shared__ int part[kCountThreads / 64];
  const int first = (int)blockIdx.x * kBlockPages + 16 * (int)threadIdx.x;
  const int n = wave_reduce<false>(__popc(used_bits(c.refs, first, c.pages)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x == 0) c.counts[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// used pages of the blocks before this one, and of all
__device__ __forceinline__ void sums_of(const int32_t* counts, int blocks, int block, int* part, int& before, int& all) {
  int b = 0, a = 0;
  for (int i = threadIdx.x; i < blocks; i += kCountThreads) {
    const int n = counts[i];
    a += n;
    b += i < block ? n : 0;
  }
  a = wave_reduce<false>(a);
  b = wave_reduce<false>(b);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    part[wave] = a;
    part[4 + wave] = b;
  }
  __syncthreads();
  all = part[0] + part[1] + part[2] + part[3];
  before = part[4] + part[5] + part[6] + part[7];
}

// The ranks of 16 pages from `first` on, `used` used ones before them, of n in all.
__device__ __forceinline__ void rank_pages(const Compact& c, int first, int bits, int used, int n) {
  for (int j = 0; j < 16 && first + j < c.pages; ++j) {
    const int p = first + j;
    const bool in_use = bits >> j & 1;
    if (p == n) *c.above = n - used;  // used pages from n on: as many as free ones below
    if (p < n) {
      if (!in_use && p - used < c.moves) c.target[p - used] = p;
    } else {
      const int r = in_use ? n - 1 - used : -1;
      c.rank[p] = r;
      if (in_use && r < c.moves) c.source[r] = p;
    }
    used += in_use;
  }
}

__device__ __forceinline__ void no_copy(const Compact& c, int64_t i) {
  c.copies[3 * i] = c.copies[3 * i + 1] = -1;
  c.copies[3 * i + 2] = 0;
}

// Item i: a move, or behind them an entry of the tables.
__device__ __forceinline__ void rename(const Compact& c, int64_t i, int n, int moved) {
  if (i >= c.moves) {
    const int32_t e = c.table[i - c.moves];
    if (e < n || e >= c.pages) return;
    const int r = c.rank[e];
    if (r >= 0 && r < moved) c.table[i - c.moves] = c.target[r];
  } else if (i < moved) {
    const int from = c.source[i], to = c.target[i];
    c.copies[3 * i] = from;
    c.copies[3 * i + 1] = to;
    c.copies[3 * i + 2] = c.page_tokens;
    c.refs[to] = c.refs[from];
    c.refs[from] = 0;
  } else {
    no_copy(c, i);
  }
}

__global__ __launch_bounds__(kCountThreads) void k_kv_rank(Compact c) {
  __shared__ int part[8], wave_used[4];
  const int blocks = (int)gridDim.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int used, n;
  sums_of(c.counts, blocks, (int)blockIdx.x, part, used, n);
  const int first = (int)blockIdx.x * kBlockPages + 16 * tid;
  const int bits = used_bits(c.refs, first, c.pages), mine = __popc(bits);
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int other = __shfl_up(sum, d, 64);
    if (lane >= d) sum += other;
  }
  if (lane == 63) wave_used[wave] = sum;
  __syncthreads();
  for (int w = 0; w < wave; ++w) used += wave_used[w];
  used += sum - mine;  // used pages before this thread's first
  if (blockIdx.x == 0 && tid == 0 && n == c.pages) *c.above = 0;
  rank_pages(c, first, bits, used, n);
}

__global__ __launch_bounds__(kCountThreads) void k_kv_rename(Compact c, int blocks) {
  __shared__ int part[8];
  int before, n;
  sums_of(c.counts, blocks, 0, part, before, n);
  const int moved = min(*c.above, c.moves);
  if (blockIdx.x == 0 && threadIdx.x == 0) *c.moved = moved;
  for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < c.moves + c.entries;
       i += (int64_t)gridDim.x * kCountThreads)
    rename(c, i, n, moved);
}

// All of it in one workgroup with its lists in LDS, for a pool and tables that
// it is done with sooner than three launches are (2048 pages, 1536 entries: 5 us
// against 12).
__global__ __launch_bounds__(kThreads) void k_kv_compact(Compact c) {
  __shared__ int part[kThreads / 64], above;
  __shared__ int rank[kOnePages], target[kOnePages / 2], source[kOnePages / 2];
  const int tid = threadIdx.x, first = 16 * tid;
  const int bits = used_bits(c.refs, first, c.pages);
  int n;
  const int used = block_prefix(__popc(bits), part, n);
  c.above = &above;
  c.rank = rank;
  c.target = target;
  c.source = source;
  if (tid == 0 && n == c.pages) above = 0;
  // no more of them than there are used pages above n, or free ones below
  c.moves = min(c.moves, kOnePages / 2);
  rank_pages(c, first, bits, used, n);
  __syncthreads();
  const int moved = min(above, c.moves);
  if (tid == 0) *c.moved = moved;
  for (int64_t i = tid; i < c.moves + c.entries; i += kThreads) rename(c, i, n, moved);
  for (int64_t i = c.moves + tid; i < c.asked; i += kThreads) no_copy(c, i);
}

// ---- bl_kv_copy ----
// A wave moves a piece of 4 KB: four 16-byte loads of a lane in flight, then
// their stores.  A piece belongs to the codes of one copy, cache, head and of k
// or v; the wave of a head's first piece moves its scale.  HBM-bound: 345 MB of
// half a batch's pages take 66 us (5.2 TB/s).  Stores go past the caches: a step
// that copies 135 MB of 192 forks' pages in four caches takes 25 us against 34,
// and 527 against 530 with the attention over them next.  Pieces of 2 KB and 8 KB: 4 us and 1 more;
// 2048 workgroups that go over the pieces in turn instead of one per four: 6 us
// more for the larger.
typedef unsigned v4u __attribute__((ext_vector_type(4)));

constexpr int kCopyThreads = 256;
constexpr int kPiece = 4096;
constexpr int64_t kCopyBlocks = 65536;

struct CopyArgs {
  int8_t* codes[kCopyCaches][2];
  float* absmax[kCopyCaches][2];
  const int32_t *copies, *count;
  int64_t n;
  int pages, heads, page_tokens, dim, caches, pieces;
};

__global__ __launch_bounds__(kCopyThreads) void k_kv_copy(CopyArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t waves = (int64_t)gridDim.x * (kCopyThreads / 64);
  int64_t n = a.n;
  if (a.count) {
    const int64_t told = *a.count;
    n = told < n ? told : n;
  }
  const int per_copy = a.caches * 2 * a.heads * a.pieces;
  for (int64_t item = (int64_t)blockIdx.x * (kCopyThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
       item < n * per_copy; item += waves) {
    const int64_t copy = item / per_copy;
    int rest = (int)(item - copy * per_copy);
    const int piece = rest % a.pieces;
    rest /= a.pieces;
    const int head = rest % a.heads;
    rest /= a.heads;
    const int which = rest & 1, cache = rest >> 1;
    const int32_t* entry = a.copies + 3 * copy;
    const int from = entry[0], to = entry[1], tokens = min(entry[2], a.page_tokens);
    if ((uint32_t)from >= (uint32_t)a.pages || (uint32_t)to >= (uint32_t)a.pages || tokens <= 0 || from == to) continue;
    const int64_t src = (int64_t)from * a.heads + head, dst = (int64_t)to * a.heads + head;
    const int64_t block = (int64_t)a.page_tokens * a.dim;
    const int bytes = tokens * a.dim;  // a multiple of 16
    const int8_t* in = a.codes[cache][which] + src * block;
    int8_t* out = a.codes[cache][which] + dst * block;
    v4u w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = piece * kPiece + (i * 64 + lane) * 16;
      w[i] = *reinterpret_cast<const v4u*>(in + min(at, bytes - 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = piece * kPiece + (i * 64 + lane) * 16;
      if (at < bytes) __builtin_nontemporal_store(w[i], reinterpret_cast<v4u*>(out + at));
    }
    if (piece == 0 && lane == 0) a.absmax[cache][which][dst] = a.absmax[cache][which][src];
  }
}

int64_t compact_blocks(int64_t pages) { return (pages + kBlockPages - 1) / kBlockPages; }

}  // namespace

hipError_t launch_kv_grow(int32_t* refs, int64_t pages, int page_tokens, const KvStep& st, int64_t seqs, int64_t max_new,
                          int32_t* table, int32_t* copies, int32_t* shortage, hipStream_t s) {
  const int touched = (int)((max_new + page_tokens - 2) / page_tokens + 1);
  const Grow g = {refs, (int)pages, page_tokens, st, seqs, touched, table, copies, shortage};
  hipLaunchKernelGGL(k_kv_grow, dim3(1), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

hipError_t launch_kv_fork(int32_t* refs, int64_t pages, int page_tokens, const int32_t* table, int64_t stride,
                          const int32_t* length, int64_t seqs, const int32_t* parent, int64_t children, bool keep_parents,
                          int32_t* table_out, int32_t* length_out, int32_t* copies, int32_t* shortage, hipStream_t s) {
  const bool here = !keep_parents && children > 0 && seqs * stride <= kReleaseHere;
  const Fork f = {refs,          (int)pages,   page_tokens, table,     length,     parent, stride,  (int)seqs,
                  (int)children, keep_parents, here,        table_out, length_out, copies, shortage};
  if (children > 0) {
    hipLaunchKernelGGL(k_kv_fork, dim3(1 + (unsigned)children), dim3(kThreads), 0, s, f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (keep_parents || seqs == 0 || here) return hipSuccess;
  hipLaunchKernelGGL(k_kv_fork_release, dim3((unsigned)seqs), dim3(256), 0, s, f);
  return hipGetLastError();
}

hipError_t launch_kv_free(int32_t* refs, int64_t pages, int page_tokens, int32_t* table, int64_t stride, int64_t seqs,
                          const int32_t* keep, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_free, dim3((unsigned)seqs), dim3(256), 0, s, refs, (int)pages, page_tokens, table, stride, keep);
  return hipGetLastError();
}

size_t kv_compact_workspace_bytes(int64_t pages, int64_t moves) {
  return 4 * (size_t)(compact_blocks(pages) + 1 + 2 * moves + pages);
}

hipError_t launch_kv_compact(int32_t* refs, int64_t pages, int page_tokens, int32_t* table, int64_t stride, int64_t seqs,
                             int64_t moves, int32_t* copies, int32_t* moved, void* workspace, hipStream_t s) {
  const int64_t blocks = compact_blocks(pages), entries = seqs * stride;
  Compact c = {refs, (int)pages, page_tokens, table, entries, (int)moves, (int)moves, copies, moved};
  if (pages <= kOnePages && entries <= kOneEntries) {
    hipLaunchKernelGGL(k_kv_compact, dim3(1), dim3(kThreads), 0, s, c);
    return hipGetLastError();
  }
  c.counts = (int32_t*)workspace;
  c.above = c.counts + blocks;
  c.source = c.above + 1;
  c.target = c.source + moves;
  c.rank = c.target + moves;
  hipLaunchKernelGGL(k_kv_count, dim3((unsigned)blocks), dim3(kCountThreads), 0, s, c);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_kv_rank, dim3((unsigned)blocks), dim3(kCountThreads), 0, s, c);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t wanted = (moves + entries + kCountThreads - 1) / kCountThreads;
  hipLaunchKernelGGL(k_kv_rename, dim3((unsigned)(wanted < 1 ? 1 : wanted < 2048 ? wanted : 2048)), dim3(kCountThreads), 0, s,
                     c, (int)blocks);
  return hipGetLastError();
}

hipError_t launch_kv_copy(const KvView* caches, int64_t count, const int32_t* copies, int64_t n, const int32_t* valid,
                          hipStream_t s) {
  for (int64_t done = 0; done < count; done += kCopyCaches) {
    CopyArgs a;
    a.caches = (int)(count - done < kCopyCaches ? count - done : kCopyCaches);
    for (int i = 0; i < a.caches; ++i) {
      const KvView& kv = caches[done + i];
      a.codes[i][0] = kv.k;
      a.codes[i][1] = kv.v;
      a.absmax[i][0] = kv.k_absmax;
      a.absmax[i][1] = kv.v_absmax;
    }
    const KvView& kv = caches[done];
    a.copies = copies;
    a.count = valid;
    a.n = n;
    a.pages = (int)kv.pages;
    a.heads = kv.heads;
    a.page_tokens = kv.page_tokens;
    a.dim = kv.dim;
    a.pieces = (kv.page_tokens * kv.dim + kPiece - 1) / kPiece;
    const int64_t items = n * a.caches * 2 * kv.heads * a.pieces, wanted = (items + 3) / 4;
    hipLaunchKernelGGL(k_kv_copy, dim3((unsigned)(wanted < kCopyBlocks ? wanted : kCopyBlocks)), dim3(kCopyThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bl
