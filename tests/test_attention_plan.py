"""The attention's split along the keys on the host: whatever stands in the
device's positions and offsets, no tile takes more steps of keys than the plan
and its workspace hold, none is left without one, and lengths that keep the
bounds are covered whole.

The planner and the arithmetic of the tiles are compiled from attention.hip
itself together with the checks below; nothing is launched."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "ternary_weight_absmean_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

CHECK = """
#include "attention.hip"

namespace {
uint64_t state;
// 0 .. below - 1, small numbers as often as large ones
int64_t draw(int64_t below) {
  auto next = [] { return (state = state * 6364136223846793005ull + 1442695040888963407ull) >> 20; };
  int64_t most = below;
  for (uint64_t halve = next() % 24; halve > 0 && most > 2; --halve) most = (most + 1) / 2;
  return (int64_t)(next() % (uint64_t)most);
}
int any_int() { return (int)(draw(2) ? draw((int64_t)1 << 31) : -draw((int64_t)1 << 31)); }
}  // namespace

// Which check fails first in `batches` random batches (0: none); the batch's numbers in `out`.
extern "C" int check(uint64_t seed, int batches, int trusted, int64_t* out) {
  using namespace bl;
  state = seed;
  for (int b = 0; b < batches; ++b) {
    const int pages_of[5] = {16, 32, 64, 128, 256};
    KvView kv = {};
    kv.heads = 1 + (int)draw(64);
    kv.page_tokens = pages_of[draw(5)];
    kv.dim = 16 * (1 + (int)draw(16));
    kv.pages = 8;
    const int group = 1 + (int)draw(32);
    const int64_t q_heads = (int64_t)kv.heads * group, seqs = 1 + draw(64);
    KvStep st = {};
    st.tokens = 1 + (int)draw(1 << 16);
    st.max_new = 1 + (int)draw(st.tokens);
    const int64_t max_len = st.max_new + draw(1 << 20);
    st.table_stride = (max_len + kv.page_tokens - 1) / kv.page_tokens + draw(1 << 16);  // room past max_len
    const int64_t window = draw(2) ? 1 + draw(1 << 18) : 0, sinks = window ? draw(512) : 0;
    const Plan p = make_plan(kv, seqs, st.max_new, max_len, q_heads, window, sinks);
    const int64_t held = most_splits(kv, seqs, st.max_new, max_len, q_heads);
    const int64_t numbers[] = {kv.heads, kv.page_tokens, kv.dim, group, seqs, st.tokens, st.max_new, max_len, window, sinks,
                               p.tile_rows, p.splits, p.per, held};
    for (int i = 0; i < 14; ++i) out[i] = numbers[i];
    if (p.splits < 1 || p.per < 1 || p.splits > held) return 1;
    if (attention_workspace_bytes(kv, seqs, st.tokens, st.max_new, max_len, q_heads) <
        (held > 1 ? (size_t)st.tokens * q_heads * p.splits * (kv.dim + 2) * 4 : 0))
      return 2;
    for (int i = 0; i < 40; ++i) {
      int from, to, start;
      if (trusted) {
        const int count = 1 + (int)draw(st.max_new);
        from = (int)draw(st.tokens - count + 1), to = from + count;
        start = draw(2) ? (int)max_len - count : (int)draw(max_len - count + 1);
      } else {
        from = any_int(), to = any_int(), start = draw(2) ? any_int() : (int)(max_len - st.max_new + draw(4096));
      }
      const int begin = st.begin_of(from), count = st.count_of(begin, to), first = st.start_from(start);
      if (begin < 0 || count < 0 || count > st.max_new || begin + count > st.tokens || first < 0) return 3;
      if (trusted && (begin != from || count != to - from || first != start)) return 4;
      const int64_t rows = (int64_t)count * group;
      if (rows > p.row_tiles * p.tile_rows) return 5;
      if (rows == 0) continue;
      for (int which = 0; which < 3; ++which) {  // the first, the last and some tile
        const int64_t last_tile = (rows - 1) / p.tile_rows;
        const int64_t row0 = p.tile_rows * (which == 0 ? 0 : which == 1 ? last_tile : draw(last_tile + 1));
        const int64_t end = row0 + p.tile_rows < rows ? row0 + p.tile_rows : rows;
        const int first_pos = first + (int)(row0 / group), last_pos = first + (int)((end - 1) / group);
        const Span s = span_of(first_pos, last_pos, (int)max_len, (int)window, (int)sinks);
        out[14] = first_pos, out[15] = last_pos, out[16] = s.steps;
        if (s.steps < 1 || s.keys < 1 || s.keys > max_len || s.keys > st.table_stride * kv.page_tokens) return 6;
        if ((s.steps + p.per - 1) / p.per > p.splits) return 7;  // a slot that the row does not have
        int before = -1;
        for (int step = 0; step < s.steps; ++step) {
          const int key = s.key0(step);
          if (key <= before || key % kStep != 0 || key >= s.keys) return 8;
          before = key;
        }
        if (!trusted) continue;
        if (s.keys != last_pos + 1 || s.key0(s.steps - 1) + kStep < s.keys) return 9;
        const int64_t low = window > 0 && first_pos - window + 1 > 0 ? first_pos - window + 1 : 0;
        if (s.key0(s.sink_steps) > low) return 10;  // a visible key is left out
        const int64_t sunk = sinks < s.base * kStep ? sinks : s.base * kStep;
        if (s.sink_steps * kStep < sunk) return 11;
      }
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is missing")
    tmp = tmp_path_factory.mktemp("plan")
    src, so = str(tmp / "plan_check.hip"), str(tmp / "plan_check.so")
    with open(src, "w") as f:
        f.write(CHECK)
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-fPIC", "-shared",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", CSRC, "-I", os.path.join(ROOT, "include"), src, "-o", so], check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(so)
    lib.check.argtypes = [ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def run(seed, batches, trusted):
        out = (ctypes.c_int64 * 17)()
        failed = lib.check(seed, batches, trusted, out)
        assert failed == 0, f"check {failed} with {list(out)}"
    return run


@pytest.mark.parametrize("seed", range(4))
def test_lengths_within_their_bounds_are_covered(check, seed):
    check(seed, 30000, 1)


@pytest.mark.parametrize("seed", range(4))
def test_no_device_integer_leads_past_the_plan(check, seed):
    check(seed, 30000, 0)
