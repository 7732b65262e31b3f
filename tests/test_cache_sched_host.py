"""How attention over the cache deals its work, run on the CPU: the dealing code
itself, cut out of the kernel source and compiled with 32 threads as a warp.

Equal runs of all items' tiles must cover every tile of every item once and
chain the parts of an item over consecutive CTAs.  Lengths live on the device
and belong to the caller: should they change while a call reads them, its
numbers are worth nothing, but every loop must end and every index stay in
range."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "sparse_attention_diffusion_mcs_b200", "csrc")

SHIM = r"""
#include <algorithm>
#include <atomic>
#include <barrier>
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>
using std::max;
using std::min;
#define __device__
#define __host__
#define __forceinline__ inline
// the caller's tensor: from the `change`-th read on it holds other numbers; a whole
// warp's reads between two exchanges see the same
static int n_seq;
static long long change = LLONG_MAX;
static std::atomic<long long> reads{0};
static std::atomic<bool> other{false};
static bool alone = false;
static long long exchanges = 0;
struct Look {
  void operator()() noexcept {
    other = reads >= change;
    if (++exchanges > 20000) std::puts("exchanges without an end"), std::fflush(stdout), std::_Exit(3);
  }
};
static std::barrier<Look> warp_bar(32);
static long long box[32];
static thread_local int lane_id;
template <typename F> static long long exchange(long long v, F pick) {
  box[lane_id] = v;
  warp_bar.arrive_and_wait();
  const long long r = pick();
  warp_bar.arrive_and_wait();
  return r;
}
template <typename T> T __shfl_xor_sync(unsigned, T v, int o) { return (T)exchange(v, [&] { return box[lane_id ^ o]; }); }
template <typename T> T __shfl_up_sync(unsigned, T v, int o) { return (T)exchange(v, [&] { return box[lane_id >= o ? lane_id - o : lane_id]; }); }
template <typename T> T __shfl_sync(unsigned, T v, int l) { return (T)exchange(v, [&] { return box[l & 31]; }); }
static unsigned __ballot_sync(unsigned, bool p) {
  return (unsigned)exchange(p, [&] { unsigned m = 0; for (int i = 0; i < 32; ++i) m |= (unsigned)(box[i] != 0) << i; return (long long)m; });
}
static int __ffs(unsigned x) { return __builtin_ffs((int)x); }
static void record_status(unsigned *, unsigned) {}
constexpr unsigned kStatusBadMeta = 6;
static void fail(const char *why, long long x) { std::printf("%s %lld\n", why, x); std::fflush(stdout); std::_Exit(3); }
struct Lens {
  const int *a = nullptr, *b = nullptr;
  int operator[](int i) const {
    if (i < 0 || i >= n_seq) fail("read of sequence", i);
    const long long n = reads++;
    if (n > 300000) fail("reads without an end", n);
    if (alone) other = n >= change;
    return (other ? b : a)[i];
  }
  explicit operator bool() const { return a != nullptr; }
};
"""

MAIN = r"""
template <int BM, bool HALVES> static void deal(const SchedArgs &s, int n_cta, int min_quota, bool stable) {
  using S = Sched<BM, HALVES>;
  const size_t items = (size_t)s.B * s.H * s.n_blocks;
  std::vector<int> next_tile(items, 0), expect(items, -1);
  for (int cta = 0; cta < n_cta; ++cta) {
    S run{};
    alone = false;
    exchanges = 0;
    std::vector<std::thread> warp;
    for (int l = 0; l < 32; ++l)
      warp.emplace_back([&, l] {
        lane_id = l;
        S mine;
        mine.start(s, cta, n_cta, min_quota, l, nullptr);
        if (l == 0) run = mine;
      });
    for (auto &t : warp) t.join();
    lane_id = 0;
    alone = true;
    Segment g;
    for (long long steps = 0; run.next(s, g); ++steps) {
      if (steps > (long long)items) fail("parts without an end", cta);
      if (g.b < 0 || g.b >= s.B || g.h < 0 || g.h >= s.H || g.block < 0 || g.block >= s.n_blocks) fail("an item out of range", g.h);
      if (g.len < 0 || g.len > s.cap || g.nq < 0 || g.nq > s.Nq || g.kmax < 0 || g.kmax > s.cap) fail("lengths out of range", g.len);
      if (g.t0 < 0 || g.t1 < g.t0 || (g.t1 > g.t0 && g.t1 > max((g.kmax + kKeyTile - 1) / kKeyTile, 1))) fail("tiles out of range", g.t1);
      if (g.go_on < 0 || (stable && cta + g.go_on >= n_cta)) fail("goes on behind the last CTA", g.go_on);
      if (!stable) continue;
      const size_t i = ((size_t)g.b * s.H + g.h) * s.n_blocks + g.block;
      if (g.t0 != next_tile[i]) fail("a tile left out or dealt twice", g.t0);
      next_tile[i] = g.t1;
      if (g.first != (expect[i] < 0)) fail("not where the item begins", cta);
      if (g.first) expect[i] = cta + g.go_on;
      else if (g.t1 > g.t0 && cta > expect[i]) fail("a part behind the item's last CTA", cta);
    }
  }
  for (int b = 0; stable && b < s.B; ++b)
    for (int h = 0; h < s.H; ++h)
      for (int k = 0; k < s.n_blocks; ++k) {
        Segment g;
        if (next_tile[((size_t)b * s.H + h) * s.n_blocks + k] != S::item(s, b, k, g)) fail("tiles left out", k);
      }
}

int main(int argc, char **argv) {
  // B H Nq share causal cap n_cta change counted, then B lengths, B other lengths, B counts, B other counts
  int p = 1;
  auto num = [&] { return std::atoi(argv[p++]); };
  SchedArgs s;
  std::memset((void *)&s, 0, sizeof(s));
  s.B = n_seq = num(); s.H = num(); s.Nq = num(); s.share = num(); s.causal = num(); s.cap = num();
  const int n_cta = num(), when = num(), counted = num();
  std::vector<int> v[4];
  for (auto &x : v) for (int i = 0; i < s.B; ++i) x.push_back(num());
  s.lengths.a = v[0].data(); s.lengths.b = v[1].data();
  if (counted) { s.counts.a = v[2].data(); s.counts.b = v[3].data(); }
  s.n_rows = s.Nq * s.share;
  for (int which = 0; which < 2; ++which) {
    change = when < 0 ? LLONG_MAX : when;
    reads = 0;
    other = change == 0;
    s.n_blocks = which ? (s.n_rows + 255) / 256 : (s.n_rows + 15) / 16;
    if (which) deal<256, true>(s, n_cta, 4, when < 0);
    else deal<16, false>(s, n_cta, 4, when < 0);
  }
  std::puts("fine");
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    src = open(os.path.join(CSRC, "cache_sched.cuh")).read()
    part = src[src.index("constexpr int kKeyTile"):src.index("// What the merge knows of a CTA")]
    part, n = re.subn(r"const int32_t \*(lengths|counts);", r"Lens \1;", part)
    assert n == 2
    at = tmp_path_factory.mktemp("sched")
    (at / "deal.cpp").write_text(SHIM + part + MAIN)
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", "-o", str(at / "deal"), str(at / "deal.cpp")], check=True)
    return str(at / "deal")


def run(program, B, H, Nq, share, causal, cap, n_cta, change, lengths, others=None, counts=None, other_counts=None):
    args = [B, H, Nq, share, int(causal), cap, n_cta, change, int(counts is not None)]
    args += lengths + (others or lengths) + (counts or [0] * B) + (other_counts or counts or [0] * B)
    r = subprocess.run([program] + [str(x) for x in args], capture_output=True, text=True, timeout=60)
    assert (r.returncode, r.stdout) == (0, "fine\n"), r.stdout


CASES = [
    (1, 1, 1, 1, True, 128, [1], None), (3, 2, 1, 4, True, 9000, [8300, 0, 700], None),
    (2, 3, 40, 2, False, 2000, [2000, 129], None), (2, 1, 300, 1, True, 1000, [300, 11], [300, 299]),
    (40, 2, 1, 8, True, 700, [(37 * i * i) % 701 for i in range(40)], None),
    (2, 2, 700, 4, True, 4096, [4096, 100], [0, 700]), (33, 1, 5, 1, False, 300, [300] * 33, [i % 6 for i in range(33)]),
]


@pytest.mark.parametrize("n_cta", [3, 16])
@pytest.mark.parametrize("case", CASES)
def test_every_tile_once(program, case, n_cta):
    B, H, Nq, share, causal, cap, lengths, counts = case
    run(program, B, H, Nq, share, causal, cap, n_cta, -1, lengths, counts=counts)


@pytest.mark.parametrize("change", [1, 7, 40, 200, 500])
@pytest.mark.parametrize("case", CASES)
def test_lengths_that_change_end_every_loop(program, case, change):
    """All of a call's later reads see shorter, none, or longer sequences."""
    B, H, Nq, share, causal, cap, lengths, counts = case
    for others, other_counts in (([-2 ** 31] * B, None), ([n // 3 for n in lengths], [-5] * B), ([2 ** 31 - 1] * B, [2 ** 31 - 1] * B)):
        run(program, B, H, Nq, share, causal, cap, 5, change, lengths, others, counts, counts and other_counts)
