// cache_sched.cuh -- how attention over the cache is dealt to CTAs, and the
// merge of what is dealt to several.
//
// A block of query rows of one (sequence, key head) is an item; its work is
// its tiles of 128 keys, each counted once per 128-row half that has rows to
// compute.  Lengths live on the device, so the CTAs deal the work themselves:
// each adds up the items' units and takes an equal run of them, which may end
// inside an item.  Whole items are finished by their CTA; of the others a CTA
// leaves (reference, sum, O) in its slots of the workspace -- at most two, its
// first item and its last -- and writes down where an item goes on, and
// cache_merge_kernel, launched behind, adds the parts up in the order of the
// keys.  No atomics: results repeat bit for bit.
//
// Lengths are read again and again, here and by the roles of a CTA.  A caller that
// changes them while a call runs gets numbers that are worth nothing; but every
// loop is bounded by sizes that the host gave, and every index is in range.
#pragma once

#include "kvcache_kernels.cuh"

namespace mcs {

constexpr int kKeyTile = 128;

struct SchedArgs {
  const int32_t *lengths;        // [B] tokens kept
  const int32_t *counts;         // [B] query tokens, or null: Nq
  int B, H, Nq, share;           // share: query heads per key head
  int causal;
  int cap;                       // places of a sequence's row of the page table
  int n_rows, n_blocks;          // Nq * share; blocks of BM rows
};

// one item, and the part of it that is this CTA's
struct Segment {
  int b, h, block;
  int len, nq;                   // the sequence's tokens and query tokens
  int kmax;                      // keys that some row of the block sees: [0, kmax)
  int halves;                    // halves of BM/2 rows with something to compute (1 or 2)
  int t0, t1;                    // key tiles [t0, t1)
  bool first, whole;             // holds the item's beginning; holds all of it
  int go_on;                     // CTAs that the item goes on in
};

template <int BM, bool HALVES>
struct Sched {
  // len, nq, kmax, halves of an item; its number of tiles, at least 1 (rows that see nothing are written too)
  static __device__ __forceinline__ int item(const SchedArgs &s, int b, int block, Segment &g) {
    g.len = min(max(s.lengths[b], 0), s.cap);
    g.nq = s.counts ? min(max(s.counts[b], 0), s.Nq) : s.Nq;
    const int row0 = block * BM;
    const int last = min(min(row0 + BM, s.n_rows), g.nq * s.share) - 1;   // last row with a query
    g.kmax = last < row0 ? 0 : s.causal ? max(g.len - g.nq + last / s.share + 1, 0) : g.len;
    g.halves = HALVES && last - row0 >= BM / 2 ? 2 : 1;
    return max((g.kmax + kKeyTile - 1) / kKeyTile, 1);
  }
  static __device__ __forceinline__ long long units(const SchedArgs &s, int b, int block) {
    Segment g;
    const int t = item(s, b, block, g);
    return static_cast<long long>(t) * g.halves;
  }

  int b, h, block;
  long long off, left;           // units of the current item before this CTA's, and units left of this CTA's
  long long quota;

  static __device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  static __device__ __forceinline__ long long warp_scan(long long v, int lane) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  }
  // one sequence's units, all its heads; by a whole warp
  static __device__ long long sequence_units(const SchedArgs &s, int b, int lane) {
    long long v = 0;
    for (int k = lane; k < s.n_blocks; k += 32) v += units(s, b, k);
    return warp_sum(v) * s.H;
  }

  // This CTA's run of units; by a whole warp.  Few blocks per sequence: a lane
  // adds up a sequence; else the warp does.
  __device__ void start(const SchedArgs &s, int cta, int n_cta, int min_quota, int lane, unsigned *status) {
    long long total = 0;
    const bool by_lane = s.n_blocks <= 4;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      const bool have = b0 + lane < s.B;
      if (have && s.lengths[b0 + lane] > s.cap) record_status(status, kStatusBadMeta);
      if (by_lane) {
        long long v = 0;
        for (int k = 0; have && k < s.n_blocks; ++k) v += units(s, b0 + lane, k);
        total += warp_sum(v) * s.H;
      } else {
        for (int i = b0; i < min(b0 + 32, s.B); ++i) total += sequence_units(s, i, lane);
      }
    }
    quota = (total + n_cta - 1) / n_cta;
    quota = quota < min_quota ? min_quota : quota;
    const long long u0 = quota * cta;
    const long long share_of = total - u0 < quota ? total - u0 : quota;
    left = 0;                                // (unless the run's beginning is found)
    b = h = block = 0;
    off = 0;
    if (share_of <= 0) return;
    long long before = 0, mine = 0;          // units before the sequence, and of one of its heads
    if (by_lane) {
      for (int b0 = 0; b0 < s.B; b0 += 32) {   // (found: u0 < total)
        long long v = 0;
        for (int k = 0; b0 + lane < s.B && k < s.n_blocks; ++k) v += units(s, b0 + lane, k);
        const long long sum = warp_scan(v * s.H, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > u0);
        if (hit) {
          const int l = __ffs(hit) - 1;
          b = b0 + l;
          mine = __shfl_sync(0xffffffffu, v, l);
          before += __shfl_sync(0xffffffffu, sum, l) - mine * s.H;
          break;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    } else {
      for (b = 0; b < s.B; ++b) {
        const long long v = sequence_units(s, b, lane);
        if (before + v > u0) {
          mine = v / s.H;
          break;
        }
        before += v;
      }
    }
    if (mine == 0) return;
    long long r = u0 - before;
    h = static_cast<int>(r / mine);
    r -= h * mine;
    for (int k0 = 0; k0 < s.n_blocks; k0 += 32) {   // (found: r < mine)
      const long long v = k0 + lane < s.n_blocks ? units(s, b, k0 + lane) : 0;
      const long long sum = warp_scan(v, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, sum > r);
      if (hit) {
        const int l = __ffs(hit) - 1;
        block = k0 + l;
        off = r - (__shfl_sync(0xffffffffu, sum, l) - __shfl_sync(0xffffffffu, v, l));
        left = share_of;
        return;
      }
      r -= __shfl_sync(0xffffffffu, sum, 31);
    }
  }

  // whether next() has another part
  __device__ __forceinline__ bool more(const SchedArgs &s) const { return left > 0 && b < s.B; }
  // the next part of this CTA's run
  __device__ __forceinline__ bool next(const SchedArgs &s, Segment &g) {
    if (!more(s)) return false;
    g.b = b;
    g.h = h;
    g.block = block;
    const int tiles = item(s, b, block, g);
    const long long all = static_cast<long long>(tiles) * g.halves;
    const long long rest = all > off ? all - off : 0, take = rest < left ? rest : left;
    // tile t is of the CTA that has the unit t * halves
    g.t0 = static_cast<int>((off + g.halves - 1) / g.halves);
    g.t1 = static_cast<int>((off + take + g.halves - 1) / g.halves);
    g.first = off == 0;
    g.whole = g.t0 == 0 && g.t1 == tiles;
    g.go_on = g.whole ? 0 : static_cast<int>((rest - take + quota - 1) / quota);
    left -= take;
    off = 0;
    if (++block == s.n_blocks) {
      block = 0;
      if (++h == s.H) {
        h = 0;
        ++b;
      }
    }
    return true;
  }
};

// What the merge knows of a CTA: the item that begins in it and goes on.
struct MergeItem {
  int b, h, block;
  int go_on;                     // CTAs that it goes on in (0: nothing to merge)
};
// A CTA's slots: 2 cta, the item that it goes on with; 2 cta + 1, the one that begins in it and goes on.

// The workspace of n_cta CTAs with blocks of `rows` rows
struct MergeSpace {
  MergeItem *items;              // [n_cta]
  float2 *ml;                    // [2 n_cta, rows]  reference (log2 units) and sum
  float4 *o;                     // [2 n_cta, d / 4, rows]: what neighbouring rows' threads write lies together
};
__host__ __device__ inline size_t merge_space(int n_cta, int rows, int d, void *base, MergeSpace *m) {
  const size_t a = (static_cast<size_t>(n_cta) * sizeof(MergeItem) + 15) / 16 * 16;
  const size_t b = static_cast<size_t>(n_cta) * 2 * rows * sizeof(float2);
  if (m) {
    uint8_t *p = static_cast<uint8_t *>(base);
    m->items = reinterpret_cast<MergeItem *>(p);
    m->ml = reinterpret_cast<float2 *>(p + a);
    m->o = reinterpret_cast<float4 *>(p + a + b);
  }
  return a + b + static_cast<size_t>(n_cta) * 2 * rows * d * sizeof(float);
}

// numbers 4 quad .. 4 quad + 3 of row r of the slot that `before` rows precede
__device__ __forceinline__ float4 *merge_part(const MergeSpace &m, size_t before, int rows, int d, int r, int quad) {
  return m.o + before * (d / 4) + static_cast<size_t>(quad) * rows + r;
}

struct MergeArgs {
  MergeSpace m;
  bf16 *O;                       // [B, H * share, Nq, d]
  float *lse;
  int H, Nq, share, n_rows, rows;
};

constexpr int kMergeThreads = 256;

// weight of a part with reference m under the joint reference mm (no keys: m = -inf, l = 0; NaN stays)
__device__ __forceinline__ float merge_factor(float m, float l, float mm) {
  return l != l ? l : m == -INFINITY ? 0.f : ex2_approx(m - mm);
}

// the parts of one row's quad of numbers, added up
struct MergeSum {
  float m, l;                    // joint reference and sum
  float4 acc;
};
__device__ __forceinline__ void merge_add(MergeSum &s, float m, float l, const float4 &x, float mm) {
  const float f = merge_factor(m, l, mm);
  if (f != 0.f) {                                          // (NaN counts; a part without keys has no O)
    s.l = fmaf(l, f, s.l);
    s.acc = make_float4(fmaf(x.x, f, s.acc.x), fmaf(x.y, f, s.acc.y), fmaf(x.z, f, s.acc.z), fmaf(x.w, f, s.acc.w));
  }
}
__device__ __forceinline__ MergeSum merge_parts(const MergeArgs &a, int c, int go_on, int d, int r, int quad, int k0,
                                                int step) {
  auto before = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)) * a.rows; };
  // two parts at once, the first two (mostly all) before anything waits for them
  float2 p[2];
  float4 x[2];
  auto load = [&](int k) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      p[u] = make_float2(-INFINITY, 0.f);
      if (k + u * step <= go_on) {
        const size_t at = before(k + u * step);
        p[u] = a.m.ml[at + r];
        x[u] = *merge_part(a.m, at, a.rows, d, r, quad);
      }
    }
  };
  load(k0);
  MergeSum s;
  s.m = fmaxf(p[0].x, p[1].x);
#pragma unroll 4
  for (int k = k0 + 2 * step; k <= go_on; k += step) s.m = fmaxf(s.m, a.m.ml[before(k) + r].x);
  s.l = 0.f;
  s.acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = k0; k <= go_on; k += 2 * step) {
    if (k > k0) load(k);
#pragma unroll
    for (int u = 0; u < 2; ++u) merge_add(s, p[u].x, p[u].y, x[u], s.m);
  }
  return s;
}

// CTA (c, y): a share of the item that begins in CTA c.  A warp takes 8 rows x 4
// quads of numbers: 128-byte lines of the parts, 32 bytes of O.  Few parts an
// item: the warps take rows y, y + gridDim.y, ... (in steps of what a CTA takes
// at once).  Many (SPLIT): all eight warps take the same 8 rows and 4 quads, of
// every eighth part each, and add up through shared memory, in the warps' order.
// Either way bound by a few reads that wait for one another: the item, then
// the parts, out of the second-level cache.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kMergeThreads, 6) cache_merge_kernel(const __grid_constant__ MergeArgs a) {
  const int c = blockIdx.x;
  MergeItem it = a.m.items[c];
  if (it.go_on == 0) return;
  it.go_on = min(it.go_on, static_cast<int>(gridDim.x) - 1 - c);   // (gridDim.x: the CTAs that computed)
  constexpr int QG = D / 16;                                 // groups of 4 quads
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row0 = it.block * a.rows;
  const int rows = min(a.rows, a.n_rows - row0);
  auto finish = [&](const MergeSum &s, int r, int quad) {
    const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
    const int row = row0 + r, i = row / a.share, hq = it.h * a.share + row % a.share;
    const size_t at = (static_cast<size_t>(it.b) * a.H * a.share + hq) * a.Nq + i;
    *reinterpret_cast<uint2 *>(a.O + at * D + 4 * quad) =
        make_uint2(pack_bf16x2(s.acc.x * inv, s.acc.y * inv), pack_bf16x2(s.acc.z * inv, s.acc.w * inv));
    if (a.lse && quad == 0) a.lse[at] = s.l == 0.f ? -INFINITY : (s.m + log2f(s.l)) * 0.6931471805599453f;
  };
  if constexpr (SPLIT) {
    __shared__ MergeSum part[8][32];
    const int r = blockIdx.y / QG * 8 + lane % 8, quad = blockIdx.y % QG * 4 + lane / 8;
    if (r < rows) part[warp][lane] = merge_parts(a, c, it.go_on, D, r, quad, warp, 8);
    __syncthreads();
    if (warp == 0 && r < rows) {
      MergeSum s;
      s.m = -INFINITY;
#pragma unroll
      for (int w = 0; w < 8; ++w) s.m = fmaxf(s.m, part[w][lane].m);
      s.l = 0.f;
      s.acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 8; ++w) merge_add(s, part[w][lane].m, part[w][lane].l, part[w][lane].acc, s.m);
      finish(s, r, quad);
    }
  } else {
    constexpr int RPC = kMergeThreads / (D / 4);             // rows at once
    const int quad = warp % QG * 4 + lane / 8;
    for (int r0 = blockIdx.y * RPC; r0 < rows; r0 += gridDim.y * RPC) {
      const int r = r0 + warp / QG * 8 + lane % 8;
      if (r < rows) finish(merge_parts(a, c, it.go_on, D, r, quad, 0, 1), r, quad);
    }
  }
}

}  // namespace mcs
