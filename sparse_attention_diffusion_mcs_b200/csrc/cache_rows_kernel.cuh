// cache_rows_kernel.cuh -- attention of few query rows over the 8-bit cache
// (single tokens, short drafts): bound by reading the cache once.
//
// For row i and token j of the page with scales ks, vs (base-2 units):
//   x_ij = scale log2(e) (q_i . k8_j) ks,     y_ij = x_ij + log2(vs),
//   O_i  = sum_j 2^(y_ij - m_i) v8_j  /  sum_j 2^(y_ij - m_i) / vs,
// m_i the running maximum of y.  2^y = 2^x vs is the weight that v8 itself
// gets, so the held numbers enter the products as they are (e4m3 is exact in
// fp16), every weight is <= 1 whatever the pages' scales, and no page is
// dequantised.  m, the sums and O are fp32; the weights, times 2^14, are
// rounded to fp16 (2^-11 relative; below 2^-28 of the row's largest weight, an
// absolute 2^-39 of it), because the products take 16-bit numbers: a second part of
// each weight would be half as many products again, for an eighth of what the
// output's own rounding to bf16 may be off by.  Against 64 bits outputs are off by
// 1.6e-3 of their norm, as ones computed in 32 bits are.  The sum that they are
// divided by takes the weights before they are rounded.
// Queries are held as fp16 of q 2^-e, 2^e the power of two at the row's
// largest magnitude: exact for bf16 numbers down to 2^-17 of it, and off by
// 2^-25 of it below.
//
// A CTA takes 16 rows -- all query heads that share a key head, times their
// tokens -- and runs of 128-key tiles, dealt in one of two ways.  Little work:
// a cluster of CTAs takes one item (cache_sched.cuh), each its share of the
// tiles, and merges (m, l, O) through distributed shared memory, in one launch.
// Much work: the CTAs that fill the SMs once take equal runs of all items'
// tiles, and a second launch merges what was split; sequences of any lengths
// then keep every SM reading to the end.  Either way the merge order is fixed,
// so results repeat bit for bit.
// Products by mma.sync m16n8k16: one row tile of 16 is all there is, while a
// tcgen05 product has at least 64 rows, needs its operands in 16 bits in
// shared memory (an extra write and read of every number), and 16 rows
// keep the tensor work far below the time of the bytes.
//
// Warps 0-3 each take 32 keys of every tile with their own online softmax
// (no barrier between them until the end); warp 4 loads: one TMA box per page,
// keys and values, into a ring of stages.  The swizzle of the boxes and the
// order in which keys are dealt to the product's columns keep every shared
// memory read free of bank conflicts (key_of below).
//
// Measured: one token of eight sequences of 73728 to 131072 tokens, 32 query heads
// on 8 of 128: 270 us, 6.2 TB/s (95 % of the measured copy), and 5 us of merge; as a
// call among others 297 to 315 us.  5 tokens of 4 sequences of 5120 to 8191, 16 heads on 4
// of 64: 15.0 us, bound by the 0.9 us that a warp takes for its 32 keys of a tile.
// 168 registers, what two CTAs an SM leave; of the four variants the dealt one for
// d = 128 spills (88 bytes written, 68 read a thread).
#pragma once

#include "cache_sched.cuh"

namespace mcs {

struct CacheAttnArgs {
  CUtensorMap tmK, tmV;          // [n_pages * H * page, d] bytes, box min(page, 128) rows
  CacheView c;
  const bf16 *Q;                 // [B, Hq, Nq, d]
  bf16 *O;                       // [B, Hq, Nq, d]
  float *lse;                    // [B, Hq, Nq] or null: log of the sum of exp (natural units)
  SchedArgs s;
  MergeSpace m;                  // (not used by clusters)
  float scale_log2;
  unsigned *status;
  unsigned long long wait_ns;
};

template <int D>
struct RowsCfg {
  static constexpr int BN = 128;                       // keys per tile
  static constexpr int TILE = BN * D;                  // bytes of a K or V tile
  static constexpr int NS = (D == 128 ? 3 : 6);
  static constexpr int OFF_KV = 0;
  static constexpr int OFF_SC = OFF_KV + NS * 2 * TILE;   // per stage: 8 x float4 (ks, log2 vs, 1 / vs, -)
  static constexpr int OFF_BAR = OFF_SC + NS * 8 * 16;
  static constexpr int OFF_MISC = OFF_BAR + 16 * NS;
  static constexpr int OFF_ML = OFF_MISC + 16;            // merged (reference, l) of 16 rows
  static constexpr int OFF_WML = OFF_ML + 16 * 8;    // per warp (reference, l)
  // the warps' O on its way into the CTA's, 32 numbers of a row at a time
  static constexpr int OLD = 32 + 4;
  static constexpr int OFF_WO = OFF_WML + 4 * 16 * 8;
  static constexpr int SMEM = OFF_WO + 4 * 16 * OLD * 4 + 1024;
  // clusters, after their only run of tiles, over the ring: the CTA's O
  static constexpr int OFF_O = 0;
  static_assert(OFF_WML % 16 == 0 && OFF_WO % 16 == 0, "16-byte aligned");
  static_assert(16 * D * 4 <= OFF_SC, "a cluster's O fits the ring");
  static constexpr int THREADS = 5 * 32;
};

// The key (of eight) in column `col` of a score tile.  A quarter warp reads the
// 16-byte chunks t = 0..3 of the keys of two neighbouring columns (scores), or
// chunks g, g + 1 of the keys of columns u, 2 + u, 4 + u, 6 + u (P.V): the order
// sends each of these to different banks under the boxes' swizzle.
// d = 128 (128B): 0 5 2 7 4 1 6 3; d = 64 (64B): 0 3 1 2 4 7 5 6.
template <int D>
__device__ __forceinline__ int key_of(int col) {
  if (D == 128) return col & 1 ? col ^ 4 : col;
  const int base = (col >> 2) * 4 + ((col >> 1) & 1);
  return col & 1 ? base ^ 3 : base;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 ld_dsmem2(uint32_t addr, uint32_t rank) {
  uint32_t r;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_dsmem4(uint32_t addr, uint32_t rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(r)
               : "memory");
  return v;
}
// a barrier of warps 0-3 that tells whether all of them are well
__device__ __forceinline__ bool group_ok(bool ok) {
  uint32_t bad;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(bad)
      : "r"(ok ? 0u : 1u)
      : "memory");
  return bad == 0;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// weights are held times 2^kRowsBias in fp16
constexpr float kRowsBias = 14.f;
constexpr int kMaxRanks = 8;     // CTAs of a cluster, at most

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(RowsCfg<D>::THREADS, 2)
    cache_rows_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = RowsCfg<D>;
  using S = Sched<16, false>;
  constexpr int NS = C::NS, BN = C::BN, SEG = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto b_full = [&](int s) { return bar0 + 8 * s; };
  auto b_empty = [&](int s) { return bar0 + 8 * (NS + s); };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC);

  const CacheView &cv = a.c;
  const SchedArgs &sa = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, ranks = gridDim.x;        // CLUSTER: it spans the x dimension
  const int share = sa.share;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), 4);
    }
    *abort_flag = 0;
    mbar_init_fence();
  }
  // every warp goes through the same parts
  S run;
  if constexpr (CLUSTER) {
    run.b = blockIdx.y / sa.H;
    run.h = blockIdx.y - run.b * sa.H;
    run.block = blockIdx.z;
    run.left = 1;
    if (tid == 0 && sa.lengths[run.b] > sa.cap) record_status(a.status, kStatusBadMeta);
  } else {
    run.start(sa, rank, ranks, 4, lane, a.status);
    if (tid == 0) a.m.items[rank].go_on = 0;
  }
  auto next = [&](Segment &g) -> bool {
    if constexpr (CLUSTER) {
      if (!run.left) return false;
      run.left = 0;
      g.b = run.b;
      g.h = run.h;
      g.block = run.block;
      S::item(sa, g.b, g.block, g);
      const int tiles = (g.kmax + BN - 1) / BN;
      g.t0 = static_cast<int>(static_cast<long long>(tiles) * rank / ranks);
      g.t1 = static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / ranks);
      return true;
    } else {
      if (!run.next(sa, g)) return false;
      g.t1 = min(g.t1, (g.kmax + BN - 1) / BN);          // an item without keys has no tile to read
      return true;
    }
  };
  __syncthreads();

  Segment sg;
  if (warp == 4) {
    // ------------------------------------------------------------------ loads
    // lane l holds page and scales of the 16-key group 32 bt + l of batch bt
    // (four tiles); the next batch's are on the way meanwhile
    if (lane == 0) {
      tma_prefetch_desc(&a.tmK);
      tma_prefetch_desc(&a.tmV);
    }
    bool ok = true;
    int it = 0;                                      // tiles so far, over all parts
    while (ok && next(sg)) {
      const int32_t *table = cv.table + static_cast<long long>(sg.b) * cv.max_pages;
      const int groups = (sg.kmax + 15) / 16;
      auto fetch_page = [&](int g) {
        int p = -1;
        if (g < groups) {
          p = table[g * 16 / cv.page];
          if (p < 0 || p >= cv.n_pages) {
            record_status(a.status, kStatusBadMeta);
            p = -1;
          }
        }
        return p;
      };
      int pid = fetch_page(8 * sg.t0 + lane);
      float ks = 0.f, vs = 0.f;
      auto fetch_scales = [&](int p, float &k, float &v) {
        k = v = 0.f;
        if (p >= 0) {
          k = cv.k_scale[static_cast<size_t>(p) * cv.H + sg.h];
          v = cv.v_scale[static_cast<size_t>(p) * cv.H + sg.h];
        }
      };
      fetch_scales(pid, ks, vs);
      auto check_scales = [&]() {
        if (pid >= 0 && !scales_fit(ks, vs)) {
          record_status(a.status, kStatusBadMeta);
          pid = -1;
        }
      };
      check_scales();
      const int gpb = cv.page / 16;                    // groups per page (a page is at most a tile)
      for (int tb = sg.t0; tb < sg.t1 && ok; tb += 4) {
        const int npid = fetch_page(8 * (tb + 4) + lane);
        float nks, nvs;
        fetch_scales(npid, nks, nvs);
        for (int t = tb; t < min(tb + 4, sg.t1); ++t, ++it) {
          const int s = it % NS;
          const int gl = 8 * (t - tb);                 // lane of the tile's first group
          ok = mbar_wait_warp(b_empty(s), ((it / NS) & 1) ^ 1, a.wait_ns, abort_flag);
          if (!ok) break;
          if (lane >= gl && lane < gl + 8)
            *reinterpret_cast<float4 *>(smem + C::OFF_SC + (s * 8 + lane - gl) * 16) = page_factors(pid >= 0, ks, vs, 0.f);
          // the first lane of each page's groups loads it
          const bool mine = lane >= gl && lane < gl + 8 && (lane - gl) % gpb == 0 && pid >= 0;
          const unsigned who = __ballot_sync(0xffffffffu, mine);
          const uint32_t page_bytes = static_cast<uint32_t>(cv.page) * D;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(b_full(s), __popc(who) * 2 * page_bytes);
          __syncwarp();
          if (mine) {
            const uint32_t dst = sbase + C::OFF_KV + s * 2 * C::TILE + (lane - gl) * 16 * D;
            const int r = static_cast<int>((static_cast<long long>(pid) * cv.H + sg.h) * cv.page);
            tma_load_2d(dst, &a.tmK, 0, r, b_full(s));
            tma_load_2d(dst + C::TILE, &a.tmV, 0, r, b_full(s));
          }
          __syncwarp();
        }
        pid = npid;
        ks = nks;
        vs = nvs;
        check_scales();
      }
    }
    if (!ok && lane == 0 && !*abort_flag) {
      *abort_flag = 1;
      record_status(a.status, kStatusTimeout);
    }
    // never leave the CTA with a copy still landing in its shared memory
    volatile int never = 0;
    for (int i = (it > NS ? it - NS : 0); i < it; ++i)
      mbar_wait(b_full(i % NS), (i / NS) & 1, 2000000000ull, &never);
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ products and softmax
    const int g = lane >> 2, t = lane & 3;
    bool ok = true;
    int it = 0;
    // the four warps have barriers between them: all go on to a part, or none
    auto more = [&]() -> bool { return CLUSTER ? run.left : run.more(sa); };
    while (group_ok(ok && more()) && next(sg)) {
    const int row0 = sg.block * 16;                 // rows are (token, query head of the group)
    const int kmax = sg.kmax;
    // keys that row i of the item sees: [0, limit)
    auto limit_of = [&](int row) {
      const int i = row / share;
      if (row >= sa.n_rows || i >= sg.nq) return 0;
      return sa.causal ? max(sg.len - sg.nq + i + 1, 0) : sg.len;
    };
    const int last_row = min(row0 + 16, sa.n_rows) - 1;
    uint32_t qa[SEG][4][4];
    float rowf[2];
    int lim[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = row0 + u * 8 + g;
      lim[u] = limit_of(row);
      uint4 w[SEG][2];
#pragma unroll
      for (int sgm = 0; sgm < SEG; ++sgm) w[sgm][0] = w[sgm][1] = make_uint4(0, 0, 0, 0);
      if (row < sa.n_rows) {
        const int i = row / share, hq = sg.h * share + row % share;
        const uint4 *q = reinterpret_cast<const uint4 *>(
            a.Q + ((static_cast<size_t>(sg.b) * sa.H * share + hq) * sa.Nq + i) * D);
#pragma unroll
        for (int sgm = 0; sgm < SEG; ++sgm) {
          w[sgm][0] = q[sgm * 8 + 2 * t];
          w[sgm][1] = q[sgm * 8 + 2 * t + 1];
        }
      }
      // the row's largest magnitude, as bf16 bits
      uint32_t am = 0;
      const uint32_t *x = reinterpret_cast<const uint32_t *>(w);
#pragma unroll
      for (int i = 0; i < SEG * 8; ++i) am = max(am, max((x[i] << 1) & 0xFFFEu, (x[i] >> 15) & 0xFFFEu));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int e = min(max(static_cast<int>(am >> 8) - 127, -100), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      rowf[u] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      if (am >> 8 == 255) rowf[u] = __uint_as_float(0x7FC00000u);   // a query that is not finite: NaN
#pragma unroll
      for (int sgm = 0; sgm < SEG; ++sgm) {
        const uint32_t *y = reinterpret_cast<const uint32_t *>(w[sgm]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t z = y[2 * j + p];
            qa[sgm][j][u + 2 * p] =
                half2_bits(__uint_as_float(z << 16) * down, __uint_as_float(z & 0xFFFF0000u) * down);
          }
      }
    }
    // keys every row of the CTA sees: no row of a block sees fewer than its first (queries behind nq: none)
    const int all = min(limit_of(row0), limit_of(last_row));

    constexpr int NT = D / 8;          // column tiles of O
    float o[NT][4];
    float m[2], l[2];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    for (int tt = sg.t0; tt < sg.t1; ++tt, ++it) {
      const int s = it % NS;
      if (!mbar_wait_warp(b_full(s), (it / NS) & 1, a.wait_ns, abort_flag)) {
        ok = false;
        if (lane == 0 && !*abort_flag) {     // the others then give up too, before the barriers below
          *abort_flag = 1;
          record_status(a.status, kStatusTimeout);
        }
        break;
      }
      const int key0 = tt * BN + warp * 32;
      if (key0 < kmax) {
        const uint8_t *kb = smem + C::OFF_KV + s * 2 * C::TILE + warp * 32 * D;
        const uint8_t *vb = kb + C::TILE;
        const float4 *scp = reinterpret_cast<const float4 *>(smem + C::OFF_SC) + s * 8 + warp * 2;
        const float4 sc0 = scp[0], sc1 = scp[1];
        const bool clean = key0 + 32 <= all && sc0.y > kHasValues && sc1.y > kHasValues;
        // ---- scores of 32 keys
        float sc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
          const int r = 8 * i + key_of<D>(g);
#pragma unroll
          for (int sgm = 0; sgm < SEG; ++sgm) {
            const int chunk = D == 128 ? ((4 * sgm + t) ^ (r & 7)) : (t ^ ((r >> 1) & 3));
            const uint4 w = *reinterpret_cast<const uint4 *>(kb + r * D + chunk * 16);
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b0 = half2_of_e4m3x2(x[j]), b1 = half2_of_e4m3x2_hi(x[j]);
              mma_f16(sc[i], qa[sgm][j][0], qa[sgm][j][1], qa[sgm][j][2], qa[sgm][j][3], b0, b1);
            }
          }
        }
        // ---- online softmax; column 2t + u of group i is key key0 + 8 i + key_of(2t + u)
        uint32_t pa[4][2];
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 f = i < 2 ? sc0 : sc1;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y = fmaf(sc[i][e], rowf[e >> 1] * f.x, f.y);
            if (!clean) {
              const int key = key0 + 8 * i + key_of<D>(2 * t + (e & 1));
              y = key < lim[e >> 1] && f.y > -INFINITY ? y : -INFINITY;
            }
            sc[i][e] = y;
            mx[e >> 1] = fmaxf(mx[e >> 1], y);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
          float al[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float nm = fmaxf(m[u], mx[u]);
            al[u] = nm == m[u] ? 1.f : ex2_approx(m[u] - nm);
            m[u] = nm;
            l[u] *= al[u];
          }
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            o[c][0] *= al[0];
            o[c][1] *= al[0];
            o[c][2] *= al[1];
            o[c][3] *= al[1];
          }
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0] - kRowsBias,
                             m[1] == -INFINITY ? 0.f : m[1] - kRowsBias};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float inv = i < 2 ? sc0.z : sc1.z;
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = ex2_approx(sc[i][e] - mu[e >> 1]);
          l[0] = fmaf(p[0] + p[1], inv, l[0]);
          l[1] = fmaf(p[2] + p[3], inv, l[1]);
          pa[i][0] = half2_bits(p[0], p[1]);
          pa[i][1] = half2_bits(p[2], p[3]);
        }
        // ---- P.V; column g of tile c is number (D / 8) g + c
#pragma unroll
        for (int ii = 0; ii < 2; ++ii) {
          uint4 w[4];   // D / 8 bytes of the keys of columns 2t, 2t + 1, of groups 2 ii and 2 ii + 1
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * ii + 8 * (q >> 1) + key_of<D>(2 * t + (q & 1));
            if (D == 128) {
              w[q] = *reinterpret_cast<const uint4 *>(vb + r * D + ((g ^ (r & 7)) * 16));
            } else {
              const uint2 z = *reinterpret_cast<const uint2 *>(vb + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16) + (g & 1) * 8);
              w[q] = make_uint4(z.x, z.y, 0, 0);
            }
            // what lies behind the last token, or was never loaded, or has a scale of 0, may be any bits
            const float lv = ii ? sc1.y : sc0.y;
            if (!clean && !(key0 + r < kmax && lv > kHasValues)) w[q] = make_uint4(0, 0, 0, 0);
          }
          const uint32_t x0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, x1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
          const uint32_t x2[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, x3[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
          for (int q = 0; q < NT / 4; ++q) {
            const uint32_t lo0 = __byte_perm(x0[q], x1[q], 0x5140), lo1 = __byte_perm(x0[q], x1[q], 0x7362);
            const uint32_t hi0 = __byte_perm(x2[q], x3[q], 0x5140), hi1 = __byte_perm(x2[q], x3[q], 0x7362);
            const uint32_t b0[4] = {half2_of_e4m3x2(lo0), half2_of_e4m3x2_hi(lo0), half2_of_e4m3x2(lo1), half2_of_e4m3x2_hi(lo1)};
            const uint32_t b1[4] = {half2_of_e4m3x2(hi0), half2_of_e4m3x2_hi(hi0), half2_of_e4m3x2(hi1), half2_of_e4m3x2_hi(hi1)};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mma_f16(o[4 * q + c], pa[2 * ii][0], pa[2 * ii][1], pa[2 * ii + 1][0], pa[2 * ii + 1][1], b0[c], b1[c]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty(s));
    }
    // ---- the four warps' parts into the CTA's, 32 numbers of every row at a time:
    // thread t holds numbers (D / 8)(2t + e) + c of rows g and 8 + g
    float2 *wml = reinterpret_cast<float2 *>(smem + C::OFF_WML);
    float *wo = reinterpret_cast<float *>(smem + C::OFF_WO);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // sums of products stay below 2^17 and scales are at most 2^90: from 2^20 on scores
      // may leave fp32.  Above it they make NaN; a row with keys and all its scores below is NaN too.
      const bool lost = rowf[u] >= 0x1p20f && m[u] == -INFINITY && sg.t0 < sg.t1 && lim[u] > sg.t0 * BN + warp * 32;
      float s = lost ? NAN : l[u];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if (t == 0)
        wml[warp * 16 + u * 8 + g] =
            make_float2(m[u] == -INFINITY ? -INFINITY : m[u] - kRowsBias, s);
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    // this thread merges 4 numbers of row r
    float2 ml;
    float f[4];
    const int r = tid / 8;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, wml[w * 16 + r].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 p = wml[w * 16 + r];
      f[w] = merge_factor(p.x, p.y, mm);
      ll = fmaf(p.y, f[w], ll);
    }
    ml = make_float2(mm, ll);
    const size_t slot = CLUSTER ? 0 : (2 * static_cast<size_t>(rank) + (sg.first ? 1 : 0)) * 16;
    if constexpr (!CLUSTER) {
      if (tid == 0 && sg.first && !sg.whole && ok) {
        MergeItem mi;
        mi.b = sg.b;
        mi.h = sg.h;
        mi.block = sg.block;
        mi.go_on = sg.go_on;
        a.m.items[rank] = mi;
      }
    }
    float2 *cml = reinterpret_cast<float2 *>(smem + C::OFF_ML);
    float *oc = reinterpret_cast<float *>(smem + C::OFF_O);
    if (tid % 8 == 0) {
      if constexpr (CLUSTER) cml[r] = ml;
      else if (!sg.whole) a.m.ml[slot + r] = ml;
    }
#pragma unroll
    for (int q = 0; q < NT / 4; ++q) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4 *>(wo + (warp * 16 + u * 8 + g) * C::OLD + 4 * (2 * t + e)) =
              make_float4(o[4 * q][2 * u + e], o[4 * q + 1][2 * u + e], o[4 * q + 2][2 * u + e],
                          o[4 * q + 3][2 * u + e]);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const int te = tid % 8, col = NT * te + 4 * q;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 x = *reinterpret_cast<const float4 *>(wo + (w * 16 + r) * C::OLD + 4 * te);
        const float y = f[w];
        acc = make_float4(fmaf(x.x, y, acc.x), fmaf(x.y, y, acc.y), fmaf(x.z, y, acc.z), fmaf(x.w, y, acc.w));
      }
      if constexpr (CLUSTER) {
        *reinterpret_cast<float4 *>(oc + r * D + col) = acc;
      } else if (!sg.whole) {
        *merge_part(a.m, slot, 16, D, r, col / 4) = acc;
      } else if (row0 + r < sa.n_rows && ok) {
        const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;      // a row that sees nothing is 0
        const int row = row0 + r, i = row / share, hq = sg.h * share + row % share;
        const size_t at = (static_cast<size_t>(sg.b) * sa.H * share + hq) * sa.Nq + i;
        *reinterpret_cast<uint2 *>(a.O + at * D + col) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        // l is in units of 2^reference: the sum of exp(score) is l 2^reference
        if (a.lse && te == 0 && q == 0)
          a.lse[at] = ml.y == 0.f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.6931471805599453f;
      }
      if (q + 1 < NT / 4) asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    }   // parts
  }
  // ---------------------------------------------------------------------- merge over the cluster
  if constexpr (CLUSTER) {
    if (ranks > 1)
      cluster_sync();
    else
      __syncthreads();
    if (!*abort_flag) {
      const int row0 = run.block * 16;
      const int rows_here = min(16, sa.n_rows - row0);
      for (int idx = rank * C::THREADS + tid; idx < rows_here * (D / 4); idx += ranks * C::THREADS) {
        const int r = idx / (D / 4), c = (idx - r * (D / 4)) * 4;
        // all ranks' reads on the way at once: one after the other they took 3 to 5 us
        float2 p[kMaxRanks];
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) p[k] = ld_dsmem2(sbase + C::OFF_ML + r * 8, min(k, ranks - 1));
        float4 x[kMaxRanks];
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) x[k] = ld_dsmem4(sbase + C::OFF_O + (r * D + c) * 4, min(k, ranks - 1));
        float mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) mm = fmaxf(mm, p[k].x);
        float ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxRanks; ++k) {
          const float f = k < ranks ? merge_factor(p[k].x, p[k].y, mm) : 0.f;
          if (f != 0.f) {                                // (NaN counts)
            ll = fmaf(p[k].y, f, ll);
            acc = make_float4(fmaf(x[k].x, f, acc.x), fmaf(x[k].y, f, acc.y), fmaf(x[k].z, f, acc.z), fmaf(x[k].w, f, acc.w));
          }
        }
        const float inv = ll == 0.f ? 0.f : 1.f / ll;      // a row that sees nothing is 0
        const int row = row0 + r, i = row / share, hq = run.h * share + row % share;
        const size_t at = (static_cast<size_t>(run.b) * sa.H * share + hq) * sa.Nq + i;
        *reinterpret_cast<uint2 *>(a.O + at * D + c) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (c == 0 && a.lse) a.lse[at] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
      }
    }
    if (ranks > 1) cluster_sync();   // no CTA leaves while another reads it
  }
}

}  // namespace mcs
