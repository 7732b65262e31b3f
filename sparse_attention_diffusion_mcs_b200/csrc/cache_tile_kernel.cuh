// cache_tile_kernel.cuh -- attention of many query rows over the 8-bit cache
// (chunks of tokens, whole frames): bound by the tensor cores and by the
// exponentials.
//
// The mathematics is cache_rows_kernel.cuh's: x_ij = scale log2(e) (q_i . k8_j) ks,
// y_ij = x_ij + log2(vs), O_i = sum_j 2^(y_ij - m) v8_j / sum_j 2^(y_ij - m) / vs.
//
// Q.K^T runs in 8 bits straight from the cache's bytes.  A bf16 number has 8
// significant bits, an e4m3 number 4: with its row scaled so that the largest
// magnitude lies in [2^7, 2^8), q is hi + lo with hi = e4m3(q), lo = e4m3(q - hi),
// exact down to 2^-10 of the row's largest and off by at most 2^-18 of it below.
// Two 8-bit products (hi, then lo) cost what one 16-bit product costs, and no
// key is converted.
// P.V runs in fp16: the weights need more than e4m3's 4 bits, and a weight
// whose 8-bit parts underflow would lose the tail of a long row.  Two warps
// turn each 128-key tile of V into fp16 once (exact) for all 256 query rows.
// Weights are 2^(y - m + 6) with m at most 2^8 behind the row's maximum: at
// most 2^14, rounded to fp16 by 2^-11 relative, normal down to 2^-20 of the
// reference's.  Sums, m and O are fp32.
//
// A CTA takes 256 query rows (two halves of 128, one TMEM lane a row) and runs
// of 128-key tiles, dealt as cache_sched.cuh describes:
//   warps 0-3, 4-7  softmax and epilogue of half 0, half 1
//   warp  8         TMEM allocation, the single MMA-issuing thread
//   warp  9         loads: one TMA box per page, keys and values; the scales
//   warps 10, 11    V from e4m3 to fp16
// The tensor pipe runs per tile j: PV0(j) QK0(j+1) PV1(j) QK1(j+1), so each
// half's softmax has the other half's two products to work in.  P (fp16 pairs)
// lies over the upper half of its own S.  TMEM: S0, S1 (128 columns each),
// O0, O1 (D columns each).  Every wait is bounded.
#pragma once

#include "cache_rows_kernel.cuh"

namespace mcs {

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptors: e4m3 (kind::f8f6f4) and fp16 (kind::f16), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// K-major rows of ROW bytes (64 or 128), swizzled by their width.
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr) {
  if (ROW == 128) return sdesc_sw128(saddr, 16, 1024);
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>(512 >> 4) << 32;   // 8 rows of 64 bytes
  d |= static_cast<uint64_t>(1u) << 46;         // descriptor version (sm_100)
  d |= static_cast<uint64_t>(4u) << 61;         // swizzle: 64B
  return d;
}
// byte offset of 16-byte chunk `chunk` of row `row`
template <int ROW>
__device__ __forceinline__ int swizzled(int row, int chunk) {
  return row * ROW + ((ROW == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

// maxima that keep NaN
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D>
struct TileCfg {
  static constexpr int BM = 128, ROWS = 256, BN = kKeyTile;
  static constexpr int NK = D == 128 ? 3 : 4;     // K ring
  static constexpr int NV = D == 128 ? 2 : 4;     // V ring, e4m3
  static constexpr int NH = 2;                    // V ring, fp16
  static constexpr int NSC = 8;                   // scales' ring (see the loads)
  static constexpr int Q_BYTES = BM * D;          // one half's hi or lo part
  static constexpr int T8 = BN * D, T16 = BN * D * 2;
  static constexpr int OFF_Q = 0;                 // hi, lo of half 0; hi, lo of half 1
  static constexpr int OFF_K = OFF_Q + 4 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * T8;
  static constexpr int OFF_H = OFF_V + NV * T8;
  static constexpr int OFF_SC = OFF_H + NH * T16;             // per tile: 8 x float4 (ks, log2 vs, 1 / vs, whole tile)
  static constexpr int OFF_BAR = OFF_SC + NSC * 8 * 16;
  static constexpr int N_BAR = 2 * NK + 2 * NV + 2 * NH + NSC + 8 + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int MMA_WARP = 8, LOAD_WARP = 9, CVT_WARP = 10, CVT_THREADS = 64;
  static constexpr int THREADS = 12 * 32;
  static constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_O = 256;   // half h: S at 128 h, O at 256 + D h
  static constexpr uint32_t COL_P = 64;           // of S
  static constexpr float kBias = 6.f, kRaise = 8.f;
  static_assert(SMEM <= 232448, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::THREADS, 1) cache_tile_kernel(const __grid_constant__ CacheAttnArgs a) {
  using C = TileCfg<D>;
  using S = Sched<C::ROWS, true>;
  constexpr int NK = C::NK, NV = C::NV, NH = C::NH, NSC = C::NSC, BN = C::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto b_kfull = [&](int i) { return bar0 + 8 * (i % NK); };
  auto b_kempty = [&](int i) { return bar0 + 8 * (NK + i % NK); };
  auto b_vfull = [&](int i) { return bar0 + 8 * (2 * NK + i % NV); };
  auto b_vempty = [&](int i) { return bar0 + 8 * (2 * NK + NV + i % NV); };
  auto b_hfull = [&](int i) { return bar0 + 8 * (2 * NK + 2 * NV + i % NH); };
  auto b_hempty = [&](int i) { return bar0 + 8 * (2 * NK + 2 * NV + NH + i % NH); };
  const uint32_t bx = bar0 + 8 * (2 * NK + 2 * NV + 2 * NH);
  auto b_sc = [&](int i) { return bx + 8 * (i % NSC); };
  const uint32_t by = bx + 8 * NSC;
  // one of each per half: a half's softmax and the MMA thread wait for each other at every tile, so none runs ahead
  auto b_q = [&](int h) { return by + 8 * h; };
  auto b_s = [&](int h) { return by + 16 + 8 * h; };
  auto b_p = [&](int h) { return by + 32 + 8 * h; };
  auto b_o = [&](int h) { return by + 48 + 8 * h; };
  const uint32_t b_drain = by + 64;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

  const CacheView &cv = a.c;
  const SchedArgs &sa = a.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(b_kfull(i), 1);
      mbar_init(b_kempty(i), 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(b_vfull(i), 1);
      mbar_init(b_vempty(i), C::CVT_THREADS);
    }
    for (int i = 0; i < NH; ++i) {
      mbar_init(b_hfull(i), C::CVT_THREADS);
      mbar_init(b_hempty(i), 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(b_sc(i), 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(b_q(h), 128);
      mbar_init(b_s(h), 1);
      mbar_init(b_p(h), 128);
      mbar_init(b_o(h), 1);
    }
    mbar_init(b_drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
    a.m.items[cta].go_on = 0;
  }
  if (warp == C::MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  S run;                                           // every warp goes through the same parts
  run.start(sa, cta, gridDim.x, 4, lane, a.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  Segment sg = {};
  // the part's key tiles to read: [t0, end)
  auto end_of = [&]() { return min(sg.t1, (sg.kmax + BN - 1) / BN); };
  auto give_up = [&]() {
    if (!*abort_flag) {
      *abort_flag = 1;
      record_status(a.status, kStatusTimeout);
    }
  };

  if (warp == C::LOAD_WARP) {
    // ------------------------------------------------------------------ loads
    // lane l holds page and scales of the 16-key group 32 bt + l of batch bt
    // (four tiles); the next batch's are on the way meanwhile.  The scales have
    // a ring of their own, read until P of their tile is published: slot i is
    // written again for tile i + NSC, after K's slot of tile i + NSC - NK is
    // free, when P of the tile before that one was.
    static_assert(NSC > NK, "scales outlive their readers");
    if (lane == 0) {
      tma_prefetch_desc(&a.tmK);
      tma_prefetch_desc(&a.tmV);
    }
    bool ok = true;
    int it = 0, ik = 0, iv = 0;                      // tiles so far, over all parts; loads issued
    const int gpb = cv.page / 16;                    // groups per page (a page is at most a tile)
    const uint32_t page_bytes = static_cast<uint32_t>(cv.page) * D;
    while (ok && run.next(sa, sg)) {
      const int end = end_of();
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
      auto fetch_scales = [&](int p, float &k, float &v) {
        k = v = 0.f;
        if (p >= 0) {
          k = cv.k_scale[static_cast<size_t>(p) * cv.H + sg.h];
          v = cv.v_scale[static_cast<size_t>(p) * cv.H + sg.h];
        }
      };
      int pid = fetch_page(8 * sg.t0 + lane);
      float ks, vs;
      fetch_scales(pid, ks, vs);
      for (int tb = sg.t0; tb < end && ok; tb += 4) {
        const int npid = fetch_page(8 * (tb + 4) + lane);
        float nks, nvs;
        fetch_scales(npid, nks, nvs);
        for (int t = tb; t < min(tb + 4, end); ++t, ++it) {
          const int gl = 8 * (t - tb);                 // lane of the tile's first group
          const bool in = lane >= gl && lane < gl + 8;
          const unsigned good = __ballot_sync(0xffffffffu, in && pid >= 0);
          // the first lane of each page's groups loads it
          const bool mine = in && (lane - gl) % gpb == 0 && pid >= 0;
          const uint32_t tx = __popc(__ballot_sync(0xffffffffu, mine)) * page_bytes;
          const int r = mine ? static_cast<int>((static_cast<long long>(pid) * cv.H + sg.h) * cv.page) : 0;
          const uint32_t at = (lane - gl) * 16 * D;
          ok = mbar_wait_warp(b_kempty(it), ((it / NK) & 1) ^ 1, a.wait_ns, abort_flag);
          if (!ok) break;
          if (in)
            *reinterpret_cast<float4 *>(smem + C::OFF_SC + ((it % NSC) * 8 + lane - gl) * 16) =
                make_float4(ks, pid >= 0 ? __log2f(vs) : -INFINITY, pid >= 0 ? 1.f / vs : 0.f,
                            __popc(good) == 8 ? 1.f : 0.f);
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(b_sc(it));
            mbar_arrive_expect_tx(b_kfull(it), tx);
          }
          __syncwarp();
          if (mine) tma_load_2d(sbase + C::OFF_K + (it % NK) * C::T8 + at, &a.tmK, 0, r, b_kfull(it));
          ++ik;
          ok = mbar_wait_warp(b_vempty(it), ((it / NV) & 1) ^ 1, a.wait_ns, abort_flag);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(b_vfull(it), tx);
          __syncwarp();
          if (mine) tma_load_2d(sbase + C::OFF_V + (it % NV) * C::T8 + at, &a.tmV, 0, r, b_vfull(it));
          ++iv;
          __syncwarp();
        }
        pid = npid;
        ks = nks;
        vs = nvs;
      }
    }
    if (!ok && lane == 0) give_up();
    // never leave the CTA with a copy still landing in its shared memory
    volatile int never = 0;
    for (int i = (ik > NK ? ik - NK : 0); i < ik; ++i) mbar_wait(b_kfull(i), (i / NK) & 1, 2000000000ull, &never);
    for (int i = (iv > NV ? iv - NV : 0); i < iv; ++i) mbar_wait(b_vfull(i), (i / NV) & 1, 2000000000ull, &never);
    __syncwarp();
  } else if (warp >= C::CVT_WARP) {
    // ------------------------------------------------------------------ V to fp16
    // A thread takes 16 numbers of a key at a time: one 16-byte read, two 16-byte
    // writes.  Eight neighbouring threads take four chunks of keys r and r ^ 5,
    // which the swizzles of both layouts send to different banks.
    constexpr int CH = D / 16, PER = BN * CH / C::CVT_THREADS;
    const int ct = tid - C::CVT_WARP * 32;
    bool ok = true;
    int it = 0;
    while (ok && run.next(sa, sg)) {
      const int end = end_of();
      for (int t = sg.t0; t < end; ++t, ++it) {
        ok = mbar_wait_warp(b_vfull(it), (it / NV) & 1, a.wait_ns, abort_flag) &&
             mbar_wait_warp(b_hempty(it), ((it / NH) & 1) ^ 1, a.wait_ns, abort_flag);
        if (!ok) break;
        const uint8_t *src = smem + C::OFF_V + (it % NV) * C::T8;
        uint8_t *dst = smem + C::OFF_H + (it % NH) * C::T16;
        const float4 *sc = reinterpret_cast<const float4 *>(smem + C::OFF_SC) + (it % NSC) * 8;
        const bool whole = sc[0].w != 0.f && (t + 1) * BN <= sg.kmax;
#pragma unroll 4
        for (int i = 0; i < PER; ++i) {
          const int id = ct + i * C::CVT_THREADS;            // (pair of keys, 4 chunks, key of the pair, chunk)
          const int c4 = id & 3, second = (id >> 2) & 1, rest = id >> 3;
          const int q4 = rest % (CH / 4), pair = rest / (CH / 4);
          // pairs (r, r ^ 5) of 8 keys: r = 0, 1, 2, 3 (bit 2 clear)
          const int r0 = (pair >> 2) * 8 + (pair & 3), r = second ? r0 ^ 5 : r0, c = q4 * 4 + c4;
          uint4 w = *reinterpret_cast<const uint4 *>(src + swizzled<D>(r, c));
          // what lies behind the last key that is seen, or was never loaded, may be any bits
          if (!whole && !(t * BN + r < sg.kmax && sc[r >> 4].y > -INFINITY)) w = make_uint4(0, 0, 0, 0);
          // 64-number blocks of 128-byte rows
          uint8_t *o = dst + (c >> 2) * (BN * 128);
          *reinterpret_cast<uint4 *>(o + swizzled<128>(r, 2 * (c & 3))) =
              make_uint4(half2_of_e4m3x2(w.x), half2_of_e4m3x2_hi(w.x), half2_of_e4m3x2(w.y), half2_of_e4m3x2_hi(w.y));
          *reinterpret_cast<uint4 *>(o + swizzled<128>(r, 2 * (c & 3) + 1)) =
              make_uint4(half2_of_e4m3x2(w.z), half2_of_e4m3x2_hi(w.z), half2_of_e4m3x2(w.w), half2_of_e4m3x2_hi(w.w));
        }
        fence_proxy_async_smem();
        mbar_arrive(b_hfull(it));
        mbar_arrive(b_vempty(it));
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------------ MMA issue
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_e4m3_f32(C::BM, BN);
      constexpr uint32_t idesc_pv = idesc_f16_f32(C::BM, D, 1);
      bool ok = true;
      int it = 0;                                    // tiles so far, over all parts
      int n_s[2] = {0, 0}, n_part[2] = {0, 0};       // a half's tiles and parts so far
      auto wait = [&](uint32_t bar, int phase) {
        if (ok) ok = mbar_wait(bar, phase & 1, a.wait_ns, abort_flag);
        return ok;
      };
      auto qk = [&](int h, int i) {
        const uint32_t q = sbase + C::OFF_Q + h * 2 * C::Q_BYTES, k = sbase + C::OFF_K + (i % NK) * C::T8;
        const uint32_t s = tbase + C::COL_S + 128 * h;
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_e4m3_ss(s, sdesc_rows<D>(q + part * C::Q_BYTES + kk * 32), sdesc_rows<D>(k + kk * 32), idesc_qk,
                         part + kk > 0 ? 1u : 0u);
        umma_commit(b_s(h));
      };
      auto pv = [&](int h, int i, bool add) {
        const uint32_t v = sbase + C::OFF_H + (i % NH) * C::T16;
        const uint32_t p = tbase + C::COL_S + 128 * h + C::COL_P, o = tbase + C::COL_O + D * h;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_bf16_ts(o, p + kk * 8, sdesc_sw128(v + kk * 16 * 128, BN * 128, 1024), idesc_pv, add || kk > 0 ? 1u : 0u);
      };
      while (ok && run.next(sa, sg)) {
        const int n = end_of() - sg.t0;
        if (n <= 0) continue;
        wait(b_kfull(it), it / NK);
        for (int h = 0; h < sg.halves && ok; ++h) {
          if (!wait(b_q(h), n_part[h])) break;
          tc_fence_after();
          qk(h, it);
        }
        if (!ok) break;
        umma_commit(b_kempty(it));
        for (int j = 0; j < n && ok; ++j, ++it) {
          const bool more = j + 1 < n;
          if (!wait(b_hfull(it), it / NH)) break;
          if (more && !wait(b_kfull(it + 1), (it + 1) / NK)) break;
          for (int h = 0; h < sg.halves && ok; ++h) {
            if (!wait(b_p(h), n_s[h])) break;
            ++n_s[h];
            tc_fence_after();
            pv(h, it, j > 0);
            if (!more) umma_commit(b_o(h));
            if (h + 1 == sg.halves) umma_commit(b_hempty(it));
            if (more) qk(h, it + 1);                 // over S and P of the tile whose P.V is ahead in the pipe
          }
          if (more && ok) umma_commit(b_kempty(it + 1));
        }
        for (int h = 0; h < sg.halves; ++h) ++n_part[h];
      }
      if (!ok) give_up();
      // make sure nothing issued is still running before TMEM is released
      umma_commit(b_drain);
      volatile int never = 0;
      mbar_wait(b_drain, 0, 2000000000ull, &never);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;              // row of the half == TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_addr + C::COL_S + 128 * half, tP = tS + C::COL_P;
    const uint32_t tO = tbase + lane_addr + C::COL_O + D * half;
    const int share = sa.share;
    bool ok = true;
    int it = 0, n_s = 0, n_part = 0;                   // all tiles so far; this half's tiles and parts
    while (ok && run.next(sa, sg)) {
      const int end = end_of(), n = max(end - sg.t0, 0);
      const int row0 = sg.block * C::ROWS + half * C::BM, row = row0 + r;
      auto limit_of = [&](int x) {                     // keys that row x sees: [0, limit)
        const int i = x / share;
        if (x >= sa.n_rows || i >= sg.nq) return 0;
        return sa.causal ? max(sg.len - sg.nq + i + 1, 0) : sg.len;
      };
      const bool active = half < sg.halves && n > 0;
      const int qi = row / share, hq = sg.h * share + row % share;
      const size_t at = (static_cast<size_t>(sg.b) * sa.H * share + hq) * sa.Nq + qi;   // row of Q and O
      float m_run = -INFINITY, l_run = 0.f;
      if (active) {
        // ---- the row's query in two e4m3 parts
        float rowf;
        {
          uint4 w[D / 8];
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = make_uint4(0, 0, 0, 0);
          if (row < sa.n_rows) {
            const uint4 *q = reinterpret_cast<const uint4 *>(a.Q + at * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) w[c] = __ldg(q + c);
          }
          uint32_t am = 0;                             // the largest magnitude, as bf16 bits
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) am = max(am, max((x[i] << 1) & 0xFFFEu, (x[i] >> 15) & 0xFFFEu));
          }
          const int e = min(max(static_cast<int>(am >> 8) - 127, -100), 100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
          rowf = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
          if (am >> 8 == 255) rowf = __uint_as_float(0x7FC00000u);   // a query that is not finite: NaN
          uint8_t *qs = smem + C::OFF_Q + half * 2 * C::Q_BYTES;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t x[8] = {w[2 * c].x,     w[2 * c].y,     w[2 * c].z,     w[2 * c].w,
                                   w[2 * c + 1].x, w[2 * c + 1].y, w[2 * c + 1].z, w[2 * c + 1].w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t hh[2], ll[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float f0 = __uint_as_float(x[2 * i + k] << 16) * up;
                const float f1 = __uint_as_float(x[2 * i + k] & 0xFFFF0000u) * up;
                hh[k] = e4m3x2(f0, f1);
                const float2 back = float2_of_half2(half2_of_e4m3x2(hh[k]));
                ll[k] = e4m3x2(f0 - back.x, f1 - back.y);
              }
              hi[i] = hh[0] | hh[1] << 16;
              lo[i] = ll[0] | ll[1] << 16;
            }
            *reinterpret_cast<uint4 *>(qs + swizzled<D>(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(qs + C::Q_BYTES + swizzled<D>(r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
          fence_proxy_async_smem();
          mbar_arrive(b_q(half));
        }
        const int lim = limit_of(row);
        const int all = min(limit_of(row0), limit_of(min(row0 + C::BM, sa.n_rows) - 1));   // keys every row sees
        for (int t = sg.t0; t < end; ++t, ++it, ++n_s) {
          if (!mbar_wait_warp(b_s(half), n_s & 1, a.wait_ns, abort_flag) ||
              !mbar_wait_warp(b_sc(it), (it / NSC) & 1, a.wait_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float4 *sc = reinterpret_cast<const float4 *>(smem + C::OFF_SC) + (it % NSC) * 8;
          const int left = lim - t * BN;               // columns that this row sees
          auto tile = [&](auto clean_tag) {
            constexpr bool CLEAN = decltype(clean_tag)::value;
            float v[64];
            // ---- the row's largest y; columns 64.. stay in registers
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tmem_ld64(tS + 64 * c, v);
              tmem_wait_ld();
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const float4 f = sc[4 * c + g];
                if (!CLEAN) {
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    v[16 * g + i] = 64 * c + 16 * g + i < left && f.y > -INFINITY ? v[16 * g + i] : -INFINITY;
                }
                float m0 = v[16 * g], m1 = v[16 * g + 1];
#pragma unroll
                for (int i = 2; i < 14; i += 4) {
                  m0 = fmax3_nan(m0, v[16 * g + i], v[16 * g + i + 1]);
                  m1 = fmax3_nan(m1, v[16 * g + i + 2], v[16 * g + i + 3]);
                }
                m0 = fmax3_nan(m0, v[16 * g + 14], v[16 * g + 15]);
                m0 = fmax_nan(m0, m1);
                float y = fmaf(m0, rowf * f.x, f.y);
                if (!CLEAN) y = m0 == -INFINITY ? -INFINITY : y;
                mx = fmax_nan(mx, y);
              }
            }
            if (mx != mx) rowf = mx;                   // NaN from here on
            const bool up = mx > m_run + C::kRaise;    // first keys of the row: always (m_run = -inf)
            if (__any_sync(0xffffffffu, up)) {
              const float alpha = up ? ex2_approx(m_run - mx) : 1.f;
              l_run *= alpha;
              if (t > sg.t0) {   // O holds the tiles before this one: their products are behind this S in the pipe
#pragma unroll 1
                for (int cc = 0; cc < D / 16; ++cc) {
                  float o[16];
                  tmem_ld16(tO + cc * 16, o);
                  tmem_wait_ld();
                  uint32_t u[16];
#pragma unroll
                  for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * alpha);
                  tmem_st16u(tO + cc * 16, u);
                }
              }
              if (up) m_run = mx;
            }
            // ---- weights, their sum (in units of 1 / vs) and P, columns 64.. first
            const float ref = m_run == -INFINITY ? 0.f : m_run - C::kBias;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int c = 1 - k;
              if (c == 0) {
                tmem_ld64(tS, v);
                tmem_wait_ld();
              }
              uint32_t pk[32];
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const float4 f = sc[4 * c + g];
                const float rk = rowf * f.x, off = f.y - ref;
                const float2 rk2 = make_float2(rk, rk), off2 = make_float2(off, off);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int e = 16 * g + 2 * i;
                  float2 x = __ffma2_rn(make_float2(v[e], v[e + 1]), rk2, off2);
                  if (!CLEAN) {
                    const int col = 64 * c + e;
                    x.x = col < left && f.y > -INFINITY ? x.x : -INFINITY;
                    x.y = col + 1 < left && f.y > -INFINITY ? x.y : -INFINITY;
                  }
                  x.x = ex2_approx(x.x);
                  x.y = ex2_approx(x.y);
                  sum = __fadd2_rn(sum, x);
                  pk[8 * g + i] = half2_bits(x.x, x.y);
                }
                l_run = fmaf(sum.x + sum.y, f.z, l_run);
              }
              tmem_st32u(tP + 32 * c, pk);
            }
          };
          if ((t + 1) * BN <= all && sc[0].w != 0.f) tile(std::true_type{});
          else tile(std::false_type{});
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(b_p(half));
        }
        if (ok && !mbar_wait_warp(b_o(half), n_part & 1, a.wait_ns, abort_flag)) ok = false;
        ++n_part;
        if (!ok) break;
        tc_fence_after();
      } else {
        it += n;
      }
      // ---------------------------------------------------------------- epilogue
      const float ref = m_run == -INFINITY ? -INFINITY : m_run - C::kBias;
      if (sg.whole) {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;      // a row that sees nothing is 0
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          float o[32];
          if (active) {
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (row < sa.n_rows) {
            uint4 *op = reinterpret_cast<uint4 *>(a.O + at * D + cc * 32);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              op[u] = make_uint4(pack_bf16x2(o[8 * u] * inv, o[8 * u + 1] * inv), pack_bf16x2(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                 pack_bf16x2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                 pack_bf16x2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
          }
          __syncwarp();
        }
        if (a.lse && row < sa.n_rows)
          a.lse[at] = l_run == 0.f ? -INFINITY : (ref + log2f(l_run)) * 0.6931471805599453f;
      } else {
        const size_t slot = (2 * static_cast<size_t>(cta) + (sg.first ? 1 : 0)) * C::ROWS + half * C::BM + r;
        a.m.ml[slot] = make_float2(ref, l_run);
        if (active) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            float o[32];
            tmem_ld32(tO + cc * 32, o);
            tmem_wait_ld();
            float4 *op = reinterpret_cast<float4 *>(a.m.o + slot * D + cc * 32);
#pragma unroll
            for (int u = 0; u < 8; ++u) op[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          }
        }
        if (tid == 0 && sg.first) {
          MergeItem mi;
          mi.b = sg.b;
          mi.h = sg.h;
          mi.block = sg.block;
          mi.go_on = sg.go_on;
          a.m.items[cta] = mi;
        }
      }
      tc_fence_before();   // O is read before the next part's first P is published
    }
    if (!ok && lane == 0) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

}  // namespace mcs
