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
// exact from 2^-2 on, where lo is a multiple of e4m3's smallest step, 2^-9, and off
// by at most half that step below: exact down to 2^-9 of the row's largest at
// worst, and off by at most 2^-17 of it below.
// Two 8-bit products (hi, then lo) cost what one 16-bit product costs, and no
// key is converted.
// P.V runs in fp16: the weights need more than e4m3's 4 bits, and a weight
// whose 8-bit parts underflow would lose the tail of a long row.  A second fp16
// part would double these products, for an eighth of what the output's own rounding
// to bf16 may be off by: outputs are off by 1.7e-3 of their norm against 64 bits, as
// ones computed in 32 bits are.  Four warps turn each 128-key tile of V into fp16
// once (exact) for all 256 query rows.
// Weights are 2^(y - m + 6) with m at most 2^8 behind the row's maximum: at
// most 2^14, rounded to fp16 by 2^-11 relative, normal down to 2^-20 of the
// reference's.  Sums, m and O are fp32.
//
// A CTA takes 256 query rows (two halves of 128, one TMEM lane a row) and runs
// of 128-key tiles, dealt as cache_sched.cuh describes:
//   warp  0         TMEM allocation, MMA issue
//   warp  1         loads: one TMA box per page, keys and values; the scales
//   warps 4-7       V from e4m3 to fp16
//   warps 8-11, 12-15  softmax and epilogue of half 0, half 1
// The tensor pipe runs per tile j: PV0(j) QK0(j+1) PV1(j) QK1(j+1), so each
// half's softmax has the other half's two products to work in.  A block of at
// most 128 rows has no second half: the two then take alternate tiles of the
// same rows, and half 0 adds half 1's O to its own at the end (PV0(j) QK0(j+2)
// PV1(j+1) QK1(j+3)).  P (fp16 pairs) lies over the lower half of its own S.
// TMEM: S0, S1 (128 columns each), O0, O1 (D columns each).  Every wait is
// bounded.
//
// Measured (4680 causal rows against 32760 tokens, 24 heads of 128): 1.69 to 1.87
// ms with the clock that the power leaves, 1.04 to 0.94 PFLOP/s; 1560 rows against
// 10920 tokens 280 us and 12 of merge.  ptxas spills 416 bytes written and 316 read a
// thread, at 128 registers for all roles before the handover below.  What follows
// was measured at 1.72 ms: without the conversion of V 1.63, without
// exponentials 1.47 ms.  Per tile a half's softmax takes 2600 cycles beside the
// other half's (1024 of them exponentials), and the products 2340 instead of
// 2048: they, the conversion and the loads ask for 2330 cycles of the shared
// memory's 128 bytes a cycle.  Tried and slower: one thread per half row (1.83),
// S read twice (1.86), tiles of 64 keys with S double-buffered (1.87: twice
// the MMA instructions, 75 cycles each to issue), an MMA warp per half (2.13:
// both halves' products then end late, together), exponentials on the FMA
// pipe (one in eight 1.81, one in four 1.98).
#pragma once

#include <type_traits>

#include "cache_rows_kernel.cuh"

namespace mcs {

// The MMA warp's lanes run its loop together, so that operands stay in uniform
// registers; each instruction is issued by one elected lane.

// the same word of every lane as a warp-uniform one
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate; descriptors by their halves.
__device__ __forceinline__ void umma_e4m3_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t hi,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
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

// the largest of 16 numbers
__device__ __forceinline__ float max16(const float *x) {
  const float a = fmax3(x[0], x[1], x[2]), b = fmax3(x[3], x[4], x[5]), c = fmax3(x[6], x[7], x[8]);
  const float d = fmax3(x[9], x[10], x[11]), e = fmax3(x[12], x[13], x[14]);
  return fmaxf(fmax3(a, b, c), fmax3(d, e, x[15]));
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
  static constexpr int N_BAR = 2 * NK + 2 * NV + 2 * NH + NSC + 10 + 1;
  static constexpr int OFF_XCH = OFF_BAR + 8 * N_BAR;         // 128 x float2: half 1's reference and sum for half 0
  static constexpr int OFF_RF = OFF_XCH + BM * 8;             // the rows' factors (scale log2(e) 2^..)
  static constexpr int OFF_MISC = OFF_RF + ROWS * 4;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int MMA_WARP = 0, LOAD_WARP = 1, CVT_WARP = 4, CVT_THREADS = 128, SOFTMAX_WARP = 8;
  static constexpr int THREADS = 16 * 32;
  static constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_O = 256;   // half h: S at 128 h, O at 256 + D h
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
  auto b_j = [&](int h) { return by + 64 + 8 * h; };
  const uint32_t b_drain = by + 80;
  float2 *xch = reinterpret_cast<float2 *>(smem + C::OFF_XCH);
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
      mbar_init(b_vempty(i), C::CVT_THREADS / 32);
    }
    for (int i = 0; i < NH; ++i) {
      mbar_init(b_hfull(i), C::CVT_THREADS / 32);
      mbar_init(b_hempty(i), 1);
    }
    for (int i = 0; i < NSC; ++i) mbar_init(b_sc(i), 1);
    for (int h = 0; h < 2; ++h) {
      mbar_init(b_q(h), 4);
      mbar_init(b_s(h), 1);
      mbar_init(b_p(h), 4);                        // (one lane a warp)
      mbar_init(b_o(h), 1);
      mbar_init(b_j(h), 4);
    }
    mbar_init(b_drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (tid == C::SOFTMAX_WARP * 32) a.m.items[cta].go_on = 0;   // (the thread that may set it)
  if (warp == C::MMA_WARP) {
    __syncwarp();                                  // (lane 0 comes from the branch above)
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

  auto warp_arrive = [&](uint32_t bar) {           // once for the warp, when all its lanes are there
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  // registers go from the helpers to the softmax, whose threads hold a whole row
  // of S: 256 x 200 + 256 x 56 = the 512 x 128 of the launch
  if (warp < C::SOFTMAX_WARP) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
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
      auto check_scales = [&]() {
        if (pid >= 0 && !scales_fit(ks, vs)) {
          record_status(a.status, kStatusBadMeta);
          pid = -1;
        }
      };
      check_scales();
      for (int tb = sg.t0; tb < end && ok; tb += 4) {
        const int npid = fetch_page(8 * (tb + 4) + lane);
        float nks, nvs;
        fetch_scales(npid, nks, nvs);
        for (int t = tb; t < min(tb + 4, end); ++t, ++it) {
          const int gl = 8 * (t - tb);                 // lane of the tile's first group
          const bool in = lane >= gl && lane < gl + 8;
          const unsigned good = __ballot_sync(0xffffffffu, in && pid >= 0 && vs > 0.f);
          // the first lane of each page's groups loads it
          const bool mine = in && (lane - gl) % gpb == 0 && pid >= 0;
          const uint32_t tx = __popc(__ballot_sync(0xffffffffu, mine)) * page_bytes;
          const int r = mine ? static_cast<int>((static_cast<long long>(pid) * cv.H + sg.h) * cv.page) : 0;
          const uint32_t at = (lane - gl) * 16 * D;
          ok = mbar_wait_warp(b_kempty(it), ((it / NK) & 1) ^ 1, a.wait_ns, abort_flag);
          if (!ok) break;
          if (in)
            *reinterpret_cast<float4 *>(smem + C::OFF_SC + ((it % NSC) * 8 + lane - gl) * 16) =
                page_factors(pid >= 0, ks, vs, __popc(good) == 8 ? 1.f : 0.f);
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
        check_scales();
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
    // A thread takes one 16-byte chunk of every RSTEP-th key: a 16-byte read, two
    // 16-byte writes at fixed distances.  Eight neighbouring threads take four
    // chunks of keys r and r ^ 5, which the swizzles of both layouts send to
    // different banks.
    constexpr int CH = D / 16, PER = BN * CH / C::CVT_THREADS, RSTEP = BN / PER;
    static_assert(RSTEP % 8 == 0 && PER % 4 == 0, "a thread's keys share their swizzle");
    const int ct = tid - C::CVT_WARP * 32;                   // (pair of keys, 4 chunks, key of the pair, chunk)
    const int rest = ct >> 3, chunk = rest % (CH / 4) * 4 + (ct & 3), pair = rest / (CH / 4);
    const int key = ((pair >> 2) * 8 + (pair & 3)) ^ (ct & 4 ? 5 : 0);   // pairs (r, r ^ 5), r = 0, 1, 2, 3 of each 8 keys
    const int from = swizzled<D>(key, chunk);
    // 64-number blocks of 128-byte rows
    const int to0 = (chunk >> 2) * (BN * 128) + swizzled<128>(key, 2 * (chunk & 3));
    const int to1 = (chunk >> 2) * (BN * 128) + swizzled<128>(key, 2 * (chunk & 3) + 1);
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
        // four reads on the way at once: the compiler cannot move one over the writes of another
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += 4) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4 *>(src + from + (i0 + i) * RSTEP * D);
          // what lies behind the last key that is seen, or was never loaded, or has a scale of 0, may be any bits
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = key + (i0 + i) * RSTEP;
              if (!(t * BN + r < sg.kmax && sc[r >> 4].y > kHasValues)) w[i] = make_uint4(0, 0, 0, 0);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = w[i];
            *reinterpret_cast<uint4 *>(dst + to0 + (i0 + i) * RSTEP * 128) =
                make_uint4(half2_of_e4m3x2(x.x), half2_of_e4m3x2_hi(x.x), half2_of_e4m3x2(x.y), half2_of_e4m3x2_hi(x.y));
            *reinterpret_cast<uint4 *>(dst + to1 + (i0 + i) * RSTEP * 128) =
                make_uint4(half2_of_e4m3x2(x.z), half2_of_e4m3x2_hi(x.z), half2_of_e4m3x2(x.w), half2_of_e4m3x2_hi(x.w));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_hfull(it));
          mbar_arrive(b_vempty(it));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) give_up();
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------------ MMA issue
    {
      constexpr uint32_t idesc_qk = idesc_e4m3_f32(C::BM, BN);
      constexpr uint32_t idesc_pv = idesc_f16_f32(C::BM, D, 1);
      // descriptors: the upper words are the layouts', the lower ones move with the address
      const uint64_t dq = sdesc_rows<D>(sbase + C::OFF_Q), dk = sdesc_rows<D>(sbase + C::OFF_K);
      const uint64_t dv = sdesc_sw128(sbase + C::OFF_H, BN * 128, 1024);
      const uint32_t q_lo = uniform(static_cast<uint32_t>(dq)), k_lo = uniform(static_cast<uint32_t>(dk));
      const uint32_t v_lo = uniform(static_cast<uint32_t>(dv));
      const uint32_t qk_hi = uniform(static_cast<uint32_t>(dq >> 32)), v_hi = uniform(static_cast<uint32_t>(dv >> 32));
      const uint32_t tb = uniform(tbase);
      bool ok = true;
      int it = 0;                                    // tiles so far, over all parts
      int n_s[2] = {0, 0}, n_part[2] = {0, 0};       // a half's tiles and parts so far
      auto wait = [&](uint32_t bar, int phase) {
        if (ok) ok = mbar_wait_warp(bar, phase & 1, a.wait_ns, abort_flag);
        return ok;
      };
      auto qk = [&](int h, int i) {
        const uint32_t q = q_lo + uniform(h * (2 * C::Q_BYTES >> 4)), k = k_lo + uniform(i % NK * (C::T8 >> 4));
        const uint32_t s = tb + uniform(C::COL_S + 128 * h);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            umma_e4m3_ss(s, q + ((part * C::Q_BYTES + kk * 32) >> 4), k + (kk * 32 >> 4), qk_hi, idesc_qk,
                         part + kk > 0 ? 1u : 0u);
        umma_commit_elect(b_s(h));
      };
      auto pv = [&](int h, int i, bool add) {
        const uint32_t v = v_lo + uniform(i % NH * (C::T16 >> 4));
        const uint32_t p = tb + uniform(C::COL_S + 128 * h), o = tb + uniform(C::COL_O + D * h);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_f16_ts(o, p + kk * 8, v + (kk * 16 * 128 >> 4), v_hi, idesc_pv, add || kk > 0 ? 1u : 0u);
      };
      while (ok && run.next(sa, sg)) {
        const int n = end_of() - sg.t0;
        if (n <= 0) continue;
        const bool two = sg.halves == 2;
        // scores of the part's tile j for half h
        auto scores = [&](int h, int j) {
          if (!wait(b_kfull(it + j), (it + j) / NK)) return;
          if (j < (two ? 1 : 2) && !wait(b_q(h), n_part[h])) return;
          tc_fence_after();
          qk(h, it + j);
          if (!two || h == 1) umma_commit_elect(b_kempty(it + j));
        };
        scores(0, 0);
        if (two) scores(1, 0);
        else if (n > 1) scores(1, 1);
        for (int j = 0; j < n && ok; ++j) {
          if (!wait(b_hfull(it + j), (it + j) / NH)) break;
          const int ahead = two ? 1 : 2;
          for (int h = two ? 0 : j & 1; h < (two ? 2 : (j & 1) + 1) && ok; ++h) {
            if (!wait(b_p(h), n_s[h])) break;
            ++n_s[h];
            tc_fence_after();
            pv(h, it + j, j >= ahead);
            if (j + ahead >= n) umma_commit_elect(b_o(h));
            if (!two || h == 1) umma_commit_elect(b_hempty(it + j));
            if (j + ahead < n) scores(h, j + ahead);   // over S and P of the tile whose P.V is ahead in the pipe
          }
        }
        it += n;
        ++n_part[0];
        if (two || n > 1) ++n_part[1];
      }
      if (!ok && lane == 0) give_up();
      // make sure nothing issued is still running before TMEM is released
      umma_commit_elect(b_drain);
      volatile int never = 0;
      mbar_wait(b_drain, 0, 2000000000ull, &never);
    }
    __syncwarp();
  }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int half = (warp - C::SOFTMAX_WARP) >> 2;
    const int r = (warp & 3) * 32 + lane;              // row of the half == TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_addr + C::COL_S + 128 * half;
    const uint32_t tO = tbase + lane_addr + C::COL_O + D * half;
    const int share = sa.share;
    bool ok = true;
    int it = 0, n_s = 0, n_part = 0, n_join = 0;       // all tiles so far; this half's tiles and parts; joint parts
    while (ok && run.next(sa, sg)) {
      const int end = end_of(), n = max(end - sg.t0, 0), it0 = it;
      const bool two = sg.halves == 2;
      const int row0 = sg.block * C::ROWS + (two ? half * C::BM : 0), row = row0 + r;   // whose scores
      const int orow = sg.block * C::ROWS + half * C::BM + r;                             // whose output
      auto limit_of = [&](int x) {                     // keys that row x sees: [0, limit)
        const int i = x / share;
        if (x >= sa.n_rows || i >= sg.nq) return 0;
        return sa.causal ? max(sg.len - sg.nq + i + 1, 0) : sg.len;
      };
      const int step = two ? 1 : 2, skip = two ? 0 : half;   // this half's tiles: t0 + skip, + step, ...
      const bool active = n > skip;
      const size_t first_row = (static_cast<size_t>(sg.b) * sa.H + sg.h) * share * sa.Nq;
      auto address = [&](int x) {                      // row x of the item in Q and O
        return first_row + (share == 1 ? x : static_cast<size_t>(x % share) * sa.Nq + x / share);
      };
      float m_run = -INFINITY, l_run = 0.f;
      if (active) {
        // ---- the queries in two e4m3 parts: a warp takes its 32 rows, D / 8 lanes a row.
        // (A thread for each row, unrolled over the row, took 7 us a part: its
        // instructions came from far away, its loads 16 bytes a line.)
        constexpr int LPR = D / 8, RPI = 32 / LPR;     // lanes per row, rows at once
        const int lane_row = (warp & 3) * 32 + lane / LPR, qc = lane % LPR;
        uint8_t *qs = smem + C::OFF_Q + half * 2 * C::Q_BYTES;
        float *rf = reinterpret_cast<float *>(smem + C::OFF_RF) + half * C::BM;
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 8 * RPI) {
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = row0 + lane_row + i0 + i * RPI;
            w[i] = make_uint4(0, 0, 0, 0);
            if (x < sa.n_rows) w[i] = __ldg(reinterpret_cast<const uint4 *>(a.Q + address(x) * D) + qc);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int qr = lane_row + i0 + i * RPI;
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t am = 0;                           // the row's largest magnitude, as bf16 bits
#pragma unroll
            for (int k = 0; k < 4; ++k) am = max(am, max((x[k] << 1) & 0xFFFEu, (x[k] >> 15) & 0xFFFEu));
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int e = min(max(static_cast<int>(am >> 8) - 127, -100), 127);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + 7 - e) << 23);
            const float down = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - 7 + e) << 23);
            if (qc == 0) rf[qr] = am >> 8 == 255 ? __uint_as_float(0x7FC00000u) : down;   // a query that is not finite: NaN
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f0 = __uint_as_float(x[k] << 16) * up, f1 = __uint_as_float(x[k] & 0xFFFF0000u) * up;
              hi[k] = e4m3x2(f0, f1);
              const float2 back = float2_of_half2(half2_of_e4m3x2(hi[k]));
              lo[k] = e4m3x2(f0 - back.x, f1 - back.y);
            }
            uint8_t *to = qs + swizzled<D>(qr, qc >> 1) + (qc & 1) * 8;
            *reinterpret_cast<uint2 *>(to) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2 *>(to + C::Q_BYTES) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(b_q(half));
        const float rowf = rf[r];
        const int lim = limit_of(row);
        const int all = min(limit_of(row0), limit_of(min(row0 + C::BM, sa.n_rows) - 1));   // keys every row sees
        it += skip;
        for (int t = sg.t0 + skip; t < end; t += step, it += step, ++n_s) {
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
            // the whole row in registers: a read of S takes hundreds of cycles beside the products
            float v[128];
            tmem_ld64(tS, *reinterpret_cast<float(*)[64]>(v));
            tmem_ld64(tS + 64, *reinterpret_cast<float(*)[64]>(v + 64));
            tmem_wait_ld();
            // ---- the row's largest y
            float mx = -INFINITY;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              const float4 f = sc[g];
              if (!CLEAN) {
#pragma unroll
                for (int i = 16 * g; i < 16 * g + 16; ++i) v[i] = i < left && f.y > -INFINITY ? v[i] : -INFINITY;
              }
              const float top = max16(v + 16 * g), y = fmaf(top, rowf * f.x, f.y);
              mx = fmaxf(mx, CLEAN || top > -INFINITY ? y : -INFINITY);
            }
            const bool up = mx > m_run + C::kRaise;    // first keys of the row: always (m_run = -inf)
            if (__any_sync(0xffffffffu, up)) {
              const float alpha = up ? ex2_approx(m_run - mx) : 1.f;
              l_run *= alpha;
              if (t >= sg.t0 + step) {   // O holds the tiles before this one: their products are behind this S in the pipe
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
            // ---- weights, their sum (in units of 1 / vs) and P, 32 keys at a time, in
            // stages, so that the exponentials follow one another without a pause (348
            // cycles for the 32 columns of a warp alone, 628 pair by pair)
            const float ref = m_run == -INFINITY ? 0.f : m_run - C::kBias;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 fs[2] = {sc[2 * c], sc[2 * c + 1]};
              float2 y[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float rk = rowf * fs[i >> 3].x, off = fs[i >> 3].y - ref;
                const float2 x = make_float2(v[32 * c + 2 * i], v[32 * c + 2 * i + 1]);
                y[i] = __ffma2_rn(x, make_float2(rk, rk), make_float2(off, off));
                if (!CLEAN) {
                  y[i].x = x.x == -INFINITY ? -INFINITY : y[i].x;
                  y[i].y = x.y == -INFINITY ? -INFINITY : y[i].y;
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = make_float2(ex2_approx(y[i].x), ex2_approx(y[i].y));
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = half2_bits(y[i].x, y[i].y);
              tmem_st16u(tS + 16 * c, pk);
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const float2 *z = y + 8 * g;
                const float2 s0 = __fadd2_rn(__fadd2_rn(z[0], z[1]), __fadd2_rn(z[2], z[3]));
                const float2 s1 = __fadd2_rn(__fadd2_rn(z[4], z[5]), __fadd2_rn(z[6], z[7]));
                const float2 sum = __fadd2_rn(s0, s1);
                l_run = fmaf(sum.x + sum.y, fs[g].z, l_run);
              }
            }
          };
          if ((t + 1) * BN <= all && sc[0].w != 0.f) tile(std::true_type{});
          else tile(std::false_type{});
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(b_p(half));
        }
        // sums of products stay below 2^24 and scales are at most 2^90: from 2^13 on scores
        // may leave fp32.  Above it they make NaN; a row with keys and all its scores below is NaN too.
        if (rowf >= 0x1p13f && m_run == -INFINITY && lim > (sg.t0 + skip) * BN) l_run = NAN;
        if (ok && !mbar_wait_warp(b_o(half), n_part & 1, a.wait_ns, abort_flag)) ok = false;
        ++n_part;
        if (!ok) break;
        tc_fence_after();
      }
      it = it0 + n;
      float ref = m_run == -INFINITY ? -INFINITY : m_run - C::kBias, f0 = 1.f, f1 = 0.f;
      // ---- a block without a second half: half 0 adds half 1's part of the row to its own
      const bool join = !two && n > 1;
      if (join && half == 1) {
        xch[r] = make_float2(ref, l_run);
        tc_fence_before();
        warp_arrive(b_j(1));
      } else if (join) {
        if (!mbar_wait_warp(b_j(1), n_join & 1, a.wait_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float2 g = xch[r];
        const float mm = fmaxf(ref, g.x);
        f0 = merge_factor(ref, l_run, mm);
        f1 = merge_factor(g.x, g.y, mm);
        l_run = fmaf(l_run, f0, g.y * f1);
        ref = mm;
      }
      const bool has = n > 0 && (two || half == 0);    // an output to write that is not empty
      if (!has) {
        ref = -INFINITY;
        l_run = 0.f;
      }
      // ---------------------------------------------------------------- epilogue
      auto load_o = [&](int cc, float (&o)[32]) {
        tmem_ld32(tO + cc * 32, o);
        if (join) {
          float o1[32];
          tmem_ld32(tO + D + cc * 32, o1);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(o1[i], f1, o[i] * f0);
        } else {
          tmem_wait_ld();
        }
      };
      if (sg.whole) {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;      // a row that sees nothing is 0
        const size_t at = orow < sa.n_rows ? address(orow) : 0;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          float o[32];
          if (has) {
            load_o(cc, o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (orow < sa.n_rows) {
            uint4 *op = reinterpret_cast<uint4 *>(a.O + at * D + cc * 32);
#pragma unroll
            for (int u = 0; u < 4; ++u)
              op[u] = make_uint4(pack_bf16x2(o[8 * u] * inv, o[8 * u + 1] * inv), pack_bf16x2(o[8 * u + 2] * inv, o[8 * u + 3] * inv),
                                 pack_bf16x2(o[8 * u + 4] * inv, o[8 * u + 5] * inv),
                                 pack_bf16x2(o[8 * u + 6] * inv, o[8 * u + 7] * inv));
          }
          __syncwarp();
        }
        if (a.lse && orow < sa.n_rows)
          a.lse[at] = l_run == 0.f ? -INFINITY : (ref + log2f(l_run)) * 0.6931471805599453f;
      } else {
        const size_t slot_rows = (2 * static_cast<size_t>(cta) + (sg.first ? 1 : 0)) * C::ROWS;   // rows before the slot's
        a.m.ml[slot_rows + half * C::BM + r] = make_float2(ref, l_run);
        if (has) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            float o[32];
            load_o(cc, o);
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *merge_part(a.m, slot_rows, C::ROWS, D, half * C::BM + r, cc * 8 + u) =
                  make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          }
        }
        if (tid == C::SOFTMAX_WARP * 32 && sg.first) {
          MergeItem mi;
          mi.b = sg.b;
          mi.h = sg.h;
          mi.block = sg.block;
          mi.go_on = sg.go_on;
          a.m.items[cta] = mi;
        }
      }
      if (join) {
        if (half == 0) {
          tc_fence_before();
          warp_arrive(b_j(0));
        } else if (!mbar_wait_warp(b_j(0), n_join & 1, a.wait_ns, abort_flag)) {   // half 0 has read O1
          ok = false;
          break;
        }
        ++n_join;
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
