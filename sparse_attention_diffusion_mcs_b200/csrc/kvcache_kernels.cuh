// kvcache_kernels.cuh -- the paged cache of keys and values held in e4m3, with
// one scale per (page, head), for keys and for values: appending tokens (keys
// rotated on the way) and reading them back as bf16.
//
// A stored number stands for e4m3 * scale.  append writes powers of two,
// scale = 2^e with the smallest e in [-60, 60] whose 448 * 2^e holds the
// page's largest finite magnitude.  With e4m3 (a floating format) a power of
// two costs no precision against the exact ratio: the relative rounding is
// 2^-4 at most for every number down to 2^-14 of the largest, e4m3's normal
// range.  What it buys: when a later token of the page needs a larger scale,
// the numbers already held move by a whole number of binades, exactly unless
// they fall below e4m3's normal range (2^-6), and dequantising is exact in
// bf16.  New numbers are rounded once, from the rotated fp32 value.
//
// Non-finite numbers: +-inf is held as the largest magnitude (+-448 * scale).
// A token with a NaN among a head's key or value has its key there held as
// NaN throughout and the value's NaN as 0: its score is then NaN in every row
// that sees it, and rows that do not see it are not reached (a NaN held in V
// would reach them as 0 * NaN).
//
// Both kernels are bound by memory (16 -> 8 bits per number, and back).
#pragma once

#include <cuda_fp8.h>

#include "rotary.cuh"

namespace mcs {

constexpr float kE4m3Max = 448.f;
constexpr int kScaleExp = 60;

struct CacheView {
  uint8_t *k, *v;                // e4m3 [n_pages, H, page, d]
  float *k_scale, *v_scale;      // [n_pages, H]
  const int32_t *table;          // [B, max_pages]
  int n_pages, max_pages, H, page, d;
};

// Scales that attention takes: of keys 0 to 2^90, of values 2^-90 to 2^90, or 0 (the
// values are 0, whatever the bytes).  Others are recorded and the page is left out.
// (Weights of 2^14 over a scale of 2^-91 sum up to less than 2^127 for 2^22 tokens;
// weights are flushed 2^140 below their row's reference, which goes by 2^x vs.)
__device__ __forceinline__ bool scales_fit(float ks, float vs) {
  return ks >= 0.f && ks <= 0x1p90f && (vs == 0.f || (vs >= 0x1p-90f && vs <= 0x1p90f));
}
// What attention reads of a page: (ks, log2 vs, 1 / vs, w); log2 vs is -inf where
// there is none, and -91 for a vs of 0: below kHasValues the bytes of V count as 0.
constexpr float kHasValues = -90.5f;
__device__ __forceinline__ float4 page_factors(bool have, float ks, float vs, float w) {
  const float v = vs == 0.f ? 0x1p-91f : vs;
  return make_float4(ks, have ? __log2f(v) : -INFINITY, have ? 1.f / v : 0.f, w);
}

// two fp32 numbers to two e4m3 bytes (lo in the low byte), to nearest, +-inf and
// what is out of range to +-448, NaN to NaN
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 bytes to two halves (exact)
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t lo16) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(lo16));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_e4m3x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ float2 float2_of_half2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// the smallest 2^e, |e| <= 60, with amax <= 448 * 2^e (amax >= 0, finite)
__device__ __forceinline__ float e4m3_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.f * 2^x: 448 * 2^e = 1.75 * 2^(8 + e)
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = min(max(e, -kScaleExp), kScaleExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

struct AppendArgs {
  CacheView c;
  const bf16 *K, *V;
  long long k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;   // strides in numbers
  const int32_t *start;                            // [B] first new token's place
  const int32_t *counts;                           // [B] new tokens of each sequence, or null: n
  const int32_t *pos;                              // [B, n, axes], or null: the token's place
  long long pos_b, pos_n;
  RotaryTable t;                                   // pairs == 0: no rotation
  int n;
  unsigned *status;
};

constexpr int kAppendThreads = 512;

// One CTA per (page that may be touched, head, sequence): grid (pages, H, B),
// one thread (or, on the largest pages, half a thread) per 16 numbers of a
// token's key and value: U units each.  A CTA's loads wait for one another
// (start, table, numbers, then the barrier), so what counts is how many CTAs an
// SM holds: keys stay in registers as rotated fp32, values as they came.
// Measured: 1560 tokens, 24 heads of 128, keys rotated: 16.3 us (29 MB; three rounds
// of two CTAs an SM, 56 % of the issue slots); one token of 16 sequences 5.7 us.
// At 64 registers, two CTAs an SM, U = 2 spills 160 bytes written and 168 read a
// thread, U = 1 8 and 24.
template <int U>
__global__ void __launch_bounds__(kAppendThreads, 2) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ unsigned s_amax[2];
  __shared__ unsigned char s_nan[128];
  const CacheView &c = a.c;
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, threads = blockDim.x;
  const int start = a.start[b];
  const int count = a.counts ? min(a.counts[b], a.n) : a.n;
  if (count <= 0) return;
  if (start < 0) {
    if (tid == 0) record_status(a.status, kStatusBadMeta);
    return;
  }
  const long long end = static_cast<long long>(start) + count;
  const long long at = start / c.page + static_cast<long long>(blockIdx.x);   // the sequence's page
  if (at * c.page >= end) return;
  int pid = -1;
  if (at < c.max_pages) pid = c.table[static_cast<long long>(b) * c.max_pages + at];   // (on its way with the numbers)
  const int base = static_cast<int>(min(at * c.page, static_cast<long long>(INT_MAX - 128)));   // (exact where there is a page)
  const int lo = max(start - base, 0);                        // new slots [lo, hi)
  const int hi = static_cast<int>(min(end - base, static_cast<long long>(c.page)));
  const int shift = c.d == 128 ? 3 : 2, upt = 1 << shift;     // units per token
  if (tid < 2) s_amax[tid] = 0;
  for (int i = tid; i < 128; i += threads) s_nan[i] = 0;
  __syncthreads();

  float kx[U][8], ky[U][8];
  RotVec<bf16> v0[U], v1[U];
  uint32_t ak = 0, av = 0;                                    // largest finite magnitudes, as their bits
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int id = tid + j * threads, slot = lo + (id >> shift), u = id & (upt - 1);
    if (slot < hi) {
      const int i = base + slot - start;                      // the call's token
      const RotUnit r = rotary_unit(a.t, u);
      const bf16 *kp = a.K + b * a.k_sb + h * a.k_sh + i * a.k_sn;
      const bf16 *vp = a.V + b * a.v_sb + h * a.v_sh + i * a.v_sn;
      RotVec<bf16> k0, k1;
      k0.load(kp + r.first);
      k1.load(kp + r.second);
      v0[j].load(vp + r.first);
      v1[j].load(vp + r.second);
      k0.get(kx[j]);
      k1.get(ky[j]);
      if (r.n_rot > 0) {
        const int32_t place = base + slot;
        float cs[8], sn[8];
        rotary_unit_angles(a.t, r, a.pos ? a.pos + b * a.pos_b + i * a.pos_n : &place, cs, sn);
        rotary_turn(a.t.interleaved, r.n_rot, cs, sn, kx[j], ky[j]);
      }
      // magnitudes by their bits, which order as they do; only a unit with a number
      // that is not finite looks at each
      constexpr uint32_t kAbs = 0x7FFFFFFFu, kInf = 0x7F800000u;
      const uint32_t w[8] = {v0[j].u.x, v0[j].u.y, v0[j].u.z, v0[j].u.w, v1[j].u.x, v1[j].u.y, v1[j].u.z, v1[j].u.w};
      uint32_t mk = 0, mv = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mk = max(mk, max(__float_as_uint(kx[j][e]) & kAbs, __float_as_uint(ky[j][e]) & kAbs));
        mv = max(mv, max(w[e] << 16 & kAbs, w[e] & 0x7FFF0000u));
      }
      if (max(mk, mv) >= kInf) {
        mk = mv = 0;
        bool bad = false;
        auto look = [&](uint32_t x, uint32_t &m) {
          x &= kAbs;
          if (x < kInf) m = max(m, x);
          bad |= x > kInf;
        };
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          look(__float_as_uint(kx[j][e]), mk);
          look(__float_as_uint(ky[j][e]), mk);
          look(w[e] << 16, mv);
          look(w[e] & 0xFFFF0000u, mv);
        }
        if (bad) s_nan[slot] = 1;
      }
      ak = max(ak, mk);
      av = max(av, mv);
    }
  }
  if (pid < 0 || pid >= c.n_pages) {   // behind the table, or no page of the pool: nothing is written
    if (tid == 0) record_status(a.status, kStatusBadMeta);
    return;
  }
  const size_t row0 = (static_cast<size_t>(pid) * c.H + h) * c.page;
  const size_t sidx = static_cast<size_t>(pid) * c.H + h;
  float ok = 0.f, ov = 0.f;                                   // the scales of the tokens held before
  if (lo > 0) {
    ok = c.k_scale[sidx];
    ov = c.v_scale[sidx];
  }
  const unsigned mk = __reduce_max_sync(0xffffffffu, ak);
  const unsigned mv = __reduce_max_sync(0xffffffffu, av);
  if ((tid & 31) == 0) {
    atomicMax(&s_amax[0], mk);
    atomicMax(&s_amax[1], mv);
  }
  __syncthreads();
  const float sk = fmaxf(e4m3_scale(__uint_as_float(s_amax[0])), ok);
  const float sv = fmaxf(e4m3_scale(__uint_as_float(s_amax[1])), ov);
  // tokens held before move to the larger scale (their slots are [0, lo))
  for (int w = 0; w < 2; ++w) {
    const float was = w ? ov : ok, now = w ? sv : sk;
    if (lo > 0 && now > was) {
      const float f = was / now;
      uint4 *p = reinterpret_cast<uint4 *>((w ? c.v : c.k) + row0 * c.d);
      for (int id = tid; id < lo * upt; id += threads) {
        uint4 q = p[id];
        uint32_t *x = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 u0 = float2_of_half2(half2_of_e4m3x2(x[e])), u1 = float2_of_half2(half2_of_e4m3x2_hi(x[e]));
          x[e] = e4m3x2(u0.x * f, u0.y * f) | e4m3x2(u1.x * f, u1.y * f) << 16;
        }
        p[id] = q;
      }
    }
  }
  const float ik = 1.f / sk, iv = 1.f / sv;                   // exact for powers of two
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int id = tid + j * threads, slot = lo + (id >> shift), u = id & (upt - 1);
    if (slot < hi) {
      const RotUnit r = rotary_unit(a.t, u);
      const bool bad = s_nan[slot] != 0;
      auto pack = [&](const float (&x)[8], float f) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = e4m3x2(x[2 * e] * f, x[2 * e + 1] * f);
        return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      };
      float x[8], y[8];
      v0[j].get(x);
      v1[j].get(y);
      uint2 k0 = pack(kx[j], ik), k1 = pack(ky[j], ik);
      if (bad) {                                              // a NaN key, its values' NaN as 0
        k0 = k1 = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = isnan(x[e]) ? 0.f : x[e];
          y[e] = isnan(y[e]) ? 0.f : y[e];
        }
      }
      uint8_t *kp = c.k + (row0 + slot) * c.d, *vp = c.v + (row0 + slot) * c.d;
      *reinterpret_cast<uint2 *>(kp + r.first) = k0;
      *reinterpret_cast<uint2 *>(kp + r.second) = k1;
      *reinterpret_cast<uint2 *>(vp + r.first) = pack(x, iv);
      *reinterpret_cast<uint2 *>(vp + r.second) = pack(y, iv);
    }
  }
  if (tid == 0) {
    c.k_scale[sidx] = sk;
    c.v_scale[sidx] = sv;
  }
}

struct ReadArgs {
  CacheView c;
  const int32_t *start, *counts;   // [B]; counts may be null: n
  bf16 *K, *V;                     // [B, H, n, d]
  int n, page_shift;
  unsigned *status;
};

constexpr int kReadThreads = 256;

// 16 numbers of a token and head, of K and of V, per thread: grid (units of one
// sequence and head, H, B).  Bound by memory: 1 byte in, 2 out (604 MB in 112 us,
// 5.4 TB/s, 82 % of the measured copy's 1:1; two and four units a thread, 128
// to 512 threads and streaming stores are all within 4 % of it).
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  const CacheView &c = a.c;
  const int b = blockIdx.z, h = blockIdx.y;
  const int shift = c.d == 128 ? 3 : 2;                 // units per token
  const long long id = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long i = id >> shift;                      // the call's token
  if (i >= a.n) return;
  const int u = static_cast<int>(id) & ((1 << shift) - 1);
  const long long pos = a.start[b] + i, at = pos >> a.page_shift;
  uint4 k = make_uint4(0, 0, 0, 0), v = k;
  float sk = 0.f, sv = 0.f;
  if (pos >= 0 && at < c.max_pages && (!a.counts || i < a.counts[b])) {
    const int pid = c.table[static_cast<long long>(b) * c.max_pages + at];
    if (pid >= 0 && pid < c.n_pages) {
      const size_t s = static_cast<size_t>(pid) * c.H + h;
      const size_t off = (s * c.page + static_cast<size_t>(pos & (c.page - 1))) * c.d + 16 * u;
      k = *reinterpret_cast<const uint4 *>(c.k + off);
      v = *reinterpret_cast<const uint4 *>(c.v + off);
      sk = c.k_scale[s];
      sv = c.v_scale[s];
    } else {
      record_status(a.status, kStatusBadMeta);
    }
  }
  const size_t to = ((static_cast<size_t>(b) * c.H + h) * a.n + i) * c.d + 16 * u;
  auto put = [&](bf16 *out, const uint4 &q, float s) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = float2_of_half2(half2_of_e4m3x2(w[e])), hi = float2_of_half2(half2_of_e4m3x2_hi(w[e]));
      o[2 * e] = pack_bf16x2(lo.x * s, lo.y * s);
      o[2 * e + 1] = pack_bf16x2(hi.x * s, hi.y * s);
    }
    uint4 *p = reinterpret_cast<uint4 *>(out + to);
    p[0] = make_uint4(o[0], o[1], o[2], o[3]);
    p[1] = make_uint4(o[4], o[5], o[6], o[7]);
  };
  put(a.K, k, sk);
  put(a.V, v, sv);
}

}  // namespace mcs
