// rotary.cuh -- rotary positions: each pair (a, b) of a head's numbers is
// turned by the angle t = pos * f of its pair,
//   a' = mag (a cos t - b sin t),   b' = mag (a sin t + b cos t),
// and the gradient is the same map with -t.
//
// Angles: f is held as the 64-bit fraction of a turn F = round(f / 2pi * 2^64).
// pos * F mod 2^64 is then the phase, exact for every 32-bit position (the
// product wraps whole turns away; F's own rounding moves it by at most
// |pos| * 2^-65 turns), so far positions lose nothing and no table of angles is
// read.  The phase's top 32 bits (what is cut off is less than 1.5e-9 rad) are
// split into a quarter turn and the rest, at most an eighth of a turn, whose sine
// and cosine are polynomials (turn_sincos): off by 1.1e-7 at most, in about half
// the instructions of sincospif.  Correct rounding would be off by 3e-8; a pair is
// off by 2.9e-7 of its length in all, which 16-bit outputs do not see (2^-9) and
// fp32 ones as their last two bits.
//
// The kernel is bound by memory: every number is read and written once.  A
// thread owns 16 numbers of one token (8 pairs, two 16-byte vectors for 16-bit
// types) and walks over the heads, so the angles are computed once for all
// heads of its group.  Measured, 24 heads, 32760 tokens of 128, 3 axes, from the
// projection's layout: bf16 and fp16 70 us in a row of calls, 5.7 TB/s (88 % of the
// measured copy), fp32 143 us, 5.6 TB/s; one bf16 call after a flush 62 us, a
// quarter of its writes still in the cache.  2 x 16 heads, 8191 tokens of 64, 48
// turned: 16 us, 4.2 TB/s.
#pragma once

#include <cuda_fp16.h>

#include "mcs_common.cuh"

namespace mcs {

struct RotaryTable {
  const unsigned long long *turns;   // [pairs] fractions of a turn per position, times 2^64
  const int32_t *axis;               // [pairs] position axis each pair goes by
  int pairs;                         // rotated pairs of a head (may be 0)
  int interleaved;                   // pairs (2i, 2i+1) instead of (i, pairs + i)
  int axes;                          // numbers per position
  float mag;                         // factor on the rotated numbers
};

// cos and sin of phase / 2^32 turns.  With q the nearest quarter turn and x the
// rest in half turns, |x| <= 1/4, z = x^2:
//   sin(pi x) ~ x (s0 + s1 z + s2 z^2 + s3 z^3),  cos(pi x) ~ 1 + z (c0 + c1 z + c2 z^2 + c3 z^3),
// the Chebyshev interpolants of sin(pi x) / x and (cos(pi x) - 1) / z in z on
// [0, 1/16]: off by 1.1e-7 at most with fp32's roundings.
__device__ __forceinline__ void turn_sincos(uint32_t phase, float &c, float &s) {
  const uint32_t q = (phase + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(phase - (q << 30))) * 4.656612873077393e-10f;   // 2^-31
  const float z = x * x;
  float u = fmaf(z, -5.890768766e-01f, 2.549767017e+00f);
  u = fmaf(u, z, -5.167707920e+00f);
  u = fmaf(u, z, 3.141592741e+00f) * x;
  float v = fmaf(z, 2.321258634e-01f, -1.335137844e+00f);
  v = fmaf(v, z, 4.058710575e+00f);
  v = fmaf(v, z, -4.934802055e+00f);
  v = fmaf(v, z, 1.f);
  // q quarter turns on: (c, s) -> (-s, c) each
  const float a = q & 1 ? u : v, b = q & 1 ? v : u;
  c = __uint_as_float(__float_as_uint(a) ^ (((q + 1) & 2) << 30));
  s = __uint_as_float(__float_as_uint(b) ^ ((q & 2) << 30));
}

// cos and sin of pair i at the position whose axis numbers are at `pos`
__device__ __forceinline__ void rotary_angle(const RotaryTable &t, int i, const int32_t *pos, float &c, float &s) {
  const unsigned long long f = t.turns[i];
  const long long p = pos[t.axis[i]];
  turn_sincos(static_cast<uint32_t>((static_cast<unsigned long long>(p) * f) >> 32), c, s);
}

// 8 numbers; keep(was, n): the neighbouring pairs from the n-th on as in `was`, bit for bit
template <typename T>
struct RotVec;
__device__ __forceinline__ void keep_words(uint4 &u, const uint4 &was, int n) {
  if (n <= 0) u.x = was.x;
  if (n <= 1) u.y = was.y;
  if (n <= 2) u.z = was.z;
  if (n <= 3) u.w = was.w;
}
template <>
struct RotVec<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void store(float *p) const {
    *reinterpret_cast<float4 *>(p) = a;
    *reinterpret_cast<float4 *>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void keep(const RotVec &was, int n) {
    if (n <= 0) a.x = was.a.x, a.y = was.a.y;
    if (n <= 1) a.z = was.a.z, a.w = was.a.w;
    if (n <= 2) b.x = was.b.x, b.y = was.b.y;
    if (n <= 3) b.z = was.b.z, b.w = was.b.w;
  }
};
template <>
struct RotVec<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
  __device__ __forceinline__ void keep(const RotVec &was, int n) { keep_words(u, was.u, n); }
};
template <>
struct RotVec<__half> {
  uint4 u;
  __device__ __forceinline__ void load(const __half *p) { u = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(__half *p) const { *reinterpret_cast<uint4 *>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void keep(const RotVec &was, int n) { keep_words(u, was.u, n); }
};

__device__ __forceinline__ float rot_get(float x) { return x; }
__device__ __forceinline__ float rot_get(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float rot_get(__half x) { return __half2float(x); }
__device__ __forceinline__ void rot_put(float *p, float x) { *p = x; }
__device__ __forceinline__ void rot_put(bf16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void rot_put(__half *p, float x) { *p = __float2half_rn(x); }

// Where unit u of a head (16 numbers) lies: its two 8-number vectors start at
// first and second; n_rot of its pairs turn, the first being pair `pair`.
// Half layout: vector `first` holds the pairs' a, `second` their b (or, behind
// the rotated part, 16 numbers that stay).  Interleaved: 16 numbers in a row.
// The half layout needs pairs % 8 == 0.
struct RotUnit {
  int first, second, pair, n_rot;
};
__device__ __forceinline__ RotUnit rotary_unit(const RotaryTable &t, int u) {
  RotUnit r;
  if (t.interleaved) {
    r.first = 16 * u;
    r.second = r.first + 8;
    r.pair = 8 * u;
    r.n_rot = min(max(t.pairs - r.pair, 0), 8);
  } else if (8 * u < t.pairs) {
    r.first = 8 * u;
    r.second = t.pairs + 8 * u;
    r.pair = 8 * u;
    r.n_rot = 8;
  } else {
    r.first = 2 * t.pairs + 16 * (u - t.pairs / 8);
    r.second = r.first + 8;
    r.pair = 0;
    r.n_rot = 0;
  }
  return r;
}

// cos and sin (times mag) of the unit's pairs that turn
__device__ __forceinline__ void rotary_unit_angles(const RotaryTable &t, const RotUnit &r, const int32_t *pos,
                                                   float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
    if (i < r.n_rot) {
      rotary_angle(t, r.pair + i, pos, c[i], s[i]);
      c[i] *= t.mag;
      s[i] *= t.mag;
    }
  }
}

// the unit's first n_rot pairs turned in place, the others untouched (b * 0 is not 0
// where b is inf or NaN): x its first vector, y its second.  Half layout: n_rot is 8.
__device__ __forceinline__ void rotary_turn(bool interleaved, int n_rot, const float (&c)[8], const float (&s)[8],
                                            float (&x)[8], float (&y)[8]) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float &p = i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)], &q = i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1];
      const float a = p, b = q;
      p = i < n_rot ? fmaf(a, c[i], -b * s[i]) : a;
      q = i < n_rot ? fmaf(a, s[i], b * c[i]) : b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = fmaf(a, c[i], -b * s[i]);
      y[i] = fmaf(a, s[i], b * c[i]);
    }
  }
}

struct RotateArgs {
  const void *x;
  void *out;                         // contiguous [B, H, N, d]
  const int32_t *pos;                // [B, N, axes], strides pos_b and pos_n
  long long sb, sh, sn;              // strides of x in numbers (d's is 1)
  long long pos_b, pos_n;
  RotaryTable t;
  int B, H, N, d;
  int heads;                         // heads per group: blockIdx.y takes [y * heads, ...)
  int back;                          // turn by -t (the gradient)
};

constexpr int kRotateThreads = 256;

// VEC: 16-byte vectors (see the host's rule); else one pair per thread, for
// any strides, alignment and number of pairs.  Numbers that stay keep their bits.
// MIXED: some unit has pairs of both kinds (interleaved, pairs no multiple of 8); a
// kernel of its own, whose kept vectors would cost the other a CTA of three on an SM.
// CTAs an SM: 8 without vectors (at 40 registers instead of 32 a head of 64 with 22
// turned took 165 us for 134), 3 with them, 2 MIXED.
template <typename T, bool VEC, bool MIXED>
__global__ void __launch_bounds__(kRotateThreads, VEC ? (MIXED ? 2 : 3) : 8)
    rotate_kernel(const __grid_constant__ RotateArgs a) {
  const int per_token = VEC ? a.d / 16 : a.d - a.t.pairs;   // units, or pairs and single numbers behind them
  const long long id = static_cast<long long>(blockIdx.x) * kRotateThreads + threadIdx.x;
  const long long token = id / per_token;
  if (token >= static_cast<long long>(a.B) * a.N) return;
  const int u = static_cast<int>(id - token * per_token);
  const int b = static_cast<int>(token / a.N), n = static_cast<int>(token - static_cast<long long>(b) * a.N);
  const int32_t *pos = a.pos + b * a.pos_b + n * a.pos_n;
  const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H);
  const T *src = static_cast<const T *>(a.x) + b * a.sb + n * a.sn;
  T *dst = static_cast<T *>(a.out) + (static_cast<size_t>(b) * a.H * a.N + n) * a.d;
  const size_t dst_h = static_cast<size_t>(a.N) * a.d;
  if constexpr (VEC) {
    const RotUnit r = rotary_unit(a.t, u);
    float c[8], s[8];
    rotary_unit_angles(a.t, r, pos, c, s);
    if (a.back) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
    auto turn = [&](RotVec<T> &vx, RotVec<T> &vy) {
      if (r.n_rot == 0) return;
      const RotVec<T> was_x = vx, was_y = vy;
      float x[8], y[8];
      vx.get(x);
      vy.get(y);
      rotary_turn(a.t.interleaved, 8, c, s, x, y);
      vx.set(x);
      vy.set(y);
      if (MIXED) {
        vx.keep(was_x, r.n_rot);
        vy.keep(was_y, r.n_rot - 4);
      }
    };
    constexpr int U = sizeof(T) == 4 ? 2 : 4;   // heads in flight
    int h = h0;
    for (; h + U <= h1; h += U) {
      RotVec<T> vx[U], vy[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        vx[i].load(src + (h + i) * a.sh + r.first);
        vy[i].load(src + (h + i) * a.sh + r.second);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        turn(vx[i], vy[i]);
        vx[i].store(dst + (h + i) * dst_h + r.first);
        vy[i].store(dst + (h + i) * dst_h + r.second);
      }
    }
    for (; h < h1; ++h) {
      RotVec<T> vx, vy;
      vx.load(src + h * a.sh + r.first);
      vy.load(src + h * a.sh + r.second);
      turn(vx, vy);
      vx.store(dst + h * dst_h + r.first);
      vy.store(dst + h * dst_h + r.second);
    }
  } else {
    if (u < a.t.pairs) {
      const int first = a.t.interleaved ? 2 * u : u, second = a.t.interleaved ? 2 * u + 1 : a.t.pairs + u;
      float c, s;
      rotary_angle(a.t, u, pos, c, s);
      c *= a.t.mag;
      s *= a.back ? -a.t.mag : a.t.mag;
      for (int h = h0; h < h1; ++h) {
        const float x = rot_get(src[h * a.sh + first]), y = rot_get(src[h * a.sh + second]);
        rot_put(dst + h * dst_h + first, fmaf(x, c, -y * s));
        rot_put(dst + h * dst_h + second, fmaf(x, s, y * c));
      }
    } else {
      const int e = a.t.pairs + u;
      for (int h = h0; h < h1; ++h) dst[h * dst_h + e] = src[h * a.sh + e];
    }
  }
}

}  // namespace mcs
