// cache_api.cu -- host side of the rotary and cache entry points of
// include/mcs.h: argument checks and launches on the caller's stream.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "../../include/mcs.h"
#include "cache_rows_kernel.cuh"
#include "cache_tile_kernel.cuh"
#include "host_shared.h"
#include "kvcache_kernels.cuh"
#include "rotary.cuh"

using namespace mcs;

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
mcs_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MCS_OK : MCS_ERR_CUDA; }
cudaStream_t cu(mcs_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kSms = 148;   // of a B200: the grids are sized for it, no result depends on it

// a kernel's dynamic shared memory limit, set once per device
template <auto *Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  const cudaError_t ge = cudaGetDevice(&dev);
  if (ge != cudaSuccess) return ge;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

mcs_status check_rotary(const mcs_rotary *r, int d, RotaryTable *t) {
  std::memset(t, 0, sizeof(*t));
  t->mag = 1.f;
  if (!r) return MCS_OK;
  if (r->pairs < 0 || 2ll * r->pairs > d || r->axes < 1) return MCS_ERR_INVALID_ARG;
  if (!(r->magnitude > 0.f) || !std::isfinite(r->magnitude)) return MCS_ERR_INVALID_ARG;
  if (r->pairs > 0 && (!r->turns || !r->axis || (reinterpret_cast<uintptr_t>(r->turns) & 7u) || !aligned4(r->axis)))
    return MCS_ERR_INVALID_ARG;
  t->turns = reinterpret_cast<const unsigned long long *>(r->turns);
  t->axis = r->axis;
  t->pairs = r->pairs;
  t->interleaved = r->interleaved != 0;
  t->axes = r->axes;
  t->mag = r->magnitude;
  return MCS_OK;
}

mcs_status check_cache(const mcs_cache *c, CacheView *v) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->page_table) return MCS_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned4(c->k_scale) || !aligned4(c->v_scale) ||
      !aligned4(c->page_table))
    return MCS_ERR_INVALID_ARG;
  if (c->B < 1 || c->H < 1 || c->n_pages < 1 || c->max_pages < 1) return MCS_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return MCS_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return MCS_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->B) * c->H > 65535) return MCS_ERR_INVALID_ARG;
  if (static_cast<long long>(c->max_pages) * c->page > (1ll << 30)) return MCS_ERR_INVALID_ARG;
  // TMA row coordinates are int32
  if (static_cast<long long>(c->n_pages) * c->H > (1ll << 31) / c->page - 1) return MCS_ERR_INVALID_ARG;
  v->k = static_cast<uint8_t *>(c->k_pages);
  v->v = static_cast<uint8_t *>(c->v_pages);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->table = c->page_table;
  v->n_pages = c->n_pages;
  v->max_pages = c->max_pages;
  v->H = c->H;
  v->page = c->page;
  v->d = c->d;
  return MCS_OK;
}

// whether [p, p + np) and [q, q + nq) have bytes in common
bool overlap(const void *p, __int128 np, const void *q, __int128 nq) {
  const __int128 a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

// ---------------------------------------------------------------- rotate
template <typename T>
cudaError_t launch_rotate(RotateArgs &a, bool vec, cudaStream_t s) {
  const long long per_token = vec ? a.d / 16 : a.d - a.t.pairs;
  const long long threads = static_cast<long long>(a.B) * a.N * per_token;
  const long long blocks = (threads + kRotateThreads - 1) / kRotateThreads;
  // A thread walks over a group of heads with one set of angles.  Few tokens:
  // smaller groups, down to one head, until the SMs have a CTA each.  (16 heads,
  // 16382 tokens: one group 15.4 us, three 17.5, eight 24.4.)
  long long groups = (kSms + blocks - 1) / blocks;
  groups = groups < 1 ? 1 : (groups > a.H ? a.H : groups);
  a.heads = static_cast<int>((a.H + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(blocks), (a.H + a.heads - 1) / a.heads);
  if (!vec)
    rotate_kernel<T, false, false><<<grid, kRotateThreads, 0, s>>>(a);
  else if (a.t.pairs % 8 == 0)
    rotate_kernel<T, true, false><<<grid, kRotateThreads, 0, s>>>(a);
  else
    rotate_kernel<T, true, true><<<grid, kRotateThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- attention over the cache
// sizes of one call: blocks of rows, and how they are computed
struct AttnPlan {
  bool rows;                     // cache_rows_kernel (blocks of 16 rows), else cache_tile_kernel (256)
  int block;                     // rows of a block
  int ctas;                      // CTAs that share the work; 0: clusters, no workspace
  int split;                     // CTAs of a cluster
};
// By sizes known here (the table's places; lengths are not):
// - Little work: clusters of 8 CTAs at most (of 16, fewer fit at once: one token
//   of 16 heads against 8000 20.7 us, of 8 16.0), as many as run at once and as
//   there can be tiles, on blocks of 16 rows.  More rows than 16 read the keys
//   once a block, but start at once: 20 rows of 16 heads against 8191 tokens take
//   15.5 us, as one block of 32 rows 26, with the tile kernel 25 and 5 of merge.
//   Both sides of the two borders, us of a call after a flush, clusters | dealt:
//   items x tiles an SM, near 28 a second round of clusters begins:
//     one token, 32 heads on 8 of 128, 32 tiles: 13.8: 28 | 37, 27.7: 41 | 50, 34.6: 61 | 56
//     one token, 8 heads of 64, 8 tiles: 27.7: 33 | 38, 31.1: 35 | 40, 34.6: 43 | 42
//     rows of 16 heads of 128, 64 tiles: 20.8: 35 | 53, 27.7: 40 | 55, 41.5: 63 | 58
//   tiles, of 16 items:
//     4 rows of 128: 32: 19 | 26, 64: 26 | 28, 96: 31 | 32, 128: 37 | 36, 192: 49 | 44
//     one row of 64: 64: 19 | 24, 128: 27 | 29, 192: 35 | 33
//     20 rows of 64: 64: 20 | 41, 128: 29 | 50, 192: 37 | 56
//   all for sequences of one length: where they differ, a cluster's share grows with
//   its own sequence, a dealt CTA's with all, so the border is below where these meet.
//   Places that are not filled count as tiles (lengths are not known here): in a table
//   of 32768, 16 heads of 64 against 300 tokens take 19.5 us dealt, in clusters 12; 20
//   rows of each of 16 items 49, in clusters 12.
// - Else 16 rows or fewer are bound by reading the keys (cache_rows_kernel: 16 rows
//   of 64 heads, 819200 tokens, 294 us; the tile kernel 467), more by the products
//   (32 rows: the tile kernel 467, blocks of 32 rows 1276).
AttnPlan plan_attention(const CacheView &c, int B, long long n_rows) {
  AttnPlan p;
  const long long tiles = (static_cast<long long>(c.max_pages) * c.page + kKeyTile - 1) / kKeyTile;
  const long long items = static_cast<long long>(B) * c.H * ((n_rows + 15) / 16);
  p.rows = true;
  p.block = 16;
  p.ctas = 2 * kSms;
  p.split = 1;
  if (tiles <= 64 && items * tiles <= 28ll * kSms) {
    // a cluster lies within one of 8 groups of 16 SMs or more: those that hold
    // whole clusters, two CTAs an SM, run all of them at once
    const long long per_group = (items + 7) / 8;
    long long split = 2 * 16 / per_group;
    split = split > kMaxRanks ? kMaxRanks : split;
    split = split > tiles ? tiles : split;
    p.split = static_cast<int>(split < 1 ? 1 : split);
    p.ctas = 0;
  } else if (n_rows > 16) {
    p.rows = false;
    p.block = 256;
    p.ctas = kSms;
  }
  return p;
}

template <int D>
cudaError_t launch_rows(CacheAttnArgs &a, const AttnPlan &p, cudaStream_t s) {
  using C = RowsCfg<D>;
  static_assert(2 * (C::SMEM + 1024) <= 233472, "two CTAs on an SM");
  if (p.ctas) {
    const cudaError_t e = allow_smem<cache_rows_kernel<D, false>>(C::SMEM);
    if (e != cudaSuccess) return e;
    cache_rows_kernel<D, false><<<p.ctas, C::THREADS, C::SMEM, s>>>(a);
    return cudaGetLastError();
  }
  const cudaError_t e = allow_smem<cache_rows_kernel<D, true>>(C::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.split), static_cast<unsigned>(a.s.B * a.s.H),
                     static_cast<unsigned>(a.s.n_blocks));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(p.split);
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_rows_kernel<D, true>, a);
}

template <int D>
cudaError_t launch_tile(CacheAttnArgs &a, const AttnPlan &p, cudaStream_t s) {
  using C = TileCfg<D>;
  const cudaError_t e = allow_smem<cache_tile_kernel<D>>(C::SMEM);
  if (e != cudaSuccess) return e;
  cache_tile_kernel<D><<<p.ctas, C::THREADS, C::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_attention(CacheAttnArgs &a, const AttnPlan &p, cudaStream_t s) {
  return p.rows ? launch_rows<D>(a, p, s) : launch_tile<D>(a, p, s);
}

template <int D>
cudaError_t launch_merge(const CacheAttnArgs &a, const AttnPlan &p, cudaStream_t s) {
  MergeArgs m;
  std::memset(&m, 0, sizeof(m));
  m.m = a.m;
  m.O = a.O;
  m.lse = a.lse;
  m.H = a.s.H;
  m.Nq = a.s.Nq;
  m.share = a.s.share;
  m.n_rows = a.s.n_rows;
  m.rows = p.block;
  // four parts an item, or more: split them
  const long long items = static_cast<long long>(a.s.B) * a.s.H * a.s.n_blocks;
  const int rows = a.s.n_rows < p.block ? a.s.n_rows : p.block;
  const int at_once = kMergeThreads / (D / 4);
  if (4 * items <= p.ctas)
    cache_merge_kernel<D, true><<<dim3(p.ctas, (rows + 7) / 8 * (D / 16)), kMergeThreads, 0, s>>>(m);
  else
    cache_merge_kernel<D, false><<<dim3(p.ctas, (rows + at_once - 1) / at_once), kMergeThreads, 0, s>>>(m);
  return cudaGetLastError();
}

}  // namespace

// ---------------------------------------------------------------- the C ABI
extern "C" {

mcs_status mcs_rotate(const void *x, int dtype, int B, int H, int N, int d, const int64_t *strides,
                      const int32_t *positions, int64_t pos_stride_b, int64_t pos_stride_n, const mcs_rotary *rotary,
                      int back, void *out, mcs_stream_t stream) {
  if (!rotary || !strides || B < 0 || H < 0 || N < 0 || d < 1) return MCS_ERR_INVALID_ARG;
  if (dtype != MCS_BF16 && dtype != MCS_FP16 && dtype != MCS_FP32) return MCS_ERR_UNSUPPORTED;
  RotateArgs a;
  std::memset(&a, 0, sizeof(a));
  const mcs_status st = check_rotary(rotary, d, &a.t);
  if (st != MCS_OK) return st;
  if (B == 0 || H == 0 || N == 0) return MCS_OK;
  if (!x || !out || !positions || !aligned4(positions)) return MCS_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > INT_MAX || H > INT_MAX / d) return MCS_ERR_INVALID_ARG;
  if (static_cast<double>(B) * N * d > 5e11) return MCS_ERR_INVALID_ARG;   // the grid's x is below 2^31 blocks
  const int elt = dtype == MCS_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % elt || reinterpret_cast<uintptr_t>(out) % elt) return MCS_ERR_INVALID_ARG;
  a.x = x;
  a.out = out;
  a.pos = positions;
  a.pos_b = pos_stride_b;
  a.pos_n = pos_stride_n;
  // a dimension of one entry has no stride
  a.sb = B > 1 ? strides[0] : 0;
  a.sh = H > 1 ? strides[1] : 0;
  a.sn = N > 1 ? strides[2] : 0;
  a.B = B;
  a.H = H;
  a.N = N;
  a.d = d;
  a.back = back != 0;
  // out over x: in place only, where every thread reads the numbers it writes first
  const bool same = x == out && (N == 1 || a.sn == d) && (H == 1 || a.sh == static_cast<long long>(N) * d) &&
                    (B == 1 || a.sb == static_cast<long long>(H) * N * d);
  __int128 lo = 0, hi = d;   // the numbers of x: [lo, hi)
  for (const __int128 reach : {static_cast<__int128>(B - 1) * a.sb, static_cast<__int128>(H - 1) * a.sh,
                               static_cast<__int128>(N - 1) * a.sn})
    (reach < 0 ? lo : hi) += reach;
  const uint8_t *first = static_cast<const uint8_t *>(x) + static_cast<ptrdiff_t>(lo * elt);
  if (!same && overlap(first, (hi - lo) * elt, out, static_cast<__int128>(B) * H * N * d * elt))
    return MCS_ERR_INVALID_ARG;
  // 16-byte vectors need whole units of 16 numbers and aligned rows
  const bool vec = d % 16 == 0 && (a.t.interleaved || a.t.pairs % 8 == 0) && aligned16(x) && aligned16(out) &&
                   a.sb * elt % 16 == 0 && a.sh * elt % 16 == 0 && a.sn * elt % 16 == 0;
  const cudaError_t e = dtype == MCS_FP32   ? launch_rotate<float>(a, vec, cu(stream))
                        : dtype == MCS_FP16 ? launch_rotate<__half>(a, vec, cu(stream))
                                            : launch_rotate<bf16>(a, vec, cu(stream));
  return cuda_status(e);
}

mcs_status mcs_cache_append(const mcs_cache *cache, const void *K, const void *V, const int64_t *k_strides,
                            const int64_t *v_strides, int n, const int32_t *start, const int32_t *counts,
                            const int32_t *positions, int64_t pos_stride_b, int64_t pos_stride_n,
                            const mcs_rotary *rotary, mcs_stream_t stream) {
  AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  mcs_status st = check_cache(cache, &a.c);
  if (st != MCS_OK) return st;
  st = check_rotary(rotary, a.c.d, &a.t);
  if (st != MCS_OK) return st;
  if (n < 0 || !k_strides || !v_strides) return MCS_ERR_INVALID_ARG;
  if (!a.t.interleaved && a.t.pairs % 8 != 0) return MCS_ERR_UNSUPPORTED;
  if (!positions && a.t.pairs > 0 && a.t.axes != 1) return MCS_ERR_INVALID_ARG;
  if (n == 0) return MCS_OK;
  if (!K || !V || !start || !aligned16(K) || !aligned16(V) || !aligned4(start) || !aligned4(counts) ||
      !aligned4(positions))
    return MCS_ERR_INVALID_ARG;
  if (n > (1 << 30) || a.c.H > 65535 || cache->B > 65535) return MCS_ERR_INVALID_ARG;
  const int sizes[3] = {cache->B, a.c.H, n};
  long long ks[3], vs[3];
  for (int i = 0; i < 3; ++i) {
    ks[i] = sizes[i] > 1 ? k_strides[i] : 0;
    vs[i] = sizes[i] > 1 ? v_strides[i] : 0;
    if (ks[i] % 8 || vs[i] % 8) return MCS_ERR_INVALID_ARG;   // rows on 16-byte boundaries
  }
  a.K = static_cast<const bf16 *>(K);
  a.V = static_cast<const bf16 *>(V);
  a.k_sb = ks[0], a.k_sh = ks[1], a.k_sn = ks[2];
  a.v_sb = vs[0], a.v_sh = vs[1], a.v_sn = vs[2];
  a.start = start;
  a.counts = counts;
  a.pos = positions;
  a.pos_b = pos_stride_b;
  a.pos_n = pos_stride_n;
  a.n = n;
  if (!(a.status = device_status_word())) return MCS_ERR_CUDA;
  // n tokens reach into ceil((n - 1) / page) + 1 pages at most
  const dim3 grid((n + a.c.page - 2) / a.c.page + 1, a.c.H, cache->B);
  const int units = a.c.page * (a.c.d / 16);
  const int threads = units < kAppendThreads ? units : kAppendThreads;
  if (units <= kAppendThreads)
    append_kernel<1><<<grid, threads, 0, cu(stream)>>>(a);
  else
    append_kernel<2><<<grid, threads, 0, cu(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

mcs_status mcs_cache_read(const mcs_cache *cache, const int32_t *start, const int32_t *counts, int n, void *K, void *V,
                          mcs_stream_t stream) {
  ReadArgs a;
  std::memset(&a, 0, sizeof(a));
  const mcs_status st = check_cache(cache, &a.c);
  if (st != MCS_OK) return st;
  if (n < 0) return MCS_ERR_INVALID_ARG;
  if (n == 0) return MCS_OK;
  if (!K || !V || !start || !aligned16(K) || !aligned16(V) || !aligned4(start) || !aligned4(counts))
    return MCS_ERR_INVALID_ARG;
  a.start = start;
  a.counts = counts;
  a.K = static_cast<bf16 *>(K);
  a.V = static_cast<bf16 *>(V);
  a.n = n;
  a.page_shift = a.c.page == 16 ? 4 : a.c.page == 32 ? 5 : a.c.page == 64 ? 6 : 7;
  const long long units = static_cast<long long>(n) * (a.c.d / 16);
  const int threads = units < kReadThreads ? static_cast<int>((units + 31) / 32 * 32) : kReadThreads;
  const long long blocks = (units + threads - 1) / threads;
  if (blocks > INT_MAX) return MCS_ERR_INVALID_ARG;
  if (!(a.status = device_status_word())) return MCS_ERR_CUDA;
  cache_read_kernel<<<dim3(static_cast<unsigned>(blocks), a.c.H, cache->B), threads, 0, cu(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

size_t mcs_cache_attention_workspace_size(const mcs_cache *cache, int Hq, int Nq) {
  CacheView c;
  if (check_cache(cache, &c) != MCS_OK || Hq < 1 || Hq % c.H != 0 || Nq < 0) return 0;
  const long long n_rows = static_cast<long long>(Nq) * (Hq / c.H);
  if (n_rows == 0 || n_rows > (1 << 20)) return 0;
  const AttnPlan p = plan_attention(c, cache->B, n_rows);
  return p.ctas ? merge_space(p.ctas, p.block, c.d, nullptr, nullptr) : 0;
}

mcs_status mcs_cache_attention(const mcs_cache *cache, const void *Q, int Hq, int Nq, const int32_t *lengths,
                               const int32_t *counts, int causal, float scale, void *O, float *lse, void *workspace,
                               size_t workspace_bytes, mcs_stream_t stream) {
  CacheAttnArgs a;
  std::memset(&a, 0, sizeof(a));
  const mcs_status st = check_cache(cache, &a.c);
  if (st != MCS_OK) return st;
  if (Hq < 1 || Hq % a.c.H != 0 || Nq < 0) return MCS_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MCS_ERR_INVALID_ARG;
  if (Nq == 0) return MCS_OK;
  if (!Q || !O || !lengths || !aligned16(Q) || !aligned16(O) || !aligned4(lengths) || !aligned4(counts) || !aligned4(lse))
    return MCS_ERR_INVALID_ARG;
  const long long n_rows = static_cast<long long>(Nq) * (Hq / a.c.H);
  if (n_rows > (1 << 20)) return MCS_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return MCS_ERR_INVALID_ARG;
  const __int128 bytes = static_cast<__int128>(cache->B) * Hq * Nq * a.c.d * 2;
  if (overlap(Q, bytes, O, bytes)) return MCS_ERR_INVALID_ARG;
  if (!(a.status = device_status_word())) return MCS_ERR_CUDA;
  const AttnPlan p = plan_attention(a.c, cache->B, n_rows);
  if (p.ctas) {
    if (!workspace || workspace_bytes < merge_space(p.ctas, p.block, a.c.d, nullptr, nullptr)) return MCS_ERR_WORKSPACE;
    merge_space(p.ctas, p.block, a.c.d, workspace, &a.m);
  }
  a.Q = static_cast<const bf16 *>(Q);
  a.O = static_cast<bf16 *>(O);
  a.lse = lse;
  a.s.lengths = lengths;
  a.s.counts = counts;
  a.s.B = cache->B;
  a.s.H = a.c.H;
  a.s.Nq = Nq;
  a.s.share = Hq / a.c.H;
  a.s.causal = causal != 0;
  a.s.cap = a.c.max_pages * a.c.page;
  a.s.n_rows = static_cast<int>(n_rows);
  a.s.n_blocks = static_cast<int>((n_rows + p.block - 1) / p.block);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.wait_ns = wait_limit_ns();
  const size_t rows = static_cast<size_t>(a.c.n_pages) * a.c.H * a.c.page;
  if (!map_byte_rows(&a.tmK, a.c.k, a.c.d, rows, a.c.page) || !map_byte_rows(&a.tmV, a.c.v, a.c.d, rows, a.c.page))
    return MCS_ERR_CUDA;
  cudaError_t e = a.c.d == 64 ? launch_attention<64>(a, p, cu(stream)) : launch_attention<128>(a, p, cu(stream));
  if (e == cudaSuccess && p.ctas) e = a.c.d == 64 ? launch_merge<64>(a, p, cu(stream)) : launch_merge<128>(a, p, cu(stream));
  return cuda_status(e);
}

}  // extern "C"
