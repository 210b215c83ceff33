// Log probabilities of given tokens, the entropy of each row's distribution and its most probable tokens, with the
// gradient of the first two.  Per row, with z = scale·x:
//   M = max x,  S = Σ_v exp(z_v − scale·M),  log p_v = z_v − scale·M − ln S,
//   logp = log p_token,  H = −Σ_v p_v log p_v = ln S − Σ_v p_v (z_v − scale·M),
//   dx_v = scale·(dlogp·([v = token] − p_v) − dH·p_v·(log p_v + H)).
//
// Forward.  One pass over the logits.  A thread keeps the sums Σ 2^t and Σ t·2^t of its elements, t = x·scale·log2(e) − b,
// against a base b of its own: the largest t of the first elements it saw, moved only where a later one lies more than
// kHeadroom above it (2^t has room for that in float32, so that almost no element pays for a rescaling, and
// Σ t·2^t / Σ 2^t loses at most kHeadroom·2⁻²⁴).  The threads' sums meet at the largest base.  What this path cannot hold (a largest logit beyond
// 2⁻¹·FLT_MAX in t, below −1e30, or no finite sum) is done over by row_safe(), two passes with differences taken first.
//
// The most probable tokens: a warp takes 512 neighbouring bytes at a time and one of its lanes in turn keeps the largest of
// these groups' maxima (a maximum over the warp, one instruction).  The k-th largest of the lanes' maxima bounds the k-th
// largest element from below, and the elements above it lie with the k lanes whose maxima reach it, so only those lanes'
// groups are read again (whole lines; with a thread's own vectors, 4 KB apart, it was 40 % more bytes out of HBM at
// 128256 logits and 20 alternatives), filtered by their vectors' maxima, and the few elements at or above the bound are put
// in order.  Elements are ordered by (value, lower index first) throughout, so that ties have one answer, and no step
// depends on timing.
//
// Bound by HBM: a logit is read once (backward: read and written).  On one GB300: 8192 x 50304 bf16 forward 142 us (5.8 TB/s),
// backward 258 us (6.4 TB/s); 4096 x 128256 with 20 alternatives 213 us (4.9 TB/s; 163 without: a quarter more instructions and 14
// block barriers at a row's end, six for either merge of the warps' lists, during which its block loads nothing); 3 x 50257 with
// 5 alternatives 7.5 us.  Six blocks per SM of 40 registers with four vectors in flight: fewer blocks or more vectors were 2 to 10 %
// slower.
#include <cfloat>
#include <cstring>

#include "internal.cuh"

namespace xt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;          // a list lives in one warp, an entry per lane
constexpr float kHeadroom = 8.f;     // log2 units
constexpr float kLowest = -200.f;    // 2^kLowest is 0 in float32, and 0·kLowest stays 0 where 0·(−∞) would not
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 16 bytes of logits: the float values and their maximum (NaN ignored).
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  static constexpr int W = 4;
  __device__ __forceinline__ static void values(const uint4& q, float (&x)[4]) {
    x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y); x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
  }
  __device__ __forceinline__ static float top(const uint4& q) {
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
};
template <> struct Chunk<bf16> {
  static constexpr int W = 8;
  __device__ __forceinline__ static void values(const uint4& q, float (&x)[8]) { Vec<bf16>::unpack(q, x); }
  __device__ __forceinline__ static float top(const uint4& q) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
};

// A row as 16-byte vectors: `head` elements before the first 16-byte boundary, `full` whole vectors, then the tail.
// Vectors are numbered 0 (head), 1 .. full, full + 1 (tail); element e of whole vector j is head + (j − 1)·W + e.
template <typename T>
struct Row {
  const T* x;
  int64_t V;
  int head;
  int64_t full;
  __device__ __forceinline__ Row(const T* p, int64_t V_) : x(p), V(V_) {
    const int64_t h = int64_t((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int64_t(sizeof(T));
    head = int(h < V ? h : V);
    full = (V - head) / Chunk<T>::W;
  }
  __device__ __forceinline__ const T* vector(int64_t j) const { return x + head + (j - 1) * Chunk<T>::W; }
  // first element of vector j and one past its last
  __device__ __forceinline__ int64_t first(int64_t j) const { return j == 0 ? 0 : head + (j - 1) * Chunk<T>::W; }
  __device__ __forceinline__ int64_t last(int64_t j) const {
    return j == 0 ? head : j <= full ? head + j * Chunk<T>::W : V;
  }
};

struct Sums {
  float b;         // base of the exponents, log2 units
  uint64_t s, w;   // Σ 2^t and Σ t·2^t, two partial sums each
  float top;       // largest element
};

__device__ __forceinline__ void rebase(Sums& a, float nb) {
  const float d = fmaxf(a.b - nb, kLowest), r = ex2(d);
  float s0, s1, w0, w1;
  f32x2_unpack(a.s, s0, s1);
  f32x2_unpack(a.w, w0, w1);
  a.w = f32x2_pack(r * fmaf(d, s0, w0), r * fmaf(d, s1, w1));
  a.s = f32x2_pack(r * s0, r * s1);
  a.b = nb;
}

template <int N>
__device__ __forceinline__ void consume(Sums& a, const float (&x)[N], float top, float c) {
  a.top = fmaxf(a.top, top);
  if (top * c > a.b + kHeadroom) rebase(a, top * c);
  const uint64_t cc = f32x2_pack(c, c), nb = f32x2_pack(-a.b, -a.b);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float t0, t1;
    f32x2_unpack(f32x2_fma(f32x2_pack(x[i], x[i + 1]), cc, nb), t0, t1);
    t0 = max_nan(t0, kLowest);
    t1 = max_nan(t1, kLowest);
    const uint64_t e = f32x2_pack(ex2(t0), ex2(t1));
    a.s = f32x2_add(a.s, e);
    a.w = f32x2_fma(e, f32x2_pack(t0, t1), a.w);
  }
}

// ------------------------------------------------------------------------------ lists of the most probable
// An element's place in the order: larger values first, among equal ones the lower number.  0 stands for none.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // −0 as +0
  return v != v ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t order(float v, uint32_t number) {
  const uint32_t k = order_key(v);
  return k ? (uint64_t(k) << 32) | uint32_t(~number) : 0ull;
}

// The warp's 32 entries in falling order (bitonic network).
__device__ __forceinline__ uint64_t sort_warp(uint64_t v, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) {
      const uint64_t o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool up = (lane & k) != 0 && k < 32, lower = (lane & j) != 0;
      v = (v > o) == (up == lower) ? v : o;
    }
  return v;
}
// The 32 largest of two lists in falling order, in falling order.
__device__ __forceinline__ uint64_t merge_warp(uint64_t a, uint64_t b, int lane) {
  b = __shfl_sync(0xffffffffu, b, 31 - lane);
  uint64_t v = a > b ? a : b;
#pragma unroll
  for (int j = 16; j > 0; j /= 2) {
    const uint64_t o = __shfl_xor_sync(0xffffffffu, v, j);
    v = (v > o) == ((lane & j) == 0) ? v : o;
  }
  return v;
}
__device__ __forceinline__ uint64_t insert_warp(uint64_t list, uint64_t c, int lane) {
  const int pos = __popc(__ballot_sync(0xffffffffu, list > c));
  const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
  return lane < pos ? list : lane == pos ? c : up;
}

__device__ __forceinline__ float order_value(uint64_t o) {
  const uint32_t k = uint32_t(o >> 32);
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Puts the elements at or above `bound` of the lanes' vectors (number j; none where j < 0; `group`: the number that the bound
// orders them by) into the warp's list: lanes whose maximum reaches the bound hand their 16 bytes round.
template <typename T>
__device__ __forceinline__ uint64_t collect(uint64_t list, const Row<T>& row, int64_t j, uint32_t group, uint64_t bound,
                                            int lane) {
  constexpr int W = Chunk<T>::W;
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  int n = 0;
  float top = -INFINITY;
  if (j >= 0) {
    n = int(row.last(j) - row.first(j));
    if (n == W && j > 0) {
      q = *reinterpret_cast<const uint4*>(row.vector(j));
      top = Chunk<T>::top(q);
    } else {
      T v[W];
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = i < n ? row.x[row.first(j) + i] : from_f<T>(-INFINITY);
      memcpy(&q, v, 16);
      top = Chunk<T>::top(q);
    }
  }
  uint32_t some = __ballot_sync(0xffffffffu, n > 0 && order(top, group) >= bound);
  while (some) {
    const int from = __ffs(some) - 1;
    some &= some - 1;
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, q.x, from);
    o.y = __shfl_sync(0xffffffffu, q.y, from);
    o.z = __shfl_sync(0xffffffffu, q.z, from);
    o.w = __shfl_sync(0xffffffffu, q.w, from);
    const int count = __shfl_sync(0xffffffffu, n, from);
    const uint32_t jj = uint32_t(__shfl_sync(0xffffffffu, int(j), from)), gg = __shfl_sync(0xffffffffu, group, from);
    float v[W], mine = 0.f;
    Chunk<T>::values(o, v);
#pragma unroll
    for (int i = 0; i < W; ++i) mine = lane == i ? v[i] : mine;
    uint64_t c = 0;
    if (lane < count && order(mine, gg) >= bound) c = order(mine, uint32_t(row.first(jj) + lane));
    uint32_t hits = __ballot_sync(0xffffffffu, c != 0);
    while (hits) {
      const int l = __ffs(hits) - 1;
      hits &= hits - 1;
      list = insert_warp(list, __shfl_sync(0xffffffffu, c, l), lane);
    }
  }
  return list;
}

// The largest entries of N warps' lists, in falling order, merged pair by pair; the result is warp 0's return value.
template <int N>
__device__ __forceinline__ uint64_t merge_lists(uint64_t (*lists)[32], uint64_t mine, int warp, int lane) {
#pragma unroll
  for (int s = 1; s < N; s *= 2) {
    lists[warp][lane] = mine;
    __syncthreads();
    if (warp % (2 * s) == 0 && warp + s < N) mine = merge_warp(mine, lists[warp + s][lane], lane);
    __syncthreads();
  }
  return mine;
}

struct Fwd {
  const void* x;
  int64_t ld, rows, V;
  const int32_t* tokens;
  float scale, c;   // c = scale·log2(e)
  int top;
  float *logp, *entropy, *stats, *top_logp;
  int32_t* top_ids;
  uint32_t* flag;
};

// The row's results from M, log2 Σ 2^(c(x − M)) and Σ p·c(x − M) (log2 units), by the lane that holds the row's token and
// its logit.
__device__ __forceinline__ void write_row(const Fwd& a, int64_t r, bool valid, float given, float M, double log2s,
                                          double mean) {
  const bool ok = isfinite(M) && isfinite(log2s) && isfinite(mean);
  const float nan = __int_as_float(0x7fc00000);
  const double ln2 = 0.69314718055994530942;
  if (!valid) flag_error(a.flag, XT_DEVERR_INDEX);
  const double z = (double(given) - double(M)) * double(a.scale);
  a.logp[r] = ok && valid ? float(z - log2s * ln2) : nan;
  if (a.entropy) a.entropy[r] = ok ? float(fmax((log2s - mean) * ln2, 0.0)) : nan;
  if (a.stats) {
    a.stats[2 * r] = ok ? M : nan;
    a.stats[2 * r + 1] = ok ? float(log2s * ln2) : nan;
  }
}
// The list's entries: one lane each.
__device__ __forceinline__ void write_top(const Fwd& a, int64_t r, uint64_t list, int lane, float M, double log2s) {
  if (lane >= a.top) return;
  const bool ok = isfinite(M) && isfinite(log2s);
  const double z = (double(order_value(list)) - double(M)) * double(a.scale) - log2s * 0.69314718055994530942;
  a.top_logp[r * a.top + lane] = ok ? float(z) : __int_as_float(0x7fc00000);
  a.top_ids[r * a.top + lane] = ok ? int32_t(~uint32_t(list)) : -1;
}

// The sums of one row by one warp, differences taken before they are scaled, double sums: any finite logits.
template <typename T>
__device__ __noinline__ void row_safe(const T* x, int64_t V, float scale, int lane, float& M, double& log2s,
                                      double& mean) {
  float m = -INFINITY;
  for (int64_t v = lane; v < V; v += 32) m = max_nan(m, to_f(x[v]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  double s = 0, w = 0;
  for (int64_t v = lane; v < V; v += 32) {
    const float t = max_nan(float((double(to_f(x[v])) - double(m)) * double(scale)) * kLog2e, kLowest);
    const float e = exp2f(t);
    s += double(e);
    w += double(e) * double(t);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    w += __shfl_xor_sync(0xffffffffu, w, o);
  }
  M = m;
  log2s = log2(s);
  mean = w / s;
}

// Sums over the warp at its largest base.
__device__ __forceinline__ void warp_join(float& b, float& s, float& w) {
  const float B = warp_max(b), d = fmaxf(b - B, kLowest), r = ex2(d);
  w = warp_sum(r * fmaf(d, s, w));
  s = warp_sum(r * s);
  b = B;
}

// log2 Σ 2^(c(x − M)) of sums to the base b.  The largest element's own term is 1, so it is nought at least: what the
// exponential rounded off would leave probabilities above 1.  (NaN stays.)
__device__ __forceinline__ double log2_sum(float b, float s, float M, float c) {
  const double l = double(log2f(s)) + (double(b) - double(M) * double(c));
  return l < 0 ? 0 : l;
}

// WARP: a warp to a row (short rows); else a CTA, or with gridDim.x a multiple of the cluster size a cluster of CTAs
// that share the row's vectors out in ranges and join in the first one's shared memory.
template <typename T, bool TOP, bool WARP>
__global__ void __launch_bounds__(kThreads, 6) token_logprobs_kernel(const __grid_constant__ Fwd a) {
  constexpr int W = Chunk<T>::W;
  constexpr int kUnroll = 4;
  constexpr int NT = WARP ? 32 : kThreads;  // threads that share the vectors
  constexpr int kMaxCluster = 8;
  __shared__ float part[3][kMaxCluster * kWarps];  // base, Σ, Σ t of every warp of the cluster (in its first CTA)
  __shared__ float part_top[kMaxCluster * kWarps];
  __shared__ uint64_t lists[TOP && !WARP ? kWarps : 1][32];
  __shared__ uint64_t cluster_lists[TOP && !WARP ? kMaxCluster : 1][32];  // of every CTA (in the first one)
  __shared__ uint64_t chosen[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = WARP ? lane : int(threadIdx.x);
  uint32_t rank = 0, cl = 1;
  if (!WARP) {
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
  }
  // the other CTAs are running before anything is stored into the first one
  if (!WARP && cl > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_begin();
  const int64_t r = WARP ? int64_t(blockIdx.x) * kWarps + warp : int64_t(blockIdx.x) / cl;
  if (WARP && r >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + r * a.ld;
  const Row<T> row(x, a.V);
  // the token's logit, on its way while the row is read
  int32_t token = -1;
  float given = 0.f;
  if (lane == 0 && (WARP || warp == 0)) {
    token = __ldg(a.tokens + r);
    if (token >= 0 && token < a.V) given = to_f(x[token]);
  }
  const bool valid = token >= 0 && token < a.V;
  // this CTA's whole vectors: (lo, hi], numbers 1 .. full
  const int64_t lo = WARP ? 0 : row.full * rank / cl, hi = WARP ? row.full : row.full * (rank + 1) / cl;

  Sums m{-1e30f, 0ull, 0ull, -INFINITY};
  // Groups (a CTA's rows with alternatives): the 32 neighbouring vectors that a warp takes together, 512 bytes, numbered
  // 1 + 8·turn + warp in the row's order.  Lane t keeps the largest of its warp's groups of turns t, t + 32, ...
  constexpr bool GROUPS = TOP && !WARP;
  // A warp's rows: each lane keeps two, of its even and of its odd vectors (the k-th largest of 64 bounds better than that
  // of 32: 50000 x 4000 with 32 alternatives 792 us with one).
  constexpr bool PAIRS = TOP && WARP;
  uint32_t best_key = 0, best_group = 0, turn = 0;
  float pair_top[2] = {-INFINITY, -INFINITY};
  uint32_t pair_at[2] = {uint32_t(lo + 1 + tid), uint32_t(lo + 1 + tid + NT)};
  bool pair_any[2] = {lo + tid < hi, lo + tid + NT < hi};
  auto take = [&](const uint4& q, int64_t j, bool in, int odd) {
    const float top = Chunk<T>::top(q);
    if constexpr (GROUPS) {
      const uint32_t key = __reduce_max_sync(0xffffffffu, in ? order_key(top) : 0u);
      if (lane == int(turn & 31) && key > best_key) {
        best_key = key;
        best_group = 1 + turn * kWarps + warp;
      }
      ++turn;
    }
    if (!in) return;
    if constexpr (PAIRS) {
      const bool more = top > pair_top[odd];
      pair_top[odd] = more ? top : pair_top[odd];
      pair_at[odd] = more ? uint32_t(j) : pair_at[odd];
    }
    float v[W];
    Chunk<T>::values(q, v);
    consume<W>(m, v, top, a.c);
  };
  const T* p = row.vector(lo + 1 + tid);
  int64_t j = lo + 1 + tid;
  for (; j - lane + 31 + (kUnroll - 1) * NT <= hi; j += kUnroll * NT, p += kUnroll * NT * W) {  // the same for the whole warp
    uint4 q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) q[u] = load_stream(p + u * NT * W);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) take(q[u], j + u * NT, true, u & 1);
  }
  {  // what is left, all of it in flight at once
    uint4 q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (j + u * NT <= hi) q[u] = load_stream(p + u * NT * W);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (j - lane + u * NT > hi) break;
      take(q[u], j + u * NT, j + u * NT <= hi, u & 1);
    }
  }
  // the elements beside the whole vectors: the head with thread 0 of the first CTA, the tail with the last thread of
  // the last one (whose vectors they follow, so that the first of equal values is kept)
  const int64_t tail = row.full + 1;
  const bool has_head = rank == 0 && tid == 0 && row.head > 0;
  const bool has_tail = rank == cl - 1 && tid == NT - 1 && row.first(tail) < a.V;
  if (has_head || has_tail) {
    const int64_t k = has_head ? 0 : tail;
    float v[W], top = -INFINITY;
    const int64_t e0 = row.first(k);
    const int n = int(row.last(k) - e0);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      v[i] = i < n ? to_f(x[e0 + i]) : -INFINITY;
      top = fmaxf(top, v[i]);
    }
    if constexpr (GROUPS) {
      // the head, group 0, comes before what the lane has seen, the tail after it
      const uint32_t key = order_key(top), group = has_head ? 0u : ~0u - 1u;
      if (key > best_key || (has_head && key == best_key)) {
        best_key = key;
        best_group = group;
      }
    } else if constexpr (PAIRS) {
      // the head comes before the lane's even vectors, the tail after its odd ones
      const int h = has_head ? 0 : 1;
      if (!pair_any[h] || top > pair_top[h] || (has_head && top == pair_top[h])) {
        pair_top[h] = top;
        pair_at[h] = uint32_t(k);
      }
      pair_any[h] = true;
    }
    consume<W>(m, v, top, a.c);
  }

  float b = m.b, s0, s1, w0, w1;
  f32x2_unpack(m.s, s0, s1);
  f32x2_unpack(m.w, w0, w1);
  float s = s0 + s1, w = w0 + w1, M = warp_max(m.top);
  warp_join(b, s, w);
  uint64_t list = 0;

  if constexpr (WARP) {
    double log2s = log2_sum(b, s, M, a.c);
    double mean = double(w / s) + (double(b) - double(M) * double(a.c));
    if (!(s > 0.f && s < FLT_MAX) || !isfinite(M) || !isfinite(w)) row_safe(x, a.V, a.scale, lane, M, log2s, mean);
    if (lane == 0) write_row(a, r, valid, given, M, log2s, mean);
    if constexpr (TOP) {
      const uint64_t even = sort_warp(pair_any[0] ? order(pair_top[0], pair_at[0]) : 0ull, lane);
      const uint64_t odd = sort_warp(pair_any[1] ? order(pair_top[1], pair_at[1]) : 0ull, lane);
      const uint64_t bound = __shfl_sync(0xffffffffu, merge_warp(even, odd, lane), a.top - 1);
      // vectors are few here: all of them are looked through
      for (int64_t j0 = 0; j0 <= tail; j0 += 32) {
        const int64_t jj = j0 + lane;
        list = collect(list, row, jj <= tail ? jj : -1, uint32_t(jj), bound, lane);
      }
      write_top(a, r, list, lane, M, log2s);
    }
    return;
  }

  // ---- the CTA's most probable elements
  if constexpr (TOP) {
    const uint64_t best = best_key ? (uint64_t(best_key) << 32) | uint32_t(~best_group) : 0ull;
    const uint64_t all = merge_lists<kWarps>(lists, sort_warp(best, lane), warp, lane);
    if (warp == 0) chosen[lane] = all;
    __syncthreads();
    const uint64_t bound = chosen[a.top - 1];
    // a warp to a chosen lane: all the groups that its maximum is taken over
    for (int k = warp; k < a.top; k += kWarps) {
      const uint64_t ch = chosen[k];
      if (ch == 0) break;
      const uint32_t group = ~uint32_t(ch);
      const bool head = group == 0, end = group == ~0u - 1u;
      const int ow = head ? 0 : end ? kWarps - 1 : int((group - 1) % kWarps);
      const uint32_t ol = head ? 0 : end ? 31 : (group - 1) / kWarps % 32;
      for (int64_t t = ol;; t += 32) {
        const int64_t j0 = lo + 1 + (t * kWarps + ow) * 32;
        if (j0 > hi) break;
        list = collect(list, row, j0 + lane <= hi ? j0 + lane : -1, uint32_t(1 + t * kWarps + ow), bound, lane);
      }
      if (ow == 0 && ol == 0 && rank == 0 && row.head > 0) list = collect(list, row, lane == 0 ? 0 : -1, 0u, bound, lane);
      if (ow == kWarps - 1 && ol == 31 && rank == cl - 1 && row.first(tail) < a.V)
        list = collect(list, row, lane == 0 ? tail : -1, ~0u - 1u, bound, lane);
    }
    list = merge_lists<kWarps>(lists, list, warp, lane);
  }

  // ---- the warps' sums and the CTAs' lists meet in the first CTA of the cluster
  const int slot = int(rank) * kWarps + warp;
  if (cl > 1) {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    auto at0 = [](const void* p) {
      uint32_t d;
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(d) : "r"(uint32_t(__cvta_generic_to_shared(p))));
      return d;
    };
    if (lane == 0) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at0(&part[0][slot])), "f"(b) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at0(&part[1][slot])), "f"(s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at0(&part[2][slot])), "f"(w) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at0(&part_top[slot])), "f"(M) : "memory");
    }
    if constexpr (TOP)
      if (warp == 0)
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at0(&cluster_lists[rank][lane])), "l"(list) : "memory");
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    if (rank != 0) return;
    if constexpr (TOP) list = merge_lists<kWarps>(lists, warp < int(cl) ? cluster_lists[warp][lane] : 0ull, warp, lane);
  } else {
    if (lane == 0) {
      part[0][slot] = b;
      part[1][slot] = s;
      part[2][slot] = w;
      part_top[slot] = M;
    }
    __syncthreads();
  }
  if (warp != 0) return;
  const int n = int(cl) * kWarps;  // ≤ 64: two slots to a lane, joined in slot order by the shuffles' fixed tree
  b = lane < n ? part[0][lane] : -1e30f;
  s = lane < n ? part[1][lane] : 0.f;
  w = lane < n ? part[2][lane] : 0.f;
  M = lane < n ? part_top[lane] : -INFINITY;
  if (lane + 32 < n) {
    const float b2 = part[0][lane + 32], s2 = part[1][lane + 32], w2 = part[2][lane + 32];
    const float B = fmaxf(b, b2), d1 = fmaxf(b - B, kLowest), d2 = fmaxf(b2 - B, kLowest);
    w = ex2(d1) * fmaf(d1, s, w) + ex2(d2) * fmaf(d2, s2, w2);
    s = ex2(d1) * s + ex2(d2) * s2;
    b = B;
    M = fmaxf(M, part_top[lane + 32]);
  }
  M = warp_max(M);
  warp_join(b, s, w);
  double log2s = log2_sum(b, s, M, a.c);
  double mean = double(w / s) + (double(b) - double(M) * double(a.c));
  if (!(s > 0.f && s < FLT_MAX) || !isfinite(M) || !isfinite(w)) row_safe(x, a.V, a.scale, lane, M, log2s, mean);
  if (lane == 0) write_row(a, r, valid, given, M, log2s, mean);
  if constexpr (TOP) write_top(a, r, list, lane, M, log2s);
}

// ------------------------------------------------------------------------------ backward

struct Bwd {
  const void* x;
  int64_t ld;
  const int32_t* tokens;
  const float *stats, *entropy, *d_logp, *d_entropy;
  float scale, c;
  void* dx;
  int64_t ld_d, rows, V;
  int segs;         // pieces of a row, loops·kSegVectors vectors for each lane
  int loops, acc;
  uint32_t* flag;
};
constexpr int kSegVectors = 4;

// 16 bytes of gradients, or as many as W values make, from and to memory.
template <typename TG, int W> struct Store {
  static constexpr int S = 16 / int(sizeof(TG)) < W ? 16 / int(sizeof(TG)) : W;  // elements to an access
  __device__ __forceinline__ static void add(const TG* p, float (&v)[W]) {
#pragma unroll
    for (int k = 0; k < W; k += S) {
      float o[S];
      if constexpr (S * sizeof(TG) == 16) Vec<TG>::load(p + k, o);
      else
#pragma unroll
        for (int i = 0; i < S; ++i) o[i] = to_f(p[k + i]);
#pragma unroll
      for (int i = 0; i < S; ++i) v[k + i] += o[i];
    }
  }
  __device__ __forceinline__ static void put(TG* p, const float (&v)[W]) {
#pragma unroll
    for (int k = 0; k < W; k += S) {
      float o[S];
#pragma unroll
      for (int i = 0; i < S; ++i) o[i] = v[k + i];
      if constexpr (S * sizeof(TG) == 16) Vec<TG>::store(p + k, o);
      else
#pragma unroll
        for (int i = 0; i < S; ++i) p[k + i] = from_f<TG>(o[i]);
    }
  }
};

// A warp to loops·kSegVectors·32 vectors of a row: dx = p·(A + B·t) (+ scale·dlogp at the token), t = log2 p.
template <typename T, typename TG>
__global__ void __launch_bounds__(kThreads, 5) token_logprobs_bwd_kernel(const __grid_constant__ Bwd a) {
  constexpr int W = Chunk<T>::W;
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t r = unit / a.segs;
  const int seg = int(unit - r * a.segs);
  if (r >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + r * a.ld;
  TG* dx = static_cast<TG*>(a.dx) + r * a.ld_d;
  const Row<T> row(x, a.V);
  const int full = int(row.full);
  int j0 = seg * a.loops * (kSegVectors * 32) + lane;
  uint4 q[kSegVectors];
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kSegVectors; ++u) {
      const int j = j0 + u * 32;
      if (j >= 1 && j <= full) q[u] = *reinterpret_cast<const uint4*>(row.vector(j));
    }
  };
  fetch();
  // 16-byte stores where the gradient's vectors are aligned as the logits' are
  const bool vec = ((reinterpret_cast<uintptr_t>(dx) + size_t(row.head) * sizeof(TG)) & 15) == 0;
  const float dl = a.d_logp ? __ldg(a.d_logp + r) : 0.f, dh = a.d_entropy ? __ldg(a.d_entropy + r) : 0.f;
  const int32_t t = __ldg(a.tokens + r);
  const bool valid = t >= 0 && t < a.V;
  if (!valid && seg == 0 && lane == 0) flag_error(a.flag, XT_DEVERR_INDEX);
  const bool none = dl == 0.f && dh == 0.f;  // zeros, whatever the row holds
  const float M = __ldg(a.stats + 2 * r), L = __ldg(a.stats + 2 * r + 1) * kLog2e;
  const float H = dh != 0.f ? __ldg(a.entropy + r) : 0.f;
  const float A = valid ? -a.scale * fmaf(dh, H, dl) : __int_as_float(0x7fc00000);
  const float B = -a.scale * dh * 0.6931471805599453f;
  const float hit = a.scale * dl;
  for (int loop = 0;;) {
#pragma unroll
    for (int u = 0; u < kSegVectors; ++u) {
      const int j = j0 + u * 32;
      if (j > full + 1) continue;
      const int e0 = int(row.first(j));
      const int n = int(row.last(j)) - e0;
      const bool whole = j >= 1 && j <= full;
      float v[W];
      if (whole) {
        Chunk<T>::values(q[u], v);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = i < n ? to_f(x[e0 + i]) : 0.f;
      }
      if (none) {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float y = max_nan(fmaf(v[i] - M, a.c, -L), kLowest);
          v[i] = ex2(y) * fmaf(B, y, A);
        }
        if (uint32_t(t - e0) < uint32_t(W)) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[i] += t - e0 == i ? hit : 0.f;
        }
      }
      TG* out = dx + e0;
      if (whole && vec) {
        if (a.acc) Store<TG, W>::add(out, v);
        Store<TG, W>::put(out, v);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (i < n) out[i] = from_f<TG>(a.acc ? to_f(out[i]) + v[i] : v[i]);
      }
    }
    if (++loop == a.loops) break;
    j0 += kSegVectors * 32;
    if (j0 - lane > full + 1) break;
    fetch();
  }
}

// Arguments that both calls check.
int check_args(const char* fn, const void* x, int64_t ld, const int32_t* tokens, float scale, int64_t rows, int64_t V,
               int dt) {
  XT_REQUIRE(valid_dtype(dt), "%s: bad dtype", fn);
  XT_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31) && V > 0 && V < (int64_t(1) << 30), "%s: bad sizes", fn);
  XT_REQUIRE(ld >= V, "%s: row stride smaller than V", fn);
  XT_REQUIRE(scale >= 1e-6f && scale <= 1e6f, "%s: scale must lie in [1e-6, 1e6]", fn);
  if (rows == 0) return XT_OK;
  XT_REQUIRE(x && tokens, "%s: NULL pointer", fn);
  if (reinterpret_cast<uintptr_t>(x) % dtype_size(dt)) return fail(XT_ERR_ALIGNMENT, "%s: logits are not aligned to their type", fn);
  return XT_OK;
}

}  // namespace
}  // namespace xt

using namespace xt;

extern "C" {

int xt_token_logprobs_fwd(const void* logits, int64_t ld, const int32_t* tokens, float scale, int top, float* logp,
                          float* entropy, float* stats, float* top_logp, int32_t* top_ids, int64_t rows, int64_t V,
                          int dt, void* stream) {
  const char* fn = "xt_token_logprobs_fwd";
  XT_TRY(check_args(fn, logits, ld, tokens, scale, rows, V, dt));
  XT_REQUIRE(top >= 0 && top <= V, "%s: top must lie in [0, V]", fn);
  if (top > kMaxTop) return fail(XT_ERR_UNSUPPORTED, "%s: at most %d alternatives", fn, kMaxTop);
  if (rows == 0) return XT_OK;
  XT_REQUIRE(logp && (top == 0 || (top_logp && top_ids)), "%s: NULL pointer", fn);
  Fwd a{logits, ld, rows, V, tokens, scale, scale * kLog2e, top, logp, entropy, stats, top_logp, top_ids, errflag()};
  cudaStream_t s = as_stream(stream);
  const int64_t bytes = V * int64_t(dtype_size(dt));
  // Short rows go to a warp each; longer ones to a CTA, and where the rows are too few to fill the GPU to a cluster of
  // CTAs, as long as each of them keeps 8 KB of the row.  With alternatives a CTA pays 14 barriers a row, and one whose part
  // of the row has fewer groups of 512 bytes than there are alternatives puts all of its elements in order: up to 16 KB a warp
  // takes the row where there are eight for every SM (25000 x 8000 with 20: 237 us, 359 by CTAs), up to 8 KB where the groups
  // are too few (100 x 4000 with 20: 25 us, 58); 3 x 8000 with 5 take 10 us by CTAs and 21 by warps.  Longer rows do not
  // look at the number of alternatives, so with 17 to 32 of them a CTA's 8 to 16 KB can have too few groups: 3 x 50257 take
  // 7.5 us with 5, 11 with 20 and 108 with 32 (eight CTAs of 24 groups), 16 x 36000 8, 88 and 89, 1000 x 5000 14, 29 and 206.
  const bool warp = bytes <= 4096 || (top && bytes <= 16384 && rows >= int64_t(num_sms()) * 8) ||
                    (top && bytes <= 8192 && bytes < int64_t(top + 1) * 512);
  int cl = 1;
  while (!warp && cl < 8 && rows * cl * 2 <= int64_t(num_sms()) * 4 && bytes >= int64_t(cl) * 2 * 8192) cl *= 2;
  const int64_t grid = warp ? ceil_div(rows, kWarps) : rows * cl;
  if (grid >= (int64_t(1) << 31)) return fail(XT_ERR_UNSUPPORTED, "%s: too many rows", fn);
#define XT_LOGPROBS(T_, TOP_)                                                                            \
  do {                                                                                                   \
    if (warp) launch(token_logprobs_kernel<T_, TOP_, true>, unsigned(grid), kThreads, 0, s, a);          \
    else if (cl == 1) launch(token_logprobs_kernel<T_, TOP_, false>, unsigned(grid), kThreads, 0, s, a); \
    else launch_clustered(token_logprobs_kernel<T_, TOP_, false>, unsigned(grid), kThreads, 0, s, cl, a); \
  } while (0)
  if (dt == XT_BF16) {
    if (top) XT_LOGPROBS(bf16, true);
    else XT_LOGPROBS(bf16, false);
  } else {
    if (top) XT_LOGPROBS(float, true);
    else XT_LOGPROBS(float, false);
  }
#undef XT_LOGPROBS
  return check_launch(fn);
}

int xt_token_logprobs_bwd(const void* logits, int64_t ld, const int32_t* tokens, const float* stats,
                          const float* entropy, const float* d_logp, const float* d_entropy, float scale,
                          void* dlogits, int64_t ld_d, int64_t rows, int64_t V, int dt, int dt_grad, int acc,
                          void* stream) {
  const char* fn = "xt_token_logprobs_bwd";
  XT_TRY(check_args(fn, logits, ld, tokens, scale, rows, V, dt));
  XT_REQUIRE(valid_dtype(dt_grad), "%s: bad gradient dtype", fn);
  XT_REQUIRE(ld_d >= V, "%s: gradient's row stride smaller than V", fn);
  XT_REQUIRE(acc == 0 || acc == 1, "%s: acc must be 0 or 1", fn);
  if (rows == 0) return XT_OK;
  XT_REQUIRE(stats && dlogits, "%s: NULL pointer", fn);
  XT_REQUIRE(d_entropy == nullptr || entropy != nullptr, "%s: d_entropy needs the forward's entropy", fn);
  XT_REQUIRE(logits != dlogits || (dt == dt_grad && ld == ld_d && !acc), "%s: in place needs one dtype and row stride, and acc = 0", fn);
  if (reinterpret_cast<uintptr_t>(dlogits) % dtype_size(dt_grad))
    return fail(XT_ERR_ALIGNMENT, "%s: dlogits are not aligned to their type", fn);
  const int w = dt == XT_BF16 ? 8 : 4;
  const int64_t vectors = V / w + 2;  // whole ones, the head and the tail
  // as long pieces as leave 64 warps to an SM, so that a row's values are fetched seldom
  int loops = 4;
  while (loops > 1 && rows * ceil_div(vectors, kSegVectors * 32 * loops) < int64_t(num_sms()) * 64) loops /= 2;
  const int64_t segs = ceil_div(vectors, kSegVectors * 32 * loops);
  Bwd a{logits, ld, tokens, stats, entropy, d_logp, d_entropy, scale, scale * kLog2e, dlogits, ld_d, rows, V, int(segs), loops, acc,
        errflag()};
  const int64_t grid = ceil_div(rows * segs, kWarps);
  if (grid >= (int64_t(1) << 31)) return fail(XT_ERR_UNSUPPORTED, "%s: too many rows", fn);
  cudaStream_t s = as_stream(stream);
  if (dt == XT_BF16) {
    if (dt_grad == XT_BF16) launch(token_logprobs_bwd_kernel<bf16, bf16>, unsigned(grid), kThreads, 0, s, a);
    else launch(token_logprobs_bwd_kernel<bf16, float>, unsigned(grid), kThreads, 0, s, a);
  } else {
    if (dt_grad == XT_BF16) launch(token_logprobs_bwd_kernel<float, bf16>, unsigned(grid), kThreads, 0, s, a);
    else launch(token_logprobs_bwd_kernel<float, float>, unsigned(grid), kThreads, 0, s, a);
  }
  return check_launch(fn);
}

}  // extern "C"
