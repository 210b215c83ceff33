// Builds the plan of masked attention (attention_plan.cuh) from the documents of a batch.
//
// Two launches, one where eight tiles or fewer make up the batch (1024 tokens: the launch is most
// of its time).  The first gives each token a thread: a binary search (in shared memory, which holds
// the offsets of up to kOffsets documents) finds its document, warps and shared memory reduce the
// intervals of a 128-token tile to the tile's ranges.  The second writes the tiles' records in the
// order of their work: a tile's place is the number of tiles with more work than it (or as much and a
// lower number), counted by one warp per tile, so the order never depends on timing.  Bound by two launches in
// a row: 4.7 us for 8192 tokens, 2.4 us for 96 (a cluster barrier in the place of the second launch: 4.5 and 2.9).
#include "attention_plan.cuh"
#include "internal.cuh"

namespace xt {
namespace attn_plan {
namespace {

constexpr int kTilesPerCta = 8;
constexpr int kThreads = BT * kTilesPerCta;
constexpr int kOffsets = 2048;  // document offsets searched in shared memory

struct Docs {
  const int32_t *off, *len, *prefix;
  int n, causal;
  int64_t T;
  int32_t* plan;
  uint32_t* flag;
};

struct Doc {
  int a, end, pe;  // first token, end of the valid part, end of the prefix
};

// `off`: p.off or its copy in shared memory.
__device__ __forceinline__ Doc doc_of(const Docs& p, const int32_t* off, int t) {
  int d, a, e;
  if (off) {
    int lo = 0, hi = p.n - 1;  // the last document that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    d = lo;
    a = p.n ? off[d] : 0;
    e = p.n ? off[d + 1] : 0;
  } else {
    const int span = p.n ? int(p.T / p.n) : 1;
    d = t / span;
    a = d * span;
    e = p.n ? a + span : 0;
  }
  // whatever the lists hold, the intervals stay inside the tokens
  const int T = int(p.T);
  a = min(max(a, 0), T);
  e = min(max(e, a), T);
  const int len = p.len && p.n ? min(max(p.len[d], 0), e - a) : e - a;
  const int pre = p.prefix && p.n ? min(max(p.prefix[d], 0), len) : 0;
  return Doc{a, a + len, a + pre};
}

// Work of a tile in opposite tiles; of a pair of query tiles in the key tiles that either meets.
__device__ __forceinline__ int cost(int4 r) { return max(r.y - r.x, 0); }
__device__ __forceinline__ int pair_cost(int4 a, int4 b) {
  if (a.y <= a.x) return cost(b);
  if (b.y <= b.x) return cost(a);
  return max(a.y, b.y) - min(a.x, b.x);
}

// One warp: the records of tile i and, for an even share of them, of pair i.
__device__ void order_tile(const Docs& p, int i) {
  const Layout l(p.T);
  const int nt = int(l.tiles), np = (nt + 1) / 2, lane = threadIdx.x & 31;
  if (i >= nt) return;
  const int4* q = reinterpret_cast<const int4*>(p.plan + l.qrange);
  const int4* k = reinterpret_cast<const int4*>(p.plan + l.krange);
  const int4 none = make_int4(0, 0, 0, 0);
  const bool has_pair = i < np;
  const int4 q0 = has_pair ? q[2 * i] : none, q1 = has_pair && 2 * i + 1 < nt ? q[2 * i + 1] : none;
  const int4 qi = q[i], ki = k[i];
  const int cq = cost(qi), ck = cost(ki), cp = pair_cost(q0, q1);
  int rq = 0, rk = 0, rp = 0;
  for (int j = lane; j < nt; j += 32) {
    const int a = cost(q[j]), b = cost(k[j]);
    rq += a > cq || (a == cq && j < i);
    rk += b > ck || (b == ck && j < i);
    if (has_pair && j < np) {
      const int c = pair_cost(q[2 * j], 2 * j + 1 < nt ? q[2 * j + 1] : none);
      rp += c > cp || (c == cp && j < i);
    }
  }
  rq = __reduce_add_sync(0xffffffffu, rq);
  rk = __reduce_add_sync(0xffffffffu, rk);
  rp = __reduce_add_sync(0xffffffffu, rp);
  if (lane != 0) return;
  int4* out = reinterpret_cast<int4*>(p.plan + l.qs) + 2 * rq;
  out[0] = make_int4(i, 0, 0, 0);
  out[1] = qi;
  out = reinterpret_cast<int4*>(p.plan + l.ks) + 2 * rk;
  out[0] = make_int4(i, 0, 0, 0);
  out[1] = ki;
  if (!has_pair) return;
  out = reinterpret_cast<int4*>(p.plan + l.pairs) + 3 * rp;
  const int first = cost(q0) == 0 ? q1.x : cost(q1) == 0 ? q0.x : min(q0.x, q1.x);
  out[0] = make_int4(2 * i, first, first + cp, 0);
  out[1] = q0;
  out[2] = q1;
}

__device__ __forceinline__ int4 tile_range(int lo_min, int hi_max, int lo_max, int hi_min) {
  if (hi_max <= lo_min) return make_int4(0, 0, 0, 0);
  const int f0 = (lo_max + BT - 1) / BT, f1 = hi_min / BT;
  return make_int4(lo_min / BT, (hi_max + BT - 1) / BT, f0, max(f0, f1));
}

__global__ void __launch_bounds__(kThreads) plan_tiles_kernel(const Docs p) {
  pdl_begin();
  __shared__ int red[8][kThreads / 32];
  const Layout l(p.T);
  const int64_t t = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.off || p.len || p.prefix)
    for (int64_t d = t; d < p.n; d += int64_t(gridDim.x) * kThreads) {
      const int64_t a = p.off ? p.off[d] : d * (p.T / p.n), e = p.off ? p.off[d + 1] : (d + 1) * (p.T / p.n);
      bool bad = a < 0 || e < a || e > p.T;
      if (p.len) bad |= p.len[d] < 0 || p.len[d] > e - a;
      if (p.prefix) bad |= p.prefix[d] < 0;
      if (bad) flag_error(p.flag, XT_DEVERR_INDEX);
    }
  __shared__ int32_t offs[kOffsets];
  const int32_t* off = p.off;
  if (p.off && p.n < kOffsets) {
    for (int d = threadIdx.x; d <= p.n; d += kThreads) offs[d] = p.off[d];
    off = offs;
    __syncthreads();
  }
  const bool real = t < p.T;
  int2 q = make_int2(0, 0), k = make_int2(0, 0);
  if (real) {
    const int i = int(t);
    const Doc d = doc_of(p, off, i);
    if (i >= d.a && i < d.end) {
      q = make_int2(d.a, p.causal ? max(i + 1, d.pe) : d.end);
      k = make_int2(p.causal && i >= d.pe ? i : d.a, d.end);
    }
  }
  if (t < l.tiles * BT) {
    reinterpret_cast<int2*>(p.plan + l.q_iv)[t] = q;
    reinterpret_cast<int2*>(p.plan + l.k_iv)[t] = k;
  }
  // per tile: the least first and largest end of rows that see something, and the largest first and
  // least end of all real rows (an empty row leaves no tile full)
  const int big = 0x7fffffff;
  const int v[8] = {q.y > q.x ? q.x : big, q.y > q.x ? q.y : 0, real ? (q.y > q.x ? q.x : big) : 0,
                    real ? q.y : big,      k.y > k.x ? k.x : big, k.y > k.x ? k.y : 0,
                    real ? (k.y > k.x ? k.x : big) : 0, real ? k.y : big};
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const int r = (m == 1 || m == 2 || m == 5 || m == 6) ? __reduce_max_sync(0xffffffffu, v[m])
                                                         : __reduce_min_sync(0xffffffffu, v[m]);
    if (lane == 0) red[m][warp] = r;
  }
  __syncthreads();
  const int64_t tile = t / BT;
  if ((threadIdx.x & (BT - 1)) < 2 && tile < l.tiles) {
    const int w = warp, m = (threadIdx.x & 1) * 4;
    auto mn = [&](int i) { return min(min(red[i][w], red[i][w + 1]), min(red[i][w + 2], red[i][w + 3])); };
    auto mx = [&](int i) { return max(max(red[i][w], red[i][w + 1]), max(red[i][w + 2], red[i][w + 3])); };
    const int lo_max = mx(m + 2);
    const int4 r = tile_range(mn(m), mx(m + 1), lo_max == big ? int(p.T) : lo_max, mn(m + 3));
    reinterpret_cast<int4*>(p.plan + (m ? l.krange : l.qrange))[tile] = r;
  }
  if (t == 0) {
    p.plan[0] = kMagic;
    p.plan[1] = int32_t(p.T);
    p.plan[2] = p.causal;
  }
  if (gridDim.x == 1) {
    __syncthreads();
    if (warp < kTilesPerCta) order_tile(p, warp);
  }
}

__global__ void __launch_bounds__(256) plan_order_kernel(const Docs p) {
  pdl_begin();
  order_tile(p, int(blockIdx.x) * 8 + int(threadIdx.x >> 5));
}

}  // namespace
}  // namespace attn_plan
}  // namespace xt

using namespace xt;
using namespace xt::attn_plan;

extern "C" {

int xt_attention_plan_size(int64_t T, size_t* bytes) {
  XT_REQUIRE(T >= 0 && T < (int64_t(1) << 30) && bytes, "xt_attention_plan_size: bad arguments");
  *bytes = size_t(Layout(T).total) * 4;
  return XT_OK;
}

int xt_attention_plan(int64_t T, int n_docs, const int32_t* doc_off, const int32_t* doc_len, const int32_t* prefix,
                      int causal, void* plan, size_t plan_bytes, void* stream) {
  XT_REQUIRE(T >= 0 && T < (int64_t(1) << 30), "xt_attention_plan: T must be in [0, 2^30)");
  XT_REQUIRE(n_docs >= 0 && n_docs < (1 << 30), "xt_attention_plan: n_docs must be in [0, 2^30)");
  XT_REQUIRE(causal == 0 || causal == 1, "xt_attention_plan: causal must be 0 or 1");
  XT_REQUIRE(doc_off || (n_docs > 0 ? T % n_docs == 0 : T == 0),
             "xt_attention_plan: without doc_off T must be a multiple of n_docs");
  XT_REQUIRE(plan, "xt_attention_plan: plan is NULL");
  if (!aligned16(plan)) return fail(XT_ERR_ALIGNMENT, "xt_attention_plan: the plan must be 16-byte aligned");
  const Layout l(T);
  XT_REQUIRE(plan_bytes >= size_t(l.total) * 4, "xt_attention_plan: plan too small (%zu < %zu)", plan_bytes,
             size_t(l.total) * 4);
  if (T == 0) return XT_OK;
  const Docs p{doc_off, doc_len, prefix, n_docs, causal, T, static_cast<int32_t*>(plan), errflag()};
  cudaStream_t s = as_stream(stream);
  const unsigned grid = unsigned(ceil_div(l.tiles, kTilesPerCta));
  launch(plan_tiles_kernel, grid, kThreads, 0, s, p);
  XT_TRY(check_launch("xt_attention_plan (tiles)"));
  if (grid > 1) {
    launch(plan_order_kernel, unsigned(ceil_div(l.tiles, 8)), 256, 0, s, p);
    XT_TRY(check_launch("xt_attention_plan (order)"));
  }
  return XT_OK;
}

}  // extern "C"
