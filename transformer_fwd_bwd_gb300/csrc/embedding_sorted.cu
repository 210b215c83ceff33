// Embedding lookup with a scale, and its gradient by sorted tokens:
//   h[t] = scale·E[ids[t]],   dE[v] (+)= scale·Σ_{t: ids[t] = v} dh[t], t ascending.
//
// xt_embedding_plan sorts the tokens by id, those of one id by t: up to kRankTokens of them by counting (below), more by
// a stable radix sort, least significant digit first,
// by one cluster of CTAs (hardware barriers, no waiting on memory; 16 CTAs for many tokens: 131072 in 35 us where 8 take
// 56), every digit of up to 9 bits two sweeps over the cluster's tokens: counts of each warp, their prefix over warps, CTAs and digits, then the moves.  One launch; 16 bits
// of id take two digits.
//
// The gradient cuts the sorted tokens into chunks of 8 to 32.  A warp takes a chunk and 256 columns, keeps the running
// sum of an id's rows in registers and writes dE where an id's tokens lie within the chunk; the sums of ids that cross
// chunks go to the workspace (at most two rows per chunk) and a second launch adds them in chunk order.  So every row
// of dh is read once, every row of dE that is touched is read and written once, nothing depends on how often an id
// occurs, and no sum depends on timing.  With acc = 0 the rows that no token touches are zeroed in the same launch: a
// warp to 32 rows, each lane looking its row up in the plan.
//
// Bound by HBM, few tokens by latency.  On one GB300 (bf16 rows, float32 gradient, us): lookup, plan, gradient of 8192 tokens x 768
// over 50304 rows 5.4, 12.8, 13.2; of 131072 x 1024 over 128256 rows, written afresh, 65, 35, 176 (0.67 of the copy rate); of
// 37 tokens 1.8, 2.4, 7.1.
#include <atomic>

#include "internal.cuh"

namespace xt {
namespace {

// ------------------------------------------------------------------------------ lookup

template <typename TE, typename TH, bool VEC>
__global__ void __launch_bounds__(256) embedding_lookup_kernel(const int32_t* __restrict__ ids, const TE* __restrict__ E,
                                                               TH* __restrict__ h, int64_t T, int64_t d, int64_t V,
                                                               float scale, uint32_t* flag) {
  constexpr int W = VEC ? 8 : 1;
  pdl_begin();
  const int64_t per = d / W, total = T * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
    const int64_t t = i / per, c = (i - t * per) * W;
    const int32_t id = __ldg(ids + t);
    float v[W];
    if (id >= 0 && id < V) {
      Acc<TE, W>::load(E + int64_t(id) * d + c, v);
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] *= scale;
    } else {
      if (c == 0) flag_error(flag, XT_DEVERR_INDEX);
#pragma unroll
      for (int k = 0; k < W; ++k) v[k] = __int_as_float(0x7fc00000);
    }
    Acc<TH, W>::store(h + t * d + c, v);
  }
}

// ------------------------------------------------------------------------------ plan

struct PlanHeader {
  int64_t T, V;
};
// [header][T entries: id << 32 | t, sorted][T entries of the sort's other buffer]; ids outside [0, V) as V
__host__ __device__ inline uint64_t* plan_entries(void* plan) {
  return reinterpret_cast<uint64_t*>(static_cast<char*>(plan) + sizeof(PlanHeader));
}

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSortCluster = 16;  // 8 is what every GPU of this kind schedules; 16 where it says it can
constexpr int kBatch = 8;
// counts of the CTA's warps, totals of every CTA of the cluster, scratch of the scan over digits
constexpr int kSortSmem = (kSortWarps * kDigits + kSortCluster * kDigits + kSortWarps) * 4;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The lanes whose digit (of `bits` bits) is this lane's, among those in `in`: a ballot per bit (about 27 instructions; the
// instruction that compares all lanes' values is slower: 131072 tokens sorted by 8 CTAs in 73 us instead of 56).
__device__ __forceinline__ uint32_t same_digit(uint32_t dg, bool in, int bits) {
  uint32_t peers = __ballot_sync(0xffffffffu, in);
  for (int b = 0; b < bits; ++b) {
    const uint32_t one = __ballot_sync(0xffffffffu, (dg >> b) & 1);
    peers &= (dg >> b) & 1 ? one : ~one;
  }
  return peers;
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(const int32_t* __restrict__ ids, void* plan,
                                                                      int64_t T, int64_t V, int passes, int bits,
                                                                      uint32_t* flag) {
  extern __shared__ uint32_t smem[];
  uint32_t* counts = smem;                              // [warp][digit]
  uint32_t* totals = smem + kSortWarps * kDigits;       // [cta][digit]
  uint32_t* scan = totals + kSortCluster * kDigits;     // [warp]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t rank, cl;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cl));
  // the other CTAs are running before anything is stored into them (waited for at the first digit's totals)
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_begin();
  if (rank == 0 && threadIdx.x == 0) *static_cast<PlanHeader*>(plan) = PlanHeader{T, V};
  uint64_t* sorted = plan_entries(plan);
  uint64_t* other = sorted + T;
  // each warp owns a contiguous piece of the input, a multiple of 32 tokens
  const int64_t warps = int64_t(cl) * kSortWarps;
  const int64_t piece = ((T + warps - 1) / warps + 31) / 32 * 32;
  const int64_t lo = (int64_t(rank) * kSortWarps + warp) * piece;
  const int64_t hi = lo + piece < T ? lo + piece : T;
  const uint32_t mask = (1u << bits) - 1u;
  for (int p = 0; p < passes; ++p) {
    // the last pass ends in `sorted`
    uint64_t* dst = (passes - 1 - p) % 2 == 0 ? sorted : other;
    const uint64_t* src = dst == sorted ? other : sorted;
    auto item = [&](int64_t i) -> uint64_t {
      if (p > 0) return __ldcg(src + i);  // written by other SMs of the cluster
      const int32_t id = __ldg(ids + i);
      const bool ok = id >= 0 && id < V;
      return (uint64_t(ok ? uint32_t(id) : uint32_t(V)) << 32) | uint32_t(i);
    };
    const int shift = 32 + p * bits;
    for (int i = threadIdx.x; i < kSortWarps * kDigits; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    uint32_t* mine = counts + warp * kDigits;
    // kBatch rounds of 32 tokens are fetched together
    auto digit = [&](uint64_t e, bool in) { return in ? uint32_t(e >> shift) & mask : uint32_t(kDigits); };
    for (int64_t b0 = lo; b0 < hi; b0 += kBatch * 32) {
      uint64_t e[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) e[k] = b0 + k * 32 + lane < hi ? item(b0 + k * 32 + lane) : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (b0 + k * 32 >= hi) break;
        const bool in = b0 + k * 32 + lane < hi;
        const uint32_t dg = digit(e[k], in);
        if (p == 0 && in && (e[k] >> 32) == uint64_t(V)) flag_error(flag, XT_DEVERR_INDEX);
        const uint32_t peers = same_digit(dg, in, bits);
        if (in && lane == __ffs(peers) - 1) mine[dg] += __popc(peers);
        __syncwarp();
      }
    }
    __syncthreads();
    // counts → prefix over the CTA's warps; the CTA's totals go to every CTA of the cluster
    if (p == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (threadIdx.x < kDigits) {
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = counts[w * kDigits + threadIdx.x];
        counts[w * kDigits + threadIdx.x] = sum;
        sum += n;
      }
      const uint32_t at = uint32_t(__cvta_generic_to_shared(totals + rank * kDigits + threadIdx.x));
      for (uint32_t c = 0; c < cl; ++c) {
        uint32_t remote;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(at), "r"(c));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(sum) : "memory");
      }
    }
    cluster_barrier();
    // this CTA's first place for each digit: all smaller digits, then the same digit of the CTAs before it
    uint32_t all = 0, before = 0;
    if (threadIdx.x < kDigits) {
      for (uint32_t c = 0; c < cl; ++c) {
        const uint32_t n = totals[c * kDigits + threadIdx.x];
        before += c < rank ? n : 0u;
        all += n;
      }
    }
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    if (threadIdx.x < kDigits) {
      uint32_t base = inc - all + before;
      for (int w = 0; w < warp; ++w) base += scan[w];
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) counts[w * kDigits + threadIdx.x] += base;
    }
    __syncthreads();
    for (int64_t b0 = lo; b0 < hi; b0 += kBatch * 32) {
      uint64_t e[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) e[k] = b0 + k * 32 + lane < hi ? item(b0 + k * 32 + lane) : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (b0 + k * 32 >= hi) break;
        const bool in = b0 + k * 32 + lane < hi;
        const uint32_t dg = digit(e[k], in);
        const uint32_t peers = same_digit(dg, in, bits);
        const uint32_t first = in ? mine[dg] : 0u;
        __syncwarp();
        if (in) {
          dst[first + __popc(peers & ((1u << lane) - 1u))] = e[k];
          if (lane == __ffs(peers) - 1) mine[dg] = first + __popc(peers);
        }
        __syncwarp();
      }
    }
    // the moves are done, and no CTA still reads the totals, before the next digit (or, at the end, the exit)
    cluster_barrier();
  }
}

// Few tokens: a token's place is the number of tokens before it in the order, counted against all of them, with nothing to
// wait for between CTAs (37 tokens: 2.4 us, the sort 8.5).  T² comparisons and 4·T bytes of shared memory per CTA: at 8192
// tokens no faster than the sort (13.2 against 12.7 us), and changing the SMs' split of shared memory cost as much again.
constexpr int kRankTokens = 2048;
constexpr int kRankThreads = 256;
constexpr int kRankPer = 32;  // tokens of a CTA: kRankThreads / 32 warps share the comparisons of a token to a lane
__global__ void __launch_bounds__(kRankThreads) embedding_rank_kernel(const int32_t* __restrict__ ids, void* plan, int T,
                                                                      int64_t V, uint32_t* flag) {
  extern __shared__ __align__(16) uint32_t keys[];  // ids of all tokens, those outside as V; padded with ~0
  __shared__ int part[kRankThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarpsHere = kRankThreads / 32;
  pdl_begin();
  if (blockIdx.x == 0 && threadIdx.x == 0) *static_cast<PlanHeader*>(plan) = PlanHeader{T, V};
  const int padded = (T + 127) / 128 * 128;
  for (int i0 = threadIdx.x; i0 < padded; i0 += 8 * kRankThreads) {
    int32_t id[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) id[k] = i0 + k * kRankThreads < T ? __ldg(ids + i0 + k * kRankThreads) : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kRankThreads;
      const bool ok = id[k] >= 0 && id[k] < V;
      if (!ok && blockIdx.x == 0) flag_error(flag, XT_DEVERR_INDEX);
      if (i < padded) keys[i] = i >= T ? 0xffffffffu : ok ? uint32_t(id[k]) : uint32_t(V);
    }
  }
  __syncthreads();
  const int t = int(blockIdx.x) * kRankPer + lane;
  const uint32_t mine = t < T ? keys[t] : 0u;
  // pieces of 128 tokens go round the warps; in those before the token's own an equal id counts
  const int own = int(blockIdx.x) * kRankPer / 128;
  int rank = 0;
  for (int p = warp; p < padded / 128; p += kWarpsHere) {
    const uint4* k4 = reinterpret_cast<const uint4*>(keys + p * 128);
    if (p == own) {
#pragma unroll 8
      for (int i = 0; i < 128; ++i) {
        const uint32_t k = keys[p * 128 + i];
        rank += k < mine || (k == mine && p * 128 + i < t);
      }
    } else {
      const uint32_t bound = p < own ? mine + 1u : mine;  // V < 2³¹: no wrap
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const uint4 k = k4[i];
        rank += int(k.x < bound) + int(k.y < bound) + int(k.z < bound) + int(k.w < bound);
      }
    }
  }
  part[warp][lane] = rank;
  __syncthreads();
  if (warp == 0 && t < T) {
#pragma unroll
    for (int w = 1; w < kWarpsHere; ++w) rank += part[w][lane];
    plan_entries(plan)[rank] = (uint64_t(mine) << 32) | uint32_t(t);
  }
}

// ------------------------------------------------------------------------------ gradient

constexpr int kCols = 256;  // columns of a warp: 8 to a lane
constexpr int kWarps = 8;

// Sorted tokens per chunk: 32, or fewer where that leaves too few warps to keep HBM busy.
constexpr int64_t kManyWarps = 4864;  // 32 on each of 152 SMs
__host__ inline int chunk_tokens(int64_t T, int64_t d) {
  const int64_t tiles = ceil_div(d, kCols);
  int c = 32;
  while (c > 8 && ceil_div(T, c) * tiles < kManyWarps) c /= 2;
  return c;
}
__host__ inline size_t part_bytes_for(int64_t chunks, int64_t d) { return size_t(chunks) * 2 * size_t(d) * 4; }
// The most chunks that a batch of up to T tokens is cut into.  Where chunks grow from c to 2c tokens their number falls: the
// last T of chunks of c has fewer than kManyWarps warps' worth of chunks of 2c, that is twice as many of c.
__host__ inline int64_t most_chunks(int64_t T, int64_t d) {
  const int c = chunk_tokens(T, d);
  const int64_t chunks = ceil_div(T, c), shorter = 2 * ((kManyWarps - 1) / ceil_div(d, kCols));
  return c > 8 && shorter > chunks ? shorter : chunks;
}

struct Grad {
  const void* plan;
  const void* dh;
  void* dE;
  float* part;  // [chunk][2][d]: the chunk's share of an id that began before it, of one that goes on after it
  int64_t T, d, V;
  int64_t chunks, tiles, zero_units;
  float scale;
  int chunk, acc;
  uint32_t* flag;
};

// A lane's 8 columns of a row: two groups of 4 neighbours 128 columns apart (so that a warp's float32 accesses fill whole
// sectors: with 8 neighbours to a lane 131072 rows of 1024 took 251 us instead of 202), or 8 columns 32 apart where rows are not
// made of aligned 16 bytes.
template <typename T> struct V4;
template <> struct V4<float> {
  __device__ __forceinline__ static void load(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  }
  __device__ __forceinline__ static void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct V4<bf16> {
  __device__ __forceinline__ static void load(const bf16* p, float* v) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
  }
  __device__ __forceinline__ static void store(bf16* p, const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};
template <typename T, bool VEC> struct Cols {
  __device__ __forceinline__ static void load(const T* row, int64_t c0, int64_t d, int lane, float (&v)[8]) {
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = c0 + h * 128 + lane * 4;
        if (c < d) V4<T>::load(row + c, v + 4 * h);
        else
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * h + i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c0 + i * 32 + lane < d ? to_f(row[c0 + i * 32 + lane]) : 0.f;
    }
  }
  __device__ __forceinline__ static void store(T* row, int64_t c0, int64_t d, int lane, const float (&v)[8]) {
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = c0 + h * 128 + lane * 4;
        if (c < d) V4<T>::store(row + c, v + 4 * h);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + i * 32 + lane < d) row[c0 + i * 32 + lane] = from_f<T>(v[i]);
    }
  }
};

template <typename TG, bool VEC>
__device__ __forceinline__ void write_row(const Grad& a, int64_t id, int64_t c0, int lane, float (&sum)[8]) {
  TG* row = static_cast<TG*>(a.dE) + id * a.d;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] *= a.scale;
  if (a.acc) {
    float old[8];
    Cols<TG, VEC>::load(row, c0, a.d, lane, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += old[i];
  }
  Cols<TG, VEC>::store(row, c0, a.d, lane, sum);
}

__device__ __forceinline__ bool plan_fits(const Grad& a) {
  const PlanHeader* h = static_cast<const PlanHeader*>(a.plan);
  if (h->T == a.T && h->V == a.V) return true;
  if (threadIdx.x == 0 && blockIdx.x == 0) flag_error(a.flag, XT_DEVERR_PLAN);
  return false;
}

template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, 4) embedding_grad_kernel(const __grid_constant__ Grad a) {
  // rows in flight: two and four blocks per SM (131072 rows of 1024: 183 us; four rows 188, eight 215)
  constexpr int U = 2;
  pdl_begin();
  if (!plan_fits(a)) return;
  const int lane = threadIdx.x & 31;
  // from the end: the rows to zero, then the higher ids, whose tokens are fewer each and whose rows more (183 -> 176 us)
  const int64_t unit = int64_t(gridDim.x - 1 - blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const uint64_t* plan = plan_entries(const_cast<void*>(a.plan));
  const int64_t units = a.chunks * a.tiles;
  if (unit >= units) {
    // rows that no token touches
    if (unit - units >= a.zero_units) return;
    const int64_t v0 = (unit - units) * 32, v = v0 + lane;
    int64_t lo = 0, hi = a.T;  // first entry with an id of at least v
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (int64_t(__ldg(plan + mid) >> 32) < v) lo = mid + 1;
      else hi = mid;
    }
    const bool untouched = v < a.V && !(lo < a.T && int64_t(__ldg(plan + lo) >> 32) == v);
    const float zero[8] = {};
    for (uint32_t m = __ballot_sync(0xffffffffu, untouched); m; m &= m - 1) {
      TG* row = static_cast<TG*>(a.dE) + (v0 + __ffs(m) - 1) * a.d;
      for (int64_t c0 = 0; c0 < a.d; c0 += kCols) Cols<TG, VEC>::store(row, c0, a.d, lane, zero);
    }
    return;
  }
  const int64_t chunk = unit / a.tiles, c0 = (unit - chunk * a.tiles) * kCols;
  const int64_t p0 = chunk * a.chunk;
  const int n = int(a.T - p0 < a.chunk ? a.T - p0 : a.chunk);
  const uint64_t e = lane < n ? __ldg(plan + p0 + lane) : 0;
  const int64_t before = p0 > 0 ? int64_t(__ldg(plan + p0 - 1) >> 32) : -1;
  const int64_t after = p0 + n < a.T ? int64_t(__ldg(plan + p0 + n) >> 32) : -1;
  const T* dh = static_cast<const T*>(a.dh);
  const int id = int(e >> 32), t = int(uint32_t(e));
  const int next = __shfl_down_sync(0xffffffffu, id, 1);
  // tokens that end their id within the chunk, or end the chunk
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < n && (lane == n - 1 || next != id));
  const int first_id = __shfl_sync(0xffffffffu, id, 0);
  float sum[8] = {};
  for (int q = 0; q < n; q += U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tu = __shfl_sync(0xffffffffu, t, (q + u) & 31);
      if (q + u < n) Cols<T, VEC>::load(dh + int64_t(tu) * a.d, c0, a.d, lane, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (q + u >= n) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += v[u][i];
      if (!((ends >> (q + u)) & 1)) continue;
      const int64_t cur = __shfl_sync(0xffffffffu, id, q + u);
      const bool began = !(cur == first_id && before == cur), done = !(q + u == n - 1 && after == cur);
      if (cur < a.V) {
        if (began && done) {
          write_row<TG, VEC>(a, cur, c0, lane, sum);
        } else {
          Cols<float, VEC>::store(a.part + (chunk * 2 + (began ? 1 : 0)) * a.d, c0, a.d, lane, sum);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    }
  }
}

// Adds the shares of the ids that cross chunks: the warp of the chunk where such an id begins.  Ids over more than
// kAlone chunks are summed by the block's warps together.
template <typename TG, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) embedding_join_kernel(const __grid_constant__ Grad a) {
  constexpr int64_t kAlone = 16;
  __shared__ int64_t wide[kWarps][4];      // id, chunk, chunks that follow, first column (id < 0: none)
  __shared__ float sums[kWarps][32][9];
  pdl_begin();
  if (!plan_fits(a)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t unit = int64_t(blockIdx.x) * kWarps + warp;
  const uint64_t* plan = plan_entries(const_cast<void*>(a.plan));
  auto id_at = [&](int64_t p) { return int64_t(__ldg(plan + p) >> 32); };
  int64_t id = -1, chunk = 0, more = 0, c0 = 0;
  if (unit < a.chunks * a.tiles) {
    chunk = unit / a.tiles;
    c0 = (unit - chunk * a.tiles) * kCols;
    const int64_t p0 = chunk * a.chunk, p1 = p0 + a.chunk;
    if (p1 < a.T) {
      const int64_t last = id_at(p1 - 1), after = id_at(p1), first = id_at(p0);
      const int64_t before = p0 > 0 ? id_at(p0 - 1) : -1;
      if (last == after && last < a.V && !(first == last && before == last)) id = last;
    }
  }
  if (id >= 0) {
    // chunks after this one that begin with the id: 32 places of the range at a time
    int64_t lo = chunk + 1, hi = a.chunks;  // lo begins with it, hi does not
    while (hi - lo > 1) {
      const int64_t step = (hi - lo + 31) / 32;
      const int64_t c = lo + (lane + 1) * step;
      const bool with = c < hi && id_at(c * a.chunk) == id;
      const int64_t k = __popc(__ballot_sync(0xffffffffu, with));  // ids rise, so these are the first k
      const int64_t nlo = lo + k * step;
      hi = lo + (k + 1) * step < hi ? lo + (k + 1) * step : hi;
      lo = nlo;
    }
    more = lo - chunk;
  }
  auto add = [&](int64_t from, int64_t to, int64_t col, float (&sum)[8]) {  // chunks [from, to), in order
    for (int64_t c = from; c < to; c += 8) {
      float v[8][8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c + u < to) Cols<float, VEC>::load(a.part + (c + u) * 2 * a.d, col, a.d, lane, v[u]);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c + u < to)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += v[u][i];
    }
  };
  if (id >= 0 && more <= kAlone) {
    float sum[8];
    Cols<float, VEC>::load(a.part + (chunk * 2 + 1) * a.d, c0, a.d, lane, sum);
    add(chunk + 1, chunk + 1 + more, c0, sum);
    write_row<TG, VEC>(a, id, c0, lane, sum);
  }
  if (lane == 0) {
    wide[warp][0] = more > kAlone ? id : -1;
    wide[warp][1] = chunk;
    wide[warp][2] = more;
    wide[warp][3] = c0;
  }
  __syncthreads();
  for (int k = 0; k < kWarps; ++k) {
    const int64_t wid = wide[k][0], wc = wide[k][1], n = wide[k][2], wc0 = wide[k][3];
    if (wid < 0) continue;
    float sum[8] = {};
    if (warp == 0) Cols<float, VEC>::load(a.part + (wc * 2 + 1) * a.d, wc0, a.d, lane, sum);
    add(wc + 1 + n * warp / kWarps, wc + 1 + n * (warp + 1) / kWarps, wc0, sum);
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][lane][i] = sum[i];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += sums[w][lane][i];
      write_row<TG, VEC>(a, wid, wc0, lane, sum);
    }
    __syncthreads();
  }
}

int sizes_ok(const char* fn, int64_t T, int64_t d, int64_t V) {
  XT_REQUIRE(T >= 0 && T < (int64_t(1) << 30), "%s: T must lie in [0, 2^30)", fn);
  XT_REQUIRE(d > 0 && d < (int64_t(1) << 30), "%s: d must be positive", fn);
  XT_REQUIRE(V > 0 && V < (int64_t(1) << 31) - 1, "%s: V must lie in [1, 2^31 - 2]", fn);
  return XT_OK;
}
size_t plan_bytes_for(int64_t T) { return sizeof(PlanHeader) + size_t(T) * 16; }

}  // namespace
}  // namespace xt

using namespace xt;

extern "C" {

int xt_embedding_lookup_fwd(const int32_t* ids, const void* E, void* h, int64_t T, int64_t d, int64_t V, float scale,
                            int dt_e, int dt_h, void* stream) {
  const char* fn = "xt_embedding_lookup_fwd";
  XT_TRY(sizes_ok(fn, T, d, V));
  XT_REQUIRE(valid_dtype(dt_e) && valid_dtype(dt_h), "%s: bad dtype", fn);
  if (T == 0) return XT_OK;
  XT_REQUIRE(ids && E && h, "%s: NULL pointer", fn);
  const bool vec = d % 8 == 0 && aligned16(E) && aligned16(h);
  const int64_t total = T * (d / (vec ? 8 : 1));
  int64_t grid = ceil_div(total, 256);
  if (grid > int64_t(num_sms()) * 64) grid = int64_t(num_sms()) * 64;
  cudaStream_t s = as_stream(stream);
#define XT_LOOKUP(TE_, TH_)                                                                                          \
  do {                                                                                                               \
    if (vec)                                                                                                         \
      launch(embedding_lookup_kernel<TE_, TH_, true>, unsigned(grid), 256, 0, s, ids, static_cast<const TE_*>(E),    \
             static_cast<TH_*>(h), T, d, V, scale, errflag());                                                       \
    else                                                                                                             \
      launch(embedding_lookup_kernel<TE_, TH_, false>, unsigned(grid), 256, 0, s, ids, static_cast<const TE_*>(E),   \
             static_cast<TH_*>(h), T, d, V, scale, errflag());                                                       \
  } while (0)
  if (dt_e == XT_BF16) {
    if (dt_h == XT_BF16) XT_LOOKUP(bf16, bf16);
    else XT_LOOKUP(bf16, float);
  } else {
    if (dt_h == XT_BF16) XT_LOOKUP(float, bf16);
    else XT_LOOKUP(float, float);
  }
#undef XT_LOOKUP
  return check_launch(fn);
}

int xt_embedding_plan_size(int64_t T, size_t* bytes) {
  XT_REQUIRE(bytes != nullptr, "xt_embedding_plan_size: NULL pointer");
  XT_TRY(sizes_ok("xt_embedding_plan_size", T, 1, 1));
  *bytes = plan_bytes_for(T);
  return XT_OK;
}

int xt_embedding_plan(const int32_t* ids, int64_t T, int64_t V, void* plan, size_t plan_bytes, void* stream) {
  const char* fn = "xt_embedding_plan";
  XT_TRY(sizes_ok(fn, T, 1, V));
  XT_REQUIRE(plan && plan_bytes >= plan_bytes_for(T), "%s: the plan holds %zu bytes, %zu are needed", fn,
             plan ? plan_bytes : size_t(0), plan_bytes_for(T));
  if (!aligned16(plan)) return fail(XT_ERR_ALIGNMENT, "%s: the plan must be 16-byte aligned", fn);
  XT_REQUIRE(T == 0 || ids, "%s: NULL pointer", fn);
  if (T > 0 && T <= kRankTokens) {
    launch(embedding_rank_kernel, unsigned(ceil_div(T, kRankPer)), kRankThreads, size_t((T + 127) / 128 * 512),
           as_stream(stream), ids, plan, int(T), V, errflag());
    return check_launch(fn);
  }
  int bits = 1;
  while ((V >> bits) != 0) ++bits;  // ids 0 .. V − 1, and V for those outside
  const int passes = int(ceil_div(bits, kDigitBits));
  const int digit = int(ceil_div(bits, passes));
  // kept as bits per device: the attribute is set once on each
  static std::atomic<uint64_t> set{0}, wide{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch(fn);
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem) != cudaSuccess ||
        cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return check_launch(fn);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kSortCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, embedding_sort_kernel, &cfg) != cudaSuccess) {
      n = 0;
      cudaGetLastError();  // a failed query leaves no launch error behind for the next check
    }
    if (dev < 64) {
      if (n > 0) wide.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
      set.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
  }
  // a CTA for every 1024 tokens up to 8, and 16 from 16384 tokens on
  int cl = 1;
  while (cl < 8 && T > int64_t(cl) * kSortThreads) cl *= 2;
  if (T >= 16384 && dev < 64 && (wide.load(std::memory_order_relaxed) >> dev & 1)) cl = 16;
  launch_clustered(embedding_sort_kernel, cl, kSortThreads, kSortSmem, as_stream(stream), cl, ids, plan, T, V, passes,
                   digit, errflag());
  return check_launch(fn);
}

int xt_embedding_sorted_bwd_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  XT_REQUIRE(bytes != nullptr, "xt_embedding_sorted_bwd_workspace_size: NULL pointer");
  XT_TRY(sizes_ok("xt_embedding_sorted_bwd_workspace_size", T, d, 1));
  *bytes = part_bytes_for(most_chunks(T, d), d);
  return XT_OK;
}

int xt_embedding_sorted_bwd(const void* plan, size_t plan_bytes, const void* dh, void* dE, int64_t T, int64_t d,
                            int64_t V, float scale, int dt_dh, int dt_grad, int acc, void* ws, size_t ws_bytes,
                            void* stream) {
  const char* fn = "xt_embedding_sorted_bwd";
  XT_TRY(sizes_ok(fn, T, d, V));
  XT_REQUIRE(valid_dtype(dt_dh) && valid_dtype(dt_grad), "%s: bad dtype", fn);
  XT_REQUIRE(acc == 0 || acc == 1, "%s: acc must be 0 or 1", fn);
  XT_REQUIRE(plan && plan_bytes >= plan_bytes_for(T), "%s: the plan holds %zu bytes, %zu are needed", fn,
             plan ? plan_bytes : size_t(0), plan_bytes_for(T));
  if (!aligned16(plan)) return fail(XT_ERR_ALIGNMENT, "%s: the plan must be 16-byte aligned", fn);
  XT_REQUIRE(dE && (T == 0 || dh), "%s: NULL pointer", fn);
  const size_t need = part_bytes_for(ceil_div(T, chunk_tokens(T, d)), d);
  XT_REQUIRE(need == 0 || (ws && ws_bytes >= need), "%s: the workspace holds %zu bytes, %zu are needed", fn,
             ws ? ws_bytes : size_t(0), need);
  if (ws && !aligned16(ws)) return fail(XT_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", fn);
  Grad a{};
  a.plan = plan;
  a.dh = dh;
  a.dE = dE;
  a.part = static_cast<float*>(ws);
  a.T = T;
  a.d = d;
  a.V = V;
  a.chunk = chunk_tokens(T, d);
  a.chunks = ceil_div(T, a.chunk);
  a.tiles = ceil_div(d, kCols);
  a.zero_units = acc ? 0 : ceil_div(V, 32);
  a.scale = scale;
  a.acc = acc;
  a.flag = errflag();
  const int64_t grid = ceil_div(a.chunks * a.tiles + a.zero_units, kWarps);
  if (grid == 0) return XT_OK;
  if (grid >= (int64_t(1) << 31)) return fail(XT_ERR_UNSUPPORTED, "%s: too many tokens", fn);
  const int64_t joins = a.chunks > 1 ? ceil_div(a.chunks * a.tiles, kWarps) : 0;
  const bool vec = d % 8 == 0 && aligned16(dh) && aligned16(dE);
  cudaStream_t s = as_stream(stream);
#define XT_GRAD(T_, TG_, VEC_)                                                                            \
  do {                                                                                                    \
    launch(embedding_grad_kernel<T_, TG_, VEC_>, unsigned(grid), kWarps * 32, 0, s, a);                   \
    XT_TRY(check_launch(fn));                                                                             \
    if (joins) {                                                                                          \
      launch(embedding_join_kernel<TG_, VEC_>, unsigned(joins), kWarps * 32, 0, s, a);                    \
      XT_TRY(check_launch(fn));                                                                           \
    }                                                                                                     \
  } while (0)
#define XT_GRAD_T(T_, TG_)                  \
  do {                                      \
    if (vec) XT_GRAD(T_, TG_, true);        \
    else XT_GRAD(T_, TG_, false);           \
  } while (0)
  if (dt_dh == XT_BF16) {
    if (dt_grad == XT_BF16) XT_GRAD_T(bf16, bf16);
    else XT_GRAD_T(bf16, float);
  } else {
    if (dt_grad == XT_BF16) XT_GRAD_T(float, bf16);
    else XT_GRAD_T(float, float);
  }
#undef XT_GRAD_T
#undef XT_GRAD
  return XT_OK;
}

}  // extern "C"
