// The Muon step over matrices W [rows, cols] with float32 master weights, gradients G and momenta M:
//   M ← μ M + s·G,   U = s·G + μ M (nesterov; else M),   X₀ = U / (‖U‖_F + ε),
//   X ← a X + (b A + c A²) X,  A = X Xᵀ   (Xᵀ X, multiplied from the right, where rows > cols),   `steps` times,
//   W ← W (1 − lr·λ) − lr·rms·√max(rows, cols)·X.
//
// Precision.  The polynomial's slope at 0 is a = 3.44, so what is rounded off X₀ grows by up to a⁵ = 485 in the
// directions of small singular values: with every operand rounded to bf16 X comes out with a relative error of a few
// 10⁻², to f16 of a few 10⁻³.  Here X, A and B = b A + c A² are held as two f16 terms each (value and remainder, scaled by
// 2¹⁰: 22 bits of what is at least 2⁻³ as held, 1.2·10⁻⁴ of X; the remainders of smaller entries are subnormal, and what is held
// is good to 2⁻²⁵, 3·10⁻¹¹ of X; singular values stay below 1.21, entries of B below 16), and a product is three:
// hi·lo + lo·hi + hi·hi, float32 sums in tensor memory.  The sums there are cut off, not rounded, after every 16 elements of K:
// the small products come first, while the sum is small.  X is then good to a few 10⁻⁶ at three times the operations of a
// single f16 product: two to five times what float32 products leave, more with a longer K (the weights of 12 layers of width 768
// after a step 2.3·10⁻⁶ against 4.9·10⁻⁷ in norm).
//
// Work.  A and A² are symmetric: only the tiles on and above the diagonal are computed, the others written from them.
// Matrices of one shape form a batch, up to kMaxGroups shapes run in one launch, so that the tiles of all of a model's
// matrices fill the GPU together: three launches per iteration whatever the list.
//
// The product kernel is warp-specialised as the GEMM is: TMA producer, MMA issuer (CTA pairs, 256 × 256 tiles,
// tcgen05 kind::f16 on f16; 128 × 128 ones of single CTAs for few matrices), eight epilogue warps; bounded waits.  Tensor-bound.
// On one GB300, 48 matrices of a 12-layer stack of width 768 (us): A 184 (1418 TFLOP/s of the three products), B 73, X 273 (1430) per
// step, the passes over 85 M weights 141, 174 and 169 (at HBM's rate): 3390 in all; four matrices of width 256 222.
#include <cuda_fp16.h>

#include <cmath>
#include <atomic>
#include <cfloat>
#include <cstring>

#include "gemm.cuh"
#include "internal.cuh"

namespace xt {
namespace muon {

using namespace gemm;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 1024.f;   // of X, A and B as held
constexpr int kMaxGroups = 8;
constexpr int kMaxMatrices = 128;  // of an elementwise launch (its table travels in the parameters)

// ------------------------------------------------------------------------------ products

// A tile's edge is BM for each of the CG CTAs that share it: pairs of CTAs with 256 × 256 tiles, or single ones with
// 128 × 128 where the others would leave most of the GPU idle (see products()).
constexpr int kBk = 128;           // K elements per stage: two swizzle atoms
constexpr int kAtom = 64, kAtoms = kBk / kAtom;
constexpr int kOperandBytes = BM * kBk * 2;  // each CTA stages 128 rows of either operand
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kStagingBytes = kEpilogueWarps * 4096;
constexpr int kSmem = 1024 + kStages * kStageBytes + kStagingBytes + 256;
constexpr int kProductThreads = 64 + 32 * kEpilogueWarps;

// Matrices of one shape: C = alpha·P Q + beta·D as two f16 terms.
struct Group {
  CUtensorMap tp, tq, tc;   // P [M, K], Q [N, K] (either of them MN-major); C; (.., .., batch, term)
  const __half* d;          // D's first term (null: beta = 0); the second d_term further
  __half* c;                // C's first term, for the mirrored tiles
  int64_t d_term, d_batch, c_term, c_batch;
  int ld, M, N;             // of C and D
  int k_blocks;             // of one term's K
  int num_m, num_n, tile0, tiles;  // tiles of a matrix; the group's first tile and number of tiles
  int p_mn, q_mn, sym;
  float alpha, beta;
};
struct Products {
  Group g[kMaxGroups];
  int groups, tiles;
  uint32_t* flag;
  uint64_t wait_ns;
};

struct Place {
  int g, batch, m, n;  // group, matrix, tile row and column
};
__device__ __forceinline__ Place place_of(const Products& a, int t) {
  Place w;
  w.g = 0;
  while (w.g + 1 < a.groups && t >= a.g[w.g + 1].tile0) ++w.g;
  const Group& g = a.g[w.g];
  const int per = g.sym ? g.num_m * (g.num_m + 1) / 2 : g.num_m * g.num_n;
  t -= g.tile0;
  w.batch = t / per;
  int r = t - w.batch * per;
  if (g.sym) {  // column by column of the upper triangle
    w.n = 0;
    while (r > w.n) {
      r -= w.n + 1;
      ++w.n;
    }
    w.m = r;
  } else {
    w.n = r / g.num_m;  // m fastest: neighbours share Q's tiles
    w.m = r - w.n * g.num_m;
  }
  return w;
}

template <int kCg>
__global__ void __launch_bounds__(kProductThreads, 1) muon_product_kernel(const __grid_constant__ Products a) {
  constexpr int kTile = BM * kCg;
  const int rank = kCg == 2 ? int(cluster_ctarank()) & 1 : 0;
  const int unit = int(blockIdx.x) / kCg, units = int(gridDim.x) / kCg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(staging + kStagingBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* tfull = bars + 2 * kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tfull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* counts = reinterpret_cast<volatile int*>(tfull + 6);  // fills asked for by either CTA (see the end)
  static_assert((2 * kStages + 6) * 8 + kCg * 4 <= 256, "room for the barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), kEpilogueWarps * kCg);
    }
    mbar_init(smem_u32(mma_done), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane < a.groups) {
    prefetch_tmap(&a.g[lane].tp);
    prefetch_tmap(&a.g[lane].tq);
    prefetch_tmap(&a.g[lane].tc);
  }
  if (warp == 1) {
    tmem_alloc_cg<kCg>(smem_u32(tmem_slot), 2 * kTile);
    tmem_relinquish_cg<kCg>();
  }
  tc_fence_before();
  if constexpr (kCg == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  auto give_up = [&]() {  // both CTAs of a pair stop
    if constexpr (kCg == 2) {
      cluster_give_up<2>(smem_u32(const_cast<int*>(abort_flag)), a.flag);
    } else {
      *abort_flag = 1;
      flag_error(a.flag, XT_DEVERR_TIMEOUT);
    }
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------------ TMA producer
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int t = unit; t < a.tiles && !*abort_flag; t += units) {
        const Place w = place_of(a, t);
        const Group& g = a.g[w.g];
        const int m0 = w.m * kTile + rank * BM, n0 = w.n * kTile + rank * BM;
        for (int kb = 0; kb < 3 * g.k_blocks; ++kb) {
          if (*abort_flag) break;
          if (!mbar_wait_spin(smem_u32(&empty[stage]), phase ^ 1, a.wait_ns)) { give_up(); break; }
          if (rank == 0) mbar_expect_tx(smem_u32(&full[stage]), kCg * kStageBytes);
          const uint32_t fb = kCg == 2 ? mapa_shared(smem_u32(&full[stage]), 0) : smem_u32(&full[stage]);
          auto load = [&](uint32_t dst, const CUtensorMap* tm, int c0, int c1, int z) {
            if constexpr (kCg == 2) tma_load_4d_pair(dst, tm, fb, c0, c1, w.batch, z);
            else tma_load_4d(dst, tm, fb, c0, c1, w.batch, z);
          };
          const uint32_t p_s = smem_u32(smem + stage * kStageBytes), q_s = p_s + kOperandBytes;
          const int term = kb / g.k_blocks, k0 = (kb - term * g.k_blocks) * kBk;
          const int zp = term == 1, zq = term == 0;  // hi·lo, lo·hi, hi·hi
#pragma unroll
          for (int c = 0; c < kAtoms; ++c) {
            if (g.p_mn) load(p_s + c * (kBk * 128), &g.tp, m0 + c * kAtom, k0, zp);
            else load(p_s + c * (BM * 128), &g.tp, k0 + c * kAtom, m0, zp);
          }
#pragma unroll
          for (int c = 0; c < kAtoms; ++c) {
            if (g.q_mn) load(q_s + c * (kBk * 128), &g.tq, n0 + c * kAtom, k0, zq);
            else load(q_s + c * (BM * 128), &g.tq, k0 + c * kAtom, n0, zq);
          }
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      // copies that may still be in flight land before the CTA exits (in a pair the MMA issuer has waited for every fill
      // unless a wait ran out: see the end)
      if constexpr (kCg == 1) {
        for (int i = 0; i < kStages && i < issued; ++i) {
          if (--stage < 0) { stage = kStages - 1; phase ^= 1; }
          if (!mbar_wait(smem_u32(&full[stage]), phase)) { give_up(); break; }
        }
      } else {
        counts[rank] = issued;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ------------------------------------------------------------------ MMA issuer
      int stage = 0, ab = 0;
      uint32_t phase = 0, aphase = 0;
      bool any = false;
      for (int t = unit; t < a.tiles && !*abort_flag; t += units) {
        const Place w = place_of(a, t);
        const Group& g = a.g[w.g];
        // f16 operands, float32 sums; a K step is 16 elements: 32 bytes along a K-major row, 16 rows MN-major
        const uint32_t idesc = (1u << 4) | (uint32_t(g.p_mn) << 15) | (uint32_t(g.q_mn) << 16) |
                               (uint32_t(kTile >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
        const int p_mn = g.p_mn, q_mn = g.q_mn, blocks = 3 * g.k_blocks;
        if (!mbar_wait_spin(smem_u32(&tempty[ab]), aphase ^ 1, a.wait_ns)) { give_up(); break; }
        tc_fence_after();
        bool ok = true;
        for (int kb = 0; kb < blocks; ++kb) {
          const bool landed = mbar_wait_spin(smem_u32(&full[stage]), phase, a.wait_ns);
          if (*abort_flag || !landed) { ok = false; break; }
          tc_fence_after();
          const uint32_t p_s = smem_u32(smem + stage * kStageBytes), q_s = p_s + kOperandBytes;
#pragma unroll
          for (int kk = 0; kk < kBk / 16; ++kk) {
            const uint32_t major = uint32_t((kk / 4) * (BM * 128) + (kk % 4) * 32), minor = uint32_t(kk * 16 * 128);
            const uint64_t pd = p_mn ? smem_desc(p_s + minor, kBk * 128, 1024) : smem_desc(p_s + major, 16, 1024);
            const uint64_t qd = q_mn ? smem_desc(q_s + minor, kBk * 128, 1024) : smem_desc(q_s + major, 16, 1024);
            tc_mma<kBf16, kCg>(tbase + uint32_t(ab * kTile), pd, qd, idesc, (kb | kk) ? 1u : 0u);
          }
          any = true;
          tc_commit_cg<kCg>(smem_u32(&empty[stage]));
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) { give_up(); break; }
        tc_commit_cg<kCg>(smem_u32(&tfull[ab]));
        if (++ab == 2) { ab = 0; aphase ^= 1; }
      }
      if (any) {
        tc_commit_cg<kCg>(smem_u32(mma_done));
        if (!mbar_wait(smem_u32(mma_done), 0)) give_up();
      }
    }
  } else {
    // -------------------------------------------------------------------- epilogue
    // Two warps to a quadrant of tensor memory's lanes, half of the columns each, 32 columns at a time: D's two terms
    // come two pieces ahead, whole sectors to a load (row 8·j + lane/4, 16 bytes of 64), pass through the warp's two
    // boxes (32 rows × 64 bytes, 64-byte swizzle) to the lanes' own rows, and the result leaves from the same boxes.
    // (Four warps that read D with a row to a lane: 20 us for a single tile, 4.1 ms a step of the 12-layer stack.)
    const int q = warp & 3, half0 = ((warp - 2) >> 2) * (kTile / 2);
    int ab = 0;
    uint32_t aphase = 0;
    const uint32_t box = smem_u32(staging) + uint32_t((warp - 2) * 4096);
    const uint32_t tempty0 = smem_u32(&tempty[0]), tempty_at = kCg == 2 ? mapa_shared(tempty0, 0) : tempty0;
    for (int t = unit; t < a.tiles; t += units) {
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const Place w = place_of(a, t);
      const Group& g = a.g[w.g];
      const int y = w.m * kTile + rank * BM + q * 32, row = y + lane, x0 = w.n * kTile + half0;
      const int M = g.M, N = g.N, ld = g.ld;
      const bool with_d = g.d != nullptr;
      const float alpha = g.alpha, beta = g.beta;
      const int dr = y + (lane >> 2), dc = (lane & 3) * 8;
      const __half* d = with_d ? g.d + w.batch * g.d_batch + int64_t(dr) * ld + dc : nullptr;
      const int64_t d_term = g.d_term;
      auto load_d = [&](uint4 (&hi)[4], uint4 (&lo)[4], int x) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = with_d && dr + 8 * j < M && x + dc < N;
          const __half* p = d + int64_t(8 * j) * ld + x;
          hi[j] = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
          lo[j] = in ? __ldg(reinterpret_cast<const uint4*>(p + d_term)) : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      uint4 hi[2][4], lo[2][4];
      load_d(hi[0], lo[0], x0);
      load_d(hi[1], lo[1], x0 + 32);
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&tfull[ab]), aphase, a.wait_ns));
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      tc_fence_after();
      const bool mirror = g.sym && w.m != w.n && row < M;
      __half* cm = g.c + w.batch * g.c_batch + row;  // the mirrored element (x + k, row)
      const int64_t c_term = g.c_term;
#pragma unroll 1
      for (int c2 = 0; c2 < kTile / 64; c2 += 2) {
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int c = c2 + o, x = x0 + c * 32;
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(tbase + (uint32_t(q * 32) << 16) + uint32_t(ab * kTile + half0 + c * 32), r);
          tmem_ld_wait();
          if (c == kTile / 64 - 1) {  // the accumulator is read: the next tile's products may start
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank) mbar_arrive_cluster(tempty_at + uint32_t(ab * 8));
              else mbar_arrive(tempty0 + uint32_t(ab * 8));
            }
          }
          if (y >= M || x >= N) continue;
          if (lane == 0) bulk_wait_read_0();  // the last piece's boxes have been read
          __syncwarp();
          if (with_d) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int rw = 8 * j + (lane >> 2);
              const uint32_t to = box + uint32_t(rw) * 64 + (uint32_t((lane & 3) ^ ((rw >> 1) & 3)) << 4);
              st_shared_v4(to, hi[o][j].x, hi[o][j].y, hi[o][j].z, hi[o][j].w);
              st_shared_v4(to + 2048, lo[o][j].x, lo[o][j].y, lo[o][j].z, lo[o][j].w);
            }
            __syncwarp();
            if (c + 2 < kTile / 64) load_d(hi[o], lo[o], x + 64);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t at = box + uint32_t(lane) * 64 + (uint32_t(j ^ ((lane >> 1) & 3)) << 4);
            uint4 vh4 = make_uint4(0u, 0u, 0u, 0u), vl4 = vh4;
            if (with_d) {
              vh4 = ld_shared_v4(at);
              vl4 = ld_shared_v4(at + 2048);
            }
            const uint32_t dh[4] = {vh4.x, vh4.y, vh4.z, vh4.w}, dl[4] = {vl4.x, vl4.y, vl4.z, vl4.w};
            uint32_t oh[4], ol[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 vh = __half22float2(*reinterpret_cast<const __half2*>(&dh[e]));
              const float2 vl = __half22float2(*reinterpret_cast<const __half2*>(&dl[e]));
              const float v0 = fmaf(beta, vh.x + vl.x, alpha * __uint_as_float(r[8 * j + 2 * e]));
              const float v1 = fmaf(beta, vh.y + vl.y, alpha * __uint_as_float(r[8 * j + 2 * e + 1]));
              const __half2 h = __floats2half2_rn(v0, v1);
              const float2 back = __half22float2(h);
              const __half2 l = __floats2half2_rn(v0 - back.x, v1 - back.y);
              oh[e] = *reinterpret_cast<const uint32_t*>(&h);
              ol[e] = *reinterpret_cast<const uint32_t*>(&l);
              if (mirror) {
                const int k = x + 8 * j + 2 * e;
                __half* m = cm + int64_t(k) * ld;
                if (k < N) {
                  m[0] = __low2half(h);
                  m[c_term] = __low2half(l);
                }
                if (k + 1 < N) {
                  m[ld] = __high2half(h);
                  m[ld + c_term] = __high2half(l);
                }
              }
            }
            st_shared_v4(at, oh[0], oh[1], oh[2], oh[3]);
            st_shared_v4(at + 2048, ol[0], ol[1], ol[2], ol[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_4d(&g.tc, box, x, y, w.batch, 0);
            tma_store_4d(&g.tc, box + 2048, x, y, w.batch, 1);
            bulk_commit();
          }
        }
      }
      if (++ab == 2) { ab = 0; aphase ^= 1; }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncthreads();
  // neither CTA releases tensor memory or exits while the other may still signal its barriers or read its operands
  if constexpr (kCg == 2) {
    cluster_sync_all();
    if (*abort_flag)  // in both alike; as in the GEMM, every copy that either CTA asked for lands before one of them exits
      cluster_finish<kStages, 1>(smem_u32(full), smem_u32(const_cast<int*>(counts)), kOperandBytes, kOperandBytes, a.flag);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<kCg>(tbase, 2 * kTile);
  }
}

// ------------------------------------------------------------------------------ elementwise passes

constexpr int kElemThreads = 256;
constexpr int kElemTile = 8192;  // elements of a block's piece

struct Matrix {
  float* p;
  const float* g;
  float* m;
  void* w;          // working copy (may be null)
  __half* x;        // X's first term; the second x_term further
  int64_t n, x_term;
  int cols, ld;
  int tile0;        // first piece
  float step;       // lr·rms·√max(rows, cols)
};
struct Table {
  Matrix m[kMaxMatrices];
  int count, tiles;
  double* part;     // Σ U² of every piece
  float momentum, scale, eps, decay;
  int nesterov;
};
__device__ __forceinline__ int matrix_of(const Table& a, int t) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.m[mid].tile0 <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The block's sum, in every thread.
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kElemThreads / 32; ++i) v += red[i];
  return v;
}

// M ← μ M + s·G and each piece's Σ U².
__global__ void __launch_bounds__(kElemThreads) muon_momentum_kernel(const __grid_constant__ Table a) {
  pdl_begin();
  __shared__ float red[kElemThreads / 32];
  const Matrix& k = a.m[matrix_of(a, blockIdx.x)];
  const int64_t base = int64_t(int(blockIdx.x) - k.tile0) * kElemTile;
  const int64_t len = k.n - base < kElemTile ? k.n - base : kElemTile;
  const float* g = k.g + base;
  float* m = k.m + base;
  float sum = 0.f;
  auto one = [&](float gv, float& mv) {
    const float sg = gv * a.scale;
    mv = fmaf(a.momentum, mv, sg);
    const float u = a.nesterov ? fmaf(a.momentum, mv, sg) : mv;
    sum = fmaf(u, u, sum);
  };
  if (((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(m)) & 15) == 0) {
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < len / 4; i += kElemThreads) {
      const float4 gv = __ldg(reinterpret_cast<const float4*>(g) + i);
      float4 mv = reinterpret_cast<const float4*>(m)[i];
      one(gv.x, mv.x);
      one(gv.y, mv.y);
      one(gv.z, mv.z);
      one(gv.w, mv.w);
      reinterpret_cast<float4*>(m)[i] = mv;
    }
    for (int64_t i = len / 4 * 4 + threadIdx.x; i < len; i += kElemThreads) one(g[i], m[i]);
  } else {
    for (int64_t i = threadIdx.x; i < len; i += kElemThreads) one(g[i], m[i]);
  }
  sum = group_reduce<false>(sum, kElemThreads, red);
  double total = double(sum);
  // squares beyond float32's range, or so small that they lost bits there: over again in doubles, from the new momentum (the
  // block's stores lie before the barriers above)
  if (!(sum >= 1e-20f && sum <= FLT_MAX)) {
    __shared__ double red64[kElemThreads / 32];
    total = 0;
    for (int64_t i = threadIdx.x; i < len; i += kElemThreads) {
      const double u = double(a.nesterov ? fmaf(a.momentum, m[i], g[i] * a.scale) : m[i]);
      total = fma(u, u, total);
    }
    total = block_sum(total, red64);
  }
  if (threadIdx.x == 0) a.part[blockIdx.x] = total;
}

// 8 elements of a row of a matrix whose rows are whole 16 bytes, or one.
template <int W> struct Terms {
  __device__ __forceinline__ static void store(__half* hi, __half* lo, const float (&v)[W]) {
    if constexpr (W == 8) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 a = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        const float2 back = __half22float2(a);
        const __half2 b = __floats2half2_rn(v[2 * i] - back.x, v[2 * i + 1] - back.y);
        h[i] = *reinterpret_cast<const uint32_t*>(&a);
        l[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
    } else {
      const __half a = __float2half_rn(v[0]);
      *hi = a;
      *lo = __float2half_rn(v[0] - __half2float(a));
    }
  }
  __device__ __forceinline__ static void load(const __half* hi, const __half* lo, float (&v)[W]) {
    if constexpr (W == 8) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(hi)), b = __ldg(reinterpret_cast<const uint4*>(lo));
      const uint32_t h[4] = {a.x, a.y, a.z, a.w}, l[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&l[i]));
        v[2 * i] = x.x + y.x;
        v[2 * i + 1] = x.y + y.y;
      }
    } else {
      v[0] = __half2float(*hi) + __half2float(*lo);
    }
  }
};

// Rows of whole vectors and aligned buffers: then no vector crosses a row.
__device__ __forceinline__ bool whole_rows(const Matrix& k, const void* a, const void* b) {
  return k.cols % 8 == 0 && ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

// X₀ from the new momentum, in two terms.
template <int W>
__device__ __forceinline__ void begin_piece(const Table& a, const Matrix& k, int64_t base, int64_t len, float f1, float f2) {
  for (int64_t i = threadIdx.x * W; i < len; i += kElemThreads * W) {
    float g[W], m[W];
    if constexpr (W == 8) {
      V8<float>::load(k.g + base + i, g);
      V8<float>::load(k.m + base + i, m);
    } else {
      g[0] = k.g[base + i];
      m[0] = k.m[base + i];
    }
#pragma unroll
    for (int e = 0; e < W; ++e) m[e] = (a.nesterov ? fmaf(a.momentum, m[e], g[e] * a.scale) : m[e]) * f1 * f2;
    const int64_t r = (base + i) / k.cols, at = r * k.ld + (base + i - r * k.cols);
    Terms<W>::store(k.x + at, k.x + k.x_term + at, m);
  }
}
__global__ void __launch_bounds__(kElemThreads) muon_begin_kernel(const __grid_constant__ Table a) {
  pdl_begin();
  __shared__ double red[kElemThreads / 32];
  const Matrix& k = a.m[matrix_of(a, blockIdx.x)];
  const int pieces = int((k.n + kElemTile - 1) / kElemTile);
  double sum = 0;
  for (int i = threadIdx.x; i < pieces; i += kElemThreads) sum += __ldcg(a.part + k.tile0 + i);
  const double f = double(kScale) / (sqrt(block_sum(sum, red)) + double(a.eps));
  // as two factors, the first a power of two: f itself may lie outside float32's range (0 or not a number: the gradient
  // is not finite)
  const int e = ((__double2hiint(f) >> 20) & 0x7ff) - 1023, half = e > -250 && e < 250 ? e / 2 : 0;
  const float f1 = __int_as_float((127 + half) << 23);
  const float f2 = float(f * __hiloint2double((1023 - half) << 20, 0));
  const int64_t base = int64_t(int(blockIdx.x) - k.tile0) * kElemTile;
  const int64_t len = k.n - base < kElemTile ? k.n - base : kElemTile;
  if (whole_rows(k, k.g, k.m)) begin_piece<8>(a, k, base, len, f1, f2);
  else begin_piece<1>(a, k, base, len, f1, f2);
}

// W ← W (1 − lr·λ) − step·X, and the working copy.
template <typename TS, int W>
__device__ __forceinline__ void apply_piece(const Table& a, const Matrix& k, int64_t base, int64_t len) {
  const float s = k.step / kScale;
  for (int64_t i = threadIdx.x * W; i < len; i += kElemThreads * W) {
    const int64_t r = (base + i) / k.cols, at = r * k.ld + (base + i - r * k.cols);
    float x[W], p[W];
    Terms<W>::load(k.x + at, k.x + k.x_term + at, x);
    if constexpr (W == 8) V8<float>::load(k.p + base + i, p);
    else p[0] = k.p[base + i];
#pragma unroll
    for (int e = 0; e < W; ++e) p[e] = fmaf(p[e], a.decay, -s * x[e]);
    Acc<float, W>::store(k.p + base + i, p);
    if (k.w) Acc<TS, W>::store(static_cast<TS*>(k.w) + base + i, p);
  }
}
template <typename TS>
__global__ void __launch_bounds__(kElemThreads) muon_apply_kernel(const __grid_constant__ Table a) {
  pdl_begin();
  const Matrix& k = a.m[matrix_of(a, blockIdx.x)];
  const int64_t base = int64_t(int(blockIdx.x) - k.tile0) * kElemTile;
  const int64_t len = k.n - base < kElemTile ? k.n - base : kElemTile;
  if (whole_rows(k, k.p, k.w)) apply_piece<TS, 8>(a, k, base, len);
  else apply_piece<TS, 1>(a, k, base, len);
}

// ------------------------------------------------------------------------------ host

// Matrices of one shape and where their workspace lies (in elements of f16 from the workspace's start).
struct Shape {
  int64_t rows, cols;
  int count;
  int64_t k, ld, ldk;          // the smaller side; row strides of X, and of A and B
  int64_t x_term, a_term;      // elements of a term: count matrices
  int64_t x0, x1, a, b;
};
constexpr int kMaxShapes = 64;

struct Layout {
  Shape shape[kMaxShapes];
  int shapes = 0;
  int64_t pieces = 0;   // of all matrices
  int64_t halves = 0;   // elements of f16 in all
  size_t bytes() const { return part_bytes() + size_t(halves) * 2; }
  size_t part_bytes() const { return (size_t(pieces) * sizeof(double) + 255) & ~size_t(255); }
  int find(int64_t rows, int64_t cols) const {
    for (int i = 0; i < shapes; ++i)
      if (shape[i].rows == rows && shape[i].cols == cols) return i;
    return -1;
  }
};

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

int plan(Layout& l, const char* fn, int n, const int64_t* rows, const int64_t* cols) {
  XT_REQUIRE(n >= 0 && (n == 0 || (rows && cols)), "%s: bad matrix list", fn);
  for (int i = 0; i < n; ++i) {
    XT_REQUIRE(rows[i] > 0 && cols[i] > 0, "%s: matrix %d has no elements", fn, i);
    XT_REQUIRE(rows[i] <= (1 << 20) && cols[i] <= (1 << 20) && rows[i] * cols[i] < (int64_t(1) << 31),
               "%s: matrix %d is too large", fn, i);
    int at = l.find(rows[i], cols[i]);
    if (at < 0) {
      if (l.shapes == kMaxShapes) return fail(XT_ERR_UNSUPPORTED, "%s: more than %d shapes", fn, kMaxShapes);
      at = l.shapes++;
      l.shape[at] = Shape{};
      l.shape[at].rows = rows[i];
      l.shape[at].cols = cols[i];
    }
    XT_REQUIRE(++l.shape[at].count < (1 << 20), "%s: too many matrices", fn);
    l.pieces += ceil_div(rows[i] * cols[i], kElemTile);
    XT_REQUIRE(l.pieces < (int64_t(1) << 30), "%s: too many elements", fn);
  }
  for (int i = 0; i < l.shapes; ++i) {
    Shape& s = l.shape[i];
    s.k = s.rows < s.cols ? s.rows : s.cols;
    s.ld = up(s.cols, 8);
    s.ldk = up(s.k, 8);
    s.x_term = up(s.count * s.rows * s.ld, 128);
    s.a_term = up(s.count * s.k * s.ldk, 128);
    s.x0 = l.halves;
    s.x1 = s.x0 + 2 * s.x_term;
    s.a = s.x1 + 2 * s.x_term;
    s.b = s.a + 2 * s.a_term;
    l.halves = s.b + 2 * s.a_term;
  }
  return XT_OK;
}

// A matrix batch [2 terms][count][rows][ld] as the product kernel reads (boxes 64 wide) or stores it (32 × 32 boxes).
int make_map(CUtensorMap* tm, __half* base, int64_t rows, int64_t cols, int64_t ld, int count, int64_t term, uint32_t bx,
             uint32_t by) {
  auto enc = encode_fn();
  if (!enc) return fail(XT_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[4] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(count), 2};
  cuuint64_t strides[3] = {cuuint64_t(ld * 2), cuuint64_t(rows * ld * 2), cuuint64_t(term * 2)};
  cuuint32_t box[4] = {bx, by, 1, 1}, estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, bx == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(XT_ERR_CUDA, "cuTensorMapEncodeTiled (muon) failed (%d)", int(r));
  return XT_OK;
}

// One of an iteration's products over the shapes [first, first + count): 0 A = X Xᵀ, 1 B = b A + c A², 2 X ← a X + B X.
int products(const Layout& l, int first, int count, int which, int flip, __half* ws, cudaStream_t s) {
  Products a{};
  a.groups = count;
  // 256 × 256 tiles where they fill half of the pairs (and pairs may be used at all)
  const int pairs = pairing() == 1 ? 0 : pair_capacity();
  int64_t big = 0;
  for (int i = 0; i < count; ++i) {
    const Shape& sh = l.shape[first + i];
    const int64_t nk = ceil_div(sh.k, 2 * BM);
    big += sh.count * (which < 2 ? nk * (nk + 1) / 2 : ceil_div(sh.rows, 2 * BM) * ceil_div(sh.cols, 2 * BM));
  }
  const int cg = pairs > 0 && 2 * big >= pairs ? 2 : 1, tile = BM * cg;
  for (int i = 0; i < count; ++i) {
    const Shape& sh = l.shape[first + i];
    Group& g = a.g[i];
    __half* x = ws + (flip ? sh.x1 : sh.x0);
    __half* xn = ws + (flip ? sh.x0 : sh.x1);
    __half *A = ws + sh.a, *B = ws + sh.b;
    const bool tall = sh.rows > sh.cols;
    auto square = [&](CUtensorMap* tm, __half* p, uint32_t by) {
      return make_map(tm, p, sh.k, sh.k, sh.ldk, sh.count, sh.a_term, by == 32 ? 32 : kAtom, by);
    };
    auto matrix = [&](CUtensorMap* tm, __half* p, uint32_t by) {
      return make_map(tm, p, sh.rows, sh.cols, sh.ld, sh.count, sh.x_term, by == 32 ? 32 : kAtom, by);
    };
    int64_t K;
    if (which == 0) {
      // the sum runs over the longer side: along X's rows, or (rows > cols) over them
      g.p_mn = g.q_mn = tall;
      K = tall ? sh.rows : sh.cols;
      XT_TRY(matrix(&g.tp, x, tall ? kBk : BM));
      g.tq = g.tp;
      XT_TRY(square(&g.tc, A, 32));
      g.alpha = 1.f / kScale;
    } else if (which == 1) {
      K = sh.k;
      XT_TRY(square(&g.tp, A, BM));
      g.tq = g.tp;
      XT_TRY(square(&g.tc, B, 32));
      g.alpha = kC / kScale;
      g.beta = kB;
      g.d = A;
    } else {
      K = sh.k;
      if (tall) {
        XT_TRY(matrix(&g.tp, x, BM));
        XT_TRY(square(&g.tq, B, BM));
      } else {
        XT_TRY(square(&g.tp, B, BM));
        XT_TRY(matrix(&g.tq, x, kBk));
        g.q_mn = 1;
      }
      XT_TRY(matrix(&g.tc, xn, 32));
      g.alpha = 1.f / kScale;
      g.beta = kA;
      g.d = x;
    }
    g.sym = which < 2;
    g.M = int(which < 2 ? sh.k : sh.rows);
    g.N = int(which < 2 ? sh.k : sh.cols);
    g.ld = int(which < 2 ? sh.ldk : sh.ld);
    g.c = which == 0 ? A : which == 1 ? B : xn;
    g.c_term = g.d_term = which < 2 ? sh.a_term : sh.x_term;
    g.c_batch = g.d_batch = int64_t(g.M) * g.ld;
    g.k_blocks = int(ceil_div(K, kBk));
    g.num_m = int(ceil_div(g.M, tile));
    g.num_n = int(ceil_div(g.N, tile));
    g.tile0 = a.tiles;
    const int64_t per = g.sym ? int64_t(g.num_m) * (g.num_m + 1) / 2 : int64_t(g.num_m) * g.num_n;
    if (a.tiles + per * sh.count >= (int64_t(1) << 30)) return fail(XT_ERR_UNSUPPORTED, "xt_muon_step: too many tiles");
    g.tiles = int(per * sh.count);
    a.tiles += g.tiles;
  }
  a.flag = errflag();
  a.wait_ns = wait_limit_ns();
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("xt_muon_step");
  if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
    if (cudaFuncSetAttribute(muon_product_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(muon_product_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return check_launch("xt_muon_step: shared memory attribute");
    if (dev < 64) set.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  if (cg == 2)
    launch_clustered(muon_product_kernel<2>, 2 * (a.tiles < pairs ? a.tiles : pairs), kProductThreads, kSmem, s, 2, a);
  else
    launch(muon_product_kernel<1>, a.tiles < num_sms() ? a.tiles : num_sms(), kProductThreads, kSmem, s, a);
  return check_launch("xt_muon_step (product)");
}

}  // namespace muon
}  // namespace xt

using namespace xt;

extern "C" {

int xt_muon_workspace_size(int n, const int64_t* rows, const int64_t* cols, size_t* bytes) {
  XT_REQUIRE(bytes != nullptr, "xt_muon_workspace_size: NULL pointer");
  muon::Layout l;
  XT_TRY(muon::plan(l, "xt_muon_workspace_size", n, rows, cols));
  *bytes = l.bytes();
  return XT_OK;
}

int xt_muon_step(const xt_muon_config* cfg, int n, float* const* param, const float* const* grad, float* const* momentum,
                 void* const* shadow, int shadow_dtype, const int64_t* rows, const int64_t* cols, void* ws,
                 size_t ws_bytes, void* stream) {
  const char* fn = "xt_muon_step";
  XT_REQUIRE(cfg != nullptr, "%s: cfg is NULL", fn);
  muon::Layout l;
  XT_TRY(muon::plan(l, fn, n, rows, cols));
  XT_REQUIRE(cfg->momentum >= 0.f && cfg->momentum < 1.f, "%s: momentum must be in [0, 1)", fn);
  XT_REQUIRE(cfg->lr >= 0.f && cfg->weight_decay >= 0.f && cfg->rms >= 0.f && cfg->eps > 0.f && std::isfinite(cfg->lr) &&
                 std::isfinite(cfg->weight_decay) && std::isfinite(cfg->rms) && std::isfinite(cfg->eps) &&
                 std::isfinite(cfg->grad_scale),
             "%s: bad hyperparameters", fn);
  XT_REQUIRE(cfg->steps >= 1 && cfg->steps <= 20, "%s: steps must lie in [1, 20]", fn);
  XT_REQUIRE(cfg->nesterov == 0 || cfg->nesterov == 1, "%s: nesterov must be 0 or 1", fn);
  XT_REQUIRE(shadow == nullptr || valid_dtype(shadow_dtype), "%s: bad shadow dtype", fn);
  if (n == 0) return XT_OK;
  XT_REQUIRE(param && grad && momentum, "%s: NULL table", fn);
  for (int i = 0; i < n; ++i) XT_REQUIRE(param[i] && grad[i] && momentum[i], "%s: NULL matrix %d", fn, i);
  XT_REQUIRE(ws && ws_bytes >= l.bytes(), "%s: workspace too small (%zu < %zu)", fn, ws ? ws_bytes : size_t(0), l.bytes());
  if (!aligned16(ws)) return fail(XT_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", fn);
  cudaStream_t s = as_stream(stream);
  double* part = static_cast<double*>(ws);
  __half* halves = reinterpret_cast<__half*>(static_cast<char*>(ws) + l.part_bytes());

  // which: 0 momentum and norms, 1 X₀, 2 the update (X is in x1 after an odd number of steps)
  auto elementwise = [&](int which) {
    int used[muon::kMaxShapes] = {};
    int64_t piece = 0;
    for (int first = 0; first < n;) {
      muon::Table a{};
      a.part = part + piece;
      a.momentum = cfg->momentum;
      a.scale = cfg->grad_scale;
      a.eps = cfg->eps;
      a.decay = float(1.0 - double(cfg->lr) * double(cfg->weight_decay));
      a.nesterov = cfg->nesterov;
      for (; first < n && a.count < muon::kMaxMatrices; ++first) {
        const int at = l.find(rows[first], cols[first]);
        const muon::Shape& sh = l.shape[at];
        muon::Matrix& m = a.m[a.count++];
        m.p = param[first];
        m.g = grad[first];
        m.m = momentum[first];
        m.w = shadow ? shadow[first] : nullptr;
        m.x = halves + (which == 2 && cfg->steps % 2 ? sh.x1 : sh.x0) + used[at]++ * sh.rows * sh.ld;
        m.x_term = sh.x_term;
        m.n = sh.rows * sh.cols;
        m.cols = int(sh.cols);
        m.ld = int(sh.ld);
        m.tile0 = a.tiles;
        m.step = float(double(cfg->lr) * double(cfg->rms) * std::sqrt(double(sh.rows > sh.cols ? sh.rows : sh.cols)));
        a.tiles += int(ceil_div(m.n, muon::kElemTile));
      }
      piece += a.tiles;
      if (which == 0) launch(muon::muon_momentum_kernel, a.tiles, muon::kElemThreads, 0, s, a);
      else if (which == 1) launch(muon::muon_begin_kernel, a.tiles, muon::kElemThreads, 0, s, a);
      else if (shadow && shadow_dtype == XT_BF16) launch(muon::muon_apply_kernel<bf16>, a.tiles, muon::kElemThreads, 0, s, a);
      else launch(muon::muon_apply_kernel<float>, a.tiles, muon::kElemThreads, 0, s, a);
      XT_TRY(check_launch(fn));
    }
    return int(XT_OK);
  };
  XT_TRY(elementwise(0));
  XT_TRY(elementwise(1));
  for (int first = 0; first < l.shapes; first += muon::kMaxGroups) {
    const int count = l.shapes - first < muon::kMaxGroups ? l.shapes - first : muon::kMaxGroups;
    for (int i = 0; i < cfg->steps; ++i)
      for (int which = 0; which < 3; ++which) XT_TRY(muon::products(l, first, count, which, i & 1, halves, s));
  }
  return elementwise(2);
}

}  // extern "C"
