// Attention over packed documents with masks, capped scores, a distance bias and shared key / value
// heads, forward and backward, for head dimensions 64 and 128 (bf16).  Per query head h, with key /
// value head h / (H / Hkv), tokens i (query) and j (key):
//   a = scale·q_i·k_j,  c = cap·tanh(a/cap) (cap > 0; else a),  s = c − slope_h·|i − j|,
//   P = softmax of s over the keys that i sees,  O = P V,  lse = log Σ exp s;
//   D_i = dO_i·O_i,  dP = dO Vᵀ,  dS = P∘(dP − D)∘(1 − tanh²),
//   dQ = scale·dS K,  dK = scale·dSᵀ Q,  dV = Pᵀ dO  (dK, dV summed over the query heads that share them).
// What a row sees is an interval of columns (attention_plan.cuh), so a tile is skipped, masked by two
// comparisons per element, or taken whole.
//
// All matrix products run on tcgen05.  P and dS, the left operands of the second products, are written
// back to tensor memory as bf16 over the scores they come from and read from there by the MMA (the
// causal kernel without masks stages P in shared memory and fences it into the async proxy for every tile);
// that also leaves shared memory for 128-wide heads.
//
// Rows whose mask leaves nothing get O = 0, lse = −∞ and zero gradients.  A masked element's P is 0 by
// selection, so whatever its score is (NaN, ∞) stays out of the row; but the products add 0·V for masked
// keys of a tile, which a NaN or ∞ in V turns into NaN.  A row whose result is not finite is therefore
// done over from its visible columns alone (redo_row): the check costs an addition per output element.
#pragma once

#include <type_traits>

#include "attention_plan.cuh"
#include "gemm.cuh"
#include "internal.cuh"

namespace xt {
namespace attnm {

using namespace gemm;
using attn_plan::BT;

constexpr int TILE = BT * 128;  // 128 rows × 64 bf16: one 128-byte-swizzled chunk, 16 KB
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // log2 growth of the running max that forces a rescale of O

struct Params {
  attn_plan::View plan;
  int H, Hkv, group;      // query heads, key / value heads, H / Hkv
  float sc;               // scale·log₂e
  float scale;
  float capk, cap2;       // 2·log₂e·scale/cap, cap·log₂e (CAP)
  const float* slopes;    // [H] (BIAS)
  const bf16 *q, *k, *v;  // rows of ldq, ldk, ldv elements
  int64_t ldq, ldk, ldv;
  bf16 *o, *o_lo;         // o_lo: O − bf16(O), or null
  const bf16 *d_o;
  int64_t ldo, lddo;
  float *lse;             // [H][T]
  float *D;               // [H][T]
  bf16 *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  uint32_t* flag;
  uint64_t wait_ns;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  return f32x2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
// 32 lanes × 16 consecutive columns into registers, and back.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// D[tmem] (+)= A[tmem]·B: A is 128 rows × 16 bf16, two per 32-bit column, row = lane.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, limit_ns));
}

template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The products of 128-row tiles held in shared memory as HD/64 swizzled chunks of TILE bytes.
template <int HD>
struct Mma {
  static constexpr uint32_t kIdescS = instr_desc_bf16(128, 128, false, false);
  static constexpr uint32_t kIdescO = instr_desc_bf16(128, HD, false, true);
  // D = A Bᵀ over the head dimension (both K-major)
  static __device__ __forceinline__ void nt(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint32_t off = uint32_t((kk >> 2) * TILE + (kk & 3) * 32);
      tc_mma<kBf16>(d, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), kIdescS, kk > 0 ? 1u : 0u);
    }
  }
  // D (+)= A B over 128 tokens: A bf16 in tensor memory (k-step kk at a + (kk/4)·skip + 8·(kk%4)), B MN-major
  static __device__ __forceinline__ void tn(uint32_t d, uint32_t a, uint32_t skip, uint32_t b, bool first) {
#pragma unroll
    for (int kk = 0; kk < BT / 16; ++kk)
      tc_mma_ts(d, a + uint32_t(kk >> 2) * skip + uint32_t(kk & 3) * 8, smem_desc(b + kk * 2048, TILE, 1024), kIdescO,
                (!first || kk > 0) ? 1u : 0u);
  }
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int head, int tile) {
#pragma unroll
    for (int c = 0; c < HD / 64; ++c) tma_load_4d(dst + c * TILE, tm, bar, c * 64, head, tile * BT, 0);
  }
};

// r[c] −= slope₂·|d0 + c|.
template <int N>
__device__ __forceinline__ void add_bias(uint32_t (&r)[N], float slope2, int d0, int side) {
  if (side != 0) {
    const float st = side > 0 ? slope2 : -slope2, b0 = st * float(d0);
#pragma unroll
    for (int c = 0; c < N; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) + fmaf(float(c), st, b0));
  } else {
    const float d = float(d0);
#pragma unroll
    for (int c = 0; c < N; ++c) r[c] = __float_as_uint(fmaf(-slope2, fabsf(d + float(c)), __uint_as_float(r[c])));
  }
}

// Scores of one row, r[c] = q·k of column base + c, to s·log₂e (CAP or BIAS; without both the caller
// scales).  d0: column 0 minus the row, in tokens; side: +1 / −1 where every column of the tile lies before
// / behind the row (the distance is then linear in c), 0 else.
template <int N, bool CAP, bool BIAS>
__device__ __forceinline__ void to_log2(uint32_t (&r)[N], const Params& p, float slope2, int d0, int side) {
  if constexpr (CAP) {
#pragma unroll
    for (int c = 0; c < N; ++c) {
      // cap·tanh(a/cap) = cap − 2·cap/(1 + e^{2a/cap}): one exponential, one reciprocal, absolute error ~2⁻²²·cap
      const float e = ex2(__uint_as_float(r[c]) * p.capk);
      r[c] = __float_as_uint(fmaf(-2.f * p.cap2, rcp(1.f + e), p.cap2));
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * p.sc);
  }
  if constexpr (BIAS) add_bias(r, slope2, d0, side);
}

// ------------------------------------------------------------------------------ the careful path

template <int HD>
__device__ __forceinline__ float dot_rows(const bf16* a, const bf16* b) {
  float acc = 0.f;
  for (int c = 0; c < HD; c += 8) {
    float x[8], y[8];
    Vec<bf16>::load(a + c, x);
    Vec<bf16>::load(b + c, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc = fmaf(x[e], y[e], acc);
  }
  return acc;
}

// s·log₂e of one pair and 1 − tanh².
template <bool CAP, bool BIAS>
__device__ __forceinline__ float pair_score(const Params& p, float dot, float slope2, int dist, float& slack) {
  slack = 1.f;
  float s = dot * p.sc;
  if constexpr (CAP) {
    const float e = ex2(dot * p.capk), u = rcp(1.f + e);
    s = fmaf(-2.f * p.cap2, u, p.cap2);
    slack = 4.f * u * (1.f - u);
  }
  if constexpr (BIAS) s = fmaf(-slope2, fabsf(float(dist)), s);
  return s;
}

// One output row from its visible columns alone, by a whole warp: 32 columns at a time, a lane scores
// one, then every lane adds the columns to its HD/32 elements.
//   FWD:  out = Σ_j p_j v_j,               row = query, m2: the running max
//   else: out = Σ dS_ij·(other row), out2 = Σ P_ij·dO_i (KEY), of the row `row` of head h
template <int HD, bool KEY, bool FWD, bool CAP, bool BIAS>
__device__ __noinline__ void redo_row(const Params& p, int h, int kh, int row, int lo, int hi, float m2, float D,
                                      float* out, float* out2) {
  constexpr int W = HD / 32;
  const int lane = threadIdx.x & 31;
  const float slope2 = BIAS ? p.slopes[h] * kLog2e : 0.f;
  const bf16* q = p.q + int64_t(h) * HD;
  const bf16* k = p.k + int64_t(kh) * HD;
  const bf16* v = p.v + int64_t(kh) * HD;
  const bf16* g = FWD ? nullptr : p.d_o + int64_t(h) * HD;
  for (int j0 = lo; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    float pj = 0.f, dsj = 0.f;
    if (j < hi) {
      const int64_t i = KEY ? j : row, c = KEY ? row : j;
      float slack;
      const float s =
          pair_score<CAP, BIAS>(p, dot_rows<HD>(q + i * p.ldq, k + c * p.ldk), slope2, int(i - c), slack);
      float mm = m2, dd = D;
      if constexpr (KEY) {
        mm = p.lse[int64_t(h) * p.plan.T + i] * kLog2e;
        dd = p.D[int64_t(h) * p.plan.T + i];
      }
      pj = ex2(s - mm);
      if constexpr (!FWD) dsj = pj * slack * (dot_rows<HD>(g + i * p.lddo, v + c * p.ldv) - dd);
    }
    for (int u = 0; u < 32 && j0 + u < hi; ++u) {
      const int64_t j2 = j0 + u;
      const float pu = __shfl_sync(0xffffffffu, pj, u), du = __shfl_sync(0xffffffffu, dsj, u);
      const bf16* x = FWD ? v + j2 * p.ldv : KEY ? q + j2 * p.ldq : k + j2 * p.ldk;
#pragma unroll
      for (int e = 0; e < W; ++e) out[e] = fmaf(FWD ? pu : du, to_f(x[lane * W + e]), out[e]);
      if constexpr (KEY && !FWD) {
        const bf16* y = g + j2 * p.lddo;
#pragma unroll
        for (int e = 0; e < W; ++e) out2[e] = fmaf(pu, to_f(y[lane * W + e]), out2[e]);
      }
    }
  }
}

// ------------------------------------------------------------------------------ forward
//
// One persistent CTA per SM.  A work item is a head and a pair of 128-query tiles, one tile per stream;
// the two streams share the K and V tiles (a tile that only one of them meets is released by the other).
// Warps: 0 TMA, 1 and 2 the streams' MMA issuers (1 owns TMEM), 3 idle, 4–7 and 8–11 the streams'
// softmax rows, one query row per thread.  While one stream's rows are at their exponentials the tensor
// core works for the other.
// TMEM per stream: S [0, 128) | P | O.  hd 64 has room for P of its own ([128, 160) … 64 columns), so S of
// the next tile is computed as soon as the rows have read this one; with hd 128 P lies over S.
constexpr int kThreadsFwd = 384;
constexpr uint32_t kFwdRegsCtl = 72, kFwdRegsRows = 216;  // 128·72 + 256·216 = 384·168

template <int HD>
struct FwdCfg {
  static constexpr int QT = HD / 64 * TILE;         // bytes of a 128-row tile
  static constexpr int RING = HD == 64 ? 4 : 2;     // K (and V) tiles in flight
  static constexpr bool OWN_P = HD == 64;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QT;
  static constexpr int V = K + RING * QT;
  static constexpr int BARS = V + RING * QT;
  static constexpr int BYTES = 1024 + BARS + 512;
};

struct FwdItem {
  int h, kh, t0;        // head, key head, first tile of the pair
  int4 r0, r1;          // the tiles' key ranges
  int a, b;             // key tiles that either meets
};

__device__ __forceinline__ int4 range_of(const int4* r, int tile, int tiles) {
  return tile < tiles ? __ldg(r + tile) : make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ FwdItem fwd_item(const Params& p, int i) {
  FwdItem it;
  const int n = i / p.H;
  it.h = i - n * p.H;
  it.kh = it.h / p.group;
  it.t0 = 2 * __ldg(p.plan.pair_order + n);
  it.r0 = range_of(p.plan.qrange, it.t0, p.plan.tiles);
  it.r1 = range_of(p.plan.qrange, it.t0 + 1, p.plan.tiles);
  const bool e0 = it.r0.y <= it.r0.x, e1 = it.r1.y <= it.r1.x;
  it.a = e0 ? it.r1.x : e1 ? it.r0.x : min(it.r0.x, it.r1.x);
  it.b = e0 ? it.r1.y : e1 ? it.r0.y : max(it.r0.y, it.r1.y);
  return it;
}
// Work item of round r for this CTA (rounds alternate direction over the CTAs; the items come longest first).
__device__ __forceinline__ int snake(int r) {
  const int G = int(gridDim.x), c = int(blockIdx.x);
  return r * G + ((r & 1) ? G - 1 - c : c);
}

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreadsFwd, 1)
    attnm_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = FwdCfg<HD>;
  constexpr uint32_t TCOLS = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);
  uint64_t* k_full = bars;                // [RING]
  uint64_t* k_empty = k_full + C::RING;   // one arrival per stream
  uint64_t* v_full = k_empty + C::RING;
  uint64_t* v_empty = v_full + C::RING;
  uint64_t* stream_bars = v_empty + C::RING;  // per stream: q_full, q_empty, s_full, s_free, p_full, pv_done, mma_done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(stream_bars + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(smem_u32(&k_full[i]), 1);
      mbar_init(smem_u32(&k_empty[i]), 2);
      mbar_init(smem_u32(&v_full[i]), 1);
      mbar_init(smem_u32(&v_empty[i]), 2);
    }
    for (int st = 0; st < 2; ++st)
      for (int i = 0; i < 7; ++i) mbar_init(smem_u32(&stream_bars[7 * st + i]), (i == 3 || i == 4) ? 4 : 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_begin();
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.flag, XT_DEVERR_TIMEOUT);
  };
  const bool ok_plan = attn_plan::valid(p.plan);
  if (!ok_plan && blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.flag, XT_DEVERR_PLAN);
  const int items = ok_plan ? (p.plan.tiles + 1) / 2 * p.H : 0;

  const int wg = warp >> 2;
  if (wg == 0) {
    regs_dec<kFwdRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer
      uint32_t nq = 0, n = 0;  // items, K / V tiles so far
      bool ok = true;
#pragma unroll 1
      for (int r = 0; r * int(gridDim.x) < items && ok && !*abort_flag; ++r) {
        const int i = snake(r);
        if (i >= items) continue;
        const FwdItem it = fwd_item(p, i);
#pragma unroll 1
        for (int st = 0; st < 2 && ok; ++st) {
          uint64_t* b = stream_bars + 7 * st;
          if (!mbar_wait(smem_u32(&b[1]), (nq & 1) ^ 1, p.wait_ns)) { ok = false; break; }
          mbar_expect_tx(smem_u32(&b[0]), C::QT);
          Mma<HD>::load(sb + C::Q + st * C::QT, &tmQ, smem_u32(&b[0]), it.h, it.t0 + st);
        }
        if (!ok) break;
        ++nq;
#pragma unroll 1
        for (int j = it.a; j < it.b; ++j, ++n) {
          const uint32_t s = n % C::RING, ph = ((n / C::RING) & 1) ^ 1;
          if (*abort_flag || !mbar_wait(smem_u32(&k_empty[s]), ph, p.wait_ns)) { ok = false; break; }
          mbar_expect_tx(smem_u32(&k_full[s]), C::QT);
          Mma<HD>::load(sb + C::K + s * C::QT, &tmK, smem_u32(&k_full[s]), it.kh, j);
          if (!mbar_wait(smem_u32(&v_empty[s]), ph, p.wait_ns)) {  // K of this tile is in flight: drained below
            ok = false;
            mbar_wait(smem_u32(&k_full[s]), (n / C::RING) & 1);
            break;
          }
          mbar_expect_tx(smem_u32(&v_full[s]), C::QT);
          Mma<HD>::load(sb + C::V + s * C::QT, &tmV, smem_u32(&v_full[s]), it.kh, j);
        }
      }
      if (!ok) give_up();
      // bounded wait for the fills that may still be in flight
      bool drained = true;
      if (nq > 0)
        for (int st = 0; st < 2; ++st) drained &= mbar_wait(smem_u32(&stream_bars[7 * st]), (nq - 1) & 1);
      for (uint32_t m = 0; m < (n < uint32_t(C::RING) ? n : uint32_t(C::RING)); ++m) {
        const uint32_t g = n - 1 - m;
        drained &= mbar_wait(smem_u32(&k_full[g % C::RING]), (g / C::RING) & 1);
        drained &= mbar_wait(smem_u32(&v_full[g % C::RING]), (g / C::RING) & 1);
      }
      if (!drained) give_up();
    } else if ((warp == 1 || warp == 2) && lane == 0) {
      // -------------------------------------------------------------- MMA issuer of stream warp − 1
      const int st = warp - 1;
      uint64_t* b = stream_bars + 7 * st;
      const uint32_t tS = tbase + uint32_t(256 * st), tP = tS + (C::OWN_P ? 128u : 0u), tO = tbase + 256 * st + (C::OWN_P ? 192u : 128u);
      const uint32_t qs = sb + C::Q + st * C::QT;
      uint32_t n0 = 0, nq = 0, g = 0;  // K / V tiles of earlier items, items, score tiles of this stream
      bool ok = true;
      auto pv = [&](uint32_t n, uint32_t gg, bool first) -> bool {  // O += P V of ring tile n, score tile gg
        const uint32_t s = n % C::RING;
        if (!mbar_wait_spin(smem_u32(&b[4]), gg & 1, p.wait_ns) ||
            !mbar_wait_spin(smem_u32(&v_full[s]), (n / C::RING) & 1, p.wait_ns)) return false;
        tc_fence_after();
        Mma<HD>::tn(tO, tP, 32, sb + C::V + s * C::QT, first);
        tc_commit(smem_u32(&v_empty[s]));
        tc_commit(smem_u32(&b[5]));
        return true;
      };
#pragma unroll 1
      for (int r = 0; r * int(gridDim.x) < items && ok && !*abort_flag; ++r) {
        const int i = snake(r);
        if (i >= items) continue;
        const FwdItem it = fwd_item(p, i);
        const int4 rg = st ? it.r1 : it.r0;
        if (!mbar_wait_spin(smem_u32(&b[0]), nq & 1, p.wait_ns)) { ok = false; break; }
        ++nq;
        tc_fence_after();
        int pend = -1;  // ring tile whose P V is still to be issued
        bool first = true;
        bool held = true;  // Q still needed
#pragma unroll 1
        for (int j = it.a; j < it.b && ok; ++j) {
          const uint32_t n = n0 + uint32_t(j - it.a), s = n % C::RING, ph = (n / C::RING) & 1;
          const bool mine = j >= rg.x && j < rg.y;
          if (*abort_flag) { ok = false; break; }
          if (pend >= 0 && (!mine || !C::OWN_P)) {
            if (!pv(uint32_t(pend), g - 1, first)) { ok = false; break; }
            first = false;
            pend = -1;
          }
          if (!mbar_wait_spin(smem_u32(&k_full[s]), ph, p.wait_ns)) { ok = false; break; }
          if (!mine) {  // the other stream's tile
            mbar_arrive(smem_u32(&k_empty[s]));
            if (!mbar_wait_spin(smem_u32(&v_full[s]), ph, p.wait_ns)) { ok = false; break; }
            mbar_arrive(smem_u32(&v_empty[s]));
            continue;
          }
          if (C::OWN_P && !mbar_wait_spin(smem_u32(&b[3]), (g & 1) ^ 1, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          Mma<HD>::nt(tS, qs, sb + C::K + s * C::QT);
          tc_commit(smem_u32(&k_empty[s]));
          tc_commit(smem_u32(&b[2]));
          if (j == rg.y - 1) {
            tc_commit(smem_u32(&b[1]));
            held = false;
          }
          if (pend >= 0) {
            if (!pv(uint32_t(pend), g - 1, first)) { ok = false; break; }
            first = false;
          }
          pend = int(n);
          ++g;
        }
        if (!ok) break;
        if (pend >= 0 && !pv(uint32_t(pend), g - 1, first)) { ok = false; break; }
        if (held) mbar_arrive(smem_u32(&b[1]));
        n0 += uint32_t(it.b - it.a);
      }
      if (!ok) give_up();
      // every MMA issued has completed (also after a give-up) before TMEM is released
      tc_commit(smem_u32(&b[6]));
      if (!mbar_wait(smem_u32(&b[6]), 0)) give_up();
    }
  } else {
    regs_inc<kFwdRegsRows>();
    // ---------------------------------------------------------------- softmax rows, epilogue
    const int st = wg - 1;
    uint64_t* b = stream_bars + 7 * st;
    const int qw = warp & 3;
    const int rr = qw * 32 + lane;
    const uint32_t lane_off = uint32_t(qw * 32) << 16;
    const uint32_t tS = tbase + uint32_t(256 * st) + lane_off, tP = tS + (C::OWN_P ? 128u : 0u),
                   tO = tS + (C::OWN_P ? 192u : 128u);
    uint32_t g = 0;
#pragma unroll 1
    for (int r = 0; r * int(gridDim.x) < items; ++r) {
      const int i = snake(r);
      if (i >= items) continue;
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const FwdItem it = fwd_item(p, i);
      const int tile = it.t0 + st;
      if (tile >= p.plan.tiles) continue;
      const int4 rg = st ? it.r1 : it.r0;
      const int row = tile * BT + rr;
      const int2 iv = __ldg(p.plan.q_iv + row);
      const float slope2 = BIAS ? __ldg(p.slopes + it.h) * kLog2e : 0.f;
      float m = -INFINITY;  // running max, of the raw scores or (CAP, BIAS) of s·log₂e
      float l = 0.f;        // running Σ 2^(s − m)
      const float unit = (CAP || BIAS) ? 1.f : p.sc;
      bool ok = true;
#pragma unroll 1
      for (int j = rg.x; j < rg.y; ++j, ++g) {
        if (!warp_wait(smem_u32(&b[2]), g & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + uint32_t(c * 32), *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
        tmem_ld_wait();
        if (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&b[3]));
        }
        if constexpr (CAP || BIAS)
          to_log2<128, CAP, BIAS>(s, p, slope2, j * BT - row, j < tile ? 1 : j > tile ? -1 : 0);
        if (j < rg.z || j >= rg.w) {
          const int lo = iv.x - j * BT, hi = iv.y - j * BT;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c < lo || c >= hi) s[c] = __float_as_uint(-INFINITY);
        }
        float mx[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) mx[t] = fmaxf(__uint_as_float(s[2 * t]), __uint_as_float(s[2 * t + 1]));
#pragma unroll
        for (int c = 8; c < 128; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        const float m_new = fmaxf(max3(m, mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool need = m_new > m && (m == -INFINITY || (m_new - m) * unit > kRescale);
        // the previous tile's P V is complete before P is rewritten and O rescaled (with P over S the
        // scores' arrival says so: they were computed after it)
        if (C::OWN_P && !warp_wait(smem_u32(&b[5]), (g & 1) ^ 1, p.wait_ns)) { ok = false; break; }
        if (j > rg.x && __any_sync(0xffffffffu, need)) {
          if (C::OWN_P) tc_fence_after();
          const float a = need ? exp2f((m - m_new) * unit) : 1.f;
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {  // few registers: the row's scores stay in theirs
            uint32_t o[16];
            tmem_ld16(tO + uint32_t(c), o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st16(tO + uint32_t(c), o);
          }
        }
        if (need) {
          l = (m == -INFINITY) ? 0.f : l * exp2f((m - m_new) * unit);
          m = m_new;
        }
        const float ms = (m == -INFINITY) ? 0.f : m * unit;
        const uint64_t sc2 = f32x2_pack(unit, unit), ms2 = f32x2_pack(-ms, -ms);
        uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 128; c += 32) {  // 32 columns at a time: 16 registers of P
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            f32x2_unpack(f32x2_fma(pair(s[c + e], s[c + e + 1]), sc2, ms2), x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            ls[(e >> 1) & 3] = f32x2_add(ls[(e >> 1) & 3], f32x2_pack(x0, x1));
            pk[e >> 1] = pack_bf16(x0, x1);
          }
          tmem_st16(tP + uint32_t(c / 2), pk);
        }
        float la, lb;
        f32x2_unpack(f32x2_add(f32x2_add(ls[0], ls[1]), f32x2_add(ls[2], ls[3])), la, lb);
        l += la + lb;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b[4]));
      }
      if (ok && rg.y > rg.x && !warp_wait(smem_u32(&b[5]), (g - 1) & 1, p.wait_ns)) ok = false;
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      // ---- epilogue: O / l
      const bool seen = m > -INFINITY || l != 0.f;  // l: a NaN score leaves m at −∞
      const float inv = seen ? 1.f / l : 0.f;
      tc_fence_after();
      bf16* orow = p.o + int64_t(row) * p.ldo + int64_t(it.h) * HD;
      bf16* lrow = p.o_lo ? p.o_lo + int64_t(row) * p.ldo + int64_t(it.h) * HD : nullptr;
      float bad = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        if (rg.y > rg.x) {
          tmem_ld32(tO + uint32_t(c * 32), o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = seen ? __uint_as_float(o[e]) * inv : 0.f;
          bad = fmaf(x, 0.f, bad);
          o[e] = __float_as_uint(x);
        }
        if (row < p.plan.T) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = __uint_as_float(o[8 * u + 2 * e]), y = __uint_as_float(o[8 * u + 2 * e + 1]);
              hi[e] = pack_bf16(x, y);
              lo[e] = pack_bf16(x - lo_bf16(hi[e]), y - hi_bf16(hi[e]));
            }
            *reinterpret_cast<uint4*>(orow + c * 32 + u * 8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if (lrow) *reinterpret_cast<uint4*>(lrow + c * 32 + u * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      tc_fence_before();
      if (row < p.plan.T)
        p.lse[int64_t(it.h) * p.plan.T + row] = seen ? (m * unit + log2f(l)) * kLn2 : -INFINITY;
      // rows that a masked NaN or infinity reached through the products
      uint32_t redo = __ballot_sync(0xffffffffu, bad != 0.f && l == l && row < p.plan.T);
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        const int rw = __shfl_sync(0xffffffffu, row, src), lo = __shfl_sync(0xffffffffu, iv.x, src),
                  hi = __shfl_sync(0xffffffffu, iv.y, src);
        const float m2 = __shfl_sync(0xffffffffu, m * unit, src), iv2 = __shfl_sync(0xffffffffu, inv, src);
        float acc[HD / 32] = {};
        redo_row<HD, false, true, CAP, BIAS>(p, it.h, it.kh, rw, lo, hi, m2, 0.f, acc, nullptr);
        __syncwarp();
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          const int64_t at = int64_t(rw) * p.ldo + int64_t(it.h) * HD + lane * (HD / 32) + e;
          const float x = acc[e] * iv2;
          const bf16 hi_x = __float2bfloat16_rn(x);
          p.o[at] = hi_x;
          if (p.o_lo) p.o_lo[at] = __float2bfloat16_rn(x - __bfloat162float(hi_x));
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TCOLS);
  }
}

// ------------------------------------------------------------------------------ backward
//
// One kernel for both directions.  KEY: an item is a key tile of a key head, a thread's row a key, the
// columns queries; dK and dV sum over the query tiles that see the tile, for every query head of the group
// in turn.  else: an item is a query tile of a head, a row a query, the columns keys; dQ sums over key tiles.
// Per tile: S = (row tile)(column tile)ᵀ and dP likewise into TMEM; the rows form P = 2^(s − lse) and (KEY)
// write it over S for dV += P dO; then dS = P∘(dP − D)∘(1 − tanh²) over dP for dK (dQ) += dS Q (K).
// Eight row warps, two per TMEM lane quadrant, each half of a tile's 128 columns.  The next S is issued
// before this tile's second products wherever its buffer allows (two S buffers, or KEY at hd 128 one), so
// the tensor core works while the rows are at their exponentials.  The query pass also forms D (its rows'
// dO·O) and leaves it in the workspace for the key pass, which follows it: no kernel of its own for D.
constexpr int kThreadsBwd = 384;  // warps 0 TMA, 1 MMA, 2 and 3 idle, 4–11 rows
constexpr uint32_t kBwdRegsCtl = 72, kBwdRegsRows = 216;  // 128·72 + 256·216 = 384·168

template <int HD, bool KEY>
struct BwdCfg {
  static constexpr int QT = HD / 64 * TILE;
  static constexpr int RING = HD == 64 ? 4 : 2;          // column tiles (pairs) in flight
  static constexpr int NS = (HD == 64 || !KEY) ? 2 : 1;  // S buffers
  static constexpr uint32_t DP = NS * 128, ACC1 = DP + 128, ACC2 = ACC1 + HD;  // TMEM columns
  static constexpr int A = 0;                            // the row tiles: K, V or Q, dO
  static constexpr int R = A + 2 * QT;                   // ring of column tile pairs: Q, dO or K, V
  static constexpr int VEC = R + RING * 2 * QT;          // 2 × (lse·log₂e, D) × 128 floats
  static constexpr int BARS = VEC + 2048;
  static constexpr int BYTES = 1024 + BARS + 256;
  static_assert(ACC2 + (KEY ? HD : 0) <= 512, "TMEM columns");
};

struct BwdItem {
  int h0, kh, tile;   // first query head, key head, row tile
  int4 rg;            // column tiles
  int heads, n;       // query heads, column tiles in all
};
template <bool KEY>
__device__ __forceinline__ BwdItem bwd_item(const Params& p, int i) {
  BwdItem it;
  const int heads = KEY ? p.Hkv : p.H, n = i / heads, h = i - n * heads;
  it.tile = __ldg((KEY ? p.plan.k_order : p.plan.q_order) + n);
  it.rg = __ldg((KEY ? p.plan.krange : p.plan.qrange) + it.tile);
  it.kh = KEY ? h : h / p.group;
  it.h0 = KEY ? h * p.group : h;
  it.heads = KEY ? p.group : 1;
  it.n = max(it.rg.y - it.rg.x, 0) * it.heads;
  return it;
}

template <int HD, bool KEY, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreadsBwd, 1)
    attnm_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ Params p) {
  using C = BwdCfg<HD, KEY>;
  constexpr uint32_t TCOLS = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);
  uint64_t* a_full = bars;
  uint64_t* a_empty = bars + 1;
  uint64_t* r_full = bars + 2;            // [RING]
  uint64_t* r_empty = bars + 6;           // [RING]
  uint64_t* s_full = bars + 10;           // [NS]
  uint64_t* dp_full = bars + 12;
  uint64_t* p_full = bars + 13;
  uint64_t* ds_full = bars + 14;
  uint64_t* acc_full = bars + 15;
  uint64_t* vec_full = bars + 16;         // [2]
  uint64_t* mma_done = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* vec = reinterpret_cast<float*>(smem + C::VEC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 19; ++i) {
      const int n = (i == 13 || i == 14) ? 8 : (i == 16 || i == 17) ? 256 : 1;
      mbar_init(smem_u32(&bars[i]), n);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmDO);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_begin();
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.flag, XT_DEVERR_TIMEOUT);
  };
  const bool ok_plan = attn_plan::valid(p.plan);
  if (!ok_plan && blockIdx.x == 0 && threadIdx.x == 0) flag_error(p.flag, XT_DEVERR_PLAN);
  const int items = ok_plan ? p.plan.tiles * (KEY ? p.Hkv : p.H) : 0;
  const CUtensorMap *tmA1 = KEY ? &tmK : &tmQ, *tmA2 = KEY ? &tmV : &tmDO;
  const CUtensorMap *tmR1 = KEY ? &tmQ : &tmK, *tmR2 = KEY ? &tmDO : &tmV;

  if (warp < 4) {
    regs_dec<kBwdRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer
      uint32_t na = 0, n = 0;
      bool ok = true;
#pragma unroll 1
      for (int r = 0; r * int(gridDim.x) < items && ok && !*abort_flag; ++r) {
        const int i = snake(r);
        if (i >= items) continue;
        const BwdItem it = bwd_item<KEY>(p, i);
        if (it.n == 0) continue;
        if (!mbar_wait(smem_u32(a_empty), (na & 1) ^ 1, p.wait_ns)) { ok = false; break; }
        mbar_expect_tx(smem_u32(a_full), 2 * C::QT);
        Mma<HD>::load(sb + C::A, tmA1, smem_u32(a_full), KEY ? it.kh : it.h0, it.tile);
        Mma<HD>::load(sb + C::A + C::QT, tmA2, smem_u32(a_full), KEY ? it.kh : it.h0, it.tile);
        ++na;
        int h = it.h0, t = it.rg.x;
#pragma unroll 1
        for (int j = 0; j < it.n; ++j, ++n) {
          const uint32_t s = n % C::RING;
          if (*abort_flag || !mbar_wait(smem_u32(&r_empty[s]), ((n / C::RING) & 1) ^ 1, p.wait_ns)) { ok = false; break; }
          const uint32_t fb = smem_u32(&r_full[s]), dst = sb + C::R + s * 2 * C::QT;
          mbar_expect_tx(fb, 2 * C::QT);
          Mma<HD>::load(dst, tmR1, fb, KEY ? h : it.kh, t);
          Mma<HD>::load(dst + C::QT, tmR2, fb, KEY ? h : it.kh, t);
          if (++t == it.rg.y) { t = it.rg.x; ++h; }
        }
      }
      if (!ok) give_up();
      bool drained = true;
      if (na > 0) drained &= mbar_wait(smem_u32(a_full), (na - 1) & 1);
      for (uint32_t m = 0; m < (n < uint32_t(C::RING) ? n : uint32_t(C::RING)); ++m) {
        const uint32_t g = n - 1 - m;
        drained &= mbar_wait(smem_u32(&r_full[g % C::RING]), (g / C::RING) & 1);
      }
      if (!drained) give_up();
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------------- MMA issuer
      uint32_t na = 0, g = 0;
      bool ok = true;
      const uint32_t a1 = sb + C::A, a2 = a1 + C::QT;
      auto slot = [&](uint32_t n) { return sb + C::R + (n % C::RING) * 2 * C::QT; };
      auto issue_s = [&](uint32_t n) -> bool {
        if (!mbar_wait_spin(smem_u32(&r_full[n % C::RING]), (n / C::RING) & 1, p.wait_ns)) return false;
        tc_fence_after();
        Mma<HD>::nt(tbase + (n % C::NS) * 128, a1, slot(n));
        tc_commit(smem_u32(&s_full[n % C::NS]));
        return true;
      };
      auto issue_dp = [&](uint32_t n) {
        Mma<HD>::nt(tbase + C::DP, a2, slot(n) + C::QT);
        tc_commit(smem_u32(dp_full));
      };
#pragma unroll 1
      for (int r = 0; r * int(gridDim.x) < items && ok && !*abort_flag; ++r) {
        const int i = snake(r);
        if (i >= items) continue;
        const BwdItem it = bwd_item<KEY>(p, i);
        if (it.n == 0) continue;
        if (!mbar_wait_spin(smem_u32(a_full), na & 1, p.wait_ns)) { ok = false; break; }
        ++na;
        tc_fence_after();
        if (!issue_s(g)) { ok = false; break; }
        issue_dp(g);
#pragma unroll 1
        for (int j = 0; j < it.n; ++j, ++g) {
          const bool next = j + 1 < it.n;
          if (*abort_flag) { ok = false; break; }
          if (C::NS == 2 && next && !issue_s(g + 1)) { ok = false; break; }
          if (KEY) {
            if (!mbar_wait_spin(smem_u32(p_full), g & 1, p.wait_ns)) { ok = false; break; }
            tc_fence_after();
            Mma<HD>::tn(tbase + C::ACC2, tbase + (g % C::NS) * 128, 64, slot(g) + C::QT, j == 0);  // dV += Pᵀ dO
          }
          if (C::NS == 1 && next && !issue_s(g + 1)) { ok = false; break; }
          if (!mbar_wait_spin(smem_u32(ds_full), g & 1, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          Mma<HD>::tn(tbase + C::ACC1, tbase + C::DP, 64, slot(g), j == 0);  // dK += dSᵀ Q, dQ += dS K
          tc_commit(smem_u32(&r_empty[g % C::RING]));
          if (next) issue_dp(g + 1);
        }
        if (!ok) break;
        tc_commit(smem_u32(acc_full));
        tc_commit(smem_u32(a_empty));
      }
      if (!ok) give_up();
      tc_commit(smem_u32(mma_done));
      if (!mbar_wait(smem_u32(mma_done), 0)) give_up();
    }
  } else {
    // ---------------------------------------------------------------- rows
    regs_inc<kBwdRegsRows>();
    const int qw = warp & 3, half = (warp - 4) >> 2, col0 = 64 * half;
    const int rr = qw * 32 + lane;
    const uint32_t lane_off = uint32_t(qw * 32) << 16;
    const uint32_t tDP = tbase + C::DP + lane_off + uint32_t(col0);
    uint32_t g = 0, na = 0, nv = 0;
#pragma unroll 1
    for (int r = 0; r * int(gridDim.x) < items; ++r) {
      const int i = snake(r);
      if (i >= items) continue;
      if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
      const BwdItem it = bwd_item<KEY>(p, i);
      const int row = it.tile * BT + rr;
      const int64_t T = p.plan.T;
      const bool real = row < T;
      const int2 iv = __ldg((KEY ? p.plan.k_iv : p.plan.q_iv) + row);
      float lse2 = INFINITY, Dr = 0.f;  // of the row (not KEY)
      bool ok = true;
      if constexpr (!KEY) {
        // D of the row: each half warp group adds its half of the columns, the halves meet in shared memory
        float acc = 0.f;
        if (real && iv.y > iv.x) {
          const int64_t c0 = int64_t(it.h0) * HD + half * (HD / 2);
          const bf16* o = p.o + int64_t(row) * p.ldo + c0;
          const bf16* ol = p.o_lo ? p.o_lo + int64_t(row) * p.ldo + c0 : nullptr;
          const bf16* go = p.d_o + int64_t(row) * p.lddo + c0;
#pragma unroll
          for (int c = 0; c < HD / 2; c += 8) {
            float x[8], y[8], z[8];
            Vec<bf16>::load(o + c, x);
            Vec<bf16>::load(go + c, y);
            if (ol) {
              Vec<bf16>::load(ol + c, z);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] += z[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc = fmaf(x[e], y[e], acc);
          }
          lse2 = p.lse[int64_t(it.h0) * T + row] * kLog2e;
          if (lse2 == -INFINITY) lse2 = INFINITY;
        }
        float* dv = vec + (nv & 1) * 256;
        dv[half * 128 + rr] = acc;
        mbar_arrive(smem_u32(&vec_full[nv & 1]));
        if (!warp_wait(smem_u32(&vec_full[nv & 1]), (nv >> 1) & 1, p.wait_ns)) {
          if (lane == 0) give_up();
          break;
        }
        ++nv;
        Dr = dv[rr] + dv[128 + rr];
        if (half == 0 && real) p.D[int64_t(it.h0) * T + row] = Dr;
      }
      int h = it.h0, t = it.rg.x;
      // KEY: this thread's entry of a column tile's −lse·log₂e (half 0) or −D (half 1), read one tile ahead
      auto vec_entry = [&](int hh, int tt) -> float {
        const int q = tt * BT + rr;
        if (half == 0) {
          const float x = q < T ? p.lse[int64_t(hh) * T + q] * -kLog2e : -INFINITY;
          return x == INFINITY ? -INFINITY : x;
        }
        return q < T ? -p.D[int64_t(hh) * T + q] : 0.f;
      };
      float vnext = 0.f;
      if (KEY && it.n > 0) vnext = vec_entry(h, t);
#pragma unroll 1
      for (int j = 0; j < it.n; ++j, ++g) {
        int h2 = h, t2 = t + 1;
        if (t2 == it.rg.y) { t2 = it.rg.x; ++h2; }
        const float* lv = vec + (g & 1) * 256;
        if constexpr (KEY) {
          // a thread refills a slot only after all have arrived for the tile in between, having read it
          vec[(g & 1) * 256 + half * 128 + rr] = vnext;
          if (j + 1 < it.n) vnext = vec_entry(h2, t2);
          mbar_arrive(smem_u32(&vec_full[g & 1]));
          if (!warp_wait(smem_u32(&vec_full[g & 1]), (g >> 1) & 1, p.wait_ns)) { ok = false; break; }
        }
        const float slope2 = BIAS ? __ldg(p.slopes + h) * kLog2e : 0.f;
        const uint32_t tS = tbase + (g % C::NS) * 128 + lane_off + uint32_t(col0);
        if (!warp_wait(smem_u32(&s_full[g % C::NS]), (g / C::NS) & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[64];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
        tmem_ld_wait();
        const float unit = (CAP || BIAS) ? 1.f : p.sc;
        const int side = t < it.tile ? 1 : t > it.tile ? -1 : 0;
        float slack[CAP ? 64 : 1];  // 1 − tanh²
        if constexpr (CAP) {
#pragma unroll
          for (int c = 0; c < 64; ++c) {  // as to_log2, keeping u = 1/(1 + e^{2a/cap}): 1 − tanh² = 4u(1 − u)
            const float u = rcp(1.f + ex2(__uint_as_float(s[c]) * p.capk));
            s[c] = __float_as_uint(fmaf(-2.f * p.cap2, u, p.cap2));
            slack[c] = 4.f * u * (1.f - u);
          }
          if constexpr (BIAS) add_bias(s, slope2, t * BT + col0 - row, side);
        } else if constexpr (BIAS) {
          to_log2<64, CAP, BIAS>(s, p, slope2, t * BT + col0 - row, side);
        }
        const bool edge = t < it.rg.z || t >= it.rg.w;
        const int lo = iv.x - t * BT - col0, hi = iv.y - t * BT - col0;
        if (edge) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < lo || c >= hi) {
              s[c] = __float_as_uint(-INFINITY);
              if constexpr (CAP) slack[c] = 0.f;
            }
        }
        const uint64_t unit2 = f32x2_pack(unit, unit), nl2 = f32x2_pack(-lse2, -lse2);
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = c; e < c + 32; e += 4) {
            float4 nl;
            if constexpr (KEY) nl = *reinterpret_cast<const float4*>(lv + col0 + e);
            float x[4];
            f32x2_unpack(f32x2_fma(pair(s[e], s[e + 1]), unit2, KEY ? f32x2_pack(nl.x, nl.y) : nl2), x[0], x[1]);
            f32x2_unpack(f32x2_fma(pair(s[e + 2], s[e + 3]), unit2, KEY ? f32x2_pack(nl.z, nl.w) : nl2), x[2], x[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = ex2(x[k]);
            if constexpr (KEY) {
              pk[(e - c) >> 1] = pack_bf16(x[0], x[1]);
              pk[((e - c) >> 1) + 1] = pack_bf16(x[2], x[3]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (CAP) x[k] *= slack[e + k];
              s[e + k] = __float_as_uint(x[k]);
            }
          }
          if constexpr (KEY) tmem_st16(tS + uint32_t(c / 2), pk);
        }
        if constexpr (KEY) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(p_full));
        }
        if (!warp_wait(smem_u32(dp_full), g & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t d[64];
        tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(d));
        tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(d + 32));
        tmem_ld_wait();
        const uint64_t nd2 = f32x2_pack(-Dr, -Dr);
        auto form_ds = [&](auto masked) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int e = c; e < c + 32; e += 4) {
              float4 nd;
              if constexpr (KEY) nd = *reinterpret_cast<const float4*>(lv + 128 + col0 + e);
              float x[4];
              f32x2_unpack(f32x2_mul(f32x2_add(pair(d[e], d[e + 1]), KEY ? f32x2_pack(nd.x, nd.y) : nd2),
                                     pair(s[e], s[e + 1])), x[0], x[1]);
              f32x2_unpack(f32x2_mul(f32x2_add(pair(d[e + 2], d[e + 3]), KEY ? f32x2_pack(nd.z, nd.w) : nd2),
                                     pair(s[e + 2], s[e + 3])), x[2], x[3]);
              if constexpr (decltype(masked)::value) {  // a masked column's dP or D may be NaN
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (e + k < lo || e + k >= hi) x[k] = 0.f;
              }
              pk[(e - c) >> 1] = pack_bf16(x[0], x[1]);
              pk[((e - c) >> 1) + 1] = pack_bf16(x[2], x[3]);
            }
            tmem_st16(tDP + uint32_t(c / 2), pk);
          }
        };
        if (edge) form_ds(std::true_type{});
        else form_ds(std::false_type{});
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(ds_full));
        h = h2;
        t = t2;
      }
      if (ok && it.n > 0) {
        if (!warp_wait(smem_u32(acc_full), na & 1, p.wait_ns)) ok = false;
        ++na;
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      // ---- epilogue: this half's HD/2 columns of the accumulators
      tc_fence_after();
      float bad = 0.f;
#pragma unroll
      for (int w = 0; w < (KEY ? 2 : 1); ++w) {
        bf16* out = w ? p.dv + int64_t(row) * p.lddv : KEY ? p.dk + int64_t(row) * p.lddk : p.dq + int64_t(row) * p.lddq;
        out += int64_t(KEY ? it.kh : it.h0) * HD + half * (HD / 2);
        const float mul = w ? 1.f : p.scale;
        const uint32_t acc = tbase + (w ? C::ACC2 : C::ACC1) + lane_off + uint32_t(half * (HD / 2));
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          uint32_t o[32];
          if (it.n > 0) {
            tmem_ld32(acc + uint32_t(c * 32), o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = it.n > 0 ? __uint_as_float(o[e]) * mul : 0.f;
            bad = fmaf(x, 0.f, bad);
            o[e] = __float_as_uint(x);
          }
          if (real) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(out + c * 32 + u * 8) =
                  make_uint4(pack_bf16(__uint_as_float(o[8 * u]), __uint_as_float(o[8 * u + 1])),
                             pack_bf16(__uint_as_float(o[8 * u + 2]), __uint_as_float(o[8 * u + 3])),
                             pack_bf16(__uint_as_float(o[8 * u + 4]), __uint_as_float(o[8 * u + 5])),
                             pack_bf16(__uint_as_float(o[8 * u + 6]), __uint_as_float(o[8 * u + 7])));
          }
        }
      }
      tc_fence_before();
      // rows that a masked NaN or infinity reached through the products: this half's columns once more
      uint32_t redo = __ballot_sync(0xffffffffu, bad != 0.f && real);
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        const int rw = __shfl_sync(0xffffffffu, row, src), lo = __shfl_sync(0xffffffffu, iv.x, src),
                  hi = __shfl_sync(0xffffffffu, iv.y, src);
        const float m2 = __shfl_sync(0xffffffffu, lse2, src), dr = __shfl_sync(0xffffffffu, Dr, src);
        float a1[HD / 32] = {}, a2[HD / 32] = {};
        for (int hh = it.h0; hh < it.h0 + it.heads; ++hh)
          redo_row<HD, KEY, false, CAP, BIAS>(p, hh, it.kh, rw, lo, hi, m2, dr, a1, a2);
        __syncwarp();
        if ((lane >> 4) != half) continue;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          const int64_t c = int64_t(KEY ? it.kh : it.h0) * HD + lane * (HD / 32) + e;
          (KEY ? p.dk + int64_t(rw) * p.lddk : p.dq + int64_t(rw) * p.lddq)[c] = __float2bfloat16_rn(a1[e] * p.scale);
          if constexpr (KEY) p.dv[int64_t(rw) * p.lddv + c] = __float2bfloat16_rn(a2[e]);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TCOLS);
  }
}

// ------------------------------------------------------------------------------ launches

// Raises the kernel's shared-memory limit on the current device and, for a kernel that splits its registers,
// checks that it was built with the count the split adds up to (any other could never be met).
int prepare_kernel(const void* kernel, int smem, int regs);

template <int HD>
int launch_fwd(bool cap, bool bias, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const Params& p, cudaStream_t s);
template <int HD, bool KEY>
int launch_bwd(bool cap, bool bias, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
               const CUtensorMap& tdo, const Params& p, cudaStream_t s);

#define XT_ATTNM_FWD(HD)                                                                                         \
  template <bool CAP, bool BIAS>                                                                                 \
  static int fwd_one(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Params& p,       \
                     cudaStream_t s) {                                                                           \
    auto k = attnm_fwd_kernel<HD, CAP, BIAS>;                                                                    \
    XT_TRY(prepare_kernel(reinterpret_cast<const void*>(k), FwdCfg<HD>::BYTES, 168));                            \
    const int64_t items = int64_t((p.plan.tiles + 1) / 2) * p.H;                                                 \
    launch(k, unsigned(items < num_sms() ? items : num_sms()), kThreadsFwd, FwdCfg<HD>::BYTES, s, tq, tk, tv, p); \
    return check_launch("xt_attention_masked_fwd");                                                              \
  }                                                                                                              \
  template <>                                                                                                    \
  int launch_fwd<HD>(bool cap, bool bias, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,   \
                     const Params& p, cudaStream_t s) {                                                          \
    if (cap) return bias ? fwd_one<true, true>(tq, tk, tv, p, s) : fwd_one<true, false>(tq, tk, tv, p, s);       \
    return bias ? fwd_one<false, true>(tq, tk, tv, p, s) : fwd_one<false, false>(tq, tk, tv, p, s);              \
  }

#define XT_ATTNM_BWD(HD, KEY)                                                                                    \
  template <bool CAP, bool BIAS>                                                                                 \
  static int bwd_one(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo, \
                     const Params& p, cudaStream_t s) {                                                          \
    auto k = attnm_bwd_kernel<HD, KEY, CAP, BIAS>;                                                               \
    XT_TRY(prepare_kernel(reinterpret_cast<const void*>(k), BwdCfg<HD, KEY>::BYTES, 168));                         \
    const int64_t items = int64_t(p.plan.tiles) * (KEY ? p.Hkv : p.H);                                           \
    launch(k, unsigned(items < num_sms() ? items : num_sms()), kThreadsBwd, BwdCfg<HD, KEY>::BYTES, s, tq, tk,   \
           tv, tdo, p);                                                                                          \
    return check_launch("xt_attention_masked_bwd");                                                              \
  }                                                                                                              \
  template <>                                                                                                    \
  int launch_bwd<HD, KEY>(bool cap, bool bias, const CUtensorMap& tq, const CUtensorMap& tk,                     \
                          const CUtensorMap& tv, const CUtensorMap& tdo, const Params& p, cudaStream_t s) {      \
    if (cap)                                                                                                     \
      return bias ? bwd_one<true, true>(tq, tk, tv, tdo, p, s) : bwd_one<true, false>(tq, tk, tv, tdo, p, s);    \
    return bias ? bwd_one<false, true>(tq, tk, tv, tdo, p, s) : bwd_one<false, false>(tq, tk, tv, tdo, p, s);    \
  }

}  // namespace attnm
}  // namespace xt
