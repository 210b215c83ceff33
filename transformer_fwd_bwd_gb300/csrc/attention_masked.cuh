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
// Rows whose mask leaves nothing get O = 0, lse = −∞ and zero gradients.  A masked element's score is −∞ by
// selection, so whatever it was (NaN, ∞) stays out of the row; but the products add 0·V for masked
// keys of a tile, which a NaN or ∞ in V turns into NaN, and in the key pass −∞ less the lse of a masked query is NaN where
// that lse is (its query sees a key that is not finite, or a score of its own overflows).  A row whose result is not finite,
// and which has such a column among its masked ones, is therefore done over from its visible columns alone (repair): the
// check costs a fused multiply-add per output element.
//
// Work items (a head and a tile or pair of tiles, the longest first) are the blocks of the grid, one per SM
// at a time; a running block takes over the next item instead of ending (clusterlaunchcontrol: the hardware
// cancels the launch of a waiting block and hands out its index), which keeps its tensor memory, barriers and
// loads in flight across items and balances them by their real times.  The producer warp takes the next item
// when its last load of this one is issued and leaves its description in shared memory for the other warps.
#pragma once

#include <cuda_fp16.h>

#include <atomic>
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
  int split, share;       // key pass: items per key head and tile, query heads of each (but the last)
  float sc;               // scale·log₂e
  float scale;
  float capy, capk, cap2; // scale/cap, 2·log₂e·scale/cap, cap·log₂e (CAP)
  uint64_t tanh_c[7];     // coefficients of tanh(y)/y in y², twice each
  const float* slopes;    // [H] (BIAS)
  const bf16 *q, *k, *v;  // rows of ldq, ldk, ldv elements
  int64_t ldq, ldk, ldv;
  bf16* o;
  const bf16* d_o;
  int64_t ldo, lddo;
  float *lse;             // [H][T]
  float *nl, *nd;         // workspace, [H][tiles·128]: −lse·log₂e (−∞ where nothing is seen) and −D
  bf16 *dq, *dk, *dv;
  int64_t lddq, lddk, lddv;
  float *part_k, *part_v; // split > 1: float32 sums [split][T][Hkv·hd] of dK (before scale) and dV
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
// NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
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

// D[tmem] (+)= A[tmem]·B: A is 128 rows × 16 bf16, two per 32-bit column, row = lane.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accum)
      : "memory");
}

__device__ __forceinline__ bool spin(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return mbar_wait_spin(bar, parity, limit_ns);
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, spin(bar, parity, limit_ns));
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
  // D [128 × N] = A Bᵀ over the head dimension (both K-major), N rows of B from b on
  template <int N = BT>
  static __device__ __forceinline__ void nt(uint32_t d, uint32_t a, uint32_t b) {
    constexpr uint32_t kIdesc = instr_desc_bf16(128, N, false, false);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint32_t off = uint32_t((kk >> 2) * TILE + (kk & 3) * 32);
      tc_mma<kBf16>(d, smem_desc(a + off, 16, 1024), smem_desc(b + off, 16, 1024), kIdesc, kk > 0 ? 1u : 0u);
    }
  }
  // D [128 × HD] (+)= A B over N tokens: A bf16 in tensor memory, GROUP tokens (two to a column) every `step` columns,
  // B's N rows from b on, MN-major
  template <int N = BT, int GROUP = 64>
  static __device__ __forceinline__ void tn(uint32_t d, uint32_t a, uint32_t step, uint32_t b, bool first) {
    constexpr uint32_t kIdesc = instr_desc_bf16(128, HD, false, true);
#pragma unroll
    for (int kk = 0; kk < N / 16; ++kk)
      tc_mma_ts(d, a + uint32_t(kk / (GROUP / 16)) * step + uint32_t(kk % (GROUP / 16)) * 8,
                smem_desc(b + kk * 2048, TILE, 1024), kIdesc,
                (!first || kk > 0) ? 1u : 0u);
  }
  static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int head, int tile) {
#pragma unroll
    for (int c = 0; c < HD / 64; ++c) tma_load_4d(dst + c * TILE, tm, bar, c * 64, head, tile * BT, 0);
  }
};

// Bits of the columns base .. base + 31 that lie in [lo, hi).
__device__ __forceinline__ uint32_t visible_bits(int lo, int hi, int base) {
  const uint32_t below_hi = uint32_t(~(~0ull << min(max(hi - base, 0), 32)));
  const uint32_t below_lo = uint32_t(~(~0ull << min(max(lo - base, 0), 32)));
  return below_hi & ~below_lo;
}

// r[c] = unit·r[c] − slope₂·|d0 + c|.  d0: column 0 minus the row, in tokens; side: +1 / −1 where every column of the
// tile lies before / behind the row (the distance is then linear in c), 0 else.
template <int N>
__device__ __forceinline__ void add_bias(uint32_t (&r)[N], float unit, float slope2, int d0, int side) {
  if (side != 0) {
    const float st = side > 0 ? slope2 : -slope2, b0 = st * float(d0);
    const uint64_t unit2 = f32x2_pack(unit, unit), step2 = f32x2_pack(2.f * st, 2.f * st);
#pragma unroll
    for (int c = 0; c < N; c += 16) {  // two columns at a time; afresh every 16, so that the steps' roundings stay few
      uint64_t b = f32x2_pack(fmaf(float(c), st, b0), fmaf(float(c + 1), st, b0));
#pragma unroll
      for (int e = c; e < c + 16; e += 2) {
        float x, y;
        f32x2_unpack(f32x2_fma(pair(r[e], r[e + 1]), unit2, b), x, y);
        r[e] = __float_as_uint(x);
        r[e + 1] = __float_as_uint(y);
        b = f32x2_add(b, step2);
      }
    }
  } else {
    const float d = float(d0);
#pragma unroll
    for (int c = 0; c < N; ++c)
      r[c] = __float_as_uint(fmaf(-slope2, fabsf(d + float(c)), unit * __uint_as_float(r[c])));
  }
}

// r[c] = tanh(scale·r[c]/cap) = 1 − 2/(1 + e^{2y}), one exponential and one reciprocal.  Where no element of the
// warp's rows is beyond the cap the special-function unit and the multipliers share the work: of four columns two go
// through y·p(y²), p of degree 6 fitted to tanh(y)/y over |y| ≤ 1 (least squares reweighted to equal extremes,
// Lawson's method; tanh(y) is off by 2.6e-8 at most, 3.0e-7 of itself near 0), and two through exponentials and the
// reciprocal of the product of their denominators, 1/a = b·1/(ab) (at most 8.4² there).  A NaN, which may stand in a masked
// column, must not reach the column it would share a reciprocal with: it counts as beyond the cap.  The choice is one for
// the warp's 32 rows and all columns, hidden ones too, so the last bits of a capped score (2⁻²³ of the cap) depend on what
// lies beside it, and the two directions may differ by as much.
// 8192 causal tokens, 12 heads of 64, forward: 233 us (128 without a cap); the special-function unit alone takes 3 %
// more than this mixture, the polynomial alone 4 %.
//
// `slack` (the backward's): 1 − tanh², times kSlack, as f16.  Beyond the cap 1 − t·t would be the rounding of t, so there it is
// 4u(1 − u) of u = 1/(1 + e^{2y}), and 1 − u is e^{2y}·u where that is less than a half.  The power of two, which the
// gradients' factors take back, keeps f16's normal range down to 1.9e-9 (|a/cap| of 10.7; 2⁻¹¹ of the value at most, half a
// step, beside dS's own bf16 rounding of 2⁻⁸), for half the registers of float32; under that it is off by 9e-13.
// (dS itself, of up to 1e34, stays in bf16's range.)
constexpr float kSlack = 32768.f;
template <int N, bool SLACK>
__device__ __forceinline__ void tanh_cap(uint32_t (&r)[N], const Params& p, __half2 (&slack)[SLACK ? N / 2 : 1]) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 2)
    top[(c >> 1) & 3] = max3_nan(top[(c >> 1) & 3], fabsf(__uint_as_float(r[c])), fabsf(__uint_as_float(r[c + 1])));
  const float most = max3_nan(max3_nan(top[0], top[1], top[2]), top[3], 0.f) * p.capy;
  if (__any_sync(0xffffffffu, !(most <= 1.f))) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float f[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float e = ex2(__uint_as_float(r[c + k]) * p.capk), u = rcp(1.f + e);
        r[c + k] = __float_as_uint(fmaf(-2.f, u, 1.f));
        if constexpr (SLACK) f[k] = 4.f * kSlack * u * (e < 1.f ? e * u : 1.f - u);
      }
      if constexpr (SLACK) slack[c / 2] = __floats2half2_rn(f[0], f[1]);
    }
  } else {
    const uint64_t y2 = f32x2_pack(p.capy, p.capy), k2 = f32x2_pack(p.capk, p.capk), one2 = f32x2_pack(1.f, 1.f);
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      float u, w;
      f32x2_unpack(f32x2_mul(pair(r[c + 2], r[c + 3]), k2), u, w);
      u = ex2(u);
      w = ex2(w);
      const uint64_t y = f32x2_mul(pair(r[c], r[c + 1]), y2), z = f32x2_mul(y, y);
      uint64_t q = p.tanh_c[6];
#pragma unroll
      for (int k = 5; k >= 0; --k) q = f32x2_fma(q, z, p.tanh_c[k]);
      f32x2_unpack(f32x2_add(f32x2_pack(u, w), one2), u, w);
      const float i = -2.f * rcp(u * w);
      r[c + 2] = __float_as_uint(fmaf(i, w, 1.f));
      r[c + 3] = __float_as_uint(fmaf(i, u, 1.f));
      f32x2_unpack(f32x2_mul(y, q), u, w);
      r[c] = __float_as_uint(u);
      r[c + 1] = __float_as_uint(w);
      if constexpr (SLACK) {
        const uint64_t all2 = f32x2_pack(kSlack, kSlack), neg2 = f32x2_pack(-kSlack, -kSlack);
#pragma unroll
        for (int k = c; k < c + 4; k += 2) {
          const uint64_t t = pair(r[k], r[k + 1]);
          f32x2_unpack(f32x2_fma(f32x2_mul(t, neg2), t, all2), u, w);
          slack[k / 2] = __floats2half2_rn(u, w);
        }
      }
    }
  }
}

// What a row warp hands to the TMA: 64 bytes of each of its 32 rows at a time, through two buffers of 2 KB with the
// 64-byte swizzle.  The copies run while the warp goes on (a lane that stores its own row touches 32 rows at a time:
// the epilogue of 128 keys and 64 columns took 3800 cycles so, 2650 with four lanes to a row, 1980 like this); rows
// behind the last token are clipped.
constexpr int STAGE = 8 * 2 * 2048;  // of the eight row warps
// w: 64 bytes of this lane's row; to columns c0 on of a head's, rows row0 on, through buffer `buf`.  ALONE: an item
// has one such piece, and all go through the same buffer.  `stage`: the eight warps' buffers.
template <bool ALONE>
__device__ __forceinline__ void put_rows(uint8_t* stage, int buf, const CUtensorMap* tm, const uint32_t (&w)[16], int c0,
                                         int head, int row0, int plane, int64_t T) {
  const int lane = threadIdx.x & 31;
  uint4* to = reinterpret_cast<uint4*>(stage + ((threadIdx.x >> 5) - 4) * 4096 + buf * 2048);
  if (lane == 0) {  // the last copy from this buffer has left it
    if (ALONE) bulk_wait_read_0();
    else bulk_wait_read_1();
  }
  __syncwarp();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    to[lane * 4 + (u ^ (lane >> 1 & 3))] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (row0 < T) tma_store_4d(tm, smem_u32(to), c0, head, row0, plane);
    bulk_commit();
  }
}
// Every copy of the warp has arrived: before a row is written again, and before the block ends.
__device__ __forceinline__ void rows_stored() {
  if ((threadIdx.x & 31) == 0) bulk_wait_all();
  __syncwarp();
}

// Products of 16 rows of a and b (of lda, ldb elements, from `row` on; row T − 1 in the place of later ones), HD / 8
// lanes to a row: the sums go to out[0 .. 15].  A thread that walks its own row takes 2700 cycles for 64 columns and 9500
// for 128, these 1850 and 3300.
template <int HD>
__device__ __forceinline__ void dots16(const bf16* a, int64_t lda, const bf16* b, int64_t ldb, int64_t row, int64_t T,
                                       float* out) {
  constexpr int LPR = HD / 8, RPL = 32 / LPR, N = 16 / RPL;
  const int lane = threadIdx.x & 31, c = lane % LPR * 8;
  uint4 u[N], w[N];  // all loads in flight together: rows behind the last are clamped, not branched around
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = min(row + i * RPL + lane / LPR, T - 1);
    u[i] = *reinterpret_cast<const uint4*>(a + r * lda + c);
    w[i] = *reinterpret_cast<const uint4*>(b + r * ldb + c);
  }
  float x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t y[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, z[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    x[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[i] = fmaf(__uint_as_float(y[e] << 16), __uint_as_float(z[e] << 16), x[i]);
      x[i] = fmaf(__uint_as_float(y[e] & 0xFFFF0000u), __uint_as_float(z[e] & 0xFFFF0000u), x[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if (lane % LPR == 0) out[i * RPL + lane / LPR] = x[i];
  }
}

// What the scores are multiplied by on their way into the exponential (base 2), after the two steps above.
template <bool CAP, bool BIAS>
__device__ __forceinline__ float score_unit(const Params& p) {
  return BIAS ? 1.f : CAP ? p.cap2 : p.sc;
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
    slack = 4.f * u * (e < 1.f ? e * u : 1.f - u);
  }
  if constexpr (BIAS) s = fmaf(-slope2, fabsf(float(dist)), s);
  return s;
}

// One output row from its visible columns alone, by a whole warp: 32 columns at a time, a lane scores
// one, then every lane adds the columns to its HD/32 elements.
//   FWD:  out = Σ_j p_j v_j,               row = query, m2: the running max
//   else: out = Σ dS_ij·(other row), out2 = Σ P_ij·dO_i (KEY), of the row `row` of head h
// False as soon as a sum is not finite: the row sees such a value itself, and its result stands.
template <int HD, bool KEY, bool FWD, bool CAP, bool BIAS>
__device__ __forceinline__ bool redo_row(const Params& p, int h, int kh, int row, int lo, int hi, float m2, float D,
                                         float* out, float* out2) {
  constexpr int W = HD / 32;
  const int lane = threadIdx.x & 31;
  const float slope2 = BIAS ? p.slopes[h] * kLog2e : 0.f;
  const bf16* q = p.q + int64_t(h) * HD;
  const bf16* k = p.k + int64_t(kh) * HD;
  const bf16* v = p.v + int64_t(kh) * HD;
  const bf16* g = FWD ? nullptr : p.d_o + int64_t(h) * HD;
#pragma unroll 1
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
        mm = -p.nl[int64_t(h) * p.plan.tiles * BT + i];
        dd = -p.nd[int64_t(h) * p.plan.tiles * BT + i];
      }
      pj = ex2(s - mm);
      if constexpr (!FWD) dsj = pj * slack * (dot_rows<HD>(g + i * p.lddo, v + c * p.ldv) - dd);
    }
    float bad = 0.f;
#pragma unroll 1
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
#pragma unroll
    for (int e = 0; e < W; ++e) {
      bad = fmaf(out[e], 0.f, bad);
      if constexpr (KEY && !FWD) bad = fmaf(out2[e], 0.f, bad);
    }
    if (__any_sync(0xffffffffu, bad != 0.f)) return false;
  }
  return true;
}

template <int HD>
__device__ __forceinline__ bool row_finite(const bf16* x) {
  float bad = 0.f;
  for (int c = 0; c < HD; c += 8) {
    float v[8];
    Vec<bf16>::load(x + c, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) bad = fmaf(v[e], 0.f, bad);
  }
  return bad == 0.f;
}

// Rows of this warp (`rows`: lanes whose result is not finite) that a masked column's NaN or ∞ reached through
// the second products or (KEY) its query's lse, over the columns [c0, c1) of the tiles the item met.  (Selecting the key
// pass's P after its exponential instead costs every call 3 % at hd 64: 8192 unmasked tokens 901 -> 934 us.)  The first and
// the last column that hold one are found once; a row is done over if it masks one of them.  A lane writes the HD/32 elements
// it summed if they are of the warp's part (part_n parts of HD/part_n columns).
template <int HD, bool KEY, bool FWD, bool CAP, bool BIAS>
__device__ __noinline__ void repair(const Params& p, int h0, int heads, int kh, int row, int2 iv, uint32_t rows,
                                    int c0, int c1, float m2, float D, float inv, int part, int part_n, int split) {
  constexpr int W = HD / 32;
  const int lane = threadIdx.x & 31;
  c1 = min(c1, int(p.plan.T));
  auto clean = [&](int c) {
    if constexpr (FWD) return row_finite<HD>(p.v + int64_t(c) * p.ldv + int64_t(kh) * HD);
    else if constexpr (!KEY) return row_finite<HD>(p.k + int64_t(c) * p.ldk + int64_t(kh) * HD);
    else for (int h = h0; h < h0 + heads; ++h)
      if (!(p.nl[int64_t(h) * p.plan.tiles * BT + c] < INFINITY) ||
          !row_finite<HD>(p.q + int64_t(c) * p.ldq + int64_t(h) * HD) ||
          !row_finite<HD>(p.d_o + int64_t(c) * p.lddo + int64_t(h) * HD)) return false;
    return true;
  };
  int first = 0x7fffffff, last = -1;
#pragma unroll 1
  for (int b = c0; b < c1 && first == 0x7fffffff; b += 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, b + lane < c1 && !clean(b + lane));
    if (m) first = b + __ffs(m) - 1;
  }
  if (first == 0x7fffffff) return;
#pragma unroll 1
  for (int e = c1; e > c0 && last < 0; e -= 32) {
    const int c = e - 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, c >= c0 && !clean(c));
    if (m) last = e - 1 - __clz(m);
  }
  rows &= __ballot_sync(0xffffffffu, first < iv.x || last >= iv.y);
#pragma unroll 1
  while (rows) {
    const int src = __ffs(rows) - 1;
    rows &= rows - 1;
    const int rw = __shfl_sync(0xffffffffu, row, src), lo = __shfl_sync(0xffffffffu, iv.x, src),
              hi = __shfl_sync(0xffffffffu, iv.y, src);
    const float mm = __shfl_sync(0xffffffffu, m2, src), dd = __shfl_sync(0xffffffffu, D, src),
                mul = __shfl_sync(0xffffffffu, inv, src);
    float a1[W] = {}, a2[W] = {};
    bool ok = true;
#pragma unroll 1
    for (int h = h0; h < h0 + heads && ok; ++h)
      ok = redo_row<HD, KEY, FWD, CAP, BIAS>(p, h, kh, rw, lo, hi, mm, dd, a1, a2);
    __syncwarp();
    if (!ok || lane / (32 / part_n) != part) continue;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int64_t c = int64_t(KEY ? kh : h0) * HD + lane * W + e;
      if constexpr (FWD) {
        p.o[int64_t(rw) * p.ldo + c] = __float2bfloat16_rn(a1[e] * mul);
      } else if constexpr (!KEY) {
        p.dq[int64_t(rw) * p.lddq + c] = __float2bfloat16_rn(a1[e] * p.scale);
      } else if (p.split > 1) {
        const int64_t at = (int64_t(split) * p.plan.T + rw) * (int64_t(p.Hkv) * HD) + c;
        p.part_k[at] = a1[e];
        p.part_v[at] = a2[e];
      } else {
        p.dk[int64_t(rw) * p.lddk + c] = __float2bfloat16_rn(a1[e] * p.scale);
        p.dv[int64_t(rw) * p.lddv + c] = __float2bfloat16_rn(a2[e]);
      }
    }
  }
}

// ------------------------------------------------------------------------------ work items

// Asks for the index of a block of this grid that has not started; 16 bytes land at dst.
__device__ __forceinline__ void take_block(uint32_t dst, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
      "r"(bar)
      : "memory");
}
// The index, or −1 where none was left (no further request may follow then).
__device__ __forceinline__ int taken_block(uint32_t src) {
  int x;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "mov.b32 %0, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
      : "=r"(x)
      : "r"(src)
      : "memory");
  return x;
}

// A contiguous copy into shared memory that completes on an mbarrier (16-byte units).
__device__ __forceinline__ void copy_in(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A work item as the producer leaves it for the other warps.
struct alignas(16) Item {
  int h;             // query head, or (key pass) key head; −1: no more
  int tile;          // first tile of the pair; the row tile
  int a, b;          // column tiles of the pair's union; (key pass) first query head, heads
  int4 r0, r1;       // ranges (r1: the pair's second tile, or (split) in x)
};
struct Queue {
  Item item[2];
  uint4 reply;
  uint64_t full[2], empty[2], got;
};

template <bool KEY, bool PAIR>
__device__ __forceinline__ Item describe(const Params& p, int i) {
  Item it;
  const int per = KEY ? p.Hkv * p.split : p.H;
  const int n = i / per, h = i - n * per;
  if constexpr (PAIR) {
    const int4 x = __ldg(p.plan.pairs + 3 * n);
    it.tile = x.x;
    it.a = x.y;
    it.b = x.z;
    it.r0 = __ldg(p.plan.pairs + 3 * n + 1);
    it.r1 = __ldg(p.plan.pairs + 3 * n + 2);
    it.h = h;
  } else {
    const int4* rec = (KEY ? p.plan.ks : p.plan.qs) + 2 * n;
    it.tile = __ldg(rec).x;
    it.r0 = __ldg(rec + 1);
    const int sp = KEY ? h / p.Hkv : 0;
    it.h = KEY ? h - sp * p.Hkv : h;
    it.a = KEY ? it.h * p.group + sp * p.share : h;
    it.b = KEY ? min(p.share, p.group - sp * p.share) : 1;
    it.r1 = make_int4(sp, 0, 0, 0);
  }
  return it;
}

// The producer's side of the queue.
struct Source {
  Queue* q;
  uint32_t n = 0;  // items published
  __device__ __forceinline__ bool publish(const Item& it, uint64_t limit) {
    const uint32_t s = n & 1;
    if (!spin(smem_u32(&q->empty[s]), ((n >> 1) & 1) ^ 1, limit)) return false;
    q->item[s] = it;
    mbar_arrive(smem_u32(&q->full[s]));
    ++n;
    return true;
  }
  // The next block's index (−1: none was left); a request always ends before the block does.  False when its reply did not
  // come: whether a block was taken over is not known then, so the call must report it.
  __device__ __forceinline__ bool take(int& next) {
    const uint32_t bar = smem_u32(&q->got);
    fence_proxy_async_smem();  // the last reply has been read
    mbar_expect_tx(bar, 16);
    take_block(smem_u32(&q->reply), bar);
    if (!mbar_wait(bar, (n - 1) & 1)) return false;
    next = taken_block(smem_u32(&q->reply));
    return true;
  }
};
// Everybody else's: item n, false when the wait ran out.  All lanes of a warp, or one thread (WARP false).
template <bool WARP>
__device__ __forceinline__ bool next_item(Queue* q, uint32_t n, Item& it, uint64_t limit) {
  const uint32_t s = n & 1;
  bool ok = spin(smem_u32(&q->full[s]), (n >> 1) & 1, limit);
  if (WARP) ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  it = q->item[s];
  if (WARP) __syncwarp();
  if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&q->empty[s]));
  return true;
}
__device__ __forceinline__ void queue_init(Queue* q, int readers) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(smem_u32(&q->full[i]), 1);
    mbar_init(smem_u32(&q->empty[i]), readers);
  }
  mbar_init(smem_u32(&q->got), 1);
}

// ------------------------------------------------------------------------------ forward
//
// A work item is a head and a pair of 128-query tiles, one tile per stream; the two streams share the K and V
// tiles (a tile that only one of them meets is released for the other).  Warps: 0 TMA, 1 (and 2) MMA issuers
// (1 owns TMEM), 4–7 and 8–11 the streams' softmax rows, one query row per thread.
// TMEM per stream, 256 columns: S [0, 128) | P | O.  With hd 64 P has 64 columns of its own, S of the next tile
// is computed as soon as the rows have read this one, and each stream has an issuer.  With hd 128 P lies over
// S, so a stream's rows wait while P V and the next S are computed: one thread issues both streams' products
// in turn (P V and S of stream 0, then of stream 1), which sets the streams half a period apart — one is
// at its exponentials while the other's products run.
// What bounds it: the rows (exponentials, their sums and conversions, tensor-memory loads) at hd 64: 8192 tokens
// without masks, 12 heads, 263 us, 784 TFLOP/s, 0.41 of measured; at hd 128 as much time goes into the products: 392 us,
// 1051 TFLOP/s, 0.55.  8192 causal tokens 128 us, where the kernel without masks takes 161.
constexpr int kThreadsFwd = 384;
constexpr uint32_t kFwdRegsCtl = 72, kFwdRegsRows = 216;  // 128·72 + 256·216 = 384·168

template <int HD>
struct FwdCfg {
  static constexpr int QT = HD / 64 * TILE;         // bytes of a 128-row tile
  static constexpr int RING = HD == 64 ? 4 : 2;     // K (and V) tiles in flight
  static constexpr bool OWN_P = HD == 64;
  static constexpr int ISSUERS = OWN_P ? 2 : 1;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * QT;
  static constexpr int V = K + RING * QT;
  static constexpr int ST = V + RING * QT;          // the row warps' output
  static constexpr int BARS = ST + STAGE;
  static constexpr int BYTES = BARS + 1024;
};

template <int HD>
struct FwdBars {
  Queue queue;
  uint64_t k_full[FwdCfg<HD>::RING], k_empty[FwdCfg<HD>::RING], v_full[FwdCfg<HD>::RING], v_empty[FwdCfg<HD>::RING];
  struct Stream {
    uint64_t q_full, q_empty, s_full, s_free, p_full, pv_done;
  } st[2];
  uint64_t mma_done[2];
  uint32_t tmem, abort;
};

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreadsFwd, 1)
    attnm_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                     const __grid_constant__ Params p) {
  using C = FwdCfg<HD>;
  constexpr uint32_t TCOLS = 512, RING = C::RING;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  FwdBars<HD>& B = *reinterpret_cast<FwdBars<HD>*>(smem + C::BARS);
  static_assert(sizeof(FwdBars<HD>) <= 1024, "barrier space");
  volatile uint32_t* abort_flag = &B.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    queue_init(&B.queue, 8 + C::ISSUERS);
    for (uint32_t i = 0; i < RING; ++i) {
      mbar_init(smem_u32(&B.k_full[i]), 1);
      mbar_init(smem_u32(&B.k_empty[i]), C::ISSUERS);
      mbar_init(smem_u32(&B.v_full[i]), 1);
      mbar_init(smem_u32(&B.v_empty[i]), C::ISSUERS);
    }
    for (int st = 0; st < 2; ++st) {
      mbar_init(smem_u32(&B.st[st].q_full), 1);
      mbar_init(smem_u32(&B.st[st].q_empty), 1);
      mbar_init(smem_u32(&B.st[st].s_full), 1);
      mbar_init(smem_u32(&B.st[st].s_free), 4);
      mbar_init(smem_u32(&B.st[st].p_full), 4);
      mbar_init(smem_u32(&B.st[st].pv_done), 1);
      mbar_init(smem_u32(&B.mma_done[st]), 1);
    }
    B.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&B.tmem), TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = B.tmem;
  pdl_begin();
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.flag, XT_DEVERR_TIMEOUT);
  };

  const int wg = warp >> 2;
  if (wg == 0) {
    regs_dec<kFwdRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer, work items
      uint32_t n = 0, nq[2] = {0, 0};  // K / V tiles and Q tiles so far
      bool ok = true;
      Source src{&B.queue};
      Item it;
      it.h = -1;
      if (attn_plan::valid(p.plan)) it = describe<false, true>(p, int(blockIdx.x));
      else if (blockIdx.x == 0) flag_error(p.flag, XT_DEVERR_PLAN);
#pragma unroll 1
      for (;;) {
        if (!src.publish(it, p.wait_ns)) { ok = false; break; }
        if (it.h < 0) break;
        const int kh = it.h / p.group;
#pragma unroll 1
        for (int st = 0; st < 2 && ok; ++st) {
          auto& b = B.st[st];
          if (!mbar_wait(smem_u32(&b.q_empty), (nq[st] & 1) ^ 1, p.wait_ns)) { ok = false; break; }
          mbar_expect_tx(smem_u32(&b.q_full), C::QT);
          Mma<HD>::load(sb + C::Q + st * C::QT, &tmQ, smem_u32(&b.q_full), it.h, it.tile + st);
          ++nq[st];
        }
#pragma unroll 1
        for (int j = it.a; j < it.b && ok; ++j, ++n) {
          const uint32_t s = n % RING, ph = ((n / RING) & 1) ^ 1;
          if (*abort_flag || !mbar_wait(smem_u32(&B.k_empty[s]), ph, p.wait_ns)) { ok = false; break; }
          mbar_expect_tx(smem_u32(&B.k_full[s]), C::QT);
          Mma<HD>::load(sb + C::K + s * C::QT, &tmK, smem_u32(&B.k_full[s]), kh, j);
          if (!mbar_wait(smem_u32(&B.v_empty[s]), ph, p.wait_ns)) {
            ok = false;
            mbar_wait(smem_u32(&B.k_full[s]), (n / RING) & 1);  // this K is in flight
            break;
          }
          mbar_expect_tx(smem_u32(&B.v_full[s]), C::QT);
          Mma<HD>::load(sb + C::V + s * C::QT, &tmV, smem_u32(&B.v_full[s]), kh, j);
        }
        if (!ok || *abort_flag) { ok = false; break; }
        int next;
        if (!src.take(next)) { ok = false; break; }
        if (next >= 0) it = describe<false, true>(p, next);
        else it.h = -1;
      }
      if (!ok) give_up();
      // bounded wait for the fills that may still be in flight
      bool drained = true;
      for (int st = 0; st < 2; ++st)
        if (nq[st] > 0) drained &= mbar_wait(smem_u32(&B.st[st].q_full), (nq[st] - 1) & 1);
      for (uint32_t m = 0; m < (n < RING ? n : RING); ++m) {
        const uint32_t g = n - 1 - m;
        drained &= mbar_wait(smem_u32(&B.k_full[g % RING]), (g / RING) & 1);
        drained &= mbar_wait(smem_u32(&B.v_full[g % RING]), (g / RING) & 1);
      }
      if (!drained) give_up();
    } else if (warp >= 1 && warp <= C::ISSUERS && lane == 0) {
      // -------------------------------------------------------------- MMA issuer: of stream warp − 1, or of both
      const int st0 = C::OWN_P ? warp - 1 : 0, st1 = C::OWN_P ? warp - 1 : 1;
      uint32_t n0 = 0;                       // K / V tiles of earlier items
      uint32_t g[2] = {0, 0};                // score tiles of each stream
      bool ok = true;
      auto tS = [&](int st) { return tbase + uint32_t(256 * st); };
      auto pv = [&](int st, uint32_t n, bool first) -> bool {  // O += P V of ring tile n, the stream's last score tile
        auto& b = B.st[st];
        const uint32_t s = n % RING;
        const uint32_t gg = C::OWN_P ? g[0] : g[st];
        if (!spin(smem_u32(&b.p_full), (gg - 1) & 1, p.wait_ns) ||
            !spin(smem_u32(&B.v_full[s]), (n / RING) & 1, p.wait_ns)) return false;
        tc_fence_after();
        Mma<HD>::tn(tS(st) + (C::OWN_P ? 192u : 128u), tS(st) + (C::OWN_P ? 128u : 0u), 32, sb + C::V + s * C::QT,
                    first);
        tc_commit(smem_u32(&b.pv_done));
        return true;
      };
#pragma unroll 1
      for (uint32_t ni = 0; ok; ++ni) {
        Item it;
        if (*abort_flag || !next_item<false>(&B.queue, ni, it, p.wait_ns)) { ok = false; break; }
        if (it.h < 0) break;
        for (int st = st0; st <= st1 && ok; ++st) ok = spin(smem_u32(&B.st[st].q_full), ni & 1, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        if constexpr (C::OWN_P) {
          // S of a tile goes ahead of P V of the one before
          auto& b = B.st[st0];
          const int4 rg = st0 ? it.r1 : it.r0;
          int pend = -1;  // ring tile whose P V is still to be issued
          bool first = true, held = true;
#pragma unroll 1
          for (int j = it.a; j < it.b; ++j) {
            const uint32_t n = n0 + uint32_t(j - it.a), s = n % RING, ph = (n / RING) & 1;
            const bool mine = j >= rg.x && j < rg.y;
            if (*abort_flag) { ok = false; break; }
            if (pend >= 0 && !mine) {
              if (!pv(st0, uint32_t(pend), first)) { ok = false; break; }
              tc_commit(smem_u32(&B.v_empty[uint32_t(pend) % RING]));
              first = false;
              pend = -1;
            }
            if (!spin(smem_u32(&B.k_full[s]), ph, p.wait_ns)) { ok = false; break; }
            if (!mine) {  // the other stream's tile
              mbar_arrive(smem_u32(&B.k_empty[s]));
              if (!spin(smem_u32(&B.v_full[s]), ph, p.wait_ns)) { ok = false; break; }
              mbar_arrive(smem_u32(&B.v_empty[s]));
              continue;
            }
            if (!spin(smem_u32(&b.s_free), (g[0] & 1) ^ 1, p.wait_ns)) { ok = false; break; }
            tc_fence_after();
            Mma<HD>::nt(tS(st0), sb + C::Q + st0 * C::QT, sb + C::K + s * C::QT);
            tc_commit(smem_u32(&B.k_empty[s]));
            tc_commit(smem_u32(&b.s_full));
            if (j == rg.y - 1) {
              tc_commit(smem_u32(&b.q_empty));
              held = false;
            }
            if (pend >= 0) {
              if (!pv(st0, uint32_t(pend), first)) { ok = false; break; }
              tc_commit(smem_u32(&B.v_empty[uint32_t(pend) % RING]));
              first = false;
            }
            pend = int(n);
            ++g[0];
          }
          if (!ok) break;
          if (pend >= 0) {
            if (!pv(st0, uint32_t(pend), first)) { ok = false; break; }
            tc_commit(smem_u32(&B.v_empty[uint32_t(pend) % RING]));
          }
          if (held) mbar_arrive(smem_u32(&b.q_empty));
        } else {
          bool pend[2] = {false, false}, first[2] = {true, true}, held[2] = {true, true};
#pragma unroll 1
          for (int j = it.a; j <= it.b && ok; ++j) {  // one step more than tiles: the last P V
            const uint32_t n = n0 + uint32_t(j - it.a), s = n % RING;
            if (*abort_flag) { ok = false; break; }
            if (j < it.b && !spin(smem_u32(&B.k_full[s]), (n / RING) & 1, p.wait_ns)) { ok = false; break; }
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              auto& b = B.st[st];
              const int4 rg = st ? it.r1 : it.r0;
              if (pend[st]) {
                if (!pv(st, n - 1, first[st])) { ok = false; break; }
                first[st] = false;
                pend[st] = false;
              }
              if (j < it.b && j >= rg.x && j < rg.y) {
                tc_fence_after();
                Mma<HD>::nt(tS(st), sb + C::Q + st * C::QT, sb + C::K + s * C::QT);
                tc_commit(smem_u32(&b.s_full));
                if (j == rg.y - 1) {
                  tc_commit(smem_u32(&b.q_empty));
                  held[st] = false;
                }
                pend[st] = true;
                ++g[st];
              }
            }
            if (!ok) break;
            if (j < it.b) tc_commit(smem_u32(&B.k_empty[s]));
            if (j > it.a) {
              const uint32_t m = n - 1;
              if (!spin(smem_u32(&B.v_full[m % RING]), (m / RING) & 1, p.wait_ns)) { ok = false; break; }
              tc_commit(smem_u32(&B.v_empty[m % RING]));
            }
          }
          if (!ok) break;
          for (int st = 0; st < 2; ++st)
            if (held[st]) mbar_arrive(smem_u32(&B.st[st].q_empty));
        }
        n0 += uint32_t(it.b - it.a);
      }
      if (!ok) give_up();
      // every MMA issued has completed (also after a give-up) before TMEM is released
      tc_commit(smem_u32(&B.mma_done[warp - 1]));
      if (!mbar_wait(smem_u32(&B.mma_done[warp - 1]), 0)) give_up();
    }
  } else {
    regs_inc<kFwdRegsRows>();
    // ---------------------------------------------------------------- softmax rows, epilogue
    const int st = wg - 1;
    auto& b = B.st[st];
    const int qw = warp & 3;
    const int rr = qw * 32 + lane;
    const uint32_t lane_off = uint32_t(qw * 32) << 16;
    const uint32_t tS = tbase + uint32_t(256 * st) + lane_off, tP = tS + (C::OWN_P ? 128u : 0u),
                   tO = tS + (C::OWN_P ? 192u : 128u);
    uint32_t g = 0;
#pragma unroll 1
    for (uint32_t ni = 0;; ++ni) {
      bool ok = !__shfl_sync(0xffffffffu, *abort_flag, 0);
      int h, tile;
      int4 rg;
      {
        Item it;
        it.h = -1;
        if (ok) ok = next_item<true>(&B.queue, ni, it, p.wait_ns);
        h = it.h;
        tile = it.tile + st;
        rg = st ? it.r1 : it.r0;
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      if (h < 0) break;
      if (tile >= p.plan.tiles) continue;
      const int row = tile * BT + rr;
      const int2 iv = __ldg(p.plan.q_iv + row);
      const float slope2 = BIAS ? __ldg(p.slopes + h) * kLog2e : 0.f;
      float m = -INFINITY;  // running max of the scores before `unit`
      float l = 0.f;        // running Σ 2^((s − m)·unit)
      const float unit = score_unit<CAP, BIAS>(p);
#pragma unroll 1
      for (int j = rg.x; j < rg.y; ++j, ++g) {
        if (!warp_wait(smem_u32(&b.s_full), g & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + uint32_t(c * 32), *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
        tmem_ld_wait();
        if (C::OWN_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&b.s_free));
        }
        if constexpr (CAP) {
          __half2 none[1];
          tanh_cap<128, false>(s, p, none);
        }
        if constexpr (BIAS) add_bias(s, CAP ? p.cap2 : p.sc, slope2, j * BT - row, j < tile ? 1 : j > tile ? -1 : 0);
        if (j < rg.z || j >= rg.w) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t seen = visible_bits(iv.x - j * BT, iv.y - j * BT, 32 * w);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen & (1u << c))) s[32 * w + c] = __float_as_uint(-INFINITY);
          }
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
        if (C::OWN_P && !warp_wait(smem_u32(&b.pv_done), (g & 1) ^ 1, p.wait_ns)) { ok = false; break; }
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
        if (lane == 0) mbar_arrive(smem_u32(&b.p_full));
      }
      if (ok && rg.y > rg.x && !warp_wait(smem_u32(&b.pv_done), (g - 1) & 1, p.wait_ns)) ok = false;
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      // ---- epilogue: O / l
      const bool seen = m > -INFINITY || l != 0.f;  // l: a NaN score leaves m at −∞
      const float inv = seen ? 1.f / l : 0.f;
      const bool real = row < p.plan.T;
      tc_fence_after();
      float bad = 0.f;
      // Not unrolled, and O is read even where no tile was met (`seen` leaves it out): with both the other way the scores'
      // loop has fewer registers (capped long text 689 us against 727).
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + uint32_t(c * 32), o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float x = seen ? __uint_as_float(o[e]) * inv : 0.f;
          bad = fmaf(x, 0.f, bad);
          o[e] = __float_as_uint(x);
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
        put_rows<false>(smem + C::ST, c & 1, &tmO, w, c * 32, h, row - lane, 0, p.plan.T);
      }
      tc_fence_before();
      if (real) p.lse[int64_t(h) * p.plan.T + row] = seen ? (m * unit + log2f(l)) * kLn2 : -INFINITY;
      const uint32_t rows = __ballot_sync(0xffffffffu, bad != 0.f && l == l && real);
      if (rows) {
        rows_stored();
        repair<HD, false, true, CAP, BIAS>(p, h, 1, h / p.group, row, iv, rows, rg.x * BT, rg.y * BT, m * unit, 0.f,
                                           inv, 0, 1, 0);
      }
    }
    rows_stored();
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
// columns queries; dK and dV sum over the query tiles that see the tile, for the query heads of the group in
// turn.  else: an item is a query tile of a head, a row a query, the columns keys; dQ sums over key tiles.
// Per tile: S = (row tile)(column tile)ᵀ and dP likewise into TMEM; the rows form P = 2^(s − lse) and write it
// over S for dV += P dO (KEY); then dS = P∘(dP − D)∘(1 − tanh²) over dP for dK (dQ) += dS Q (K).
//
// D.  D = Σ_j P dP over a whole row, but is wanted from the row's first tile on; dO·O has it up to the rounding of
// the stored O, 2⁻⁹ of |dO||O|, which where P is peaked is several times the error of everything else in dS (dQ
// off by 5.8e-3 against 2.5e-3, texts of 12 tokens).  So the query pass takes D₀ = dO·O for its dS, sums
// T = Σ_j P(dP − D₀) beside it in float32, and adds up W K, W = P∘(1 − tanh²), as a second product: with
// D = D₀ + T,  dQ = scale·(Σ dS₀ K − T·Σ W K)  exactly.  It leaves −lse·log₂e and −D in the workspace, rows padded
// to whole tiles, from where the key pass, which follows it, copies them in with each query tile.
//
// Rounding dS to bf16 puts as much error into dK and dQ as their own rounding (2.4e-3 of both against float64, 1.7e-3
// without).  Where few elements carry a row, the total varies most: so an edge tile's dS, and short documents have no other tiles,
// is multiplied as the sum of two bf16s, the rounded value and what the rounding left, which has room in the chunk's own
// columns: their dK and dQ (without a cap: 1 − tanh² has 11 bits) are as exact as float32 arithmetic rounded once, for 9 % of
// the backward where most tiles are edges (23 packed texts: 102 us, 93 without) and 2 % in a long text.  One loop issues both
// terms: a second copy of the products' code makes their issuer spill (8192 unmasked tokens at hd 128: 1574 us against 1317).
//
// A tile's time is the rows' chain of tensor-memory loads, exponentials, stores and barriers, several times the
// work in it, so two chains run side by side: each half of a tile's 128 columns has its own MMA issuer, four row
// warps (one per TMEM lane quadrant), S and dP buffers, accumulators and barriers; P and dS are elementwise, so
// the halves never need each other until their accumulators are added at the end of an item, in the halves' order
// (deterministic).  One chain's products and loads run during the other's exponentials.  At hd 128 there is tensor
// memory for one set of accumulators: there the halves' rows share one chain of 128 columns.
//
// What bounds it: the rows' chain at hd 64 (issue slots and tensor-memory latency: 8192 tokens without masks, 12 heads,
// both passes: 900 us, 573 TFLOP/s of the formulas' five products and 917 of the eight that run, 0.48 of measured; one
// chain of whole tiles instead of two took 8 % more), at hd 128 the products beside it (1317 us, 782 and 1252 TFLOP/s,
// 0.66 of measured).  Packed short texts pay for the parts of tiles that their masks hide, and some 4000 cycles per item
// for D₀, the last products' arrival and the epilogue, where an unmasked tile takes 2100 (hd 64) to 2900 (hd 128): together
// three quarters of the time of 23 packed texts and half that of 40 capped ones, the rest being what edge tiles (masks, two
// terms of dS) and caps take on top.
constexpr int kThreadsBwd = 384;  // warps 0 TMA, 1 (and 2) MMA, 4–7 and 8–11 the halves' rows
constexpr uint32_t kBwdRegsCtl = 88, kBwdRegsRows = 208;  // 128·88 + 256·208 = 384·168; at 72 the query pass's issuer
// spills at hd 128 (8192 unmasked tokens: 1383 us against 1300), where the forward's does not (above)
constexpr int PW = BT / 2;        // columns of a row warp

template <int HD, bool KEY>
struct BwdCfg {
  static constexpr int QT = HD / 64 * TILE;
  static constexpr int RING = HD == 64 ? 4 : 2;          // column tiles (pairs) in flight
  static constexpr int CH = HD == 128 ? 1 : 2;           // chains
  // TMEM columns: S, dP (the halves' side by side), each chain's dK or dQ, each chain's dV or W K
  static constexpr uint32_t DP = 128, ACC1 = 256, ACC2 = ACC1 + CH * HD;
  static constexpr int A = 0;                            // the row tiles: K, V or Q, dO
  static constexpr int R = A + 2 * QT;                   // ring of column tile pairs: Q, dO or K, V
  static constexpr int VEC = R + RING * 2 * QT;          // (KEY) ring of −lse·log₂e and −D, 128 floats each; or sums of halves
  static constexpr int ST = VEC + RING * 1024;           // the row warps' output
  static constexpr int BARS = ST + STAGE;
  static constexpr int BYTES = BARS + 512;
  static_assert(BYTES <= 227 * 1024, "shared memory");
  static_assert(ACC2 + CH * HD <= 512, "TMEM columns");
};

template <int HD, bool KEY>
struct BwdBars {
  Queue queue;
  uint64_t a_full, a_empty, r_full[BwdCfg<HD, KEY>::RING], r_empty[BwdCfg<HD, KEY>::RING];
  struct Chain {
    uint64_t s_full, dp_full, p_full, ds_full, acc_full, mma_done;
  } ch[2];
  uint64_t acc_free, met[4];
  uint32_t tmem, abort;
};

template <int HD, bool KEY, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreadsBwd, 1)
    attnm_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmG1, const __grid_constant__ CUtensorMap tmG2,
                     const __grid_constant__ Params p) {
  using C = BwdCfg<HD, KEY>;
  constexpr uint32_t TCOLS = 512, RING = C::RING;
  constexpr int CH = C::CH;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  BwdBars<HD, KEY>& B = *reinterpret_cast<BwdBars<HD, KEY>*>(smem + C::BARS);
  static_assert(sizeof(BwdBars<HD, KEY>) <= 512, "barrier space");
  volatile uint32_t* abort_flag = &B.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    queue_init(&B.queue, 8 + CH);
    mbar_init(smem_u32(&B.a_full), 1);
    mbar_init(smem_u32(&B.a_empty), CH);
    for (uint32_t i = 0; i < RING; ++i) {
      mbar_init(smem_u32(&B.r_full[i]), 1);
      mbar_init(smem_u32(&B.r_empty[i]), CH);
    }
    for (int c = 0; c < CH; ++c) {
      mbar_init(smem_u32(&B.ch[c].s_full), 1);
      mbar_init(smem_u32(&B.ch[c].dp_full), 1);
      mbar_init(smem_u32(&B.ch[c].p_full), 8 / CH);
      mbar_init(smem_u32(&B.ch[c].ds_full), 8 / CH);
      mbar_init(smem_u32(&B.ch[c].acc_full), 1);
      mbar_init(smem_u32(&B.ch[c].mma_done), 1);
    }
    mbar_init(smem_u32(&B.acc_free), 8);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&B.met[i]), 2);
    B.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmDO);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&B.tmem), TCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = B.tmem;
  pdl_begin();
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.flag, XT_DEVERR_TIMEOUT);
  };
  const int64_t Tp = int64_t(p.plan.tiles) * BT;  // row stride of nl and nd

  if (warp < 4) {
    regs_dec<kBwdRegsCtl>();
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------------- TMA producer, work items
      const CUtensorMap *tmA1 = KEY ? &tmK : &tmQ, *tmA2 = KEY ? &tmV : &tmDO;
      const CUtensorMap *tmR1 = KEY ? &tmQ : &tmK, *tmR2 = KEY ? &tmDO : &tmV;
      uint32_t na = 0, n = 0;
      bool ok = true;
      Source src{&B.queue};
      Item it;
      it.h = -1;
      if (attn_plan::valid(p.plan)) it = describe<KEY, false>(p, int(blockIdx.x));
      else if (blockIdx.x == 0) flag_error(p.flag, XT_DEVERR_PLAN);
#pragma unroll 1
      for (;;) {
        if (!src.publish(it, p.wait_ns)) { ok = false; break; }
        if (it.h < 0) break;
        const int tiles = it.r0.y - it.r0.x, kh = KEY ? it.h : it.h / p.group;
        if (tiles > 0) {
          if (!mbar_wait(smem_u32(&B.a_empty), (na & 1) ^ 1, p.wait_ns)) { ok = false; break; }
          mbar_expect_tx(smem_u32(&B.a_full), 2 * C::QT);
          Mma<HD>::load(sb + C::A, tmA1, smem_u32(&B.a_full), it.h, it.tile);
          Mma<HD>::load(sb + C::A + C::QT, tmA2, smem_u32(&B.a_full), it.h, it.tile);
          ++na;
        }
#pragma unroll 1
        for (int u = 0; u < it.b && ok; ++u)
#pragma unroll 1
          for (int t = it.r0.x; t < it.r0.y; ++t, ++n) {
            const uint32_t s = n % RING;
            if (*abort_flag || !mbar_wait(smem_u32(&B.r_empty[s]), ((n / RING) & 1) ^ 1, p.wait_ns)) {
              ok = false;
              break;
            }
            const uint32_t fb = smem_u32(&B.r_full[s]), dst = sb + C::R + s * 2 * C::QT;
            mbar_expect_tx(fb, 2 * C::QT + (KEY ? 1024 : 0));
            Mma<HD>::load(dst, tmR1, fb, KEY ? it.a + u : kh, t);
            Mma<HD>::load(dst + C::QT, tmR2, fb, KEY ? it.a + u : kh, t);
            if constexpr (KEY) {
              const int64_t at = int64_t(it.a + u) * Tp + int64_t(t) * BT;
              copy_in(sb + C::VEC + s * 1024, p.nl + at, 512, fb);
              copy_in(sb + C::VEC + s * 1024 + 512, p.nd + at, 512, fb);
            }
          }
        if (!ok || *abort_flag) { ok = false; break; }
        int next;
        if (!src.take(next)) { ok = false; break; }
        if (next >= 0) it = describe<KEY, false>(p, next);
        else it.h = -1;
      }
      if (!ok) give_up();
      bool drained = true;
      if (na > 0) drained &= mbar_wait(smem_u32(&B.a_full), (na - 1) & 1);
      for (uint32_t m = 0; m < (n < RING ? n : RING); ++m) {
        const uint32_t g = n - 1 - m;
        drained &= mbar_wait(smem_u32(&B.r_full[g % RING]), (g / RING) & 1);
      }
      if (!drained) give_up();
    } else if (warp >= 1 && warp <= CH && lane == 0) {
      // -------------------------------------------------------------- MMA issuer of chain warp − 1
      const int c = warp - 1;
      auto& b = B.ch[c];
      uint32_t na = 0, g = 0;  // items with tiles, tiles
      bool ok = true;
      const uint32_t a1 = sb + C::A, a2 = a1 + C::QT;
      const uint32_t tS = tbase + PW * c, tDP = tS + C::DP, acc1 = tbase + C::ACC1 + HD * c, acc2 = tbase + C::ACC2 + HD * c;
      auto slot = [&](uint32_t n) { return sb + C::R + (n % RING) * 2 * C::QT + uint32_t(c) * (PW * 128); };
      auto issue_s = [&](uint32_t n) -> bool {
        if (!spin(smem_u32(&B.r_full[n % RING]), (n / RING) & 1, p.wait_ns)) return false;
        tc_fence_after();
        Mma<HD>::template nt<BT / CH>(tS, a1, slot(n));
        tc_commit(smem_u32(&b.s_full));
        return true;
      };
      auto issue_dp = [&](uint32_t n) {
        Mma<HD>::template nt<BT / CH>(tDP, a2, slot(n) + C::QT);
        tc_commit(smem_u32(&b.dp_full));
      };
#pragma unroll 1
      for (uint32_t ni = 0; ok; ++ni) {
        Item it;
        if (*abort_flag || !next_item<false>(&B.queue, ni, it, p.wait_ns)) { ok = false; break; }
        if (it.h < 0) break;
        const int n = (it.r0.y - it.r0.x) * it.b;
        if (n <= 0) continue;
        int t = it.r0.x;
        if (!spin(smem_u32(&B.a_full), na & 1, p.wait_ns)) { ok = false; break; }
        ++na;
        tc_fence_after();
        if (!issue_s(g)) { ok = false; break; }
        issue_dp(g);
        if (n == 1) tc_commit(smem_u32(&B.a_empty));
        // the rows of both halves have read the last item's accumulators
        if (!spin(smem_u32(&B.acc_free), na & 1, p.wait_ns)) { ok = false; break; }
#pragma unroll 1
        for (int j = 0; j < n; ++j, ++g) {
          const bool next = j + 1 < n;
          if (*abort_flag) { ok = false; break; }
          // the next S follows as soon as P has been multiplied (it lies over S)
          if (!spin(smem_u32(&b.p_full), g & 1, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          Mma<HD>::template tn<BT / CH>(acc2, tS, PW, slot(g) + (KEY ? C::QT : 0), j == 0);  // dV += Pᵀ dO, or W K
          if (next && !issue_s(g + 1)) { ok = false; break; }
          if (!spin(smem_u32(&b.ds_full), g & 1, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          const int terms = t < it.r0.z || t >= it.r0.w ? 2 : 1;  // dS of an edge tile: with its remainders
#pragma unroll 1
          for (int r = 0; r < terms; ++r)  // dK += dSᵀ Q, dQ += dS K
            Mma<HD>::template tn<BT / CH, 32>(acc1, tDP + uint32_t(16 * r), 32, slot(g), j == 0 && r == 0);
          if (++t == it.r0.y) t = it.r0.x;
          tc_commit(smem_u32(&B.r_empty[g % RING]));
          if (next) {
            issue_dp(g + 1);
            if (j + 2 == n) tc_commit(smem_u32(&B.a_empty));  // the last tile's S and dP: the row tiles are free
          }
        }
        if (!ok) break;
        tc_commit(smem_u32(&b.acc_full));
      }
      if (!ok) give_up();
      tc_commit(smem_u32(&b.mma_done));
      if (!mbar_wait(smem_u32(&b.mma_done), 0)) give_up();
    }
  } else {
    regs_inc<kBwdRegsRows>();
    // ---------------------------------------------------------------- rows
    const int qw = warp & 3, half = (warp - 4) >> 2, col0 = PW * half;
    const int rr = qw * 32 + lane;
    const uint32_t lane_off = uint32_t(qw * 32) << 16;
    const uint32_t tS = tbase + lane_off + uint32_t(col0);
    const uint32_t tDP = tS + C::DP;
    auto& b = B.ch[CH == 2 ? half : 0];
    const int64_t T = p.plan.T;
    uint32_t g = 0, na = 0, nm = 0;
    // The two halves' warps of a row have written their parts; false when the wait ran out.
    auto meet_halves = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&B.met[qw]));
      return warp_wait(smem_u32(&B.met[qw]), nm++ & 1, p.wait_ns);
    };
#pragma unroll 1
    for (uint32_t ni = 0;; ++ni) {
      bool ok = !__shfl_sync(0xffffffffu, *abort_flag, 0);
      int h, tile, h0, heads, sp;
      int4 rg;
      {
        Item it;
        it.h = -1;
        if (ok) ok = next_item<true>(&B.queue, ni, it, p.wait_ns);
        h = it.h;
        tile = it.tile;
        h0 = it.a;
        heads = it.b;
        rg = it.r0;
        sp = it.r1.x;
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      if (h < 0) break;
      const int row = tile * BT + rr;
      const bool real = row < T;
      const int2 iv = __ldg((KEY ? p.plan.k_iv : p.plan.q_iv) + row);
      const int n = max(rg.y - rg.x, 0) * heads;
      float nlse = -INFINITY, nD = 0.f, T1 = 0.f;  // not KEY: −lse·log₂e, −D₀ and this half's share of T of the row
      if constexpr (!KEY) {
        // each half takes 16 of the warp's 32 rows
        if (n > 0) {
          float lse = -INFINITY;
          if (real) lse = p.lse[int64_t(h) * T + row];
          float* meet = reinterpret_cast<float*>(smem + C::VEC) + (nm & 1) * 256 + qw * 32;
          dots16<HD>(p.o + int64_t(h) * HD, p.ldo, p.d_o + int64_t(h) * HD, p.lddo,
                     int64_t(tile) * BT + qw * 32 + half * 16, T, meet + half * 16);
          ok = meet_halves();
          if (iv.y > iv.x) {
            nD = -meet[lane];
            if (lse != -INFINITY) nlse = lse * -kLog2e;
          }
        }
      }
      int hq = KEY ? h0 : h, t = rg.x;
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j, ++g) {
        const float* lv = reinterpret_cast<const float*>(smem + C::VEC + (g % RING) * 1024) + col0;
        const float slope2 = BIAS ? __ldg(p.slopes + hq) * kLog2e : 0.f;
        if (!warp_wait(smem_u32(&b.s_full), g & 1, p.wait_ns)) { ok = false; break; }
        // (complete: S was computed from the same arrival; the wait makes the copied vectors visible here)
        if (KEY && !warp_wait(smem_u32(&B.r_full[g % RING]), (g / RING) & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[PW];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(s));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
        tmem_ld_wait();
        const float unit = score_unit<CAP, BIAS>(p);
        __half2 slack[CAP ? PW / 2 : 1];  // kSlack (1 − tanh²)
        if constexpr (CAP) tanh_cap<PW, true>(s, p, slack);
        if constexpr (BIAS)
          add_bias(s, CAP ? p.cap2 : p.sc, slope2, t * BT + col0 - row, t < tile ? 1 : t > tile ? -1 : 0);
        const bool edge = t < rg.z || t >= rg.w;
        uint32_t seen[2] = {~0u, ~0u};
        if (edge) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            seen[w] = visible_bits(iv.x - t * BT, iv.y - t * BT, col0 + 32 * w);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen[w] & (1u << c))) s[32 * w + c] = __float_as_uint(-INFINITY);
          }
        }
        const uint64_t unit2 = f32x2_pack(unit, unit);
#pragma unroll
        for (int c = 0; c < PW; c += 32) {  // 32 columns at a time: 16 registers of P
          uint32_t pk[16];
#pragma unroll
          for (int e = c; e < c + 32; e += 4) {
            float4 nl = make_float4(nlse, nlse, nlse, nlse);
            if constexpr (KEY) nl = *reinterpret_cast<const float4*>(lv + e);
            float x[4];
            f32x2_unpack(f32x2_fma(pair(s[e], s[e + 1]), unit2, f32x2_pack(nl.x, nl.y)), x[0], x[1]);
            f32x2_unpack(f32x2_fma(pair(s[e + 2], s[e + 3]), unit2, f32x2_pack(nl.z, nl.w)), x[2], x[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = ex2(x[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) s[e + k] = __float_as_uint(x[k]);
            if constexpr (!KEY && CAP) {  // W (a masked column's tanh may be NaN: its P stays 0)
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const float2 u = __half22float2(slack[(e + k) / 2]);
                x[k] = x[k] == 0.f ? 0.f : x[k] * u.x;
                x[k + 1] = x[k + 1] == 0.f ? 0.f : x[k + 1] * u.y;
              }
            }
            pk[(e - c) >> 1] = pack_bf16(x[0], x[1]);
            pk[((e - c) >> 1) + 1] = pack_bf16(x[2], x[3]);
          }
          tmem_st16(tS + uint32_t(c / 2), pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b.p_full));
        if (!warp_wait(smem_u32(&b.dp_full), g & 1, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        uint64_t dot[2] = {0, 0};
        auto form_ds = [&](auto masked) {
#pragma unroll
          for (int c = 0; c < PW; c += 32) {
            uint32_t d[32], pk[16], rest[16];
            tmem_ld32(tDP + uint32_t(c), d);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 nd = make_float4(nD, nD, nD, nD);
              if constexpr (KEY) nd = *reinterpret_cast<const float4*>(lv + 128 + c + e);
              float x[4];
              f32x2_unpack(f32x2_mul(f32x2_add(pair(d[e], d[e + 1]), f32x2_pack(nd.x, nd.y)), pair(s[c + e], s[c + e + 1])),
                           x[0], x[1]);
              f32x2_unpack(f32x2_mul(f32x2_add(pair(d[e + 2], d[e + 3]), f32x2_pack(nd.z, nd.w)),
                                     pair(s[c + e + 2], s[c + e + 3])), x[2], x[3]);
              auto hide = [&]() {  // a masked column's dP, D or tanh may be NaN
                if constexpr (decltype(masked)::value) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    if (!(seen[c / 32] & (1u << (e + k)))) x[k] = 0.f;
                }
              };
              if constexpr (!KEY) {
                hide();
                dot[0] = f32x2_add(dot[0], f32x2_pack(x[0], x[1]));
                dot[1] = f32x2_add(dot[1], f32x2_pack(x[2], x[3]));
              }
              if constexpr (CAP) {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const float2 u = __half22float2(slack[(c + e + k) / 2]);
                  x[k] *= u.x;
                  x[k + 1] *= u.y;
                }
              }
              if constexpr (KEY || CAP) hide();
              pk[e >> 1] = pack_bf16(x[0], x[1]);
              pk[(e >> 1) + 1] = pack_bf16(x[2], x[3]);
              if constexpr (decltype(masked)::value) {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                  const uint32_t w = pk[(e + k) >> 1];
                  rest[(e + k) >> 1] =
                      pack_bf16(x[k] - __uint_as_float(w << 16), x[k + 1] - __uint_as_float(w & 0xFFFF0000u));
                }
              }
            }
            tmem_st16(tDP + uint32_t(c), pk);
            if constexpr (decltype(masked)::value) tmem_st16(tDP + uint32_t(c + 16), rest);
          }
        };
        if (edge) form_ds(std::true_type{});
        else form_ds(std::false_type{});
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b.ds_full));
        if constexpr (!KEY) {
          float u, w;
          f32x2_unpack(f32x2_add(dot[0], dot[1]), u, w);
          T1 += u + w;
        }
        if (++t == rg.y) {
          t = rg.x;
          ++hq;
        }
      }
      if (ok && n > 0) {
        for (int c = 0; c < CH; ++c) ok = ok && warp_wait(smem_u32(&B.ch[c].acc_full), na & 1, p.wait_ns);
        ++na;
      }
      float Tr = 0.f;
      if constexpr (!KEY) {
        if (ok && n > 0) {  // added in the halves' order
          float* meet = reinterpret_cast<float*>(smem + C::VEC) + (nm & 1) * 256;
          meet[half * 128 + rr] = T1;
          ok = meet_halves();
          Tr = meet[rr] + meet[128 + rr];
        }
        if (ok && half == 0) {
          p.nl[int64_t(h) * Tp + row] = nlse;
          p.nd[int64_t(h) * Tp + row] = nD - Tr;
        }
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      // ---- epilogue: this half's HD/2 columns of the accumulators
      tc_fence_after();
      float bad = 0.f;
      auto load_acc = [&](uint32_t at, uint32_t(&o)[32]) {  // 32 columns of both chains' accumulators
        tmem_ld32(at, o);
        if constexpr (CH == 2) {
          uint32_t o1[32];
          tmem_ld32(at + HD, o1);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(o1[e]));
        } else {
          tmem_ld_wait();
        }
      };
      // Not unrolled, and the accumulators are read even where no tile was met (the select leaves them out): with both the
      // other way the tiles' loop has fewer registers (capped texts, heads of 128: backward 70 us against 78).
#pragma unroll 1
      for (int w = 0; w < (KEY ? 2 : 1); ++w) {
        const CUtensorMap* tm = w ? &tmG2 : &tmG1;
        const bool raw = KEY && p.split > 1;  // the part's float32 sums
        const float mul = w ? 1.f : (CAP ? 1.f / kSlack : 1.f) * (raw ? 1.f : p.scale);
        const uint32_t acc = tbase + (w ? C::ACC2 : C::ACC1) + lane_off + uint32_t(half * (HD / 2));
#pragma unroll 1
        for (int c = 0; c < HD / 2; c += 32) {
          uint32_t o[32];
          load_acc(acc + uint32_t(c), o);
          if constexpr (!KEY) {
            uint32_t wk[32];
            load_acc(tbase + C::ACC2 + lane_off + uint32_t(half * (HD / 2) + c), wk);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(fmaf(-Tr, __uint_as_float(wk[e]), __uint_as_float(o[e])));
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = n > 0 ? __uint_as_float(o[e]) * mul : 0.f;
            bad = fmaf(x, 0.f, bad);
            o[e] = __float_as_uint(x);
          }
          uint32_t x[16];
          const int col = half * (HD / 2) + c;
          if (raw) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = o[16 * u + e];
              put_rows<false>(smem + C::ST, u, tm, x, col + 16 * u, h, row - lane, sp, T);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            put_rows<!KEY && HD == 64>(smem + C::ST, (w * (HD / 64) + c / 32) & 1, tm, x, col, h, row - lane, 0, T);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (n > 0 && lane == 0) mbar_arrive(smem_u32(&B.acc_free));
      const uint32_t rows = __ballot_sync(0xffffffffu, bad != 0.f && real);
      if (rows) {
        rows_stored();
        repair<HD, KEY, false, CAP, BIAS>(p, KEY ? h0 : h, heads, KEY ? h : h / p.group, row, iv, rows, rg.x * BT,
                                          rg.y * BT, -nlse, Tr - nD, 0.f, half, 2, sp);
      }
    }
    rows_stored();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TCOLS);
  }
}

// ------------------------------------------------------------------------------ launches

// Raises the kernel's shared-memory limit on the current device and, for a kernel that splits its registers,
// checks that it was built with the count the split adds up to (any other could never be met).  `ready` has a bit
// for each device where that is done.
int prepare_kernel(std::atomic<uint64_t>& ready, const void* kernel, int smem, int regs);

template <int HD>
int launch_fwd(bool cap, bool bias, const CUtensorMap (&tm)[4], const Params& p, cudaStream_t s);
template <int HD, bool KEY>
int launch_bwd(bool cap, bool bias, const CUtensorMap (&tm)[4], const CUtensorMap& g1, const CUtensorMap& g2,
               const Params& p, cudaStream_t s);

#define XT_ATTNM_FWD(HD)                                                                                         \
  template <bool CAP, bool BIAS>                                                                                 \
  static int fwd_one(const CUtensorMap (&tm)[4], const Params& p, cudaStream_t s) {                              \
    static std::atomic<uint64_t> ready{0};                                                                       \
    auto k = attnm_fwd_kernel<HD, CAP, BIAS>;                                                                    \
    XT_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(k), FwdCfg<HD>::BYTES, 168));                     \
    const int64_t items = int64_t((p.plan.tiles + 1) / 2) * p.H;                                                 \
    launch(k, unsigned(items), kThreadsFwd, FwdCfg<HD>::BYTES, s, tm[0], tm[1], tm[2], tm[3], p);                \
    return check_launch("xt_attention_masked_fwd");                                                              \
  }                                                                                                              \
  template <>                                                                                                    \
  int launch_fwd<HD>(bool cap, bool bias, const CUtensorMap (&tm)[4], const Params& p, cudaStream_t s) {         \
    if (cap) return bias ? fwd_one<true, true>(tm, p, s) : fwd_one<true, false>(tm, p, s);                       \
    return bias ? fwd_one<false, true>(tm, p, s) : fwd_one<false, false>(tm, p, s);                              \
  }

#define XT_ATTNM_BWD(HD, KEY)                                                                                    \
  template <bool CAP, bool BIAS>                                                                                 \
  static int bwd_one(const CUtensorMap (&tm)[4], const CUtensorMap& g1, const CUtensorMap& g2, const Params& p,  \
                     cudaStream_t s) {                                                                           \
    static std::atomic<uint64_t> ready{0};                                                                       \
    auto k = attnm_bwd_kernel<HD, KEY, CAP, BIAS>;                                                               \
    XT_TRY(prepare_kernel(ready, reinterpret_cast<const void*>(k), BwdCfg<HD, KEY>::BYTES, 168));                \
    const int64_t items = int64_t(p.plan.tiles) * (KEY ? p.Hkv * p.split : p.H);                                 \
    launch(k, unsigned(items), kThreadsBwd, BwdCfg<HD, KEY>::BYTES, s, tm[0], tm[1], tm[2], tm[3], g1, g2, p);   \
    return check_launch("xt_attention_masked_bwd");                                                              \
  }                                                                                                              \
  template <>                                                                                                    \
  int launch_bwd<HD, KEY>(bool cap, bool bias, const CUtensorMap (&tm)[4], const CUtensorMap& g1,                \
                          const CUtensorMap& g2, const Params& p, cudaStream_t s) {                              \
    if (cap) return bias ? bwd_one<true, true>(tm, g1, g2, p, s) : bwd_one<true, false>(tm, g1, g2, p, s);       \
    return bias ? bwd_one<false, true>(tm, g1, g2, p, s) : bwd_one<false, false>(tm, g1, g2, p, s);              \
  }

}  // namespace attnm
}  // namespace xt
