// AdamW over many tensors with the two moments held in 8 bits, and their decoding.
//
// Held state.  256 consecutive elements of a tensor share two scales.  The first moment is an
// int8 code c with m = ms·c·|c|; of the second the root is held, as a uint8 code c with r = rs·c²
// and v = r².  The square law spends its codes where the values are: a code step is 2/c of the
// value, 0.8 % (v) and 1.6 % (m) at the block's largest, and values down to 1/65025 of the largest
// root stay apart from zero (a linear code's smallest is 1/255: a weight with a small second moment
// would be stepped with none).  A positive v keeps a code of at least 1 for the same reason.
//
// The step, on float32 values (f = grad_scale times the clip factor):
//   g' = f·g,  m' = β₁ m + (1−β₁) g',  v' = β₂ v + ((1−β₂) g')·g',
//   θ  = θ(1 − lr·λ) − lr·(m'/bc₁)/(√(v'/bc₂) + ε)      (from m', v' before they are coded),
//   ms = max|m'|/127²,  c = sign(m')·rint(√(|m'|/ms)),   rs = √(max v')/255²,  c = rint(√(√v'/rs)).
// Codes are whole numbers, so the value that is coded is defined to the last bit: every operation of
// m', v' and of the codes is rounded to float32 by itself (no fused multiply-add).  The code is found
// with approximate roots, and only an element that lies within their error of a border between two
// codes is done over with the exactly rounded ones.  The gradient norm behind f is a sum in pairs of
// float32 (relative error ~2⁻⁴⁴; GB300's float64 units are too few to add every element, or for every
// thread to take the norm's root), so f is the rounding of the true value.
//
// Memory-bound: 18 bytes per element (weight 8, gradient 4, codes 4, bf16 working copy 2) and 4 more
// for the norm's pass.  A warp takes one block of 256 at a time: its lanes hold the block's values in
// registers between the two maxima and the coding.  104.7 M weights in 74 tensors with a bf16 working copy: update 353 us
// (5.34 TB/s, 0.79 of the measured copy rate), with the norm's pass 435 us; decoding both moments 167 us
// (1.05 GB, 6.27 TB/s, 0.92).  In the update a block's loads wait on one another's arithmetic (45 % of the issue slots).
#include <cmath>

#include "internal.cuh"

namespace xt {
namespace {

constexpr int kBlock = 256;          // elements per scale
constexpr int kTile = 4096;          // elements per CTA and turn: 16 blocks, two per warp
constexpr int kThreads = 256;
constexpr int kMaxTensors = 128;     // tensors per launch (the table travels in the kernel parameters)
constexpr int kNormThreads = 512;
constexpr int kNormTile = 8192;      // elements per CTA and turn of the norm's pass
constexpr int kMaxCtas = 456;        // CTAs of a norm launch, three per SM: partial sums per launch

struct Table {
  float* p[kMaxTensors];
  const float* g[kMaxTensors];
  int8_t* m[kMaxTensors];
  uint8_t* r[kMaxTensors];
  float* ms[kMaxTensors];
  float* rs[kMaxTensors];
  void* sh[kMaxTensors];
  int64_t n[kMaxTensors];
  int tile0[kMaxTensors + 1];  // first tile of each tensor; tile0[count] = the group's tiles
  int count;
};

// The table in shared memory.  Reads of the parameters at an index of its own wait for one another, several before
// every tile's data where tensors are small (104.7 M weights in 74 tensors: step with norm 522 us with a search there,
// 492 with the walk below, 435 with both).
template <int THREADS>
__device__ __forceinline__ void table_in(Table& to, const Table& from) {
  constexpr int kWords = sizeof(Table) / 8;
  static_assert(sizeof(Table) % 8 == 0, "words");
#pragma unroll
  for (int u = 0; u < (kWords + THREADS - 1) / THREADS; ++u) {
    const int i = u * THREADS + threadIdx.x;
    if (i < kWords) reinterpret_cast<uint64_t*>(&to)[i] = reinterpret_cast<const uint64_t*>(&from)[i];
  }
  __syncthreads();
}
// The tensor of tile t, from that of an earlier tile: a block's tiles only go forward.
template <typename TB>
__device__ __forceinline__ int tensor_of(const TB& tb, int t, int k) {
  while (tb.tile0[k + 1] <= t) ++k;
  return k;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (hi, lo) += x² without loss: the product's rounding error by a fused multiply-add, the sum's by
// Knuth's two-sum.
__device__ __forceinline__ void add_square(float& hi, float& lo, float x) {
  const float p = x * x, e = fmaf(x, x, -p);
  const float s = __fadd_rn(hi, p), z = __fadd_rn(s, -hi);
  lo += __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -z)), __fadd_rn(p, -z)) + e;
  hi = s;
}

// Partial sums of g² of one group: one per CTA (the grid is fixed by the tile count and the device,
// so the order of the sums is too).
__global__ void __launch_bounds__(kNormThreads, 3) sq8_kernel(const __grid_constant__ Table table,
                                                             double* __restrict__ part) {
  __shared__ Table tb;
  table_in<kNormThreads>(tb, table);
  pdl_begin();
  __shared__ double sh[kNormThreads / 32];
  const int tiles = tb.tile0[tb.count];
  double acc = 0.0;
  float hi = 0.f, lo = 0.f;
  int first = 0, end = 0;  // tiles of the tensor at hand; its entry is read when it changes
  int64_t n = 0;
  const float* g0 = nullptr;
  for (int t = blockIdx.x, k = 0; t < tiles; t += gridDim.x) {
    if (t >= end) {
      k = tensor_of(tb, t, k);
      first = tb.tile0[k];
      end = tb.tile0[k + 1];
      n = tb.n[k];
      g0 = tb.g[k];
    }
    const int64_t base = int64_t(t - first) * kNormTile;
    const int64_t len = n - base < kNormTile ? n - base : kNormTile;
    const float* g = g0 + base;
    float x[16];
    if (len == kNormTile && (reinterpret_cast<uintptr_t>(g) & 15u) == 0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 q = reinterpret_cast<const float4*>(g)[u * kNormThreads + threadIdx.x];
        x[4 * u] = q.x; x[4 * u + 1] = q.y; x[4 * u + 2] = q.z; x[4 * u + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int i = u * kNormThreads + threadIdx.x;
        x[u] = i < len ? g[i] : 0.f;
      }
    }
    float top = 0.f, h1 = 0.f, l1 = 0.f;
#pragma unroll
    for (int u = 0; u < 16; ++u) top = fmaxf(top, fabsf(x[u]));
#pragma unroll
    for (int u = 0; u < 16; ++u) add_square(h1, l1, x[u]);
    // squares that leave float32's normal range are summed in float64 (NaN also lands here and stays)
    if (h1 == h1 && (top == 0.f || (top > 1e-13f && top < 1e17f))) {
      const float s = __fadd_rn(hi, h1), z = __fadd_rn(s, -hi);
      lo += __fadd_rn(__fadd_rn(hi, -__fadd_rn(s, -z)), __fadd_rn(h1, -z)) + l1;
      hi = s;
    } else {
      for (int u = 0; u < 16; ++u) acc = fma(double(x[u]), double(x[u]), acc);
    }
  }
  const double s = warp_sum_f64(acc + (double(hi) + double(lo)));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double r = 0.0;
    for (int w = 0; w < kNormThreads / 32; ++w) r += sh[w];
    part[blockIdx.x] = r;
  }
}

struct Hyper {
  float beta1, beta2, omb1, omb2;  // omb = 1 − β
  float decay;                     // 1 − lr·λ
  float step, root_bc2, eps;       // lr/bc₁, √(1/bc₂), ε
  float scale, max_norm;
  const double* part;              // the norm's partial sums
  int parts, norm;                 // their number (0 where all tensors are empty); whether the norm is wanted
  float* norm_out;
};

__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// √x of x ≥ 0 by the approximate reciprocal root (2⁻²² relative; values under 1e-36 come out too small, by 1e-18 at most, and
// 0 stays 0)
__device__ __forceinline__ float sqrt_fast(float x) { return x * rsqrt_fast(fmaxf(x, 1e-36f)); }
// The larger magnitude; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// Adding 1.5·2²³ to |x| < 2²² leaves rint(x), to even on ties, in the low bits (two's complement), without the
// conversion unit; a byte put under 2²³'s exponent is that number plus 2²³.
constexpr float kRound = 12582912.f;
constexpr float kByte = 8388608.f;
// Distance from half way between two codes within which the fast √(x/d) may round to the other one: its relative
// error is below 2⁻²¹ (quotient 2⁻²²·⁴, root 2⁻²², and for √v' its own root, halved), 1.2e-4 at 255.
constexpr float kBorder = 1.5e-4f;
__device__ __forceinline__ float code_exact(float x, float d) { return rintf(__fsqrt_rn(__fdiv_rn(x, d))); }

template <typename TS>
struct Four;  // four working-copy values in one store
template <> struct Four<float> {
  __device__ __forceinline__ static void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Four<bf16> {
  __device__ __forceinline__ static void store(bf16* p, const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// One block of up to 256 elements by one warp; lane l holds elements 128k + 4l + e.  EXACT: the update's root and quotient are
// the exactly rounded ones (exact_update says when).
template <typename TS, bool EXACT, bool VEC>
__device__ __forceinline__ void step_block(float* p, const float* g, int8_t* mc, uint8_t* rc, float* ms_p, float* rs_p,
                                           TS* sh, int len, int lane, float f, const Hyper& h) {
  float P[8], G[8];
  uint32_t M[2] = {0u, 0u}, R[2] = {0u, 0u};
  const float ms0 = *ms_p, rs0 = *rs_p;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 128 * k + 4 * lane;
    if (VEC) {
      const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(g + i);
      P[4 * k] = a.x; P[4 * k + 1] = a.y; P[4 * k + 2] = a.z; P[4 * k + 3] = a.w;
      G[4 * k] = b.x; G[4 * k + 1] = b.y; G[4 * k + 2] = b.z; G[4 * k + 3] = b.w;
      M[k] = *reinterpret_cast<const uint32_t*>(mc + i);
      R[k] = *reinterpret_cast<const uint32_t*>(rc + i);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = i + e < len;
        P[4 * k + e] = in ? p[i + e] : 0.f;
        G[4 * k + e] = in ? g[i + e] : 0.f;
        M[k] |= (in ? uint32_t(uint8_t(mc[i + e])) : 0u) << (8 * e);
        R[k] |= (in ? uint32_t(rc[i + e]) : 0u) << (8 * e);
      }
    }
  }
  float m[8], v[8];
  float mtop = 0.f, vtop = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = __uint_as_float(__byte_perm(M[j >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (j & 3))) - (kByte + 128.f);
    const float q = __uint_as_float(__byte_perm(R[j >> 2], 0x4B000000u, 0x7440 + (j & 3))) - kByte;
    const float gg = __fmul_rn(G[j], f);
    const float r0 = __fmul_rn(q * q, rs0);
    m[j] = __fadd_rn(__fmul_rn(__fmul_rn(c * fabsf(c), ms0), h.beta1), __fmul_rn(gg, h.omb1));
    v[j] = __fadd_rn(__fmul_rn(__fmul_rn(r0, r0), h.beta2), __fmul_rn(__fmul_rn(gg, h.omb2), gg));
    mtop = max_nan(mtop, fabsf(m[j]));
    vtop = max_nan(vtop, v[j]);
  }
  // magnitudes compared as bits: a NaN is the largest
  const float mmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop)));
  const float vmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop)));
  const float ms = __fdiv_rn(mmax, 16129.f), rs = __fdiv_rn(__fsqrt_rn(vmax), 65025.f);
  // a scale that is zero, infinite or NaN leaves codes of 0 (0·∞ and NaN then read back as NaN)
  const bool mok = ms > 0.f && ms < INFINITY, rok = rs > 0.f && rs < INFINITY;
  // below these the flush-to-zero approximations would lose values that still have a code
  const bool tiny = ms < 1e-33f || vmax < 1e-26f;
  const float mi = rcp_fast(ms), ri = rcp_fast(rs);
  uint32_t tm[8], tr[8], close = tiny ? 0xffu : 0u;  // rounded sums; elements to be done over
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float r = sqrt_fast(v[j]);
    const float xm = sqrt_fast(fabsf(m[j]) * mi), xr = sqrt_fast(r * ri);
    const float sm = copysignf(xm, m[j]) + kRound;
    float sr = xr + kRound;
    if (fabsf(xm - fabsf(sm - kRound)) > 0.5f - kBorder || fabsf(xr - (sr - kRound)) > 0.5f - kBorder) close |= 1u << j;
    if (v[j] > 0.f) sr = fmaxf(sr, kRound + 1.f);
    tm[j] = __float_as_uint(sm);
    tr[j] = __float_as_uint(sr);
    if (!EXACT) P[j] = fmaf(-h.step, m[j] * rcp_fast(fmaf(r, h.root_bc2, h.eps)), P[j] * h.decay);
  }
  if (EXACT) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      P[j] = fmaf(-h.step, __fdiv_rn(m[j], fmaf(__fsqrt_rn(v[j]), h.root_bc2, h.eps)), P[j] * h.decay);
  }
  if (close) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (close & (1u << j)) {
        const float cm = code_exact(fabsf(m[j]), ms), cr = code_exact(__fsqrt_rn(v[j]), rs);
        tm[j] = __float_as_uint(copysignf(cm, m[j]) + kRound);
        tr[j] = __float_as_uint((v[j] > 0.f ? fmaxf(cr, 1.f) : cr) + kRound);
      }
  }
  uint32_t mo[2], ro[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    mo[k] = __byte_perm(__byte_perm(tm[4 * k], tm[4 * k + 1], 0x0040), __byte_perm(tm[4 * k + 2], tm[4 * k + 3], 0x0040),
                        0x5410);
    ro[k] = __byte_perm(__byte_perm(tr[4 * k], tr[4 * k + 1], 0x0040), __byte_perm(tr[4 * k + 2], tr[4 * k + 3], 0x0040),
                        0x5410);
    if (!mok) mo[k] = 0u;
    if (!rok) ro[k] = 0u;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 128 * k + 4 * lane;
    if (VEC) {
      *reinterpret_cast<float4*>(p + i) = make_float4(P[4 * k], P[4 * k + 1], P[4 * k + 2], P[4 * k + 3]);
      *reinterpret_cast<uint32_t*>(mc + i) = mo[k];
      *reinterpret_cast<uint32_t*>(rc + i) = ro[k];
      if (sh) Four<TS>::store(sh + i, P + 4 * k);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e >= len) break;
        p[i + e] = P[4 * k + e];
        mc[i + e] = int8_t(mo[k] >> (8 * e));
        rc[i + e] = uint8_t(ro[k] >> (8 * e));
        if (sh) sh[i + e] = from_f<TS>(P[4 * k + e]);
      }
    }
  }
  if (lane == 0) {
    *ms_p = ms;
    *rs_p = rs;
  }
}

template <typename TS, bool EXACT>
__global__ void __launch_bounds__(kThreads, 3) adamw8_kernel(const __grid_constant__ Table table, const Hyper h) {
  __shared__ Table tb;
  table_in<kThreads>(tb, table);
  pdl_begin();
  __shared__ float sh_f;
  float f = h.scale;
  if (h.norm) {  // every CTA adds the same partial sums in the same order
    if (threadIdx.x < 32) {
      double acc = 0.0;
      for (int i = threadIdx.x; i < h.parts; i += 32) acc += h.part[i];
      acc = warp_sum_f64(acc);
      if (threadIdx.x == 0) {
        const double norm = fabs(double(h.scale)) * sqrt(acc);
        double c = 1.0;
        if (h.max_norm > 0.f) {
          c = double(h.max_norm) / (norm + 1e-6);
          c = c > 1.0 ? 1.0 : c;  // a NaN norm stays
        }
        sh_f = float(double(h.scale) * c);
        if (h.norm_out && blockIdx.x == 0) *h.norm_out = float(norm);
      }
    }
    __syncthreads();
    f = sh_f;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = tb.tile0[tb.count];
  for (int t = blockIdx.x, k = 0; t < tiles; t += gridDim.x) {
    k = tensor_of(tb, t, k);
    const int64_t tile = int64_t(t - tb.tile0[k]) * kTile;
    float* p = tb.p[k];
    const float* g = tb.g[k];
    int8_t* m = tb.m[k];
    uint8_t* r = tb.r[k];
    TS* w = static_cast<TS*>(tb.sh[k]);
    const bool aligned = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(g)) & 15u) == 0 &&
                         ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(r)) & 3u) == 0 &&
                         (reinterpret_cast<uintptr_t>(w) & (4 * sizeof(TS) - 1)) == 0;
#pragma unroll
    for (int u = 0; u < kTile / kBlock / (kThreads / 32); ++u) {
      const int64_t b = tile + int64_t(u * (kThreads / 32) + warp) * kBlock;
      const int64_t left = tb.n[k] - b;
      if (left <= 0) continue;
      TS* wb = w ? w + b : nullptr;
      float *ms = tb.ms[k] + b / kBlock, *rs = tb.rs[k] + b / kBlock;
      if (aligned && left >= kBlock)
        step_block<TS, EXACT, true>(p + b, g + b, m + b, r + b, ms, rs, wb, kBlock, lane, f, h);
      else
        step_block<TS, EXACT, false>(p + b, g + b, m + b, r + b, ms, rs, wb, int(left < kBlock ? left : kBlock), lane, f, h);
    }
  }
}

struct DecodeTable {
  const int8_t* m[kMaxTensors];
  const uint8_t* r[kMaxTensors];
  const float* ms[kMaxTensors];
  const float* rs[kMaxTensors];
  float* mo[kMaxTensors];
  float* vo[kMaxTensors];
  int64_t n[kMaxTensors];
  int tile0[kMaxTensors + 1];
  int count;
};

__global__ void __launch_bounds__(kThreads) decode8_kernel(const __grid_constant__ DecodeTable tb) {
  pdl_begin();
  const int tiles = tb.tile0[tb.count];
  for (int t = blockIdx.x, k = 0; t < tiles; t += gridDim.x) {
    k = tensor_of(tb, t, k);
    const int64_t base = int64_t(t - tb.tile0[k]) * kTile;
    const int8_t* m = tb.m[k] + base;
    const uint8_t* r = tb.r[k] + base;
    const float *ms = tb.ms[k] + base / kBlock, *rs = tb.rs[k] + base / kBlock;
    float* mo = tb.mo[k] ? tb.mo[k] + base : nullptr;
    float* vo = tb.vo[k] ? tb.vo[k] + base : nullptr;
    const int64_t left = tb.n[k] - base;
    const bool vec = left >= kTile &&
                     ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(r)) & 3u) == 0 &&
                     ((reinterpret_cast<uintptr_t>(mo) | reinterpret_cast<uintptr_t>(vo)) & 15u) == 0;
#pragma unroll
    for (int u = 0; u < kTile / (4 * kThreads); ++u) {
      const int i = (u * kThreads + int(threadIdx.x)) * 4;
      float a[4], b[4];
      if (i >= left) continue;
      const float s1 = ms[i / kBlock], s2 = rs[i / kBlock];
      if (vec) {
        const uint32_t cw = *reinterpret_cast<const uint32_t*>(m + i) ^ 0x80808080u;
        const uint32_t qw = *reinterpret_cast<const uint32_t*>(r + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = __uint_as_float(__byte_perm(cw, 0x4B000000u, 0x7440 + e)) - (kByte + 128.f);
          const float q = __uint_as_float(__byte_perm(qw, 0x4B000000u, 0x7440 + e)) - kByte;
          a[e] = c * fabsf(c) * s1;
          const float x = q * q * s2;
          b[e] = x * x;
        }
        if (mo) *reinterpret_cast<float4*>(mo + i) = make_float4(a[0], a[1], a[2], a[3]);
        if (vo) *reinterpret_cast<float4*>(vo + i) = make_float4(b[0], b[1], b[2], b[3]);
      } else {
        for (int e = 0; e < 4 && i + e < left; ++e) {
          const int c = m[i + e], q = r[i + e];
          const float x = float(q * q) * s2;
          if (mo) mo[i + e] = float(c * abs(c)) * s1;
          if (vo) vo[i + e] = x * x;
        }
      }
    }
  }
}

// The fast root is off by up to 1e-18 and the fast reciprocal takes a denominator outside 2⁻¹²⁶ .. 2¹²⁶ for 0 or ∞: beside an ε
// of 2²⁵·1e-18/√bc₂ or more the first is under 2⁻²⁵ of the denominator (ε = 1e-8 is, up to 1/√bc₂ = 297), and from an ε of 1e37
// on the second could show.  104.7 M weights, step with norm: 575 us so, 470 with the fast ones.
bool exact_update(float eps, float root_bc2) { return !(eps >= 3.4e-11f * root_bc2 && eps < 1e37f); }

int64_t tiles_of(int64_t n, int tile = kTile) { return ceil_div(n, tile); }

// Fills tile0, n and count of a table for up to kMaxTensors tensors from `first` on.
template <typename TB>
int plan(TB& tb, int n, const int64_t* numel, int first, int tile = kTile) {
  int tiles = 0;
  tb.count = 0;
  for (int i = first; i < n && tb.count < kMaxTensors; ++i) {
    tb.tile0[tb.count] = tiles;
    tb.n[tb.count] = numel[i];
    tiles += int(tiles_of(numel[i], tile));
    ++tb.count;
  }
  tb.tile0[tb.count] = tiles;
  return tiles;
}

int check_sizes(const char* fn, int n, const int64_t* numel) {
  XT_REQUIRE(n >= 0 && (n == 0 || numel), "%s: bad tensor list", fn);
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    XT_REQUIRE(numel[i] >= 0, "%s: negative size", fn);
    XT_REQUIRE(tiles_of(numel[i]) < (int64_t(1) << 30), "%s: tensor too large", fn);
    tiles += tiles_of(numel[i]);
    XT_REQUIRE(tiles < (int64_t(1) << 30), "%s: too many elements", fn);
  }
  return XT_OK;
}

int norm_grid(int tiles) {
  return tiles < kMaxCtas ? tiles : kMaxCtas;
}

}  // namespace
}  // namespace xt

using namespace xt;

extern "C" {

int xt_adamw8_scales(int64_t numel, int64_t* count) {
  XT_REQUIRE(numel >= 0 && count, "xt_adamw8_scales: bad arguments");
  *count = ceil_div(numel, kBlock);
  return XT_OK;
}

int xt_adamw8_workspace_size(int n, const int64_t* numel, size_t* bytes) {
  XT_REQUIRE(bytes, "xt_adamw8_workspace_size: bad arguments");
  XT_TRY(check_sizes("xt_adamw8_workspace_size", n, numel));
  size_t parts = 0;
  for (int first = 0; first < n; first += kMaxTensors) {
    int64_t tiles = 0;
    for (int i = first; i < n && i < first + kMaxTensors; ++i) tiles += tiles_of(numel[i], kNormTile);
    parts += size_t(tiles < kMaxCtas ? tiles : kMaxCtas);
  }
  *bytes = (parts * sizeof(double) + 255) & ~size_t(255);
  return XT_OK;
}

int xt_adamw8_step(const xt_adamw_config* cfg, int n, float* const* param, const float* const* grad,
                   int8_t* const* m_code, uint8_t* const* r_code, float* const* m_scale, float* const* r_scale,
                   void* const* shadow, int shadow_dtype, const int64_t* numel, float* norm_out, void* ws,
                   size_t ws_bytes, void* stream) {
  XT_REQUIRE(cfg != nullptr, "xt_adamw8_step: cfg is NULL");
  XT_TRY(check_sizes("xt_adamw8_step", n, numel));
  if (n == 0) return XT_OK;
  XT_REQUIRE(param && grad && m_code && r_code && m_scale && r_scale, "xt_adamw8_step: NULL table");
  XT_REQUIRE(cfg->step >= 1, "xt_adamw8_step: step must be >= 1");
  XT_REQUIRE(cfg->beta1 >= 0.f && cfg->beta1 < 1.f && cfg->beta2 >= 0.f && cfg->beta2 < 1.f,
             "xt_adamw8_step: betas must be in [0, 1)");
  XT_REQUIRE(cfg->eps > 0.f && cfg->lr >= 0.f && cfg->weight_decay >= 0.f, "xt_adamw8_step: bad hyperparameters");
  XT_REQUIRE(shadow == nullptr || valid_dtype(shadow_dtype), "xt_adamw8_step: bad shadow dtype");
  for (int i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    XT_REQUIRE(param[i] && grad[i] && m_code[i] && r_code[i] && m_scale[i] && r_scale[i],
               "xt_adamw8_step: NULL tensor %d", i);
  }
  const bool need_norm = cfg->max_grad_norm > 0.f || norm_out != nullptr;
  size_t need = 0;
  XT_TRY(xt_adamw8_workspace_size(n, numel, &need));
  if (need_norm) {
    XT_REQUIRE(need == 0 || (ws && ws_bytes >= need), "xt_adamw8_step: workspace too small (%zu < %zu)", ws_bytes,
               need);
    if ((reinterpret_cast<uintptr_t>(ws) & 7u) != 0)
      return fail(XT_ERR_ALIGNMENT, "xt_adamw8_step: the workspace must be 8-byte aligned");
  }
  cudaStream_t s = as_stream(stream);
  double* part = static_cast<double*>(ws);
  int parts = 0;
  if (need_norm)
    for (int first = 0; first < n; first += kMaxTensors) {
      Table tb{};
      const int tiles = plan(tb, n, numel, first, kNormTile);
      for (int j = 0; j < tb.count; ++j) tb.g[j] = grad[first + j];
      if (tiles == 0) continue;
      const int grid = norm_grid(tiles);
      launch(sq8_kernel, grid, kNormThreads, 0, s, tb, part + parts);
      XT_TRY(check_launch("xt_adamw8_step (norm)"));
      parts += grid;
    }
  Hyper h{};
  h.beta1 = cfg->beta1;
  h.beta2 = cfg->beta2;
  h.omb1 = 1.f - cfg->beta1;
  h.omb2 = 1.f - cfg->beta2;
  h.decay = float(1.0 - double(cfg->lr) * double(cfg->weight_decay));
  h.step = float(double(cfg->lr) / (1.0 - std::pow(double(cfg->beta1), double(cfg->step))));
  h.root_bc2 = float(std::sqrt(1.0 / (1.0 - std::pow(double(cfg->beta2), double(cfg->step)))));
  h.eps = cfg->eps;
  h.scale = cfg->grad_scale;
  h.max_norm = cfg->max_grad_norm;
  h.part = part;
  h.norm = need_norm;
  h.parts = parts;
  h.norm_out = norm_out;
  bool any = false;
  for (int first = 0; first < n; first += kMaxTensors) {
    Table tb{};
    const int tiles = plan(tb, n, numel, first);
    for (int j = 0; j < tb.count; ++j) {
      const int i = first + j;
      tb.p[j] = param[i];
      tb.g[j] = grad[i];
      tb.m[j] = m_code[i];
      tb.r[j] = r_code[i];
      tb.ms[j] = m_scale[i];
      tb.rs[j] = r_scale[i];
      tb.sh[j] = shadow ? shadow[i] : nullptr;
    }
    // a launch without tiles still reports the norm of tensors that are all empty
    if (tiles == 0 && (any || !norm_out || first + kMaxTensors < n)) continue;
    any = true;
    // the blocks that fit at once (three per SM), each walking its tiles: 104.7 M weights 353 us, 378 with a grid of
    // six per SM; asking L2 for the next tile ahead of time made it 428
    const int cap = num_sms() * 3;
    const int grid = tiles < 1 ? 1 : tiles < cap ? tiles : cap;
    const bool exact = exact_update(h.eps, h.root_bc2);
    if (shadow && shadow_dtype == XT_BF16)
      launch(exact ? adamw8_kernel<bf16, true> : adamw8_kernel<bf16, false>, grid, kThreads, 0, s, tb, h);
    else
      launch(exact ? adamw8_kernel<float, true> : adamw8_kernel<float, false>, grid, kThreads, 0, s, tb, h);
    XT_TRY(check_launch("xt_adamw8_step (update)"));
  }
  return XT_OK;
}

int xt_adamw8_decode(int n, const int8_t* const* m_code, const uint8_t* const* r_code, const float* const* m_scale,
                     const float* const* r_scale, float* const* m, float* const* v, const int64_t* numel,
                     void* stream) {
  XT_TRY(check_sizes("xt_adamw8_decode", n, numel));
  if (n == 0) return XT_OK;
  XT_REQUIRE(m_code && r_code && m_scale && r_scale && (m || v), "xt_adamw8_decode: NULL table");
  for (int i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    XT_REQUIRE(m_code[i] && r_code[i] && m_scale[i] && r_scale[i], "xt_adamw8_decode: NULL tensor %d", i);
  }
  cudaStream_t s = as_stream(stream);
  for (int first = 0; first < n; first += kMaxTensors) {
    DecodeTable tb{};
    const int tiles = plan(tb, n, numel, first);
    for (int j = 0; j < tb.count; ++j) {
      const int i = first + j;
      tb.m[j] = m_code[i];
      tb.r[j] = r_code[i];
      tb.ms[j] = m_scale[i];
      tb.rs[j] = r_scale[i];
      tb.mo[j] = m ? m[i] : nullptr;
      tb.vo[j] = v ? v[i] : nullptr;
    }
    if (tiles == 0) continue;
    // 104.7 M weights: 167 us with 64 blocks per SM (several waves even out what each of them waits for memory), 182
    // with eight
    const int cap = num_sms() * 64;
    launch(decode8_kernel, tiles < cap ? tiles : cap, kThreads, 0, s, tb);
    XT_TRY(check_launch("xt_adamw8_decode"));
  }
  return XT_OK;
}

}  // extern "C"
