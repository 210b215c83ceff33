// Rotary positions with several axes (time, height, width, ...) given per token, forward and
// backward.  For a token t and the rotation pair (i, i + h), h = hd/2, of any head,
//   θ = pos[axis(i)][t] · f_i,
//   y_i = x_i cos θ − x_{i+h} sin θ,   y_{i+h} = x_{i+h} cos θ + x_i sin θ
// (the backward is the transposed rotation), with the pairs shared out among the axes in order by
// `sections` and f_i = base^(−2i/hd), or base^(−k/sections[a]) for pair k of axis a.
//
// Angles.  An angle matters modulo a turn only, and pos is an integer, so f_i/2π is held as a
// 64-bit fraction of a turn and pos·(f_i/2π) mod 1 is one 64-bit integer product, whose wrap-around
// is the reduction: no position is too far (a float32 product is off by 0.06 rad at position 10⁶).
// The nearest quarter turn comes off in integers too, and what is left, at most an eighth of a turn,
// goes through the Taylor series of sin and cos (next terms below 2⁻²⁵), some twenty instructions for
// the pair of them.
//
// Memory-bound: x is read once and y written once.  A thread keeps one token's VW pairs: it forms
// their cos and sin once and applies them to several heads, the loads of some heads in flight.
#include <cmath>

#include "internal.cuh"

namespace xt {
namespace {

constexpr int kMaxPairs = 128;  // hd ≤ 256
constexpr int kMaxAxes = 4;
constexpr int kThreads = 256;

// sin and cos of a turn's fraction u·2⁻³².
__device__ __forceinline__ void sincos_turn(uint32_t u, float& sn, float& cs) {
  const uint32_t q = (u + 0x20000000u) >> 30;                            // nearest quarter turn
  const float y = float(int32_t(u - (q << 30))) * 1.46291807926716e-9f;  // 2π·2⁻³²; |y| ≤ π/4
  const float z = y * y;
  const float s = fmaf(y * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), y);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float a = (q & 1) ? c : s, b = (q & 1) ? s : c;
  sn = __uint_as_float(__float_as_uint(a) ^ ((q & 2) << 30));
  cs = __uint_as_float(__float_as_uint(b) ^ (((q + 1) & 2) << 30));
}

struct RopeAxes {
  uint64_t turn[kMaxPairs];  // f_i / 2π mod 1, in units of 2⁻⁶⁴
  uint8_t axis[kMaxPairs];
  const int32_t* pos;        // [n_axes][T]
  int64_t T, ld_x, ld_y;
  int n_axes, H, half;
  int groups;                // a thread's heads are group, group + groups, ...
  int acc;
};

template <typename T, bool BWD, int VW>
__global__ void __launch_bounds__(kThreads, VW == 8 ? 6 : 3) rope_axes_kernel(const T* x, T* y, const __grid_constant__ RopeAxes a) {
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ uint8_t axis[kMaxPairs];
  for (int i = threadIdx.x; i < a.half; i += kThreads) {
    turn[i] = a.turn[i];
    axis[i] = a.axis[i];
  }
  __syncthreads();
  pdl_begin();
  // Heads whose loads are in flight, and blocks per SM: eight bf16 pairs fill a thread, so one head at a time and
  // many threads (50001 tokens x 40 heads of 128, forward and backward: 338 us, 6.06 TB/s; two heads and four blocks
  // 378, four heads at 112 registers 510); four float32 pairs leave room for four heads (8192 x 24 x 64: 37.6 us
  // against 39.2 with one).
  constexpr int kInFlight = VW == 8 ? 1 : 4;
  const int chunks = a.half / VW;
  const int64_t total = a.T * a.groups * chunks;
  for (int64_t v = int64_t(blockIdx.x) * kThreads + threadIdx.x; v < total; v += int64_t(gridDim.x) * kThreads) {
    const int64_t tg = v / chunks;
    const int i0 = int(v - tg * chunks) * VW;
    const int64_t t = tg / a.groups;
    const int g = int(tg - t * a.groups);
    uint32_t pos[kMaxAxes];
#pragma unroll
    for (int k = 0; k < kMaxAxes; ++k) pos[k] = k < a.n_axes ? uint32_t(__ldg(a.pos + k * a.T + t)) : 0u;
    float c[VW], s[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int ax = axis[i0 + e];
      const uint32_t p = ax == 0 ? pos[0] : ax == 1 ? pos[1] : ax == 2 ? pos[2] : pos[3];
      sincos_turn(uint32_t((uint64_t(int64_t(int32_t(p))) * turn[i0 + e]) >> 32), s[e], c[e]);
      if (BWD) s[e] = -s[e];
    }
    const T* xr = x + t * a.ld_x + i0;
    T* yr = y + t * a.ld_y + i0;
    const int64_t hd = 2 * int64_t(a.half);
    for (int h0 = g; h0 < a.H; h0 += kInFlight * a.groups) {
      float u[kInFlight][VW], w[kInFlight][VW];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int h = h0 + k * a.groups;
        if (h < a.H) {
          Acc<T, VW>::load(xr + h * hd, u[k]);
          Acc<T, VW>::load(xr + h * hd + a.half, w[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int h = h0 + k * a.groups;
        if (h >= a.H) continue;
        float o1[VW], o2[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          o1[e] = u[k][e] * c[e] - w[k][e] * s[e];
          o2[e] = w[k][e] * c[e] + u[k][e] * s[e];
        }
        if (BWD && a.acc) {
          float p1[VW], p2[VW];
          Acc<T, VW>::load(yr + h * hd, p1);
          Acc<T, VW>::load(yr + h * hd + a.half, p2);
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            o1[e] += p1[e];
            o2[e] += p2[e];
          }
        }
        Acc<T, VW>::store(yr + h * hd, o1);
        Acc<T, VW>::store(yr + h * hd + a.half, o2);
      }
    }
  }
}

int rope_axes_run(const char* fn, bool bwd, const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* pos,
                  int n_axes, const int32_t* sections, int per_axis, double base, int64_t T, int H, int hd, int dt,
                  int acc, void* stream) {
  XT_REQUIRE(valid_dtype(dt), "%s: bad dtype", fn);
  XT_REQUIRE(T >= 0 && T < (int64_t(1) << 31) && H > 0, "%s: bad sizes", fn);
  XT_REQUIRE(hd > 0 && hd % 2 == 0, "%s: hd must be even", fn);
  if (hd > 2 * kMaxPairs) return fail(XT_ERR_UNSUPPORTED, "%s: hd must be at most %d", fn, 2 * kMaxPairs);
  XT_REQUIRE(n_axes >= 1 && n_axes <= kMaxAxes && sections, "%s: 1 to %d axes with their sections", fn, kMaxAxes);
  XT_REQUIRE(std::isfinite(base) && base > 0, "%s: base must be positive", fn);
  XT_REQUIRE(per_axis == 0 || per_axis == 1, "%s: per_axis must be 0 or 1", fn);
  XT_REQUIRE(ld_x >= int64_t(H) * hd && ld_y >= int64_t(H) * hd, "%s: row stride smaller than H*hd", fn);
  RopeAxes a{};
  a.half = hd / 2;
  int64_t pairs = 0;
  for (int k = 0; k < n_axes; ++k) {
    XT_REQUIRE(sections[k] >= 0, "%s: negative section", fn);
    pairs += sections[k];
  }
  XT_REQUIRE(pairs == a.half, "%s: the sections add up to %lld pairs, not hd/2 = %d", fn, (long long)pairs, a.half);
  if (T == 0) return XT_OK;
  XT_REQUIRE(x && y && pos, "%s: NULL pointer", fn);
  XT_REQUIRE(x != y || ld_x == ld_y, "%s: in place needs one row stride", fn);
  for (int k = 0, i = 0; k < n_axes; ++k)
    for (int j = 0; j < sections[k]; ++j, ++i) {
      const double f = per_axis ? std::pow(base, -double(j) / sections[k]) : std::pow(base, -2.0 * i / hd);
      const double turns = f * 0.15915494309189533577;  // 1/2π
      XT_REQUIRE(std::isfinite(turns), "%s: base is out of range", fn);
      a.turn[i] = uint64_t(std::ldexp(turns - std::floor(turns), 64));
      a.axis[i] = uint8_t(k);
    }
  a.pos = pos;
  a.T = T;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.n_axes = n_axes;
  a.H = H;
  a.acc = acc;
  const int vw = dt == XT_BF16 ? 8 : 4;
  const size_t e = dtype_size(dt);
  const bool vec = a.half % vw == 0 && (ld_x * e) % 16 == 0 && (ld_y * e) % 16 == 0 && aligned16(x) && aligned16(y);
  const int64_t chunks = a.half / (vec ? vw : 1);
  // As many heads to a thread as leave 1024 threads per SM (cos and sin are formed once per thread), eight at
  // most; few tokens spread their heads over more threads.
  int per = 8;
  while (per > 1 && T * chunks * ceil_div(H, per) < int64_t(num_sms()) * 1024) per /= 2;
  a.groups = int(ceil_div(H, per));
  const int64_t total = T * chunks * a.groups;
  int64_t grid = ceil_div(total, kThreads);
  if (grid > int64_t(num_sms()) * 64) grid = int64_t(num_sms()) * 64;
  cudaStream_t s = as_stream(stream);
#define XT_ROPE_AXES(T_, VW_)                                                                                   \
  do {                                                                                                          \
    if (bwd)                                                                                                    \
      launch(rope_axes_kernel<T_, true, VW_>, unsigned(grid), kThreads, 0, s, static_cast<const T_*>(x),        \
             static_cast<T_*>(y), a);                                                                           \
    else                                                                                                        \
      launch(rope_axes_kernel<T_, false, VW_>, unsigned(grid), kThreads, 0, s, static_cast<const T_*>(x),       \
             static_cast<T_*>(y), a);                                                                           \
  } while (0)
  if (dt == XT_BF16) {
    if (vec) XT_ROPE_AXES(bf16, 8);
    else XT_ROPE_AXES(bf16, 1);
  } else {
    if (vec) XT_ROPE_AXES(float, 4);
    else XT_ROPE_AXES(float, 1);
  }
#undef XT_ROPE_AXES
  return check_launch(fn);
}

}  // namespace
}  // namespace xt

using namespace xt;

extern "C" {

int xt_rope_axes_fwd(const void* x, int64_t ld_x, void* y, int64_t ld_y, const int32_t* pos, int n_axes,
                     const int32_t* sections, int per_axis, double base, int64_t T, int H, int hd, int dt,
                     void* stream) {
  return rope_axes_run("xt_rope_axes_fwd", false, x, ld_x, y, ld_y, pos, n_axes, sections, per_axis, base, T, H, hd,
                       dt, 0, stream);
}

int xt_rope_axes_bwd(const void* d, int64_t ld_d, void* dx, int64_t ld_dx, const int32_t* pos, int n_axes,
                     const int32_t* sections, int per_axis, double base, int64_t T, int H, int hd, int dt, int acc,
                     void* stream) {
  XT_REQUIRE(acc == 0 || acc == 1, "xt_rope_axes_bwd: acc must be 0 or 1");
  XT_REQUIRE(!(acc && d == dx), "xt_rope_axes_bwd: accumulate cannot be in place");
  return rope_axes_run("xt_rope_axes_bwd", true, d, ld_d, dx, ld_dx, pos, n_axes, sections, per_axis, base, T, H, hd,
                       dt, acc, stream);
}

}  // extern "C"
