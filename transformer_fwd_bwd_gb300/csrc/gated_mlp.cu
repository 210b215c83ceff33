// The gated feed-forward block: h = act(x Wg)∘(x Wu), y = h Wd, and its backward:
//   dh = dy Wdᵀ,  dg = dh∘u∘act'(g),  du = dh∘act(g),  dx = dg Wgᵀ + du Wuᵀ,  dWg = xᵀ dg,  dWu = xᵀ du,  dWd = hᵀ dy.
// The first product of each direction carries the activation in its epilogue (gemm_kernel.cuh): the forward's one kernel
// runs both projections, the activation and the product, the backward's forms dg and du where dh is still in tensor
// memory.  [dg | du] stands as Wg and Wu stand beside each other, so dx is one product over 2F and dW_up another.
//
// Roundings.  The products' operands are bf16, so h, dg and du are rounded once where they are formed (from float32 sums), and
// g and u are kept for the backward as bf16, half of the bytes that its epilogue waits for: act' is taken at the rounded g.
// y is then within 2.4e-3 of the formulas in norm (1.7e-3 with one rounding at the end), dx and dW_up within 3.0e-3.
//
// Bound by the tensor cores: 6·T·d·F operations forward, 12·T·d·F backward.  On one GB300, T x d x F = 8192 x 768 x 2048 silu (us):
// projections with activation 42 (1230 TFLOP/s), down 28, dh with its epilogue 51 (504: reads of g and u compete with the
// operands'), dx 41, dW 44 and 27; 12001 x 2048 x 5464 gelu: 359 (1500 TFLOP/s), 172, 303 (886), 325, 309 and 194.
#include "gemm.cuh"
#include "internal.cuh"

using namespace xt;

namespace {

xt_matmul_desc product(int64_t M, int64_t N, int64_t K, int trans_a, int trans_b, int64_t lda, int64_t ldb, int64_t ldc,
                       int dt_c, int acc) {
  xt_matmul_desc m{};
  m.M = int32_t(M);
  m.N = int32_t(N);
  m.K = int32_t(K);
  m.trans_a = trans_a;
  m.trans_b = trans_b;
  m.batch_outer = m.batch_inner = 1;
  m.dtype_ab = XT_BF16;
  m.dtype_c = dt_c;
  m.accumulate = acc;
  m.alpha = 1.f;
  m.lda = lda;
  m.ldb = ldb;
  m.ldc = ldc;
  return m;
}
// y = h Wd;  dx = dgu W_upᵀ;  dW_up = xᵀ dgu;  dW_down = hᵀ dy
xt_matmul_desc down(int64_t T, int64_t d, int64_t F) { return product(T, d, F, 0, 0, F, d, d, XT_BF16, 0); }
xt_matmul_desc grad_x(int64_t T, int64_t d, int64_t F, int acc) {
  return product(T, d, 2 * F, 0, 1, 2 * F, 2 * F, d, XT_BF16, acc);
}
xt_matmul_desc grad_up(int64_t T, int64_t d, int64_t F, int dt, int acc) {
  return product(d, 2 * F, T, 1, 0, d, 2 * F, 2 * F, dt, acc);
}
xt_matmul_desc grad_down(int64_t T, int64_t d, int64_t F, int dt, int acc) {
  return product(F, d, T, 1, 0, F, d, d, dt, acc);
}

int check_sizes(const char* fn, int64_t T, int64_t d, int64_t F, int act) {
  XT_REQUIRE(T >= 0 && d > 0 && F > 0, "%s: sizes must be positive", fn);
  XT_REQUIRE(T < (int64_t(1) << 30) && d < (int64_t(1) << 24) && F < (int64_t(1) << 24), "%s: sizes are too large", fn);
  XT_REQUIRE(act == XT_GATE_SILU || act == XT_GATE_GELU, "%s: bad activation", fn);
  if (d % 8 || F % 8) return fail(XT_ERR_ALIGNMENT, "%s: d and F must be multiples of 8", fn);
  return XT_OK;
}
int check_ptr(const char* fn, const char* name, const void* p) {
  XT_REQUIRE(p != nullptr, "%s: %s is NULL", fn, name);
  if (!aligned16(p)) return fail(XT_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned", fn, name);
  return XT_OK;
}

}  // namespace

extern "C" {

int xt_gated_mlp_workspace_size(int64_t T, int64_t d, int64_t F, size_t* bytes) {
  const char* fn = "xt_gated_mlp_workspace_size";
  XT_REQUIRE(bytes != nullptr, "%s: NULL pointer", fn);
  XT_TRY(check_sizes(fn, T, d, F, XT_GATE_SILU));
  size_t most = gemm::kSkFlagBytes;
  for (const xt_matmul_desc& m : {down(T, d, F), grad_x(T, d, F, 0), grad_up(T, d, F, XT_F32, 0), grad_down(T, d, F, XT_F32, 0)}) {
    const size_t b = matmul_workspace(m);
    if (b > most) most = b;
  }
  *bytes = most;
  return XT_OK;
}

int xt_gated_mlp_fwd(const void* x, const void* w_up, const void* w_down, void* gu, void* h, void* y, int64_t T,
                     int64_t d, int64_t F, int act, int dt, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "xt_gated_mlp_fwd";
  XT_TRY(check_sizes(fn, T, d, F, act));
  if (dt != XT_BF16) return fail(XT_ERR_UNSUPPORTED, "%s: bf16 only", fn);
  if (T == 0) return XT_OK;
  XT_TRY(check_ptr(fn, "x", x));
  XT_TRY(check_ptr(fn, "w_up", w_up));
  XT_TRY(check_ptr(fn, "h", h));
  if (gu) XT_TRY(check_ptr(fn, "gu", gu));
  if (y) {
    XT_TRY(check_ptr(fn, "y", y));
    XT_TRY(check_ptr(fn, "w_down", w_down));
  }
  if (ws) XT_TRY(check_ptr(fn, "ws", ws));
  cudaStream_t s = as_stream(stream);
  gemm::Problem pb{};
  pb.M = T;
  pb.N = F;
  pb.K = d;
  pb.A = gemm::Operand{x, false, T, d, d, 0, 0, 1, 1};
  pb.B = gemm::Operand{w_up, true, 2 * F, d, 2 * F, 0, 0, 1, 1};
  pb.C = h;
  pb.C2 = gu;
  pb.act = act == XT_GATE_SILU ? gemm::kGateFwdSilu : gemm::kGateFwdGelu;
  XT_TRY(gemm::run_gated(pb, s));
  return y ? matmul(down(T, d, F), h, w_down, y, ws, ws_bytes, s) : XT_OK;
}

int xt_gated_mlp_bwd(const void* x, const void* w_up, const void* w_down, const void* gu, const void* h, const void* dy,
                     void* dgu, void* dx, void* dw_up, void* dw_down, int64_t T, int64_t d, int64_t F, int act, int dt,
                     int dt_grad, int acc_dx, int acc_dw, void* ws, size_t ws_bytes, void* stream) {
  const char* fn = "xt_gated_mlp_bwd";
  XT_TRY(check_sizes(fn, T, d, F, act));
  if (dt != XT_BF16) return fail(XT_ERR_UNSUPPORTED, "%s: bf16 only", fn);
  XT_REQUIRE(valid_dtype(dt_grad), "%s: bad gradient dtype", fn);
  XT_REQUIRE((acc_dx == 0 || acc_dx == 1) && (acc_dw == 0 || acc_dw == 1), "%s: accumulate flags must be 0 or 1", fn);
  if (ws) XT_TRY(check_ptr(fn, "ws", ws));
  if (dx) XT_TRY(check_ptr(fn, "dx", dx));
  if (dw_up) XT_TRY(check_ptr(fn, "dw_up", dw_up));
  if (dw_down) XT_TRY(check_ptr(fn, "dw_down", dw_down));
  cudaStream_t s = as_stream(stream);
  if (T > 0) {
    XT_TRY(check_ptr(fn, "dy", dy));
    if (dx || dw_up) {
      XT_TRY(check_ptr(fn, "w_down", w_down));
      XT_TRY(check_ptr(fn, "gu", gu));
      XT_TRY(check_ptr(fn, "dgu", dgu));
    }
    if (dx) XT_TRY(check_ptr(fn, "w_up", w_up));
    if (dw_up) XT_TRY(check_ptr(fn, "x", x));
    if (dw_down) XT_TRY(check_ptr(fn, "h", h));
  }
  if (T > 0 && (dx || dw_up)) {
    gemm::Problem pb{};
    pb.M = T;
    pb.N = F;
    pb.K = d;
    pb.A = gemm::Operand{dy, false, T, d, d, 0, 0, 1, 1};
    pb.B = gemm::Operand{w_down, false, F, d, d, 0, 0, 1, 1};
    pb.C2 = dgu;
    pb.aux = gu;
    pb.act = act == XT_GATE_SILU ? gemm::kGateBwdSilu : gemm::kGateBwdGelu;
    XT_TRY(gemm::run_gated(pb, s));
  }
  // no tokens: the weights' gradients are nought (products over nothing)
  if (dx) XT_TRY(matmul(grad_x(T, d, F, acc_dx), dgu, w_up, dx, ws, ws_bytes, s));
  if (dw_up) XT_TRY(matmul(grad_up(T, d, F, dt_grad, acc_dw), x, dgu, dw_up, ws, ws_bytes, s));
  if (dw_down) XT_TRY(matmul(grad_down(T, d, F, dt_grad, acc_dw), h, dy, dw_down, ws, ws_bytes, s));
  return XT_OK;
}

}  // extern "C"
