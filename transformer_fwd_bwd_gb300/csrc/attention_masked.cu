// Entry points of masked attention: argument checks, tensor maps, launches (the kernels: attention_masked.cuh).
#include <cstring>

#include "attention_masked.cuh"

namespace xt {
namespace attnm {

int prepare_kernel(std::atomic<uint64_t>& ready, const void* kernel, int smem, int regs) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(XT_ERR_CUDA, "masked attention: no current device");
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return XT_OK;
  cudaFuncAttributes fa{};
  cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return fail(XT_ERR_CUDA, "masked attention: kernel attributes: %s", cudaGetErrorString(e));
  if (regs && fa.numRegs != regs)
    return fail(XT_ERR_UNSUPPORTED, "masked attention: kernel built with %d registers, not %d", fa.numRegs, regs);
  ready.fetch_or(bit, std::memory_order_release);
  return XT_OK;
}

namespace {

// dK and dV of a split key pass: the splits' sums added in order, scaled and rounded.
__global__ void __launch_bounds__(256) attnm_join_kernel(const __grid_constant__ attnm::Params p, int width) {
  pdl_begin();
  if (!attn_plan::valid(p.plan)) return;  // the passes have refused the plan: there are no sums
  const int64_t n = p.plan.T * width, per = n / 4;
  for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < 2 * per; v += int64_t(gridDim.x) * 256) {
    const bool is_v = v >= per;
    const int64_t e = (is_v ? v - per : v) * 4, t = e / width;
    const float* src = (is_v ? p.part_v : p.part_k) + e;
    float4 a = *reinterpret_cast<const float4*>(src);
    for (int s = 1; s < p.split; ++s) {
      const float4 b = *reinterpret_cast<const float4*>(src + s * n);
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
    }
    const float mul = is_v ? 1.f : p.scale;
    bf16* out = (is_v ? p.dv + t * p.lddv : p.dk + t * p.lddk) + (e - t * width);
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(a.x * mul, a.y * mul), pack_bf16(a.z * mul, a.w * mul));
  }
}

// [planes, T, heads, hd] view of bf16 or (f32) float32 with rows of ld elements.  To be read: boxes of 128 tokens × 64
// elements of one head, 128-byte swizzle; to be written (out): 32 tokens × 64 bytes, 64-byte swizzle.
int token_map(CUtensorMap* tm, const void* base, int64_t ld, int64_t T, int heads, int hd, bool out = false,
              bool f32 = false, int planes = 1) {
  auto enc = encode_fn();
  if (!enc) return fail(XT_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int64_t e = f32 ? 4 : 2;
  cuuint64_t dims[4] = {cuuint64_t(hd), cuuint64_t(heads), cuuint64_t(T), cuuint64_t(planes)};
  cuuint64_t strides[3] = {cuuint64_t(hd * e), cuuint64_t(ld * e), cuuint64_t(T * ld * e)};
  cuuint32_t box[4] = {out ? cuuint32_t(64 / e) : 64u, 1, out ? 32u : cuuint32_t(BT), 1}, estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         out ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(XT_ERR_CUDA, "masked attention: cuTensorMapEncodeTiled failed (%d)", int(r));
  return XT_OK;
}

struct Strided {
  const void* p;
  int64_t ld;
  int heads;
};

// The part of the kernels' parameters that the desc gives.
attnm::Params params_of(const xt_attention_desc* d) {
  Params p{};
  p.H = d->H;
  p.Hkv = d->Hkv;
  p.group = d->H / d->Hkv;
  const double scale = d->scale > 0.f ? double(d->scale) : 1.0 / std::sqrt(double(d->hd)), log2e = 1.4426950408889634;
  p.scale = float(scale);
  p.sc = float(scale * log2e);
  if (d->cap > 0.f) {
    p.capy = float(scale / double(d->cap));
    p.capk = float(2.0 * log2e * scale / double(d->cap));
    constexpr float kTanh[7] = {0.9999997019767761f,  -0.33332130312919617f,  0.13319583237171173f, -0.05326583608984947f,
                                0.019973281770944595f, -0.005951280705630779f, 0.0009637721814215183f};
    for (int k = 0; k < 7; ++k) {
      uint32_t w;
      std::memcpy(&w, &kTanh[k], 4);
      p.tanh_c[k] = uint64_t(w) << 32 | w;
    }
    p.cap2 = float(double(d->cap) * log2e);
  }
  p.slopes = d->slopes;
  return p;
}

int check(const char* fn, const xt_attention_desc* d, const void* plan, size_t plan_bytes, const void* lse,
          std::initializer_list<Strided> xs) {
  XT_REQUIRE(d != nullptr, "%s: desc is NULL", fn);
  XT_REQUIRE(d->T >= 0 && d->T < (int64_t(1) << 30), "%s: T must be in [0, 2^30)", fn);
  XT_REQUIRE(d->H > 0 && d->Hkv > 0 && d->H % d->Hkv == 0, "%s: H must be a positive multiple of Hkv", fn);
  if (d->dtype != XT_BF16) return fail(XT_ERR_UNSUPPORTED, "%s: only bf16 is supported", fn);
  if (d->hd != 64 && d->hd != 128) return fail(XT_ERR_UNSUPPORTED, "%s: head_dim must be 64 or 128", fn);
  XT_REQUIRE(std::isfinite(d->scale) && d->scale >= 0.f, "%s: scale must be finite and not negative", fn);
  // the capped scores' exponential form is off by 2⁻²³ of the cap, 1.2e-4 at the largest one taken; the scores'
  // multiplier of a tiny cap must stay finite
  XT_REQUIRE(d->cap >= 0.f && d->cap <= 1024.f, "%s: cap must be in [0, 1024]", fn);
  XT_REQUIRE(d->cap == 0.f || std::isfinite(params_of(d).capk), "%s: cap too small for this scale", fn);
  const attn_plan::Layout l(d->T);
  if (l.tiles * d->H >= (int64_t(1) << 30)) return fail(XT_ERR_UNSUPPORTED, "%s: too many tokens times heads", fn);
  if (d->T == 0) return XT_OK;
  XT_REQUIRE(plan && lse, "%s: NULL pointer", fn);
  if (!aligned16(plan)) return fail(XT_ERR_ALIGNMENT, "%s: the plan must be 16-byte aligned", fn);
  XT_REQUIRE(plan_bytes >= size_t(l.total) * 4, "%s: plan too small (%zu < %zu)", fn, plan_bytes, size_t(l.total) * 4);
  for (const Strided& x : xs) {
    XT_REQUIRE(x.p, "%s: NULL pointer", fn);
    XT_REQUIRE(x.ld >= int64_t(x.heads) * d->hd, "%s: row stride smaller than the heads' columns", fn);
    if (x.ld % 8) return fail(XT_ERR_ALIGNMENT, "%s: row strides must be multiples of 8", fn);
    if (!aligned16(x.p)) return fail(XT_ERR_ALIGNMENT, "%s: pointers must be 16-byte aligned", fn);
  }
  return XT_OK;
}

attnm::Params params(const xt_attention_desc* d, const void* plan) {
  Params p = params_of(d);
  p.plan = attn_plan::view(plan, d->T);
  p.flag = errflag();
  p.wait_ns = wait_limit_ns();
  return p;
}

// Items of the key pass per key tile and head: shared key heads leave few of them, each over the whole group
// of query heads.  Where they are fewer than four per SM of a GB300 the group is cut into up to its heads, the
// parts' float32 sums being joined by a second kernel (4 x 1023 tokens, 16 query and 4 key heads of 128:
// backward 91 us, 103 without the cut, both with one bf16 of dS everywhere).  A constant SM count keeps the workspace's
// size a function of the problem alone.
int key_split(const xt_attention_desc* d) {
  constexpr int64_t kWanted = 4 * 152;
  const int64_t items = attn_plan::Layout(d->T).tiles * d->Hkv;
  const int group = d->H / d->Hkv;
  int split = 1;
  while (split < group && items * split < kWanted) split = split * 2 < group ? split * 2 : group;
  const int share = (group + split - 1) / split;
  return (group + share - 1) / share;
}
size_t d_bytes(const xt_attention_desc* d) {  // nl and nd, rows of whole tiles
  return 2 * size_t(attn_plan::Layout(d->T).tiles) * BT * size_t(d->H) * 4;
}
size_t part_bytes(const xt_attention_desc* d, int split) {
  return (size_t(split) * size_t(d->T) * size_t(d->Hkv) * size_t(d->hd) * 4 + 255) & ~size_t(255);
}

}  // namespace
}  // namespace attnm
}  // namespace xt

using namespace xt;
using namespace xt::attnm;

extern "C" {

int xt_attention_masked_fwd(const xt_attention_desc* desc, const void* plan, size_t plan_bytes, const void* q,
                            int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, void* o,
                            int64_t ld_o, float* lse, void* stream) {
  const char* fn = "xt_attention_masked_fwd";
  const int H = desc ? desc->H : 0, Hkv = desc ? desc->Hkv : 0;
  XT_TRY(check(fn, desc, plan, plan_bytes, lse, {{q, ld_q, H}, {k, ld_k, Hkv}, {v, ld_v, Hkv}, {o, ld_o, H}}));
  if (desc->T == 0) return XT_OK;
  attnm::Params p = attnm::params(desc, plan);
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.ldq = ld_q;
  p.ldk = ld_k;
  p.ldv = ld_v;
  p.o = static_cast<bf16*>(o);
  p.ldo = ld_o;
  p.lse = lse;
  CUtensorMap tm[4];
  XT_TRY(token_map(&tm[0], q, ld_q, desc->T, H, desc->hd));
  XT_TRY(token_map(&tm[1], k, ld_k, desc->T, Hkv, desc->hd));
  XT_TRY(token_map(&tm[2], v, ld_v, desc->T, Hkv, desc->hd));
  XT_TRY(token_map(&tm[3], o, ld_o, desc->T, H, desc->hd, true));
  const bool cap = desc->cap > 0.f, bias = desc->slopes != nullptr;
  return desc->hd == 64 ? launch_fwd<64>(cap, bias, tm, p, as_stream(stream))
                        : launch_fwd<128>(cap, bias, tm, p, as_stream(stream));
}

int xt_attention_masked_bwd_workspace_size(const xt_attention_desc* desc, size_t* bytes) {
  XT_REQUIRE(desc && bytes && desc->T >= 0 && desc->T < (int64_t(1) << 30) && desc->H > 0 && desc->Hkv > 0 &&
                 desc->H % desc->Hkv == 0 && desc->hd > 0,
             "xt_attention_masked_bwd_workspace_size: bad arguments");
  const int split = key_split(desc);
  *bytes = d_bytes(desc) + (split > 1 ? 2 * part_bytes(desc, split) : 0);
  return XT_OK;
}

int xt_attention_masked_bwd(const xt_attention_desc* desc, const void* plan, size_t plan_bytes, const void* q,
                            int64_t ld_q, const void* k, int64_t ld_k, const void* v, int64_t ld_v, const void* o,
                            int64_t ld_o, const void* d_o, int64_t ld_do, const float* lse, void* dq,
                            int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv, void* ws, size_t ws_bytes,
                            void* stream) {
  const char* fn = "xt_attention_masked_bwd";
  const int H = desc ? desc->H : 0, Hkv = desc ? desc->Hkv : 0;
  XT_TRY(check(fn, desc, plan, plan_bytes, lse,
               {{q, ld_q, H}, {k, ld_k, Hkv}, {v, ld_v, Hkv}, {o, ld_o, H}, {d_o, ld_do, H}, {dq, ld_dq, H},
                {dk, ld_dk, Hkv}, {dv, ld_dv, Hkv}}));
  if (desc->T == 0) return XT_OK;
  size_t need = 0;
  XT_TRY(xt_attention_masked_bwd_workspace_size(desc, &need));
  XT_REQUIRE(ws && ws_bytes >= need, "%s: workspace too small (%zu < %zu)", fn, ws_bytes, need);
  if (!aligned16(ws)) return fail(XT_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", fn);
  attnm::Params p = attnm::params(desc, plan);
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.ldq = ld_q;
  p.ldk = ld_k;
  p.ldv = ld_v;
  p.o = const_cast<bf16*>(static_cast<const bf16*>(o));
  p.ldo = ld_o;
  p.d_o = static_cast<const bf16*>(d_o);
  p.lddo = ld_do;
  p.lse = const_cast<float*>(lse);
  p.nl = static_cast<float*>(ws);
  p.nd = p.nl + int64_t(p.plan.tiles) * BT * H;
  p.dq = static_cast<bf16*>(dq);
  p.dk = static_cast<bf16*>(dk);
  p.dv = static_cast<bf16*>(dv);
  p.lddq = ld_dq;
  p.lddk = ld_dk;
  p.lddv = ld_dv;
  CUtensorMap tm[4], tdq, tdk, tdv;
  XT_TRY(token_map(&tm[0], q, ld_q, desc->T, H, desc->hd));
  XT_TRY(token_map(&tm[1], k, ld_k, desc->T, Hkv, desc->hd));
  XT_TRY(token_map(&tm[2], v, ld_v, desc->T, Hkv, desc->hd));
  XT_TRY(token_map(&tm[3], d_o, ld_do, desc->T, H, desc->hd));
  XT_TRY(token_map(&tdq, dq, ld_dq, desc->T, H, desc->hd, true));
  const bool cap = desc->cap > 0.f, bias = desc->slopes != nullptr;
  cudaStream_t s = as_stream(stream);
  p.split = key_split(desc);
  p.share = (p.group + p.split - 1) / p.split;
  if (p.split > 1) {
    p.part_k = reinterpret_cast<float*>(static_cast<char*>(ws) + d_bytes(desc));
    p.part_v = reinterpret_cast<float*>(reinterpret_cast<char*>(p.part_k) + part_bytes(desc, p.split));
    const int64_t ld = int64_t(Hkv) * desc->hd;
    XT_TRY(token_map(&tdk, p.part_k, ld, desc->T, Hkv, desc->hd, true, true, p.split));
    XT_TRY(token_map(&tdv, p.part_v, ld, desc->T, Hkv, desc->hd, true, true, p.split));
  } else {
    XT_TRY(token_map(&tdk, dk, ld_dk, desc->T, Hkv, desc->hd, true));
    XT_TRY(token_map(&tdv, dv, ld_dv, desc->T, Hkv, desc->hd, true));
  }
  if (desc->hd == 64) {
    XT_TRY((launch_bwd<64, false>(cap, bias, tm, tdq, tdq, p, s)));
    XT_TRY((launch_bwd<64, true>(cap, bias, tm, tdk, tdv, p, s)));
  } else {
    XT_TRY((launch_bwd<128, false>(cap, bias, tm, tdq, tdq, p, s)));
    XT_TRY((launch_bwd<128, true>(cap, bias, tm, tdk, tdv, p, s)));
  }
  if (p.split == 1) return XT_OK;
  const int width = Hkv * desc->hd;
  const int64_t blocks = ceil_div(desc->T * width / 2, 256), most = int64_t(num_sms()) * 8;
  launch(attnm_join_kernel, unsigned(blocks < most ? blocks : most), 256, 0, s, p, width);
  return check_launch("xt_attention_masked_bwd (join)");
}

}  // extern "C"
