// GEMM instantiations with the gated feed-forward block's epilogues.
#include "gemm.cuh"

namespace xt {
namespace gemm {

template <int ACT, bool B_MN>
static int pick(int bn, int cg, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                const CUtensorMap& tc2, const Params& p, int grid, cudaStream_t s) {
  if (cg == 2) return launch_one<kBf16, 256, false, B_MN, ACT, 2>(ta, tb, tc, tc2, p, grid, s);
  if (bn == 128) return launch_one<kBf16, 128, false, B_MN, ACT>(ta, tb, tc, tc2, p, grid, s);
  return launch_one<kBf16, 256, false, B_MN, ACT>(ta, tb, tc, tc2, p, grid, s);
}

int launch_gated(int act, int bn, int cg, const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                 const CUtensorMap& tc2, const Params& p, int grid, cudaStream_t s) {
  switch (act) {
    case kGateFwdSilu: return pick<kGateFwdSilu, true>(bn, cg, ta, tb, tc, tc2, p, grid, s);
    case kGateFwdGelu: return pick<kGateFwdGelu, true>(bn, cg, ta, tb, tc, tc2, p, grid, s);
    case kGateBwdSilu: return pick<kGateBwdSilu, false>(bn, cg, ta, tb, tc, tc2, p, grid, s);
    case kGateBwdGelu: return pick<kGateBwdGelu, false>(bn, cg, ta, tb, tc, tc2, p, grid, s);
    default: return fail(XT_ERR_UNSUPPORTED, "gemm: gated epilogue %d", act);
  }
}

}  // namespace gemm
}  // namespace xt
