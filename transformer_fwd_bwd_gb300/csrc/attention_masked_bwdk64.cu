// Masked attention backward, key pass (dK, dV), head dimension 64.
#include "attention_masked.cuh"

namespace xt {
namespace attnm {
XT_ATTNM_BWD(64, true)
}  // namespace attnm
}  // namespace xt
