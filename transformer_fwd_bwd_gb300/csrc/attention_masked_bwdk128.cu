// Masked attention backward, key pass (dK, dV), head dimension 128.
#include "attention_masked.cuh"

namespace xt {
namespace attnm {
XT_ATTNM_BWD(128, true)
}  // namespace attnm
}  // namespace xt
