// Masked attention backward, query pass (dQ, D), head dimension 64.
#include "attention_masked.cuh"

namespace xt {
namespace attnm {
XT_ATTNM_BWD(64, false)
}  // namespace attnm
}  // namespace xt
