// Masked attention backward, query pass (dQ, D), head dimension 128.
#include "attention_masked.cuh"

namespace xt {
namespace attnm {
XT_ATTNM_BWD(128, false)
}  // namespace attnm
}  // namespace xt
