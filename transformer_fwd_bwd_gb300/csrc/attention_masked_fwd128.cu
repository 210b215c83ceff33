// Masked attention forward, head dimension 128 (a translation unit of its own: they compile in parallel).
#include "attention_masked.cuh"

namespace xt {
namespace attnm {
XT_ATTNM_FWD(128)
}  // namespace attnm
}  // namespace xt
