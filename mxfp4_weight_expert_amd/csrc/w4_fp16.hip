// The 4-bit products of half tokens, and the choice between the token types.
#include "w4_kernel.h"

namespace moe {
hipError_t launch_w4(const W4Args& a, hipStream_t st) {
  return a.dtype == MOE_DTYPE_BF16 ? launch_w4_bf16(a, st) : w4_formats<MOE_DTYPE_FP16>(a, st);
}
}  // namespace moe
