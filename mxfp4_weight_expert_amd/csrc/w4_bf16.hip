// The 4-bit products of bfloat16 tokens.
#include "w4_kernel.h"

namespace moe {
hipError_t launch_w4_bf16(const W4Args& a, hipStream_t st) {
  return w4_formats<MOE_DTYPE_BF16>(a, st);
}
}  // namespace moe
