// Products with 4-bit weights, bfloat16 x, scales and y.
#include "q4_kernels.h"

namespace lora {

hipError_t launch_q4_bf16(const Q4Args& a, int sub, hipStream_t s) { return launch_type<1>(a, sub, s); }

}  // namespace lora
