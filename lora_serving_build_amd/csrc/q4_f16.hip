// Products with 4-bit weights, binary16 x, scales and y.
#include "q4_kernels.h"

namespace lora {

hipError_t launch_q4_f16(const Q4Args& a, int sub, hipStream_t s) { return launch_type<0>(a, sub, s); }

size_t q4_workspace(int32_t T, int32_t n, int32_t k, int32_t group) {
  const Q4Layout l = q4_layout(n, k, group, false);
  const Q4Plan p = q4_plan(T, l.tiles, l.blocks, l.sub);
  return p.splits > 1 ? (size_t)p.splits * (size_t)T * (size_t)l.tiles * 64 : 0;
}

}  // namespace lora
