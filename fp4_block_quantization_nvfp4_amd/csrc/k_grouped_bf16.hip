// Grouped products of bf16 rows; nvfp4_grouped.hpp has the kernel.
#include "nvfp4_grouped.hpp"

namespace nvfp4 {

int launch_grouped_bf16(const MatmulArgs& a, void* stream) { return grouped_launch<false>(a, stream); }

}  // namespace nvfp4
