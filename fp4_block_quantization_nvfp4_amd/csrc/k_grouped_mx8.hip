// Grouped products of 8-bit rows (mx8); nvfp4_grouped.hpp has the kernel.
#include "nvfp4_grouped.hpp"

namespace nvfp4 {

int launch_grouped_mx8(const MatmulArgs& a, void* stream) { return grouped_launch<true>(a, stream); }

}  // namespace nvfp4
