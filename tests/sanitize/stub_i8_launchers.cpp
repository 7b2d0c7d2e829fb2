// Stand-ins for the kernel launchers of the 8-bit operators, as stub_launchers.cpp for the others:
// every launch reports that no device is present.
#include "i8_launch.h"

namespace gdr {

hipError_t launch_add_rmsnorm_i8(const NormArgs&) { return hipErrorNoDevice; }
hipError_t launch_gated_rmsnorm_i8(const NormArgs&) { return hipErrorNoDevice; }
hipError_t launch_matmul_i8(const MatmulArgs&) { return hipErrorNoDevice; }

}  // namespace gdr
