// Stand-ins for the kernel launchers of the layer operators, as stub_launchers.cpp for the others:
// every launch reports that no device is present.
#include "layer_launch.h"

namespace gdr {

hipError_t launch_causal_conv(const ConvArgs&) { return hipErrorNoDevice; }
hipError_t launch_qk_norm_rope(const QkArgs&) { return hipErrorNoDevice; }
hipError_t launch_selective_scan(const ScanArgs&) { return hipErrorNoDevice; }
hipError_t launch_selective_scan_step(const ScanArgs&) { return hipErrorNoDevice; }

}  // namespace gdr
