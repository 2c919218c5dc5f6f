// Host-only stand-ins for the kernel launchers that the front end of the
// operators around the recurrence (kda_layer_api.cpp) calls, as
// host_stubs.cpp is for kda_api.cpp: a launch does nothing and succeeds.  Not
// part of the library.
#include "kda_layer.h"

namespace kda {

int launch_conv_forward(int, int, int, const ConvArgs&, void*, void*, void*) { return 0; }
int launch_conv_step(int, int, int, const ConvArgs&, void*, void*, void*) { return 0; }
int launch_conv_backward(int, int, int, const ConvArgs&, const void*, const void*, void*, float*, float*, void*, float*,
                         void*) {
  return 0;
}
int launch_scan_forward(int, const ScanArgs&, const ScanPlan&, void*, float*, void*, void*) { return 0; }
int launch_scan_step(int, const ScanArgs&, float*, void*, void*) { return 0; }
int launch_scan_backward(int, const ScanArgs&, const ScanBwdPlan&, const ScanGrads&, void*, void*) { return 0; }
int launch_norm_forward(int, const NormArgs&, void*, void*, void*) { return 0; }
int launch_norm_backward(int, const NormArgs&, const void*, const void*, void*, void*, float*, float*, float*, void*) {
  return 0;
}

}  // namespace kda
