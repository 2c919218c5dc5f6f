// Host-only stand-ins for the kernel launchers that the front end of linear
// attention and of the norms at a block's end (kda_block_api.cpp) calls, as
// layer_stubs.cpp is for kda_layer_api.cpp: a launch does nothing and
// succeeds.  Not part of the library.
#include "kda_block.h"
#include "kda_linear.h"

namespace kda {

int launch_linear_forward(int, const LinearArgs&, const LinearPlan&, void*, float*, void*, void*) { return 0; }
int launch_linear_step(int, const LinearArgs&, float*, void*, void*) { return 0; }
int launch_linear_backward(int, const LinearArgs&, const LinearPlan&, const LinearGrads&, void*, void*) { return 0; }
int launch_gated_norm_forward(int, const BlockNormArgs&, void*, void*) { return 0; }
int launch_gated_norm_backward(int, const BlockNormArgs&, const void*, void*, void*, float*, float*, void*) { return 0; }
int launch_residual_norm_forward(int, const BlockNormArgs&, void*, void*, void*) { return 0; }
int launch_residual_norm_backward(int, const BlockNormArgs&, const void*, const void*, void*, void*, float*, float*,
                                  float*, void*) {
  return 0;
}

}  // namespace kda
