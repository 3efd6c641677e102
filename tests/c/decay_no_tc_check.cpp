// The decayed attention's entry points in a build whose tensor-core path is off (vdn_host.cu's VDN_HAVE_TC = 0): linked
// with decay.o and these stand-ins for the rest of the library.  Prints the statuses of calls on addresses that are never
// read: bf16 sequences have to be refused before any launch, as have their workspace sizes.
#include <cstdint>
#include <cstdio>

#include "decay.h"
#include "internal.h"

static int launches = 0;

namespace vdn {
bool use_tc(const vdn_shape&, int) { return false; }
vdn_status check_shape(const vdn_shape*) { return VDN_OK; }
cudaError_t launch_decay_segments_tc(const DecayScan&, const DecayPlan&, float*) { return ++launches, cudaErrorUnknown; }
cudaError_t launch_decay_scan_tc(const DecayScan&, const DecayPlan&) { return ++launches, cudaErrorUnknown; }
}  // namespace vdn

int main() {
  auto at = [](int i) { return (float*)((uintptr_t)1 << 40) + ((size_t)i << 32); };
  const vdn_shape bf16 = {2, 4, 1, 3000, 128, 1, VDN_DTYPE_BF16}, f32 = {2, 4, 1, 3000, 128, 1, VDN_DTYPE_F32};
  std::printf("forward %d\n", (int)vdn_decay_forward(&bf16, at(0), at(1), at(2), at(3), nullptr, nullptr, 0, 0.f, at(4),
                                                     (size_t)1 << 40, at(5), at(6), nullptr));
  std::printf("backward %d\n", (int)vdn_decay_backward(&bf16, at(0), at(1), at(2), at(3), nullptr, nullptr, 0, 0.f, at(4),
                                                       nullptr, at(5), (size_t)1 << 40, at(6), at(7), at(8), nullptr, nullptr));
  std::printf("bf16 sizes %zu %zu\n", vdn_decay_workspace_size(&bf16), vdn_decay_backward_workspace_size(&bf16));
  std::printf("f32 sizes %d %d\n", vdn_decay_workspace_size(&f32) > 0, vdn_decay_backward_workspace_size(&f32) > 0);
  std::printf("launches %d\n", launches);
  return 0;
}
