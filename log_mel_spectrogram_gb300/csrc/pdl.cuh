// pdl.cuh -- programmatic dependent launch from a kernel's side (launch_dependent() is the host's).
#pragma once

namespace lm {

// The grid before has finished and its writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next grid may start.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace lm
