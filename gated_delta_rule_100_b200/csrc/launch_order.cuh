// launch_order.cuh -- hints between a kernel and the next one on its stream.
#pragma once

namespace kda {

// The next kernel's blocks may be placed now (they still wait for this one's end).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// The kernel before this one has ended and its writes are visible.
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace kda
