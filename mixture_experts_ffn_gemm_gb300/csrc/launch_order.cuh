// launch_order.cuh -- the order of kernels of one stream that may start while the one in front of them ends
// (programmatic launches).
#pragma once

namespace moe {

// The next kernel of the stream may start as SMs become free, if it was launched to wait by itself for this
// one's results (wait_for_prior_kernel); any other waits for this kernel's end as ever.
__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Nothing that a kernel before this one wrote, or still reads, may be touched in front of this; __ldg, which
// takes its data for constant while the kernel runs, may be moved there and does not belong behind it either.
__device__ __forceinline__ void wait_for_prior_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace moe
