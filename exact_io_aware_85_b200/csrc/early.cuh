// early.cuh — kernels that are launched while those before them on the stream still run.
#pragma once

namespace fa {

// For kernels launched before the ones ahead of them on the stream have ended: everything those
// wrote is visible behind this.  Nothing that they may write or read is touched before it.  The
// next kernel may then be brought onto the SMs (it waits in the same way for this one's end).
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

}  // namespace fa
