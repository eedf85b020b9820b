// Programmatic dependent launch: a kernel lets the next one of its stream start while it runs, and that one waits for
// its end (and its writes) where it needs them.  A kernel launched so must wait in at least one thread before it ends:
// its own end is all that the stream's later work waits for.
#pragma once

namespace msa {

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace msa
