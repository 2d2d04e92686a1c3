// A tag for flags in memory that nothing clears between calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// The dispatch packet's index in its queue (a hardware-provided value).
extern "C" __device__ uint64_t qlora_dispatch_index() __asm("llvm.amdgcn.dispatch.id");

// A tag unique to this dispatch among those of the queues that live: dispatch
// indices count up per queue, and queues differ in address bits 12-39, so the
// value repeats only after 2^36 dispatches on one queue. A queue made at the
// address of a destroyed one would count from 0 again. The runtime keeps its
// queues when streams are destroyed (48 streams made and destroyed in turn, two
// dispatches each: one queue, 96 different tags). Flags that are left set after
// a call (the few-token NF4 forward's) rely on that; the rows of logits clear
// theirs.
__device__ __forceinline__ uint64_t call_tag() {
  const uint64_t q = (uint64_t)(uintptr_t)__builtin_amdgcn_queue_ptr();
  return qlora_dispatch_index() ^ (q << 24);
}

}  // namespace qlora
