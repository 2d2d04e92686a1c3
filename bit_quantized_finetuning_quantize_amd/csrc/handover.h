// A tag for flags in memory that nothing clears between calls.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// The dispatch packet's index in its queue (a hardware-provided value).
extern "C" __device__ uint64_t qlora_dispatch_index() __asm("llvm.amdgcn.dispatch.id");

// A tag unique to this dispatch within the process: dispatch indices count
// up per queue, and queues differ in address bits 12-39, so the value
// repeats only after 2^36 dispatches on one queue.
__device__ __forceinline__ uint64_t call_tag() {
  const uint64_t q = (uint64_t)(uintptr_t)__builtin_amdgcn_queue_ptr();
  return qlora_dispatch_index() ^ (q << 24);
}

}  // namespace qlora
