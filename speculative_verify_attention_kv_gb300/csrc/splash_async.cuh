// Copies from global to shared memory that run in the background, in groups.
#pragma once

#include <cstdint>

namespace splash {

__device__ inline uint32_t shared_address(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// The first `bytes` of kBytes (4, 8 or 16, both addresses multiples of it); zeros
// for the rest.
template <int kBytes>
__device__ inline void copy_async(uint32_t dst, const void* src, int bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
                 "r"(bytes) : "memory");
}
// Ends the thread's group of copies (an empty one too).
__device__ inline void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All groups of the thread but the last kOpen have arrived.
template <int kOpen>
__device__ inline void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kOpen) : "memory");
}

}  // namespace splash
