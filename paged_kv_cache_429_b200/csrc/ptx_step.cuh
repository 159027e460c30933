// Inline-PTX wrappers of the serving-step kernels (tables.cuh, rope.cuh,
// shared_prefix.cuh), beside those of ptx.cuh.
#pragma once

#include <cstdint>

namespace pa {

// Programmatic dependent launch: let the next kernel of the stream start
// beside this one, and wait until the one before has finished (its writes
// visible). Without the launch attribute neither does anything.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// 32 bytes, a whole sector, of one thread (32-byte aligned).
__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

}  // namespace pa
