// store_through.hpp -- stores that go through the L2 cache of their XCD to memory's own
// cache at once.  Plain stores stay in the eight L2 caches until the kernel ends, which
// then waits for up to 32 MB to be written back; stores past all caches (non-temporal)
// make what reads the values next wait for memory.  8-bit product 4000 x 8192 x 4096,
// alone and with the convolution that reads its output behind it: 159 and 189 us with
// plain stores, 131 and 170 non-temporal, 140 and 160 through.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

typedef unsigned through_u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned through_u32x4 __attribute__((ext_vector_type(4)));

// 8 or 16 bytes at p.  A store has no result to wait for, but the registers of one of
// more than 8 bytes must not be written for two wait states behind it, which the
// compiler does not see to for inline assembly.
__device__ __forceinline__ void store_through(void* p, through_u32x4 v) {
  asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" ::"v"(p), "v"(v) : "memory");
}
__device__ __forceinline__ void store_through(void* p, through_u32x2 v) {
  asm volatile("global_store_dwordx2 %0, %1, off sc1" ::"v"(p), "v"(v) : "memory");
}

}  // namespace gdr
