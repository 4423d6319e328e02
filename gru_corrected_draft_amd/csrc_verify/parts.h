// Results in parts, joined by the last workgroup of a launch to bring one.
#pragma once
#include "common.h"

// Parts of a result pass between workgroups of one launch on any XCD: written
// through to and read from where all see them, 8 bytes at a time.  A fence in
// their place writes a whole L2 back (27.5 us for those 10.8).
__device__ __forceinline__ void share2(float* p, float x, float y) {
  const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
  __hip_atomic_store((uint64_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 shared2(const float* p) {
  const uint64_t v = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float4 shared4(const float* p) {
  const float2 a = shared2(p), b = shared2(p + 2);
  return make_float4(a.x, a.y, b.x, b.y);
}
// Called by all threads of a workgroup after they shared a part of a segment:
// whether it was the last of `parts`, in which case all of them can be read.
__device__ __forceinline__ bool last_of(int32_t* arrived, int parts, int* s_last) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's are where all see them
  __syncthreads();
  if (threadIdx.x == 0) {
    *s_last = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    if (*s_last) __hip_atomic_store(arrived, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *s_last;
}
