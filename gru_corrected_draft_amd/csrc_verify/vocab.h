// Device helpers of the kernels that read rows of logits.
#pragma once
#include "common.h"

namespace {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
};
template <>
struct Elem<bf16_t> {
  static constexpr int kVec = 8;
};

// kVec consecutive logits as they lie in memory.  Rows of an odd vocabulary are
// aligned to the element only; the copy still compiles to one 16-byte load,
// which the memory path takes at any alignment.  Past the n that there are, -inf.
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T* p, int n) {
  constexpr int V = Elem<T>::kVec;
  u32x4 raw;
  if (n >= V) {
    __builtin_memcpy(&raw, p, 16);
    return raw;
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t lo = 2 * w < n ? p[2 * w] : 0xFF80u, hi = 2 * w + 1 < n ? p[2 * w + 1] : 0xFF80u;
      raw[w] = lo | hi << 16;
    } else {
      raw[w] = w < n ? __float_as_uint(p[w]) : 0xFF800000u;
    }
  }
  return raw;
}
template <typename T>
__device__ __forceinline__ void unpack(const u32x4& raw, float* x) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (sizeof(T) == 2) {
      x[2 * w] = __uint_as_float(raw[w] << 16);
      x[2 * w + 1] = __uint_as_float(raw[w] & 0xFFFF0000u);
    } else {
      x[w] = __uint_as_float(raw[w]);
    }
  }
}
__device__ __forceinline__ float load_one(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }

// the largest fp32 number for +inf, -inf for NaN
__device__ __forceinline__ float tame(float x) {
  return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);
}

// e^x's power of two; results below 2^-126 become zero
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The largest of n; a quiet NaN is passed over, a signaling one takes its two
// neighbours with it.  Written out because fmaxf first makes each operand
// canonical, one more instruction apiece.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
  float top = max3(x[0], x[1], x[2]);
#pragma unroll
  for (int j = 3; j + 1 < N; j += 2) top = max3(top, x[j], x[j + 1]);
  return max3(top, x[N - 1], x[N - 1]);
}

// Lane exchange for reductions over a wave: neighbours, pairs, halves of eight
// and sixteen by data-parallel moves, then halves of 32 and 64 by swaps.
template <int STEP>
__device__ __forceinline__ uint32_t other(uint32_t x) {
  if constexpr (STEP == 0) return __builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false);   // quad_perm 1 0 3 2
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(x, x, 0x4E, 0xF, 0xF, false);   // quad_perm 2 3 0 1
  if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(x, x, 0x141, 0xF, 0xF, false);  // row_half_mirror
  if constexpr (STEP == 3) return __builtin_amdgcn_update_dpp(x, x, 0x140, 0xF, 0xF, false);  // row_mirror
  return x;
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, F f) {
  x = f(x, other<0>(x));
  x = f(x, other<1>(x));
  x = f(x, other<2>(x));
  x = f(x, other<3>(x));
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_max(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ int wave_min(int x) {
  return (int)wave_reduce((uint32_t)x, [](uint32_t a, uint32_t b) { return (uint32_t)min((int)a, (int)b); });
}

}  // namespace
