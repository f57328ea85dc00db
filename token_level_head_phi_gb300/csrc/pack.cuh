// Short vectors of a row and the approximate functions of the streaming
// operators (gated recurrence, normalised queries and keys, short convolution).
#pragma once

#include "common.cuh"

namespace mhla {

// N consecutive elements, at most 16 bytes; `whole` takes them in one access,
// otherwise the first `n` one by one.
template <typename T, int N>
struct Pack {
  static_assert(sizeof(T) * N <= 16, "one access");
  alignas(sizeof(T) * N) T v[N];
  __device__ __forceinline__ float f(int i) const { return to_f32(v[i]); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void load(const T* p, bool whole, int n = N) {
    if (whole) {
      if constexpr (sizeof(T) * N == 16)
        *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
      else if constexpr (sizeof(T) * N == 8)
        *reinterpret_cast<uint2*>(v) = __ldcs(reinterpret_cast<const uint2*>(p));
      else if constexpr (sizeof(T) * N == 4)
        *reinterpret_cast<unsigned int*>(v) = __ldcs(reinterpret_cast<const unsigned int*>(p));
      else
        v[0] = p[0];
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void store(T* p, bool whole, int n = N) const {
    if (whole) {
      if constexpr (sizeof(T) * N == 16)
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
      else if constexpr (sizeof(T) * N == 8)
        __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(v));
      else if constexpr (sizeof(T) * N == 4)
        __stcs(reinterpret_cast<unsigned int*>(p), *reinterpret_cast<const unsigned int*>(v));
      else
        p[0] = v[0];
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = v[i];
  }
};

// Asynchronous copies into shared memory: `bytes` of BYTES (4, 8 or 16), zeros
// behind them.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from, int bytes) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at), "l"(from), "n"(BYTES), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Programmatic launches: a kernel waits here for all of its predecessor's results;
// its predecessor lets it start early.
__device__ __forceinline__ void after_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Entry i of a parameter vector that is bf16 or float32.
__device__ __forceinline__ float param_at(const void* p, int is_f32, int64_t i) {
  return is_f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The smaller one, a NaN if either is.
__device__ __forceinline__ float least(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
// The larger one, a NaN if either is.
__device__ __forceinline__ float most(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
constexpr float kLog2e = 1.4426950408889634f;

// Pairs of float32 in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 splat(float a) { return make_float2(a, a); }
// With a constant.
__device__ __forceinline__ float2 addc(float2 a, float c) { return add2(a, splat(c)); }
__device__ __forceinline__ float2 mulc(float2 a, float c) { return mul2(a, splat(c)); }
__device__ __forceinline__ float2 fmac(float2 a, float2 b, float c) { return fma2(a, b, splat(c)); }

// Elements 2 i and 2 i + 1 of a pack.
template <int N>
__device__ __forceinline__ float2 pair_of(const Pack<__nv_bfloat16, N>& x, int i) {
  const uint32_t v = reinterpret_cast<const uint32_t*>(x.v)[i];
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <int N>
__device__ __forceinline__ float2 pair_of(const Pack<float, N>& x, int i) {
  return make_float2(x.v[2 * i], x.v[2 * i + 1]);
}
template <int N>
__device__ __forceinline__ void put_pair(Pack<__nv_bfloat16, N>* x, int i, float2 v) {
  reinterpret_cast<__nv_bfloat162*>(x->v)[i] = __floats2bfloat162_rn(v.x, v.y);
}
template <int N>
__device__ __forceinline__ void put_pair(Pack<float, N>* x, int i, float2 v) {
  x->v[2 * i] = v.x;
  x->v[2 * i + 1] = v.y;
}

}  // namespace mhla
