// numbers.cuh -- numbers of the 16-bit types and of binary32 on the device, and
// short vectors of them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace zo {

// Two numbers of the data's type as binary32, and back with one rounding each.
template <typename T> struct Num;
template <> struct Num<__half> {
  static __device__ float get(__half x) { return __half2float(x); }
  static __device__ float2 get2(const __half* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
  static __device__ __half put(float x) { return __float2half_rn(x); }
  static __device__ void put2(__half* p, float2 x) { *reinterpret_cast<__half2*>(p) = __float22half2_rn(x); }
  static __device__ float2 of_word(uint32_t u) {
    return __half22float2(__halves2half2(__ushort_as_half((unsigned short)u), __ushort_as_half((unsigned short)(u >> 16))));
  }
  static __device__ uint32_t word(float2 x) {
    const __half2 h = __float22half2_rn(x);
    return (uint32_t)__half_as_ushort(__high2half(h)) << 16 | __half_as_ushort(__low2half(h));
  }
};
template <> struct Num<__nv_bfloat16> {
  static __device__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ float2 get2(const __nv_bfloat16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
  static __device__ void put2(__nv_bfloat16* p, float2 x) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(x);
  }
  static __device__ float2 of_word(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ uint32_t word(float2 x) {
    const __nv_bfloat162 h = __float22bfloat162_rn(x);
    return (uint32_t)__bfloat16_as_ushort(__high2bfloat16(h)) << 16 | __bfloat16_as_ushort(__low2bfloat16(h));
  }
};
template <> struct Num<float> {
  static __device__ float get(float x) { return x; }
  static __device__ float2 get2(const float* p) { return make_float2(p[0], p[1]); }
  static __device__ float put(float x) { return x; }
  static __device__ void put2(float* p, float2 x) { p[0] = x.x; p[1] = x.y; }
};

// Numbers of 16 bytes, held as words, as pairs of binary32 and back.
template <typename E> __device__ __forceinline__ void unpack(uint4 w, float2* x) {
  if constexpr (sizeof(E) == 4) {
    x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = Num<E>::of_word(u[k]);
  }
}
template <typename E> __device__ __forceinline__ uint4 pack(const float2* x) {
  if constexpr (sizeof(E) == 4)
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  else
    return make_uint4(Num<E>::word(x[0]), Num<E>::word(x[1]), Num<E>::word(x[2]), Num<E>::word(x[3]));
}

// V numbers at an address that is a multiple of their size, of 16 bytes at most.
template <typename T, int V> struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Vec { T v[V]; };

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// 16 bytes from global to shared memory, in the background.
__device__ __forceinline__ void copy16(void* to, const char* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}

// The same of which only the first `bytes` are read; the rest becomes zero.
__device__ __forceinline__ void copy16(void* to, const char* from, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(bytes)
               : "memory");
}

}  // namespace zo
