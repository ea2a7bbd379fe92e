// Element types of the training-step operators: fp32, bf16 and fp16 arrays
// are read into fp32 and rounded once (to nearest even) when written.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace sparcml {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements, moved as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};

// V elements as they lie in memory: a 16-byte word group (V > 1), or one element.
template <typename T, int V>
struct Raw {
  uint4 w;
  // Hides where the value came from: a later unpack() is then done anew, instead of the
  // floats of an earlier one being kept in four or eight registers.
  __device__ __forceinline__ void forget() {
    asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
  }
};
template <typename T>
struct Raw<T, 1> {
  T w;
  __device__ __forceinline__ void forget() {}
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = to_f32(r.w);
  } else if constexpr (V == 4) {
    f[0] = __uint_as_float(r.w.x); f[1] = __uint_as_float(r.w.y);
    f[2] = __uint_as_float(r.w.z); f[3] = __uint_as_float(r.w.w);
  } else {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = unpack2<T>(w[e]);
      f[2 * e] = p.x;
      f[2 * e + 1] = p.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float (&f)[V]) {
  Raw<T, V> r;
  if constexpr (V == 1) {
    r.w = from_f32<T>(f[0]);
  } else if constexpr (V == 4) {
    r.w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
  } else {
    r.w = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                     pack2<T>(f[6], f[7]));
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  Raw<T, V> r;
  r.w = *reinterpret_cast<const decltype(r.w)*>(p);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& r) {
  *reinterpret_cast<decltype(Raw<T, V>::w)*>(p) = r.w;
}

// One element of an array whose type is a run-time code (enum sparcml_type).
__device__ __forceinline__ float load_any(const void* p, int32_t type, uint64_t i) {
  if (type == SPARCML_F32) return static_cast<const float*>(p)[i];
  if (type == SPARCML_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

inline size_t type_bytes(int32_t type) { return type == SPARCML_F32 ? 4 : 2; }
inline bool type_ok(int32_t type) { return type >= SPARCML_F32 && type <= SPARCML_F16; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace sparcml
