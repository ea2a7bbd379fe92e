// Element types of the training-step operators: fp32, bf16 and fp16 arrays
// are read into fp32 and rounded once (to nearest even) when written.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// Two fp32 values; PACKED: one f32x2 instruction for both, which wants them in an aligned
// register pair. (The forward norm of long rows is 6 % faster packed, the backward one 4 %
// slower, by the moves.)
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float a, float b) { return {a, b}; }
__device__ __forceinline__ float2 split(F2 a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ unsigned long long pair(F2 a) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a.x), "f"(a.y));
  return v;
}
__device__ __forceinline__ F2 unpair(unsigned long long v) {
  F2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
template <bool PACKED>
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  if constexpr (!PACKED) return {a.x + b.x, a.y + b.y};
  unsigned long long v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(pair(a)), "l"(pair(b)));
  return unpair(v);
}
template <bool PACKED>
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  if constexpr (!PACKED) return {a.x * b.x, a.y * b.y};
  unsigned long long v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(pair(a)), "l"(pair(b)));
  return unpair(v);
}
template <bool PACKED>
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  if constexpr (!PACKED) return {fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)};
  unsigned long long v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
  return unpair(v);
}

// V elements as they lie in memory (a 16-byte group of words), or, for V = 2, two elements
// already in fp32.
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
struct Raw<T, 2> {
  F2 w;
  __device__ __forceinline__ void forget() {}
};

template <typename T>
__device__ __forceinline__ F2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ F2 unpack2<__nv_bfloat16>(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ F2 unpack2<__half>(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f2(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(F2 a);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(F2 a) {
  const float2 f = split(a);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(F2 a) {
  const float2 f = split(a);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Raw values as V / 2 fp32 pairs.
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, F2 (&f)[V / 2]) {
  if constexpr (V == 2) {
    f[0] = r.w;
  } else if constexpr (V == 4) {
    f[0] = f2(__uint_as_float(r.w.x), __uint_as_float(r.w.y));
    f[1] = f2(__uint_as_float(r.w.z), __uint_as_float(r.w.w));
  } else {
    f[0] = unpack2<T>(r.w.x);
    f[1] = unpack2<T>(r.w.y);
    f[2] = unpack2<T>(r.w.z);
    f[3] = unpack2<T>(r.w.w);
  }
}
template <typename T, int V>
__device__ __forceinline__ uint4 pack(const F2 (&f)[V / 2]) {
  if constexpr (V == 4) {
    const float2 p = split(f[0]), q = split(f[1]);
    return make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(q.x),
                      __float_as_uint(q.y));
  } else {
    return make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
  }
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  Raw<T, V> r;
  r.w = *reinterpret_cast<const uint4*>(p);
  return r;
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

template <typename T>
constexpr int32_t type_of() {
  return sizeof(T) == 4 ? SPARCML_F32
         : std::is_same_v<T, __half> ? SPARCML_F16 : SPARCML_BF16;
}
inline size_t type_bytes(int32_t type) { return type == SPARCML_F32 ? 4 : 2; }
inline bool type_ok(int32_t type) { return type >= SPARCML_F32 && type <= SPARCML_F16; }
inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace sparcml
