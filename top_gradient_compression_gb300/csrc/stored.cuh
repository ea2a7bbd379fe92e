// Activations kept in 8 bits: codes int8, and an exponent byte for every 128 columns of a row.
#pragma once

#include "types.cuh"

namespace sparcml {

constexpr uint32_t kGroup = 128;       // columns that share an exponent
constexpr uint32_t kNanExponent = 255;  // the group held a NaN or an inf

// 2^(b - 127), a NaN for 255. (Below b = 1 the float is subnormal.)
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b == kNanExponent ? __uint_as_float(0x7fffffffu)
                           : __uint_as_float(b ? b << 23 : 0x00400000u);
}
// Byte i of w, a code, as a float: its bits with the sign's turned, as the low ones of 2^23 + c +
// 128, from which that is taken away.
__device__ __forceinline__ float code_at(uint32_t w, int i) {
  return __uint_as_float(__byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
}

}  // namespace sparcml
