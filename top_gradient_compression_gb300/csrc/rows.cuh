// What the row-wise operators share: the threads that share a row with their sums, and the
// join of the blocks' sums over columns.
#pragma once

#include <algorithm>

#include "types.cuh"

namespace sparcml {

constexpr uint32_t kSms = 152;

namespace {

// The `threads` threads that share a row: 8, 16 or 32 lanes of a warp, or whole warps
// with a named barrier and 2 * 33 float2 of shared memory of their own.
struct Group {
  uint32_t threads, index, t;  // their number, which group of the block, this thread's place
  float2* scratch;
  uint32_t turn;

  __device__ __forceinline__ void sync() const {
    if (threads > 32)
      asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(threads) : "memory");
    else
      __syncwarp();
  }
  template <int D>
  static __device__ __forceinline__ void add(float2& v) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, D);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, D);
  }
  __device__ __forceinline__ float sum(float2 two) {
    float v = two.x + two.y;
    if (threads >= 32) v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (threads >= 16) v += __shfl_xor_sync(0xffffffffu, v, 8);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threads <= 32) return v;
    float2* s = scratch + 33 * (turn & 1u);
    ++turn;
    const uint32_t lane = lane_id(), nw = threads >> 5;
    if (lane == 0) s[t >> 5].x = v;
    sync();
    v = lane < nw ? s[lane].x : 0.f;
    if (nw > 8) {
      if (nw > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return __shfl_sync(0xffffffffu, v, 0);
  }
  // Sums of two values. `turn` alternates between the halves of the scratch from call to
  // call, so that one barrier per call is enough.
  __device__ __forceinline__ float2 sum2(float2 v) {
    if (threads >= 32) add<16>(v);
    if (threads >= 16) add<8>(v);
    add<4>(v);
    add<2>(v);
    add<1>(v);
    if (threads <= 32) return v;
    float2* s = scratch + 33 * (turn & 1u);
    ++turn;
    const uint32_t lane = lane_id(), nw = threads >> 5;
    if (lane == 0) s[t >> 5] = v;
    sync();
    v = lane < nw ? s[lane] : make_float2(0.f, 0.f);
    if (nw > 8) {
      if (nw > 16) add<16>(v);
      add<8>(v);
    }
    add<4>(v);
    add<2>(v);
    add<1>(v);
    // the lanes that were added up hold the sum; the first one tells the rest
    v.x = __shfl_sync(0xffffffffu, v.x, 0);
    v.y = __shfl_sync(0xffffffffu, v.y, 0);
    return v;
  }
};
__device__ __forceinline__ Group make_group(uint32_t threads, float2* scratch) {
  const uint32_t index = threadIdx.x / threads;
  return {threads, index, threadIdx.x - index * threads, scratch + 66 * index, 0};
}

// out[c] (+)= sum of the `parts` partial sums of column c: 32 columns per block,
// 16 warps over the parts, joined in warp order. blockIdx.y: 0 dw, 1 db.
__global__ void __launch_bounds__(512)
join_columns_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b,
                 uint32_t parts, uint64_t dim, float* dw, float* db, int32_t accumulate) {
  griddep_wait();
  __shared__ float sums[16][33];
  const float* part = blockIdx.y ? part_b : part_w;
  float* out = blockIdx.y ? db : dw;
  if (out == nullptr) return;
  const uint32_t lane = lane_id(), warp = threadIdx.x >> 5;
  const uint64_t c = (uint64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < dim) {
    for (uint32_t p = warp; p < parts; p += 16 * 20) {
      float v[20];  // on their way together
#pragma unroll
      for (uint32_t k = 0; k < 20; ++k)
        v[k] = p + 16 * k < parts ? part[(uint64_t)(p + 16 * k) * dim + c] : 0.f;
#pragma unroll
      for (uint32_t k = 0; k < 20; ++k) s += v[k];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < dim) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += sums[k][lane];
    out[c] = accumulate ? out[c] + v : v;
  }
}

// Threads that share a row, in whole warps, when each holds `per` elements.
inline uint32_t threads_for(uint64_t dim, uint32_t per) {
  return (uint32_t)((dim + 32ull * per - 1) / (32ull * per)) * 32u;
}

constexpr uint32_t kBackwardPer = 16;  // elements per thread

// Threads of a row and of a block, and the blocks, each with a row of partial sums: what
// the registers of the SMs hold at one time (kFit blocks of 256 threads each; with a
// second, partial wave 16384 x 4096 fp32 took 271 us), no more than there are rows.
constexpr uint32_t kFit = 2;
struct BackwardShape {
  uint32_t threads, block, parts;
};
inline BackwardShape backward_shape(uint64_t rows, uint64_t dim) {
  const uint32_t threads = dim <= 128   ? 8
                           : dim <= 256 ? 16
                                        : (uint32_t)std::min<uint64_t>(
                                              512, threads_for(dim, kBackwardPer));
  const uint32_t groups = std::max(1u, 256 / threads);
  const uint64_t most = kSms * (threads <= 256 ? kFit : 1);
  return {threads, threads * groups,
          (uint32_t)std::max<uint64_t>(1, std::min((rows + groups - 1) / groups, most))};
}

}  // namespace
}  // namespace sparcml
