// Layer norm over rows, forward and backward, for the training step around
// the gradient exchange.
//
//   y  = (x - mean) * rstd * w + b
//   dx = rstd * (d - mean(d) - xh * mean(d * xh)),  d = dy * w, xh = (x - mean) * rstd
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Both passes are bound by memory: forward moves 2 elements per element of x,
// backward 3. A row is read once, into the registers of the threads that share
// it, and every sum over it (the mean, then the sum of squared deviations from
// that mean, which loses nothing to cancellation) is taken from there.

#include <algorithm>

#include "types.cuh"

namespace sparcml {
namespace {

// Sum of two values over the threads that share a row: a warp, or the whole
// block. `scratch` holds 2 * 33 float2 of shared memory; `turn` alternates
// between its halves from call to call, so that one barrier per call is enough.
template <bool BLOCK>
__device__ __forceinline__ float2 row_sum(float2 v, float2* scratch, uint32_t& turn) {
  v.x = warp_sum_f(v.x);
  v.y = warp_sum_f(v.y);
  if (!BLOCK) return v;
  float2* s = scratch + 33 * (turn & 1u);
  ++turn;
  const uint32_t lane = lane_id(), nw = blockDim.x >> 5;
  if (lane == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? s[lane] : make_float2(0.f, 0.f);
  v.x = warp_sum_f(v.x);
  v.y = warp_sum_f(v.y);
  return v;
}

// V weights from column c; 1 where there is no weight.
template <int V>
__device__ __forceinline__ void load_affine(const void* w, int32_t type, bool vec, uint64_t c,
                                            float none, float (&out)[V]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = none;
  } else if (V > 1 && vec) {
    if (type == SPARCML_F32) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + 4 * q);
        out[4 * q] = f.x; out[4 * q + 1] = f.y; out[4 * q + 2] = f.z; out[4 * q + 3] = f.w;
      }
    } else if (type == SPARCML_BF16) {
      const auto p = *reinterpret_cast<const Pack<__nv_bfloat16, V>*>(
          static_cast<const __nv_bfloat16*>(w) + c);
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = to_f32(p.e[i]);
    } else {
      const auto p =
          *reinterpret_cast<const Pack<__half, V>*>(static_cast<const __half*>(w) + c);
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = to_f32(p.e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = load_any(w, type, c + i);
  }
}

struct NormArgs {
  const void* x;
  int64_t x_stride;  // elements between rows
  const void* w;     // may be null: all ones
  const void* b;     // may be null: all zeros
  int32_t w_type;
  int32_t vec_w;  // w and b may be read V at a time
  uint64_t rows;
  uint64_t dim;
  float eps;
  void* y;
  int64_t y_stride;
  float* mean;
  float* rstd;
};

// NV packs of V elements per thread; pack j of thread t starts at column
// (j * threads + t) * V.
template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128) norm_forward_kernel(const NormArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  uint32_t turn = 0;
  const uint32_t threads = BLOCK ? blockDim.x : 32u;
  const uint32_t t = BLOCK ? threadIdx.x : lane_id();
  const uint64_t row = BLOCK ? blockIdx.x
                             : (uint64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (!BLOCK && row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + (int64_t)row * a.x_stride;
  Pack<T, V> v[NV];
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t c = (uint64_t)(j * threads + t) * V;
    if (c < a.dim) v[j] = *reinterpret_cast<const Pack<T, V>*>(x + c);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((uint64_t)(j * threads + t) * V < a.dim) {
#pragma unroll
      for (int i = 0; i < V; ++i) s.x += to_f32(v[j].e[i]);
    }
  const float inv = 1.0f / (float)a.dim;
  const float mean = row_sum<BLOCK>(s, scratch, turn).x * inv;
  s.x = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if ((uint64_t)(j * threads + t) * V < a.dim) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = to_f32(v[j].e[i]) - mean;
        s.x += d * d;
      }
    }
  const float var = row_sum<BLOCK>(s, scratch, turn).x * inv;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (t == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + (int64_t)row * a.y_stride;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t c = (uint64_t)(j * threads + t) * V;
    if (c < a.dim) {
      float w[V], b[V];
      load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
      load_affine<V>(a.b, a.w_type, a.vec_w, c, 0.f, b);
      Pack<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i)
        o.e[i] = from_f32<T>((to_f32(v[j].e[i]) - mean) * rstd * w[i] + b[i]);
      *reinterpret_cast<Pack<T, V>*>(y + c) = o;
    }
  }
}

// Rows too long for a block's registers: the row is read again for each sum
// (from L2, where one row of any such length fits).
template <typename T>
__global__ void __launch_bounds__(1024) norm_forward_long_kernel(const NormArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  uint32_t turn = 0;
  const T* x = static_cast<const T*>(a.x) + (int64_t)blockIdx.x * a.x_stride;
  T* y = static_cast<T*>(a.y) + (int64_t)blockIdx.x * a.y_stride;
  const float inv = 1.0f / (float)a.dim;
  float2 s = make_float2(0.f, 0.f);
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) s.x += to_f32(x[c]);
  const float mean = row_sum<true>(s, scratch, turn).x * inv;
  s.x = 0.f;
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(x[c]) - mean;
    s.x += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum<true>(s, scratch, turn).x * inv + a.eps);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = rstd;
  }
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float w = a.w ? load_any(a.w, a.w_type, c) : 1.f;
    const float b = a.b ? load_any(a.b, a.w_type, c) : 0.f;
    y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * w + b);
  }
}

struct NormGradArgs {
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* w;
  int32_t w_type;
  int32_t vec_w;
  const float* mean;
  const float* rstd;
  uint64_t rows;
  uint64_t dim;
  void* dx;
  int64_t dx_stride;
  float* part_w;  // [gridDim.x][dim] partial sums over the block's rows
  float* part_b;
};

// A block walks rows blockIdx.x, blockIdx.x + gridDim.x, ...; each thread keeps
// the running dw and db of its own columns in registers, so x and dy are read
// once for dx, dw and db together. Where a warp has a row of its own, the warps'
// sums are joined in warp order at the end. Every order is fixed.
template <typename T, int V, int NV, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(const NormGradArgs a) {
  griddep_wait();
  extern __shared__ float join[];  // !BLOCK: [2][dim]
  __shared__ float2 scratch[66];
  uint32_t turn = 0;
  const uint32_t threads = BLOCK ? blockDim.x : 32u;
  const uint32_t t = BLOCK ? threadIdx.x : lane_id();
  const uint32_t per = BLOCK ? 1u : blockDim.x >> 5;
  const uint32_t slot = BLOCK ? 0u : threadIdx.x >> 5;
  float gw[NV][V], gb[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) gw[j][i] = gb[j][i] = 0.f;
  }
  const float inv = 1.0f / (float)a.dim;
  for (uint64_t row = (uint64_t)blockIdx.x * per + slot; row < a.rows;
       row += (uint64_t)gridDim.x * per) {
    const T* x = static_cast<const T*>(a.x) + (int64_t)row * a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride;
    const float mean = a.mean[row], rstd = a.rstd[row];
    Pack<T, V> vx[NV], vd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) {
        vx[j] = *reinterpret_cast<const Pack<T, V>*>(x + c);
        vd[j] = *reinterpret_cast<const Pack<T, V>*>(dy + c);
      }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) {
        float w[V];
        load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float g = to_f32(vd[j].e[i]);
          const float xh = (to_f32(vx[j].e[i]) - mean) * rstd;
          gw[j][i] += g * xh;
          gb[j][i] += g;
          s.x += g * w[i];
          s.y += g * w[i] * xh;
        }
      }
    }
    s = row_sum<BLOCK>(s, scratch, turn);
    const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) {
        float w[V];
        load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
        Pack<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (to_f32(vx[j].e[i]) - mean) * rstd;
          o.e[i] = from_f32<T>(rstd * (to_f32(vd[j].e[i]) * w[i] - c1 - xh * c2));
        }
        *reinterpret_cast<Pack<T, V>*>(dx + c) = o;
      }
    }
  }
  if constexpr (!BLOCK) {
    for (uint32_t k = 0; k < per; ++k) {
      if (slot == k) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const uint64_t c = (uint64_t)(j * threads + t) * V + i;
            if (c < a.dim) {
              join[c] = (k ? join[c] : 0.f) + gw[j][i];
              join[a.dim + c] = (k ? join[a.dim + c] : 0.f) + gb[j][i];
            }
          }
        }
      }
      __syncthreads();
    }
    for (uint32_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
      a.part_w[(uint64_t)blockIdx.x * a.dim + c] = join[c];
      a.part_b[(uint64_t)blockIdx.x * a.dim + c] = join[a.dim + c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t c = (uint64_t)(j * threads + t) * V + i;
        if (c < a.dim) {
          a.part_w[(uint64_t)blockIdx.x * a.dim + c] = gw[j][i];
          a.part_b[(uint64_t)blockIdx.x * a.dim + c] = gb[j][i];
        }
      }
    }
  }
}

// Rows too long for a block's registers: dx by re-reading the row, the column
// sums by norm_columns_kernel.
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const NormGradArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  uint32_t turn = 0;
  const T* x = static_cast<const T*>(a.x) + (int64_t)blockIdx.x * a.x_stride;
  const T* dy = static_cast<const T*>(a.dy) + (int64_t)blockIdx.x * a.dy_stride;
  T* dx = static_cast<T*>(a.dx) + (int64_t)blockIdx.x * a.dx_stride;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  const float inv = 1.0f / (float)a.dim;
  float2 s = make_float2(0.f, 0.f);
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (a.w ? load_any(a.w, a.w_type, c) : 1.f);
    s.x += d;
    s.y += d * ((to_f32(x[c]) - mean) * rstd);
  }
  s = row_sum<true>(s, scratch, turn);
  const float c1 = s.x * inv, c2 = s.y * inv;
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (a.w ? load_any(a.w, a.w_type, c) : 1.f);
    const float xh = (to_f32(x[c]) - mean) * rstd;
    dx[c] = from_f32<T>(rstd * (d - c1 - xh * c2));
  }
}

// part[blockIdx.y][c] = sums over the rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradArgs a) {
  griddep_wait();
  const uint64_t c = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.dim) return;
  float gw = 0.f, gb = 0.f;
  for (uint64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float g = to_f32(static_cast<const T*>(a.dy)[(int64_t)r * a.dy_stride + c]);
    const float v = to_f32(static_cast<const T*>(a.x)[(int64_t)r * a.x_stride + c]);
    gw += g * ((v - a.mean[r]) * a.rstd[r]);
    gb += g;
  }
  a.part_w[(uint64_t)blockIdx.y * a.dim + c] = gw;
  a.part_b[(uint64_t)blockIdx.y * a.dim + c] = gb;
}

// out[c] (+)= sum of the `parts` partial sums of column c: 32 columns per block,
// 16 warps over the parts, joined in warp order. blockIdx.y: 0 dw, 1 db.
__global__ void __launch_bounds__(512)
norm_join_kernel(const float* __restrict__ part_w, const float* __restrict__ part_b,
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
#pragma unroll 4
    for (uint32_t p = warp; p < parts; p += 16) s += part[(uint64_t)p * dim + c];
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
uint32_t threads_for(uint64_t dim, uint32_t per) {
  return (uint32_t)((dim + 32ull * per - 1) / (32ull * per)) * 32u;
}

constexpr uint32_t kForwardPer = 32, kForwardPer1 = 16;  // elements per thread, V > 1 and V = 1
constexpr uint32_t kBackwardPer = 16;

template <typename T, int V, int NV>
void launch_forward(const NormArgs& a, cudaStream_t s) {
  const uint32_t threads = threads_for(a.dim, V * NV);
  if (threads == 32)
    launch_pdl(norm_forward_kernel<T, V, NV, false>, (unsigned)((a.rows + 3) / 4), 128, 0, s, a);
  else
    launch_pdl(norm_forward_kernel<T, V, NV, true>, (unsigned)a.rows, threads, 0, s, a);
}

// Packs of 16 bytes need 16-byte aligned rows and a whole number of packs; other
// rows are read element by element.
template <typename T>
void forward_typed(const NormArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.x_stride % V == 0 && a.y_stride % V == 0 &&
                   aligned_to(a.x, 16) && aligned_to(a.y, 16);
  if (vec && a.dim <= 1024ull * kForwardPer)
    launch_forward<T, V, kForwardPer / V>(a, s);
  else if (a.dim <= 1024ull * kForwardPer1)
    launch_forward<T, 1, kForwardPer1>(a, s);
  else
    launch_pdl(norm_forward_long_kernel<T>, (unsigned)a.rows, 1024, 0, s, a);
}

// Blocks of the backward pass, each with a row of partial sums: enough to fill
// 152 SMs, no more than there are rows. A function of the sizes alone, so that
// the workspace and the order of the sums do not depend on the device's state.
uint32_t backward_parts(uint64_t rows, uint64_t dim) {
  const uint32_t threads = threads_for(dim, kBackwardPer);
  uint64_t groups = rows, most = 152;
  if (threads == 32) {
    groups = (rows + 7) / 8;
    most = 152 * 4;
  } else if (threads <= 512) {
    most = 152ull * std::min(4u, 1024u / threads);
  }
  return (uint32_t)std::max<uint64_t>(1, std::min(groups, most));
}

template <typename T, int V>
void launch_backward(const NormGradArgs& a, uint32_t parts, cudaStream_t s) {
  constexpr int NV = kBackwardPer / V;
  const uint32_t threads = threads_for(a.dim, kBackwardPer);
  if (threads == 32)
    launch_pdl(norm_backward_kernel<T, V, NV, false, 256>, parts, 256, 2 * a.dim * sizeof(float),
               s, a);
  else if (threads <= 256)
    launch_pdl(norm_backward_kernel<T, V, NV, true, 256>, parts, threads, 0, s, a);
  else
    launch_pdl(norm_backward_kernel<T, V, NV, true, 512>, parts, threads, 0, s, a);
}

template <typename T>
void backward_typed(const NormGradArgs& a, uint32_t parts, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 &&
                   a.dx_stride % V == 0 && aligned_to(a.x, 16) && aligned_to(a.dy, 16) &&
                   aligned_to(a.dx, 16);
  if (a.dim > 512ull * kBackwardPer) {
    launch_pdl(norm_backward_long_kernel<T>, (unsigned)a.rows, 1024, 0, s, a);
    launch_pdl(norm_columns_kernel<T>, dim3((unsigned)((a.dim + 255) / 256), parts), 256, 0, s, a);
    note_launches(2);
    return;
  }
  if (vec)
    launch_backward<T, V>(a, parts, s);
  else
    launch_backward<T, 1>(a, parts, s);
  note_launches(1);
}

bool rows_ok(uint64_t rows, uint64_t dim) {
  return rows <= 0x7fffffffull && dim >= 1 && dim <= 0x7fffffffull;
}

}  // namespace
}  // namespace sparcml

using namespace sparcml;

extern "C" int sparcml_layer_norm(const void* x, int32_t type, int64_t x_stride, const void* weight,
                                  const void* bias, int32_t weight_type, uint64_t rows,
                                  uint64_t dim, float eps, void* y, int64_t y_stride, float* mean,
                                  float* rstd, void* stream) {
  const ApiRange nvtx_range(__func__);
  if (!type_ok(type) || !type_ok(weight_type) || !rows_ok(rows, dim) || !(eps >= 0.f))
    return SPARCML_ERR_INVALID_ARG;
  if (rows == 0) return SPARCML_OK;
  const size_t e = type_bytes(type), we = type_bytes(weight_type);
  if (!x || !y || !mean || !rstd || x_stride < 0 || (rows > 1 && y_stride < (int64_t)dim) ||
      !aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, we) || !aligned_to(bias, we))
    return SPARCML_ERR_INVALID_ARG;
  const NormArgs a{x,    x_stride, weight, bias, weight_type,
                   aligned_to(weight, 16) && aligned_to(bias, 16), rows, dim, eps, y,
                   rows > 1 ? y_stride : 0, mean, rstd};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == SPARCML_F32) forward_typed<float>(a, s);
  else if (type == SPARCML_BF16) forward_typed<__nv_bfloat16>(a, s);
  else forward_typed<__half>(a, s);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  note_launches(1);
  return SPARCML_OK;
}

extern "C" size_t sparcml_layer_norm_backward_workspace_size(uint64_t rows, uint64_t dim) {
  if (!rows_ok(rows, dim)) return 0;
  return 256 + align_up(2 * sizeof(float) * dim * backward_parts(rows, dim), 256);
}

extern "C" int sparcml_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                           int64_t x_stride, int32_t type, const void* weight,
                                           int32_t weight_type, const float* mean,
                                           const float* rstd, uint64_t rows, uint64_t dim,
                                           void* dx, int64_t dx_stride, float* dweight,
                                           float* dbias, int32_t accumulate, void* ws,
                                           size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  if (!type_ok(type) || !type_ok(weight_type) || !rows_ok(rows, dim) || !ws ||
      !aligned_to(ws, 256) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return SPARCML_ERR_INVALID_ARG;
  const size_t e = type_bytes(type);
  if (rows > 0 &&
      (!dy || !x || !mean || !rstd || !dx || dy_stride < 0 || x_stride < 0 ||
       (rows > 1 && dx_stride < (int64_t)dim) || !aligned_to(x, e) || !aligned_to(dy, e) ||
       !aligned_to(dx, e) || !aligned_to(weight, type_bytes(weight_type))))
    return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < sparcml_layer_norm_backward_workspace_size(rows, dim))
    return SPARCML_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint32_t parts = rows ? backward_parts(rows, dim) : 0;
  float* part_w = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  float* part_b = part_w + (uint64_t)parts * dim;
  if (rows) {
    const NormGradArgs a{dy,   dy_stride, x,   x_stride, weight, weight_type,
                         aligned_to(weight, 16), mean, rstd, rows, dim, dx,
                         rows > 1 ? dx_stride : 0, part_w, part_b};
    if (type == SPARCML_F32) backward_typed<float>(a, parts, s);
    else if (type == SPARCML_BF16) backward_typed<__nv_bfloat16>(a, parts, s);
    else backward_typed<__half>(a, parts, s);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  }
  if (dweight || dbias) {
    launch_pdl(norm_join_kernel, dim3((unsigned)((dim + 31) / 32), 2), 512, 0, s, part_w, part_b,
               parts, dim, dweight, dbias, accumulate);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  return SPARCML_OK;
}
