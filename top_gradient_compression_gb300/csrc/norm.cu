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

// Sum of two values over the `threads` threads that share a row: a warp, or a group of
// whole warps with a named barrier and 2 * 33 float2 of shared memory of its own. `turn`
// alternates between the halves of that from call to call, so that one barrier per
// call is enough.
__device__ __forceinline__ float2 row_sum(float2 v, uint32_t threads, uint32_t group,
                                          float2* scratch, uint32_t& turn) {
  v.x = warp_sum_f(v.x);
  v.y = warp_sum_f(v.y);
  if (threads == 32) return v;
  float2* s = scratch + 33 * (turn & 1u);
  ++turn;
  const uint32_t lane = lane_id(), nw = threads >> 5;
  if (lane == 0) s[(threadIdx.x >> 5) - group * nw] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
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
    // V = 4: one 16- or 8-byte access; V = 8: one of 16 bytes, or two
    if (type == SPARCML_F32) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + 4 * q);
        out[4 * q] = f.x; out[4 * q + 1] = f.y; out[4 * q + 2] = f.z; out[4 * q + 3] = f.w;
      }
    } else {
      uint32_t h[V / 2 ? V / 2 : 1];
      const uint16_t* p = static_cast<const uint16_t*>(w) + c;
      if constexpr (V == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        h[0] = q.x; h[1] = q.y; h[2] = q.z; h[3] = q.w;
      } else if constexpr (V == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        h[0] = q.x; h[1] = q.y;
      }
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float2 f = type == SPARCML_BF16 ? unpack2<__nv_bfloat16>(h[e]) : unpack2<__half>(h[e]);
        out[2 * e] = f.x;
        out[2 * e + 1] = f.y;
      }
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
// (j * threads + t) * V. A persistent grid: while a row is reduced and written, the next
// one is already on its way into registers, which keeps 64 to 96 KB per SM in flight
// (without it 16384 x 4096 bf16 took 62 us).
template <typename T, int V, int NV, bool BLOCK, int MINB>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128, MINB) norm_forward_kernel(const NormArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  uint32_t turn = 0;
  const uint32_t threads = BLOCK ? blockDim.x : 32u;
  const uint32_t t = BLOCK ? threadIdx.x : lane_id();
  const uint32_t per = BLOCK ? 1u : blockDim.x >> 5;
  const uint64_t step = (uint64_t)gridDim.x * per;
  uint64_t row = (uint64_t)blockIdx.x * per + (BLOCK ? 0u : threadIdx.x >> 5);
  const float inv = 1.0f / (float)a.dim;
  Raw<T, V> v[NV], next[NV];
  auto fetch = [&](Raw<T, V>(&to)[NV], uint64_t r) {
    const T* x = static_cast<const T*>(a.x) + (int64_t)r * a.x_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) to[j] = load_raw<T, V>(x + c);
    }
  };
  if (row < a.rows) fetch(next, row);
  for (; row < a.rows; row += step) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = next[j];
    if (row + step < a.rows) fetch(next, row + step);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((uint64_t)(j * threads + t) * V < a.dim) {
        float f[V];
        unpack<T, V>(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) s.x += f[i];
        v[j].forget();
      }
    const float mean = row_sum(s, threads, 0, scratch, turn).x * inv;
    s.x = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if ((uint64_t)(j * threads + t) * V < a.dim) {
        float f[V];
        unpack<T, V>(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = f[i] - mean;
          s.x += d * d;
        }
        v[j].forget();
      }
    const float var = row_sum(s, threads, 0, scratch, turn).x * inv;
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
        float w[V], b[V], f[V];
        load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
        load_affine<V>(a.b, a.w_type, a.vec_w, c, 0.f, b);
        unpack<T, V>(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd * w[i] + b[i];
        store_raw<T, V>(y + c, pack<T, V>(f));
      }
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
  const float mean = row_sum(s, blockDim.x, 0, scratch, turn).x * inv;
  s.x = 0.f;
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(x[c]) - mean;
    s.x += d * d;
  }
  const float rstd = 1.0f / sqrtf(row_sum(s, blockDim.x, 0, scratch, turn).x * inv + a.eps);
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
  float* part_w;  // [gridDim.x][dim] partial sums over the block's rows, or null
  float* part_b;
  uint32_t threads;  // that share a row
  uint32_t* ticket;  // null: norm_join_kernel joins the blocks' sums
  float* dweight;
  float* dbias;
  int32_t accumulate;
};

// A block's groups of `threads` threads walk the rows; each thread keeps the running dw and
// db of its own columns in registers, so x and dy are read once for dx, dw and db
// together. Rows of whole packs come through a ring in shared memory, in which each thread
// copies ahead and reads back its own packs alone, so the ring needs no barrier. At the
// end the groups' sums are joined in their order, and the blocks' by the last block to
// finish (`ticket`, few sums) or by norm_join_kernel. Every order is fixed.
constexpr int kRing = 3;

template <typename T, int V, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
norm_backward_kernel(const NormGradArgs a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float2 scratch[8 * 66];
  __shared__ uint32_t last;
  uint32_t turn = 0;
  const uint32_t threads = a.threads, groups = blockDim.x / threads;
  const uint32_t group = threadIdx.x / threads, t = threadIdx.x - group * threads;
  float gw[NV][V], gb[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) gw[j][i] = gb[j][i] = 0.f;
  }
  const float inv = 1.0f / (float)a.dim;
  const uint64_t step = (uint64_t)gridDim.x * groups;
  const uint64_t row0 = (uint64_t)blockIdx.x * groups + group;
  auto fetch = [&](uint64_t row, uint32_t slot) {
    if (row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + (int64_t)row * a.x_stride;
      const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
      uint8_t* to = dynamic + ((uint64_t)slot * 2 * NV * blockDim.x + threadIdx.x) * 16;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint64_t c = (uint64_t)(j * threads + t) * V;
        if (c < a.dim) {
          cp_async16(to + (uint64_t)j * blockDim.x * 16, x + c);
          cp_async16(to + (uint64_t)(NV + j) * blockDim.x * 16, dy + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (V > 1) {
#pragma unroll
    for (int k = 0; k < kRing - 1; ++k) fetch(row0 + k * step, k);
  }
  uint32_t slot = 0;
  for (uint64_t row = row0; row < a.rows; row += step) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    Raw<T, V> vx[NV], vd[NV];
    if constexpr (V > 1) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      const uint8_t* from = dynamic + ((uint64_t)slot * 2 * NV * blockDim.x + threadIdx.x) * 16;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        vx[j].w = *reinterpret_cast<const uint4*>(from + (uint64_t)j * blockDim.x * 16);
        vd[j].w = *reinterpret_cast<const uint4*>(from + (uint64_t)(NV + j) * blockDim.x * 16);
      }
      fetch(row + (kRing - 1) * step, slot == 0 ? kRing - 1 : slot - 1);
      slot = slot + 1 == kRing ? 0 : slot + 1;
    } else {
      const T* x = static_cast<const T*>(a.x) + (int64_t)row * a.x_stride;
      const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint64_t c = (uint64_t)(j * threads + t) * V;
        if (c < a.dim) {
          vx[j] = load_raw<T, V>(x + c);
          vd[j] = load_raw<T, V>(dy + c);
        }
      }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) {
        float w[V], g[V], f[V];
        load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
        unpack<T, V>(vd[j], g);
        unpack<T, V>(vx[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (f[i] - mean) * rstd;
          gw[j][i] += g[i] * xh;
          gb[j][i] += g[i];
          s.x += g[i] * w[i];
          s.y += g[i] * w[i] * xh;
        }
        vx[j].forget();
        vd[j].forget();
      }
    }
    s = row_sum(s, threads, group, scratch + 66 * group, turn);
    const float c1 = s.x * inv, c2 = s.y * inv;
    T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(j * threads + t) * V;
      if (c < a.dim) {
        float w[V], g[V], f[V];
        load_affine<V>(a.w, a.w_type, a.vec_w, c, 1.f, w);
        unpack<T, V>(vd[j], g);
        unpack<T, V>(vx[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i)
          f[i] = rstd * (g[i] * w[i] - c1 - (f[i] - mean) * rstd * c2);
        store_raw<T, V>(dx + c, pack<T, V>(f));
      }
    }
  }
  if (a.part_w == nullptr) return;  // neither sum is wanted
  float* to_w = a.part_w + (uint64_t)blockIdx.x * a.dim;
  float* to_b = a.part_b + (uint64_t)blockIdx.x * a.dim;
  if (groups > 1) {
    float* join = reinterpret_cast<float*>(dynamic);  // [2][dim]
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    for (uint32_t k = 0; k < groups; ++k) {
      if (group == k) {
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
      to_w[c] = join[c];
      to_b[c] = join[a.dim + c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint64_t c = (uint64_t)(j * threads + t) * V + i;
        if (c < a.dim) {
          to_w[c] = gw[j][i];
          to_b[c] = gb[j][i];
        }
      }
    }
  }
  if (a.ticket == nullptr) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (uint32_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    float w = 0.f, b = 0.f;
#pragma unroll 4
    for (uint32_t p = 0; p < gridDim.x; ++p) {
      w += __ldcg(a.part_w + (uint64_t)p * a.dim + c);
      b += __ldcg(a.part_b + (uint64_t)p * a.dim + c);
    }
    if (a.dweight) a.dweight[c] = a.accumulate ? a.dweight[c] + w : w;
    if (a.dbias) a.dbias[c] = a.accumulate ? a.dbias[c] + b : b;
  }
  if (threadIdx.x == 0) *a.ticket = 0;  // as the next call needs it
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
  s = row_sum(s, blockDim.x, 0, scratch, turn);
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

constexpr uint32_t kSms = 152;

template <typename T, int V, int NV, bool BLOCK, int MINB>
void launch_forward(const NormArgs& a, cudaStream_t s) {
  const uint32_t threads = BLOCK ? threads_for(a.dim, V * NV) : 128;
  const uint64_t work = BLOCK ? a.rows : (a.rows + 3) / 4;
  const uint32_t fit = kSms * (BLOCK ? std::max(1u, std::min(16u, 1024 / threads)) : MINB);
  launch_pdl(norm_forward_kernel<T, V, NV, BLOCK, MINB>, (unsigned)std::min<uint64_t>(work, fit),
             threads, 0, s, a);
}

// Packs of 16 bytes need 16-byte aligned rows and a whole number of packs; other rows
// are read element by element. A warp takes a row of up to 16 packs per lane, which needs
// no barrier; a block takes longer ones.
template <typename T>
void forward_typed(const NormArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.x_stride % V == 0 && a.y_stride % V == 0 &&
                   aligned_to(a.x, 16) && aligned_to(a.y, 16);
  const uint64_t packs = a.dim / V;
  if (vec && packs <= 32) launch_forward<T, V, 1, false, 11>(a, s);
  else if (vec && packs <= 64) launch_forward<T, V, 2, false, 10>(a, s);
  else if (vec && packs <= 128) launch_forward<T, V, 4, false, 7>(a, s);
  else if (vec && packs <= 256) launch_forward<T, V, 8, false, 4>(a, s);
  else if (vec && packs <= 512) launch_forward<T, V, 16, false, 3>(a, s);
  else if (vec && packs <= 4 * 1024) launch_forward<T, V, 4, true, 1>(a, s);
  else if (a.dim <= 32 * 16) launch_forward<T, 1, 16, false, 5>(a, s);
  else if (a.dim <= 1024 * 8) launch_forward<T, 1, 8, true, 1>(a, s);
  else launch_pdl(norm_forward_long_kernel<T>, (unsigned)a.rows, 1024, 0, s, a);
}

constexpr uint32_t kBackwardPer = 16;  // elements per thread

// Threads of a row and of a block, and the blocks, each with a row of partial sums:
// three blocks per SM, no more than there are rows. A function of the sizes alone, so
// that the workspace and the order of the sums do not depend on the device's state.
struct BackwardShape {
  uint32_t threads, block, parts;
};
BackwardShape backward_shape(uint64_t rows, uint64_t dim) {
  const uint32_t threads = (uint32_t)std::min<uint64_t>(512, threads_for(dim, kBackwardPer));
  const uint32_t groups = std::max(1u, 256 / threads);
  const uint64_t most = kSms * (threads <= 256 ? 3 : 1);
  return {threads, threads * groups,
          (uint32_t)std::max<uint64_t>(1, std::min((rows + groups - 1) / groups, most))};
}
// One block joins up to this many partial sums in less time than a launch takes.
constexpr uint64_t kTicketSums = 16 * 1024;

template <typename T, int V, int MAXT, int MINB>
bool launch_backward(const NormGradArgs& a, const BackwardShape& h, cudaStream_t s) {
  constexpr int NV = kBackwardPer / V;
  auto kernel = norm_backward_kernel<T, V, NV, MAXT, MINB>;
  const size_t ring = V > 1 ? (size_t)kRing * 2 * NV * h.block * 16 : 0;
  const size_t join = h.block > h.threads ? 2 * a.dim * sizeof(float) : 0;
  const size_t smem = std::max(ring, join);
  if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
  launch_pdl(kernel, h.parts, h.block, smem, s, a);
  return true;
}

template <typename T>
bool backward_typed(const NormGradArgs& a, const BackwardShape& h, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 &&
                   a.dx_stride % V == 0 && aligned_to(a.x, 16) && aligned_to(a.dy, 16) &&
                   aligned_to(a.dx, 16);
  if (a.dim > 512ull * kBackwardPer) {
    launch_pdl(norm_backward_long_kernel<T>, (unsigned)a.rows, 1024, 0, s, a);
    note_launches(1);
    if (a.part_w) {
      launch_pdl(norm_columns_kernel<T>, dim3((unsigned)((a.dim + 255) / 256), h.parts), 256, 0, s,
                 a);
      note_launches(1);
    }
    return true;
  }
  note_launches(1);
  if (h.block <= 256)
    return vec ? launch_backward<T, V, 256, sizeof(T) == 2 ? 3 : 2>(a, h, s)
               : launch_backward<T, 1, 256, 2>(a, h, s);
  return vec ? launch_backward<T, V, 512, 1>(a, h, s) : launch_backward<T, 1, 512, 1>(a, h, s);
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
  return 256 + align_up(2 * sizeof(float) * dim * backward_shape(rows, dim).parts, 256);
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
  const BackwardShape h = backward_shape(rows, dim);
  const bool sums = dweight || dbias;
  float* part_w = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  float* part_b = part_w + (uint64_t)h.parts * dim;
  bool joined = !sums;
  if (rows) {
    NormGradArgs a{dy, dy_stride, x, x_stride, weight, weight_type, aligned_to(weight, 16), mean,
                   rstd, rows, dim, dx, rows > 1 ? dx_stride : 0, sums ? part_w : nullptr, part_b,
                   h.threads, nullptr, dweight, dbias, accumulate};
    if (sums && dim <= 512ull * kBackwardPer && h.parts * dim <= kTicketSums) {
      a.ticket = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kTicketOffset);
      joined = true;
    }
    const bool ok = type == SPARCML_F32    ? backward_typed<float>(a, h, s)
                    : type == SPARCML_BF16 ? backward_typed<__nv_bfloat16>(a, h, s)
                                           : backward_typed<__half>(a, h, s);
    if (launch_status() != SPARCML_OK || !ok) return SPARCML_ERR_CUDA;
  }
  if (!joined) {
    launch_pdl(norm_join_kernel, dim3((unsigned)((dim + 31) / 32), 2), 512, 0, s, part_w, part_b,
               rows ? h.parts : 0u, dim, dweight, dbias, accumulate);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  return SPARCML_OK;
}
