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

// A row on its way into shared memory, as the aligned pieces of 16 bytes that cover it;
// element c comes to lie at slot + row_skew + c. What a first piece holds before the row
// is not used; where it could lie before the array, its elements are copied one by one.
template <typename T>
__device__ __forceinline__ uint32_t row_skew(const T* row) {
  return (uint32_t)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}
template <typename T>
__device__ __forceinline__ void copy_row(T* slot, const T* row, uint32_t dim, uint64_t before,
                                         const Group& g) {
  const uint32_t skew = row_skew(row), per = 16 / sizeof(T);
  const uint32_t pieces = (skew + dim + per - 1) / per;
  const T* start = row - skew;
  for (uint32_t p = g.t; p < pieces; p += g.threads) {
    if (p == 0 && before < skew) {
      for (uint32_t e = skew; e < min(per, skew + dim); ++e) slot[e] = start[e];
    } else {
      const uint32_t bytes = (uint32_t)min(16u, (skew + dim - p * per) * (uint32_t)sizeof(T));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(slot + p * per)),
                   "l"(start + p * per), "r"(bytes)
                   : "memory");
    }
  }
}
// Elements that a slot for such a row takes: the row, its skew and the last piece's rest.
__host__ __device__ constexpr uint32_t slot_elements(uint32_t dim, uint32_t bytes) {
  const uint32_t per = 16 / bytes;
  return (dim + 2 * per - 2) / per * per + per;
}

// V weights of type W at `at`, as fp32 pairs; `none` where there are none.
template <typename W, int V>
__device__ __forceinline__ void load_affine(bool there, const W* at, float none,
                                            F2 (&out)[V / 2]) {
  if (!there) {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) out[e] = f2(none, none);
    return;
  }
  if constexpr (sizeof(W) == 4) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const float4 f = *reinterpret_cast<const float4*>(at + 4 * q);
      out[2 * q] = f2(f.x, f.y);
      out[2 * q + 1] = f2(f.z, f.w);
    }
  } else {
    unpack<W, 8>(load_raw<W, 8>(at), out);
  }
}

// Columns of a thread: `first` and constant offsets from it, which the compiler folds into the
// accesses' addresses (with offsets from the number of threads, 16384 x 4095 bf16 took 48
// instructions per element). LANES neighbouring threads own LANES * NV * V columns in a row.
// Whole packs (V = 4 or 8): pack j of a thread is LANES packs after its pack j - 1. Else (V = 2)
// its pair j is two columns LANES apart, so that a warp's accesses are consecutive elements.
template <int V, int NV, int LANES>
__device__ __forceinline__ int first_column(uint32_t t) {
  return (int)((t / LANES) * (NV * LANES * V) + (t % LANES) * (V == 2 ? 1 : V));
}
template <int V, int LANES>
__device__ __forceinline__ constexpr int offset(int j, int i) {
  return V == 2 ? (2 * j + i) * LANES : j * LANES * V + i;
}
// A pack or pair to `to`, of whose row `left` columns are left.
template <typename T, int V, int LANES>
__device__ __forceinline__ void store_pack(T* to, int j, int left, const F2 (&f)[V / 2]) {
  if constexpr (V == 2) {
    const float2 p = split(f[0]);
    to[offset<V, LANES>(j, 0)] = from_f32<T>(p.x);
    if (offset<V, LANES>(j, 1) < left) to[offset<V, LANES>(j, 1)] = from_f32<T>(p.y);
  } else {
    *reinterpret_cast<uint4*>(to + offset<V, LANES>(j, 0)) = pack<T, V>(f);
  }
}
// Such a pair of a vector in shared memory; zero beyond its end.
template <typename T, int LANES>
__device__ __forceinline__ F2 pair_at(const T* v, int j, int left) {
  return f2(to_f32(v[offset<2, LANES>(j, 0)]),
            offset<2, LANES>(j, 1) < left ? to_f32(v[offset<2, LANES>(j, 1)]) : 0.f);
}

struct NormArgs {
  const void* x;
  int64_t x_stride;  // elements between rows
  const void* w;     // may be null: all ones
  const void* b;     // may be null: all zeros
  int32_t w_type;
  uint64_t rows;
  uint64_t dim;
  float eps;
  void* y;
  int64_t y_stride;
  float* mean;
  float* rstd;
  uint32_t threads;  // that share a row
  bool w_packs;      // long rows: weights of the rows' type, 16-byte aligned
};

// A persistent grid: while a row is reduced and written, the next one is already on its
// way, which keeps 64 to 96 KB per SM in flight. Rows of whole, aligned packs go into
// registers; others (V = 2) through shared memory, where the weights wait in fp32. (Loaded
// from memory one element at a time, 16384 x 4095 bf16 took 181 us.)
//
// In 16 bits no unit is busy all the time: 16384 x 4096 bf16 takes 49 us (0.81 of the copy rate),
// with 55 % of the issue slots filled and no pipe above 50 %, by the 12 warps of an SM that 160
// registers a thread allow (1,830 warp instructions per row, 460 issue cycles of the 700 that its
// bytes take); more warps would hide more latency. Each pass over a row converts it
// anew: fp32 copies of the row cost as much in registers as they save (48.2 us either way at
// 8192 x 8192). fp32 rows run at the copy rate less 7 %.
template <typename T, typename W, int V, int NV, int LANES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_forward_kernel(const NormArgs a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float2 scratch[MAXT >= 64 ? 66 * (MAXT / 64) : 1];
  constexpr bool PACKS = V > 2;
  constexpr int P = V / 2;
  Group g = make_group(a.threads, scratch);
  const uint32_t threads = a.threads, groups = blockDim.x / threads, dim = (uint32_t)a.dim;
  const uint32_t t = g.t;
  const uint64_t step = (uint64_t)gridDim.x * groups;
  const float inv = 1.0f / (float)dim;
  const int first = first_column<V, NV, LANES>(t), all = (int)dim - first;
  const T* xs = static_cast<const T*>(a.x);
  // V = 2: [2][dim] weights, then two slots for each group
  float* affine = reinterpret_cast<float*>(dynamic);
  const uint32_t slot_size = slot_elements(dim, sizeof(T));
  T* slots = reinterpret_cast<T*>(dynamic + (2 * dim * sizeof(float) + 15) / 16 * 16) +
             (uint64_t)g.index * 2 * slot_size;
  uint32_t turn = 0;
  Raw<T, V> v[NV], next[NV];
  auto fetch = [&](uint64_t row, uint32_t slot) {
    if (row < a.rows) {
      const T* x = xs + (int64_t)row * a.x_stride;
      if constexpr (PACKS) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (offset<V, LANES>(j, 0) < all)
            next[j] = load_raw<T, V>(x + first + offset<V, LANES>(j, 0));
      } else {
        copy_row(slots + slot * slot_size, x, dim, row * (uint64_t)a.x_stride, g);
      }
    }
    if constexpr (!PACKS) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (!PACKS) {
    for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x) {
      affine[c] = a.w ? load_any(a.w, a.w_type, c) : 1.f;
      affine[dim + c] = a.b ? load_any(a.b, a.w_type, c) : 0.f;
    }
  }
  uint64_t base = (uint64_t)blockIdx.x * groups;
  fetch(base + g.index, 0);
  if constexpr (!PACKS) __syncthreads();
  for (; base < a.rows; base += step) {  // the same turns for all groups
    const uint64_t row = base + g.index;
    const bool active = row < a.rows;
    const int left = active ? all : 0;
    if constexpr (PACKS) {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = next[j];
      fetch(row + step, 0);
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      g.sync();
      const T* x = slots + turn * slot_size + first +
                   (active ? row_skew(xs + (int64_t)row * a.x_stride) : 0);
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (offset<V, LANES>(j, 0) < left) v[j].w = pair_at<T, LANES>(x, j, left);
      turn ^= 1u;
      fetch(row + step, turn);
    }
    F2 s = f2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (offset<V, LANES>(j, 0) < left) {
        F2 f[P];
        unpack<T, V>(v[j], f);
        v[j].forget();
#pragma unroll
        for (int d = 1; d < P; d *= 2) {
#pragma unroll
          for (int i = 0; i < P; i += 2 * d) f[i] = add2<PACKS>(f[i], f[i + d]);
        }
        s = add2<PACKS>(s, f[0]);
      }
    const float mean = g.sum(split(s)) * inv;
    s = f2(0.f, 0.f);
    const F2 minus = f2(-mean, -mean);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (offset<V, LANES>(j, 0) < left) {
        F2 f[P], q = f2(0.f, 0.f);
        unpack<T, V>(v[j], f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f[i] = add2<PACKS>(f[i], minus);
          if (!PACKS && offset<V, LANES>(j, 1) >= left) f[i] = f2(split(f[i]).x, 0.f);
          q = fma2<PACKS>(f[i], f[i], q);
        }
        s = add2<PACKS>(s, q);
        v[j].forget();
      }
    const float var = g.sum(split(s)) * inv;
    const float rstd = rsqrtf(var + a.eps);
    if (!active) continue;
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    const F2 by = f2(rstd, rstd);
    T* y = static_cast<T*>(a.y) + (int64_t)row * a.y_stride + first;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (offset<V, LANES>(j, 0) < all) {
        F2 w[P], b[P], f[P];
        if constexpr (PACKS) {
          load_affine<W, V>(a.w, static_cast<const W*>(a.w) + first + offset<V, LANES>(j, 0), 1.f,
                            w);
          load_affine<W, V>(a.b, static_cast<const W*>(a.b) + first + offset<V, LANES>(j, 0), 0.f,
                            b);
        } else {
          w[0] = pair_at<float, LANES>(affine + first, j, all);
          b[0] = pair_at<float, LANES>(affine + dim + first, j, all);
        }
        unpack<T, V>(v[j], f);
#pragma unroll
        for (int i = 0; i < P; ++i)
          f[i] = fma2<PACKS>(mul2<PACKS>(add2<PACKS>(f[i], minus), by), w[i], b[i]);
        store_pack<T, V, LANES>(y, j, all, f);
      }
    }
  }
}

// Rows too long for a block's registers: the row is read again for each sum (from L2, where
// one row of any such length fits), in packs where it consists of them (V > 1).
template <typename T, int V>
__device__ __forceinline__ void load_floats(const T* p, uint64_t c, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = to_f32(p[c]);
  } else {
    F2 q[V / 2];
    unpack<T, V>(load_raw<T, V>(p + c), q);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i & 1 ? q[i / 2].y : q[i / 2].x;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_floats(T* p, uint64_t c, const float (&f)[V]) {
  if constexpr (V == 1) {
    p[c] = from_f32<T>(f[0]);
  } else {
    F2 q[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = f2(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(p + c) = pack<T, V>(q);
  }
}
// Weights at column c; `packs`: they have the rows' type and lie on 16 bytes. (Read one by one,
// the gradients of 4096 x 16384 bf16 took 205 us, and 183 so.)
template <typename T, int V>
__device__ __forceinline__ void weight_floats(const void* w, int32_t type, bool packs, uint64_t c,
                                              float none, float (&f)[V]) {
  if (packs && w) {
    load_floats<T, V>(static_cast<const T*>(w), c, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = w ? load_any(w, type, c + i) : none;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(1024, V == 8 ? 1 : 2) norm_forward_long_kernel(const NormArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  Group g = make_group(blockDim.x, scratch);
  const T* x = static_cast<const T*>(a.x) + (int64_t)blockIdx.x * a.x_stride;
  T* y = static_cast<T*>(a.y) + (int64_t)blockIdx.x * a.y_stride;
  const float inv = 1.0f / (float)a.dim;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
  for (uint64_t c = threadIdx.x * V; c < a.dim; c += blockDim.x * V) {
    float f[V];
    load_floats<T, V>(x, c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) (i & 1 ? s.y : s.x) += f[i];
  }
  const float mean = g.sum(s) * inv;
  s = make_float2(0.f, 0.f);
#pragma unroll 2
  for (uint64_t c = threadIdx.x * V; c < a.dim; c += blockDim.x * V) {
    float f[V];
    load_floats<T, V>(x, c, f);
#pragma unroll
    for (int i = 0; i < V; ++i) (i & 1 ? s.y : s.x) += (f[i] - mean) * (f[i] - mean);
  }
  const float rstd = rsqrtf(g.sum(s) * inv + a.eps);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = rstd;
  }
#pragma unroll 2
  for (uint64_t c = threadIdx.x * V; c < a.dim; c += blockDim.x * V) {
    float f[V], w[V], b[V];
    load_floats<T, V>(x, c, f);
    weight_floats<T, V>(a.w, a.w_type, a.w_packs, c, 1.f, w);
    weight_floats<T, V>(a.b, a.w_type, a.w_packs, c, 0.f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (f[i] - mean) * rstd * w[i] + b[i];
    store_floats<T, V>(y, c, f);
  }
}

struct NormGradArgs {
  const void* dy;
  int64_t dy_stride;
  const void* x;
  int64_t x_stride;
  const void* w;
  int32_t w_type;
  const float* mean;
  const float* rstd;
  uint64_t rows;
  uint64_t dim;
  void* dx;
  int64_t dx_stride;
  float* part_w;  // [gridDim.x][dim] partial sums over the block's rows, or null
  float* part_b;
  uint32_t threads;  // that share a row
  bool w_packs;      // as in NormArgs
  uint32_t* ticket;  // null: norm_join_kernel joins the blocks' sums
  float* dweight;
  float* dbias;
  int32_t accumulate;
};

// A block's groups of `threads` threads walk the rows; each thread keeps the running dw and
// db of its own columns in registers, so x and dy are read once for dx, dw and db
// together. Rows of whole, aligned packs come through a ring in shared memory, in which
// each thread copies ahead and reads back its own packs alone, so the ring needs no
// barrier; other rows (V = 2) as in the forward pass. At the
// end the groups' sums are joined, and then the blocks', by the last block to
// finish (`ticket`, few sums) or by norm_join_kernel. Every order is fixed.
constexpr int kRing = 3;

template <typename T, typename W, int V, int NV, int LANES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB)
norm_backward_kernel(const NormGradArgs a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float2 scratch[66 * (MAXT / 64)];
  __shared__ uint32_t last;
  Group g = make_group(a.threads, scratch);
  const uint32_t threads = a.threads, groups = blockDim.x / threads, t = g.t;
  const uint32_t dim = (uint32_t)a.dim;
  constexpr bool PACKS = V > 2;
  constexpr int P = V / 2;
  constexpr int kWide = sizeof(W) > sizeof(T) ? 2 : 1;  // 16-byte groups of weights per pack
  F2 gw[NV][P], gb[NV][P];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < P; ++i) gw[j][i] = gb[j][i] = f2(0.f, 0.f);
  }
  const float inv = 1.0f / (float)dim;
  const int first = first_column<V, NV, LANES>(t), all = (int)dim - first;
  const uint64_t step = (uint64_t)gridDim.x * groups;
  const T* xs = static_cast<const T*>(a.x);
  const T* ds = static_cast<const T*>(a.dy);
  // Packs: kRing slots of this thread's packs of x and dy; V = 2: [dim] weights, then two
  // slots for x and for dy of each group
  constexpr int kSlots = PACKS ? kRing : 2;
  float* weights = reinterpret_cast<float*>(dynamic);
  const uint32_t slot_size = slot_elements(dim, sizeof(T));
  T* slots = reinterpret_cast<T*>(dynamic + (dim * sizeof(float) + 15) / 16 * 16) +
             (uint64_t)g.index * 4 * slot_size;
  auto fetch = [&](uint64_t row, uint32_t slot) {
    if (row < a.rows) {
      const T* x = xs + (int64_t)row * a.x_stride;
      const T* dy = ds + (int64_t)row * a.dy_stride;
      if constexpr (PACKS) {
        uint8_t* to = dynamic + (slot * 2 * NV * MAXT + threadIdx.x) * 16;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int o = offset<V, LANES>(j, 0);
          if (o < all) {
            cp_async16(to + j * MAXT * 16, x + first + o);
            cp_async16(to + (NV + j) * MAXT * 16, dy + first + o);
          }
        }
      } else {
        copy_row(slots + (2 * slot) * slot_size, x, dim, row * (uint64_t)a.x_stride, g);
        copy_row(slots + (2 * slot + 1) * slot_size, dy, dim, row * (uint64_t)a.dy_stride, g);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if constexpr (!PACKS) {
    for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x)
      weights[c] = a.w ? load_any(a.w, a.w_type, c) : 1.f;
  }
  // a thread's weights stay in its registers
  Raw<W, V> own[PACKS ? NV : 1][PACKS ? kWide : 1];
  if constexpr (PACKS) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int o = offset<V, LANES>(j, 0);
#pragma unroll
      for (int q = 0; q < kWide; ++q)
        if (a.w && o < all)
          own[j][q].w =
              *reinterpret_cast<const uint4*>(static_cast<const W*>(a.w) + first + o + 4 * q);
    }
  }
  auto weights_at = [&](int j, F2(&w)[P]) {
    if constexpr (!PACKS) {
      w[0] = pair_at<float, LANES>(weights + first, j, all);
    } else if (a.w == nullptr) {
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = f2(1.f, 1.f);
    } else if constexpr (kWide == 1) {
      unpack<W, V>(own[j][0], w);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 f = own[j][q].w;
        w[2 * q] = f2(__uint_as_float(f.x), __uint_as_float(f.y));
        w[2 * q + 1] = f2(__uint_as_float(f.z), __uint_as_float(f.w));
      }
    }
  };
  uint64_t base = (uint64_t)blockIdx.x * groups;
  float next_mean = 0.f, next_rstd = 0.f;
  if (base + g.index < a.rows) {
    next_mean = a.mean[base + g.index];
    next_rstd = a.rstd[base + g.index];
  }
#pragma unroll
  for (int k = 0; k < kSlots - 1; ++k) fetch(base + g.index + k * step, k);
  if constexpr (!PACKS) __syncthreads();
  uint32_t slot = 0;
  for (; base < a.rows; base += step) {  // the same turns for all groups
    const uint64_t row = base + g.index;
    const bool active = row < a.rows;
    const int left = active ? all : 0;
    const float mean = next_mean, rstd = next_rstd;
    if (row + step < a.rows) {
      next_mean = a.mean[row + step];
      next_rstd = a.rstd[row + step];
    }
    Raw<T, V> vx[NV], vd[NV];
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
    if constexpr (PACKS) {
      const uint8_t* from = dynamic + (slot * 2 * NV * MAXT + threadIdx.x) * 16;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        vx[j].w = *reinterpret_cast<const uint4*>(from + j * MAXT * 16);
        vd[j].w = *reinterpret_cast<const uint4*>(from + (NV + j) * MAXT * 16);
      }
    } else {
      g.sync();
      const T* x = slots + (2 * slot) * slot_size + first;
      const T* dy = slots + (2 * slot + 1) * slot_size + first;
      if (active) {
        x += row_skew(xs + (int64_t)row * a.x_stride);
        dy += row_skew(ds + (int64_t)row * a.dy_stride);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (offset<V, LANES>(j, 0) < left) {
          vx[j].w = pair_at<T, LANES>(x, j, left);
          vd[j].w = pair_at<T, LANES>(dy, j, left);
        }
      }
    }
    fetch(row + (kSlots - 1) * step, slot == 0 ? kSlots - 1 : slot - 1);
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    F2 s0 = f2(0.f, 0.f), s1 = s0;
    const F2 minus = f2(-mean, -mean), by = f2(rstd, rstd);
    // 16-bit packs keep x - mean and dy w in fp32 for the second pass (82.6 us against 88.5 at
    // 16384 x 4096); fp32 ones and pairs have no registers left, or nothing to convert.
    constexpr bool KEEP = PACKS && sizeof(T) == 2;
    F2 xc[KEEP ? NV : 1][P], kept[KEEP ? NV : 1][P];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (offset<V, LANES>(j, 0) < left) {
        F2 w[P], d[P], f[P];
        weights_at(j, w);
        unpack<T, V>(vd[j], d);
        unpack<T, V>(vx[j], f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          f[i] = add2<false>(f[i], minus);
          const F2 xh = mul2<false>(f[i], by);
          gw[j][i] = fma2<false>(d[i], xh, gw[j][i]);
          gb[j][i] = add2<false>(gb[j][i], d[i]);
          d[i] = mul2<false>(d[i], w[i]);
          s0 = add2<false>(s0, d[i]);
          s1 = fma2<false>(d[i], xh, s1);
          if constexpr (KEEP) {
            xc[j][i] = f[i];
            kept[j][i] = d[i];
          }
        }
        vx[j].forget();
        vd[j].forget();
      }
    }
    const float2 t0 = split(s0), t1 = split(s1);
    const float2 s = g.sum2(make_float2(t0.x + t0.y, t1.x + t1.y));
    if (!active) continue;
    // dx = (x - mean) k2 + (d rstd + k1)
    const float k1s = -s.x * inv * rstd, k2s = -s.y * inv * rstd * rstd;
    const F2 k1 = f2(k1s, k1s), k2 = f2(k2s, k2s);
    T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride + first;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (offset<V, LANES>(j, 0) < all) {
        F2 w[P], d[P], f[P];
        if constexpr (!KEEP) {
          weights_at(j, w);
          unpack<T, V>(vd[j], d);
          unpack<T, V>(vx[j], f);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const F2 dv = KEEP ? kept[KEEP ? j : 0][i] : mul2<false>(d[i], w[i]);
          const F2 xv = KEEP ? xc[KEEP ? j : 0][i] : add2<false>(f[i], minus);
          f[i] = fma2<false>(xv, k2, fma2<false>(dv, by, k1));
        }
        store_pack<T, V, LANES>(dx, j, all, f);
      }
    }
  }
  if (a.part_w == nullptr) return;  // neither sum is wanted
  auto part = [](F2 v, int i) { return i & 1 ? split(v).y : split(v).x; };
  float* to_w = a.part_w + (uint64_t)blockIdx.x * a.dim;
  float* to_b = a.part_b + (uint64_t)blockIdx.x * a.dim;
  if (groups > 1) {
    // Groups that share a warp by shuffles, then a row of sums per warp or wider group, then
    // a thread per column. (One group after the other, 1025 x 64 took 25 us in all.)
    if (threads < 32) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float2 w = split(gw[j][i]), b = split(gb[j][i]);
          if (threads == 8) {
            Group::add<8>(w);
            Group::add<8>(b);
          }
          Group::add<16>(w);
          Group::add<16>(b);
          gw[j][i] = f2(w.x, w.y);
          gb[j][i] = f2(b.x, b.y);
        }
      }
    }
    const uint32_t sets = min(groups, blockDim.x / 32);
    float* join = reinterpret_cast<float*>(dynamic);  // [sets][2][dim]
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (threads >= 32 || lane_id() < threads) {
      float* set = join + (uint64_t)(threads < 32 ? threadIdx.x >> 5 : g.index) * 2 * dim;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; i += PACKS ? 4 : 1) {
          const uint32_t c = (uint32_t)(first + offset<V, LANES>(j, i));
          if (c >= dim) continue;
          if constexpr (PACKS) {
            const float2 w0 = split(gw[j][i / 2]), w1 = split(gw[j][i / 2 + 1]);
            const float2 b0 = split(gb[j][i / 2]), b1 = split(gb[j][i / 2 + 1]);
            *reinterpret_cast<float4*>(set + c) = make_float4(w0.x, w0.y, w1.x, w1.y);
            *reinterpret_cast<float4*>(set + dim + c) = make_float4(b0.x, b0.y, b1.x, b1.y);
          } else {
            set[c] = part(gw[j][0], i);
            set[dim + c] = part(gb[j][0], i);
          }
        }
      }
    }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x) {
      float w = 0.f, b = 0.f;
      for (uint32_t k = 0; k < sets; ++k) {
        w += join[2 * k * dim + c];
        b += join[(2 * k + 1) * dim + c];
      }
      to_w[c] = w;
      to_b[c] = b;
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t c = (uint32_t)(first + offset<V, LANES>(j, i));
        if (c < a.dim) {
          to_w[c] = part(gw[j][i / 2], i);
          to_b[c] = part(gb[j][i / 2], i);
        }
      }
    }
  }
  if (a.ticket == nullptr) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  // Slices of `span` threads, a column each, share the blocks' sums of a narrow row.
  const uint32_t span = min(blockDim.x, (dim + 31) / 32 * 32), slices = blockDim.x / span;
  const uint32_t slice = threadIdx.x / span;
  for (uint32_t c = threadIdx.x - slice * span; c < (dim + span - 1) / span * span; c += span) {
    float2 sum = make_float2(0.f, 0.f);
    if (c < dim && slice < slices) {
      for (uint32_t p = slice; p < gridDim.x; p += 8 * slices) {
        float2 v[8];  // on their way together
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          const uint64_t at = (uint64_t)(p + k * slices) * dim + c;
          const bool in = p + k * slices < gridDim.x;
          v[k] = in ? make_float2(__ldcg(a.part_w + at), __ldcg(a.part_b + at))
                    : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) {
          sum.x += v[k].x;
          sum.y += v[k].y;
        }
      }
    }
    if (slices > 1) {  // then span covers the row
      scratch[threadIdx.x] = sum;
      __syncthreads();
      for (uint32_t k = 1; k < slices && slice == 0; ++k) {
        sum.x += scratch[k * span + c].x;
        sum.y += scratch[k * span + c].y;
      }
    }
    if (c < dim && slice == 0) {
      if (a.dweight) a.dweight[c] = a.accumulate ? a.dweight[c] + sum.x : sum.x;
      if (a.dbias) a.dbias[c] = a.accumulate ? a.dbias[c] + sum.y : sum.y;
    }
  }
  if (threadIdx.x == 0) *a.ticket = 0;  // as the next call needs it
}

// Rows too long for a block's registers: dx by re-reading the row, the column sums by
// norm_columns_kernel.
template <typename T, int V>
__global__ void __launch_bounds__(1024, V == 8 ? 1 : 2)
norm_backward_long_kernel(const NormGradArgs a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  Group g = make_group(blockDim.x, scratch);
  const T* x = static_cast<const T*>(a.x) + (int64_t)blockIdx.x * a.x_stride;
  const T* dy = static_cast<const T*>(a.dy) + (int64_t)blockIdx.x * a.dy_stride;
  T* dx = static_cast<T*>(a.dx) + (int64_t)blockIdx.x * a.dx_stride;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  const float inv = 1.0f / (float)a.dim;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
  for (uint64_t c = threadIdx.x * V; c < a.dim; c += blockDim.x * V) {
    float f[V], d[V], w[V];
    load_floats<T, V>(x, c, f);
    load_floats<T, V>(dy, c, d);
    weight_floats<T, V>(a.w, a.w_type, a.w_packs, c, 1.f, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s.x += d[i] * w[i];
      s.y += d[i] * w[i] * ((f[i] - mean) * rstd);
    }
  }
  s = g.sum2(s);
  const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll 2
  for (uint64_t c = threadIdx.x * V; c < a.dim; c += blockDim.x * V) {
    float f[V], d[V], w[V];
    load_floats<T, V>(x, c, f);
    load_floats<T, V>(dy, c, d);
    weight_floats<T, V>(a.w, a.w_type, a.w_packs, c, 1.f, w);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = rstd * (d[i] * w[i] - c1 - (f[i] - mean) * rstd * c2);
    store_floats<T, V>(dx, c, f);
  }
}

// part[blockIdx.y][c] = sums over the rows blockIdx.y, blockIdx.y + gridDim.y, ... of x and dy
// as they were: this kernel runs before the one above, which may write dx over either.
template <typename T, int V>
__global__ void __launch_bounds__(128) norm_columns_kernel(const NormGradArgs a) {
  griddep_wait();
  const uint64_t c = ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= a.dim) return;
  float gw[V], gb[V];
#pragma unroll
  for (int i = 0; i < V; ++i) gw[i] = gb[i] = 0.f;
#pragma unroll 4
  for (uint64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    float f[V], d[V];
    load_floats<T, V>(static_cast<const T*>(a.dy) + (int64_t)r * a.dy_stride, c, d);
    load_floats<T, V>(static_cast<const T*>(a.x) + (int64_t)r * a.x_stride, c, f);
    const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      gw[i] += d[i] * ((f[i] - mean) * rstd);
      gb[i] += d[i];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a.part_w[(uint64_t)blockIdx.y * a.dim + c + i] = gw[i];
    a.part_b[(uint64_t)blockIdx.y * a.dim + c + i] = gb[i];
  }
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
uint32_t threads_for(uint64_t dim, uint32_t per) {
  return (uint32_t)((dim + 32ull * per - 1) / (32ull * per)) * 32u;
}

constexpr uint32_t kSms = 152;

// Threads of a block for a row beyond registers: two blocks of an SM, of 1024 threads where 32
// registers are enough, else (packs of eight) of 512 (4096 x 16384 bf16 161 us against 183 for
// the gradients with one block of 1024; fp32 229, against 251 with blocks of 512).
unsigned long_threads(int v, uint64_t rows) { return v == 8 && rows > kSms ? 512 : 1024; }

// `threads` for a row, blocks of at least `block` threads, `fit` of them per SM.
template <typename T, typename W, int V, int NV, int LANES, int MAXT, int MINB>
bool launch_forward(NormArgs a, uint32_t threads, uint32_t block, uint32_t fit, cudaStream_t s) {
  auto kernel = norm_forward_kernel<T, W, V, NV, LANES, MAXT, MINB>;
  a.threads = threads;
  const uint32_t groups = std::max(1u, block / threads);
  size_t smem = 0;
  if (V == 2) {
    smem = align_up(2 * a.dim * sizeof(float), 16) +
           2ull * groups * slot_elements((uint32_t)a.dim, sizeof(T)) * sizeof(T);
    if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem))
      return false;
    fit = (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(fit, 220 * 1024 / (smem + 2048)));
  }
  launch_pdl(kernel, (unsigned)std::min<uint64_t>((a.rows + groups - 1) / groups, kSms * fit),
             threads * groups, smem, s, a);
  return true;
}

// Up to 16 packs per lane a warp takes a row alone, which needs no barrier (2048 fp32
// columns: 53 us against 61 with four warps); longer ones take several. Shorter rows share a
// warp, four packs per lane: 65536 x 256 bf16 15 us, against 24 with a warp for a row, of
// which fewer are on their way at a time. For few rows the fewest steps count: 2432 x 256 bf16
// 2.0 us against 2.6, 4864 rows 3.3 against 3.0.
template <typename T, typename W>
bool forward_packs(const NormArgs& a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const uint64_t packs = a.dim / V;
  const bool few = a.rows <= 16 * kSms;
  if (packs <= 8) return launch_forward<T, W, V, 1, 8, 128, 10>(a, 8, 128, 10, s);
  if (few && packs <= 16) return launch_forward<T, W, V, 1, 16, 128, 10>(a, 16, 128, 10, s);
  if (few && packs <= 32) return launch_forward<T, W, V, 1, 32, 128, 10>(a, 32, 128, 10, s);
  if (packs <= 16) return launch_forward<T, W, V, 2, 8, 128, 8>(a, 8, 128, 8, s);
  if (few && packs <= 64) return launch_forward<T, W, V, 2, 32, 128, 8>(a, 32, 128, 8, s);
  if (packs <= 32) return launch_forward<T, W, V, 4, 8, 128, 7>(a, 8, 128, 7, s);
  if (packs <= 64) return launch_forward<T, W, V, 4, 16, 128, 7>(a, 16, 128, 7, s);
  if (packs <= 128) return launch_forward<T, W, V, 4, 32, 128, 7>(a, 32, 128, 7, s);
  if (packs <= 256) return launch_forward<T, W, V, 8, 32, 128, 4>(a, 32, 128, 4, s);
  if (packs <= 512) return launch_forward<T, W, V, 16, 32, 128, 3>(a, 32, 128, 3, s);
  const uint32_t threads = threads_for(packs, 4);
  if (packs <= 2048)
    return launch_forward<T, W, V, 4, 32, 512, 1>(a, threads, threads,
                                                  std::max(1u, 640 / threads), s);
  return launch_forward<T, W, V, 4, 32, 1024, 1>(a, threads, threads, 1, s);
}

// Whole packs: 16-byte aligned rows and weights of the rows' type or fp32. Everything else
// goes element by element.
template <typename T>
bool forward_typed(NormArgs a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.dim <= 4096 * V && a.x_stride % V == 0 &&
                   a.y_stride % V == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16) &&
                   aligned_to(a.w, 16) && aligned_to(a.b, 16);
  if (vec && (type_of<T>() == a.w_type || (!a.w && !a.b))) return forward_packs<T, T>(a, s);
  if (sizeof(T) == 2 && vec && a.w_type == SPARCML_F32) return forward_packs<T, float>(a, s);
  if (a.dim <= 512 * 16) {
    const uint32_t threads = threads_for(a.dim, 16);
    if (a.dim <= 128) return launch_forward<T, T, 2, 8, 8, 256, 3>(a, 8, 256, 3, s);
    if (a.dim <= 256) return launch_forward<T, T, 2, 8, 16, 256, 3>(a, 16, 256, 3, s);
    if (threads <= 256)
      return launch_forward<T, T, 2, 8, 32, 256, 3>(a, threads, 256, 3, s);
    return launch_forward<T, T, 2, 8, 32, 512, 1>(a, threads, threads, 2, s);
  }
  const bool wide = a.dim % V == 0 && a.x_stride % V == 0 && a.y_stride % V == 0 &&
                    aligned_to(a.x, 16) && aligned_to(a.y, 16);
  a.w_packs = type_of<T>() == a.w_type && aligned_to(a.w, 16) && aligned_to(a.b, 16);
  launch_pdl(wide ? norm_forward_long_kernel<T, V> : norm_forward_long_kernel<T, 1>,
             (unsigned)a.rows, long_threads(wide ? V : 1, a.rows), 0, s, a);
  return true;
}

constexpr uint32_t kBackwardPer = 16;  // elements per thread

// Threads of a row and of a block, and the blocks, each with a row of partial sums: what
// the registers of the SMs hold at one time (kFit blocks of 256 threads each; with a
// second, partial wave 16384 x 4096 fp32 took 271 us), no more than there are rows.
constexpr uint32_t kFit = 2;
struct BackwardShape {
  uint32_t threads, block, parts;
};
BackwardShape backward_shape(uint64_t rows, uint64_t dim) {
  const uint32_t threads = dim <= 128   ? 8
                           : dim <= 256 ? 16
                                        : (uint32_t)std::min<uint64_t>(
                                              512, threads_for(dim, kBackwardPer));
  const uint32_t groups = std::max(1u, 256 / threads);
  const uint64_t most = kSms * (threads <= 256 ? kFit : 1);
  return {threads, threads * groups,
          (uint32_t)std::max<uint64_t>(1, std::min((rows + groups - 1) / groups, most))};
}
// Up to this many partial sums the last block to finish joins them: that saves the host a
// launch, 2 us of a call that waits for the host (10.7 against 12.7 at every size up to 16 K
// sums), and costs time on the device, ticket against launch: 450 sums 4.5 and 3.6 us, 2 K 5.3 and
// 3.8, 4 K 5.8 to 6.6 and 4.1, 6 K 7.1 and 4.0, 8 K 7.0 to 9.1 and 4.2, 16 K 9.6 to 11.8 and 4.3,
// 32 K 14 to 26 and 4.2 to 7.6. So it is worth it to a caller who is bound by launches up to where
// the device loses as much as the host gains, and to no other; rows of more than 1,024 columns
// lose it earlier (3 x 2048 fp32 9.0 and 4.4).
constexpr uint64_t kTicketSums = 4 * 1024;

template <typename T, typename W, int V, int LANES, int MAXT, int MINB>
bool launch_backward(const NormGradArgs& a, const BackwardShape& h, cudaStream_t s) {
  constexpr int NV = kBackwardPer / V;
  auto kernel = norm_backward_kernel<T, W, V, NV, LANES, MAXT, MINB>;
  const uint32_t groups = h.block / h.threads;
  const size_t ring = V > 2 ? (size_t)kRing * 2 * NV * MAXT * 16
                            : align_up(a.dim * sizeof(float), 16) +
                                  4ull * groups * slot_elements((uint32_t)a.dim, sizeof(T)) *
                                      sizeof(T);
  const size_t join = groups > 1 ? 2 * std::min(groups, h.block / 32) * a.dim * sizeof(float) : 0;
  const size_t smem = std::max(ring, join);
  if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
  launch_pdl(kernel, h.parts, h.block, smem, s, a);
  return true;
}

template <typename T, typename W, int V>
bool launch_backward_shape(const NormGradArgs& a, const BackwardShape& h, cudaStream_t s) {
  if (h.threads == 8) return launch_backward<T, W, V, 8, 256, kFit>(a, h, s);
  if (h.threads == 16) return launch_backward<T, W, V, 16, 256, kFit>(a, h, s);
  if (h.block <= 256) return launch_backward<T, W, V, 32, 256, kFit>(a, h, s);
  return launch_backward<T, W, V, 32, 512, 1>(a, h, s);
}

template <typename T>
bool backward_typed(NormGradArgs a, bool sums, uint8_t* ws, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.dim % V == 0 && a.x_stride % V == 0 && a.dy_stride % V == 0 &&
                   a.dx_stride % V == 0 && aligned_to(a.x, 16) && aligned_to(a.dy, 16) &&
                   aligned_to(a.dx, 16) && aligned_to(a.w, 16);
  const bool same = type_of<T>() == a.w_type || !a.w;
  const bool packs = vec && (same || a.w_type == SPARCML_F32);
  const bool longer = a.dim > 512ull * kBackwardPer;
  const BackwardShape h = backward_shape(a.rows, a.dim);
  a.threads = h.threads;
  a.part_w = sums ? reinterpret_cast<float*>(ws + 256) : nullptr;
  a.part_b = reinterpret_cast<float*>(ws + 256) + (uint64_t)h.parts * a.dim;
  const bool ticket = sums && !longer && h.parts * a.dim <= kTicketSums;
  if (ticket) a.ticket = reinterpret_cast<uint32_t*>(ws + kTicketOffset);
  bool ok = true;
  a.w_packs = same && aligned_to(a.w, 16);
  if (longer) {
    // the column sums first: dx may be written over x or dy
    const unsigned across = (unsigned)((a.dim + 128 * V - 1) / (128 * V));
    if (sums && vec)
      launch_pdl(norm_columns_kernel<T, V>, dim3(across, h.parts), 128, 0, s, a);
    else if (sums)
      launch_pdl(norm_columns_kernel<T, 1>, dim3((unsigned)((a.dim + 127) / 128), h.parts), 128, 0,
                 s, a);
    launch_pdl(vec ? norm_backward_long_kernel<T, V> : norm_backward_long_kernel<T, 1>,
               (unsigned)a.rows, long_threads(vec ? V : 1, a.rows), 0, s, a);
  } else if (packs && same) {
    ok = launch_backward_shape<T, T, V>(a, h, s);
  } else if (sizeof(T) == 2 && packs) {
    ok = launch_backward_shape<T, float, V>(a, h, s);
  } else {
    ok = launch_backward_shape<T, T, 2>(a, h, s);
  }
  const bool join = sums && !ticket;
  if (join)
    launch_pdl(norm_join_kernel, dim3((unsigned)((a.dim + 31) / 32), 2), 512, 0, s, a.part_w,
               a.part_b, h.parts, a.dim, a.dweight, a.dbias, a.accumulate);
  note_launches(1 + (longer && sums) + join);
  return ok;
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
      !aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, we) || !aligned_to(bias, we) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return SPARCML_ERR_INVALID_ARG;
  const NormArgs a{x,   x_stride, weight,   bias, weight_type, rows,
                   dim, eps,      y,        rows > 1 ? y_stride : 0, mean, rstd, 0, false};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ok = type == SPARCML_F32    ? forward_typed<float>(a, s)
                  : type == SPARCML_BF16 ? forward_typed<__nv_bfloat16>(a, s)
                                         : forward_typed<__half>(a, s);
  if (launch_status() != SPARCML_OK || !ok) return SPARCML_ERR_CUDA;
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
       !aligned_to(dx, e) || !aligned_to(weight, type_bytes(weight_type)) ||
       !aligned_to(mean, 4) || !aligned_to(rstd, 4)))
    return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < sparcml_layer_norm_backward_workspace_size(rows, dim))
    return SPARCML_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sums = dweight || dbias;
  if (rows) {
    const NormGradArgs a{dy,   dy_stride, x,    x_stride, weight, weight_type, mean,
                         rstd, rows,      dim,  dx,       rows > 1 ? dx_stride : 0,
                         nullptr, nullptr, 0,   false, nullptr, dweight, dbias, accumulate};
    uint8_t* w = static_cast<uint8_t*>(ws);
    const bool ok = type == SPARCML_F32    ? backward_typed<float>(a, sums, w, s)
                    : type == SPARCML_BF16 ? backward_typed<__nv_bfloat16>(a, sums, w, s)
                                           : backward_typed<__half>(a, sums, w, s);
    return launch_status() == SPARCML_OK && ok ? SPARCML_OK : SPARCML_ERR_CUDA;
  }
  if (sums) {  // of no rows
    launch_pdl(norm_join_kernel, dim3((unsigned)((dim + 31) / 32), 2), 512, 0, s,
               static_cast<const float*>(nullptr), static_cast<const float*>(nullptr), 0u, dim,
               dweight, dbias, accumulate);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  return SPARCML_OK;
}
