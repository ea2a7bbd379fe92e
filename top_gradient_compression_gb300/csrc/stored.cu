// Activations kept in 8 bits between the forward and the backward pass, and the layer norm's
// gradients from them.
//
// A group of 128 columns of a row has one exponent e, the least with max |x| 2^-e < 127.5, and an
// element the code c = rint(x 2^-e): it stands for c 2^e. A scale that is a power of two costs at
// most one of the eight bits against max |x| / 127, and in return c 2^e is a bf16, an fp16 and an
// fp32 number: what reads it can use it as it is, the tensor cores included, and rounds nothing a
// second time. All that is done here is exact but for that one rounding.
//
// Writing, reading back and the gradients are bound by memory: e + 1 bytes per element, the same,
// and 2 e + 1.

#include "rows.cuh"
#include "stored.cuh"

namespace sparcml {
namespace {

// An octet of lanes has a group of 128 columns, a lane sixteen of them: 16 / V pieces of V, the 16
// bytes of an access, so that the octet's accesses are whole stretches of 128 bytes.
template <int V>
__device__ __forceinline__ uint32_t piece_column(uint32_t octet_lane, int q) {
  return 8 * V * q + V * octet_lane;
}
// A lane's V elements to p, those before `left` alone where that is less.
template <typename T, int V = 16 / sizeof(T)>
__device__ __forceinline__ void store_piece(T* p, int64_t left, const F2 (&f)[V / 2]) {
  if (left >= V) {
    *reinterpret_cast<uint4*>(p) = pack<T, V>(f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) p[i] = from_f32<T>(i & 1 ? f[i / 2].y : f[i / 2].x);
  }
}
// V codes, as one access.
template <int V>
struct Codes {
  uint32_t w[V / 4];
};
template <int V>
__device__ __forceinline__ Codes<V> load_codes(const int8_t* p) {
  Codes<V> c;
  if constexpr (V == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x;
    c.w[1] = v.y;
  } else {
    c.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return c;
}
template <int V>
__device__ __forceinline__ void store_codes(int8_t* p, const Codes<V>& c) {
  if constexpr (V == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = c.w[0];
}
template <int V>
__device__ __forceinline__ void codes_f2(const Codes<V>& c, F2 (&f)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    f[i] = f2(code_at(c.w[i / 2], 2 * i % 4), code_at(c.w[i / 2], 2 * i % 4 + 1));
}

struct StoreArgs {
  void* x;  // read by the writing of codes, written by reading them back
  int64_t x_stride;
  uint64_t rows, dim;
  int8_t* codes;
  int64_t codes_stride;
  uint8_t* exponents;
  int64_t exponents_stride;
  uint32_t groups;  // of a row
};

// Where an octet of lanes is in the sequence of all groups; neighbouring octets take
// neighbouring groups, a warp four of them at a time.
struct GroupWalk {
  uint64_t row, rows_on;
  uint32_t group, groups, groups_on;
  __device__ __forceinline__ explicit GroupWalk(uint32_t per_row) : groups(per_row) {
    const uint64_t octet = ((uint64_t)blockIdx.x * blockDim.x + threadIdx.x) / 8;
    const uint64_t on = (uint64_t)gridDim.x * blockDim.x / 8;
    row = octet / groups;
    group = (uint32_t)(octet - row * groups);
    rows_on = on / groups;
    groups_on = (uint32_t)(on - rows_on * groups);
  }
  __device__ __forceinline__ void next() {
    row += rows_on;
    group += groups_on;
    if (group >= groups) {
      group -= groups;
      ++row;
    }
  }
};

// The exponent byte of a group whose largest magnitude has these bits as a float: with m = 1.f
// 2^p, 64 2^(p - e) 1.f is below 127.5 for e = p - 6 where 1.f is below 255 / 128. `least` and
// `most` keep every c 2^e a finite number of the type.
__device__ __forceinline__ uint32_t exponent_byte(uint32_t bits, int least, int most) {
  if (bits >= 0x7f800000u) return kNanExponent;
  const int b = (int)(bits >> 23) - 6 + ((bits & 0x7fffffu) >= 0x7f0000u);
  return (uint32_t)min(max(b, least), most);
}

// The largest of the magnitudes' bits in a word of two 16-bit elements, or in an fp32.
template <typename T>
__device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t w) {
  if constexpr (sizeof(T) == 4) return max(a, w & 0x7fffffffu);
  return __vmaxu2(a, w & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t float_bits(uint32_t a) {
  if constexpr (sizeof(T) == 4) return a;
  a = max(a & 0xffffu, a >> 16);
  if constexpr (std::is_same_v<T, __nv_bfloat16>) return a << 16;
  return __float_as_uint(__half2float(__ushort_as_half((uint16_t)a)));
}

// What an octet of lanes has of a group: its elements, and the largest of their bits.
template <typename T, bool PACKS>
struct Loaded {
  static constexpr int V = 16 / sizeof(T), Q = 16 / V;
  Raw<T, V> r[Q];
  __device__ __forceinline__ void load(const T* x, uint32_t lane, int64_t left) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t c = piece_column<V>(lane, q);
      if (PACKS && left >= c + V) {
        r[q] = load_raw<T, V>(x + c);
      } else {
        Pack<T, V> e;
#pragma unroll
        for (int i = 0; i < V; ++i) e.e[i] = c + i < left ? x[c + i] : from_f32<T>(0.f);
        r[q].w = *reinterpret_cast<const uint4*>(&e);
      }
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      t = largest<T>(largest<T>(largest<T>(largest<T>(t, r[q].w.x), r[q].w.y), r[q].w.z), r[q].w.w);
    return float_bits<T>(t);
  }
};

template <typename T, bool PACKS>
__global__ void __launch_bounds__(256) store_kernel(const StoreArgs a) {
  griddep_wait();
  constexpr bool kHalf = std::is_same_v<T, __half>;
  constexpr int V = 16 / sizeof(T), Q = 16 / V;
  constexpr int kLeast = kHalf ? 103 : 1, kMost = kHalf ? 136 : 248;
  const uint32_t lane = lane_id() & 7u;
  auto write = [&](const GroupWalk& at, const Loaded<T, PACKS>& x) {
    const bool active = at.row < a.rows;
    const uint64_t c0 = (uint64_t)at.group * kGroup;
    const int64_t left = active ? (int64_t)(a.dim - c0) : 0;
    uint32_t top = x.top();
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const uint32_t b = exponent_byte(top, kLeast, kMost);
    const bool fine = b != kNanExponent;
    const float scale = __uint_as_float((fine ? 254u - b : 127u) << 23);  // 2^-e
    const F2 by = f2(scale, scale), magic = f2(12582912.f, 12582912.f);  // 1.5 2^23
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      F2 f[V / 2];
      unpack<T, V>(x.r[q], f);
      if (b == (uint32_t)kMost) {  // the largest step, of which there may be more than 127
        const float most = 127.f / scale;
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
          f[i] = f2(fminf(fmaxf(f[i].x, -most), most), fminf(fmaxf(f[i].y, -most), most));
      }
      Codes<V> codes;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        // the product is exact, the sum rounds it to a whole number, in the low byte
        const F2 lo = fma2<true>(f[2 * k], by, magic), hi = fma2<true>(f[2 * k + 1], by, magic);
        const uint32_t w =
            __byte_perm(__byte_perm(__float_as_uint(lo.x), __float_as_uint(lo.y), 0x0040),
                        __byte_perm(__float_as_uint(hi.x), __float_as_uint(hi.y), 0x0040), 0x5410);
        codes.w[k] = fine ? w : 0u;
      }
      // the row's padding to whole 16 bytes is written as zeros
      const uint32_t c = piece_column<V>(lane, q);
      if (left > 0 && c < (uint32_t)(left >= kGroup ? kGroup : (left + 15) / 16 * 16))
        store_codes<V>(a.codes + (int64_t)at.row * a.codes_stride + c0 + c, codes);
    }
    if (active && lane == 0)
      a.exponents[(int64_t)at.row * a.exponents_stride + at.group] = (uint8_t)b;
  };
  auto load = [&](const GroupWalk& at, Loaded<T, PACKS>& x) {
    const uint64_t c0 = (uint64_t)at.group * kGroup;
    x.load(static_cast<const T*>(a.x) + (int64_t)at.row * a.x_stride + c0, lane,
           at.row < a.rows ? (int64_t)(a.dim - c0) : 0);
  };
  // Every lane of a warp takes part in its shuffles: the warp goes on while any octet has work. The
  // next group is on its way while one is written.
  GroupWalk at(a.groups), next = at;
  Loaded<T, PACKS> x, y;
  load(at, x);
  while (__any_sync(0xffffffffu, at.row < a.rows)) {
    next.next();
    load(next, y);
    write(at, x);
    at = next;
    next.next();
    load(next, x);
    write(at, y);
    at = next;
  }
}

// Rows that start anywhere are written element by element, neighbouring lanes neighbouring ones: by a
// warp, the groups of its octets two at a time: 16384 x 4095 bf16 takes 74 us, 1237 x 777 fp32 with
// its writing of codes 6.2. (Each octet its own, eight elements of a lane after one another, 234 and
// 6.6; one group at a time 74 and 8.4, all four at once 78 and 6.0.)
template <typename T>
__device__ __forceinline__ void restore_any(const StoreArgs& a) {
  const uint32_t lane = lane_id();
  GroupWalk at(a.groups);
  for (; __any_sync(0xffffffffu, at.row < a.rows); at.next()) {
#pragma unroll 1
    for (int first = 0; first < 32; first += 16) {
      T* y[2];
      int64_t left[2];
      uint32_t e[2];
      int8_t codes[2][4];  // all on their way at once
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint64_t row = __shfl_sync(0xffffffffu, at.row, first + 8 * k);
        const uint32_t group = __shfl_sync(0xffffffffu, at.group, first + 8 * k);
        const uint64_t c0 = (uint64_t)group * kGroup;
        left[k] = row < a.rows ? (int64_t)(a.dim - c0) : 0;
        y[k] = static_cast<T*>(a.x) + (int64_t)row * a.x_stride + c0;
        const int8_t* from = a.codes + (int64_t)row * a.codes_stride + c0;
        if (left[k] > 0) e[k] = a.exponents[(int64_t)row * a.exponents_stride + group];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < left[k]) codes[k][i] = from[lane + 32 * i];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (lane + 32 * i < left[k])
            y[k][lane + 32 * i] = from_f32<T>((float)codes[k][i] * scale_of(e[k]));
      }
    }
  }
}

template <typename T, bool PACKS>
__global__ void __launch_bounds__(256) restore_kernel(const StoreArgs a) {
  griddep_wait();
  if constexpr (!PACKS) return restore_any<T>(a);
  constexpr int V = 16 / sizeof(T), Q = 16 / V;
  GroupWalk at(a.groups);
  const uint32_t lane = lane_id() & 7u;
  for (; at.row < a.rows; at.next()) {
    const uint64_t c0 = (uint64_t)at.group * kGroup;
    const int64_t left = (int64_t)(a.dim - c0);
    const int8_t* from = a.codes + (int64_t)at.row * a.codes_stride + c0;
    const float scale =
        scale_of(a.exponents[(int64_t)at.row * a.exponents_stride + at.group]);
    T* y = static_cast<T*>(a.x) + (int64_t)at.row * a.x_stride + c0;
    Codes<V> codes[Q] = {};
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (piece_column<V>(lane, q) < left)
        codes[q] = load_codes<V>(from + piece_column<V>(lane, q));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t c = piece_column<V>(lane, q);
      F2 f[V / 2];
      codes_f2<V>(codes[q], f);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[i] = mul2<true>(f[i], f2(scale, scale));
      if (c < left) store_piece<T>(y + c, left - c, f);
    }
  }
}

// ---------------------------------------------------------------------------
// The layer norm's gradients.

struct Norm8Args {
  const void* dy;
  int64_t dy_stride;
  const int8_t* codes;
  int64_t codes_stride;
  const uint8_t* exponents;
  int64_t exponents_stride;
  const void* w;
  int32_t w_type;
  const float* mean;
  const float* rstd;
  uint64_t rows, dim;
  void* dx;
  int64_t dx_stride;
  float* part_w;  // [gridDim.x][dim] partial sums over the block's rows, or null
  float* part_b;
  uint32_t threads;  // that share a row
};

// The sums of a block's rows: of its groups of threads one after the other, in shared memory
// (`join`: [groups][2][dim]), or as they are. `column(i)`: of the thread's i-th sum.
template <typename F>
__device__ __forceinline__ void write_sums(const Norm8Args& a, const Group& g, uint32_t groups,
                                           float* join, const float (&gw)[16],
                                           const float (&gb)[16], F column) {
  const uint32_t dim = (uint32_t)a.dim;
  float* to_w = a.part_w + (uint64_t)blockIdx.x * a.dim;
  float* to_b = a.part_b + (uint64_t)blockIdx.x * a.dim;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (column(i) < dim) {
        to_w[column(i)] = gw[i];
        to_b[column(i)] = gb[i];
      }
    return;
  }
  __syncthreads();
  float* set = join + (uint64_t)g.index * 2 * dim;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (column(i) < dim) {
      set[column(i)] = gw[i];
      set[dim + column(i)] = gb[i];
    }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x) {
    float sw = 0.f, sb = 0.f;
    for (uint32_t k = 0; k < groups; ++k) {
      sw += join[2 * k * dim + c];
      sb += join[(2 * k + 1) * dim + c];
    }
    to_w[c] = sw;
    to_b[c] = sb;
  }
}

// Sixteen columns per thread, whose sums over the rows stay in its registers, as do its weights.
// Here the rows are whole, aligned pieces, which come through a ring in shared memory: a thread
// copies ahead and reads back its own pieces alone, so that the ring needs no barrier.
//
// 16384 x 4096 bf16 takes 70 us, 4.8 TB/s: half of the issue slots are filled by the 16 warps of an
// SM that 127 registers allow (its traffic alone takes 57 in this shape). What it took to come from
// 79 was fewer instructions, 46 to 35 million: pointers that go on by a stride in place of a
// product each, rows and columns that do not exist as zeros in place of branches, and sums over a
// row by half the shuffles. Not faster: what was read kept in place of the floats made of it (80
// registers, 24 warps), two rows at a time, a row's result in the turn after that of its sums (76),
// arithmetic single in place of packed, three rows in the ring (71) or five.
constexpr int kRing = 4;

// The sums of two values over a row's threads. Of more than a warp: the halves of a warp add up one
// of the values each, and all threads add up the warps' sums, of WARPS at most (those that are not
// there are zeros, which the group's scratch, [2][16], holds from the start).
template <int WARPS>
__device__ __forceinline__ F2 row_sums(Group& g, float2 v) {
  if (g.threads <= 32) {
    v = g.sum2(v);
    return f2(v.x, v.y);
  }
  const uint32_t lane = lane_id();
  const bool second = lane & 16;
  float u = second ? v.y : v.x;
  u += __shfl_xor_sync(0xffffffffu, second ? v.x : v.y, 16);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) u += __shfl_xor_sync(0xffffffffu, u, d);
  float2* s = g.scratch + 16 * (g.turn & 1u);
  ++g.turn;
  if ((lane & 15u) == 0) reinterpret_cast<float*>(s)[g.t / 16] = u;
  g.sync();
  F2 sum = f2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < WARPS; k += 2) {
    const float4 two = *reinterpret_cast<const float4*>(s + k);
    sum = add2<true>(sum, add2<true>(f2(two.x, two.y), f2(two.z, two.w)));
  }
  return sum;
}

template <typename T, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm8_backward_kernel(const Norm8Args a) {
  griddep_wait();
  constexpr int V = 16 / sizeof(T), Q = 16 / V, P = V / 2;
  // [kRing][Q of dy, 1 of codes][MAXT] of 16 bytes
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ alignas(16) float2 scratch[32 * (MAXT / 8)];
  const uint32_t threads = a.threads, groups = blockDim.x / threads;
  for (uint32_t i = threadIdx.x; i < 32 * groups; i += blockDim.x)
    scratch[i] = make_float2(0.f, 0.f);
  __syncthreads();
  const uint32_t index = threadIdx.x / threads, t = threadIdx.x - index * threads;
  Group g = {threads, index, t, scratch + 32 * index, 0};
  const uint32_t dim = (uint32_t)a.dim, rows = (uint32_t)a.rows, first = t / 8 * kGroup;
  const float inv = 1.0f / (float)dim;
  auto column = [&](int i) { return first + piece_column<V>(t & 7u, i / V) + i % V; };
  bool there[Q];
  F2 w[Q][P], gw[Q][P], gb[Q][P];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    there[q] = column(q * V) < dim;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t c = column(q * V + 2 * i);
      gw[q][i] = gb[q][i] = f2(0.f, 0.f);
      w[q][i] = a.w && there[q] ? f2(load_any(a.w, a.w_type, c), load_any(a.w, a.w_type, c + 1))
                                : f2(1.f, 1.f);
    }
  }
  const uint32_t step = gridDim.x * groups;
  constexpr uint32_t kSlot = (Q + 1) * MAXT * 16;
  uint8_t* const mine = dynamic + threadIdx.x * 16;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  float mean_of[kRing], rstd_of[kRing];
  uint32_t exp_of[kRing];
  // Rows are read in order, kRing - 1 ahead; what is not there, of a row or of rows, as zeros, so
  // that its turn adds nothing to any sum.
  uint32_t base = blockIdx.x * groups, next = base + index;
  const T* dy = static_cast<const T*>(a.dy) + (int64_t)next * a.dy_stride + column(0);
  const int8_t* x = a.codes + (int64_t)next * a.codes_stride + column(0);
  const uint8_t* e = a.exponents + (int64_t)next * a.exponents_stride + first / kGroup;
  T* dx = static_cast<T*>(a.dx) + (int64_t)next * a.dx_stride + column(0);
  const int64_t dy_on = step * a.dy_stride, x_on = step * a.codes_stride,
                e_on = step * a.exponents_stride, dx_on = step * a.dx_stride;
  auto fetch = [&](uint32_t slot, float& mean, float& rstd, uint32_t& exponent) {
    const bool active = next < rows;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t to = ring + slot * kSlot + q * MAXT * 16;
      const bool here = active && there[q];
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                   "l"(dy + 8 * V * q), "r"(here ? 16 : 0)
                   : "memory");
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                       ring + slot * kSlot + Q * MAXT * 16 + q * V),
                   "l"(x + 8 * V * q), "n"(V), "r"(here ? V : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    mean = rstd = 0.f;
    exponent = 0;
    if (active) {
      mean = a.mean[next];
      rstd = a.rstd[next];
      if (there[0]) exponent = *e;
    }
    next += step;
    dy += dy_on;
    x += x_on;
    e += e_on;
  };
#pragma unroll
  for (int k = 0; k < kRing - 1; ++k) fetch(k, mean_of[k], rstd_of[k], exp_of[k]);
  // A row, whose small parts are the k-th; those of the one that is fetched become the `later`-th.
  auto turn = [&](uint32_t slot, uint32_t free, int k, int later) {
    const bool active = base + index < rows;
    const float mean = mean_of[k], rstd = rstd_of[k], scale = scale_of(exp_of[k]);
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    const F2 by = f2(scale, scale), minus = f2(-mean, -mean), r2 = f2(rstd, rstd);
    F2 xh[Q][P], d[Q][P], s0 = f2(0.f, 0.f), s1 = s0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint8_t* from = mine + slot * kSlot;
      Raw<T, V> raw;
      raw.w = *reinterpret_cast<const uint4*>(from + q * MAXT * 16);
      unpack<T, V>(raw, d[q]);
      codes_f2<V>(load_codes<V>(reinterpret_cast<const int8_t*>(from + Q * MAXT * 16 + q * V)),
                  xh[q]);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // c 2^e is exact, and so its difference from the mean is rounded once
        xh[q][i] = mul2<true>(fma2<true>(xh[q][i], by, minus), r2);
        gw[q][i] = fma2<true>(d[q][i], xh[q][i], gw[q][i]);
        gb[q][i] = add2<true>(gb[q][i], d[q][i]);
        d[q][i] = mul2<true>(d[q][i], w[q][i]);
        s0 = add2<true>(s0, d[q][i]);
        s1 = fma2<true>(d[q][i], xh[q][i], s1);
      }
    }
    fetch(free, mean_of[later], rstd_of[later], exp_of[later]);
    const F2 s = row_sums<MAXT / 32>(g, make_float2(s0.x + s0.y, s1.x + s1.y));
    // dx = rstd (d - sum(d) / dim - xh sum(d xh) / dim)
    const float k1s = -s.x * inv * rstd, k2s = -s.y * inv * rstd;
    const F2 k1 = f2(k1s, k1s), k2 = f2(k2s, k2s);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        d[q][i] = fma2<true>(xh[q][i], k2, fma2<true>(d[q][i], r2, k1));
      if (active && there[q])
        *reinterpret_cast<uint4*>(dx + 8 * V * q) = pack<T, V>(d[q]);
    }
    dx += dx_on;
  };
  // The same turns for all groups of threads. In 16 bits the ring's turns are written out, so that
  // no small part has to be there before its row's turn to be handed on; in fp32 that makes four
  // times the code slower (16384 x 4096: 105 us in place of 95).
  if constexpr (sizeof(T) == 2) {
    while (base < rows) {
#pragma unroll
      for (int k = 0; k < kRing; ++k) {
        if (base >= rows) break;
        turn(k, (k + kRing - 1) % kRing, k, (k + kRing - 1) % kRing);
        base += step;
      }
    }
  } else {
    for (uint32_t slot = 0; base < rows; base += step) {
      const uint32_t free = slot == 0 ? kRing - 1 : slot - 1;
      turn(slot, free, 0, kRing - 1);
#pragma unroll
      for (int k = 0; k < kRing - 1; ++k) {
        mean_of[k] = mean_of[k + 1];
        rstd_of[k] = rstd_of[k + 1];
        exp_of[k] = exp_of[k + 1];
      }
      slot = slot + 1 == kRing ? 0 : slot + 1;
    }
  }
  // also the zeros in place of rows behind the last one have to have come before the block leaves
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (a.part_w == nullptr) return;  // neither sum is wanted
  float fw[16], fb[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const F2 u = gw[i / V][i % V / 2], v = gb[i / V][i % V / 2];
    fw[i] = i & 1 ? u.y : u.x;
    fb[i] = i & 1 ? v.y : v.x;
  }
  write_sums(a, g, groups, reinterpret_cast<float*>(dynamic), fw, fb, column);
}

// Any width, stride and alignment, element by element: a thread's columns are LANES apart, so
// that neighbouring threads read neighbouring elements.
template <typename T, int LANES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm8_backward_any_kernel(const Norm8Args a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float2 scratch[66 * (MAXT / 64)];
  Group g = make_group(a.threads, scratch);
  const uint32_t threads = a.threads, groups = blockDim.x / threads, t = g.t;
  const uint32_t dim = (uint32_t)a.dim;
  const float inv = 1.0f / (float)dim;
  const uint32_t first = t / LANES * (16 * LANES) + t % LANES;
  const int left = (int)dim - (int)first;
  auto column = [&](int i) { return first + i * LANES; };
  float w[16], gw[16], gb[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    gw[i] = gb[i] = 0.f;
    w[i] = a.w && i * LANES < left ? load_any(a.w, a.w_type, column(i)) : 1.f;
  }
  const uint64_t step = (uint64_t)gridDim.x * groups;
  constexpr int kScales = LANES / 8;  // groups of 128 that the columns lie in
  float mean_of = 0.f, rstd_of = 0.f;
  auto fetch = [&](uint64_t row) {
    if (row >= a.rows) return;
    mean_of = a.mean[row];
    rstd_of = a.rstd[row];
  };
  uint64_t base = (uint64_t)blockIdx.x * groups;
  fetch(base + g.index);
  for (; base < a.rows; base += step) {  // the same turns for all groups of threads
    const uint64_t row = base + g.index;
    const int in = row < a.rows ? left : 0;
    const float mean = mean_of, rstd = rstd_of;
    const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
    const int8_t* x = a.codes + (int64_t)row * a.codes_stride;
    const uint8_t* e = a.exponents + (int64_t)row * a.exponents_stride;
    float xh[16], d[16], scale[kScales];
#pragma unroll
    for (int k = 0; k < kScales; ++k)
      scale[k] = k * kGroup < in ? scale_of(e[first / kGroup + k]) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const bool there = i * LANES < in;
      d[i] = there ? to_f32(dy[column(i)]) : 0.f;
      xh[i] = there ? ((float)x[column(i)] * scale[i * kScales / 16] - mean) * rstd : 0.f;
    }
    fetch(row + step);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      gw[i] += d[i] * xh[i];
      gb[i] += d[i];
      d[i] *= w[i];
      s.x += d[i];
      s.y += d[i] * xh[i];
    }
    s = g.sum2(s);
    const float k1 = -s.x * inv * rstd, k2 = -s.y * inv * rstd;
    T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i * LANES < in) dx[column(i)] = from_f32<T>(xh[i] * k2 + (d[i] * rstd + k1));
  }
  if (a.part_w == nullptr) return;  // neither sum is wanted
  write_sums(a, g, groups, reinterpret_cast<float*>(dynamic), gw, gb, column);
}

// Rows too long for a block's registers: dx by reading the row twice, the column sums by a
// kernel of their own before it (dx may be written over dy).
__device__ __forceinline__ float stored_at(const Norm8Args& a, uint64_t row, uint64_t c) {
  return (float)a.codes[(int64_t)row * a.codes_stride + c] *
         scale_of(a.exponents[(int64_t)row * a.exponents_stride + c / kGroup]);
}
template <typename T>
__global__ void __launch_bounds__(1024, 2) norm8_backward_long_kernel(const Norm8Args a) {
  griddep_wait();
  __shared__ float2 scratch[66];
  Group g = make_group(blockDim.x, scratch);
  const uint64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
  T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride;
  const float mean = a.mean[row], rstd = a.rstd[row], inv = 1.0f / (float)a.dim;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll 4
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (a.w ? load_any(a.w, a.w_type, c) : 1.f);
    s.x += d;
    s.y += d * ((stored_at(a, row, c) - mean) * rstd);
  }
  s = g.sum2(s);
  const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll 4
  for (uint64_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
    const float d = to_f32(dy[c]) * (a.w ? load_any(a.w, a.w_type, c) : 1.f);
    dx[c] = from_f32<T>(rstd * (d - c1 - (stored_at(a, row, c) - mean) * rstd * c2));
  }
}
template <typename T>
__global__ void __launch_bounds__(128) norm8_columns_kernel(const Norm8Args a) {
  griddep_wait();
  const uint64_t c = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.dim) return;
  float gw = 0.f, gb = 0.f;
#pragma unroll 4
  for (uint64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float d = to_f32(static_cast<const T*>(a.dy)[(int64_t)r * a.dy_stride + c]);
    gw += d * ((stored_at(a, r, c) - a.mean[r]) * a.rstd[r]);
    gb += d;
  }
  a.part_w[(uint64_t)blockIdx.y * a.dim + c] = gw;
  a.part_b[(uint64_t)blockIdx.y * a.dim + c] = gb;
}

template <typename T, int MAXT, int MINB>
bool launch_norm8(const Norm8Args& a, const BackwardShape& h, cudaStream_t s) {
  auto kernel = norm8_backward_kernel<T, MAXT, MINB>;
  const uint32_t groups = h.block / h.threads;
  const size_t ring = (size_t)kRing * (sizeof(T) + 1) * MAXT * 16;
  const size_t join = groups > 1 ? (size_t)2 * groups * a.dim * sizeof(float) : 0;
  const size_t smem = std::max(ring, join);
  if (!ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
  launch_pdl(kernel, h.parts, h.block, smem, s, a);
  return true;
}
template <typename T, int LANES, int MAXT, int MINB>
bool launch_norm8_any(const Norm8Args& a, const BackwardShape& h, cudaStream_t s) {
  auto kernel = norm8_backward_any_kernel<T, LANES, MAXT, MINB>;
  const uint32_t groups = h.block / h.threads;
  const size_t smem = groups > 1 ? 2ull * groups * a.dim * sizeof(float) : 0;
  if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
  launch_pdl(kernel, h.parts, h.block, smem, s, a);
  return true;
}
template <typename T>
bool launch_norm8_shape(const Norm8Args& a, const BackwardShape& h, bool packs, cudaStream_t s) {
  if (packs && h.block <= 256) return launch_norm8<T, 256, kFit>(a, h, s);
  if (packs) return launch_norm8<T, 512, 1>(a, h, s);
  if (h.threads == 8) return launch_norm8_any<T, 8, 256, kFit>(a, h, s);
  if (h.threads == 16) return launch_norm8_any<T, 16, 256, kFit>(a, h, s);
  if (h.block <= 256) return launch_norm8_any<T, 32, 256, kFit>(a, h, s);
  return launch_norm8_any<T, 32, 512, 1>(a, h, s);
}

template <typename T>
bool norm8_typed(Norm8Args a, float* dweight, float* dbias, int32_t accumulate, uint8_t* ws,
                 cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool packs = a.dim % V == 0 && a.dy_stride % V == 0 && a.dx_stride % V == 0 &&
                     aligned_to(a.dy, 16) && aligned_to(a.dx, 16);
  const bool sums = dweight || dbias;
  const BackwardShape h = backward_shape(a.rows, a.dim);
  a.threads = h.threads;
  a.part_w = sums ? reinterpret_cast<float*>(ws + 256) : nullptr;
  a.part_b = reinterpret_cast<float*>(ws + 256) + (uint64_t)h.parts * a.dim;
  bool ok = true;
  const bool longer = a.dim > 512ull * kBackwardPer;
  if (longer) {
    if (sums)
      launch_pdl(norm8_columns_kernel<T>, dim3((unsigned)((a.dim + 127) / 128), h.parts), 128, 0,
                 s, a);
    launch_pdl(norm8_backward_long_kernel<T>, (unsigned)a.rows, 1024, 0, s, a);
  } else {
    ok = launch_norm8_shape<T>(a, h, packs, s);
  }
  if (sums)
    launch_pdl(join_columns_kernel, dim3((unsigned)((a.dim + 31) / 32), 2), 512, 0, s, a.part_w,
               a.part_b, h.parts, a.dim, dweight, dbias, accumulate);
  note_launches(1 + (longer && sums) + sums);
  return ok;
}

// A block's eight warps take 32 groups at a time; four of them per SM's 2,048 threads twice over.
unsigned store_grid(uint64_t rows, uint32_t groups) {
  return (unsigned)std::min<uint64_t>((rows * groups + 31) / 32, kSms * 8);
}
uint64_t groups_of(uint64_t dim) { return (dim + kGroup - 1) / kGroup; }
bool sizes_ok(uint64_t rows, uint64_t dim) {
  return rows <= 0x7fffffffull && dim >= 1 && dim <= 0x7fffffffull;
}
// The 8-bit form: 16-byte aligned rows with room for whole 16 bytes.
bool stored_ok(const int8_t* codes, int64_t codes_stride, const uint8_t* exponents,
               int64_t exponents_stride, uint64_t dim) {
  return codes && exponents && aligned_to(codes, 16) && codes_stride % 16 == 0 &&
         codes_stride >= (int64_t)align_up(dim, 16) && exponents_stride >= (int64_t)groups_of(dim);
}

template <typename T>
void store_typed(const StoreArgs& a, bool restore, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool packs = aligned_to(a.x, 16) && a.x_stride % V == 0;
  auto kernel = restore ? (packs ? restore_kernel<T, true> : restore_kernel<T, false>)
                        : (packs ? store_kernel<T, true> : store_kernel<T, false>);
  launch_pdl(kernel, store_grid(a.rows, a.groups), 256, 0, s, a);
}

int store_or_restore(const StoreArgs& a, int32_t type, bool restore, cudaStream_t s) {
  if (type == SPARCML_F32) store_typed<float>(a, restore, s);
  else if (type == SPARCML_BF16) store_typed<__nv_bfloat16>(a, restore, s);
  else store_typed<__half>(a, restore, s);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  note_launches(1);
  return SPARCML_OK;
}

}  // namespace
}  // namespace sparcml

using namespace sparcml;

extern "C" int sparcml_checkpoint8(const void* x, int32_t type, int64_t x_stride, uint64_t rows,
                                   uint64_t dim, int8_t* codes, int64_t codes_stride,
                                   uint8_t* exponents, int64_t exponents_stride, void* stream) {
  const ApiRange nvtx_range(__func__);
  if (!type_ok(type) || !sizes_ok(rows, dim)) return SPARCML_ERR_INVALID_ARG;
  if (rows == 0) return SPARCML_OK;
  if (!x || !aligned_to(x, type_bytes(type)) || x_stride < 0 ||
      !stored_ok(codes, codes_stride, exponents, exponents_stride, dim))
    return SPARCML_ERR_INVALID_ARG;
  const StoreArgs a{const_cast<void*>(x), x_stride,  rows,      dim, codes,
                    codes_stride,         exponents, exponents_stride, (uint32_t)groups_of(dim)};
  return store_or_restore(a, type, false, static_cast<cudaStream_t>(stream));
}

extern "C" int sparcml_restore8(const int8_t* codes, int64_t codes_stride,
                                const uint8_t* exponents, int64_t exponents_stride, uint64_t rows,
                                uint64_t dim, void* y, int32_t type, int64_t y_stride,
                                void* stream) {
  const ApiRange nvtx_range(__func__);
  if (!type_ok(type) || !sizes_ok(rows, dim)) return SPARCML_ERR_INVALID_ARG;
  if (rows == 0) return SPARCML_OK;
  if (!y || !aligned_to(y, type_bytes(type)) || (rows > 1 && y_stride < (int64_t)dim) ||
      !stored_ok(codes, codes_stride, exponents, exponents_stride, dim))
    return SPARCML_ERR_INVALID_ARG;
  const StoreArgs a{y,
                    rows > 1 ? y_stride : 0,
                    rows,
                    dim,
                    const_cast<int8_t*>(codes),
                    codes_stride,
                    const_cast<uint8_t*>(exponents),
                    exponents_stride,
                    (uint32_t)groups_of(dim)};
  return store_or_restore(a, type, true, static_cast<cudaStream_t>(stream));
}

extern "C" int sparcml_layer_norm_backward8(
    const void* dy, int64_t dy_stride, int32_t type, const int8_t* codes, int64_t codes_stride,
    const uint8_t* exponents, int64_t exponents_stride, const void* weight, int32_t weight_type,
    const float* mean, const float* rstd, uint64_t rows, uint64_t dim, void* dx, int64_t dx_stride,
    float* dweight, float* dbias, int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  if (!type_ok(type) || !type_ok(weight_type) || !sizes_ok(rows, dim) || !ws ||
      !aligned_to(ws, 256) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4))
    return SPARCML_ERR_INVALID_ARG;
  const size_t e = type_bytes(type);
  if (rows > 0 &&
      (!dy || !mean || !rstd || !dx || dy_stride < 0 || (rows > 1 && dx_stride < (int64_t)dim) ||
       !aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(weight, type_bytes(weight_type)) ||
       !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
       !stored_ok(codes, codes_stride, exponents, exponents_stride, dim)))
    return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < sparcml_layer_norm_backward_workspace_size(rows, dim))
    return SPARCML_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // the sums of no rows
    if (!dweight && !dbias) return SPARCML_OK;
    launch_pdl(join_columns_kernel, dim3((unsigned)((dim + 31) / 32), 2), 512, 0, s,
               static_cast<const float*>(nullptr), static_cast<const float*>(nullptr), 0u, dim,
               dweight, dbias, accumulate);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
    return SPARCML_OK;
  }
  const Norm8Args a{dy,     dy_stride, codes, codes_stride, exponents, exponents_stride,
                    weight, weight_type, mean, rstd,        rows,      dim,
                    dx,     rows > 1 ? dx_stride : 0,       nullptr,   nullptr, 0};
  uint8_t* w = static_cast<uint8_t*>(ws);
  const bool ok = type == SPARCML_F32 ? norm8_typed<float>(a, dweight, dbias, accumulate, w, s)
                  : type == SPARCML_BF16
                      ? norm8_typed<__nv_bfloat16>(a, dweight, dbias, accumulate, w, s)
                      : norm8_typed<__half>(a, dweight, dbias, accumulate, w, s);
  return launch_status() == SPARCML_OK && ok ? SPARCML_OK : SPARCML_ERR_CUDA;
}
