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
// A lane's V elements from p, those from `left` on as zeros; `packs`: they are aligned.
template <typename T, int V = 16 / sizeof(T)>
__device__ __forceinline__ void load_piece(const T* p, int64_t left, bool packs, F2 (&f)[V / 2]) {
  if (packs && left >= V) {
    unpack<T, V>(load_raw<T, V>(p), f);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      f[i] = f2(2 * i < left ? to_f32(p[2 * i]) : 0.f,
                2 * i + 1 < left ? to_f32(p[2 * i + 1]) : 0.f);
  }
}
template <typename T, int V = 16 / sizeof(T)>
__device__ __forceinline__ void store_piece(T* p, int64_t left, bool packs,
                                            const F2 (&f)[V / 2]) {
  if (packs && left >= V) {
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

template <typename T, bool PACKS>
__global__ void __launch_bounds__(256) restore_kernel(const StoreArgs a) {
  griddep_wait();
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
      if (piece_column<V>(lane, q) < left) codes[q] = load_codes<V>(from + piece_column<V>(lane, q));
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint32_t c = piece_column<V>(lane, q);
      F2 f[V / 2];
      codes_f2<V>(codes[q], f);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[i] = mul2<true>(f[i], f2(scale, scale));
      if (c < left) store_piece<T>(y + c, left - c, PACKS, f);
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

// Sums of four values over the threads of a group, two values of each of two rows. `room`: of the
// group, [2][16][4] floats; `turn` alternates between its halves, so that one barrier is enough.
__device__ __forceinline__ void sum4(const Group& g, float* room, uint32_t turn, float (&v)[4]) {
  const uint32_t lane = lane_id();
  if (g.threads <= 32) {
    for (uint32_t d = g.threads / 2; d > 0; d >>= 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
    return;
  }
  // each half of the lanes goes on with half of the values: lane bits 4 and 3 say which one
  const bool up = lane & 16, right = lane & 8;
  const float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
  const float c = a + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
  const float d = b + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
  float e = (right ? d : c) + __shfl_xor_sync(0xffffffffu, right ? c : d, 8);
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) e += __shfl_xor_sync(0xffffffffu, e, k);
  room += 64 * (turn & 1u);
  const uint32_t warps = g.threads / 32;
  if ((lane & 7u) == 0) room[(g.t / 32) * 4 + lane / 8] = e;
  g.sync();
  // lane: value lane % 4 of warp lane / 4, and of warp lane / 4 + 8
  e = lane / 4 < warps ? room[lane] : 0.f;
  if (lane / 4 + 8 < warps) e += room[lane + 32];
#pragma unroll
  for (int k = 16; k > 2; k >>= 1) e += __shfl_xor_sync(0xffffffffu, e, k);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, e, i);
}

// Sixteen columns per thread, whose sums over the rows stay in its registers. Here the rows are
// whole, aligned pieces, which come through a ring in shared memory: a thread copies ahead and
// reads back its own pieces alone, so that the ring needs no barrier. Two rows are taken at a time
// and read from the ring twice, before and after their sums: what one row waits for, the
// reduction above all, the other fills. (One row at a time, kept in registers between, allows 16
// warps per SM and took 79 us for 16384 x 4096 bf16, whether its loads were ahead by one row or by
// three, and its arithmetic single or packed.) One block per SM, so that few partial sums are left.
constexpr int kTurns = 2;  // pairs of rows in the ring
template <typename T>
constexpr int kNorm8Threads = sizeof(T) == 2 ? 768 : 512;
template <typename T>
constexpr uint32_t kNorm8Slot = (sizeof(T) + 1) * kNorm8Threads<T> * 16;  // a row

template <typename T>
__global__ void __launch_bounds__(kNorm8Threads<T>, 1) norm8_backward_kernel(const Norm8Args a) {
  griddep_wait();
  constexpr int V = 16 / sizeof(T), Q = 16 / V, P = V / 2, MAXT = kNorm8Threads<T>;
  constexpr uint32_t kSlot = kNorm8Slot<T>;
  // [kTurns][2][Q of dy, 1 of codes][MAXT] of 16 bytes; weights [dim]
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float room[(MAXT / 64) * 128];
  const Group g = make_group(a.threads, nullptr);
  const uint32_t threads = a.threads, groups = blockDim.x / threads, t = g.t;
  const uint32_t dim = (uint32_t)a.dim, first = t / 8 * kGroup;
  const float inv = 1.0f / (float)dim;
  auto column = [&](int i) { return first + piece_column<V>(t & 7u, i / V) + i % V; };
  float* const weights = reinterpret_cast<float*>(dynamic + kTurns * 2 * kSlot);
  for (uint32_t c = threadIdx.x; c < dim; c += blockDim.x)
    weights[c] = a.w ? load_any(a.w, a.w_type, c) : 1.f;
  bool there[Q];
  F2 gw[Q][P], gb[Q][P];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    there[q] = column(q * V) < dim;
#pragma unroll
    for (int i = 0; i < P; ++i) gw[q][i] = gb[q][i] = f2(0.f, 0.f);
  }
  const uint64_t step = (uint64_t)gridDim.x * groups * 2;
  uint8_t* const mine = dynamic + threadIdx.x * 16;
  float mean_next[2] = {0.f, 0.f}, rstd_next[2] = {0.f, 0.f};
  uint32_t exp_next[2] = {0, 0};
  auto fetch = [&](uint64_t row0, uint32_t turn) {
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
      const uint64_t row = row0 + r;
      if (row >= a.rows) continue;
      const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride;
      const int8_t* x = a.codes + (int64_t)row * a.codes_stride;
      uint8_t* to = mine + (2 * turn + r) * kSlot;
#pragma unroll
      for (int q = 0; q < Q; ++q)
        if (there[q]) {
          cp_async16(to + q * MAXT * 16, dy + column(q * V));
          const uint32_t at =
              static_cast<uint32_t>(__cvta_generic_to_shared(to + Q * MAXT * 16 + q * V));
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at),
                       "l"(x + column(q * V)), "n"(V)
                       : "memory");
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch_small = [&](uint64_t row0) {
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r)
      if (row0 + r < a.rows) {
        mean_next[r] = a.mean[row0 + r];
        rstd_next[r] = a.rstd[row0 + r];
        if (first < dim)
          exp_next[r] = a.exponents[(int64_t)(row0 + r) * a.exponents_stride + first / kGroup];
      }
  };
  uint64_t base = (uint64_t)blockIdx.x * groups * 2;
  const uint64_t of = 2 * g.index;
#pragma unroll
  for (int k = 0; k < kTurns; ++k) fetch(base + of + k * step, k);
  fetch_small(base + of);
  __syncthreads();
  uint32_t turn = 0, sums = 0;
  for (; base < a.rows; base += step) {  // the same turns for all groups of threads
    const uint64_t row0 = base + of;
    F2 by[2], minus[2], r2[2];
    float rstd[2];
    bool active[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float scale = scale_of(exp_next[r]);
      rstd[r] = rstd_next[r];
      by[r] = f2(scale, scale);
      minus[r] = f2(-mean_next[r], -mean_next[r]);
      r2[r] = f2(rstd[r], rstd[r]);
      active[r] = row0 + r < a.rows;
    }
    fetch_small(row0 + step);
    // dy and xh of piece q of row r; c 2^e is exact, so its difference from the mean is rounded
    // once
    auto read = [&](int q, int r, F2(&d)[P], F2(&xh)[P]) {
      const uint8_t* from = mine + (2 * turn + r) * kSlot;
      Raw<T, V> raw;
      raw.w = *reinterpret_cast<const uint4*>(from + q * MAXT * 16);
      unpack<T, V>(raw, d);
      codes_f2<V>(load_codes<V>(reinterpret_cast<const int8_t*>(from + Q * MAXT * 16 + q * V)), xh);
#pragma unroll
      for (int i = 0; i < P; ++i) xh[i] = mul2<true>(fma2<true>(xh[i], by[r], minus[r]), r2[r]);
    };
    auto read_weights = [&](int q, F2(&w)[P]) {
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float4 f = *reinterpret_cast<const float4*>(weights + column(q * V) + 2 * i);
        w[i] = f2(f.x, f.y);
        w[i + 1] = f2(f.z, f.w);
      }
    };
    asm volatile("cp.async.wait_group %0;" ::"n"(kTurns - 1) : "memory");
    F2 s0[2], s1[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) s0[r] = s1[r] = f2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (!there[q]) continue;
      F2 w[P];
      read_weights(q, w);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!active[r]) continue;
        F2 d[P], xh[P];
        read(q, r, d, xh);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          gw[q][i] = fma2<true>(d[i], xh[i], gw[q][i]);
          gb[q][i] = add2<true>(gb[q][i], d[i]);
          d[i] = mul2<true>(d[i], w[i]);
          s0[r] = add2<true>(s0[r], d[i]);
          s1[r] = fma2<true>(d[i], xh[i], s1[r]);
        }
      }
    }
    float s[4] = {s0[0].x + s0[0].y, s1[0].x + s1[0].y, s0[1].x + s0[1].y, s1[1].x + s1[1].y};
    sum4(g, room + 128 * g.index, sums++, s);
    // dx = rstd (d - sum(d) / dim - xh sum(d xh) / dim)
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (!there[q]) continue;
      F2 w[P];
      read_weights(q, w);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (!active[r]) continue;
        const float k1 = -s[2 * r] * inv * rstd[r], k2 = -s[2 * r + 1] * inv * rstd[r];
        F2 d[P], xh[P];
        read(q, r, d, xh);
#pragma unroll
        for (int i = 0; i < P; ++i)
          d[i] = fma2<true>(xh[i], f2(k2, k2),
                            fma2<true>(mul2<true>(d[i], w[i]), r2[r], f2(k1, k1)));
        T* dx = static_cast<T*>(a.dx) + (int64_t)(row0 + r) * a.dx_stride;
        *reinterpret_cast<uint4*>(dx + column(q * V)) = pack<T, V>(d);
      }
    }
    fetch(row0 + kTurns * step, turn);
    turn = turn + 1 == kTurns ? 0 : turn + 1;
  }
  if (a.part_w == nullptr) return;  // neither sum is wanted
  asm volatile("cp.async.wait_all;" ::: "memory");
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
  float mean_next = 0.f, rstd_next = 0.f;
  auto fetch = [&](uint64_t row) {
    if (row >= a.rows) return;
    mean_next = a.mean[row];
    rstd_next = a.rstd[row];
  };
  uint64_t base = (uint64_t)blockIdx.x * groups;
  fetch(base + g.index);
  for (; base < a.rows; base += step) {  // the same turns for all groups of threads
    const uint64_t row = base + g.index;
    const int in = row < a.rows ? left : 0;
    const float mean = mean_next, rstd = rstd_next;
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

// One block per SM of as many groups of threads as fit, fewer where there are few rows; never more
// blocks than backward_shape has, by which the workspace is sized.
template <typename T>
bool launch_norm8(const Norm8Args& a, BackwardShape& h, cudaStream_t s) {
  auto kernel = norm8_backward_kernel<T>;
  const uint32_t least = std::max(1u, 256 / h.threads), most = kNorm8Threads<T> / h.threads;
  const uint32_t groups = (uint32_t)std::min<uint64_t>(
      most, std::max<uint64_t>(least, align_up((a.rows + 2 * kSms - 1) / (2 * kSms), least)));
  h.block = groups * h.threads;
  h.parts = (uint32_t)std::min<uint64_t>(kSms, (a.rows + 2 * groups - 1) / (2 * groups));
  const size_t smem = kTurns * 2 * kNorm8Slot<T> + a.dim * sizeof(float);
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
bool launch_norm8_shape(const Norm8Args& a, BackwardShape& h, bool packs, cudaStream_t s) {
  if (packs) return launch_norm8<T>(a, h, s);
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
  BackwardShape h = backward_shape(a.rows, a.dim);  // as launched, in the end
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
