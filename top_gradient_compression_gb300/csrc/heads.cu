// Norms of queries and keys, head by head, and the rotation by their positions in the same pass,
// forward and backward.
//
//   r = 1 / sqrt(mean(x^2) + eps),  u = x r w,  and each pair (u0, u1) of the head's first `turned`
//   elements turns by the angle p f_i of its position p: (u0 c - u1 s, u0 s + u1 c)
//   backward, with g the gradient turned back and xh = x r:
//   dx = r (g w - xh mean(g w xh)),  dw = sum over tokens and heads of g xh
//
// Both passes are bound by memory: an element is read and written once, backward two are read.
//
// A head belongs to L neighbouring lanes, each with the same pairs of elements whatever the head:
// both members of a pair are in one lane, so that the rotation exchanges nothing, and its weights
// stay in registers. A warp takes 32 / L heads of a token at a time, and many of one token's after
// another, for which the sines and cosines are worked out once.
//
// Angles. A frequency is kept as 64 bits of a turn, f / 2 pi 2^64, so that position times
// frequency modulo 2^64 is the angle without whole turns and without a rounding, however far the
// position: the error is 2^-64 of a turn times the position, for frequencies up to 2^40. Its upper
// 32 bits go to sincospif.

#include "rows.cuh"

namespace sparcml {
namespace {

constexpr uint32_t kWarps = 8;      // per block
constexpr uint32_t kMostDim = 512;  // elements of a head

struct Heads {  // an array [tokens][heads][dim]
  const void* p;
  int64_t token, head;  // strides in elements
};
struct Side {  // queries, or keys
  Heads x, g, out;  // g: the gradient of the result (backward)
  const void* w;    // may be null: all ones
  uint32_t heads, jobs;  // jobs of a token: 32 / L heads each
};
struct HeadArgs {
  Side side[2];
  uint64_t tokens;
  uint32_t dim, turned, units, lanes;  // units of V pairs each; L
  const void* positions;
  int32_t wide;  // positions are int64, else int32
  const float* freqs;
  int32_t w_type;
  float eps;
  uint32_t warps[2];  // of the grid, for each side
  float* part[2];     // [gridDim.x][dim] sums of dw, one array after the other; or null
};

// f / 2 pi of a turn, in 2^-64: the product with 1 / 2 pi in two parts, of which whole turns
// are dropped. What is left of the first one is at most half a turn of either sign, exactly.
__device__ __forceinline__ uint64_t turn_fraction(float freq) {
  const double inv = 0.15915494309189535, low = -9.839338337591243e-18;  // 1 / 2 pi = inv + low
  const double f = freq, hi = f * inv, rest = fma(f, inv, -hi) + f * low;
  const uint64_t a = (uint64_t)__double2ll_rn((hi - rint(hi)) * 0x1p64);
  return a + (uint64_t)__double2ll_rn(rest * 0x1p64);
}

// Where a unit's two pieces lie in a head, which is V elements each: of a turned unit the members
// of its pairs (PAIRS: neighbours, both pieces holding whole pairs), of the others any two
// pieces. `second`: whether the second one exists (the last element of an odd head is alone).
struct Place {
  uint32_t at0, at1;
  bool there, second;
};
template <int V, bool PAIRS>
__device__ __forceinline__ Place place_of(const HeadArgs& a, uint32_t unit) {
  Place p;
  const uint32_t half = a.turned / 2, p0 = unit * V;
  const bool turns = p0 < half;
  p.there = unit < a.units;
  const uint32_t from = turns ? 0 : a.turned, q = turns ? p0 : p0 - half;
  const uint32_t apart = turns ? half : (a.dim - a.turned + 1) / 2;
  p.at0 = from + (PAIRS ? 2 * q : q);
  p.at1 = p.at0 + (PAIRS ? V : apart);
  p.second = p.there && p.at1 < a.dim;
  return p;
}
// The elements of the unit's pair i.
template <int V, bool PAIRS>
__device__ __forceinline__ uint2 pair_elements(const Place& p, uint32_t i) {
  return PAIRS && V > 1 ? make_uint2(p.at0 + 2 * i, p.at0 + 2 * i + 1)
                        : make_uint2(p.at0 + i, p.at1 + i);
}

// What a lane reads of one head: NU units of V pairs, each as two pieces, of which those that do
// not exist are zeros. RING: on its way through shared memory, kRing jobs ahead, where a lane
// copies and reads back its own pieces alone; else (16-bit elements one by one, which no
// asynchronous copy takes) in registers, one job ahead. (With one job ahead in registers 24 KB of
// an SM's reads were on their way at a time, and 16384 x 40 x 128 bf16 took 95 us.)
constexpr int kRing = 4;
template <typename T, int V, int NU>
struct Piece {
  static constexpr bool RING = V * sizeof(T) >= 4;
  static constexpr uint32_t kBytes = V * sizeof(T);
  static constexpr uint32_t kSlot = RING ? 2 * NU * kBytes : 0;  // of a lane
  Pack<T, V> a[NU], b[NU];

  // `to`: the lane's place in the slot's first piece, of 32 lanes each
  __device__ __forceinline__ void load(const T* p, const Place (&at)[NU], bool active,
                                       uint32_t to) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if constexpr (RING) {
        copy(to + 2 * j * 32 * kBytes, p + (at[j].there ? at[j].at0 : 0), active && at[j].there);
        copy(to + (2 * j + 1) * 32 * kBytes, p + (at[j].second ? at[j].at1 : 0),
             active && at[j].second);
      } else {
        a[j] = b[j] = Pack<T, V>{};
        if (active && at[j].there) a[j] = *reinterpret_cast<const Pack<T, V>*>(p + at[j].at0);
        if (active && at[j].second) b[j] = *reinterpret_cast<const Pack<T, V>*>(p + at[j].at1);
      }
    }
  }
  static __device__ __forceinline__ void copy(uint32_t to, const T* from, bool there) {
    const uint32_t bytes = there ? kBytes : 0;  // the rest is filled with zeros
    if constexpr (kBytes == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to),
                   "l"(from), "r"(bytes)
                   : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(to),
                   "l"(from), "r"(bytes), "n"(kBytes)
                   : "memory");
  }
  __device__ __forceinline__ void arrive(const uint8_t* from) {
    if constexpr (RING) {
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        a[j] = *reinterpret_cast<const Pack<T, V>*>(from + 2 * j * 32 * kBytes);
        b[j] = *reinterpret_cast<const Pack<T, V>*>(from + (2 * j + 1) * 32 * kBytes);
      }
    }
  }
  // lo and hi: the members of its pairs, two pairs to an F2. With V = 1 its units are the pairs.
  template <bool PAIRS>
  __device__ __forceinline__ void get(F2 (&lo)[V * NU / 2], F2 (&hi)[V * NU / 2]) const {
#pragma unroll
    for (int k = 0; k < V * NU; k += 2) {
      const int j = k / V, i = k % V;
      if constexpr (PAIRS && V > 1) {
        const Pack<T, V>& from = 2 * i < V ? a[j] : b[j];
        const F2 u = two(from, 2 * i % V), v = two(from, 2 * i % V + 2);
        lo[k / 2] = f2(u.x, v.x);
        hi[k / 2] = f2(u.y, v.y);
      } else if constexpr (V > 1) {
        lo[k / 2] = two(a[j], i);
        hi[k / 2] = two(b[j], i);
      } else {
        lo[k / 2] = f2(to_f32(a[k].e[0]), to_f32(a[k + 1].e[0]));
        hi[k / 2] = f2(to_f32(b[k].e[0]), to_f32(b[k + 1].e[0]));
      }
    }
  }
  // Elements i and i + 1 of a piece.
  static __device__ __forceinline__ F2 two(const Pack<T, V>& p, int i) {
    if constexpr (sizeof(T) == 4)
      return f2(p.e[i], p.e[i + 1]);
    else
      return unpack2<T>(reinterpret_cast<const uint32_t*>(&p)[i / 2]);
  }
};
template <typename T, int V>
__device__ __forceinline__ void set_two(Pack<T, V>& p, int i, F2 v) {
  if constexpr (sizeof(T) == 4) {
    p.e[i] = v.x;
    p.e[i + 1] = v.y;
  } else {
    reinterpret_cast<uint32_t*>(&p)[i / 2] = pack2<T>(v);
  }
}
template <typename T, int V, int NU, bool PAIRS>
__device__ __forceinline__ void put_members(T* to, const Place (&at)[NU],
                                            const F2 (&lo)[V * NU / 2],
                                            const F2 (&hi)[V * NU / 2]) {
  auto one = [](const F2& v, int i) { return i & 1 ? v.y : v.x; };
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    Pack<T, V> x, y;
    if constexpr (V == 1) {
      x.e[0] = from_f32<T>(one(lo[j / 2], j));
      y.e[0] = from_f32<T>(one(hi[j / 2], j));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        // elements i, i + 1 of the first piece are pair i / 2, of the second V / 2 + i / 2
        const int p = j * V + i / 2, q = p + V / 2, k = (j * V + i) / 2;
        set_two(x, i, PAIRS ? f2(one(lo[p / 2], p), one(hi[p / 2], p)) : lo[k]);
        set_two(y, i, PAIRS ? f2(one(lo[q / 2], q), one(hi[q / 2], q)) : hi[k]);
      }
    }
    if (at[j].there) *reinterpret_cast<Pack<T, V>*>(to + at[j].at0) = x;
    if (at[j].second) *reinterpret_cast<Pack<T, V>*>(to + at[j].at1) = y;
  }
}

// A lane's V * NU pairs of a vector in shared memory that holds one value for each pair.
template <int V, int NU>
__device__ __forceinline__ void from_table(const float* t, uint32_t l, uint32_t lanes,
                                           F2 (&v)[V * NU / 2]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int j = 0; j < NU; j += 2) v[j / 2] = f2(t[l + j * lanes], t[l + (j + 1) * lanes]);
  } else {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(t + (l + j * lanes) * V + i);
        v[(j * V + i) / 2] = f2(f.x, f.y);
        v[(j * V + i) / 2 + 1] = f2(f.z, f.w);
      }
    }
  }
}

// Where the rings begin in shared memory.
__host__ __device__ __forceinline__ uint32_t ring_offset(uint32_t all, uint32_t half) {
  return ((4 + 2 * kWarps) * all * 4 + half * 8 + 15) / 16 * 16;
}

// BACK: the gradients, else the forward pass. NU units of V pairs per lane. Arithmetic is on two
// pairs at a time.
template <typename T, int V, int NU, bool PAIRS, bool BACK, int MINB>
__global__ void __launch_bounds__(32 * kWarps, MINB) heads_kernel(const HeadArgs a) {
  griddep_wait();
  constexpr int N = V * NU / 2;  // of F2
  // Shared memory, `all` being the pairs of 32 lanes: both sides' weights of the pairs' first and
  // second members [2][2][all], for each warp the cosines and the sines [2][all], the fractions
  // of a turn [turned / 2], for each warp the ring of what it reads (x, and g); at the end of the
  // backward pass [warps][dim] sums.
  extern __shared__ __align__(16) uint8_t dynamic[];
  const uint32_t half = a.turned / 2, lane = lane_id(), warp = threadIdx.x >> 5;
  const uint32_t all = a.lanes * V * NU;
  float* const weights = reinterpret_cast<float*>(dynamic);
  float* const cosine = weights + 4 * all + 2 * all * warp;
  float* const sine = cosine + all;
  uint64_t* const fraction = reinterpret_cast<uint64_t*>(weights + (4 + 2 * kWarps) * all);
  using Mine = Piece<T, V, NU>;
  constexpr uint32_t kSlot = 32 * Mine::kSlot * (BACK ? 2 : 1);
  uint8_t* const ring = dynamic + ring_offset(all, half) + warp * kRing * kSlot +
                        lane * Mine::kBytes;
  for (uint32_t i = threadIdx.x; i < half; i += blockDim.x) fraction[i] = turn_fraction(a.freqs[i]);
  for (uint32_t i = threadIdx.x; i < 2 * all; i += blockDim.x) {
    const uint32_t k = i >= all, c = i - k * all, unit = c / V;
    const Place p = place_of<V, PAIRS>(a, unit);
    const uint2 e = pair_elements<V, PAIRS>(p, c - unit * V);
    const void* w = a.side[k].w;
    weights[2 * k * all + c] = w && p.there ? load_any(w, a.w_type, e.x) : 1.f;
    weights[(2 * k + 1) * all + c] = w && p.second ? load_any(w, a.w_type, e.y) : 1.f;
  }
  for (uint32_t i = lane; i < all; i += 32) {  // what is not turned: once and for all
    cosine[i] = 1.f;
    sine[i] = 0.f;
  }
  __syncthreads();

  // this warp's side and run of jobs
  const uint32_t id = blockIdx.x * kWarps + warp;
  const bool keys = id >= a.warps[0];
  const Side& side = a.side[keys];
  const uint32_t among = a.warps[keys], index = keys ? id - a.warps[0] : id;
  const bool works = index < among;
  const uint64_t jobs = a.tokens * side.jobs;
  const uint64_t job = works ? jobs * index / among : 0;
  const uint64_t end = works ? jobs * (index + 1) / among : 0;
  const uint32_t slots = 32 / a.lanes, slot = lane / a.lanes, l = lane - slot * a.lanes;
  const float inv = 1.f / (float)a.dim;
  Place place[NU];
#pragma unroll
  for (int j = 0; j < NU; ++j) place[j] = place_of<V, PAIRS>(a, l + j * a.lanes);
  // Backward: weights, and the sums of their gradients. Forward: the four products of weights
  // with cosines and sines.
  F2 w0[N], w1[N], s0[N], s1[N];
  const float* const w_lo = weights + 2 * keys * all;
  if constexpr (BACK) {
    from_table<V, NU>(w_lo, l, a.lanes, w0);
    from_table<V, NU>(w_lo + all, l, a.lanes, w1);
#pragma unroll
    for (int i = 0; i < N; ++i) s0[i] = s1[i] = f2(0.f, 0.f);
  }
  uint64_t token = side.jobs ? job / side.jobs : 0;
  uint32_t part = (uint32_t)(job - token * side.jobs);

  Mine x, g;
  // The jobs are fetched in order, kAhead before their turn; pointers go on from head to head and
  // from token to token.
  constexpr uint32_t kAhead = Mine::RING ? kRing - 1 : 1;
  struct Walk {
    const T* at;     // this lane's head
    // to the next job of the token, and from its last one to the next token
    int64_t heads_on, token_on;
    __device__ __forceinline__ Walk(const Heads& h, uint64_t token, uint32_t part, uint32_t jobs,
                                    uint32_t slots, uint32_t slot) {
      heads_on = (int64_t)slots * h.head;
      token_on = h.token - (int64_t)(jobs - 1) * heads_on;
      at = static_cast<const T*>(h.p) + (int64_t)token * h.token +
           (int64_t)(part * slots + slot) * h.head;
    }
    __device__ __forceinline__ void next(bool last) { at += last ? token_on : heads_on; }
  };
  Walk from_x(side.x, token, part, side.jobs, slots, slot);
  Walk from_g(side.g, token, part, side.jobs, slots, slot);
  Walk to_out(side.out, token, part, side.jobs, slots, slot);
  const uint32_t in_last = side.heads - (side.jobs - 1) * slots;  // heads of a token's last job
  uint32_t next_part = part, left = (uint32_t)(end - job);
  uint32_t to_fetch = left;
  const uint32_t ring0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  uint32_t slot_in = 0, slot_out = 0;
  auto fetch = [&]() {
    if (to_fetch > 0) {
      const bool last = next_part + 1 == side.jobs;
      // a lane without a head in the last job reads nothing, and so its pointer does not matter
      const bool active = !last || slot < in_last;
      x.load(from_x.at, place, active, ring0 + slot_in);
      from_x.next(last);
      if constexpr (BACK) {
        g.load(from_g.at, place, active, ring0 + slot_in + 32 * Mine::kSlot);
        from_g.next(last);
      }
      --to_fetch;
      next_part = last ? 0 : next_part + 1;
      slot_in = slot_in == (kRing - 1) * kSlot ? 0 : slot_in + kSlot;
    }
    if constexpr (Mine::RING) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (uint32_t k = 0; k < kAhead; ++k) fetch();
  bool known = false;
  for (; left > 0; --left) {
    const bool last = part + 1 == side.jobs, active = !last || slot < in_last;
    F2 lo[N], hi[N], glo[N], ghi[N];
    if constexpr (Mine::RING) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
      x.arrive(ring + slot_out);
      if constexpr (BACK) g.arrive(ring + slot_out + 32 * Mine::kSlot);
      slot_out = slot_out == (kRing - 1) * kSlot ? 0 : slot_out + kSlot;
    }
    x.template get<PAIRS>(lo, hi);
    if constexpr (BACK) g.template get<PAIRS>(glo, ghi);
    T* const out = const_cast<T*>(to_out.at);
    to_out.next(last);
    part = last ? 0 : part + 1;
    fetch();
    if (!known) {
      if (half) {
        const int64_t position = a.wide ? static_cast<const int64_t*>(a.positions)[token]
                                        : static_cast<const int32_t*>(a.positions)[token];
        __syncwarp();
        for (uint32_t i = lane; i < half; i += 32) {
          const uint64_t turn = (uint64_t)position * fraction[i];
          sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, sine + i, cosine + i);
        }
        __syncwarp();
      }
      if constexpr (!BACK) {  // out = r (lo w0 c - hi w1 s), r (lo w0 s + hi w1 c)
        F2 c[N], s[N], u[N], v[N];
        from_table<V, NU>(cosine, l, a.lanes, c);
        from_table<V, NU>(sine, l, a.lanes, s);
        from_table<V, NU>(w_lo, l, a.lanes, u);
        from_table<V, NU>(w_lo + all, l, a.lanes, v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          w0[i] = mul2<true>(u[i], c[i]);
          s0[i] = mul2<true>(u[i], s[i]);
          w1[i] = mul2<true>(v[i], c[i]);
          s1[i] = mul2<true>(v[i], f2(-s[i].x, -s[i].y));
        }
      }
    }
    known = !last;
    token += last;

    // (Lanes without a head would make an infinity of 0 here, times zeros in the weights' sums. As a
    // choice on the root itself it took 92 us in place of 90 at 16384 x 40 x 128.)
    const float eps = BACK && !active ? 1.f : a.eps;
    F2 ss = f2(0.f, 0.f), dot = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ss = fma2<true>(lo[i], lo[i], ss);
      ss = fma2<true>(hi[i], hi[i], ss);
    }
    if constexpr (BACK) {
      F2 c[N], s[N];
      from_table<V, NU>(cosine, l, a.lanes, c);
      from_table<V, NU>(sine, l, a.lanes, s);
#pragma unroll
      for (int i = 0; i < N; ++i) {  // the gradient turned back
        const F2 t = fma2<true>(ghi[i], s[i], mul2<true>(glo[i], c[i]));
        ghi[i] = fma2<true>(glo[i], f2(-s[i].x, -s[i].y), mul2<true>(ghi[i], c[i]));
        glo[i] = t;
        dot = fma2<true>(mul2<true>(glo[i], w0[i]), lo[i], dot);
        dot = fma2<true>(mul2<true>(ghi[i], w1[i]), hi[i], dot);
      }
    }
    float2 sum = make_float2(ss.x + ss.y, dot.x + dot.y);
    for (uint32_t d = a.lanes / 2; d > 0; d >>= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, d);
      if constexpr (BACK) sum.y += __shfl_xor_sync(0xffffffffu, sum.y, d);
    }
    const float r = rsqrtf(sum.x * inv + eps);
    const F2 by = f2(r, r);
    if constexpr (BACK) {
      const float k = -sum.y * inv * r * r * r;
      const F2 kk = f2(k, k);
#pragma unroll
      for (int i = 0; i < N; ++i) {  // dx = r g w + k x
        s0[i] = fma2<true>(glo[i], mul2<true>(lo[i], by), s0[i]);
        s1[i] = fma2<true>(ghi[i], mul2<true>(hi[i], by), s1[i]);
        lo[i] = fma2<true>(mul2<true>(glo[i], w0[i]), by, mul2<true>(lo[i], kk));
        hi[i] = fma2<true>(mul2<true>(ghi[i], w1[i]), by, mul2<true>(hi[i], kk));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const F2 u = mul2<true>(lo[i], by), v = mul2<true>(hi[i], by);
        lo[i] = fma2<true>(v, s1[i], mul2<true>(u, w0[i]));
        hi[i] = fma2<true>(u, s0[i], mul2<true>(v, w1[i]));
      }
    }
    if (active) put_members<T, V, NU, PAIRS>(out, place, lo, hi);
  }
  if constexpr (BACK) {
    if (a.part[0] == nullptr) return;  // neither sum is wanted
    // a warp's slots by shuffles, then the block's warps in order
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(dynamic) + warp * a.dim;
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) {
      float u = k & 1 ? s0[k / 2].y : s0[k / 2].x, v = k & 1 ? s1[k / 2].y : s1[k / 2].x;
      for (uint32_t d = a.lanes; d < 32; d <<= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, d);
        v += __shfl_xor_sync(0xffffffffu, v, d);
      }
      const uint2 e = pair_elements<V, PAIRS>(place[k / V], k % V);
      if (slot == 0 && place[k / V].there) sums[e.x] = u;
      if (slot == 0 && place[k / V].second) sums[e.y] = v;
    }
    __syncthreads();
    const uint32_t id0 = blockIdx.x * kWarps;
    for (uint32_t c = threadIdx.x; c < a.dim; c += blockDim.x) {
      float of[2] = {0.f, 0.f};
      for (uint32_t k = 0; k < kWarps; ++k) {
        const float v = reinterpret_cast<const float*>(dynamic)[k * a.dim + c];
        if (id0 + k >= a.warps[0]) of[1] += v;
        else of[0] += v;
      }
      a.part[0][(uint64_t)blockIdx.x * a.dim + c] = of[0];
      a.part[1][(uint64_t)blockIdx.x * a.dim + c] = of[1];
    }
  }
}

// Blocks: what the registers of the SMs hold at one time (FIT per SM, two backward at most), no
// more than there are jobs.
constexpr uint32_t kBackFit = 2;
uint32_t grid_for(uint64_t jobs, uint32_t fit) {
  const uint64_t blocks = std::min<uint64_t>((jobs + kWarps - 1) / kWarps, kSms * fit);
  return (uint32_t)std::max<uint64_t>(1, blocks);
}

// Each returns the blocks of its grid, 0 if the launch failed.
template <typename T, int V, int NU, bool PAIRS, bool BACK, int FIT>
uint32_t launch_heads(HeadArgs a, cudaStream_t s) {
  const uint32_t slots = 32 / a.lanes;
  uint64_t jobs = 0;
  for (Side& d : a.side) {
    d.jobs = (d.heads + slots - 1) / slots;
    jobs += a.tokens * d.jobs;
  }
  // The warps are shared out by the jobs, at least one to a side that has any. Where a warp has
  // several tokens, each one's sines count as two jobs, backward as one, which is more of the few
  // keys' time. 16384 tokens, bf16: 59 us for 32 + 8 heads of 128, 63 without, backward 88 and 91;
  // 50 and 57 for 64 + 4 of 64, backward 77 and 81.
  uint32_t grid = grid_for(jobs, FIT);
  const uint32_t warps = grid * kWarps;
  const uint32_t extra = a.turned && jobs > 2ull * warps ? (BACK ? 1 : 2) : 0;
  auto cost = [extra](const Side& d) { return d.jobs ? d.jobs + extra : 0u; };
  const uint32_t each = cost(a.side[0]) + cost(a.side[1]);
  a.warps[0] = (uint32_t)(((uint64_t)warps * cost(a.side[0]) + each / 2) / each);
  if (a.side[0].jobs) a.warps[0] = std::max(1u, a.warps[0]);
  if (a.side[1].jobs) a.warps[0] = std::min(warps - 1, a.warps[0]);
  a.warps[1] = warps - a.warps[0];
  if (a.part[0]) a.part[1] = a.part[0] + (uint64_t)grid * a.dim;
  const size_t all = (size_t)a.lanes * V * NU;
  size_t smem = ring_offset((uint32_t)all, a.turned / 2) +
                kWarps * kRing * 32 * Piece<T, V, NU>::kSlot * (BACK ? 2 : 1);
  if (BACK) smem = std::max(smem, kWarps * a.dim * sizeof(float));
  auto kernel = heads_kernel<T, V, NU, PAIRS, BACK, FIT>;
  if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return 0;
  launch_pdl(kernel, grid, 32 * kWarps, smem, s, a);
  return grid;
}

// L: the least power of two of lanes that hold a head with NU units each.
uint32_t lanes_for(uint32_t units, uint32_t nu) {
  uint32_t l = 1;
  while (l * nu < units) l *= 2;
  return l;
}

// `pack` neighbouring elements are one access, 1 where they are not aligned.
template <typename T, bool PAIRS, bool BACK>
uint32_t heads_typed(HeadArgs a, uint32_t pack, cudaStream_t s) {
  a.units = (a.dim + 1) / 2 / pack;
  if (pack == 1) {
    a.units = (a.dim + 1) / 2;
    if (a.units <= 64) {
      a.lanes = lanes_for(a.units, 2);
      return launch_heads<T, 1, 2, PAIRS, BACK, BACK ? 2 : 4>(a, s);
    }
    a.lanes = 32;
    return launch_heads<T, 1, 8, PAIRS, BACK, 1>(a, s);
  }
  if constexpr (sizeof(T) == 2) {
    if (pack == 8) {
      a.lanes = lanes_for(a.units, 1);
      // (three blocks per SM forward, of 80 registers: 68 us where two took 63, 16384 x 40 x 128)
      return launch_heads<T, 8, 1, PAIRS, BACK, 2>(a, s);
    }
  }
  // two units per lane where 32 lanes do not hold a head: more than 256 elements
  if (a.units <= 32) {
    a.lanes = lanes_for(a.units, 1);
    return launch_heads<T, 4, 1, PAIRS, BACK, BACK ? 2 : 4>(a, s);
  }
  a.lanes = 32;
  return launch_heads<T, 4, 2, PAIRS, BACK, BACK ? 1 : 2>(a, s);
}

template <typename T>
uint32_t heads_any(const HeadArgs& a, bool pairs, bool back, cudaStream_t s) {
  auto packs = [&](uint32_t v) {
    bool fit = a.turned % (2 * v) == 0 && (a.dim - a.turned) % (2 * v) == 0;
    for (const Side& d : a.side)
      for (const Heads* h : {&d.x, &d.g, &d.out})
        fit = fit && (!d.heads || (aligned_to(h->p, v * sizeof(T)) && h->token % v == 0 &&
                                   h->head % v == 0));
    return fit;
  };
  const uint32_t pack = sizeof(T) == 2 && packs(8) ? 8 : packs(4) ? 4 : 1;
  if (back)
    return pairs ? heads_typed<T, true, true>(a, pack, s)
                 : heads_typed<T, false, true>(a, pack, s);
  return pairs ? heads_typed<T, true, false>(a, pack, s)
               : heads_typed<T, false, false>(a, pack, s);
}

// Whether no two elements of [tokens][heads][dim] share an address: heads within tokens, or
// tokens within heads.
bool heads_apart(uint64_t tokens, uint64_t heads, uint64_t dim, int64_t token, int64_t head) {
  if (token < 0 || head < 0) return false;
  const uint64_t t = tokens > 1 ? token : 0, h = heads > 1 ? head : 0, n = dim;
  const bool within = (heads <= 1 || h >= n) && (tokens <= 1 || t >= (heads - 1) * h + n);
  const bool around = (tokens <= 1 || t >= n) && (heads <= 1 || h >= (tokens - 1) * t + n);
  return within || around;
}

bool input_ok(const Heads& h, uint32_t heads, size_t bytes) {
  return heads == 0 || (h.p && aligned_to(h.p, bytes) && h.token >= 0 && h.head >= 0);
}

// What both passes check.
int check_heads(const HeadArgs& a, int64_t type, int64_t weight_type) {
  const auto known = [](int64_t t) { return t >= SPARCML_F32 && t <= SPARCML_F16; };
  if (!known(type) || !known(weight_type) || a.tokens > 0x7fffffffull || a.dim < 1 ||
      a.dim > kMostDim || a.turned > a.dim || a.turned % 2 || !(a.eps >= 0.f))
    return SPARCML_ERR_INVALID_ARG;
  for (const Side& d : a.side)
    if (d.heads > 65535 || (d.heads && !aligned_to(d.w, type_bytes((int32_t)weight_type))))
      return SPARCML_ERR_INVALID_ARG;
  if (a.tokens == 0 || a.side[0].heads + a.side[1].heads == 0) return SPARCML_OK;
  const size_t e = type_bytes((int32_t)type);
  if (a.turned && (!a.positions || !aligned_to(a.positions, a.wide ? 8 : 4) || !a.freqs ||
                   !aligned_to(a.freqs, 4)))
    return SPARCML_ERR_INVALID_ARG;
  for (const Side& d : a.side)
    if (!input_ok(d.x, d.heads, e) || !input_ok(d.out, d.heads, e) ||
        (d.heads && !heads_apart(a.tokens, d.heads, a.dim, d.out.token, d.out.head)))
      return SPARCML_ERR_INVALID_ARG;
  return SPARCML_OK;
}

}  // namespace
}  // namespace sparcml

using namespace sparcml;

// The arguments of both passes; false where one is out of range.
static bool read_args(const sparcml_head_args* p, bool back, HeadArgs& a) {
  if (!p || p->tokens < 0 || p->dim < 0 || p->dim > kMostDim || p->q_heads < 0 ||
      p->q_heads > 65535 || p->k_heads < 0 || p->k_heads > 65535 || p->turned < 0 ||
      p->turned > kMostDim)
    return false;
  a = {};
  a.side[0] = {{p->q, p->q_token_stride, p->q_head_stride}, {nullptr, 0, 0},
               {p->q_out, p->q_out_token_stride, p->q_out_head_stride}, p->q_weight,
               (uint32_t)p->q_heads, 0};
  a.side[1] = {{p->k, p->k_token_stride, p->k_head_stride}, {nullptr, 0, 0},
               {p->k_out, p->k_out_token_stride, p->k_out_head_stride}, p->k_weight,
               (uint32_t)p->k_heads, 0};
  if (back) {
    a.side[0].g = {p->dq, p->dq_token_stride, p->dq_head_stride};
    a.side[1].g = {p->dk, p->dk_token_stride, p->dk_head_stride};
  }
  a.tokens = (uint64_t)p->tokens;
  a.dim = (uint32_t)p->dim;
  a.turned = (uint32_t)p->turned;
  a.positions = p->positions;
  a.wide = p->positions_int64 != 0;
  a.freqs = p->freqs;
  a.w_type = (int32_t)p->weight_type;
  a.eps = (float)p->eps;
  return true;
}

extern "C" int sparcml_head_norm_rotary(const sparcml_head_args* args, void* stream) {
  const ApiRange nvtx_range(__func__);
  HeadArgs a;
  if (!read_args(args, false, a)) return SPARCML_ERR_INVALID_ARG;
  const int64_t type = args->type;
  const int r = check_heads(a, type, args->weight_type);
  if (r != SPARCML_OK) return r;
  if (a.tokens == 0 || a.side[0].heads + a.side[1].heads == 0) return SPARCML_OK;
  const bool pairs = args->interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint32_t blocks = type == SPARCML_F32    ? heads_any<float>(a, pairs, false, s)
                          : type == SPARCML_BF16 ? heads_any<__nv_bfloat16>(a, pairs, false, s)
                                                 : heads_any<__half>(a, pairs, false, s);
  if (launch_status() != SPARCML_OK || !blocks) return SPARCML_ERR_CUDA;
  note_launches(1);
  return SPARCML_OK;
}

extern "C" size_t sparcml_head_norm_rotary_backward_workspace_size(uint64_t tokens,
                                                                   uint32_t q_heads,
                                                                   uint32_t k_heads,
                                                                   uint32_t dim) {
  if (tokens > 0x7fffffffull || dim < 1 || dim > kMostDim || q_heads > 65535 || k_heads > 65535)
    return 0;
  // a block for eight heads at most
  const uint32_t most = grid_for(tokens * (q_heads + k_heads), kBackFit);
  return 256 + align_up(2ull * most * dim * sizeof(float), 256);
}

extern "C" int sparcml_head_norm_rotary_backward(const sparcml_head_args* args, void* stream) {
  const ApiRange nvtx_range(__func__);
  HeadArgs a;
  if (!read_args(args, true, a)) return SPARCML_ERR_INVALID_ARG;
  const int64_t type = args->type;
  const int r = check_heads(a, type, args->weight_type);
  if (r != SPARCML_OK) return r;
  float *const dq = args->q_dweight, *const dk = args->k_dweight;
  uint8_t* const ws = static_cast<uint8_t*>(args->ws);
  if (!ws || !aligned_to(ws, 256) || !aligned_to(dq, 4) || !aligned_to(dk, 4))
    return SPARCML_ERR_INVALID_ARG;
  const uint32_t heads[2] = {a.side[0].heads, a.side[1].heads};
  const bool work = a.tokens && heads[0] + heads[1];
  for (const Side& d : a.side)
    if (work && !input_ok(d.g, d.heads, type_bytes((int32_t)type))) return SPARCML_ERR_INVALID_ARG;
  if (args->ws_bytes < 0 ||
      (uint64_t)args->ws_bytes < sparcml_head_norm_rotary_backward_workspace_size(
                                     a.tokens, heads[0], heads[1], a.dim))
    return SPARCML_ERR_WORKSPACE;
  const bool sums = dq || dk, pairs = args->interleaved != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t parts = 0;
  if (work) {
    if (sums) a.part[0] = reinterpret_cast<float*>(ws + 256);
    parts = type == SPARCML_F32    ? heads_any<float>(a, pairs, true, s)
            : type == SPARCML_BF16 ? heads_any<__nv_bfloat16>(a, pairs, true, s)
                                   : heads_any<__half>(a, pairs, true, s);
    if (launch_status() != SPARCML_OK || !parts) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  if (sums) {
    const float* part = reinterpret_cast<const float*>(ws + 256);
    launch_pdl(join_columns_kernel, dim3((a.dim + 31) / 32, 2), 512, 0, s, part,
               part + (uint64_t)parts * a.dim, parts, (uint64_t)a.dim, dq, dk,
               (int32_t)(args->accumulate != 0));
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  return SPARCML_OK;
}
