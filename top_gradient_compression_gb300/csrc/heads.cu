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
// position: the error is 2^-65 of a turn times the position. Its upper 32 bits go to sincospif.

#include "rows.cuh"

namespace sparcml {
namespace {

constexpr uint32_t kWarps = 8;      // per block
constexpr uint32_t kMostDim = 512;  // elements of a head

// V consecutive elements as they lie in memory: four (in 16 bits, 8 bytes: eight of them per lane
// leave too few registers), or one.
constexpr int kPack = 4;
template <typename T, int V>
struct Piece {
  Pack<T, V> r;
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const Pack<T, V>*>(p); }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(r.e[i]);
  }
  static __device__ __forceinline__ void put(T* p, const float (&f)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(f[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = r;
  }
};
template <typename T>
struct Piece<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f32(v); }
  static __device__ __forceinline__ void put(T* p, const float (&f)[1]) { *p = from_f32<T>(f[0]); }
};

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
  uint32_t dim, turned, units, lanes;  // units of V pairs; L
  const void* positions;
  int32_t wide;  // positions are int64, else int32
  const float* freqs;
  int32_t w_type;
  float eps;
  uint32_t warps[2];  // of the grid, for each side
  float* part[2];     // [gridDim.x][dim] sums of dw, one array after the other; or null
};

// f / 2 pi of a turn, in 2^-64: the product with 1 / 2 pi in two parts, of which whole turns
// are dropped.
__device__ __forceinline__ uint64_t turn_fraction(float freq) {
  const double inv = 0.15915494309189535, low = -9.839338337591243e-18;  // 1 / 2 pi = inv + low
  const double f = freq, hi = f * inv, rest = fma(f, inv, -hi) + f * low;
  const uint64_t a = __double2ull_rn((hi - floor(hi)) * 0x1p64);
  return a + (uint64_t)__double2ll_rn(rest * 0x1p64);
}

// Where a unit's two pieces lie in a head, which is V elements each: of a turned unit the members
// of its pairs (PAIRS: neighbours, both pieces holding whole pairs), of the others any two
// pieces. `second`: whether the second one exists (the last element of an odd head is alone).
struct Place {
  uint32_t at0, at1, pair;
  bool there, second, turns;
};
template <int V, bool PAIRS>
__device__ __forceinline__ Place place_of(const HeadArgs& a, uint32_t unit) {
  Place p;
  const uint32_t half = a.turned / 2, p0 = unit * V;
  p.there = unit < a.units;
  p.turns = p0 < half;
  p.pair = p0;
  const uint32_t from = p.turns ? 0 : a.turned, q = p.turns ? p0 : p0 - half;
  const uint32_t apart = p.turns ? half : (a.dim - a.turned + 1) / 2;
  p.at0 = from + (PAIRS ? 2 * q : q);
  p.at1 = p.at0 + (PAIRS ? V : apart);
  p.second = p.there && p.at1 < a.dim;
  return p;
}

// A lane's elements of one head: lo and hi are the members of its pairs.
template <typename T, int V, bool PAIRS>
__device__ __forceinline__ void members(const Piece<T, V>& a, const Piece<T, V>& b,
                                        float (&lo)[V], float (&hi)[V]) {
  float x[V], y[V];
  a.get(x);
  b.get(y);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (PAIRS && V > 1) {
      lo[i] = 2 * i < V ? x[2 * i % V] : y[2 * i % V];
      hi[i] = 2 * i < V ? x[2 * i % V + 1] : y[2 * i % V + 1];
    } else {
      lo[i] = x[i];
      hi[i] = y[i];
    }
  }
}
template <typename T, int V, bool PAIRS>
__device__ __forceinline__ void put_members(T* to, const Place& p, const float (&lo)[V],
                                            const float (&hi)[V]) {
  float x[V], y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (PAIRS && V > 1) {
      x[i] = i & 1 ? hi[i / 2] : lo[i / 2];
      y[i] = i & 1 ? hi[V / 2 + i / 2] : lo[V / 2 + i / 2];
    } else {
      x[i] = lo[i];
      y[i] = hi[i];
    }
  }
  if (p.there) Piece<T, V>::put(to + p.at0, x);
  if (p.second) Piece<T, V>::put(to + p.at1, y);
}

// Weights of a lane's elements, in the order of lo and hi.
template <int V, bool PAIRS>
__device__ __forceinline__ void load_weights(const HeadArgs& a, const void* w, const Place& p,
                                             float (&lo)[V], float (&hi)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    lo[i] = hi[i] = 1.f;
    const uint32_t c0 = PAIRS && V > 1 ? p.at0 + 2 * i : p.at0 + i;
    const uint32_t c1 = PAIRS && V > 1 ? c0 + 1 : p.at1 + i;
    if (w && p.there) lo[i] = load_any(w, a.w_type, c0);
    if (w && p.second) hi[i] = load_any(w, a.w_type, c1);
  }
}

// BACK: the gradients, else the forward pass. NU units of V pairs per lane.
template <typename T, int V, int NU, bool PAIRS, bool BACK, int MINB>
__global__ void __launch_bounds__(32 * kWarps, MINB) heads_kernel(const HeadArgs a) {
  griddep_wait();
  // [turned / 2] fractions of a turn, then for each warp [turned / 2] cosines and sines; at the
  // end of the backward pass [warps][dim] sums
  extern __shared__ __align__(16) uint8_t dynamic[];
  const uint32_t half = a.turned / 2, lane = lane_id(), warp = threadIdx.x >> 5;
  uint64_t* const fraction = reinterpret_cast<uint64_t*>(dynamic);
  float2* const table = reinterpret_cast<float2*>(fraction + half) + warp * half;
  for (uint32_t i = threadIdx.x; i < half; i += blockDim.x) fraction[i] = turn_fraction(a.freqs[i]);
  __syncthreads();

  // this warp's side and run of jobs
  const uint32_t id = blockIdx.x * kWarps + warp;
  const bool keys = id >= a.warps[0];
  const Side& side = a.side[keys];
  const uint32_t among = a.warps[keys], index = keys ? id - a.warps[0] : id;
  const bool works = index < among;
  const uint64_t jobs = a.tokens * side.jobs;
  uint64_t job = works ? jobs * index / among : 0;
  const uint64_t end = works ? jobs * (index + 1) / among : 0;
  const uint32_t slots = 32 / a.lanes, slot = lane / a.lanes, l = lane - slot * a.lanes;
  const float inv = 1.f / (float)a.dim;
  Place place[NU];
  float w0[NU][V], w1[NU][V], s0[BACK ? NU : 1][V], s1[BACK ? NU : 1][V];
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    place[j] = place_of<V, PAIRS>(a, l + j * a.lanes);
    load_weights<V, PAIRS>(a, side.w, place[j], w0[j], w1[j]);
    if constexpr (BACK) {
#pragma unroll
      for (int i = 0; i < V; ++i) s0[j][i] = s1[j][i] = 0.f;
    }
  }
  uint64_t token = side.jobs ? job / side.jobs : 0;
  uint32_t part = (uint32_t)(job - token * side.jobs);

  Piece<T, V> x0[NU], x1[NU], g0[BACK ? NU : 1], g1[BACK ? NU : 1];
  auto fetch = [&](uint64_t tok, uint32_t part_) {
    const uint32_t head = part_ * slots + slot;
    if (head >= side.heads) return;
    const T* x = static_cast<const T*>(side.x.p) + (int64_t)tok * side.x.token +
                 (int64_t)head * side.x.head;
    const T* g = static_cast<const T*>(side.g.p) + (int64_t)tok * side.g.token +
                 (int64_t)head * side.g.head;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (place[j].there) x0[j].load(x + place[j].at0);
      if (place[j].second) x1[j].load(x + place[j].at1);
      if constexpr (BACK) {
        if (place[j].there) g0[j].load(g + place[j].at0);
        if (place[j].second) g1[j].load(g + place[j].at1);
      }
    }
  };
  if (job < end) fetch(token, part);
  bool known = false;
  float cs[NU][V], sn[NU][V];
  for (; job < end; ++job) {
    const uint32_t head = part * slots + slot;
    const bool active = head < side.heads;
    float lo[NU][V], hi[NU][V], glo[BACK ? NU : 1][V], ghi[BACK ? NU : 1][V];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      members<T, V, PAIRS>(x0[j], x1[j], lo[j], hi[j]);
      if constexpr (BACK) members<T, V, PAIRS>(g0[j], g1[j], glo[j], ghi[j]);
      // what was not loaded counts as zero
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!active || !place[j].there) lo[j][i] = 0.f;
        if (!active || !place[j].second) hi[j][i] = 0.f;
        if constexpr (BACK) {
          if (!active || !place[j].there) glo[j][i] = 0.f;
          if (!active || !place[j].second) ghi[j][i] = 0.f;
        }
      }
    }
    const uint64_t now = token;
    if (++part == side.jobs) {
      part = 0;
      ++token;
    }
    if (job + 1 < end) fetch(token, part);
    if (!known) {
      const int64_t position = a.wide ? static_cast<const int64_t*>(a.positions)[now]
                                      : static_cast<const int32_t*>(a.positions)[now];
      __syncwarp();
      for (uint32_t i = lane; i < half; i += 32) {
        const uint64_t turn = (uint64_t)position * fraction[i];
        float sine, cosine;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sine, &cosine);
        table[i] = make_float2(cosine, sine);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NU; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 t = place[j].turns && place[j].there ? table[place[j].pair + i]
                                                            : make_float2(1.f, 0.f);
          cs[j][i] = t.x;
          sn[j][i] = t.y;
        }
      }
    }
    known = token == now;

    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s.x += lo[j][i] * lo[j][i];
        s.x += hi[j][i] * hi[j][i];
        if constexpr (BACK) {
          const float t = glo[j][i] * cs[j][i] + ghi[j][i] * sn[j][i];
          ghi[j][i] = ghi[j][i] * cs[j][i] - glo[j][i] * sn[j][i];
          glo[j][i] = t;
          s.y += t * w0[j][i] * lo[j][i];
          s.y += ghi[j][i] * w1[j][i] * hi[j][i];
        }
      }
    }
    for (uint32_t d = a.lanes / 2; d > 0; d >>= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, d);
      if constexpr (BACK) s.y += __shfl_xor_sync(0xffffffffu, s.y, d);
    }
    const float r = rsqrtf(s.x * inv + a.eps);
    T* out = static_cast<T*>(const_cast<void*>(side.out.p)) + (int64_t)now * side.out.token +
             (int64_t)head * side.out.head;
    const float k = BACK ? -s.y * inv * r * r * r : 0.f;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      float o0[V], o1[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (BACK) {
          s0[j][i] += glo[j][i] * (lo[j][i] * r);
          s1[j][i] += ghi[j][i] * (hi[j][i] * r);
          o0[i] = glo[j][i] * w0[j][i] * r + lo[j][i] * k;
          o1[i] = ghi[j][i] * w1[j][i] * r + hi[j][i] * k;
        } else {
          const float u0 = lo[j][i] * r * w0[j][i], u1 = hi[j][i] * r * w1[j][i];
          o0[i] = u0 * cs[j][i] - u1 * sn[j][i];
          o1[i] = u0 * sn[j][i] + u1 * cs[j][i];
        }
      }
      if (active) put_members<T, V, PAIRS>(out, place[j], o0, o1);
    }
  }
  if constexpr (BACK) {
    if (a.part[0] == nullptr) return;  // neither sum is wanted
    // a warp's slots by shuffles, then the block's warps in order
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(dynamic) + warp * a.dim;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        for (uint32_t d = a.lanes; d < 32; d <<= 1) {
          s0[j][i] += __shfl_xor_sync(0xffffffffu, s0[j][i], d);
          s1[j][i] += __shfl_xor_sync(0xffffffffu, s1[j][i], d);
        }
        const uint32_t c0 = PAIRS && V > 1 ? place[j].at0 + 2 * i : place[j].at0 + i;
        const uint32_t c1 = PAIRS && V > 1 ? c0 + 1 : place[j].at1 + i;
        if (slot == 0 && place[j].there) sums[c0] = s0[j][i];
        if (slot == 0 && place[j].second) sums[c1] = s1[j][i];
      }
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
  return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>((jobs + kWarps - 1) / kWarps, kSms * fit));
}

// Each returns the blocks of its grid.
template <typename T, int V, int NU, bool PAIRS, bool BACK, int FIT>
uint32_t launch_heads(HeadArgs a, cudaStream_t s) {
  const uint32_t slots = 32 / a.lanes;
  uint64_t jobs = 0;
  for (Side& d : a.side) {
    d.jobs = (d.heads + slots - 1) / slots;
    jobs += a.tokens * d.jobs;
  }
  // the warps are shared out by the jobs, at least one to a side that has any
  uint32_t grid = grid_for(jobs, FIT);
  const uint32_t warps = grid * kWarps, each = a.side[0].jobs + a.side[1].jobs;
  a.warps[0] = (uint32_t)(((uint64_t)warps * a.side[0].jobs + each / 2) / each);
  if (a.side[0].jobs) a.warps[0] = std::max(1u, a.warps[0]);
  if (a.side[1].jobs) a.warps[0] = std::min(warps - 1, a.warps[0]);
  a.warps[1] = warps - a.warps[0];
  if (a.part[0]) a.part[1] = a.part[0] + (uint64_t)grid * a.dim;
  const size_t half = a.turned / 2;
  const size_t smem = std::max(half * 8 * (1 + kWarps), BACK ? kWarps * a.dim * sizeof(float) : 0);
  launch_pdl(heads_kernel<T, V, NU, PAIRS, BACK, FIT>, grid, 32 * kWarps, smem, s, a);
  return grid;
}

// L: the least power of two of lanes that hold a head with NU units each.
uint32_t lanes_for(uint32_t units, uint32_t nu) {
  uint32_t l = 1;
  while (l * nu < units) l *= 2;
  return l;
}

template <typename T, bool PAIRS, bool BACK>
uint32_t heads_typed(HeadArgs a, bool packs, cudaStream_t s) {
  const uint32_t pairs = (a.dim + 1) / 2;
  a.units = packs ? pairs / kPack : pairs;
  // two units per lane where 32 lanes do not hold a head: more than 256 elements
  if (packs && a.units <= 32) {
    a.lanes = lanes_for(a.units, 1);
    return launch_heads<T, kPack, 1, PAIRS, BACK, BACK ? 2 : 4>(a, s);
  }
  if (packs) {
    a.lanes = 32;
    return launch_heads<T, kPack, 2, PAIRS, BACK, BACK ? 1 : 2>(a, s);
  }
  if (a.units <= 64) {
    a.lanes = lanes_for(a.units, 2);
    return launch_heads<T, 1, 2, PAIRS, BACK, BACK ? 2 : 4>(a, s);
  }
  a.lanes = 32;
  return launch_heads<T, 1, 8, PAIRS, BACK, 1>(a, s);
}

template <typename T>
uint32_t heads_any(const HeadArgs& a, bool pairs, bool back, cudaStream_t s) {
  bool packs = a.turned % (2 * kPack) == 0 && (a.dim - a.turned) % (2 * kPack) == 0;
  for (const Side& d : a.side)
    for (const Heads* h : {&d.x, &d.g, &d.out})
      packs = packs && (!d.heads || (aligned_to(h->p, sizeof(Pack<T, kPack>)) &&
                                   h->token % kPack == 0 && h->head % kPack == 0));
  if (back)
    return pairs ? heads_typed<T, true, true>(a, packs, s)
                 : heads_typed<T, false, true>(a, packs, s);
  return pairs ? heads_typed<T, true, false>(a, packs, s)
               : heads_typed<T, false, false>(a, packs, s);
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
int check_heads(const HeadArgs& a, int32_t type, int32_t weight_type) {
  if (!type_ok(type) || !type_ok(weight_type) || a.tokens > 0x7fffffffull || a.dim < 1 ||
      a.dim > kMostDim || a.turned > a.dim || a.turned % 2 || !(a.eps >= 0.f))
    return SPARCML_ERR_INVALID_ARG;
  for (const Side& d : a.side)
    if (d.heads > 65535 || (d.heads && !aligned_to(d.w, type_bytes(weight_type))))
      return SPARCML_ERR_INVALID_ARG;
  if (a.tokens == 0 || a.side[0].heads + a.side[1].heads == 0) return SPARCML_OK;
  const size_t e = type_bytes(type);
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

extern "C" int sparcml_head_norm_rotary(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, uint32_t q_heads, const void* k,
    int64_t k_token_stride, int64_t k_head_stride, uint32_t k_heads, int32_t type, uint64_t tokens,
    uint32_t dim, const void* positions, int32_t positions_int64, const float* freqs,
    uint32_t turned, int32_t interleaved, const void* q_weight, const void* k_weight,
    int32_t weight_type, float eps, void* q_out, int64_t q_out_token_stride,
    int64_t q_out_head_stride, void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
    void* stream) {
  const ApiRange nvtx_range(__func__);
  HeadArgs a = {};
  const Heads none = {nullptr, 0, 0};
  a.side[0] = {{q, q_token_stride, q_head_stride}, none,
               {q_out, q_out_token_stride, q_out_head_stride}, q_weight, q_heads, 0};
  a.side[1] = {{k, k_token_stride, k_head_stride}, none,
               {k_out, k_out_token_stride, k_out_head_stride}, k_weight, k_heads, 0};
  a.tokens = tokens;
  a.dim = dim;
  a.turned = turned;
  a.positions = positions;
  a.wide = positions_int64;
  a.freqs = freqs;
  a.w_type = weight_type;
  a.eps = eps;
  const int r = check_heads(a, type, weight_type);
  if (r != SPARCML_OK) return r;
  if (tokens == 0 || q_heads + k_heads == 0) return SPARCML_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == SPARCML_F32) heads_any<float>(a, interleaved, false, s);
  else if (type == SPARCML_BF16) heads_any<__nv_bfloat16>(a, interleaved, false, s);
  else heads_any<__half>(a, interleaved, false, s);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
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

extern "C" int sparcml_head_norm_rotary_backward(
    const void* dq, int64_t dq_token_stride, int64_t dq_head_stride, const void* dk,
    int64_t dk_token_stride, int64_t dk_head_stride, const void* q, int64_t q_token_stride,
    int64_t q_head_stride, uint32_t q_heads, const void* k, int64_t k_token_stride,
    int64_t k_head_stride, uint32_t k_heads, int32_t type, uint64_t tokens, uint32_t dim,
    const void* positions, int32_t positions_int64, const float* freqs, uint32_t turned,
    int32_t interleaved, const void* q_weight, const void* k_weight, int32_t weight_type, float eps,
    void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride, void* k_out,
    int64_t k_out_token_stride, int64_t k_out_head_stride, float* q_dweight, float* k_dweight,
    int32_t accumulate, void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  HeadArgs a = {};
  a.side[0] = {{q, q_token_stride, q_head_stride}, {dq, dq_token_stride, dq_head_stride},
               {q_out, q_out_token_stride, q_out_head_stride}, q_weight, q_heads, 0};
  a.side[1] = {{k, k_token_stride, k_head_stride}, {dk, dk_token_stride, dk_head_stride},
               {k_out, k_out_token_stride, k_out_head_stride}, k_weight, k_heads, 0};
  a.tokens = tokens;
  a.dim = dim;
  a.turned = turned;
  a.positions = positions;
  a.wide = positions_int64;
  a.freqs = freqs;
  a.w_type = weight_type;
  a.eps = eps;
  const int r = check_heads(a, type, weight_type);
  if (r != SPARCML_OK) return r;
  if (!ws || !aligned_to(ws, 256) || !aligned_to(q_dweight, 4) || !aligned_to(k_dweight, 4))
    return SPARCML_ERR_INVALID_ARG;
  const bool work = tokens && q_heads + k_heads;
  for (const Side& d : a.side)
    if (work && !input_ok(d.g, d.heads, type_bytes(type))) return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < sparcml_head_norm_rotary_backward_workspace_size(tokens, q_heads, k_heads, dim))
    return SPARCML_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool sums = q_dweight || k_dweight;
  uint32_t parts = 0;
  if (work) {
    if (sums) a.part[0] = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    parts = type == SPARCML_F32    ? heads_any<float>(a, interleaved, true, s)
            : type == SPARCML_BF16 ? heads_any<__nv_bfloat16>(a, interleaved, true, s)
                                   : heads_any<__half>(a, interleaved, true, s);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  if (sums) {
    launch_pdl(join_columns_kernel, dim3((dim + 31) / 32, 2), 512, 0, s,
               static_cast<const float*>(a.part[0]),
               static_cast<const float*>(a.part[0] + (uint64_t)parts * dim), parts, (uint64_t)dim,
               q_dweight, k_dweight, accumulate);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
    note_launches(1);
  }
  return SPARCML_OK;
}
