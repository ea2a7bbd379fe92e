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

// Sixteen consecutive elements, those from `left` on as zeros; PACKS: they are aligned and all
// there.
template <typename T, bool PACKS>
__device__ __forceinline__ void load16(const T* p, int left, float (&f)[16]) {
  if constexpr (PACKS) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < 16 / V; ++q) {
      F2 two[V / 2];
      unpack<T, V>(load_raw<T, V>(p + q * V), two);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        f[q * V + 2 * i] = two[i].x;
        f[q * V + 2 * i + 1] = two[i].y;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = i < left ? to_f32(p[i]) : 0.f;
  }
}
template <typename T, bool PACKS>
__device__ __forceinline__ void store16(T* p, int left, const float (&f)[16]) {
  if constexpr (PACKS) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int q = 0; q < 16 / V; ++q) {
      F2 two[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) two[i] = f2(f[q * V + 2 * i], f[q * V + 2 * i + 1]);
      *reinterpret_cast<uint4*>(p + q * V) = pack<T, V>(two);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) p[i] = from_f32<T>(f[i]);
  }
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

template <typename T, bool PACKS>
__global__ void __launch_bounds__(256) store_kernel(const StoreArgs a) {
  griddep_wait();
  constexpr bool kHalf = std::is_same_v<T, __half>;
  GroupWalk at(a.groups);
  const uint32_t lane = lane_id() & 7u;
  // every lane of a warp takes part in its shuffles: the warp goes on while any octet has work
  for (; __any_sync(0xffffffffu, at.row < a.rows); at.next()) {
    const bool active = at.row < a.rows;
    const uint64_t c = (uint64_t)at.group * kGroup + 16 * lane;
    const int left = active && c < a.dim ? (a.dim - c < 16 ? (int)(a.dim - c) : 16) : 0;
    float f[16];
    const T* x = static_cast<const T*>(a.x) + (int64_t)at.row * a.x_stride + c;
    if (left == 16) {
      load16<T, PACKS>(x, 16, f);
    } else {
      load16<T, false>(x, left, f);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const uint32_t b = exponent_byte(top, kHalf ? 103 : 1, kHalf ? 136 : 248);
    const bool fine = b != kNanExponent;
    const float by = __uint_as_float((fine ? 254u - b : 127u) << 23);  // 2^-e
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // clamped for the largest exponent's sake; 1.5 2^23 leaves the code in the low byte
        const float v = fminf(fmaxf(f[4 * q + i] * by, -127.f), 127.f);
        r[i] = __float_as_uint(v + 12582912.f);
      }
      w[q] = fine ? __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040),
                                0x5410)
                  : 0u;
    }
    if (left > 0)  // the row's padding to whole 16 bytes is written as zeros
      *reinterpret_cast<uint4*>(a.codes + (int64_t)at.row * a.codes_stride + c) =
          make_uint4(w[0], w[1], w[2], w[3]);
    if (active && lane == 0)
      a.exponents[(int64_t)at.row * a.exponents_stride + at.group] = (uint8_t)b;
  }
}

// Sixteen codes as floats, without their scale.
__device__ __forceinline__ void codes16(uint4 v, float (&f)[16]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * q + i] = code_at(w[q], i);
  }
}

template <typename T, bool PACKS>
__global__ void __launch_bounds__(256) restore_kernel(const StoreArgs a) {
  griddep_wait();
  GroupWalk at(a.groups);
  const uint32_t lane = lane_id() & 7u;
  for (; at.row < a.rows; at.next()) {
    const uint64_t c = (uint64_t)at.group * kGroup + 16 * lane;
    if (c >= a.dim) continue;
    const int left = a.dim - c < 16 ? (int)(a.dim - c) : 16;
    const float scale =
        scale_of(a.exponents[(int64_t)at.row * a.exponents_stride + at.group]);
    float f[16];
    codes16(*reinterpret_cast<const uint4*>(a.codes + (int64_t)at.row * a.codes_stride + c), f);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= scale;
    T* y = static_cast<T*>(a.x) + (int64_t)at.row * a.x_stride + c;
    if (left == 16)
      store16<T, PACKS>(y, 16, f);
    else
      store16<T, false>(y, left, f);
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

// Sixteen columns per thread, whose sums over the rows stay in its registers, as do its weights.
// PACKS: the columns are consecutive; else LANES apart, so that neighbouring threads read
// neighbouring elements at any alignment.
template <typename T, bool PACKS, int LANES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm8_backward_kernel(const Norm8Args a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ float2 scratch[66 * (MAXT / 64)];
  Group g = make_group(a.threads, scratch);
  const uint32_t threads = a.threads, groups = blockDim.x / threads, t = g.t;
  const uint32_t dim = (uint32_t)a.dim;
  const float inv = 1.0f / (float)dim;
  const uint32_t first = PACKS ? 16 * t : t / LANES * (16 * LANES) + t % LANES;
  const int left = (int)dim - (int)first;
  auto column = [&](int i) { return PACKS ? i : i * LANES; };  // from the first
  float w[16], gw[16], gb[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    gw[i] = gb[i] = 0.f;
    w[i] = a.w && column(i) < left ? load_any(a.w, a.w_type, first + column(i)) : 1.f;
  }
  const uint64_t step = (uint64_t)gridDim.x * groups;
  constexpr int kScales = PACKS ? 1 : LANES / 8;  // groups of 128 that the columns lie in
  constexpr int kDy = PACKS ? (int)sizeof(T) : 1;  // 16-byte pieces of dy
  uint4 dy_next[kDy], codes_next;
  uint32_t exp_next = 0;
  float mean_next = 0.f, rstd_next = 0.f;
  auto fetch = [&](uint64_t row) {
    if (row >= a.rows) return;
    mean_next = a.mean[row];
    rstd_next = a.rstd[row];
    if constexpr (PACKS) {
      if (left <= 0) return;
      const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride + first;
#pragma unroll
      for (int q = 0; q < kDy; ++q) dy_next[q] = reinterpret_cast<const uint4*>(dy)[q];
      codes_next =
          *reinterpret_cast<const uint4*>(a.codes + (int64_t)row * a.codes_stride + first);
      exp_next = a.exponents[(int64_t)row * a.exponents_stride + first / kGroup];
    }
  };
  uint64_t base = (uint64_t)blockIdx.x * groups;
  fetch(base + g.index);
  for (; base < a.rows; base += step) {  // the same turns for all groups of threads
    const uint64_t row = base + g.index;
    const bool active = row < a.rows;
    const int in = active ? left : 0;
    const float mean = mean_next, rstd = rstd_next;
    float xh[16], d[16];
    if constexpr (PACKS) {
      if (in > 0) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < kDy; ++q) {
          Raw<T, V> r;
          r.w = dy_next[q];
          F2 two[V / 2];
          unpack<T, V>(r, two);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            d[q * V + 2 * i] = two[i].x;
            d[q * V + 2 * i + 1] = two[i].y;
          }
        }
        codes16(codes_next, xh);
        const float by = scale_of(exp_next);
#pragma unroll
        for (int i = 0; i < 16; ++i) xh[i] = (xh[i] * by - mean) * rstd;
      }
      fetch(row + step);
    } else {
      const T* dy = static_cast<const T*>(a.dy) + (int64_t)row * a.dy_stride + first;
      const int8_t* x = a.codes + (int64_t)row * a.codes_stride + first;
      const uint8_t* ex = a.exponents + (int64_t)row * a.exponents_stride + first / kGroup;
      float by[kScales];
#pragma unroll
      for (int k = 0; k < kScales; ++k) by[k] = k * 128 < in ? scale_of(ex[k]) : 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool there = column(i) < in;
        d[i] = there ? to_f32(dy[column(i)]) : 0.f;
        xh[i] = there ? ((float)x[column(i)] * by[i * kScales / 16] - mean) * rstd : 0.f;
      }
      fetch(row + step);
    }
    float2 s = make_float2(0.f, 0.f);
    if (!PACKS || in > 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        gw[i] += d[i] * xh[i];
        gb[i] += d[i];
        d[i] *= w[i];
        s.x += d[i];
        s.y += d[i] * xh[i];
      }
    }
    s = g.sum2(s);
    if (in <= 0) continue;
    // dx = rstd (d - sum(d) / dim - xh sum(d xh) / dim)
    const float k1 = -s.x * inv * rstd, k2 = -s.y * inv * rstd;
#pragma unroll
    for (int i = 0; i < 16; ++i) d[i] = xh[i] * k2 + (d[i] * rstd + k1);
    T* dx = static_cast<T*>(a.dx) + (int64_t)row * a.dx_stride + first;
    if constexpr (PACKS) {
      store16<T, true>(dx, 16, d);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (column(i) < in) dx[column(i)] = from_f32<T>(d[i]);
    }
  }
  if (a.part_w == nullptr) return;  // neither sum is wanted
  float* to_w = a.part_w + (uint64_t)blockIdx.x * a.dim;
  float* to_b = a.part_b + (uint64_t)blockIdx.x * a.dim;
  if (groups == 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (column(i) < left) {
        to_w[first + column(i)] = gw[i];
        to_b[first + column(i)] = gb[i];
      }
    return;
  }
  // the groups' sums one after the other, in shared memory
  float* join = reinterpret_cast<float*>(dynamic);  // [groups][2][dim]
  float* set = join + (uint64_t)g.index * 2 * dim;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (column(i) < left) {
      set[first + column(i)] = gw[i];
      set[dim + first + column(i)] = gb[i];
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

template <typename T, bool PACKS, int LANES, int MAXT, int MINB>
bool launch_norm8(const Norm8Args& a, const BackwardShape& h, cudaStream_t s) {
  auto kernel = norm8_backward_kernel<T, PACKS, LANES, MAXT, MINB>;
  const uint32_t groups = h.block / h.threads;
  const size_t smem = groups > 1 ? 2ull * groups * a.dim * sizeof(float) : 0;
  if (smem > 40 * 1024 && !ensure_smem(reinterpret_cast<const void*>(kernel), smem)) return false;
  launch_pdl(kernel, h.parts, h.block, smem, s, a);
  return true;
}
template <typename T, bool PACKS>
bool launch_norm8_shape(const Norm8Args& a, const BackwardShape& h, cudaStream_t s) {
  if (h.threads == 8) return launch_norm8<T, PACKS, 8, 256, kFit>(a, h, s);
  if (h.threads == 16) return launch_norm8<T, PACKS, 16, 256, kFit>(a, h, s);
  if (h.block <= 256) return launch_norm8<T, PACKS, 32, 256, kFit>(a, h, s);
  return launch_norm8<T, PACKS, 32, 512, 1>(a, h, s);
}

template <typename T>
bool norm8_typed(Norm8Args a, float* dweight, float* dbias, int32_t accumulate, uint8_t* ws,
                 cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool packs = a.dim % 16 == 0 && a.dy_stride % V == 0 && a.dx_stride % V == 0 &&
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
    ok = packs ? launch_norm8_shape<T, true>(a, h, s) : launch_norm8_shape<T, false>(a, h, s);
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
