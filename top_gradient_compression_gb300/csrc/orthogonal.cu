// Orthogonalisation of an update by Newton-Schulz products, and the weight
// step built on it.
//
// With k the smaller side of X and S = X X' (or X' X where X is tall), a step is
//     S = X X',  P = b S + c S S,  X <- a X + P X   (X <- a X + X P)
// five products of which the first two are symmetric: only their tiles on and
// below the diagonal are computed, each written a second time as its mirror
// image. The tall case needs no transpose: the same row-major X is read by the
// tensor cores with its other side as the contiguous one.
//
// Operands are fp16 with fp32 accumulators. X is scaled by 2^12, S by 2^12 and
// P by 2^11: singular values stay near 1 at most, so nothing overflows, and
// entries far below the usual 1 / sqrt(m n) still have all their bits. bf16 operands
// would lose 8 times as much: the result would be 1 % off where fp16 is 0.15 % off.
// X itself is kept as a pair of fp16, hi + lo. The products read hi. The term
// a X, repeated over the steps, multiplies small singular values several
// hundred times, and with them any rounding of X, which has no rank of its
// own: from the single fp16 a quickly decaying spectrum comes out 2 % off, from
// the pair 0.02 %. The rounding of S and P is not multiplied so.

#include <algorithm>

#include "tensor.cuh"
#include "types.cuh"

namespace sparcml {
namespace {

constexpr float kScaleX = 4096.f, kScaleS = 4096.f, kScaleP = 2048.f;

// ---------------------------------------------------------------------------
// Momentum, norm and split of the input.

struct GatherArgs {
  const void* g;
  int32_t g_type;
  int64_t g_batch, g_stride;
  float* mom;  // null: the input is g itself
  int64_t m_batch, m_stride;
  float mu;
  int32_t nesterov;
  uint64_t m, n;
  uint32_t blocks;  // per matrix
  float* sums;      // [batch][blocks][3]
  __half* hi;       // [batch][m][pitch]
  __half* lo;
  uint64_t pitch;
};

// Sums of squares in three ranges (Blue, ACM TOMS 4, 1978), so that no square
// overflows or vanishes: entries above 2^40 scaled by 2^-90, below 2^-50 by 2^80.
__device__ __forceinline__ void add_square(float v, float (&s)[3]) {
  const float a = fabsf(v);
  if (a > 0x1p40f) {
    const float t = a * 0x1p-90f;
    s[2] += t * t;
  } else if (a < 0x1p-50f) {
    const float t = a * 0x1p80f;
    s[0] += t * t;
  } else {
    s[1] += a * a;
  }
}

// M <- mu M + G where there is a momentum, and the partial sums of squares of U.
__global__ void __launch_bounds__(256) gather_norm_kernel(const GatherArgs a) {
  griddep_wait();
  __shared__ float warp_sums[8][3];
  const uint64_t b = blockIdx.y, total = a.m * a.n;
  float s[3] = {0.f, 0.f, 0.f};
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (uint64_t)a.blocks * 256) {
    const uint64_t r = i / a.n, c = i % a.n;
    float u = load_any(a.g, a.g_type, b * a.g_batch + r * a.g_stride + c);
    if (a.mom) {
      float* mp = a.mom + b * a.m_batch + r * a.m_stride + c;
      const float m = a.mu * *mp + u;
      *mp = m;
      u = a.nesterov ? u + a.mu * m : m;
    }
    add_square(u, s);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    s[q] = warp_sum_f(s[q]);
    if (lane_id() == 0) warp_sums[threadIdx.x >> 5][q] = s[q];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float t = 0.f;
    for (int w = 0; w < 8; ++w) t += warp_sums[w][threadIdx.x];
    a.sums[(b * a.blocks + blockIdx.x) * 3 + threadIdx.x] = t;
  }
}

// The scaled input as a pair of fp16. 2^12 / |U| is applied as two factors, each a
// normal number, whatever the size of |U|.
__global__ void __launch_bounds__(256) split_kernel(const GatherArgs a) {
  griddep_wait();
  __shared__ float factors[2];
  const uint64_t b = blockIdx.y, total = a.m * a.n;
  if (threadIdx.x < 32) {
    double t[3] = {0.0, 0.0, 0.0};
    for (uint32_t k = threadIdx.x; k < a.blocks; k += 32)
      for (int q = 0; q < 3; ++q) t[q] += a.sums[(b * a.blocks + k) * 3 + q];
    for (int d = 16; d > 0; d >>= 1)
      for (int q = 0; q < 3; ++q) t[q] += __shfl_xor_sync(0xffffffffu, t[q], d);
    const double norm = sqrt(t[0] * 0x1p-160 + t[1] + t[2] * 0x1p180);
    if (threadIdx.x == 0) {
      float f0 = 0.f, f1 = 0.f;
      if (!(norm < __longlong_as_double(0x7ff0000000000000ll))) {
        f0 = f1 = __int_as_float(0x7fffffff);  // an inf or a NaN in U: all of X is NaN
      } else if (norm > 0.0) {
        int e;
        const double mant = frexp(norm, &e);
        f0 = ldexpf(1.f, -e / 2);
        f1 = (float)(ldexp((double)kScaleX, -(e - e / 2)) / mant);
      }
      factors[0] = f0;
      factors[1] = f1;
    }
  }
  __syncthreads();
  const float f0 = factors[0], f1 = factors[1];
  for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (uint64_t)gridDim.x * 256) {
    const uint64_t r = i / a.n, c = i % a.n;
    float u = load_any(a.g, a.g_type, b * a.g_batch + r * a.g_stride + c);
    if (a.mom) {
      const float m = a.mom[b * a.m_batch + r * a.m_stride + c];
      u = a.nesterov ? u + a.mu * m : m;
    }
    const float x = u * f0 * f1;
    const __half h = __float2half_rn(x);
    const uint64_t o = (b * a.m + r) * a.pitch + c;
    a.hi[o] = h;
    a.lo[o] = __float2half_rn(x - __half2float(h));
  }
}

// ---------------------------------------------------------------------------
// The products.

enum Epilogue { kGram = 0, kPoly = 1, kApply = 2, kOrthogonal = 3, kWeight = 4 };

struct ProductArgs {
  uint32_t rows, cols, depth;  // of the product, per matrix
  uint32_t tiles;              // per matrix
  uint32_t tile_cols;          // 0: the tiles on and below the diagonal
  float alpha, beta;           // result = alpha * product + beta * (what stands there)
  const __half* in_hi;         // kPoly: S; kApply and on: X
  __half* lo;
  __half* out_hi;
  uint64_t pitch;  // of in_hi, lo and out_hi
  void* out;       // kOrthogonal: O; kWeight: W
  int32_t out_type;
  int64_t out_batch, out_stride;
  float keep;  // kWeight: W <- keep W + (result)
  int32_t* status;
};

constexpr uint32_t kTile = 128, kDepth = 64, kStages = 4;
constexpr uint32_t kOperandBytes = kTile * kDepth * 2;
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kProductSmem = kStages * kStageBytes + 1024;

// One operand's tile of 128 rows and 64 k: two loads of 64 x 64.
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t row,
                                             uint32_t k, uint32_t b, uint32_t bar) {
#pragma unroll
  for (uint32_t h = 0; h < 2; ++h) {
    if (MN)
      tma_load_3d(dst + h * 8192, map, (int32_t)(row + 64 * h), (int32_t)k, (int32_t)b, bar);
    else
      tma_load_3d(dst + h * 8192, map, (int32_t)k, (int32_t)(row + 64 * h), (int32_t)b, bar);
  }
}

template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t step) {
  return MN ? tile_desc(addr + step * 2048, 8192, 1024) : tile_desc(addr + step * 32, 16, 1024);
}

// C = A B for one 128 x 128 tile per block: warp 0 loads, warp 1 issues the
// products, warps 2 to 5 write the result.
template <bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(192)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const ProductArgs p) {
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[2 * kStages + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t gave_up;
  const uint32_t warp = threadIdx.x >> 5;
  const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kStages, done = full + 16 * kStages;

  const uint32_t b = blockIdx.x / p.tiles, t = blockIdx.x % p.tiles;
  uint32_t ti, tj;
  if (p.tile_cols) {
    ti = t / p.tile_cols;
    tj = t % p.tile_cols;
  } else {
    ti = (uint32_t)((sqrtf(8.f * (float)t + 1.f) - 1.f) * 0.5f);
    while (ti * (ti + 1) / 2 > t) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= t) ++ti;
    tj = t - ti * (ti + 1) / 2;
  }
  const uint32_t row0 = ti * kTile, col0 = tj * kTile;

  if (threadIdx.x == 0) {
    gave_up = 0;
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(
                     smem_addr(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t steps = (p.depth + kDepth - 1) / kDepth;
  griddep_wait();

  if (warp == 0) {
    if (elect_one()) {
      uint32_t issued = 0;
      for (uint32_t i = 0; i < steps; ++i) {
        const uint32_t s = i % kStages;
        if (i >= kStages && !mbar_wait(empty + 8 * s, ((i / kStages) & 1u) ^ 1u, &gave_up)) break;
        mbar_expect_tx(full + 8 * s, kStageBytes);
        load_operand<A_MN>(base + s * kStageBytes, &map_a, row0, i * kDepth, b, full + 8 * s);
        load_operand<B_MN>(base + s * kStageBytes + kOperandBytes, &map_b, col0, i * kDepth, b,
                           full + 8 * s);
        ++issued;
      }
      // nothing of this block may still be in flight when it ends
      if (gave_up) {
        volatile uint32_t alone = 0;
        for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          mbar_wait(full + 8 * (i % kStages), (i / kStages) & 1u, &alone);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t idesc = mma_desc(kTile, kTile, A_MN, B_MN);
      for (uint32_t i = 0; i < steps; ++i) {
        const uint32_t s = i % kStages;
        if (!mbar_wait(full + 8 * s, (i / kStages) & 1u, &gave_up)) break;
        tmem_fence_after();
        const uint32_t sa = base + s * kStageBytes, sb = sa + kOperandBytes;
#pragma unroll
        for (uint32_t k = 0; k < kDepth / 16; ++k) {
          const uint64_t da = operand_desc<A_MN>(sa, k), db = operand_desc<B_MN>(sb, k);
          const uint32_t add = i > 0 || k > 0;
          asm volatile(
              "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
              "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}" ::"r"(tmem),
              "l"(da), "l"(db), "r"(idesc), "r"(add)
              : "memory");
        }
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                empty + 8 * s)
            : "memory");
      }
      asm volatile(
          "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(done)
          : "memory");
      if (gave_up) {  // tensor memory is freed below: no product may still run then
        volatile uint32_t alone = 0;
        mbar_wait(done, 0, &alone);
      }
    }
  } else if (__all_sync(0xffffffffu, mbar_wait(done, 0, &gave_up))) {
    tmem_fence_after();
    const uint32_t quarter = warp & 3u, lane = lane_id();
    const uint32_t row = row0 + quarter * 32 + lane;
    const uint64_t line = ((uint64_t)b * p.rows + row) * p.pitch;
    for (uint32_t c0 = 0; c0 < kTile; c0 += 32) {
      const uint32_t col = col0 + c0;
      if (col >= p.cols) break;
      float v[32];
      tmem_load32(tmem + (quarter << 21) + c0, v);
      tmem_load_wait();
#pragma unroll
      for (uint32_t i = 0; i < 32; ++i) v[i] *= p.alpha;
      if (EPI != kGram && row < p.rows) {
        if (EPI == kPoly) {
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            if (col + i < p.cols) v[i] += p.beta * __half2float(p.in_hi[line + col + i]);
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            if (col + i < p.cols)
              v[i] += p.beta * (__half2float(p.in_hi[line + col + i]) +
                                __half2float(p.lo[line + col + i]));
        }
      }
      if (EPI == kGram || EPI == kPoly) {
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) {
          const __half h = __float2half_rn(v[i]);
          if (row < p.rows && col + i < p.cols) {
            p.out_hi[line + col + i] = h;
            if (ti != tj)
              p.out_hi[((uint64_t)b * p.rows + col + i) * p.pitch + row] = h;
          }
        }
      } else if (row < p.rows) {
#pragma unroll
        for (uint32_t i = 0; i < 32; ++i) {
          if (col + i >= p.cols) continue;
          if (EPI == kApply) {
            const __half h = __float2half_rn(v[i]);
            p.out_hi[line + col + i] = h;
            p.lo[line + col + i] = __float2half_rn(v[i] - __half2float(h));
          } else {
            const int64_t o = (int64_t)b * p.out_batch + (int64_t)row * p.out_stride + col + i;
            float r = v[i];
            if (EPI == kWeight) r += p.keep * load_any(p.out, p.out_type, o);
            if (p.out_type == SPARCML_F32) static_cast<float*>(p.out)[o] = r;
            else if (p.out_type == SPARCML_BF16)
              static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(r);
            else static_cast<__half*>(p.out)[o] = __float2half_rn(r);
          }
        }
      }
    }
    tmem_fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && gave_up) set_status(p.status, SPARCML_ERR_TIMEOUT);
  if (warp == 0) {
    __syncwarp();
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem));
  }
}

// ---------------------------------------------------------------------------
// Host side.

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// fp16 [batch][rows][pitch], of which `cols` columns exist; boxes of 64 x 64.
bool make_map(CUtensorMap* map, const void* p, uint64_t batch, uint64_t rows, uint64_t cols,
              uint64_t pitch) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, batch};
  const cuuint64_t strides[2] = {pitch * 2, rows * pitch * 2};
  const cuuint32_t box[3] = {64, 64, 1}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  uint64_t batch, m, n, k, pitch, kpitch;
  uint32_t blocks;
  size_t sums, hi0, hi1, lo, s, p, bytes;
};

bool make_plan(int32_t batch, uint64_t m, uint64_t n, Plan& q) {
  if (batch < 0 || batch > 65535 || m < 1 || n < 1 || m > (1u << 24) || n > (1u << 24) ||
      std::min(m, n) > 32768)
    return false;
  q.batch = batch;
  q.m = m;
  q.n = n;
  q.k = std::min(m, n);
  q.pitch = align_up(n, 64);
  q.kpitch = align_up(q.k, 64);
  q.blocks = (uint32_t)std::min<uint64_t>((m * n + 4095) / 4096, 152 * 4);
  const size_t x = align_up(q.batch * m * q.pitch * 2, 256);
  const size_t s = align_up(q.batch * q.k * q.kpitch * 2, 256);
  size_t at = 256;
  auto take = [&](size_t bytes) { const size_t o = at; at += align_up(bytes, 256); return o; };
  q.sums = take(q.batch * q.blocks * 3 * sizeof(float));
  q.hi0 = take(x);
  q.hi1 = take(x);
  q.lo = take(x);
  q.s = take(s);
  q.p = take(s);
  q.bytes = at;
  return true;
}

template <bool A_MN, bool B_MN, int EPI>
bool launch_product(const CUtensorMap& a, const CUtensorMap& b, ProductArgs p, uint64_t batch,
                    bool symmetric, cudaStream_t s) {
  auto kernel = product_kernel<A_MN, B_MN, EPI>;
  if (!ensure_smem(reinterpret_cast<const void*>(kernel), kProductSmem)) return false;
  const uint64_t tr = (p.rows + kTile - 1) / kTile, tc = (p.cols + kTile - 1) / kTile;
  p.tile_cols = symmetric ? 0 : (uint32_t)tc;
  p.tiles = (uint32_t)(symmetric ? tr * (tr + 1) / 2 : tr * tc);
  if (p.tiles * batch > 0x7fffffffull) return false;
  launch_pdl(kernel, (unsigned)(p.tiles * batch), 192, kProductSmem, s, a, b, p);
  return true;
}

struct Target {  // where the result goes
  int epilogue;  // kOrthogonal or kWeight
  void* out;
  int32_t type;
  int64_t batch, stride;
  float alpha, keep;
};

int run_steps(GatherArgs g, const Plan& q, const Target& to, const float* coeffs, int32_t steps,
              void* ws, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  __half* hi[2] = {reinterpret_cast<__half*>(w + q.hi0), reinterpret_cast<__half*>(w + q.hi1)};
  __half* lo = reinterpret_cast<__half*>(w + q.lo);
  __half* gram = reinterpret_cast<__half*>(w + q.s);
  __half* poly = reinterpret_cast<__half*>(w + q.p);
  CUtensorMap map_x[2], map_s, map_p;
  if (!make_map(&map_x[0], hi[0], q.batch, q.m, q.n, q.pitch) ||
      !make_map(&map_x[1], hi[1], q.batch, q.m, q.n, q.pitch) ||
      !make_map(&map_s, gram, q.batch, q.k, q.k, q.kpitch) ||
      !make_map(&map_p, poly, q.batch, q.k, q.k, q.kpitch))
    return SPARCML_ERR_CUDA;
  g.m = q.m;
  g.n = q.n;
  g.blocks = q.blocks;
  g.sums = reinterpret_cast<float*>(w + q.sums);
  g.hi = hi[0];
  g.lo = lo;
  g.pitch = q.pitch;
  const dim3 grid(q.blocks, (unsigned)q.batch);
  launch_pdl(gather_norm_kernel, grid, 256, 0, s, g);
  launch_pdl(split_kernel, grid, 256, 0, s, g);
  const bool tall = q.m > q.n;
  const uint32_t k = (uint32_t)q.k, l = (uint32_t)std::max(q.m, q.n);
  int32_t* status = reinterpret_cast<int32_t*>(w);
  bool ok = true;
  for (int32_t i = 0; i < steps && ok; ++i) {
    const float ca = coeffs[3 * i], cb = coeffs[3 * i + 1], cc = coeffs[3 * i + 2];
    const CUtensorMap& x = map_x[i & 1];
    ProductArgs p = {};
    p.status = status;
    p.rows = p.cols = k;
    p.depth = l;
    p.pitch = q.kpitch;
    p.alpha = kScaleS / (kScaleX * kScaleX);
    p.out_hi = gram;
    ok = tall ? launch_product<true, true, kGram>(x, x, p, q.batch, true, s)
              : launch_product<false, false, kGram>(x, x, p, q.batch, true, s);
    p.depth = k;
    p.alpha = cc * kScaleP / (kScaleS * kScaleS);
    p.beta = cb * kScaleP / kScaleS;
    p.in_hi = gram;
    p.out_hi = poly;
    ok = ok && launch_product<false, false, kPoly>(map_s, map_s, p, q.batch, true, s);
    p.rows = (uint32_t)q.m;
    p.cols = (uint32_t)q.n;
    p.pitch = q.pitch;
    p.in_hi = hi[i & 1];
    p.lo = lo;
    p.out_hi = hi[(i + 1) & 1];
    const bool last = i + 1 == steps;
    const float f = last ? to.alpha / kScaleX : 1.f;
    p.alpha = f / kScaleP;
    p.beta = f * ca;
    p.out = to.out;
    p.out_type = to.type;
    p.out_batch = to.batch;
    p.out_stride = to.stride;
    p.keep = to.keep;
    const CUtensorMap& first = tall ? x : map_p;
    const CUtensorMap& second = tall ? map_p : x;
    auto apply = [&](auto epi) {
      constexpr int E = decltype(epi)::value;
      return tall ? launch_product<false, false, E>(first, second, p, q.batch, false, s)
                  : launch_product<false, true, E>(first, second, p, q.batch, false, s);
    };
    ok = ok && (!last ? apply(std::integral_constant<int, kApply>{})
                : to.epilogue == kWeight ? apply(std::integral_constant<int, kWeight>{})
                                         : apply(std::integral_constant<int, kOrthogonal>{}));
  }
  if (launch_status() != SPARCML_OK || !ok) return SPARCML_ERR_CUDA;
  note_launches(2 + 3 * steps);
  return SPARCML_OK;
}

// Whether no two elements of a batch of matrices share an address: the matrices
// lie one after the other, or their rows alternate.
bool apart(int64_t batch, uint64_t m, uint64_t n, int64_t batch_stride, int64_t stride) {
  if (batch_stride < 0 || stride < 0 || (m > 1 && stride < (int64_t)n)) return false;
  if (batch <= 1) return true;
  const int64_t w = (int64_t)n, h = (int64_t)m - 1;
  return batch_stride >= h * stride + w ||
         (batch_stride >= w && (h == 0 || stride >= (batch - 1) * batch_stride + w));
}

bool finite(float v) { return v - v == 0.f; }

int check_steps(const float* coeffs, int32_t steps) {
  if (steps < 1 || steps > 64 || !coeffs) return SPARCML_ERR_INVALID_ARG;
  for (int32_t i = 0; i < 3 * steps; ++i)
    if (!finite(coeffs[i])) return SPARCML_ERR_INVALID_ARG;
  return SPARCML_OK;
}

}  // namespace
}  // namespace sparcml

using namespace sparcml;

extern "C" size_t sparcml_orthogonalize_workspace_size(int32_t batch, uint64_t m, uint64_t n) {
  Plan q;
  return make_plan(batch, m, n, q) ? q.bytes : 0;
}

extern "C" int sparcml_orthogonalize(const void* g, int32_t g_type, int64_t g_batch_stride,
                                     int64_t g_stride, void* out, int32_t out_type,
                                     int64_t out_batch_stride, int64_t out_stride, int32_t batch,
                                     uint64_t m, uint64_t n, const float* coeffs, int32_t steps,
                                     void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  Plan q;
  if (!make_plan(batch, m, n, q) || !type_ok(g_type) ||
      (out_type != SPARCML_BF16 && out_type != SPARCML_F16) ||
      check_steps(coeffs, steps) != SPARCML_OK || !ws || !aligned_to(ws, 256))
    return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < q.bytes) return SPARCML_ERR_WORKSPACE;
  if (batch == 0) return SPARCML_OK;
  if (!g || !out || !aligned_to(g, type_bytes(g_type)) || !aligned_to(out, 2) ||
      g_batch_stride < 0 || g_stride < 0 || !apart(batch, m, n, out_batch_stride, out_stride))
    return SPARCML_ERR_INVALID_ARG;
  GatherArgs a = {};
  a.g = g;
  a.g_type = g_type;
  a.g_batch = g_batch_stride;
  a.g_stride = g_stride;
  const Target to{kOrthogonal, out, out_type, out_batch_stride, out_stride, 1.f, 0.f};
  return run_steps(a, q, to, coeffs, steps, ws, static_cast<cudaStream_t>(stream));
}

extern "C" int sparcml_muon_step(void* weight, int32_t w_type, int64_t w_batch_stride,
                                 int64_t w_stride, const void* grad, int32_t g_type,
                                 int64_t g_batch_stride, int64_t g_stride, float* momentum,
                                 int64_t m_batch_stride, int64_t m_stride, int32_t batch,
                                 uint64_t m, uint64_t n, float mu, int32_t nesterov, float lr,
                                 float weight_decay, float scale, const float* coeffs,
                                 int32_t steps, void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  Plan q;
  if (!make_plan(batch, m, n, q) || !type_ok(w_type) || !type_ok(g_type) ||
      check_steps(coeffs, steps) != SPARCML_OK || !finite(mu) || !finite(lr) ||
      !finite(weight_decay) || !finite(scale) || !ws || !aligned_to(ws, 256))
    return SPARCML_ERR_INVALID_ARG;
  if (ws_bytes < q.bytes) return SPARCML_ERR_WORKSPACE;
  if (batch == 0) return SPARCML_OK;
  if (!weight || !grad || !momentum || !aligned_to(weight, type_bytes(w_type)) ||
      !aligned_to(grad, type_bytes(g_type)) || !aligned_to(momentum, 4) || g_batch_stride < 0 || g_stride < 0 ||
      !apart(batch, m, n, w_batch_stride, w_stride) ||
      !apart(batch, m, n, m_batch_stride, m_stride))
    return SPARCML_ERR_INVALID_ARG;
  GatherArgs a = {};
  a.g = grad;
  a.g_type = g_type;
  a.g_batch = g_batch_stride;
  a.g_stride = g_stride;
  a.mom = momentum;
  a.m_batch = m_batch_stride;
  a.m_stride = m_stride;
  a.mu = mu;
  a.nesterov = nesterov;
  const Target to{kWeight,  weight,      w_type, w_batch_stride,
                  w_stride, -lr * scale, 1.f - lr * weight_decay};
  return run_steps(a, q, to, coeffs, steps, ws, static_cast<cudaStream_t>(stream));
}
