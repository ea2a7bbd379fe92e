// Orthogonalisation of an update by Newton-Schulz products, and the weight
// step built on it.
//
// With k the smaller side of X and S = X X' (or X' X where X is tall), a step is
//     S = X X',  P = b S + c S S,  X <- a X + P X   (X <- a X + X P)
// three products of which the first two are symmetric: only their tiles on and
// below the diagonal are computed, each written a second time as its mirror
// image. The tall case needs no transpose: the same row-major X is read by the
// tensor cores with its other side as the contiguous one.
//
// One launch runs all steps: a persistent grid of one block per SM, whose
// blocks wait for one another between the products (15 products of five steps;
// as launches of their own each would cost the host 2 us and the device a start and an
// end). The matrices of a batch form two chains: a block works
// on one while the other's results are on their way, and neither waits for the other.
//
// Numbers. Operands are fp16 with fp32 accumulators. X and S are scaled by 2^12
// and P by 2^11: singular values stay near 1, so nothing overflows, and entries
// far below the usual 1 / sqrt(m n) still have all their bits. bf16 operands
// would lose 8 times as much. Two things are kept beyond that:
//   - X is a pair of fp16, hi + lo. The products read hi, the term a X both. It
//     multiplies small singular values several hundred times over the steps, and
//     with them any rounding of X: from hi alone a 1/i^2 spectrum comes out 2 %
//     off, from the pair 0.02 to 0.06 %. The rounding of S and P is not multiplied so.
//   - The diagonals of S and P are fp32 vectors s and p, and the fp16 matrices
//     hold zeros there: with S = s + S', S S = S' S' + s S' + S' s + s s and
//     P X = p X + P' X. X near orthogonal has S near the identity, and rounding
//     that diagonal was most of the error (in a simulation 0.15 to 0.2 % on flat
//     spectra). As it is, 100 x 300 to 4096 x 1024 come out 0.01 to 0.14 % off in the
//     Frobenius norm over flat, 1/sqrt(i), 1/i and 1/i^2 spectra and noise.

// A side of at most 64 needs no step of its own products. With S kept in fp32 all steps are
// polynomials of it, X <- q(S) X with
//     P = a + b S + c S S,  q <- P q,  S <- P S P,
// which one block works out in shared memory; X is read for S and for q(S) X alone, in
// products of all three leading pairs of the halves hi and lo. Three products in a row
// in place of fifteen, and exact to 1e-3 even on a 1/i^4 spectrum. S loses its sign where it
// is small against its own rounding, so this is left to coefficients that multiply small
// singular values 1800 times at most.

#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>

#include "tensor.cuh"
#include "types.cuh"

namespace sparcml {
namespace {

constexpr float kScaleX = 4096.f, kScaleS = 4096.f, kScaleP = 2048.f, kScaleQ = 32.f;
constexpr uint32_t kSmall = 64;  // the smaller side that one block takes

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
  int32_t vec_g, vec_m;  // rows of g, of mom: four elements are one aligned access
  int32_t flat;          // the rows of a matrix follow one another in both
  int32_t vec_flat_g, vec_flat_m;  // and four elements of that one row are such an access
  uint64_t m, n;
  uint32_t blocks;  // per matrix
  float* sums;      // [batch][blocks][3]
  uint32_t* turns;  // counters of arrivals, zeroed here: of the grid, of each chain
};
constexpr uint32_t kTurnStep = 8;  // words between counters

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

// Four consecutive elements of a row, those from `n` on as zeros; `vec`: all rows allow
// one access of four.
__device__ __forceinline__ void load4(const void* p, int32_t type, uint64_t at, uint64_t c,
                                      uint64_t n, bool vec, float (&v)[4]) {
  if (vec && c + 4 <= n) {
    if (type == SPARCML_F32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else if (type == SPARCML_BF16) {
      const auto f = *reinterpret_cast<const Pack<__nv_bfloat16, 4>*>(
          static_cast<const __nv_bfloat16*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = to_f32(f.e[i]);
    } else {
      const auto f =
          *reinterpret_cast<const Pack<__half, 4>*>(static_cast<const __half*>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = to_f32(f.e[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = c + i < n ? load_any(p, type, at + i) : 0.f;
  }
}

// A matrix is walked in pieces, a warp at a time, each lane with four groups of four columns:
// 64 or 128 bytes per lane in flight. A piece is 512 columns of a row, or several whole rows of
// at most 256 columns.
constexpr uint32_t kPiece = 512;

struct Pieces {
  uint32_t groups;  // of four columns, in a row
  uint32_t rows;    // in a piece, if there are several; else 1
  uint64_t across, total;  // pieces in a row (of one row each), in a matrix

  __host__ __device__ Pieces(uint64_t m, uint64_t n) {
    const uint64_t all = (n + 3) / 4;
    groups = all > 64 ? 0 : (uint32_t)all;
    rows = groups ? 128 / groups : 1;
    across = groups ? 1 : (n + kPiece - 1) / kPiece;
    total = groups ? (m + rows - 1) / rows : m * across;
  }
};
// Lane's group q of a piece: its row within the piece, and its first column.
struct Slots {
  uint32_t row[4], col[4];
  __device__ __forceinline__ explicit Slots(const Pieces& p) {
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint32_t at = 32 * q + lane_id();
      row[q] = p.groups ? at / p.groups : 0;
      col[q] = 4 * (p.groups ? at - row[q] * p.groups : at);
    }
  }
};

// M <- mu M + G where there is a momentum, and the partial sums of squares of U.
__global__ void __launch_bounds__(256) gather_norm_kernel(const GatherArgs a) {
  griddep_wait();
  __shared__ float warp_sums[8][3];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 3) a.turns[threadIdx.x * kTurnStep] = 0;
  const uint64_t b = blockIdx.y;
  // where rows follow one another they are one long row here
  const uint64_t m = a.flat ? 1 : a.m, n = a.flat ? a.m * a.n : a.n;
  const bool vec_g = a.flat ? a.vec_flat_g : a.vec_g, vec_m = a.flat ? a.vec_flat_m : a.vec_m;
  const Pieces pieces(m, n);
  const Slots slots(pieces);
  const uint64_t warps = (uint64_t)a.blocks * 8, id = blockIdx.x * 8ull + (threadIdx.x >> 5);
  const uint64_t end = pieces.total * (id + 1) / warps;
  uint64_t u = pieces.total * id / warps;
  uint64_t r0 = u / pieces.across * pieces.rows, piece = u % pieces.across;
  float s[3] = {0.f, 0.f, 0.f};
  for (; u < end; ++u) {
    float v[4][4], mo[4][4];
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint64_t r = r0 + slots.row[q], c = piece * kPiece + slots.col[q];
      const uint64_t in = slots.row[q] < pieces.rows && r < m ? n : 0;  // no columns, if no row
      load4(a.g, a.g_type, b * a.g_batch + r * a.g_stride + c, c, in, vec_g, v[q]);
      if (a.mom)
        load4(a.mom, SPARCML_F32, b * a.m_batch + r * a.m_stride + c, c, in, vec_m, mo[q]);
    }
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint64_t r = r0 + slots.row[q], c = piece * kPiece + slots.col[q];
      const uint64_t in = slots.row[q] < pieces.rows && r < m ? n : 0;
      if (a.mom) {
        float* mp = a.mom + b * a.m_batch + r * a.m_stride + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float t = a.mu * mo[q][i] + v[q][i];
          mo[q][i] = t;
          v[q][i] = a.nesterov ? v[q][i] + a.mu * t : t;
        }
        if (vec_m && c + 4 <= in) {
          *reinterpret_cast<float4*>(mp) = make_float4(mo[q][0], mo[q][1], mo[q][2], mo[q][3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < in) mp[i] = mo[q][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) add_square(v[q][i], s);
    }
    if (++piece == pieces.across) {
      piece = 0;
      r0 += pieces.rows;
    }
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

// ---------------------------------------------------------------------------
// The steps.

constexpr uint32_t kMaxSteps = 64;

struct Product {       // one product of a step, of every matrix of the batch
  uint32_t n;          // columns of a tile (rows: 128 per block)
  uint32_t rows, cols;  // of the result
  uint32_t blocks;     // of 64 along the summed axis
  uint32_t tile_rows;  // tiles down, or 0: those on and below the diagonal
  uint32_t tiles;      // per matrix
  uint32_t splits;     // parts of the summed axis, each an item of its own
  uint32_t whole;      // items of full width; those after them are halves of tiles
  uint32_t items;
  uint32_t b0;         // the chain's first matrix
  uint32_t offset;     // which block or pair takes item 0
  uint32_t part0;      // the chain's first partial tile
};

struct Maps {
  // What is added to the products, in boxes of 32 x 32, 64-byte swizzled.
  CUtensorMap x_out[2], lo_out, s_out;
  // Operands, one load of 128 rows (or one tile's columns) by 64 of the summed axis, 128-byte
  // swizzled: [0] the first operand, [1] the second. With a load per 64 x 64 the issue of
  // loads, over 100 cycles each, was what bounded the products.
  CUtensorMap x_gram[2][2], s_poly[2], x_apply[2], p_apply;
  CUtensorMap lo_gram[2], lo_apply, q_lo;  // for a small side: the lower halves
};

struct StepArgs {
  GatherArgs g;
  uint32_t batch, steps, tall, chains;
  Product product[2][3];  // of each chain: S, P, X
  float coeffs[3 * kMaxSteps];
  __half* hi[2];  // [batch][m][pitch]
  __half* lo;
  __half* s;  // [batch][k][kpitch]
  __half* p;
  uint64_t pitch, kpitch;
  float* diag_s;  // [batch][k]
  float* diag_p;
  float* part;  // partial tiles of a split product
  uint32_t k;
  uint32_t weight;  // result: 1 the weight step, 0 the orthogonal matrix itself
  void* out;
  int32_t out_type;
  int64_t out_batch, out_stride;
  float alpha, keep;  // weight: W <- keep W + alpha X; else X
  int32_t* status;
  const uint32_t* inject;  // the workspace's fault-injection word
};

enum Kind { kGram, kPart, kJoin, kSolve, kPoly, kApply, kLast };

constexpr uint32_t kWriters = 8;  // warps that write results; then a loader and an issuer
constexpr uint32_t kThreads = 32 * (kWriters + 2);
constexpr uint32_t kRingBytes = 160 * 1024, kMaxStages = 6;
constexpr uint32_t kStageBuf = 4096;  // per writer, twice
constexpr uint32_t kStepsSmem = kRingBytes + kWriters * 2 * kStageBuf + 1024;
constexpr uint32_t kAccColumns = 256;  // two accumulators in the 512 columns of tensor memory

struct Tile {
  uint32_t b, row0, col0, n, first, last;  // blocks [first, last) of the summed axis
  bool mirror;                          // write its mirror image too
  bool none;                            // beyond the last column
};

// Item i of a product: the splits of one tile are neighbours, and tiles run down
// the columns first, so that the blocks working at one time share few columns
// of the larger operand.
template <int CG>
__device__ __forceinline__ Tile tile_of(const Product& p, uint32_t item) {
  Tile t;
  uint32_t split = 0, u = item, half = 0;
  t.n = p.n;
  if (p.splits > 1) {
    u = item / p.splits;
    split = item - u * p.splits;
  } else if (item >= p.whole) {
    u = p.whole + (item - p.whole) / 2;
    half = (item - p.whole) & 1u;
    t.n = p.n / 2;
  }
  t.b = u / p.tiles;
  u -= t.b * p.tiles;
  t.b += p.b0;
  uint32_t i, j;
  t.mirror = false;
  if (p.tile_rows) {
    j = u / p.tile_rows;
    i = u - j * p.tile_rows;
  } else {
    const uint32_t ratio = 128 * CG / p.n, v = u / ratio;
    i = (uint32_t)((sqrtf(8.f * (float)v + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > v) --i;
    while ((i + 1) * (i + 2) / 2 <= v) ++i;
    j = u - ratio * (i * (i + 1) / 2);
    t.mirror = j < ratio * i;
  }
  t.row0 = i * 128 * CG;
  t.col0 = j * p.n + half * t.n;
  t.none = t.col0 >= p.cols;
  t.first = 0;
  t.last = p.blocks;
  if (p.splits > 1) {  // at most 2^18 blocks in at most 152 parts
    t.first = p.blocks * split / p.splits;
    t.last = p.blocks * (split + 1) / p.splits;
  }
  return t;
}
// Has the tile worked out, or the product's parameters read, here and not where they are
// first used.
__device__ __forceinline__ void pin(Tile& t) {
  asm volatile("" : "+r"(t.b), "+r"(t.row0), "+r"(t.col0), "+r"(t.n), "+r"(t.first), "+r"(t.last));
}
__device__ __forceinline__ void pin(Product& p) {
  asm volatile("" : "+r"(p.n), "+r"(p.rows), "+r"(p.cols), "+r"(p.items), "+r"(p.splits),
               "+r"(p.tiles), "+r"(p.part0));
}

// Byte offset of 16-byte piece c of row r in a 32 x 32 fp16 box, 64-byte swizzled.
__device__ __forceinline__ uint32_t box_at(uint32_t r, uint32_t c) {
  return r * 64 + ((c ^ ((r >> 1) & 3u)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// The state of one block.
template <int CG>
struct Worker {
  __device__ __forceinline__ void next_stage() {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }

  uint32_t ring, stages, stage_bytes;      // operand ring
  uint32_t full, empty, acc_full, acc_empty, in_bar;  // barriers
  uint32_t lead_full, lead_acc_empty;      // the same of the pair's first block
  uint32_t buf;                            // this writer's two buffers
  uint32_t rank, cluster, clusters, tmem;
  bool leader;                             // the lane that issues for its warp
  Waits* waits;
  uint32_t stage = 0, phase = 0;  // next operand stage and its turn's parity (loader, issuer)
  uint32_t acc = 0;       // accumulators used so far (issuer, writers)
  uint32_t in_phase = 0;  // bit s: parity of buffer s's next load
  uint32_t turn = 0;      // chunks written so far

  // The first of this block's items.
  __device__ __forceinline__ uint32_t first_item(const Product& p) const {
    return cluster >= p.offset ? cluster - p.offset : cluster + clusters - p.offset;
  }
};

// The loader and the issuer run as whole warps, of which one lane issues: so the addresses
// and the control flow are known to be uniform (a lane on its own took 700 cycles per
// block of the summed axis, where the products take 512).
template <int CG, bool SMALL>
__device__ __forceinline__ bool load_operands(Worker<CG>& w, const Product& p,
                                              const CUtensorMap* ma, const CUtensorMap* mb,
                                              const CUtensorMap* ma_lo, const CUtensorMap* mb_lo,
                                              bool a_mn, bool b_mn, Tile t) {
  for (uint32_t item = w.first_item(p); item < p.items; item += w.clusters) {
    if (item >= w.clusters) t = tile_of<CG>(p, item);
    if (t.none) continue;
    const uint32_t bytes = 128 * 128 + p.n / CG * 128;  // halves of tiles use half of theirs
    const uint32_t ra = t.row0 + 128 * w.rank, rb = t.col0 + t.n / CG * w.rank;
    uint32_t rep = 0;
    for (uint32_t i = t.first; i < t.last; w.next_stage()) {
      const uint32_t s = w.stage;
      if (!mbar_wait_warp(w.empty + 8 * s, w.phase ^ 1u, w.waits)) return false;
      // of a small side's operands hi hi, hi lo, lo hi; else hi hi alone
      const CUtensorMap* const ua = SMALL && rep == 2 ? ma_lo : ma;
      const CUtensorMap* const ub = SMALL && rep == 1 ? mb_lo : mb;
      if (w.leader) {
        if (w.rank == 0) mbar_expect_tx(w.full + 8 * s, CG * bytes);
        const uint32_t bar = w.lead_full + 8 * s, k = i * 64;
        const uint32_t dst = w.ring + s * w.stage_bytes;
        tma_load_4d<CG>(dst, ua, a_mn ? 0 : k, a_mn ? k : ra, a_mn ? ra / 64 : 0, t.b, bar);
        tma_load_4d<CG>(dst + 128 * 128, ub, b_mn ? 0 : k, b_mn ? k : rb, b_mn ? rb / 64 : 0, t.b,
                        bar);
      }
      __syncwarp();
      if (!SMALL || ++rep == 3) {
        rep = 0;
        ++i;
      }
    }
  }
  return true;
}

template <int CG, bool SMALL>
__device__ __forceinline__ bool issue_products(Worker<CG>& w, const Product& p, bool a_mn, bool b_mn, Tile t) {
  const uint32_t step_a = a_mn ? 2048 : 32, step_b = b_mn ? 2048 : 32;
  for (uint32_t item = w.first_item(p); item < p.items; item += w.clusters) {
    if (item >= w.clusters) t = tile_of<CG>(p, item);
    if (t.none) continue;
    const uint32_t idesc = mma_desc(128 * CG, t.n, a_mn, b_mn);
    const uint32_t a = w.acc & 1u;
    if (!mbar_wait_warp(w.acc_empty + 8 * a, ((w.acc >> 1) & 1u) ^ 1u, w.waits)) return false;
    tmem_fence_after();
    const uint32_t d = w.tmem + a * kAccColumns;
    const uint32_t blocks = (t.last - t.first) * (SMALL ? 3 : 1);
    for (uint32_t i = 0; i < blocks; ++i, w.next_stage()) {
      const uint32_t s = w.stage;
      if (!mbar_wait_warp(w.full + 8 * s, w.phase, w.waits)) return false;
      tmem_fence_after();
      if (w.leader) {
        const uint32_t sa = w.ring + s * w.stage_bytes, sb = sa + 128 * 128;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          mma_f16<CG>(d, tile_desc(sa + k * step_a, 8192, 1024),
                      tile_desc(sb + k * step_b, 8192, 1024), idesc, i > 0 || k > 0);
        mma_commit<CG>(w.empty + 8 * s);
      }
      __syncwarp();
    }
    if (w.leader) mma_commit<CG>(w.acc_full + 8 * a);
    __syncwarp();
    ++w.acc;
  }
  return true;
}

// A 32 x 32 fp16 box in shared memory to rows [row0, row0 + 32) below `rows`, from column
// col, of a matrix whose padded rows hold whole boxes: eight rows of 64 bytes at a
// time. (A TMA store of such a box takes over a microsecond when all SMs issue them:
// 4096 x 4096 took 2.4 ms with it.)
__device__ __forceinline__ void store_box(uint32_t box, __half* out, uint64_t pitch, uint32_t row0,
                                          uint32_t rows, uint32_t col) {
  const uint32_t lane = lane_id(), r = lane >> 2, c = lane & 3u;
  __half* o = out + (uint64_t)(row0 + r) * pitch + col + 8 * c;
#pragma unroll
  for (uint32_t q = 0; q < 32; q += 8, o += 8 * pitch)
    if (row0 + q + r < rows) *reinterpret_cast<uint4*>(o) = lds128(box + box_at(q + r, c));
}

// Before a block leaves that gave up, or whose partner did: until the operands have landed. A
// pair's loads all report to the first block, in one phase per stage for both blocks; where the
// two stopped at different stages (`apart`) some phases never complete, and the loads get their
// time instead.
__device__ __noinline__ void land_operands(uint32_t full, uint32_t stages, uint32_t stage,
                                           uint32_t phase, bool apart) {
  if (apart) {
    const uint64_t end = global_ns() + 1000ull * kLandUs;
    while (global_ns() < end) __nanosleep(1000);
    return;
  }
  Waits alone = {0, kLandUs};
  for (uint32_t s = 0; s < stages; ++s)
    mbar_wait(full + 8 * s, s < stage ? phase : phase ^ 1u, &alone);
}

// What becomes of a product's entry, for all products alike:
//     r = f acc + (r0 + r1 d_j) in_ij
// with d the diagonal vector of column j, and in what stands at that place:
//     S = X X'                                    (nothing)
//     P' = c S' S' + (b + c s_i + c s_j) S'       S', rows' s in r0, columns' s by r1
//     X <- P' X + (a + p_i) X                     hi + lo; p_i in r0
//     X <- X P' + (a + p_j) X                     (tall) hi + lo; p_j by r1
// and on the diagonal of S and P the sum goes to an fp32 vector, with `on` added.
struct Rule {
  float f, r0, r1, on, diag_scale;
  float* diag;   // this matrix's, or null
  __half* out;   // this matrix's
  __half* low;   // X: the lower half of the pair
  uint64_t pitch;
  uint32_t rows;  // of out
};

// Sixteen columns from column 16 h of the 32 x 32 box: v holds this lane's row. All reads
// come before all arithmetic: a writer's time is the latency of its chain (with eight
// columns at a time a box took 1.2 us).
__device__ __forceinline__ void finish16(float (&v)[16], uint32_t h, uint32_t buf, bool reads,
                                         bool pairs, bool by_column, float other, const Rule& u,
                                         bool on_diag, uint32_t row) {
  const uint32_t lane = lane_id();
  if (reads) {
    uint4 h4[2], l4[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) h4[c] = lds128(buf + box_at(lane, 2 * h + c));
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = u.r0;
    if (by_column) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] += u.r1 * __shfl_sync(0xffffffffu, other, (int)(16 * h) + i);
    }
    if (pairs) {
#pragma unroll
      for (int c = 0; c < 2; ++c) l4[c] = lds128(buf + 2048 + box_at(lane, 2 * h + c));
    } else {
      l4[0] = l4[1] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t hw[4] = {h4[c].x, h4[c].y, h4[c].z, h4[c].w};
      const uint32_t lw[4] = {l4[c].x, l4[c].y, l4[c].z, l4[c].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 h2 = unpack_half(hw[e]), l2 = unpack_half(lw[e]);
        const int i = 8 * c + 2 * e;
        v[i] = v[i] * u.f + w[i] * (h2.x + l2.x);
        v[i + 1] = v[i + 1] * u.f + w[i + 1] * (h2.y + l2.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= u.f;
  }
  if (on_diag) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (lane == 16 * h + i) {
        if (row < u.rows) u.diag[row] = (v[i] + u.on) * u.diag_scale;
        v[i] = 0.f;
      }
  }
}

// The sixteen results as fp16 (and what that rounding left, for a pair) into the box, and
// into the box of its mirror image.
__device__ __forceinline__ void stage16(const float (&v)[16], uint32_t h, uint32_t buf, bool pairs,
                                        bool mirror) {
  const uint32_t lane = lane_id();
  uint32_t hw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) hw[e] = pack_half(v[2 * e], v[2 * e + 1]);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    sts128(buf + box_at(lane, 2 * h + c),
           make_uint4(hw[4 * c], hw[4 * c + 1], hw[4 * c + 2], hw[4 * c + 3]));
  if (pairs) {
    uint32_t lw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 back = unpack_half(hw[e]);
      lw[e] = pack_half(v[2 * e] - back.x, v[2 * e + 1] - back.y);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
      sts128(buf + 2048 + box_at(lane, 2 * h + c),
             make_uint4(lw[4 * c], lw[4 * c + 1], lw[4 * c + 2], lw[4 * c + 3]));
  } else if (mirror) {
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(buf + 2048 + box_at(16 * h + i, lane >> 3) +
                                                   (lane & 7u) * 2),
                   "h"((uint16_t)(i & 1 ? hw[i / 2] >> 16 : hw[i / 2]))
                   : "memory");
  }
}

__device__ __forceinline__ void store_boxes(uint32_t buf, const Rule& u, uint32_t row0,
                                            uint32_t col, bool pairs, bool mirror) {
  __syncwarp();
  store_box(buf, u.out, u.pitch, row0, u.rows, col);
  if (pairs) store_box(buf + 2048, u.low, u.pitch, row0, u.rows, col);
  if (mirror) store_box(buf + 2048, u.out, u.pitch, col, u.rows, row0);
  __syncwarp();
}

__device__ __forceinline__ Rule gram_rule(const StepArgs& a, uint32_t b) {
  return {kScaleS / (kScaleX * kScaleX), 0.f, 0.f, 0.f, 1.f / kScaleS,
          a.diag_s + (uint64_t)b * a.k, a.s + (uint64_t)b * a.k * a.kpitch, nullptr, a.kpitch,
          a.k};
}

// The last step's 32 x 32 results, turned in shared memory (`box`: 4 KB) so that a warp
// writes 32 elements of a row at once, whatever the alignment of the caller's rows.
__device__ __forceinline__ void store_result(const StepArgs& a, uint32_t box, uint32_t b,
                                             uint32_t row0, uint32_t rows, uint32_t col,
                                             uint32_t cols) {
  const uint32_t lane = lane_id();
  __syncwarp();
  if (col + lane < cols) {
    const int64_t o0 = (int64_t)b * a.out_batch + (int64_t)row0 * a.out_stride + col + lane;
    const uint32_t n = min(32u, rows - row0);
    for (uint32_t r0 = 0; r0 < n; r0 += 8) {
      float old[8];
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r)
        old[r] = a.weight && r0 + r < n
                     ? load_any(a.out, a.out_type, o0 + (int64_t)(r0 + r) * a.out_stride)
                     : 0.f;
#pragma unroll
      for (uint32_t r = 0; r < 8; ++r) {
        if (r0 + r >= n) break;
        float x;
        asm volatile("ld.shared.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(box + (r0 + r) * 128 + ((lane ^ (r0 + r)) << 2))
                     : "memory");
        if (a.weight) x += a.keep * old[r];
        const int64_t o = o0 + (int64_t)(r0 + r) * a.out_stride;
        if (a.out_type == SPARCML_F32) static_cast<float*>(a.out)[o] = x;
        else if (a.out_type == SPARCML_BF16)
          static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x);
        else static_cast<__half*>(a.out)[o] = __float2half_rn(x);
      }
    }
  }
  __syncwarp();
}

// Before a writer gives up: until buffer s's load, of parity `phase`'s bit s, has landed, for
// each bit s of `slots`. (Not inlined, as all that only a wait beyond its first tries needs:
// beside the loops it cost 8 x 1024 x 1024 3 %.)
__device__ __noinline__ void land(uint32_t in_bar, uint32_t phase, uint32_t slots) {
  Waits alone = {0, kLandUs};
  for (uint32_t s = 0; s < 2; ++s)
    if (slots >> s & 1u) mbar_wait_warp(in_bar + 8 * s, (phase >> s) & 1u, &alone);
}

template <int CG, bool SMALL>
__device__ __forceinline__ bool write_results(Worker<CG>& w, const StepArgs& a, const Maps& m, const Product& p,
                              int kind, uint32_t step, Tile t) {
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t quarter = warp & 3u, half = warp >> 2;
  const float ca = a.coeffs[3 * step], cb = a.coeffs[3 * step + 1], cc = a.coeffs[3 * step + 2];
  const bool pairs = kind == kApply || kind == kLast, reads = kind == kPoly || pairs;
  for (uint32_t item = w.first_item(p); item < p.items; item += w.clusters) {
    if (item >= w.clusters) t = tile_of<CG>(p, item);
    if (t.none) continue;
    const uint32_t row0 = t.row0 + 128 * w.rank + 32 * quarter, row = row0 + lane;
    // the 32-column chunks of a tile alternate between the two warps of its rows
    const uint32_t tile_col = half * 32, col0 = t.col0 + tile_col;
    uint32_t count = 0;  // of this warp's chunks, those that exist
    if (row0 < p.rows && col0 < p.cols) count = min(t.n / 64, (p.cols - col0 + 63) / 64);
    const uint32_t turn0 = w.turn;
    auto fetch = [&](uint32_t q) {  // what is added to chunk q
      if (lane == 0) {
        const uint32_t slot = kind == kLast ? 0 : (turn0 + q) & 1u;
        const uint32_t dst = w.buf + slot * kStageBuf, bar = w.in_bar + 8 * slot;
        const uint32_t c = col0 + 64 * q;
        proxy_fence_shared();  // the buffer's last ordinary accesses come first
        mbar_expect_tx(bar, pairs ? 4096 : 2048);
        tma_load_3d(dst, pairs ? &m.x_out[step & 1] : &m.s_out, c, row0, t.b, bar);
        if (pairs) tma_load_3d(dst + 2048, &m.lo_out, c, row0, t.b, bar);
      }
    };
    if (reads && count) fetch(0);

    Rule u = gram_rule(a, t.b);
    const float* columns = nullptr;  // the diagonal vector that columns go by
    if (kind == kPoly) {
      const float s = row < p.rows ? __ldcg(u.diag + row) : 0.f;
      columns = u.diag;
      u.f = cc * kScaleP / (kScaleS * kScaleS);
      u.r0 = (cb + cc * s) * (kScaleP / kScaleS);
      u.r1 = cc * (kScaleP / kScaleS);
      u.on = (cb + cc * s) * s * kScaleP;
      u.diag_scale = 1.f / kScaleP;
      u.diag = a.diag_p + (uint64_t)t.b * a.k;
      u.out = a.p + (uint64_t)t.b * a.k * a.kpitch;
    } else if (pairs) {
      const float* d = a.diag_p + (uint64_t)t.b * a.k;
      columns = a.tall ? d : nullptr;
      u.f = SMALL ? 1.f / kScaleQ : 1.f / kScaleP;
      u.r0 = (SMALL ? 0.f : ca) + (!a.tall && row < p.rows ? __ldcg(d + row) : 0.f);
      u.r1 = a.tall ? 1.f : 0.f;
      if (kind == kLast) {
        const float g = a.alpha / kScaleX;
        u.f *= g;
        u.r0 *= g;
        u.r1 *= g;
      }
      u.diag = nullptr;
      u.out = a.hi[(step + 1) & 1] + (uint64_t)t.b * p.rows * a.pitch;
      u.low = a.lo + (uint64_t)t.b * p.rows * a.pitch;
      u.pitch = a.pitch;
      u.rows = p.rows;
    }
    auto column_diag = [&](uint32_t q) {
      const uint32_t c = col0 + 64 * q + lane;
      return columns && q < count && c < p.cols ? __ldcg(columns + c) : 0.f;
    };
    float other = column_diag(0);

    const uint32_t acc = w.acc & 1u;
    if (!mbar_wait_warp(w.acc_full + 8 * acc, (w.acc >> 1) & 1u, w.waits)) {
      if (reads && count) land(w.in_bar, w.in_phase, kind == kLast ? 1u : 1u << (turn0 & 1u));
      return false;
    }
    tmem_fence_after();
    const uint32_t src = w.tmem + acc * kAccColumns + (quarter << 21) + tile_col;
    if (kind == kPart) count = t.n / 64;
#pragma unroll 1
    for (uint32_t q = 0; q < count; ++q) {
      const uint32_t col = col0 + 64 * q;
      const uint32_t slot = kind == kLast ? 0 : w.turn & 1u;
      const uint32_t buf = w.buf + slot * kStageBuf, turned = w.buf + kStageBuf;
      if (reads && kind != kLast && q + 1 < count) fetch(q + 1);
      const float next = column_diag(q + 1);
      if (reads) {
        if (!mbar_wait_warp(w.in_bar + 8 * slot, (w.in_phase >> slot) & 1u, w.waits)) {
          land(w.in_bar, w.in_phase, kind != kLast && q + 1 < count ? 3u : 1u << slot);
          return false;
        }
        w.in_phase ^= 1u << slot;
      }
      const bool on_diag = !pairs && row0 == col;
#pragma unroll 1
      for (uint32_t h = 0; h < 2; ++h) {
        float v[16];
        tmem_load16(src + 64 * q + 16 * h, v);
        tmem_load_wait(v);
        if (kind == kPart) {
          // columns of 128 rows, or of the 64 that a small side has
          const uint32_t high = SMALL ? kSmall : 128;
          float* o = a.part +
                     ((uint64_t)((p.part0 + item) * CG + w.rank) * p.n + tile_col + 64 * q +
                      16 * h) * high + quarter * 32 + lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (quarter * 32 < high) o[i * high] = v[i];
          continue;
        }
        finish16(v, h, buf, reads, pairs, columns != nullptr, other, u, on_diag, row);
        if (kind == kLast) {
#pragma unroll
          for (uint32_t i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(turned + lane * 128 +
                                                         (((16 * h + i) ^ lane) << 2)),
                         "f"(v[i])
                         : "memory");
        } else {
          stage16(v, h, buf, pairs, t.mirror);
        }
      }
      if (kind == kLast) {
        __syncwarp();
        if (q + 1 < count) fetch(q + 1);
        store_result(a, turned, t.b, row0, p.rows, col, p.cols);
      } else if (kind != kPart) {
        store_boxes(buf, u, row0, col, pairs, t.mirror);
      }
      other = next;
      ++w.turn;
    }
    tmem_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(w.lead_acc_empty + 8 * acc);
    ++w.acc;
  }
  return true;
}

// S from the partial tiles of a split product, in the order of the splits: a warp takes
// 32 rows and 8 columns, so that a few tiles give work to many SMs.
template <int CG>
__device__ __forceinline__ uint32_t join_units(const Product& p) {
  return p.items / p.splits * 4 * CG * (p.n / 8);
}
template <int CG>
__device__ void join_parts(const StepArgs& a, Product p) {
  pin(p);
  const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t across = p.n / 8, per = 4 * CG * across, total = join_units<CG>(p);
  for (uint32_t x = blockIdx.x + gridDim.x * warp; x < total; x += gridDim.x * kWriters) {
    const uint32_t tile = x / per, r = x % per / across, q = x % across;
    const Tile t = tile_of<CG>(p, tile * p.splits);
    const uint32_t row0 = t.row0 + 32 * r, col = t.col0 + 8 * q, row = row0 + lane;
    if (row0 >= p.rows || col >= p.cols) continue;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint64_t step = (uint64_t)CG * p.n * 128;
    const float* o = a.part + ((uint64_t)((p.part0 + tile * p.splits) * CG + r / 4) * p.n + 8 * q) * 128 +
                     (r & 3u) * 32 + lane;
#pragma unroll 8
    for (uint32_t s = 0; s < p.splits; ++s, o += step) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += __ldcg(o + i * 128);
    }
    const Rule u = gram_rule(a, t.b);
    uint16_t half[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= u.f;
      if (row == col + i) {
        if (row < u.rows) u.diag[row] = v[i] * u.diag_scale;
        v[i] = 0.f;
      }
      half[i] = __half_as_ushort(__float2half_rn(v[i]));
    }
    if (row < u.rows) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = half[2 * e] | (uint32_t)half[2 * e + 1] << 16;
      *reinterpret_cast<uint4*>(u.out + (uint64_t)row * u.pitch + col) =
          make_uint4(w[0], w[1], w[2], w[3]);
      if (t.mirror) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < u.rows)
            u.out[(uint64_t)(col + i) * u.pitch + row] = __ushort_as_half(half[i]);
      }
    }
  }
}

// M consecutive floats of shared memory.
template <int M>
__device__ __forceinline__ void lds_floats(uint32_t a, float (&x)[M]) {
  if constexpr (M == 4)
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                 : "r"(a)
                 : "memory");
  else if constexpr (M == 2)
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[0]) : "r"(a) : "memory");
}
__device__ __forceinline__ void writers_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// A B[0], ..., A B[N - 1] of symmetric matrices in shared memory, k <= 64 rows of 64 floats, zeros
// beyond; f(n, e, i, j, value) takes a thread's entries e. A warp has R rows, a lane C
// columns of them, 32 apart: A's R entries of a row are the same for all lanes, B's are
// consecutive, so that each load is one access of shared memory (with tiles of 4 x 4 or
// 4 x 8 entries, 16 bytes per lane, loads bound it: 5,200 cycles for a product of 64).
template <int R, int C, int N, typename F>
__device__ __forceinline__ void small_products(uint32_t a, const uint32_t (&b)[N], uint32_t k, F f) {
  constexpr int ROWS = R == 8 ? 2 : 4;
  const uint32_t i0 = (threadIdx.x >> 5) * R, lane = lane_id();
  if (i0 < k) {
    float v[N][R][C];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < R * C; ++e) v[n][e / C][e % C] = 0.f;
    }
#pragma unroll 2
    for (uint32_t r = 0; r < k; r += ROWS) {
      float x[ROWS][R], y[ROWS][N][C];
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const uint32_t at = a + ((r + u) * kSmall + i0) * 4;
        if constexpr (R == 8) {
          float lo[4], hi[4];
          lds_floats<4>(at, lo);
          lds_floats<4>(at + 16, hi);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[u][i] = lo[i];
            x[u][4 + i] = hi[i];
          }
        } else {
          lds_floats<R>(at, x[u]);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float one[1];
            lds_floats<1>(b[n] + ((r + u) * kSmall + lane + 32 * c) * 4, one);
            y[u][n][c] = one[0];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
          for (int e = 0; e < R * C; ++e) v[n][e / C][e % C] += x[u][e / C] * y[u][n][e % C];
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int e = 0; e < R * C; ++e) f(n, e, i0 + e / C, lane + 32 * (e % C), v[n][e / C][e % C]);
    }
  }
  writers_sync();
}

// q(S) of one matrix, by its block's writers: S from the partial tiles in the order of the
// splits, in fp32 as all that follows; then q's diagonal and the two halves of the rest.
// `room`: four matrices of 64 x 64 floats.
template <int R, int C>
__device__ __noinline__ void solve_one(const StepArgs& a, uint32_t splits, uint32_t b,
                                       uint32_t tile, float* room) {
  constexpr uint32_t kCount = kSmall * kSmall;
  const uint32_t k = a.k;
  // the room is the writers' buffers: each has to be done with its own
  writers_sync();
  float *s = room, *pm = s + kCount, *q = pm + kCount, *t = q + kCount;
  {
    const float4* o = reinterpret_cast<const float4*>(a.part + (uint64_t)tile * kCount);
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (uint32_t c = 0; c < splits; ++c, o += kCount / 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4 x = __ldcg(o + u * 256 + threadIdx.x);
        v[u].x += x.x;
        v[u].y += x.y;
        v[u].z += x.z;
        v[u].w += x.w;
      }
    }
    const float f = 1.f / (kScaleX * kScaleX);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t e = 4 * (u * 256 + threadIdx.x), i = e / kSmall, j = e % kSmall;
      // beyond the matrix the operands hold whatever its padding does
      const bool row = i < k;
      reinterpret_cast<float4*>(s)[e / 4] =
          make_float4(row && j < k ? v[u].x * f : 0.f, row && j + 1 < k ? v[u].y * f : 0.f,
                      row && j + 2 < k ? v[u].z * f : 0.f, row && j + 3 < k ? v[u].w * f : 0.f);
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      reinterpret_cast<float4*>(pm)[e / 4] = zero;
      reinterpret_cast<float4*>(q)[e / 4] = zero;
      reinterpret_cast<float4*>(t)[e / 4] = zero;
    }
  }
  writers_sync();
  for (uint32_t step = 0; step < a.steps; ++step) {
    const float ca = a.coeffs[3 * step], cb = a.coeffs[3 * step + 1], cc = a.coeffs[3 * step + 2];
    const bool last = step + 1 == a.steps;
    float* const to = step == 0 ? q : pm;
    {
      const uint32_t other[1] = {smem_addr(s)};
      small_products<R, C, 1>(smem_addr(s), other, k, [&](int, int, uint32_t i, uint32_t j, float v) {
        const float x = (i == j && i < k ? ca : 0.f) + cb * s[i * kSmall + j] + cc * v;
        to[i * kSmall + j] = x;
      });
    }
    if (step == 0) {  // q = P
      if (last) break;
      const uint32_t other[1] = {smem_addr(s)};
      small_products<R, C, 1>(smem_addr(q), other, k, [&](int, int, uint32_t i, uint32_t j, float v) {
        t[i * kSmall + j] = v;
      });
      const uint32_t other2[1] = {smem_addr(q)};
      small_products<R, C, 1>(smem_addr(t), other2, k, [&](int, int, uint32_t i, uint32_t j, float v) {
        s[i * kSmall + j] = v;
      });
      continue;
    }
    if (last) {
      const uint32_t other[1] = {smem_addr(q)};
      small_products<R, C, 1>(smem_addr(pm), other, k, [&](int, int, uint32_t i, uint32_t j, float v) {
        t[i * kSmall + j] = v;
      });
      q = t;
      break;
    }
    // P q and P S in one pass; the second's entries wait in registers until S has been read
    float keep[R * C];
    const uint32_t both[2] = {smem_addr(q), smem_addr(s)};
    small_products<R, C, 2>(smem_addr(pm), both, k, [&](int n, int e, uint32_t i, uint32_t j, float v) {
      if (n == 0) t[i * kSmall + j] = v;
      else keep[e] = v;
    });
    {
      const uint32_t i0 = (threadIdx.x >> 5) * R;
      if (i0 < k) {
#pragma unroll
        for (int e = 0; e < R * C; ++e)
          q[(i0 + e / C) * kSmall + lane_id() + 32 * (e % C)] = keep[e];
      }
      writers_sync();
    }
    const uint32_t other[1] = {smem_addr(pm)};
    small_products<R, C, 1>(smem_addr(q), other, k, [&](int, int, uint32_t i, uint32_t j, float v) {
      s[i * kSmall + j] = v;
    });
    float* const now = t;
    t = q;
    q = now;
  }
  for (uint32_t e = threadIdx.x; e < k * kSmall; e += 32 * kWriters) {
    const uint32_t i = e / kSmall, j = e % kSmall;
    const float v = i == j ? 0.f : q[e] * kScaleQ;
    if (i == j) a.diag_p[(uint64_t)b * k + i] = q[e];
    const __half h = __float2half_rn(v);
    a.p[((uint64_t)b * k) * kSmall + e] = h;  // k <= 64: the pitch is 64
    a.s[((uint64_t)b * k) * kSmall + e] = __float2half_rn(v - __half2float(h));
  }
  writers_sync();
}

// 2^12 / |U| as two factors, each a normal number whatever the size of |U|.
__device__ __forceinline__ void norm_factors(const GatherArgs& g, uint64_t b, float& f0,
                                             float& f1) {
  float t[3] = {0.f, 0.f, 0.f};
  for (uint32_t k = lane_id(); k < g.blocks; k += 32)
    for (int q = 0; q < 3; ++q) t[q] += __ldcg(g.sums + (b * g.blocks + k) * 3 + q);
  for (int q = 0; q < 3; ++q) t[q] = warp_sum_f(t[q]);
  // |U|^2 = t0 2^-160 + t1 + t2 2^180, in the unit of the largest range that has any
  const float all = t[0] + t[1] + t[2];
  if (!(all < __int_as_float(0x7f800000))) {
    f0 = f1 = __int_as_float(0x7fffffff);  // an inf or a NaN in U: all of X is NaN
  } else if (t[2] > 0.f) {
    f0 = 0x1p-90f;
    f1 = kScaleX / sqrtf(t[2] + t[1] * 0x1p-90f * 0x1p-90f);
  } else if (t[1] > 0.f) {
    f0 = 1.f;
    f1 = kScaleX / sqrtf(t[1] + t[0] * 0x1p-80f * 0x1p-80f);
  } else {
    f0 = 0x1p80f;
    f1 = t[0] > 0.f ? kScaleX / sqrtf(t[0]) : 0.f;
  }
}

// The scaled input as a pair of fp16.
__device__ void split_input(const StepArgs& a) {
  const GatherArgs& g = a.g;
  const Pieces pieces(g.m, g.n);
  const Slots slots(pieces);
  const uint64_t total = a.batch * pieces.total;
  const uint64_t warps = (uint64_t)gridDim.x * (kThreads / 32);
  const uint64_t id = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  // each warp takes a run of pieces, which lies in few matrices
  const uint64_t end = total * (id + 1) / warps;
  uint64_t u = total * id / warps, b = u / pieces.total, rest = u - b * pieces.total;
  uint64_t r0 = rest / pieces.across * pieces.rows, piece = rest % pieces.across;
  bool known = false;
  float f0 = 0.f, f1 = 0.f;
#pragma unroll 2
  for (; u < end; ++u) {
    if (!known) norm_factors(g, b, f0, f1);
    known = true;
    float v[4][4], mo[4][4];
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint64_t r = r0 + slots.row[q], c = piece * kPiece + slots.col[q];
      const uint64_t in = slots.row[q] < pieces.rows && r < g.m ? g.n : 0;
      load4(g.g, g.g_type, b * g.g_batch + r * g.g_stride + c, c, in, g.vec_g, v[q]);
      if (g.mom)
        load4(g.mom, SPARCML_F32, b * g.m_batch + r * g.m_stride + c, c, in, g.vec_m, mo[q]);
    }
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {
      const uint64_t r = r0 + slots.row[q], c = piece * kPiece + slots.col[q];
      // the row's padding takes what is left of the last four
      if (slots.row[q] >= pieces.rows || r >= g.m || c >= g.n) continue;
      uint32_t hw[2], lw[2];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = v[q][i + e];
          if (g.mom) t = g.nesterov ? t + g.mu * mo[q][i + e] : mo[q][i + e];
          x[e] = t * f0 * f1;
        }
        hw[i / 2] = pack_half(x[0], x[1]);
        const float2 back = unpack_half(hw[i / 2]);
        lw[i / 2] = pack_half(x[0] - back.x, x[1] - back.y);
      }
      const uint64_t at = (b * g.m + r) * a.pitch + c;
      *reinterpret_cast<uint2*>(a.hi[0] + at) = make_uint2(hw[0], hw[1]);
      *reinterpret_cast<uint2*>(a.lo + at) = make_uint2(lw[0], lw[1]);
    }
    if (++piece == pieces.across) {
      piece = 0;
      r0 += pieces.rows;
      if (r0 >= g.m) {
        r0 = 0;
        ++b;
        known = false;
      }
    }
  }
}

// Whether a counter of arrivals has come to `want`; what the arriving blocks wrote before
// is then visible. wait_count ends after four times the waits' limit at worst.
__device__ __forceinline__ bool count_is(const uint32_t* count, uint32_t want) {
  uint32_t now;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(now) : "l"(count) : "memory");
  return (int32_t)(now - want) >= 0;
}
__device__ __noinline__ bool wait_count_long(const uint32_t* count, uint32_t want, Waits* waits) {
  const uint64_t end = global_ns() + 4000ull * waits->limit_us;
  for (uint32_t polls = 1;; ++polls) {
    if (count_is(count, want)) return true;
    if ((polls & 63u) == 0) {
      if (waits->gave_up != 0) return false;
      if (global_ns() > end) {
        waits->gave_up = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_count(const uint32_t* count, uint32_t want, Waits* waits) {
  for (uint32_t i = 0; i < 64; ++i)
    if (count_is(count, want)) return true;
  return wait_count_long(count, want, waits);
}
__device__ __forceinline__ void add_count(uint32_t* count) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
}

// The order of work, the same for the loader, the issuer and the writers of every block:
// step by step, product by product, chain by chain. f(step, kind, product, chain, count
// of the chain's arrivals that the work has to wait for).
template <int CG, bool SMALL, typename F>
__device__ __forceinline__ void in_order(const StepArgs& a, F f) {
  uint32_t need[2] = {0, 0};
  const uint32_t steps = SMALL ? 1 : a.steps;
#pragma unroll 1
  for (uint32_t step = 0; step < steps; ++step) {
#pragma unroll 1
    for (uint32_t ph = 0; ph < 4; ++ph) {
#pragma unroll 1
      for (uint32_t chain = 0; chain < a.chains; ++chain) {
        const Product& p = a.product[chain][ph < 2 ? 0 : ph - 1];
        if (ph == 1 && (SMALL || p.splits == 1)) continue;  // nothing to join
        const int kind = ph == 0   ? (SMALL || p.splits > 1 ? kPart : kGram)
                         : ph == 1 ? kJoin
                         : ph == 2 ? (SMALL ? kSolve : kPoly)
                                   : (step + 1 == steps ? kLast : kApply);
        const uint32_t blocks = kind == kJoin ? min(join_units<CG>(p), gridDim.x)
                                              : min(p.items, gridDim.x / CG) * CG;
        const uint32_t n = chain ? need[1] : need[0];
        if (!f(step, kind, p, chain, n)) return;
        if (chain) need[1] += blocks;
        else need[0] += blocks;
      }
    }
  }
}

template <int CG, bool SMALL>
__global__ void __launch_bounds__(kThreads, 1)
steps_kernel(const __grid_constant__ Maps m, const __grid_constant__ StepArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[2 * kMaxStages + 7 + 2 * kWriters];
  __shared__ uint32_t tmem_slot, written[2];
  __shared__ Waits waits;
  // What the other block of a pair says at the end: whether it gave up, and the next stage that
  // it would have loaded.
  __shared__ uint32_t partner[2];
  griddep_wait();
  const uint32_t warp = threadIdx.x >> 5;
  Worker<CG> w;
  w.ring = (smem_addr(raw) + 1023u) & ~1023u;
  const Product* shape = a.product[0];
  const uint32_t widest = max(shape[0].n, max(shape[1].n, shape[2].n));
  w.stage_bytes = 128 * 128 + widest / CG * 128;
  w.stages = min(kMaxStages, kRingBytes / w.stage_bytes);
  w.full = smem_addr(bars);
  w.empty = w.full + 8 * kMaxStages;
  w.acc_full = w.empty + 8 * kMaxStages;
  w.acc_empty = w.acc_full + 16;
  const uint32_t ready = w.acc_empty + 16, finished = ready + 16 + 16 * kWriters;
  w.in_bar = ready + 16 + 16 * (warp % kWriters);
  w.buf = w.ring + kRingBytes + (warp % kWriters) * 2 * kStageBuf;
  w.rank = CG == 1 ? 0 : cluster_rank();
  w.cluster = blockIdx.x / CG;
  w.clusters = gridDim.x / CG;
  w.waits = &waits;
  w.lead_full = CG == 1 ? w.full : cluster_addr(w.full, 0);
  w.lead_acc_empty = cluster_addr(w.acc_empty, 0);
  w.leader = elect_one();

  if (threadIdx.x < sizeof(Maps) / sizeof(CUtensorMap))
    tma_prefetch_map(reinterpret_cast<const CUtensorMap*>(&m) + threadIdx.x);
  if (threadIdx.x == 0) {
    waits.gave_up = written[0] = written[1] = 0;
    waits.limit_us = kWaitUs;
    partner[0] = partner[1] = 0;
    for (uint32_t s = 0; s < kMaxStages; ++s) {
      mbar_init(w.full + 8 * s, 1);
      mbar_init(w.empty + 8 * s, 1);
    }
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(w.acc_full + 8 * s, 1);
      mbar_init(w.acc_empty + 8 * s, CG * kWriters);
      mbar_init(ready + 8 * s, 1);
    }
    for (uint32_t s = 0; s < 2 * kWriters; ++s) mbar_init(ready + 16 + 8 * s, 1);
    mbar_init(finished, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWriters) tmem_alloc<CG>(smem_addr(&tmem_slot), 2 * kAccColumns);
  tmem_fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();
  tmem_fence_after();
  w.tmem = tmem_slot;

  const bool tall = a.tall != 0;
  const bool armed = threadIdx.x == 0 && injected(a.inject);
  split_input(a);
  proxy_fence_global();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (armed) waits.limit_us = kInjectWaitUs;
    add_count(a.g.turns);
    wait_count(a.g.turns, gridDim.x, &waits);
  }
  __syncthreads();

  auto a_major = [&](int kind) { return (kind == kGram || kind == kPart) && tall; };
  auto b_major = [&](int kind) {
    return kind == kGram || kind == kPart ? tall : kind != kPoly && !tall;
  };
  uint32_t* const turns = a.g.turns + kTurnStep;
  // The loader waits for what the products read, and tells the block's writers; at most
  // two of its messages can be unread (of three in a row two are of one chain, and the
  // later one comes after the writers' arrival for the earlier), so two barriers in
  // turn carry them.
  uint32_t told = 0;
  if (warp == kWriters) {
    in_order<CG, SMALL>(a, [&](uint32_t step, int kind, const Product& p, uint32_t chain, uint32_t need) {
      const uint32_t item = w.first_item(p);
      if (kind == kJoin ? blockIdx.x >= join_units<CG>(p) : item >= p.items) return true;
      Tile t = {};
      if (kind != kJoin && kind != kSolve) t = tile_of<CG>(p, item);
      pin(t);
      bool come = true;
      if (w.leader) {
        come = wait_count(turns + chain * kTurnStep, need, &waits);
        if (come) mbar_arrive(ready + 8 * (told & 1u));
      }
      if (!__all_sync(0xffffffffu, come)) return false;
      ++told;
      if (kind == kJoin || kind == kSolve) return true;
      const CUtensorMap *ma = &m.x_gram[step & 1][0], *mb = &m.x_gram[step & 1][1];
      if (kind == kPoly) {
        ma = &m.s_poly[0];
        mb = &m.s_poly[1];
      } else if (kind != kGram && kind != kPart) {
        ma = tall ? &m.x_apply[step & 1] : &m.p_apply;
        mb = tall ? &m.p_apply : &m.x_apply[step & 1];
      }
      // the lower halves, where they take part
      const CUtensorMap *ma_lo = &m.lo_gram[0], *mb_lo = &m.lo_gram[1];
      if (kind == kLast) {
        ma_lo = tall ? &m.lo_apply : &m.q_lo;
        mb_lo = tall ? &m.q_lo : &m.lo_apply;
      }
      return load_operands<CG, SMALL>(w, p, ma, mb, ma_lo, mb_lo, a_major(kind), b_major(kind), t);
    });
  } else if (warp == kWriters + 1) {
    // An injected fault: the first block (or pair) withholds its products from one on that adds
    // to something, so that full stages, loads of writers and the grid's counters are waited for.
    const bool withhold = w.cluster == 0 && waits.limit_us == kInjectWaitUs;
    if (w.rank == 0)
      in_order<CG, SMALL>(a, [&](uint32_t, int kind, const Product& p, uint32_t, uint32_t) {
        const uint32_t item = w.first_item(p);
        if (kind == kJoin || kind == kSolve || item >= p.items) return true;
        if (withhold && (SMALL || kind == kPoly)) return false;
        Tile t = tile_of<CG>(p, item);
        pin(t);
        return issue_products<CG, SMALL>(w, p, a_major(kind), b_major(kind), t);
      });
  } else {
    // A writer that gives up leaves, but for solve_one, whose barriers take all of a block's
    // writers and have no limit: there it still works along, on whatever is there.
    bool lost = false;
    in_order<CG, SMALL>(a, [&](uint32_t step, int kind, const Product& p, uint32_t chain, uint32_t) {
      const uint32_t item = w.first_item(p);
      if (kind == kJoin ? blockIdx.x >= join_units<CG>(p) : item >= p.items) return true;
      Tile t = {};
      if (kind != kJoin && kind != kSolve) t = tile_of<CG>(p, item);
      pin(t);
      if (!lost && !mbar_wait_warp(ready + 8 * (told & 1u), (told >> 1) & 1u, &waits)) {
        if (!SMALL) return false;
        lost = true;
      }
      ++told;
      if (SMALL && lost && kind != kSolve) return true;
      if (kind == kJoin) {
        join_parts<CG>(a, p);
      } else if (SMALL && kind == kSolve) {
        float* room = reinterpret_cast<float*>(raw + (w.ring - smem_addr(raw)) + kRingBytes);
        const Product& gram = a.product[chain][0];
        for (uint32_t i = item; i < p.items; i += w.clusters) {
          const uint32_t tile = gram.part0 + i * gram.splits;
          if (a.k > 32) solve_one<8, 2>(a, gram.splits, p.b0 + i, tile, room);
          else if (a.k > 16) solve_one<4, 1>(a, gram.splits, p.b0 + i, tile, room);
          else solve_one<2, 1>(a, gram.splits, p.b0 + i, tile, room);
        }
      } else if (!write_results<CG, SMALL>(w, a, m, p, kind, step, t)) {
        lost = true;
        return SMALL;
      }
      if (lost || kind == kLast) return true;
      // what was written is read by asynchronous copies; the last of the block's writers
      // reports to the grid
      proxy_fence_global();
      __syncwarp();
      if (w.leader) {
        uint32_t before;
        asm volatile("atom.acq_rel.cta.shared::cta.add.u32 %0, [%1], 1;"
                     : "=r"(before)
                     : "r"(smem_addr(&written[chain]))
                     : "memory");
        if (before == kWriters - 1) {
          written[chain] = 0;
          add_count(turns + chain * kTurnStep);
        }
      }
      __syncwarp();
      return true;
    });
  }
  tmem_fence_before();
  __syncthreads();  // now it is settled whether this block gave up
  if constexpr (CG > 1) {
    const uint32_t to = cluster_addr(smem_addr(partner), w.rank ^ 1u);
    if (threadIdx.x == 0) store_cluster(to, waits.gave_up);
    if (warp == kWriters && w.leader) store_cluster(to + 4, 2 * w.stage + w.phase);
    __syncwarp();
    cluster_sync();
  }
  if (waits.gave_up || (CG > 1 && partner[0])) {
    // Nothing may still be in flight when the shared and tensor memory go: wait, again with a
    // limit, for the loads and products that were begun. (Writers have waited for their own.)
    if (warp == kWriters && w.leader) {
      const bool apart = CG > 1 && partner[1] != 2 * w.stage + w.phase;
      if (w.rank == 0 || apart) land_operands(w.full, w.stages, w.stage, w.phase, apart);
    }
    if (warp == kWriters + 1 && w.leader) {
      // arrives, in both blocks of a pair, once all products have completed
      Waits alone = {0, kWaitUs};
      if (w.rank == 0) mma_commit<CG>(finished);
      mbar_wait(finished, 0, &alone);
    }
    __syncwarp();
    if (threadIdx.x == 0) set_status(a.status, SPARCML_ERR_TIMEOUT);
    __syncthreads();
    if constexpr (CG > 1) cluster_sync();
  }
  tmem_fence_after();
  if (warp == kWriters) tmem_free<CG>(w.tmem, 2 * kAccColumns);
}

// ---------------------------------------------------------------------------
// Host side.

bool encode(CUtensorMap* map, const void* p, uint32_t rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, rank, dims, strides, box, swizzle);
}

struct Matrices {  // fp16 [batch][rows][pitch], of which `cols` columns exist
  const void* p;
  uint64_t batch, rows, cols, pitch;
};

// Boxes of 32 x 32.
bool box_map(CUtensorMap* map, const Matrices& a) {
  const cuuint64_t dims[3] = {a.cols, a.rows, a.batch};
  const cuuint64_t strides[2] = {a.pitch * 2, a.rows * a.pitch * 2};
  const cuuint32_t box[3] = {32, 32, 1};
  return encode(map, a.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

// An operand with `size` rows of the result's side per load. K-major: `size` rows of 64
// columns, the columns being the summed axis. MN-major: 64 rows, the summed axis, of `size`
// columns as groups of 64; the last group's columns beyond the matrix are the pitch's
// padding, whatever it holds, and lead to rows or columns of the result that do not exist.
bool operand_map(CUtensorMap* map, const Matrices& a, bool mn, uint32_t size) {
  const cuuint64_t row = a.pitch * 2, all = a.rows * row;
  const cuuint64_t k_dims[4] = {a.cols, a.rows, 1, a.batch}, k_strides[3] = {row, all, all};
  const cuuint32_t k_box[4] = {64, size, 1, 1};
  const cuuint64_t m_dims[4] = {64, a.rows, a.pitch / 64, a.batch}, m_strides[3] = {row, 128, all};
  const cuuint32_t m_box[4] = {64, 64, size / 64, 1};
  return encode(map, a.p, 4, mn ? m_dims : k_dims, mn ? m_strides : k_strides, mn ? m_box : k_box,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr uint32_t kSms = 152;

struct Plan {
  uint64_t batch, m, n, k, l, pitch, kpitch;
  uint32_t blocks;  // of the norm, per matrix
  uint32_t pair;    // blocks that share a tile: 1 or 2
  uint32_t chains;
  Product product[2][3];
  Product small[2][3];  // for a small side
  size_t sums, hi0, hi1, lo, s, p, ds, dp, part, bytes;
};

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// Tiles of a product and the time of its slowest worker, in units of 128 cycles. A block
// of 64 along the summed axis takes n / 64 of them on the tensor cores, and its operands
// 58 bytes per cycle and SM from L2 when all SMs fetch; writing 64 columns of a tile takes
// about 16, beside the next tile's product.
Product shape_product(uint64_t batch, uint64_t rows, uint64_t cols, uint64_t depth, bool symmetric,
                      uint32_t pair, uint32_t n, bool may_split, uint64_t all, double* time) {
  Product p = {};
  const uint64_t workers = kSms / pair, tr = ceil_div(rows, 128 * pair), tc = ceil_div(cols, n);
  const uint64_t ratio = std::max<uint64_t>(1, 128 * pair / n);
  p.n = n;
  p.rows = (uint32_t)rows;
  p.cols = (uint32_t)cols;
  p.blocks = (uint32_t)ceil_div(depth, 64);
  p.tile_rows = symmetric ? 0 : (uint32_t)tr;
  const uint64_t tiles = symmetric ? ratio * tr * (tr + 1) / 2 : tr * tc;
  p.tiles = (uint32_t)tiles;
  p.splits = 1;
  // joining the parts costs a turn of the grid
  if (may_split && tiles * all * 2 <= workers && p.blocks >= 64)
    p.splits = (uint32_t)std::min<uint64_t>(workers / (tiles * all), p.blocks / 8);
  uint64_t items = tiles * batch * p.splits;
  // a last round that at most half of the workers would have work in is done in half
  // tiles, of 64 operand rows per block at least
  const uint64_t left = items % workers;
  const bool halves = p.splits == 1 && all == 1 && items > workers && n >= 128 * pair && left * 2 <= workers;
  p.whole = (uint32_t)(halves ? items - left : items);
  if (halves) items += left;
  p.items = items > 0x7fffffffull ? 0 : (uint32_t)items;
  const double busy = std::min(1.0, (double)items / (double)workers);
  const double each = std::max(n / 64.0, (128 + n / pair) / 58.0 * busy);
  const double product = (double)ceil_div(p.blocks, p.splits) * each;
  const double write = 6 + std::min<uint64_t>(n, align_up(cols, 64)) / 4.0;
  const double rounds = (double)ceil_div(p.whole, workers) + (halves && left ? 0.5 : 0.0);
  *time = product + (rounds - 1) * std::max(product, write) + write;
  if (p.splits > 1)  // a turn of the grid, and the partial tiles' way to L2 and back
    *time += 60.0 + (double)items * pair * 128 * n * 8 / (kSms * 40.0 * 128.0);
  if (all > 1)  // two chains: each one's latency, or the work of both
    *time = std::max((*time + product + write) / 2 + 20, rounds * std::max(product, write));
  return p;
}

Product best_product(uint64_t batch, uint64_t rows, uint64_t cols, uint64_t depth, bool symmetric,
                     uint32_t pair, bool may_split, double* best) {
  Product p = {};
  *best = 0;
  for (uint32_t n = 64 * pair; n <= 128 * pair; n *= 2) {
    double t;
    const Product q =
        shape_product(batch, rows, cols, depth, symmetric, pair, n, may_split, batch, &t);
    if (n == 64 * pair || t <= *best) {
      p = q;
      *best = t;
    }
  }
  return p;
}

bool make_plan(int32_t batch, uint64_t m, uint64_t n, Plan& q) {
  if (batch < 0 || batch > 65535 || m < 1 || n < 1 || m > (1u << 24) || n > (1u << 24) ||
      std::min(m, n) > 32768)
    return false;
  if (batch == 0) {  // nothing to shape: a workspace of a header, and no launch
    q = Plan{};
    q.bytes = 256;
    return true;
  }
  q.batch = batch;
  q.m = m;
  q.n = n;
  q.k = std::min(m, n);
  q.l = std::max(m, n);
  q.pitch = align_up(n, 64);
  q.kpitch = align_up(q.k, 64);
  q.blocks = (uint32_t)std::min<uint64_t>(ceil_div(m * n, 8 * kPiece), kSms * 2);
  double best = 0;
  uint32_t width[3] = {0, 0, 0};
  for (uint32_t pair = 1; pair <= 2; ++pair) {
    double t[3];
    const Product g = best_product(batch, q.k, q.k, q.l, true, pair, true, &t[0]);
    const Product p = best_product(batch, q.k, q.k, q.k, true, pair, false, &t[1]);
    const Product a = best_product(batch, m, n, q.k, false, pair, false, &t[2]);
    const double sum = t[0] + t[1] + t[2];
    if (pair == 1 || sum <= best) {
      best = sum;
      q.pair = pair;
      width[0] = g.n;
      width[1] = p.n;
      width[2] = a.n;
    }
  }
  q.chains = batch > 1 ? 2 : 1;
  size_t parts = 0;
  for (uint32_t c = 0; c < q.chains; ++c) {
    const uint64_t b0 = c ? (batch + 1) / 2 : 0;
    const uint64_t some = q.chains == 1 ? batch : c ? batch / 2 : (batch + 1) / 2;
    for (int i = 0; i < 3; ++i) {
      double t;
      Product& p = q.product[c][i];
      p = shape_product(some, i < 2 ? q.k : m, i < 2 ? q.k : n, i == 0 ? q.l : q.k, i < 2, q.pair,
                        width[i], i == 0, batch, &t);
      if (!p.items) return false;
      p.b0 = (uint32_t)b0;
      if (p.splits > 1) {
        p.part0 = (uint32_t)parts;
        parts += p.items;
      }
    }
  }
  size_t small_parts = 0;
  if (q.k <= kSmall) {
    // S in few parts, which one block adds up; then a block per matrix; then q(S) X
    const uint64_t blocks = ceil_div(q.l, 64);
    const uint32_t splits = (uint32_t)std::max<uint64_t>(
        1, std::min({(uint64_t)16, blocks / 4, kSms / q.batch}));
    for (uint32_t c = 0; c < q.chains; ++c) {
      const uint64_t some = q.chains == 1 ? batch : c ? batch / 2 : (batch + 1) / 2;
      double t;
      for (int i = 0; i < 3; ++i) {
        Product& p = q.small[c][i];
        p = shape_product(some, i < 2 ? q.k : m, i < 2 ? q.k : n, i == 0 ? q.l : q.k, i < 2, 1,
                          i < 2 ? 64 : 128, false, batch, &t);
        p.b0 = q.product[c][i].b0;
        if (i == 0) {
          p.splits = splits;
          p.tiles = 1;
          p.part0 = (uint32_t)small_parts;
          small_parts += some * splits;
        }
        if (i < 2) p.whole = p.items = (uint32_t)(some * (i == 0 ? splits : 1));
      }
    }
  }
  const size_t x = q.batch * m * q.pitch * 2, s = q.batch * q.k * q.kpitch * 2;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, 256);
    return o;
  };
  q.sums = take(q.batch * q.blocks * 3 * sizeof(float));
  q.hi0 = take(x);
  q.hi1 = take(x);
  q.lo = take(x);
  q.s = take(s);
  q.p = take(s);
  q.ds = take(q.batch * q.k * sizeof(float));
  q.dp = take(q.batch * q.k * sizeof(float));
  q.part = take(std::max(parts * q.pair * 128 * width[0], small_parts * kSmall * kSmall) *
                sizeof(float));
  q.bytes = at;
  return true;
}

// Whether the steps may be taken as one polynomial of S: q(S) stays within 1800 and S's
// own rounding within 1/64 of the largest singular value's square, over all singular values
// that X can have.
bool one_polynomial(const float* coeffs, int32_t steps) {
  for (int j = 0; j <= 64; ++j) {
    double s = (j / 64.0) * (j / 64.0), q = 1.0, grown = 1.0;
    for (int32_t i = 0; i < steps; ++i) {
      const double p = coeffs[3 * i] + s * (coeffs[3 * i + 1] + s * coeffs[3 * i + 2]);
      q *= p;
      s *= p * p;
      if (!(std::abs(q) <= 1800.0) || !(s <= 16.0)) return false;
      if (i + 1 < steps) grown *= p * p;
      if (!(grown <= 262144.0)) return false;
    }
  }
  return true;
}

struct Target {  // where the result goes
  bool weight;
  void* out;
  int32_t type;
  int64_t batch, stride;
  float alpha, keep;
};

// Blocks (or pairs of blocks) of a kernel that run at one time on the current device, up to
// one per SM; 0 if that cannot be found out. Asked for once per device.
template <int CG, bool SMALL>
unsigned resident() {
  static std::mutex lock;
  static std::map<int, unsigned> known;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> hold(lock);
  const auto it = known.find(device);
  if (it != known.end()) return it->second;
  auto kernel = steps_kernel<CG, SMALL>;
  if (!ensure_smem(reinterpret_cast<const void*>(kernel), kStepsSmem)) return 0;
  int count = 0;
  if (CG == 1) {
    int per = 0, sms = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, kStepsSmem) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
      return 0;
    count = std::min(per, 1) * sms;
  } else {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kStepsSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CG;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) return 0;
  }
  const unsigned fit = (unsigned)std::min<int>(count, kSms / CG);
  known[device] = fit;
  return fit;
}

template <int CG, bool SMALL>
int launch_steps(const Maps& m, StepArgs& a, cudaStream_t s) {
  auto kernel = steps_kernel<CG, SMALL>;
  const unsigned clusters = resident<CG, SMALL>();
  if (clusters == 0 || !ensure_smem(reinterpret_cast<const void*>(kernel), kStepsSmem))
    return SPARCML_ERR_CUDA;
  for (int i = 0; i < 3; ++i)  // the second chain starts beside the first one
    a.product[1][i].offset = a.product[0][i].items % clusters;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kStepsSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;  // all blocks run at one time
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  (void)cudaLaunchKernelEx(&cfg, kernel, m, a);
  return launch_status();
}

int run_steps(GatherArgs g, const Plan& q, const Target& to, const float* coeffs, int32_t steps,
              void* ws, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  char *hi0 = w + q.hi0, *hi1 = w + q.hi1, *lo = w + q.lo, *sm = w + q.s, *pm = w + q.p;
  Maps m;
  const bool tall = q.m > q.n;
  const bool small = q.k <= kSmall && one_polynomial(coeffs, steps);
  const Product(*const product)[3] = small ? q.small : q.product;
  const uint32_t pair = small ? 1 : q.pair;
  const Matrices x[2] = {{hi0, q.batch, q.m, q.n, q.pitch}, {hi1, q.batch, q.m, q.n, q.pitch}};
  const Matrices low = {lo, q.batch, q.m, q.n, q.pitch};
  const Matrices sq = {sm, q.batch, q.k, q.k, q.kpitch}, pq = {pm, q.batch, q.k, q.k, q.kpitch};
  uint32_t second[3];  // rows of the second operand that one block loads
  for (int i = 0; i < 3; ++i) second[i] = product[0][i].n / pair;
  bool ok = box_map(&m.lo_out, low) && box_map(&m.s_out, sq) &&
            operand_map(&m.s_poly[0], sq, false, 128) &&
            operand_map(&m.s_poly[1], sq, false, second[1]) &&
            operand_map(&m.p_apply, pq, false, tall ? second[2] : 128);
  for (int i = 0; i < 2 && ok; ++i)
    ok = box_map(&m.x_out[i], x[i]) && operand_map(&m.x_gram[i][0], x[i], tall, 128) &&
         operand_map(&m.x_gram[i][1], x[i], tall, second[0]) &&
         operand_map(&m.x_apply[i], x[i], !tall, tall ? 128 : second[2]);
  if (small)
    ok = ok && operand_map(&m.lo_gram[0], low, tall, 128) &&
         operand_map(&m.lo_gram[1], low, tall, second[0]) &&
         operand_map(&m.lo_apply, low, !tall, tall ? 128 : second[2]) &&
         operand_map(&m.q_lo, sq, false, tall ? second[2] : 128);
  else
    m.lo_gram[0] = m.lo_gram[1] = m.lo_apply = m.q_lo = m.s_out;  // not used
  if (!ok) return SPARCML_ERR_CUDA;
  const int64_t ge = g.g_type == SPARCML_F32 ? 16 : 8;
  g.vec_g = aligned_to(g.g, ge) && g.g_batch % 4 == 0 && g.g_stride % 4 == 0;
  g.vec_m = aligned_to(g.mom, 16) && g.m_batch % 4 == 0 && g.m_stride % 4 == 0;
  g.flat = g.g_stride == (int64_t)q.n && (!g.mom || g.m_stride == (int64_t)q.n);
  if (g.flat) {  // then only a matrix's start has to be aligned
    g.vec_flat_g = aligned_to(g.g, ge) && g.g_batch % 4 == 0;
    g.vec_flat_m = aligned_to(g.mom, 16) && g.m_batch % 4 == 0;
  }
  g.m = q.m;
  g.n = q.n;
  g.blocks = q.blocks;
  g.sums = reinterpret_cast<float*>(w + q.sums);
  g.turns = reinterpret_cast<uint32_t*>(w + 128);
  StepArgs a = {};
  a.g = g;
  a.batch = (uint32_t)q.batch;
  a.steps = (uint32_t)steps;
  a.tall = tall;
  a.chains = q.chains;
  for (uint32_t c = 0; c < q.chains; ++c) std::copy(product[c], product[c] + 3, a.product[c]);
  std::copy(coeffs, coeffs + 3 * steps, a.coeffs);
  a.hi[0] = reinterpret_cast<__half*>(hi0);
  a.hi[1] = reinterpret_cast<__half*>(hi1);
  a.lo = reinterpret_cast<__half*>(lo);
  a.s = reinterpret_cast<__half*>(sm);
  a.p = reinterpret_cast<__half*>(pm);
  a.pitch = q.pitch;
  a.kpitch = q.kpitch;
  a.diag_s = reinterpret_cast<float*>(w + q.ds);
  a.diag_p = reinterpret_cast<float*>(w + q.dp);
  a.part = reinterpret_cast<float*>(w + q.part);
  a.k = (uint32_t)q.k;
  a.weight = to.weight;
  a.out = to.out;
  a.out_type = to.type;
  a.out_batch = to.batch;
  a.out_stride = to.stride;
  a.alpha = to.alpha;
  a.keep = to.keep;
  a.status = reinterpret_cast<int32_t*>(w);
  a.inject = reinterpret_cast<const uint32_t*>(w + kInjectOffset);
  launch_pdl(gather_norm_kernel, dim3(q.blocks, (unsigned)q.batch), 256, 0, s, g);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  const int r = small       ? launch_steps<1, true>(m, a, s)
                : pair == 1 ? launch_steps<1, false>(m, a, s)
                            : launch_steps<2, false>(m, a, s);
  if (r != SPARCML_OK) return r;
  note_launches(2);
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

extern "C" int sparcml_orthogonalize_plan(int32_t batch, uint64_t m, uint64_t n, int32_t* plan) {
  Plan q;
  if (!plan || batch < 1 || !make_plan(batch, m, n, q)) return SPARCML_ERR_INVALID_ARG;
  plan[0] = (int32_t)q.pair;
  plan[1] = (int32_t)q.chains;
  plan[5] = (int32_t)q.product[0][0].splits;
  plan[6] = 0;
  for (int i = 0; i < 3; ++i) {
    plan[2 + i] = (int32_t)q.product[0][i].n;
    for (uint32_t c = 0; c < q.chains; ++c)
      if (q.product[c][i].whole < q.product[c][i].items) plan[6] |= 1 << i;
  }
  plan[7] = q.k <= kSmall;
  return SPARCML_OK;
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
  const Target to{false, out, out_type, out_batch_stride, out_stride, 1.f, 0.f};
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
  const Target to{true,     weight,      w_type, w_batch_stride,
                  w_stride, -lr * scale, 1.f - lr * weight_decay};
  return run_steps(a, q, to, coeffs, steps, ws, static_cast<cudaStream_t>(stream));
}
