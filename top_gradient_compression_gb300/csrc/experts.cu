// Linear layers of experts, each on its own run of the rows, and their gradients:
//
//   y[r] = x[r] W_e',  dx[r] = dy[r] W_e,  dW_e = sum over the expert's rows of dy[r]' x[r]
//
// All three are one product on the tensor cores, out[j][i] = sum over s of P[i][s] Q[j][s]:
//
//            i     j     s     P                           Q
//   forward  n     rows  k     W_e, s contiguous           x, s contiguous
//   dx       k     rows  n     W_e, i contiguous           dy, s contiguous
//   dW       k     n     rows  x, i contiguous             dy, j contiguous
//
// i, the results' contiguous axis, is what a pair of SMs has 256 of: a matrix's side, of any
// size, while the ragged rows are the instruction's N, any multiple of 16 up to 256. So an expert
// with few rows costs what reading its matrix costs and no more. No operand is transposed: the
// tensor cores read either axis as the contiguous one.
//
// One launch, a persistent grid of pairs of SMs. Of a block's twelve warps one loads operands by
// TMA, one issues the products (for both blocks of a pair), eight turn accumulators into results
// while the next tile is under way, one clears rows (below). Where the experts' runs begin and end
// is read on the device: every block works out the same list of tiles from them, and they are
// handed out as pairs get to them. A long summed axis is split where there are few tiles, and for
// dW, whose tiles are as deep as the experts' runs, in those tiles that no whole round of all pairs
// is left for; the parts are added in order by a second launch.
//
// Numbers. Operands as they are (16 bits), sums in fp32, one rounding at the end. The tensor cores
// drop the bits that do not fit when they add to an accumulator, always towards zero: over 16,384
// rows dW came out 1.9e-5 off, and over 2^20 products of one sign y 6e-3, 15 half steps of fp16.
// So an accumulator takes 512 rows of dW, and 1024 of y's and dx's summed axis, and the writers'
// registers add those sums, rounded: dW 5e-7. For dW, the rows of the last 64 that belong to the
// next expert are zeros in both operands, so that what stands there, a NaN say, does not count.
//
// What bounds it is the tensor cores' rate. 16384 rows of one expert, 2048 x 4096 bf16 (143 us at
// the rate of a large library product) in loops of a few ms: forward 147 us, dx 158, dW 163; 8 runs
// of unequal lengths, 4096 x 2048: 170, 169, 188. (Call after call for half a second, under the power
// cap, that forward pass takes 190.) With few rows it is reading the matrices: 9 us for a batch of
// single tokens whose matrices take 5 at the copy rate.

#include <algorithm>
#include <map>
#include <mutex>

#include "stored.cuh"
#include "tensor.cuh"
#include "types.cuh"

namespace sparcml {
namespace {

constexpr uint32_t kMostExperts = 1024;
constexpr uint32_t kSide = 256;      // i and j of a tile, at most
constexpr uint32_t kPairs = 76;      // of SMs
constexpr uint32_t kWriters = 8;     // warps that write results; then loader, issuer, clearer
constexpr uint32_t kThreads = 32 * (kWriters + 4);
constexpr uint32_t kOperand = 128 * 128;  // bytes of one operand's 64 of the summed axis, per block
constexpr uint32_t kStageBytes = 2 * kOperand, kStages = 6;
constexpr uint32_t kSmem = kStages * kStageBytes + 1024;
constexpr uint32_t kBox = 32;        // rows of Q per load
constexpr uint32_t kLeastBlocks = 8;  // forward, dx: of 64 in a part of a split sum, at least
constexpr uint32_t kJoinBlocks = 28;  // dW: blocks of 64 rows that take as long as adding up parts
constexpr uint32_t kSorted = 256;     // dW: experts, at most, that are taken by falling depth
constexpr uint32_t kFeed = 4;         // items that a pair's first loader can be ahead
constexpr uint32_t kBand = 8;        // tiles along j that are taken together, for L2's sake

enum Form { kForward, kInput, kWeight };

// Blocks of 64 of the summed axis that an accumulator takes. What y and dx lose in 1024, 6e-6 where
// all products have one sign, is a 40th of fp16's least half step; dW is an fp32 result. (With 512
// forward took 166 us in place of 162, 16384 rows of 4096 x 2048, one call by itself; in one
// accumulator for the whole axis 159.)
template <int FORM>
constexpr uint32_t kRun = FORM == kWeight ? 8 : 16;

// x from its 8 bits into 16, for dW: a side job of the two warps that dx has nothing to do for, 16
// columns per lane at a time. c 2^e is a number of either type, so nothing is rounded. (Converting
// in the dW kernel itself, on the way to the products, took 500 us in all for 16384 x 2048 x 4096
// against 165 for x in 16 bits: four warps are too few for it, and shared memory, whose bandwidth
// the products' operands take up, is written and read twice more. A kernel of its own takes 32.)
struct Restore {
  const int8_t* codes;  // or null: nothing to do
  int64_t codes_stride;
  const uint8_t* exponents;
  int64_t exponents_stride;
  void* to;        // [rows][pitch]
  uint64_t pitch;  // a multiple of 8
  uint32_t rows, dim;
};

struct ExpertArgs {
  const int32_t* offsets;  // or null: one expert with all rows
  uint32_t experts, rows;
  uint32_t i_size, j_size, s_size;  // j_size for dW, s_size for the others; the rest is rows
  uint32_t tall;        // forward, dx: j of a tile, at most
  uint32_t splits;      // forward, dx: parts of the summed axis
  uint32_t may_split;   // dW: whether tiles may be taken in parts
  uint32_t wide;        // j of a partial tile
  uint32_t shared;      // one matrix for all experts
  void* out;
  int64_t out_batch, out_stride;
  int32_t accumulate;
  uint32_t bf16;        // operands; else fp16
  float* part;          // [slot][wide][256]
  int32_t* status;
  const uint32_t* inject;
  uint32_t* handed_out;
  Restore restore;      // dx: the side job
};
struct ExpertMaps {
  CUtensorMap p, q;
};

// The experts' runs and items, in shared memory. An item is a tile, or a part of its summed axis.
// Of forward and dx all tiles are in `splits` parts. dW takes the experts by falling depth: whole
// tiles first, of which `whole` fill rounds of all pairs, then `rest` tiles in `splits` parts.
struct Table {
  int32_t begin[kMostExperts + 1];   // of the expert's rows; the last: where they end
  uint32_t first[kMostExperts + 1];  // the first item (dW: tile) of the experts in their order
  uint16_t order[kMostExperts];      // dW
  uint32_t items, whole, rest, splits;
};

constexpr uint32_t kNone = 0xffffffffu;
struct Item {
  uint32_t e, i0, j0, width;  // j0: a row of all rows (forward, dx), or of dW's matrix
  uint32_t count;             // of its j, those that exist
  uint32_t row, rows;         // the expert's run
  uint32_t s0, s1;            // blocks of 64 of the summed axis
  uint32_t slot;              // where it is a part: which one, else kNone
};

__device__ __forceinline__ uint32_t ceil_of(uint32_t a, uint32_t b) { return (a + b - 1) / b; }
__device__ __forceinline__ uint32_t rows_of(const Table& t, uint32_t e) {
  return (uint32_t)(t.begin[e + 1] - t.begin[e]);
}

// Where the experts' runs begin, by one warp. An offset out of order or range counts as the
// nearest that is not; returns whether there was one.
__device__ __forceinline__ bool make_runs(const ExpertArgs& a, Table& t) {
  const uint32_t lane = lane_id();
  bool bad = false;
  int32_t carry = 0;
  for (uint32_t base = 0; base <= a.experts; base += 32) {
    const uint32_t e = base + lane;
    const bool there = e <= a.experts;
    const int32_t given = !there ? 0 : a.offsets ? a.offsets[e] : e ? (int32_t)a.rows : 0;
    int32_t v = min(max(given, 0), (int32_t)a.rows);
    if (lane == 0) v = max(v, carry);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= (uint32_t)d) v = max(v, o);
    }
    if (there) t.begin[e] = v;
    bad |= there && v != given;
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  return __any_sync(0xffffffffu, bad);
}

// The rest of the table, from all of a block's threads (and between their barriers).
template <int FORM>
__device__ __forceinline__ void make_items(const ExpertArgs& a, Table& t, uint32_t pairs) {
  // By falling depth, so that the last tiles are the short ones: an expert's place is how many go
  // before it. (Beyond kSorted that count would take longer than it is worth.)
  if (FORM == kWeight) {
    for (uint32_t e = threadIdx.x; e < a.experts; e += blockDim.x) {
      uint32_t place = e;
      if (a.experts <= kSorted) {
        const uint32_t rows = rows_of(t, e);
        place = 0;
        for (uint32_t o = 0; o < a.experts; ++o) {
          const uint32_t r = rows_of(t, o);
          place += r > rows || (r == rows && o < e);
        }
      }
      t.order[place] = (uint16_t)e;
    }
    __syncthreads();
  }
  if (threadIdx.x >= 32) return;
  const uint32_t lane = lane_id();
  const uint32_t ti = ceil_of(a.i_size, kSide), tj = ceil_of(a.j_size, kSide);
  uint32_t sum = 0;
  for (uint32_t base = 0; base < a.experts; base += 32) {
    const uint32_t e = base + lane;
    uint32_t n = 0;
    if (e < a.experts)
      n = FORM == kWeight ? ti * tj : ti * ceil_of(rows_of(t, e), a.tall) * a.splits;
    const uint32_t upto = warp_incl_sum(n);
    if (e < a.experts) t.first[e] = sum + upto - n;
    sum += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (FORM != kWeight) {
    if (lane == 0) {
      t.first[a.experts] = t.items = sum;
      t.splits = a.splits;
    }
    return;
  }
  // The rest after whole rounds, in as many parts as it is done soonest with. Rounds of parts of
  // the rest's deepest tile count, and kJoinBlocks for adding the parts up.
  const uint32_t rest = sum % pairs, whole = sum - rest;
  uint32_t splits = 1;
  if (a.may_split && rest) {
    // The deepest's rows, wherever it stands: experts may be unsorted. (By the first one's, 16384
    // rows of the last of 308 experts of 64 x 64 took 95 us in place of 37.)
    uint32_t rows = 0;
    for (uint32_t place = whole / (ti * tj) + lane; place < a.experts; place += 32)
      rows = max(rows, rows_of(t, t.order[place]));
    const uint32_t depth = ceil_of(__reduce_max_sync(0xffffffffu, rows), 64);
    const uint32_t most = min(2 * pairs / rest, depth / kLeastBlocks);
    auto cost = [](uint32_t blocks, uint32_t parts) {  // blocks, then parts (at most 152)
      return min(blocks, 0xffffffu) << 8 | parts;
    };
    uint32_t best = cost(depth, 1);
    for (uint32_t c = 2 + lane; c <= most; c += 32)
      best = min(best, cost(ceil_of(rest * c, pairs) * ceil_of(depth, c) + kJoinBlocks, c));
    splits = __reduce_min_sync(0xffffffffu, best) & 255u;
  }
  if (lane == 0) {
    t.first[a.experts] = sum;
    t.whole = whole;
    t.rest = rest;
    t.splits = splits;
    t.items = whole + rest * splits;
  }
}

template <int FORM>
__device__ __forceinline__ Item item_of(const ExpertArgs& a, const Table& t, uint32_t index) {
  uint32_t tile = index, split = 0, splits = 1;
  if (FORM == kWeight && index >= t.whole) {
    // all tiles' first parts, then their second ones: neighbours read the same rows
    split = (index - t.whole) / t.rest;
    tile = index - split * t.rest;
    splits = t.splits;
  }
  uint32_t lo = 0, hi = a.experts;  // first[lo] <= tile < first[hi]
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (t.first[mid] <= tile) lo = mid;
    else hi = mid;
  }
  uint32_t u = tile - t.first[lo];
  Item it;
  it.e = FORM == kWeight ? t.order[lo] : lo;
  it.row = (uint32_t)t.begin[it.e];
  it.rows = rows_of(t, it.e);
  if (FORM != kWeight && a.splits > 1) {
    splits = a.splits;
    split = u % splits;
    u /= splits;
  }
  it.slot = splits == 1 ? kNone : FORM == kWeight ? index - t.whole : index;
  const uint32_t blocks = ceil_of(FORM == kWeight ? it.rows : a.s_size, 64);
  it.s0 = (uint32_t)((uint64_t)blocks * split / splits);
  it.s1 = (uint32_t)((uint64_t)blocks * (split + 1) / splits);
  const uint32_t j_size = FORM == kWeight ? a.j_size : it.rows;
  const uint32_t tj = ceil_of(j_size, FORM == kWeight ? kSide : a.tall);
  const uint32_t ti = ceil_of(a.i_size, kSide);
  // the rows of an expert are shared out evenly; of dW's matrix only the last tile is narrower
  it.width = FORM == kWeight ? kSide : (ceil_of(j_size, tj) + 15) / 16 * 16;
  const uint32_t band = u / (ti * kBand), rest = u - band * ti * kBand;
  const uint32_t across = min(kBand, tj - band * kBand), i = rest / across;
  const uint32_t j = (band * kBand + rest - i * across) * it.width;
  it.i0 = i * kSide;
  it.count = min(it.width, j_size - j);
  it.j0 = FORM == kWeight ? j : it.row + j;
  return it;
}

struct Worker {
  uint32_t ring, full, empty, acc_full, acc_empty, tail;  // shared-memory addresses
  uint32_t fed, lead_fed_empty, feed_full;  // of the feed: its values and barriers
  uint32_t lead_full, lead_acc_empty, own_tail;           // in the cluster's shared memory
  uint32_t rank, pair, pairs, items, tmem;
  bool leader;  // the lane that issues for its warp
  Waits* waits;
  uint32_t stage = 0, phase = 0, acc = 0, tails = 0;
  uint32_t feed = 0, feed_phase = 0;  // the feed's next slot, and its turn's parity
  __device__ __forceinline__ void next_stage() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void skip(uint32_t blocks) {  // stages that others go through
    const uint32_t at = stage + blocks;
    stage = at % kStages;
  }
  __device__ __forceinline__ void next_feed() {
    if (++feed == kFeed) {
      feed = 0;
      feed_phase ^= 1u;
    }
  }
};

// Items are handed out as pairs get to them: the first of each is its own number, of the others the
// loader of a pair's first block draws the number when it begins the one before, and feeds it to
// all other warps of both blocks. (With every 76th tile to each pair, 16384 rows in 8 unequal runs
// took 234 us for 4096 x 2048, and with shares of one stream of blocks, which no longer read the
// same rows at the same time, 237.)
//
// Every pair draws until it gets a number past the end; who draws the last of those resets the
// counter for the next kernel.
__device__ __forceinline__ uint32_t draw_item(const Worker& w, const ExpertArgs& a) {
  uint32_t drawn = 0;
  if (w.leader) drawn = atomicAdd(a.handed_out, 1u);
  return drawn;
}
__device__ __forceinline__ uint32_t drawn_item(const Worker& w, const ExpertArgs& a,
                                               uint32_t drawn) {
  if (w.leader && drawn == w.items - 1) *a.handed_out = 0;
  const uint32_t lane = __ffs(__ballot_sync(0xffffffffu, w.leader)) - 1;
  const uint32_t x = w.pairs + __shfl_sync(0xffffffffu, drawn, lane);
  return x < w.items ? x : kNone;
}
// Tells both blocks' warps; kNone if they do not get to it in time.
__device__ __forceinline__ uint32_t feed_item(Worker& w, uint32_t fed_empty, uint32_t x) {
  const uint32_t s = w.feed;
  if (!mbar_wait_warp_inline<true>(fed_empty + 8 * s, w.feed_phase ^ 1u, w.waits)) return kNone;
  if (w.leader) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(w.fed + 4 * s), "r"(x) : "memory");
    mbar_arrive(w.feed_full + 8 * s);
    // (released for the pair by an arrival, it would take this warp a microsecond)
    store_cluster_async(cluster_addr(w.fed + 4 * s, 1), x, cluster_addr(w.feed_full + 8 * s, 1));
  }
  __syncwarp();
  w.next_feed();
  return x;
}
// The next item of any other warp. LOADER: the second block's, which has the feed's barrier expect
// the word.
template <bool LOADER = false>
__device__ __forceinline__ uint32_t next_item(Worker& w) {
  if (w.items <= w.pairs) return kNone;
  const uint32_t s = w.feed;
  if (LOADER && w.leader) mbar_expect_tx(w.feed_full + 8 * s, 4);
  if (!mbar_wait_warp_inline<true>(w.feed_full + 8 * s, w.feed_phase, w.waits)) return kNone;
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(w.fed + 4 * s) : "memory");
  // All lanes have read the same word, so this is always true; but it takes the word itself to find
  // out, and so the reads are over before the arrival that lets the feeder write the slot again. (The
  // arrival is relaxed: releasing, it would also wait for what the warp has stored, 194 us against
  // 187 for dx of 16384 rows in 8 runs, 4096 x 2048, 210 against 204 for dW.)
  const bool read = __all_sync(0xffffffffu, x == __shfl_sync(0xffffffffu, x, 0));
  if (w.leader && read) mbar_arrive_cluster(w.lead_fed_empty + 8 * s);
  __syncwarp();
  w.next_feed();
  return x;
}

// Both blocks of a pair load their halves of P and Q; the first one's barriers count for both. The
// last rows of an expert's run go to a barrier of the block's own, and are reported by its clearer
// once those of the next expert are zeros.
template <int FORM>
__device__ __forceinline__ bool load_item(Worker& w, const ExpertMaps& m, const ExpertArgs& a,
                                          const Item& it) {
  const uint32_t i0 = it.i0 + 128 * w.rank, j0 = it.j0 + it.width / 2 * w.rank;
  const uint32_t boxes = (it.width / 2 + kBox - 1) / kBox;
  const uint32_t bytes = kOperand + (FORM == kWeight ? kOperand : boxes * kBox * 128);
  for (uint32_t b = it.s0; b < it.s1; ++b, w.next_stage()) {
    const uint32_t s = w.stage;
    if (!mbar_wait_warp_inline(w.empty + 8 * s, w.phase ^ 1u, w.waits)) return false;
    const bool cut = FORM == kWeight && it.rows - b * 64 < 64;
    const uint32_t bar = cut ? w.own_tail + 8 * s : w.lead_full + 8 * s;
    const uint32_t p = w.ring + s * kStageBytes, q = p + kOperand;
    if (w.leader) {
      if (cut) mbar_expect_tx(w.tail + 8 * s, bytes);
      else if (w.rank == 0) mbar_expect_tx(w.full + 8 * s, 2 * bytes);
      else mbar_arrive_cluster(w.lead_full + 8 * s);
      const uint32_t at = FORM == kWeight ? it.row + b * 64 : b * 64;
      if constexpr (FORM == kForward) {
        tma_load_3d_pair(p, &m.p, at, i0, a.shared ? 0 : it.e, bar);
      } else {
        const uint32_t z = FORM == kInput && !a.shared ? it.e : 0;
        tma_load_3d_pair(p, &m.p, i0, at, z, bar);
        tma_load_3d_pair(p + kOperand / 2, &m.p, i0 + 64, at, z, bar);
      }
      if constexpr (FORM == kWeight) {
        tma_load_3d_pair(q, &m.q, j0, at, 0, bar);
        tma_load_3d_pair(q + kOperand / 2, &m.q, j0 + 64, at, 0, bar);
      } else {
        for (uint32_t k = 0; k < boxes; ++k)
          tma_load_3d_pair(q + k * kBox * 128, &m.q, at, j0 + k * kBox, 0, bar);
      }
    }
    __syncwarp();
  }
  return true;
}

// The clearer: waits for an item's last block where that is cut, and clears the rows behind the
// run. (When the loader did so, it began the next loads 3 us later: 190 us in place of 161 for 4
// runs of odd lengths.)
__device__ __forceinline__ bool clear_item(Worker& w, const Item& it) {
  const uint32_t blocks = it.s1 - it.s0;
  if (blocks > 0) {
    const uint32_t left = it.rows - (it.s1 - 1) * 64;  // rows of the last block
    w.skip(blocks - 1);
    if (left < 64) {
      const uint32_t s = w.stage, p = w.ring + s * kStageBytes;
      if (!mbar_wait_warp_inline(w.tail + 8 * s, w.tails >> s & 1u, w.waits)) {
        Waits alone = {0, kLandUs};  // what was begun has to land before the block leaves
        mbar_wait_warp_inline(w.tail + 8 * s, w.tails >> s & 1u, &alone);
        return false;
      }
      w.tails ^= 1u << s;
      // a row is 128 bytes of each of the boxes of 8 KB: two of P, two of Q
#pragma unroll
      for (uint32_t box = 0; box < 4; ++box)
        for (uint32_t at = left * 128 + 16 * lane_id(); at < 64 * 128; at += 512)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                           p + box * (kOperand / 2) + at),
                       "r"(0)
                       : "memory");
      proxy_fence_shared();
      __syncwarp();
      if (w.leader) mbar_arrive_cluster_release(w.lead_full + 8 * s);
      __syncwarp();
    }
    w.skip(1);
  }
  return true;
}

// Eight pieces of a lane are on their way at a time. (With two the side job took 100 us longer than
// the products beside it.)
template <typename T>
__device__ __forceinline__ void restore_rows(const Restore& x, uint32_t thread, uint32_t threads) {
  constexpr int kBatch = 8;
  const uint32_t pieces = ceil_of(x.dim, 16);
  uint32_t row = thread / pieces, piece = thread - row * pieces;
  const uint32_t rows_on = threads / pieces, pieces_on = threads - rows_on * pieces;
  while (row < x.rows) {
    uint4 w[kBatch];
    uint32_t e[kBatch];
    uint4* to[kBatch];
    bool both[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      to[q] = nullptr;
      if (row < x.rows) {
        w[q] = __ldg(reinterpret_cast<const uint4*>(x.codes + (int64_t)row * x.codes_stride) +
                     piece);
        e[q] = __ldg(x.exponents + (int64_t)row * x.exponents_stride + piece / (kGroup / 16));
        to[q] = reinterpret_cast<uint4*>(static_cast<T*>(x.to) + row * x.pitch + 16 * piece);
        both[q] = 16 * piece + 8 < x.pitch;
      }
      row += rows_on;
      piece += pieces_on;
      if (piece >= pieces) {
        piece -= pieces;
        ++row;
      }
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (!to[q]) continue;
      const float scale = scale_of(e[q]);
      const uint32_t words[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
      F2 lo[4], hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        lo[k] = f2(code_at(words[k / 2], 2 * k % 4) * scale,
                   code_at(words[k / 2], 2 * k % 4 + 1) * scale);
        hi[k] = f2(code_at(words[2 + k / 2], 2 * k % 4) * scale,
                   code_at(words[2 + k / 2], 2 * k % 4 + 1) * scale);
      }
      to[q][0] = pack<T, 8>(lo);
      if (both[q]) to[q][1] = pack<T, 8>(hi);
    }
  }
}

template <int FORM>
__device__ __forceinline__ bool issue_item(Worker& w, const ExpertArgs& a, const Item& it) {
  constexpr bool P_MN = FORM != kForward, Q_MN = FORM == kWeight;
  constexpr uint32_t step_p = P_MN ? 2048 : 32, step_q = Q_MN ? 2048 : 32;
  const uint32_t idesc = mma_desc(256, it.width, P_MN, Q_MN, a.bf16);
  for (uint32_t b = it.s0; b < it.s1;) {
    const uint32_t from = b, end = min(b + kRun<FORM>, it.s1);
    const uint32_t acc = w.acc & 1u;
    if (!mbar_wait_warp_inline(w.acc_empty + 8 * acc, ((w.acc >> 1) & 1u) ^ 1u, w.waits))
      return false;
    tmem_fence_after();
    const uint32_t d = w.tmem + acc * kSide;
    for (; b < end; ++b, w.next_stage()) {
      const uint32_t s = w.stage;
      // With dW, ordinary stores of either block may be part of the stage, so the wait acquires for
      // the pair. (As a fence of its own that took a microsecond for every block: 572 us against
      // 190 for 16384 x 2048 x 4096.)
      if (!mbar_wait_warp_inline<FORM == kWeight>(w.full + 8 * s, w.phase, w.waits)) return false;
      tmem_fence_after();
      if (w.leader) {
        const uint32_t p = w.ring + s * kStageBytes, q = p + kOperand;
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          mma_f16<2>(d, tile_desc(p + k * step_p, 8192, 1024),
                     tile_desc(q + k * step_q, 8192, 1024), idesc, b > from || k > 0);
        mma_commit<2>(w.empty + 8 * s);
      }
      __syncwarp();
    }
    if (w.leader) mma_commit<2>(w.acc_full + 8 * acc);
    __syncwarp();
    ++w.acc;
  }
  return true;
}

// N sums of a thread to their results, `step` elements apart, of which `count` exist. dW alone
// (fp32) is added to what is there, by the memory itself: one addition to each element, so that
// nothing depends on an order. (Read, added and written by the thread, 8 at a time, 16384 rows in 8
// unequal runs took 308 us for 4096 x 2048, one by one 921; so it is 205, and 188 without adding.)
template <int FORM, int N>
__device__ __forceinline__ void put(const ExpertArgs& a, int64_t at, int64_t step, uint32_t count,
                                    const float* v) {
  if (FORM != kWeight) {
    uint16_t* const o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
    for (uint32_t q = 0; q < N; q += 2) {
      const F2 two = f2(v[q], v[q + 1]);
      const uint32_t b = pack2<__nv_bfloat16>(two), h = pack2<__half>(two), w = a.bf16 ? b : h;
      if (q < count) o[(int64_t)q * step] = (uint16_t)w;
      if (q + 1 < count) o[(int64_t)(q + 1) * step] = (uint16_t)(w >> 16);
    }
    return;
  }
  float* const o = static_cast<float*>(a.out) + at;
  if (a.accumulate) {
#pragma unroll
    for (uint32_t q = 0; q < N; ++q)
      if (q < count)
        asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(o + (int64_t)q * step),
                     "f"(v[q])
                     : "memory");
  } else {
#pragma unroll
    for (uint32_t q = 0; q < N; ++q)
      if (q < count) o[(int64_t)q * step] = v[q];
  }
}

// Sixteen sums of a thread's i, from column c of the tile: to their results, or where the parts of
// a split sum wait to be added up.
template <int FORM>
__device__ __forceinline__ void put16(const ExpertArgs& a, const Item& it, uint32_t side,
                                      uint32_t c, const float (&v)[16]) {
  const uint32_t i = it.i0 + side;
  if (it.slot != kNone) {
    float* o = a.part + ((uint64_t)it.slot * a.wide + c) * kSide + side;
#pragma unroll
    for (int q = 0; q < 16; ++q) o[q * kSide] = v[q];
  } else if (i < a.i_size) {
    const int64_t out = (FORM == kWeight ? (int64_t)it.e * a.out_batch : 0) +
                        (int64_t)(it.j0 + c) * a.out_stride + i;
    put<FORM, 16>(a, out, a.out_stride, it.count - c, v);
  }
}

// An accumulator's rows are i, its columns j: a warp has 32 neighbouring i, so that it writes
// whole stretches of a result's row as they come. The two warps of a quarter of the i alternate
// over the columns, sixteen at a time. A warp that is done with its columns leaves what is written
// out for the others by one jump: instructions that were not used yet take long to come. (With a jump
// over each of them, and a way of its own for either type of y, 1024 rows of 4864 x 4096 took 29.2 us
// in place of 27.0, in pieces of 512.)
template <int FORM>
__device__ __forceinline__ bool write_item(Worker& w, const ExpertArgs& a, const Item& it) {
  const uint32_t warp = threadIdx.x >> 5, quarter = warp & 3u, half = warp >> 2;
  const uint32_t side = 128 * w.rank + 32 * quarter + lane_id();
  const uint32_t src = w.tmem + (quarter << 21);
  auto next = [&]() {  // the next accumulator, once it is full
    const uint32_t acc = w.acc & 1u;
    if (!mbar_wait_warp_inline(w.acc_full + 8 * acc, (w.acc >> 1) & 1u, w.waits)) return false;
    tmem_fence_after();
    return true;
  };
  auto done = [&]() {
    tmem_fence_before();
    __syncwarp();
    if (lane_id() == 0) mbar_arrive_cluster(w.lead_acc_empty + 8 * (w.acc & 1u));
    ++w.acc;
  };
  auto from = [&](uint32_t c) { return src + (w.acc & 1u) * kSide + c; };
  if (it.s1 - it.s0 <= kRun<FORM>) {  // one accumulator, or (dW) none
    const bool any = it.s1 > it.s0;
    if (any && !next()) return false;
#pragma unroll 1
    for (uint32_t c = 16 * half; c < it.count; c += 64) {  // two loads on their way at a time
      float u[16] = {}, v[16] = {};
      if (any) {
        tmem_load16(from(c), u);
        tmem_load16(from(min(c + 32, kSide - 16)), v);
        tmem_load_wait(u);
        tmem_load_wait(v);
      }
      put16<FORM>(a, it, side, c, u);
      if (c + 32 < it.count) put16<FORM>(a, it, side, c + 32, v);
    }
    if (any) done();
    return true;
  }
  // The accumulators' sums are added up here, rounded to nearest.
  float sum[8][16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int q = 0; q < 16; ++q) sum[k][q] = 0.f;
  }
  for (uint32_t b = it.s0; b < it.s1; b += kRun<FORM>) {
    if (!next()) return false;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t c = 32 * k + 16 * half;
      if (c >= it.count) break;
      float v[16];
      tmem_load16(from(c), v);
      tmem_load_wait(v);
#pragma unroll
      for (int q = 0; q < 16; ++q) sum[k][q] += v[q];
    }
    done();
  }
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) {
    const uint32_t c = 32 * k + 16 * half;
    if (c >= it.count) break;
    put16<FORM>(a, it, side, c, sum[k]);
  }
  return true;
}

template <int FORM>
__global__ void __launch_bounds__(kThreads, 1)
experts_kernel(const __grid_constant__ ExpertMaps m, const __grid_constant__ ExpertArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ alignas(8) uint64_t bars[3 * kStages + 5 + 2 * kFeed];
  // partner: whether the other block gave up; armed: whether a fault is injected
  __shared__ uint32_t tmem_slot, partner, armed, fed[kFeed];
  __shared__ Waits waits;
  __shared__ Table table;
  const uint32_t warp = threadIdx.x >> 5;
  Worker w;
  w.ring = (smem_addr(raw) + 1023u) & ~1023u;
  w.full = smem_addr(bars);
  w.empty = w.full + 8 * kStages;
  w.acc_full = w.empty + 8 * kStages;
  w.acc_empty = w.acc_full + 16;
  w.tail = w.acc_empty + 16;
  w.feed_full = w.tail + 8 * kStages;
  const uint32_t fed_empty = w.feed_full + 8 * kFeed, finished = fed_empty + 8 * kFeed;
  w.fed = smem_addr(fed);
  w.rank = cluster_rank();
  w.pair = blockIdx.x / 2;
  w.pairs = gridDim.x / 2;
  w.waits = &waits;
  w.lead_full = cluster_addr(w.full, 0);
  w.lead_acc_empty = cluster_addr(w.acc_empty, 0);
  w.own_tail = cluster_addr(w.tail, w.rank);
  w.lead_fed_empty = cluster_addr(fed_empty, 0);
  w.leader = elect_one();
  if (threadIdx.x < 2) tma_prefetch_map(threadIdx.x ? &m.q : &m.p);
  if (threadIdx.x == 0) {
    waits.gave_up = 0;
    partner = 0;
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(w.full + 8 * s, 2);
      mbar_init(w.empty + 8 * s, 1);
      mbar_init(w.tail + 8 * s, 1);
    }
    for (uint32_t s = 0; s < 2; ++s) {
      mbar_init(w.acc_full + 8 * s, 1);
      mbar_init(w.acc_empty + 8 * s, 2 * kWriters);
    }
    mbar_init(finished, 1);
    for (uint32_t s = 0; s < kFeed; ++s) {
      mbar_init(w.feed_full + 8 * s, 1);
      // both blocks' writers and clearers, one issuer and one loader
      mbar_init(fed_empty + 8 * s, 2 * (kWriters + (FORM == kWeight ? 1 : 0)) + 2);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWriters) tmem_alloc<2>(smem_addr(&tmem_slot), 2 * kSide);
  griddep_wait();  // up to here nothing is read or written that another kernel may have
  if (threadIdx.x == 0) {
    // A warp may have to wait for a whole tile (the clearer for its end, all for the next one), of up
    // to 2^25 blocks of 64, which take 0.25 us each. So a block adds 4 us.
    armed = injected(a.inject);
    waits.limit_us = (armed ? kInjectWaitUs : kWaitUs) + (FORM == kWeight ? a.rows : a.s_size) / 16;
  }
  if (warp == 1) {
    const bool bad = make_runs(a, table);
    if (bad && blockIdx.x == 0 && w.leader) set_status(a.status, SPARCML_ERR_BAD_STREAM);
  }
  __syncthreads();
  make_items<FORM>(a, table, w.pairs);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  w.tmem = tmem_slot;
  w.items = table.items;

  uint32_t x = w.pair;
  if (warp < kWriters) {
    for (; x < w.items; x = next_item(w))
      if (!write_item<FORM>(w, a, item_of<FORM>(a, table, x))) break;
  } else if (warp == kWriters && w.rank == 0) {
    const bool draws = w.items > w.pairs;
    while (x < w.items) {
      uint32_t drawn = draws ? draw_item(w, a) : 0;
      const bool loaded = load_item<FORM>(w, m, a, item_of<FORM>(a, table, x));
      x = draws ? drawn_item(w, a, drawn) : kNone;
      if (!draws || (loaded && feed_item(w, fed_empty, x) == x)) continue;
      while (x != kNone) {  // given up: the counter is left as the next kernel needs it
        drawn = draw_item(w, a);
        x = drawn_item(w, a, drawn);
      }
    }
  } else if (warp == kWriters) {
    for (; x < w.items; x = next_item<true>(w))
      if (!load_item<FORM>(w, m, a, item_of<FORM>(a, table, x))) break;
  } else if (warp == kWriters + 1) {
    // An injected fault: the first pair withholds its products.
    const bool withhold = w.pair == 0 && armed;
    if (w.rank == 0 && !withhold)
      for (; x < w.items; x = next_item(w))
        if (!issue_item<FORM>(w, a, item_of<FORM>(a, table, x))) break;
  } else if (FORM == kWeight) {
    if (warp == kWriters + 2)
      for (; x < w.items; x = next_item(w))
        if (!clear_item(w, item_of<FORM>(a, table, x))) break;
  } else if (FORM == kInput && a.restore.codes) {
    const uint32_t thread = 64 * blockIdx.x + (threadIdx.x - 32 * (kWriters + 2));
    if (a.bf16) restore_rows<__nv_bfloat16>(a.restore, thread, 64 * gridDim.x);
    else restore_rows<__half>(a.restore, thread, 64 * gridDim.x);
  }
  tmem_fence_before();
  __syncthreads();  // now it is settled whether this block gave up
  if (threadIdx.x == 0)
    store_cluster(cluster_addr(smem_addr(&partner), w.rank ^ 1u), waits.gave_up);
  __syncwarp();
  cluster_sync();
  if (waits.gave_up || partner) {
    // Nothing may still be in flight when the shared and tensor memory go: loads and what was fed
    // get their time to land, products are waited for.
    if (warp == kWriters && w.leader) {
      const uint64_t end = global_ns() + 1000ull * kLandUs;
      while (global_ns() < end) __nanosleep(1000);
    }
    if (warp == kWriters + 1 && w.leader) {
      // arrives, in both blocks of a pair, once all products have completed
      Waits alone = {0, kWaitUs};
      if (w.rank == 0) mma_commit<2>(finished);
      mbar_wait_inline(finished, 0, &alone);
    }
    __syncwarp();
    if (threadIdx.x == 0) set_status(a.status, SPARCML_ERR_TIMEOUT);
    __syncthreads();
    cluster_sync();
  }
  tmem_fence_after();
  if (warp == kWriters) tmem_free<2>(w.tmem, 2 * kSide);
}

// The parts of split sums, added in their order: four rows of 256 i for a block at a time, four
// neighbouring i for a thread.
template <int FORM>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ ExpertArgs a,
                                                         uint32_t pairs) {
  __shared__ Table table;
  griddep_wait();
  if (threadIdx.x < 32) make_runs(a, table);
  __syncthreads();
  make_items<FORM>(a, table, pairs);
  __syncthreads();
  const uint32_t groups = a.wide / 4, splits = table.splits;
  if (splits == 1) return;
  const uint32_t tiles = FORM == kWeight ? table.rest : table.items / splits;
  const uint32_t from = FORM == kWeight ? table.whole : 0;
  // a tile's parts: neighbours, or (dW) a round apart
  const uint32_t on = FORM == kWeight ? table.rest : 1, step = FORM == kWeight ? 1 : splits;
  for (uint32_t x = blockIdx.x; x < tiles * groups; x += gridDim.x) {
    const uint32_t tile = x / groups, slot = tile * step;
    const Item it = item_of<FORM>(a, table, from + slot);
    const uint32_t j = 4 * (x - tile * groups) + threadIdx.x / 64, i = 4 * (threadIdx.x % 64);
    if (j >= it.count || it.i0 + i >= a.i_size) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (uint32_t s = 0; s < splits; ++s) {
      const float4 q = __ldcg(reinterpret_cast<const float4*>(
          a.part + ((uint64_t)(slot + s * on) * a.wide + j) * kSide + i));
      v.x += q.x;
      v.y += q.y;
      v.z += q.z;
      v.w += q.w;
    }
    const int64_t out = (FORM == kWeight ? (int64_t)it.e * a.out_batch : 0) +
                        (int64_t)(it.j0 + j) * a.out_stride + it.i0 + i;
    const float f[4] = {v.x, v.y, v.z, v.w};
    put<FORM, 4>(a, out, 1, a.i_size - it.i0 - i, f);
  }
}

// Operands whose rows are not what TMA takes (16-byte aligned, 16 bytes a step), copied into rows
// of `pitch` elements; 16 bytes per thread and turn.
struct Copy {
  const uint16_t* from;
  int64_t batch, stride;
  uint16_t* to;
  uint64_t pitch, rows, cols, all;  // all: rows of all matrices
};
struct CopyArgs {
  Copy of[3];
};
__global__ void __launch_bounds__(256) copy_rows_kernel(const __grid_constant__ CopyArgs args) {
  griddep_wait();
  const Copy& a = args.of[blockIdx.y];
  const uint64_t per = a.pitch / 8, total = a.all * per;
  for (uint64_t x = blockIdx.x * (uint64_t)blockDim.x + threadIdx.x; x < total;
       x += (uint64_t)gridDim.x * blockDim.x) {
    const uint64_t r = x / per, c = (x - r * per) * 8, b = r / a.rows;
    const uint16_t* p = a.from + (int64_t)b * a.batch + (int64_t)(r - b * a.rows) * a.stride + c;
    uint32_t v[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = c + i < a.cols ? p[i] : 0u;
    reinterpret_cast<uint4*>(a.to)[x] =
        make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

// ---------------------------------------------------------------------------
// Host side.

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

struct Sizes {
  uint64_t rows, experts, n, k;
  bool ok() const {
    return rows <= 0x7fffffffull && experts >= 1 && experts <= kMostExperts && n >= 1 &&
           n <= (1u << 24) && k >= 1 && k <= (1u << 24) &&
           // counted in 32 bits on the device (more would not fit the memory, or take minutes)
           ceil_div(std::max(n, k), kSide) * (rows / kSide + experts) < (1ull << 31) &&
           (rows / 64 + experts) * ceil_div(n, kSide) * ceil_div(k, kSide) < (1ull << 31);
  }
  // Forward and dx: the most tiles that the rows can make where one takes `tall` of them.
  uint64_t most_tiles(uint64_t i, uint32_t tall) const {
    return ceil_div(i, kSide) * (std::min(experts, rows) + rows / tall);
  }
  // Forward and dx: the most rows of a tile, and the parts of the summed axis, where all tiles and
  // parts together are one round of all pairs (else 256, and one part): what takes least by times
  // in ns that were measured on short calls. A block of 64 takes 240 with 64 rows and 272 with
  // 256, writing 12.5 a row, adding up parts 3,000. (64 rows in place of 256, us: 1237 rows of 5 x 776
  // x 336 dx 9.9 for 12.2, 512 of 2048 x 2048 14.2 for 17.0; but dx of 300 rows of 8192 x 2048
  // 22 with 256 rows and 4 parts, 36 with 64 and one.)
  struct Plan {
    uint32_t tall, splits;
  };
  Plan plan(uint64_t i, uint64_t s) const {
    const uint64_t blocks = ceil_div(s, 64);
    Plan best = {kSide, 1};
    uint64_t least = ~0ull;
    for (uint32_t tall = kSide; tall >= 64; tall /= 2) {
      const uint64_t tiles = most_tiles(i, tall);
      for (uint64_t c = 1; c * tiles <= kPairs && (c == 1 || c * kLeastBlocks <= blocks); ++c) {
        const uint64_t ns = ceil_div(blocks, c) * (230 + tall / 6) + tall * 25 / 2 +
                            (c > 1 ? 3000 : 0);
        if (ns < least) {
          least = ns;
          best = {tall, (uint32_t)c};
        }
      }
    }
    return best;
  }
  uint64_t weight_tiles() const { return experts * ceil_div(n, kSide) * ceil_div(k, kSide); }
  bool weight_splits() const { return rows > 64 * kJoinBlocks; }
  size_t part_bytes() const {
    size_t r = 0;
    if (plan(n, k).splits > 1 || plan(k, n).splits > 1)
      r = (size_t)kPairs * std::min<uint64_t>(kSide, align_up(rows, 16)) * kSide * 4;
    if (weight_splits()) r = std::max(r, (size_t)2 * kPairs * kSide * kSide * 4);
    return align_up(r, 256);
  }
};

struct Operand {  // `batches` matrices of `rows` rows of `cols` elements of 16 bits
  const void* p;
  int64_t batch, stride;
  uint64_t batches, rows, cols;

  // The matrices of all experts, of which there is one where they lie at one place.
  static Operand matrices(const void* p, int64_t batch, int64_t stride, const Sizes& z) {
    return {p, batch, stride, batch == 0 ? 1 : z.experts, z.n, z.k};
  }

  uint64_t pitch() const { return align_up(cols, 8); }
  size_t copy_bytes() const { return align_up(batches * rows * pitch() * 2, 256); }
  bool fits() const {
    return aligned_to(p, 16) && (rows == 1 || (stride % 8 == 0 && stride >= (int64_t)cols)) &&
           (batches == 1 || (batch % 8 == 0 && batch >= (int64_t)cols));
  }
};

// Has operands (null: none) as TMA takes them, by copies where they are not; bytes(): what these
// take.
struct Settle {
  Operand* of[3];
  size_t bytes() const {
    size_t r = 0;
    for (const Operand* o : of)
      if (o && o->rows && !o->fits()) r += o->copy_bytes();
    return r;
  }
  void run(uint8_t* room, cudaStream_t s) const {
    CopyArgs a = {};
    unsigned count = 0;
    uint64_t most = 0;
    for (Operand* o : of) {
      if (!o || !o->rows || o->fits()) continue;
      Copy& c = a.of[count++];
      c = {static_cast<const uint16_t*>(o->p), o->batch, o->stride,
           reinterpret_cast<uint16_t*>(room), o->pitch(), o->rows, o->cols, o->rows * o->batches};
      most = std::max(most, c.all * c.pitch);
      room += o->copy_bytes();
      o->p = c.to;
      o->stride = (int64_t)c.pitch;
      o->batch = (int64_t)(c.pitch * c.rows);
    }
    if (!count) return;
    launch_pdl(copy_rows_kernel,
               dim3((unsigned)std::min<uint64_t>(ceil_div(most, 8 * 256), 152 * 8), count), 256, 0,
               s, a);
    note_launches(1);
  }
};

bool map_of(CUtensorMap* map, const Operand& o, bool bf16, uint32_t box_rows) {
  const cuuint64_t row = (o.rows == 1 ? o.pitch() : (uint64_t)o.stride) * 2;
  const cuuint64_t dims[3] = {o.cols, o.rows, o.batches};
  const cuuint64_t strides[2] = {row, o.batches == 1 ? row : (uint64_t)o.batch * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  return encode_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    o.p, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Pairs of SMs that run the kernel at one time on the current device; 0 if that cannot be found
// out. Asked for once per device.
template <int FORM>
unsigned resident() {
  static std::mutex lock;
  static std::map<int, unsigned> known;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> hold(lock);
  const auto it = known.find(device);
  if (it != known.end()) return it->second;
  auto kernel = experts_kernel<FORM>;
  if (!ensure_smem(reinterpret_cast<const void*>(kernel), kSmem)) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * kPairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int count = 0;
  if (cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) != cudaSuccess) return 0;
  const unsigned fit = (unsigned)std::min<int>(count, kPairs);
  known[device] = fit;
  return fit;
}

template <int FORM>
int launch_experts(const ExpertMaps& m, const ExpertArgs& a, uint64_t most_items,
                   uint64_t join_units, cudaStream_t s) {
  const bool join = join_units > 0;
  auto kernel = experts_kernel<FORM>;
  const unsigned fit = resident<FORM>();
  if (fit == 0 || !ensure_smem(reinterpret_cast<const void*>(kernel), kSmem))
    return SPARCML_ERR_CUDA;
  const unsigned pairs = (unsigned)std::min<uint64_t>(fit, most_items);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  (void)cudaLaunchKernelEx(&cfg, kernel, m, a);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  if (join) {
    launch_pdl(join_parts_kernel<FORM>, (unsigned)std::min<uint64_t>(join_units, 152 * 8), 256, 0,
               s, a, pairs);
    if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  }
  note_launches(1 + join);
  return SPARCML_OK;
}

struct Call {
  Sizes z;
  int32_t type;
  const int32_t* offsets;
  void* ws;
  size_t ws_bytes;
  cudaStream_t stream;
};

struct Stored {  // x in 8 bits
  const int8_t* codes;
  int64_t codes_stride;
  const uint8_t* exponents;
  int64_t exponents_stride;
};

// The product of operands that TMA takes; dx with a side job, or none.
template <int FORM>
int run(const Call& c, Operand p, Operand q, void* out, int64_t out_batch, int64_t out_stride,
        int32_t accumulate, const Restore& side = {}) {
  const Sizes& z = c.z;
  uint8_t* w = static_cast<uint8_t*>(c.ws);
  ExpertArgs a = {};
  a.offsets = c.offsets;
  a.experts = (uint32_t)z.experts;
  a.rows = (uint32_t)z.rows;
  a.i_size = (uint32_t)(FORM == kForward ? z.n : z.k);
  a.j_size = FORM == kWeight ? (uint32_t)z.n : 0;
  a.s_size = (uint32_t)(FORM == kForward ? z.k : FORM == kInput ? z.n : 0);
  const Sizes::Plan plan = FORM == kWeight ? Sizes::Plan{kSide, 1} : z.plan(a.i_size, a.s_size);
  a.tall = plan.tall;
  a.splits = plan.splits;
  a.may_split = FORM == kWeight && z.weight_splits();
  a.wide = FORM == kWeight ? kSide : (uint32_t)std::min<uint64_t>(a.tall, align_up(z.rows, 16));
  a.out = out;
  a.out_batch = out_batch;
  a.out_stride = out_stride;
  a.accumulate = accumulate;
  a.shared = FORM != kWeight && p.batches == 1;
  a.bf16 = c.type == SPARCML_BF16;
  a.part = reinterpret_cast<float*>(w + 256);
  a.status = reinterpret_cast<int32_t*>(w);
  a.inject = reinterpret_cast<const uint32_t*>(w + kInjectOffset);
  a.handed_out = reinterpret_cast<uint32_t*>(w + kItemsOffset);
  a.restore = side;
  ExpertMaps m;
  if (z.rows == 0) p = q = Operand{w, 64, 64, 1, 1, 64};  // no operand is read
  if (!map_of(&m.p, p, a.bf16, FORM == kForward ? 128 : 64) ||
      !map_of(&m.q, q, a.bf16, FORM == kWeight ? 64 : kBox))
    return SPARCML_ERR_CUDA;
  const uint64_t tiles = FORM == kWeight ? z.weight_tiles() : z.most_tiles(a.i_size, a.tall);
  const uint64_t joined = a.may_split ? kPairs : a.splits > 1 ? tiles : 0;
  const uint64_t most = a.may_split ? kPairs : tiles * a.splits;
  return launch_experts<FORM>(m, a, std::max<uint64_t>(1, most), joined * (a.wide / 4), c.stream);
}

bool half_type(int32_t type) { return type == SPARCML_BF16 || type == SPARCML_F16; }

// Whether rows of `cols` elements at these strides share no address.
bool rows_apart(uint64_t rows, uint64_t cols, int64_t stride) {
  return rows <= 1 || stride >= (int64_t)cols;
}

int check_call(const Call& c) {
  if (!c.z.ok() || !half_type(c.type) || (!c.offsets && c.z.experts != 1) ||
      !aligned_to(c.offsets, 4) || !c.ws || !aligned_to(c.ws, 256))
    return SPARCML_ERR_INVALID_ARG;
  return SPARCML_OK;
}
bool operand_ok(const Operand& o) {
  return o.rows == 0 || (o.p && aligned_to(o.p, 2) && o.stride >= 0 && o.batch >= 0);
}

bool result_ok(const void* p, uint64_t rows, uint64_t cols, int64_t stride) {
  return rows == 0 || (p && aligned_to(p, 2) && rows_apart(rows, cols, stride));
}
// dW: matrices one after the other, or their rows in turn.
bool matrices_ok(const float* p, const Sizes& z, int64_t batch, int64_t stride) {
  const int64_t n = (int64_t)z.n, k = (int64_t)z.k, e = (int64_t)z.experts;
  if (!aligned_to(p, 4) || batch < 0 || stride < 0 || (n > 1 && stride < k)) return false;
  return e == 1 || batch >= (n - 1) * stride + k ||
         (batch >= k && (n == 1 || stride >= (e - 1) * batch + k));
}

// dx and dW, each where it is wanted; x as it is, or in 8 bits.
int backward(const Call& c, Operand dy, Operand x, const Stored* stored, Operand w, void* dx,
             int64_t dx_stride, float* dweight, int64_t dw_batch, int64_t dw_stride,
             int32_t accumulate) {
  const Sizes& z = c.z;
  int r = check_call(c);
  if (r != SPARCML_OK) return r;
  if (!operand_ok(dy) || (dx && (!operand_ok(w) || !result_ok(dx, z.rows, z.k, dx_stride))) ||
      (dweight && ((!stored && !operand_ok(x)) || !matrices_ok(dweight, z, dw_batch, dw_stride))))
    return SPARCML_ERR_INVALID_ARG;
  const bool rows = z.rows > 0;
  const bool input = dx && rows, weights = dweight != nullptr;
  if (!input && !weights) return SPARCML_OK;
  const bool restored = stored && weights && rows;
  Operand plain = x;
  if (restored) plain = {nullptr, 0, (int64_t)align_up(z.k, 8), 1, z.rows, z.k};
  const Settle copies{{&dy, input ? &w : nullptr,
                       weights && !stored ? &plain : nullptr}};
  const size_t parts = z.part_bytes(), more = restored ? plain.copy_bytes() : 0;
  if (c.ws_bytes < 256 + parts + more + copies.bytes()) return SPARCML_ERR_WORKSPACE;
  uint8_t* room = static_cast<uint8_t*>(c.ws) + 256 + parts;
  Restore side = {};
  if (restored) {  // beside dx, or before dW
    plain.p = room;
    if (input)
      side = {stored->codes, stored->codes_stride, stored->exponents, stored->exponents_stride,
              room, plain.pitch(), (uint32_t)z.rows, (uint32_t)z.k};
    else
      r = sparcml_restore8(stored->codes, stored->codes_stride, stored->exponents,
                           stored->exponents_stride, z.rows, z.k, room, c.type, plain.stride,
                           c.stream);
    if (r != SPARCML_OK) return r;
  }
  copies.run(room + more, c.stream);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  if (input) {
    r = run<kInput>(c, w, dy, dx, 0, dx_stride, 0, side);
    if (r != SPARCML_OK) return r;
  }
  return weights ? run<kWeight>(c, plain, dy, dweight, dw_batch, dw_stride, accumulate)
                 : SPARCML_OK;
}

}  // namespace
}  // namespace sparcml

using namespace sparcml;

extern "C" size_t sparcml_expert_linear_workspace_size(uint64_t rows, uint32_t experts, uint64_t n,
                                                       uint64_t k, int32_t aligned) {
  const Sizes z{rows, experts, n, k};
  if (!z.ok()) return 0;
  const Operand x{nullptr, 0, 0, 1, rows, k}, dy{nullptr, 0, 0, 1, rows, n},
      w{nullptr, 0, 0, experts, n, k};
  const bool odd_n = !aligned || n % 8 != 0, odd_k = !aligned || k % 8 != 0;
  // x also where it is kept in 8 bits
  return 256 + z.part_bytes() + x.copy_bytes() + (odd_k ? w.copy_bytes() : 0) +
         (odd_n ? dy.copy_bytes() : 0);
}

extern "C" int sparcml_expert_linear(const void* x, int64_t x_stride, const void* weight,
                                     int64_t weight_batch_stride, int64_t weight_stride,
                                     int32_t type, const int32_t* offsets, uint32_t experts,
                                     uint64_t rows, uint64_t n, uint64_t k, void* y,
                                     int64_t y_stride, void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  const Call c{{rows, experts, n, k}, type, offsets, ws, ws_bytes,
               static_cast<cudaStream_t>(stream)};
  const int r = check_call(c);
  if (r != SPARCML_OK) return r;
  Operand w = Operand::matrices(weight, weight_batch_stride, weight_stride, c.z);
  Operand q{x, 0, x_stride, 1, rows, k};
  if (rows == 0) return SPARCML_OK;
  if (!operand_ok(w) || !operand_ok(q) || !result_ok(y, rows, n, y_stride))
    return SPARCML_ERR_INVALID_ARG;
  const Settle copies{{&w, &q, nullptr}};
  const size_t parts = c.z.part_bytes();
  if (ws_bytes < 256 + parts + copies.bytes()) return SPARCML_ERR_WORKSPACE;
  copies.run(static_cast<uint8_t*>(ws) + 256 + parts, c.stream);
  if (launch_status() != SPARCML_OK) return SPARCML_ERR_CUDA;
  return run<kForward>(c, w, q, y, 0, y_stride, 0);
}

extern "C" int sparcml_expert_linear_backward(
    const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, const void* weight,
    int64_t weight_batch_stride, int64_t weight_stride, int32_t type, const int32_t* offsets,
    uint32_t experts, uint64_t rows, uint64_t n, uint64_t k, void* dx, int64_t dx_stride,
    float* dweight, int64_t dweight_batch_stride, int64_t dweight_stride, int32_t accumulate,
    void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  const Call c{{rows, experts, n, k}, type, offsets, ws, ws_bytes,
               static_cast<cudaStream_t>(stream)};
  return backward(c, {dy, 0, dy_stride, 1, rows, n}, {x, 0, x_stride, 1, rows, k}, nullptr,
                  Operand::matrices(weight, weight_batch_stride, weight_stride, c.z), dx, dx_stride,
                  dweight, dweight_batch_stride, dweight_stride, accumulate);
}

extern "C" int sparcml_expert_linear_backward8(
    const void* dy, int64_t dy_stride, const int8_t* codes, int64_t codes_stride,
    const uint8_t* exponents, int64_t exponents_stride, const void* weight,
    int64_t weight_batch_stride, int64_t weight_stride, int32_t type, const int32_t* offsets,
    uint32_t experts, uint64_t rows, uint64_t n, uint64_t k, void* dx, int64_t dx_stride,
    float* dweight, int64_t dweight_batch_stride, int64_t dweight_stride, int32_t accumulate,
    void* ws, size_t ws_bytes, void* stream) {
  const ApiRange nvtx_range(__func__);
  const Call c{{rows, experts, n, k}, type, offsets, ws, ws_bytes,
               static_cast<cudaStream_t>(stream)};
  const Stored x{codes, codes_stride, exponents, exponents_stride};
  if (dweight && rows &&
      (!codes || !exponents || !aligned_to(codes, 16) || codes_stride % 16 != 0 ||
       codes_stride < (int64_t)align_up(k, 16) || exponents_stride < (int64_t)ceil_div(k, kGroup)))
    return SPARCML_ERR_INVALID_ARG;
  return backward(c, {dy, 0, dy_stride, 1, rows, n}, {}, &x,
                  Operand::matrices(weight, weight_batch_stride, weight_stride, c.z), dx, dx_stride,
                  dweight, dweight_batch_stride, dweight_stride, accumulate);
}
