// fcc_paged_tiles.cu -- attention of a step's rows over the paged cache in tiles of
// 128 rows on tcgen05 (prompts, chunks of prompts, mixed steps).
//
// A row is a token and one of the G query heads that share a key/value head, so a
// tile's rows read the same keys whatever G is, and few tokens fill it.  An item is
// a pair of tiles (256 rows of one sequence, rank and head) and its blocks of 128
// positions, from the first that any row sees to the last.  plan_kernel adds up what
// all items cost (their blocks, and three more each), and the list is cut into as many
// equal runs as there are CTAs, one to an SM: causal, windowed and ragged steps load all
// SMs alike, and a few rows over a long context are spread over all of them.  (Without
// the three, the CTAs with a causal prompt's many short items came last: 1.60 against
// 1.05 ms for 8192 rows of 64 heads, which take 0.86 to 0.88 now.)  What a cut leaves of an item are partial sums, at
// most two from a CTA, added in order by join_kernel.  Rows that tiles cannot give (Again)
// are computed behind them by launch_again's kernel, which waits for nothing: inside a
// tile, where a warp alone needs 0.8 us a position, long rows would let the other warps'
// waits run out.  The launch costs 2.3 us where no row is marked.
//
// Within an item, for tile t and block j (all f32 in TMEM):
//   S_t = Q_t K_j^T;  P_t = 2^(S_t c - ref), in 16 bits over S_t's first columns;
//   O_t += P_t V_j, A from TMEM.
// A row's reference is raised (and its O_t rescaled) only when a block's maximum
// passes it by far.  The two tiles alternate on the tensor core: one
// tile's exponentials run under the other's products.  A new item's queries are
// loaded, and its first S computed, before the old one's O has been stored.
//
// Warps: 0-3 and 4-7 softmax and output of tiles A and B (a thread owns a row and its
// 128 columns), then those that load keys and values and the one that issues the
// products.  The loaders look up every position's page for itself (any page size).
// bf16 rows go by TMA into the swizzled tile, 32 positions to a warp.  e4m3 rows pass
// through registers and become f16 there, times their powers of two relative to
// 2^A of the keys and 2^B of the values, 2^-7 of each 32 positions' largest; those enter at
// the exponent (see fcc_paged.cu): t = 2^A (S c) + B, P = 2^(t - ref), l += 2^-B sum P.
//
// What bounds it: 2048 rows of 32 heads over 32768 positions take 718 us in bf16
// (1483 TFLOP/s, 0.75 of the measured burst peak; 760 to 780 in a loop of calls, 0.70, where
// power holds the clock down), 1.7 us a block and pair.  A
// 128 x 128 x 16 product alone takes 64 clocks, 2048 for a block and pair: the tensor
// pipe is busy 63 % of the time, the schedulers issue in 45 % and the exponentials'
// unit works in 32 %.  No unit is full: the rest is the way from the last score to the
// first P V and back, of which two tiles cover one another's only in part, and shared
// memory, which the operands of S fill by themselves while they run.  e4m3 (1005 us)
// waits for its loaders, busy 0.85 of the time with conversions and addresses, and for
// the maximum that f16 needs before the exponentials.
// Shared memory (128-byte swizzle): Q_t and four slots of [128 rows][D] 16-bit
// values in atoms of 64 columns, K_0, V_0, K_1, V_1, ... in the slots; K is the
// K-major and V the MN-major B operand of the same layout.
#include "fcc_paged.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <mutex>

namespace fcc {
namespace ptx {

// 4-D tiled load global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Stores 16 consecutive 32-bit columns of each thread's TMEM lane.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// mma_f16 and mma_f16_tmem_a (fcc_ptx.cuh) with the descriptors as words: their low ones,
// and a high one that both share.
__device__ __forceinline__ void mma_f16_words(uint32_t d_tmem, uint32_t a_low, uint32_t b_low,
                                              uint32_t high, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(high), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_tmem_a_words(uint32_t d_tmem, uint32_t a_tmem,
                                                     uint32_t b_low, uint32_t high, uint32_t idesc,
                                                     uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(high), "r"(idesc), "r"(accumulate)
      : "memory");
}

}  // namespace ptx

namespace {

constexpr int kTileRows = 128;
constexpr int kPairRows = 256;
constexpr int kBlock = 128;                    // positions of a block
constexpr int kSlots = 4;
constexpr int kCols = 4;                       // blocks whose column constants are kept
constexpr uint32_t kAtom = 128 * 128;
// A row's reference is raised when a block's maximum passes it by this much (log2
// units).  bf16 has f32's exponents: P may grow far, and the raise (which rescales O_t
// in tensor memory) can wait for the next block.  A row whose sums overflow all the
// same (2^127 within one block) is not finite at the end and is computed again.  f16
// ends at 2^16: there the maximum is taken before the exponentials, and a row's largest P
// is kept between 2^8 and 2^16, as in fcc_paged.cu.
template <bool E4M3>
constexpr float kRaise = E4M3 ? 7.9f : 32.f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;                // S_t at 128 t, O_t at 256 + 128 t
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;
// Warps: 8 softmax, 4 loading (e4m3: 4 for the keys and 4 for the values), 1 issuing and
// its 3 idle neighbours.  Registers: the launch's are dealt out anew.  Little may spill
// (62 bytes of 128-column e4m3 do, 4 of the others): what shared memory leaves of the L1 is
// too small to hold it (200 bytes a thread made a 2048-row prompt three times as slow).
template <bool E4M3>
struct Roles {
  static constexpr int kLoadWarps = E4M3 ? 8 : 4;
  static constexpr int kIssuer = 8 + kLoadWarps;         // the issuing warp
  static constexpr int kThreads = (kIssuer + 4) * 32;
  static constexpr int kLaunch = E4M3 ? 96 : 128;
  static constexpr int kSoftmax = E4M3 ? 112 : 176, kLoad = E4M3 ? 96 : 80, kIssue = E4M3 ? 64 : 80;
  static_assert(kThreads * kLaunch <= 65536 && 256 * kSoftmax + 32 * kLoadWarps * kLoad + 128 * kIssue <= kThreads * kLaunch);
};
constexpr int kMaxCtas = 512;

struct Start {                                 // where a CTA's run begins (and the one before it ends)
  int b, rh, pair, j;
  __device__ __forceinline__ bool same_item(const Start& o) const { return b == o.b && rh == o.rh && pair == o.pair; }
};
struct Header {                                // of the item that a CTA begins last and does not finish
  int parts, b, rh, pair;
};

// Workspace: the plan's totals, the headers, the cost of what is before each sequence,
// two partial results for each CTA, then a bit for every row (see Again).
struct Layout {
  size_t headers, units, parts, part_bytes, again;
};
// References, sums, then [D / 4][256] float4.
template <int D>
constexpr size_t kPartBytes = kPairRows * static_cast<size_t>(D + 2) * 4;
__host__ __device__ inline Layout layout_of(int64_t d, int B, int ctas) {
  Layout l;
  l.headers = 256;
  l.units = l.headers + static_cast<size_t>(ctas) * sizeof(Header);
  l.parts = (l.units + static_cast<size_t>(B) * 8 + 255) & ~size_t{255};
  l.part_bytes = kPairRows * static_cast<size_t>(d + 2) * 4;
  l.again = l.parts + 2 * static_cast<size_t>(ctas) * l.part_bytes;
  return l;
}
struct Totals {                                // at the workspace's start
  long long cost;                              // of all items
  int ctas;                                    // with work
  int again;                                   // some row's bit is set (tests read it here, 12 bytes in)
};

__device__ __forceinline__ int pairs_of(const PagedArgs& a, const Seq& q) {
  return (q.n * a.G + (kPairRows - 1)) / kPairRows;   // (T * G stays below 2^31 - 256)
}

// What an item costs beside its blocks, in blocks: its queries' loads, the first S and
// the last P V that nothing runs beside, its output.
constexpr int kItemBlocks = 3;

// Blocks [j0, j1) that rows [first, last] of a sequence see.
struct Range {
  int j0, j1;
};
__device__ __forceinline__ Range blocks_of(const PagedArgs& a, const Seq& q, int first, int last) {
  if (!q.ok) return Range{0, 1};               // (one, of which nothing is seen)
  const int p0 = q.L - q.n + a.by_g(first), p1 = q.L - q.n + a.by_g(last);
  const int j0 = max(0, p0 - a.window + 1) / kBlock;
  return Range{j0, max(j0, min(p1, a.held - 1) / kBlock) + 1};
}
__device__ __forceinline__ Range pair_blocks(const PagedArgs& a, const Seq& q, int pair) {
  const int first = pair * kPairRows;
  return blocks_of(a, q, first, min(q.n * a.G - first, kPairRows) + first - 1);
}

constexpr int kPlanThreads = 1024;
constexpr int kFewPairs = 8;                   // up to here a thread counts a sequence's blocks alone

// Division by 32-bit means where they will do: 64-bit ones are long.
__device__ __forceinline__ long long divide(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// Adds up what all items cost, in blocks.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PagedArgs a, int grid) {
  __shared__ long long s_scan[32];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Layout lay = layout_of(a.pool.d, a.step.B, grid);
  long long* units = reinterpret_cast<long long*>(a.ws + lay.units);
  const long long rh = static_cast<long long>(a.R) * a.pool.H;
  for (int b0 = warp * 32; b0 < a.step.B; b0 += kPlanThreads) {
    const int b = b0 + lane;
    Seq q{0, 0, 0, false, false};
    int np = 0;
    long long n = 0;
    if (b < a.step.B) {
      q = load_seq(a.step, b);
      if (bad_sequence(a, q)) record_invalid(a.status);
      np = pairs_of(a, q);
      if (np <= kFewPairs)
        for (int p = 0; p < np; ++p) {
          const Range g = pair_blocks(a, q, p);
          n += g.j1 - g.j0 + kItemBlocks;
        }
    }
    for (unsigned m = __ballot_sync(0xffffffffu, np > kFewPairs); m != 0; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const Seq o = load_seq(a.step, b0 + src);
      const int onp = pairs_of(a, o);
      long long sum = 0;
      for (int p = lane; p < onp; p += 32) {
        const Range g = pair_blocks(a, o, p);
        sum += g.j1 - g.j0 + kItemBlocks;
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      if (lane == src) n = sum;
    }
    if (b < a.step.B) units[b] = n * rh;
  }
  __syncthreads();
  const int per = (a.step.B + kPlanThreads - 1) / kPlanThreads;
  const int b_first = min(a.step.B, static_cast<int>(threadIdx.x) * per), b_last = min(a.step.B, b_first + per);
  long long mine = 0;
  for (int b = b_first; b < b_last; ++b) mine += units[b];
  long long upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += v;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long total = 0, from = upto - mine;
  for (int i = 0; i < 32; ++i) {
    if (i < warp) from += s_scan[i];
    total += s_scan[i];
  }
  const long long ctas = min(static_cast<long long>(grid), total);
  const int64_t words = rh * a.again.words;
  for (int64_t i = threadIdx.x; i < words; i += kPlanThreads) a.again.rows[i] = 0;
  // (from here on units[b] is the cost of what is before sequence b)
  for (int b = b_first; b < b_last; ++b) {
    const long long n = units[b];
    units[b] = from;
    from += n;
  }
  if (threadIdx.x == 0) *reinterpret_cast<Totals*>(a.ws) = Totals{total, static_cast<int>(ctas), 0};
}

// Where the run that begins `u` blocks into the list begins; cost0: what is before its
// item.  A whole warp calls it; every lane gets the answer.
__device__ __forceinline__ Start find_start(const PagedArgs& a, const long long* units, long long total, long long u, long long& cost0) {
  const int lane = threadIdx.x & 31;
  // the last sequence whose items begin at or before u
  int b = 0;
  for (int count = a.step.B; count > 1;) {
    const int step = (count + 31) >> 5, i = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, i < count && units[b + i] <= u);
    const int k = 31 - __clz(m);
    b += k * step;
    count = min(step, count - k * step);
  }
  const Seq q = load_seq(a.step, b);
  const long long off = u - units[b];
  const long long each = divide((b + 1 < a.step.B ? units[b + 1] : total) - units[b], static_cast<long long>(a.R) * a.pool.H);
  const int rh = static_cast<int>(divide(off, each));
  long long rest = off - rh * each;
  const int np = pairs_of(a, q);
  for (int p0 = 0; p0 < np; p0 += 32) {
    const int p = p0 + lane;
    int n = 0;
    if (p < np) {
      const Range g = pair_blocks(a, q, p);
      n = g.j1 - g.j0 + kItemBlocks;
    }
    int incl = n;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += v;
    }
    const unsigned m = __ballot_sync(0xffffffffu, rest < incl);
    if (m != 0) {
      const int src = __ffs(m) - 1;
      const int within = static_cast<int>(rest) - __shfl_sync(0xffffffffu, incl - n, src);
      cost0 = u - within;
      // (an item's own cost comes before its first block: no cut falls into it)
      return Start{b, rh, p0 + src, max(0, within - kItemBlocks)};
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
  return Start{a.step.B, 0, 0, 0};             // (not reached: u lies before the list's end)
}

// This CTA's run of blocks.
struct alignas(16) Run {
  Start start, stop;
  long long cost, cost0;                       // of all items; of what is before the first one here
  int ctas;                                    // with work
  bool busy;
};

// A walk over a CTA's run: item after item, each from block ja to block jb.
struct Walk {
  int b, rh, pair, pairs;
  Seq q;
  int j0, j1;                                  // the item's blocks
  int ja, jb;                                  // the CTA's part of them
  long long cost0;                             // of what is before the item
  Start stop;                                  // where the run ends
  int lo[2], hi[2];                            // tile t's blocks of [ja, jb): none if lo >= hi
  bool more;                                   // there is such an item

  __device__ __forceinline__ bool take(const PagedArgs& a, int skip) {
    const int rows = q.n * a.G, first = pair * kPairRows;
    const Range g = pair_blocks(a, q, pair);
    j0 = g.j0;
    j1 = g.j1;
    ja = j0 + skip;
    jb = stop.same_item(Start{b, rh, pair, 0}) ? j0 + stop.j : j1;
    if (ja >= jb) return false;                // (the run ends where the item begins)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r0 = first + t * kTileRows;
      lo[t] = hi[t] = 0;
      if (r0 >= rows) continue;
      const Range s = blocks_of(a, q, r0, min(rows - r0, kTileRows) + r0 - 1);
      lo[t] = max(ja, s.j0);
      hi[t] = min(jb, s.j1);
    }
    return true;
  }
  __device__ __forceinline__ bool begin(const PagedArgs& a, const Run& r) {
    if (!r.busy) return false;                 // (its start says nothing then)
    stop = r.stop;
    cost0 = r.cost0;
    b = r.start.b;
    rh = r.start.rh;
    pair = r.start.pair;
    q = load_seq(a.step, b);
    pairs = pairs_of(a, q);
    return take(a, r.start.j);
  }
  __device__ __forceinline__ bool next_item(const PagedArgs& a) {
    if (stop.same_item(Start{b, rh, pair, 0})) return false;
    cost0 += j1 - j0 + kItemBlocks;
    if (++pair == pairs) {
      pair = 0;
      if (++rh == a.R * a.pool.H) {
        rh = 0;
        do {
          if (++b >= a.step.B) return false;
          q = load_seq(a.step, b);
        } while (q.n == 0);
        pairs = pairs_of(a, q);
      }
    }
    return take(a, 0);
  }
  // Tile t has a block here.  Where it has none, its softmax warps and the issuing
  // warp pass the item without a word: a barrier's phases stay one to an exchange.
  __device__ __forceinline__ bool active(int t) const { return lo[t] < hi[t]; }
  __device__ __forceinline__ int rank(const PagedArgs& a) const { return rh / a.pool.H; }
  __device__ __forceinline__ int head(const PagedArgs& a) const { return rh % a.pool.H; }
};

// A warp's walk, kept in shared memory (the softmax threads have no registers to
// spare): lane 0 takes the steps.  The softmax warps also keep the item before.
struct alignas(16) WarpWalk {
  Walk now, old;
  __device__ __forceinline__ void begin(const PagedArgs& a, const Run& r, int lane) {
    if (lane == 0) now.more = now.begin(a, r);
    __syncwarp();
  }
  __device__ __forceinline__ void next(const PagedArgs& a, int lane) {
    __syncwarp();                              // (every lane has read what it needs)
    if (lane == 0) {
      old = now;
      now.more = now.next_item(a);
    }
    __syncwarp();
  }
};
constexpr int kWalks = 17;

// What the softmax warps need to know of a block's columns, for each 32 of them: e4m3
// the largest powers of two of their keys and values; which positions the pages hold.
struct alignas(16) Columns {
  float ka[4], vb[4], vi[4];                   // 2^A, B and 2^-B, 2^kLift below the largest
  uint32_t there[4];
  uint32_t wide[2][4];                         // keys', values' powers too far apart for f16, see f16_power()
};

// 2^(byte - top + kLift) in f16 (both halves): codes end at 448 * 2^7 = 57344, below f16's
// largest, and a code (a multiple of 2^-9) times a power is exact down to 2^-15, with f16's
// subnormal numbers: over 22 powers.  A group with powers further apart is `wide`: the rows
// that met it are computed again (Again).  (P's 33 bits: of an output of values 2^22 below
// their neighbours', which they outweigh by more than that, a neighbour's lost part is 2^-11.
// To mark such rows by the size of their sums took 1 to 4 % of every chunk, and marked one
// in a hundred of rows with a quiet position near their query that lost nothing.)
constexpr int kLift = 7;
__device__ __forceinline__ uint32_t f16_power(int byte, int top) {
  const int k = byte - top + kLift;
  const uint32_t h = k >= -14 ? static_cast<uint32_t>(15 + k) << 10 : k == -15 ? 1u << 9 : 0u;
  return h | (h << 16);
}
constexpr int kWide = 15 + kLift;
constexpr int kZeroByte = 63;                  // append's least, and what a row of zeros has
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr int kStageRow = 80;                  // 64 bytes of output and 16 that keep lanes apart
constexpr int kBars = 2 * kSlots + kCols + 2 + 2 + 2 + 2 + 1;

template <int D>
constexpr uint32_t kTileBytes = (D / 64) * kAtom;
template <int D>
constexpr int kSmem = 1024 + (2 + kSlots) * static_cast<int>(kTileBytes<D>) + kCols * static_cast<int>(sizeof(Columns)) +
                      kWalks * static_cast<int>(sizeof(WarpWalk)) + 8 * 32 * kStageRow +
                      static_cast<int>(sizeof(Run)) + kBars * 8 + 16;
static_assert(kSmem<128> <= 232448, "shared memory per CTA");

// The low words of the operands' descriptors (address and leading offset, in 16 bytes;
// the K steps of 16 are added there) and the high word that all share: 1024 bytes
// between groups of 8 rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t desc_low(const uint8_t* tile, uint32_t lbo) {
  return static_cast<uint32_t>(ptx::smem_desc_sw128(ptx::smem_addr(tile), lbo, 1024));
}
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__host__ __device__ constexpr uint32_t step_kmajor(int kk) { return ((kk >> 2) * kAtom + (kk & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t step_mnmajor(int kk) { return (kk * 2048) >> 4; }
// The byte of 16-byte chunk `chunk` (8 values) of a tile's row.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (chunk >> 3) * kAtom + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tmem_ld_wait_regs(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

__device__ __forceinline__ float sum2(const uint64_t (&v)[2]) {
  float a, b;
  ptx::f32x2_unpack(ptx::f32x2_add(v[0], v[1]), a, b);
  return a + b;
}

// The place of column group c4 (4 values) of a row in a partial result.
__device__ __forceinline__ float4* part_at(char* part, int c4, int row) {
  return reinterpret_cast<float4*>(part + kPairRows * 8) + c4 * kPairRows + row;
}

struct PoolMaps {                              // bf16 pools with pages of 16 rows and more
  CUtensorMap K[FCC_MAX_RANKS], V[FCC_MAX_RANKS];
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(Roles<E4M3>::kThreads, 1) tiles_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ PoolMaps maps, unsigned long long timeout_ns) {
  constexpr uint32_t kTile = kTileBytes<D>;
  constexpr int kIssuer = Roles<E4M3>::kIssuer;
  constexpr uint32_t kFormat = E4M3 ? 0u : (1u << 7) | (1u << 10);   // f16 or bf16 operands
  constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);
  constexpr uint32_t kIdescS = (ptx::idesc_bf16_f32(kTileRows, kBlock, false, false) & ~kBf16) | kFormat;
  constexpr uint32_t kIdescO = (ptx::idesc_bf16_f32(kTileRows, D, false, true) & ~kBf16) | kFormat;
  constexpr float kOff = E4M3 ? 8.f : 0.f;     // p up to 2^(kOff + kRaise) in f16

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = sQ + 2 * kTile;
  Columns* cols = reinterpret_cast<Columns*>(sR + kSlots * kTile);
  WarpWalk* walks = reinterpret_cast<WarpWalk*>(cols + kCols);
  uint8_t* stages = reinterpret_cast<uint8_t*>(walks + kWalks);
  Run* run = reinterpret_cast<Run*>(stages + 8 * 32 * kStageRow);
  uint64_t* r_full = reinterpret_cast<uint64_t*>(run + 1);  // [kSlots], four loading warps
  uint64_t* r_empty = r_full + kSlots;         // [kSlots]
  uint64_t* c_full = r_empty + kSlots;         // [kCols], the loading warps
  uint64_t* q_full = c_full + kCols;           // [2]: Q_t written, the tile's four softmax warps
  uint64_t* s_full = q_full + 2;               // [2]: S_t complete
  uint64_t* p_full = s_full + 2;               // [2]: P_t written (and O_t rescaled)
  uint64_t* o_full = p_full + 2;               // [2]: an item's products of tile t complete
  uint64_t* mma_done = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&r_full[i], 4);
      ptx::mbar_init(&r_empty[i], 1);
    }
    for (int i = 0; i < kCols; ++i) ptx::mbar_init(&c_full[i], Roles<E4M3>::kLoadWarps);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&q_full[t], 4);
      ptx::mbar_init(&s_full[t], 1);
      ptx::mbar_init(&p_full[t], 4);
      ptx::mbar_init(&o_full[t], 1);
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kIssuer) {
    ptx::tmem_alloc(tmem_slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const ptx::Waiter W{abort_flag, a.status, timeout_ns};
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (warp < 2) {                              // where this run begins, and where the next one does
    const Layout lay = layout_of(D, a.step.B, gridDim.x);
    const Totals tot = *reinterpret_cast<const Totals*>(a.ws);
    const int c = static_cast<int>(blockIdx.x) + warp;
    Start s{a.step.B, 0, 0, 0};                // (behind all items)
    long long cost0 = 0;
    if (c < tot.ctas)
      s = find_start(a, reinterpret_cast<const long long*>(a.ws + lay.units), tot.cost, divide(c * tot.cost, tot.ctas), cost0);
    if (lane == 0) {
      (warp == 0 ? run->start : run->stop) = s;
      if (warp == 0) {
        run->cost = tot.cost;
        run->cost0 = cost0;
        run->ctas = tot.ctas;
        run->busy = c < tot.ctas;
        reinterpret_cast<Header*>(a.ws + lay.headers)[blockIdx.x] = Header{0, 0, 0, 0};
      }
    }
  }
  __syncthreads();

  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, W.wait(bar, parity) ? 1 : 0) != 0;
  };

  if (warp >= kIssuer) {
    // ----------------------------------------------------------- MMA issue
    regs_dec<Roles<E4M3>::kIssue>();
    if (warp == kIssuer) {
      // The whole warp walks and waits, and one lane issues: what a product takes stays
      // in registers that the warp shares.  What the loop over blocks needs is in
      // registers too: this warp's own instructions stand between one product and the next.
      WarpWalk& ww = walks[kIssuer];
      const bool lead = elect_one();
      bool any = false, ok = true;
      ww.begin(a, *run, lane);
      uint32_t q_phase = 0, p_phase = 0;       // bit t: the parity that Q_t / P_t will complete
      uint32_t u = 0;                          // ring position of the block's K, V is at u + 1
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
      const uint32_t qd0 = __shfl_sync(0xffffffffu, desc_low(sQ, 16), 0), kd0 = __shfl_sync(0xffffffffu, desc_low(sR, 16), 0),
                     vd0 = __shfl_sync(0xffffffffu, desc_low(sR, kAtom), 0);
      // O_t += P_t V, the V at ring position `pos`.
      auto issue_pv = [&](int t, uint32_t pos, bool first) -> bool {
        const uint32_t vd = vd0 + (pos % kSlots) * (kTile >> 4);
        const uint32_t pa = tmem + t * 128, o = tmem + kColO + t * 128;
        // (P as a whole: its halves as they come, on a barrier each, were 4 to 13 % slower)
        if (!wait_warp(&p_full[t], p_phase >> t & 1u)) return false;
        ptx::tc_fence_after();
        if (lead) {
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            ptx::mma_f16_tmem_a_words(o, pa + kk * 8, vd + step_mnmajor(kk), kDescHigh, kIdescO, (!first || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
        p_phase ^= 1u << t;
        return true;
      };
      auto issue_s = [&](int t) {
        const uint32_t qd = qd0 + t * (kTile >> 4), kd = kd0 + (u % kSlots) * (kTile >> 4);
        if (lead) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_f16_words(tmem + t * 128, qd + step_kmajor(kk), kd + step_kmajor(kk), kDescHigh, kIdescS, kk > 0 ? 1u : 0u);
          ptx::mma_commit(&s_full[t]);
        }
        __syncwarp();
      };
      while (ok && __shfl_sync(0xffffffffu, ww.now.more ? 1 : 0, 0) != 0) {
        auto same = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const int ja = same(ww.now.ja), jb = same(ww.now.jb), lo0 = same(ww.now.lo[0]), hi0 = same(ww.now.hi[0]),
                  lo1 = same(ww.now.lo[1]), hi1 = same(ww.now.hi[1]);
        any = true;
        if (lo0 < hi0) ok = wait_warp(&q_full[0], q_phase & 1u), q_phase ^= 1u;
        if (ok && lo1 < hi1) ok = wait_warp(&q_full[1], q_phase >> 1 & 1u), q_phase ^= 2u;
        // one step more than there are blocks: the last one's P V
        for (int j = ja; j <= jb && ok; ++j, u += 2) {
          if (j < jb && !(ok = wait_warp(&r_full[u % kSlots], u / kSlots & 1u))) break;
          if (j > ja && !(ok = wait_warp(&r_full[(u - 1) % kSlots], (u - 1) / kSlots & 1u))) break;
          ptx::tc_fence_after();
          if (j > lo0 && j <= hi0 && !(ok = issue_pv(0, u - 1, j == lo0 + 1))) break;
          if (j >= lo0 && j < hi0) issue_s(0);
          if (j > lo1 && j <= hi1 && !(ok = issue_pv(1, u - 1, j == lo1 + 1))) break;
          if (j >= lo1 && j < hi1) issue_s(1);
          // K_j is free once both tiles' S are done, V_{j-1} once both P V are
          if (lead) {
            if (j < jb) ptx::mma_commit(&r_empty[u % kSlots]);
            if (j > ja) ptx::mma_commit(&r_empty[(u - 1) % kSlots]);
          }
          __syncwarp();
        }
        if (!ok) break;
        u -= 2;                                // (the step more had no block)
        if (lead) {
          if (lo0 < hi0) ptx::mma_commit(&o_full[0]);
          if (lo1 < hi1) ptx::mma_commit(&o_full[1]);
        }
        ww.next(a, lane);
      }
      if (any && lead) {
        ptx::mma_commit(mma_done);
        W.drain(mma_done, 0, kDrainNs);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------- loading
    // Warp 8 + i brings positions 32 i .. 32 i + 31 of each block (e4m3: their keys,
    // warp 12 + i their values).  A lane looks up one of them, a block ahead.
    regs_dec<Roles<E4M3>::kLoad>();
    const int wl = (warp - 8) & 3, kind = (warp - 8) >> 2;   // kind 1: e4m3 values
    constexpr int kRow = D * (E4M3 ? 1 : 2), kLanes = kRow / 16, kAtOnce = 32 / kLanes, kN = 32 / kAtOnce;
    if (run->busy) {
      WarpWalk& ww = walks[warp];
      Walk& w = ww.now;
      ww.begin(a, *run, lane);
      int j = w.ja;                            // the block that is looked up next
      int page = -1, in_page = 0, r = 0, h = 0;  // this lane's position in the block looked up last
      bool have = false, needed = false, left = w.more;
      // The item: its rank, head, end, table and positions.  Those in (see_from, see_to]
      // are seen by some row of it: others need no page.
      int item_r = 0, item_h = 0, item_end = 0, see_from = 0, see_to = 0;
      uint32_t positions = 0;
      const int* table = nullptr;
      auto new_item = [&]() {
        j = w.ja;
        item_r = w.rank(a);
        item_h = w.head(a);
        item_end = w.jb;
        positions = w.q.ok ? w.q.L : 0;
        table = a.step.table + w.b * a.step.max_pages;
        const int row0 = w.pair * kPairRows, first = w.q.L - w.q.n;
        see_from = max(-1, first + a.by_g(row0) - a.window);
        see_to = first + a.by_g(min(w.q.n * a.G - row0, kPairRows) + row0 - 1);
      };
      // Asks for the page of the next block's position; answer() takes what has come.
      auto ask = [&]() {
        page = -1;
        needed = false;
        have = left;
        if (!have) return;
        const uint32_t pos = static_cast<uint32_t>(j) * kBlock + 32 * wl + lane;
        r = item_r;
        h = item_h;
        if (pos < positions) {
          const uint32_t idx = pos >> a.pool.log2P;
          if (idx < static_cast<uint32_t>(a.step.max_pages)) page = __ldg(table + idx);
          in_page = static_cast<int>(pos) & ((1 << a.pool.log2P) - 1);
          needed = static_cast<int>(pos) <= see_to && static_cast<int>(pos) > see_from;
        }
        if (++j == item_end) {
          ww.next(a, lane);
          left = w.more;
          if (left) new_item();
        }
      };
      auto answer = [&]() {
        if (page >= 0 && page < a.pool.pages) return;
        page = -1;
        if (needed) record_invalid(a.status);
      };
      auto look_up = [&]() {
        ask();
        answer();
      };
      if (left) new_item();
      // Number of this lane's position's row in its rank's pools, -1 for none.
      auto row_of = [&]() -> int64_t {
        return page < 0 ? -1 : ((static_cast<int64_t>(page) * a.pool.H + h) << a.pool.log2P) + in_page;
      };
      uint32_t u = 0, blk = 0;
      bool ok = true;
      auto wait_slot = [&]() -> bool { return wait_warp(&r_empty[u % kSlots], ((u / kSlots) & 1u) ^ 1u); };
      // What the softmax warps are told of the block (called once the block's slot is
      // free: the products of the block that had these constants four blocks ago were
      // issued before the slot was handed back).  e4m3: returns this position's factor.
      // least: the least byte of the warp's rows that are not zero (any power leaves those what they are).
      auto constants = [&](int64_t row, int byte, int least) -> uint32_t {
        Columns& cc = cols[blk % kCols];
        uint32_t factor = 0;
        if constexpr (E4M3) {
          byte = min(byte, 254);
          // (a group without positions: a power that leaves its factor of the masked scores above zero)
          const int most = __reduce_max_sync(0xffffffffu, row >= 0 ? byte : 0), top = most > 0 ? max(most, kLift + 1) : 127;
          const bool wide = least < top - kWide;
          factor = row >= 0 ? f16_power(byte, top) : 0u;   // (where there is no position, byte is an earlier block's)
          if (lane == 0) {
            const int scale = top - kLift;
            cc.wide[kind][wl] = wide;
            if (kind == 0) {
              cc.ka[wl] = __int_as_float(scale << 23);
            } else {
              cc.vb[wl] = static_cast<float>(scale - 127);
              cc.vi[wl] = __int_as_float((254 - scale) << 23);
            }
          }
        }
        const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0) {
          if (kind == 0) cc.there[wl] = there;
          ptx::mbar_arrive(&c_full[blk % kCols]);
        }
        ++blk;
        return factor;
      };
      if constexpr (E4M3) {
        // Eight lanes hold four 16-byte pieces of one 64-column atom of two rows next to
        // each other: their f16 stores fall into different banks.
        constexpr int kAtoms = D / 64;
        const int piece = (lane >> 3) % kAtoms * 4 + (lane & 3);
        const int sub = (lane >> 3) / kAtoms * 2 + (lane >> 2 & 1);  // row of the kAtOnce
        uint4 x[kN];
        int byte = 1;
        u = kind;
        auto fetch = [&](int64_t row, int r) {
          const char* pool = (kind == 0 ? a.pool.K[r] : a.pool.V[r]) + piece * 16;
          if (a.pool.log2P >= 5 && __all_sync(0xffffffffu, row >= 0)) {   // one piece of a page
            pool += (__shfl_sync(0xffffffffu, row, 0) + sub) * kRow;
#pragma unroll
            for (int i = 0; i < kN; ++i) x[i] = *reinterpret_cast<const uint4*>(pool + i * kAtOnce * kRow);
          } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const int64_t src = __shfl_sync(0xffffffffu, row, i * kAtOnce + sub);
              x[i] = make_uint4(0, 0, 0, 0);
              if (src >= 0) x[i] = *reinterpret_cast<const uint4*>(pool + src * kRow);
            }
          }
          if (row >= 0) byte = (kind == 0 ? a.pool.Ke[r] : a.pool.Ve[r])[row];
        };
        // Which of the 32 rows are not zero, by rows i * kAtOnce + sub of the lanes that hold them.
        auto not_zero = [&]() -> uint32_t {
          uint32_t rows = 0;
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const uint32_t m = __ballot_sync(0xffffffffu, ((x[i].x | x[i].y | x[i].z | x[i].w) & 0x7f7f7f7fu) != 0);
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n)
              rows |= (m >> (kAtoms * 8 * (n >> 1) + 4 * (n & 1)) & (kAtoms == 2 ? 0xf0fu : 0xfu)) != 0 ? 1u << (i * kAtOnce + n) : 0u;
          }
          return rows;
        };
        // (Pages taken as soon as they were asked for, an address for each load and the
        // item's fields from shared memory each time: 1034 instead of 1005 us for the chunk.)
        // A block's pages are asked for two blocks ahead; what has come a block later is
        // brought into the L2, before that block's own loads: they would wait for DRAM
        // between one block's conversion and the next.
        look_up();
        int64_t row = row_of();
        bool full = have;
        if (full) fetch(row, r);
        ask();
        while (full) {
          const bool next = have;
          answer();
          const int64_t next_row = row_of();
          const int next_r = r;
          if (next_row >= 0) {
            ptx::prefetch_l2((kind == 0 ? a.pool.K[r] : a.pool.V[r]) + next_row * kRow);
            ptx::prefetch_l2((kind == 0 ? a.pool.Ke[r] : a.pool.Ve[r]) + next_row);
          }
          ask();
          if (!(ok = wait_slot())) break;
          int least = __reduce_min_sync(0xffffffffu, row >= 0 ? byte : 255);
          if (least == kZeroByte) {
            const uint32_t rows = not_zero();
            least = __reduce_min_sync(0xffffffffu, row >= 0 && (rows >> lane & 1) != 0 ? byte : 255);
          }
          const uint32_t power = constants(row, byte, least);
          uint8_t* dst = sR + (u % kSlots) * kTile;
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int tok = i * kAtOnce + sub;
            const uint32_t f = __shfl_sync(0xffffffffu, power, tok);
            uint32_t y[8];
            f16x4_of_e4m3(x[i].x, y[0], y[1]);
            f16x4_of_e4m3(x[i].y, y[2], y[3]);
            f16x4_of_e4m3(x[i].z, y[4], y[5]);
            f16x4_of_e4m3(x[i].w, y[6], y[7]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = mul_f16x2(y[e], f);
            *reinterpret_cast<uint4*>(dst + tile_at(32 * wl + tok, 2 * piece)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + tile_at(32 * wl + tok, 2 * piece + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&r_full[u % kSlots]);
          u += 2;
          full = next;
          row = next_row;
          if (full) fetch(row, next_r);
        }
      } else {
        // A warp's 32 positions come by TMA, a box of a page's rows and 64 columns at a
        // time, if they are all there (kBoxes: pages of 16 rows and more); otherwise,
        // at a sequence's end, through registers, with zeros for what is not.
        const int box = min(32, 1 << a.pool.log2P);
        look_up();
        while (have) {
          const int64_t row = row_of();
          const int page_now = page, in_page_now = in_page, rr = r, hh = h;
          const bool boxes = a.boxes && __all_sync(0xffffffffu, page >= 0);
          look_up();
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++u) {
            if (!(ok = wait_slot())) break;
            if (kv == 0) constants(row, 0, 0);
            uint8_t* dst = sR + (u % kSlots) * kTile;
            uint64_t* bar = &r_full[u % kSlots];
            if (boxes) {
              if (lane == 0) ptx::mbar_arrive_expect_tx(bar, 32 * D * 2);
              __syncwarp();                    // the bytes are expected before any arrive
              if ((lane & (box - 1)) == 0) {
                const CUtensorMap* map = kv == 0 ? &maps.K[rr] : &maps.V[rr];
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                  ptx::tma_load_4d(dst + x * kAtom + (32 * wl + lane) * 128, map, bar, 64 * x, in_page_now, hh, page_now);
              }
            } else {
              const char* pool = kv == 0 ? a.pool.K[rr] : a.pool.V[rr];
              const int chunk = lane % kLanes;
#pragma unroll 4
              for (int i = 0; i < kN; ++i) {
                const int tok = i * kAtOnce + lane / kLanes;
                const int64_t src = __shfl_sync(0xffffffffu, row, tok);
                uint4 x = make_uint4(0, 0, 0, 0);
                if (src >= 0) x = *reinterpret_cast<const uint4*>(pool + src * kRow + chunk * 16);
                *reinterpret_cast<uint4*>(dst + tile_at(32 * wl + tok, chunk)) = x;
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar);
            }
          }
          if (!ok) break;
        }
        if (a.boxes)                           // copies in flight land before the block ends
          for (uint32_t v = u >= kSlots ? u - kSlots : 0; v < u; ++v)
            W.drain(&r_full[v % kSlots], (v / kSlots) & 1u, kDrainNs);
      }
    }
  } else {
    // ------------------------------------------------- softmax and output
    regs_inc<Roles<E4M3>::kSoftmax>();
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;       // of the tile
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_addr = lane_addr + t * 128;
    const uint32_t o_addr = lane_addr + kColO + t * 128;
    uint32_t ns = 0, items = 0, blk0 = 0;      // this tile's blocks and items, the CTA's blocks before this item
    bool ok = true;
    WarpWalk& ww = walks[warp];
    Walk& w = ww.now;
    ww.begin(a, *run, lane);
    float c = 0.f;                             // what a score is multiplied by
    // This thread's row of a new item's Q_t; its place among the token rows.
    int64_t token = 0;
    int head = 0, qpos = -1;
    bool live = false;
    auto load_q = [&]() {
      const int rho = w.pair * kPairRows + t * kTileRows + row;
      live = rho < w.q.n * a.G;
      const int i = a.by_g(rho);
      token = static_cast<int64_t>(w.q.s) + i;
      head = w.head(a) * a.G + (rho - i * a.G);
      qpos = live && w.q.ok ? w.q.L - w.q.n + i : -1;
      if (!w.active(t)) return;
      // A row's 16-byte pieces lie on kQ neighbouring lanes, for whole lines of memory.
      constexpr int kQ = D / 8, kRows = 32 / kQ;
      const char* mine = live ? a.Q[w.rank(a)] + (token * a.ldq + static_cast<int64_t>(head) * D) * 2 : nullptr;
      uint8_t* dst = sQ + t * kTile;
      c = a.scale_log2;
      uint4 in[kQ];                            // (all loads in flight)
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int from = i * kRows + lane / kQ;
        const char* src = reinterpret_cast<const char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), from));
        in[i] = make_uint4(0, 0, 0, 0);
        if (src != nullptr) in[i] = *reinterpret_cast<const uint4*>(src + (lane % kQ) * 16);
      }
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int from = i * kRows + lane / kQ;
        uint4 v = in[i];
        if constexpr (E4M3) {
          unsigned top = 0;
          for (uint32_t y : {v.x, v.y, v.z, v.w}) {
            const unsigned m0 = y & 0x7fffu, m1 = (y >> 16) & 0x7fffu;
            top = max(top, max(m0 < 0x7f80u ? m0 : 0u, m1 < 0x7f80u ? m1 : 0u));
          }
#pragma unroll
          for (int k = 1; k < kQ; k *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
          // (a row of zeros keeps 2^0: the least power, times a group's 2^A, may round to 0, and a masked
          // score of -inf times that is NaN)
          const int e = top == 0 ? 0 : max(static_cast<int>(top >> 7) - 127, -100) - 14;
          const float f = power_of_two(-e);
          auto f16 = [&](uint32_t y) { return pack_f16x2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f); };
          v = make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w));
          const int own = __shfl_sync(0xffffffffu, e, lane % kRows * kQ);   // of row i kRows + lane % kRows
          if (lane / kRows == i) c = a.scale_log2 * power_of_two(own);
        }
        *reinterpret_cast<uint4*>(dst + tile_at(32 * quarter + from, lane % kQ)) = v;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&q_full[t]);
    };
    bool more = w.more;
    if (more) load_q();
    while (more) {
      float ref = -INFINITY, l = 0.f;
      uint32_t wide = 0;
      float late = -INFINITY;                  // the last block's largest t - ref
      int n = 0;
      const int j_end = w.hi[t];
      uint32_t blk = blk0 + (w.lo[t] - w.ja);
      for (int j = w.lo[t]; j < j_end; ++j, ++blk) {
        if (!wait_warp(&s_full[t], ns & 1u) || !wait_warp(&c_full[blk % kCols], (blk / kCols) & 1u)) {
          ok = false;
          break;
        }
        ++ns;
        ptx::tc_fence_after();
        const Columns& cc = cols[blk % kCols];
        // which of the block's positions the row sees
        const int base = j * kBlock;
        const long long first = static_cast<long long>(qpos) - a.window + 1 - base;
        const int cmax = qpos - base, cmin = first > 0 ? static_cast<int>(min(first, 128ll)) : 0;
        const uint4 there = *reinterpret_cast<const uint4*>(cc.there);
        const bool whole = cmin <= 0 && cmax >= kBlock - 1 && (there.x & there.y & there.z & there.w) == 0xffffffffu;
        auto seen = [&](int k) -> uint32_t {   // columns 32 k .. 32 k + 31
          const int hi = cmax - 32 * k, lo = cmin - 32 * k;
          uint32_t m = k == 0 ? there.x : k == 1 ? there.y : k == 2 ? there.z : there.w;
          m &= hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1;
          return m & (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1));
        };
        const bool mask = !__all_sync(0xffffffffu, whole || !live);
        bool raise;                            // the row asks for a new reference
        float to;
        if (!E4M3 && !mask && __all_sync(0xffffffffu, ref != -INFINITY || !live)) {
          // bf16, and every row of the warp has a reference: the exponentials follow the
          // scores as they come, and a block's maximum counts for the next one.
          raise = late > kRaise<E4M3>;
          to = ref + late;
        } else {
          float top = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t x[32];
            ptx::tmem_ld_32x32b_x32(s_addr + 32 * k, x);
            tmem_ld_wait_regs(x);
            if (mask) {                        // what the row does not see, here and for the exponentials
              const uint32_t m = seen(k);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(m >> i & 1)) x[i] = 0xff800000u;
              ptx::tmem_st_32x32b_x32(s_addr + 32 * k, x);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx[i / 2 & 3] = ptx::max3(mx[i / 2 & 3], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            const float m32 = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
            top = fmaxf(top, E4M3 ? fmaf(m32, c * cc.ka[k], cc.vb[k]) : m32 * c);
          }
          if (mask) ptx::tmem_st_wait();
          raise = top > ref + (kOff + kRaise<E4M3>);
          to = top - kOff;
        }
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2_from(ref, to) : 1.f;
          if (raise) ref = to;
          l *= f;
          // S_t was issued after the last P_t V: O_t has no product in flight
#pragma unroll 1
          for (int k = 0; k < D && n > 0; k += 16) {
            uint32_t o[16];
            ptx::tmem_ld_32x32b_x16(o_addr + k, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            ptx::tmem_st_32x32b_x16(o_addr + k, o);
          }
        }
        late = -INFINITY;
        // (a row that has seen nothing yet: 2^(-inf - 0) = 0)
        const float sub = ref == -INFINITY ? 0.f : ref;
        // l takes P as it is in f32, the product with V takes it in 16 bits: off by 2^-8 of it
        // at most in bf16, by 2^-11 in f16.  In bf16, where a row's largest P is any number up to 2^32, its
        // rounding shows: an output is off by 0.0023 of itself where its own rounding is
        // 0.0017.  With the rounded P in l that was 0.0017 too, but the chunk took 743 instead of
        // 719 us, and lse was off by 0.004 instead of 5e-6.
        auto exponentials = [&](uint32_t (&x)[32], int k) {
          const float ck = E4M3 ? c * cc.ka[k] : c, rk = E4M3 ? cc.vb[k] - sub : -sub;
          const uint64_t c2 = ptx::f32x2_pack(ck, ck), r2 = ptx::f32x2_pack(rk, rk);
          uint64_t l2[2] = {0, 0};
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float y0, y1;
            ptx::f32x2_unpack(ptx::f32x2_fma(ptx::f32x2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, r2), y0, y1);
            if constexpr (!E4M3) late = ptx::max3(late, y0, y1);
            const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
            l2[i / 2 & 1] = ptx::f32x2_add(l2[i / 2 & 1], ptx::f32x2_pack(p0, p1));
            pk[i / 2] = pack16<E4M3>(p0, p1);
          }
          const float l32 = sum2(l2);
          l = E4M3 ? fmaf(l32, cc.vi[k], l) : l + l32;
          // (P's columns 16 k .. 16 k + 15 lie over scores already read)
          ptx::tmem_st_32x32b_x16(s_addr + 16 * k, pk);
        };
        // (Rolled: the warps of five roles share the instruction caches, and what they do
        // not hold costs more than a load's latency.  Two chunks a step, one under the
        // other's load, took 832 instead of 800 us for 2048 rows over 32768 positions.)
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t x[32];
          ptx::tmem_ld_32x32b_x32(s_addr + 32 * k, x);
          tmem_ld_wait_regs(x);
          exponentials(x, k);
        }
        // (before P is handed over: nothing that this tile does later holds back the block
        // that has these constants next)
        if constexpr (E4M3) {
          const uint4 wk = *reinterpret_cast<const uint4*>(cc.wide[0]), wv = *reinterpret_cast<const uint4*>(cc.wide[1]);
          wide |= wk.x | wk.y | wk.z | wk.w | wv.x | wv.y | wv.z | wv.w;
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_full[t]);
        ++n;
      }
      if (!ok) break;
      // The next item's queries: this tile's S are all complete.
      const Walk& cur = ww.old;
      const int64_t o_token = token;
      const int o_head = head;
      const bool o_live = live;
      ww.next(a, lane);
      more = w.more;
      if (more) load_q();
      blk0 += cur.jb - cur.ja;
      if (n > 0) {
        if (!wait_warp(&o_full[t], items & 1u)) {
          ok = false;
          break;
        }
        ++items;
        ptx::tc_fence_after();
      }
      const int r = cur.rank(a);
      const bool complete = cur.ja == cur.j0 && cur.jb == cur.j1;
      char* part = a.ws + layout_of(D, a.step.B, gridDim.x).parts + static_cast<size_t>(2 * blockIdx.x + (cur.ja == cur.j0 ? 1 : 0)) * kPartBytes<D>;
      const int prow = t * kTileRows + row;
      const bool none = l == 0.f;
      const float inv = complete ? 1.f / l : 1.f;
      const char* const dst = o_live ? a.O[r] + (o_token * a.ldo + static_cast<int64_t>(o_head) * D) * 2 : nullptr;
      bool odd = !(fabsf(l) < INFINITY) || wide != 0;
      uint8_t* const stage = stages + warp * (32 * kStageRow);
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32x32b_x32(o_addr + k, v);
        tmem_ld_wait_regs(v);
        uint32_t top = 0;                      // the largest magnitude, as bits
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          top = max(top, v[i] & 0x7fffffffu);
          v[i] = __float_as_uint(__uint_as_float(v[i]) * inv);
        }
        odd |= n > 0 && top >= 0x7f800000u;
        if (n == 0 || none) {                  // (O_t holds nothing of this row)
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (complete) {
          // 32 columns of the warp's rows pass through shared memory: four lanes store
          // 64 bytes of a row
          uint8_t* const st = stage + lane * kStageRow;
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 y;
            y.x = ptx::pack_bf16x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            y.y = ptx::pack_bf16x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            y.z = ptx::pack_bf16x2(__uint_as_float(v[i + 4]), __uint_as_float(v[i + 5]));
            y.w = ptx::pack_bf16x2(__uint_as_float(v[i + 6]), __uint_as_float(v[i + 7]));
            *reinterpret_cast<uint4*>(st + i * 2) = y;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int from = 8 * i + lane / 4;
            char* to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), from));
            const uint4 y = *reinterpret_cast<const uint4*>(stage + from * kStageRow + (lane & 3) * 16);
            if (to != nullptr) *reinterpret_cast<uint4*>(to + k * 2 + (lane & 3) * 16) = y;
          }
          __syncwarp();
        } else if (o_live) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *part_at(part, (k + i) / 4, prow) = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                            __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
        }
      }
      // Rows that this form cannot give are left to launch_again's kernel: nothing that
      // could take long stands between two barriers here.
      const unsigned m = __ballot_sync(0xffffffffu, odd && o_live);
      if (m != 0 && lane == 0) {
        a.again.mark(cur.rh, cur.q.s * a.G + cur.pair * kPairRows + t * kTileRows + quarter * 32, m);
        *a.again.any = 1;
      }
      if (complete) {
        if (o_live && a.lse[r] != nullptr)
          a.lse[r][o_token * a.Hq + o_head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
      } else {
        float* st = reinterpret_cast<float*>(part);
        if (o_live) {
          st[prow] = ref;
          st[kPairRows + prow] = l;
        }
        if (cur.ja == cur.j0 && threadIdx.x == 0) {
          // the CTA that has the item's last block
          const long long last = divide((cur.cost0 + (cur.j1 - cur.j0) + kItemBlocks) * run->ctas - 1, run->cost);
          reinterpret_cast<Header*>(a.ws + layout_of(D, a.step.B, gridDim.x).headers)[blockIdx.x] =
              Header{static_cast<int>(last) - static_cast<int>(blockIdx.x) + 1, cur.b, cur.rh, cur.pair};
        }
      }
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
}

// Adds the parts of the item that CTA blockIdx.x of tiles_kernel began last and did
// not finish, in the CTAs' order; a thread has 16 columns of a row.
template <int D>
__global__ void __launch_bounds__(kPairRows) join_kernel(const __grid_constant__ PagedArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const Layout lay = layout_of(D, a.step.B, gridDim.x);
  const Header hd = reinterpret_cast<const Header*>(a.ws + lay.headers)[blockIdx.x];
  if (hd.parts == 0) return;
  const Seq q = load_seq(a.step, hd.b);
  const int row = threadIdx.x;
  const int rho = hd.pair * kPairRows + row;
  if (rho >= q.n * a.G) return;
  auto part = [&](int i) {
    return a.ws + lay.parts + static_cast<size_t>(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * lay.part_bytes;
  };
  float ref = -INFINITY, l = 0.f, o[16] = {};
  for (int v = 0; v < hd.parts; ++v) ref = fmaxf(ref, reinterpret_cast<const float*>(part(v))[row]);
  for (int v = 0; v < hd.parts; ++v) {
    const float* st = reinterpret_cast<const float*>(part(v));
    const float f = ex2_from(st[row], ref);
    l = fmaf(st[kPairRows + row], f, l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = *part_at(part(v), 4 * blockIdx.y + i, row);
      o[4 * i] = fmaf(x.x, f, o[4 * i]);
      o[4 * i + 1] = fmaf(x.y, f, o[4 * i + 1]);
      o[4 * i + 2] = fmaf(x.z, f, o[4 * i + 2]);
      o[4 * i + 3] = fmaf(x.w, f, o[4 * i + 3]);
    }
  }
  const int r = hd.rh / a.pool.H, head = hd.rh % a.pool.H * a.G + rho % a.G;
  const int64_t token = q.s + rho / a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = l == 0.f ? 0u : ptx::pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(a.O[r] + (token * a.ldo + static_cast<int64_t>(head) * D + 16 * blockIdx.y) * 2);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (blockIdx.y == 0 && a.lse[r] != nullptr) a.lse[r][token * a.Hq + head] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// 4-D bf16 tensor map of a pool [pages, H, P, d], box [1, 1, box_rows, 64], 128-byte
// swizzle.  An encoding is a pure function of what it is given: calls on the same pools
// reuse it (direct-mapped).
bool pool_map(CUtensorMap* m, const void* ptr, int64_t pages, int H, int P, int d, uint32_t box_rows) {
  struct Entry {
    const void* ptr = nullptr;
    int64_t pages = 0;
    int H = 0, P = 0, d = 0;
    uint32_t box_rows = 0;
    CUtensorMap map{};
  };
  constexpr size_t kEntries = 256;
  static Entry entries[kEntries];
  static EncodeTiledFn encode = nullptr;
  static std::mutex mu;
  uint64_t hash = reinterpret_cast<uintptr_t>(ptr) * 0x9E3779B97F4A7C15ull;
  hash ^= static_cast<uint64_t>(pages) * 0xC2B2AE3D27D4EB4Full;
  std::lock_guard<std::mutex> lk(mu);
  Entry& e = entries[(hash >> 32) % kEntries];
  if (e.ptr == ptr && e.pages == pages && e.H == H && e.P == P && e.d == d && e.box_rows == box_rows) {
    *m = e.map;
    return true;
  }
  if (encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return false;
    encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(P), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {row, row * P, row * P * H};
  const cuuint32_t box[4] = {64, box_rows, 1, 1}, steps[4] = {1, 1, 1, 1};
  if (encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, steps,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  e.ptr = ptr;
  e.pages = pages;
  e.H = H;
  e.P = P;
  e.d = d;
  e.box_rows = box_rows;
  e.map = *m;
  return true;
}

template <int D, bool E4M3>
cudaError_t launch(PagedArgs a, int ctas, unsigned long long timeout_ns, cudaStream_t st) {
  PoolMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const int P = 1 << a.pool.log2P;
  a.boxes = !E4M3 && P >= 16 ? 1 : 0;
  for (int r = 0; r < a.R && a.boxes; ++r)
    if (!pool_map(&maps.K[r], a.pool.K[r], a.pool.pages, a.pool.H, P, D, std::min(P, 32)) ||
        !pool_map(&maps.V[r], a.pool.V[r], a.pool.pages, a.pool.H, P, D, std::min(P, 32)))
      return cudaErrorUnknown;
  static bool attr_set[64] = {};
  cudaError_t e = smem_attr_once(attr_set, tiles_kernel<D, E4M3>, kSmem<D>);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1u, a, ctas)) != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(ctas);
  if ((e = launch_pdl(tiles_kernel<D, E4M3>, dim3(grid), dim3(Roles<E4M3>::kThreads), kSmem<D>, st, 1u, a, maps, timeout_ns)) != cudaSuccess) return e;
  return launch_pdl(join_kernel<D>, dim3(grid, D / 16), dim3(kPairRows), 0, st, 1u, a);
}

}  // namespace

size_t tiles_ws_bytes(int64_t d, int B, int ctas, int64_t rows, int64_t rank_heads) {
  return layout_of(d, B, std::min(ctas, kMaxCtas)).again + static_cast<size_t>(rank_heads) * Again::words_of(rows) * 4;
}

cudaError_t launch_tiles(PagedArgs& a, bool e4m3, int ctas, unsigned long long timeout_ns, cudaStream_t st) {
  ctas = std::min(ctas, kMaxCtas);
  a.again.rows = reinterpret_cast<uint32_t*>(a.ws + layout_of(a.pool.d, a.step.B, ctas).again);
  a.again.any = &reinterpret_cast<Totals*>(a.ws)->again;
  a.again.words = Again::words_of(static_cast<int64_t>(a.step.T) * a.G);
  return a.pool.d == 128 ? (e4m3 ? launch<128, true>(a, ctas, timeout_ns, st) : launch<128, false>(a, ctas, timeout_ns, st))
                         : (e4m3 ? launch<64, true>(a, ctas, timeout_ns, st) : launch<64, false>(a, ctas, timeout_ns, st));
}

}  // namespace fcc
