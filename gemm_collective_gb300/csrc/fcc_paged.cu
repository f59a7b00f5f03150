// fcc_paged.cu -- attention of a step's rows over the paged key/value cache: the
// entry point, and the kernel for few rows to a sequence and head (decoding).
//
// With few rows every byte of the cache is used once or twice, so DRAM bounds the
// kernel: it is built to keep loads in flight and every SM busy.
//
//  * The work is the list of all (sequence, rank, head, tile of 8 NQ rows) items, each
//    a run of units of kWarps kTok positions.  The list is cut into as many equal runs
//    of units as there are CTAs (two to an SM), wherever the cuts fall: sequences of
//    all lengths, or a single long one, load all SMs alike.  An item that a cut goes
//    through leaves partial sums (O, its reference exponent and l) in the
//    workspace, at most two from a CTA, and combine_kernel adds an item's in order.
//  * A unit is kWarps slices of kTok positions, one for each warp.  A warp has a ring of
//    kStages slices of its own in shared memory, filled by its own cp.async, and
//    runs through the positions without ever waiting for another warp; the
//    loads run ahead over the ends of items, and one CTA's sums are added up while
//    the SM's other one still loads.  Any page size works: a position's place is
//    looked up for itself, one slice before its loads.
//  * S^T = K Q^T and O^T += V^T P^T on m16n8k16 products of the warp: positions (and
//    columns of V) fill the 16 rows, the tile's rows come 8 at a time as n, so 8 heads
//    of one token leave nothing empty.  At 23 bytes a clock and SM these products run
//    at a fraction of their rate (8.6 clocks each); tensor memory would only add its
//    round trip.
//  * e4m3 codes become f16 exactly.  The powers of two never touch them: with
//    k_j = 2^a_j K_j and v_j = 2^b_j V_j in codes K, V, the exponent of
//    position j is t_j = 2^a_j (q . K_j) c + b_j in one multiply-add, the sum over V
//    takes 2^(t_j - ref) V_j and l takes 2^(t_j - ref) 2^-b_j.  Queries become f16
//    after a power of two has brought their row's largest to 2^14 (what f16
//    cannot hold then is below 2^-38 of it).
#include "fcc_paged.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "fcc_ptx.cuh"

namespace fcc {
namespace {

// Rows to a sequence and key/value head up to which items of 16 rows are faster than
// tiles of 128, although an item reads the cache for every 16 rows: 40 sequences of 6000
// positions, 8 heads take 155 us by items with 16 rows in bf16 and 300 with 24, and 202 by
// tiles with any number up to 128; e4m3 192 by items with 24 and 32 rows, 293 with 40, and
// 261 by tiles.  For sequences alike: the average says nothing of a chunk among single rows,
// which one call takes in 1.02 to 3.5 times the two parts' time (fcc.h says how to split it).
constexpr int kFewRowsBf16 = 16, kFewRowsE4m3 = 32;
// The reference is raised past this (log2 units).  f16 is used to its end: a row's largest
// p lies between 2^8 and 2^16, and what vanishes, p below 2^-25, is below 2^-33 of it.
template <bool E4M3>
constexpr float kRaise = E4M3 ? 7.9f : 8.f;

struct Header {                                // of the item whose first part CTA c holds last
  int parts;                                   // CTAs from c on (0: none)
  int b, item;
};

__host__ __device__ inline size_t header_bytes(int ctas) {
  return (static_cast<size_t>(ctas) * sizeof(Header) + 255) & ~size_t{255};
}

// Partial sums of an item: its rows' references and sums, then the values as the
// threads hold them.
__host__ __device__ constexpr size_t part_floats(int d, int nq) { return 8 * static_cast<size_t>(nq) * (d + 2); }

template <int D, bool E4M3, int NQ>
struct Few {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);        // bytes of a position's key
  // Bytes of a slice's keys (and of its values): long slices, because a slice's look-ups
  // and addresses are as many instructions as 16 positions' products.
  static constexpr int kHalf = 4096;
  static constexpr int kTok = kHalf / kRow;              // positions of a slice: 16, 32 or 64
  // 96 KB of rings, two CTAs to an SM: more warps where the registers allow it (8 rows to
  // an item: 6 warps of 2 slices read 201 x 8000 e4m3 in 330 us, 4 of 3 in 334, 64 x 8192
  // bf16 in 205 and 210; 16 rows: 4 of 3 take 106 us for 40 x 1-5 rows, 6 of 2 143).
  static constexpr int kWarps = NQ == 1 ? 6 : 4;
  static constexpr int kStages = NQ == 1 ? 2 : 3;
  static constexpr int kUnit = kWarps * kTok;
  static constexpr int kRows = 8 * NQ;                   // of a tile
  static constexpr int kLanes = kRow / 16;               // lanes that load a row
  static constexpr int kRowsAtOnce = 32 / kLanes;
  static constexpr int kPer = (kTok + 31) / 32;          // positions that a lane looks up
  // a slice in the ring: keys, values, e4m3: the bytes of their powers
  static constexpr int kStage = 2 * kHalf + (E4M3 ? 2 * kTok : 0);
  static constexpr int kSmem = kWarps * kStages * kStage;
  // a warp's values pass through the place of its last slice, a part of the rows at a time
  static constexpr int kRounds = NQ * 8 * D * 4 > 2 * kHalf ? NQ * 8 * D * 4 / (2 * kHalf) : 1;
  static constexpr int kQTiles = NQ / kRounds;           // tiles of 8 rows in a round
  static_assert(kQTiles * kRounds == NQ && kQTiles * 8 * D * 4 <= 2 * kHalf, "a round's values fit a slice's place");
  // 16-byte chunks are permuted so that eight rows' chunks of one number lie in
  // eight different groups of banks
  static __device__ __forceinline__ uint32_t at(int row, int chunk) {
    return row * kRow + ((chunk ^ (kRow == 64 ? (row >> 1) & 3 : row & 7)) << 4);
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of the warp's 8 x 8 16-bit values.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A walk over a CTA's run of units: item after item, each from unit k to unit end.
// AGAIN: over whole items, every gridDim.x-th one, those that have rows to be computed again.
template <int kRows, int kUnit, bool AGAIN>
struct Walk {
  int b, item, k, end;
  Seq q;
  int seen;          // the first position that a row sees
  int first;         // the first position of unit 0: 16 positions from a multiple of 16 on lie together
  int nk;            // units of each of the sequence's items
  int tiles;         // tiles of kRows rows
  int items;         // R * H * tiles
  long long left;    // units of the CTA behind this item's
  int r, h, row0;    // the item's rank, head and first row
  int hi;            // the position of its last row (-1: nothing is seen)
  int whole_from, whole_to;   // positions in (from, to] are seen by every row

  // What sequence `seq` has to do (units of all its items).
  __device__ __forceinline__ long long measure(const PagedArgs& a, int seq) {
    b = seq;
    q = load_seq(a.step, seq);
    tiles = (q.n * a.G + kRows - 1) / kRows;
    items = a.R * a.pool.H * tiles;
    seen = max(0, q.L - q.n - a.window + 1);
    first = seen & ~15;
    const int L = min(q.L, a.held);
    nk = q.ok && L > first ? static_cast<int>((static_cast<long long>(L) - first + kUnit - 1) / kUnit) : 1;
    return static_cast<long long>(items) * nk;
  }
  __device__ __forceinline__ void take(const PagedArgs& a) {
    const int n = static_cast<int>(min(static_cast<long long>(nk - k), left));
    end = k + n;
    left -= n;
    const int rh = item / tiles;
    row0 = (item - rh * tiles) * kRows;
    r = rh / a.pool.H;
    h = rh - r * a.pool.H;
    hi = q.ok ? q.L - q.n + a.by_g(min(q.n * a.G - row0, kRows) + row0 - 1) : -1;
    whole_from = hi - a.window;
    whole_to = q.ok ? q.L - q.n + a.by_g(row0) : -1;
  }
  // The item's rows that are to be computed again.
  __device__ __forceinline__ uint32_t marked(const PagedArgs& a) const {
    const int rh = item / tiles, row = (item - rh * tiles) * kRows;
    const uint32_t m = a.again.bits(rh, q.s * a.G + row);
    return m & ((1u << min(kRows, q.n * a.G - row)) - 1);
  }
  __device__ __forceinline__ bool find_marked(const PagedArgs& a) {
    for (;; item += gridDim.x) {
      while (item >= items) {
        item -= items;
        if (b + 1 >= a.step.B) return false;
        measure(a, b + 1);
      }
      if (marked(a) != 0) break;
    }
    k = 0;
    left = nk;
    take(a);
    return true;
  }
  __device__ __forceinline__ bool next_item(const PagedArgs& a) {
    if constexpr (AGAIN) {
      item += gridDim.x;
      return find_marked(a);
    }
    if (left <= 0) return false;
    if (++item == items) {
      item = 0;
      do {
        if (b + 1 >= a.step.B) return false;
      } while (measure(a, b + 1) == 0);
    }
    k = 0;
    take(a);
    return true;
  }
};

// An item's sums for one product's 16 columns and 8 rows: thread `lane` holds columns
// lane / 4 and + 8 (in V's order) of rows 2 (lane % 4) and + 1.
struct Sums {
  float o[4] = {};
  float ref[2] = {-INFINITY, -INFINITY}, l[2] = {};
  __device__ __forceinline__ void add(const float4& x, const float (&f)[2]) {
    o[0] = fmaf(x.x, f[0], o[0]);
    o[1] = fmaf(x.y, f[1], o[1]);
    o[2] = fmaf(x.z, f[0], o[2]);
    o[3] = fmaf(x.w, f[1], o[3]);
  }
};

// Stores columns 16 j .. 16 j + 15 of rows row0 .. row0 + 7 of a sequence, those whose bits are set.
template <int D, bool E4M3>
__device__ __forceinline__ void store_rows(const PagedArgs& a, const Seq& q, int r, int h, int row0, int j, int lane,
                                           const Sums& m, uint32_t rows = 0xff) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool none = m.l[i] == 0.f;
    const float inv = 1.f / m.l[i];
    float x = none ? 0.f : m.o[i] * inv, y = none ? 0.f : m.o[2 + i] * inv;
    int col = 2 * g;                           // e4m3: columns 2 g and 2 g + 1
    if constexpr (!E4M3) {                     // columns g and g + 8: neighbours are brought together
      const float other = __shfl_xor_sync(0xffffffffu, g & 1 ? x : y, 4);
      col = g & 1 ? g + 7 : g;
      x = g & 1 ? other : x;
      y = g & 1 ? y : other;
    }
    const int rho = row0 + 2 * c + i;
    if (rho >= q.n * a.G || !(rows >> (2 * c + i) & 1)) continue;
    const int t = a.by_g(rho), head = h * a.G + (rho - t * a.G);
    const int64_t token = static_cast<int64_t>(q.s) + t;
    *reinterpret_cast<uint32_t*>(a.O[r] + (token * a.ldo + static_cast<int64_t>(head) * D + 16 * j + col) * 2) = ptx::pack_bf16x2(x, y);
    if (j == 0 && g == 0 && a.lse[r] != nullptr)
      a.lse[r][token * a.Hq + head] = none ? -INFINITY : (m.ref[i] + log2f(m.l[i])) * kLn2;
  }
}

// AGAIN: the rows that tiles of 128 left (Again), an item to a CTA from its first position
// to its last: where they are summed does not depend on which others there are.  All 65536
// rows over 32768 positions take 6.4 ms in bf16 and 37 in e4m3, beside 0.7 and 1.0 in tiles.
template <int D, bool E4M3, int NQ, bool AGAIN>
__global__ void __launch_bounds__(Few<D, E4M3, NQ>::kWarps * 32, 2) few_rows_kernel(const __grid_constant__ PagedArgs a) {
  using F = Few<D, E4M3, NQ>;
  constexpr int kTok = F::kTok, kUnit = F::kUnit, kPer = F::kPer, kWarps = F::kWarps, kHalf = F::kHalf, kStages = F::kStages;
  constexpr int kM = kTok / 16;                // products' rows of 16 positions
  constexpr int kD = D / 16;
  constexpr float kOff = E4M3 ? 8.f : 0.f;     // p up to 2^(kOff + kRaise)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps], s_off;
  __shared__ int s_b;
  __shared__ float s_ref[kWarps][F::kRows], s_l[kWarps][F::kRows];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ---------------------------------------------- this CTA's run of units
  Walk<F::kRows, kUnit, AGAIN> w;
  long long total = 0, ctas = 0, u0 = 0;
  Header* const headers = reinterpret_cast<Header*>(a.ws);
  if constexpr (AGAIN) {
    if (*a.again.any == 0) return;
    w.measure(a, 0);
    w.item = blockIdx.x;
    if (!w.find_marked(a)) return;
  } else {
    const int per = (a.step.B + kWarps * 32 - 1) / (kWarps * 32);
    const int b_first = min(a.step.B, static_cast<int>(threadIdx.x) * per), b_last = min(a.step.B, b_first + per);
    long long mine = 0;
    for (int b = b_first; b < b_last; ++b) {
      mine += w.measure(a, b);
      if (blockIdx.x == 0 && bad_sequence(a, w.q)) record_invalid(a.status);
    }
    long long upto = mine;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, s);
      if (lane >= s) upto += v;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long from = upto - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) from += s_scan[i];
      total += s_scan[i];
    }
    ctas = min(static_cast<long long>(gridDim.x), total);
    if (threadIdx.x == 0) headers[blockIdx.x].parts = 0;
    if (blockIdx.x >= ctas) return;
    u0 = blockIdx.x * total / ctas;
    const long long u1 = (blockIdx.x + 1) * total / ctas;
    if (u0 >= from && u0 < from + mine) {
      long long off = u0 - from;
      for (int b = b_first; b < b_last; ++b) {
        const long long n = w.measure(a, b);
        if (off < n) {
          s_b = b;
          s_off = off;
          break;
        }
        off -= n;
      }
    }
    __syncthreads();
    w.measure(a, s_b);
    w.item = static_cast<int>(s_off / w.nk);
    w.k = static_cast<int>(s_off % w.nk);
    w.left = u1 - u0;
    w.take(a);
  }

  // ------------------------------------------------------------- loading
  // The loads' own walk runs kStages - 1 slices ahead of the products, and the
  // look-up of the pages one slice more.
  uint8_t* const ring = smem + warp * (kStages * F::kStage);
  const uint32_t ring_addr = ptx::smem_addr(ring);
  struct Slice {
    uint32_t there[kPer];                      // which positions the pages hold
  };
  Walk<F::kRows, kUnit, AGAIN> lw = w;
  bool more = true;
  int page[kPer], in_page[kPer] = {}, pool_r = 0, pool_h = 0;
  const int* table = a.step.table + static_cast<int64_t>(lw.b) * a.step.max_pages;   // of lw's sequence
  uint32_t pos = static_cast<uint32_t>(lw.first) + static_cast<uint32_t>(lw.k) * kUnit + warp * kTok + lane;   // of the next slice's
  // A page's number is checked where it was asked for, which waits for it, or with 16 rows
  // to an item of e4m3 a slice later (40 x 2 tokens 104 instead of 110 us, 40 x 1-5 103
  // instead of 105).  Where DRAM is the bound, later was slower: 1 x 1000003 e4m3 309
  // instead of 304 us, 64 x 8192 bf16 201.2 instead of 199.7, 40 x 2 bf16 154.7 instead
  // of 153.7.
  constexpr bool kLater = E4M3 && NQ > 1;
  bool asked[kPer];
  auto check = [&](int i) {
    if (static_cast<uint32_t>(page[i]) >= static_cast<uint32_t>(a.pool.pages)) {
      page[i] = -1;
      if (asked[i]) record_invalid(a.status);
    }
  };
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      page[i] = -1;
      asked[i] = false;
    }
    if (!more) return;
    pool_r = lw.r;
    pool_h = lw.h;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t p = pos + 32 * i;
      if ((kTok >= 32 || lane < kTok) && p < static_cast<uint32_t>(lw.hi + 1) && p >= static_cast<uint32_t>(lw.seen)) {
        const uint32_t idx = p >> a.pool.log2P;
        if (idx < static_cast<uint32_t>(a.step.max_pages)) page[i] = __ldg(table + idx);
        in_page[i] = p & ((1u << a.pool.log2P) - 1);
        asked[i] = true;
        if constexpr (!kLater) check(i);
      }
    }
    pos += kUnit;
    if (++lw.k == lw.end) {
      more = lw.next_item(a);
      table = a.step.table + static_cast<int64_t>(lw.b) * a.step.max_pages;
      pos = static_cast<uint32_t>(lw.first) + static_cast<uint32_t>(lw.k) * kUnit + warp * kTok + lane;
    }
  };
  auto issue = [&](int slot) -> Slice {
    Slice s;
    uint32_t any = 0, run = 0xffffffffu;       // run: each 16 positions lie one after another in a page
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kLater) check(i);
      s.there[i] = __ballot_sync(0xffffffffu, page[i] >= 0);
      any |= s.there[i];
      const int page0 = __shfl_sync(0xffffffffu, page[i], lane & 16), in_page0 = __shfl_sync(0xffffffffu, in_page[i], lane & 16);
      const bool next = page[i] >= 0 && page[i] == page0 && in_page[i] == in_page0 + (lane & 15);
      run &= __ballot_sync(0xffffffffu, next || (kTok < 32 && lane >= kTok));
    }
    if (any != 0) {
      int64_t row[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        row[i] = page[i] < 0 ? 0 : ((static_cast<int64_t>(page[i]) * a.pool.H + pool_h) << a.pool.log2P) + in_page[i];
      const int chunk = lane % F::kLanes, sub = lane / F::kLanes;
      const uint32_t dst = ring_addr + slot * F::kStage;
      if (run == 0xffffffffu) {                // 16 positions are one piece of memory, 512 bytes to a step
        constexpr int kSteps = 16 / F::kRowsAtOnce;
        const char* K = a.pool.K[pool_r] + lane * 16;
        const char* V = a.pool.V[pool_r] + lane * 16;
#pragma unroll
        for (int n = 0; n < kTok / 16; ++n) {
          const int64_t off = __shfl_sync(0xffffffffu, row[n / 2], 16 * (n & 1)) * F::kRow;
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const uint32_t to = dst + F::at(n * 16 + i * F::kRowsAtOnce + sub, chunk);
            cp_async16(to, K + off + i * 512, true);
            cp_async16(to + kHalf, V + off + i * 512, true);
          }
        }
        if constexpr (E4M3) {                  // (through memory like the rest: a register waits for its load)
          const int64_t at = __shfl_sync(0xffffffffu, row[kPer - 1], lane * 16 & 31);
          const int64_t at0 = __shfl_sync(0xffffffffu, row[0], lane * 16 & 31);
          if (lane < 2 * (kTok / 16)) {
            const int n = lane % (kTok / 16);  // 16 bytes of keys or values
            const uint8_t* e = lane < kTok / 16 ? a.pool.Ke[pool_r] : a.pool.Ve[pool_r];
            cp_async16(dst + 2 * kHalf + lane * 16, e + (n < 2 ? at0 : at), true);
          }
        }
      } else {
        const char* K = a.pool.K[pool_r] + chunk * 16;
        const char* V = a.pool.V[pool_r] + chunk * 16;
#pragma unroll
        for (int i = 0; i < kTok / F::kRowsAtOnce; ++i) {
          const int tok = i * F::kRowsAtOnce + sub;
          const int64_t off = __shfl_sync(0xffffffffu, row[(i * F::kRowsAtOnce) / 32], tok & 31) * F::kRow;
          const bool there = s.there[(i * F::kRowsAtOnce) / 32] >> (tok & 31) & 1;
          cp_async16(dst + F::at(tok, chunk), K + off, there);
          cp_async16(dst + kHalf + F::at(tok, chunk), V + off, there);
        }
        if constexpr (E4M3) {
          uint8_t* const e = ring + slot * F::kStage + 2 * kHalf;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const bool there = page[i] >= 0;
            e[lane + 32 * i] = there ? a.pool.Ke[pool_r][row[i]] : 127;
            e[kTok + lane + 32 * i] = there ? a.pool.Ve[pool_r][row[i]] : 127;
          }
        }
      }
    }
    cp_async_commit();
    return s;
  };

  Slice queue[kStages - 1];
  look_up();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    queue[s] = issue(s);
    look_up();
  }

  // ------------------------------------------------------------ products
  int slot = 0;
  long long at = u0;                           // unit that the walk stands at
  do {
    const int k0 = w.k, rows = w.q.n * a.G;
    // Queries: the thread's row (of n) is g; the scales of its columns' rows 2 c, 2 c + 1.
    uint32_t qb[NQ][kD][2];
    float scale[NQ][2], ref[NQ][2], l[NQ][2];
    int qpos[NQ][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const int rho = min(w.row0 + 8 * nq + g, rows - 1), t = a.by_g(rho);   // (a row past the last repeats it)
      const char* src = a.Q[w.r] + ((static_cast<int64_t>(w.q.s) + t) * a.ldq + static_cast<int64_t>(w.h * a.G + rho - t * a.G) * D) * 2;
#pragma unroll
      for (int kk = 0; kk < kD; ++kk) {
        if constexpr (E4M3) {
          const uint2 x = *reinterpret_cast<const uint2*>(src + kk * 32 + 8 * c);
          qb[nq][kk][0] = x.x;
          qb[nq][kk][1] = x.y;
        } else {
          qb[nq][kk][0] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + 4 * c);
          qb[nq][kk][1] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + 16 + 4 * c);
        }
      }
      float mine = a.scale_log2;
      if constexpr (E4M3) {
        // the row's largest finite magnitude, as bf16 bits
        unsigned top = 0;
#pragma unroll
        for (int kk = 0; kk < kD; ++kk)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned m = (qb[nq][kk][j >> 1] >> (16 * (j & 1))) & 0x7fffu;
            top = max(top, m < 0x7f80u ? m : 0u);
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -100) - 14;
        const float f = power_of_two(-e);
        mine *= power_of_two(e);
#pragma unroll
        for (int kk = 0; kk < kD; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x = qb[nq][kk][j];
            qb[nq][kk][j] = pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        scale[nq][i] = __shfl_sync(0xffffffffu, mine, (2 * c + i) * 4);
        qpos[nq][i] = w.q.ok ? w.q.L - w.q.n + a.by_g(min(w.row0 + 8 * nq + 2 * c + i, rows - 1)) : -1;
        ref[nq][i] = -INFINITY;
        l[nq][i] = 0.f;
      }
    }
    float o[kD][NQ][4] = {};

    for (; w.k < w.end; ++w.k) {
      cp_async_wait<kStages - 2>();
      __syncwarp();                            // every lane's part of the slice is there
      const Slice cur = queue[0];
#pragma unroll
      for (int s = 0; s + 1 < kStages - 1; ++s) queue[s] = queue[s + 1];
      queue[kStages - 2] = issue(slot == 0 ? kStages - 1 : slot - 1);
      look_up();
      const uint32_t ks = ring_addr + slot * F::kStage, vs = ks + kHalf;
      uint8_t* const scratch = ring + slot * F::kStage;
      slot = slot + 1 == kStages ? 0 : slot + 1;

      uint32_t any = 0, all = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        any |= cur.there[i];
        all &= kTok < 32 ? cur.there[i] | ~((1u << (kTok & 31)) - 1) : cur.there[i];
      }
      if (any == 0) continue;
      const int pos0 = w.first + w.k * kUnit + warp * kTok;   // (some position of it is there)
      // every row sees every position (a window reaches back from the last row)
      const bool whole = all == 0xffffffffu && pos0 <= w.whole_to - (kTok - 1) && pos0 > w.whole_from;
      auto sees = [&](int mt, int nq, int i) -> bool {
        const int tok = mt * 16 + g + 8 * (i >> 1), q = qpos[nq][i & 1];
        const long long pos = static_cast<long long>(pos0) + tok;
        return (cur.there[mt / 2] >> (tok & 31) & 1) && pos <= q && pos > static_cast<long long>(q) - a.window;
      };

      // S^T: element i of a product is position g + 8 (i / 2), row 2 c + i % 2
      float s[kM][NQ][4];
#pragma unroll
      for (int mt = 0; mt < kM; ++mt) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][nq][i] = 0.f;
        const int row = mt * 16 + (lane & 15);
        uint32_t x[4], y[4];
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {   // two steps of 16: chunks 2 j and 2 j + 1
            ldsm4(x, ks + F::at(row, 2 * j + (lane >> 4)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              f16x4_of_e4m3(x[2 * i], y[0], y[2]);
              f16x4_of_e4m3(x[2 * i + 1], y[1], y[3]);
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq) mma<true>(s[mt][nq], y, qb[nq][2 * j + i][0], qb[nq][2 * j + i][1]);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < kD; ++kk) {
            ldsm4(x, ks + F::at(row, 2 * kk + (lane >> 4)));
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) mma<false>(s[mt][nq], x, qb[nq][kk][0], qb[nq][kk][1]);
          }
        }
      }
      // exponents (log2 units), and whether a row asks for a new reference
      float inv[kM][2];                        // e4m3: what brings p back to the sum's units
      bool raise = false;
#pragma unroll
      for (int mt = 0; mt < kM; ++mt) {
        float kx[2], vx[2];
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint8_t* e = scratch + 2 * kHalf + mt * 16 + g + 8 * j;
            const int ev = min(static_cast<int>(e[kTok]), 254);
            kx[j] = __int_as_float(static_cast<int>(e[0]) << 23);
            vx[j] = static_cast<float>(ev - 127);
            inv[mt][j] = __int_as_float((254 - ev) << 23);
          }
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& t = s[mt][nq][i];
            t = E4M3 ? fmaf(t * scale[nq][i & 1], kx[i >> 1], vx[i >> 1]) : t * scale[nq][i & 1];
            if (!whole && !sees(mt, nq, i)) t = -INFINITY;
            raise |= t > ref[nq][i & 1] + (kOff + kRaise<E4M3>);
          }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -INFINITY;             // the row's largest
#pragma unroll
            for (int mt = 0; mt < kM; ++mt) top = ptx::max3(top, s[mt][nq][i], s[mt][nq][2 + i]);
#pragma unroll
            for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            f[i] = 1.f;
            if (top > ref[nq][i] + (kOff + kRaise<E4M3>)) {
              f[i] = ex2_from(ref[nq][i], top - kOff);
              ref[nq][i] = top - kOff;
              l[nq][i] *= f[i];
            }
          }
#pragma unroll
          for (int j = 0; j < kD; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][nq][i] *= f[i & 1];
        }
      }
      // (e4m3 rows that are computed again saw powers far apart: their sums are f32 throughout)
      constexpr bool kExact = AGAIN && E4M3;
      bool plain = !kExact;
      if (!kExact && !whole) {
        // A value that is not finite must not reach rows that do not see it through
        // a product with their p = 0.
        bool odd = false;
        const uint4* v = reinterpret_cast<const uint4*>(scratch + kHalf);
#pragma unroll
        for (int i = 0; i < kHalf / 512; ++i) {
          const uint4 x = v[i * 32 + lane];
          for (uint32_t y : {x.x, x.y, x.z, x.w})
            odd |= E4M3 ? (((y & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0
                        : (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
        }
        plain = !__any_sync(0xffffffffu, odd);
      }
      if (plain) {
#pragma unroll
        for (int mt = 0; mt < kM; ++mt) {
          uint32_t pb[NQ][2];
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (a row that has seen nothing yet: 2^(-inf - 0) = 0)
              p[i] = ptx::ex2_approx(s[mt][nq][i] - (ref[nq][i & 1] == -INFINITY ? 0.f : ref[nq][i & 1]));
              l[nq][i & 1] = E4M3 ? fmaf(p[i], inv[mt][i >> 1], l[nq][i & 1]) : l[nq][i & 1] + p[i];
            }
            pb[nq][0] = transpose8(pack16<E4M3>(p[0], p[1]));
            pb[nq][1] = transpose8(pack16<E4M3>(p[2], p[3]));
          }
          uint32_t x[4], y[4];
          if constexpr (E4M3) {
            const int row = mt * 16 + (lane & 15);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              ldsm4_t(x, vs + F::at(row, 2 * j + (lane >> 4)));
#pragma unroll
              for (int i = 0; i < 2; ++i) {    // columns 2 g in the products' rows g, 2 g + 1 in g + 8
                f16x4_of_e4m3(__byte_perm(x[2 * i], 0, 0x3120), y[0], y[1]);
                f16x4_of_e4m3(__byte_perm(x[2 * i + 1], 0, 0x3120), y[2], y[3]);
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) mma<true>(o[2 * j + i][nq], y, pb[nq][0], pb[nq][1]);
              }
            }
          } else {
            const int row = mt * 16 + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < kD; ++j) {
              ldsm4_t(x, vs + F::at(row, 2 * j + half));
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq) mma<false>(o[j][nq], x, pb[nq][0], pb[nq][1]);
            }
          }
        }
      } else {
        // One position after another, in f32; the probabilities of 8 rows at a time pass
        // through the keys' place, -1 for a position that the row does not see.
        float* const ps = reinterpret_cast<float*>(scratch);   // [8][kTok]
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          __syncwarp();
#pragma unroll
          for (int mt = 0; mt < kM; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool there = sees(mt, nq, i);
              const float p = ptx::ex2_approx(s[mt][nq][i] - (ref[nq][i & 1] == -INFINITY ? 0.f : ref[nq][i & 1]));
              if (there) l[nq][i & 1] = E4M3 ? fmaf(p, inv[mt][i >> 1], l[nq][i & 1]) : l[nq][i & 1] + p;
              ps[(2 * c + (i & 1)) * kTok + mt * 16 + g + 8 * (i >> 1)] = there ? p : -1.f;
            }
          __syncwarp();
#pragma unroll 1
          for (int tok = 0; tok < kTok; ++tok) {
            const float p[2] = {ps[2 * c * kTok + tok], ps[(2 * c + 1) * kTok + tok]};
#pragma unroll
            for (int j = 0; j < kD; ++j) {
              float v[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int col = 16 * j + (E4M3 ? 2 * g + i : g + 8 * i);
                if constexpr (E4M3) {
                  const uint32_t code = scratch[kHalf + F::at(tok, col >> 4) + (col & 15)];
                  v[i] = __low2float(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(code), __NV_E4M3)));
                } else {
                  v[i] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                      scratch + kHalf + F::at(tok, col >> 3) + (col & 7) * 2));
                }
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!(p[i & 1] < 0.f)) o[j][nq][i] = fmaf(p[i & 1], v[i >> 1], o[j][nq][i]);
            }
          }
        }
        __syncwarp();
      }
    }

    // ------------------------------------- the warps' sums, added in order
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[nq][i] += __shfl_xor_sync(0xffffffffu, l[nq][i], x);
        if (g == 0) {
          s_ref[warp][8 * nq + 2 * c + i] = ref[nq][i];
          s_l[warp][8 * nq + 2 * c + i] = l[nq][i];
        }
      }
    const bool complete = AGAIN || (k0 == 0 && w.end == w.nk);
    const uint32_t wanted = AGAIN ? w.marked(a) : 0xffffffffu;
    // (the slice just used: its place is loaded again by the next item's first step)
    const int used = slot == 0 ? kStages - 1 : slot - 1;
    float4* const mine_o = reinterpret_cast<float4*>(ring + used * F::kStage);
    // an item that begins here and does not end goes to the second place of this CTA
    float* const part = reinterpret_cast<float*>(a.ws + header_bytes(gridDim.x)) +
                        (2 * static_cast<size_t>(blockIdx.x) + (k0 == 0 ? 1 : 0)) * part_floats(D, NQ);
#pragma unroll
    for (int round = 0; round < F::kRounds; ++round) {
      __syncwarp();
#pragma unroll
      for (int n = 0; n < F::kQTiles; ++n)
#pragma unroll
        for (int j = 0; j < kD; ++j) {
          const float (&x)[4] = o[j][round * F::kQTiles + n];
          mine_o[(n * kD + j) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
        }
      __syncthreads();
#pragma unroll 1
      for (int f4 = warp; f4 < F::kQTiles * kD; f4 += kWarps) {
        const int n = f4 / kD, j = f4 % kD, row = 8 * (round * F::kQTiles + n) + 2 * c;
        Sums m;
#pragma unroll
        for (int v = 0; v < kWarps; ++v)
#pragma unroll
          for (int i = 0; i < 2; ++i) m.ref[i] = fmaxf(m.ref[i], s_ref[v][row + i]);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f[i] = ex2_from(s_ref[v][row + i], m.ref[i]);
            m.l[i] = fmaf(s_l[v][row + i], f[i], m.l[i]);
          }
          m.add(reinterpret_cast<const float4*>(smem + (v * kStages + used) * F::kStage)[f4 * 32 + lane], f);
        }
        if (complete) {
          store_rows<D, E4M3>(a, w.q, w.r, w.h, w.row0 + row - 2 * c, j, lane, m, wanted >> (row - 2 * c));
        } else {
          if (j == 0 && g == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              part[row + i] = m.ref[i];
              part[F::kRows + row + i] = m.l[i];
            }
          }
          reinterpret_cast<float4*>(part + 2 * F::kRows)[(round * F::kQTiles * kD + f4) * 32 + lane] =
              make_float4(m.o[0], m.o[1], m.o[2], m.o[3]);
        }
      }
      __syncthreads();
    }
    if (!complete && k0 == 0 && threadIdx.x == 0) {
      const long long last = at + w.nk;        // behind the item's last unit
      headers[blockIdx.x] = Header{static_cast<int>((last * ctas - 1) / total) - static_cast<int>(blockIdx.x) + 1, w.b, w.item};
    }
    at += w.end - k0;
  } while (w.next_item(a));
  cp_async_wait<0>();
}

// Adds the parts of the item that CTA blockIdx.x of few_rows_kernel began last
// and did not finish, in the CTAs' order; blockIdx.y counts tiles of 8 rows.
template <int D, bool E4M3, int NQ>
__global__ void __launch_bounds__(D * 2) combine_kernel(const __grid_constant__ PagedArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const Header hd = reinterpret_cast<const Header*>(a.ws)[blockIdx.x];
  if (hd.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 8 * blockIdx.y + 2 * (lane & 3);
  const float* parts = reinterpret_cast<const float*>(a.ws + header_bytes(gridDim.x));
  auto part = [&](int i) { return parts + (2 * static_cast<size_t>(blockIdx.x + i) + (i == 0 ? 1 : 0)) * part_floats(D, NQ); };
  // (four parts' loads at a time: a long item's parts are a chain of them otherwise)
  constexpr int kAtOnce = 4;
  Sums m;
  for (int v0 = 0; v0 < hd.parts; v0 += kAtOnce) {
    float2 ref[kAtOnce], l[kAtOnce];
    float4 x[kAtOnce];
#pragma unroll
    for (int v = 0; v < kAtOnce; ++v) {
      const float* p = part(min(v0 + v, hd.parts - 1));
      ref[v] = *reinterpret_cast<const float2*>(p + row);
      l[v] = *reinterpret_cast<const float2*>(p + 8 * NQ + row);
      x[v] = reinterpret_cast<const float4*>(p + 16 * NQ)[(blockIdx.y * (D / 16) + warp) * 32 + lane];
    }
    float top[2] = {m.ref[0], m.ref[1]}, f[2];
#pragma unroll
    for (int v = 0; v < kAtOnce; ++v) {
      top[0] = fmaxf(top[0], ref[v].x);
      top[1] = fmaxf(top[1], ref[v].y);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = ex2_from(m.ref[i], top[i]);
      m.ref[i] = top[i];
      m.l[i] *= f[i];
      m.o[i] *= f[i];
      m.o[2 + i] *= f[i];
    }
#pragma unroll
    for (int v = 0; v < kAtOnce; ++v) {
      if (v0 + v >= hd.parts) break;
      f[0] = ex2_from(ref[v].x, top[0]);
      f[1] = ex2_from(ref[v].y, top[1]);
      m.l[0] = fmaf(l[v].x, f[0], m.l[0]);
      m.l[1] = fmaf(l[v].y, f[1], m.l[1]);
      m.add(x[v], f);
    }
  }
  const Seq q = load_seq(a.step, hd.b);
  const int tiles = (q.n * a.G + 8 * NQ - 1) / (8 * NQ), rh = hd.item / tiles;
  store_rows<D, E4M3>(a, q, rh / a.pool.H, rh % a.pool.H, (hd.item - rh * tiles) * 8 * NQ + 8 * blockIdx.y, warp, lane, m);
}

template <int D, bool E4M3, int NQ>
cudaError_t launch_few(const PagedArgs& a, int ctas, cudaStream_t st) {
  using F = Few<D, E4M3, NQ>;
  static bool attr_set[64] = {};
  cudaError_t e = smem_attr_once(attr_set, few_rows_kernel<D, E4M3, NQ, false>, F::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(ctas);
  if ((e = launch_pdl(few_rows_kernel<D, E4M3, NQ, false>, dim3(grid), dim3(F::kWarps * 32), F::kSmem, st, 1u, a)) != cudaSuccess)
    return e;
  return launch_pdl(combine_kernel<D, E4M3, NQ>, dim3(grid, NQ), dim3(D * 2), 0, st, 1u, a);
}

template <int NQ>
cudaError_t launch_few(const PagedArgs& a, bool e4m3, int ctas, cudaStream_t st) {
  return a.pool.d == 128 ? (e4m3 ? launch_few<128, true, NQ>(a, ctas, st) : launch_few<128, false, NQ>(a, ctas, st))
                         : (e4m3 ? launch_few<64, true, NQ>(a, ctas, st) : launch_few<64, false, NQ>(a, ctas, st));
}

// After launch_tiles: the rows that it left.
template <int D, bool E4M3>
cudaError_t launch_again(const PagedArgs& a, int ctas, cudaStream_t st) {
  using F = Few<D, E4M3, 2>;
  static bool attr_set[64] = {};
  const cudaError_t e = smem_attr_once(attr_set, few_rows_kernel<D, E4M3, 2, true>, F::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(few_rows_kernel<D, E4M3, 2, true>, dim3(static_cast<unsigned>(ctas)), dim3(F::kWarps * 32), F::kSmem, st, 1u, a);
}
cudaError_t launch_again(const PagedArgs& a, bool e4m3, int ctas, cudaStream_t st) {
  return a.pool.d == 128 ? (e4m3 ? launch_again<128, true>(a, ctas, st) : launch_again<128, false>(a, ctas, st))
                         : (e4m3 ? launch_again<64, true>(a, ctas, st) : launch_again<64, false>(a, ctas, st));
}

// The form for a step: NQ tiles of 8 rows to an item, or 0 for tiles of 128 rows on
// the tensor cores' own memory.  By the rows to a sequence and key/value head on
// average, which is all that the host knows; every form takes every step.
int form_of(int64_t T, int B, int G, bool e4m3) {
  const int64_t rows = T * G, each = B;
  if (rows <= 8 * each) return 1;
  return rows <= (e4m3 ? kFewRowsE4m3 : kFewRowsBf16) * each ? 2 : 0;
}

// CTAs of a form's kernel: two to an SM, or one of tiles_kernel's.
int ctas_of(int form, const fcc_opts* o) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 256;  // (no device: sizes for the largest grid)
  }
  const int ctas = sms * (form != 0 ? 2 : 1);
  return o != nullptr && o->max_ctas > 0 ? std::min(ctas, o->max_ctas) : ctas;
}

size_t form_ws_bytes(int form, int R, int64_t T, int B, int G, int H, int64_t d, int ctas) {
  return form != 0 ? header_bytes(ctas) + 2 * static_cast<size_t>(ctas) * part_floats(static_cast<int>(d), form) * sizeof(float)
                   : tiles_ws_bytes(d, B, ctas, T * G, static_cast<int64_t>(R) * H);
}

// What a call asks for: enough for either type of cache.
size_t paged_ws_bytes(int R, int64_t T, int B, int G, int H, int64_t d, const fcc_opts* o) {
  size_t most = 0;
  for (bool e4m3 : {false, true}) {
    const int form = form_of(T, B, G, e4m3);
    most = std::max(most, form_ws_bytes(form, R, T, B, G, H, d, ctas_of(form, o)));
  }
  return most;
}

}  // namespace
}  // namespace fcc

using namespace fcc;

extern "C" {

size_t fcc_paged_attention_workspace_size(int R, int64_t T, int B, int Hq, int H, int64_t d,
                                          const fcc_opts* opts) {
  if (R < 1 || R > FCC_MAX_RANKS || T < 1 || B < 1 || H < 1 || Hq < H || Hq % H != 0 ||
      (d != 64 && d != 128))
    return 0;
  return paged_ws_bytes(R, T, B, Hq / H, H, d, opts);
}

fcc_status fcc_paged_attention(int R, const void* const* Q, int64_t ldq, const fcc_cache* cache,
                               const fcc_batch* batch, int Hq, void* const* O, int64_t ldo,
                               float* const* lse, float scale, int64_t window, fcc_dtype in,
                               fcc_dtype out, const fcc_opts* opts, fcc_stream_t stream) {
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  const fcc_status described = cache_args(R, cache, batch, &a.pool, &a.step);
  if (described == FCC_ERR_INVALID) return described;
  if (Hq < 1 || Hq > 1024 || Hq % cache->H != 0) return FCC_ERR_INVALID;
  if (Q == nullptr || O == nullptr) return FCC_ERR_INVALID;
  for (int r = 0; r < R; ++r) {
    for (const void* p : {Q[r], static_cast<const void*>(O[r])})
      if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u)) return FCC_ERR_INVALID;
    if (lse != nullptr && (lse[r] == nullptr || (reinterpret_cast<uintptr_t>(lse[r]) & 15u)))
      return FCC_ERR_INVALID;
  }
  const int64_t width = static_cast<int64_t>(Hq) * cache->d;
  if (ldq == 0) ldq = width;
  if (ldo == 0) ldo = width;
  for (int64_t ld : {ldq, ldo})
    if (ld < width || ld % 8 != 0 || ld > INT_MAX) return FCC_ERR_INVALID;
  if (!(scale >= 0.f) || std::isinf(scale) || window < 0) return FCC_ERR_INVALID;
  a.scale_log2 = static_cast<float>((scale > 0.f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(cache->d))) *
                                    1.4426950408889634);
  if (std::isinf(a.scale_log2)) return FCC_ERR_INVALID;
  for (fcc_dtype t : {in, out})
    if (t != FCC_BF16 && t != FCC_F16 && t != FCC_F32) return FCC_ERR_INVALID;
  if (described != FCC_OK) return described;
  if (in != FCC_BF16 || out != FCC_BF16) return FCC_ERR_UNSUPPORTED;
  if (opts != nullptr && opts->algo != FCC_ALGO_AUTO && opts->algo != FCC_ALGO_FUSED)
    return FCC_ERR_UNSUPPORTED;
  // rows (tokens times a group's heads) and tiles of 8 of them are counted in 32 bits
  const int64_t rows = batch->T * (Hq / cache->H);
  if (rows > INT_MAX - 256 ||
      static_cast<int64_t>(R) * cache->H * (rows / 8 + batch->B) > INT_MAX)
    return FCC_ERR_INVALID;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (opts == nullptr || opts->workspace == nullptr) {
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &capture) != cudaSuccess) return FCC_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) return FCC_ERR_WORKSPACE;
  }
  a.G = Hq / cache->H;
  const bool e4m3 = cache->dtype == FCC_E4M3;
  const int form = form_of(batch->T, batch->B, a.G, e4m3), ctas = ctas_of(form, opts);
  void* ws = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  const fcc_status s = internal_prepare(opts, paged_ws_bytes(R, batch->T, batch->B, a.G, cache->H, cache->d, opts),
                                        &ws, &a.status, &sms, &timeout_ns);
  if (s != FCC_OK) return s;
  for (int r = 0; r < R; ++r) {
    a.Q[r] = static_cast<const char*>(Q[r]);
    a.O[r] = static_cast<char*>(O[r]);
    a.lse[r] = lse != nullptr ? lse[r] : nullptr;
  }
  a.ldq = ldq;
  a.ldo = ldo;
  a.R = R;
  a.Hq = Hq;
  while ((1 << a.g_shift) < a.G) ++a.g_shift;
  a.g_mul = static_cast<uint32_t>(((uint64_t{1} << (31 + a.g_shift)) + a.G - 1) / a.G);
  a.held = static_cast<int>(std::min<int64_t>(batch->max_pages << a.pool.log2P, INT_MAX));
  a.window = window == 0 ? INT_MAX : static_cast<int>(std::min<int64_t>(window, INT_MAX));
  a.ws = static_cast<char*>(ws);
  cudaError_t e = form == 1   ? launch_few<1>(a, e4m3, ctas, st)
                  : form == 2 ? launch_few<2>(a, e4m3, ctas, st)
                              : launch_tiles(a, e4m3, ctas, timeout_ns, st);
  if (form == 0 && e == cudaSuccess) e = launch_again(a, e4m3, ctas_of(2, opts), st);
  if (e != cudaSuccess) return FCC_ERR_CUDA;
  bump_launch_count(form != 0 ? 2 : 4);
  return FCC_OK;
}

}  // extern "C"
