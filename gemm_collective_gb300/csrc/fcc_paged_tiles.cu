// fcc_paged_tiles.cu -- attention of a step's rows over the paged cache in tiles of
// 128 rows on tcgen05 (prompts, chunks of prompts, mixed steps).
//
// A row is a token and one of the G query heads that share a key/value head, so a
// tile's rows read the same keys whatever G is, and few tokens fill it.  An item is
// a pair of tiles (256 rows of one sequence, rank and head) and its blocks of 128
// positions, from the first that any row sees to the last.  plan_kernel counts all
// items' blocks and cuts their list into as many equal runs as there are CTAs, one
// to an SM: causal, windowed and ragged steps load all SMs alike, and a few rows
// over a long context are spread over all of them.  What a cut leaves of an item
// are partial sums, at most two from a CTA, added in order by join_kernel.
//
// Within an item, for tile t and block j (all f32 in TMEM):
//   S_t = Q_t K_j^T;  P_t = 2^(S_t c - ref), in 16 bits over S_t's first columns;
//   O_t += P_t V_j, A from TMEM.
// A row's reference is raised (and its O_t rescaled) only when a block's maximum
// passes it by 8 (log2 units).  The two tiles alternate on the tensor core: one
// tile's exponentials run under the other's products.  A new item's queries are
// loaded, and its first S computed, before the old one's O has been stored.
//
// Warps: 0-3 and 4-7 softmax and output of tiles A and B (a thread owns a row and
// its 128 columns), 8-11 load keys and values, 12 issues the products.  The
// loaders look up every position's page for itself (any page size), bf16 rows go
// by cp.async into the swizzled tile.  e4m3 rows pass through registers and become
// f16 there, exactly; their powers of two enter at the exponent (see
// fcc_paged.cu): t = 2^a (S c) + b, P = 2^(t - ref), l += P 2^-b.
// Shared memory (128-byte swizzle): Q_t and four slots of [128 rows][D] 16-bit
// values in atoms of 64 columns, K_0, V_0, K_1, V_1, ... in the slots; K is the
// K-major and V the MN-major B operand of the same layout.
#include "fcc_paged.cuh"

#include <cuda_bf16.h>

#include <algorithm>
#include <climits>

namespace fcc {
namespace {

constexpr int kTileRows = 128;
constexpr int kPairRows = 256;
constexpr int kBlock = 128;                    // positions of a block
constexpr int kSlots = 4;
constexpr int kCols = 4;                       // blocks whose column constants are kept
constexpr uint32_t kAtom = 128 * 128;
constexpr float kRaise = 8.f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;                // S_t at 128 t, O_t at 256 + 128 t
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;
constexpr int kThreads = 512;                  // 16 warps: 8 softmax, 4 loading, 1 issuing, 3 idle
// Registers: 512 x 128 at launch = 256 x 192 + 128 x 72 + 128 x 56 afterwards.
constexpr int kRegsSoftmax = 192, kRegsLoad = 72, kRegsIssue = 56;
static_assert(256 * kRegsSoftmax + 128 * kRegsLoad + 128 * kRegsIssue == kThreads * 128);
constexpr int kMaxCtas = 512;

struct Start {                                 // where a CTA's run begins
  int b, rh, pair, j;
};
struct Header {                                // of the item that a CTA begins last and does not finish
  int parts, b, rh, pair;
};

// Workspace: the plan's totals, the runs' starts, the headers, the sequences'
// blocks, then two partial results for each CTA.
struct Layout {
  size_t starts, headers, units, parts, part_bytes, total;
};
__host__ __device__ inline Layout layout_of(int64_t d, int B, int ctas) {
  Layout l;
  l.starts = 256;
  l.headers = l.starts + static_cast<size_t>(ctas) * sizeof(Start);
  l.units = l.headers + static_cast<size_t>(ctas) * sizeof(Header);
  l.parts = (l.units + static_cast<size_t>(B) * 8 + 255) & ~size_t{255};
  l.part_bytes = kPairRows * static_cast<size_t>(d + 2) * 4;   // references, sums, [D / 4][256] float4
  l.total = l.parts + 2 * static_cast<size_t>(ctas) * l.part_bytes;
  return l;
}
struct Totals {                                // at the workspace's start
  long long units;
  int ctas;
};

__device__ __forceinline__ int pairs_of(const PagedArgs& a, const Seq& q) {
  return static_cast<int>((static_cast<long long>(q.n) * a.G + kPairRows - 1) / kPairRows);
}

// Blocks [j0, j1) that rows [first, last] of a sequence see.
struct Range {
  int j0, j1;
};
__device__ __forceinline__ Range blocks_of(const PagedArgs& a, const Seq& q, long long first, long long last) {
  if (!q.ok) return Range{0, 1};               // (one, of which nothing is seen)
  const int p0 = q.L - q.n + static_cast<int>(first / a.G), p1 = q.L - q.n + static_cast<int>(last / a.G);
  return Range{max(0, p0 - a.window + 1) / kBlock, p1 / kBlock + 1};
}
__device__ __forceinline__ Range pair_blocks(const PagedArgs& a, const Seq& q, int pair) {
  const long long first = static_cast<long long>(pair) * kPairRows;
  return blocks_of(a, q, first, min(static_cast<long long>(q.n) * a.G, first + kPairRows) - 1);
}

constexpr int kPlanThreads = 1024;
constexpr int kFewPairs = 8;                   // up to here a thread counts a sequence's blocks alone

// Counts the blocks of all items and finds where each CTA's run begins.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PagedArgs a, int grid) {
  __shared__ long long s_scan[32], s_off[kMaxCtas];
  __shared__ int s_b[kMaxCtas];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Layout lay = layout_of(a.pool.d, a.step.B, grid);
  long long* units = reinterpret_cast<long long*>(a.ws + lay.units);
  const long long rh = static_cast<long long>(a.R) * a.pool.H;
  long long np_all = 0;
  for (int b0 = warp * 32; b0 < a.step.B; b0 += kPlanThreads) {
    const int b = b0 + lane;
    Seq q{0, 0, 0, false, false};
    int np = 0;
    long long n = 0;
    if (b < a.step.B) {
      q = load_seq(a.step, b);
      if (!q.ok) record_invalid(a.status);
      np = pairs_of(a, q);
      np_all += np;
      if (np <= kFewPairs)
        for (int p = 0; p < np; ++p) {
          const Range g = pair_blocks(a, q, p);
          n += g.j1 - g.j0;
        }
    }
    for (unsigned m = __ballot_sync(0xffffffffu, np > kFewPairs); m != 0; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const Seq o = load_seq(a.step, b0 + src);
      const int onp = pairs_of(a, o);
      long long sum = 0;
      for (int p = lane; p < onp; p += 32) {
        const Range g = pair_blocks(a, o, p);
        sum += g.j1 - g.j0;
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
  if (mine > 0) {
    // runs c with from <= c total / ctas < from + mine
    long long c = (from * ctas + total - 1) / total;
    while (c > 0 && (c - 1) * total / ctas >= from) --c;
    while (c * total / ctas < from) ++c;
    long long at = from;
    int b = b_first;
    for (; c < ctas; ++c) {
      const long long u = c * total / ctas;
      if (u >= from + mine) break;
      while (u >= at + units[b]) at += units[b++];
      s_b[c] = b;
      s_off[c] = u - at;
    }
  }
  __syncthreads();
  Start* starts = reinterpret_cast<Start*>(a.ws + lay.starts);
  for (int c = warp; c < ctas; c += 32) {
    const int b = s_b[c];
    const long long each = units[b] / rh;
    long long rest = s_off[c] % each;
    const Seq q = load_seq(a.step, b);
    const int np = pairs_of(a, q);
    for (int p0 = 0; p0 < np; p0 += 32) {
      const int p = p0 + lane;
      int n = 0;
      if (p < np) {
        const Range g = pair_blocks(a, q, p);
        n = g.j1 - g.j0;
      }
      int incl = n;
#pragma unroll
      for (int s = 1; s < 32; s *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += v;
      }
      const unsigned m = __ballot_sync(0xffffffffu, rest < incl);
      if (m != 0) {
        if (lane == __ffs(m) - 1)
          starts[c] = Start{b, static_cast<int>(s_off[c] / each), p, static_cast<int>(rest - (incl - n))};
        break;
      }
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (threadIdx.x == 0) *reinterpret_cast<Totals*>(a.ws) = Totals{total, static_cast<int>(ctas)};
}

// A walk over a CTA's run: item after item, each from block ja to block jb.
struct Walk {
  int b, rh, pair, pairs;
  Seq q;
  int j0, j1;                                  // the item's blocks
  int ja, jb;                                  // the CTA's part of them
  long long left;                              // blocks of the CTA behind this item's
  int lo[2], hi[2];                            // tile t's blocks of [ja, jb): none if lo >= hi

  __device__ __forceinline__ void take(const PagedArgs& a, int skip) {
    const long long rows = static_cast<long long>(q.n) * a.G, first = static_cast<long long>(pair) * kPairRows;
    const Range g = pair_blocks(a, q, pair);
    j0 = g.j0;
    j1 = g.j1;
    ja = j0 + skip;
    const int n = static_cast<int>(min(static_cast<long long>(j1 - ja), left));
    jb = ja + n;
    left -= n;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const long long r0 = first + t * kTileRows;
      lo[t] = hi[t] = 0;
      if (r0 >= rows) continue;
      const Range s = blocks_of(a, q, r0, min(rows, r0 + kTileRows) - 1);
      lo[t] = max(ja, s.j0);
      hi[t] = min(jb, s.j1);
    }
  }
  __device__ __forceinline__ bool begin(const PagedArgs& a, const Start& s, long long units) {
    b = s.b;
    rh = s.rh;
    pair = s.pair;
    q = load_seq(a.step, b);
    pairs = pairs_of(a, q);
    left = units;
    if (left <= 0) return false;
    take(a, s.j);
    return true;
  }
  __device__ __forceinline__ bool next_item(const PagedArgs& a) {
    if (left <= 0) return false;
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
    take(a, 0);
    return true;
  }
  __device__ __forceinline__ bool sees(int j, int t) const { return j >= lo[t] && j < hi[t]; }
  // Tile t has a block here.  Where it has none, its softmax warps and the issuing
  // warp pass the item without a word: a barrier's phases stay one to an exchange.
  __device__ __forceinline__ bool active(int t) const { return lo[t] < hi[t]; }
  __device__ __forceinline__ int rank(const PagedArgs& a) const { return rh / a.pool.H; }
  __device__ __forceinline__ int head(const PagedArgs& a) const { return rh % a.pool.H; }
};

// Column constants of a block: for position i its key's power 2^a, its value's
// exponent b and 2^-b; which positions the pages hold.
struct Columns {
  float ka[kBlock], vb[kBlock], vi[kBlock];
  uint32_t there[4];
};

constexpr int kBars = 2 * kSlots + kCols + 2 + 2 + 2 + 2 + 1;

template <int D>
constexpr uint32_t kTileBytes = (D / 64) * kAtom;
template <int D>
constexpr int kSmem = 1024 + (2 + kSlots) * static_cast<int>(kTileBytes<D>) + kCols * static_cast<int>(sizeof(Columns)) + kBars * 8 + 16;
static_assert(kSmem<128> <= 232448, "shared memory per CTA");

__device__ __forceinline__ uint64_t desc_kmajor(uint32_t base, int kk) {
  return ptx::smem_desc_sw128(base + (kk >> 2) * kAtom + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t base, int kk) {
  return ptx::smem_desc_sw128(base + kk * 2048, kAtom, 1024);
}
// The byte of 16-byte chunk `chunk` (8 values) of a tile's row.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (chunk >> 3) * kAtom + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
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

// 32 scores of a row: y = t - ref for columns col .. col + 31, and p = 2^y as 16-bit
// pairs.  MASK: columns whose bit in `seen` is clear get p = 0.
template <bool E4M3, bool MASK>
__device__ __forceinline__ void exponentials(const uint32_t (&x)[32], float c, float ref, const Columns& cc, int col,
                                             uint32_t seen, uint32_t* pk, uint64_t (&l2)[4], float (&mx)[4]) {
  const uint64_t c2 = ptx::f32x2_pack(c, c), r2 = ptx::f32x2_pack(-ref, -ref);
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    float4 ka, vb, vi;
    if constexpr (E4M3) {
      ka = *reinterpret_cast<const float4*>(&cc.ka[col + k]);
      vb = *reinterpret_cast<const float4*>(&cc.vb[col + k]);
      vi = *reinterpret_cast<const float4*>(&cc.vi[col + k]);
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t x2 = ptx::f32x2_pack(__uint_as_float(x[k + i]), __uint_as_float(x[k + i + 1]));
      uint64_t y2;
      if constexpr (E4M3) {
        const uint64_t ka2 = i == 0 ? ptx::f32x2_pack(ka.x, ka.y) : ptx::f32x2_pack(ka.z, ka.w);
        const uint64_t vb2 = i == 0 ? ptx::f32x2_pack(vb.x, vb.y) : ptx::f32x2_pack(vb.z, vb.w);
        y2 = ptx::f32x2_fma(ptx::f32x2_mul(x2, c2), ka2, ptx::f32x2_add(vb2, r2));
      } else {
        y2 = ptx::f32x2_fma(x2, c2, r2);
      }
      float y0, y1;
      ptx::f32x2_unpack(y2, y0, y1);
      if constexpr (MASK) {
        if (!(seen >> (k + i) & 1)) y0 = -INFINITY;
        if (!(seen >> (k + i + 1) & 1)) y1 = -INFINITY;
      }
      const int n = (k + i) / 2 & 3;
      mx[n] = ptx::max3(mx[n], y0, y1);
      const float p0 = ptx::ex2_approx(y0), p1 = ptx::ex2_approx(y1);
      if constexpr (E4M3)
        l2[n] = ptx::f32x2_fma(ptx::f32x2_pack(p0, p1), i == 0 ? ptx::f32x2_pack(vi.x, vi.y) : ptx::f32x2_pack(vi.z, vi.w), l2[n]);
      else
        l2[n] = ptx::f32x2_add(l2[n], ptx::f32x2_pack(p0, p1));
      pk[(k + i) / 2] = pack16<E4M3>(p0, p1);
    }
  }
}

__device__ __forceinline__ float sum4(const uint64_t (&v)[4]) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    ptx::f32x2_unpack(v[i], a, b);
    s[i] = a + b;
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The place of column group c4 (4 values) of a row in a partial result.
__device__ __forceinline__ float4* part_at(char* part, int c4, int row) {
  return reinterpret_cast<float4*>(part + kPairRows * 8) + c4 * kPairRows + row;
}

// One row over positions [from, to], computed again by a warp from the definition:
// lanes hold D / 32 columns each.  Rows whose sums are not finite come here, because
// in a product with P = 0 a value that is not finite reaches rows that do not see it.
template <int D, bool E4M3>
__device__ __forceinline__ void row_again(const PagedArgs& a, int b, int r, int h, int head, int64_t t, int from, int to, int lane,
                                       float (&o)[D / 32], float& ref, float& l) {
  constexpr int N = D / 32;
  float x[N];
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.Q[r]) + t * a.ldq + static_cast<int64_t>(head) * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __bfloat162float(src[i]);
    o[i] = 0.f;
  }
  ref = -INFINITY;
  l = 0.f;
  for (int64_t j = from; j <= to; ++j) {
    const int page = page_of(a.step, a.pool.pages, b, static_cast<int>(j >> a.pool.log2P));
    if (page < 0) continue;
    const int64_t row = ((static_cast<int64_t>(page) * a.pool.H + h) << a.pool.log2P) + (j & ((1 << a.pool.log2P) - 1));
    float k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = row * D + lane * N + i;
      if constexpr (E4M3) {
        const float fk = __int_as_float(a.pool.Ke[r][row] << 23), fv = __int_as_float(a.pool.Ve[r][row] << 23);
        k[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(a.pool.K[r][at]), __NV_E4M3))) * fk;
        v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(a.pool.V[r][at]), __NV_E4M3))) * fv;
      } else {
        k[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.pool.K[r])[at]);
        v[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.pool.V[r])[at]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], k[i], s);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= a.scale_log2;
    const float top = fmaxf(ref, s);
    const float f = ex2_from(ref, top), e = ex2_from(s, top);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + (s == -INFINITY ? 0.f : e * v[i]);
    ref = top;
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ PagedArgs a, unsigned long long timeout_ns) {
  constexpr uint32_t kTile = kTileBytes<D>;
  constexpr uint32_t kFormat = E4M3 ? 0u : (1u << 7) | (1u << 10);   // f16 or bf16 operands
  constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);
  constexpr uint32_t kIdescS = (ptx::idesc_bf16_f32(kTileRows, kBlock, false, false) & ~kBf16) | kFormat;
  constexpr uint32_t kIdescO = (ptx::idesc_bf16_f32(kTileRows, D, false, true) & ~kBf16) | kFormat;
  constexpr float kOff = E4M3 ? 6.f : 0.f;     // p up to 2^14 in f16, see fcc_paged.cu

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sR = sQ + 2 * kTile;
  Columns* cols = reinterpret_cast<Columns*>(sR + kSlots * kTile);
  uint64_t* r_full = reinterpret_cast<uint64_t*>(cols + kCols);  // [kSlots], four loading warps
  uint64_t* r_empty = r_full + kSlots;         // [kSlots]
  uint64_t* c_full = r_empty + kSlots;         // [kCols], four loading warps
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
    for (int i = 0; i < kCols; ++i) ptx::mbar_init(&c_full[i], 4);
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
  if (warp == 12) {
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
  const Layout lay = layout_of(D, a.step.B, gridDim.x);
  const Totals tot = *reinterpret_cast<const Totals*>(a.ws);
  Header* const headers = reinterpret_cast<Header*>(a.ws + lay.headers);
  if (threadIdx.x == 0) headers[blockIdx.x] = Header{0, 0, 0, 0};
  const bool busy = static_cast<int>(blockIdx.x) < tot.ctas;
  const long long u0 = busy ? blockIdx.x * tot.units / tot.ctas : 0;
  const long long u1 = busy ? (blockIdx.x + 1) * tot.units / tot.ctas : 0;
  const Start start = busy ? reinterpret_cast<const Start*>(a.ws + lay.starts)[blockIdx.x] : Start{0, 0, 0, 0};

  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, W.wait(bar, parity) ? 1 : 0) != 0;
  };

  if (warp >= 12) {
    // ----------------------------------------------------------- MMA issue
    regs_dec<kRegsIssue>();
    if (warp == 12 && lane == 0 && busy) {
      Walk w;
      bool any = false, ok = true;
      bool more = w.begin(a, start, u1 - u0);
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
      uint32_t u = 0;                          // ring position of the item's first K
      while (more && ok) {
        bool first[2] = {true, true};          // O_t holds nothing of this item yet
        uint32_t pend[2] = {0, 0};                      // ring position of the V whose product is next
        bool pending[2] = {false, false};
        for (int t = 0; t < 2 && ok; ++t)
          if (w.active(t)) ok = W.wait(&q_full[t], nq[t]++ & 1u);
        auto issue_pv = [&](int t) -> bool {
          const uint32_t pos = pend[t];
          pending[t] = false;
          if (!W.wait(&r_full[pos % kSlots], (pos / kSlots) & 1u)) return false;
          if (!W.wait(&p_full[t], np[t] & 1u)) return false;
          ++np[t];
          ptx::tc_fence_after();
          const uint32_t va = ptx::smem_addr(sR + (pos % kSlots) * kTile);
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            ptx::mma_f16_tmem_a(tmem_base + kColO + t * 128, tmem_base + t * 128 + kk * 8, desc_mnmajor(va, kk), kIdescO,
                                (!first[t] || kk > 0) ? 1u : 0u);
          first[t] = false;
          any = true;
          return true;
        };
        for (int j = w.ja; j < w.jb && ok; ++j, u += 2) {
          if (!(ok = W.wait(&r_full[u % kSlots], (u / kSlots) & 1u))) break;
          ptx::tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && pending[t]) ok = issue_pv(t);
            if (ok && w.sees(j, t)) {
              const uint32_t qa = ptx::smem_addr(sQ + t * kTile), ka = ptx::smem_addr(sR + (u % kSlots) * kTile);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                ptx::mma_f16(tmem_base + t * 128, desc_kmajor(qa, kk), desc_kmajor(ka, kk), kIdescS, kk > 0 ? 1u : 0u);
              ptx::mma_commit(&s_full[t]);
              any = true;
              pending[t] = true;
              pend[t] = u + 1;
            }
          }
          if (!ok) break;
          // K_j is free once both tiles' S are done, V_{j-1} once both P V are
          ptx::mma_commit(&r_empty[u % kSlots]);
          if (j > w.ja) ptx::mma_commit(&r_empty[(u - 1) % kSlots]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && pending[t]) ok = issue_pv(t);
        if (ok) {
          // (a V that no tile's last block used has to have arrived all the same)
          ok = W.wait(&r_full[(u - 1) % kSlots], ((u - 1) / kSlots) & 1u);
          ptx::mma_commit(&r_empty[(u - 1) % kSlots]);
          for (int t = 0; t < 2; ++t)
            if (w.active(t)) ptx::mma_commit(&o_full[t]);
          any = true;
        }
        more = ok && w.next_item(a);
      }
      if (any) {
        ptx::mma_commit(mma_done);
        W.drain(mma_done, 0, kDrainNs);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------- loading
    // Warp 8 + i brings positions 32 i .. 32 i + 31 of each block.  A lane looks up
    // one of them, a block ahead.
    regs_dec<kRegsLoad>();
    const int wl = warp - 8;
    constexpr int kRow = D * (E4M3 ? 1 : 2), kLanes = kRow / 16, kAtOnce = 32 / kLanes, kN = 32 / kAtOnce;
    const int chunk = lane % kLanes;
    if (busy) {
      Walk w;
      bool more = w.begin(a, start, u1 - u0);
      int j = w.ja;                            // the block that is looked up next
      int page = -1, in_page = 0, nr = 0, nh = 0;
      bool have = false;                       // a block has been looked up
      auto look_up = [&]() {
        have = more;
        page = -1;
        if (!more) return;
        const long long rows = min(static_cast<long long>(w.q.n) * a.G, (w.pair + 1ll) * kPairRows);
        const int last = w.q.ok ? w.q.L - w.q.n + static_cast<int>((rows - 1) / a.G) : -1;
        const long long pos = static_cast<long long>(j) * kBlock + 32 * wl + lane;
        nr = w.rank(a);
        nh = w.head(a);
        if (pos <= last) {
          page = page_of(a.step, a.pool.pages, w.b, static_cast<int>(pos >> a.pool.log2P));
          in_page = static_cast<int>(pos) & ((1 << a.pool.log2P) - 1);
          // (positions before every row's window were given back, perhaps)
          if (page < 0 && pos > static_cast<long long>(w.q.L - w.q.n + static_cast<int>(static_cast<long long>(w.pair) * kPairRows / a.G)) - a.window)
            record_invalid(a.status);
        }
        if (++j == w.jb) {
          more = w.next_item(a);
          j = w.ja;
        }
      };
      look_up();
      uint32_t u = 0;
      bool ok = true;
      while (have && ok) {
        const int64_t row = page < 0 ? -1 : ((static_cast<int64_t>(page) * a.pool.H + nh) << a.pool.log2P) + in_page;
        const int r = nr;
        const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
        uint32_t ke = 127, ve = 127;
        if constexpr (E4M3) {
          if (row >= 0) {
            ke = a.pool.Ke[r][row];
            ve = a.pool.Ve[r][row];
          }
        }
        uint4 x[kN];
        auto fetch = [&](const char* pool) {   // e4m3: into registers
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            const int64_t src = __shfl_sync(0xffffffffu, row, i * kAtOnce + lane / kLanes);
            x[i] = make_uint4(0, 0, 0, 0);
            if (src >= 0) x[i] = *reinterpret_cast<const uint4*>(pool + src * kRow + chunk * 16);
          }
        };
        if constexpr (E4M3) fetch(a.pool.K[r]);
        look_up();
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++u) {
          const uint32_t slot = u % kSlots;
          if (!(ok = wait_warp(&r_empty[slot], ((u / kSlots) & 1u) ^ 1u))) break;
          if (kv == 0) {
            // (the block that used these constants four blocks ago is done: its
            // products were issued before the slot's last occupant was handed back)
            const uint32_t blk = u / 2;
            Columns& cc = cols[blk % kCols];
            if constexpr (E4M3) {
              const int ev = min(static_cast<int>(ve), 254), i = 32 * wl + lane;
              cc.ka[i] = __int_as_float(static_cast<int>(ke) << 23);
              cc.vb[i] = static_cast<float>(ev - 127);
              cc.vi[i] = __int_as_float((254 - ev) << 23);
            }
            if (lane == 0) cc.there[wl] = there;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&c_full[blk % kCols]);
          }
          uint8_t* dst = sR + slot * kTile;
          if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const int tok = 32 * wl + i * kAtOnce + lane / kLanes;
              uint4 lo, hi;
              lo.x = f16x2_of_e4m3(x[i].x);
              lo.y = f16x2_of_e4m3(x[i].x >> 16);
              lo.z = f16x2_of_e4m3(x[i].y);
              lo.w = f16x2_of_e4m3(x[i].y >> 16);
              hi.x = f16x2_of_e4m3(x[i].z);
              hi.y = f16x2_of_e4m3(x[i].z >> 16);
              hi.z = f16x2_of_e4m3(x[i].w);
              hi.w = f16x2_of_e4m3(x[i].w >> 16);
              *reinterpret_cast<uint4*>(dst + tile_at(tok, 2 * chunk)) = lo;
              *reinterpret_cast<uint4*>(dst + tile_at(tok, 2 * chunk + 1)) = hi;
            }
            if (kv == 0) fetch(a.pool.V[r]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&r_full[slot]);
          } else {
            const char* pool = kv == 0 ? a.pool.K[r] : a.pool.V[r];
            const uint32_t d32 = ptx::smem_addr(dst);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const int tok = i * kAtOnce + lane / kLanes;
              const int64_t src = __shfl_sync(0xffffffffu, row, tok);
              cp_async16(d32 + tile_at(32 * wl + tok, chunk), pool + max(src, static_cast<int64_t>(0)) * kRow + chunk * 16, src >= 0);
            }
            cp_async_commit();
            // the slot filled two steps ago: every lane's loads have arrived
            if (u >= 2) {
              cp_async_wait<2>();
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(&r_full[(u - 2) % kSlots]);
            }
          }
        }
      }
      if constexpr (!E4M3) {
        cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (ok && lane == 0)
          for (uint32_t v = u >= 2 ? u - 2 : 0; v < u; ++v) ptx::mbar_arrive(&r_full[v % kSlots]);
      }
    }
  } else {
    // ------------------------------------------------- softmax and output
    regs_inc<kRegsSoftmax>();
    const int t = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;       // of the tile
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_addr = lane_addr + t * 128;
    const uint32_t o_addr = lane_addr + kColO + t * 128;
    uint32_t ns = 0, items = 0, blk0 = 0;      // this tile's blocks and items, the CTA's blocks before this item
    bool ok = true;
    Walk w;
    bool more = busy && w.begin(a, start, u1 - u0);
    float c = 0.f;                             // what a score is multiplied by
    long long at = u0;
    // This thread's row of a new item's Q_t; its place among the token rows.
    int64_t token = 0;
    int head = 0, qpos = -1;
    bool live = false;
    auto load_q = [&]() {
      const long long rho = static_cast<long long>(w.pair) * kPairRows + t * kTileRows + row;
      live = rho < static_cast<long long>(w.q.n) * a.G;
      const int i = static_cast<int>(rho / a.G);
      token = static_cast<int64_t>(w.q.s) + i;
      head = w.head(a) * a.G + static_cast<int>(rho % a.G);
      qpos = live && w.q.ok ? w.q.L - w.q.n + i : -1;
      if (!w.active(t)) return;
      const char* src = a.Q[w.rank(a)] + (token * a.ldq + static_cast<int64_t>(head) * D) * 2;
      uint8_t* dst = sQ + t * kTile;
      c = a.scale_log2;
      float f = 1.f;
      if constexpr (E4M3) {
        unsigned top = 0;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 v = live ? *reinterpret_cast<const uint4*>(src + k * 16) : make_uint4(0, 0, 0, 0);
          for (uint32_t y : {v.x, v.y, v.z, v.w}) {
            const unsigned m0 = y & 0x7fffu, m1 = (y >> 16) & 0x7fffu;
            top = max(top, max(m0 < 0x7f80u ? m0 : 0u, m1 < 0x7f80u ? m1 : 0u));
          }
        }
        const int e = max(static_cast<int>(top >> 7) - 127, -100) - 14;
        f = power_of_two(-e);
        c *= power_of_two(e);
      }
#pragma unroll 4
      for (int k = 0; k < D / 8; ++k) {
        uint4 v = live ? *reinterpret_cast<const uint4*>(src + k * 16) : make_uint4(0, 0, 0, 0);
        if constexpr (E4M3) {
          auto f16 = [&](uint32_t y) {
            return pack_f16x2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xffff0000u) * f);
          };
          v = make_uint4(f16(v.x), f16(v.y), f16(v.z), f16(v.w));
        }
        *reinterpret_cast<uint4*>(dst + tile_at(row, k)) = v;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&q_full[t]);
    };
    if (more) load_q();
    while (more && ok) {
      float ref = -INFINITY, l = 0.f;
      int n = 0;
      for (int j = w.lo[t]; j < w.hi[t]; ++j) {
        const uint32_t blk = blk0 + (j - w.ja);
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
        const bool whole = cmin == 0 && cmax >= kBlock - 1 && (there.x & there.y & there.z & there.w) == 0xffffffffu;
        auto seen = [&](int k) -> uint32_t {   // columns 32 k .. 32 k + 31
          const int hi = cmax - 32 * k, lo = cmin - 32 * k;
          uint32_t m = k == 0 ? there.x : k == 1 ? there.y : k == 2 ? there.z : there.w;
          m &= hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1;
          return m & (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1));
        };
        uint32_t vb[2][32];
        bool done = false;
        if (n > 0 && __all_sync(0xffffffffu, (whole && ref != -INFINITY) || !live)) {
          // A whole block is exponentiated against the reference as it stands while the
          // next 32 columns come from TMEM; only a maximum that calls for a raise starts over.
          uint64_t l2[4] = {0, 0, 0, 0};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          uint32_t pk[64];
          const float sub = live ? ref : 0.f;
          ptx::tmem_ld_32x32b_x32(s_addr, vb[0]);
          tmem_ld_wait_regs(vb[0]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < 3) ptx::tmem_ld_32x32b_x32(s_addr + 32 * (k + 1), vb[(k + 1) & 1]);
            exponentials<E4M3, false>(vb[k & 1], c, sub, cc, 32 * k, 0, pk + 16 * k, l2, mx);
            if (k < 3) tmem_ld_wait_regs(vb[(k + 1) & 1]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          if (!__any_sync(0xffffffffu, live && top > kOff + kRaise)) {
            ptx::tmem_st_32x32b_x32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(pk));
            ptx::tmem_st_32x32b_x32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
            l += sum4(l2);
            done = true;
          }
        }
        if (!done) {
          // The maximum first, then the exponentials, in two passes over S.
          float top = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            ptx::tmem_ld_32x32b_x32(s_addr + 32 * k, vb[0]);
            tmem_ld_wait_regs(vb[0]);
            const uint32_t m = seen(k);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float y = __uint_as_float(vb[0][i]) * c;
              if constexpr (E4M3) y = fmaf(y, cc.ka[32 * k + i], cc.vb[32 * k + i]);
              if (m >> i & 1) top = fmaxf(top, y);
            }
          }
          const bool raise = top > ref + (kOff + kRaise);
          const float ref_new = raise ? top - kOff : ref;
          const float f = raise ? ex2_from(ref, ref_new) : 1.f;
          ref = ref_new;
          l *= f;
          const float sub = ref == -INFINITY ? 0.f : ref;
          uint64_t l2[4] = {0, 0, 0, 0};
          float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t pk[16];
            ptx::tmem_ld_32x32b_x32(s_addr + 32 * k, vb[0]);
            tmem_ld_wait_regs(vb[0]);
            exponentials<E4M3, true>(vb[0], c, sub, cc, 32 * k, seen(k), pk, l2, mx);
            // (P's columns 16 k .. 16 k + 15 lie over scores already read)
            ptx::tmem_st_32x32b_x16(s_addr + 16 * k, pk);
          }
          l += sum4(l2);
          // S_t was issued after the last P_t V: O_t has no product in flight
          if (n > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              ptx::tmem_ld_32x32b_x32(o_addr + k, vb[0]);
              tmem_ld_wait_regs(vb[0]);
#pragma unroll
              for (int i = 0; i < 32; ++i) vb[0][i] = __float_as_uint(__uint_as_float(vb[0][i]) * f);
              ptx::tmem_st_32x32b_x32(o_addr + k, vb[0]);
            }
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&p_full[t]);
        ++n;
      }
      if (!ok) break;
      // The next item's queries: this tile's S are all complete.
      const Walk cur = w;
      const int64_t o_token = token;
      const int o_head = head, o_qpos = qpos;
      const bool o_live = live;
      more = w.next_item(a);
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
      char* part = a.ws + lay.parts + static_cast<size_t>(2 * blockIdx.x + (cur.ja == cur.j0 ? 1 : 0)) * lay.part_bytes;
      const int prow = t * kTileRows + row;
      const bool none = l == 0.f;
      const float inv = complete ? (none ? 0.f : 1.f / l) : 1.f;
      char* dst = a.O[r] + (o_token * a.ldo + static_cast<int64_t>(o_head) * D) * 2;
      bool odd = !(fabsf(l) < INFINITY);
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t v[32];
        if (n > 0) {                           // (the same for the whole tile)
          ptx::tmem_ld_32x32b_x32(o_addr + k, v);
          tmem_ld_wait_regs(v);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = n > 0 && !none ? __uint_as_float(v[i]) * inv : 0.f;
          odd |= n > 0 && !(fabsf(__uint_as_float(v[i])) < INFINITY);
          v[i] = __float_as_uint(y);
        }
        if (!o_live) continue;
        if (complete) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 y;
            y.x = ptx::pack_bf16x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            y.y = ptx::pack_bf16x2(__uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
            y.z = ptx::pack_bf16x2(__uint_as_float(v[i + 4]), __uint_as_float(v[i + 5]));
            y.w = ptx::pack_bf16x2(__uint_as_float(v[i + 6]), __uint_as_float(v[i + 7]));
            *reinterpret_cast<uint4*>(dst + (k + i) * 2) = y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *part_at(part, (k + i) / 4, prow) = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                                            __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
        }
      }
      for (unsigned m = __ballot_sync(0xffffffffu, odd && o_live); m != 0; m &= m - 1) {
        const int src = __ffs(m) - 1;
        const int64_t tok = __shfl_sync(0xffffffffu, o_token, src);
        const int hd = __shfl_sync(0xffffffffu, o_head, src), p = __shfl_sync(0xffffffffu, o_qpos, src);
        const int from = static_cast<int>(max(static_cast<long long>(cur.ja) * kBlock, static_cast<long long>(p) - a.window + 1));
        const int to = static_cast<int>(min(static_cast<long long>(cur.jb) * kBlock - 1, static_cast<long long>(p)));
        float o[D / 32], ref1, l1;
        row_again<D, E4M3>(a, cur.b, r, cur.head(a), hd, tok, from, to, lane, o, ref1, l1);
        const int prow1 = t * kTileRows + quarter * 32 + src;
        const float inv1 = l1 == 0.f ? 0.f : 1.f / l1;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int col = lane * (D / 32) + i;
          if (complete)
            reinterpret_cast<__nv_bfloat16*>(a.O[r])[tok * a.ldo + static_cast<int64_t>(hd) * D + col] = __float2bfloat16(o[i] * inv1);
          else
            reinterpret_cast<float*>(part_at(part, col >> 2, prow1))[col & 3] = o[i];
        }
        if (lane == src) {
          ref = ref1;
          l = l1;
        }
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
          const long long last = at + (cur.j1 - cur.j0);
          headers[blockIdx.x] = Header{static_cast<int>((last * tot.ctas - 1) / tot.units) - static_cast<int>(blockIdx.x) + 1,
                                       cur.b, cur.rh, cur.pair};
        }
      }
      at += cur.jb - cur.ja;
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
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
  const long long rho = static_cast<long long>(hd.pair) * kPairRows + row;
  if (rho >= static_cast<long long>(q.n) * a.G) return;
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
  const int r = hd.rh / a.pool.H, head = hd.rh % a.pool.H * a.G + static_cast<int>(rho % a.G);
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

template <int D, bool E4M3>
cudaError_t launch(const PagedArgs& a, int ctas, unsigned long long timeout_ns, cudaStream_t st) {
  static bool attr_set[64] = {};
  cudaError_t e = smem_attr_once(attr_set, tiles_kernel<D, E4M3>, kSmem<D>);
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1u, a, ctas)) != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(ctas);
  if ((e = launch_pdl(tiles_kernel<D, E4M3>, dim3(grid), dim3(kThreads), kSmem<D>, st, 1u, a, timeout_ns)) != cudaSuccess) return e;
  return launch_pdl(join_kernel<D>, dim3(grid, D / 16), dim3(kPairRows), 0, st, 1u, a);
}

}  // namespace

size_t tiles_ws_bytes(int64_t d, int B, int ctas) { return layout_of(d, B, std::min(ctas, kMaxCtas)).total; }

cudaError_t launch_tiles(const PagedArgs& a, bool e4m3, int ctas, unsigned long long timeout_ns, cudaStream_t st) {
  ctas = std::min(ctas, kMaxCtas);
  return a.pool.d == 128 ? (e4m3 ? launch<128, true>(a, ctas, timeout_ns, st) : launch<128, false>(a, ctas, timeout_ns, st))
                         : (e4m3 ? launch<64, true>(a, ctas, timeout_ns, st) : launch<64, false>(a, ctas, timeout_ns, st));
}

}  // namespace fcc
