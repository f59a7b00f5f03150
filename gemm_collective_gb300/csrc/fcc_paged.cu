// fcc_paged.cu -- attention of a step's rows over the paged key/value cache: the
// entry point, and the kernel for few rows to a sequence and head (decoding).
//
// With few rows every byte of the cache is used once or twice, so DRAM bounds the
// kernel: it is built to keep loads in flight and every SM busy.
//
//  * The work is the list of all (sequence, rank, head, 16 rows) items, each a
//    run of units of 8 kTok positions.  The list is cut into as many equal runs of
//    units as there are CTAs (one to an SM), wherever the cuts fall: sequences of all
//    lengths, or a single long one, load all SMs alike.  An item that a cut goes
//    through leaves partial sums (O, its reference exponent and l) in the
//    workspace, at most two from a CTA, and combine_kernel adds an item's in order.
//  * A unit is 8 slices of kTok positions, one for each warp.  A warp has a ring of
//    kStages slices of its own in shared memory, filled by its own cp.async, and
//    runs through the positions without ever waiting for another warp; the
//    loads run ahead over the ends of items.  Any page size works: a
//    position's place is looked up for itself, one slice before its loads.
//  * S = Q K^T and O += P V on m16n8k16 products of the warp: 16 query rows (a
//    group's heads, and a few tokens).  At 23 bytes a clock and SM these run
//    at a fraction of their rate; tensor memory would only add its round trip.
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

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kHalf = 4096;                    // bytes of a slice's keys (and of its values)
constexpr float kRaise = 8.f;                  // the reference is raised past this (log2 units)
constexpr int kRowTile = 16;

// Partial sums of an item: 16 references, 16 sums, 16 x D values as the threads hold them.
template <int D>
constexpr int kPartFloats = 2 * kRowTile + kRowTile * D;

struct Header {                                // of the item whose first part CTA c holds last
  int parts;                                   // CTAs from c on (0: none)
  int b, item;
};

__host__ __device__ inline size_t header_bytes(int ctas) { return (static_cast<size_t>(ctas) * sizeof(Header) + 255) & ~size_t{255}; }

template <int D, bool E4M3>
struct Few {
  static constexpr int kRow = D * (E4M3 ? 1 : 2);        // bytes of a position's key
  static constexpr int kTok = kHalf / kRow;              // positions of a slice: 16, 32 or 64
  static constexpr int kUnit = kWarps * kTok;
  static constexpr int kLanes = kRow / 16;               // lanes that load a row
  static constexpr int kRowsAtOnce = 32 / kLanes;
  static constexpr int kPer = (kTok + 31) / 32;          // positions that a lane looks up
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
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A walk over a CTA's run of units: item after item, each from unit k to unit end.
struct Walk {
  int b, item, k, end;
  Seq q;
  int first;         // the first position of unit 0
  int nk;            // units of each of the sequence's items
  int tiles;         // tiles of 16 rows
  int items;         // R * H * tiles
  long long left;    // units of the CTA behind this item's

  // What sequence `seq` has to do (units of all its items).
  template <int kUnit>
  __device__ __forceinline__ long long measure(const PagedArgs& a, int seq) {
    b = seq;
    q = load_seq(a.step, seq);
    tiles = static_cast<int>((static_cast<long long>(q.n) * a.G + kRowTile - 1) / kRowTile);
    items = a.R * a.pool.H * tiles;
    first = max(0, q.L - q.n - a.window + 1);
    nk = q.ok ? static_cast<int>((static_cast<long long>(q.L) - first + kUnit - 1) / kUnit) : 1;
    return static_cast<long long>(items) * nk;
  }
  __device__ __forceinline__ void take() {
    const int n = static_cast<int>(min(static_cast<long long>(nk - k), left));
    end = k + n;
    left -= n;
  }
  template <int kUnit>
  __device__ __forceinline__ bool next_item(const PagedArgs& a) {
    if (left <= 0) return false;
    if (++item == items) {
      item = 0;
      do {
        if (b + 1 >= a.step.B) return false;
      } while (measure<kUnit>(a, b + 1) == 0);
    }
    k = 0;
    take();
    return true;
  }
  __device__ __forceinline__ int rank(const PagedArgs& a) const { return item / (a.pool.H * tiles); }
  __device__ __forceinline__ int head(const PagedArgs& a) const { return item / tiles % a.pool.H; }
  __device__ __forceinline__ int tile() const { return item % tiles; }
  // The position of row rho of the sequence's rows (tokens times a group's heads).
  __device__ __forceinline__ int position(const PagedArgs& a, long long rho) const {
    return q.L - q.n + static_cast<int>(rho / a.G);
  }
  __device__ __forceinline__ long long last_row(const PagedArgs& a) const {
    return min(static_cast<long long>(q.n) * a.G, (tile() + 1ll) * kRowTile) - 1;
  }
};

// An item's sums for the 16 columns that a warp handles: thread `lane` holds rows
// lane / 4 and + 8 of n-tiles 2 j and 2 j + 1.
struct Sums {
  float o[8] = {};
  float ref[2] = {-INFINITY, -INFINITY}, l[2] = {};
  __device__ __forceinline__ void add(const float4& x, const float4& y, const float (&f)[2]) {
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(v[i], f[(i >> 1) & 1], o[i]);
  }
};

template <int D, bool E4M3>
__device__ __forceinline__ void store_rows(const PagedArgs& a, const Seq& q, int item, int tiles, int j, int lane,
                                           const Sums& m) {
  const int r = item / (a.pool.H * tiles), h = item / tiles % a.pool.H, c = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const long long rho = static_cast<long long>(item % tiles) * kRowTile + (lane >> 2) + 8 * i;
    if (rho >= static_cast<long long>(q.n) * a.G) continue;
    const int64_t t = q.s + rho / a.G;
    const int head = h * a.G + static_cast<int>(rho % a.G);
    const bool none = m.l[i] == 0.f;
    const float inv = none ? 0.f : 1.f / m.l[i];
    float v[4];                                // (x0, x1) of n-tile 2 j, (y0, y1) of 2 j + 1
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = none ? 0.f : m.o[(k >> 1) * 4 + 2 * i + (k & 1)] * inv;
    char* dst = a.O[r] + (t * a.ldo + static_cast<int64_t>(head) * D + 16 * j) * 2;
    if constexpr (E4M3) {                      // even columns in 2 j, odd ones in 2 j + 1
      *reinterpret_cast<uint2*>(dst + 8 * c) = make_uint2(ptx::pack_bf16x2(v[0], v[2]), ptx::pack_bf16x2(v[1], v[3]));
    } else {
      *reinterpret_cast<uint32_t*>(dst + 4 * c) = ptx::pack_bf16x2(v[0], v[1]);
      *reinterpret_cast<uint32_t*>(dst + 16 + 4 * c) = ptx::pack_bf16x2(v[2], v[3]);
    }
    if (j == 0 && c == 0 && a.lse[r] != nullptr)
      a.lse[r][t * a.Hq + head] = none ? -INFINITY : (m.ref[i] + log2f(m.l[i])) * kLn2;
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32, 1) few_rows_kernel(const __grid_constant__ PagedArgs a) {
  using F = Few<D, E4M3>;
  constexpr int kTok = F::kTok, kUnit = F::kUnit, kPer = F::kPer;
  constexpr int kNT = kTok / 8;                // n-tiles of 8 positions
  constexpr float kOff = E4M3 ? 6.f : 0.f;     // p up to 2^(kOff + kRaise): f16 holds 2^14, and 2^-38 of it
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps], s_off;
  __shared__ int s_b;
  __shared__ float s_ref[kWarps][kRowTile], s_l[kWarps][kRowTile];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // ---------------------------------------------- this CTA's run of units
  Walk w;
  const int per = (a.step.B + kWarps * 32 - 1) / (kWarps * 32);
  const int b_first = min(a.step.B, static_cast<int>(threadIdx.x) * per), b_last = min(a.step.B, b_first + per);
  long long mine = 0;
  for (int b = b_first; b < b_last; ++b) {
    mine += w.measure<kUnit>(a, b);
    if (blockIdx.x == 0 && !w.q.ok) record_invalid(a.status);
  }
  long long upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s *= 2) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += v;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  long long total = 0, from = upto - mine;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) from += s_scan[i];
    total += s_scan[i];
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  Header* const headers = reinterpret_cast<Header*>(a.ws);
  if (threadIdx.x == 0) headers[blockIdx.x].parts = 0;
  if (blockIdx.x >= ctas) return;
  const long long u0 = blockIdx.x * total / ctas, u1 = (blockIdx.x + 1) * total / ctas;
  if (u0 >= from && u0 < from + mine) {
    long long off = u0 - from;
    for (int b = b_first; b < b_last; ++b) {
      const long long n = w.measure<kUnit>(a, b);
      if (off < n) {
        s_b = b;
        s_off = off;
        break;
      }
      off -= n;
    }
  }
  __syncthreads();
  w.measure<kUnit>(a, s_b);
  w.item = static_cast<int>(s_off / w.nk);
  w.k = static_cast<int>(s_off % w.nk);
  w.left = u1 - u0;
  w.take();

  // ------------------------------------------------------------- loading
  // The loads' own walk runs kStages - 1 slices ahead of the products, and the
  // look-up of the pages one slice more.
  uint8_t* const ring = smem + warp * (kStages * 2 * kHalf);
  const uint32_t ring_addr = ptx::smem_addr(ring);
  struct Slice {
    uint32_t there[kPer];                      // which positions the pages hold
    uint32_t exps[kPer];                       // e4m3: this lane's positions' two bytes
  };
  Walk lw = w;
  bool more = true;
  int page[kPer], in_page[kPer], pool_r = 0, pool_h = 0;
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i < kPer; ++i) page[i] = -1;
    if (!more) return;
    const int hi = lw.q.ok ? lw.position(a, lw.last_row(a)) : -1;
    pool_r = lw.rank(a);
    pool_h = lw.head(a);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int tok = lane + 32 * i;
      const long long pos = static_cast<long long>(lw.first) + static_cast<long long>(lw.k) * kUnit + warp * kTok + tok;
      if (tok < kTok && pos <= hi) {
        page[i] = page_of(a.step, a.pool.pages, lw.b, static_cast<int>(pos >> a.pool.log2P));
        in_page[i] = static_cast<int>(pos) & ((1 << a.pool.log2P) - 1);
        if (page[i] < 0) record_invalid(a.status);
      }
    }
    if (++lw.k == lw.end) more = lw.next_item<kUnit>(a);
  };
  auto issue = [&](int slot) -> Slice {
    Slice s;
    int64_t row[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.there[i] = __ballot_sync(0xffffffffu, page[i] >= 0);
      s.exps[i] = 0;
      row[i] = page[i] < 0 ? 0 : ((static_cast<int64_t>(page[i]) * a.pool.H + pool_h) << a.pool.log2P) + in_page[i];
    }
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) any |= s.there[i];
    if (any != 0) {
      const char* K = a.pool.K[pool_r];
      const char* V = a.pool.V[pool_r];
      if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (page[i] >= 0) s.exps[i] = a.pool.Ke[pool_r][row[i]] | (a.pool.Ve[pool_r][row[i]] << 8);
      }
      const uint32_t dst = ring_addr + slot * (2 * kHalf);
#pragma unroll
      for (int i = 0; i < kTok / F::kRowsAtOnce; ++i) {
        const int tok = i * F::kRowsAtOnce + lane / F::kLanes;
        const int chunk = lane % F::kLanes;
        const int64_t off = __shfl_sync(0xffffffffu, row[(i * F::kRowsAtOnce) / 32], tok & 31) * F::kRow + chunk * 16;
        const bool there = s.there[(i * F::kRowsAtOnce) / 32] >> (tok & 31) & 1;
        cp_async16(dst + F::at(tok, chunk), K + off, there);
        cp_async16(dst + kHalf + F::at(tok, chunk), V + off, there);
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
    const int r = w.rank(a), h = w.head(a);
    const long long row0 = static_cast<long long>(w.tile()) * kRowTile;
    const int k0 = w.k;
    const int lo = w.position(a, row0), hi = w.position(a, w.last_row(a));  // the rows' positions
    int qpos[2];
    uint32_t qa[D / 16][4];
    float scale[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const long long rho = min(row0 + g + 8 * i, w.last_row(a));  // (a row past the last repeats it)
      qpos[i] = w.position(a, rho);
      const char* src = a.Q[r] + ((w.q.s + rho / a.G) * a.ldq + (static_cast<int64_t>(h) * a.G + rho % a.G) * D) * 2;
      scale[i] = a.scale_log2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (E4M3) {
          const uint2 x = *reinterpret_cast<const uint2*>(src + kk * 32 + 8 * c);
          qa[kk][i] = x.x;
          qa[kk][i + 2] = x.y;
        } else {
          qa[kk][i] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + 4 * c);
          qa[kk][i + 2] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + 16 + 4 * c);
        }
      }
      if constexpr (E4M3) {
        // the row's largest finite magnitude, as bf16 bits
        unsigned top = 0;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned m = (qa[kk][i + 2 * (j >> 1)] >> (16 * (j & 1))) & 0x7fffu;
            top = max(top, m < 0x7f80u ? m : 0u);
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top >> 7) - 127, -100) - 14;
        const float f = power_of_two(-e);
        scale[i] *= power_of_two(e);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const uint32_t x = qa[kk][i + j];
            qa[kk][i + j] = pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
          }
      }
    }
    float o[D / 8][4] = {}, ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (; w.k < w.end; ++w.k) {
      cp_async_wait<kStages - 2>();
      __syncwarp();                            // every lane's part of the slice is there
      const Slice cur = queue[0];
#pragma unroll
      for (int s = 0; s + 1 < kStages - 1; ++s) queue[s] = queue[s + 1];
      queue[kStages - 2] = issue(slot == 0 ? kStages - 1 : slot - 1);
      look_up();
      const uint32_t ks = ring_addr + slot * (2 * kHalf), vs = ks + kHalf;
      uint8_t* const scratch = ring + slot * (2 * kHalf);
      slot = slot + 1 == kStages ? 0 : slot + 1;

      uint32_t any = 0, all = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        any |= cur.there[i];
        all &= kTok < 32 ? cur.there[i] | ~((1u << (kTok & 31)) - 1) : cur.there[i];
      }
      if (any == 0) continue;
      const int pos0 = static_cast<int>(w.first + static_cast<long long>(w.k) * kUnit + warp * kTok);
      // every row sees every position (a window reaches back from the last row)
      const bool whole = all == 0xffffffffu && pos0 <= lo - (kTok - 1) && static_cast<long long>(pos0) > static_cast<long long>(hi) - a.window;

      float s[kNT][4];
#pragma unroll
      for (int np = 0; np < kNT / 2; ++np) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[2 * np][i] = s[2 * np + 1][i] = 0.f;
        const int row = np * 16 + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
        uint32_t x[4];
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            ldsm4(x, ks + F::at(row, 2 * j + half));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma<true>(s[2 * np], qa[2 * j + i], f16x2_of_e4m3(x[i]), f16x2_of_e4m3(x[i] >> 16));
              mma<true>(s[2 * np + 1], qa[2 * j + i], f16x2_of_e4m3(x[2 + i]), f16x2_of_e4m3(x[2 + i] >> 16));
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            ldsm4(x, ks + F::at(row, 2 * kk + half));
            mma<false>(s[2 * np], qa[kk], x[0], x[1]);
            mma<false>(s[2 * np + 1], qa[kk], x[2], x[3]);
          }
        }
      }
      // exponents (log2 units), and the rows' largest
      float inv[kNT][2];                       // e4m3: what brings p back to the sum's units
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float kx[2] = {1.f, 1.f}, vx[2] = {0.f, 0.f};
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t e = __shfl_sync(0xffffffffu, cur.exps[nt / 4], (nt * 8 + 2 * c + j) & 31);
            const int ev = min(static_cast<int>(e >> 8), 254);
            kx[j] = __int_as_float(static_cast<int>(e & 0xff) << 23);
            vx[j] = static_cast<float>(ev - 127);
            inv[nt][j] = __int_as_float((254 - ev) << 23);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[nt][i] = E4M3 ? fmaf(s[nt][i] * scale[i >> 1], kx[i & 1], vx[i & 1]) : s[nt][i] * scale[i >> 1];
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = nt * 8 + 2 * c + (i & 1), q = qpos[i >> 1];
            const long long pos = static_cast<long long>(pos0) + tok;
            if (!(cur.there[nt / 4] >> (tok & 31) & 1) || pos > q || pos <= static_cast<long long>(q) - a.window)
              s[nt][i] = -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i >> 1] = fmaxf(top[i >> 1], s[nt][i]);
      }
      bool raise = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        raise |= top[i] > ref[i] + (kOff + kRaise);
      }
      if (__any_sync(0xffffffffu, raise)) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[i] = 1.f;
          if (top[i] > ref[i] + (kOff + kRaise)) {
            f[i] = ex2_from(ref[i], top[i] - kOff);
            ref[i] = top[i] - kOff;
            l[i] *= f[i];
          }
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= f[i >> 1];
      }
      // (a row that has seen nothing yet: 2^(-inf - 0) = 0)
      const float sub[2] = {ref[0] == -INFINITY ? 0.f : ref[0], ref[1] == -INFINITY ? 0.f : ref[1]};
      bool plain = true;
      if (!whole) {
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
        for (int tg = 0; tg < kNT / 2; ++tg) {
          uint32_t pa[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[i] = ptx::ex2_approx(s[2 * tg + j][i] - sub[i >> 1]);
              l[i >> 1] = E4M3 ? fmaf(p[i], inv[2 * tg + j][i & 1], l[i >> 1]) : l[i >> 1] + p[i];
            }
            pa[2 * j] = pack16<E4M3>(p[0], p[1]);
            pa[2 * j + 1] = pack16<E4M3>(p[2], p[3]);
          }
          const int row = tg * 16 + (lane & 15);
          uint32_t x[4];
          if constexpr (E4M3) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              ldsm4_t(x, vs + F::at(row, 2 * j + (lane >> 4)));
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = __byte_perm(x[i], 0, 0x3120);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                mma<true>(o[4 * j + 2 * i], pa, f16x2_of_e4m3(x[2 * i]), f16x2_of_e4m3(x[2 * i + 1]));
                mma<true>(o[4 * j + 2 * i + 1], pa, f16x2_of_e4m3(x[2 * i] >> 16), f16x2_of_e4m3(x[2 * i + 1] >> 16));
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              ldsm4_t(x, vs + F::at(row, 2 * j + (lane >> 4)));
              mma<false>(o[2 * j], pa, x[0], x[1]);
              mma<false>(o[2 * j + 1], pa, x[2], x[3]);
            }
          }
        }
      } else {
        // One position after another, in f32; the probabilities pass through the
        // keys' place, -1 for a position that the row does not see.
        float* const ps = reinterpret_cast<float*>(scratch);   // [16][kTok]
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = nt * 8 + 2 * c + (i & 1), q = qpos[i >> 1];
            const long long pos = static_cast<long long>(pos0) + tok;
            const bool sees = (cur.there[nt / 4] >> (tok & 31) & 1) && pos <= q && pos > static_cast<long long>(q) - a.window;
            const float p = ptx::ex2_approx(s[nt][i] - sub[i >> 1]);
            if (sees) l[i >> 1] = E4M3 ? fmaf(p, inv[nt][i & 1], l[i >> 1]) : l[i >> 1] + p;
            ps[(g + 8 * (i >> 1)) * kTok + tok] = sees ? p : -1.f;
          }
        __syncwarp();
#pragma unroll 1
        for (int tok = 0; tok < kTok; ++tok) {
          const float p[2] = {ps[g * kTok + tok], ps[(g + 8) * kTok + tok]};
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            float v[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int col = E4M3 ? 16 * (j >> 1) + 4 * c + 2 * i + (j & 1) : 8 * j + 2 * c + i;
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
              if (!(p[i >> 1] < 0.f)) o[j][i] = fmaf(p[i >> 1], v[i & 1], o[j][i]);
          }
        }
        __syncwarp();
      }
    }

    // ------------------------------------- the warps' sums, added in order
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (c == 0) {
        s_ref[warp][g + 8 * i] = ref[i];
        s_l[warp][g + 8 * i] = l[i];
      }
    }
    // (the slice just used: its place is loaded again by the next item's first step)
    const int used = slot == 0 ? kStages - 1 : slot - 1;
    __syncwarp();
    float4* const mine_o = reinterpret_cast<float4*>(ring + used * (2 * kHalf));
#pragma unroll
    for (int j = 0; j < D / 8; ++j) mine_o[j * 32 + lane] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
    __syncthreads();
    const bool complete = k0 == 0 && w.end == w.nk;
    if (warp < D / 16) {
      Sums m;
#pragma unroll
      for (int v = 0; v < kWarps; ++v)
#pragma unroll
        for (int i = 0; i < 2; ++i) m.ref[i] = fmaxf(m.ref[i], s_ref[v][g + 8 * i]);
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[i] = ex2_from(s_ref[v][g + 8 * i], m.ref[i]);
          m.l[i] = fmaf(s_l[v][g + 8 * i], f[i], m.l[i]);
        }
        const float4* src = reinterpret_cast<const float4*>(smem + (v * kStages + used) * (2 * kHalf));
        m.add(src[2 * warp * 32 + lane], src[(2 * warp + 1) * 32 + lane], f);
      }
      if (complete) {
        store_rows<D, E4M3>(a, w.q, w.item, w.tiles, warp, lane, m);
      } else {
        // an item that begins here goes to the second place of this CTA
        float* part = reinterpret_cast<float*>(a.ws + header_bytes(gridDim.x)) +
                      static_cast<size_t>(2 * blockIdx.x + (k0 == 0 ? 1 : 0)) * kPartFloats<D>;
        if (warp == 0 && c == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            part[g + 8 * i] = m.ref[i];
            part[kRowTile + g + 8 * i] = m.l[i];
          }
        }
        float4* dst = reinterpret_cast<float4*>(part + 2 * kRowTile);
        dst[2 * warp * 32 + lane] = make_float4(m.o[0], m.o[1], m.o[2], m.o[3]);
        dst[(2 * warp + 1) * 32 + lane] = make_float4(m.o[4], m.o[5], m.o[6], m.o[7]);
        if (k0 == 0 && threadIdx.x == 0) {
          const long long last = at + w.nk;    // behind the item's last unit
          headers[blockIdx.x] = Header{static_cast<int>((last * ctas - 1) / total) - static_cast<int>(blockIdx.x) + 1, w.b, w.item};
        }
      }
    }
    at += w.end - k0;
    __syncthreads();
  } while (w.next_item<kUnit>(a));
  cp_async_wait<0>();
}

// Adds the parts of the item that CTA blockIdx.x of few_rows_kernel began last
// and did not finish, in the CTAs' order.
template <int D, bool E4M3>
__global__ void __launch_bounds__(D * 2) combine_kernel(const __grid_constant__ PagedArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const Header hd = reinterpret_cast<const Header*>(a.ws)[blockIdx.x];
  if (hd.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const float* parts = reinterpret_cast<const float*>(a.ws + header_bytes(gridDim.x));
  auto part = [&](int i) {
    return parts + static_cast<size_t>(2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kPartFloats<D>;
  };
  Sums m;
  for (int v = 0; v < hd.parts; ++v)
#pragma unroll
    for (int i = 0; i < 2; ++i) m.ref[i] = fmaxf(m.ref[i], part(v)[g + 8 * i]);
  for (int v = 0; v < hd.parts; ++v) {
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = ex2_from(part(v)[g + 8 * i], m.ref[i]);
      m.l[i] = fmaf(part(v)[kRowTile + g + 8 * i], f[i], m.l[i]);
    }
    const float4* src = reinterpret_cast<const float4*>(part(v) + 2 * kRowTile);
    m.add(src[2 * warp * 32 + lane], src[(2 * warp + 1) * 32 + lane], f);
  }
  const Seq q = load_seq(a.step, hd.b);
  const int tiles = static_cast<int>((static_cast<long long>(q.n) * a.G + kRowTile - 1) / kRowTile);
  store_rows<D, E4M3>(a, q, hd.item, tiles, warp, lane, m);
}

template <int D, bool E4M3>
cudaError_t launch_few(const PagedArgs& a, int ctas, cudaStream_t st) {
  constexpr int kSmem = kWarps * kStages * 2 * kHalf;
  static bool attr_set[64] = {};
  cudaError_t e = smem_attr_once(attr_set, few_rows_kernel<D, E4M3>, kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(ctas));
  if ((e = launch_pdl(few_rows_kernel<D, E4M3>, grid, dim3(kWarps * 32), kSmem, st, 1u, a)) != cudaSuccess) return e;
  return launch_pdl(combine_kernel<D, E4M3>, grid, dim3(D * 2), 0, st, 1u, a);
}

size_t few_rows_ws_bytes(int64_t d, int ctas) {
  const size_t part = (2 * kRowTile + kRowTile * static_cast<size_t>(d)) * sizeof(float);
  return header_bytes(ctas) + 2 * static_cast<size_t>(ctas) * part;
}

// Up to 16 rows to a sequence and key/value head on average: the tensor cores'
// tiles of 128 rows would be mostly empty, and their latency is what a short
// item waits for.
bool few_rows(int64_t T, int B, int G) { return T * G <= static_cast<int64_t>(kRowTile) * B; }

size_t paged_ws_bytes(int64_t T, int B, int G, int64_t d, int ctas) {
  return few_rows(T, B, G) ? few_rows_ws_bytes(d, ctas) : tiles_ws_bytes(d, B, ctas);
}

int usable_sms(const fcc_opts* o) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 256;  // (no device: sizes for the largest grid)
  }
  return o != nullptr && o->max_ctas > 0 ? std::min(sms, o->max_ctas) : sms;
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
  return paged_ws_bytes(T, B, Hq / H, d, usable_sms(opts));
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
  for (fcc_dtype t : {in, out})
    if (t != FCC_BF16 && t != FCC_F16 && t != FCC_F32) return FCC_ERR_INVALID;
  if (described != FCC_OK) return described;
  if (in != FCC_BF16 || out != FCC_BF16) return FCC_ERR_UNSUPPORTED;
  if (opts != nullptr && opts->algo != FCC_ALGO_AUTO && opts->algo != FCC_ALGO_FUSED)
    return FCC_ERR_UNSUPPORTED;
  // rows (tokens times a group's heads) and tiles of 16 of them are counted in 32 bits
  const int64_t rows = batch->T * (Hq / cache->H);
  if (rows > INT_MAX - 256 ||
      static_cast<int64_t>(R) * cache->H * (rows / kRowTile + batch->B) > INT_MAX)
    return FCC_ERR_INVALID;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (opts == nullptr || opts->workspace == nullptr) {
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &capture) != cudaSuccess) return FCC_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) return FCC_ERR_WORKSPACE;
  }
  const int ctas = usable_sms(opts);
  a.G = Hq / cache->H;
  void* ws = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  const fcc_status s = internal_prepare(opts, paged_ws_bytes(batch->T, batch->B, a.G, cache->d, ctas), &ws,
                                        &a.status, &sms, &timeout_ns);
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
  a.window = window == 0 ? INT_MAX : static_cast<int>(std::min<int64_t>(window, INT_MAX));
  a.scale_log2 = static_cast<float>((scale > 0.f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(cache->d))) *
                                    1.4426950408889634);
  a.ws = static_cast<char*>(ws);
  const bool e4m3 = cache->dtype == FCC_E4M3;
  const bool few = few_rows(batch->T, batch->B, a.G);
  const cudaError_t e =
      !few ? launch_tiles(a, e4m3, ctas, timeout_ns, st)
      : cache->d == 128 ? (e4m3 ? launch_few<128, true>(a, ctas, st) : launch_few<128, false>(a, ctas, st))
                        : (e4m3 ? launch_few<64, true>(a, ctas, st) : launch_few<64, false>(a, ctas, st));
  if (e != cudaSuccess) return FCC_ERR_CUDA;
  bump_launch_count(few ? 2 : 3);
  return FCC_OK;
}

}  // extern "C"
