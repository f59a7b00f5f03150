// fcc_loss.cu -- vocabulary-parallel losses on a linear head, forward and
// backward, without keeping the logits (sm_103a).
//
// The head W [V, D] is split by rows over R ranks; every rank holds the tokens'
// hidden states X [T, D].  With l_v = X_t . W_v (f32; optionally capped,
// l = c tanh(x / c)) two losses share these kernels:
//   cross entropy   lse - (1 - eps) l_y - eps/V sum_v l_v + z lse^2
//   distillation    tau^2 ( sum_k q_k (log q_k - l_{i_k}/tau) + lse ),
//                   lse of l/tau, q = softmax of a teacher's top logits / tau
// Both gradients have the form
//   dl_v = a p_v - b - sum_k w_k [v = i_k],   p_v = exp(l_v/tau - lse)
// with a, b, w_k per token (cross entropy: one target, its label).
//
// Forward, one GEMM over (token tile, vocabulary tile of any rank): each
// epilogue thread owns one token's logits of the tile in TMEM and reduces them
// to a maximum and a sum (base 2), their plain sum when smoothing asks for it,
// and the logits at the token's targets; one partial per (tile, token) goes to
// memory and loss_combine_kernel merges the partials of all ranks: the
// all-reduce of the softmax statistics.
// Backward: target_logit_kernel computes the logits of the labels (or of a
// teacher's heavy entries) by themselves, as the forward pass did; then, per
// piece of the vocabulary, the same product again, whose epilogue turns logits
// into dl (bf16) for the piece; then, in one launch,
// dX += dl W (the K loop runs over all ranks: the all-reduce) and dW = dl^T X.
// Only one piece of dl is ever held.
//
// All products run on tcgen05 (bf16 x bf16 -> f32 in TMEM), fed by TMA through
// an mbarrier ring: warp 0 loads, warp 1 issues the MMAs into one of two TMEM
// accumulators, warps 2-9 are the epilogue of the other.  CG = 1: one CTA per
// tile of 128 rows; CG = 2: a CTA pair per tile of 256.  dX and dW tiles are 256
// wide, in stages of 48 (pair: 32) KiB a CTA; logit tiles and their stages are
// sized by the call.  Each CTA is alone on its SM and loops over tiles.
//
// What bounds it, measured (tensor pipe busy, 4096 tokens x 32768 x 4096):
// forward 96 %, dl 96 %, dX 94 %, dW 93 %.  A training-sized call then runs at
// the chip's power limit, where what the waiting warps do not issue counts: with
// every wait suspended in hardware instead of spinning the forward pass of 8192
// tokens x 131072 x 4096 took 4.89 ms, spinning 5.07.  A few tokens are bound
// by reading W: 64 tokens x 131072 x 8192 in 306-313 us, 6.9 TB/s.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "fcc.h"
#include "fcc_internal.h"
#include "fcc_ptx.cuh"

namespace fcc {
namespace {

constexpr int kBN = 256;                            // tile columns
constexpr uint32_t kABytes = kBM * kBK * 2;         // 16 KiB per CTA and stage
constexpr uint32_t kBoxBytes = kBK * 64 * 2;        // 8 KiB: an MN-major box [64 k][64 mn]
constexpr uint32_t kTmemCols = 2 * kBN;             // double-buffered accumulator
constexpr uint64_t kDrainNs = 50ull * 1000 * 1000;  // unwinding limit after an abort
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum LossKind : int {
  LK_FWD = 0,   // logits -> softmax statistics and target logits
  LK_DL = 1,    // logits -> dl of one vocabulary piece
  LK_GRAD = 2,  // dX (+)= dl W over the ranks' pieces, and dW rows of the piece = dl^T X
};
// Operand layouts: X and W rows are contiguous along D.  dl, the library's own,
// is kept in panels of 64 vocabulary entries, [panel][token][64], tokens padded
// to 32 with zeros: every box of dl that a product loads is one contiguous run.
// (Row-major over the whole piece, a box's 128-byte rows lie a piece apart: the
// tensor pipe was busy 86 % of dX, against 92 % this way; 4096 tokens x 32768 x
// 4096.)
// Logits contract D (both operands K-major); dX contracts the vocabulary (dl
// K-major, W MN-major); dW contracts the tokens (dl and X both MN-major).
constexpr bool b_mn(int kind) { return kind == LK_GRAD; }

// The tensor core cuts its accumulator off instead of rounding it, once for
// every 16 of D, so a logit comes out too small.  By how much depends on the
// terms; measured on this chip, of the logit, per 16 of D: 1.4e-8 to 1.6e-8 where
// the products have random signs and outweigh their sum, as a head's do, at
// every D from 1024 to 131072; 0 where a single product is not zero; 4e-8 to
// 9e-8 where all products are positive; up to 1.6e-7 where the first outweighs
// the sum of the rest.  Every logit is multiplied by what the first kind loses
// (8.2e-6 at D = 8192): that is an error of as much where nothing was cut off, and
// a part of the loss where more was.  No D past the measured ones adds to it, so
// it is 1.3e-4 at most.  Adding up shorter chains in registers needs no such
// assumption; it costs 4 % (chains of 1024) to 34 % (of 256) of the forward pass.
// The logits that a loss takes from lse one by one are summed by themselves.
constexpr float kCutPerStep = 1.6e-8f;
constexpr int64_t kCutSteps = 131072 / 16;
constexpr float kHeavy = 0.125f;  // a teacher entry whose logit is also computed by itself
constexpr int kMaxHeavy = 8;      // (a token has at most so many: their sum is 1)

// Up to this many tokens dl is kept as the sum of two bf16 numbers, the second
// in the rows kSplit further on of its panels.  With few tokens there is no
// averaging of dl's rounding in dW (one token: an error of up to 2^-8 of the
// label's whole row), and the rows of the 128-row tile are free: dX's two halves
// are rows of one product, dW's a second K step of a pass bound by its output.
constexpr int kSplit = 64;

constexpr int kEpiWarps = 8;   // two per TMEM lane quarter, each with every other 64 columns
// Warps: producer, MMA, epilogue; FWD two more for the labels' own logits.
constexpr int threads_of(int kind) { return 64 + 32 * kEpiWarps + (kind == LK_FWD ? 64 : 0); }
// A warp's staging: 32 rows x 64 bf16 (dX, dW: 128-byte swizzle; dl: half of it,
// 32 columns, 64-byte swizzle).
constexpr uint32_t kOutBytes = 32 * 128;
// bf16 results leave by TMA stores from shared memory.
constexpr bool stages_out(int kind) { return kind != LK_FWD; }

template <int KIND, int CG>
struct Cfg {
  static constexpr int kTileM = kBM * CG;
  static constexpr int kBNcta = kBN / CG;                  // B columns this CTA holds
  // GRAD: stages of full size.  FWD, DL: as many as the tile's rows and width
  // leave room for (LossParams), up to kMaxStages: a few words' or tokens' tiles
  // are bound by the loads, of which more are then in flight (64 tokens x 131072
  // x 8192: 327 -> 313 us).
  static constexpr int kMaxStages = KIND == LK_GRAD ? (CG == 2 ? 6 : 4) : 16;
  static constexpr uint32_t kBBytes = kBK * kBNcta * 2;    // 32 or 16 KiB
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  static constexpr uint32_t kOut = stages_out(KIND) ? kEpiWarps * kOutBytes : 0;
  static constexpr uint32_t kRing = 7 * 32768 - kOut;      // bytes for the stages
  static_assert(KIND != LK_GRAD || kMaxStages * kStageBytes <= kRing, "ring");
  // Instruction descriptor of a tile `width` columns wide.
  __device__ static constexpr uint32_t idesc(int width, bool a_mn) {
    return ptx::idesc_bf16_f32(kTileM, width, a_mn, b_mn(KIND));
  }
  static constexpr int kSmem = 1024 + static_cast<int>(kRing + kOut) + (2 * kMaxStages + 5) * 8 +
                               16 + (KIND == LK_FWD ? 128 * 12 : 0);
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// How the dX tiles that would make up a last, partly filled round (all tiles,
// when they are fewer than the CTAs) are shared: `tiles` tiles of k steps over
// `ctas` CTAs (pairs).  Each of `groups` CTAs per tile takes `len` steps of
// it, so that the CTAs of a group walk the same rows of dl and W side by side
// (equal shares of the tiles' steps laid end to end start everywhere in k and
// read dl and W from memory once per tile: 321 us against 224 for 1999 tokens x
// 50257 x 2048); the helpers, the CTAs left over, share the tiles' remaining
// tails, laid end to end.  A tile's parts are summed at the end in a fixed
// order.
struct Shares {
  int tiles, ctas, k;
  int groups, len, tail, helpers;  // tail = k - groups * len
  int max_parts;
  __host__ __device__ __forceinline__ long long tails() const {
    return static_cast<long long>(tiles) * tail;
  }
  // The helper that holds step x of the tails: helper h has steps
  // [h tails / helpers, (h + 1) tails / helpers).
  __host__ __device__ __forceinline__ int helper_of(long long x) const {
    return static_cast<int>(((x + 1) * helpers - 1) / tails());
  }
  // No tile is shared after all: as many CTAs as tiles.
  __host__ __device__ __forceinline__ bool alone() const { return groups == 1 && tail <= 0; }
  // Parts of shared tile i.
  __host__ __device__ __forceinline__ int parts(int i) const {
    if (tail <= 0) return groups;
    const long long x = static_cast<long long>(i) * tail;
    return groups + helper_of(x + tail - 1) - helper_of(x) + 1;
  }
};

// Division of 0 <= n < 2^31 by a divisor fixed on the host: n m >> (31 + s),
// m = ceil(2^(31+s) / d), 2^(s-1) < d <= 2^s.  m d exceeds 2^(31+s) by less
// than d <= 2^s, so the product's error, n (m d - 2^(31+s)) / (d 2^(31+s)), is
// below 1 / d: the quotient is exact.  (The loading and the issuing thread find
// their next tile with it: plain divisions cost 1.5-2 us of a 40-70 us call.)
struct FastDiv {
  uint32_t m, s;
  int d;
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> (31 + s));
  }
};
FastDiv fast_div(int d) {
  FastDiv f;
  f.d = d;
  f.s = 0;
  while ((1ll << f.s) < d) ++f.s;
  f.m = static_cast<uint32_t>(((1ull << (31 + f.s)) + d - 1) / d);
  return f;
}

// The order of a grid of tiles: groups of `group` rows of tiles, column by
// column within a group, so that CTAs running at the same time share operands.
struct Raster {
  FastDiv per_group, height, last_height;
  int last_first;  // the first row of the last group
  __device__ __forceinline__ void at(int t, int& mt, int& nt) const {
    const int g = per_group.div(t);
    const int first = g * height.d;
    const int local = t - g * per_group.d;
    const bool last = first == last_first;
    nt = last ? last_height.div(local) : height.div(local);
    mt = first + local - nt * (last ? last_height.d : height.d);
  }
};
Raster raster_of(int tiles_m, int tiles_n, int group) {
  Raster r;
  r.last_first = (tiles_m - 1) / group * group;
  r.per_group = fast_div(group * tiles_n);
  r.height = fast_div(group);
  r.last_height = fast_div(tiles_m - r.last_first);
  return r;
}

// A few tokens' products read W once each, and the next product reads it again
// (forward, dl, dX, the next forward).  Evicted by age, a W larger than the L2
// leaves nothing to hit; so a fixed part of its lines (the hardware's choice by
// address) is held as usual and the rest marked to go first.  48 MB of W of 262
// (96 tokens x 32000 x 4096): backward 159 -> 151 us, 526 MB 272 -> 268; 32 or 64
// MB the same within 1 us, 96 MB 154.  Below kKeepFrom bytes of W it loses (100 MB:
// 87 -> 88), past kKeepTo too (2.1 GB: 961 -> 974; 820 MB: 393 -> 390).
constexpr double kKeepBytes = 48e6, kKeepFrom = 128e6, kKeepTo = 1e9;

constexpr int kGroupM = 16;  // against 8: forward 5.33 -> 5.18 ms, backward unchanged; 32: slower

struct LossParams {
  CUtensorMap mapA[FCC_MAX_RANKS];
  CUtensorMap mapB[FCC_MAX_RANKS];
  CUtensorMap mapO[FCC_MAX_RANKS];  // DL: dl, box 32 tokens x 32; GRAD: dW, 32 rows x 64
  CUtensorMap mapA2[FCC_MAX_RANKS];  // GRAD: mapA, mapB of dX are dl and W, of dW these:
  CUtensorMap mapB2[FCC_MAX_RANKS];  // dl and X in boxes of k_rows tokens
  CUtensorMap mapX[FCC_MAX_RANKS];   // GRAD: dX, box 32 x 64
  int R, T, D;
  int Vs;                  // vocabulary rows per rank
  int v0, vn;              // this piece: rows [v0, v0 + vn) of every rank (FWD: 0, Vs)
  int tpad;                // rows of a dl panel: the tokens, to a multiple of 32 (split: 2 kSplit)
  int split;               // GRAD, DL: dl in two halves, see kSplit
  int width;               // tile columns (FWD, DL: a multiple of 32), else kBN
  int tiles_m, tiles_n;    // tiles of one rank (GRAD: of dX, over all)
  int full_tiles;          // tiles run whole, round-robin (dX: the others are shared, see Shares)
  int k_iters;             // 64-deep K steps of a whole tile (GRAD: of dX)
  int kb_per_rank;         // dX: K steps per rank
  int dw_tiles_m, dw_tiles;  // dW: row tiles of one rank, tiles over all
  Shares shares;           // DX: the tiles past full_tiles, by the first piece's K steps
  int a_rows;              // rows of an A box (K-major A: fewer than 128 when T is)
  uint32_t stages, a_size, stage_size;  // FWD, DL: the ring (a_size: the A box, to 1 KiB)
  int k_rows;              // DW: tokens of a K step (fewer than 64 when T is)
  Raster order, dw_order;  // of the logit or dX tiles, and of the dW tiles
  FastDiv by_tiles_n, by_dw_tiles_m;  // tile columns / dW tile rows of a rank
  float keep;              // the share of W's lines that the L2 is to hold, 0: no hint
  // tokens' targets: labels (cross entropy), or per token K sorted vocabulary
  // indices (INT_MAX past the last) and their teacher probabilities
  const int32_t* labels;
  const int32_t* hit_idx;  // [T, K]
  const float* hit_q;      // [T, K]
  // [T][start_ld]: the first of them at or past a logit tile, by (rank, piece, tile)
  const uint16_t* hit_start;
  long long start_ld;
  int npieces, piece, piece_tiles;
  int K;
  int ignore_index;
  float cap, inv_cap;      // soft cap, 0 = none
  float c2;                // log2(e) / tau
  float grow;              // what the tensor core's sums lose on average, see kCutPerStep
  float tau, smoothing, z;
  // FWD
  float2* part;            // [R * tiles_n][T]: base-2 maximum and sum
  float* part_sum;         // the same layout: sum of the logits (smoothing), or NULL
  float* pick;             // [T, K] logits at the targets
  const void* X[FCC_MAX_RANKS];   // the matrices themselves and the labels' (or the heavy
  const void* Wr[FCC_MAX_RANKS];  // entries') logits computed from them, DL: capped
  float* own_logit;               // [T, K]
  const int16_t* heavy;    // [T, kMaxHeavy]: a token's heavy entries' places, then -1
  // DL
  const float* lse[FCC_MAX_RANKS];
  const float* dloss;
  // dX: f32 sums [T][D] (split: [2 kSplit][D]) of whole tiles and of shared tiles' first parts, and
  // one [rows][kBN] block for each further part; first = 1: overwrite, else add
  float* acc;
  float* parts;
  int first;
  int direct;              // dX tiles that one CTA sums to the end leave in bf16 here (last piece)
  int* status;
  unsigned long long timeout_ns;
};

struct Tile {
  int rank, mt, nt;
  int it_lo, it_hi;  // K steps
  int part;          // dX: which part of a shared tile (0: goes to acc)
  int shared;        // dX: index among the shared tiles
  bool dw;           // GRAD: a tile of dW, else of dX
  bool alone;        // dX: no other CTA has a part of the tile
};

template <int KIND>
__device__ __forceinline__ Tile tile_of(const LossParams& p, int t) {
  Tile tl;
  tl.rank = 0;
  tl.part = 0;
  tl.shared = 0;
  tl.dw = false;
  tl.alone = true;
  tl.it_lo = 0;
  tl.it_hi = p.k_iters;
  p.order.at(t, tl.mt, tl.nt);
  if constexpr (KIND == LK_FWD || KIND == LK_DL) {
    tl.rank = p.by_tiles_n.div(tl.nt);
    tl.nt -= tl.rank * p.tiles_n;
  }
  return tl;
}

__device__ __forceinline__ Tile dw_tile_of(const LossParams& p, int t) {
  Tile tl;
  tl.part = 0;
  tl.shared = 0;
  tl.dw = true;
  tl.alone = true;
  tl.it_lo = 0;
  tl.it_hi = p.split ? 2 : (p.T + kBK - 1) / kBK;
  p.dw_order.at(t, tl.mt, tl.nt);
  tl.rank = p.by_dw_tiles_m.div(tl.mt);
  tl.mt -= tl.rank * p.dw_tiles_m;
  return tl;
}

// What one CTA (pair) works on: whole tiles round-robin; GRAD: whole dX tiles,
// its share of the others, and dW tiles round-robin.
template <int KIND>
struct Work {
  const LossParams& p;
  int t, tw, npairs, pair;
  long long cur, end;  // of the tails (a helper); cur = -1: a group's share to do
  __device__ __forceinline__ Work(const LossParams& p_, int pair_, int npairs_)
      : p(p_), t(pair_), tw(pair_), npairs(npairs_), pair(pair_), cur(0), end(0) {
    if constexpr (KIND == LK_GRAD) {
      const Shares& s = p.shares;
      const int h = pair - s.groups * s.tiles;
      if (s.tiles > 0 && h < 0) {
        cur = -1;
      } else if (s.tail > 0 && h < s.helpers) {
        cur = s.tails() * h / s.helpers;
        end = s.tails() * (h + 1) / s.helpers;
      }
    }
  }
  __device__ __forceinline__ bool next_dw(Tile& tl) {
    if (tw >= p.dw_tiles) return false;
    tl = dw_tile_of(p, tw);
    tw += npairs;
    return true;
  }
  __device__ __forceinline__ bool next_dx(Tile& tl) {
    if (t < p.full_tiles) {
      tl = tile_of<KIND>(p, t);
      t += npairs;
      return true;
    }
    if constexpr (KIND == LK_GRAD) {
      const Shares& s = p.shares;
      int i, lo, n, part;
      if (cur < 0) {
        const int g = pair / s.tiles;
        i = pair - g * s.tiles;
        lo = g * s.len;
        n = s.len;
        part = g;
        cur = 0;
      } else if (cur < end) {
        i = static_cast<int>(cur / s.tail);
        const int x = static_cast<int>(cur - static_cast<long long>(i) * s.tail);
        n = static_cast<int>(min(static_cast<long long>(s.tail - x), end - cur));
        lo = s.groups * s.len + x;
        part = s.groups + pair - s.groups * s.tiles - s.helper_of(static_cast<long long>(i) * s.tail);
        cur += n;
      } else {
        return false;
      }
      tl = tile_of<KIND>(p, p.full_tiles + i);
      tl.shared = i;
      tl.part = part;
      tl.alone = s.alone();
      // (a shorter last piece has fewer steps than planned, or none)
      tl.it_lo = min(lo, p.k_iters);
      tl.it_hi = min(lo + n, p.k_iters);
      return true;
    }
    return false;
  }
  __device__ __forceinline__ bool next(Tile& tl) {
    return next_dx(tl) || (KIND == LK_GRAD && next_dw(tl));
  }
};

// 32 f32 columns of each lane's row as bf16 into the warp's staging: half 0 / 1
// of 64 columns (WIDE, 128-byte swizzle) or all of 32 (64-byte swizzle), in
// 16-byte pieces without bank conflicts.
template <bool WIDE>
__device__ __forceinline__ void stage_bf16(uint8_t* buf, int lane, int half,
                                           const uint32_t (&v)[32]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint4 w;
    w.x = ptx::pack_bf16x2(__uint_as_float(v[8 * g]), __uint_as_float(v[8 * g + 1]));
    w.y = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 2]), __uint_as_float(v[8 * g + 3]));
    w.z = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 4]), __uint_as_float(v[8 * g + 5]));
    w.w = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 6]), __uint_as_float(v[8 * g + 7]));
    const int at = WIDE ? lane * 128 + (((half * 4 + g) ^ (lane & 7)) << 4)
                        : lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4);
    *reinterpret_cast<uint4*>(buf + at) = w;
  }
}

// l = c tanh(x / c) of a lane's 32 logits, to 2^-20 of l for any c.  |x| < c/2:
// the Taylor series x (1 - w/3 + 2 w^2/15 - ...), w = (x/c)^2, to w^6 (the first
// term left out is 9e-8 of x).  Past it c - 2c / (1 + e^{2|x|/c}) with the sign of
// x, by the approximate exponential and reciprocal (an exponential past the range
// gives +-c); near zero that form would be off by c 2^-23, whatever x is.  A
// warp's chunk is hardly ever past c/2, and the series alone, without special
// functions, is also the faster form.  An element's result does not depend on the
// others': both paths compute the series with the same roundings.
__device__ __forceinline__ float soft_cap_series(float w) {
  float s = fmaf(w, 21844.f / 6081075.f, -1382.f / 155925.f);
  s = fmaf(s, w, 62.f / 2835.f);
  s = fmaf(s, w, -17.f / 315.f);
  s = fmaf(s, w, 2.f / 15.f);
  s = fmaf(s, w, -1.f / 3.f);
  return fmaf(s, w, 1.f);
}
__device__ __forceinline__ void soft_cap(uint32_t (&v)[32], float cap, float inv_cap) {
  float far = 0.f;  // (a NaN is passed over: it stays one in either path)
#pragma unroll
  for (int k = 0; k < 32; k += 2)
    far = ptx::max3(far, fabsf(__uint_as_float(v[k])), fabsf(__uint_as_float(v[k + 1])));
  if (__all_sync(0xffffffffu, far * inv_cap < 0.5f)) {
    const uint64_t inv2 = ptx::f32x2_pack(inv_cap, inv_cap);
    auto both = [](float a) { return ptx::f32x2_pack(a, a); };
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const uint64_t x = ptx::f32x2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
      const uint64_t u = ptx::f32x2_mul(x, inv2);
      const uint64_t w = ptx::f32x2_mul(u, u);
      uint64_t s = ptx::f32x2_fma(w, both(21844.f / 6081075.f), both(-1382.f / 155925.f));
      s = ptx::f32x2_fma(s, w, both(62.f / 2835.f));
      s = ptx::f32x2_fma(s, w, both(-17.f / 315.f));
      s = ptx::f32x2_fma(s, w, both(2.f / 15.f));
      s = ptx::f32x2_fma(s, w, both(-1.f / 3.f));
      s = ptx::f32x2_fma(s, w, both(1.f));
      float y0, y1;
      ptx::f32x2_unpack(ptx::f32x2_mul(x, s), y0, y1);
      v[k] = __float_as_uint(y0);
      v[k + 1] = __float_as_uint(y1);
    }
  } else {
    const float step = 2.f * kLog2e * inv_cap;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float x = __uint_as_float(v[k]);
      const float u = __fmul_rn(x, inv_cap);
      const float near = __fmul_rn(x, soft_cap_series(__fmul_rn(u, u)));
      const float rest = ptx::rcp_approx(1.f + ptx::ex2_approx(fabsf(x) * step));
      const float past = copysignf(fmaf(-2.f * cap, rest, cap), x);
      v[k] = __float_as_uint(fabsf(u) < 0.5f ? near : past);
    }
  }
}

// v[at] by halving: 31 selections.
__device__ __forceinline__ float pick32(const uint32_t (&v)[32], int at) {
  uint32_t h[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) h[k] = at & 16 ? v[k + 16] : v[k];
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) h[k] = at & n ? h[k + n] : h[k];
  return __uint_as_float(h[0]);
}

// (m, s) of both: base-2 maximum and sum.
__device__ __forceinline__ void merge(float& m, float& s, float m1, float s1) {
  const float mn = fmaxf(m, m1);
  const float off = mn == -INFINITY ? 0.f : mn;
  // (a sum whose maximum is -inf is 0, or NaN after a NaN logit: kept as it is)
  s = (m == -INFINITY ? s : s * exp2f(m - off)) + (m1 == -INFINITY ? s1 : s1 * exp2f(m1 - off));
  m = mn;
}

// What a logit tile's epilogue thread needs of its token, fetched a tile ahead.
struct Token {
  int y;       // the label, or the place of the first target at or past the tile
  int first;   // DL, teacher: the token's first target (INT_MAX: it has none)
  float lse, g;
  float own;   // DL, labels: the label's logit by itself
};

template <int KIND>
__device__ __forceinline__ Token token_of(const LossParams& p, const Tile& tl, long long row) {
  Token k{0, INT_MAX, 0.f, 0.f, 0.f};
  if (row >= p.T) return k;
  if (p.labels != nullptr) {
    k.y = __ldg(p.labels + row);
    if (KIND == LK_DL) k.own = __ldg(p.own_logit + row);
  } else {
    k.y = __ldg(p.hit_start + row * p.start_ld +
                (tl.rank * p.npieces + p.piece) * p.piece_tiles + tl.nt);
    if (KIND == LK_DL) k.first = __ldg(p.hit_idx + row * p.K);
  }
  if (KIND == LK_DL) {
    k.g = __ldg(p.dloss + row);
    k.lse = __ldg(p.lse[tl.rank] + row);
  }
  return k;
}

// A token's targets in ascending vocabulary order: `next` is the next one at
// or past the tile (INT_MAX: none), `cur` its place in the token's list.
struct Targets {
  const int32_t* list;
  int cur, n, next;
};

__device__ __forceinline__ Targets targets_from(const LossParams& p, const Token& k, long long row,
                                                int col0) {
  Targets g{nullptr, 0, 0, INT_MAX};
  if (row >= p.T) return g;
  if (p.labels != nullptr) {
    if (k.y >= col0) g.next = k.y;  // (an ignored or bad label is dealt with by the caller)
    return g;
  }
  g.list = p.hit_idx + row * p.K;
  g.n = p.K;
  g.cur = k.y;
  if (g.cur < g.n) g.next = __ldg(g.list + g.cur);
  return g;
}

__device__ __forceinline__ void targets_advance(Targets& g) {
  ++g.cur;
  g.next = g.cur < g.n ? __ldg(g.list + g.cur) : INT_MAX;
}

__device__ __forceinline__ bool label_live(const LossParams& p, int y) {
  return y != p.ignore_index && y >= 0 && y < p.R * p.Vs;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(threads_of(KIND), 1)
loss_gemm_kernel(const __grid_constant__ LossParams p) {
  using C = Cfg<KIND, CG>;
  constexpr int TM = C::kTileM;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // The ring: stage s at s * stage_size, its A and, a_size on, its B.
  const uint32_t kStages = KIND == LK_GRAD ? C::kMaxStages : p.stages;
  const uint32_t a_size = KIND == LK_GRAD ? kABytes : p.a_size;
  const uint32_t stage_size = KIND == LK_GRAD ? C::kStageBytes : p.stage_size;
  uint8_t* sO = smem + C::kRing;  // DL, GRAD: the epilogue warps' staging blocks
  uint64_t* full = reinterpret_cast<uint64_t*>(sO + C::kOut);
  uint64_t* empty = full + C::kMaxStages;
  uint64_t* tfull = empty + C::kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sStat = reinterpret_cast<float*>(tmem_slot + 4);  // FWD: [128][3]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = kPair ? ptx::cluster_ctarank() : 0u;  // 0 issues the pair's MMAs
  const int pair = blockIdx.x / CG;
  const int npairs = gridDim.x / CG;

  if (threadIdx.x < kStages) {
    ptx::mbar_init(&full[threadIdx.x], 1);
    ptx::mbar_init(&empty[threadIdx.x], 1);
    ptx::fence_mbar_init();
  } else if (threadIdx.x == 32) {
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], kEpiWarps * CG);  // every epilogue warp of the pair
    }
    ptx::mbar_init(mma_done, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    for (int r = 0; r < p.R; ++r) {
      ptx::tma_prefetch_desc(&p.mapA[r]);
      ptx::tma_prefetch_desc(&p.mapB[r]);
    }
  }
  if (warp == 1) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(tmem_slot, kTmemCols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tmem_slot, kTmemCols);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  if constexpr (kPair) {
    ptx::cluster_sync_all();  // the peer's barriers exist before anyone signals them
  } else {
    __syncthreads();
  }
  ptx::tc_fence_after();
  // Launched with programmatic stream serialization: nothing above touches
  // global memory.
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  const ptx::Waiter W{abort_flag, p.status, p.timeout_ns};
  Work<KIND> work(p, pair, npairs);
  Tile tl;
  // B columns per CTA: of a logit tile its width's half or whole, else fixed
  const int bn_cta = (KIND == LK_FWD || KIND == LK_DL) ? p.width / CG : C::kBNcta;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      int64_t loads = 0;  // stages filled so far
      // (rows of A past a short box stay as they are: they only make rows of
      // the result that nothing reads)
      const uint32_t bytes_x =
          static_cast<uint32_t>(p.a_rows) * kBK * 2 + static_cast<uint32_t>(bn_cta) * kBK * 2;
      const uint32_t bytes_w = static_cast<uint32_t>(kBM + C::kBNcta) * p.k_rows * 2;
      // (a pair's bytes are counted on the leader's barriers)
      const uint32_t full0 = kPair ? ptx::mapa(ptx::smem_addr(full), 0) : 0u;
      bool ok = true;
      const uint64_t policy = kPair || !(p.keep > 0) ? 0 : ptx::policy_keep(p.keep);
      while (ok && work.next(tl)) {
        const int m0 = tl.mt * TM + static_cast<int>(cta) * kBM;  // this CTA's A rows
        const int n0 = tl.nt * (bn_cta * CG) + static_cast<int>(cta) * bn_cta;  // and B columns
        // The tile's loads, for one of the two products of GRAD (dW, or dX and
        // the logits): as little as possible per K step, for one thread issues
        // them all.
        auto k_loop = [&](auto w) {
          constexpr bool kDw = decltype(w)::value;
          const uint32_t stage_bytes = kDw ? bytes_w : bytes_x;
          int r = tl.rank, kb = tl.it_lo;
          if (KIND == LK_GRAD && !kDw) {
            r = tl.it_lo / p.kb_per_rank;
            kb = tl.it_lo - r * p.kb_per_rank;
          }
          const CUtensorMap* ma = kDw ? &p.mapA2[r] : &p.mapA[r];
          const CUtensorMap* mb = kDw ? &p.mapB2[r] : &p.mapB[r];
          // A: (x, y) and their steps; dW a second box, one panel on
          int ax = 0, ay = m0, by = 0;
          if constexpr (kDw) {
            ay = (m0 >> 6) * p.tpad;
          } else if constexpr (KIND == LK_GRAD) {
            ay = kb * p.tpad + m0;  // (panel kb)
            by = p.v0 + kb * kBK;
          }
          for (int it = tl.it_lo; it < tl.it_hi; ++it) {
            if (!W.wait_suspended(&empty[stage], phase ^ 1u)) return false;
            uint8_t* a_dst = smem + stage * stage_size;
            uint8_t* b_dst = a_dst + a_size;
            if (!kPair || cta == 0) ptx::mbar_arrive_expect_tx(&full[stage], CG * stage_bytes);
            auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
              if constexpr (kPair)
                ptx::tma_load_2d_pair(dst, map, full0 + stage * 8, x, y);
              else
                ptx::tma_load_2d(dst, map, &full[stage], x, y);
            };
            auto load_w = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
              if (!kPair && !kDw && p.keep > 0)
                ptx::tma_load_2d_hint(dst, map, &full[stage], x, y, policy);
              else
                load(dst, map, x, y);
            };
            load(a_dst, ma, ax, ay);
            if constexpr (kDw) load(a_dst + kBoxBytes, ma, ax, ay + p.tpad);
            if constexpr (b_mn(KIND)) {
              // W rows of the piece (dX) or tokens (dW) down, D across
#pragma unroll
              for (int i = 0; i < C::kBNcta / 64; ++i)
                load_w(b_dst + i * kBoxBytes, mb, n0 + 64 * i, by);
            } else {
              load_w(b_dst, mb, ax, p.v0 + n0);
            }
            ++loads;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            if constexpr (kDw) {
              ay += p.split ? kSplit : kBK;
              by += p.split ? 0 : kBK;
            } else if constexpr (KIND == LK_GRAD) {
              ay += p.tpad;
              by += kBK;
              if (++kb == p.kb_per_rank) {
                kb = 0;
                ++r;
                ++ma;
                ++mb;
                ay = m0;
                by = p.v0;
              }
            } else {
              ax += kBK;
            }
          }
          return true;
        };
        if (KIND == LK_GRAD && tl.dw)
          ok = k_loop(std::true_type{});
        else
          ok = k_loop(std::false_type{});
      }
      if (*abort_flag && cta == 0) {
        // Loads in flight write into shared memory: let them land (in a pair
        // all are counted on the leader's barriers).
        for (int64_t i = loads > kStages ? loads - kStages : 0; i < loads; ++i)
          W.drain(&full[i % kStages], static_cast<uint32_t>((i / kStages) & 1), kDrainNs);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue
    if (lane == 0 && cta == 0) {
      uint32_t stage = 0, phase = 0;
      uint32_t acc = 0, acc_phase = 0;
      bool any = false, ok = true;
      while (ok && work.next(tl)) {
        if (!W.wait_suspended(&tempty[acc], acc_phase ^ 1u)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kBN;
        // The tile's K steps, for one layout of A (dW: dl MN-major, else K-major).
        auto k_loop = [&](auto mn) {
          constexpr bool kDw = decltype(mn)::value;
          const uint32_t idesc = C::idesc(bn_cta * CG, kDw);
          const uint64_t a_desc0 = ptx::smem_desc_sw128(ptx::smem_addr(smem), kDw ? kBoxBytes : 16, 1024);
          const uint64_t b_desc0 =
              ptx::smem_desc_sw128(ptx::smem_addr(smem) + a_size, b_mn(KIND) ? kBoxBytes : 16, 1024);
          for (int it = tl.it_lo; it < tl.it_hi; ++it) {
            if (!W.wait_suspended(&full[stage], phase)) return false;
            ptx::tc_fence_after();
            // The stage's descriptors; a K step of 16 on is 32 B within the
            // swizzled row (K-major) or 2 KiB (MN-major, 64-wide boxes 8 KiB
            // apart), added to the address field.
            const uint64_t ad = a_desc0 + stage * (stage_size >> 4);
            const uint64_t bd = b_desc0 + stage * (stage_size >> 4);
            auto mma = [&](int kk) {
              const uint32_t accum = (it > tl.it_lo || kk > 0) ? 1u : 0u;
              const uint64_t a_kk = ad + kk * ((kDw ? 2048 : 32) >> 4);
              const uint64_t b_kk = bd + kk * ((b_mn(KIND) ? 2048 : 32) >> 4);
              if constexpr (kPair)
                ptx::mma_f16_pair(d_tmem, a_kk, b_kk, idesc, accum);
              else
                ptx::mma_f16(d_tmem, a_kk, b_kk, idesc, accum);
            };
            // (dW: no MMA for 16 rows past the last token, which a short box
            // does not fill; the usual step has no such test, which the one
            // thread that issues would feel)
            const int tokens = kDw ? p.T - (p.split ? 0 : it * kBK) : kBK;
            if (tokens > kBK - 16) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) mma(kk);
            } else {
              for (int kk = 0; 16 * kk < tokens; ++kk) mma(kk);
            }
            if constexpr (kPair)
              ptx::mma_commit_pair_arrive_ctas(&empty[stage], 0x3);
            else
              ptx::mma_commit(&empty[stage]);
            any = true;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          return true;
        };
        if (KIND == LK_GRAD && tl.dw)
          ok = k_loop(std::true_type{});
        else
          ok = k_loop(std::false_type{});
        if (!ok) break;
        if constexpr (kPair)
          ptx::mma_commit_pair_arrive_ctas(&tfull[acc], 0x3);
        else
          ptx::mma_commit(&tfull[acc]);
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (any) {
        if constexpr (kPair)
          ptx::mma_commit_pair(mma_done);
        else
          ptx::mma_commit(mma_done);
        W.drain(mma_done, 0, kDrainNs);
      }
    }
  } else if (warp < 2 + kEpiWarps) {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;            // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // it takes every other 64 columns, from 64 half on
    const int trow = q * 32 + lane;    // its row of the CTA's 128
    uint8_t* buf = sO + (warp - 2) * kOutBytes;
    const uint32_t tempty_leader0 = kPair ? ptx::mapa(ptx::smem_addr(&tempty[0]), 0) : 0u;
    uint32_t acc = 0, acc_phase = 0;
    // The whole warp polls and stops as one (the TMEM loads are collective);
    // FWD: both warps of a lane quarter, which meet at a named barrier below.
    auto wait_tile = [&]() -> bool {
      bool ok = __all_sync(0xffffffffu, W.wait_suspended(&tfull[acc], acc_phase) ? 1 : 0) != 0;
      if constexpr (KIND == LK_FWD) ok = !ptx::named_barrier_or(1 + q, 64, !ok);
      if (ok) ptx::tc_fence_after();
      return ok;
    };
    // Hands the accumulator back (every warp): dX and dW after the last read of
    // it, before its columns are stored (dX of 1024 x 50257 x 256 30.5 -> 28 us,
    // dW 21 -> 18.5); the logits' epilogues at their end (earlier was slower: dl
    // 54 -> 61 us).
    auto release_acc = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair)
          ptx::mbar_arrive_cluster_tmem(tempty_leader0 + acc * 8);
        else
          ptx::mbar_arrive(&tempty[acc]);
      }
    };
    // The staged columns leave by TMA, issued by one lane: dW and dX, 64 columns
    // to (x, y) of each of `n` maps; dl, 32 columns from piece column x on.
    auto store_rows = [&](const CUtensorMap* maps, int n, int x, int y) {
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        for (int r = 0; r < n; ++r) ptx::tma_store_2d(maps + r, buf, x, y);
        ptx::bulk_commit();
      }
    };
    auto store_dl = [&](const CUtensorMap* map, int x, int row) {
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::tma_store_2d(map, buf, x & 63, (x >> 6) * p.tpad + row);
        ptx::bulk_commit();
      }
    };
    auto buf_free = [&]() {
      if (lane == 0) ptx::bulk_wait_read();
      __syncwarp();
    };
    bool more = work.next(tl);
    Tile ahead = tl;
    Token token_ahead{};
    auto row_of = [&](const Tile& w) {  // the warp's first row
      return w.mt * TM + static_cast<int>(cta) * kBM + q * 32;
    };
    if constexpr (KIND == LK_FWD || KIND == LK_DL) {
      if (more) token_ahead = token_of<KIND>(p, ahead, row_of(ahead) + lane);
    }
    while (more) {
      tl = ahead;
      const Token tok = token_ahead;
      more = work.next(ahead);
      const int row0 = row_of(tl);
      const long long row = row0 + lane;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kBN;
      if constexpr (KIND == LK_FWD || KIND == LK_DL) {
        const bool row_ok = row < p.T;
        const int col0 = tl.nt * p.width;                // within the piece
        const int vcol0 = tl.rank * p.Vs + p.v0 + col0;  // the tile's first vocabulary index
        const int ncols = min(p.width, p.vn - col0);
        // (the other half's targets are passed over below)
        Targets tg = targets_from(p, tok, row, vcol0);
        if (more) token_ahead = token_of<KIND>(p, ahead, row_of(ahead) + lane);
        // DL: the token's coefficients (not live: an ignored row, all zeros)
        float ca = 0.f, cb = 0.f, cw = 0.f, off2 = 0.f;
        bool live = false;
        if constexpr (KIND == LK_DL) {
          if (row_ok) {
            off2 = tok.lse * kLog2e;
            if (p.labels != nullptr) {
              live = label_live(p, tok.y);
              if (vcol0 == 0 && !live && tok.y != p.ignore_index)
                atomicCAS(p.status, 0, FCC_ERR_INVALID);
              ca = tok.g * (1.f + 2.f * p.z * tok.lse);
              cb = tok.g * (p.smoothing / static_cast<float>(p.R * p.Vs));
              cw = tok.g * (1.f - p.smoothing);
            } else {
              live = tok.first != INT_MAX;
              ca = tok.g * p.tau;
              cw = tok.g * p.tau;
            }
          }
        }
        if (!wait_tile()) break;
        float m2 = -INFINITY, sum = 0.f, lsum = 0.f;  // FWD: base-2 maximum, sum; plain sum
        // One chunk of 32 columns from c on, of which nc > 0 exist.
        auto chunk = [&](uint32_t (&v)[32], int c, int nc) {
          const uint64_t grow2 = ptx::f32x2_pack(p.grow, p.grow);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x0, x1;
            ptx::f32x2_unpack(
                ptx::f32x2_mul(ptx::f32x2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                               grow2), x0, x1);
            v[k] = __float_as_uint(x0);
            v[k + 1] = __float_as_uint(x1);
          }
          if (p.cap > 0.f) soft_cap(v, p.cap, p.inv_cap);
          const int vc = vcol0 + c, vend = vc + min(32, nc);
          if constexpr (KIND == LK_FWD) {
            if (nc < 32) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k >= nc) v[k] = 0xff800000u;  // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              mx[(k / 2) & 3] = ptx::max3(mx[(k / 2) & 3], __uint_as_float(v[k]),
                                          __uint_as_float(v[k + 1]));
            const float cm = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.c2;
            const float mn = fmaxf(m2, cm);
            const float off = mn == -INFINITY ? 0.f : mn;
            // (before any finite logit the sum is 0, or the NaN of a NaN logit)
            const float before = m2 == -INFINITY ? sum : sum * ptx::ex2_approx(m2 - off);
            const uint64_t c22 = ptx::f32x2_pack(p.c2, p.c2), off22 = ptx::f32x2_pack(-off, -off);
            uint64_t s2[4] = {ptx::f32x2_pack(before, 0.f), 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float y0, y1;
              ptx::f32x2_unpack(
                  ptx::f32x2_fma(ptx::f32x2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                 c22, off22), y0, y1);
              s2[(k / 2) & 3] = ptx::f32x2_add(
                  s2[(k / 2) & 3], ptx::f32x2_pack(ptx::ex2_approx(y0), ptx::ex2_approx(y1)));
            }
            float s0, s1;
            ptx::f32x2_unpack(
                ptx::f32x2_add(ptx::f32x2_add(s2[0], s2[1]), ptx::f32x2_add(s2[2], s2[3])), s0, s1);
            sum = s0 + s1;
            m2 = mn;
            if (p.part_sum != nullptr) {
              float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k < nc) l4[k & 3] += __uint_as_float(v[k]);
              lsum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
            }
            // Targets in the chunk; those before it are the other half's.
            while (tg.next < vc) targets_advance(tg);
            while (tg.next < vend) {
              p.pick[row * p.K + tg.cur] = pick32(v, tg.next - vc);
              targets_advance(tg);
            }
          } else {
            float d[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float pv = ptx::ex2_approx(fmaf(__uint_as_float(v[k]), p.c2, -off2));
              d[k] = fmaf(ca, pv, -cb);
            }
            // Targets.  A label's or heavy entry's logit known by itself takes the
            // place of the tensor core's, as it did in lse: of a confident token
            // p - 1 leaves little but the difference of the two.
            while (tg.next < vc) targets_advance(tg);
            while (tg.next < vend) {
              const int at = tg.next - vc;
              float w = cw, l = tok.own;
              bool exact = p.labels != nullptr;
              if (!exact) {
                const float q = __ldg(p.hit_q + row * p.K + tg.cur);
                l = __ldg(p.own_logit + row * p.K + tg.cur);  // (unset if not heavy)
                w = cw * q;
                exact = q >= kHeavy;
              }
              if (exact) {
                // (of an index given twice, the second time changes nothing)
                const float x = pick32(v, at);
                w -= ca * (ptx::ex2_approx(fmaf(l, p.c2, -off2)) -
                           ptx::ex2_approx(fmaf(x, p.c2, -off2)));
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (k == at) v[k] = __float_as_uint(l);
              }
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k == at) d[k] -= w;
              targets_advance(tg);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float x = d[k];
              if (p.cap > 0.f) {
                const float u = __uint_as_float(v[k]) * p.inv_cap;
                x *= 1.f - u * u;
              }
              v[k] = __float_as_uint(x);
            }
            // Exact zeros for ignored rows and past the piece's end.
            __syncwarp();
            if (!__all_sync(0xffffffffu, live && nc >= 32)) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!live || k >= nc) v[k] = 0u;
            }
          }
          __syncwarp();
        };
        // 64 columns at a time.  DL: a piece's last tile also writes the zeros
        // up to the end of its last panel.
        int end = ncols;
        if (KIND == LK_DL && tl.nt == p.tiles_n - 1) end = ((p.vn + 63) & ~63) - col0;
        if (row0 >= p.T) end = 0;  // (no token in the warp's rows)
#pragma unroll 1
        for (int c = 64 * half; c < end; c += (c & 32) ? 96 : 32) {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(taddr + c, v);
          ptx::tmem_ld_wait();
          const int nc = ncols - c;
          if (KIND == LK_DL || nc > 0) chunk(v, c, nc);
          if constexpr (KIND == LK_DL) {
            buf_free();
            stage_bf16<false>(buf, lane, 0, v);
            if (row0 < p.T) store_dl(&p.mapO[tl.rank], col0 + c, row0);
            if (p.split && row0 < p.T) {  // what the rounding left
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float x = __uint_as_float(v[k]);
                v[k] = __float_as_uint(x - __uint_as_float(ptx::pack_bf16x2(0.f, x) & 0xffff0000u));
              }
              buf_free();
              stage_bf16<false>(buf, lane, 0, v);
              store_dl(&p.mapO[tl.rank], col0 + c, row0 + kSplit);
            }
          }
        }
        release_acc();
        if constexpr (KIND == LK_FWD) {
          // The second warp of the lane quarter hands its part to the first.
          float* stat = sStat + trow * 3;
          if (half == 1) {
            stat[0] = m2;
            stat[1] = sum;
            stat[2] = lsum;
          }
          ptx::named_barrier_sync(1 + q, 64);
          if (half == 0 && row_ok) {
            merge(m2, sum, stat[0], stat[1]);
            const long long o = static_cast<long long>(tl.rank * p.tiles_n + tl.nt) * p.T + row;
            p.part[o] = make_float2(m2, sum);
            if (p.part_sum != nullptr) p.part_sum[o] = lsum + stat[2];
          }
        }
      } else if (!tl.dw) {
        const bool row_ok = p.split ? row < 2 * kSplit && row % kSplit < p.T : row < p.T;
        const int col0 = tl.nt * kBN;
        const int width = __any_sync(0xffffffffu, row_ok) ? min(kBN, p.D - col0) : 0;
        const bool none = tl.it_lo >= tl.it_hi;  // (no steps of a short last piece: adds nothing)
        if (!wait_tile()) break;
        float* dst = tl.part == 0
                         ? p.acc + row * p.D + col0
                         : p.parts + (static_cast<long long>(tl.shared) * (p.shares.max_parts - 1) +
                                      tl.part - 1) * (TM * kBN) +
                               (cta * kBM + trow) * kBN;
        if (p.direct && tl.alone) {
          // The sum is complete: bf16 to every rank (the all-reduce).
#pragma unroll 1
          for (int c = 64 * half; c < width; c += 128) {
            uint32_t v[2][32];
            ptx::tmem_ld_32x32b_x32(taddr + c, v[0]);
            ptx::tmem_ld_32x32b_x32(taddr + c + 32, v[1]);
            ptx::tmem_ld_wait();
            if (c + 128 >= width) release_acc();
            if (!p.first && row_ok) {
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float4 y[8];
#pragma unroll
                for (int g = 0; g < 8; ++g)
                  y[g] = c + 32 * b + 4 * g + 4 <= width
                             ? __ldcg(reinterpret_cast<const float4*>(dst + c + 32 * b + 4 * g))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  v[b][k] = __float_as_uint((none ? 0.f : __uint_as_float(v[b][k])) +
                                            reinterpret_cast<const float*>(y)[k]);
              }
            }
            __syncwarp();
            buf_free();
            stage_bf16<true>(buf, lane, 0, v[0]);
            stage_bf16<true>(buf, lane, 1, v[1]);
            store_rows(p.mapX, p.R, col0 + c, row0);
          }
        } else {
#pragma unroll 1
          for (int c = 64 * half; c < width; c += 128) {
            uint32_t v[64];
            ptx::tmem_ld_32x32b_x32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(v));
            ptx::tmem_ld_32x32b_x32(taddr + c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
            ptx::tmem_ld_wait();
            if (c + 128 >= width) release_acc();
            if (row_ok && (p.first || !none)) {
#pragma unroll
              for (int g = 0; g < 16; ++g) {
                if (c + 4 * g + 4 > width) continue;
                float4 x = make_float4(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]),
                                       __uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3]));
                if (none) x = make_float4(0.f, 0.f, 0.f, 0.f);
                // (one CTA adds to an element once per piece, so the sum's order
                // is the pieces'; the additions need no answer)
                float* o = dst + c + 4 * g;
                if (p.first)
                  *reinterpret_cast<float4*>(o) = x;
                else
                  ptx::red_add_v4_f32(o, x.x, x.y, x.z, x.w);
              }
            }
            __syncwarp();
          }
        }
        if (64 * half >= width) release_acc();
      } else {
        const int col0 = tl.nt * kBN;
        const int width = min(kBN, p.D - col0);
        if (!wait_tile()) break;
#pragma unroll 1
        for (int c = 64 * half; c < width; c += 128) {
          uint32_t v[2][32];
          ptx::tmem_ld_32x32b_x32(taddr + c, v[0]);
          ptx::tmem_ld_32x32b_x32(taddr + c + 32, v[1]);
          ptx::tmem_ld_wait();
          if (c + 128 >= width) release_acc();
          buf_free();
          stage_bf16<true>(buf, lane, 0, v[0]);
          stage_bf16<true>(buf, lane, 1, v[1]);
          // (columns past D, and rows past the piece, which are past the
          // shard, are not stored)
          if (row0 < p.vn) store_rows(&p.mapO[tl.rank], 1, col0 + c, p.v0 + row0);
        }
        if (64 * half >= width) release_acc();
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
    if constexpr (stages_out(KIND)) {
      if (lane == 0) ptx::bulk_wait_all();
    }
  } else {
    // ------------------------------------------ the targets' own logits (FWD)
    // Two warps beside the GEMM compute X_t . W_i in f32, with short chains of
    // additions, for every token's label or its teacher entries of probability
    // 1/8 or more: the logits that the loss takes from lse one by one, whose
    // errors do not average out.  2 D products for each are hidden behind the
    // 2 V D of the GEMM.  A lane holds a (token, entry); the warp computes four
    // products at a time, so that their loads are in flight together (one at a
    // time took longer than a GEMM over a small vocabulary).
    if constexpr (KIND == LK_FWD) {
      const int vecs = p.D / 8;
      const int slots = p.labels != nullptr ? 1 : kMaxHeavy;   // entries of a token
      const long long warps = 2 * static_cast<long long>(gridDim.x);
      const int group = static_cast<int>(  // tokens of a warp at a time
          min(static_cast<long long>(32 / slots), (p.T + warps - 1) / warps));
      for (long long t0 = (2 * static_cast<long long>(blockIdx.x) + warp - 2 - kEpiWarps) * group;
           t0 < p.T; t0 += warps * group) {
        const long long t = t0 + lane / slots;
        int y = -1;
        long long at = t;
        if (lane < group * slots && t < p.T) {
          if (p.labels != nullptr) {
            y = __ldg(p.labels + t);
            if (!label_live(p, y)) y = -1;
          } else {
            const int k = __ldg(p.heavy + t * kMaxHeavy + lane % kMaxHeavy);
            if (k >= 0) {
              at = t * p.K + k;
              y = __ldg(p.hit_idx + at);
            }
          }
        }
        unsigned left = __ballot_sync(0xffffffffu, y >= 0);
        while (left != 0) {
          const uint4* x[4];
          const uint4* w[4];
          int from[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            // (past the last one: the same again)
            if (u == 0 || left != 0) {
              from[u] = __ffs(left) - 1;
              left &= left - 1;
            } else {
              from[u] = from[u - 1];
            }
            const int yu = __shfl_sync(0xffffffffu, y, from[u]);
            const int r = yu / p.Vs;
            x[u] = reinterpret_cast<const uint4*>(p.X[r]) + (t0 + from[u] / slots) * vecs;
            w[u] = reinterpret_cast<const uint4*>(p.Wr[r]) +
                   static_cast<long long>(yu - r * p.Vs) * vecs;
          }
          float s[4][4] = {};
          for (int i = lane; i < vecs; i += 32) {
            uint4 a[4], b[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              a[u] = __ldg(x[u] + i);
              b[u] = __ldg(w[u] + i);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t au[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
              const uint32_t bu[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                s[u][k] = fmaf(__uint_as_float(au[k] << 16), __uint_as_float(bu[k] << 16), s[u][k]);
                s[u][k] = fmaf(__uint_as_float(au[k] & 0xffff0000u),
                               __uint_as_float(bu[k] & 0xffff0000u), s[u][k]);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float d = (s[u][0] + s[u][1]) + (s[u][2] + s[u][3]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
            if (lane == from[u]) p.own_logit[at] = d;
          }
        }
      }
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  if constexpr (kPair) {
    // The leader's MMAs read the peer's shared memory and write the peer's
    // TMEM: neither CTA frees anything before both are done.
    ptx::cluster_sync_all();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (kPair)
      ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      ptx::tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------ teacher entries
// One warp per token: the valid entries' probabilities q = softmax(teacher /
// tau) and their order by vocabulary index, written as hit_idx (INT_MAX past
// the last) and hit_q; then, per logit tile, the place of the first entry at
// or past it.  E entries per lane (lane i: places iE .. iE + E - 1) are sorted
// by (index, place in the list) with a bitonic network, whose short strides
// stay within a lane and whose long ones are shuffles.
struct TeacherArgs {
  const int32_t* idx;   // [T, K], negative = no entry
  const float* logits;  // [T, K]
  int32_t* hit_idx;
  float* hit_q;
  uint16_t* hit_start;  // [T][start_ld]
  int16_t* heavy;       // [T][kMaxHeavy]: the places of entries of probability >= kHeavy
  long long start_ld;
  FastDiv by_piece_tiles, by_npieces;
  int T, K, V, Vs;
  int npieces, piece_tiles, piece_rows, width;  // logit tiles of a rank
  float inv_tau;
  int* status;
};

constexpr int kTeacherWarps = 4;

template <int E>
__global__ void __launch_bounds__(32 * kTeacherWarps) teacher_kernel(const TeacherArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  constexpr int N = 32 * E;
  __shared__ float prob[kTeacherWarps][N];
  __shared__ int sorted[kTeacherWarps][N];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long row = static_cast<long long>(blockIdx.x) * kTeacherWarps + w;
  if (row >= a.T) return;
  int id[E];
  float x[E];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = 32 * e + lane;
    id[e] = INT_MAX;
    x[e] = -INFINITY;
    if (k < a.K) {
      const int i = __ldg(a.idx + row * a.K + k);
      if (i >= 0 && i < a.V) {
        x[e] = __ldg(a.logits + row * a.K + k);
        if (x[e] != -INFINITY) id[e] = i;  // (a logit of -inf is no entry)
      } else if (i >= a.V) {
        atomicCAS(a.status, 0, FCC_ERR_INVALID);
      }
    }
    m = fmaxf(m, x[e]);  // (drops a NaN; the sum keeps it)
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    // (the difference is taken before the scaling, which could overflow)
    x[e] = id[e] != INT_MAX ? expf((x[e] - m) * a.inv_tau) : 0.f;
    s += x[e];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  unsigned long long key[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    prob[w][32 * e + lane] = id[e] != INT_MAX ? x[e] / s : 0.f;
    key[e] = (static_cast<unsigned long long>(id[e]) << 8) | static_cast<unsigned>(32 * e + lane);
  }
  // (any start order will do: the place in the list is part of the key)
#pragma unroll
  for (int size = 2; size <= N; size <<= 1) {
#pragma unroll
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = lane * E + e;
        const bool up = (i & size) == 0;
        if (stride >= E) {
          const unsigned long long o = __shfl_xor_sync(0xffffffffu, key[e], stride / E);
          const bool low = (i & stride) == 0;
          key[e] = (low == up) == (o < key[e]) ? o : key[e];
        } else if ((e & stride) == 0) {
          unsigned long long &u = key[e], &v = key[e | (stride & (E - 1))];
          if ((v < u) == up) {
            const unsigned long long t = u;
            u = v;
            v = t;
          }
        }
      }
    }
  }
  __syncwarp();
  if (lane < kMaxHeavy) a.heavy[row * kMaxHeavy + lane] = -1;
  __syncwarp();
  int heavies = 0;  // those found so far
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int place = lane * E + e, at = static_cast<int>(key[e] >> 8);
    const float q = prob[w][key[e] & 255u];
    sorted[w][place] = at;
    if (place < a.K) {
      a.hit_idx[row * a.K + place] = at;
      a.hit_q[row * a.K + place] = q;
    }
    const unsigned those = __ballot_sync(0xffffffffu, at != INT_MAX && q >= kHeavy);
    const int mine = heavies + __popc(those & ((1u << lane) - 1u));
    if ((those >> lane & 1u) && mine < kMaxHeavy)
      a.heavy[row * kMaxHeavy + mine] = static_cast<int16_t>(place);
    heavies += __popc(those);
  }
  __syncwarp();
  for (int t = lane; t < a.start_ld; t += 32) {
    const int rp = a.by_piece_tiles.div(t);
    const int r = a.by_npieces.div(rp);
    const int col = min((rp - r * a.npieces) * a.piece_rows + (t - rp * a.piece_tiles) * a.width, a.Vs);
    const int first = r * a.Vs + col;
    int lo = 0;  // entries before `first`: all of the first lo, and maybe more
#pragma unroll
    for (int half = N / 2; half > 0; half >>= 1)
      if (sorted[w][lo + half - 1] < first) lo += half;
    if (sorted[w][lo] < first) ++lo;
    a.hit_start[row * a.start_ld + t] = static_cast<uint16_t>(lo);
  }
}

// ------------------------------------------------------------ target logits
// The backward pass's own logits of the labels or heavy entries, capped: X_t .
// W_i in f32 with short chains of additions, as the forward pass's side warps
// compute them.  There is no product to hide behind, so a token is given
// 2^log_warps warps of a CTA's eight, enough for up to four vectors of a row a
// thread, all in flight at once.  Bound by reading the rows, and by its launch
// for few: 96 tokens x 4096 5-7 us, 4096 tokens x 4096 with a teacher's entries
// 22 us (four entries at a time, for more loads in flight, took 36: 128
// registers, two CTAs to an SM).
struct TargetArgs {
  const void* X[FCC_MAX_RANKS];
  const void* W[FCC_MAX_RANKS];
  const int32_t* labels;
  const int32_t* hit_idx;
  const int16_t* heavy;
  float* own_logit;
  float cap;
  int T, D, K, V, Vs, ignore_index, log_warps;
};

__global__ void __launch_bounds__(256) target_logit_kernel(const __grid_constant__ TargetArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  __shared__ float sums[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = 32 << a.log_warps;  // threads of a token
  const int sub = threadIdx.x & (group - 1);
  const long long t = (static_cast<long long>(blockIdx.x) << (3 - a.log_warps)) +
                      (warp >> a.log_warps);
  const int vecs = a.D / 8;
  const int entries = a.labels != nullptr ? 1 : kMaxHeavy;
  for (int j = 0; j < entries; ++j) {
    int y = -1;
    long long at = t;
    if (t < a.T) {
      if (a.labels != nullptr) {
        y = __ldg(a.labels + t);
        if (y == a.ignore_index || y >= a.V) y = -1;
      } else {
        const int k = __ldg(a.heavy + t * kMaxHeavy + j);
        if (k >= 0) {
          at = t * a.K + k;
          y = __ldg(a.hit_idx + at);
        }
      }
    }
    // (a token's heavy entries come first, then -1)
    if (!__syncthreads_or(y >= 0)) break;
    float s[4] = {};
    if (y >= 0) {
      const int r = y / a.Vs;
      const uint4* x = reinterpret_cast<const uint4*>(a.X[r]) + t * vecs;
      const uint4* w =
          reinterpret_cast<const uint4*>(a.W[r]) + static_cast<long long>(y - r * a.Vs) * vecs;
#pragma unroll 4
      for (int i = sub; i < vecs; i += group) {
        const uint4 b = __ldg(x + i), c = __ldg(w + i);
        const uint32_t bu[4] = {b.x, b.y, b.z, b.w};
        const uint32_t cu[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[k] = fmaf(__uint_as_float(bu[k] << 16), __uint_as_float(cu[k] << 16), s[k]);
          s[k] = fmaf(__uint_as_float(bu[k] & 0xffff0000u), __uint_as_float(cu[k] & 0xffff0000u),
                      s[k]);
        }
      }
    }
    float d = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) sums[warp] = d;
    __syncthreads();
    if (sub == 0 && y >= 0) {
      for (int i = 1; i < 1 << a.log_warps; ++i) d += sums[warp + i];
      a.own_logit[at] = a.cap > 0.f ? a.cap * tanhf(d / a.cap) : d;
    }
  }
}

// ------------------------------------------------------------------- combine
// Merges the tiles' partials of a token over all ranks (in a fixed order) and
// writes its lse and loss to every rank.  A CTA of 256 threads takes `tok`
// tokens (a power of two up to 32); thread (token, part) merges every
// (256/tok)-th partial, then shared memory the parts.
struct CombineArgs {
  const float2* part;
  const float* part_sum;
  const float* pick;
  const float* own_logit;
  const int32_t* labels;
  const int32_t* hit_idx;
  const float* hit_q;
  float* loss[FCC_MAX_RANKS];
  float* lse[FCC_MAX_RANKS];
  int R, T, V, K, nparts, tok, ignore_index;
  float tau, c2, smoothing, z, cap;
  int* status;
};

__global__ void __launch_bounds__(256) loss_combine_kernel(const CombineArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  __shared__ float sm[256], ss[256], sl[256], sg[256];
  const int token = threadIdx.x & (a.tok - 1), part = threadIdx.x / a.tok;
  const int parts = 256 / a.tok;
  const long long t = static_cast<long long>(blockIdx.x) * a.tok + token;
  float m = -INFINITY, s = 0.f, l = 0.f;
  if (t < a.T) {
    for (int i = part; i < a.nparts; i += parts) {
      const float2 x = __ldg(a.part + static_cast<long long>(i) * a.T + t);
      merge(m, s, x.x, x.y);
      if (a.part_sum != nullptr) l += __ldg(a.part_sum + static_cast<long long>(i) * a.T + t);
    }
  }
  sm[threadIdx.x] = m;
  ss[threadIdx.x] = s;
  sl[threadIdx.x] = l;
  __syncthreads();
  for (int n = parts / 2; n > 0; n >>= 1) {
    if (part < n) {
      const int o = threadIdx.x + n * a.tok;
      merge(sm[threadIdx.x], ss[threadIdx.x], sm[o], ss[o]);
      sl[threadIdx.x] += sl[o];
    }
    __syncthreads();
  }
  m = sm[token];
  const float log2s = log2f(ss[token]);
  const float lsum = sl[token];
  __syncthreads();
  // The targets.  lse - l_k is taken in base 2 from the sum's own maximum
  // (rounded as the target's logit is here), so that a target that is the
  // maximum loses nothing.  Where the logit is also known by itself, l + e, it
  // takes the place of the tensor core's l; in the sum too, whose logarithm
  // then grows by log(1 + sum_k p_k (exp(e_k / tau) - 1)).
  float gap = 0.f, more = 0.f, own = 0.f;  // own: the label's logit
  bool live = false;
  auto target = [&](long long at, bool exact, bool in_sum) {
    const float x = __ldg(a.pick + at);
    const float x2 = __fmul_rn(x, a.c2);
    float e = 0.f;
    if (exact) {
      const float y = __ldg(a.own_logit + at);
      e = (a.cap > 0.f ? a.cap * tanhf(y / a.cap) : y) - x;
      if (in_sum) more += exp2f(x2 - m - log2s) * expm1f(e / a.tau);
    }
    own = x + e;
    return (m - x2 + log2s) * kLn2 - e / a.tau;
  };
  if (t < a.T) {
    if (a.labels != nullptr) {
      const int y = __ldg(a.labels + t);
      live = y != a.ignore_index && y >= 0 && y < a.V;
      if (part == 0) {
        if (live)
          gap = target(t, true, true);
        else if (y != a.ignore_index)
          atomicCAS(a.status, 0, FCC_ERR_INVALID);
      }
    } else {
      live = __ldg(a.hit_idx + t * a.K) != INT_MAX;
      for (int k = part; k < a.K; k += parts) {
        const long long at = t * a.K + k;
        const int id = __ldg(a.hit_idx + at);
        const float q = id != INT_MAX ? __ldg(a.hit_q + at) : 0.f;
        if (q == 0.f) continue;  // (an entry of probability 0 adds nothing)
        // (an index given often is in the sum once: with its first heavy entry,
        // whatever lies between)
        const bool exact = q >= kHeavy;
        bool again = false;
        for (long long o = at - 1; exact && !again && o >= t * a.K && __ldg(a.hit_idx + o) == id; --o)
          again = __ldg(a.hit_q + o) >= kHeavy;
        gap += q * (logf(q) + target(at, exact, !again));
      }
    }
  }
  ss[threadIdx.x] = gap;
  sg[threadIdx.x] = more;
  __syncthreads();
  for (int n = parts / 2; n > 0; n >>= 1) {
    if (part < n) {
      ss[threadIdx.x] += ss[threadIdx.x + n * a.tok];
      sg[threadIdx.x] += sg[threadIdx.x + n * a.tok];
    }
    __syncthreads();
  }
  if (part != 0 || t >= a.T) return;
  const float grow = log1pf(sg[threadIdx.x]);
  const float lse = (m + log2s) * kLn2 + grow;
  float loss = 0.f;
  if (live) {
    loss = a.tau * a.tau * (ss[threadIdx.x] + grow);  // (labels: tau = 1)
    if (a.labels != nullptr) loss += a.z * lse * lse;
    // lse - (1 - eps) l_y - eps / V sum l = (lse - l_y) + eps (l_y - mean l)
    if (a.part_sum != nullptr) loss += a.smoothing * (own - lsum / static_cast<float>(a.V));
  }
  for (int r = 0; r < a.R; ++r) {
    a.loss[r][t] = loss;
    a.lse[r][t] = lse;
  }
}

// ------------------------------------------------------------------ dX finish
// dX[r] = bf16(acc + the further parts of shared tiles) for every rank.  64
// threads of 4 columns take a row of a tile; a CTA has four such groups, for
// four rows, or (SPLIT, for tiles of many parts: a few tokens' sums over the
// whole vocabulary) for one row, each group with every fourth part.  The order
// of the sums is fixed.  (The whole backward pass of 16 tokens x 131072 x 256, whose
// one dX tile has 152 parts: 94 us with one group, 69 so.)
struct FinishArgs {
  const float* acc;
  const float* parts;
  void* out[FCC_MAX_RANKS];
  int T, D, R, split;
  int tile_m, full_tiles, first_tile;  // first_tile: those before it have left already
  Raster order;
  Shares shares;
};

template <bool SPLIT>
__global__ void __launch_bounds__(256) dx_finish_kernel(const __grid_constant__ FinishArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  constexpr int kRows = SPLIT ? 1 : 4, kGroups = SPLIT ? 4 : 1;
  __shared__ float4 red[SPLIT ? 256 : 1];
  const int per = a.tile_m / kRows;
  const int t = a.first_tile + blockIdx.x / per;
  const int group = threadIdx.x >> 6;
  const int rr = (blockIdx.x % per) * kRows + (SPLIT ? 0 : group);
  int mt, nt;
  a.order.at(t, mt, nt);
  const long long row = static_cast<long long>(mt) * a.tile_m + rr;
  if (SPLIT && row >= a.T) return;  // (the whole CTA)
  const int c = (threadIdx.x & 63) * 4;
  const int col = nt * kBN + c;
  const bool in = row < a.T && col + 4 <= a.D;
  int n = 1;
  long long part0 = 0;
  if (t >= a.full_tiles) {
    n = a.shares.parts(t - a.full_tiles);
    part0 = static_cast<long long>(t - a.full_tiles) * (a.shares.max_parts - 1);
  }
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& y) {
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  };
  if (in) {
    const long long step = static_cast<long long>(a.tile_m) * kBN;  // from part to part
    for (int half = 0; half <= a.split; ++half) {  // (the rows kSplit on are dl's second half's)
      if (!SPLIT || group == 0)
        add(__ldcs(reinterpret_cast<const float4*>(a.acc + (row + half * kSplit) * a.D + col)));
      const float* src = a.parts + part0 * step + static_cast<long long>(rr + half * kSplit) * kBN + c;
      int i = SPLIT ? group : 0;
      for (; i + 7 * kGroups < n - 1; i += 8 * kGroups) {  // (eight loads in flight)
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = __ldcs(reinterpret_cast<const float4*>(src + (i + j * kGroups) * step));
#pragma unroll
        for (int j = 0; j < 8; ++j) add(y[j]);
      }
#pragma unroll 4
      for (; i < n - 1; i += kGroups) add(__ldcs(reinterpret_cast<const float4*>(src + i * step)));
    }
  }
  if constexpr (SPLIT) {
    red[threadIdx.x] = x;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) {
      const float4 y = red[64 * g + threadIdx.x];
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
  }
  if (!in) return;
  const uint2 o = make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
  for (int r = 0; r < a.R; ++r)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out[r]) + row * a.D + col) = o;
}

// ------------------------------------------------------------------ host side
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool al(const void* p, uintptr_t a) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

template <int KIND, int CG>
cudaError_t launch_kind(const LossParams& p, int grid, cudaStream_t st) {
  auto kern = loss_gemm_kernel<KIND, CG>;
  static bool attr_set[64] = {};
  constexpr int kSmem = Cfg<KIND, CG>::kSmem;
  const cudaError_t e = smem_attr_once(attr_set, kern, kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid, 1, 1), dim3(threads_of(KIND), 1, 1), kSmem, st,
                    CG == 2 ? 2u : 1u, p);
}

// A CTA pair per tile when the rows exceed 128 and the single-CTA tiles
// outnumber the CTAs, or the caller's shape.
int choose_cg(const fcc_opts* o, int64_t rows, int64_t single_tiles, int sms) {
  if (sms < 2) return 1;
  if (o != nullptr && (o->cta_pair == 1 || o->cta_pair == 2)) return o->cta_pair;
  return rows > kBM && single_tiles > sms ? 2 : 1;
}

// Width of the logit tiles, a multiple of 32: the widest within 5 % of the least
// (rounds of tiles x clocks per 16 of D).  An MMA takes about 82 + 0.18 width
// clocks (a 128-wide one 0.81 of a 256-wide one's), so few rounds count most;
// where each tile of W is read by one CTA only (one row of tiles), its share of
// the memory bandwidth, 21 bytes per clock, is what counts: one token on 32000
// words takes 143 tiles of 224 columns in one round, not 125 of 256 (48 us
// against 54); 64 tokens on 131072 words four rounds of 224, not nine of 96 (313
// against 325).
int choose_width(int R, int64_t tiles_m, int64_t vn, int slots) {
  auto cost = [&](int w) {
    const double mma = 82 + 0.18 * w, mem = tiles_m == 1 ? w * 32 / 21.0 : 0;
    return static_cast<double>(cdiv(tiles_m * R * cdiv(vn, w), slots)) * std::max(mma, mem);
  };
  double least = cost(kBN);
  for (int w = kBN - 32; w >= 32; w -= 32) least = std::min(least, cost(w));
  int w = kBN;
  while (cost(w) > 1.05 * least) w -= 32;
  return w;
}

// The shares of `rest` tiles of k steps over at most `slots` CTAs (pairs), of
// eight steps at least: shorter ones make more parts to sum than they save (64
// tokens x 8000 x 1024: 35 us, against 53 with four and 42 with sixteen).
Shares plan_shares(int rest, int k, int slots) {
  Shares s;
  std::memset(&s, 0, sizeof(s));
  s.max_parts = 1;
  if (rest == 0) return s;
  const int64_t total = static_cast<int64_t>(rest) * k;
  s.tiles = rest;
  s.k = k;
  s.ctas = static_cast<int>(std::max<int64_t>(rest, std::min<int64_t>(slots, total / 8)));
  s.groups = s.ctas / rest;
  s.helpers = s.ctas - s.groups * rest;
  s.len = static_cast<int>(s.helpers > 0 ? cdiv(total, s.ctas) : cdiv(k, s.groups));
  s.tail = std::max(0, k - s.groups * s.len);
  s.helpers = static_cast<int>(std::min<int64_t>(s.helpers, s.tails()));  // (none of them idle)
  for (int i = 0; i < rest; ++i) s.max_parts = std::max(s.max_parts, s.parts(i));
  return s;
}

int slots_of(int cg, int sms) { return std::max(1, std::min(sms / cg, gemm_max_clusters(cg))); }

// One of the products over at most `sms` CTAs.  The logit tiles are counted
// here; the gradients' tiles are planned by the caller.
template <int KIND>
cudaError_t launch_loss_gemm(LossParams& p, int cg, int sms, cudaStream_t st) {
  const int64_t tm = static_cast<int64_t>(kBM) * cg;
  const int slots = slots_of(cg, sms);
  int64_t busy = 0;
  if (KIND != LK_GRAD) {
    p.tiles_m = static_cast<int>(cdiv(p.T, tm));
    p.tiles_n = static_cast<int>(cdiv(p.vn, p.width));
    p.k_iters = static_cast<int>(cdiv(p.D, kBK));
    busy = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.R;
    if (busy > (1ll << 30)) return cudaErrorInvalidValue;
    p.full_tiles = static_cast<int>(busy);
    if (kGroupM * static_cast<int64_t>(p.R) * p.tiles_n > (1ll << 30)) return cudaErrorInvalidValue;
    p.order = raster_of(p.tiles_m, p.R * p.tiles_n, kGroupM);
    p.by_tiles_n = fast_div(p.tiles_n);
    // (the MMA reads 128 rows of A from every stage, whatever lies past its box)
    p.a_size = static_cast<uint32_t>(cdiv(p.a_rows, 8) * 1024);
    p.stage_size = p.a_size + static_cast<uint32_t>(p.width / cg) * kBK * 2;
    const uint32_t ring = cg == 2 ? Cfg<KIND, 2>::kRing : Cfg<KIND, 1>::kRing;
    p.stages = std::min<uint32_t>((ring - kABytes) / p.stage_size + 1, ring / p.stage_size);
    p.stages = std::min<uint32_t>(p.stages, cg == 2 ? Cfg<KIND, 2>::kMaxStages : Cfg<KIND, 1>::kMaxStages);
  } else {
    busy = std::max({p.full_tiles, p.shares.groups * p.shares.tiles + p.shares.helpers, p.dw_tiles});
  }
  const double w_bytes = 2.0 * p.R * p.vn * p.D;
  p.keep = p.tiles_m == 1 && w_bytes > kKeepFrom && w_bytes < kKeepTo
               ? static_cast<float>(kKeepBytes / w_bytes) : 0.f;
  const int grid = cg * static_cast<int>(std::min<int64_t>(slots, busy));
  return cg == 2 ? launch_kind<KIND, 2>(p, grid, st) : launch_kind<KIND, 1>(p, grid, st);
}

// What one call is about, checked.
struct Call {
  int R;
  const void* const* X;
  const void* const* W;
  const int32_t* labels;
  const int32_t* teacher_idx;
  const float* teacher;
  int64_t T, V, D;
  int K;
  int32_t ignore_index;
  float smoothing, z, softcap, tau;
  fcc_dtype in;
  const fcc_opts* opts;
  cudaStream_t st;
};

fcc_status check_call(const Call& c) {
  if (c.R < 1 || c.R > FCC_MAX_RANKS) return FCC_ERR_INVALID;
  if (c.T < 1 || c.V < 1 || c.D < 8 || c.D % 8 != 0 || c.V % c.R != 0) return FCC_ERR_INVALID;
  if (c.T > (1ll << 28) || c.V > (1ll << 30) || c.D > (1ll << 24)) return FCC_ERR_INVALID;
  if (c.X == nullptr || c.W == nullptr) return FCC_ERR_INVALID;
  for (int r = 0; r < c.R; ++r)
    if (!al(c.X[r], 16) || !al(c.W[r], 16)) return FCC_ERR_INVALID;
  if (c.in != FCC_BF16 && c.in != FCC_F16 && c.in != FCC_F32) return FCC_ERR_INVALID;
  // (a cap's double and reciprocal, a temperature's square: normal numbers)
  if (!(c.softcap == 0.f || (c.softcap >= 0x1p-126f && c.softcap <= 0x1p126f))) return FCC_ERR_INVALID;
  if (c.K == 0) {
    if (!al(c.labels, 4)) return FCC_ERR_INVALID;
    if (!(c.smoothing >= 0.f && c.smoothing < 1.f)) return FCC_ERR_INVALID;
    if (!(c.z >= 0.f) || std::isinf(c.z)) return FCC_ERR_INVALID;
  } else {
    if (c.K < 1 || c.K > FCC_MAX_TEACHER) return FCC_ERR_INVALID;
    if (!al(c.teacher_idx, 4) || !al(c.teacher, 4)) return FCC_ERR_INVALID;
    if (!(c.tau >= 0x1p-63f && c.tau <= 0x1p63f)) return FCC_ERR_INVALID;
  }
  const fcc_opts* o = c.opts;
  if (o != nullptr) {
    if (o->algo < FCC_ALGO_AUTO || o->algo > FCC_ALGO_CE) return FCC_ERR_INVALID;
    if (o->cta_pair < 0 || o->cta_pair > 2 || o->chunks < 0) return FCC_ERR_INVALID;
    if (o->algo != FCC_ALGO_AUTO && o->algo != FCC_ALGO_FUSED) return FCC_ERR_UNSUPPORTED;
  }
  return c.in == FCC_BF16 ? FCC_OK : FCC_ERR_UNSUPPORTED;
}

int usable_sms(const fcc_opts* o) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms = 256;  // (no device: sizes for the largest plan)
  }
  return o != nullptr && o->max_ctas > 0 ? std::min(sms, o->max_ctas) : sms;
}

// Scratch layout.  Target logits; distillation also the sorted teacher entries.
// Forward: partials.  Backward: the piece's dl, the f32 sums of dX.
struct Plan {
  size_t hit_idx = 0, hit_q = 0, hit_start = 0, heavy = 0, pick = 0, own_logit = 0, part = 0, part_sum = 0;
  size_t dl = 0, acc = 0, parts = 0, total = 0;
  int cg = 1, width = kBN;  // logit tiles
  int nparts = 0;
  int64_t piece = 0;        // vocabulary rows of a piece, per rank (forward: all)
  int npieces = 1, piece_tiles = 0;
};

constexpr size_t kPieceBytes = size_t(512) << 20;  // dl held at a time

// Rows of a dl panel.
int64_t tpad_of(int64_t T) { return T <= kSplit ? 2 * kSplit : cdiv(T, 32) * 32; }

Plan plan_of(int R, int64_t T, int64_t V, int64_t D, int K, bool grad, bool smoothing, bool want_dx,
             int sms, const fcc_opts* o) {
  Plan p;
  size_t off = 0;
  const int64_t Vs = V / R, tpad = tpad_of(T);
  if (K > 0) {
    p.hit_idx = off;
    off += up256(static_cast<size_t>(T) * K * 4);
    p.hit_q = off;
    off += up256(static_cast<size_t>(T) * K * 4);
  }
  int64_t rows = Vs;  // vocabulary rows of a launch, per rank
  p.piece = Vs;
  if (grad) {
    // Equal pieces, whole tiles of 256 rows, as few as hold kPieceBytes of dl
    // (or the caller's count).
    const int64_t most = std::max<int64_t>(
        kBN, static_cast<int64_t>(kPieceBytes / (static_cast<size_t>(tpad) * R * 2)) / kBN * kBN);
    int64_t n = o != nullptr && o->chunks > 0 ? o->chunks : cdiv(Vs, most);
    n = std::max<int64_t>(1, std::min(n, cdiv(Vs, kBN)));
    p.piece = cdiv(cdiv(Vs, n), kBN) * kBN;
    rows = std::min(p.piece, Vs);
    p.npieces = static_cast<int>(cdiv(Vs, p.piece));
  }
  p.cg = choose_cg(o, T, cdiv(T, kBM) * R * cdiv(rows, kBN), sms);
  p.width = choose_width(R, cdiv(T, kBM * p.cg), rows, std::max(1, sms / p.cg));
  p.piece_tiles = static_cast<int>(cdiv(rows, p.width));
  if (K > 0) {
    p.hit_start = off;
    off += up256(static_cast<size_t>(T) * R * p.npieces * p.piece_tiles * 2);
    p.heavy = off;
    off += up256(static_cast<size_t>(T) * kMaxHeavy * 2);
  }
  p.own_logit = off;
  off += up256(static_cast<size_t>(T) * std::max(K, 1) * 4);
  if (!grad) {
    p.nparts = static_cast<int>(R * cdiv(Vs, p.width));
    p.pick = off;
    off += up256(static_cast<size_t>(T) * std::max(K, 1) * 4);
    p.part = off;
    off += up256(static_cast<size_t>(p.nparts) * T * 8);
    p.part_sum = off;
    if (smoothing) off += up256(static_cast<size_t>(p.nparts) * T * 4);
  } else {
    p.dl = off;
    off += up256(static_cast<size_t>(R) * tpad * p.piece * 2);
    if (want_dx) {
      p.acc = off;
      off += up256(static_cast<size_t>(T <= kSplit ? 2 * kSplit : T) * D * 4);
      // Blocks for the shared tiles' further parts: fewer than the shares and
      // the shared tiles together, each at most the CTAs (pairs).
      const int64_t tiles = cdiv(T, kBM) * cdiv(D, kBN);
      const int64_t steps = tiles * R * cdiv(rows, kBK);
      p.parts = off;
      off += up256(std::min(static_cast<size_t>(2 * sms) * (kBM * kBN * 4),
                            static_cast<size_t>(steps / 4 + tiles + 1) * (2 * kBM * kBN * 4)));
    }
  }
  p.total = off;
  return p;
}

void common_params(LossParams& p, const Call& c, const Plan& pl, char* base, int* status,
                   unsigned long long timeout_ns) {
  std::memset(&p, 0, sizeof(p));
  p.R = c.R;
  p.T = static_cast<int>(c.T);
  p.D = static_cast<int>(c.D);
  p.Vs = static_cast<int>(c.V / c.R);
  p.v0 = 0;
  p.vn = p.Vs;
  p.width = pl.width;
  p.npieces = pl.npieces;
  p.piece_tiles = pl.piece_tiles;
  p.start_ld = static_cast<long long>(c.R) * pl.npieces * pl.piece_tiles;
  p.split = c.T <= kSplit ? 1 : 0;
  p.tpad = static_cast<int>(tpad_of(c.T));
  p.a_rows = static_cast<int>(std::min<int64_t>(c.T, kBM));
  p.k_rows = static_cast<int>(std::min<int64_t>(cdiv(c.T, 16) * 16, kBK));
  p.K = std::max(c.K, 1);
  if (c.K == 0) {
    p.labels = c.labels;
  } else {
    p.hit_idx = reinterpret_cast<int32_t*>(base + pl.hit_idx);
    p.hit_q = reinterpret_cast<float*>(base + pl.hit_q);
    p.hit_start = reinterpret_cast<uint16_t*>(base + pl.hit_start);
    p.heavy = reinterpret_cast<int16_t*>(base + pl.heavy);
  }
  p.own_logit = reinterpret_cast<float*>(base + pl.own_logit);
  for (int r = 0; r < c.R; ++r) {
    p.X[r] = c.X[r];
    p.Wr[r] = c.W[r];
  }
  p.ignore_index = c.ignore_index;
  p.cap = c.softcap;
  p.inv_cap = c.softcap > 0.f ? 1.f / c.softcap : 0.f;
  p.tau = c.tau;
  p.c2 = static_cast<float>(1.4426950408889634 / c.tau);
  p.grow = 1.f + kCutPerStep * static_cast<float>(std::min(cdiv(c.D, 16), kCutSteps));
  p.smoothing = c.smoothing;
  p.z = c.z;
  p.status = status;
  p.timeout_ns = timeout_ns;
}

// Teacher entries: probabilities and vocabulary order.
cudaError_t launch_teacher(const Call& c, const Plan& pl, char* base, int* status) {
  TeacherArgs a;
  a.idx = c.teacher_idx;
  a.logits = c.teacher;
  a.hit_idx = reinterpret_cast<int32_t*>(base + pl.hit_idx);
  a.hit_q = reinterpret_cast<float*>(base + pl.hit_q);
  a.T = static_cast<int>(c.T);
  a.K = c.K;
  a.V = static_cast<int>(c.V);
  a.inv_tau = 1.f / c.tau;
  a.status = status;
  a.hit_start = reinterpret_cast<uint16_t*>(base + pl.hit_start);
  a.heavy = reinterpret_cast<int16_t*>(base + pl.heavy);
  a.by_piece_tiles = fast_div(pl.piece_tiles);
  a.by_npieces = fast_div(pl.npieces);
  a.start_ld = static_cast<long long>(c.R) * pl.npieces * pl.piece_tiles;
  a.Vs = static_cast<int>(c.V / c.R);
  a.npieces = pl.npieces;
  a.piece_tiles = pl.piece_tiles;
  a.piece_rows = static_cast<int>(pl.piece);
  a.width = pl.width;
  const auto kern = c.K <= 32 ? teacher_kernel<1> : c.K <= 64 ? teacher_kernel<2>
                    : c.K <= 128 ? teacher_kernel<4> : teacher_kernel<8>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(cdiv(c.T, kTeacherWarps))),
                    dim3(32 * kTeacherWarps), 0, c.st, 1u, a);
}

// The labels' or heavy entries' own logits, for the backward pass.
cudaError_t launch_targets(const Call& c, const LossParams& p) {
  TargetArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int r = 0; r < c.R; ++r) {
    a.X[r] = c.X[r];
    a.W[r] = c.W[r];
  }
  a.labels = p.labels;
  a.hit_idx = p.hit_idx;
  a.heavy = p.heavy;
  a.own_logit = p.own_logit;
  a.cap = p.cap;
  a.T = p.T;
  a.D = p.D;
  a.K = p.K;
  a.V = static_cast<int>(c.V);
  a.Vs = p.Vs;
  a.ignore_index = p.ignore_index;
  while (a.log_warps < 3 && (128 << a.log_warps) < p.D / 8) ++a.log_warps;
  const int64_t tokens = 8 >> a.log_warps;  // of a CTA
  return launch_pdl(target_logit_kernel, dim3(static_cast<unsigned>(cdiv(c.T, tokens))), dim3(256),
                    0, c.st, 1u, a);
}

// Tensor maps of the logit product: X rows and W rows, both K-major.
fcc_status logit_maps(LossParams& p, const Call& c, const Plan& pl) {
  for (int r = 0; r < c.R; ++r) {
    fcc_status s = internal_encode_map(&p.mapA[r], c.X[r], c.T, c.D, c.D,
                                       static_cast<uint32_t>(p.a_rows));
    if (s == FCC_OK)
      s = internal_encode_map(&p.mapB[r], c.W[r], c.V / c.R, c.D, c.D,
                              static_cast<uint32_t>(pl.width / pl.cg));
    if (s != FCC_OK) return s;
  }
  return FCC_OK;
}

fcc_status forward(const Call& c, float* const* loss, float* const* lse) {
  fcc_status s = check_call(c);
  if (s == FCC_ERR_INVALID) return s;
  if (loss == nullptr || lse == nullptr) return FCC_ERR_INVALID;
  for (int r = 0; r < c.R; ++r)
    if (!al(loss[r], 4) || !al(lse[r], 4)) return FCC_ERR_INVALID;
  if (s != FCC_OK) return s;
  const Plan pl = plan_of(c.R, c.T, c.V, c.D, c.K, false, c.smoothing > 0.f, false,
                          usable_sms(c.opts), c.opts);
  void* ws = nullptr;
  int* status = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  if ((s = internal_prepare(c.opts, pl.total, &ws, &status, &sms, &timeout_ns)) != FCC_OK) return s;
  char* base = static_cast<char*>(ws);
  LossParams p;
  common_params(p, c, pl, base, status, timeout_ns);
  p.part = reinterpret_cast<float2*>(base + pl.part);
  p.part_sum = c.smoothing > 0.f ? reinterpret_cast<float*>(base + pl.part_sum) : nullptr;
  p.pick = reinterpret_cast<float*>(base + pl.pick);
  if ((s = logit_maps(p, c, pl)) != FCC_OK) return s;
  uint64_t launches = 2;
  if (c.K > 0) {
    if (launch_teacher(c, pl, base, status) != cudaSuccess) return FCC_ERR_CUDA;
    ++launches;
  }
  if (launch_loss_gemm<LK_FWD>(p, pl.cg, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
  CombineArgs a;
  std::memset(&a, 0, sizeof(a));
  a.part = p.part;
  a.part_sum = p.part_sum;
  a.pick = p.pick;
  a.own_logit = p.own_logit;
  a.labels = p.labels;
  a.hit_idx = p.hit_idx;
  a.hit_q = p.hit_q;
  for (int r = 0; r < c.R; ++r) {
    a.loss[r] = loss[r];
    a.lse[r] = lse[r];
  }
  a.R = c.R;
  a.T = p.T;
  a.V = static_cast<int>(c.V);
  a.K = p.K;
  a.nparts = pl.nparts;
  a.ignore_index = c.ignore_index;
  a.tau = c.tau;
  a.c2 = p.c2;
  a.smoothing = c.smoothing;
  a.z = c.z;
  a.cap = c.softcap;
  a.status = status;
  // Tokens per CTA: 32 when that still fills the SMs, fewer for few tokens.
  a.tok = 32;
  while (a.tok > 1 && cdiv(c.T, a.tok) < sms) a.tok >>= 1;
  if (launch_pdl(loss_combine_kernel, dim3(static_cast<unsigned>(cdiv(c.T, a.tok))), dim3(256), 0, c.st,
                 1u, a) != cudaSuccess)
    return FCC_ERR_CUDA;
  bump_launch_count(launches);
  return FCC_OK;
}

fcc_status backward(const Call& c, const float* const* lse, const float* dloss, void* const* dX,
                    void* const* dW, fcc_dtype out_dtype) {
  fcc_status s = check_call(c);
  if (s == FCC_ERR_INVALID) return s;
  if (lse == nullptr || !al(dloss, 4) || (dX == nullptr && dW == nullptr)) return FCC_ERR_INVALID;
  for (int r = 0; r < c.R; ++r) {
    if (!al(lse[r], 4)) return FCC_ERR_INVALID;
    if (dX != nullptr && !al(dX[r], 16)) return FCC_ERR_INVALID;
    if (dW != nullptr && !al(dW[r], 16)) return FCC_ERR_INVALID;
  }
  if (out_dtype != FCC_BF16 && out_dtype != FCC_F16 && out_dtype != FCC_F32) return FCC_ERR_INVALID;
  if (s != FCC_OK) return s;
  if (out_dtype != FCC_BF16) return FCC_ERR_UNSUPPORTED;
  const bool want_dx = dX != nullptr, want_dw = dW != nullptr;
  const int usable = usable_sms(c.opts);
  const Plan pl = plan_of(c.R, c.T, c.V, c.D, c.K, true, false, want_dx, usable, c.opts);
  void* ws = nullptr;
  int* status = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  if ((s = internal_prepare(c.opts, pl.total, &ws, &status, &sms, &timeout_ns)) != FCC_OK) return s;
  char* base = static_cast<char*>(ws);
  LossParams base_p;
  common_params(base_p, c, pl, base, status, timeout_ns);
  base_p.dloss = dloss;
  for (int r = 0; r < c.R; ++r) base_p.lse[r] = lse[r];
  const int64_t Vs = c.V / c.R, rows = std::min(pl.piece, Vs);
  uint64_t launches = 0;
  if (c.K > 0) {
    if (launch_teacher(c, pl, base, status) != cudaSuccess) return FCC_ERR_CUDA;
    ++launches;
  }
  if (launch_targets(c, base_p) != cudaSuccess) return FCC_ERR_CUDA;
  ++launches;
  LossParams p_dl = base_p, p = base_p;
  if ((s = logit_maps(p_dl, c, pl)) != FCC_OK) return s;
  // Gradient tiles: a CTA pair each when there are more than 128 tokens.
  const int cg = sms < 2 ? 1
                 : c.opts != nullptr && c.opts->cta_pair != 0 ? c.opts->cta_pair
                 : c.T > kBM ? 2 : 1;
  const int slots = slots_of(cg, sms);
  const int64_t tm = static_cast<int64_t>(kBM) * cg;
  p.width = kBN;
  if (p.split) p.a_rows = kSplit + p.T;
  p.tiles_m = static_cast<int>(cdiv(c.T, tm));
  p.tiles_n = static_cast<int>(cdiv(c.D, kBN));
  p.order = raster_of(p.tiles_m, p.tiles_n, kGroupM);
  int dx_tiles = 0;
  if (want_dx) {
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (tiles > (1ll << 24)) return FCC_ERR_INVALID;
    dx_tiles = static_cast<int>(tiles);
    p.full_tiles = dx_tiles / slots * slots;
    p.shares = plan_shares(dx_tiles - p.full_tiles, static_cast<int>(c.R * cdiv(rows, kBK)), slots);
    const size_t blocks = static_cast<size_t>(p.shares.tiles) * (p.shares.max_parts - 1);
    if (blocks * cg * (kBM * kBN * 4) > pl.total - pl.parts) return FCC_ERR_INVALID;
    p.acc = reinterpret_cast<float*>(base + pl.acc);
    p.parts = reinterpret_cast<float*>(base + pl.parts);
  }
  if (want_dw && cdiv(rows, tm) * c.R * p.tiles_n > (1ll << 30)) return FCC_ERR_INVALID;
  const int64_t panels = pl.piece / 64;
  if (panels * p.tpad > INT32_MAX) return FCC_ERR_INVALID;
  for (int r = 0; r < c.R; ++r) {
    // W and X again, MN-major boxes
    if ((s = internal_encode_map(&p.mapB[r], c.W[r], Vs, c.D, c.D, kBK)) != FCC_OK ||
        (s = internal_encode_map(&p.mapB2[r], c.X[r], c.T, c.D, c.D, p.k_rows)) != FCC_OK)
      return s;
    if (want_dw && (s = internal_encode_map(&p.mapO[r], dW[r], Vs, c.D, c.D, 32)) != FCC_OK)
      return s;
    if (want_dx && (s = internal_encode_map(&p.mapX[r], dX[r], c.T, c.D, c.D, 32)) != FCC_OK)
      return s;
    // dl's panels, one below another
    const char* d = base + pl.dl + static_cast<size_t>(r) * panels * p.tpad * 128;
    const int64_t dl_rows = panels * p.tpad;
    if ((s = internal_encode_map(&p_dl.mapO[r], d, dl_rows, 64, 64, 32, 32)) != FCC_OK ||
        (s = internal_encode_map(&p.mapA[r], d, dl_rows, 64, 64, p.a_rows)) != FCC_OK ||
        (s = internal_encode_map(&p.mapA2[r], d, dl_rows, 64, 64, p.k_rows)) != FCC_OK)
      return s;
  }
  for (int64_t v0 = 0; v0 < Vs; v0 += pl.piece) {
    const int vn = static_cast<int>(std::min(pl.piece, Vs - v0));
    p_dl.v0 = p.v0 = static_cast<int>(v0);
    p_dl.vn = p.vn = vn;
    p_dl.piece = static_cast<int>(v0 / pl.piece);
    if (launch_loss_gemm<LK_DL>(p_dl, pl.cg, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
    p.first = v0 == 0 ? 1 : 0;
    p.direct = want_dx && v0 + vn == Vs && !p.split ? 1 : 0;
    p.kb_per_rank = static_cast<int>(cdiv(vn, kBK));
    p.k_iters = c.R * p.kb_per_rank;
    if (want_dw) {
      p.dw_tiles_m = static_cast<int>(cdiv(vn, tm));
      p.dw_tiles = p.dw_tiles_m * c.R * p.tiles_n;
      p.dw_order = raster_of(p.dw_tiles_m * c.R, p.tiles_n, kGroupM);
      p.by_dw_tiles_m = fast_div(p.dw_tiles_m);
    }
    if (launch_loss_gemm<LK_GRAD>(p, cg, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
    launches += 2;
  }
  // (direct: nothing is left to sum but the shared tiles)
  const int first_tile = p.direct ? p.full_tiles : 0;
  if (want_dx && first_tile < dx_tiles && !(p.direct && p.shares.alone())) {
    FinishArgs f;
    std::memset(&f, 0, sizeof(f));
    f.acc = p.acc;
    f.parts = p.parts;
    for (int r = 0; r < c.R; ++r) f.out[r] = dX[r];
    f.T = p.T;
    f.D = p.D;
    f.R = c.R;
    f.split = p.split;
    f.tile_m = static_cast<int>(tm);
    f.order = p.order;
    f.full_tiles = p.full_tiles;
    f.first_tile = first_tile;
    f.shares = p.shares;
    const bool many = p.shares.max_parts > 8;
    const int blocks = (dx_tiles - first_tile) * (many ? f.tile_m : f.tile_m / 4);
    if (launch_pdl(many ? dx_finish_kernel<true> : dx_finish_kernel<false>,
                   dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.st, 1u, f) != cudaSuccess)
      return FCC_ERR_CUDA;
    ++launches;
  }
  bump_launch_count(launches);
  return FCC_OK;
}

}  // namespace
}  // namespace fcc

using namespace fcc;

extern "C" {

size_t fcc_linear_loss_workspace_size(int R, int64_t T, int64_t V, int64_t D, int topk, int grad,
                                      const fcc_opts* opts) {
  if (R < 1 || R > FCC_MAX_RANKS || T < 1 || V < R || D < 1 || topk < 0 || topk > FCC_MAX_TEACHER)
    return 0;
  return plan_of(R, T, V, D, topk, grad != 0, topk == 0, true, usable_sms(opts), opts).total;
}

fcc_status fcc_linear_xent(int R, const void* const* X, const void* const* W, const int32_t* labels,
                           int64_t T, int64_t V, int64_t D, float* const* loss, float* const* lse,
                           int32_t ignore_index, float smoothing, float z_weight, float softcap,
                           fcc_dtype in, const fcc_opts* opts, fcc_stream_t stream) {
  const Call c{R, X, W, labels, nullptr, nullptr, T, V, D, 0, ignore_index, smoothing, z_weight,
               softcap, 1.f, in, opts, reinterpret_cast<cudaStream_t>(stream)};
  return forward(c, loss, lse);
}

fcc_status fcc_linear_xent_grad(int R, const void* const* X, const void* const* W,
                                const int32_t* labels, const float* const* lse, const float* dloss,
                                int64_t T, int64_t V, int64_t D, void* const* dX, void* const* dW,
                                int32_t ignore_index, float smoothing, float z_weight,
                                float softcap, fcc_dtype in, fcc_dtype out_dtype,
                                const fcc_opts* opts, fcc_stream_t stream) {
  const Call c{R, X, W, labels, nullptr, nullptr, T, V, D, 0, ignore_index, smoothing, z_weight,
               softcap, 1.f, in, opts, reinterpret_cast<cudaStream_t>(stream)};
  return backward(c, lse, dloss, dX, dW, out_dtype);
}

fcc_status fcc_linear_distill(int R, const void* const* X, const void* const* W,
                              const int32_t* teacher_idx, const float* teacher_logits, int64_t T,
                              int64_t V, int64_t D, int topk, float* const* loss,
                              float* const* lse, float temperature, float softcap, fcc_dtype in,
                              const fcc_opts* opts, fcc_stream_t stream) {
  if (topk < 1) return FCC_ERR_INVALID;
  const Call c{R, X, W, nullptr, teacher_idx, teacher_logits, T, V, D, topk, 0, 0.f, 0.f, softcap,
               temperature, in, opts, reinterpret_cast<cudaStream_t>(stream)};
  return forward(c, loss, lse);
}

fcc_status fcc_linear_distill_grad(int R, const void* const* X, const void* const* W,
                                   const int32_t* teacher_idx, const float* teacher_logits,
                                   const float* const* lse, const float* dloss, int64_t T,
                                   int64_t V, int64_t D, int topk, void* const* dX,
                                   void* const* dW, float temperature, float softcap, fcc_dtype in,
                                   fcc_dtype out_dtype, const fcc_opts* opts,
                                   fcc_stream_t stream) {
  if (topk < 1) return FCC_ERR_INVALID;
  const Call c{R, X, W, nullptr, teacher_idx, teacher_logits, T, V, D, topk, 0, 0.f, 0.f, softcap,
               temperature, in, opts, reinterpret_cast<cudaStream_t>(stream)};
  return backward(c, lse, dloss, dX, dW, out_dtype);
}

}  // extern "C"
