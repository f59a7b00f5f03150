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
// epilogue thread owns one token's 256 logits of the tile in TMEM and reduces
// them to a running maximum and sum (base 2), their plain sum when smoothing
// asks for it, and the logits at the token's targets; one partial per (tile,
// token) goes to memory and combine_kernel merges the partials of all ranks:
// the all-reduce of the softmax statistics.
// Backward, per piece of the vocabulary: the same product again, whose
// epilogue turns logits into dl (bf16) for the piece; then dX += dl W (the K
// loop runs over all ranks: the all-reduce) and dW = dl^T X.  Only one piece
// of dl is ever held.
//
// All products run on tcgen05 (bf16 x bf16 -> f32 in TMEM), fed by TMA through
// an mbarrier ring: warp 0 loads, warp 1 issues the MMAs into one of two TMEM
// accumulators, warps 2-5 are the epilogue of the other.  CG = 1: one CTA per
// 128 x 256 tile; CG = 2: a CTA pair per 256 x 256 tile.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

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
  LK_FWD = 0,  // logits -> softmax statistics and target logits
  LK_DL = 1,   // logits -> dl of one vocabulary piece
  LK_DX = 2,   // dX (+)= dl W over the ranks' pieces
  LK_DW = 3,   // dW rows of the piece = dl^T X
};
// Operand layouts: X and W rows are contiguous along D, dl rows along the
// vocabulary.  Logits contract D (both K-major); dX contracts the vocabulary
// (dl K-major, W MN-major); dW contracts the tokens (both MN-major).
constexpr bool a_mn(int kind) { return kind == LK_DW; }
constexpr bool b_mn(int kind) { return kind == LK_DX || kind == LK_DW; }

template <int KIND, int CG>
struct Cfg {
  static constexpr int kTileM = kBM * CG;
  static constexpr int kBNcta = kBN / CG;                  // B columns this CTA holds
  static constexpr int kStages = CG == 2 ? 7 : 4;
  static constexpr uint32_t kBBytes = kBK * kBNcta * 2;    // 32 or 16 KiB
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  static constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(kTileM, kBN, a_mn(KIND), b_mn(KIND));
  static constexpr int kSmem =
      1024 + kStages * static_cast<int>(kStageBytes) + (2 * kStages + 5) * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct LossParams {
  CUtensorMap mapA[FCC_MAX_RANKS];
  CUtensorMap mapB[FCC_MAX_RANKS];
  int R, T, D;
  int Vs;                  // vocabulary rows per rank
  int v0, vn;              // this piece: rows [v0, v0 + vn) of every rank (FWD: 0, Vs)
  int tiles_m, tiles_n;    // tiles of one rank (DX: of all)
  int num_tiles;
  int k_iters;             // 64-deep K steps of a whole tile
  int kb_per_rank;         // DX: K steps per rank
  int splits;              // DX: parts of the K loop, each with its own f32 slab
  int group_m;             // raster group height (tiles)
  // tokens' targets: labels (cross entropy), or per token K sorted vocabulary
  // indices (INT_MAX past the last) and their teacher probabilities
  const int32_t* labels;
  const int32_t* hit_idx;  // [T, K]
  const float* hit_q;      // [T, K]
  int K;
  int ignore_index;
  float cap, inv_cap;      // soft cap, 0 = none
  float c2;                // log2(e) / tau
  float tau, smoothing, z;
  // FWD
  float2* part;            // [R * tiles_n][T]: base-2 maximum and sum
  float* part_sum;         // the same layout: sum of the logits (smoothing), or NULL
  float* pick;             // [T, K] logits at the targets
  // DL
  const float* lse[FCC_MAX_RANKS];
  const float* dloss;
  // dl: [R][T][ldl] bf16 (DL writes it, the tensor maps of DX and DW read it)
  uint16_t* dl;
  long long ldl;
  // DX: f32 slabs [splits][T][D]; first = 1: overwrite, else add
  float* acc;
  int first;
  // DW
  void* out[FCC_MAX_RANKS];  // [Vs, D] bf16
  int* status;
  unsigned long long timeout_ns;
};

struct Tile {
  int rank, mt, nt;
  int it_lo, it_hi;  // K steps
  int split;
};

__device__ __forceinline__ void raster(int t, int tiles_m, int tiles_n, int group, int& mt,
                                       int& nt) {
  const int per_group = group * tiles_n;
  const int g = t / per_group;
  const int first = g * group;
  const int gm = min(group, tiles_m - first);
  const int local = t - g * per_group;
  mt = first + local % gm;
  nt = local / gm;
}

template <int KIND>
__device__ __forceinline__ Tile tile_of(const LossParams& p, int t) {
  Tile tl;
  tl.rank = 0;
  tl.split = 0;
  tl.it_lo = 0;
  tl.it_hi = p.k_iters;
  if constexpr (KIND == LK_FWD || KIND == LK_DL) {
    raster(t, p.tiles_m, p.R * p.tiles_n, p.group_m, tl.mt, tl.nt);
    tl.rank = tl.nt / p.tiles_n;
    tl.nt -= tl.rank * p.tiles_n;
  } else if constexpr (KIND == LK_DX) {
    const int per = p.tiles_m * p.tiles_n;
    tl.split = t / per;
    raster(t - tl.split * per, p.tiles_m, p.tiles_n, p.group_m, tl.mt, tl.nt);
    tl.it_lo = static_cast<int>(static_cast<long long>(p.k_iters) * tl.split / p.splits);
    tl.it_hi = static_cast<int>(static_cast<long long>(p.k_iters) * (tl.split + 1) / p.splits);
  } else {
    raster(t, p.R * p.tiles_m, p.tiles_n, p.group_m, tl.mt, tl.nt);
    tl.rank = tl.mt / p.tiles_m;
    tl.mt -= tl.rank * p.tiles_m;
  }
  return tl;
}

// A warp's 32 x 32 block (lane i: 32 columns of its row) as bf16 in 16-byte
// pieces, four lanes to a row: emit(src, k, piece) stores columns 8k .. 8k + 7
// of lane src's row; every lane calls it.
template <class Emit>
__device__ __forceinline__ void store_block_bf16(const uint32_t (&v)[32], int lane, Emit&& emit) {
  uint4 w[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    w[g].x = ptx::pack_bf16x2(__uint_as_float(v[8 * g]), __uint_as_float(v[8 * g + 1]));
    w[g].y = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 2]), __uint_as_float(v[8 * g + 3]));
    w[g].z = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 4]), __uint_as_float(v[8 * g + 5]));
    w[g].w = ptx::pack_bf16x2(__uint_as_float(v[8 * g + 6]), __uint_as_float(v[8 * g + 7]));
  }
  const int k = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int src = 8 * j + (lane >> 2);
    uint4 piece = w[0];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint4 x;
      x.x = __shfl_sync(0xffffffffu, w[kk].x, src);
      x.y = __shfl_sync(0xffffffffu, w[kk].y, src);
      x.z = __shfl_sync(0xffffffffu, w[kk].z, src);
      x.w = __shfl_sync(0xffffffffu, w[kk].w, src);
      if (kk == k) piece = x;
    }
    emit(src, k, piece);
  }
}

// A token's targets in ascending vocabulary order: `next` is the next one at
// or past the tile (INT_MAX: none), `cur` its place in the token's list.
struct Targets {
  const int32_t* list;
  int cur, n, next;
};

__device__ __forceinline__ Targets targets_from(const LossParams& p, bool row_ok, long long row,
                                                int col0) {
  Targets g{nullptr, 0, 0, INT_MAX};
  if (!row_ok) return g;
  if (p.labels != nullptr) {
    const int y = __ldg(p.labels + row);
    if (y >= col0) g.next = y;  // (an ignored or bad label is dealt with by the caller)
    g.n = 1;
    return g;
  }
  g.list = p.hit_idx + row * p.K;
  g.n = p.K;
  int lo = 0, hi = p.K;  // the first entry >= col0
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(g.list + mid) < col0)
      lo = mid + 1;
    else
      hi = mid;
  }
  g.cur = lo;
  if (lo < p.K) g.next = __ldg(g.list + lo);
  return g;
}

__device__ __forceinline__ void targets_advance(Targets& g) {
  ++g.cur;
  g.next = g.cur < g.n && g.list != nullptr ? __ldg(g.list + g.cur) : INT_MAX;
}

__device__ __forceinline__ bool label_live(const LossParams& p, int y) {
  return y != p.ignore_index && y >= 0 && y < p.R * p.Vs;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
loss_gemm_kernel(const __grid_constant__ LossParams p) {
  using C = Cfg<KIND, CG>;
  constexpr int kStages = C::kStages;
  constexpr int TM = C::kTileM;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + kStages * C::kBBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = kPair ? ptx::cluster_ctarank() : 0u;  // 0 issues the pair's MMAs
  const int pair = blockIdx.x / CG;
  const int npairs = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&tfull[b], 1);
      ptx::mbar_init(&tempty[b], 4 * CG);  // every epilogue warp of the pair
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

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      uint32_t issued = 0, last_parity = 0;
      bool ok = true;
      for (int t = pair; t < p.num_tiles && ok; t += npairs) {
        const Tile tl = tile_of<KIND>(p, t);
        const int m0 = tl.mt * TM + static_cast<int>(cta) * kBM;       // this CTA's A rows
        const int n0 = tl.nt * kBN + static_cast<int>(cta) * C::kBNcta;  // and B columns
        for (int it = tl.it_lo; it < tl.it_hi; ++it) {
          if (!W.wait(&empty[stage], phase ^ 1u)) {
            ok = false;
            break;
          }
          int r = tl.rank, kb = it;
          if constexpr (KIND == LK_DX) {
            r = it / p.kb_per_rank;
            kb = it - r * p.kb_per_rank;
          }
          const CUtensorMap* ma = &p.mapA[r];
          const CUtensorMap* mb = &p.mapB[r];
          uint8_t* a_dst = sA + stage * kABytes;
          uint8_t* b_dst = sB + stage * C::kBBytes;
          uint32_t bar = 0;
          if constexpr (kPair) {
            bar = ptx::mapa(ptx::smem_addr(&full[stage]), 0);
            if (cta == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          } else {
            ptx::mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
          }
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int x, int y) {
            if constexpr (kPair)
              ptx::tma_load_2d_pair(dst, map, bar, x, y);
            else
              ptx::tma_load_2d(dst, map, &full[stage], x, y);
          };
          if constexpr (a_mn(KIND)) {
            for (int i = 0; i < kBM / 64; ++i)
              load(a_dst + i * kBoxBytes, ma, m0 + 64 * i, kb * kBK);
          } else {
            load(a_dst, ma, kb * kBK, m0);
          }
          if constexpr (b_mn(KIND)) {
            // W rows of the piece (DX) or tokens (DW) down, D across
            const int y = (KIND == LK_DX ? p.v0 : 0) + kb * kBK;
            for (int i = 0; i < C::kBNcta / 64; ++i)
              load(b_dst + i * kBoxBytes, mb, n0 + 64 * i, y);
          } else {
            load(b_dst, mb, kb * kBK, p.v0 + n0);
          }
          issued |= 1u << stage;
          last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_flag && cta == 0) {
        // Loads in flight write into shared memory: let them land (in a pair
        // all are counted on the leader's barriers).
        for (int s = 0; s < kStages; ++s)
          if (issued & (1u << s)) W.drain(&full[s], (last_parity >> s) & 1u, kDrainNs);
      }
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issue
    if (lane == 0 && cta == 0) {
      uint32_t stage = 0, phase = 0;
      uint32_t acc = 0, acc_phase = 0;
      bool any = false, ok = true;
      for (int t = pair; t < p.num_tiles && ok; t += npairs) {
        const Tile tl = tile_of<KIND>(p, t);
        if (!W.wait(&tempty[acc], acc_phase ^ 1u)) break;
        ptx::tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kBN;
        for (int it = tl.it_lo; it < tl.it_hi; ++it) {
          if (!W.wait(&full[stage], phase)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a_addr = ptx::smem_addr(sA + stage * kABytes);
          const uint32_t b_addr = ptx::smem_addr(sB + stage * C::kBBytes);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            // K-major: 16 elements (32 B) on inside the swizzled row;
            // MN-major: 16 k rows (2 KiB) on, 64-wide boxes 8 KiB apart.
            const uint64_t ad = a_mn(KIND)
                                    ? ptx::smem_desc_sw128(a_addr + kk * 2048, kBoxBytes, 1024)
                                    : ptx::smem_desc_sw128(a_addr + kk * 32, 16, 1024);
            const uint64_t bd = b_mn(KIND)
                                    ? ptx::smem_desc_sw128(b_addr + kk * 2048, kBoxBytes, 1024)
                                    : ptx::smem_desc_sw128(b_addr + kk * 32, 16, 1024);
            const uint32_t accum = (it > tl.it_lo || kk > 0) ? 1u : 0u;
            if constexpr (kPair)
              ptx::mma_f16_pair(d_tmem, ad, bd, C::kIdesc, accum);
            else
              ptx::mma_f16(d_tmem, ad, bd, C::kIdesc, accum);
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
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const uint32_t tempty_leader0 = kPair ? ptx::mapa(ptx::smem_addr(&tempty[0]), 0) : 0u;
    uint32_t acc = 0, acc_phase = 0;
    // The whole warp polls and stops as one (the TMEM loads are collective).
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, W.wait(bar, parity) ? 1 : 0) != 0;
    };
    for (int t = pair; t < p.num_tiles; t += npairs) {
      const Tile tl = tile_of<KIND>(p, t);
      const long long row = static_cast<long long>(tl.mt) * TM + cta * kBM + q * 32 + lane;
      const int col0 = tl.nt * kBN;  // within the piece (FWD, DL) or D (DX, DW)
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * kBN;
      auto release_acc = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            ptx::mbar_arrive_cluster(tempty_leader0 + acc * 8);
          else
            ptx::mbar_arrive(&tempty[acc]);
        }
      };
      if constexpr (KIND == LK_FWD || KIND == LK_DL) {
        const bool row_ok = row < p.T;
        const int vcol0 = tl.rank * p.Vs + p.v0 + col0;  // the tile's first vocabulary index
        const int ncols = min(kBN, p.vn - col0);
        Targets tg = targets_from(p, row_ok, row, vcol0);
        // DL: the token's coefficients (all zero and not live: an ignored row)
        float ca = 0.f, cb = 0.f, cw = 0.f, off2 = 0.f;
        bool live = false;
        if constexpr (KIND == LK_DL) {
          if (row_ok) {
            const float g = __ldg(p.dloss + row);
            const float lse = __ldg(p.lse[tl.rank] + row);
            off2 = lse * kLog2e;
            if (p.labels != nullptr) {
              const int y = __ldg(p.labels + row);
              live = label_live(p, y);
              if (tl.rank == 0 && vcol0 == 0 && !live && y != p.ignore_index)
                atomicCAS(p.status, 0, FCC_ERR_INVALID);
              ca = g * (1.f + 2.f * p.z * lse);
              cb = g * (p.smoothing / static_cast<float>(p.R * p.Vs));
              cw = g * (1.f - p.smoothing);
            } else {
              live = __ldg(p.hit_idx + row * p.K) != INT_MAX;
              ca = g * p.tau;
              cw = g * p.tau;
            }
          }
        }
        if (!wait_warp(&tfull[acc], acc_phase)) break;
        ptx::tc_fence_after();
        float m2 = -INFINITY, sum = 0.f, lsum = 0.f;  // FWD: base-2 maximum, sum; plain sum
#pragma unroll 1
        for (int c = 0; c < kBN; c += 32) {
          uint32_t v[32];
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(taddr + c, v);
          ptx::tmem_ld_wait();
          if (c == kBN - 32) release_acc();
          const int nc = ncols - c;  // valid columns of the chunk
          if (nc <= 0) continue;
          if (p.cap > 0.f) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              v[k] = __float_as_uint(p.cap * tanhf(__uint_as_float(v[k]) * p.inv_cap));
          }
          if constexpr (KIND == LK_FWD) {
            while (tg.next < vcol0 + c + 32) {
              const int at = tg.next - (vcol0 + c);
              float x = 0.f;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k == at) x = __uint_as_float(v[k]);
              if (at < nc) p.pick[row * p.K + tg.cur] = x;
              if (at >= nc) break;  // (the next rank's columns)
              targets_advance(tg);
            }
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
            float s4[4] = {m2 == -INFINITY ? sum : sum * ptx::ex2_approx(m2 - off), 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 32; ++k)
              s4[k & 3] += ptx::ex2_approx(fmaf(__uint_as_float(v[k]), p.c2, -off));
            sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
            m2 = mn;
            if (p.part_sum != nullptr) {
              float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k < nc) l4[k & 3] += __uint_as_float(v[k]);
              lsum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
            }
          } else {
            float d[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float pv = ptx::ex2_approx(fmaf(__uint_as_float(v[k]), p.c2, -off2));
              d[k] = fmaf(ca, pv, -cb);
            }
            while (tg.next < vcol0 + c + 32) {
              const int at = tg.next - (vcol0 + c);
              const float w = p.labels != nullptr ? cw : cw * __ldg(p.hit_q + row * p.K + tg.cur);
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k == at) d[k] -= w;
              if (at >= nc) break;
              targets_advance(tg);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              float x = d[k];
              if (p.cap > 0.f) {
                const float u = __uint_as_float(v[k]) * p.inv_cap;
                x *= 1.f - u * u;
              }
              v[k] = live ? __float_as_uint(x) : 0u;
            }
            __syncwarp();
            const int ok = row_ok ? 1 : 0;
            uint16_t* dst0 = p.dl + static_cast<long long>(tl.rank) * p.T * p.ldl + col0 + c;
            store_block_bf16(v, lane, [&](int src, int k, const uint4& x) {
              const long long srow = row - lane + src;
              if (__shfl_sync(0xffffffffu, ok, src) && col0 + c + 8 * k + 8 <= p.ldl)
                ptx::st_global_v4(dst0 + srow * p.ldl + 8 * k, x.x, x.y, x.z, x.w);
            });
          }
        }
        if constexpr (KIND == LK_FWD) {
          if (row_ok) {
            const long long o = static_cast<long long>(tl.rank * p.tiles_n + tl.nt) * p.T + row;
            p.part[o] = make_float2(m2, sum);
            if (p.part_sum != nullptr) p.part_sum[o] = lsum;
          }
        }
      } else if constexpr (KIND == LK_DX) {
        const bool row_ok = row < p.T;
        if (!wait_warp(&tfull[acc], acc_phase)) break;
        ptx::tc_fence_after();
        float* dst = p.acc + (static_cast<long long>(tl.split) * p.T + row) * p.D + col0;
#pragma unroll 1
        for (int c = 0; c < kBN; c += 32) {
          uint32_t v[32];
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(taddr + c, v);
          ptx::tmem_ld_wait();
          if (c == kBN - 32) release_acc();
          if (!row_ok) continue;
          if (tl.it_lo >= tl.it_hi) {  // (a short last piece leaves this part no K steps)
            if (!p.first) continue;
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = 0u;
          }
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (col0 + c + 4 * g + 4 > p.D) continue;
            float4 x = make_float4(__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]),
                                   __uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3]));
            float4* o = reinterpret_cast<float4*>(dst + c + 4 * g);
            if (!p.first) {
              const float4 y = *o;
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            *o = x;
          }
        }
      } else {
        const bool row_ok = row < p.vn;
        if (!wait_warp(&tfull[acc], acc_phase)) break;
        ptx::tc_fence_after();
        uint16_t* dst = static_cast<uint16_t*>(p.out[tl.rank]) +
                        (static_cast<long long>(p.v0)) * p.D + col0;
        const int ok = row_ok ? 1 : 0;
#pragma unroll 1
        for (int c = 0; c < kBN; c += 32) {
          uint32_t v[32];
          __syncwarp();
          ptx::tmem_ld_32x32b_x32(taddr + c, v);
          ptx::tmem_ld_wait();
          if (c == kBN - 32) release_acc();
          store_block_bf16(v, lane, [&](int src, int k, const uint4& x) {
            const long long srow = row - lane + src;
            if (__shfl_sync(0xffffffffu, ok, src) && col0 + c + 8 * k + 8 <= p.D)
              ptx::st_global_v4(dst + srow * p.D + c + 8 * k, x.x, x.y, x.z, x.w);
          });
        }
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
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
// One CTA of `n2` threads (a power of two >= K, at least 32) per token: the
// valid entries' probabilities q = softmax(teacher / tau) and their order by
// vocabulary index (a bitonic sort in shared memory; equal indices stay
// separate entries), written as hit_idx (INT_MAX past the last) and hit_q.
struct TeacherArgs {
  const int32_t* idx;   // [T, K], negative = no entry
  const float* logits;  // [T, K]
  int32_t* hit_idx;
  float* hit_q;
  int T, K, V;
  float inv_tau;
  int* status;
};

__global__ void __launch_bounds__(256) teacher_kernel(const TeacherArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  __shared__ int key[FCC_MAX_TEACHER];
  __shared__ float val[FCC_MAX_TEACHER];
  __shared__ float red[8];
  const int n2 = blockDim.x, k = threadIdx.x, lane = k & 31, warp = k >> 5;
  const long long row = blockIdx.x;
  int id = INT_MAX;
  float x = -INFINITY;
  if (k < a.K) {
    const int i = __ldg(a.idx + row * a.K + k);
    if (i >= 0 && i < a.V) {
      x = __ldg(a.logits + row * a.K + k);
      if (x != -INFINITY) id = i;  // (a logit of -inf is no entry)
    } else if (i >= a.V) {
      atomicCAS(a.status, 0, FCC_ERR_INVALID);
    }
  }
  // softmax over the valid entries (fmaxf drops a NaN; the sum keeps it)
  float m = x;
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
  for (int w = 1; w < n2 / 32; ++w) m = fmaxf(m, red[w]);
  __syncthreads();
  // (the difference is taken before the scaling, which could overflow)
  const float e = id != INT_MAX ? expf((x - m) * a.inv_tau) : 0.f;
  float s = e;
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  s = red[0];
  for (int w = 1; w < n2 / 32; ++w) s += red[w];
  key[k] = id;
  val[k] = id != INT_MAX ? e / s : 0.f;
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const int j = k ^ stride;
      if (j > k) {
        const bool up = (k & size) == 0;
        if ((key[k] > key[j]) == up) {
          const int ti = key[k];
          key[k] = key[j];
          key[j] = ti;
          const float tv = val[k];
          val[k] = val[j];
          val[j] = tv;
        }
      }
      __syncthreads();
    }
  }
  if (k < a.K) {
    a.hit_idx[row * a.K + k] = key[k];
    a.hit_q[row * a.K + k] = val[k];
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
  const int32_t* labels;
  const int32_t* hit_idx;
  const float* hit_q;
  float* loss[FCC_MAX_RANKS];
  float* lse[FCC_MAX_RANKS];
  int R, T, V, K, nparts, tok, ignore_index;
  float tau, smoothing, z;
  int* status;
};

__device__ __forceinline__ void merge(float& m, float& s, float m1, float s1) {
  const float mn = fmaxf(m, m1);
  const float off = mn == -INFINITY ? 0.f : mn;
  // (a sum whose maximum is -inf is 0, or NaN after a NaN logit: kept as it is)
  s = (m == -INFINITY ? s : s * exp2f(m - off)) + (m1 == -INFINITY ? s1 : s1 * exp2f(m1 - off));
  m = mn;
}

__global__ void __launch_bounds__(256) loss_combine_kernel(const CombineArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  __shared__ float sm[256], ss[256], sl[256], sh[256];
  const int token = threadIdx.x & (a.tok - 1), part = threadIdx.x / a.tok;
  const int parts = 256 / a.tok;
  const long long t = static_cast<long long>(blockIdx.x) * a.tok + token;
  float m = -INFINITY, s = 0.f, l = 0.f, h = 0.f;
  if (t < a.T) {
    for (int i = part; i < a.nparts; i += parts) {
      const float2 x = __ldg(a.part + static_cast<long long>(i) * a.T + t);
      merge(m, s, x.x, x.y);
      if (a.part_sum != nullptr) l += __ldg(a.part_sum + static_cast<long long>(i) * a.T + t);
    }
    if (a.labels == nullptr) {
      // sum_k q_k (log q_k - l_k / tau); an entry of probability 0 adds nothing
      for (int k = part; k < a.K; k += parts) {
        if (__ldg(a.hit_idx + t * a.K + k) == INT_MAX) continue;
        const float q = __ldg(a.hit_q + t * a.K + k);
        if (q != 0.f) h += q * (logf(q) - __ldg(a.pick + t * a.K + k) / a.tau);
      }
    }
  }
  sm[threadIdx.x] = m;
  ss[threadIdx.x] = s;
  sl[threadIdx.x] = l;
  sh[threadIdx.x] = h;
  __syncthreads();
  for (int n = parts / 2; n > 0; n >>= 1) {
    if (part < n) {
      const int o = threadIdx.x + n * a.tok;
      merge(sm[threadIdx.x], ss[threadIdx.x], sm[o], ss[o]);
      sl[threadIdx.x] += sl[o];
      sh[threadIdx.x] += sh[o];
    }
    __syncthreads();
  }
  if (part != 0 || t >= a.T) return;
  const float lse = (sm[threadIdx.x] + log2f(ss[threadIdx.x])) * kLn2;
  float loss = 0.f;
  if (a.labels != nullptr) {
    const int y = __ldg(a.labels + t);
    if (y != a.ignore_index) {
      if (y < 0 || y >= a.V) {
        atomicCAS(a.status, 0, FCC_ERR_INVALID);
      } else {
        loss = lse - (1.f - a.smoothing) * __ldg(a.pick + t) + a.z * lse * lse;
        if (a.part_sum != nullptr) loss -= a.smoothing / static_cast<float>(a.V) * sl[threadIdx.x];
      }
    }
  } else if (__ldg(a.hit_idx + t * a.K) != INT_MAX) {
    loss = a.tau * a.tau * (sh[threadIdx.x] + lse);
  }
  for (int r = 0; r < a.R; ++r) {
    a.loss[r][t] = loss;
    a.lse[r][t] = lse;
  }
}

// ------------------------------------------------------------------ dX finish
// dX[r] = bf16(sum of the f32 slabs, in order) for every rank.
struct FinishArgs {
  const float* acc;
  void* out[FCC_MAX_RANKS];
  long long n;  // T * D, a multiple of 8
  int splits, R;
};

__global__ void __launch_bounds__(256) dx_finish_kernel(const FinishArgs a) {
  ptx::griddep_wait();  // launched with programmatic stream serialization
  ptx::griddep_launch_dependents();
  const long long nv = a.n / 8;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < nv;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) {
      const float4* p = reinterpret_cast<const float4*>(a.acc + s * a.n) + 2 * i;
      const float4 u = __ldcs(p), w = __ldcs(p + 1);
      x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
      x[4] += w.x; x[5] += w.y; x[6] += w.z; x[7] += w.w;
    }
    uint4 o;
    o.x = ptx::pack_bf16x2(x[0], x[1]);
    o.y = ptx::pack_bf16x2(x[2], x[3]);
    o.z = ptx::pack_bf16x2(x[4], x[5]);
    o.w = ptx::pack_bf16x2(x[6], x[7]);
    for (int r = 0; r < a.R; ++r) reinterpret_cast<uint4*>(a.out[r])[i] = o;
  }
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
  return launch_pdl(kern, dim3(grid, 1, 1), dim3(kGemmThreads, 1, 1), kSmem, st,
                    CG == 2 ? 2u : 1u, p);
}

// One of the four products: tile counts for the shape, then the launch over
// at most `sms` CTAs.
template <int KIND>
cudaError_t launch_loss_gemm(LossParams& p, int cg, int sms, cudaStream_t st) {
  const int64_t tm = static_cast<int64_t>(kBM) * cg;
  int64_t tiles = 0;
  if (KIND == LK_FWD || KIND == LK_DL) {
    p.tiles_m = static_cast<int>(cdiv(p.T, tm));
    p.tiles_n = static_cast<int>(cdiv(p.vn, kBN));
    p.k_iters = static_cast<int>(cdiv(p.D, kBK));
    tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.R;
  } else if (KIND == LK_DX) {
    p.tiles_m = static_cast<int>(cdiv(p.T, tm));
    p.tiles_n = static_cast<int>(cdiv(p.D, kBN));
    p.kb_per_rank = static_cast<int>(cdiv(p.vn, kBK));
    p.k_iters = p.R * p.kb_per_rank;
    tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.splits;
  } else {
    p.tiles_m = static_cast<int>(cdiv(p.vn, tm));
    p.tiles_n = static_cast<int>(cdiv(p.D, kBN));
    p.k_iters = static_cast<int>(cdiv(p.T, kBK));
    tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n * p.R;
  }
  if (tiles > (1ll << 30)) return cudaErrorInvalidValue;
  p.num_tiles = static_cast<int>(tiles);
  p.group_m = 8;
  const int slots = std::max(1, std::min(sms / cg, gemm_max_clusters(cg)));
  const int grid = cg * std::min(slots, p.num_tiles);
  return cg == 2 ? launch_kind<KIND, 2>(p, grid, st) : launch_kind<KIND, 1>(p, grid, st);
}

// A CTA pair per tile when the rows exceed 128 and the single-CTA tiles
// outnumber the CTAs, or the caller's shape.
int choose_cg(const fcc_opts* o, int64_t rows, int64_t single_tiles, int sms) {
  if (sms < 2) return 1;
  if (o != nullptr && (o->cta_pair == 1 || o->cta_pair == 2)) return o->cta_pair;
  return rows > kBM && single_tiles > sms ? 2 : 1;
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
  if (!(c.softcap >= 0.f) || std::isinf(c.softcap)) return FCC_ERR_INVALID;
  if (c.K == 0) {
    if (!al(c.labels, 4)) return FCC_ERR_INVALID;
    if (!(c.smoothing >= 0.f && c.smoothing < 1.f)) return FCC_ERR_INVALID;
    if (!(c.z >= 0.f) || std::isinf(c.z)) return FCC_ERR_INVALID;
  } else {
    if (c.K < 1 || c.K > FCC_MAX_TEACHER) return FCC_ERR_INVALID;
    if (!al(c.teacher_idx, 4) || !al(c.teacher, 4)) return FCC_ERR_INVALID;
    if (!(c.tau > 0.f) || std::isinf(c.tau)) return FCC_ERR_INVALID;
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

// Scratch layout.  Forward: partials, target logits; distillation also the
// sorted teacher entries.  Backward: the piece's dl, the dX slabs.
struct Plan {
  size_t hit_idx = 0, hit_q = 0, pick = 0, part = 0, part_sum = 0;
  size_t dl = 0, acc = 0, total = 0;
  int nparts = 0;
  int64_t piece = 0;  // vocabulary rows of a piece, per rank
  int splits = 1;     // K parts of dX
};

constexpr size_t kPieceBytes = size_t(512) << 20;  // dl held at a time

Plan plan_of(int R, int64_t T, int64_t V, int64_t D, int K, bool grad, bool smoothing, bool want_dx,
             int sms, const fcc_opts* o) {
  Plan p;
  size_t off = 0;
  const int64_t Vs = V / R;
  if (K > 0) {
    p.hit_idx = off;
    off += up256(static_cast<size_t>(T) * K * 4);
    p.hit_q = off;
    off += up256(static_cast<size_t>(T) * K * 4);
  }
  if (!grad) {
    p.nparts = static_cast<int>(R * cdiv(Vs, kBN));
    p.pick = off;
    off += up256(static_cast<size_t>(T) * std::max(K, 1) * 4);
    p.part = off;
    off += up256(static_cast<size_t>(p.nparts) * T * 8);
    p.part_sum = off;
    if (smoothing) off += up256(static_cast<size_t>(p.nparts) * T * 4);
  } else {
    // Equal pieces, whole tiles of 256 rows, as few as hold kPieceBytes of dl
    // (or the caller's count).
    const int64_t most = std::max<int64_t>(
        kBN, static_cast<int64_t>(kPieceBytes / (static_cast<size_t>(T) * R * 2)) / kBN * kBN);
    int64_t n = o != nullptr && o->chunks > 0 ? o->chunks : cdiv(Vs, most);
    n = std::max<int64_t>(1, std::min(n, cdiv(Vs, kBN)));
    p.piece = cdiv(cdiv(Vs, n), kBN) * kBN;
    p.dl = off;
    off += up256(static_cast<size_t>(R) * T * p.piece * 2);
    if (want_dx) {
      // Few dX tiles: split the vocabulary's K loop so that all SMs have work.
      const int64_t tiles = cdiv(T, kBM) * cdiv(D, kBN);
      const int64_t k_iters = R * cdiv(std::min(p.piece, Vs), kBK);
      p.splits = static_cast<int>(
          std::max<int64_t>(1, std::min<int64_t>(sms / std::max<int64_t>(tiles, 1), k_iters / 4)));
      p.acc = off;
      off += up256(static_cast<size_t>(p.splits) * T * D * 4);
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
  p.splits = pl.splits;
  p.K = std::max(c.K, 1);
  if (c.K == 0) {
    p.labels = c.labels;
  } else {
    p.hit_idx = reinterpret_cast<int32_t*>(base + pl.hit_idx);
    p.hit_q = reinterpret_cast<float*>(base + pl.hit_q);
  }
  p.ignore_index = c.ignore_index;
  p.cap = c.softcap;
  p.inv_cap = c.softcap > 0.f ? 1.f / c.softcap : 0.f;
  p.tau = c.tau;
  p.c2 = static_cast<float>(1.4426950408889634 / c.tau);
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
  unsigned n2 = 32;
  while (n2 < static_cast<unsigned>(c.K)) n2 <<= 1;
  return launch_pdl(teacher_kernel, dim3(static_cast<unsigned>(c.T)), dim3(n2), 0, c.st, 1u, a);
}

// Tensor maps of the logit product: X rows and W rows, both K-major.
fcc_status logit_maps(LossParams& p, const Call& c, int cg) {
  for (int r = 0; r < c.R; ++r) {
    fcc_status s = internal_encode_map(&p.mapA[r], c.X[r], c.T, c.D, c.D, kBM);
    if (s == FCC_OK)
      s = internal_encode_map(&p.mapB[r], c.W[r], c.V / c.R, c.D, c.D,
                              static_cast<uint32_t>(kBN / cg));
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
  const Plan pl = plan_of(c.R, c.T, c.V, c.D, c.K, false, c.smoothing > 0.f, false, 1, c.opts);
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
  const int cg = choose_cg(c.opts, c.T, cdiv(c.T, kBM) * pl.nparts, sms);
  if ((s = logit_maps(p, c, cg)) != FCC_OK) return s;
  uint64_t launches = 2;
  if (c.K > 0) {
    if (launch_teacher(c, pl, base, status) != cudaSuccess) return FCC_ERR_CUDA;
    ++launches;
  }
  if (launch_loss_gemm<LK_FWD>(p, cg, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
  CombineArgs a;
  std::memset(&a, 0, sizeof(a));
  a.part = p.part;
  a.part_sum = p.part_sum;
  a.pick = p.pick;
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
  a.smoothing = c.smoothing;
  a.z = c.z;
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
  base_p.dl = reinterpret_cast<uint16_t*>(base + pl.dl);
  base_p.ldl = pl.piece;
  base_p.acc = want_dx ? reinterpret_cast<float*>(base + pl.acc) : nullptr;
  base_p.dloss = dloss;
  for (int r = 0; r < c.R; ++r) {
    base_p.lse[r] = lse[r];
    base_p.out[r] = want_dw ? dW[r] : nullptr;
  }
  const int64_t Vs = c.V / c.R;
  const int cg_dl = choose_cg(c.opts, c.T, cdiv(c.T, kBM) * c.R * cdiv(std::min(pl.piece, Vs), kBN), sms);
  const int cg_dx = choose_cg(c.opts, c.T, cdiv(c.T, kBM) * cdiv(c.D, kBN) * pl.splits, sms);
  const int cg_dw = choose_cg(c.opts, std::min(pl.piece, Vs),
                              cdiv(std::min(pl.piece, Vs), kBM) * cdiv(c.D, kBN) * c.R, sms);
  uint64_t launches = 0;
  if (c.K > 0) {
    if (launch_teacher(c, pl, base, status) != cudaSuccess) return FCC_ERR_CUDA;
    ++launches;
  }
  LossParams p_dl = base_p;
  if ((s = logit_maps(p_dl, c, cg_dl)) != FCC_OK) return s;
  LossParams p_dx = base_p, p_dw = base_p;
  for (int r = 0; r < c.R; ++r) {
    // W and X again, MN-major boxes of 64 rows
    if ((s = internal_encode_map(&p_dx.mapB[r], c.W[r], Vs, c.D, c.D, kBK)) != FCC_OK) return s;
    if ((s = internal_encode_map(&p_dw.mapB[r], c.X[r], c.T, c.D, c.D, kBK)) != FCC_OK) return s;
  }
  for (int64_t v0 = 0; v0 < Vs; v0 += pl.piece) {
    const int vn = static_cast<int>(std::min(pl.piece, Vs - v0));
    for (LossParams* p : {&p_dl, &p_dx, &p_dw}) {
      p->v0 = static_cast<int>(v0);
      p->vn = vn;
    }
    // dl holds vn valid columns: the maps end there (reads past them give zeros)
    if (v0 == 0 || v0 + vn == Vs) {
      for (int r = 0; r < c.R; ++r) {
        const uint16_t* d = base_p.dl + static_cast<size_t>(r) * c.T * pl.piece;
        if ((s = internal_encode_map(&p_dx.mapA[r], d, c.T, vn, pl.piece, kBM)) != FCC_OK) return s;
        if ((s = internal_encode_map(&p_dw.mapA[r], d, c.T, vn, pl.piece, kBK)) != FCC_OK) return s;
      }
    }
    if (launch_loss_gemm<LK_DL>(p_dl, cg_dl, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
    ++launches;
    if (want_dx) {
      p_dx.first = v0 == 0 ? 1 : 0;
      if (launch_loss_gemm<LK_DX>(p_dx, cg_dx, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
      ++launches;
    }
    if (want_dw) {
      if (launch_loss_gemm<LK_DW>(p_dw, cg_dw, sms, c.st) != cudaSuccess) return FCC_ERR_CUDA;
      ++launches;
    }
  }
  if (want_dx) {
    FinishArgs f;
    std::memset(&f, 0, sizeof(f));
    f.acc = base_p.acc;
    for (int r = 0; r < c.R; ++r) f.out[r] = dX[r];
    f.n = c.T * c.D;
    f.splits = pl.splits;
    f.R = c.R;
    const int64_t blocks = std::min<int64_t>(cdiv(f.n / 8, 256), static_cast<int64_t>(sms) * 8);
    if (launch_pdl(dx_finish_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.st, 1u,
                   f) != cudaSuccess)
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
