// fcc_paged.cuh -- arguments and launchers of the paged attention's kernels.
#pragma once

#include "fcc_cache.cuh"
#include "fcc_ptx.cuh"

namespace fcc {

// Rows that the tiles of 128 cannot give, one bit for each row of a rank's key/value
// head: because in a product with P = 0 a value that is not finite reaches rows that do
// not see it, and e4m3 rows that saw powers too far apart.  launch_again's kernel
// computes them from all their positions.
struct Again {
  uint32_t* rows;              // [R * H][words]: bit i of a (rank, head) is row i % G of token i / G
  int* any;                    // some bit is set
  int64_t words;

  __host__ __device__ static int64_t words_of(int64_t rows) { return (rows + 31) / 32 + 1; }   // (one for a mask's upper part)
  __device__ __forceinline__ uint32_t* word(int rh, int row) const { return rows + rh * words + (row >> 5); }
  // Rows row .. row + 31 whose bits in m are set (m has none behind the last row).
  __device__ __forceinline__ void mark(int rh, int row, uint32_t m) const {
    uint32_t* w = word(rh, row);
    const int shift = row & 31;
    atomicOr(w, m << shift);
    if (shift != 0 && m >> (32 - shift) != 0) atomicOr(w + 1, m >> (32 - shift));
  }
  // The bits of rows row .. row + 31.
  __device__ __forceinline__ uint32_t bits(int rh, int row) const {
    const uint32_t* w = word(rh, row);
    return __funnelshift_r(w[0], w[1], row & 31);
  }
};

struct PagedArgs {
  PoolArgs pool;
  StepArgs step;
  const char* Q[FCC_MAX_RANKS];
  char* O[FCC_MAX_RANKS];
  float* lse[FCC_MAX_RANKS];   // all NULL: not wanted
  int64_t ldq, ldo;
  int R, Hq, G;
  int window;                  // INT_MAX: none
  int held;                    // positions that max_pages pages hold: no work for others
  float scale_log2;            // scale * log2(e)
  int* status;
  char* ws;
  uint32_t g_mul, g_shift;     // rows / G for rows < 2^31: see by_g()
  int boxes;                   // pages come by TMA
  Again again;                 // tiles only

  // x / G by multiplication: g_mul = ceil(2^(31 + g_shift) / G) with 2^(g_shift - 1) < G
  // <= 2^g_shift is exact for x < 2^31.
  __device__ __forceinline__ int by_g(int x) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(x)) * g_mul) >> (31 + g_shift));
  }
};

// A sequence that needs a page past its table's end, or that is not valid.
__device__ __forceinline__ bool bad_sequence(const PagedArgs& a, const Seq& q) {
  return !q.ok || (q.n > 0 && q.L > a.held);
}

constexpr float kLn2 = 0.6931471805599453f;

// 2^(x - ref), 0 for x = -inf.
__device__ __forceinline__ float ex2_from(float x, float ref) {
  return x == -INFINITY ? 0.f : ptx::ex2_approx(x - ref);
}

// Four e4m3 codes as two pairs of f16: exact.
__device__ __forceinline__ void f16x4_of_e4m3(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) return pack_f16x2(lo, hi);
  return ptx::pack_bf16x2(lo, hi);
}

// Tiles of 128 rows on the tensor cores' own memory (fcc_paged_tiles.cu).
// rows: tokens times G; rank_heads: R * H.  launch_tiles fills a.again.
size_t tiles_ws_bytes(int64_t d, int B, int ctas, int64_t rows, int64_t rank_heads);
cudaError_t launch_tiles(PagedArgs& a, bool e4m3, int ctas, unsigned long long timeout_ns,
                         cudaStream_t st);

}  // namespace fcc
