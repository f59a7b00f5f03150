// fcc_paged.cuh -- arguments and launchers of the paged attention's kernels.
#pragma once

#include "fcc_cache.cuh"
#include "fcc_ptx.cuh"

namespace fcc {

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
size_t tiles_ws_bytes(int64_t d, int B, int ctas);
cudaError_t launch_tiles(const PagedArgs& a, bool e4m3, int ctas, unsigned long long timeout_ns,
                         cudaStream_t st);

}  // namespace fcc
