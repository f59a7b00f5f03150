// fcc_paged.cu -- attention of a step's rows over the paged key/value cache.
//
// The simplest form: a warp for each row and query head walks the positions
// one after another with a running maximum and sum.
#include "fcc_cache.cuh"

#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "fcc_ptx.cuh"

namespace fcc {
namespace {

struct PagedArgs {
  PoolArgs pool;
  StepArgs step;
  const char* Q[FCC_MAX_RANKS];
  char* O[FCC_MAX_RANKS];
  float* lse[FCC_MAX_RANKS];   // all NULL: not wanted
  int64_t ldq, ldo;
  int R, Hq, G;
  int64_t window;              // 0: none
  float scale;
  int* status;
};

// 2^(byte - 127) of an e4m3 row.
__device__ __forceinline__ float exp_byte(uint8_t e) { return __int_as_float(static_cast<int>(e) << 23); }

template <int N, bool E4M3>
__device__ __forceinline__ void load_row(const char* pool, const uint8_t* exps, int64_t row, int lane,
                                         float (&x)[N]) {
  if constexpr (E4M3) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(pool) + row * (N * 32) + lane * N;
    const float f = exp_byte(exps[row]);
#pragma unroll
    for (int i = 0; i < N; ++i)
      x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3))) * f;
  } else {
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(pool) + row * (N * 32) + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(p[i]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) row_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t b = i0; b < a.step.B; b += static_cast<int64_t>(gridDim.x) * blockDim.x)
    if (!load_seq(a.step, static_cast<int>(b)).ok) record_invalid(a.status);
  const int64_t task = i0 >> 5;
  if (task >= static_cast<int64_t>(a.step.T) * a.R * a.Hq) return;
  const int h = static_cast<int>(task % a.Hq);
  const int r = static_cast<int>(task / a.Hq % a.R);
  const int t = static_cast<int>(task / a.Hq / a.R);
  const int b = warp_find_seq(a.step, t);
  const Seq q = load_seq(a.step, b);
  if (!q.rows_ok || t < q.s || t >= q.s + q.n) return;
  const int p = q.ok ? q.L - q.n + (t - q.s) : -1;
  float x[N], o[N] = {}, m = -INFINITY, l = 0.f;
  const __nv_bfloat16* src = reinterpret_cast<const __nv_bfloat16*>(a.Q[r]) + t * a.ldq + h * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __bfloat162float(src[i]);
  const int64_t lo = a.window > 0 ? max(static_cast<int64_t>(0), p - a.window + 1) : 0;
  const int mask = (1 << a.pool.log2P) - 1;
  for (int j = static_cast<int>(lo); j <= p; ++j) {
    const int page = page_of(a.step, a.pool.pages, b, j >> a.pool.log2P);
    if (page < 0) {
      record_invalid(a.status);
      continue;
    }
    const int64_t row = ((static_cast<int64_t>(page) * a.pool.H + h / a.G) << a.pool.log2P) + (j & mask);
    float k[N], v[N];
    load_row<N, E4M3>(a.pool.K[r], a.pool.Ke[r], row, lane, k);
    load_row<N, E4M3>(a.pool.V[r], a.pool.Ve[r], row, lane, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(x[i], k[i], s);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= a.scale;
    const float top = fmaxf(m, s);
    const float f = top == -INFINITY ? 1.f : __expf(m - top);
    const float e = s == -INFINITY ? 0.f : __expf(s - top);   // (NaN stays NaN)
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * f + (e == 0.f ? 0.f : e * v[i]);
    m = top;
  }
  __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.O[r]) + t * a.ldo + h * D + lane * N;
  const bool none = l == 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) dst[i] = __float2bfloat16(none ? 0.f : o[i] / l);
  if (a.lse[r] != nullptr && lane == 0)
    a.lse[r][static_cast<int64_t>(t) * a.Hq + h] = none ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace fcc

using namespace fcc;

extern "C" {

size_t fcc_paged_attention_workspace_size(int R, int64_t T, int B, int Hq, int H, int64_t d,
                                          const fcc_opts* opts) {
  (void)opts;
  if (R < 1 || R > FCC_MAX_RANKS || T < 1 || B < 1 || H < 1 || Hq < H || Hq % H != 0 || d < 1)
    return 0;
  return 0;
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
    if (ld < width || ld % 8 != 0 || ld > (1ll << 31) - 1) return FCC_ERR_INVALID;
  if (!(scale >= 0.f) || std::isinf(scale) || window < 0) return FCC_ERR_INVALID;
  for (fcc_dtype t : {in, out})
    if (t != FCC_BF16 && t != FCC_F16 && t != FCC_F32) return FCC_ERR_INVALID;
  if (described != FCC_OK) return described;
  if (in != FCC_BF16 || out != FCC_BF16) return FCC_ERR_UNSUPPORTED;
  if (opts != nullptr && opts->algo != FCC_ALGO_AUTO && opts->algo != FCC_ALGO_FUSED)
    return FCC_ERR_UNSUPPORTED;
  void* ws = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  const fcc_status s = internal_prepare(opts, 0, &ws, &a.status, &sms, &timeout_ns);
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
  a.G = Hq / cache->H;
  a.window = window;
  a.scale = scale > 0.f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(cache->d)));
  const int64_t blocks = (batch->T * R * Hq + 3) / 4;
  if (blocks > (1ll << 31) - 1) return FCC_ERR_INVALID;
  const bool e4m3 = cache->dtype == FCC_E4M3;
  void (*kern)(const PagedArgs) = cache->d == 128 ? (e4m3 ? row_kernel<128, true> : row_kernel<128, false>)
                                                  : (e4m3 ? row_kernel<64, true> : row_kernel<64, false>);
  kern<<<static_cast<unsigned>(blocks), 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  if (cudaGetLastError() != cudaSuccess) return FCC_ERR_CUDA;
  bump_launch_count(1);
  return FCC_OK;
}

}  // extern "C"
