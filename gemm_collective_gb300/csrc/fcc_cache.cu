// fcc_cache.cu -- writing a step's keys and values into the paged cache, and
// reading positions back out of it.
//
// Both move every byte once and compute next to nothing: DRAM bounds them, or
// the launch where the rows are few.  A warp serves up to kHeads heads of one row of the
// token arrays: d = 128 puts a head's key on lanes 0-15 and its value on lanes
// 16-31 (16 bytes of bf16 each), d = 64 two heads at once.  The token array's side
// needs no look-up, so append loads it before it knows the sequence and the page.
#include "fcc_cache.cuh"

#include <cuda_bf16.h>

#include <cstring>

#include "fcc_ptx.cuh"

namespace fcc {
namespace {

constexpr int kHeads = 4;      // heads of a row that one warp serves
constexpr int kWarps = 8;

struct MoveArgs {
  PoolArgs pool;
  StepArgs step;
  char* K[FCC_MAX_RANKS];      // token arrays, rows ld elements apart
  char* V[FCC_MAX_RANKS];
  int64_t ld;
  int R;
  int chunks;                  // ceil(H / kHeads)
  int64_t tasks;               // T * R * chunks
  int* status;
};

// Each sequence's own description, checked once per call.
__device__ __forceinline__ void check_step(const MoveArgs& a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t b = i; b < a.step.B; b += static_cast<int64_t>(gridDim.x) * blockDim.x)
    if (!load_seq(a.step, static_cast<int>(b)).ok) record_invalid(a.status);
}

// Where row t's position lies: number of the row (page, head 0, row) of the
// pools, or -1.  All lanes of a warp call it with the same t.
__device__ __forceinline__ int64_t place_of(const MoveArgs& a, int t) {
  const int b = warp_find_seq(a.step, t);
  const Seq q = load_seq(a.step, b);
  if (!q.ok || t < q.s || t >= q.s + q.n) return -1;
  const int pos = q.L - q.n + (t - q.s);
  const int page = page_of(a.step, a.pool.pages, b, pos >> a.pool.log2P);
  if (page < 0) {
    record_invalid(a.status);
    return -1;
  }
  return ((static_cast<int64_t>(page) * a.pool.H) << a.pool.log2P) +
         (pos & ((1 << a.pool.log2P) - 1));
}

// The power of two of a row whose largest finite magnitude has these bf16 bits:
// the least k >= -64 with a <= 448 * 2^k = 1.75 * 2^(k + 8).
__device__ __forceinline__ int row_power(unsigned a) {
  const int k = static_cast<int>(a >> 7) - 127 - 8 + ((a & 0x7f) > 0x60 ? 1 : 0);
  return max(k, -64);
}

// Lanes of one row (D / 8 of them, 8 values each).
template <int D>
struct Lanes {
  static constexpr int kRow = D / 8;
  static constexpr int kHeadsAtOnce = 32 / (2 * kRow);   // a key and a value row each
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const __grid_constant__ MoveArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  check_step(a);
  using L = Lanes<D>;
  constexpr int kN = kHeads / L::kHeadsAtOnce;
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (task >= a.tasks) return;
  const int chunk = static_cast<int>(task % a.chunks);
  const int r = static_cast<int>(task / a.chunks % a.R);
  const int t = static_cast<int>(task / a.chunks / a.R);
  const int part = lane % L::kRow;                       // 8 values of the row
  const bool value = (lane / L::kRow) & 1;
  const int h0 = chunk * kHeads + lane / (2 * L::kRow);
  const char* src = (value ? a.V[r] : a.K[r]) + (static_cast<int64_t>(t) * a.ld) * 2;
  uint4 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * L::kHeadsAtOnce;
    if (h < a.pool.H) x[i] = *reinterpret_cast<const uint4*>(src + (h * D + part * 8) * 2);
  }
  const int64_t place = place_of(a, t);
  if (place < 0) return;
  char* dst = value ? a.pool.V[r] : a.pool.K[r];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * L::kHeadsAtOnce;
    const bool there = h < a.pool.H;
    const int64_t row = place + (static_cast<int64_t>(h) << a.pool.log2P);
    if constexpr (!E4M3) {
      if (there) *reinterpret_cast<uint4*>(dst + row * (D * 2) + part * 16) = x[i];
    } else {
      const unsigned w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      unsigned top = 0;                                  // largest finite magnitude, as bits
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int s = 0; s < 32; s += 16) {
          const unsigned m = (w[j] >> s) & 0x7fffu;
          top = max(top, there && m < 0x7f80u ? m : 0u);
        }
#pragma unroll
      for (int s = 1; s < L::kRow; s *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
      const int k = row_power(top);
      const float f = power_of_two(-k);
      unsigned q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const unsigned m = (w[2 * j + s / 2] >> (16 * (s & 1))) & 0xffffu;
          // (an infinity would saturate to 448: it becomes NaN as well)
          v[s] = (m & 0x7fffu) == 0x7f80u ? __int_as_float(0x7fffffff) : __uint_as_float(m << 16) * f;
        }
        const unsigned lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
        const unsigned hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
        q[j] = lo | (hi << 16);
      }
      if (there) {
        *reinterpret_cast<uint2*>(dst + row * D + part * 8) = make_uint2(q[0], q[1]);
        if (part == 0) (value ? a.pool.Ve[r] : a.pool.Ke[r])[row] = static_cast<uint8_t>(k + 127);
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const __grid_constant__ MoveArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  check_step(a);
  using L = Lanes<D>;
  constexpr int kN = kHeads / L::kHeadsAtOnce;
  const int lane = threadIdx.x & 31;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (task >= a.tasks) return;
  const int chunk = static_cast<int>(task % a.chunks);
  const int r = static_cast<int>(task / a.chunks % a.R);
  const int t = static_cast<int>(task / a.chunks / a.R);
  const int part = lane % L::kRow;
  const bool value = (lane / L::kRow) & 1;
  const int h0 = chunk * kHeads + lane / (2 * L::kRow);
  const int64_t place = place_of(a, t);
  if (place < 0) return;
  const char* src = value ? a.pool.V[r] : a.pool.K[r];
  const uint8_t* exps = value ? a.pool.Ve[r] : a.pool.Ke[r];
  uint4 x[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * L::kHeadsAtOnce;
    const int64_t row = place + (static_cast<int64_t>(h) << a.pool.log2P);
    if (h >= a.pool.H) continue;
    if constexpr (E4M3) {
      const uint2 c = *reinterpret_cast<const uint2*>(src + row * D + part * 8);
      x[i] = make_uint4(c.x, c.y, exps[row], 0);
    } else {
      x[i] = *reinterpret_cast<const uint4*>(src + row * (D * 2) + part * 16);
    }
  }
  char* dst = (value ? a.V[r] : a.K[r]) + static_cast<int64_t>(t) * a.ld * 2;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int h = h0 + i * L::kHeadsAtOnce;
    if (h >= a.pool.H) continue;
    uint4 o = x[i];
    if constexpr (E4M3) {
      // (a byte of 0 or 255 is no power that append writes; 2^-127 needs two steps)
      const int k = static_cast<int>(x[i].z) - 127;
      const float f = power_of_two(max(k, -126)), g = k < -126 ? 0.5f : 1.f;
      unsigned w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned c = ((j < 2 ? x[i].x : x[i].y) >> (16 * (j & 1))) & 0xffffu;
        const __half2_raw h2 = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
        const float2 v = __half22float2(__half2(h2));
        w[j] = ptx::pack_bf16x2(v.x * f * g, v.y * f * g);
      }
      o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(dst + (h * D + part * 8) * 2) = o;
  }
}

bool aligned(const void* p, unsigned n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

fcc_status move_call(bool append, int R, const void* const* K, const void* const* V, int64_t ld,
                     const fcc_cache* cache, const fcc_batch* batch, fcc_dtype type,
                     const fcc_opts* opts, fcc_stream_t stream) {
  MoveArgs a;
  std::memset(&a, 0, sizeof(a));
  fcc_status s = cache_args(R, cache, batch, &a.pool, &a.step);
  if (s == FCC_ERR_INVALID) return s;
  if (K == nullptr || V == nullptr) return FCC_ERR_INVALID;
  for (int r = 0; r < R; ++r)
    if (!aligned(K[r], 16) || !aligned(V[r], 16)) return FCC_ERR_INVALID;
  const int64_t width = static_cast<int64_t>(cache->H) * cache->d;
  if (ld == 0) ld = width;
  if (ld < width || ld % 8 != 0 || ld > (1ll << 31) - 1) return FCC_ERR_INVALID;
  if (type != FCC_BF16 && type != FCC_F16 && type != FCC_F32) return FCC_ERR_INVALID;
  if (s != FCC_OK) return s;
  if (type != FCC_BF16) return FCC_ERR_UNSUPPORTED;
  if (opts != nullptr && opts->algo != FCC_ALGO_AUTO && opts->algo != FCC_ALGO_FUSED)
    return FCC_ERR_UNSUPPORTED;
  a.chunks = (cache->H + kHeads - 1) / kHeads;
  a.tasks = batch->T * R * a.chunks;
  const int64_t blocks = (a.tasks + kWarps - 1) / kWarps;
  if (blocks > (1ll << 31) - 1) return FCC_ERR_INVALID;
  void* ws = nullptr;
  int sms = 0;
  unsigned long long timeout_ns = 0;
  if ((s = internal_prepare(opts, 0, &ws, &a.status, &sms, &timeout_ns)) != FCC_OK) return s;
  for (int r = 0; r < R; ++r) {
    a.K[r] = static_cast<char*>(const_cast<void*>(K[r]));
    a.V[r] = static_cast<char*>(const_cast<void*>(V[r]));
  }
  a.ld = ld;
  a.R = R;
  const bool e4m3 = cache->dtype == FCC_E4M3;
  void (*kern)(const MoveArgs) =
      append ? (cache->d == 128 ? (e4m3 ? append_kernel<128, true> : append_kernel<128, false>)
                                : (e4m3 ? append_kernel<64, true> : append_kernel<64, false>))
             : (cache->d == 128 ? (e4m3 ? gather_kernel<128, true> : gather_kernel<128, false>)
                                : (e4m3 ? gather_kernel<64, true> : gather_kernel<64, false>));
  if (launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0,
                 reinterpret_cast<cudaStream_t>(stream), 1u, a) != cudaSuccess)
    return FCC_ERR_CUDA;
  bump_launch_count(1);
  return FCC_OK;
}

}  // namespace

fcc_status cache_args(int R, const fcc_cache* cache, const fcc_batch* batch, PoolArgs* pool,
                      StepArgs* step) {
  constexpr int64_t kMax = (1ll << 31) - 1;
  if (R < 1 || R > FCC_MAX_RANKS || cache == nullptr || batch == nullptr) return FCC_ERR_INVALID;
  if (batch->B < 1 || batch->B > 65536 || batch->T < 1 || batch->T > kMax ||
      batch->max_pages < 1 || batch->max_pages > kMax)
    return FCC_ERR_INVALID;
  for (const int32_t* p : {batch->start, batch->len, batch->table})
    if (!aligned(p, 4)) return FCC_ERR_INVALID;
  const int P = cache->page_size;
  if (cache->H < 1 || cache->H > 1024 || cache->d < 1 || cache->pages < 1 || cache->pages > kMax ||
      P < 1 || P > 65536 || (P & (P - 1)) != 0)
    return FCC_ERR_INVALID;
  if (cache->dtype != FCC_BF16 && cache->dtype != FCC_F16 && cache->dtype != FCC_F32 &&
      cache->dtype != FCC_E4M3)
    return FCC_ERR_INVALID;
  const bool e4m3 = cache->dtype == FCC_E4M3;
  if (cache->K == nullptr || cache->V == nullptr ||
      (e4m3 && (cache->K_exp == nullptr || cache->V_exp == nullptr)))
    return FCC_ERR_INVALID;
  for (int r = 0; r < R; ++r) {
    if (!aligned(cache->K[r], 16) || !aligned(cache->V[r], 16)) return FCC_ERR_INVALID;
    if (e4m3 && (!aligned(cache->K_exp[r], 16) || !aligned(cache->V_exp[r], 16)))
      return FCC_ERR_INVALID;
    pool->K[r] = static_cast<char*>(cache->K[r]);
    pool->V[r] = static_cast<char*>(cache->V[r]);
    pool->Ke[r] = e4m3 ? cache->K_exp[r] : nullptr;
    pool->Ve[r] = e4m3 ? cache->V_exp[r] : nullptr;
  }
  pool->pages = cache->pages;
  pool->log2P = 0;
  while ((1 << pool->log2P) < P) ++pool->log2P;
  pool->H = cache->H;
  pool->d = cache->d;
  step->start = batch->start;
  step->len = batch->len;
  step->table = batch->table;
  step->max_pages = batch->max_pages;
  step->B = batch->B;
  step->T = static_cast<int>(batch->T);
  if ((cache->d != 64 && cache->d != 128) || cache->dtype == FCC_F16 || cache->dtype == FCC_F32)
    return FCC_ERR_UNSUPPORTED;
  return FCC_OK;
}

}  // namespace fcc

using namespace fcc;

extern "C" {

fcc_status fcc_cache_append(int R, const void* const* K, const void* const* V, int64_t ld,
                            const fcc_cache* cache, const fcc_batch* batch, fcc_dtype in,
                            const fcc_opts* opts, fcc_stream_t stream) {
  return move_call(true, R, K, V, ld, cache, batch, in, opts, stream);
}

fcc_status fcc_cache_gather(int R, const fcc_cache* cache, const fcc_batch* batch, void* const* K,
                            void* const* V, int64_t ld, fcc_dtype out, const fcc_opts* opts,
                            fcc_stream_t stream) {
  return move_call(false, R, K, V, ld, cache, batch, out, opts, stream);
}

}  // extern "C"
