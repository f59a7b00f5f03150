// fcc_cache.cu -- writing a step's keys and values into the paged cache, and
// reading positions back out of it.
//
// Both move every byte once and compute next to nothing: DRAM bounds them, or
// the launch and a chain of look-ups where the rows are few.  A warp serves 16
// neighbouring rows of the token arrays for one head: a row's key lies on kRow lanes
// and its value on as many (16 bytes of bf16 each).  Many warps with four steps in
// flight hide the look-ups best: 16 x 8192 e4m3 rows are read back in 122 us (6.6 TB/s)
// with 48 warps to an SM, in 146 with eight steps and 24, 197 with sixteen.
// The 16 rows' places are looked up by a lane each, their powers' bytes are
// stored or loaded together (one byte a warp, row by row, cost as much time as the
// values: 58.6 us for 4 x 4096 rows of 8 heads on two ranks).  The token array's side
// needs no look-up, so append loads its first rows before it knows where they go.
#include "fcc_cache.cuh"

#include <cuda_bf16.h>

#include <cstring>

#include "fcc_ptx.cuh"

namespace fcc {
namespace {

constexpr int kGroup = 16;     // rows of a warp
constexpr int kWarps = 8;
constexpr int kAhead = 4;      // steps of a warp's rows in flight

struct MoveArgs {
  PoolArgs pool;
  StepArgs step;
  char* K[FCC_MAX_RANKS];      // token arrays, rows ld elements apart
  char* V[FCC_MAX_RANKS];
  int64_t ld;
  int R;
  int64_t tasks;               // ceil(T / kGroup) * R * H
  int* status;
};

// Where the position of row t0 + lane % 16 lies: number of the row (page, head 0, row)
// of the pools, or -1.
__device__ __forceinline__ int64_t places_of(const MoveArgs& a, int t0) {
  const int lane = threadIdx.x & 31, t = t0 + (lane & (kGroup - 1));
  // the 16 rows' sequences: the one of t0, plus the starts up to t behind it
  int b = warp_find_seq(a.step, t0);
  for (int from = b + 1; from < a.step.B; from += 32) {
    const bool there = from + lane < a.step.B;
    const int s = there ? __ldg(a.step.start + from + lane) : 0;
    unsigned more = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, there && s <= t0 + i);   // (t0 + i may be the largest int)
      if ((lane & (kGroup - 1)) == i) b += __popc(m);
      more = m;
    }
    if (more != 0xffffffffu) break;            // (sequences without rows may fill a whole step)
  }
  const Seq q = load_seq(a.step, b);
  if (!q.ok || t < q.s || t >= q.s + q.n) return -1;
  const int pos = q.L - q.n + (t - q.s);
  const int page = page_of(a.step, a.pool.pages, b, pos >> a.pool.log2P);
  if (page < 0) {
    record_invalid(a.status);
    return -1;
  }
  return ((static_cast<int64_t>(page) * a.pool.H) << a.pool.log2P) + (pos & ((1 << a.pool.log2P) - 1));
}

// The power of two of a row whose largest finite magnitude has these bf16 bits:
// the least k >= -64 with a <= 448 * 2^k = 1.75 * 2^(k + 8).
__device__ __forceinline__ int row_power(unsigned a) {
  const int k = static_cast<int>(a >> 7) - 127 - 8 + ((a & 0x7f) > 0x60 ? 1 : 0);
  return max(k, -64);
}

// Two f32 to two codes (the low one in the low byte).
__device__ __forceinline__ uint32_t codes_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger magnitude of bf16 pairs, and over a row's lanes; `odd`: of those that are finite.
template <int kRow>
__device__ __forceinline__ unsigned row_top(const uint4& x, bool odd) {
  unsigned m[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
  if (odd)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = ((m[j] & 0xffffu) < 0x7f80u ? m[j] & 0xffffu : 0u) | (m[j] < 0x7f800000u ? m[j] & 0xffff0000u : 0u);
  const unsigned two = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
  unsigned top = max(two & 0xffffu, two >> 16);
#pragma unroll
  for (int s = 1; s < kRow; s *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
  return top;
}

// One lane's 8 values of a row as codes; k: the row's power.  All lanes of a warp call it.
template <int kRow>
__device__ __forceinline__ uint2 quantise(const uint4& x, int& k) {
  unsigned top = row_top<kRow>(x, false);
  const bool odd = __any_sync(0xffffffffu, top >= 0x7f80u);   // some value of the warp's rows is not finite
  if (odd) top = row_top<kRow>(x, true);
  k = row_power(top);
  const float f = power_of_two(-k);
  const uint64_t f2 = ptx::f32x2_pack(f, f);
  const unsigned w[4] = {x.x, x.y, x.z, x.w};
  unsigned q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    ptx::f32x2_unpack(ptx::f32x2_mul(ptx::f32x2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)), f2), lo, hi);
    if (odd) {                                 // (an infinity would saturate to 448: it becomes NaN as well)
      if (!(fabsf(lo) < INFINITY)) lo = __int_as_float(0x7fffffff);
      if (!(fabsf(hi) < INFINITY)) hi = __int_as_float(0x7fffffff);
    }
    q[j] = codes_of(lo, hi);
  }
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// 8 codes of a row of power byte - 127 as bf16 pairs.
__device__ __forceinline__ uint4 values(const uint2& c, int byte) {
  // (2^-127, which append does not write, is a subnormal number)
  const float f = __int_as_float(byte != 0 ? byte << 23 : 1 << 22);
  const uint64_t f2 = ptx::f32x2_pack(f, f);
  unsigned w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned two = ((j < 2 ? c.x : c.y) >> (16 * (j & 1))) & 0xffffu;
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
    float lo, hi;
    ptx::f32x2_unpack(ptx::f32x2_mul(ptx::f32x2_pack(v.x, v.y), f2), lo, hi);
    w[j] = ptx::pack_bf16x2(lo, hi);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool E4M3, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32, 6) move_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int kRow = D / 8;                  // lanes of a row
  constexpr int kAtOnce = 32 / (2 * kRow);     // token rows of a step: a key and a value row each
  constexpr int kSteps = kGroup / kAtOnce;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t b = i0; b < a.step.B; b += static_cast<int64_t>(gridDim.x) * blockDim.x)
    if (!load_seq(a.step, static_cast<int>(b)).ok) record_invalid(a.status);   // each sequence's description, once
  const int64_t task = i0 >> 5;
  if (task >= a.tasks) return;
  const int h = static_cast<int>(task % a.pool.H);
  const int64_t rest = task / a.pool.H;
  const int r = static_cast<int>(rest % a.R), t0 = static_cast<int>(rest / a.R) * kGroup;
  const int part = lane % kRow, value = lane / kRow & 1, sub = lane / (2 * kRow);
  char* const rows = (value ? a.V[r] : a.K[r]) + static_cast<int64_t>(h) * D * 2 + part * 16;
  char* const pool = value ? a.pool.V[r] : a.pool.K[r];
  auto token_row = [&](int n) { return reinterpret_cast<uint4*>(rows + (static_cast<int64_t>(t0) + n) * a.ld * 2); };
  uint4 x[kAhead];
  if constexpr (APPEND) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = i * kAtOnce + sub;
      x[i] = t0 + n < a.step.T ? *token_row(n) : make_uint4(0, 0, 0, 0);
    }
  }
  int64_t place = places_of(a, t0);            // of row t0 + lane % 16
  if (place >= 0) place += static_cast<int64_t>(h) << a.pool.log2P;
  // e4m3: lanes 0-15 hold the rows' key bytes, 16-31 their value bytes
  int byte = 0;
  uint8_t* const exps = E4M3 ? (lane < kGroup ? a.pool.Ke[r] : a.pool.Ve[r]) : nullptr;
  if constexpr (E4M3 && !APPEND) {
    if (place >= 0) byte = exps[place];
  }
#pragma unroll
  for (int first = 0; first < kSteps; first += kAhead) {
    int64_t at[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = (first + i) * kAtOnce + sub;
      at[i] = __shfl_sync(0xffffffffu, place, n);
      if constexpr (APPEND) {
        if (first > 0) x[i] = t0 + n < a.step.T ? *token_row(n) : make_uint4(0, 0, 0, 0);
      } else if (at[i] >= 0) {
        if constexpr (E4M3) {
          const uint2 c = *reinterpret_cast<const uint2*>(pool + at[i] * D + part * 8);
          x[i] = make_uint4(c.x, c.y, 0, 0);
        } else {
          x[i] = *reinterpret_cast<const uint4*>(pool + at[i] * (D * 2) + part * 16);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int n = (first + i) * kAtOnce + sub;
      if constexpr (APPEND && E4M3) {
        int k;
        const uint2 c = quantise<kRow>(x[i], k);
        if (at[i] >= 0) *reinterpret_cast<uint2*>(pool + at[i] * D + part * 8) = c;
        // to the lane that stores it: row lane % 16, keys below 16, values above
        const int from = __shfl_sync(0xffffffffu, k, (lane % kGroup) % kAtOnce * 2 * kRow + lane / kGroup * kRow);
        if (lane % kGroup / kAtOnce == first + i) byte = from + 127;
      } else if constexpr (APPEND) {
        if (at[i] >= 0) *reinterpret_cast<uint4*>(pool + at[i] * (D * 2) + part * 16) = x[i];
      } else if constexpr (E4M3) {
        const int e = __shfl_sync(0xffffffffu, byte, n + kGroup * value);
        if (at[i] >= 0) *token_row(n) = values(make_uint2(x[i].x, x[i].y), e);
      } else {
        if (at[i] >= 0) *token_row(n) = x[i];
      }
    }
  }
  if constexpr (APPEND && E4M3) {
    if (place >= 0) exps[place] = static_cast<uint8_t>(byte);
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
  a.tasks = (batch->T + kGroup - 1) / kGroup * R * cache->H;
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
      append ? (cache->d == 128 ? (e4m3 ? move_kernel<128, true, true> : move_kernel<128, false, true>)
                                : (e4m3 ? move_kernel<64, true, true> : move_kernel<64, false, true>))
             : (cache->d == 128 ? (e4m3 ? move_kernel<128, true, false> : move_kernel<128, false, false>)
                                : (e4m3 ? move_kernel<64, true, false> : move_kernel<64, false, false>));
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
