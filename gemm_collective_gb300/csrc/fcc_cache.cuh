// fcc_cache.cuh -- the paged key/value cache as the kernels see it: addresses of
// rows, the sequences of a step and what is checked of them, e4m3 codes.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fcc.h"

namespace fcc {

// One step's sequences (fcc_batch) on the device.
struct StepArgs {
  const int* start;   // [B + 1]
  const int* len;     // [B]
  const int* table;   // [B, max_pages]
  int64_t max_pages;
  int B, T;
};

// The pools of every rank.  Row (page, h, row) of a pool is number
// (page * H + h) * P + row, which passes 32 bits: it is kept in 64.
struct PoolArgs {
  char* K[FCC_MAX_RANKS];
  char* V[FCC_MAX_RANKS];
  uint8_t* Ke[FCC_MAX_RANKS];   // e4m3 only
  uint8_t* Ve[FCC_MAX_RANKS];
  int64_t pages;
  int log2P;
  int H, d;
};

__device__ __forceinline__ void record_invalid(int* status) {
  if (status != nullptr) atomicCAS(status, 0, 1 /* FCC_ERR_INVALID */);
}

// A sequence of the step: rows [s, s + n) of the token arrays, L positions (n where
// it has fewer, which leaves it without any: ok is false).
struct Seq {
  int s, n, L;
  bool rows_ok;   // the rows lie inside the token arrays
  bool ok;        // ... and there are positions for them
};

__device__ __forceinline__ Seq load_seq(const StepArgs& a, int b) {
  Seq q;
  q.s = __ldg(a.start + b);
  const int e = __ldg(a.start + b + 1);
  q.L = __ldg(a.len + b);
  q.rows_ok = q.s >= 0 && e >= q.s && e <= a.T;
  q.n = q.rows_ok ? e - q.s : 0;
  q.ok = q.rows_ok && q.L >= q.n;
  if (!q.ok) q.L = q.n;
  return q;
}

// The page of positions [idx * P, (idx + 1) * P) of sequence b, or -1.
__device__ __forceinline__ int page_of(const StepArgs& a, int64_t pages, int b, int idx) {
  if (idx < 0 || idx >= a.max_pages) return -1;
  const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + idx);
  return page >= 0 && page < pages ? page : -1;
}

// The sequence that row t may belong to: the last b with start[b] <= t, found by
// a whole warp 32 ways at a time.  Only for non-decreasing starts is it the one;
// the caller checks that t lies in it.
__device__ __forceinline__ int warp_find_seq(const StepArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, count = a.B;
  while (count > 1) {
    const int step = (count + 31) >> 5;
    const int i = lane * step;
    const bool le = i < count && __ldg(a.start + lo + i) <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int k = m == 0 ? 0 : 31 - __clz(m);
    lo += k * step;
    count = min(step, count - k * step);
  }
  return lo;
}

// 2^k for k in [-126, 127].
__device__ __forceinline__ float power_of_two(int k) {
  return __int_as_float((k + 127) << 23);
}

}  // namespace fcc

#include "fcc_internal.h"

namespace fcc {
// Checks the descriptions (before anything touches CUDA) and fills the kernels'
// arguments (fcc_cache.cu).
fcc_status cache_args(int R, const fcc_cache* cache, const fcc_batch* batch, PoolArgs* pool,
                      StepArgs* step);
}  // namespace fcc
