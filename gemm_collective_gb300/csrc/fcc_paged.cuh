// fcc_paged.cuh -- arguments and launchers of the paged attention's kernels.
#pragma once

#include "fcc_cache.cuh"

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
  float scale_log2;            // scale * log2(e)
  int* status;
  char* ws;
};

constexpr float kLn2 = 0.6931471805599453f;

}  // namespace fcc
