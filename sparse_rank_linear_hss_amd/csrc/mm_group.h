// Grouped small matrix products (mm_group.hip): up to kMmGroup independent
// C = A . B^T in one launch, for products too small to fill the chip alone.
#pragma once

#include "hss_internal.h"

namespace hss {

static constexpr int kMmGroup = 2;

// C (M x N) = sum_k A[m][k] B[n][k], k < K, fp32.  A and B are bf16 with
// 16-byte aligned rows; K is a multiple of 32.  C[m * ldc + n], or C[n * ldc +
// m] with trans; split z < splits of K writes to C + z * zstride.  terms3: A's
// rows hold three terms of K columns each, whose sum is meant.
struct MmProblem {
  const uint16_t* A;
  const uint16_t* B;
  float* C;
  int64_t ldc, zstride;
  int M, N, K, lda, ldb, trans;
  int splits, stages_per_split, tiles_n, blocks;  // the last three: set by launch_mm_group
};

// K splits that give about `target` blocks (at least two K stages each).
int mm_splits(int M, int N, int K, int target);
// The splits that a request for `splits` of K gives (whole K stages, none empty).
int mm_actual_splits(int K, int splits);
void launch_mm_group(const MmProblem* p, int count, bool terms3, hipStream_t s);

}  // namespace hss
