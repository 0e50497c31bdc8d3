// Grouped small matrix products (mm_group.hip): up to kMmGroup independent
// C = A . B^T in one launch, for products too small to fill the chip alone.
#pragma once

#include "hss_internal.h"

namespace hss {

static constexpr int kMmGroup = 2;

// C (M x N) = sum_k A[m][ka] B[n][kb], k < K, fp32.  A and B are bf16 with
// 16-byte aligned rows; K and the wraps are multiples of 32.  An operand with
// wrap w < K repeats: its column is k mod w (w >= K / 3).  C[m * ldc + n], or
// C[n * ldc + m] with trans; split z < splits of K writes to C + z * zstride.
struct MmProblem {
  const uint16_t* A;
  const uint16_t* B;
  float* C;
  int64_t ldc, zstride;
  int M, N, K, lda, ldb, wrap_a, wrap_b, trans;
  int splits, stages_per_split, tiles_n, blocks;  // set by launch_mm_group
};

// K splits that give about `target` blocks (at least two K stages each).
int mm_splits(int M, int N, int K, int target);
// The splits that a request for `splits` of K gives (whole K stages, none empty).
int mm_actual_splits(int K, int splits);
void launch_mm_group(const MmProblem* p, int count, hipStream_t s);

}  // namespace hss
