// Large bf16 products on the matrix cores (gemm256.hip).
#pragma once

#include "hss_internal.h"

namespace hss {

enum : int { G256_BF16 = 0, G256_PART = 1, G256_DS = 2 /* + the kind of S's pattern */ };

// Whether the operands suit k_gemm256: K segments in whole stages of 64, rows
// of whole 16-byte chunks (aligned bases), 32-bit byte offsets.
bool gemm256_ok(int M, int N, int K1, int lda, int ldb1, int K2, int ldb2);

// Bytes of the partial products where K is split, enough for every N from
// `from` to N (of one count of tiles: 64 t < from <= N <= 64 (t + 1)).
size_t gemm256_part_bytes(int M, int from, int N, int K);

// C[n * ldc + m] (bf16) = A . [B1 | B2]^T: A's rows hold K1 + K2 columns
// (K2 = 0: no second segment).
void launch_gemm256_bf16(int M, int N, const uint16_t* A, int lda, int K1, const uint16_t* B1, int ldb1, int K2,
                         const uint16_t* B2, int ldb2, void* C, int64_t ldc, float* part, hipStream_t s);

// dS[p] = sum_k Gt[row of p][k] Xt[column of p][k] for the stored entries p of
// S, k < K (K a multiple of 64; rows of ld): the product's tiles stay on the
// chip, only S's entries are written.  tptr: gemm256_ds_bytes(A) bytes.
size_t gemm256_ds_bytes(const hss_matrix* A);
void launch_gemm256_ds(const hss_matrix* A, int K, const uint16_t* Gt, const uint16_t* Xt, int ld, float* dS,
                       int32_t* tptr, hipStream_t s);

}  // namespace hss
