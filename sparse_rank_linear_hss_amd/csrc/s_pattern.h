// The stored positions of S, for the kernels that walk them.
#pragma once

#include "hss_internal.h"

namespace hss {

// S's stored positions: CSR (int32 or 16-bit columns) or 2:4 (row i holds
// n / 2 entries, entry 2g + s the s-th kept column of group g, from the
// nibble at bits 4 (g % 8) of metadata word g / 8).
enum : int { PAT_CSR32 = 0, PAT_CSR16 = 1, PAT_NM24 = 2 };

struct SPattern {
  const int32_t* row_ptr;  // CSR
  const void* col;         // CSR columns
  const uint32_t* meta;    // 2:4 metadata, m x ceil(n / 32)
  int n;
};

template <int PAT>
__device__ __forceinline__ void pat_row(const SPattern& P, int i, int64_t& rs, int64_t& re) {
  if constexpr (PAT == PAT_NM24) {
    rs = (int64_t)i * (P.n >> 1);
    re = rs + (P.n >> 1);
  } else {
    rs = P.row_ptr[i];
    re = P.row_ptr[i + 1];
  }
}

template <int PAT>
__device__ __forceinline__ int pat_col(const SPattern& P, int i, int64_t rs, int64_t p) {
  if constexpr (PAT == PAT_CSR32) {
    return static_cast<const int32_t*>(P.col)[p];
  } else if constexpr (PAT == PAT_CSR16) {
    return static_cast<const uint16_t*>(P.col)[p];
  } else {
    const int q = (int)(p - rs), g = q >> 1;
    const uint32_t w = P.meta[(int64_t)i * ((P.n + 31) >> 5) + (g >> 3)];
    const uint32_t nib = (w >> (4 * (g & 7))) & 15u;
    return 4 * g + (int)((q & 1) ? (nib >> 2) & 3u : nib & 3u);
  }
}

inline SPattern s_pattern(const hss_matrix* A) {
  SPattern P = {};
  P.row_ptr = A->row_ptr;
  P.col = A->col_idx;
  P.meta = A->nm_meta;
  P.n = A->n;
  return P;
}

inline int s_pattern_kind(const hss_matrix* A) {
  return A->fmt == HSS_FMT_2OF4 ? PAT_NM24 : ((A->flags & HSS_COL16) ? PAT_CSR16 : PAT_CSR32);
}

}  // namespace hss
