// Microscaled formats (OCP MX element types E2M1 and INT8 with a shared
// E8M0 power-of-two scale), as the kernels read them.
//
// A group is 32 consecutive columns of one row; a row holds ng =
// ceil(cols / 32) groups, the last one padded with zero codes, so that every
// group starts on a 16-byte boundary whatever cols is.
//   fp4   16 bytes per group: byte j holds columns 2j (low nibble) and 2j + 1;
//         nibble = sign << 3 | code, codes 0..7 = 0, .5, 1, 1.5, 2, 3, 4, 6;
//         value = code value * 2^(scale byte - 127)
//   int8  32 bytes per group, two's complement, -127..127;
//         value = code * 2^(scale byte - 127 - 6)
// Scale byte 255 marks a group that held a NaN or an infinity: every value of
// it reads as NaN.
#pragma once

#include "hss_internal.h"

namespace hss {

static constexpr int kMxGroup = 32;

__host__ __device__ inline int mx_groups(int cols) { return (cols + kMxGroup - 1) / kMxGroup; }

typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t mx_u32x2 __attribute__((ext_vector_type(2)));

// 16 bytes at any 2-byte aligned address (one global_load_dwordx4: the
// hardware takes unaligned vector accesses to global memory).
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t w[4];
};

// The scale of a byte as fp32; `sub` = 0 (fp4) or 6 (int8).
__device__ __forceinline__ float mx_scale(uint32_t byte, uint32_t sub) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((byte > sub ? byte - sub : 0u) << 23);
}

// Eight fp4 codes (one dword) -> eight bf16 values in four dwords, exact (a
// value has two significant bits).  `scale` is a power of two, or NaN.
__device__ __forceinline__ u32x4 mx4_to_bf16x8(uint32_t codes, float scale) {
  u32x4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return r;
}

// Two fp32 values, exact in bf16, packed (their upper halves).
__device__ __forceinline__ uint32_t mx_pack_hi(float lo, float hi) {
  return (__float_as_uint(lo) >> 16) | (__float_as_uint(hi) & 0xffff0000u);
}

// Four int8 codes (one dword) times scale -> four fp32 values (exact).
__device__ __forceinline__ void mx8_to_f32x4(uint32_t codes, float scale, float* v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = (float)((int32_t)(codes << (24 - 8 * k)) >> 24) * scale;
}

// Eight bf16 at any 2-byte aligned address.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ p) {
  const Bytes16 a = *reinterpret_cast<const Bytes16*>(p);
  return u32x4{a.w[0], a.w[1], a.w[2], a.w[3]};
}

// Eight bf16 of a row of n at column k, zeros past the end.  WHOLE: n is a
// multiple of 8 (no column-by-column tail, whose loads the compiler waits for
// one by one -- so callers branch on n once for a whole kernel).
template <bool WHOLE = false>
__device__ __forceinline__ u32x4 load_row8(const uint16_t* __restrict__ row, int k, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (WHOLE ? k < n : k + 8 <= n) {
    v = load8(row + k);
  } else if (!WHOLE && k < n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = k + 2 * e < n ? row[k + 2 * e] : 0u, hi = k + 2 * e + 1 < n ? row[k + 2 * e + 1] : 0u;
      v[e] = lo | hi << 16;
    }
  }
  return v;
}

// ---------------------------------------------------------------------------
// k_mx_prep (mx_skinny.hip): T = X V in K splits, X^T, padded X and U.
// ---------------------------------------------------------------------------
// Most K splits of T (4096 x 11008, one column, r 64: 11.4 us in all, with 8
// splits 12.2).
static constexpr int kMxPrepSplits = 16;

struct MxPrep {
  const uint16_t* X;
  const uint16_t* Vt;
  float* Tp;      // [splits][b][rp], with r > 0
  uint16_t* Xt;   // n x ldt; null = none
  uint16_t* Xp;   // b x np;  null = none
  uint16_t* Xo;   // X in k_mx_skinny's operand order, nch chunks of 2048 values; null = none
  const uint16_t* U;
  uint16_t* Up;   // m x rp;  null = none
  int m, b, n, r, rp, ltiles, splits, steps_per_split, tb, xb, ldt, np, nch;
};

MxPrep mx_prep_plan(const hss_matrix* A, int b);  // the sizes of T
void launch_mx_prep(MxPrep p, hipStream_t s);

}  // namespace hss
