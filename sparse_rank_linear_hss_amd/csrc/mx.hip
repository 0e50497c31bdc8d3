// Microscaled quantisation: hss_mx_quantize and hss_mx_dequantize.
//
// For a group of 32 columns with largest magnitude a (finite), p the code's
// significant bits (fp4 2, int8 7) and q the exponent of its largest power of
// two (fp4 2: 4 = 2^2; int8 6: 64 = 2^6):
//   e     = exponent of a rounded to p bits, nearest (a carry raises it)
//   scale = 2^(e - q),  code = nearest code to w / scale, ties to even
// Rounding a first keeps the largest magnitude within half a step too: a
// plain floor(log2 a) would clip it (fp4: from 7.99 to 6 steps).  The scale is
// a power of two, so w / scale and every value read back are exact, and so is
// the residual w - value (the two are within a factor of two of each other, or
// the value is 0).  e stops at 127 (a magnitude that would round to 2^128 is
// clipped to the largest code) and at -123 (fp4) / -120 (int8), where the
// smallest code is still a normal bf16.
//
// Four lanes take a group, 8 columns each: one or two 16-byte loads, the
// group's maximum by two DPP quad exchanges, and 4 (fp4) or 8 (int8) bytes of
// codes.  The kernels are bound by HBM.
#include <algorithm>

#include "mx_common.h"

namespace hss {

template <int DT>
__device__ __forceinline__ void load8(const void* src, int64_t at, int valid, uint32_t (&bits)[8]) {
  if constexpr (DT == HSS_F32) {
    const uint32_t* p = static_cast<const uint32_t*>(src) + at;
    if (valid == 8) {
      const Bytes16 a = *reinterpret_cast<const Bytes16*>(p), b = *reinterpret_cast<const Bytes16*>(p + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) bits[k] = a.w[k], bits[4 + k] = b.w[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) bits[k] = k < valid ? p[k] : 0u;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(src) + at;
    if (valid == 8) {
      const Bytes16 a = *reinterpret_cast<const Bytes16*>(p);
#pragma unroll
      for (int k = 0; k < 4; ++k) bits[2 * k] = a.w[k] << 16, bits[2 * k + 1] = a.w[k] & 0xffff0000u;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) bits[k] = k < valid ? (uint32_t)p[k] << 16 : 0u;
    }
  }
}

// Eight fp32 values, exact in the storage type, to dst[at ..].
template <int DT>
__device__ __forceinline__ void store8(void* dst, int64_t at, int valid, const float (&v)[8]) {
  if constexpr (DT == HSS_F32) {
    float* p = static_cast<float*>(dst) + at;
    if (valid == 8) {
      Bytes16 a, b;
#pragma unroll
      for (int k = 0; k < 4; ++k) a.w[k] = __float_as_uint(v[k]), b.w[k] = __float_as_uint(v[4 + k]);
      *reinterpret_cast<Bytes16*>(p) = a;
      *reinterpret_cast<Bytes16*>(p + 4) = b;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < valid) p[k] = v[k];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(dst) + at;
    if (valid == 8) {
      Bytes16 a;
#pragma unroll
      for (int k = 0; k < 4; ++k) a.w[k] = mx_pack_hi(v[2 * k], v[2 * k + 1]);
      *reinterpret_cast<Bytes16*>(p) = a;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < valid) p[k] = (uint16_t)(__float_as_uint(v[k]) >> 16);
    }
  }
}

template <int FMT, int DT>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* src, int cols, int ng, uint32_t groups,
                                                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                     void* residual) {
  constexpr int P = FMT == HSS_MXFP4 ? 2 : 7, Q = FMT == HSS_MXFP4 ? 2 : 6;
  constexpr int EMIN = FMT == HSS_MXFP4 ? -123 : -120;
  const int q = threadIdx.x & 3;
  const uint32_t step = gridDim.x * 64u;
  // groups < 2^26 and step < 2^19: no wrap
  for (uint32_t g = blockIdx.x * 64u + (threadIdx.x >> 2); g < groups; g += step) {
    const uint32_t row = g / (uint32_t)ng;
    const int c0 = (int)(g - row * (uint32_t)ng) * kMxGroup + 8 * q;
    const int valid = min(max(cols - c0, 0), 8);
    const int64_t at = (int64_t)row * cols + c0;
    uint32_t bits[8];
    load8<DT>(src, at, valid, bits);
    uint32_t a = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) a = max(a, bits[k] & 0x7fffffffu);
    // the four lanes of the group are active together
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, false));
    const bool bad = a >= 0x7f800000u;
    const int e = min(max((int)((a + (1u << (23 - P))) >> 23) - 127, EMIN), 127);
    const int s = e - Q;  // within -126 .. 125: 2^s and 2^-s are normal
    const float up = __uint_as_float((uint32_t)(s + 127) << 23), down = __uint_as_float((uint32_t)(127 - s) << 23);
    float rest[8];
    if constexpr (FMT == HSS_MXFP4) {
      uint32_t word = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __uint_as_float(bits[k]);
        const float v = fabsf(w) * down;
        // to a multiple of 1/2, 1 or 2 (ties to even) by adding a power of
        // two whose last place is that step
        const uint32_t i0 = __float_as_uint(v + 4194304.f) - 0x4a800000u;
        const uint32_t i1 = __float_as_uint(v + 8388608.f) - 0x4b000000u;
        const uint32_t i2 = __float_as_uint(v + 16777216.f) - 0x4b800000u;
        const uint32_t code = v < 2.f ? i0 : (v < 4.f ? i1 + 2u : min(i2 + 4u, 7u));
        word |= (bad ? 0u : code | (bits[k] >> 31) << 3) << (4 * k);
        const float grid = code < 4u ? 0.5f * (float)code : (float)(2u + (code & 1u)) * (code < 6u ? 1.f : 2.f);
        rest[k] = w - copysignf(grid, w) * up;
      }
      *reinterpret_cast<uint32_t*>(codes + (int64_t)g * 16 + 4 * q) = word;
    } else {
      uint32_t word[2] = {0u, 0u};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __uint_as_float(bits[k]);
        const float v = fminf(fmaxf(rintf(w * down), -127.f), 127.f);
        word[k >> 2] |= (bad ? 0u : (uint32_t)(int)v & 255u) << (8 * (k & 3));
        rest[k] = w - v * up;
      }
      *reinterpret_cast<mx_u32x2*>(codes + (int64_t)g * 32 + 8 * q) = mx_u32x2{word[0], word[1]};
    }
    if (q == 0) scales[g] = (uint8_t)(bad ? 255 : (FMT == HSS_MXFP4 ? s : e) + 127);
    if (residual) {
      if (bad) {
#pragma unroll
        for (int k = 0; k < 8; ++k) rest[k] = __uint_as_float(0x7fc00000u);
      }
      store8<DT>(residual, at, valid, rest);
    }
  }
}

template <int FMT, int DT>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int cols, int ng,
                                                       uint32_t groups, void* __restrict__ dst) {
  const int q = threadIdx.x & 3;
  const uint32_t step = gridDim.x * 64u;
  for (uint32_t g = blockIdx.x * 64u + (threadIdx.x >> 2); g < groups; g += step) {
    const uint32_t row = g / (uint32_t)ng;
    const int c0 = (int)(g - row * (uint32_t)ng) * kMxGroup + 8 * q;
    const int valid = min(max(cols - c0, 0), 8);
    const int64_t at = (int64_t)row * cols + c0;
    float v[8];
    if constexpr (FMT == HSS_MXFP4) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + (int64_t)g * 16 + 4 * q);
      const u32x4 h = mx4_to_bf16x8(word, mx_scale(scales[g], 0));
#pragma unroll
      for (int k = 0; k < 4; ++k) v[2 * k] = bf16lo(h[k]), v[2 * k + 1] = bf16hi(h[k]);
    } else {
      const mx_u32x2 word = *reinterpret_cast<const mx_u32x2*>(codes + (int64_t)g * 32 + 8 * q);
      const float scale = mx_scale(scales[g], 6);
      mx8_to_f32x4(word.x, scale, v);
      mx8_to_f32x4(word.y, scale, v + 4);
    }
    if (valid > 0) store8<DT>(dst, at, valid, v);
  }
}

static unsigned mx_grid(int64_t groups) { return (unsigned)std::min<int64_t>((groups + 63) / 64, 8192); }

hss_status launch_mx_quantize(int fmt, int dt, int rows, int cols, const void* src, void* codes, uint8_t* scales,
                              void* residual, hipStream_t s) {
  const int ng = mx_groups(cols);
  const int64_t groups = (int64_t)rows * ng;
  const dim3 grid(mx_grid(groups)), block(256);
  uint8_t* c = static_cast<uint8_t*>(codes);
  if (fmt == HSS_MXFP4) {
    if (dt == HSS_F32)
      hipLaunchKernelGGL((k_mx_quantize<HSS_MXFP4, HSS_F32>), grid, block, 0, s, src, cols, ng, (uint32_t)groups, c, scales, residual);
    else
      hipLaunchKernelGGL((k_mx_quantize<HSS_MXFP4, HSS_BF16>), grid, block, 0, s, src, cols, ng, (uint32_t)groups, c, scales, residual);
  } else {
    if (dt == HSS_F32)
      hipLaunchKernelGGL((k_mx_quantize<HSS_MXINT8, HSS_F32>), grid, block, 0, s, src, cols, ng, (uint32_t)groups, c, scales, residual);
    else
      hipLaunchKernelGGL((k_mx_quantize<HSS_MXINT8, HSS_BF16>), grid, block, 0, s, src, cols, ng, (uint32_t)groups, c, scales, residual);
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

hss_status launch_mx_dequantize(int fmt, int dt, int rows, int cols, const void* codes, const uint8_t* scales,
                                void* dst, hipStream_t s) {
  const int ng = mx_groups(cols);
  const int64_t groups = (int64_t)rows * ng;
  const dim3 grid(mx_grid(groups)), block(256);
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  if (fmt == HSS_MXFP4) {
    if (dt == HSS_F32)
      hipLaunchKernelGGL((k_mx_dequantize<HSS_MXFP4, HSS_F32>), grid, block, 0, s, c, scales, cols, ng, (uint32_t)groups, dst);
    else
      hipLaunchKernelGGL((k_mx_dequantize<HSS_MXFP4, HSS_BF16>), grid, block, 0, s, c, scales, cols, ng, (uint32_t)groups, dst);
  } else {
    if (dt == HSS_F32)
      hipLaunchKernelGGL((k_mx_dequantize<HSS_MXINT8, HSS_F32>), grid, block, 0, s, c, scales, cols, ng, (uint32_t)groups, dst);
    else
      hipLaunchKernelGGL((k_mx_dequantize<HSS_MXINT8, HSS_BF16>), grid, block, 0, s, c, scales, cols, ng, (uint32_t)groups, dst);
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
