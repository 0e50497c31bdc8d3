// hss_apply of layers with a microscaled 4-bit dense part (HSS_MX4):
//   Y = X (S + U V^T + D)^T,  D MXFP4, m x n; with HSS_MX4_T the stored array
//   is D^T (n x m), so that a layer and its transposed layer share one copy.
//
// Up to 16 columns, D not transposed: mx_skinny.hip.  General route, any batch:
//   W'  = D + S as dense bf16 in the workspace, rows padded to 64 columns
//   T   = X V in fp32 (matrix cores), kept as two bf16 terms T = T1 + T2 (16
//         significant bits, so that rounding T does not show beside the
//         rounding of Y)
//   Y   = [X | T1 | T2] . [W' | U | U]^T, one matrix-core product with fp32
//         accumulation, rounded to bf16 once.
// D is exact in bf16 and S is bf16: W' rounds only where an entry of S falls
// on a non-zero of D.  Operands whose rows the matrix-core kernels cannot read
// in 16-byte pieces (n not a multiple of 64, unaligned bases) are copied
// into padded rows first.
#include <algorithm>

#include "gemm256.h"
#include "mx_common.h"

namespace hss {

// mfma.hip
void launch_gemm_bf16x2(int M, int N, int K1, const uint16_t* A1, int64_t lda1, const uint16_t* B1, int64_t ldb1,
                        int K2, const uint16_t* A2, int64_t lda2, const uint16_t* B2, int64_t ldb2, void* C,
                        int64_t ldc, bool out_bf16, float* part, hipStream_t s);
size_t gemm_bf16x2_part_bytes(int M, int N, int K1, int K2, int64_t ldc);

// mx_skinny.hip
bool mx_skinny_supported(const hss_matrix* A, int b);
size_t mx_skinny_ws_bytes(const hss_matrix* A, int b);
hss_status launch_mx_skinny(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s);

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

// ---------------------------------------------------------------------------
// W' = D + S, one wave per row, kMxSeg columns at a time through LDS: the
// decoded codes first, then the row's entries of S added to them (an entry's
// column occurs once per row, so no two lanes meet), then 16-byte stores.
// ---------------------------------------------------------------------------
static constexpr int kMxSeg = 4096;  // columns per segment: 8 KiB of LDS per wave

template <typename COL>
__global__ __launch_bounds__(256) void k_mx_densify(const uint8_t* __restrict__ codes,
                                                    const uint8_t* __restrict__ scales,
                                                    const int32_t* __restrict__ row_ptr,
                                                    const COL* __restrict__ col_idx,
                                                    const uint16_t* __restrict__ vals, int m, int n, int np,
                                                    int ldw, uint16_t* __restrict__ W) {
  __shared__ __align__(16) uint16_t seg[4][kMxSeg];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int row = blockIdx.x * 4 + w;
  if (row >= m) return;  // no block-wide barrier below
  const int ng = mx_groups(n);
  uint16_t* L = seg[w];
  const int p0 = row_ptr[row], p1 = row_ptr[row + 1];
  for (int c0 = 0; c0 < np; c0 += kMxSeg) {
    const int len = min(kMxSeg, np - c0);  // a multiple of 32
    for (int j = 8 * lane; j < len; j += 512) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (((c0 + j) >> 5) < ng) {
        const int64_t g = (int64_t)row * ng + ((c0 + j) >> 5);
        const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + g * 16 + ((j >> 1) & 12));
        v = mx4_to_bf16x8(word, mx_scale(scales[g], 0));
      }
      *reinterpret_cast<u32x4*>(L + j) = v;
    }
    // A wave's LDS accesses complete in issue order; the empty asm keeps the
    // compiler from reordering the three phases.
    asm volatile("" ::: "memory");
    for (int p = p0 + lane; p < p1; p += 64) {
      const int c = (int)col_idx[p];
      if ((unsigned)(c - c0) < (unsigned)len && c < n)
        L[c - c0] = f32_to_bf16(__uint_as_float((uint32_t)L[c - c0] << 16) + __uint_as_float((uint32_t)vals[p] << 16));
    }
    asm volatile("" ::: "memory");
    for (int j = 8 * lane; j < len; j += 512)
      *reinterpret_cast<u32x4*>(W + (int64_t)row * ldw + c0 + j) = *reinterpret_cast<const u32x4*>(L + j);
    asm volatile("" ::: "memory");
  }
}

// W' = D^T, m x np from the stored n x m codes: tiles of 64 stored rows (W'
// columns) x 128 stored columns (4 groups, 64 bytes of codes per row).
static constexpr int kTrI = 64, kTrJ = 128;
__global__ __launch_bounds__(256) void k_mx_densify_t(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int m, int n, int np,
                                                      int ldw, int tiles_j,
                                                      uint16_t* __restrict__ W) {
  __shared__ __align__(16) uint16_t tile[kTrJ][kTrI + 8];
  const int i0 = (int)(blockIdx.x / (unsigned)tiles_j) * kTrI, j0 = (int)(blockIdx.x % (unsigned)tiles_j) * kTrJ;
  const int ng = mx_groups(m);
  const int t = threadIdx.x;
  {
    const int i = t >> 2, g = (j0 >> 5) + (t & 3);
    u32x4 cw = {0u, 0u, 0u, 0u};
    float sc = 0.f;
    if (i0 + i < n && g < ng) {
      const int64_t at = (int64_t)(i0 + i) * ng + g;
      cw = *reinterpret_cast<const u32x4*>(codes + at * 16);
      sc = mx_scale(scales[at], 0);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const u32x4 h = sc != 0.f ? mx4_to_bf16x8(cw[k], sc) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        tile[32 * (t & 3) + 8 * k + 2 * e][i] = (uint16_t)h[e];
        tile[32 * (t & 3) + 8 * k + 2 * e + 1][i] = (uint16_t)(h[e] >> 16);
      }
    }
  }
  __syncthreads();
  for (int q = t; q < kTrJ * (kTrI / 8); q += 256) {
    const int j = q >> 3, c = (q & 7) * 8;
    if (j0 + j < m && i0 + c < np)
      *reinterpret_cast<u32x4*>(W + (int64_t)(j0 + j) * ldw + i0 + c) = *reinterpret_cast<const u32x4*>(&tile[j][c]);
  }
}

// W' += S: one wave per row, one entry per lane and step.
template <typename COL>
__global__ __launch_bounds__(256) void k_mx_add_csr(const int32_t* __restrict__ row_ptr,
                                                    const COL* __restrict__ col_idx,
                                                    const uint16_t* __restrict__ vals, int m, int n, int ldw,
                                                    uint16_t* __restrict__ W) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= m) return;
  uint16_t* Wr = W + (int64_t)row * ldw;
  const int p1 = row_ptr[row + 1];
  for (int p = row_ptr[row] + lane_id(); p < p1; p += 64) {
    const int c = (int)col_idx[p];
    if ((unsigned)c < (unsigned)n)
      Wr[c] = f32_to_bf16(__uint_as_float((uint32_t)Wr[c] << 16) + __uint_as_float((uint32_t)vals[p] << 16));
  }
}

// `rep` copies of [src row | zeros] (colsp columns each, a multiple of 8) in
// rows of ldd.
__global__ __launch_bounds__(256) void k_mx_pad(const uint16_t* __restrict__ src, int rows, int cols, int colsp,
                                                int rep, int64_t ldd, uint16_t* __restrict__ dst) {
  const uint32_t per = (uint32_t)colsp >> 3, total = (uint32_t)rows * per;
  for (uint32_t q = blockIdx.x * 256u + threadIdx.x; q < total; q += gridDim.x * 256u) {
    const uint32_t row = q / per;
    const int c = (int)(q - row * per) * 8;
    const uint16_t* p = src + (int64_t)row * cols + c;
    u32x4 v;
    if (c + 8 <= cols) {
      const Bytes16 a = *reinterpret_cast<const Bytes16*>(p);
      v = u32x4{a.w[0], a.w[1], a.w[2], a.w[3]};
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = c + 2 * k < cols ? p[2 * k] : 0u, hi = c + 2 * k + 1 < cols ? p[2 * k + 1] : 0u;
        v[k] = lo | hi << 16;
      }
    }
    for (int z = 0; z < rep; ++z) *reinterpret_cast<u32x4*>(dst + row * ldd + (int64_t)z * colsp + c) = v;
  }
}

// T (rows x cols fp32) as `terms` bf16 terms side by side (colsp columns
// each, zero past cols): term z is the rest after the terms before it,
// rounded to nearest.
__global__ __launch_bounds__(256) void k_mx_terms(const float* __restrict__ T, int rows, int cols, int64_t ld,
                                                  int colsp, int terms, uint16_t* __restrict__ dst) {
  const uint32_t total = (uint32_t)rows * (uint32_t)colsp;
  for (uint32_t q = blockIdx.x * 256u + threadIdx.x; q < total; q += gridDim.x * 256u) {
    const uint32_t row = q / (uint32_t)colsp;
    const int c = (int)(q - row * (uint32_t)colsp);
    float v = c < cols ? T[row * ld + c] : 0.f;
    for (int z = 0; z < terms; ++z) {
      const uint16_t h = f32_to_bf16(v);
      dst[((int64_t)row * terms + z) * colsp + c] = h;
      // (an infinity leaves 0, not the NaN of inf - inf)
      const float hf = __uint_as_float((uint32_t)h << 16);
      v = (h & 0x7fffu) == 0x7f80u ? 0.f : v - hf;
    }
  }
}

void launch_mx_pad(const uint16_t* src, int rows, int cols, int colsp, int rep, int64_t ldd, uint16_t* dst,
                   hipStream_t s) {
  const int64_t total = (int64_t)rows * (colsp >> 3);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 4096);
  hipLaunchKernelGGL(k_mx_pad, dim3(grid), dim3(256), 0, s, src, rows, cols, colsp, rep, ldd, dst);
}

void launch_mx_terms(const float* T, int rows, int cols, int64_t ld, int colsp, int terms, uint16_t* dst,
                     hipStream_t s) {
  const int64_t total = (int64_t)rows * colsp;
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 4096);
  hipLaunchKernelGGL(k_mx_terms, dim3(grid), dim3(256), 0, s, T, rows, cols, ld, colsp, terms, dst);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static constexpr int kG256MinTiles = 128;

struct MxPlan {
  int np, rp;
  size_t w, x, vt, tf, tb, part, total;
};

static MxPlan plan_mx(const hss_matrix* A, int b) {
  MxPlan p;
  const int m = A->m, n = A->n, r = A->r;
  p.np = (n + 63) & ~63;
  p.rp = r > 0 ? round32(r) : 0;
  size_t off = 0;
  p.w = off;  off += al256((size_t)m * (p.np + 2 * p.rp) * 2);
  p.x = off;  off += al256((size_t)b * p.np * 2);
  p.vt = off; off += al256((size_t)r * p.np * 2);
  p.tf = off; off += al256((size_t)b * r * 4);
  p.tb = off; off += al256((size_t)b * p.rp * 4);
  p.part = off;
  const size_t pt = r > 0 ? gemm_bf16x2_part_bytes(r, b, p.np, 0, r) : 0;
  off += al256(std::max(pt, gemm_bf16x2_part_bytes(m, b, p.np, 2 * p.rp, m)));
  p.total = off;
  return p;
}

size_t mx_apply_ws_bytes(const hss_matrix* A, int b) {
  return mx_skinny_supported(A, b) ? mx_skinny_ws_bytes(A, b) : plan_mx(A, b).total;
}

static bool rows_ok(const void* p, int cols) { return (uintptr_t)p % 16 == 0 && cols % 64 == 0; }

hss_status launch_mx_apply(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s) {
  if (mx_skinny_supported(A, b)) return launch_mx_skinny(A, b, X, Y, ws, s);
  const MxPlan p = plan_mx(A, b);
  char* base = static_cast<char*>(ws);
  uint16_t* W = reinterpret_cast<uint16_t*>(base + p.w);
  float* Tf = reinterpret_cast<float*>(base + p.tf);
  uint16_t* Tb = reinterpret_cast<uint16_t*>(base + p.tb);
  float* part = reinterpret_cast<float*>(base + p.part);
  const int m = A->m, n = A->n, r = A->r, np = p.np, rp = p.rp, ldw = np + 2 * rp;
  uint16_t* Ub = W + np;  // [W' | U | U]
  const dim3 rows4((unsigned)((m + 3) / 4));
  const uint8_t* codes = A->dq_codes;
  const uint8_t* scales = static_cast<const uint8_t*>(A->dq_levels);
  const uint16_t* vals = static_cast<const uint16_t*>(A->values);
  const uint16_t* col16 = reinterpret_cast<const uint16_t*>(A->col_idx);
  if (A->flags & HSS_MX4_T) {
    const int tiles_j = (m + kTrJ - 1) / kTrJ;
    hipLaunchKernelGGL(k_mx_densify_t, dim3((unsigned)tiles_j * (unsigned)((np + kTrI - 1) / kTrI)), dim3(256), 0, s,
                       codes, scales, m, n, np, ldw, tiles_j, W);
    if (A->nnz > 0) {
      if (A->flags & HSS_COL16)
        hipLaunchKernelGGL(k_mx_add_csr<uint16_t>, rows4, dim3(256), 0, s, A->row_ptr, col16, vals, m, n, ldw, W);
      else
        hipLaunchKernelGGL(k_mx_add_csr<int32_t>, rows4, dim3(256), 0, s, A->row_ptr, A->col_idx, vals, m, n, ldw, W);
    }
  } else if (A->flags & HSS_COL16) {
    hipLaunchKernelGGL(k_mx_densify<uint16_t>, rows4, dim3(256), 0, s, codes, scales, A->row_ptr, col16,
                       vals, m, n, np, ldw, W);
  } else {
    hipLaunchKernelGGL(k_mx_densify<int32_t>, rows4, dim3(256), 0, s, codes, scales, A->row_ptr,
                       A->col_idx, vals, m, n, np, ldw, W);
  }
  const uint16_t* Xb = static_cast<const uint16_t*>(X);
  if (!rows_ok(X, n)) {
    uint16_t* xp = reinterpret_cast<uint16_t*>(base + p.x);
    launch_mx_pad(Xb, b, n, np, 1, np, xp, s);
    Xb = xp;
  }
  if (r > 0) {
    const uint16_t* Vb = static_cast<const uint16_t*>(A->Vt);
    if (!rows_ok(A->Vt, n)) {
      uint16_t* vp = reinterpret_cast<uint16_t*>(base + p.vt);
      launch_mx_pad(Vb, r, n, np, 1, np, vp, s);
      Vb = vp;
    }
    launch_gemm_bf16x2(r, b, np, Vb, np, Xb, np, 0, nullptr, 0, nullptr, 0, Tf, r, false, part, s);
    launch_mx_terms(Tf, b, r, r, rp, 2, Tb, s);
    launch_mx_pad(static_cast<const uint16_t*>(A->U), m, r, rp, 2, ldw, Ub, s);
  }
  if (((m + 255) / 256) * ((b + 255) / 256) >= kG256MinTiles && gemm256_ok(m, b, np, ldw, np, 2 * rp, 2 * rp))
    launch_gemm256_bf16(m, b, W, ldw, np, Xb, np, 2 * rp, Tb, 2 * rp, Y, m, s);
  else
    launch_gemm_bf16x2(m, b, np, W, ldw, Xb, np, 2 * rp, Ub, ldw, Tb, 2 * rp, Y, m, true, part, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
