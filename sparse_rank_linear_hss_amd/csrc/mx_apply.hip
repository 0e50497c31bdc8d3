// hss_apply of layers with a microscaled 4-bit dense part (HSS_MX4):
//   Y = X (S + U V^T + D)^T,  D MXFP4, m x n; with HSS_MX4_T the stored array
//   is D^T (n x m), so that a layer and its transposed layer share one copy.
//
// Up to 16 columns, D not transposed: mx_skinny.hip; else up to 256 columns:
// mx_gemm.hip.  Beyond:
//   W'  = D + S as dense bf16 in the workspace, rows padded to 64 columns
//   T   = X V in fp32 (matrix cores), kept as two bf16 terms T = T1 + T2 (16
//         significant bits, so that rounding T does not show beside the
//         rounding of Y)
//   Y   = [X | T1 | T2] . [W' | U | U]^T, one matrix-core product with fp32
//         accumulation, rounded to bf16 once.
// D is exact in bf16 and S is bf16: W' rounds only where an entry of S falls
// on a non-zero of D.  There it has the precision of a bf16 weight, which S's
// values and the matrix they were taken from have too; the remainders would
// take a gather over X^T next to the product (4096^2, 3 % of S, 55 % of it on
// non-zeros: the relative error of Y is 1.683e-3 with the rounding, 1.659e-3
// without, as up to 256 columns, nearly all of it Y's own rounding).  Operands
// whose rows the matrix-core kernels cannot read in 16-byte pieces (n not a
// multiple of 64, unaligned bases) are copied into padded rows first.
#include <algorithm>

#include "gemm256.h"
#include "mm_group.h"
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

// mx_gemm.hip
bool mx_gemm_supported(int b);
size_t mx_gemm_ws_bytes(const hss_matrix* A, int b);
hss_status launch_mx_gemm(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s);
void launch_mx_tsum(const float* Tp, int splits, int b, int r, int rp, uint16_t* Tb, hipStream_t s);

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

// ---------------------------------------------------------------------------
// W' = D + S.  A wave takes 2048 columns of a row, a lane one group of them
// (16 bytes of codes): decoded into LDS, then the row's entries of S there
// added (an entry's column occurs once per row, so no two lanes meet), then
// 16-byte stores, 1 KiB a wave.  Bound by the stores (8192^2: 34.6 us, 4.9 TB/s).
// ---------------------------------------------------------------------------
// The row's two copies of U, rp columns each (zero past r), by one wave.
__device__ __forceinline__ void put_u(const uint16_t* __restrict__ U, int row, int r, int rp, uint16_t* __restrict__ dst) {
  for (int l = 8 * lane_id(); l < rp; l += 512) {
    const u32x4 v = r % 8 == 0 ? load_row8<true>(U + (int64_t)row * r, l, r) : load_row8(U + (int64_t)row * r, l, r);
    *reinterpret_cast<u32x4*>(dst + l) = v;
    *reinterpret_cast<u32x4*>(dst + rp + l) = v;
  }
}

static constexpr int kMxSeg = 2048;  // columns of one wave: 4 KiB of LDS

// Where column c of a wave's segment lies: the group's 16-byte pieces are
// permuted by the group, so that the lanes' stores of them do not conflict.
__device__ __forceinline__ int seg_at(int c) { return (c & ~31) | ((((c >> 3) ^ (c >> 6)) & 3) << 3) | (c & 7); }

template <typename COL>
__global__ __launch_bounds__(256) void k_mx_densify(const uint8_t* __restrict__ codes,
                                                    const uint8_t* __restrict__ scales,
                                                    const int32_t* __restrict__ row_ptr,
                                                    const COL* __restrict__ col_idx,
                                                    const uint16_t* __restrict__ vals, int m, int n, int np,
                                                    int ldw, const uint16_t* __restrict__ U, int r, int rp,
                                                    int segs, uint16_t* __restrict__ W) {
  __shared__ __align__(16) uint16_t seg[4][kMxSeg];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t unit = blockIdx.x * 4u + (uint32_t)w;
  const int row = (int)(unit / (uint32_t)segs), c0 = (int)(unit - (uint32_t)row * (uint32_t)segs) * kMxSeg;
  if (row >= m) return;  // no block-wide barrier below
  const int ng = mx_groups(n), g = (c0 >> 5) + lane;
  uint16_t* L = seg[w];
  u32x4 code = {0u, 0u, 0u, 0u};
  float sc = 1.f;
  if (g < ng) {
    const int64_t at = (int64_t)row * ng + g;
    code = *reinterpret_cast<const u32x4*>(codes + at * 16);
    sc = mx_scale(scales[at], 0);
  }
  const int p0 = row_ptr[row], p1 = row_ptr[row + 1];
  if (c0 == 0) put_u(U, row, r, rp, W + (int64_t)row * ldw + np);
#pragma unroll
  for (int k = 0; k < 4; ++k) *reinterpret_cast<u32x4*>(L + seg_at(32 * lane + 8 * k)) = mx4_to_bf16x8(code[k], sc);
  // A wave's LDS accesses complete in issue order; the empty asm keeps the
  // compiler from reordering the three phases.
  asm volatile("" ::: "memory");
  for (int p = p0 + lane; p < p1; p += 64) {
    const int c = (int)col_idx[p] - c0;
    if ((unsigned)c < (unsigned)min(kMxSeg, n - c0)) {
      uint16_t* at = L + seg_at(c);
      *at = f32_to_bf16(__uint_as_float((uint32_t)*at << 16) + __uint_as_float((uint32_t)vals[p] << 16));
    }
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = 8 * lane + 512 * k;
    if (c0 + j < np)
      *reinterpret_cast<u32x4*>(W + (int64_t)row * ldw + c0 + j) = *reinterpret_cast<const u32x4*>(L + seg_at(j));
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

// W' += S, and U behind it: one wave per row, one entry per lane and step.
template <typename COL>
__global__ __launch_bounds__(256) void k_mx_add_csr(const int32_t* __restrict__ row_ptr,
                                                    const COL* __restrict__ col_idx,
                                                    const uint16_t* __restrict__ vals, int m, int n, int np, int ldw,
                                                    const uint16_t* __restrict__ U, int r, int rp,
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
  put_u(U, row, r, rp, Wr + np);
}

// [src row | zeros] in rows of colsp (a multiple of 8).
__global__ __launch_bounds__(256) void k_mx_pad(const uint16_t* __restrict__ src, int rows, int cols, int colsp,
                                                uint16_t* __restrict__ dst) {
  const uint32_t per = (uint32_t)colsp >> 3, total = (uint32_t)rows * per;
  for (uint32_t q = blockIdx.x * 256u + threadIdx.x; q < total; q += gridDim.x * 256u) {
    const uint32_t row = q / per;
    const int c = (int)(q - row * per) * 8;
    *reinterpret_cast<u32x4*>(dst + (int64_t)row * colsp + c) = load_row8(src + (int64_t)row * cols, c, cols);
  }
}

static void launch_mx_pad(const uint16_t* src, int rows, int cols, int colsp, uint16_t* dst, hipStream_t s) {
  const int64_t total = (int64_t)rows * (colsp >> 3);
  const unsigned grid = (unsigned)std::min<int64_t>((total + 255) / 256, 4096);
  hipLaunchKernelGGL(k_mx_pad, dim3(grid), dim3(256), 0, s, src, rows, cols, colsp, dst);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct MxPlan {
  int np, rp, zt;
  size_t w, x, vt, tp, tb, part, total;
};

// from: the least batch that the workspace is to serve besides b (b's own
// plan, or one of the same 64 columns).
static MxPlan plan_mx(const hss_matrix* A, int b, int from) {
  MxPlan p;
  const int m = A->m, n = A->n, r = A->r;
  p.np = (n + 63) & ~63;
  p.rp = r > 0 ? round32(r) : 0;
  // a block per CU; two cost more in partial products (8192^2, 1024 columns, r
  // 256: 191 us in all against 211)
  p.zt = r > 0 ? mm_splits(r, b, p.np, 256) : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += al256(bytes); return at; };
  p.w = take((size_t)m * (p.np + 2 * p.rp) * 2);
  p.x = take((size_t)b * p.np * 2);
  p.vt = take((size_t)r * p.np * 2);
  p.tp = take((size_t)p.zt * b * p.rp * 4);
  p.tb = take((size_t)b * p.rp * 4);
  p.part = take(std::max(gemm_bf16x2_part_bytes(m, b, p.np, 2 * p.rp, m), gemm256_part_bytes(m, from, b, p.np + 2 * p.rp)));
  p.total = off;
  return p;
}

size_t mx_apply_ws_bytes(const hss_matrix* A, int b) {
  if (mx_skinny_supported(A, b)) return mx_skinny_ws_bytes(A, b);
  return mx_gemm_supported(b) ? mx_gemm_ws_bytes(A, b) : plan_mx(A, b, b).total;
}

// The most that a batch of up to b columns needs: a plan depends on b through
// its count of 16 columns (of 64 beyond the middle route) and grows with b
// among those of one count, but for the K splits of the large products.
size_t mx_apply_ws_bytes_up_to(const hss_matrix* A, int b) {
  size_t most = 0;
  for (int c = 1; c <= b && c < 16; ++c) most = std::max(most, mx_apply_ws_bytes(A, c));
  int c = 16;
  for (; c < b && mx_gemm_supported(c); c += 16) most = std::max(most, mx_apply_ws_bytes(A, c));
  if (c >= b) return std::max(most, mx_apply_ws_bytes(A, b));
  // c is the first multiple of 16 beyond the middle route, whose last batch is a multiple of 64
  for (int from = c - 15; from <= b; from += 64) most = std::max(most, plan_mx(A, std::min(from + 63, b), from).total);
  return most;
}

static bool rows_ok(const void* p, int cols) { return (uintptr_t)p % 16 == 0 && cols % 64 == 0; }

hss_status launch_mx_apply(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s) {
  if (mx_skinny_supported(A, b)) return launch_mx_skinny(A, b, X, Y, ws, s);
  if (mx_gemm_supported(b)) return launch_mx_gemm(A, b, X, Y, ws, s);
  const MxPlan p = plan_mx(A, b, b);
  char* base = static_cast<char*>(ws);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  auto f32 = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  const int m = A->m, n = A->n, r = A->r, np = p.np, rp = p.rp, ldw = np + 2 * rp;
  uint16_t* W = u16(p.w);  // [W' | U | U]
  const dim3 rows4((unsigned)((m + 3) / 4));
  const uint8_t* codes = A->dq_codes;
  const uint8_t* scales = static_cast<const uint8_t*>(A->dq_levels);
  const uint16_t* vals = static_cast<const uint16_t*>(A->values);
  const uint16_t* col16 = reinterpret_cast<const uint16_t*>(A->col_idx);
  const uint16_t* U = static_cast<const uint16_t*>(A->U);
  const bool c16 = (A->flags & HSS_COL16) != 0;
  if (A->flags & HSS_MX4_T) {
    const int tiles_j = (m + kTrJ - 1) / kTrJ;
    hipLaunchKernelGGL(k_mx_densify_t, dim3((unsigned)tiles_j * (unsigned)((np + kTrI - 1) / kTrI)), dim3(256), 0, s,
                       codes, scales, m, n, np, ldw, tiles_j, W);
    if (A->nnz > 0 || r > 0) {
      if (c16)
        hipLaunchKernelGGL(k_mx_add_csr<uint16_t>, rows4, dim3(256), 0, s, A->row_ptr, col16, vals, m, n, np, ldw, U, r,
                           rp, W);
      else
        hipLaunchKernelGGL(k_mx_add_csr<int32_t>, rows4, dim3(256), 0, s, A->row_ptr, A->col_idx, vals, m, n, np, ldw,
                           U, r, rp, W);
    }
  } else {
    const int segs = (np + kMxSeg - 1) / kMxSeg;
    const dim3 grid((unsigned)(((int64_t)m * segs + 3) / 4));
    if (c16)
      hipLaunchKernelGGL(k_mx_densify<uint16_t>, grid, dim3(256), 0, s, codes, scales, A->row_ptr, col16, vals, m, n,
                         np, ldw, U, r, rp, segs, W);
    else
      hipLaunchKernelGGL(k_mx_densify<int32_t>, grid, dim3(256), 0, s, codes, scales, A->row_ptr, A->col_idx, vals, m,
                         n, np, ldw, U, r, rp, segs, W);
  }
  const uint16_t* Xb = static_cast<const uint16_t*>(X);
  if (!rows_ok(X, n)) {
    launch_mx_pad(Xb, b, n, np, u16(p.x), s);
    Xb = u16(p.x);
  }
  if (r > 0) {
    const uint16_t* Vb = static_cast<const uint16_t*>(A->Vt);
    if (!rows_ok(A->Vt, n)) {
      launch_mx_pad(Vb, r, n, np, u16(p.vt), s);
      Vb = u16(p.vt);
    }
    MmProblem q = {};
    q.A = Vb; q.lda = np; q.M = r;
    q.B = Xb; q.ldb = np; q.N = b;
    q.K = np;
    q.C = f32(p.tp); q.ldc = rp; q.trans = 1; q.zstride = (int64_t)b * rp;
    q.splits = p.zt;
    launch_mm_group(&q, 1, false, s);
    launch_mx_tsum(f32(p.tp), p.zt, b, r, rp, u16(p.tb), s);
  }
  // measured against k_gemm_h from 300 columns on: 5 - 20 % faster throughout
  if (gemm256_ok(m, b, np, ldw, np, 2 * rp, 2 * rp))
    launch_gemm256_bf16(m, b, W, ldw, np, Xb, np, 2 * rp, u16(p.tb), 2 * rp, Y, m, f32(p.part), s);
  else
    launch_gemm_bf16x2(m, b, np, W, ldw, Xb, np, 2 * rp, W + np, ldw, u16(p.tb), 2 * rp, Y, m, true, f32(p.part), s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
