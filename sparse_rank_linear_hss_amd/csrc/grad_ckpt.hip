// Parameter gradients from an 8-bit checkpoint of the layer's input
// (hss_grad_ckpt).  With X' the values the checkpoint stands for (exact in
// bf16: a code has 7 bits, its scale is a power of two):
//
//   dS_p = sum_c G[c][i_p] X'[c][j_p]      as hss_grad, from X'
//   dU   = G^T T,  T = X' V
//   dV^T = P^T X', P = G U
//
// T and P are sums of n (m) products held in fp32.  The matrix cores take
// bf16, so each is split into three bf16 terms (24 significant bits) and the
// products with G and X' are summed over the terms: the gradients are as
// exact as fp32 products would be.
#include <algorithm>

#include "mx_common.h"

namespace hss {

void launch_gemm_bf16x2(int M, int N, int K1, const uint16_t* A1, int64_t lda1, const uint16_t* B1, int64_t ldb1,
                        int K2, const uint16_t* A2, int64_t lda2, const uint16_t* B2, int64_t ldb2, void* C,
                        int64_t ldc, bool out_bf16, float* part, hipStream_t s);
size_t gemm_bf16x2_part_bytes(int M, int N, int K1, int K2, int64_t ldc);
void launch_mx_pad(const uint16_t* src, int rows, int cols, int colsp, int rep, uint16_t* dst, hipStream_t s);
void launch_mx_terms(const float* T, int rows, int cols, int64_t ld, int colsp, int terms, uint16_t* dst,
                     hipStream_t s);
void launch_ds(const hss_matrix* A, int b, int kb, int ldt, const uint16_t* Xt, const uint16_t* Gt, float* dA,
               float* part, float* dS, hipStream_t s);
bool ds_dense(int b);

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

// ---------------------------------------------------------------------------
// dst (cols x ldt) = src (rows x cols)^T in bf16, zero for rows <= c < ldt
// (ldt a multiple of 32), and a row-major copy with rows padded to colsp
// (zero past cols; null = none).  64 x 64 tiles through LDS; thread t holds
// 16 columns of tile row t / 4.  CKPT: src is an int8 checkpoint.
// ---------------------------------------------------------------------------
template <bool CKPT>
__global__ __launch_bounds__(256) void k_ck_transpose(const void* __restrict__ src, const uint8_t* __restrict__ scales,
                                                      int rows, int cols, int ldt, uint16_t* __restrict__ dst,
                                                      uint16_t* __restrict__ copy, int colsp, int tiles_c) {
  __shared__ __align__(16) uint16_t tile[64][64 + 8];
  const int r0 = (int)(blockIdx.x / (unsigned)tiles_c) * 64, c0 = (int)(blockIdx.x % (unsigned)tiles_c) * 64;
  const int t = threadIdx.x;
  const int row = r0 + (t >> 2), col = c0 + 16 * (t & 3);
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};  // 16 bf16
  if (row < rows && col < cols) {
    if constexpr (CKPT) {
      const int64_t g = (int64_t)row * mx_groups(cols) + (col >> 5);
      const u32x4 code = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(src) + g * 32 + (col & 16));
      const float scale = mx_scale(scales[g], 6);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4];
        mx8_to_f32x4(code[k], scale, v);
        w[2 * k] = mx_pack_hi(v[0], v[1]);
        w[2 * k + 1] = mx_pack_hi(v[2], v[3]);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(src) + (int64_t)row * cols + col;
      if (col + 16 <= cols) {
        const Bytes16 a = reinterpret_cast<const Bytes16*>(p)[0], b = reinterpret_cast<const Bytes16*>(p)[1];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = a.w[k], w[4 + k] = b.w[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t lo = col + 2 * k < cols ? p[2 * k] : 0u, hi = col + 2 * k + 1 < cols ? p[2 * k + 1] : 0u;
          w[k] = lo | hi << 16;
        }
      }
    }
  }
  if (copy && row < rows && col < colsp) {
    u32x4* o = reinterpret_cast<u32x4*>(copy + (int64_t)row * colsp + col);
    o[0] = u32x4{w[0], w[1], w[2], w[3]};
    o[1] = u32x4{w[4], w[5], w[6], w[7]};
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    tile[16 * (t & 3) + 2 * k][t >> 2] = (uint16_t)w[k];
    tile[16 * (t & 3) + 2 * k + 1][t >> 2] = (uint16_t)(w[k] >> 16);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int q = t + 256 * h, j = q >> 3, c = (q & 7) * 8;
    if (c0 + j < cols && r0 + c < ldt)
      *reinterpret_cast<u32x4*>(dst + (int64_t)(c0 + j) * ldt + r0 + c) = *reinterpret_cast<const u32x4*>(&tile[j][c]);
  }
}

static void launch_ck_transpose(bool ckpt, const void* src, const uint8_t* scales, int rows, int cols, int ldt,
                                uint16_t* dst, uint16_t* copy, int colsp, hipStream_t s) {
  // the grid covers the padded columns too when a copy is written
  const int tiles_c = (std::max(cols, copy ? colsp : 0) + 63) / 64;
  const dim3 grid((unsigned)tiles_c * (unsigned)((ldt + 63) / 64));
  if (ckpt)
    hipLaunchKernelGGL(k_ck_transpose<true>, grid, dim3(256), 0, s, src, scales, rows, cols, ldt, dst, copy, colsp,
                       tiles_c);
  else
    hipLaunchKernelGGL(k_ck_transpose<false>, grid, dim3(256), 0, s, src, scales, rows, cols, ldt, dst, copy, colsp,
                       tiles_c);
}

// out[k] = a[k] + b[k]
__global__ __launch_bounds__(256) void k_ck_add(const float* __restrict__ a, const float* __restrict__ b, int64_t count,
                                                float* __restrict__ out) {
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < count; k += (int64_t)gridDim.x * 256)
    out[k] = a[k] + b[k];
}

// ---------------------------------------------------------------------------
// Workspace
// ---------------------------------------------------------------------------
struct CkPlan {
  int ldt, np, mp;
  size_t xb, xt, gt, gb, vt, ut, tf, t3, s0, s1, da, part, total;
};

static CkPlan plan_ck(const hss_matrix* A, int b) {
  CkPlan p;
  const int m = A->m, n = A->n, r = A->r;
  p.ldt = round32(b);
  p.np = round32(n);
  p.mp = round32(m);
  size_t off = 0;
  p.xb = off; off += al256((size_t)b * p.np * 2);
  p.xt = off; off += al256((size_t)n * p.ldt * 2);
  p.gt = off; off += al256((size_t)m * p.ldt * 2);
  p.gb = off; off += al256((size_t)b * p.mp * 2);
  p.vt = off; off += al256((size_t)r * p.np * 2);
  p.ut = off; off += al256((size_t)r * p.mp * 2);
  p.tf = off; off += al256((size_t)r * p.ldt * 4);
  p.t3 = off; off += al256((size_t)r * p.ldt * 6);
  p.s0 = off; off += al256((size_t)r * std::max(m, n) * 4);
  p.s1 = off; off += al256((size_t)r * std::max(m, n) * 4);
  p.da = off; off += ds_dense(b) ? al256((size_t)m * n * 4) : 0;
  size_t part = 0;
  if (r > 0) {
    part = std::max(part, gemm_bf16x2_part_bytes(b, r, p.np, 0, p.ldt));
    part = std::max(part, gemm_bf16x2_part_bytes(b, r, p.mp, 0, p.ldt));
    for (int k2 = 0; k2 <= p.ldt; k2 += p.ldt) {
      part = std::max(part, gemm_bf16x2_part_bytes(r, m, p.ldt, k2, r));
      part = std::max(part, gemm_bf16x2_part_bytes(n, r, p.ldt, k2, n));
    }
  }
  if (ds_dense(b)) part = std::max(part, gemm_bf16x2_part_bytes(n, m, p.ldt, 0, n));
  p.part = off; off += al256(part);
  p.total = off;
  return p;
}

size_t grad_ckpt_ws_bytes(const hss_matrix* A, int b) { return plan_ck(A, b).total; }

static bool rows_ok(const void* p, int cols) { return (uintptr_t)p % 16 == 0 && cols % 32 == 0; }

hss_status launch_grad_ckpt(const hss_matrix* A, int b, const void* codes, const uint8_t* scales, const void* G,
                            float* dS, float* dU, float* dVt, void* ws, hipStream_t s) {
  const CkPlan p = plan_ck(A, b);
  char* base = static_cast<char*>(ws);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  uint16_t *Xb = u16(p.xb), *Xt = u16(p.xt), *Gt = u16(p.gt), *T3 = u16(p.t3);
  float* Tf = reinterpret_cast<float*>(base + p.tf);
  float* part = reinterpret_cast<float*>(base + p.part);
  float* S0 = reinterpret_cast<float*>(base + p.s0);
  float* S1 = reinterpret_cast<float*>(base + p.s1);
  const int m = A->m, n = A->n, r = A->r, ldt = p.ldt;
  const int64_t stored = A->fmt == HSS_FMT_2OF4 ? (int64_t)m * (n / 2) : A->nnz;
  const bool want_s = dS && stored > 0, want_u = dU && r > 0, want_v = dVt && r > 0;
  if (!want_s && !want_u && !want_v) return HSS_OK;
  launch_ck_transpose(true, codes, scales, b, n, ldt, Xt, want_u ? Xb : nullptr, p.np, s);
  const uint16_t* Gb = static_cast<const uint16_t*>(G);
  const bool copy_g = want_v && !rows_ok(G, m);
  if (want_u || want_s || copy_g)
    launch_ck_transpose(false, G, nullptr, b, m, ldt, Gt, copy_g ? u16(p.gb) : nullptr, p.mp, s);
  if (copy_g) Gb = u16(p.gb);
  // C[n * ldc + m] over the three terms of T3, in a fixed order: (t1 + t2) + t3
  auto sum3 = [&](int M, int N, const uint16_t* A3, bool a_terms, const uint16_t* B3, float* out, int ldc) {
    const int la = a_terms ? 3 * ldt : ldt, lb = a_terms ? ldt : 3 * ldt;
    const int oa = a_terms ? ldt : 0, ob = a_terms ? 0 : ldt;
    launch_gemm_bf16x2(M, N, ldt, A3, la, B3, lb, ldt, A3 + oa, la, B3 + ob, lb, S0, ldc, false, part, s);
    launch_gemm_bf16x2(M, N, ldt, A3 + 2 * oa, la, B3 + 2 * ob, lb, 0, nullptr, 0, nullptr, 0, S1, ldc, false, part, s);
    const int64_t count = (int64_t)N * ldc;
    hipLaunchKernelGGL(k_ck_add, dim3((unsigned)std::min<int64_t>((count + 255) / 256, 4096)), dim3(256), 0, s, S0, S1,
                       count, out);
  };
  if (want_u) {
    const uint16_t* Vb = static_cast<const uint16_t*>(A->Vt);
    if (!rows_ok(A->Vt, n)) {
      launch_mx_pad(Vb, r, n, p.np, 1, u16(p.vt), s);
      Vb = u16(p.vt);
    }
    launch_gemm_bf16x2(b, r, p.np, Xb, p.np, Vb, p.np, 0, nullptr, 0, nullptr, 0, Tf, ldt, false, part, s);
    launch_mx_terms(Tf, r, b, ldt, ldt, 3, T3, s);
    sum3(r, m, T3, true, Gt, dU, r);
  }
  if (want_v) {
    uint16_t* Ut = u16(p.ut);
    launch_ck_transpose(false, A->U, nullptr, m, r, p.mp, Ut, nullptr, 0, s);
    launch_gemm_bf16x2(b, r, p.mp, Gb, p.mp, Ut, p.mp, 0, nullptr, 0, nullptr, 0, Tf, ldt, false, part, s);
    launch_mx_terms(Tf, r, b, ldt, ldt, 3, T3, s);
    sum3(n, r, Xt, false, T3, dVt, n);
  }
  if (want_s) launch_ds(A, b, ldt, ldt, Xt, Gt, reinterpret_cast<float*>(base + p.da), part, dS, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
