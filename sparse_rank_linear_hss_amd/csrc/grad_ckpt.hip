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
// products with G and X' are summed over the terms: the gradients are as exact
// as fp32 products would be.
//
// Launches: k_ck_prep (X'^T, G^T, U^T and padded rows where a product needs
// them), one grouped product for T^T and P^T with K split, k_ck_terms (the
// splits' sums, as terms), one grouped product for dU and dV^T (with a sum
// where K is split), and dS: sampled products, or dense tiles of
// G^T X' of which only S's entries leave the chip (gemm256.hip).
#include <algorithm>

#include "gemm256.h"
#include "mm_group.h"
#include "mx_common.h"

namespace hss {

// grad.hip
void launch_sddmm(const hss_matrix* A, int ldt, const uint16_t* Xt, const uint16_t* Gt, float* dS, hipStream_t s);

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

// ---------------------------------------------------------------------------
// A task turns src (rows x cols, bf16 or an int8 checkpoint) into bf16
//   dst  (cols x ldt) = src^T, zero for rows <= c < ldt; null = none
//   copy (rows x colsp), src with rows padded by zeros;  null = none
// (ldt and colsp multiples of 32).  64 x 64 tiles through LDS; thread t holds
// 16 columns of tile row t / 4.  Up to four tasks share a launch.
// ---------------------------------------------------------------------------
struct CkTask {
  const void* src;
  const uint8_t* scales;  // of a checkpoint; null: src is bf16
  uint16_t* dst;
  uint16_t* copy;
  int rows, cols, ldt, colsp, tiles_c, blocks;
};
struct CkTasks {
  CkTask t[4];
  int count;
};

__global__ __launch_bounds__(256) void k_ck_prep(CkTasks tasks) {
  __shared__ __align__(16) uint16_t tile[64][64 + 8];
  int block = (int)blockIdx.x, which = 0;
  while (which + 1 < tasks.count && block >= tasks.t[which].blocks) block -= tasks.t[which++].blocks;
  const CkTask& k_ = tasks.t[which];
  const int rows = k_.rows, cols = k_.cols;
  const int r0 = block / k_.tiles_c * 64, c0 = block % k_.tiles_c * 64;
  const int t = threadIdx.x;
  const int row = r0 + (t >> 2), col = c0 + 16 * (t & 3);
  uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};  // 16 bf16
  if (row < rows && col < cols) {
    if (k_.scales) {
      const int64_t g = (int64_t)row * mx_groups(cols) + (col >> 5);
      const u32x4 code = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(k_.src) + g * 32 + (col & 16));
      const float scale = mx_scale(k_.scales[g], 6);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4];
        mx8_to_f32x4(code[k], scale, v);
        w[2 * k] = mx_pack_hi(v[0], v[1]);
        w[2 * k + 1] = mx_pack_hi(v[2], v[3]);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(k_.src) + (int64_t)row * cols + col;
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
  if (k_.copy && row < rows && col < k_.colsp) {
    u32x4* o = reinterpret_cast<u32x4*>(k_.copy + (int64_t)row * k_.colsp + col);
    o[0] = u32x4{w[0], w[1], w[2], w[3]};
    o[1] = u32x4{w[4], w[5], w[6], w[7]};
  }
  if (!k_.dst) return;  // the same for the whole block
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    tile[16 * (t & 3) + 2 * k][t >> 2] = (uint16_t)w[k];
    tile[16 * (t & 3) + 2 * k + 1][t >> 2] = (uint16_t)(w[k] >> 16);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int q = t + 256 * h, j = q >> 3, c = (q & 7) * 8;
    if (c0 + j < cols && r0 + c < k_.ldt)
      *reinterpret_cast<u32x4*>(k_.dst + (int64_t)(c0 + j) * k_.ldt + r0 + c) = *reinterpret_cast<const u32x4*>(&tile[j][c]);
  }
}

static void add_task(CkTasks& ts, const void* src, const uint8_t* scales, int rows, int cols, uint16_t* dst, int ldt,
                     uint16_t* copy, int colsp) {
  CkTask t = {src, scales, dst, copy, rows, cols, ldt, colsp, 0, 0};
  t.tiles_c = (std::max(cols, copy ? colsp : 0) + 63) / 64;
  t.blocks = t.tiles_c * ((std::max(rows, dst ? ldt : 0) + 63) / 64);
  ts.t[ts.count++] = t;
}

// ---------------------------------------------------------------------------
// Terms of T^T and P^T: dst[l][z][ldt], z < 3, from the sum of the splits'
// partial products [split][l][ldt]; zero for c >= b.  Term z is what the terms
// before it leave, rounded to nearest.
// ---------------------------------------------------------------------------
struct CkTerms {
  const float* src[2];
  uint16_t* dst[2];
  int splits[2];
  int count, r, b, ldt;
};

__global__ __launch_bounds__(256) void k_ck_terms(CkTerms a) {
  const uint32_t per = (uint32_t)a.ldt >> 2, total = (uint32_t)a.r * per;
  for (uint32_t e = blockIdx.x * 256u + threadIdx.x; e < total * (uint32_t)a.count; e += gridDim.x * 256u) {
    const int which = e >= total;
    const uint32_t q = e - (which ? total : 0u);
    const uint32_t l = q / per, c = (q - l * per) * 4;
    const float* src = a.src[which] + (int64_t)l * a.ldt + c;
    const int64_t zs = (int64_t)a.r * a.ldt;
    float4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int z = 0; z < a.splits[which]; ++z) {
      const float4 v = *reinterpret_cast<const float4*>(src + z * zs);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (int)c + k < a.b ? v[k] : 0.f;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = f32_to_bf16(v[k]);
        // (an infinity leaves 0, not the NaN of inf - inf)
        v[k] = (h[k] & 0x7fffu) == 0x7f80u ? 0.f : v[k] - __uint_as_float(h[k] << 16);
      }
      *reinterpret_cast<mx_u32x2*>(a.dst[which] + ((int64_t)l * 3 + z) * a.ldt + c) =
          mx_u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
    }
  }
}

// dst[e] = the splits' partial products of it, added in order.
struct CkSum {
  const float* src[2];
  float* dst[2];
  int64_t size[2];
  int splits[2];
  int count;
};

__global__ __launch_bounds__(256) void k_ck_sum(CkSum a) {
  const int64_t total = a.size[0] + a.size[1];
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int which = e >= a.size[0];
    const int64_t q = which ? e - a.size[0] : e;
    float v = 0.f;
#pragma unroll 4
    for (int z = 0; z < a.splits[which]; ++z) v += a.src[which][z * a.size[which] + q];
    a.dst[which][q] = v;
  }
}

// ---------------------------------------------------------------------------
// Workspace
// ---------------------------------------------------------------------------
struct CkPlan {
  bool dense;  // dense_ds()
  int ldt, np, mp, zt, zp, zo;  // padded sizes; K splits of T, of P and of dU and dV
  size_t xb, xt, gt, gb, vt, ut, tf, pf, t3, p3, o, tptr, total;
};

// dS by dense tiles of G^T X' (k_gemm256) or by sampled products (k_sddmm):
// the less of the two estimates, in us, unless HSS_OPT_GRAD_DS_ROUTE forces
// one.  Both were fitted to sampled / dense measurements: 8192^2 3 % of S, 128
// tokens 47 / 61, 256 90 / 72, 512 175 / 97, 1024 444 / 147; 4096^2 3 %, 128
// 20 / 21, 512 70 / 35; 4096^2 0.5 %, 512 26 / 32, 1024 32 / 43.
static bool dense_ds(const hss_matrix* A, int b) {
  const int forced = option(HSS_OPT_GRAD_DS_ROUTE);
  if (forced) return forced == 2;
  const double stored = A->fmt == HSS_FMT_2OF4 ? 0.5 * A->m * A->n : (double)A->nnz;
  const int64_t tiles = (int64_t)((A->m + 255) / 256) * ((A->n + 255) / 256);
  return 8 + 0.17e-6 * stored * b > 10 + (double)((tiles + 255) / 256) * (0.0225 * b + 10);
}

static constexpr int kCkBlocks = 256;  // blocks of the T and P launch

// K splits of the products for dU and dV^T (one launch): enough for two blocks
// per CU (8192^2, 2048 tokens, r 128, us for all gradients: 338; for one block
// 346; unsplit 368), where K is long enough for the sum of the partial products
// to pay.
static int uv_splits(int r, int m, int n, int ldt) {
  const int tiles = (r + 127) / 128 * ((m + 127) / 128 + (n + 127) / 128);
  return std::max(1, std::min((511 + tiles) / tiles, ldt / 512));
}

static CkPlan plan_ck(const hss_matrix* A, int b, bool dense) {
  CkPlan p;
  const int m = A->m, n = A->n, r = A->r;
  p.dense = dense;
  p.ldt = p.dense ? (b + 63) & ~63 : round32(b);  // whole stages of k_gemm256
  p.np = round32(n);
  p.mp = round32(m);
  p.zt = r > 0 ? mm_splits(r, b, p.np, kCkBlocks / 2) : 0;
  p.zp = r > 0 ? mm_splits(r, b, p.mp, kCkBlocks / 2) : 0;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += al256(bytes); return at; };
  p.xb = take((size_t)b * p.np * 2);
  p.xt = take((size_t)n * p.ldt * 2);
  p.gt = take((size_t)m * p.ldt * 2);
  p.gb = take((size_t)b * p.mp * 2);
  p.vt = take((size_t)r * p.np * 2);
  p.ut = take((size_t)r * p.mp * 2);
  p.tf = take((size_t)p.zt * r * p.ldt * 4);
  p.pf = take((size_t)p.zp * r * p.ldt * 4);
  p.t3 = take((size_t)r * p.ldt * 6);
  p.p3 = take((size_t)r * p.ldt * 6);
  p.zo = r > 0 ? uv_splits(r, m, n, p.ldt) : 1;
  p.o = take(p.zo > 1 ? (size_t)p.zo * r * (m + n) * 4 : 0);
  p.tptr = take(p.dense ? gemm256_ds_bytes(A) : 0);
  p.total = off;
  return p;
}

size_t grad_ckpt_ws_bytes(const hss_matrix* A, int b) { return plan_ck(A, b, dense_ds(A, b)).total; }

// The most that a batch of up to b columns needs, on either route of dS: the
// dense one has the longer rows and a table more; its plan depends on b through
// its count of 64 columns, and grows with b among those of one count.
size_t grad_ckpt_ws_bytes_up_to(const hss_matrix* A, int b) {
  size_t most = plan_ck(A, b, true).total;
  for (int c = 64; c < b; c += 64) most = std::max(most, plan_ck(A, c, true).total);
  return most;
}

static bool rows_ok(const void* p, int cols) { return (uintptr_t)p % 16 == 0 && cols % 32 == 0; }

hss_status launch_grad_ckpt(const hss_matrix* A, int b, const void* codes, const uint8_t* scales, const void* G,
                            float* dS, float* dU, float* dVt, void* ws, hipStream_t s) {
  const CkPlan p = plan_ck(A, b, dense_ds(A, b));
  char* base = static_cast<char*>(ws);
  auto u16 = [&](size_t off) { return reinterpret_cast<uint16_t*>(base + off); };
  auto f32 = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  const int m = A->m, n = A->n, r = A->r, ldt = p.ldt;
  const int64_t stored = A->fmt == HSS_FMT_2OF4 ? (int64_t)m * (n / 2) : A->nnz;
  const bool want_s = dS && stored > 0, want_u = dU && r > 0, want_v = dVt && r > 0;
  if (!want_s && !want_u && !want_v) return HSS_OK;

  CkTasks ts = {};
  const bool want_xt = want_v || want_s, want_gt = want_u || want_s;
  add_task(ts, codes, scales, b, n, want_xt ? u16(p.xt) : nullptr, ldt, want_u ? u16(p.xb) : nullptr, p.np);
  const bool copy_g = want_v && !rows_ok(G, m), copy_v = want_u && !rows_ok(A->Vt, n);
  if (want_gt || copy_g)
    add_task(ts, G, nullptr, b, m, want_gt ? u16(p.gt) : nullptr, ldt, copy_g ? u16(p.gb) : nullptr, p.mp);
  if (want_v) add_task(ts, A->U, nullptr, m, r, u16(p.ut), p.mp, nullptr, 0);
  if (copy_v) add_task(ts, A->Vt, nullptr, r, n, nullptr, 0, u16(p.vt), p.np);
  unsigned blocks = 0;
  for (int k = 0; k < ts.count; ++k) blocks += (unsigned)ts.t[k].blocks;
  hipLaunchKernelGGL(k_ck_prep, dim3(blocks), dim3(256), 0, s, ts);

  if (want_u || want_v) {
    MmProblem q[2] = {};
    CkTerms t = {};
    t.r = r; t.b = b; t.ldt = ldt;
    int k = 0;
    auto product = [&](const uint16_t* a_rows, const uint16_t* b_rows, int K, int splits, size_t out, size_t terms) {
      q[k].A = a_rows; q[k].lda = K; q[k].M = r;
      q[k].B = b_rows; q[k].ldb = K; q[k].N = b;
      q[k].K = K;
      q[k].C = f32(out); q[k].ldc = ldt; q[k].zstride = (int64_t)r * ldt;
      q[k].splits = splits;
      t.src[k] = f32(out); t.dst[k] = u16(terms); t.splits[k] = splits;
      t.count = ++k;
    };
    if (want_u) product(copy_v ? u16(p.vt) : static_cast<const uint16_t*>(A->Vt), u16(p.xb), p.np, p.zt, p.tf, p.t3);
    if (want_v) product(u16(p.ut), copy_g ? u16(p.gb) : static_cast<const uint16_t*>(G), p.mp, p.zp, p.pf, p.p3);
    launch_mm_group(q, k, false, s);
    const int64_t work = (int64_t)t.count * r * (ldt / 4);
    hipLaunchKernelGGL(k_ck_terms, dim3((unsigned)std::min<int64_t>((work + 255) / 256, 4096)), dim3(256), 0, s, t);
    MmProblem o[2] = {};
    CkSum sum = {};
    k = 0;
    size_t at = p.o;
    auto gradient = [&](size_t terms, size_t rows, int count, float* out, int64_t ldc, int trans) {
      const int64_t size = (int64_t)r * count;
      o[k].A = u16(terms); o[k].lda = 3 * ldt; o[k].M = r;
      o[k].B = u16(rows); o[k].ldb = ldt; o[k].N = count; o[k].K = ldt;
      o[k].C = p.zo > 1 ? f32(at) : out; o[k].ldc = ldc; o[k].trans = trans;
      o[k].splits = p.zo; o[k].zstride = size;
      sum.src[k] = f32(at); sum.dst[k] = out; sum.size[k] = size; sum.splits[k] = mm_actual_splits(ldt, p.zo);
      sum.count = ++k;
      at += (size_t)p.zo * size * 4;
    };
    if (want_u) gradient(p.t3, p.gt, m, dU, r, 1);
    if (want_v) gradient(p.p3, p.xt, n, dVt, n, 0);
    launch_mm_group(o, k, true, s);
    if (p.zo > 1)
      hipLaunchKernelGGL(k_ck_sum, dim3((unsigned)std::min<int64_t>((sum.size[0] + sum.size[1] + 255) / 256, 4096)),
                         dim3(256), 0, s, sum);
  }
  if (want_s) {
    if (p.dense)
      launch_gemm256_ds(A, ldt, u16(p.gt), u16(p.xt), ldt, dS, reinterpret_cast<int32_t*>(base + p.tptr), s);
    else
      launch_sddmm(A, ldt, u16(p.xt), u16(p.gt), dS, s);
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
