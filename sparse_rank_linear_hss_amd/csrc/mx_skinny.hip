// HSS_MX4 apply for up to 16 columns (decode): Y = X (S + U V^T + D)^T straight
// from the 4-bit codes, in one launch (two when there is a low-rank term, or
// an S and more than one column).  Bound by the codes' stream from HBM.
//
// A block owns 16 rows of D.  Its waves split the columns into chunks of 128:
// lane l of a wave reads the 16 bytes of row l % 16, group l / 16 of the chunk
// -- one group, one scale byte -- and decodes them (v_cvt_scalef32, two values
// an instruction) into four A operands of v_mfma_f32_16x16x32_bf16.  The
// product's order along K is free as long as both operands share it: operand t
// holds codes 8 t .. 8 t + 7 of the lane's group, and the B operand of lane l
// the 16 bytes of X[l % 16] at the same columns.  So the codes go from memory
// to the matrix cores without passing through LDS, and one column costs as
// much as sixteen.  Columns past b repeat column b - 1 and are dropped.
//
// U (T1 + T2) runs on the same accumulators, S on the vector units: a wave
// takes a row, its lanes the row's entries.  The waves' partial tiles and S
// meet in LDS and are added in a fixed order.
//
// k_mx_prep makes what the main launch needs of X: T = X V in fp32, K split
// over blocks (the partial sums are added by the reader, in order), and X^T
// for the gathers of S.
#include <algorithm>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

static constexpr int kSkCols = 16;       // columns of one call
static constexpr int kSkBatch = 4;       // chunks whose loads are in flight together
static constexpr int kPrepSplits = 8;    // most K splits of T

// Eight bf16 of a row of n at column k, zeros past the end.
__device__ __forceinline__ u32x4 load_row8(const uint16_t* __restrict__ row, int k, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + 8 <= n) {
    const Bytes16 a = *reinterpret_cast<const Bytes16*>(row + k);
    v = u32x4{a.w[0], a.w[1], a.w[2], a.w[3]};
  } else if (k < n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = k + 2 * e < n ? row[k + 2 * e] : 0u, hi = k + 2 * e + 1 < n ? row[k + 2 * e + 1] : 0u;
      v[e] = lo | hi << 16;
    }
  }
  return v;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Blocks 0 .. tb - 1: 16 rows of V^T over one K split, T partial sums
// Tp[ks][c][rp] (c < b).  Blocks from tb: X^T (n x 16, columns past b zero).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_mx_prep(const uint16_t* __restrict__ X, const uint16_t* __restrict__ Vt, int b,
                                                 int n, int r, int rp, int ltiles, int steps_per_split, int tb,
                                                 float* __restrict__ Tp, uint16_t* __restrict__ Xt) {
  __shared__ float red[4][256];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  if ((int)blockIdx.x >= tb) {
    for (int j = ((int)blockIdx.x - tb) * 256 + t; j < n; j += ((int)gridDim.x - tb) * 256) {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t lo = 2 * k < b ? X[(int64_t)(2 * k) * n + j] : 0u;
        const uint32_t hi = 2 * k + 1 < b ? X[(int64_t)(2 * k + 1) * n + j] : 0u;
        v[k] = lo | hi << 16;
      }
      u32x4* o = reinterpret_cast<u32x4*>(Xt + (int64_t)j * kSkCols);
      o[0] = u32x4{v[0], v[1], v[2], v[3]};
      o[1] = u32x4{v[4], v[5], v[6], v[7]};
    }
    return;
  }
  const int lt = (int)blockIdx.x % ltiles, ks = (int)blockIdx.x / ltiles;
  const int steps = (n + 31) >> 5;
  const int s0 = ks * steps_per_split, s1 = min(s0 + steps_per_split, steps);
  const uint16_t* vrow = Vt + (int64_t)min(16 * lt + (lane & 15), r - 1) * n;
  const uint16_t* xrow = X + (int64_t)min(lane & 15, b - 1) * n;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0 + w; s < s1; s += 16) {
    u32x4 va[4], xa[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = s + 4 * u < s1 ? 32 * (s + 4 * u) + 8 * (lane >> 4) : n;  // n: zeros
      va[u] = load_row8(vrow, k, n);
      xa[u] = load_row8(xrow, k, n);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) acc = mfma16(va[u], xa[u], acc);
  }
  // lane holds rows 4 (lane / 16) + i of column lane % 16
#pragma unroll
  for (int i = 0; i < 4; ++i) red[w][(lane & 15) * 16 + 4 * (lane >> 4) + i] = acc[i];
  __syncthreads();
  const int c = t >> 4, l = 16 * lt + (t & 15);
  if (c < b && l < rp) Tp[((int64_t)ks * b + c) * rp + l] = l < r ? (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]) : 0.f;
}

struct SkinnyArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const int32_t* row_ptr;
  const void* col;
  const uint16_t* vals;
  const uint16_t* X;
  const uint16_t* Xt;  // n x 16, b > 1 and S not empty
  const uint16_t* U;
  const float* Tp;
  uint16_t* Y;
  int m, n, b, r, rp, ng, splits, has_s, col16;
};

// S's part of one row for one column (b == 1): the lanes take its entries.
template <typename COL>
__device__ __forceinline__ float s_row1(const SkinnyArgs& a, const COL* __restrict__ col, int p0, int p1) {
  float s = 0.f;
  for (int p = p0 + lane_id(); p < p1; p += 64) {
    const int j = (int)col[p];
    if ((unsigned)j < (unsigned)a.n) s = fmaf(bf16lo(a.vals[p]), bf16lo(a.X[j]), s);
  }
  return wave_sum(s);
}

// S's part of one row for 16 columns: lane 2 e + h takes entries e, e + 32, ..
// and columns 8 h .. 8 h + 7; the 32 lanes of a half are then added up in a
// fixed tree, in which the lanes first share out the eight columns.  Column
// 8 h + k ends in the lanes with lane % 2 = h and (lane / 2) % 8 = k.
template <typename COL>
__device__ __forceinline__ float s_row16(const SkinnyArgs& a, const COL* __restrict__ col, int p0, int p1) {
  const int lane = lane_id(), h = lane & 1;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = p0 + (lane >> 1); p < p1; p += 32) {
    const int j = (int)col[p];
    if ((unsigned)j >= (unsigned)a.n) continue;
    const float v = bf16lo(a.vals[p]);
    const u32x4 x = *reinterpret_cast<const u32x4*>(a.Xt + (int64_t)j * kSkCols + 8 * h);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s[2 * k] = fmaf(v, bf16lo(x[k]), s[2 * k]);
      s[2 * k + 1] = fmaf(v, bf16hi(x[k]), s[2 * k + 1]);
    }
  }
  // lane bits 1..3 pick the column's bits 0..2
#pragma unroll
  for (int bit = 0; bit < 3; ++bit) {
    const bool up = (lane >> (bit + 1)) & 1;
#pragma unroll
    for (int k = 0; k < (4 >> bit); ++k) {
      const float mine = up ? s[2 * k + 1] : s[2 * k], other = up ? s[2 * k] : s[2 * k + 1];
      s[k] = mine + __shfl_xor(other, 2 << bit, 64);
    }
  }
  s[0] += __shfl_xor(s[0], 16, 64);
  s[0] += __shfl_xor(s[0], 32, 64);
  return s[0];
}

template <int WV>
__global__ __launch_bounds__(64 * WV, 4) void k_mx_skinny(SkinnyArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  float* red = reinterpret_cast<float*>(lds);                       // [WV][16 columns][16 rows]
  float* sred = red + WV * 256;                                     // [16 columns][16 rows]
  uint16_t* Tl = reinterpret_cast<uint16_t*>(sred + 256);           // [b][2][rp + 8]
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int row0 = (int)blockIdx.x * 16;
  const int q = lane >> 4;
  const int nch = (a.ng + 3) >> 2;
  const int64_t grow = (int64_t)min(row0 + (lane & 15), a.m - 1) * a.ng;
  const uint16_t* __restrict__ xrow = a.X + (int64_t)min(lane & 15, a.b - 1) * a.n;

  u32x4 cw[kSkBatch], xv[kSkBatch][4];
  uint32_t sb[kSkBatch];
  // chunk c0 + WV u: past the end, a valid group's codes against zeros of X
  auto issue = [&](int c0) {
#pragma unroll
    for (int u = 0; u < kSkBatch; ++u) {
      const int g = 4 * (c0 + WV * u) + q;
      const int64_t at = grow + min(g, a.ng - 1);
      cw[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.codes + at * 16));
      sb[u] = g < a.ng ? a.scales[at] : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) xv[u][k] = load_row8(xrow, g * 32 + 8 * k, a.n);
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&]() {
#pragma unroll
    for (int u = 0; u < kSkBatch; ++u) {
      const float sc = mx_scale(sb[u], 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u32x4 av = sb[u] ? mx4_to_bf16x8(cw[u][k], sc) : u32x4{0u, 0u, 0u, 0u};
        acc = mfma16(av, xv[u][k], acc);
      }
    }
  };
  if (w < nch) issue(w);

  const int ldt = a.rp + 8;  // rows 16 bytes apart modulo the banks
  if (a.r > 0) {
    for (int e = t; e < a.b * a.rp; e += 64 * WV) {
      float v = 0.f;
      for (int ks = 0; ks < a.splits; ++ks) v += a.Tp[(int64_t)ks * a.b * a.rp + e];
      const int c = e / a.rp, l = e - c * a.rp;
      const uint16_t hi = f32_to_bf16(v);
      // an infinity leaves 0, not the NaN of inf - inf
      const uint16_t lo = (hi & 0x7fffu) == 0x7f80u ? (uint16_t)0 : f32_to_bf16(v - bf16lo(hi));
      Tl[(2 * c) * ldt + l] = hi;
      Tl[(2 * c + 1) * ldt + l] = lo;
    }
  }
  if (a.has_s) {
    for (int i = w; i < 16; i += WV) {
      const int row = row0 + i;
      int p0 = 0, p1 = 0;
      if (row < a.m) p0 = a.row_ptr[row], p1 = a.row_ptr[row + 1];
      if (a.b == 1) {
        const float s = a.col16 ? s_row1(a, static_cast<const uint16_t*>(a.col), p0, p1)
                                : s_row1(a, static_cast<const int32_t*>(a.col), p0, p1);
        if (lane == 0) sred[i] = s;
      } else {
        const float s = a.col16 ? s_row16(a, static_cast<const uint16_t*>(a.col), p0, p1)
                                : s_row16(a, static_cast<const int32_t*>(a.col), p0, p1);
        if (lane < 16) sred[(8 * (lane & 1) + (lane >> 1)) * 16 + i] = s;
      }
    }
  }
  for (int c0 = w; c0 < nch; c0 += WV * kSkBatch) {
    compute();
    if (c0 + WV * kSkBatch < nch) issue(c0 + WV * kSkBatch);
  }
  if (a.r > 0) {
    __syncthreads();
    const uint16_t* __restrict__ urow = a.U + (int64_t)min(row0 + (lane & 15), a.m - 1) * a.r;
    const uint16_t* tl = Tl + 2 * min(lane & 15, a.b - 1) * ldt + 8 * q;
    for (int j = w; j < (a.rp >> 5); j += WV) {
      const u32x4 uv = load_row8(urow, 32 * j + 8 * q, a.r);
      acc = mfma16(uv, *reinterpret_cast<const u32x4*>(tl + 32 * j), acc);
      acc = mfma16(uv, *reinterpret_cast<const u32x4*>(tl + ldt + 32 * j), acc);
    }
  }
  // lane holds rows 4 q + i of column lane % 16
  *reinterpret_cast<f32x4*>(red + w * 256 + (lane & 15) * 16 + 4 * q) = acc;
  __syncthreads();
  if (t < 256) {
    const int c = t >> 4, row = row0 + (t & 15);
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < WV; ++k) y += red[k * 256 + t];
    if (a.has_s) y += sred[t];
    if (c < a.b && row < a.m) a.Y[(int64_t)c * a.m + row] = f32_to_bf16(y);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

struct SkinnyPlan {
  int rp, ltiles, splits, steps_per_split;
  size_t tp, xt, total;
};

static SkinnyPlan plan_skinny(const hss_matrix* A, int b) {
  SkinnyPlan p = {};
  p.rp = A->r > 0 ? round32(A->r) : 0;
  p.ltiles = p.rp / 16;
  const int steps = (A->n + 31) / 32;
  // four waves of up to four steps each per split
  p.splits = std::max(1, std::min(kPrepSplits, (steps + 15) / 16));
  p.steps_per_split = (steps + p.splits - 1) / p.splits;
  p.tp = 0;
  p.xt = al256((size_t)p.splits * b * p.rp * 4);
  p.total = p.xt + ((b > 1 && A->nnz > 0) ? al256((size_t)A->n * kSkCols * 2) : 0);
  return p;
}

// The T terms of one block must fit beside the reduction buffers (64 KiB).
bool mx_skinny_supported(const hss_matrix* A, int b) {
  if ((A->flags & HSS_MX4_T) || b > kSkCols) return false;
  return (size_t)b * 2 * (round32(A->r) + 8) * 2 <= 40 * 1024;
}

size_t mx_skinny_ws_bytes(const hss_matrix* A, int b) { return plan_skinny(A, b).total; }

hss_status launch_mx_skinny(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s) {
  const SkinnyPlan p = plan_skinny(A, b);
  char* base = static_cast<char*>(ws);
  const int m = A->m, n = A->n, r = A->r;
  SkinnyArgs a = {};
  a.codes = A->dq_codes;
  a.scales = static_cast<const uint8_t*>(A->dq_levels);
  a.row_ptr = A->row_ptr;
  a.col = A->col_idx;
  a.vals = static_cast<const uint16_t*>(A->values);
  a.X = static_cast<const uint16_t*>(X);
  a.Xt = reinterpret_cast<const uint16_t*>(base + p.xt);
  a.U = static_cast<const uint16_t*>(A->U);
  a.Tp = reinterpret_cast<const float*>(base + p.tp);
  a.Y = static_cast<uint16_t*>(Y);
  a.m = m; a.n = n; a.b = b; a.r = r; a.rp = p.rp;
  a.ng = mx_groups(n);
  a.splits = p.splits;
  a.has_s = A->nnz > 0;
  a.col16 = (A->flags & HSS_COL16) != 0;
  const bool need_xt = a.has_s && b > 1;
  const int tb = r > 0 ? p.ltiles * p.splits : 0;
  const int xb = need_xt ? std::min((n + 255) / 256, 256) : 0;
  if (tb + xb > 0)
    hipLaunchKernelGGL(k_mx_prep, dim3((unsigned)(tb + xb)), dim3(256), 0, s, a.X,
                       static_cast<const uint16_t*>(A->Vt), b, n, r, p.rp, std::max(p.ltiles, 1), p.steps_per_split,
                       tb, reinterpret_cast<float*>(base + p.tp), reinterpret_cast<uint16_t*>(base + p.xt));
  const unsigned grid = (unsigned)((m + 15) / 16);
  const size_t tl = r > 0 ? (size_t)b * 2 * (p.rp + 8) * 2 : 0;
  const int nch = (a.ng + 3) / 4;
  // Waves per block: enough to hold a row tile's codes in flight, fewer when
  // the blocks fill the chip anyway.
  if (nch <= 4 * kSkBatch || grid > 512)
    hipLaunchKernelGGL(k_mx_skinny<4>, dim3(grid), dim3(256), 5 * 1024 + tl, s, a);
  else if (nch <= 8 * kSkBatch)
    hipLaunchKernelGGL(k_mx_skinny<8>, dim3(grid), dim3(512), 9 * 1024 + tl, s, a);
  else
    hipLaunchKernelGGL(k_mx_skinny<16>, dim3(grid), dim3(1024), 17 * 1024 + tl, s, a);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
