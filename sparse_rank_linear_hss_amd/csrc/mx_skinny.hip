// HSS_MX4 apply for up to 16 columns (decode): Y = X (S + U V^T + D)^T straight
// from the 4-bit codes, in one launch (two when there is a low-rank term, an S
// and more than four columns, or X's rows are long or off the 16-byte grid).
// Bound by the codes' stream from HBM.  Up to four columns: k_mx_gemv, on the vector units, below.
// From five on: k_mx_skinny, on the matrix cores.
//
// k_mx_skinny: a block owns 16 rows of D.  Its waves split the columns into chunks of 128:
// lane l of a wave reads the 16 bytes of row l % 16, group l / 16 of the chunk
// -- one group, one scale byte -- and decodes them (v_cvt_scalef32, two values
// an instruction) into four A operands of v_mfma_f32_16x16x32_bf16.  The
// product's order along K is free as long as both operands share it: operand t
// holds codes 8 t .. 8 t + 7 of the lane's group, and the B operand of lane l
// the 16 bytes of X[l % 16] at the same columns, from X's rows or from a copy
// of X in just that order.  So the codes go from memory
// to the matrix cores without passing through LDS, and one column costs as
// much as sixteen.  Columns past b repeat column b - 1 and are dropped.
//
// U (T1 + T2) runs on the same accumulators, S on the vector units: a wave
// takes a row, its lanes the row's entries.  The waves' partial tiles and S
// meet in LDS and are added in a fixed order.
//
// k_mx_prep makes what the main launch needs of X: T = X V in fp32, K split
// over blocks (the partial sums are added by the reader, in order), X^T for
// the gathers of S, and X in operand order.
#include <algorithm>
#include <type_traits>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

static constexpr int kSkCols = 16;       // columns of one call
static constexpr int kSkGather = 4;      // columns up to which S gathers from X, not X^T
static constexpr int kSkBatch = 6;       // most chunks of a wave whose loads are in flight together

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// What a launch needs of X.  Blocks 0 .. tb - 1: 16 rows of V^T times 16
// columns over one K split, T partial sums Tp[ks][c][rp] (c < b).  Blocks from
// tb: X^T (n x ldt, zero past b), X with rows of np (zero past n) and U with
// rows of rp, each where its pointer is not null.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_mx_prep(MxPrep a) {
  __shared__ float red[4][256];
  const uint16_t* __restrict__ X = a.X;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, b = a.b, n = a.n;
  if ((int)blockIdx.x >= a.tb) {
    // item counts are below 2^28 and a step below 2^18: no wrap
    const uint32_t first = (blockIdx.x - (uint32_t)a.tb) * 256u + t, step = (uint32_t)a.xb * 256u;
    const uint32_t per = (uint32_t)a.np >> 3, peru = (uint32_t)a.rp >> 3;
    for (uint32_t e = first; a.Xp && e < (uint32_t)b * per; e += step) {
      const int c = (int)(e / per), k = (int)(e - (uint32_t)c * per) * 8;
      *reinterpret_cast<u32x4*>(a.Xp + (int64_t)c * a.np + k) = load_row8(X + (int64_t)c * n, k, n);
    }
    // X in k_mx_skinny's operand order: piece 256 c + 64 k + l holds, for row l %
    // 16, columns 128 c + 32 (l / 16) + 8 k ..
    for (uint32_t e = first; a.Xo && e < (uint32_t)a.nch * 256u; e += step) {
      const int l = (int)(e & 63u), k = 128 * (int)(e >> 8) + 32 * (l >> 4) + 8 * (int)((e >> 6) & 3u);
      *reinterpret_cast<u32x4*>(a.Xo + (int64_t)e * 8) = load_row8(X + (int64_t)min(l & 15, b - 1) * n, k, n);
    }
    for (uint32_t e = first; a.Up && e < (uint32_t)a.m * peru; e += step) {
      const int i = (int)(e / peru), l = (int)(e - (uint32_t)i * peru) * 8;
      *reinterpret_cast<u32x4*>(a.Up + (int64_t)i * a.rp + l) = load_row8(a.U + (int64_t)i * a.r, l, a.r);
    }
    for (uint32_t e = first; a.Xt && e < (uint32_t)n * (uint32_t)(a.ldt >> 3); e += step) {
      const int c0 = (int)(e / (uint32_t)n) * 8, j = (int)(e - (uint32_t)(c0 >> 3) * (uint32_t)n);
      u32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = c0 + 2 * k < b ? X[(int64_t)(c0 + 2 * k) * n + j] : 0u;
        const uint32_t hi = c0 + 2 * k + 1 < b ? X[(int64_t)(c0 + 2 * k + 1) * n + j] : 0u;
        v[k] = lo | hi << 16;
      }
      *reinterpret_cast<u32x4*>(a.Xt + (int64_t)j * a.ldt + c0) = v;
    }
    return;
  }
  const int lt = (int)blockIdx.x % a.ltiles, rest = (int)blockIdx.x / a.ltiles;
  const int ks = rest % a.splits, c0 = rest / a.splits * 16;
  const int steps = (n + 31) >> 5, full = n >> 5;
  const int s0 = ks * a.steps_per_split, s1 = min(s0 + a.steps_per_split, steps), f1 = min(s1, full);
  const uint16_t* vrow = a.Vt + (int64_t)min(16 * lt + (lane & 15), a.r - 1) * n;
  const uint16_t* xrow = X + (int64_t)min(c0 + (lane & 15), b - 1) * n;
  const int k0 = 8 * (lane >> 4);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0 + w; s < f1; s += 16) {  // whole steps; past the last one that one again, not used
    u32x4 va[4], xa[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = 32 * min(s + 4 * u, f1 - 1) + k0;
      va[u] = load8(vrow + k);
      xa[u] = load8(xrow + k);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s + 4 * u < f1) acc = mfma16(va[u], xa[u], acc);
  }
  if (s1 > f1 && w == 0) acc = mfma16(load_row8(vrow, 32 * f1 + k0, n), load_row8(xrow, 32 * f1 + k0, n), acc);
  // lane holds rows 4 (lane / 16) + i of column lane % 16
#pragma unroll
  for (int i = 0; i < 4; ++i) red[w][(lane & 15) * 16 + 4 * (lane >> 4) + i] = acc[i];
  __syncthreads();
  const int c = c0 + (t >> 4), l = 16 * lt + (t & 15);
  if (c < b && l < a.rp)
    a.Tp[((int64_t)ks * b + c) * a.rp + l] = l < a.r ? (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]) : 0.f;
}

MxPrep mx_prep_plan(const hss_matrix* A, int b) {
  MxPrep p = {};
  p.m = A->m; p.b = b; p.n = A->n; p.r = A->r;
  p.rp = A->r > 0 ? (A->r + 31) & ~31 : 0;
  p.ltiles = std::max(p.rp / 16, 1);
  const int steps = (A->n + 31) / 32, tiles = p.ltiles * ((b + 15) / 16);
  // four waves of up to four steps each per split, fewer splits where the
  // tiles fill the chip by themselves
  p.splits = std::max(1, std::min({kMxPrepSplits, (steps + 15) / 16, (1024 + tiles - 1) / tiles}));
  p.steps_per_split = (steps + p.splits - 1) / p.splits;
  p.tb = A->r > 0 ? tiles * p.splits : 0;
  return p;
}

void launch_mx_prep(MxPrep p, hipStream_t s) {
  if (p.Xt || p.Xp || p.Xo || p.Up) {
    const int64_t work = std::max({p.Xt ? (int64_t)p.n * (p.ldt / 8) : 0, p.Xp ? (int64_t)p.b * (p.np / 8) : 0, (int64_t)(p.Xo ? p.nch * 256 : 0),
                                   p.Up ? (int64_t)p.m * (p.rp / 8) : 0});
    p.xb = (int)std::min<int64_t>((work + 255) / 256, 1024);
  }
  if (p.tb + p.xb > 0) hipLaunchKernelGGL(k_mx_prep, dim3((unsigned)(p.tb + p.xb)), dim3(256), 0, s, p);
}

struct SkinnyArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const int32_t* row_ptr;
  const void* col;
  const uint16_t* vals;
  const uint16_t* X;   // rows of ldx, 16-byte aligned unless b == 1
  const uint16_t* Xo;  // X in operand order; null = none
  const uint16_t* Xt;  // n x 16, b > 1 and S not empty
  const uint16_t* U;
  const float* Tp;
  uint16_t* Y;
  int m, n, b, r, rp, ng, ldx, splits, has_s, col16;
};

// Element e of T: its K splits' partial sums, loaded together, added in order.
__device__ __forceinline__ float t_sum(const SkinnyArgs& a, int e) {
  float p[kMxPrepSplits];
#pragma unroll
  for (int ks = 0; ks < kMxPrepSplits; ++ks) p[ks] = a.Tp[(uint32_t)min(ks, a.splits - 1) * (uint32_t)(a.b * a.rp) + e];
  float v = p[0];
#pragma unroll
  for (int ks = 1; ks < kMxPrepSplits; ++ks) v += ks < a.splits ? p[ks] : 0.f;
  return v;
}

// S's part of the block's 16 rows.  A wave takes R rows at once, LG = 64 / R
// lanes each; a lane's entries are loaded four at a time (past the end the
// last one again, with value 0), so that the chain of dependent loads -- row
// pointers, columns, X -- is walked once for up to 4 LG (2 LG) entries.
// Up to CB (1 or 4) columns: the lanes of a row take its entries and gather
// each column's value of X.
template <int LG, int CB, typename COL>
__device__ __forceinline__ void s_rows(const SkinnyArgs& a, const COL* __restrict__ col, int p0, int p1, float (&s)[CB]) {
  const int sl = lane_id() % LG;
#pragma unroll
  for (int c = 0; c < CB; ++c) s[c] = 0.f;
  for (int p = p0 + sl; p < p1; p += 4 * LG) {
    int j[4];
    float v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int pp = min(p + u * LG, p1 - 1);
      j[u] = (int)col[pp];
      v[u] = bf16lo(a.vals[pp]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = p + u * LG < p1 && (unsigned)j[u] < (unsigned)a.n;
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const float x = bf16lo(a.X[(uint32_t)(min(c, a.b - 1) * a.ldx + (ok ? j[u] : 0))]);
        s[c] = fmaf(ok ? v[u] : 0.f, ok ? x : 0.f, s[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int off = 1; off < LG; off <<= 1) s[c] += __shfl_xor(s[c], off, 64);
}

// Sixteen columns: lane 2 e + h of a row takes entries e, e + LG / 2, .. and
// columns 8 h .. 8 h + 7; the lanes of a half are then added up in a fixed
// tree, in which they first share out the eight columns: column 8 h + k ends
// in the lanes with lane % 2 = h and (lane / 2) % 8 = k.
// The first four entries come in j, v (s_request16), requested before the codes.
template <int LG, typename COL>
__device__ __forceinline__ void s_request16(const SkinnyArgs& a, const COL* __restrict__ col, int p, int p1,
                                            int (&j)[4], uint32_t (&v)[4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int pp = max(min(p + u * (LG / 2), p1 - 1), 0);  // an empty S has no call here
    j[u] = (int)col[pp];
    v[u] = a.vals[pp];
  }
}

template <int LG, typename COL>
__device__ __forceinline__ float s_rows16(const SkinnyArgs& a, const COL* __restrict__ col, int p0, int p1, int (&j)[4],
                                          uint32_t (&v)[4]) {
  const int lane = lane_id(), sl = lane % LG, h = lane & 1;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = p0 + (sl >> 1); p < p1; p += 2 * LG) {
    u32x4 x[4];
    float f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool ok = p + u * (LG / 2) < p1 && (unsigned)j[u] < (unsigned)a.n;
      x[u] = *reinterpret_cast<const u32x4*>(a.Xt + (int64_t)(ok ? j[u] : 0) * kSkCols + 8 * h);
      f[u] = bf16lo(v[u]);
      if (!ok) f[u] = 0.f, x[u] = u32x4{0u, 0u, 0u, 0u};
    }
    if (p + 2 * LG < p1) s_request16<LG>(a, col, p + 2 * LG, p1, j, v);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[2 * k] = fmaf(f[u], bf16lo(x[u][k]), s[2 * k]);
        s[2 * k + 1] = fmaf(f[u], bf16hi(x[u][k]), s[2 * k + 1]);
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
#pragma unroll
  for (int off = 16; off < LG; off <<= 1) s[0] += __shfl_xor(s[0], off, 64);
  return s[0];
}

// WV waves, B chunks of a wave in flight (at least 2: X comes two chunks ahead).
// XO: X comes in operand order (k_mx_prep), whole chunks with zeros past n.
template <int WV, int B, bool XO>
__global__ __launch_bounds__(64 * WV, 4) void k_mx_skinny(SkinnyArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  float* red = reinterpret_cast<float*>(lds);                       // [WV][16 columns][16 rows]
  float* sred = red + WV * 256;                                     // [16 columns][16 rows]
  uint16_t* Tl = reinterpret_cast<uint16_t*>(sred + 256);           // [b][2][rp + 8]
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int row0 = (int)blockIdx.x * 16;
  const int q = lane >> 4;
  const int nch = (a.ng + 3) >> 2, nfull = XO ? nch : a.n >> 7;  // else the last chunk may be short
  const uint32_t grow = (uint32_t)min(row0 + (lane & 15), a.m - 1) * (uint32_t)a.ng;
  const uint32_t xoff = (uint32_t)min(lane & 15, a.b - 1) * (uint32_t)a.ldx;

  u32x4 cw[B], xv[2][4];
  uint32_t sb[B];
  // whole chunks c0 + WV u; past the last one, that one again, not used.  The
  // codes of a batch are in flight together, X two chunks ahead.
  auto load_x = [&](int c, u32x4 (&x)[4]) {
    if constexpr (XO) {
      const u32x4* xp = reinterpret_cast<const u32x4*>(a.Xo) + (256 * (uint32_t)min(c, nfull - 1) + lane);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = xp[64 * k];
    } else {
      const Bytes16* xp = reinterpret_cast<const Bytes16*>(a.X + (xoff + 128 * (uint32_t)min(c, nfull - 1) + 32 * q));
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = u32x4{xp[k].w[0], xp[k].w[1], xp[k].w[2], xp[k].w[3]};
    }
  };
  auto issue = [&](int c0) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      uint32_t g = 4 * (uint32_t)min(c0 + WV * u, nfull - 1) + q;
      if constexpr (XO) g = min(g, (uint32_t)a.ng - 1u);  // past the row: its last group again, against zeros
      const uint32_t at = grow + g;
      cw[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a.codes + at * 16));
      sb[u] = a.scales[at];
    }
    load_x(c0, xv[0]);
    load_x(c0 + WV, xv[1]);
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int c0) {
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (c0 + WV * u >= nfull) break;  // the same for the whole wave
      const float sc = mx_scale(sb[u], 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) acc = mfma16(mx4_to_bf16x8(cw[u][k], sc), xv[u & 1][k], acc);
      if (u + 2 < B) load_x(c0 + WV * (u + 2), xv[u & 1]);
    }
  };
  constexpr int LG = 4 * WV;  // lanes per row of S
  int p0 = 0, p1 = 0;
  if (a.has_s && row0 + w * (16 / WV) + lane / LG < a.m) {
    p0 = a.row_ptr[row0 + w * (16 / WV) + lane / LG];
    p1 = a.row_ptr[row0 + w * (16 / WV) + lane / LG + 1];
  }
  int sj[4] = {0, 0, 0, 0};
  uint32_t sv[4] = {0u, 0u, 0u, 0u};
  if (a.has_s && a.b > kSkGather) {
    if (a.col16) s_request16<LG>(a, static_cast<const uint16_t*>(a.col), p0 + (lane % LG >> 1), p1, sj, sv);
    else s_request16<LG>(a, static_cast<const int32_t*>(a.col), p0 + (lane % LG >> 1), p1, sj, sv);
  }
  if (w < nfull) issue(w);

  const int ldt = a.rp + 8;  // rows 16 bytes apart modulo the banks
  if (a.r > 0) {
    for (int e = t; e < a.b * a.rp; e += 64 * WV) {
      const float v = t_sum(a, e);
      const int c = e / a.rp, l = e - c * a.rp;
      const uint16_t hi = f32_to_bf16(v);
      // an infinity leaves 0, not the NaN of inf - inf
      const uint16_t lo = (hi & 0x7fffu) == 0x7f80u ? (uint16_t)0 : f32_to_bf16(v - bf16lo(hi));
      Tl[(2 * c) * ldt + l] = hi;
      Tl[(2 * c + 1) * ldt + l] = lo;
    }
  }
  if (a.has_s) {
    const int i = w * (16 / WV) + lane / LG;
    const uint16_t* c16 = static_cast<const uint16_t*>(a.col);
    const int32_t* c32 = static_cast<const int32_t*>(a.col);
    if (a.b == 1) {
      float s[1];
      if (a.col16) s_rows<LG, 1>(a, c16, p0, p1, s);
      else s_rows<LG, 1>(a, c32, p0, p1, s);
      if (lane % LG == 0) sred[i] = s[0];
    } else if (a.b <= kSkGather) {
      float s[kSkGather];
      if (a.col16) s_rows<LG, kSkGather>(a, c16, p0, p1, s);
      else s_rows<LG, kSkGather>(a, c32, p0, p1, s);
#pragma unroll
      for (int c = 0; c < kSkGather; ++c)
        if (lane % LG == c) sred[c * 16 + i] = s[c];
    } else {
      const float s = a.col16 ? s_rows16<LG>(a, c16, p0, p1, sj, sv) : s_rows16<LG>(a, c32, p0, p1, sj, sv);
      if (lane % LG < 16) sred[(8 * (lane & 1) + ((lane >> 1) & 7)) * 16 + i] = s;
    }
  }
  for (int c0 = w; c0 < nfull; c0 += WV * B) {
    compute(c0);
    if (c0 + WV * B < nfull) issue(c0 + WV * B);
  }
  if (!XO && nch > nfull && w == nfull % WV) {  // the short chunk: lanes past its groups hold zeros of X
    const int g = 4 * nfull + q;
    const uint32_t at = grow + (uint32_t)min(g, a.ng - 1);
    const u32x4 code = *reinterpret_cast<const u32x4*>(a.codes + at * 16);
    const float sc = g < a.ng ? mx_scale(a.scales[at], 0) : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      acc = mfma16(mx4_to_bf16x8(code[k], sc), load_row8(a.X + xoff, 32 * g + 8 * k, a.n), acc);
  }
  if (a.r > 0) {
    __syncthreads();
    const uint16_t* __restrict__ urow = a.U + (int64_t)min(row0 + (lane & 15), a.m - 1) * a.r;
    const uint16_t* tl = Tl + 2 * min(lane & 15, a.b - 1) * ldt + 8 * q;
    const bool whole = a.r % 8 == 0;
    for (int j = w; j < (a.rp >> 5); j += WV) {
      const u32x4 uv = whole ? load_row8<true>(urow, 32 * j + 8 * q, a.r) : load_row8(urow, 32 * j + 8 * q, a.r);
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
// One to four columns, k_mx_gemv<BC, RW>: a wave owns RW rows and walks their
// columns in chunks of 2048, one group (16 bytes of codes, 32 columns) per
// lane, so that a row's codes come in whole lines.  A group's values meet the
// lane's 32 columns of X, read once from LDS for all RW rows, in
// v_dot2_f32_bf16: 16 conversions and 16 BC products per group, where the
// matrix cores would fill 16 columns whatever BC is and want four times the
// codes' bytes of X from the vector memory path.  S and U T are added to the
// lanes' partial sums, and one wave sum per row and column ends it.
// X sits in LDS piece-major: 16-byte piece k of group g of a chunk at 64 k + g,
// so that neighbouring lanes read neighbouring pieces.
// ---------------------------------------------------------------------------
static constexpr int kGvWaves = 4;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}

// bf16 index of column j within X's LDS image.
__device__ __forceinline__ int gv_at(int j) {
  return ((((j >> 11) * 4 + ((j >> 3) & 3)) * 64 + ((j >> 5) & 63)) << 3) + (j & 7);
}

template <int BC, int RW>
__global__ __launch_bounds__(64 * kGvWaves) void k_mx_gemv(SkinnyArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  const int nch = (a.ng + 63) >> 6;                  // chunks of 64 groups
  const int plane = nch * 2048;                      // bf16 of one column's image
  uint16_t* xs = reinterpret_cast<uint16_t*>(lds);   // [BC][plane]
  float* Ts = reinterpret_cast<float*>(xs + BC * plane);  // [BC][rp]
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int row0 = ((int)blockIdx.x * kGvWaves + w) * RW;
  uint32_t grow[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) grow[i] = (uint32_t)min(row0 + i, a.m - 1) * (uint32_t)a.ng;

  u32x4 cw[2][RW];
  uint32_t sb[2][RW];
  // lanes past the row's last group read that one again, against zeros of X
  auto issue = [&](int c, u32x4 (&cv)[RW], uint32_t (&sv)[RW]) {
    const uint32_t g = (uint32_t)min(64 * c + lane, a.ng - 1);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      cv[i] = *reinterpret_cast<const u32x4*>(a.codes + (grow[i] + g) * 16);
      sv[i] = a.scales[grow[i] + g];
    }
  };
  issue(0, cw[0], sb[0]);
  // the first 64 entries of each row of S
  int p0[RW], p1[RW], j0[RW];
  uint32_t v0[RW];
  if (a.has_s) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      p0[i] = a.row_ptr[min(row0 + i, a.m - 1)];
      p1[i] = a.row_ptr[min(row0 + i, a.m - 1) + 1];
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int p = p0[i] + lane;
      j0[i] = -1, v0[i] = 0u;
      if (p < p1[i]) {
        j0[i] = a.col16 ? (int)static_cast<const uint16_t*>(a.col)[p] : static_cast<const int32_t*>(a.col)[p];
        v0[i] = a.vals[p];
      }
    }
  }
  auto stage_x = [&](auto whole) {
    for (int e0 = t; e0 < nch * 256; e0 += 256 * kGvWaves) {
      u32x4 x[4][BC];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int c = 0; c < BC; ++c)
          x[u][c] = load_row8<decltype(whole)::value>(a.X + (int64_t)min(c, a.b - 1) * a.n, 8 * (e0 + 64 * kGvWaves * u), a.n);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + 64 * kGvWaves * u;
        const int at = ((((e >> 8) * 4 + (e & 3)) * 64 + ((e >> 2) & 63)) << 3);
#pragma unroll
        for (int c = 0; c < BC; ++c)
          if (e < nch * 256) *reinterpret_cast<u32x4*>(xs + c * plane + at) = x[u][c];
      }
    }
  };
  if (a.n % 8 == 0) stage_x(std::true_type());
  else stage_x(std::false_type());
  if (a.r > 0) {
    for (int e = t; e < a.b * a.rp; e += 64 * kGvWaves) Ts[e] = t_sum(a, e);
  }
  __syncthreads();

  float acc[RW][BC];
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int c = 0; c < BC; ++c) acc[i][c] = 0.f;
  auto compute = [&](int ch, const u32x4 (&cv)[RW], const uint32_t (&sv)[RW]) {
    float sc[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) sc[i] = mx_scale(sv[i], 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u32x4 x[BC];
#pragma unroll
      for (int c = 0; c < BC; ++c)
        x[c] = *reinterpret_cast<const u32x4*>(xs + c * plane + (((ch * 4 + k) * 64 + lane) << 3));
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const u32x4 d = mx4_to_bf16x8(cv[i][k], sc[i]);
#pragma unroll
        for (int c = 0; c < BC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][c] = dot2(d[e], x[c][e], acc[i][c]);
      }
    }
  };
  // pairs of chunks, so that the two register sets are named at compile time
  for (int ch = 0; ch < nch; ch += 2) {
    if (ch + 1 < nch) issue(ch + 1, cw[1], sb[1]);
    compute(ch, cw[0], sb[0]);
    if (ch + 1 < nch) {
      if (ch + 2 < nch) issue(ch + 2, cw[0], sb[0]);
      compute(ch + 1, cw[1], sb[1]);
    }
  }
  if (a.has_s) {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      for (int p = p0[i] + lane;;) {
        if ((unsigned)j0[i] < (unsigned)a.n) {
          const float v = bf16lo(v0[i]);
#pragma unroll
          for (int c = 0; c < BC; ++c) acc[i][c] = fmaf(v, bf16lo(xs[c * plane + gv_at(j0[i])]), acc[i][c]);
        }
        p += 64;
        if (p >= p1[i]) break;
        j0[i] = a.col16 ? (int)static_cast<const uint16_t*>(a.col)[p] : static_cast<const int32_t*>(a.col)[p];
        v0[i] = a.vals[p];
      }
    }
  }
  auto add_ut = [&](auto whole) {
    for (int l = 8 * lane; l < a.r; l += 512) {
      u32x4 u[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i)
        u[i] = load_row8<decltype(whole)::value>(a.U + (int64_t)min(row0 + i, a.m - 1) * a.r, l, a.r);
#pragma unroll
      for (int c = 0; c < BC; ++c) {
        const float* T = Ts + min(c, a.b - 1) * a.rp + l;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            acc[i][c] = fmaf(bf16lo(u[i][e]), T[2 * e], acc[i][c]);
            acc[i][c] = fmaf(bf16hi(u[i][e]), T[2 * e + 1], acc[i][c]);
          }
      }
    }
  };
  if (a.r % 8 == 0) add_ut(std::true_type());
  else add_ut(std::false_type());
  // result q = i BC + c goes to lane q
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int c = 0; c < BC; ++c) {
      const float v = wave_sum(acc[i][c]);
      if (lane == i * BC + c) y = v;
    }
  const int c = lane % BC, row = row0 + lane / BC;
  if (lane < RW * BC && c < a.b && row < a.m) a.Y[(int64_t)c * a.m + row] = f32_to_bf16(y);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static int round32(int x) { return (x + 31) & ~31; }

static size_t gv_plane_bytes(int n) { return (size_t)((mx_groups(n) + 63) / 64) * 4096; }

// Up to four columns whose X (and T) fit 64 KiB of LDS, of rows long enough
// to give most lanes a group.
static bool gv_supported(const hss_matrix* A, int b) {
  if (b > 4 || A->n < 1024) return false;
  return (size_t)(b > 2 ? 4 : b) * gv_plane_bytes(A->n) + (size_t)b * round32(A->r) * 4 <= 64 * 1024;
}

struct SkinnyPlan {
  MxPrep prep;
  size_t tp, xt, xp, total;
};

static SkinnyPlan plan_skinny(const hss_matrix* A, int b) {
  SkinnyPlan p = {};
  p.prep = mx_prep_plan(A, b);
  p.tp = 0;
  p.xt = al256((size_t)p.prep.splits * b * p.prep.rp * 4);
  p.xp = p.xt + ((b > kSkGather && A->nnz > 0) ? al256((size_t)A->n * kSkCols * 2) : 0);
  p.total = p.xp + (b > 1 ? (size_t)((mx_groups(A->n) + 3) / 4) * 4096 : 0);
  return p;
}

// The T terms of one block must fit beside the reduction buffers (64 KiB).
bool mx_skinny_supported(const hss_matrix* A, int b) {
  if ((A->flags & HSS_MX4_T) || b > kSkCols) return false;
  return (size_t)b * 2 * (round32(A->r) + 8) * 2 <= 40 * 1024;
}

size_t mx_skinny_ws_bytes(const hss_matrix* A, int b) { return plan_skinny(A, b).total; }

template <int WV, bool XO>
static void launch_skinny(const SkinnyArgs& a, int batch, unsigned grid, size_t tl, hipStream_t s) {
  const dim3 block(64 * WV);
  const size_t lds = (WV + 1) * 1024 + tl;
  switch (batch) {
    case 1:
    case 2: hipLaunchKernelGGL((k_mx_skinny<WV, 2, XO>), dim3(grid), block, lds, s, a); break;
    case 3: hipLaunchKernelGGL((k_mx_skinny<WV, 3, XO>), dim3(grid), block, lds, s, a); break;
    case 4: hipLaunchKernelGGL((k_mx_skinny<WV, 4, XO>), dim3(grid), block, lds, s, a); break;
    case 5: hipLaunchKernelGGL((k_mx_skinny<WV, 5, XO>), dim3(grid), block, lds, s, a); break;
    default: hipLaunchKernelGGL((k_mx_skinny<WV, 6, XO>), dim3(grid), block, lds, s, a); break;
  }
}

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
  a.m = m; a.n = n; a.b = b; a.r = r; a.rp = p.prep.rp;
  a.ng = mx_groups(n);
  a.splits = p.prep.splits;
  a.has_s = A->nnz > 0;
  a.col16 = (A->flags & HSS_COL16) != 0;
  a.ldx = n;
  const bool gemv = gv_supported(A, b);
  const bool need_xt = a.has_s && b > kSkGather && !gemv;
  // X in operand order: a load is then 1 KiB in a row, where rows of X make a
  // line of every lane's 64 bytes (us in all, 5 - 13 columns: 2731 x 5003
  // 12.3 against 13.7, 4096 x 11008 18.3 against 21.9, 8192^2 23.1 against
  // 25.5).  With neither S nor a low-rank term it costs a launch of its own,
  // about 2 us, which pays only where every block reads much of X (and for rows
  // off the 16-byte grid).  D alone, us for the rows / the copy, in graphs over
  // 0.4 GB of matrices: 4096 x 4096, 13 columns 7.4 / 7.9, 16 8.1 / 8.1; 4096 x
  // 8192, 5 columns 10.4 / 12.2, 8 11.4 / 12.2, 13 12.7 / 12.2; 4096 x 11008, 5
  // columns 12.0 / 14.2, 8 13.7 / 14.1, 13 16.0 / 14.2.  With more blocks than
  // fit at once (grid > 512) from a smaller X on: 11008 x 2528, 13 columns 12.0
  // / 10.9; 11008 x 4096, 8 columns 14.9 / 15.0, 13 17.2 / 14.8; 11008 x 8192,
  // 5 columns 25.6 / 27.8, 8 29.7 / 27.9.
  const unsigned grid = (unsigned)((m + 15) / 16);
  const bool long_x = (int64_t)b * n > (grid > 512 ? 40960 : 65536);
  const bool need_xo = !gemv && b > 1 && (r > 0 || need_xt || long_x || n % 8 != 0 || (uintptr_t)X % 16 != 0);
  MxPrep pr = p.prep;
  pr.X = a.X;
  pr.Vt = static_cast<const uint16_t*>(A->Vt);
  pr.Tp = reinterpret_cast<float*>(base + p.tp);
  pr.ldt = kSkCols;
  pr.nch = (a.ng + 3) / 4;
  if (need_xt) pr.Xt = reinterpret_cast<uint16_t*>(base + p.xt);
  if (need_xo) pr.Xo = reinterpret_cast<uint16_t*>(base + p.xp);
  launch_mx_prep(pr, s);
  a.Xo = pr.Xo;
  if (gemv) {
    const size_t lds = (size_t)(b > 2 ? 4 : b) * gv_plane_bytes(n) + (size_t)b * a.rp * 4;
    // Two rows a wave, four where the rows are many: fewer waves then read X
    // from LDS (us at two / four, D alone, in graphs over 0.4 GB of matrices:
    // n 4096, one column 8192 rows 5.9 / 6.3, 9216 6.5 / 7.1, 11008 7.2 / 7.3,
    // 16384 9.5 / 9.0, 32768 15.1 / 14.7; two columns 9216 7.7 / 8.2, 11008 8.5 /
    // 8.3, 16384 10.8 / 10.4; four columns 6144 8.0 / 8.5, 8192 9.3 / 8.8, 11008
    // 12.1 / 11.0, 16384 15.0 / 13.6.  n 1024 alike.  The one exception: n
    // 8192, one column, 16384 rows 15.3 / 16.4).
    const bool four = m > (b > 2 ? 8192 : 12288);
    const unsigned gv = (unsigned)((m + kGvWaves * (four ? 4 : 2) - 1) / (kGvWaves * (four ? 4 : 2)));
    const dim3 block(64 * kGvWaves);
    if (b == 1) {
      if (four) hipLaunchKernelGGL((k_mx_gemv<1, 4>), dim3(gv), block, lds, s, a);
      else hipLaunchKernelGGL((k_mx_gemv<1, 2>), dim3(gv), block, lds, s, a);
    } else if (b == 2) {
      if (four) hipLaunchKernelGGL((k_mx_gemv<2, 4>), dim3(gv), block, lds, s, a);
      else hipLaunchKernelGGL((k_mx_gemv<2, 2>), dim3(gv), block, lds, s, a);
    } else {
      if (four) hipLaunchKernelGGL((k_mx_gemv<4, 4>), dim3(gv), block, lds, s, a);
      else hipLaunchKernelGGL((k_mx_gemv<4, 2>), dim3(gv), block, lds, s, a);
    }
    return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
  }
  const size_t tl = r > 0 ? (size_t)b * 2 * (a.rp + 8) * 2 : 0;
  // Four waves a block where rows are short or the blocks fill the chip anyway,
  // else eight (4096 x 11008, 8 columns, D alone: 13.5 us; 16 waves 16.1).  A
  // wave's chunks in as few batches as possible, all of about the same size,
  // since a short batch loads its last chunk over again: 2731 x 5024, 13
  // columns, D alone, five chunks a wave: 7.4 us in one batch, 8.6 as 4 + 1.
  const int nfull = a.Xo ? pr.nch : n >> 7;
  const bool wide = nfull > 16 && grid <= 512;
  const int per = std::max(1, (nfull + (wide ? 7 : 3)) / (wide ? 8 : 4));
  const int batches = (per + kSkBatch - 1) / kSkBatch, batch = (per + batches - 1) / batches;
  if (a.Xo && wide) launch_skinny<8, true>(a, batch, grid, tl, s);
  else if (a.Xo) launch_skinny<4, true>(a, batch, grid, tl, s);
  else if (wide) launch_skinny<8, false>(a, batch, grid, tl, s);
  else launch_skinny<4, false>(a, batch, grid, tl, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
