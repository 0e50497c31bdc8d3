// Low-rank adapters of many requests beside a shared projection
// (hss_adapters_apply) and their backward pass (hss_adapters_grad).  Row t has
// the adapter l = ids[t], its factors U_l (m x r) and Vt_l (r x n):
//
//   forward   T = X Vt_l^T            Y  = base + scale_l T U_l^T
//   backward  P = G U_l               dX = base + scale_l P Vt_l
//             dU_l = scale_l G_l^T T_l,   dVt_l = scale_l P_l^T X_l
//
// The products are short on one side (r), so all of it is bound by reading X, G
// and the factors and by writing Y, dX and the gradients.  Rows of one adapter
// are worked on together, so that its factors are read once for up to 32 of
// them: a tile is an adapter and up to 16 or 32 of its rows, found by each block
// from ids (no launch for a plan, nothing on the host).
//
// Two launches each way: k_ad_rank makes T (and P), K split over blocks into
// partial sums in fp32, for a few tiles would not fill the chip; the second
// kernel adds the splits in order as it reads them.  T and P then go to the
// matrix cores in bf16 terms: two (16 significant bits) where the result is
// rounded to bf16 anyway, three (24 bits) for the fp32 gradients.
#include <algorithm>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

static constexpr int kAdRows = HSS_MAX_BATCH;
static constexpr int kAdSmall = 64;     // batches up to here: tiles of 16 rows, found by one ballot
static constexpr int kAdRank = 64;      // ranks of one pass
static constexpr int kAdUnit = 256;     // columns of K that a block takes at a time, 64 a wave
static constexpr int kAdBlocks = 512;   // blocks of k_ad_rank that K is split for

struct AdArgs {
  const uint16_t* U;
  const uint16_t* Vt;
  const float* scale;
  const int32_t* ids;
  const uint16_t* X;
  const uint16_t* G;
  const uint16_t* base;
  uint16_t* Y;    // forward: Y; backward: dX
  float* dU;
  float* dVt;
  float* T;       // [splits_x][b][ldr]
  float* P;       // [splits_g][b][ldr]
  int m, n, r, count, b;
  int ldr;        // r rounded up to 16
  int tiles;      // most tiles that ids can make
  int splits_x, splits_g, units_x, units_g;  // K splits of T and P, units of each
  int chunks;     // passes over the ranks
  int blocks_y, blocks_u, blocks_v;          // of the backward's second launch
  int cols_y, cols_u, cols_v;                // column blocks of each
};

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct AdTile {
  int adapter;  // -1: rows without one
  int rows;     // 0: no such tile
};

// Exclusive prefix sum over the block's 256 threads, and the total.
__device__ __forceinline__ int ad_scan(int v, int* part, int* total) {
  const int w = threadIdx.x >> 6;
  const int before = (int)wave_excl_scan_u32((uint32_t)v);
  if ((threadIdx.x & 63) == 63) part[w] = before + v;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < w) base += part[k];
    all += part[k];
  }
  __syncthreads();
  *total = all;
  return base + before;
}

__device__ __forceinline__ int ad_id(const int32_t* ids, int t, int count) {
  const int id = ids[t];
  return id >= 0 && id < count ? id : -1;
}

// rows[] (LDS): the rows of adapter l with ranks first .. first + most - 1 among
// its rows, in order; returns how many rows it has in all.
__device__ __forceinline__ int ad_collect(const int32_t* ids, int b, int count, int l, int first, int most,
                                          uint16_t* rows, int* part) {
  const int per = kAdRows / 256;
  const int t0 = threadIdx.x * per;
  int mine = 0;
#pragma unroll
  for (int k = 0; k < per; ++k)
    if (t0 + k < b && ad_id(ids, t0 + k, count) == l) mine |= 1 << k;
  int total;
  int at = ad_scan(__popc(mine), part, &total) - first;
#pragma unroll
  for (int k = 0; k < per; ++k)
    if (mine >> k & 1) {
      if (at >= 0 && at < most) rows[at] = (uint16_t)(t0 + k);
      ++at;
    }
  __syncthreads();
  return total;
}

// Tile `tile` of the batch: its adapter and its rows (in LDS).  Up to 64 rows
// tile t starts at row t, if that is the 1st, 17th, .. row of its adapter; beyond,
// tiles are counted through the adapters, rows without one last.
template <int TM>
__device__ __forceinline__ AdTile ad_tile(const int32_t* ids, int b, int count, int tile, uint16_t* rows, int* part,
                                          int* bins) {
  AdTile r = {-1, 0};
  if (TM == 16) {
    const int lane = threadIdx.x & 63;
    const int id = lane < b ? ad_id(ids, lane, count) : -2;
    const int own = __builtin_amdgcn_readlane(id, tile);
    const uint64_t same = __ballot(id == own);
    const int before = __popcll(same & ((1ull << tile) - 1));
    if (before % TM) return r;
    const int rank = __popcll(same & lanemask_lt()) - before;
    if (threadIdx.x < 64 && id == own && rank >= 0 && rank < TM) rows[rank] = (uint16_t)lane;
    __syncthreads();
    r.adapter = own;
    r.rows = min(TM, __popcll(same) - before);
    return r;
  }
  const int t = threadIdx.x;
  for (int k = t; k <= count; k += 256) bins[k] = 0;
  __syncthreads();
  for (int j = t; j < b; j += 256) {  // a wave of one adapter's rows adds once
    int id = ad_id(ids, j, count);
    if (id < 0) id = count;
    const int head = __builtin_amdgcn_readfirstlane(id);
    const uint64_t same = __ballot(id == head);
    if (same == __ballot(1)) {
      if (__popcll(same & lanemask_lt()) == 0) atomicAdd(&bins[id], __popcll(same));
    } else {
      atomicAdd(&bins[id], 1);
    }
  }
  __syncthreads();
  const int per = (count + 256) / 256, k0 = t * per;
  int own = 0, total;
  for (int k = k0; k < min(k0 + per, count + 1); ++k) own += (bins[k] + TM - 1) / TM;
  int at = ad_scan(own, part, &total);
  if (tile >= total) return r;
  if (tile >= at && tile < at + own) {
    int k = k0;
    while (tile >= at + (bins[k] + TM - 1) / TM) at += (bins[k++] + TM - 1) / TM;
    part[4] = k, part[5] = tile - at;
  }
  __syncthreads();
  const int bin = part[4], first = part[5] * TM;
  r.adapter = bin == count ? -1 : bin;
  r.rows = min(TM, bins[bin] - first);
  ad_collect(ids, b, count, r.adapter, first, TM, rows, part);
  return r;
}

// ---------------------------------------------------------------------------
// 8 x 8 transposition: eight rows of eight bf16 (v[e], column f) into operand f =
// the eight rows' values of column f, two of them a dword.
// ---------------------------------------------------------------------------
template <int CW, typename V>
__device__ __forceinline__ u32x4 ad_column(const V (&v)[8], int f) {
  u32x4 o;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    o[d] = __builtin_amdgcn_perm(v[2 * d + 1].w[f >> 1], v[2 * d].w[f >> 1], f & 1 ? 0x07060302u : 0x05040100u);
  return o;
}

template <int CW>
struct AdPiece {  // CW bf16 of a row
  uint32_t w[CW / 2];
};

// CW bf16 of a row of n at column k, zeros past the end.
template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_piece(const uint16_t* row, int k, int n) {
  struct __attribute__((packed, aligned(2))) Raw {
    uint32_t w[CW / 2];
  };
  AdPiece<CW> p;
  if (k + CW <= n) {
    const Raw raw = *reinterpret_cast<const Raw*>(row + k);
#pragma unroll
    for (int d = 0; d < CW / 2; ++d) p.w[d] = raw.w[d];
  } else {
#pragma unroll
    for (int d = 0; d < CW / 2; ++d) {
      const uint32_t lo = k + 2 * d < n ? row[k + 2 * d] : 0u, hi = k + 2 * d + 1 < n ? row[k + 2 * d + 1] : 0u;
      p.w[d] = lo | hi << 16;
    }
  }
  return p;
}

// ---------------------------------------------------------------------------
// T = X Vt^T and P = G U, partial sums over a block's part of K.
//   D[rank][row] += A[rank][k] B[row][k]: A = Vt_l as stored, or U_l transposed
//   through LDS.  Wave w takes 64 of each unit's 256 columns (a whole cache line of
//   each row); the four waves' sums meet in LDS.
// grid: (tiles, splits_x + splits_g, passes over the ranks)
// ---------------------------------------------------------------------------
static constexpr int kAdPitch = kAdUnit + 8;  // of U^T in LDS

template <int TM, int NR, bool WHOLE>
__global__ __launch_bounds__(256) void k_ad_rank(AdArgs a) {
  constexpr int MF = TM / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ uint16_t rows[TM];
  __shared__ int part[8];
  const int tile = blockIdx.x, rank0 = (int)blockIdx.z * kAdRank;
  const bool side = (int)blockIdx.y >= a.splits_x;  // P
  const AdTile at = ad_tile<TM>(a.ids, a.b, a.count, tile, rows, part, reinterpret_cast<int*>(smem));
  if (at.rows == 0 || at.adapter < 0) return;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int z = side ? (int)blockIdx.y - a.splits_x : (int)blockIdx.y;
  const int K = side ? a.m : a.n;
  const int units = (K + kAdUnit - 1) / kAdUnit, per = side ? a.units_g : a.units_x;
  const int u0 = z * per, u1 = min(u0 + per, units);
  const uint16_t* xrow[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f)
    xrow[f] = (side ? a.G : a.X) + (int64_t)rows[min(16 * f + i, at.rows - 1)] * K;

  f32x4 acc[MF][NR];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (!side) {
    const uint16_t* vrow[NR];
#pragma unroll
    for (int g = 0; g < NR; ++g)
      vrow[g] = a.Vt + ((int64_t)at.adapter * a.r + min(rank0 + 16 * g + i, a.r - 1)) * K;
    for (int u = u0; u < u1; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = u * kAdUnit + 64 * w + 32 * h + 8 * q;
        u32x4 x[MF], v[NR];
#pragma unroll
        for (int f = 0; f < MF; ++f) x[f] = load_row8<WHOLE>(xrow[f], k, K);
#pragma unroll
        for (int g = 0; g < NR; ++g) v[g] = load_row8<WHOLE>(vrow[g], k, K);
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int g = 0; g < NR; ++g)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(v[g]), as_bf16(x[f]), acc[f][g], 0, 0, 0);
      }
    }
  } else {
    uint16_t* ut = reinterpret_cast<uint16_t*>(smem);  // [16 NR][kAdPitch]
    const uint16_t* U = a.U + (int64_t)at.adapter * a.m * a.r;
    for (int u = u0; u < u1; ++u) {
      __syncthreads();
      // 8 x 8 pieces: 32 of the unit's rows j times 2 NR of the ranks
      for (int p = threadIdx.x; p < 64 * NR; p += 256) {
        const int kb = p % (2 * NR), jb = p / (2 * NR), j0 = u * kAdUnit + 8 * jb;
        AdPiece<8> v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (j0 + e < K) v[e] = ad_piece<8>(U + (int64_t)(j0 + e) * a.r, rank0 + 8 * kb, a.r);
          else v[e] = AdPiece<8>{{0u, 0u, 0u, 0u}};
        }
#pragma unroll
        for (int f = 0; f < 8; ++f)
          *reinterpret_cast<u32x4*>(ut + (8 * kb + f) * kAdPitch + 8 * jb) = ad_column<8>(v, f);
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kl = 64 * w + 32 * h + 8 * q, k = u * kAdUnit + kl;
        u32x4 x[MF];
#pragma unroll
        for (int f = 0; f < MF; ++f) x[f] = load_row8<WHOLE>(xrow[f], k, K);
#pragma unroll
        for (int g = 0; g < NR; ++g) {
          const bf16x8 v = *reinterpret_cast<const bf16x8*>(ut + (16 * g + i) * kAdPitch + kl);
#pragma unroll
          for (int f = 0; f < MF; ++f)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, as_bf16(x[f]), acc[f][g], 0, 0, 0);
        }
      }
    }
  }
  // the waves' sums, added in order
  f32x4* sum = reinterpret_cast<f32x4*>(smem);  // [4][MF NR][64]
  __syncthreads();
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) sum[(w * MF * NR + f * NR + g) * 64 + lane] = acc[f][g];
  __syncthreads();
  float* out = (side ? a.P : a.T) + (int64_t)z * a.b * a.ldr;
  for (int s = w; s < MF * NR; s += 4) {
    const int f = s / NR, g = s % NR;
    f32x4 v = sum[s * 64 + lane];
#pragma unroll
    for (int k = 1; k < 4; ++k) v += sum[(k * MF * NR + s) * 64 + lane];
    const int rank = rank0 + 16 * g + 4 * q;
    if (16 * f + i < at.rows && rank < a.ldr)
      *reinterpret_cast<f32x4*>(out + (int64_t)rows[16 * f + i] * a.ldr + rank) = v;
  }
}

// ---------------------------------------------------------------------------
// Terms of T or P (times the adapter's scale) of up to TM rows and 64 ranks from
// rank0 on, in LDS as out[row][term][64 ranks]; zeros past r and past the rows.
// ---------------------------------------------------------------------------
static constexpr int kAdTermPitch = 2 * kAdRank + 8;

template <int TM>
__device__ __forceinline__ void ad_terms2(const float* part, int splits, const AdArgs& a, const AdTile& at,
                                          const uint16_t* rows, int rank0, uint16_t* out) {
  const float scale = a.scale ? a.scale[at.adapter] : 1.f;
  for (int e = threadIdx.x; e < TM * kAdRank; e += 256) {
    const int row = e / kAdRank, k = e % kAdRank;
    float v = 0.f;
    if (row < at.rows && rank0 + k < a.r) {
      const float* p = part + (int64_t)rows[row] * a.ldr + rank0 + k;
      for (int z = 0; z < splits; ++z) v += p[(int64_t)z * a.b * a.ldr];
      v *= scale;
    }
    const uint16_t hi = f32_to_bf16(v);
    const float rest = (hi & 0x7fffu) == 0x7f80u ? 0.f : v - __uint_as_float((uint32_t)hi << 16);  // inf leaves 0
    out[row * kAdTermPitch + k] = hi;
    out[row * kAdTermPitch + kAdRank + k] = f32_to_bf16(rest);
  }
}

__device__ __forceinline__ uint32_t ad_pack(float lo, float hi) { return f32_to_bf16(lo) | (uint32_t)f32_to_bf16(hi) << 16; }

// N (a multiple of 8) columns of a row of the output: base + v, in bf16.
template <int N>
__device__ __forceinline__ void ad_store(const AdArgs& a, int64_t row, int col, int cols, const float* v) {
  const uint16_t* in = a.base ? a.base + row * cols : nullptr;
  uint16_t* out = a.Y + row * cols;
#pragma unroll
  for (int c = 0; c < N; c += 8) {
    if (col + c + 8 <= cols) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = v[c + k];
      if (in) {
        const Bytes16 old = *reinterpret_cast<const Bytes16*>(in + col + c);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[2 * k] += bf16lo(old.w[k]), x[2 * k + 1] += bf16hi(old.w[k]);
      }
      Bytes16 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o.w[k] = ad_pack(x[2 * k], x[2 * k + 1]);
      *reinterpret_cast<Bytes16*>(out + col + c) = o;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + c + k < cols)
          out[col + c + k] = f32_to_bf16((in ? __uint_as_float((uint32_t)in[col + c + k] << 16) : 0.f) + v[c + k]);
    }
  }
}

// Rows without an adapter: the output is base (nothing to do in place).
__device__ __forceinline__ void ad_copy(const AdArgs& a, const AdTile& at, const uint16_t* rows, int col, int width,
                                        int cols) {
  if (a.base == a.Y) return;
  for (int e = threadIdx.x; e < at.rows * width; e += 256) {
    const int c = col + e % width;
    const int64_t row = rows[e / width];
    if (c < cols) a.Y[row * cols + c] = a.base ? a.base[row * cols + c] : (uint16_t)0;
  }
}

// ---------------------------------------------------------------------------
// Y = base + scale T U^T.  D[column][row], A = U_l as stored: row i of piece f is
// column 16 (i / 4) + 4 f + i % 4 of the wave's 64, so that a lane ends up with
// 16 adjacent columns of one row.
// grid: (tiles, ceil(m / 256))
// ---------------------------------------------------------------------------
template <int TM, bool WHOLE>
__global__ __launch_bounds__(256) void k_ad_expand(AdArgs a) {
  constexpr int MF = TM / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ uint16_t rows[TM];
  __shared__ int part[8];
  __shared__ __align__(16) uint16_t terms[TM * kAdTermPitch];
  const AdTile at = ad_tile<TM>(a.ids, a.b, a.count, blockIdx.x, rows, part, reinterpret_cast<int*>(smem));
  if (at.rows == 0) return;
  const int cb = (int)blockIdx.y * 256;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 256, a.m);
    return;
  }
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int c0 = cb + 64 * w;
  f32x4 acc[4][MF];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int g = 0; g < MF; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int rank0 = 0; rank0 < a.r; rank0 += kAdRank) {
    __syncthreads();
    ad_terms2<TM>(a.T, a.splits_x, a, at, rows, rank0, terms);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kAdRank; s += 32) {
      if (rank0 + s >= a.r) break;
      bf16x8 t[2][MF];
#pragma unroll
      for (int g = 0; g < MF; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          t[h][g] = *reinterpret_cast<const bf16x8*>(terms + (16 * g + i) * kAdTermPitch + h * kAdRank + s + 8 * q);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int col = min(c0 + 16 * (i >> 2) + 4 * f + (i & 3), a.m - 1);
        const bf16x8 u = as_bf16(load_row8<WHOLE>(a.U + ((int64_t)at.adapter * a.m + col) * a.r, rank0 + s + 8 * q, a.r));
#pragma unroll
        for (int g = 0; g < MF; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, t[h][g], acc[f][g], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < MF; ++g) {
    if (16 * g + i >= at.rows) continue;
    float v[16];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * f + e] = acc[f][g][e];
    ad_store<16>(a, rows[16 * g + i], c0 + 16 * q, a.m, v);
  }
}

// ---------------------------------------------------------------------------
// The backward's second launch: blocks of dX, then of dU, then of dVt.
// ---------------------------------------------------------------------------
// dX = base + scale P Vt: as k_ad_expand, with Vt's 8 x 8 pieces transposed in
// registers: a lane's eight ranks and eight columns are eight operands.  128
// columns a wave.
template <int TM>
__device__ __forceinline__ void ad_dx(const AdArgs& a, int block, char* smem, uint16_t* rows, int* part,
                                      uint16_t* terms) {
  constexpr int MF = TM / 16;
  const AdTile at = ad_tile<TM>(a.ids, a.b, a.count, block / a.cols_y, rows, part, reinterpret_cast<int*>(smem));
  if (at.rows == 0) return;
  const int cb = block % a.cols_y * 512;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 512, a.n);
    return;
  }
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int c0 = cb + 128 * w;
  f32x4 acc[8][MF];
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int g = 0; g < MF; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int rank0 = 0; rank0 < a.r; rank0 += kAdRank) {
    __syncthreads();
    ad_terms2<TM>(a.P, a.splits_g, a, at, rows, rank0, terms);
    __syncthreads();
    for (int s = 0; s < kAdRank && rank0 + s < a.r; s += 32) {
      AdPiece<8> v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int rank = rank0 + s + 8 * q + e;
        if (rank < a.r) v[e] = ad_piece<8>(a.Vt + ((int64_t)at.adapter * a.r + rank) * a.n, c0 + 8 * i, a.n);
        else v[e] = AdPiece<8>{{0u, 0u, 0u, 0u}};
      }
      bf16x8 t[2][MF];
#pragma unroll
      for (int g = 0; g < MF; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          t[h][g] = *reinterpret_cast<const bf16x8*>(terms + (16 * g + i) * kAdTermPitch + h * kAdRank + s + 8 * q);
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const bf16x8 u = as_bf16(ad_column<8>(v, f));
#pragma unroll
        for (int g = 0; g < MF; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, t[h][g], acc[f][g], 0, 0, 0);
      }
    }
  }
  // row 4 q + e of piece f is column 8 (4 q + e) + f
#pragma unroll
  for (int g = 0; g < MF; ++g) {
    if (16 * g + i >= at.rows) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) v[f] = acc[f][g][e];
      ad_store<8>(a, rows[16 * g + i], c0 + 8 * (4 * q + e), a.n, v);
    }
  }
}

// dU_l (m x r) = scale G_l^T T_l, or dVt_l (r x n) = scale P_l^T X_l, for 16 CW
// columns of G or X and 16 NR ranks.  Rows of the adapter 32 at a time, a wave
// each; its G (X) comes as 8 rows x CW columns a lane, transposed in registers,
// its T (P) as three terms through LDS.  The waves' sums are added in order.
static constexpr int kAdStepPitch = 32 + 8;

// What this wave wrote to its part of LDS before is read after (LDS takes a
// wave's accesses in order; this keeps the compiler to it).
__device__ __forceinline__ void ad_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int NR, int CW, bool DV>
__device__ __forceinline__ void ad_dfactor(const AdArgs& a, int block, char* smem, uint16_t* list, int* part) {
  const int cols = DV ? a.n : a.m, blocks = DV ? a.cols_v : a.cols_u;
  const int c0 = block % blocks * 16 * CW, rest = block / blocks;
  const int rank0 = rest % a.chunks * kAdRank, l = rest / a.chunks;
  const int total = ad_collect(a.ids, a.b, a.count, l, 0, kAdRows, list, part);
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const uint16_t* src = DV ? a.X : a.G;
  const float* partial = DV ? a.P : a.T;
  const int splits = DV ? a.splits_g : a.splits_x;
  const float scale = a.scale ? a.scale[l] : 1.f;
  f32x4 acc[CW][NR];
#pragma unroll
  for (int f = 0; f < CW; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint16_t* terms = reinterpret_cast<uint16_t*>(smem) + w * 3 * 16 * kAdStepPitch;  // the wave's: [3][16][kAdStepPitch]
  for (int s = 32 * w; s < total; s += 128) {
    AdPiece<CW> v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (s + 8 * q + e < total) {
        v[e] = ad_piece<CW>(src + (int64_t)list[s + 8 * q + e] * cols, c0 + CW * i, cols);
      } else {
#pragma unroll
        for (int d = 0; d < CW / 2; ++d) v[e].w[d] = 0u;
      }
    }
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      // lane: rank lane % 16 of the group, rows q, q + 4, ..
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int row = 4 * e + q, k = rank0 + 16 * g + i;
        float x = 0.f;
        if (s + row < total && k < a.r) {
          const float* p = partial + (int64_t)list[s + row] * a.ldr + k;
          for (int z = 0; z < splits; ++z) x += p[(int64_t)z * a.b * a.ldr];
          x *= scale;
        }
#pragma unroll
        for (int h = 0; h < 3; ++h) {
          const uint16_t t = f32_to_bf16(x);
          x = (t & 0x7fffu) == 0x7f80u ? 0.f : x - __uint_as_float((uint32_t)t << 16);
          terms[(h * 16 + i) * kAdStepPitch + row] = t;
        }
      }
      ad_wave_sync();
      bf16x8 t[3];
#pragma unroll
      for (int h = 0; h < 3; ++h)
        t[h] = *reinterpret_cast<const bf16x8*>(terms + (h * 16 + i) * kAdStepPitch + 8 * q);
      ad_wave_sync();
#pragma unroll
      for (int f = 0; f < CW; ++f) {
        const bf16x8 x = as_bf16(ad_column<CW>(v, f));
#pragma unroll
        for (int h = 0; h < 3; ++h)
          acc[f][g] = DV ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[h], x, acc[f][g], 0, 0, 0)
                         : __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, t[h], acc[f][g], 0, 0, 0);
      }
    }
  }
  f32x4* sum = reinterpret_cast<f32x4*>(smem);  // [CW NR][64]
#pragma unroll
  for (int other = 1; other < 4; ++other) {
    __syncthreads();
    if (w == other) {
#pragma unroll
      for (int f = 0; f < CW; ++f)
#pragma unroll
        for (int g = 0; g < NR; ++g) sum[(f * NR + g) * 64 + lane] = acc[f][g];
    }
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int f = 0; f < CW; ++f)
#pragma unroll
        for (int g = 0; g < NR; ++g) acc[f][g] += sum[(f * NR + g) * 64 + lane];
    }
  }
  if (w != 0) return;
#pragma unroll
  for (int g = 0; g < NR; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int f = 0; f < CW; ++f) {
        // a lane holds rows 4 q + e, column i of D: columns of G (X) are CW apart
        const int rank = rank0 + 16 * g + (DV ? 4 * q + e : i), col = c0 + CW * (DV ? i : 4 * q + e) + f;
        if (rank < a.r && col < cols) {
          if (DV) a.dVt[((int64_t)l * a.r + rank) * a.n + col] = acc[f][g][e];
          else a.dU[((int64_t)l * a.m + col) * a.r + rank] = acc[f][g][e];
        }
      }
}

template <int TM, int NR, int CW>
__global__ __launch_bounds__(256) void k_ad_back(AdArgs a) {
  extern __shared__ __align__(16) char smem[];
  __shared__ uint16_t rows[kAdRows];
  __shared__ int part[8];
  int block = blockIdx.x;
  if (block < a.blocks_u) {
    ad_dfactor<NR, CW, false>(a, block, smem, rows, part);
    return;
  }
  block -= a.blocks_u;
  if (block < a.blocks_v) {
    ad_dfactor<NR, CW, true>(a, block, smem, rows, part);
    return;
  }
  block -= a.blocks_v;
  // the terms lie behind the bins that ad_tile uses, which it is done with then
  ad_dx<TM>(a, block, smem, rows, part, reinterpret_cast<uint16_t*>(smem));
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct AdPlan {
  int tm, tiles, splits_x, splits_g, units_x, units_g, ldr, chunks;
  size_t t_bytes, p_bytes;
};

static void ad_split(int K, int blocks, int* splits, int* per) {
  const int units = (K + kAdUnit - 1) / kAdUnit;
  const int want = std::max(1, std::min(units, kAdBlocks / std::max(1, blocks)));
  *per = (units + want - 1) / want;
  *splits = (units + *per - 1) / *per;
}

static AdPlan ad_plan(const hss_adapters* A, int b, bool grad) {
  AdPlan p;
  p.tm = b <= kAdSmall ? 16 : 32;
  p.tiles = b <= kAdSmall ? b : b / p.tm + std::min(b, A->count + 1);
  p.ldr = (A->r + 15) / 16 * 16;
  p.chunks = (A->r + kAdRank - 1) / kAdRank;
  // tiles with rows: between those of one adapter and one for each row
  const int busy = std::max((b + p.tm - 1) / p.tm, std::min(b, A->count)) * p.chunks * (grad ? 2 : 1);
  ad_split(A->n, busy, &p.splits_x, &p.units_x);
  ad_split(A->m, busy, &p.splits_g, &p.units_g);
  const size_t one = (size_t)b * p.ldr * 4;
  p.t_bytes = (p.splits_x * one + 255) / 256 * 256;
  p.p_bytes = grad ? p.splits_g * one : 0;
  return p;
}

size_t adapters_ws_bytes(const hss_adapters* A, int b, bool grad) {
  const AdPlan p = ad_plan(A, b, grad);
  return p.t_bytes + p.p_bytes;
}

// The most that a batch of up to b rows needs.
size_t adapters_ws_bytes_up_to(const hss_adapters* A, int b, bool grad) {
  size_t most = 0;
  for (int c = 1; c <= b; ++c) most = std::max(most, adapters_ws_bytes(A, c, grad));
  return most;
}

static AdArgs ad_args(const hss_adapters* A, int b, const AdPlan& p, const void* X, const int32_t* ids,
                      const void* base, void* Y, void* ws) {
  AdArgs a = {};
  a.U = static_cast<const uint16_t*>(A->U), a.Vt = static_cast<const uint16_t*>(A->Vt), a.scale = A->scale;
  a.ids = ids, a.X = static_cast<const uint16_t*>(X), a.base = static_cast<const uint16_t*>(base);
  a.Y = static_cast<uint16_t*>(Y);
  a.T = static_cast<float*>(ws), a.P = reinterpret_cast<float*>(static_cast<char*>(ws) + p.t_bytes);
  a.m = A->m, a.n = A->n, a.r = A->r, a.count = A->count, a.b = b;
  a.ldr = p.ldr, a.tiles = p.tiles, a.chunks = p.chunks;
  a.splits_x = p.splits_x, a.units_x = p.units_x;
  return a;
}

template <int TM, int NR>
static void launch_rank_nr(const AdArgs& a, int chunks, bool whole, hipStream_t s) {
  size_t lds = std::max<size_t>((size_t)4 * (TM / 16) * NR * 64 * 16, (size_t)(a.count + 1) * 4);
  if (a.splits_g) lds = std::max<size_t>(lds, (size_t)16 * NR * kAdPitch * 2);
  const dim3 grid(a.tiles, a.splits_x + a.splits_g, chunks);
  if (whole) hipLaunchKernelGGL((k_ad_rank<TM, NR, true>), grid, dim3(256), lds, s, a);
  else hipLaunchKernelGGL((k_ad_rank<TM, NR, false>), grid, dim3(256), lds, s, a);
}

template <int TM>
static void launch_rank(const AdArgs& a, hipStream_t s) {
  const bool whole = (!a.splits_x || a.n % 8 == 0) && (!a.splits_g || a.m % 8 == 0);
  if (a.r <= 16) launch_rank_nr<TM, 1>(a, a.chunks, whole, s);
  else if (a.r <= 32) launch_rank_nr<TM, 2>(a, a.chunks, whole, s);
  else launch_rank_nr<TM, 4>(a, a.chunks, whole, s);
}

template <int TM>
static void launch_expand(const AdArgs& a, hipStream_t s) {
  const dim3 grid(a.tiles, (a.m + 255) / 256);
  const size_t lds = (size_t)(a.count + 1) * 4;
  if (a.r % 8 == 0) hipLaunchKernelGGL((k_ad_expand<TM, true>), grid, dim3(256), lds, s, a);
  else hipLaunchKernelGGL((k_ad_expand<TM, false>), grid, dim3(256), lds, s, a);
}

hss_status launch_adapters_apply(const hss_adapters* A, int b, const void* X, const int32_t* ids, const void* base,
                                 void* Y, void* ws, hipStream_t s) {
  const AdPlan p = ad_plan(A, b, false);
  const AdArgs a = ad_args(A, b, p, X, ids, base, Y, ws);
  if (p.tm == 16) launch_rank<16>(a, s), launch_expand<16>(a, s);
  else launch_rank<32>(a, s), launch_expand<32>(a, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

template <int TM, int NR, int CW>
static void launch_back_cw(AdArgs a, hipStream_t s) {
  size_t lds = (size_t)std::max(4 * 3 * 16 * kAdStepPitch * 2, CW * NR * 64 * 16);
  if (a.Y) lds = std::max<size_t>(lds, std::max<size_t>((size_t)(a.count + 1) * 4, (size_t)TM * kAdTermPitch * 2));
  a.cols_u = (a.m + 16 * CW - 1) / (16 * CW), a.cols_v = (a.n + 16 * CW - 1) / (16 * CW);
  a.cols_y = (a.n + 511) / 512;
  a.blocks_u = a.dU ? a.cols_u * a.chunks * a.count : 0;
  a.blocks_v = a.dVt ? a.cols_v * a.chunks * a.count : 0;
  a.blocks_y = a.Y ? a.cols_y * a.tiles : 0;
  const dim3 grid(a.blocks_u + a.blocks_v + a.blocks_y);
  hipLaunchKernelGGL((k_ad_back<TM, NR, CW>), grid, dim3(256), lds, s, a);
}

template <int TM>
static void launch_back(const AdArgs& a, hipStream_t s) {
  // few blocks of dU and dVt: narrower ones
  const int64_t wide = (int64_t)a.count * a.chunks * (a.m + a.n) / 128;
  if (a.r <= 16) wide < 256 ? launch_back_cw<TM, 1, 2>(a, s) : launch_back_cw<TM, 1, 8>(a, s);
  else if (a.r <= 32) wide < 256 ? launch_back_cw<TM, 2, 2>(a, s) : launch_back_cw<TM, 2, 8>(a, s);
  else wide < 256 ? launch_back_cw<TM, 4, 2>(a, s) : launch_back_cw<TM, 4, 8>(a, s);
}

hss_status launch_adapters_grad(const hss_adapters* A, int b, const void* X, const void* G, const int32_t* ids,
                                const void* base, void* dX, float* dU, float* dVt, void* ws, hipStream_t s) {
  if (!dX && !dU && !dVt) return HSS_OK;
  const AdPlan p = ad_plan(A, b, true);
  AdArgs a = ad_args(A, b, p, X, ids, base, dX, ws);
  a.G = static_cast<const uint16_t*>(G), a.dU = dU, a.dVt = dVt;
  a.splits_g = dX || dVt ? p.splits_g : 0, a.units_g = p.units_g;
  if (!dU) a.splits_x = 0;
  if (p.tm == 16) launch_rank<16>(a, s), launch_back<16>(a, s);
  else launch_rank<32>(a, s), launch_back<32>(a, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
