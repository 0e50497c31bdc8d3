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
// Forward: two launches.  k_ad_rank makes T, K split over blocks into partial sums in
// fp32, for a few tiles would not fill the chip, and k_ad_expand adds the splits in
// order on its way to the matrix cores.  Backward: k_ad_rank makes T and P,
// k_ad_terms adds the splits once for all that read them, k_ad_back makes dU, dVt and
// dX.  T and P, times scale in fp32, go to the matrix cores as bf16 terms: two (16
// significant bits) where the result is rounded to bf16 anyway, three (24 bits)
// for the fp32 gradients.
#include <algorithm>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

static constexpr int kAdSmall = 64;     // batches up to here: tiles found by one ballot
static constexpr int kAdUnit = 64;      // columns of K that a wave takes at a time: a cache line of each row
static constexpr int kAdBlocks = 768;   // blocks of k_ad_rank that K is split for
static constexpr int kAdChunk = 256;    // ranks of T that k_ad_expand keeps in LDS

struct AdArgs {
  const uint16_t* U;
  const uint16_t* Vt;
  const float* scale;
  const int32_t* ids;
  const uint16_t* X;
  const uint16_t* G;
  const uint16_t* base;
  uint16_t* Y;      // forward: Y; backward: dX
  float* dU;
  float* dVt;
  // Workspace.  A tile's rows have the slots TM tile .. TM tile + rows - 1.
  float* part[2];   // partial sums of T and P: [split][slots][rg]
  uint16_t* t2;     // two terms of P: [slots][2][rp], zeros past r; null = none
  uint16_t* t3[2];  // three terms of T and P: [3][rg][slots]; null = none
  int2* info;       // [tiles]: adapter (-1: none) and rows (0: no such tile)
  uint16_t* rows;   // [slots]
  int2* first;      // [count]: an adapter's first tile and its rows (more than kAdSmall rows)
  int m, n, r, count, b;
  int rp, rg;       // r rounded up to 32 and to 16
  int slots, tiles;
  int splits[2], units[2];           // K splits of T and P (0: not wanted), units of each
  int blocks_u, blocks_v;            // of k_ad_back
  int cols_y, cols_u, cols_v;        // column blocks of dX, dU, dVt
  int chunks;                        // passes of dU and dVt over the ranks
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

// Tile `tile` of the batch: its adapter and its rows (in LDS).  Up to 64 rows
// tile t starts at row t, if that is the first, or TM rows after the last start,
// of its adapter; beyond, tiles are counted through the adapters, rows without one
// last.  bins: count + 1 ints; part: 6.  table: null, or where each adapter's
// first tile and rows go.
template <int TM>
__device__ __forceinline__ AdTile ad_tile(const AdArgs& a, int tile, uint16_t* rows, int* part, int* bins, int2* table) {
  AdTile r = {-1, 0};
  const int t = threadIdx.x, b = a.b, count = a.count;
  if (b <= kAdSmall) {
    const int lane = t & 63;
    const int id = lane < b ? ad_id(a.ids, lane, count) : -2;
    const int own = __builtin_amdgcn_readlane(id, tile);
    const uint64_t same = __ballot(id == own);
    const int before = __popcll(same & ((1ull << tile) - 1));
    if (before % TM) return r;
    const int rank = __popcll(same & lanemask_lt()) - before;
    if (t < 64 && id == own && rank >= 0 && rank < TM) rows[rank] = (uint16_t)lane;
    __syncthreads();
    r.adapter = own;
    r.rows = min(TM, __popcll(same) - before);
    return r;
  }
  constexpr int per = HSS_MAX_BATCH / 256;
  int id[per];
#pragma unroll
  for (int k = 0; k < per; ++k) {
    id[k] = per * t + k < b ? ad_id(a.ids, per * t + k, count) : -2;
    if (id[k] == -1) id[k] = count;
  }
  for (int k = t; k <= count; k += 256) bins[k] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < per; ++k) {  // lanes of one adapter's rows add once
    const int head = __builtin_amdgcn_readfirstlane(id[k]);
    const uint64_t same = __ballot(id[k] == head);
    if (id[k] == head) {
      if (head >= 0 && __popcll(same & lanemask_lt()) == 0) atomicAdd(&bins[head], __popcll(same));
    } else if (id[k] >= 0) {
      atomicAdd(&bins[id[k]], 1);
    }
  }
  __syncthreads();
  const int many = (count + 256) / 256, k0 = t * many;
  int own = 0, total;
  for (int k = k0; k < min(k0 + many, count + 1); ++k) own += (bins[k] + TM - 1) / TM;
  int at = ad_scan(own, part, &total);
  if (table) {
    int next = at;
    for (int k = k0; k < min(k0 + many, count); ++k) {
      table[k] = make_int2(next, bins[k]);
      next += (bins[k] + TM - 1) / TM;
    }
  }
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
  int mine = 0;
#pragma unroll
  for (int k = 0; k < per; ++k) mine += id[k] == bin;
  int rank = ad_scan(mine, part, &total) - first;
#pragma unroll
  for (int k = 0; k < per; ++k)
    if (id[k] == bin) {
      if (rank >= 0 && rank < TM) rows[rank] = (uint16_t)(per * t + k);
      ++rank;
    }
  __syncthreads();
  return r;
}

// ---------------------------------------------------------------------------
// 8 x 8 transposition: eight rows of CW bf16 (v[e], column f) into operand f =
// the eight rows' values of column f, two of them a dword.
// ---------------------------------------------------------------------------
template <int CW>
struct AdPiece {  // CW bf16 of a row
  uint32_t w[CW / 2];
};

template <int CW>
__device__ __forceinline__ u32x4 ad_column(const AdPiece<CW> (&v)[8], int f) {
  u32x4 o;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    o[d] = __builtin_amdgcn_perm(v[2 * d + 1].w[f >> 1], v[2 * d].w[f >> 1], f & 1 ? 0x07060302u : 0x05040100u);
  return o;
}

// CW bf16 at any 2-byte aligned address.
template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_piece(const uint16_t* at) {
  struct __attribute__((packed, aligned(2))) Raw {
    uint32_t w[CW / 2];
  };
  const Raw raw = *reinterpret_cast<const Raw*>(at);
  AdPiece<CW> p;
#pragma unroll
  for (int d = 0; d < CW / 2; ++d) p.w[d] = raw.w[d];
  return p;
}

// The first `left` of them, zeros behind: the slow way, for ends.
template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_piece_end(const uint16_t* at, int left) {
  AdPiece<CW> p;
#pragma unroll
  for (int d = 0; d < CW / 2; ++d) {
    const uint32_t lo = 2 * d < left ? at[2 * d] : 0u, hi = 2 * d + 1 < left ? at[2 * d + 1] : 0u;
    p.w[d] = lo | hi << 16;
  }
  return p;
}

// What this wave wrote to its part of LDS before is read after (LDS takes a
// wave's accesses in order; this keeps the compiler to it).
__device__ __forceinline__ void ad_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The next bf16 term of x, which loses it (an infinity leaves 0, not the NaN of
// inf - inf).
__device__ __forceinline__ uint32_t ad_term(float& x) {
  const uint32_t t = f32_to_bf16(x);
  x = (t & 0x7fffu) == 0x7f80u ? 0.f : x - __uint_as_float(t << 16);
  return t;
}

// ---------------------------------------------------------------------------
// T = X Vt^T and P = G U, partial sums over a block's part of K; the blocks of split
// 0 also write the table of tiles.
//   D[rank][row] += A[rank][k] B[row][k]: A = Vt_l as stored, or U_l transposed
//   through the wave's part of LDS.  Wave w takes units w, w + 4, .. of the block's;
//   the next one's loads are in flight while one is multiplied.  The four waves'
//   sums meet in LDS.
// grid: (splits of T and of P, tiles, groups of 16 NR ranks)
// ---------------------------------------------------------------------------
static constexpr int kAdPitch = kAdUnit + 8;  // of U^T in LDS

template <int TM, int NR>
__global__ __launch_bounds__(256, NR == 4 ? 3 : 4) void k_ad_rank(AdArgs a) {
  constexpr int MF = TM / 16;
  extern __shared__ __align__(16) char smem[];
  __shared__ uint16_t rows[TM];
  __shared__ int part[6];
  const int tile = blockIdx.y, rank0 = (int)blockIdx.z * 16 * NR;
  const int side = (int)blockIdx.x >= a.splits[0];
  const int z = (int)blockIdx.x - (side ? a.splits[0] : 0);
  const bool lead = blockIdx.x == 0 && blockIdx.z == 0;
  const AdTile at = ad_tile<TM>(a, tile, rows, part, reinterpret_cast<int*>(smem), lead && tile == 0 ? a.first : nullptr);
  if (lead) {
    if (threadIdx.x == 0) a.info[tile] = make_int2(at.adapter, at.rows);
    if ((int)threadIdx.x < at.rows) a.rows[TM * tile + threadIdx.x] = rows[threadIdx.x];
  }
  if (at.rows == 0 || at.adapter < 0) return;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int K = side ? a.m : a.n;
  const int u0 = z * a.units[side], u1 = min(u0 + a.units[side], (K + kAdUnit - 1) / kAdUnit);
  const uint16_t* xrow[MF];
#pragma unroll
  for (int f = 0; f < MF; ++f)
    xrow[f] = (side ? a.G : a.X) + (int64_t)rows[min(16 * f + i, at.rows - 1)] * K;

  f32x4 acc[MF][NR];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int whole = min(u1, K / kAdUnit);  // units before here end inside the row
  if (!side) {
    const uint16_t* vrow[NR];
#pragma unroll
    for (int g = 0; g < NR; ++g)
      vrow[g] = a.Vt + ((int64_t)at.adapter * a.r + min(rank0 + 16 * g + i, a.r - 1)) * K;
    struct Regs {
      u32x4 x[2][MF], v[2][NR];
    };
    auto load = [&](int u, Regs& r) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = u * kAdUnit + 32 * h + 8 * q;
#pragma unroll
        for (int f = 0; f < MF; ++f) r.x[h][f] = load8(xrow[f] + k);
#pragma unroll
        for (int g = 0; g < NR; ++g) r.v[h][g] = load8(vrow[g] + k);
      }
    };
    auto multiply = [&](const Regs& r) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < MF; ++f)
#pragma unroll
          for (int g = 0; g < NR; ++g)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(r.v[h][g]), as_bf16(r.x[h][f]), acc[f][g], 0, 0, 0);
    };
    int u = u0 + w;
    if (u < whole) {
      Regs ra, rb;
      load(u, ra);
      for (; u + 4 < whole; u += 8) {
        load(u + 4, rb);
        __builtin_amdgcn_sched_barrier(0);  // the loads first: the compiler would sink them
        multiply(ra);
        load(min(u + 8, whole - 1), ra);
        __builtin_amdgcn_sched_barrier(0);
        multiply(rb);
      }
      if (u < whole) multiply(ra), u += 4;
    }
    if (u < u1) {  // the unit in which the rows end
      Regs re;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = u * kAdUnit + 32 * h + 8 * q;
#pragma unroll
        for (int f = 0; f < MF; ++f) re.x[h][f] = load_row8(xrow[f], k, K);
#pragma unroll
        for (int g = 0; g < NR; ++g) re.v[h][g] = load_row8(vrow[g], k, K);
      }
      multiply(re);
    }
  } else {
    uint16_t* ut = reinterpret_cast<uint16_t*>(smem) + w * 16 * NR * kAdPitch;  // the wave's: [16 NR][kAdPitch]
    // 8 x 8 pieces, one a lane: 8 of the unit's j times 2 NR of the ranks.  A piece
    // in which the ranks end holds the next row's first values (its ranks are not
    // stored), so the factors' last rows are read the slow way.
    const int kb = lane % (2 * NR), jb = lane / (2 * NR), rank = min(rank0 + 8 * kb, (a.r - 1) & ~7);
    const uint16_t* U = a.U + (int64_t)at.adapter * a.m * a.r + rank;
    const bool over = (a.r & 7) != 0 && at.adapter == a.count - 1;
    const int safe = over ? min(whole, (K - 8) / kAdUnit) : whole;
    AdPiece<8> v[8];
    auto load_x = [&](int u, u32x4 (&x)[2][MF]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < MF; ++f) x[h][f] = load8(xrow[f] + u * kAdUnit + 32 * h + 8 * q);
    };
    auto load_v = [&](int u) {
      if (jb < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ad_piece<8>(U + (int64_t)(u * kAdUnit + 8 * jb + e) * a.r);
      }
    };
    auto put = [&]() {
      if (jb < 8) {
#pragma unroll
        for (int f = 0; f < 8; ++f) *reinterpret_cast<u32x4*>(ut + (8 * kb + f) * kAdPitch + 8 * jb) = ad_column<8>(v, f);
      }
      ad_wave_sync();
    };
    auto multiply = [&](const u32x4 (&x)[2][MF]) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int g = 0; g < NR; ++g) {
          const u32x4 t = *reinterpret_cast<const u32x4*>(ut + (16 * g + i) * kAdPitch + 32 * h + 8 * q);
#pragma unroll
          for (int f = 0; f < MF; ++f)
            acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t), as_bf16(x[h][f]), acc[f][g], 0, 0, 0);
        }
      ad_wave_sync();
    };
    int u = u0 + w;
    if (u < safe) {
      u32x4 xa[2][MF], xb[2][MF];
      load_v(u), load_x(u, xa);
      for (; u + 4 < safe; u += 8) {
        put();
        load_v(u + 4), load_x(u + 4, xb);
        multiply(xa);
        put();
        const int next = min(u + 8, safe - 1);
        load_v(next), load_x(next, xa);
        multiply(xb);
      }
      if (u < safe) put(), multiply(xa), u += 4;
    }
    for (; u < u1; u += 4) {
      u32x4 x[2][MF];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < MF; ++f) x[h][f] = load_row8(xrow[f], u * kAdUnit + 32 * h + 8 * q, K);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = u * kAdUnit + 8 * jb + e;
        v[e] = ad_piece_end<8>(U + (int64_t)min(j, K - 1) * a.r, jb < 8 && j < K ? a.r - rank : 0);
      }
      put();
      multiply(x);
    }
  }

  f32x4* sum = reinterpret_cast<f32x4*>(smem);  // [4][MF NR][64]
  __syncthreads();
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) sum[(w * MF * NR + f * NR + g) * 64 + lane] = acc[f][g];
  __syncthreads();
  float* out = a.part[side] + ((int64_t)z * a.slots + TM * tile) * a.rg;
#pragma unroll
  for (int c = w; c < MF * NR; c += 4) {
    const int f = c / NR, g = c % NR;
    f32x4 v = sum[c * 64 + lane];
#pragma unroll
    for (int k = 1; k < 4; ++k) v += sum[(k * MF * NR + c) * 64 + lane];
    const int rank = rank0 + 16 * g + 4 * q;  // .. rank + 3 of row 16 f + i
    if (16 * f + i < at.rows && rank < a.rg) *reinterpret_cast<f32x4*>(out + (16 * f + i) * a.rg + rank) = v;
  }
}

// The splits' sum of N values at p, added in order; 8 loads in flight.
template <typename V>
__device__ __forceinline__ V ad_sum(const float* p, int splits, int64_t stride) {
  V s = *reinterpret_cast<const V*>(p);
  int z = 1;
  for (; z + 8 <= splits; z += 8) {
    V v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const V*>(p + (z + k) * stride);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  if (z < splits) {
    V v[7];
#pragma unroll
    for (int k = 0; k < 7; ++k) v[k] = *reinterpret_cast<const V*>(p + min(z + k, splits - 1) * stride);
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (z + k < splits) s += v[k];
  }
  return s;
}

// ---------------------------------------------------------------------------
// Backward: the terms of T and P.  A lane has one rank of eight slots.
// grid: (tiles, ranks / 64, sides)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_ad_terms(AdArgs a) {
  const int tile = blockIdx.x, side = a.splits[0] == 0 ? 1 : (int)blockIdx.z;
  const int2 at = a.info[tile];
  if (at.x < 0 || at.y == 0) return;
  const int rank = (int)blockIdx.y * 64 + (threadIdx.x & 63), i0 = 8 * (threadIdx.x >> 6);
  if (rank >= a.rp) return;
  const float scale = a.scale ? a.scale[at.x] : 1.f;
  const int splits = a.splits[side];
  const int64_t stride = (int64_t)a.slots * a.rg;
  const float* p = a.part[side] + (int64_t)(32 * tile + i0) * a.rg + min(rank, a.rg - 1);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int z = 0; z < splits; ++z)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += p[z * stride + e * a.rg];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = rank < a.r && i0 + e < at.y ? v[e] * scale : 0.f;  // a slot without a row holds anything
  uint16_t* three = a.t3[side];
#pragma unroll
  for (int h = 0; h < 3; ++h) {
    uint32_t t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = ad_term(v[e]);
    if (three && rank < a.rg)
      *reinterpret_cast<u32x4*>(three + ((int64_t)h * a.rg + rank) * a.slots + 32 * tile + i0) =
          u32x4{t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16};
    if (a.t2 && side && h < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) a.t2[((int64_t)(32 * tile + i0 + e) * 2 + h) * a.rp + rank] = (uint16_t)t[e];
    }
  }
}

// ---------------------------------------------------------------------------
// Outputs in bf16
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t ad_pack(float lo, float hi) { return f32_to_bf16(lo) | (uint32_t)f32_to_bf16(hi) << 16; }

// Eight values in bf16: old + v.
__device__ __forceinline__ void ad_store8_on(uint16_t* out, const Bytes16& old, const float* v) {
  Bytes16 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) o.w[k] = ad_pack(v[2 * k] + bf16lo(old.w[k]), v[2 * k + 1] + bf16hi(old.w[k]));
  *reinterpret_cast<Bytes16*>(out) = o;
}

// Eight columns of a row of the output: base + v, in bf16.
__device__ __forceinline__ void ad_store8(const AdArgs& a, int64_t row, int col, int cols, const float* v) {
  const uint16_t* in = a.base ? a.base + row * cols : nullptr;
  uint16_t* out = a.Y + row * cols;
  if (col + 8 <= cols) {
    Bytes16 old = {{0u, 0u, 0u, 0u}};
    if (in) old = *reinterpret_cast<const Bytes16*>(in + col);
    ad_store8_on(out + col, old, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (col + k < cols) out[col + k] = f32_to_bf16((in ? __uint_as_float((uint32_t)in[col + k] << 16) : 0.f) + v[k]);
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
// column 32 (f / 2) + 8 (i / 4) + 4 (f % 2) + i % 4 of the wave's 64, so that a
// lane ends up with two runs of eight columns of one row, and four lanes with 64
// adjacent bytes.
// The block's terms of T are made first, in LDS, for all its columns.
// grid: (tiles, column blocks of 256 NC)
// ---------------------------------------------------------------------------
// Eight ranks from k on of a row of r, zeros past r (what lies there is the next
// row's).  `inside`: the 16 bytes are inside the factors.
__device__ __forceinline__ u32x4 ad_ranks(const uint16_t* row, int k, int r, bool inside) {
  if (inside) {
    u32x4 v = load8(row + min(k, (r - 1) & ~7));
    const int keep = r - k;
    if (__builtin_amdgcn_ballot_w64(keep < 8)) {
#pragma unroll
      for (int d = 0; d < 4; ++d) v[d] &= (keep > 2 * d ? 0xffffu : 0u) | (keep > 2 * d + 1 ? 0xffff0000u : 0u);
    }
    return v;
  }
  return __builtin_bit_cast(u32x4, ad_piece_end<8>(row + min(k, r - 1), r - k));
}

template <int TM>
__global__ __launch_bounds__(256) void k_ad_expand(AdArgs a, int nc) {
  constexpr int MF = TM / 16;
  extern __shared__ __align__(16) uint16_t terms[];  // [TM][2][ranks of a chunk, + 4]
  const int tile = blockIdx.x, cb = (int)blockIdx.y * 256 * nc;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int2 info = a.info[tile];
  const uint16_t* rows = a.rows + TM * tile;
  int64_t out[MF];  // (of a tile that is not there: any number, not used)
#pragma unroll
  for (int g = 0; g < MF; ++g) out[g] = rows[16 * g + i];
  const AdTile at = {info.x, info.y};
  if (at.rows == 0) return;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 256 * nc, a.m);
    return;
  }
  const int wide = min(a.rp, kAdChunk), pitch = 2 * wide + 8;
  const float scale = a.scale ? a.scale[at.adapter] : 1.f;
  auto fill = [&](int rank0) {  // two terms of a chunk's ranks, zeros past r
    const int quads = min(wide, a.rp - rank0) / 4;
    const float* p = a.part[0] + (int64_t)TM * tile * a.rg + rank0;
    for (int e = threadIdx.x; e < at.rows * quads; e += 256) {
      const int row = e / quads, k = e % quads * 4;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
      if (rank0 + k < a.rg) v = ad_sum<f32x4>(p + row * a.rg + k, a.splits[0], (int64_t)a.slots * a.rg);
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = rank0 + k + c < a.r ? v[c] * scale : 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t t[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) t[c] = ad_term(x[c]);
        *reinterpret_cast<mx_u32x2*>(terms + row * pitch + h * wide + k) = mx_u32x2{t[0] | t[1] << 16, t[2] | t[3] << 16};
      }
    }
  };
  const uint16_t* trow[MF];
#pragma unroll
  for (int g = 0; g < MF; ++g) trow[g] = terms + min(16 * g + i, at.rows - 1) * pitch + 8 * q;
  const int64_t end = (int64_t)a.count * a.m * a.r;
  const bool one = a.rp <= kAdChunk;
  bool filled = false;
  for (int c0 = cb + 64 * w; c0 < cb + 256 * nc; c0 += 256) {
    const uint16_t* urow[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
      urow[f] = a.U + ((int64_t)at.adapter * a.m + min(c0 + 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3), a.m - 1)) * a.r;
    const bool inside = ((int64_t)at.adapter * a.m + min(c0 + 64, a.m)) * a.r + 8 <= end;
    const bool full = c0 + 64 <= a.m && a.base;
    // the first ranks of U and the rows' base are on their way while the terms are made
    u32x4 u[4];
    Bytes16 old[MF][2];
#pragma unroll
    for (int f = 0; f < 4; ++f) u[f] = ad_ranks(urow[f], 8 * q, a.r, inside);
    if (full) {
#pragma unroll
      for (int g = 0; g < MF; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (16 * g + i < at.rows)
            old[g][h] = *reinterpret_cast<const Bytes16*>(a.base + out[g] * a.m + c0 + 32 * h + 8 * q);
    }
    f32x4 acc[4][MF];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int g = 0; g < MF; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int rank0 = 0; rank0 < a.rp; rank0 += kAdChunk) {
      if (!one || !filled) {  // every wave comes here as often
        __syncthreads();
        fill(rank0);
        __syncthreads();
        filled = true;
      }
      for (int s = 0; s < min(wide, a.rp - rank0); s += 32) {
        u32x4 t[2][MF];
#pragma unroll
        for (int g = 0; g < MF; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) t[h][g] = *reinterpret_cast<const u32x4*>(trow[g] + h * wide + s);
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int g = 0; g < MF; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(u[f]), as_bf16(t[h][g]), acc[f][g], 0, 0, 0);
        if (rank0 + s + 32 < a.rp) {
#pragma unroll
          for (int f = 0; f < 4; ++f) u[f] = ad_ranks(urow[f], rank0 + s + 32 + 8 * q, a.r, inside);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < MF; ++g) {
      if (16 * g + i >= at.rows) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = acc[2 * h + (k >> 2)][g][k & 3];
        const int col = c0 + 32 * h + 8 * q;
        if (full) ad_store8_on(a.Y + out[g] * a.m + col, old[g][h], v);
        else ad_store8(a, out[g], col, a.m, v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The backward's last launch: blocks of dU, then of dVt, then of dX.
// ---------------------------------------------------------------------------
// dX = base + scale P Vt: as k_ad_expand, with Vt's 8 x 8 pieces transposed in
// registers: a lane's eight ranks and eight columns are eight operands.  128
// columns a wave; row i of each operand is the run of eight columns i / 4 + 4 (i %
// 4), so that four lanes store 64 adjacent bytes.
__device__ __forceinline__ void ad_dx(const AdArgs& a, int block) {
  constexpr int MF = 2;
  const int tile = block / a.cols_y, cb = block % a.cols_y * 512;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int2 info = a.info[tile];
  const uint16_t* rows = a.rows + 32 * tile;
  const uint16_t* trow[MF];
  int64_t out[MF];  // (of a tile that is not there: any number, not used)
#pragma unroll
  for (int g = 0; g < MF; ++g) {
    out[g] = rows[16 * g + i];
    trow[g] = a.t2 + (int64_t)(32 * tile + 16 * g + i) * 2 * a.rp + 8 * q;
  }
  const AdTile at = {info.x, info.y};
  if (at.rows == 0) return;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 512, a.n);
    return;
  }
  const int c0 = cb + 128 * w, col = c0 + 8 * ((i >> 2) + 4 * (i & 3));
  if (c0 >= a.n) return;
  const uint16_t* V = a.Vt + (int64_t)at.adapter * a.r * a.n + col;
  const bool inside = c0 + 128 <= a.n, full = inside && a.base;
  Bytes16 old[MF][4];
  if (full) {
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (16 * g + i < at.rows) old[g][e] = *reinterpret_cast<const Bytes16*>(a.base + out[g] * a.n + c0 + 8 * (q + 4 * e));
  }
  f32x4 acc[8][MF];
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int g = 0; g < MF; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.rp; s += 32) {
    // past the ranks: the last one again, times the zeros that the terms hold there
    AdPiece<8> v[8];
    if (inside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ad_piece<8>(V + (int64_t)min(s + 8 * q + e, a.r - 1) * a.n);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = ad_piece_end<8>(V + (int64_t)min(s + 8 * q + e, a.r - 1) * a.n, a.n - col);
    }
    u32x4 t[2][MF];
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) t[h][g] = *reinterpret_cast<const u32x4*>(trow[g] + h * a.rp + s);
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const bf16x8 u = as_bf16(ad_column<8>(v, f));
#pragma unroll
      for (int g = 0; g < MF; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, as_bf16(t[h][g]), acc[f][g], 0, 0, 0);
    }
  }
#pragma unroll
  for (int g = 0; g < MF; ++g) {
    if (16 * g + i >= at.rows) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) v[f] = acc[f][g][e];
      if (full) ad_store8_on(a.Y + out[g] * a.n + c0 + 8 * (q + 4 * e), old[g][e], v);
      else ad_store8(a, out[g], c0 + 8 * (q + 4 * e), a.n, v);
    }
  }
}

// dU_l (m x r) = scale G_l^T T_l, or dVt_l (r x n) = scale P_l^T X_l, for 16 CW
// columns of G or X and 16 NR ranks.  Rows of the adapter 32 at a time (a tile),
// a wave each; its G (X) comes as 8 rows x CW columns a lane, transposed in
// registers, its T (P) as the three terms that k_ad_terms left.  The waves' sums are
// added in order.
template <int NR, int CW, bool DV>
__device__ __forceinline__ void ad_dfactor(const AdArgs& a, int block, char* smem) {
  const int cols = DV ? a.n : a.m, blocks = DV ? a.cols_v : a.cols_u;
  const int c0 = block % blocks * 16 * CW, rest = block / blocks;
  const int rank0 = rest % a.chunks * 16 * NR, l = rest / a.chunks;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  int total, tile0 = 0;
  const uint16_t* list = a.rows;  // the adapter's rows, 32 of a tile
  uint64_t same = 0;
  if (a.b > kAdSmall) {
    const int2 first = a.first[l];
    tile0 = first.x, total = first.y;
  } else {  // a tile starts at each 32nd of its rows
    same = __ballot(lane < a.b && a.ids[min(lane, a.b - 1)] == l);
    total = __popcll(same);
  }
  const uint16_t* src = DV ? a.X : a.G;
  const uint16_t* terms[NR];
#pragma unroll
  for (int g = 0; g < NR; ++g)
    terms[g] = a.t3[DV] + (int64_t)min(rank0 + 16 * g + i, a.rg - 1) * a.slots + 8 * q;
  const int64_t term = (int64_t)a.rg * a.slots;
  f32x4 acc[CW][NR];
#pragma unroll
  for (int f = 0; f < CW; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Rows past the end: a row of the tile again, times the zeros that the terms
  // hold there.
  const bool inside = c0 + 16 * CW <= cols;
  const uint16_t* at = src + c0 + CW * i;
  auto tile_of = [&](int s) {
    if (a.b > kAdSmall) return tile0 + s;
    uint64_t rest = same;
    for (int k = 0; k < 32 * s; ++k) rest &= rest - 1;
    return __ffsll((unsigned long long)rest) - 1;
  };
  struct Regs {
    AdPiece<CW> v[8];
    u32x4 t[NR <= 2 ? NR : 1][3];
  };
  auto load_terms = [&](int pos, int g, u32x4 (&t)[3]) {
#pragma unroll
    for (int h = 0; h < 3; ++h) t[h] = *reinterpret_cast<const u32x4*>(terms[g] + h * term + pos);
  };
  auto load = [&](int s, Regs& r) {
    const int pos = 32 * tile_of(s), left = total - 32 * s;
    if (NR <= 2) {
#pragma unroll
      for (int g = 0; g < NR; ++g) load_terms(pos, g, r.t[g]);
    }
    int64_t row[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) row[e] = (int64_t)list[pos + min(8 * q + e, left - 1)] * cols;
    if (inside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_piece<CW>(at + row[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_piece_end<CW>(at + row[e], cols - (c0 + CW * i));
    }
  };
  auto multiply = [&](int s, const Regs& r) {
    const int pos = 32 * tile_of(s);
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      u32x4 t[3];
      if (NR <= 2) {
#pragma unroll
        for (int h = 0; h < 3; ++h) t[h] = r.t[g][h];
      } else {
        load_terms(pos, g, t);
      }
#pragma unroll
      for (int f = 0; f < CW; ++f) {
        const bf16x8 x = as_bf16(ad_column<CW>(r.v, f));
#pragma unroll
        for (int h = 0; h < 3; ++h)
          acc[f][g] = DV ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t[h]), x, acc[f][g], 0, 0, 0)
                         : __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, as_bf16(t[h]), acc[f][g], 0, 0, 0);
      }
    }
  };
  const int steps = (total + 31) / 32;
  int s = w;
  if (s < steps) {
    Regs ra, rb;
    load(s, ra);
    for (; s + 4 < steps; s += 8) {
      load(s + 4, rb);
      __builtin_amdgcn_sched_barrier(0);
      multiply(s, ra);
      load(min(s + 8, steps - 1), ra);
      __builtin_amdgcn_sched_barrier(0);
      multiply(s + 4, rb);
    }
    if (s < steps) multiply(s, ra);
  }
  f32x4* sum = reinterpret_cast<f32x4*>(smem);  // [CW NR][64]
#pragma unroll
  for (int other = 1; other < 4; ++other) {
    if (other >= steps) break;  // that wave had no rows
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

template <int NR, int CW>
__global__ __launch_bounds__(256, 2) void k_ad_back(AdArgs a) {
  extern __shared__ __align__(16) char smem[];
  int block = blockIdx.x;
  if (block < a.blocks_u) {
    ad_dfactor<NR, CW, false>(a, block, smem);
    return;
  }
  block -= a.blocks_u;
  if (block < a.blocks_v) {
    ad_dfactor<NR, CW, true>(a, block, smem);
    return;
  }
  ad_dx(a, block - a.blocks_v);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct AdPlan {
  int tm, nr, tiles, slots, rp, rg, splits[2], units[2];
  size_t part[2], t2, t3[2], info, rows, first, total;  // offsets in the workspace
};

// K splits that give about kAdBlocks blocks in all, of whole units for the four
// waves.
static void ad_split(int K, int blocks, int* splits, int* per) {
  const int units = (K + kAdUnit - 1) / kAdUnit;
  const int want = std::max(1, std::min((units + 3) / 4, kAdBlocks / std::max(1, blocks)));
  *per = (units + want - 1) / want;
  *splits = (units + *per - 1) / *per;
}

static AdPlan ad_plan(const hss_adapters* A, int b, bool grad) {
  AdPlan p;
  p.tm = b <= kAdSmall && !grad ? 16 : 32;
  p.nr = A->r <= 16 ? 1 : A->r <= 32 ? 2 : 4;
  p.tiles = b <= kAdSmall ? b : b / p.tm + std::min(b, A->count + 1);
  p.slots = p.tm * p.tiles;
  p.rp = (A->r + 31) / 32 * 32;
  p.rg = (A->r + 15) / 16 * 16;
  // tiles with rows: at least those of one adapter, as if all had some
  const int groups = (p.rg + 16 * p.nr - 1) / (16 * p.nr);
  const int busy = std::max((b + p.tm - 1) / p.tm, std::min(b, A->count)) * groups * (grad ? 2 : 1);
  ad_split(A->n, busy, &p.splits[0], &p.units[0]);
  ad_split(A->m, busy, &p.splits[1], &p.units[1]);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  for (int k = 0; k < 2; ++k) {
    const bool wanted = k == 0 || grad;
    p.part[k] = take(wanted ? (size_t)p.splits[k] * p.slots * p.rg * 4 : 0);
    p.t3[k] = take(grad ? (size_t)3 * p.rg * p.slots * 2 : 0);
  }
  p.t2 = take(grad ? (size_t)p.slots * 2 * p.rp * 2 : 0);
  p.info = take((size_t)p.tiles * sizeof(int2));
  p.rows = take((size_t)p.slots * 2);
  p.first = take((size_t)A->count * sizeof(int2));
  p.total = off;
  return p;
}

size_t adapters_ws_bytes(const hss_adapters* A, int b, bool grad) { return ad_plan(A, b, grad).total; }

// The most that a batch of up to b rows needs.
size_t adapters_ws_bytes_up_to(const hss_adapters* A, int b, bool grad) {
  size_t most = 0;
  for (int c = 1; c <= b; ++c) most = std::max(most, adapters_ws_bytes(A, c, grad));
  return most;
}

static AdArgs ad_args(const hss_adapters* A, int b, const AdPlan& p, const void* X, const int32_t* ids,
                      const void* base, void* Y, void* ws) {
  AdArgs a = {};
  char* at = static_cast<char*>(ws);
  a.U = static_cast<const uint16_t*>(A->U), a.Vt = static_cast<const uint16_t*>(A->Vt), a.scale = A->scale;
  a.ids = ids, a.X = static_cast<const uint16_t*>(X), a.base = static_cast<const uint16_t*>(base);
  a.Y = static_cast<uint16_t*>(Y);
  for (int k = 0; k < 2; ++k) a.part[k] = reinterpret_cast<float*>(at + p.part[k]);
  a.info = reinterpret_cast<int2*>(at + p.info);
  a.rows = reinterpret_cast<uint16_t*>(at + p.rows);
  a.first = reinterpret_cast<int2*>(at + p.first);
  a.m = A->m, a.n = A->n, a.r = A->r, a.count = A->count, a.b = b;
  a.rp = p.rp, a.rg = p.rg, a.slots = p.slots, a.tiles = p.tiles;
  a.splits[0] = p.splits[0], a.units[0] = p.units[0];
  return a;
}

template <int TM, int NR>
static void launch_rank_nr(const AdArgs& a, hipStream_t s) {
  size_t lds = std::max<size_t>((size_t)4 * (TM / 16) * NR * 64 * 16, (size_t)(a.count + 1) * 4);
  if (a.splits[1]) lds = std::max<size_t>(lds, (size_t)4 * 16 * NR * kAdPitch * 2);
  const dim3 grid(a.splits[0] + a.splits[1], a.tiles, (a.rg + 16 * NR - 1) / (16 * NR));
  hipLaunchKernelGGL((k_ad_rank<TM, NR>), grid, dim3(256), lds, s, a);
}

template <int TM>
static void launch_rank(const AdArgs& a, int nr, hipStream_t s) {
  if (nr == 1) launch_rank_nr<TM, 1>(a, s);
  else if (nr == 2) launch_rank_nr<TM, 2>(a, s);
  else launch_rank_nr<TM, 4>(a, s);
}

template <int TM>
static void launch_expand(const AdArgs& a, hipStream_t s) {
  const int busy = std::max((a.b + TM - 1) / TM, std::min(a.b, a.count));
  const int cols = (a.m + 255) / 256;
  const int nc = std::max(1, std::min(cols, cols * busy / 512));
  const dim3 grid(a.tiles, (cols + nc - 1) / nc);
  const size_t lds = (size_t)TM * (2 * std::min(a.rp, kAdChunk) + 8) * 2;
  hipLaunchKernelGGL(k_ad_expand<TM>, grid, dim3(256), lds, s, a, nc);
}

hss_status launch_adapters_apply(const hss_adapters* A, int b, const void* X, const int32_t* ids, const void* base,
                                 void* Y, void* ws, hipStream_t s) {
  const AdPlan p = ad_plan(A, b, false);
  AdArgs a = ad_args(A, b, p, X, ids, base, Y, ws);
  a.first = nullptr;
  if (p.tm == 16) launch_rank<16>(a, p.nr, s), launch_expand<16>(a, s);
  else launch_rank<32>(a, p.nr, s), launch_expand<32>(a, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

template <int NR, int CW>
static void launch_back(AdArgs a, hipStream_t s) {
  const size_t lds = (size_t)CW * NR * 64 * 16;
  a.chunks = (a.rg + 16 * NR - 1) / (16 * NR);
  a.cols_u = (a.m + 16 * CW - 1) / (16 * CW), a.cols_v = (a.n + 16 * CW - 1) / (16 * CW);
  a.cols_y = (a.n + 511) / 512;
  a.blocks_u = a.dU ? a.cols_u * a.chunks * a.count : 0;
  a.blocks_v = a.dVt ? a.cols_v * a.chunks * a.count : 0;
  const dim3 grid(a.blocks_u + a.blocks_v + (a.Y ? a.cols_y * a.tiles : 0));
  hipLaunchKernelGGL((k_ad_back<NR, CW>), grid, dim3(256), lds, s, a);
}

hss_status launch_adapters_grad(const hss_adapters* A, int b, const void* X, const void* G, const int32_t* ids,
                                const void* base, void* dX, float* dU, float* dVt, void* ws, hipStream_t s) {
  if (!dX && !dU && !dVt) return HSS_OK;
  const AdPlan p = ad_plan(A, b, true);
  AdArgs a = ad_args(A, b, p, X, ids, base, dX, ws);
  char* at = static_cast<char*>(ws);
  a.G = static_cast<const uint16_t*>(G), a.dU = dU, a.dVt = dVt;
  a.t2 = dX ? reinterpret_cast<uint16_t*>(at + p.t2) : nullptr;
  a.t3[0] = dU ? reinterpret_cast<uint16_t*>(at + p.t3[0]) : nullptr;
  a.t3[1] = dVt ? reinterpret_cast<uint16_t*>(at + p.t3[1]) : nullptr;
  if (!dU) a.splits[0] = 0;
  if (dX || dVt) a.splits[1] = p.splits[1], a.units[1] = p.units[1];
  launch_rank<32>(a, p.nr, s);
  const dim3 grid(a.tiles, (a.rp + 63) / 64, a.splits[0] && a.splits[1] ? 2 : 1);
  hipLaunchKernelGGL(k_ad_terms, grid, dim3(256), 0, s, a);
  // few blocks of dU and dVt: narrower ones
  const bool narrow = (int64_t)A->count * ((A->r + 63) / 64) * ((int64_t)A->m + A->n) / 128 < 256;
  if (p.nr == 1) narrow ? launch_back<1, 2>(a, s) : launch_back<1, 8>(a, s);
  else if (p.nr == 2) narrow ? launch_back<2, 2>(a, s) : launch_back<2, 4>(a, s);
  else narrow ? launch_back<4, 2>(a, s) : launch_back<4, 4>(a, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
