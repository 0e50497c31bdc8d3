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
// Forward: k_ad_rank makes T, K split over blocks into partial sums in fp32, for a few
// tiles would not fill the chip, and k_ad_expand adds the splits in order on its way to
// the matrix cores.  A few rows and small factors take one launch, k_ad_fused.
// Backward: k_ad_rank makes T and P, k_ad_terms adds the splits once for all that read
// them (short K is not split, and k_ad_rank makes the terms), k_ad_back makes dU, dVt
// and dX.  T and P, times scale in fp32, go to the matrix cores as bf16 terms: two (16
// significant bits) where the result is rounded to bf16 anyway, three (24 bits)
// for the fp32 gradients.
//
// Measured (calls back to back over three sets of arrays, bytes moved at least / time): 64 requests of
// their own 11008 x 4096 r 64 127 MB in 32 us, 3.9 TB/s; 2048 rows of 4 4096 x 11008 r 64
// 86 MB in 36 us, 2.4 TB/s, of which 5 us are launches, 5 the search for tiles and 5
// the way from the partial sums to the first product; gradients of 2048 rows of 8
// 11008 x 4096 r 64 142 MB in 70 us (X and G are read twice: 204 MB, 2.9 TB/s).  One
// row 4096 x 4096 r 16: 6.6 us, of which a launch takes 2.
#include <algorithm>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Batches up to here (a lane for each row): tiles found by one ballot, of 16 rows in
// the forward pass; beyond, by a histogram, of 32.  4096 x 4096 r 64, the last batch
// of the one and the first of the other: of 4 adapters 10.8 and 13.0 us, an adapter a
// row 18.7 and 23.9.
static constexpr int kAdSmall = 64;
static constexpr int kAdUnit = 64;      // columns of K that a wave takes at a time: a cache line of each row
// Blocks of k_ad_rank that K is split for, of at least four units, one a wave.  128,
// 256, 512, 1024: 2048 rows 4096 x 11008 43.1, 41.0, 40.1, 43.7 us.  At least 4, 8, 16
// units: 77 rows 2731 x 5003 14.7, 15.3, 16.6.
static constexpr int kAdBlocks = 512;
// Ranks of T that k_ad_expand keeps in LDS, 1 KB a row (two terms of two bytes): with
// U's 32 KB two blocks of 32 rows (65 KB) or three of 16 (49 KB) share a compute unit's
// 160 KB, as many as their registers allow.
static constexpr int kAdChunk = 256;
// Units of K that the backward pass does not split, so that k_ad_rank makes the terms
// and a launch is saved: not split and split, 64 rows of 4 512 x 512 9.2 and 11.0 us,
// 16 rows 1024 x 1024 10.1 and 10.6, past the limit 2048 x 2048 12.8 and 10.9.
static constexpr int kAdWhole = 16;

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
  // Terms as the matrix cores' operands, 64 lanes of 8 values (null = none):
  uint16_t* t2;     // two of P: [tile][rp / 32][term][half of the rows], lane: row % 16 + 16 (rank / 8 % 4)
  uint16_t* t3[2];  // three of T and P: [tile][rg / 16][term], lane: rank % 16 + 16 (slot / 8 % 4)
  int2* info;       // [tiles]: adapter (-1: none) and rows (0: no such tile)
  uint16_t* rows;   // [slots]
  int2* first;      // [count]: an adapter's first tile and its rows (more than kAdSmall rows)
  int m, n, r, count, b;
  int rp, rg;       // r rounded up to 32 and to 16
  int slots, tiles;
  int splits[2], units[2];           // K splits of T and P (0: not wanted), units of each
  int blocks_u, blocks_v, blocks_y;  // of k_ad_back
  int cols_y, cols_u, cols_v;        // column blocks of dX, dU, dVt
  int chunks;                        // passes of dU and dVt over the ranks
  int direct;                        // K is not split: k_ad_rank makes the terms (backward)
};

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// 16 bytes at a byte offset from a base that the whole wave shares (arrays have
// fewer than 2^31 elements of two bytes: one register an address).
__device__ __forceinline__ u32x4 ad_load(const void* base, uint32_t at) {
  const Bytes16 v = *reinterpret_cast<const Bytes16*>(static_cast<const char*>(base) + at);
  return u32x4{v.w[0], v.w[1], v.w[2], v.w[3]};
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
// Blocks go to the chip's eight dies in turn, each with a cache of its own.  Work is
// (tile, part), and adjacent tiles mostly share an adapter: eight of them with the
// same part of its factors go to one die.  (Gradients of 2048 rows 11008 x 4096 of 8,
// r 64, whose 64 tiles read 124 MB of U and Vt: k_ad_rank 34 -> 25 us, with a quicker
// search for the tiles, which alone took 1.5 us off a forward pass of 2048 rows.)
struct AdWork {
  int tile, part;  // tile: may lie past the last one
};

__device__ __forceinline__ AdWork ad_work(uint32_t block, uint32_t parts) {
  const uint32_t group = (block & 7) + 8 * (block >> 6);
  return {(int)(8 * (group / parts) + ((block >> 3) & 7)), (int)(group % parts)};
}

static inline int ad_work_blocks(int tiles, int parts) { return ((tiles + 7) / 8 * parts + 7) / 8 * 64; }

struct AdTile {
  int adapter;  // -1: rows without one
  int rows;     // 0: no such tile
};

template <int CTRL, int ROWS>
__device__ __forceinline__ int ad_dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}

// Exclusive prefix sum over the block's 256 threads, and the total.  (In a wave by
// DPP shifts within rows of 16 lanes, then each row's last lane to the rows behind.)
__device__ __forceinline__ int ad_scan(int v, int* part, int* total) {
  const int w = threadIdx.x >> 6;
  int incl = ad_dpp_add<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  incl = ad_dpp_add<0x112, 0xF>(incl);
  incl = ad_dpp_add<0x114, 0xF>(incl);
  incl = ad_dpp_add<0x118, 0xF>(incl);
  incl = ad_dpp_add<0x142, 0xA>(incl);    // row_bcast 15 into rows 1 and 3
  incl = ad_dpp_add<0x143, 0xC>(incl);    // row_bcast 31 into rows 2 and 3
  const int before = incl - v;
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

// Copies of the bins, and the bins in all.
__host__ __device__ __forceinline__ int ad_copies(int count) { return count < 512 ? 8 : 1; }
__host__ __device__ __forceinline__ int ad_bins(int count) { return (count + 1) * (ad_copies(count) == 1 ? 1 : 9); }

__device__ __forceinline__ int ad_id(const int32_t* ids, int t, int count) {
  const int id = ids[t];
  return id >= 0 && id < count ? id : -1;
}

// Tile `tile` of the batch: its adapter and its rows (in LDS).  Up to 64 rows
// tile t starts at row t, if that is the first, or TM rows after the last start,
// of its adapter; beyond, tiles are counted through the adapters, rows without one
// last.  bins: ad_bins ints; part: 6.  table: null, or where each adapter's
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
  static_assert(per == 8, "two loads of 16 bytes a thread");
  int id[per];
  if (per * t + per <= b) {
    const u32x4 lo = ad_load(a.ids, 4 * per * t), hi = ad_load(a.ids, 4 * per * t + 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) id[k] = (int)lo[k], id[4 + k] = (int)hi[k];
  } else {
#pragma unroll
    for (int k = 0; k < per; ++k) id[k] = a.ids[min(per * t + k, b - 1)];  // all in flight
  }
  // A batch of few adapters would have lanes add to the same places: eight copies of
  // the bins, summed below.
  const int copies = ad_copies(count);
  int* bin8 = copies == 1 ? bins : bins + count + 1;
  for (int k = t; k < (count + 1) * copies; k += 256) bin8[k] = 0;
#pragma unroll
  for (int k = 0; k < per; ++k) {
    if (id[k] < 0 || id[k] >= count) id[k] = count;
    if (per * t + k >= b) id[k] = -2;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < per; ++k)
    if (id[k] >= 0) atomicAdd(&bin8[id[k] * copies + (t & (copies - 1))], 1);
  __syncthreads();
  const int many = (count + 256) / 256, k0 = t * many;
  int own = 0, total;
  for (int k = k0; k < min(k0 + many, count + 1); ++k) {
    if (copies == 8) {
      int sum = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) sum += bin8[8 * k + c];
      bins[k] = sum;
    }
    own += (bins[k] + TM - 1) / TM;
  }
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

// CW bf16 at a byte offset (a multiple of 2) from a base that the wave shares.
template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_piece_at(const void* base, uint32_t at) {
  struct __attribute__((packed, aligned(2))) Raw {
    uint32_t w[CW / 2];
  };
  const Raw raw = *reinterpret_cast<const Raw*>(static_cast<const char*>(base) + at);
  AdPiece<CW> p;
#pragma unroll
  for (int d = 0; d < CW / 2; ++d) p.w[d] = raw.w[d];
  return p;
}

// The first `left` of them, zeros behind: element by element, for the ends of rows
// shorter than a piece.
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

template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_nothing() {
  AdPiece<CW> p;
#pragma unroll
  for (int d = 0; d < CW / 2; ++d) p.w[d] = 0u;
  return p;
}

// Eight bf16 without the first s, zeros behind (s >= 8: zeros).  A row's last
// columns are loaded as the eight that end with the row, and shifted.
__device__ __forceinline__ u32x4 ad_drop(u32x4 v, int s) {
  uint64_t lo = v.x | (uint64_t)v.y << 32, hi = v.z | (uint64_t)v.w << 32;
  if (s >= 4) lo = hi, hi = 0, s -= 4;
  const int bits = 16 * min(s, 3);
  lo = lo >> bits | (hi << 1) << (63 - bits);
  hi >>= bits;
  if (s >= 4) lo = 0, hi = 0;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

template <int CW>
__device__ __forceinline__ AdPiece<CW> ad_drop(const AdPiece<CW>& p, int s) {
  u32x4 v = {p.w[0], 0u, 0u, 0u};
#pragma unroll
  for (int d = 1; d < CW / 2; ++d) v[d] = p.w[d];
  v = ad_drop(v, s);
  AdPiece<CW> o;
#pragma unroll
  for (int d = 0; d < CW / 2; ++d) o.w[d] = v[d];
  return o;
}

// Eight bf16 of a row of n at column k, zeros past the end, in one load (n >= 8).
__device__ __forceinline__ u32x4 ad_tail8(const uint16_t* row, int k, int n) {
  const int from = min(k, n - 8);
  return ad_drop(load8(row + from), k - from);
}

// What this wave wrote to its part of LDS before is read after (LDS takes a
// wave's accesses in order; this keeps the compiler to it).
__device__ __forceinline__ void ad_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Two fp32 values as bf16 (to nearest even), in a dword.
__device__ __forceinline__ uint32_t ad_pack(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, mx_bf16x2));
}

// A finite value past bf16's largest, which would round to an infinity, cut to the
// largest; any other as it is.
__device__ __forceinline__ float ad_cut(float x) {
  return fabsf(x) > 0x1.fep127f ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : x;
}

// The next bf16 terms of two values, which lose them (an infinity leaves 0, not the
// NaN of inf - inf).
__device__ __forceinline__ uint32_t ad_term2(float& x, float& y) {
  const uint32_t t = ad_pack(ad_cut(x), ad_cut(y));
  x = (t & 0x7fffu) == 0x7f80u ? 0.f : x - bf16lo(t);
  y = (t & 0x7fff0000u) == 0x7f800000u ? 0.f : y - bf16hi(t);
  return t;
}

// ---------------------------------------------------------------------------
// T = X Vt^T and P = G U, partial sums over a block's part of K; the blocks of split
// 0 also write the table of tiles.
//   D[rank][row] += A[rank][k] B[row][k]: A = Vt_l as stored, or U_l transposed.
//   Wave w takes units w, w + 4, .. of the block's, each through the wave's own part
//   of LDS, with no barrier: eight lanes load 128 adjacent bytes of a row (loaded as
//   the matrix cores take it, neighbouring lanes would have different rows, and each
//   lane's 16 bytes be an access of its own to the cache: 4 times as many; prefill
//   of 2048 rows 4096 x 11008 r 64: 37 us).  The next unit's loads are in flight
//   while one is multiplied.  The four waves' sums meet in LDS.
//   2048 rows 4096 x 11008 of 4, r 64: 17 us for 51 MB, 3 of them the search for the
//   tile, 1 the sums; gradients of 2048 rows 11008 x 4096 of 8: 25 us for 77 MB.
// grid: (tiles by splits of T and of P, groups of 16 NR ranks)
// ---------------------------------------------------------------------------
// Where 16-byte chunk c of a 128-byte row lies in LDS.  A read takes one chunk of 16
// rows, half of them in each half of the 256 bytes of banks: (row / 2) % 8 tells
// each half's eight apart.  A transposed piece's write takes one chunk of eight rows
// that are 8 apart: (row / 8) % 8 tells those apart.
__device__ __forceinline__ int ad_slot(int row, int c) { return row * kAdUnit + 8 * (c ^ ((row >> 1) & 7) ^ ((row >> 3) & 7)); }

template <int TM, int NR>
__global__ __launch_bounds__(256, NR == 4 ? 3 : 4) void k_ad_rank(AdArgs a) {
  constexpr int MF = TM / 16, XL = TM / 8, VL = 2 * NR;
  extern __shared__ __align__(16) char smem[];
  __shared__ uint16_t rows[TM];
  __shared__ int part[6];
  const AdWork work = ad_work(blockIdx.x, a.splits[0] + a.splits[1]);
  const int tile = work.tile, rank0 = (int)blockIdx.y * 16 * NR;
  if (tile >= a.tiles) return;
  const int side = work.part >= a.splits[0], z = work.part - (side ? a.splits[0] : 0);
  const bool lead = work.part == 0 && blockIdx.y == 0;
  AdTile at = ad_tile<TM>(a, tile, rows, part, reinterpret_cast<int*>(smem), lead && tile == 0 ? a.first : nullptr);
  at = {uniform(at.adapter), uniform(at.rows)};
  if (lead) {  // (a tile's free slots repeat its last row, so that all of them may be read)
    if (threadIdx.x == 0) a.info[tile] = make_int2(at.adapter, at.rows);
    if (threadIdx.x < TM && at.rows) a.rows[TM * tile + threadIdx.x] = rows[min((int)threadIdx.x, at.rows - 1)];
  }
  if (at.rows == 0 || at.adapter < 0) return;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int K = side ? a.m : a.n;
  const int u0 = z * a.units[side], u1 = min(u0 + a.units[side], (K + kAdUnit - 1) / kAdUnit);
  const int whole = min(u1, K / kAdUnit);  // units before here end inside the row
  const int c8 = lane & 7, r8 = lane >> 3;
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem) + w * (TM + 16 * NR) * kAdUnit;  // the wave's: [TM][64]
  uint16_t* vs = xs + TM * kAdUnit;  // [16 NR][64], of Vt or U^T
  const uint16_t* X = side ? a.G : a.X;
  int xrow[XL];
#pragma unroll
  for (int j = 0; j < XL; ++j) xrow[j] = rows[min(8 * j + r8, at.rows - 1)] * K;

  f32x4 acc[MF][NR];
#pragma unroll
  for (int f = 0; f < MF; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 x[XL];
  auto put_x = [&]() {
#pragma unroll
    for (int j = 0; j < XL; ++j) *reinterpret_cast<u32x4*>(xs + ad_slot(8 * j + r8, c8)) = x[j];
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 xf[MF], vf[NR];
#pragma unroll
      for (int f = 0; f < MF; ++f) xf[f] = *reinterpret_cast<const u32x4*>(xs + ad_slot(16 * f + i, 4 * h + q));
#pragma unroll
      for (int g = 0; g < NR; ++g) vf[g] = *reinterpret_cast<const u32x4*>(vs + ad_slot(16 * g + i, 4 * h + q));
      __builtin_amdgcn_sched_barrier(0);  // the reads first: one wait instead of one for each product
#pragma unroll
      for (int g = 0; g < NR; ++g)
#pragma unroll
        for (int f = 0; f < MF; ++f)
          acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(vf[g]), as_bf16(xf[f]), acc[f][g], 0, 0, 0);
    }
    ad_wave_sync();
  };

  if (!side) {
    const uint16_t* V = a.Vt + (int64_t)at.adapter * a.r * K;
    int vrow[VL];
#pragma unroll
    for (int j = 0; j < VL; ++j) vrow[j] = min(rank0 + 8 * j + r8, a.r - 1) * K;
    u32x4 v[VL];
    auto load = [&](int u) {
#pragma unroll
      for (int j = 0; j < XL; ++j) x[j] = ad_load(X, 2u * (xrow[j] + u * kAdUnit + 8 * c8));
#pragma unroll
      for (int j = 0; j < VL; ++j) v[j] = ad_load(V, 2u * (vrow[j] + u * kAdUnit + 8 * c8));
    };
    auto put = [&]() {
      put_x();
#pragma unroll
      for (int j = 0; j < VL; ++j) *reinterpret_cast<u32x4*>(vs + ad_slot(8 * j + r8, c8)) = v[j];
      ad_wave_sync();
    };
    int u = u0 + w;
    if (u < whole) {
      load(u);
      for (; u + 4 < whole; u += 4) {
        put();
        load(u + 4);
        multiply();
      }
      put(), multiply();
      u += 4;
    }
    if (u < u1) {  // the unit in which the rows end
      const int k = u * kAdUnit + 8 * c8;
      if (K >= 8) {
#pragma unroll
        for (int j = 0; j < XL; ++j) x[j] = ad_tail8(X + xrow[j], k, K);
#pragma unroll
        for (int j = 0; j < VL; ++j) v[j] = ad_tail8(V + vrow[j], k, K);
      } else {
#pragma unroll
        for (int j = 0; j < XL; ++j) x[j] = __builtin_bit_cast(u32x4, ad_piece_end<8>(X + xrow[j], k < K ? K - k : 0));
#pragma unroll
        for (int j = 0; j < VL; ++j) v[j] = __builtin_bit_cast(u32x4, ad_piece_end<8>(V + vrow[j], k < K ? K - k : 0));
      }
      put(), multiply();
    }
  } else {
    // 8 x 8 pieces, one a lane: 8 of the unit's j times 2 NR of the ranks.  The piece
    // in which the ranks end is loaded as the row's last eight, and stored behind the
    // one before it.
    const int kb = lane % (2 * NR), jb = lane / (2 * NR), want = rank0 + 8 * kb, rank = max(0, min(want, a.r - 8));
    const uint16_t* U = a.U + (int64_t)at.adapter * a.m * a.r;
    const int off = 8 * kb - (want - rank);  // its row in LDS; below 0 or past the ranks: none
    const bool mine = jb < 8 && want < a.r;
    const int safe = a.r >= 8 ? whole : u0;  // rows shorter than a piece: the slow way
    AdPiece<8> v[8];
    auto load = [&](int u) {
#pragma unroll
      for (int j = 0; j < XL; ++j) x[j] = ad_load(X, 2u * (xrow[j] + u * kAdUnit + 8 * c8));
      if (mine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(AdPiece<8>, ad_load(U, 2u * ((u * kAdUnit + 8 * jb + e) * a.r + rank)));
      }
    };
    auto put = [&]() {
      put_x();
      if (mine) {
#pragma unroll
        for (int f = 0; f < 8; ++f)
          if (off + f >= 0) *reinterpret_cast<u32x4*>(vs + ad_slot(off + f, jb)) = ad_column<8>(v, f);
      }
      ad_wave_sync();
    };
    int u = u0 + w;
    if (u < safe) {
      load(u);
      for (; u + 4 < safe; u += 4) {
        put();
        load(u + 4);
        multiply();
      }
      put(), multiply();
      u += 4;
    }
    for (; u < u1; u += 4) {
      const int k = u * kAdUnit + 8 * c8;
      if (K >= 8) {
#pragma unroll
        for (int j = 0; j < XL; ++j) x[j] = ad_tail8(X + xrow[j], k, K);
      } else {
#pragma unroll
        for (int j = 0; j < XL; ++j) x[j] = __builtin_bit_cast(u32x4, ad_piece_end<8>(X + xrow[j], k < K ? K - k : 0));
      }
      if (mine) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = u * kAdUnit + 8 * jb + e;
          const uint16_t* from = U + min(j, K - 1) * a.r + rank;
          v[e] = a.r >= 8 ? ad_piece_at<8>(from, 0) : ad_piece_end<8>(from, a.r);
          if (j >= K) v[e] = ad_nothing<8>();
        }
      }
      put(), multiply();
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
    const int rank = rank0 + 16 * g + 4 * q, slot = 16 * f + i;  // ranks .. rank + 3 of a slot
    if (rank >= a.rg) continue;
    if (!a.direct) {
      if (slot < at.rows) *reinterpret_cast<f32x4*>(out + slot * a.rg + rank) = v;
      continue;
    }
    // K was not split: the terms at once, as k_ad_terms writes them
    const float scale = a.scale ? a.scale[at.adapter] : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = slot < at.rows && rank + e < a.r ? v[e] * scale : 0.f;
    float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int h = 0; h < 3; ++h) {
      const uint32_t lo = ad_term2(x[0], x[1]), hi = ad_term2(x[2], x[3]);
      if (a.t3[side]) {
        uint16_t* to = a.t3[side] + ((((int64_t)tile * (a.rg >> 4) + (rank >> 4)) * 3 + h) * 64 + 2 * (slot & ~7) + 4 * q) * 8 + (slot & 7);
        to[0] = (uint16_t)lo, to[8] = (uint16_t)(lo >> 16), to[16] = (uint16_t)hi, to[24] = (uint16_t)(hi >> 16);
      }
      if (a.t2 && side && h < 2) {
        uint16_t* to = a.t2 + ((((int64_t)tile * (a.rp >> 5) + (rank >> 5)) * 4 + 2 * h + f) * 64 + 16 * ((rank >> 3) & 3) + i) * 8 + (rank & 7);
        *reinterpret_cast<mx_u32x2*>(to) = mx_u32x2{lo, hi};
        if (rank + 16 >= a.rg && a.rg < a.rp) *reinterpret_cast<mx_u32x2*>(to + 2 * 16 * 8) = mx_u32x2{0u, 0u};  // ranks + 16
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: the terms of T and P.  A lane has one rank of eight slots.  4 to 6 us, most
// of it a launch and one chain of loads, instead of the sums in each block of dU, dVt and
// dX (2048 rows 11008 x 4096 of 8, r 64: 1056 of them).
// grid: (tiles, ranks / 64, sides)
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_ad_terms(AdArgs a) {
  const int tile = blockIdx.x, side = a.splits[0] == 0 ? 1 : (int)blockIdx.z;
  const int rank = (int)blockIdx.y * 64 + (threadIdx.x & 63), i0 = 8 * (threadIdx.x >> 6);
  if (rank >= a.rp) return;
  const int2 info = a.info[tile];
  const int splits = a.splits[side];
  const int64_t stride = (int64_t)a.slots * a.rg;
  const float* p = a.part[side] + (int64_t)(32 * tile + i0) * a.rg + min(rank, a.rg - 1);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int z = 0; z < splits; z += 8) {  // (the tile's adapter and rows are on their way with the first ones)
    float x[8][8];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[c][e] = p[min(z + c, splits - 1) * stride + e * a.rg];
    if (z + 4 < splits) {
#pragma unroll
      for (int c = 4; c < 8; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[c][e] = p[min(z + c, splits - 1) * stride + e * a.rg];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (z + c < splits) v[e] += x[c][e];
  }
  const int2 at = make_int2(uniform(info.x), uniform(info.y));
  if (at.x < 0 || at.y == 0) return;
  const float scale = a.scale ? a.scale[at.x] : 1.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = rank < a.r && i0 + e < at.y ? v[e] * scale : 0.f;  // a slot without a row holds anything
  // the lane of an operand that holds these eight slots of this rank (dU, dVt), or
  // slot i0 + e of this rank's eight (dX)
  uint16_t* three = a.t3[side];
  const int g = rank >> 4, step = rank >> 5;
#pragma unroll
  for (int h = 0; h < 3; ++h) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = ad_term2(v[2 * e], v[2 * e + 1]);
    if (three && rank < a.rg)
      *reinterpret_cast<u32x4*>(three + ((((int64_t)tile * (a.rg >> 4) + g) * 3 + h) * 64 + 2 * i0 + (rank & 15)) * 8) =
          u32x4{t[0], t[1], t[2], t[3]};
    if (a.t2 && side && h < 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        a.t2[((((int64_t)tile * (a.rp >> 5) + step) * 4 + 2 * h + ((i0 + e) >> 4)) * 64 + 16 * ((rank >> 3) & 3) +
              ((i0 + e) & 15)) * 8 + (rank & 7)] = (uint16_t)(t[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// ---------------------------------------------------------------------------
// Outputs in bf16
// ---------------------------------------------------------------------------
// Eight columns of 4 MF rows of base, from byte offsets `at` + 2 c0 on.  Where a row
// ends before them (`back` columns too many), its last eight, which ad_store8_end
// shifts; rows of fewer than eight one by one.
template <int MF>
__device__ __forceinline__ void ad_load_base(u32x4 (&old)[MF][4], const void* base, const uint32_t (&at)[MF][4], int c0,
                                             int back, int cols) {
  if (!base) return;
  if (cols >= 8) {
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) old[g][e] = ad_load(base, at[g][e] + 2u * (c0 - back));
    return;
  }
#pragma unroll 1
  for (int k = 0; k < 8 - back; ++k)
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t raw = *reinterpret_cast<const uint16_t*>(static_cast<const char*>(base) + at[g][e] + 2 * (c0 + k));
        const uint32_t x = (uint32_t)raw << 16 * (k & 1);
        u32x4& v = old[g][e];
        v.x |= k >> 1 == 0 ? x : 0u, v.y |= k >> 1 == 1 ? x : 0u, v.z |= k >> 1 == 2 ? x : 0u, v.w |= k >> 1 == 3 ? x : 0u;
      }
}

__device__ __forceinline__ u32x4 ad_sum8(const u32x4& old, const float* v) {
  u32x4 o;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = ad_pack(v[2 * k] + bf16lo(old[k]), v[2 * k + 1] + bf16hi(old[k]));
  return o;
}

// Eight values in bf16, old + v, at a byte offset of the output.
__device__ __forceinline__ void ad_store8(void* base, uint32_t at, const u32x4& old, const float* v) {
  const u32x4 o = ad_sum8(old, v);
  *reinterpret_cast<Bytes16*>(static_cast<char*>(base) + at) = Bytes16{{o.x, o.y, o.z, o.w}};
}

// The same where the row ends after 8 - back of them: by fours, twos and ones.
__device__ __forceinline__ void ad_store8_end(void* base, uint32_t at, u32x4 old, const float* v, int back, int cols) {
  struct __attribute__((packed, aligned(2))) Two { uint32_t w[1]; };
  struct __attribute__((packed, aligned(2))) Four { uint32_t w[2]; };
  if (cols >= 8) old = ad_drop(old, back);
  u32x4 o = ad_sum8(old, v);
  char* to = static_cast<char*>(base) + at;
  const int left = 8 - back;
  if (left >= 8) *reinterpret_cast<Bytes16*>(to) = Bytes16{{o.x, o.y, o.z, o.w}};
  if (left <= 0 || left >= 8) return;
  if (left & 4) *reinterpret_cast<Four*>(to) = Four{{o.x, o.y}}, to += 8, o = u32x4{o.z, o.w, 0u, 0u};
  if (left & 2) *reinterpret_cast<Two*>(to) = Two{{o.x}}, to += 4, o.x = o.y;
  if (left & 1) *reinterpret_cast<uint16_t*>(to) = (uint16_t)o.x;
}

// Rows without an adapter: the output is base (nothing to do in place).  Eight
// columns a lane, four of them in flight.
__device__ __forceinline__ void ad_copy(const AdArgs& a, const AdTile& at, const uint16_t* rows, int col, int width,
                                        int cols) {
  if (a.base == a.Y) return;
  const int pieces = (min(width, cols - col) + 7) / 8, total = at.rows * pieces;
  const int threads = blockDim.x;
  for (int e0 = threadIdx.x; e0 < total; e0 += 4 * threads) {
    uint32_t to[4];
    int left[4];
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = min(e0 + threads * j, total - 1), c = col + e % pieces * 8;
      to[j] = rows[e / pieces] * cols + c;
      left[j] = cols - c;
      v[j] = u32x4{0u, 0u, 0u, 0u};
    }
    if (a.base) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (left[j] >= 8) v[j] = ad_load(a.base, 2u * to[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e0 + threads * j >= total) continue;
      if (left[j] >= 8) {
        *reinterpret_cast<Bytes16*>(a.Y + to[j]) = Bytes16{{v[j].x, v[j].y, v[j].z, v[j].w}};
      } else {
#pragma unroll 1
        for (int k = 0; k < left[j]; ++k) a.Y[to[j] + k] = a.base ? a.base[to[j] + k] : (uint16_t)0;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Y = base + scale T U^T.  D[row][column], B = U_l as stored, 128 columns a wave:
// piece f of the operand holds columns 8 i + f, so that a lane ends up with eight
// adjacent columns of four rows, and 16 lanes read and write 256 bytes of a row.  U
// comes through the wave's own part of LDS, 32 ranks at a time (four lanes a row),
// the next ones in flight.  The block's terms of T are made first, in LDS, for all
// its columns, of which it takes about as many as give each compute unit a block (64
// requests 11008 x 4096 r 64, NC 1, 2, 4, 6, 8: 37.0, 35.0, 34.1, 33.2, 36.3 us a call;
// 2048 rows 4096 x 11008: 43.8, 39.7, 39.9, 45.3, 50.0).  Bound by memory where U is
// read once (64 requests: 20 us, 4.6 TB/s), by the way to the first product where
// blocks are short (2048 rows: 17 us for 36 MB, 5 until the terms are made).
// grid: (tiles, column blocks of 512 NC)
// ---------------------------------------------------------------------------
// Where 16-byte chunk q of U's row 8 i + f (32 ranks, 64 bytes) lies in LDS: the 16
// rows of a piece side by side, so that a read's 16 fall on different banks (chunks
// spread by i / 4), and the four rows of a write too (rows spread by f).
__device__ __forceinline__ int ad_place(int i, int f, int q) { return (16 * f + (i ^ (f & 3))) * 32 + 8 * (q ^ ((i >> 2) & 3)); }

// Ranks k .. k + 31 of U's rows c0 .. c0 + 127, four lanes a row; at the end of the
// ranks the row's last eight, which ad_put_u shifts.
__device__ __forceinline__ void ad_load_u(u32x4 (&u)[8], const uint16_t* U, int m, int r, int c0, int k) {
  const int lane = threadIdx.x & 63, col = lane >> 2, from = min(k + 8 * (lane & 3), r - 8);
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = ad_load(U, 2u * (min(c0 + 16 * j + col, m - 1) * r + from));
}

// The same to the wave's part of LDS: column 16 j + col = 8 (2 j + col / 8) + col % 8.
__device__ __forceinline__ void ad_put_u(u32x4 (&u)[8], uint16_t* us, int r, int k) {
  const int lane = threadIdx.x & 63, col = lane >> 2, c4 = lane & 3;
  if (k + 32 > r && r >= 8) {
    const int drop = k + 8 * c4 - min(k + 8 * c4, r - 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = ad_drop(u[j], drop);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<u32x4*>(us + ad_place(2 * j + (col >> 3), col & 7, c4)) = u[j];
  ad_wave_sync();
}

// SHORT: rows of U with fewer than eight ranks, loaded one by one.
template <int TM, bool SHORT>
__global__ __launch_bounds__(256, TM == 16 ? 3 : 2) void k_ad_expand(AdArgs a, int nc) {
  constexpr int MF = TM / 16;
  extern __shared__ __align__(16) uint16_t lds[];
  const int tile = blockIdx.x, cb = (int)blockIdx.y * 512 * nc;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int2 info = a.info[tile];
  const uint16_t* rows = a.rows + TM * tile;
  uint32_t out[MF][4];  // byte offsets (of a tile that is not there: any number, not used)
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[g][e] = 2u * (rows[16 * g + 4 * q + e] * a.m + 8 * i);
  const AdTile at = {uniform(info.x), uniform(info.y)};
  if (at.rows == 0) return;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 512 * nc, a.m);
    return;
  }
  uint16_t* us = lds + w * 128 * 32;
  uint16_t* terms = lds + 4 * 128 * 32;  // [TM][2][ranks of a chunk, + 4]
  const int wide = min(a.rp, kAdChunk), pitch = 2 * wide + 8;
  const float scale = a.scale ? a.scale[at.adapter] : 1.f;
  auto fill = [&](int rank0) {  // two terms of a chunk's ranks, zeros past r; 4 J loads in flight
    const uint32_t quads = (uint32_t)min(wide, a.rp - rank0) / 4, items = at.rows * quads;
    const float* p = a.part[0] + (int64_t)TM * tile * a.rg + rank0;
    const int64_t stride = (int64_t)a.slots * a.rg;
    const int splits = a.splits[0];
    constexpr int J = MF;
    for (uint32_t e0 = threadIdx.x; e0 < items; e0 += 256 * J) {
      int row[J], k[J];
      const float* from[J];
      f32x4 sum[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t e = min(e0 + 256 * j, items - 1);
        row[j] = e / quads, k[j] = e % quads * 4;
        from[j] = p + row[j] * a.rg + min(k[j], a.rg - 4 - rank0);
        sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      for (int z = 0; z < splits; z += 4) {
        f32x4 v[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) v[j][c] = *reinterpret_cast<const f32x4*>(from[j] + min(z + c, splits - 1) * stride);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (z + c < splits) sum[j] += v[j][c];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (e0 + 256 * j >= items) continue;
        float x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = rank0 + k[j] + c < a.r ? sum[j][c] * scale : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = ad_term2(x[0], x[1]), hi = ad_term2(x[2], x[3]);
          *reinterpret_cast<mx_u32x2*>(terms + row[j] * pitch + h * wide + k[j]) = mx_u32x2{lo, hi};
        }
      }
    }
  };
  const uint16_t* trow[MF];
#pragma unroll
  for (int g = 0; g < MF; ++g) trow[g] = terms + min(16 * g + i, at.rows - 1) * pitch + 8 * q;
  const uint16_t* U = a.U + (int64_t)at.adapter * a.m * a.r;
  const bool one = a.rp <= kAdChunk;
  u32x4 u[8];
  auto load = [&](int c0, int k) {
    if constexpr (!SHORT) {
      ad_load_u(u, U, a.m, a.r, c0, k);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = u32x4{0u, 0u, 0u, 0u};
      if ((lane & 3) != 0) return;
#pragma unroll 1
      for (int e = 0; e < a.r; ++e) {
        const int d = e >> 1, sh = 16 * (e & 1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t x = (uint32_t)U[min(c0 + 16 * j + (lane >> 2), a.m - 1) * a.r + e] << sh;
          u[j].x |= d == 0 ? x : 0u, u[j].y |= d == 1 ? x : 0u, u[j].z |= d == 2 ? x : 0u, u[j].w |= d == 3 ? x : 0u;
        }
      }
    }
  };
  u32x4 old[MF][4];
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) old[g][e] = u32x4{0u, 0u, 0u, 0u};
  // the first columns' U and base are on their way while the terms are made, the
  // next ones' while a column block is multiplied
  load(cb + 128 * w, 0);
  auto back = [&](int c0) { return max(0, c0 + 8 * i + 8 - a.m); };  // columns past the end of a row
  if (cb + 128 * w < a.m) ad_load_base<MF>(old, a.base, out, cb + 128 * w, back(cb + 128 * w), a.m);
  if (one) {
    fill(0);
    __syncthreads();
  }
  const int stop = cb + 512 * nc;
  for (int c0 = cb + 128 * w; c0 < stop; c0 += 512) {
    f32x4 acc[MF][8];
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int f = 0; f < 8; ++f) acc[g][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int rank0 = 0; rank0 < a.rp; rank0 += kAdChunk) {
      if (!one) {  // every wave comes here as often
        __syncthreads();
        fill(rank0);
        __syncthreads();
      }
      for (int s = 0; s < min(wide, a.rp - rank0); s += 32) {
        ad_put_u(u, us, a.r, rank0 + s);
        if (rank0 + s + 32 < a.rp) load(c0, rank0 + s + 32);
        else if (c0 + 512 < stop) load(c0 + 512, 0);
        u32x4 t[2][MF];
#pragma unroll
        for (int g = 0; g < MF; ++g)
#pragma unroll
          for (int h = 0; h < 2; ++h) t[h][g] = *reinterpret_cast<const u32x4*>(trow[g] + h * wide + s);
#pragma unroll
        for (int f0 = 0; f0 < 8; f0 += 4) {
          u32x4 uf[4];
#pragma unroll
          for (int f = 0; f < 4; ++f) uf[f] = *reinterpret_cast<const u32x4*>(us + ad_place(i, f0 + f, q));
          __builtin_amdgcn_sched_barrier(0);  // four reads, then their products
#pragma unroll
          for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int g = 0; g < MF; ++g)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                acc[g][f0 + f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t[h][g]), as_bf16(uf[f]), acc[g][f0 + f], 0, 0, 0);
        }
        ad_wave_sync();
      }
    }
    if (c0 >= a.m) continue;
    const bool full = c0 + 128 <= a.m;
#pragma unroll
    for (int g = 0; g < MF; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) v[f] = acc[g][f][e];
        if (16 * g + 4 * q + e >= at.rows) continue;
        if (full) ad_store8(a.Y, out[g][e] + 2u * c0, old[g][e], v);
        else ad_store8_end(a.Y, out[g][e] + 2u * c0, old[g][e], v, back(c0), a.m);
      }
    if (c0 + 512 < min(stop, a.m)) ad_load_base<MF>(old, a.base, out, c0 + 512, back(c0 + 512), a.m);
  }
}

// ---------------------------------------------------------------------------
// Both in one launch, for a few rows and small factors: each block makes all of its
// tile's T for itself (16 waves share K), then its columns of Y.  Vt_l comes from L2
// for all blocks but the first; a launch, a round trip of T through memory and a
// workspace are saved.  One row 4096 x 4096 r 16: 7.0 us, a launch and a chain of loads.
// grid: (tiles, column blocks of 512 NC)
// ---------------------------------------------------------------------------
static constexpr int kAdFusedWaves = 16, kAdFusedColumns = 8;

template <int NR>
__global__ __launch_bounds__(64 * kAdFusedWaves) void k_ad_fused(AdArgs a, int nc) {
  constexpr int TM = 16, XL = TM / 8, VL = 2 * NR, UN = NR == 1 ? 4 : 2;  // units in flight
  constexpr int kStage = (TM + 16 * NR) * kAdUnit, kPitch = 2 * 32 + 8;
  __shared__ __align__(16) uint16_t lds[kAdFusedWaves * kStage];  // a wave's unit; the waves' sums; U of the columns
  __shared__ __align__(16) uint16_t terms[TM * kPitch];           // [row][term][32]
  __shared__ uint16_t rows[TM];
  static_assert(kAdFusedWaves * kStage >= kAdFusedWaves * NR * 64 * 8 &&
                    kAdFusedWaves * kStage >= kAdFusedColumns * 128 * 32, "what shares LDS fits");
  const AdTile at = ad_tile<TM>(a, blockIdx.x, rows, nullptr, nullptr, nullptr);
  if (at.rows == 0) return;
  const int cb = (int)blockIdx.y * 512 * nc;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 512 * nc, a.m);
    return;
  }
  const int adapter = uniform(at.adapter), live = uniform(at.rows);
  const int w = uniform((int)threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int c8 = lane & 7, r8 = lane >> 3, K = a.n, units = (K + kAdUnit - 1) / kAdUnit, whole = K / kAdUnit;
  uint16_t* xs = lds + w * kStage;
  uint16_t* vs = xs + TM * kAdUnit;
  const uint16_t* V = a.Vt + (int64_t)adapter * a.r * K;
  const float scale = a.scale ? a.scale[adapter] : 1.f;
  int xrow[XL], vrow[VL];
#pragma unroll
  for (int j = 0; j < XL; ++j) xrow[j] = rows[min(8 * j + r8, live - 1)] * K;
#pragma unroll
  for (int j = 0; j < VL; ++j) vrow[j] = min(8 * j + r8, a.r - 1) * K;
  f32x4 acc[NR];
#pragma unroll
  for (int g = 0; g < NR; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const u32x4 (&x)[XL], const u32x4 (&v)[VL]) {
#pragma unroll
    for (int j = 0; j < XL; ++j) *reinterpret_cast<u32x4*>(xs + ad_slot(8 * j + r8, c8)) = x[j];
#pragma unroll
    for (int j = 0; j < VL; ++j) *reinterpret_cast<u32x4*>(vs + ad_slot(8 * j + r8, c8)) = v[j];
    ad_wave_sync();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 xf = *reinterpret_cast<const u32x4*>(xs + ad_slot(i, 4 * h + q));
#pragma unroll
      for (int g = 0; g < NR; ++g) {
        const u32x4 vf = *reinterpret_cast<const u32x4*>(vs + ad_slot(16 * g + i, 4 * h + q));
        acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(vf), as_bf16(xf), acc[g], 0, 0, 0);
      }
    }
    ad_wave_sync();
  };
  for (int u0 = w; u0 < units; u0 += UN * kAdFusedWaves) {
    u32x4 x[UN][XL] = {}, v[UN][VL];  // (rows that the tile lacks: zeros)
#pragma unroll
    for (int p = 0; p < UN; ++p) {
      const int u = u0 + p * kAdFusedWaves;
      if (u < whole) {
#pragma unroll
        for (int j = 0; j < XL; ++j)
          if (8 * j + r8 < live) x[p][j] = ad_load(a.X, 2u * (xrow[j] + u * kAdUnit + 8 * c8));
#pragma unroll
        for (int j = 0; j < VL; ++j) v[p][j] = ad_load(V, 2u * (vrow[j] + u * kAdUnit + 8 * c8));
      }
    }
#pragma unroll
    for (int p = 0; p < UN; ++p) {
      const int u = u0 + p * kAdFusedWaves;
      if (u >= units) break;
      if (u >= whole) {  // the unit in which the rows end
#pragma unroll
        for (int j = 0; j < XL; ++j) x[p][j] = ad_tail8(a.X + xrow[j], u * kAdUnit + 8 * c8, K);
#pragma unroll
        for (int j = 0; j < VL; ++j) v[p][j] = ad_tail8(V + vrow[j], u * kAdUnit + 8 * c8, K);
      }
      multiply(x[p], v[p]);
    }
  }
  // the columns' U and base are on their way while the waves' sums meet
  const uint16_t* U = a.U + (int64_t)adapter * a.m * a.r;
  const int stop = min(cb + 512 * nc, a.m);
  uint32_t out[1][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) out[0][e] = 2u * (rows[min(4 * q + e, live - 1)] * a.m + 8 * i);
  u32x4 u[8], old[1][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) old[0][e] = u32x4{0u, 0u, 0u, 0u};
  auto back = [&](int c0) { return max(0, c0 + 8 * i + 8 - a.m); };  // columns past the end of a row
  auto load = [&](int c0) {
    ad_load_u(u, U, a.m, a.r, c0, 0);
    ad_load_base<1>(old, a.base, out, c0, back(c0), a.m);
  };
  const int first = cb + 128 * w;
  if (first < stop && w < kAdFusedColumns) load(first);
  f32x4* sum = reinterpret_cast<f32x4*>(lds);  // [waves][NR][64]
  __syncthreads();
#pragma unroll
  for (int g = 0; g < NR; ++g) sum[(w * NR + g) * 64 + lane] = acc[g];
  __syncthreads();
  if (w < 2) {  // wave g: ranks 16 g + 4 q .. + 3 of row i, as terms; zeros past r
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
    if (w < NR) {
      f32x4 part[kAdFusedWaves];
#pragma unroll
      for (int k = 0; k < kAdFusedWaves; ++k) part[k] = sum[(k * NR + w) * 64 + lane];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kAdFusedWaves; ++k) t += part[k];
    }
    const int rank = 16 * w + 4 * q;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = rank + e < a.r ? t[e] * scale : 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = ad_term2(x[0], x[1]), hi = ad_term2(x[2], x[3]);
      *reinterpret_cast<mx_u32x2*>(terms + i * kPitch + 32 * h + rank) = mx_u32x2{lo, hi};
    }
  }
  __syncthreads();
  u32x4 t[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) t[h] = *reinterpret_cast<const u32x4*>(terms + i * kPitch + 32 * h + 8 * q);
  // 8 KB of LDS a wave: the first half of the waves take columns at a time
  uint16_t* us = lds + w * 128 * 32;
  for (int c0 = first; c0 < stop && w < kAdFusedColumns; c0 += 128 * kAdFusedColumns) {
    ad_put_u(u, us, a.r, 0);
    f32x4 y[8];
    u32x4 uf[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) uf[f] = *reinterpret_cast<const u32x4*>(us + ad_place(i, f, q));
    __builtin_amdgcn_sched_barrier(0);  // all reads, then the products: one wait instead of eight
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      y[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) y[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t[h]), as_bf16(uf[f]), y[f], 0, 0, 0);
    }
    ad_wave_sync();
    const bool full = c0 + 128 <= a.m;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) v[f] = y[f][e];
      if (4 * q + e >= live) continue;
      if (full) ad_store8(a.Y, out[0][e] + 2u * c0, old[0][e], v);
      else ad_store8_end(a.Y, out[0][e] + 2u * c0, old[0][e], v, back(c0), a.m);
    }
    if (c0 + 128 * kAdFusedColumns < stop) load(c0 + 128 * kAdFusedColumns);
  }
}

// ---------------------------------------------------------------------------
// The backward's last launch: blocks of dU, then of dVt (the long ones first), then of
// dX.  Bound by memory (2048 rows 4096 x 4096 r 16: 19 us for 68 MB, 3.6 TB/s) unless one
// adapter has most of the rows, whose blocks are a chain of 32 at a time, 1 us each (2048
// rows 11008 x 4096 of 8, r 64: 31 us for 126 MB with the rows about even, 42 else).
// ---------------------------------------------------------------------------
// dX = base + scale P Vt: as k_ad_expand, with Vt's 8 x 8 pieces transposed in
// registers: a lane's eight ranks and eight columns are eight operands.
__device__ __forceinline__ void ad_dx(const AdArgs& a, int block) {
  constexpr int MF = 2;
  const int tile = block / a.cols_y, cb = block % a.cols_y * 512;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int2 info = a.info[tile];
  const uint16_t* rows = a.rows + 32 * tile;
  const uint16_t* t2 = a.t2 + ((int64_t)tile * (a.rp >> 5) * 4 * 64 + lane) * 8;
  uint32_t out[MF][4];  // byte offsets (of a tile that is not there: any number, not used)
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) out[g][e] = 2u * (rows[16 * g + 4 * q + e] * a.n + 8 * i);
  const AdTile at = {uniform(info.x), uniform(info.y)};
  if (at.rows == 0) return;
  if (at.adapter < 0) {
    ad_copy(a, at, rows, cb, 512, a.n);
    return;
  }
  const int c0 = cb + 128 * w, col = c0 + 8 * i;
  if (c0 >= a.n) return;
  const uint16_t* V = a.Vt + (int64_t)at.adapter * a.r * a.n;
  const bool full = c0 + 128 <= a.n;
  u32x4 old[MF][4];
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) old[g][e] = u32x4{0u, 0u, 0u, 0u};
  const int back = max(0, col + 8 - a.n);  // columns past the end of a row
  ad_load_base<MF>(old, a.base, out, c0, back, a.n);
  f32x4 acc[MF][8];
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[g][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int from = col - back;
  for (int s = 0; s < a.rp; s += 32) {
    // past the ranks: the last one again, times the zeros that the terms hold there
    AdPiece<8> v[8];
    if (a.n >= 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(AdPiece<8>, ad_load(V, 2u * (min(s + 8 * q + e, a.r - 1) * a.n + from)));
      if (!full) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = ad_drop<8>(v[e], col - from);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = ad_piece_end<8>(V + min(s + 8 * q + e, a.r - 1) * a.n, i == 0 ? a.n : 0);
    }
    u32x4 t[2][MF];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < MF; ++g) t[h][g] = *reinterpret_cast<const u32x4*>(t2 + (4 * (s >> 5) + 2 * h + g) * 64 * 8);
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const bf16x8 u = as_bf16(ad_column<8>(v, f));
#pragma unroll
      for (int g = 0; g < MF; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[g][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t[h][g]), u, acc[g][f], 0, 0, 0);
    }
  }
#pragma unroll
  for (int g = 0; g < MF; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) v[f] = acc[g][f][e];
      if (16 * g + 4 * q + e >= at.rows) continue;
      if (full) ad_store8(a.Y, out[g][e] + 2u * c0, old[g][e], v);
      else ad_store8_end(a.Y, out[g][e] + 2u * c0, old[g][e], v, back, a.n);
    }
}

// A wave's part of dU_l (m x r) or dVt_l (r x n): D[rank][column], a lane has ranks
// 4 q .. 4 q + 3 of columns CW i + f.  Four ranks of a row of dU, or CW columns of
// a row of dVt, are one store.
template <int NR, int CW, bool DV>
__device__ __forceinline__ void ad_store_factor(const AdArgs& a, int l, int rank0, int c0, const f32x4 (&acc)[CW][NR]) {
  typedef float Packed __attribute__((ext_vector_type(DV ? CW : 4), aligned(4)));
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4, cols = DV ? a.n : a.m, col0 = c0 + CW * i;
  float* out = (DV ? a.dVt : a.dU) + (int64_t)l * a.r * cols;
#pragma unroll
  for (int g = 0; g < NR; ++g) {
    const int rank = rank0 + 16 * g + 4 * q;
    if constexpr (DV) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (rank + e >= a.r) break;
        float* at = out + (int64_t)(rank + e) * cols + col0;
        if (col0 + CW <= cols) {
          Packed v;
#pragma unroll
          for (int f = 0; f < CW; ++f) v[f] = acc[f][g][e];
          *reinterpret_cast<Packed*>(at) = v;
        } else {
#pragma unroll
          for (int f = 0; f < CW; ++f)
            if (col0 + f < cols) at[f] = acc[f][g][e];
        }
      }
    } else {
#pragma unroll
      for (int f = 0; f < CW; ++f) {
        if (col0 + f >= cols) break;
        float* at = out + (int64_t)(col0 + f) * a.r + rank;
        if (rank + 4 <= a.r) {
          *reinterpret_cast<Packed*>(at) = acc[f][g];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (rank + e < a.r) at[e] = acc[f][g][e];
        }
      }
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
    tile0 = uniform(first.x), total = uniform(first.y);
  } else {  // a tile starts at each 32nd of its rows
    same = __ballot(lane < a.b && a.ids[min(lane, a.b - 1)] == l);
    total = __popcll(same);
  }
  const uint16_t* src = DV ? a.X : a.G;
  const uint16_t* terms = a.t3[DV] + lane * 8;
  const int groups = a.rg >> 4;
  f32x4 acc[CW][NR];
#pragma unroll
  for (int f = 0; f < CW; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Rows past the end: a row of the tile again, times the zeros that the terms
  // hold there.
  const bool inside = c0 + 16 * CW <= cols;
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
  auto load_terms = [&](int tile, int g, u32x4 (&t)[3]) {  // (past the ranks: the last ones, not stored)
    const int64_t from = ((int64_t)tile * groups + min(rank0 / 16 + g, groups - 1)) * 3 * 64 * 8;
#pragma unroll
    for (int h = 0; h < 3; ++h) t[h] = *reinterpret_cast<const u32x4*>(terms + from + h * 64 * 8);
  };
  auto load = [&](int s, Regs& r) {
    const int tile = tile_of(s), pos = 32 * tile, left = total - 32 * s;
    if (NR <= 2) {
#pragma unroll
      for (int g = 0; g < NR; ++g) load_terms(tile, g, r.t[g]);
    }
    int row[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) row[e] = list[pos + min(8 * q + e, left - 1)] * cols;
    if (inside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_piece_at<CW>(src, 2u * (row[e] + c0 + CW * i));
    } else if (cols >= CW) {
      const int from = min(c0 + CW * i, cols - CW);
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_drop<CW>(ad_piece_at<CW>(src, 2u * (row[e] + from)), c0 + CW * i - from);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_piece_end<CW>(src + row[e], i == 0 ? cols : 0);
    }
  };
  auto multiply = [&](int s, const Regs& r) {
    const int tile = tile_of(s);
#pragma unroll
    for (int g = 0; g < NR; ++g) {
      u32x4 t[3];
      if (NR <= 2) {
#pragma unroll
        for (int h = 0; h < 3; ++h) t[h] = r.t[g][h];
      } else {
        load_terms(tile, g, t);
      }
#pragma unroll
      for (int f = 0; f < CW; ++f) {
        const bf16x8 x = as_bf16(ad_column<CW>(r.v, f));
#pragma unroll
        for (int h = 0; h < 3; ++h)
          acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(t[h]), x, acc[f][g], 0, 0, 0);
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
  ad_store_factor<NR, CW, DV>(a, l, rank0, c0, acc);
}

// The same where there are many columns in all: the block's waves take 64 columns
// each and all of the adapter's rows, and share a tile's terms through LDS (12 KB of
// 64 ranks, one contiguous piece in memory; the next tile's are on their way).
template <bool DV>
__device__ __forceinline__ void ad_dfactor_wide(const AdArgs& a, int block, char* smem) {
  constexpr int NR = 4, CW = 4, kTerms = NR * 3 * 64;  // 16-byte pieces of a tile's terms
  const int cols = DV ? a.n : a.m, blocks = DV ? a.cols_v : a.cols_u;
  const int rest = block / blocks, rank0 = rest % a.chunks * 16 * NR, l = rest / a.chunks;
  const int t = threadIdx.x, w = t >> 6, lane = t & 63, i = lane & 15, q = lane >> 4;
  const int c0 = block % blocks * 64 * CW + w * 16 * CW;
  const int2 first = a.first[l];
  const int tile0 = uniform(first.x), total = uniform(first.y), steps = (total + 31) / 32;
  const int groups = a.rg >> 4, pieces = min(NR, groups - rank0 / 16) * 3 * 64;
  const uint16_t* src = DV ? a.X : a.G;
  const u32x4* terms = reinterpret_cast<const u32x4*>(a.t3[DV]) + rank0 / 16 * 3 * 64;
  u32x4* buf = reinterpret_cast<u32x4*>(smem);  // [2][kTerms]
  f32x4 acc[CW][NR];
#pragma unroll
  for (int f = 0; f < CW; ++f)
#pragma unroll
    for (int g = 0; g < NR; ++g) acc[f][g] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool inside = c0 + 16 * CW <= cols;
  const int from = min(c0 + CW * i, cols - CW), drop = c0 + CW * i - from;
  struct Regs {
    AdPiece<CW> v[8];
  };
  auto load = [&](int s, Regs& r) {
    const int pos = 32 * (tile0 + s);
    int row[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) row[e] = a.rows[pos + 8 * q + e] * cols;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = ad_piece_at<CW>(src, 2u * (row[e] + from));
  };
  u32x4 next[3];
  auto load_terms = [&](int s) {  // (past the ranks: the last piece again, not stored)
    const u32x4* p = terms + (int64_t)(tile0 + s) * groups * 3 * 64;
#pragma unroll
    for (int k = 0; k < 3; ++k) next[k] = p[min(256 * k + t, pieces - 1)];
  };
  auto put_terms = [&](int s) {
#pragma unroll
    for (int k = 0; k < 3; ++k) buf[(s & 1) * kTerms + 256 * k + t] = next[k];
  };
  auto multiply = [&](int s, Regs& r) {
    if (!inside) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r.v[e] = ad_drop<CW>(r.v[e], drop);
    }
    u32x4 x[CW];
#pragma unroll
    for (int f = 0; f < CW; ++f) x[f] = ad_column<CW>(r.v, f);
#pragma unroll
    for (int g = 0; g < NR; ++g)
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        const u32x4 y = buf[(s & 1) * kTerms + (3 * g + h) * 64 + lane];
#pragma unroll
        for (int f = 0; f < CW; ++f)
          acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(y), as_bf16(x[f]), acc[f][g], 0, 0, 0);
      }
  };
  if (steps > 0) {
    Regs ra, rb;
    load_terms(0), load(0, ra);
    put_terms(0);
    __syncthreads();
    for (int s = 0; s < steps; s += 2) {  // the block's waves go through it together
      load_terms(min(s + 1, steps - 1)), load(min(s + 1, steps - 1), rb);
      multiply(s, ra);
      put_terms(s + 1);
      __syncthreads();
      if (s + 1 >= steps) break;
      load_terms(min(s + 2, steps - 1)), load(min(s + 2, steps - 1), ra);
      multiply(s + 1, rb);
      put_terms(s + 2);
      __syncthreads();
    }
  }
  ad_store_factor<NR, CW, DV>(a, l, rank0, c0, acc);
}

__global__ __launch_bounds__(256, 2) void k_ad_back_wide(AdArgs a) {
  extern __shared__ __align__(16) char smem[];
  int block = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (block >= a.blocks_u + a.blocks_v + a.blocks_y) return;
  if (block < a.blocks_u) {
    ad_dfactor_wide<false>(a, block, smem);
    return;
  }
  block -= a.blocks_u;
  if (block < a.blocks_v) {
    ad_dfactor_wide<true>(a, block, smem);
    return;
  }
  ad_dx(a, block - a.blocks_v);
}

template <int NR, int CW>
__global__ __launch_bounds__(256, 2) void k_ad_back(AdArgs a) {
  extern __shared__ __align__(16) char smem[];
  int block = (int)(blockIdx.y * gridDim.x + blockIdx.x);
  if (block >= a.blocks_u + a.blocks_v + a.blocks_y) return;
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
  int tm, nr, tiles, slots, rp, rg, splits[2], units[2], direct;
  size_t part[2], t2, t3[2], info, rows, first, total;  // offsets in the workspace
};

// K splits of `units` a block takes `per` of (whole ones for the four waves).
static void ad_split(int K, int per, int* splits, int* units) {
  const int all = (K + kAdUnit - 1) / kAdUnit;
  *splits = (all + per - 1) / per;
  *units = (all + *splits - 1) / *splits;
  *splits = (all + *units - 1) / *units;
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
  const int busy = std::max((b + p.tm - 1) / p.tm, std::min(b, A->count)) * groups;
  // the same share of K for each block, whatever side it is on
  const int64_t all = (int64_t)busy * ((A->n + kAdUnit - 1) / kAdUnit + (grad ? (A->m + kAdUnit - 1) / kAdUnit : 0));
  int per = (int)std::max<int64_t>(4, (all + kAdBlocks - 1) / kAdBlocks);
  // Short rows of a few tiles are not split: a launch (k_ad_terms) less.
  const int longest = (std::max(A->m, A->n) + kAdUnit - 1) / kAdUnit;
  if (grad && longest <= kAdWhole) per = std::max(per, longest);
  p.direct = grad && per >= longest;
  ad_split(A->n, per, &p.splits[0], &p.units[0]);
  ad_split(A->m, per, &p.splits[1], &p.units[1]);
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
  const size_t lds = std::max<size_t>((size_t)4 * (TM + 16 * NR) * kAdUnit * 2, (size_t)ad_bins(a.count) * 4);
  static_assert(4 * (TM + 16 * NR) * kAdUnit * 2 >= 4 * (TM / 16) * NR * 64 * 16, "the waves' sums fit");
  const dim3 grid(ad_work_blocks(a.tiles, a.splits[0] + a.splits[1]), (a.rg + 16 * NR - 1) / (16 * NR));
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
  const int cols = (a.m + 511) / 512;
  const int nc = std::max(1, std::min(cols, cols * busy / 256));
  const dim3 grid(a.tiles, (cols + nc - 1) / nc);
  const size_t lds = (size_t)(4 * 128 * 32 + TM * (2 * std::min(a.rp, kAdChunk) + 8)) * 2;
  if (a.r >= 8) hipLaunchKernelGGL((k_ad_expand<TM, false>), grid, dim3(256), lds, s, a, nc);
  else hipLaunchKernelGGL((k_ad_expand<TM, true>), grid, dim3(256), lds, s, a, nc);
}

// One launch: up to 64 rows, and a Vt_l that a block reads in the time that a launch
// takes (at most 256 KB with its ranks rounded up to 16).  In one / in two, 4096
// columns of Y and an adapter a row: n 4096 r 16, 1 row 6.9 / 8.4 us, 64 rows 8.6 /
// 11.6; n 4096 r 32, 64 rows 11.8 / 13.2; n 8192 r 16, 1 row 9.0 / 9.8, 64 rows
// 11.8 / 12.6; past the limit n 16384 r 16, 1 row 13.7 / 12.9, 64 rows 16.9 / 14.7.
static bool ad_fused(const hss_adapters* A, int b) {
  const int nr = (A->r + 15) / 16;
  return b <= kAdSmall && A->r >= 8 && nr <= 2 && A->n >= 8 && nr * (int64_t)A->n <= 8192;
}

hss_status launch_adapters_apply(const hss_adapters* A, int b, const void* X, const int32_t* ids, const void* base,
                                 void* Y, void* ws, hipStream_t s) {
  const AdPlan p = ad_plan(A, b, false);
  AdArgs a = ad_args(A, b, p, X, ids, base, Y, ws);
  a.first = nullptr;
  if (ad_fused(A, b)) {
    // at most a block for each compute unit: each makes its tile's T again (64 rows
    // 11008 x 4096 r 16: 11.7 us, 16.5 with 320 blocks)
    const int cols = (a.m + 511) / 512, nc = std::max(1, (int)std::min<int64_t>(cols, ((int64_t)cols * a.tiles + 255) / 256));
    const dim3 grid(a.tiles, (cols + nc - 1) / nc), block(64 * kAdFusedWaves);
    if (a.r <= 16) hipLaunchKernelGGL(k_ad_fused<1>, grid, block, 0, s, a, nc);
    else hipLaunchKernelGGL(k_ad_fused<2>, grid, block, 0, s, a, nc);
  } else if (p.tm == 16) launch_rank<16>(a, p.nr, s), launch_expand<16>(a, s);
  else launch_rank<32>(a, p.nr, s), launch_expand<32>(a, s);
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

// k_ad_back's blocks for dU and dVt of `width` columns by `ranks` ranks.
static dim3 ad_back_grid(AdArgs& a, int width, int ranks) {
  a.chunks = (a.rg + ranks - 1) / ranks;
  a.cols_u = (a.m + width - 1) / width, a.cols_v = (a.n + width - 1) / width, a.cols_y = (a.n + 511) / 512;
  a.blocks_u = a.dU ? a.cols_u * a.chunks * a.count : 0;
  a.blocks_v = a.dVt ? a.cols_v * a.chunks * a.count : 0;
  a.blocks_y = a.Y ? a.cols_y * a.tiles : 0;
  // (a launch takes fewer than 2^32 threads along x)
  const unsigned all = (unsigned)a.blocks_u + a.blocks_v + a.blocks_y, x = std::min(all, 1u << 22);
  return dim3(x, (all + x - 1) / x);
}

template <int NR, int CW>
static void launch_back(AdArgs a, hipStream_t s) {
  const dim3 grid = ad_back_grid(a, 16 * CW, 16 * NR);
  hipLaunchKernelGGL((k_ad_back<NR, CW>), grid, dim3(256), (size_t)CW * NR * 64 * 16, s, a);
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
  a.direct = p.direct;
  launch_rank<32>(a, p.nr, s);
  if (!a.direct) {
    const dim3 grid(a.tiles, (a.rp + 63) / 64, a.splits[0] && a.splits[1] ? 2 : 1);
    hipLaunchKernelGGL(k_ad_terms, grid, dim3(256), 0, s, a);
  }
  // dU and dVt by blocks of 256 columns that share the terms, where there are enough of
  // them; else by blocks of 64 whose waves share the rows.  The first walk all of an
  // adapter's rows one tile after another, so that many rows an adapter ask for more of
  // them (us with 256 and with 64, rows even):
  //   2048 rows an adapter: 118 blocks (11008 x 4096 r 128 of 1) 103 and 90, 128 (8192 x
  //     8192 r 128) 103 and 93, 144 (8192 x 4096 r 192) 104 and 111, 236 (11008 x 4096 r 256) 123 and 143
  //   1024: 118 (11008 x 4096 r 64 of 2) 64.9 and 60.6, 128 (4096 x 4096 r 256 of 1) 54.8
  //     and 51.9, (8192 x 8192 r 64 of 2) 65.7 and 68.0, 150 (11008 x 8192 of 2) 75.6 and 83.9
  //   682: 96 (4096 x 4096 r 64 of 3) 45.4 and 42.2, 177 (11008 x 4096 of 3) 57.8 and 68.6
  //   512: 118 (11008 x 4096 r 128 of 1) 38.4 and 38.9, 128 (4096 x 4096 r 64 of 4) 39.1 and 41.2
  //   256: 64 (4096 x 4096 r 64 of 2) 27.0 and 26.9, 118 (11008 x 4096 of 2) 29.0 and 31.0, 472
  //     (of 8) 61.6 and 76.7; with half of the 2048 rows on one adapter of the 8 76.7 and 75.7,
  //     all of them 110.6 and 75.5, which the host does not see.
  // With up to 32 ranks there are few terms to share.
  // Very few columns in all are split further, 32 a block (r 16, 512 rows 1024 x 1024
  // of 1 13.8 and 15.1 us, of 4, where the rule ends, 13.9 and 12.8; r 64, 201 rows
  // 1501 x 2777 of 1 18.8 and 21.0, of 2 20.1 and 19.6).
  const int64_t passes = (int64_t)A->count * ((A->r + 63) / 64);
  const int64_t wide = passes * (((int64_t)A->m + 255) / 256 + (A->n + 255) / 256);
  const int64_t enough = b / std::min(b, A->count) >= 640 ? 136 : 96;
  const bool narrow = passes * ((int64_t)A->m + A->n) < 64 * 128;
  if (b > kAdSmall && p.nr == 4 && wide >= enough && std::min(A->m, A->n) >= 4) {  // (rows of a piece at least)
    const dim3 grid = ad_back_grid(a, 256, 64);
    hipLaunchKernelGGL(k_ad_back_wide, grid, dim3(256), 2 * 4 * 3 * 64 * 16, s, a);
  } else if (p.nr == 1) {
    narrow ? launch_back<1, 2>(a, s) : launch_back<1, 8>(a, s);
  } else if (p.nr == 2) {
    narrow ? launch_back<2, 2>(a, s) : launch_back<2, 4>(a, s);
  } else {
    narrow ? launch_back<4, 2>(a, s) : launch_back<4, 4>(a, s);
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
