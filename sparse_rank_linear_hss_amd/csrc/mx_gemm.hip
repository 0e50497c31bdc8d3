// HSS_MX4 apply for a middle range of columns, in both directions, straight
// from the 4-bit codes:  P = X [D | U]^T with T behind X, then Y = P + X S^T.
//
// k_mx_gemm: tiles of 128 outputs x BN columns, K in stages of 64 through two
// LDS buffers.  The codes' tile is decoded on its way to LDS: a thread takes
// one group (16 bytes, 32 columns) of one row or, where the stored array is
// the transpose, 8 columns x 4 rows of it, decoded row by row (a scale belongs
// to a stored row) and paired up along K by byte permutes.  So a stage brings
// 4 KiB of codes where a dense copy would bring 16, and no dense copy is made.
// K is split over blocks where the tiles are few; the partial products are
// added in order by k_mx_finish, which also adds S: eight lanes per entry read
// the entry's row of X^T (64 columns).
//
// Against the dense copy and the large tiles: chosen by mx_gemm_supported.
#include <algorithm>

#include "mx_common.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

static constexpr int kMgM = 128, kMgK = 64;
static constexpr int kMgBlocks = 256;                // blocks wanted: one per CU
static constexpr int kMgMaxCols = 256;
static constexpr int kFinRows = 32, kFinCols = 64;  // k_mx_finish's tile

struct MxGemmArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const uint16_t* X;   // b rows of ldx (a multiple of 64, zero past n)
  const uint16_t* U;   // m rows of rp (a multiple of 32, zero past r)
  const uint16_t* Tb;  // b rows of 2 rp: the two terms of T
  void* C;             // bf16 Y (b x m), or fp32 partial products [z][m][ldp]
  int m, n, b, r, rp, ldx, ldp, ng;
  int nst1, nst, stages_per_split, tiles_m, tiles_n, partial;
};

// Slot of 16-byte chunk c (0..7) of a 128-byte LDS row r: distinct over the
// rows that a fragment read takes together, and spread over rows 8 apart, as
// the transposed decode writes them.
__device__ __forceinline__ int mg_slot(int r, int c) { return c ^ ((r >> 1) & 7) ^ ((r & 1) << 2) ^ ((r >> 3) & 3); }

template <bool TRANS, int BN>
__global__ __launch_bounds__(256, 2) void k_mx_gemm(MxGemmArgs a) {
  constexpr int FN = BN / 32, BV = BN / 32;  // column blocks per wave; 16-byte loads of X per thread
  __shared__ __align__(16) uint16_t lds[2][(kMgM + BN) * kMgK];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int tn = (int)blockIdx.x % a.tiles_n, rest = (int)blockIdx.x / a.tiles_n;
  const int tm = rest % a.tiles_m, z = rest / a.tiles_m;
  const int m0 = tm * kMgM, n0 = tn * BN;
  const int s0 = z * a.stages_per_split, s1 = min(s0 + a.stages_per_split, a.nst);

  f32x16 acc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[j][v] = 0.f;

  // A stage in registers.  Direct codes: cw is the thread's group (row t / 2,
  // half t % 2).  Transposed: cw[i] the codes of stored row 4 (t / 16) + i,
  // columns 8 (t % 16) ..  U's stages: u[0..3], the 32 columns of the group's
  // place.  xb: 8 columns of rows t / 8 + 32 i of X (of T's terms).
  const int arow = t >> 1, ah = t & 1, jb = t & 15, ib = t >> 4;
  struct CodeRegs {
    u32x4 cw, xb[BV];
    uint32_t sc[4];
  };
  struct URegs {
    u32x4 u[4], xb[BV];
  };
  const uint16_t* xrow[BV];
#pragma unroll
  for (int i = 0; i < BV; ++i) xrow[i] = a.X + (int64_t)min(n0 + (t >> 3) + 32 * i, a.b - 1) * a.ldx + 8 * (t & 7);
  auto load_codes = [&](int s, CodeRegs& r) {
    if constexpr (TRANS) {
      const int g = min((m0 >> 5) + (jb >> 2), a.ng - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // stored rows past the end repeat the last one, against zeros of X;
        // store_codes gives them a finite scale
        const uint32_t at = (uint32_t)min(s * kMgK + 4 * ib + i, a.n - 1) * (uint32_t)a.ng + (uint32_t)g;
        r.cw[i] = *reinterpret_cast<const uint32_t*>(a.codes + at * 16 + 4 * (jb & 3));
        r.sc[i] = a.scales[at];
      }
    } else {  // a group past the end: the row's last one, against zeros of X
      const uint32_t at = (uint32_t)min(m0 + arow, a.m - 1) * (uint32_t)a.ng + (uint32_t)min(2 * s + ah, a.ng - 1);
      r.cw = *reinterpret_cast<const u32x4*>(a.codes + at * 16);
      r.sc[0] = a.scales[at];
    }
#pragma unroll
    for (int i = 0; i < BV; ++i) r.xb[i] = *reinterpret_cast<const u32x4*>(xrow[i] + s * kMgK);
  };
  auto store_x = [&](uint16_t* buf, const u32x4 (&xb)[BV]) {
#pragma unroll
    for (int i = 0; i < BV; ++i) {
      const int row = (t >> 3) + 32 * i;
      *reinterpret_cast<u32x4*>(buf + (kMgM + row) * kMgK + 8 * mg_slot(row, t & 7)) = xb[i];
    }
  };
  auto store_codes = [&](int s, uint16_t* buf, const CodeRegs& r) {
    if constexpr (TRANS) {
      u32x4 d[4];  // d[i][p]: columns 2 p, 2 p + 1 of stored row i
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = mx4_to_bf16x8(r.cw[i], s * kMgK + 4 * ib + i < a.n ? mx_scale(r.sc[i], 0) : 1.f);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 8 * jb + 2 * p + h;
          const uint32_t sel = h ? 0x07060302u : 0x05040100u;  // the upper or lower halves of (row i, row i + 1)
          *reinterpret_cast<mx_u32x2*>(buf + row * kMgK + 8 * mg_slot(row, ib >> 1) + 4 * (ib & 1)) =
              mx_u32x2{__builtin_amdgcn_perm(d[1][p], d[0][p], sel), __builtin_amdgcn_perm(d[3][p], d[2][p], sel)};
        }
    } else {
      const float scale = mx_scale(r.sc[0], 0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<u32x4*>(buf + arow * kMgK + 8 * mg_slot(arow, 4 * ah + e)) = mx4_to_bf16x8(r.cw[e], scale);
    }
    store_x(buf, r.xb);
  };
  auto load_u = [&](int s, URegs& r) {
    const int k = (s - a.nst1) * kMgK + 32 * ah;  // of 2 rp; 32 columns lie within one term
    const uint16_t* row = a.U + (int64_t)min(m0 + arow, a.m - 1) * a.rp + (k < a.rp ? k : k - a.rp);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.u[e] = *reinterpret_cast<const u32x4*>(row + 8 * e);
#pragma unroll
    for (int i = 0; i < BV; ++i)
      r.xb[i] = *reinterpret_cast<const u32x4*>(a.Tb + (int64_t)min(n0 + (t >> 3) + 32 * i, a.b - 1) * (2 * a.rp) +
                                                (s - a.nst1) * kMgK + 8 * (t & 7));
  };
  auto store_u = [&](int, uint16_t* buf, const URegs& r) {
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<u32x4*>(buf + arow * kMgK + 8 * mg_slot(arow, 4 * ah + e)) = r.u[e];
    store_x(buf, r.xb);
  };
  auto compute = [&](const uint16_t* buf) {  // wave w: rows 32 w .. of the tile
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int c = 2 * ks + (lane >> 5), row = 32 * w + (lane & 31);
      const bf16x8 af = *reinterpret_cast<const bf16x8*>(buf + row * kMgK + 8 * mg_slot(row, c));
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int rb = 32 * j + (lane & 31);
        const bf16x8 bf = *reinterpret_cast<const bf16x8*>(buf + (kMgM + rb) * kMgK + 8 * mg_slot(rb, c));
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af, bf, acc[j], 0, 0, 0);
      }
    }
  };
  // Stages from .. to: one computes from one LDS buffer while the next goes
  // from registers to the other and the one after that is on its way to the
  // other register set (past the end: the last one again, not used).
  auto run = [&](int from, int to, auto& ra, auto& rb, auto load, auto store) {
    if (from >= to) return;
    load(from, ra);
    load(min(from + 1, to - 1), rb);
    store(from, lds[0], ra);
    __syncthreads();
    // pairs of stages, then an odd last one: with an exit from the middle the
    // compiler moves the register sets about, and waits for their loads
    int s = from;
    for (; s + 1 < to; s += 2) {
      load(min(s + 2, to - 1), ra);
      __builtin_amdgcn_sched_barrier(0);  // the loads first: the compiler would sink them
      compute(lds[0]);
      store(s + 1, lds[1], rb);
      __syncthreads();
      load(min(s + 3, to - 1), rb);
      __builtin_amdgcn_sched_barrier(0);
      compute(lds[1]);
      store(min(s + 2, to - 1), lds[0], ra);
      __syncthreads();
    }
    if (s < to) {
      compute(lds[0]);
      __syncthreads();
    }
  };
  {
    CodeRegs ra, rb;
    run(s0, min(s1, a.nst1), ra, rb, load_codes, store_codes);
  }
  {
    URegs ra, rb;
    run(max(s0, a.nst1), s1, ra, rb, load_u, store_u);
  }
  // lane holds rows 8 (v / 4) + 4 (lane / 32) + v % 4 of column lane % 32
  const int nl = lane & 31, h = lane >> 5;
  if (a.partial) {  // part[z][row][c], rows of ldp
    float* P = static_cast<float*>(a.C) + (int64_t)z * a.m * a.ldp;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = m0 + 32 * w + 8 * (v >> 2) + 4 * h + (v & 3), c = n0 + 32 * j + nl;
        if (row < a.m && c < a.ldp) P[(int64_t)row * a.ldp + c] = acc[j][v];
      }
    return;
  }
  // Y: each wave stages 32 columns x its 32 rows (16-byte chunk k of column c
  // at k ^ c / 2 % 4), then writes 64 bytes per column
  uint16_t* stg = lds[0] + w * 1024;
  uint16_t* Y = static_cast<uint16_t*>(a.C);
  const bool vec = (uintptr_t)Y % 16 == 0 && a.m % 8 == 0;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
#pragma unroll
    for (int vg = 0; vg < 4; ++vg) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = f32_to_bf16(acc[j][4 * vg + e]);
      *reinterpret_cast<mx_u32x2*>(stg + nl * 32 + 8 * (vg ^ ((nl >> 1) & 3)) + 4 * h) =
          mx_u32x2{o[0] | o[1] << 16, o[2] | o[3] << 16};
    }
    // a wave's LDS accesses complete in order; the compiler is kept from moving them
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int cl = 16 * q + (lane >> 2), k = lane & 3;
      const u32x4 v = *reinterpret_cast<const u32x4*>(stg + cl * 32 + 8 * (k ^ ((cl >> 1) & 3)));
      const int c = n0 + 32 * j + cl, row = m0 + 32 * w + 8 * k;
      if (c < a.b) {
        uint16_t* o = Y + (int64_t)c * a.m + row;
        if (vec && row + 8 <= a.m) {
          *reinterpret_cast<u32x4*>(o) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row + e < a.m) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

// Tb[c][term][rp] = the two bf16 terms of T[c][l], the sum of its K splits
// Tp[z][c][rp] (zero for l >= r).
__global__ __launch_bounds__(256) void k_mx_tsum(const float* __restrict__ Tp, int splits, int b, int r, int rp,
                                                 uint16_t* __restrict__ Tb) {
  const int total = b * rp;
  for (int e = blockIdx.x * 256 + threadIdx.x; e < total; e += gridDim.x * 256) {
    const int c = e / rp, l = e - c * rp;
    float v = 0.f;
#pragma unroll 4
    for (int z = 0; z < splits; ++z) v += Tp[(int64_t)z * total + e];
    v = l < r ? v : 0.f;
    const uint16_t hi = f32_to_bf16(v);
    Tb[(int64_t)c * 2 * rp + l] = hi;
    // an infinity leaves 0, not the NaN of inf - inf
    Tb[((int64_t)c * 2 + 1) * rp + l] = (hi & 0x7fffu) == 0x7f80u ? (uint16_t)0 : f32_to_bf16(v - bf16lo(hi));
  }
}

void launch_mx_tsum(const float* Tp, int splits, int b, int r, int rp, uint16_t* Tb, hipStream_t s) {
  hipLaunchKernelGGL(k_mx_tsum, dim3((unsigned)std::min((b * rp + 255) / 256, 2048)), dim3(256), 0, s, Tp, splits, b, r,
                     rp, Tb);
}

// ---------------------------------------------------------------------------
// Y = the partial products, added in order, + X S^T.  A block owns 32 outputs
// (four rows of S per wave, 16 lanes each) and 64 columns; lane 8 e + h of a
// row takes its entries e, e + 2, .. and columns 8 h .. 8 h + 7 of X^T, eight
// entries in flight.
// ---------------------------------------------------------------------------
struct MxFinishArgs {
  const float* P;
  const int32_t* row_ptr;
  const void* col;
  const uint16_t* vals;
  const uint16_t* Xt;  // n x ldt
  uint16_t* Y;
  int m, n, b, ldt, ldp, splits, has_s, tiles_m;
};

template <typename COL>
__global__ __launch_bounds__(512) void k_mx_finish(MxFinishArgs a) {
  __shared__ float sy[kFinCols][kFinRows + 1];
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int row0 = (int)blockIdx.x % a.tiles_m * kFinRows, c0 = (int)blockIdx.x / a.tiles_m * kFinCols;
  // this thread's sums: column t % 64, rows t / 64 + 8 k
  float y[4];
  const float* p[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    p[k] = a.P + (int64_t)min(row0 + (t >> 6) + 8 * k, a.m - 1) * a.ldp + min(c0 + (t & 63), a.ldp - 1);
    y[k] = 0.f;
  }
#pragma unroll 4
  for (int z = 0; z < a.splits; ++z)
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] += p[k][(int64_t)z * a.m * a.ldp];
  if (a.has_s) {
    const int h = lane & 7, slot = (lane >> 3) & 1, i = 4 * w + (lane >> 4);
    const COL* col = static_cast<const COL*>(a.col);
    const uint16_t* xt = a.Xt + min(c0 + 8 * h, a.ldt - 8);
    int p0 = 0, p1 = 0;
    if (row0 + i < a.m) p0 = a.row_ptr[row0 + i], p1 = a.row_ptr[row0 + i + 1];
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int p = p0 + slot; p < p1; p += 16) {
      int j[8];
      float v[8];
      u32x4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int pp = min(p + 2 * q, p1 - 1);
        j[q] = (int)col[pp];
        v[q] = bf16lo(a.vals[pp]);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const bool ok = p + 2 * q < p1 && (unsigned)j[q] < (unsigned)a.n;
        x[q] = *reinterpret_cast<const u32x4*>(xt + (int64_t)(ok ? j[q] : 0) * a.ldt);
        if (!ok) v[q] = 0.f, x[q] = u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[2 * k] = fmaf(v[q], bf16lo(x[q][k]), s[2 * k]);
          s[2 * k + 1] = fmaf(v[q], bf16hi(x[q][k]), s[2 * k + 1]);
        }
    }
    // the two slots share out the eight columns: columns 8 h + 2 k + slot
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float mine = slot ? s[2 * k + 1] : s[2 * k], other = slot ? s[2 * k] : s[2 * k + 1];
      sy[8 * h + 2 * k + slot][i] = mine + __shfl_xor(other, 8, 64);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] += sy[t & 63][(t >> 6) + 8 * k];  // nobody else reads or writes these
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sy[t & 63][(t >> 6) + 8 * k] = y[k];
  __syncthreads();
  const int row = row0 + (t & 31);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = c0 + (t >> 5) + 16 * k;
    if (row < a.m && c < a.b) a.Y[(int64_t)c * a.m + row] = f32_to_bf16(sy[(t >> 5) + 16 * k][t & 31]);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

struct MxGemmPlan {
  MxPrep prep;
  int bn, nst1, nst, splits, stages_per_split, tiles_m, tiles_n, ldt, np;
  bool finish;  // partial products and k_mx_finish
  size_t tp, tb, xt, xp, up, part, total;
};

static MxGemmPlan plan_mx_gemm(const hss_matrix* A, int b) {
  MxGemmPlan p = {};
  p.prep = mx_prep_plan(A, b);
  // 128 columns a tile decode the codes once for twice the columns, in half the
  // blocks: for large products (us at 64 / 128: 8192^2, 128 columns 60 / 55,
  // input gradient 77 / 63; 4096^2, 256 columns 41 / 39, 49 / 44; but 128
  // columns 29 / 31, 33 / 32; 2049 x 1999, 256 columns 26 / 30, 25 / 27)
  const int64_t work = (int64_t)A->m * A->n * ((b + 127) / 128);
  const bool wide = b > 64 && work >= (int64_t)1 << ((A->flags & HSS_MX4_T) ? 24 : 25);
  p.bn = b <= 32 ? 32 : wide ? 128 : 64;
  p.tiles_m = (A->m + kMgM - 1) / kMgM;
  p.tiles_n = (b + p.bn - 1) / p.bn;
  p.nst1 = (A->n + kMgK - 1) / kMgK;
  p.nst = p.nst1 + (2 * p.prep.rp + kMgK - 1) / kMgK;
  const int tiles = p.tiles_m * p.tiles_n;
  // as few K splits as give every CU a block: 4096^2, 64 columns 14.4 us in 8
  // splits, 18.4 in 16 (twice the partial products)
  const int want = std::max(1, std::min({(kMgBlocks + tiles - 1) / tiles, p.nst / 4, 16}));
  p.stages_per_split = (p.nst + want - 1) / want;
  p.splits = (p.nst + p.stages_per_split - 1) / p.stages_per_split;
  p.finish = p.splits > 1 || A->nnz > 0;
  p.ldt = (b + 7) & ~7;
  p.np = (A->n + 63) & ~63;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += al256(bytes); return at; };
  p.tp = take((size_t)p.prep.splits * b * p.prep.rp * 4);
  p.tb = take((size_t)b * p.prep.rp * 4);
  p.xt = take(A->nnz > 0 ? (size_t)A->n * p.ldt * 2 : 0);
  p.xp = take((size_t)b * p.np * 2);
  p.up = take((size_t)A->m * p.prep.rp * 2);
  p.part = take(p.finish ? (size_t)p.splits * p.ldt * A->m * 4 : 0);
  p.total = off;
  return p;
}

size_t mx_gemm_ws_bytes(const hss_matrix* A, int b) { return plan_mx_gemm(A, b).total; }

template <bool TRANS>
static void launch_tile(const MxGemmArgs& a, int bn, unsigned grid, hipStream_t s) {
  if (bn == 32) hipLaunchKernelGGL((k_mx_gemm<TRANS, 32>), dim3(grid), dim3(256), 0, s, a);
  else if (bn == 64) hipLaunchKernelGGL((k_mx_gemm<TRANS, 64>), dim3(grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_mx_gemm<TRANS, 128>), dim3(grid), dim3(256), 0, s, a);
}

hss_status launch_mx_gemm(const hss_matrix* A, int b, const void* X, void* Y, void* ws, hipStream_t s) {
  const MxGemmPlan p = plan_mx_gemm(A, b);
  char* base = static_cast<char*>(ws);
  const int m = A->m, n = A->n, r = A->r;
  const bool trans = (A->flags & HSS_MX4_T) != 0;
  MxGemmArgs a = {};
  a.codes = A->dq_codes;
  a.scales = static_cast<const uint8_t*>(A->dq_levels);
  a.X = static_cast<const uint16_t*>(X);
  a.ldx = n;
  a.U = static_cast<const uint16_t*>(A->U);
  a.Tb = reinterpret_cast<const uint16_t*>(base + p.tb);
  a.m = m; a.n = n; a.b = b; a.r = r; a.rp = p.prep.rp;
  a.ng = mx_groups(trans ? m : n);
  a.nst1 = p.nst1; a.nst = p.nst; a.stages_per_split = p.stages_per_split;
  a.tiles_m = p.tiles_m; a.tiles_n = p.tiles_n;
  a.partial = p.finish;
  a.ldp = p.ldt;
  a.C = p.finish ? reinterpret_cast<void*>(base + p.part) : Y;

  MxPrep pr = p.prep;
  pr.X = a.X;
  pr.Vt = static_cast<const uint16_t*>(A->Vt);
  pr.Tp = reinterpret_cast<float*>(base + p.tp);
  pr.ldt = p.ldt;
  pr.np = p.np;
  if (A->nnz > 0) pr.Xt = reinterpret_cast<uint16_t*>(base + p.xt);
  if (n % 64 != 0 || (uintptr_t)X % 16 != 0) pr.Xp = reinterpret_cast<uint16_t*>(base + p.xp);
  if (r > 0 && (r % 32 != 0 || (uintptr_t)A->U % 16 != 0)) {
    pr.U = a.U;
    pr.Up = reinterpret_cast<uint16_t*>(base + p.up);
    a.U = pr.Up;
  }
  launch_mx_prep(pr, s);
  if (pr.Xp) {
    a.X = pr.Xp;
    a.ldx = p.np;
  }
  if (r > 0) launch_mx_tsum(pr.Tp, p.prep.splits, b, r, p.prep.rp, reinterpret_cast<uint16_t*>(base + p.tb), s);
  const unsigned grid = (unsigned)(p.tiles_m * p.tiles_n * p.splits);
  if (trans) launch_tile<true>(a, p.bn, grid, s);
  else launch_tile<false>(a, p.bn, grid, s);
  if (p.finish) {
    MxFinishArgs f = {};
    f.P = reinterpret_cast<const float*>(base + p.part);
    f.row_ptr = A->row_ptr;
    f.col = A->col_idx;
    f.vals = static_cast<const uint16_t*>(A->values);
    f.Xt = pr.Xt;
    f.Y = static_cast<uint16_t*>(Y);
    f.m = m; f.n = n; f.b = b; f.ldt = f.ldp = p.ldt;
    f.splits = p.splits;
    f.has_s = A->nnz > 0;
    f.tiles_m = (m + kFinRows - 1) / kFinRows;
    const dim3 fg((unsigned)(f.tiles_m * ((b + kFinCols - 1) / kFinCols)));
    if (A->flags & HSS_COL16) hipLaunchKernelGGL(k_mx_finish<uint16_t>, fg, dim3(512), 0, s, f);
    else hipLaunchKernelGGL(k_mx_finish<int32_t>, fg, dim3(512), 0, s, f);
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

// Columns up to which this route is taken.  Measured against the dense copy
// and its products (0.5 % of S, r 64, us; forward, input gradient):
//   4096^2         128 columns 28 against 42, 32 against 47;  256: 39 against 47, 44 against 51;  384: 58 against 51
//   4096 x 11008   128 columns 48 against 70, 60 against 76;  256: 73 against 77, 85 against 87
//   8192^2         128 columns 55 against 79, 63 against 95;  256: 89 against 96, 106 against 112
bool mx_gemm_supported(int b) { return b <= kMgMaxCols; }

}  // namespace hss
