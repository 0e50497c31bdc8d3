// Large bf16 products on the matrix cores, C = A . [B1 | B2]^T with A (M x K)
// and B (N x K) K-contiguous: 256 x 256 tiles, fp32 accumulation (or
// 256 x 192, where that leaves fewer CUs idle in the last round).
//
// Four waves, one per SIMD, each 128 x 128 of the tile: 4 x 4 blocks of
// v_mfma_f32_32x32x16_bf16 with 256 accumulators.  Per 16 columns of K a wave
// reads 8 fragments (8 KiB) from LDS for 16 MFMAs (512 cycles), so the LDS
// serves four waves in half of the matrix cores' time.  K runs in stages of 64
// through two LDS buffers of 64 KiB, filled by loads that go to LDS directly
// (no registers, no store instructions); a row is 128 bytes, its 16-byte
// chunks permuted by the row (on the source side) so that fragment reads do
// not conflict.
//
// A stage's fragments are read one step (16 columns) ahead of their MFMAs, and
// the barrier stands before a stage's last step: behind it the next stage's
// first fragments are read and the loads of the stage after that are issued
// while those MFMAs run, so the matrix cores cross the barrier with work in
// hand.
//
// Measured: 2048 x 8192, K 8192, 60 launches back to back: 231 us on average,
// 1.19 PFLOP/s (202 in the first ones: the clock falls from 1.9 GHz under this
// load; matrix cores busy in 69 % of the cycles).  The BLAS library's product,
// counted the same way: 207 (177).  In short runs, where the clock holds: 192,
// k_gemm_h's 128 x 256 tiles 250.  Loads through registers with two stages more
// in flight waited less (7 against 11 % of the wave cycles) and were 3 % slower.
#include <algorithm>
#include <type_traits>

#include "gemm256.h"
#include "s_pattern.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct G256Args {
  const uint16_t *A, *B1, *B2;
  int M, N, K1, K2;
  int lda, ldb1, ldb2;
  void* C;
  int64_t ldc;
  int tiles_m, tiles_n, stages_per_split;
  SPattern S;             // G256_DS
  const int32_t* tptr;    // G256_DS, CSR: k_ds_tiles' table
};

static constexpr int kKS = 64;  // K per stage
static constexpr int FM = 4;    // a wave's 32 x 32 blocks along M; FN (4 or 3) along N

// A tile of 256 x (64 FN): four waves, each 128 x 32 FN.
template <int FN>
struct GTile {
  static constexpr int TM = 64 * FM, TN = 64 * FN;
  static constexpr int BUF = (TM + TN) * kKS;  // bf16 per LDS buffer: A rows, then B rows
  static constexpr int AI = 2 * FM, BI = 2 * FN;  // load instructions per wave and stage, 8 rows each
};

// Slot of 16-byte chunk c (0..7) of a 128-byte LDS row r; its own inverse.
// Rows that a fragment read takes together get distinct slots, whether the LDS
// serves 8 rows in a 128-byte bank window or every second of 16 in a 256-byte one.
__device__ __forceinline__ int g_slot(int r, int c) { return c ^ ((r >> 1) & 7) ^ ((r & 1) << 2); }

// Tile of block b: the XCD that block b runs on (b % 8) gets a contiguous run
// of tile numbers, which go down groups of 8 tiles along M before moving along
// N, so that the blocks of one XCD share rows of A and B in its L2.
__device__ __forceinline__ void g_tile(int b, int G, int tiles_m, int tiles_n, int& tm, int& tn, int& tz) {
  const int per = (G + 7) / 8, x = b % 8, full = G % 8 == 0 ? 8 : G % 8;
  // XCDs 0 .. full - 1 hold `per` tiles, the others one less
  int t = x * per - max(x - full, 0) + b / 8;
  tz = t / (tiles_m * tiles_n);
  t -= tz * tiles_m * tiles_n;
  const int group = 8 * tiles_n, first = (t / group) * 8, gm = min(tiles_m - first, 8);
  const int v = t - (t / group) * group;
  tm = first + v % gm;
  tn = v / gm;
}

typedef __attribute__((address_space(3))) void lds_void;

// TWO: there is a second K segment (else its selects are left out).
template <int FN, int OUT, bool TWO>
__global__ __launch_bounds__(256, 1) void k_gemm256(G256Args g) {
  using TL = GTile<FN>;
  constexpr int KS = kKS;
  __shared__ __align__(16) uint16_t buf0[TL::BUF];
  __shared__ __align__(16) uint16_t buf1[TL::BUF];
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int wm = (w >> 1) * 32 * FM, wn = (w & 1) * 32 * FN;
  int tm, tn, tz;
  g_tile((int)blockIdx.x, (int)gridDim.x, g.tiles_m, g.tiles_n, tm, tn, tz);
  const int m0 = tm * TL::TM, n0 = tn * TL::TN;
  const int nst1 = g.K1 / KS, nst = nst1 + g.K2 / KS;
  const int s_begin = tz * g.stages_per_split, s_end = min(s_begin + g.stages_per_split, nst);
  // An AGPR named in an (empty) asm makes the compiler treat the kernel as
  // one that uses AGPRs: the accumulators live there.
  asm volatile("" ::: "a0");

  // This wave's loads: instruction i of A fills 8 rows of A's part from row 16 FM
  // w + 8 i on, and likewise for B; lane l writes row l / 8, slot l % 8.
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.A), 0, (int)((int64_t)g.M * g.lda * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb1 =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.B1), 0, (int)((int64_t)g.N * g.ldb1 * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb2 =
      TWO ? __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.B2), 0, (int)((int64_t)g.N * g.ldb2 * 2), 0x00020000)
          : rb1;
  uint32_t va[TL::AI], vb1[TL::BI], vb2[TL::BI];
  const int lr = lane >> 3, ls = lane & 7;
  // rows past the end repeat the last one; their results are dropped
#pragma unroll
  for (int i = 0; i < TL::AI; ++i) {
    const int row = 16 * FM * w + 8 * i + lr;
    va[i] = 2u * ((uint32_t)min(m0 + row, g.M - 1) * (uint32_t)g.lda + 8u * g_slot(row, ls));
  }
#pragma unroll
  for (int i = 0; i < TL::BI; ++i) {
    const int row = 16 * FN * w + 8 * i + lr;
    const uint32_t n = (uint32_t)min(n0 + row, g.N - 1), c = 8u * g_slot(row, ls);
    vb1[i] = 2u * (n * (uint32_t)g.ldb1 + c);
    vb2[i] = TWO ? 2u * (n * (uint32_t)g.ldb2 + c) : vb1[i];
  }
  // The loads of stage s; past the last one that one again, which nobody
  // reads, so that the loop has no branch around them.
  auto issue = [&](int s, uint16_t* buf) {
    s = min(s, s_end - 1);
    const bool second = TWO && s >= nst1;
    const int ka = 2 * KS * s, kb = 2 * KS * (second ? s - nst1 : s);
    const __amdgpu_buffer_rsrc_t rb = second ? rb2 : rb1;
#pragma unroll
    for (int i = 0; i < TL::AI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(buf + (16 * FM * w + 8 * i) * KS), 16, (int)va[i],
                                               ka, 0, 0);
#pragma unroll
    for (int i = 0; i < TL::BI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(buf + (TL::TM + 16 * FN * w + 8 * i) * KS), 16,
                                               (int)(second ? vb2[i] : vb1[i]), kb, 0, 0);
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  bf16x8 af[2][FM], bf[2][FN];
  auto frags = [&](const uint16_t* buf, int ks, bf16x8 (&a)[FM], bf16x8 (&b)[FN]) {
    const int c = 2 * ks + (lane >> 5);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = wm + 32 * i + (lane & 31);
      a[i] = *reinterpret_cast<const bf16x8*>(buf + row * KS + 8 * g_slot(row, c));
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int row = wn + 32 * j + (lane & 31);
      b[j] = *reinterpret_cast<const bf16x8*>(buf + (TL::TM + row) * KS + 8 * g_slot(row, c));
    }
  };
  auto mfmas = [&](const bf16x8 (&a)[FM], const bf16x8 (&b)[FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
  };
  // FM + FN times (an LDS read, its share of the loads, its share of the MFMAs)
  auto interleave = [](auto vm) {
    constexpr int R = FM + FN, PER = FM * FN / R;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if constexpr (decltype(vm)::value) __builtin_amdgcn_sched_group_barrier(0x20, (TL::AI + TL::BI) / R, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, PER, 0);
    }
    if constexpr (FM * FN > PER * R) __builtin_amdgcn_sched_group_barrier(0x8, FM * FN - PER * R, 0);
  };
  // From behind one barrier to behind the next: the last step of the stage
  // before (set 1), then this one's steps but the last; `prev` takes the loads
  // of stage s + 1.  The loop's back edge thus has no load to LDS in flight.
  auto stage = [&](int s, const uint16_t* cur, uint16_t* prev) {
    frags(cur, 0, af[0], bf[0]);
    issue(s + 1, prev);
    mfmas(af[1], bf[1]);
    interleave(std::true_type());
#pragma unroll
    for (int ks = 1; ks < KS / 16; ++ks) {
      frags(cur, ks, af[ks & 1], bf[ks & 1]);
      mfmas(af[(ks & 1) ^ 1], bf[(ks & 1) ^ 1]);
      interleave(std::false_type());
    }
    __syncthreads();  // the loads have landed, and nobody reads cur any more
  };
  issue(s_begin, buf0);
#pragma unroll
  for (int e = 0; e < 8; ++e) {  // no step before the first
#pragma unroll
    for (int i = 0; i < FM; ++i) af[1][i][e] = (__bf16)0.f;
#pragma unroll
    for (int j = 0; j < FN; ++j) bf[1][j][e] = (__bf16)0.f;
  }
  __syncthreads();
  int s = s_begin;
  for (; s + 1 < s_end; s += 2) {
    stage(s, buf0, buf1);
    stage(s + 1, buf1, buf0);
  }
  if (s < s_end) stage(s, buf0, buf1);
  mfmas(af[1], bf[1]);

  // lane holds rows 8 (v / 4) + 4 (lane / 32) + v % 4 of column lane % 32 of
  // each 32 x 32 block
  if constexpr (OUT == G256_BF16) {
    // C[n * ldc + m]: each wave stages 32 columns n x its 32 FM rows m (16-byte
    // chunk cm of row n at cm ^ n % (4 FM)), then writes 64 FM bytes per row n.
    constexpr int CH = 4 * FM, RP = 64 / CH;  // chunks per staged row, rows per read
    uint16_t* stg = buf0 + w * 32 * 32 * FM;
    uint16_t* C = static_cast<uint16_t*>(g.C);
    const bool vec = (uintptr_t)C % 16 == 0 && g.ldc % 8 == 0;
    const int nl = lane & 31, h = lane >> 5;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int vg = 0; vg < 4; ++vg) {
          u32x2 v2;
          const f32x2_t lo = {acc[i][j][4 * vg], acc[i][j][4 * vg + 1]}, hi = {acc[i][j][4 * vg + 2], acc[i][j][4 * vg + 3]};
          v2.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t));
          v2.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t));
          *reinterpret_cast<u32x2*>(stg + nl * 8 * CH + 8 * ((4 * i + vg) ^ (nl % CH)) + 4 * h) = v2;
        }
#pragma unroll
      for (int q = 0; q < 32 / RP; ++q) {
        const int nr = RP * q + lane / CH, cm = lane % CH;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + nr * 8 * CH + 8 * (cm ^ (nr % CH)));
        const int n = n0 + wn + 32 * j + nr, m = m0 + wm + 8 * cm;
        if (n < g.N) {
          uint16_t* dst = C + (int64_t)n * g.ldc + m;
          if (vec && m + 8 <= g.M) {
            *reinterpret_cast<u32x4*>(dst) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (m + e < g.M) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  } else if constexpr (OUT == G256_PART) {
    // partial product of this split: part[tz][n][m], rows of ldc (a multiple of 4)
    float* C = static_cast<float*>(g.C) + (int64_t)tz * g.N * g.ldc;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int n = n0 + wn + 32 * j + (lane & 31);
        if (n >= g.N) continue;
#pragma unroll
        for (int vg = 0; vg < 4; ++vg) {
          const int m = m0 + wm + 32 * i + 8 * vg + 4 * (lane >> 5);
          if (m < g.ldc)
            *reinterpret_cast<float4*>(C + (int64_t)n * g.ldc + m) =
                float4{acc[i][j][4 * vg], acc[i][j][4 * vg + 1], acc[i][j][4 * vg + 2], acc[i][j][4 * vg + 3]};
        }
      }
  } else {  // G256_DS32, 16, NM: dS[p] = C[row of p][column of p] for S's entries within the tile
    constexpr int PAT = OUT - G256_DS;
    float* dS = static_cast<float*>(g.C);
    // the entries' ranges of this thread's rows, requested together
    int32_t pb[FM], pt[FM];
    int64_t rs[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = min(m0 + 128 * (t >> 7) + 32 * i + ((t >> 2) & 31), g.M - 1);
      if constexpr (PAT == PAT_NM24) {
        rs[i] = (int64_t)row * (g.N >> 1);
        pb[i] = n0 >> 1, pt[i] = min(n0 + TL::TN, g.N) >> 1;
      } else {
        rs[i] = 0;
        pb[i] = g.tptr[(int64_t)row * (g.tiles_n + 1) + tn], pt[i] = g.tptr[(int64_t)row * (g.tiles_n + 1) + tn + 1];
      }
    }
    // 64 rows at a time through LDS (rows 128 g + 32 i + 0..31 at 32 g + 0..31), the
    // two buffers in turn; four threads take a row's entries
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      float* L = reinterpret_cast<float*>(i & 1 ? buf1 : buf0);
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          L[(32 * (w >> 1) + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3)) * TL::TN + wn + 32 * j + (lane & 31)] = acc[i][j][v];
      __syncthreads();
      const int lrow = t >> 2, row = m0 + 128 * (lrow >> 5) + 32 * i + (lrow & 31);
      if (row < g.M) {
        const int64_t pe = rs[i] + pt[i];
        for (int64_t p = rs[i] + pb[i] + (t & 3); p < pe; p += 4) {
          const int c = pat_col<PAT>(g.S, row, rs[i], p) - n0;
          if ((unsigned)c < (unsigned)TL::TN) dS[p] = L[lrow * TL::TN + c];
        }
      }
    }
  }
}

// tptr[row][t] = the first entry of the row at or past column 256 t (t = 0:
// its first, t = tiles: its end), by binary search.
template <int PAT>
__global__ __launch_bounds__(256) void k_ds_tiles(SPattern S, int m, int tiles, int32_t* __restrict__ tptr) {
  const int64_t total = (int64_t)m * (tiles + 1);
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int row = (int)(e / (tiles + 1)), t = (int)(e - (int64_t)row * (tiles + 1));
    const int32_t rs = S.row_ptr[row];
    int32_t lo = rs, hi = S.row_ptr[row + 1];
    if (t == 0) hi = lo;
    if (t == tiles) lo = hi;
    while (lo < hi) {
      const int32_t mid = lo + (hi - lo) / 2;
      if (pat_col<PAT>(S, row, rs, mid) < 256 * t) lo = mid + 1;
      else hi = mid;
    }
    tptr[e] = lo;
  }
}

// C[n * ldc + m] (bf16) = the splits' partial products [z][n][mp], added in order.
__global__ __launch_bounds__(256) void k_gemm256_sum(const float* __restrict__ part, int splits, int M, int N, int mp,
                                                     int64_t ldc, uint16_t* __restrict__ C) {
  const uint32_t per = (uint32_t)mp >> 2, total = (uint32_t)N * per;
  const int64_t zs = (int64_t)N * mp;
  for (uint32_t q = blockIdx.x * 256u + threadIdx.x; q < total; q += gridDim.x * 256u) {
    const uint32_t n = q / per, m = (q - n * per) * 4;
    const float* p = part + (int64_t)n * mp + m;
    float4 s = *reinterpret_cast<const float4*>(p);
    for (int z = 1; z < splits; ++z) {
      const float4 v = *reinterpret_cast<const float4*>(p + z * zs);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((int)m + e < M) C[(int64_t)n * ldc + m + e] = f32_to_bf16(v[e]);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct G256Cfg {
  int fn, splits;
};

// Tile width and K splits with the least estimated time, in us: rounds of
// tiles over the 256 CUs, one tile a CU, 0.0225 us per column of K for a 256 x
// 256 tile (measured at K 8192) and 0.77 of it for a 256 x 192 one; splitting
// K writes and reads z partial products at 5 TB/s and adds a launch.
static G256Cfg g256_cfg(int M, int N, int K) {
  G256Cfg best = {4, 1};
  double least = 1e30;
  for (int fn = 4; fn >= 3; --fn)
    for (int z = 1; z <= 8; ++z) {
      if (z > 1 && K / z < 512) break;
      const int64_t tiles = (int64_t)((M + 255) / 256) * ((N + 64 * fn - 1) / (64 * fn)) * z;
      double t = (double)((tiles + 255) / 256) * (fn == 4 ? 1.0 : 0.77) * 0.0225 * K / z;
      if (z > 1) t += 5 + 8.0 * z * M * N / 5e6;
      if (t < least) least = t, best = {fn, z};
    }
  return best;
}

bool gemm256_ok(int M, int N, int K1, int lda, int ldb1, int K2, int ldb2) {
  const int64_t lim = (int64_t)1 << 31;
  auto fits = [&](int64_t rows, int64_t ld) { return rows * ld * 2 < lim && ld % 8 == 0; };
  return K1 > 0 && K1 % 64 == 0 && K2 % 64 == 0 && fits(M, lda) && fits(N, ldb1) && (K2 == 0 || fits(N, ldb2));
}

size_t gemm256_part_bytes(int M, int from, int N, int K) {
  // as N grows among the same tiles, only the cost of the partial products
  // does, by its number of them: the choice moves to fewer
  const int splits = std::max(g256_cfg(M, from, K).splits, g256_cfg(M, N, K).splits);
  return splits > 1 ? (size_t)splits * N * ((M + 3) / 4 * 4) * 4 : 0;
}

template <int FN, int OUT>
static void launch_cfg(const G256Args& g, int splits, hipStream_t s) {
  const dim3 grid((unsigned)(g.tiles_m * g.tiles_n * splits));
  if (g.K2 > 0)
    hipLaunchKernelGGL((k_gemm256<FN, OUT, true>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((k_gemm256<FN, OUT, false>), grid, dim3(256), 0, s, g);
}

void launch_gemm256_bf16(int M, int N, const uint16_t* A, int lda, int K1, const uint16_t* B1, int ldb1, int K2,
                         const uint16_t* B2, int ldb2, void* C, int64_t ldc, float* part, hipStream_t s) {
  const G256Cfg c = g256_cfg(M, N, K1 + K2);
  G256Args g = {};
  g.A = A; g.B1 = B1; g.B2 = B2;
  g.M = M; g.N = N; g.K1 = K1; g.K2 = K2;
  g.lda = lda; g.ldb1 = ldb1; g.ldb2 = ldb2;
  g.tiles_m = (M + 255) / 256;
  g.tiles_n = (N + 64 * c.fn - 1) / (64 * c.fn);
  const int stages = (K1 + K2) / kKS;
  g.stages_per_split = (stages + c.splits - 1) / c.splits;
  const int splits = (stages + g.stages_per_split - 1) / g.stages_per_split;
  if (splits == 1) {
    g.C = C; g.ldc = ldc;
    if (c.fn == 4) launch_cfg<4, G256_BF16>(g, 1, s);
    else launch_cfg<3, G256_BF16>(g, 1, s);
    return;
  }
  const int mp = (M + 3) / 4 * 4;
  g.C = part; g.ldc = mp;
  if (c.fn == 4) launch_cfg<4, G256_PART>(g, splits, s);
  else launch_cfg<3, G256_PART>(g, splits, s);
  const int64_t work = (int64_t)N * mp / 4;
  hipLaunchKernelGGL(k_gemm256_sum, dim3((unsigned)std::min<int64_t>((work + 255) / 256, 8192)), dim3(256), 0, s, part,
                     splits, M, N, mp, ldc, static_cast<uint16_t*>(C));
}

size_t gemm256_ds_bytes(const hss_matrix* A) {
  return A->fmt == HSS_FMT_2OF4 ? 0 : (size_t)A->m * ((A->n + 255) / 256 + 1) * 4;
}

void launch_gemm256_ds(const hss_matrix* A, int K, const uint16_t* Gt, const uint16_t* Xt, int ld, float* dS,
                       int32_t* tptr, hipStream_t s) {
  G256Args g = {};
  g.A = Gt; g.B1 = Xt;
  g.M = A->m; g.N = A->n; g.K1 = K;
  g.lda = g.ldb1 = ld;
  g.C = dS;
  g.tiles_m = (g.M + 255) / 256;
  g.tiles_n = (g.N + 255) / 256;
  g.stages_per_split = K / kKS;
  g.S = s_pattern(A);
  g.tptr = tptr;
  const dim3 grid((unsigned)(g.tiles_m * g.tiles_n));
  const int pat = s_pattern_kind(A);
  if (pat == PAT_NM24) {
    hipLaunchKernelGGL((k_gemm256<4, G256_DS + PAT_NM24, false>), grid, dim3(256), 0, s, g);
    return;
  }
  const int64_t work = (int64_t)g.M * (g.tiles_n + 1);
  const dim3 tg((unsigned)std::min<int64_t>((work + 255) / 256, 8192));
  if (pat == PAT_CSR16) {
    hipLaunchKernelGGL(k_ds_tiles<PAT_CSR16>, tg, dim3(256), 0, s, g.S, g.M, g.tiles_n, tptr);
    hipLaunchKernelGGL((k_gemm256<4, G256_DS + PAT_CSR16, false>), grid, dim3(256), 0, s, g);
  } else {
    hipLaunchKernelGGL(k_ds_tiles<PAT_CSR32>, tg, dim3(256), 0, s, g.S, g.M, g.tiles_n, tptr);
    hipLaunchKernelGGL((k_gemm256<4, G256_DS + PAT_CSR32, false>), grid, dim3(256), 0, s, g);
  }
}

}  // namespace hss
