// Large bf16 products on the matrix cores, C = A . [B1 | B2]^T with A (M x K)
// and B (N x K) K-contiguous: 256 x 256 tiles, fp32 accumulation.
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
// Measured: 2048 x 8192, K 8192: 192 us, 1.43 PFLOP/s (k_gemm_h's 128 x 256
// tiles: 250); matrix cores busy in 68 % of the cycles at the 1.93 GHz the
// chip holds under this load.  Loads through registers with two stages more in
// flight waited less (7 against 11 % of the wave cycles) and were 3 % slower.
#include <algorithm>
#include <type_traits>

#include "gemm256.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

static constexpr int kT = 256, kKS = 64;            // tile side, K per stage
static constexpr int kBuf = 2 * kT * kKS;           // bf16 per LDS buffer: A rows, then B rows

struct G256Args {
  const uint16_t *A, *B1, *B2;
  int M, N, K1, K2;
  int lda, ldb1, ldb2;
  void* C;
  int64_t ldc;
  int tiles_m, tiles_n;
  // OUT_DS
  const int32_t* tile_ptr;  // m x (tiles_n + 1): first stored entry of a row at or past column 256 t
  const void* col;
  const uint32_t* meta;
  int pat, n;
};

// Slot of chunk c (0..7) of LDS row r; its own inverse.  Rows a fragment read
// takes together (8 in a 128-byte bank window, every second of 16 in a
// 256-byte one) get distinct slots.
__device__ __forceinline__ int g_slot(int r, int c) { return c ^ ((r >> 1) & 7) ^ ((r & 1) << 2); }

// Tile of block b: the XCD that block b runs on (b % 8) gets a contiguous run
// of tile numbers, which go down groups of 8 tiles along M before moving along
// N, so that the blocks of one XCD share rows of A and B in its L2.
__device__ __forceinline__ void g_tile(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int G = tiles_m * tiles_n, per = (G + 7) / 8, x = b % 8, full = G % 8 == 0 ? 8 : G % 8;
  // XCDs 0 .. full - 1 hold `per` tiles, the others one less
  const int t = x * per - max(x - full, 0) + b / 8;
  const int group = 8 * tiles_n, first = (t / group) * 8, gm = min(tiles_m - first, 8);
  const int v = t - (t / group) * group;
  tm = first + v % gm;
  tn = v / gm;
}

typedef __attribute__((address_space(3))) void lds_void;

// TWO: there is a second K segment (else its selects are left out).
template <int OUT, bool TWO>
__global__ __launch_bounds__(256, 1) void k_gemm256(G256Args g) {
  __shared__ __align__(16) uint16_t buf0[kBuf];
  __shared__ __align__(16) uint16_t buf1[kBuf];
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int wm = (w >> 1) * 128, wn = (w & 1) * 128;
  int tm, tn;
  g_tile((int)blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
  const int m0 = tm * kT, n0 = tn * kT;
  const int nst1 = g.K1 / kKS, nst = nst1 + g.K2 / kKS;
  // An AGPR named in an (empty) asm makes the compiler treat the kernel as
  // one that uses AGPRs: the accumulators live there.
  asm volatile("" ::: "a0");

  // This wave's loads: instruction i < 8 fills rows 64 w + 8 i .. + 7 of A's
  // half, instruction i >= 8 the same rows of B's; lane l writes row l / 8,
  // slot l % 8.
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.A), 0, (int)((int64_t)g.M * g.lda * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb1 =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.B1), 0, (int)((int64_t)g.N * g.ldb1 * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb2 =
      TWO ? __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(g.B2), 0, (int)((int64_t)g.N * g.ldb2 * 2), 0x00020000)
          : rb1;
  uint32_t va[8], vb1[8], vb2[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // rows past the end repeat the last one; their results are dropped
    const int row = 64 * w + 8 * i + (lane >> 3), c = g_slot(row, lane & 7);
    const uint32_t n = (uint32_t)min(n0 + row, g.N - 1);
    va[i] = 2u * ((uint32_t)min(m0 + row, g.M - 1) * (uint32_t)g.lda + 8u * c);
    vb1[i] = 2u * (n * (uint32_t)g.ldb1 + 8u * c);
    vb2[i] = TWO ? 2u * (n * (uint32_t)g.ldb2 + 8u * c) : vb1[i];
  }
  // The loads of stage s; past the last one that one again, which nobody
  // reads, so that the loop has no branch around them.
  auto issue = [&](int s, uint16_t* buf) {
    s = min(s, nst - 1);
    const bool second = TWO && s >= nst1;
    const int ka = 2 * kKS * s, kb = 2 * kKS * (second ? s - nst1 : s);
    const __amdgpu_buffer_rsrc_t rb = second ? rb2 : rb1;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(buf + (64 * w + 8 * i) * kKS), 16, (int)va[i], ka, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(buf + (kT + 64 * w + 8 * i) * kKS), 16,
                                               (int)(second ? vb2[i] : vb1[i]), kb, 0, 0);
  };

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  bf16x8 af[2][4], bf[2][4];
  auto frags = [&](const uint16_t* buf, int ks, bf16x8 (&a)[4], bf16x8 (&b)[4]) {
    const int c = 2 * ks + (lane >> 5);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = wm + 32 * i + (lane & 31);
      a[i] = *reinterpret_cast<const bf16x8*>(buf + row * kKS + 8 * g_slot(row, c));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = wn + 32 * j + (lane & 31);
      b[j] = *reinterpret_cast<const bf16x8*>(buf + (kT + row) * kKS + 8 * g_slot(row, c));
    }
  };
  auto mfmas = [&](const bf16x8 (&a)[4], const bf16x8 (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
  };
  // 8 x (one LDS read, VM loads to LDS, two MFMAs)
  auto interleave = [](auto vm) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if constexpr (decltype(vm)::value) __builtin_amdgcn_sched_group_barrier(0x20, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
    }
  };
  // From behind one barrier to behind the next: the last step of the stage
  // before (set 1), then this one's first three; `prev` takes the loads of
  // stage s + 1.  The loop's back edge thus has no load to LDS in flight.
  auto stage = [&](int s, const uint16_t* cur, uint16_t* prev) {
    frags(cur, 0, af[0], bf[0]);
    issue(s + 1, prev);
    mfmas(af[1], bf[1]);
    interleave(std::true_type());
    frags(cur, 1, af[1], bf[1]);
    mfmas(af[0], bf[0]);
    interleave(std::false_type());
    frags(cur, 2, af[0], bf[0]);
    mfmas(af[1], bf[1]);
    interleave(std::false_type());
    frags(cur, 3, af[1], bf[1]);
    mfmas(af[0], bf[0]);
    interleave(std::false_type());
    __syncthreads();  // the loads have landed, and nobody reads cur any more
  };
  issue(0, buf0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) af[1][i][e] = bf[1][i][e] = (__bf16)0.f;  // no step before the first
  __syncthreads();
  int s = 0;
  for (; s + 1 < nst; s += 2) {
    stage(s, buf0, buf1);
    stage(s + 1, buf1, buf0);
  }
  if (s < nst) stage(s, buf0, buf1);
  mfmas(af[1], bf[1]);

  // lane holds rows 8 (v / 4) + 4 (lane / 32) + v % 4 of column lane % 32 of
  // each 32 x 32 block
  if constexpr (OUT == G256_BF16) {
    // C[n * ldc + m]: each wave stages 32 columns n x its 128 rows m (16-byte
    // chunk cm of row n at cm ^ n % 16), then writes 256 bytes per row n.
    uint16_t* stg = buf0 + w * 32 * 128;
    uint16_t* C = static_cast<uint16_t*>(g.C);
    const bool vec = (uintptr_t)C % 16 == 0 && g.ldc % 8 == 0;
    const int nl = lane & 31, h = lane >> 5;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int vg = 0; vg < 4; ++vg) {
          u32x2 v2;
          const f32x2_t lo = {acc[i][j][4 * vg], acc[i][j][4 * vg + 1]}, hi = {acc[i][j][4 * vg + 2], acc[i][j][4 * vg + 3]};
          v2.x = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t));
          v2.y = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t));
          *reinterpret_cast<u32x2*>(stg + nl * 128 + 8 * ((4 * i + vg) ^ (nl & 15)) + 4 * h) = v2;
        }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int nr = 4 * q + (lane >> 4), cm = lane & 15;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stg + nr * 128 + 8 * (cm ^ (nr & 15)));
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
  }
}

bool gemm256_ok(int M, int N, int K1, int lda, int ldb1, int K2, int ldb2) {
  const int64_t lim = (int64_t)1 << 31;
  auto fits = [&](int64_t rows, int64_t ld) { return rows * ld * 2 < lim && ld % 8 == 0; };
  return K1 > 0 && K1 % kKS == 0 && K2 % kKS == 0 && fits(M, lda) && fits(N, ldb1) && (K2 == 0 || fits(N, ldb2));
}

void launch_gemm256_bf16(int M, int N, const uint16_t* A, int lda, int K1, const uint16_t* B1, int ldb1, int K2,
                         const uint16_t* B2, int ldb2, void* C, int64_t ldc, hipStream_t s) {
  G256Args g = {};
  g.A = A; g.B1 = B1; g.B2 = B2;
  g.M = M; g.N = N; g.K1 = K1; g.K2 = K2;
  g.lda = lda; g.ldb1 = ldb1; g.ldb2 = ldb2;
  g.C = C; g.ldc = ldc;
  g.tiles_m = (M + kT - 1) / kT;
  g.tiles_n = (N + kT - 1) / kT;
  const dim3 grid((unsigned)(g.tiles_m * g.tiles_n));
  if (K2 > 0)
    hipLaunchKernelGGL((k_gemm256<G256_BF16, true>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((k_gemm256<G256_BF16, false>), grid, dim3(256), 0, s, g);
}

}  // namespace hss
