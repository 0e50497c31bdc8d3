// Grouped small matrix products on the matrix cores, C = A . B^T in fp32.
//
// The products of a gradient with a low rank have one short side (r) and a
// long K or a long other side: alone they fill a part of the chip, and a
// launch costs as much as the work.  So independent ones share a launch, and
// K is split where the tiles are few (the reader adds the partial products in
// order).  Tile BM x 128 (BM = 64 or 128, the rank's side), 4 waves, K in
// stages of 64 through two LDS buffers with the next stage's loads in flight;
// one barrier per stage.
#include <algorithm>

#include "mm_group.h"

namespace hss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

static constexpr int kMmN = 128, kMmK = 64;

struct MmArgs {
  MmProblem p[kMmGroup];
  int count;
};

// Slot of 16-byte chunk c (0..7) of a 128-byte LDS row: the rows that a
// fragment read takes together (8 in a 128-byte bank window, or every second
// of 16 in a 256-byte one) get distinct slots.
__device__ __forceinline__ int mm_slot(int row, int c) { return c ^ ((row >> 1) & 7) ^ ((row & 1) << 2); }

// This wave's part of C: 16 x 16 blocks from row0, col0 on, whose lane holds
// rows 4 (lane / 16) + e of column lane % 16.
template <int FM, int FN>
__device__ __forceinline__ void mm_write(const MmProblem& p, int z, int row0, int col0, const f32x4 (&acc)[FM][FN]) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  float* C = p.C + (int64_t)z * p.zstride;
  const int M = p.M, N = p.N;
  const int mleft = M - (row0 + 4 * q), nleft = N - (col0 + (lane & 15));
  if (p.trans) {  // a lane's four rows lie side by side
    float* at = C + (row0 + 4 * q) + (col0 + (lane & 15)) * p.ldc;
    const bool vec = ((p.ldc | p.zstride) & 3) == 0 && ((uintptr_t)p.C & 15) == 0;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (16 * j >= nleft) continue;
        float* o = at + 16 * j * p.ldc + 16 * i;
        if (vec && 16 * i + 4 <= mleft) {
          *reinterpret_cast<f32x4*>(o) = acc[i][j];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * i + e < mleft) o[e] = acc[i][j][e];
        }
      }
    return;
  }
  float* at = C + (row0 + 4 * q) * p.ldc + (col0 + (lane & 15));
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float* row = at + (16 * i + e) * p.ldc;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if (16 * i + e < mleft && 16 * j < nleft) row[16 * j] = acc[i][j][e];
    }
}

template <int BM>
__global__ __launch_bounds__(256, BM == 64 ? 3 : 2) void k_mm(MmArgs args) {
  constexpr int FM = BM / 32, FN = 4;
  constexpr int AV = BM / 32, BV = kMmN / 32;  // 16-byte chunks per thread and stage
  __shared__ __align__(16) uint16_t lds[2][(BM + kMmN) * kMmK];
  int block = (int)blockIdx.x, which = 0;
  while (which + 1 < args.count && block >= args.p[which].blocks) block -= args.p[which++].blocks;
  const MmProblem& p = args.p[which];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, q = lane >> 4;
  const int tn = block % p.tiles_n, rest = block / p.tiles_n;
  const int z = rest % p.splits, tm = rest / p.splits;
  const int m0 = tm * BM, n0 = tn * kMmN;
  const int s0 = z * p.stages_per_split, s1 = min(s0 + p.stages_per_split, (p.K + kMmK - 1) / kMmK);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Regs {
    u32x4 a[AV], b[BV];
  };
  const int c = t & 7, r0 = t >> 3;  // chunk and first row of this thread's loads
  auto load = [&](int s, Regs& r) {
    const int k = min(s * kMmK + 8 * c, p.K - 8);  // past the end: a valid chunk, stored as zeros
#pragma unroll
    for (int i = 0; i < AV; ++i)
      r.a[i] = *reinterpret_cast<const u32x4*>(p.A + (int64_t)min(m0 + r0 + 32 * i, p.M - 1) * p.lda + k);
#pragma unroll
    for (int i = 0; i < BV; ++i)
      r.b[i] = *reinterpret_cast<const u32x4*>(p.B + (int64_t)min(n0 + r0 + 32 * i, p.N - 1) * p.ldb + k);
  };
  auto store = [&](int s, uint16_t* buf, const Regs& r) {
    const bool in = s * kMmK + 8 * c < p.K;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < AV; ++i)
      *reinterpret_cast<u32x4*>(buf + (r0 + 32 * i) * kMmK + 8 * mm_slot(r0 + 32 * i, c)) = in ? r.a[i] : zero;
#pragma unroll
    for (int i = 0; i < BV; ++i)
      *reinterpret_cast<u32x4*>(buf + (BM + r0 + 32 * i) * kMmK + 8 * mm_slot(r0 + 32 * i, c)) = in ? r.b[i] : zero;
  };
  const int wm = (w >> 1) * (BM / 2), wn = (w & 1) * 64;
  auto compute = [&](const uint16_t* buf) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8 af[FM], bf[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int row = wm + 16 * i + (lane & 15);
        af[i] = *reinterpret_cast<const bf16x8*>(buf + row * kMmK + 8 * mm_slot(row, 4 * ks + q));
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn + 16 * j + (lane & 15);
        bf[j] = *reinterpret_cast<const bf16x8*>(buf + (BM + row) * kMmK + 8 * mm_slot(row, 4 * ks + q));
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
  };
  if (s0 < s1) {
    Regs ra, rb;
    load(s0, ra);
    load(min(s0 + 1, s1 - 1), rb);
    store(s0, lds[0], ra);
    __syncthreads();
    // pairs of stages, then an odd last one: with an exit from the middle the
    // compiler moves the register sets about, and waits for their loads
    int s = s0;
    for (; s + 1 < s1; s += 2) {
      load(min(s + 2, s1 - 1), ra);
      __builtin_amdgcn_sched_barrier(0);  // the loads first: the compiler would sink them
      compute(lds[0]);
      store(s + 1, lds[1], rb);
      __syncthreads();
      load(min(s + 3, s1 - 1), rb);
      __builtin_amdgcn_sched_barrier(0);
      compute(lds[1]);
      store(min(s + 2, s1 - 1), lds[0], ra);
      __syncthreads();
    }
    if (s < s1) compute(lds[0]);
  }
  mm_write<FM, FN>(p, z, m0 + wm, n0 + wn, acc);
}

// The same with A in three terms side by side (terms of K columns each), all
// times the same B: C = (A1 + A2 + A3) . B^T.  A stage's B is loaded once for
// the three, into one LDS buffer with the next stage in registers.
template <int BM>
__global__ __launch_bounds__(256, 2) void k_mm3(MmArgs args) {
  constexpr int FM = BM / 32, FN = 4;
  constexpr int AV = BM / 32, BV = kMmN / 32;
  __shared__ __align__(16) uint16_t lds[(3 * BM + kMmN) * kMmK];
  int block = (int)blockIdx.x, which = 0;
  while (which + 1 < args.count && block >= args.p[which].blocks) block -= args.p[which++].blocks;
  const MmProblem& p = args.p[which];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, q = lane >> 4;
  const int tn = block % p.tiles_n, rest = block / p.tiles_n;
  const int z = rest % p.splits, tm = rest / p.splits;
  const int m0 = tm * BM, n0 = tn * kMmN, K = p.K;
  const int s0 = z * p.stages_per_split, s1 = min(s0 + p.stages_per_split, (K + kMmK - 1) / kMmK);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int c = t & 7, r0 = t >> 3;
  const uint16_t *pa[AV], *pb[BV];
#pragma unroll
  for (int i = 0; i < AV; ++i) pa[i] = p.A + (int64_t)min(m0 + r0 + 32 * i, p.M - 1) * p.lda;
#pragma unroll
  for (int i = 0; i < BV; ++i) pb[i] = p.B + (int64_t)min(n0 + r0 + 32 * i, p.N - 1) * p.ldb;
  u32x4 ra[3][AV], rb[BV];
  auto load = [&](int s) {
    const int k = min(s * kMmK + 8 * c, K - 8);  // past the end: a valid chunk, stored as zeros
#pragma unroll
    for (int i = 0; i < BV; ++i) rb[i] = *reinterpret_cast<const u32x4*>(pb[i] + k);
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
      for (int i = 0; i < AV; ++i) ra[e][i] = *reinterpret_cast<const u32x4*>(pa[i] + e * K + k);
  };
  auto store = [&](int s) {
    const bool in = s * kMmK + 8 * c < K;
    const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
      for (int i = 0; i < AV; ++i)
        *reinterpret_cast<u32x4*>(lds + (e * BM + r0 + 32 * i) * kMmK + 8 * mm_slot(r0 + 32 * i, c)) =
            in ? ra[e][i] : zero;
#pragma unroll
    for (int i = 0; i < BV; ++i)
      *reinterpret_cast<u32x4*>(lds + (3 * BM + r0 + 32 * i) * kMmK + 8 * mm_slot(r0 + 32 * i, c)) = in ? rb[i] : zero;
  };
  const int wm = (w >> 1) * (BM / 2), wn = (w & 1) * 64;
  load(s0);
  for (int s = s0; s < s1; ++s) {
    store(s);
    __syncthreads();
    load(min(s + 1, s1 - 1));
    __builtin_amdgcn_sched_barrier(0);  // the loads first: the compiler would sink them
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8 bf[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = wn + 16 * j + (lane & 15);
        bf[j] = *reinterpret_cast<const bf16x8*>(lds + (3 * BM + row) * kMmK + 8 * mm_slot(row, 4 * ks + q));
      }
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const int row = wm + 16 * i + (lane & 15);
          const bf16x8 af = *reinterpret_cast<const bf16x8*>(lds + (e * BM + row) * kMmK + 8 * mm_slot(row, 4 * ks + q));
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, bf[j], acc[i][j], 0, 0, 0);
        }
    }
    __syncthreads();
  }
  mm_write<FM, FN>(p, z, m0 + wm, n0 + wn, acc);
}

static int mm_tile_m(int M) { return M > 64 ? 128 : 64; }

int mm_splits(int M, int N, int K, int target) {
  const int tiles = ((M + mm_tile_m(M) - 1) / mm_tile_m(M)) * ((N + kMmN - 1) / kMmN);
  const int stages = (K + kMmK - 1) / kMmK;
  const int want = std::max(1, std::min(target / tiles, stages / 2));
  const int per = (stages + want - 1) / want;
  return (stages + per - 1) / per;
}

int mm_actual_splits(int K, int splits) {
  const int stages = (K + kMmK - 1) / kMmK, per = (stages + splits - 1) / splits;
  return (stages + per - 1) / per;
}

void launch_mm_group(const MmProblem* p, int count, bool terms3, hipStream_t s) {
  MmArgs a = {};
  int bm = 64, blocks = 0;
  for (int i = 0; i < count; ++i) bm = std::max(bm, mm_tile_m(p[i].M));
  for (int i = 0; i < count; ++i) {
    MmProblem& q = a.p[a.count++];
    q = p[i];
    const int stages = (q.K + kMmK - 1) / kMmK;
    q.splits = mm_actual_splits(q.K, std::max(q.splits, 1));
    q.stages_per_split = (stages + q.splits - 1) / q.splits;
    q.tiles_n = (q.N + kMmN - 1) / kMmN;
    q.blocks = q.tiles_n * q.splits * ((q.M + bm - 1) / bm);
    blocks += q.blocks;
  }
  const dim3 grid((unsigned)blocks), block(256);
  if (terms3) {
    if (bm == 64) hipLaunchKernelGGL(k_mm3<64>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_mm3<128>, grid, block, 0, s, a);
  } else {
    if (bm == 64) hipLaunchKernelGGL(k_mm<64>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_mm<128>, grid, block, 0, s, a);
  }
}

}  // namespace hss
