// One AdamW step over many tensors (hss_adamw).
//
//   g = grad * grad_scale
//   m <- b1 m + (1 - b1) g        v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Each element is read and written once, so the step is bound by memory.  The
// unit of work is a block of 256 elements: half a wave, eight elements a lane,
// so that the arrays of two and four bytes move in 16-byte accesses and the
// block's largest magnitude (the scale of the 8-bit moments) is one reduction
// over 32 lanes.  All tensors of a launch share its grid; the table of tensors
// travels in the kernel's arguments, so that the call copies nothing and can
// be captured.  38 M elements in bf16 with an fp32 copy, gradients fp32: 210 us with
// fp32 moments (1140 MB, 5.4 TB/s, more than a copy of 1 GiB reaches), 128 with 8-bit
// ones (686 MB, 5.3 TB/s); one small tensor 6.4 us, a launch and a chain of loads.
//
// 8-bit moments: m and sqrt(v) as e4m3 times one fp32 scale per block, the
// block's largest magnitude / 448.  sqrt(v) is kept rather than v because it has
// half the range in powers of two; one fp32 scale rather than a power of two lets
// the block's largest value follow its average exactly.  A step of b2 moves
// sqrt(v) by 0.05 %, far less than the 6 to 12 % between two codes: rounded to the
// nearest, most averages would never move again (and sqrt(v) would stay small
// when gradients grow).  So each value is rounded up or down at random in
// proportion, with bits that hash the element's position and the step: the
// average moves as it should in the mean, and the same call gives the same
// bits.  sqrt(v) > 0 is never rounded to 0, which would leave m / eps.
#include <algorithm>
#include <cmath>

#include "hss_internal.h"

namespace hss {

static constexpr int kAwBlock = 256;    // elements that share a scale
static constexpr int kAwChunk = 8;      // blocks of one tensor that a workgroup takes at a time
static constexpr int kAwTensors = 48;   // tensors of one launch: 3.8 KB of the 4 KB of kernel arguments

struct AwTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t count;
  uint32_t first, pos;  // its first chunk among the launch's, its first block among the call's
};

struct AwHyper {
  float b1, c1, b2, c2, eps, decay, size, root, gscale;
  double beta1, beta2, lr, wd, bias1;  // bias1 = 1 - beta1^step
  const float* lr_dev;
  const int32_t* step_dev;
  const float* gscale_dev;
  uint32_t key;  // step * 0xBB67AE85
};

struct AwArgs {
  AwHyper h;
  AwTensor t[kAwTensors];
  uint32_t first[64];  // the tensors' first chunks, then the largest number: a lane each
  int tensors;
  uint32_t chunks;
};
static_assert(sizeof(AwArgs) <= 4096, "kernel arguments");

struct __attribute__((packed, aligned(1))) AwF8 { float f[8]; };
struct __attribute__((packed, aligned(1))) AwU4 { uint32_t w[4]; };
struct __attribute__((packed, aligned(1))) AwU2 { uint32_t w[2]; };

// Eight elements from i on; `left` of them are inside the tensor.  The
// addresses may have any alignment (the hardware takes unaligned vectors).
__device__ __forceinline__ void aw_load(const float* a, int64_t i, int left, float* x) {
  if (left >= 8) {
    const AwF8 f = *reinterpret_cast<const AwF8*>(a + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = f.f[k];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < left ? a[i + k] : 0.f;
  }
}
__device__ __forceinline__ void aw_load(const uint16_t* a, int64_t i, int left, float* x) {
  if (left >= 8) {
    const AwU4 w = *reinterpret_cast<const AwU4*>(a + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[2 * k] = bf16lo(w.w[k]), x[2 * k + 1] = bf16hi(w.w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < left ? __uint_as_float((uint32_t)a[i + k] << 16) : 0.f;
  }
}
__device__ __forceinline__ void aw_store(float* a, int64_t i, int left, const float* x) {
  if (left >= 8) {
    AwF8 f;
#pragma unroll
    for (int k = 0; k < 8; ++k) f.f[k] = x[k];
    *reinterpret_cast<AwF8*>(a + i) = f;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) a[i + k] = x[k];
  }
}
__device__ __forceinline__ void aw_store(uint16_t* a, int64_t i, int left, const float* x) {
  if (left >= 8) {
    AwU4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w.w[k] = f32_to_bf16(x[2 * k]) | (uint32_t)f32_to_bf16(x[2 * k + 1]) << 16;
    *reinterpret_cast<AwU4*>(a + i) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) a[i + k] = f32_to_bf16(x[k]);
  }
}
__device__ __forceinline__ AwU2 aw_load_codes(const uint8_t* a, int64_t i, int left) {
  AwU2 c = {{0u, 0u}};
  if (left >= 8) {
    c = *reinterpret_cast<const AwU2*>(a + i);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) c.w[k >> 2] |= (uint32_t)a[i + k] << (8 * (k & 3));
  }
  return c;
}
__device__ __forceinline__ void aw_store_codes(uint8_t* a, int64_t i, int left, AwU2 c) {
  if (left >= 8) {
    *reinterpret_cast<AwU2*>(a + i) = c;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) a[i + k] = (uint8_t)(c.w[k >> 2] >> (8 * (k & 3)));
  }
}

// e4m3 (sign, 4 exponent bits, 3 mantissa bits, exponent 0 = subnormal), exact.
__device__ __forceinline__ float aw_decode(uint32_t code) {
  const uint32_t k = code & 0x7fu;
  const float a = k < 8u ? (float)k * 0x1p-9f : __uint_as_float((k + 960u) << 20);
  return __uint_as_float(__float_as_uint(a) | (code & 0x80u) << 24);
}

// x / scale (inv = 1 / scale) as a code: u / 2^16 of a step is added, and what is
// then below the step dropped, in integers: a sum in fp32 would round up to the next
// code where little is missing.  `least`: the smallest code of an x that is not 0.
__device__ __forceinline__ uint32_t aw_encode(float x, float inv, uint32_t u, uint32_t least) {
  const float a = fminf(fabsf(x) * inv, 448.f);
  const uint32_t normal = ((__float_as_uint(a) + (u << 4)) >> 20) - 960u;
  const uint32_t small = ((uint32_t)fminf(a * 0x1p25f, 0x1p20f) + u) >> 16;  // steps of 2^-9 (below 2^-6: less than 2^19)
  uint32_t k = min(a < 0x1p-6f ? small : normal, 126u);
  if (x != 0.f) k = max(k, least);
  return k | (__float_as_uint(x) >> 31) << 7;
}

// 32 bits of the position and the step: products with odd constants (the first
// digits of the golden ratio and of the square roots of 3, 2 and 19), the upper
// bits folded onto the lower ones in between.
__device__ __forceinline__ uint32_t aw_hash(uint32_t i, uint32_t key) {
  uint32_t h = i * 0x9E3779B1u + key;
  h = (h ^ h >> 16) * 0x6A09E667u;
  h = (h ^ h >> 15) * 0x5BE0CD19u;
  return h ^ h >> 16;
}

// The largest of 32 lanes' magnitudes (as bits, so that a NaN is the largest).
__device__ __forceinline__ uint32_t aw_max32(uint32_t v) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, HSS_WAVE));
  return v;
}

// The scale of a block and 1 / scale; one below 2^-100 (whose inverse could
// overflow) keeps zeros, one that is not finite makes the block read as NaN.
__device__ __forceinline__ float aw_scale(const float* x, float* inv) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
  float s = __uint_as_float(aw_max32(top)) * (float)(1.0 / 448);
  if (s < 0x1p-100f) s = 0.f;
  *inv = s > 0.f && s <= 3.4e38f ? 1.f / s : 0.f;
  return s;
}

// PT: 0 = fp32 parameters, 1 = bf16, 2 = bf16 with an fp32 master copy.
// GT: 0 = fp32 gradients, 1 = bf16.
template <int PT, int GT, int BITS>
__global__ __launch_bounds__(256) void k_adamw(AwArgs a) {
#pragma clang fp contract(off)  // the moments round after each operation, as they are defined
  AwHyper h = a.h;
  if (h.lr_dev || h.step_dev || h.gscale_dev) {
    __shared__ float s[6];
    if (threadIdx.x == 0) {
      const double lr = h.lr_dev ? (double)*h.lr_dev : h.lr;
      double bias1 = h.bias1;
      s[2] = h.root;
      s[3] = h.gscale_dev ? *h.gscale_dev : h.gscale;
      s[4] = __uint_as_float(h.key);
      if (h.step_dev) {
        const int t = max(*h.step_dev, 1);
        s[4] = __uint_as_float((uint32_t)t * 0xBB67AE85u);
        s[2] = (float)(1.0 / sqrt(1.0 - pow(h.beta2, (double)t)));
        bias1 = 1.0 - pow(h.beta1, (double)t);
      }
      s[1] = (float)(lr / bias1);
      s[0] = (float)(1.0 - lr * h.wd);
    }
    __syncthreads();
    h.decay = s[0], h.size = s[1], h.root = s[2], h.gscale = s[3], h.key = __float_as_uint(s[4]);
  }
  const int lane = threadIdx.x & 31;
  // (walking the table takes a round trip to memory for each tensor)
  const uint32_t first = a.first[threadIdx.x & 63];
  for (uint32_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const AwTensor& t = a.t[__popcll(__ballot(first <= chunk)) - 1];
    const uint32_t own = (chunk - t.first) * kAwChunk + (threadIdx.x >> 5);
    const int64_t i = (int64_t)own * kAwBlock + 8 * lane, rest = t.count - i;
    const int left = rest >= 8 ? 8 : rest > 0 ? (int)rest : 0;
    float g[8], m[8], v[8], p[8];
    if constexpr (GT == 0) aw_load(static_cast<const float*>(t.g), i, left, g);
    else aw_load(static_cast<const uint16_t*>(t.g), i, left, g);
    if constexpr (PT == 0) aw_load(static_cast<const float*>(t.p), i, left, p);
    else if constexpr (PT == 1) aw_load(static_cast<const uint16_t*>(t.p), i, left, p);
    else aw_load(t.master, i, left, p);
    if constexpr (BITS == 32) {
      aw_load(static_cast<const float*>(t.m), i, left, m);
      aw_load(static_cast<const float*>(t.v), i, left, v);
    } else {
      const AwU2 mc = aw_load_codes(static_cast<const uint8_t*>(t.m), i, left);
      const AwU2 vc = aw_load_codes(static_cast<const uint8_t*>(t.v), i, left);
      const float ms = left > 0 ? t.ms[own] : 0.f, vs = left > 0 ? t.vs[own] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] = aw_decode(mc.w[k >> 2] >> (8 * (k & 3)) & 0xffu) * ms;
        const float root = aw_decode(vc.w[k >> 2] >> (8 * (k & 3)) & 0xffu) * vs;
        v[k] = root * root;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = g[k] * h.gscale;
      m[k] = h.b1 * m[k] + h.c1 * x;
      v[k] = h.b2 * v[k] + h.c2 * (x * x);
      const float root = sqrtf(v[k]);
      p[k] = p[k] * h.decay - h.size * (m[k] / (root * h.root + h.eps));
      if constexpr (BITS == 8) v[k] = root;
    }
    if constexpr (PT == 0) aw_store(static_cast<float*>(t.p), i, left, p);
    else aw_store(static_cast<uint16_t*>(t.p), i, left, p);
    if constexpr (PT == 2) aw_store(t.master, i, left, p);
    if constexpr (BITS == 32) {
      aw_store(static_cast<float*>(t.m), i, left, m);
      aw_store(static_cast<float*>(t.v), i, left, v);
    } else {
      float mi, vi;
      const float ms = aw_scale(m, &mi), vs = aw_scale(v, &vi);
      const uint32_t at = (t.pos + own) * kAwBlock + 8u * lane;
      AwU2 mc = {{0u, 0u}}, vc = {{0u, 0u}};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t u = aw_hash(at + k, h.key);
        if (mi > 0.f) mc.w[k >> 2] |= aw_encode(m[k], mi, u & 0xffffu, 0u) << (8 * (k & 3));
        if (vi > 0.f) vc.w[k >> 2] |= aw_encode(v[k], vi, u >> 16, 1u) << (8 * (k & 3));
      }
      aw_store_codes(static_cast<uint8_t*>(t.m), i, left, mc);
      aw_store_codes(static_cast<uint8_t*>(t.v), i, left, vc);
      if (lane == 0 && left > 0) t.ms[own] = ms, t.vs[own] = vs;
    }
  }
}

template <int PT, int GT>
static void launch_aw(int bits, unsigned grid, const AwArgs& a, hipStream_t s) {
  if (bits == 32) hipLaunchKernelGGL((k_adamw<PT, GT, 32>), dim3(grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_adamw<PT, GT, 8>), dim3(grid), dim3(256), 0, s, a);
}

hss_status launch_adamw(const hss_adamw_config* c, const hss_adamw_tensor* tensors, const void* const* grads, int count,
                        hipStream_t s) {
  AwArgs a;
  AwHyper& h = a.h;
  h.b1 = (float)c->beta1, h.c1 = (float)(1.0 - c->beta1);
  h.b2 = (float)c->beta2, h.c2 = (float)(1.0 - c->beta2);
  h.beta1 = c->beta1, h.beta2 = c->beta2, h.lr = c->lr, h.wd = c->weight_decay;
  h.eps = (float)c->eps;
  h.decay = (float)(1.0 - c->lr * c->weight_decay);
  h.gscale = (float)c->grad_scale;
  h.lr_dev = c->lr_dev, h.step_dev = c->step_dev, h.gscale_dev = c->grad_scale_dev;
  h.bias1 = 1.0 - std::pow(c->beta1, (double)c->step);
  h.size = (float)(c->lr / h.bias1);
  h.root = (float)(1.0 / std::sqrt(1.0 - std::pow(c->beta2, (double)c->step)));
  h.key = (uint32_t)c->step * 0xBB67AE85u;
  if (count == 0) return HSS_OK;
  uint32_t pos = 0;
  for (int at = 0; at < count;) {
    a.tensors = 0, a.chunks = 0;
    bool master = false;
    for (; at < count && a.tensors < kAwTensors; ++at) {
      const hss_adamw_tensor& q = tensors[at];
      if (q.count == 0 || !grads[at]) continue;
      const bool own = q.master != nullptr;
      if (a.tensors && own != master) break;  // one kernel variant a launch
      const uint32_t blocks = (uint32_t)((q.count + kAwBlock - 1) / kAwBlock);
      master = own;
      a.t[a.tensors++] = AwTensor{q.param, q.master, grads[at], q.m, q.v, q.m_scale, q.v_scale, q.count, a.chunks, pos};
      a.chunks += (blocks + kAwChunk - 1) / kAwChunk;
      pos += blocks;
    }
    for (int k = 0; k < 64; ++k) a.first[k] = k < a.tensors ? a.t[k].first : 0xffffffffu;
    if (!a.tensors) {  // only tensors without elements or gradients were left
      if (!pos) return HSS_OK;  // nothing was launched
      break;
    }
    // A workgroup for each chunk (38 M elements, fp32 and 8-bit moments: 210 and 130
    // us; 2048 workgroups that go round 237 and 150), but for device scalars, whose
    // powers each workgroup computes.  (A launch takes fewer than 2^32 threads.)
    const bool scalars = c->lr_dev || c->step_dev || c->grad_scale_dev;
    const unsigned grid = std::min<uint32_t>(a.chunks, scalars ? 2048 : 1u << 23);
    const int pt = c->dtype == HSS_F32 ? 0 : master ? 2 : 1;
    if (c->grad_dtype == HSS_F32) {
      if (pt == 0) launch_aw<0, 0>(c->bits, grid, a, s);
      else if (pt == 1) launch_aw<1, 0>(c->bits, grid, a, s);
      else launch_aw<2, 0>(c->bits, grid, a, s);
    } else {
      if (pt == 0) launch_aw<0, 1>(c->bits, grid, a, s);
      else if (pt == 1) launch_aw<1, 1>(c->bits, grid, a, s);
      else launch_aw<2, 1>(c->bits, grid, a, s);
    }
  }
  return hipGetLastError() == hipSuccess ? HSS_OK : HSS_ERR_HIP;
}

}  // namespace hss
