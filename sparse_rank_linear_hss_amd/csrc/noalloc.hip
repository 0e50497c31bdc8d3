// hss_apply_noalloc: hss_apply with the library's own device scratch instead
// of a caller workspace, for callers that cannot allocate device memory.
//
// The scratch is one file-scope device array per GPU (kScratchBytes, held
// until the process ends).  In host code the array's name is only a host-side
// stand-in, so its device address is looked up once per device with
// hipGetSymbolAddress (with that device current) and only that address is
// passed on.  The first call on a device also clears the whole array with the
// zero-fill kernel, on that call's stream: the fused decode kernel keeps its
// call epoch, arrival counters and tagged T words in the first bytes and needs
// them to start from zeros.  Later calls keep the state the previous call
// left, as the decode kernel expects.  Every call on one GPU shares the array:
// calls that overlap in time on one GPU race and may return wrong values.
//
// HSS_MX4 matrices have a second array of the same size: their scratch holds
// dense data and keeps no state, and a word of it left among the decode
// kernel's T words could carry the tag of a later call.
#include <mutex>

#include "hss_internal.h"

namespace hss {

static constexpr size_t kScratchBytes = (size_t)16 << 20;  // 16 MiB per GPU
static constexpr int kMaxDevices = 64;

static __device__ __align__(256) unsigned char scratch[kScratchBytes];
static __device__ __align__(256) unsigned char scratch_mx[kScratchBytes];

namespace {
std::mutex g_mu;
// device addresses of `scratch` and `scratch_mx` on each device, once looked up
void* g_ptr[kMaxDevices] = {};
void* g_ptr_mx[kMaxDevices] = {};

// The device address of this device's scratch; clears it on the first call
// (on `stream`; the one for HSS_MX4 needs none).  nullptr (and *st set) if the lookup or the clear fails.
void* device_scratch(bool mx, hipStream_t stream, hss_status* st) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
    *st = HSS_ERR_HIP;
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  void** slot = mx ? &g_ptr_mx[dev] : &g_ptr[dev];
  if (!*slot) {
    void* p = nullptr;
    const hipError_t e = mx ? hipGetSymbolAddress(&p, HIP_SYMBOL(scratch_mx)) : hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p) {
      *st = HSS_ERR_HIP;
      return nullptr;
    }
    if (!mx && launch_zero_fill(p, kScratchBytes, stream) != HSS_OK) {
      *st = HSS_ERR_HIP;
      return nullptr;
    }
    *slot = p;
  }
  *st = HSS_OK;
  return *slot;
}
}  // namespace

}  // namespace hss

extern "C" size_t hss_noalloc_scratch_bytes(void) { return hss::kScratchBytes; }

extern "C" hss_status hss_apply_noalloc(const hss_matrix* A, int32_t b, const void* X, void* Y,
                                        hipStream_t stream) {
  const hss_status st = hss::check_apply_args(A, b, X, Y);
  if (st != HSS_OK) return st;
  if (hss::apply_route_ws_bytes(A, b, X) > hss::kScratchBytes) return HSS_ERR_WORKSPACE;
  hss_status sst = HSS_OK;
  void* ws = hss::device_scratch((A->flags & HSS_MX4) != 0, stream, &sst);
  if (!ws) return sst;
  return hss::launch_apply(A, b, X, Y, ws, stream);
}
