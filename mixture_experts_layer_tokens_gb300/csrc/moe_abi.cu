// moe_abi: host-side helpers shared by the entry points -- status strings,
// the device status word, SM counts.
#include "moe_vec.cuh"

#include <atomic>
#include <initializer_list>

namespace moe {

int num_sms() {
  static std::atomic<int> cached[64];  // (host threads may come at once)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  int n = dev >= 0 && dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
  if (n) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 1;
  if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool fits_int32(long long v) { return v >= 0 && v < 2147483647LL; }

}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_device_status(int clear) {
  if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
  const moe_status_t a = experts_status(clear);
  const moe_status_t b = align_status(clear);
  const moe_status_t c = prepare_status(clear);
  const moe_status_t d = finalize_status(clear);
  const moe_status_t e = route_grouped_status(clear);
  const moe_status_t f = linear_status(clear);
  const moe_status_t g = finalize_backward_status(clear);
  for (const moe_status_t st : {a, b, c, d, e, f, g})
    if (st != MOE_OK) return st;
  return MOE_OK;
}

extern "C" const char* moe_status_string(moe_status_t status) {
  switch (status) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARG: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported configuration";
    case MOE_ERR_WORKSPACE: return "workspace missing or too small";
    case MOE_ERR_CUDA: return "CUDA error";
    case MOE_ERR_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}
