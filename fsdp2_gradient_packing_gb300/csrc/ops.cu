// Host side that the training operators (fsdp_ops.h) share: device queries,
// argument checks, launches, and the counts of waits that gave up.
#include "ops.h"

#include <mutex>

namespace fsdp {
namespace {
constexpr int kMaxDevices = 64;
__device__ uint32_t g_gave_up[GAVE_UP_KINDS];

// The current device's counts, and its index.
cudaError_t counts(uint32_t **at, int *device) {
  static std::mutex lock;
  static uint32_t *known[kMaxDevices];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> hold(lock);
  if (!known[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_gave_up);
    if (e != cudaSuccess) return e;
    known[dev] = static_cast<uint32_t *>(p);
  }
  *at = known[dev], *device = dev;
  return cudaSuccess;
}
}  // namespace

cudaError_t gave_up_count(GaveUp kind, uint32_t **count) {
  int dev;
  cudaError_t e = counts(count, &dev);
  if (e == cudaSuccess) *count += kind;
  return e;
}

int device_sms() {
  static std::mutex lock;
  static int sms[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> hold(lock);
  if (dev < kMaxDevices && sms[dev] > 0) return sms[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < kMaxDevices) sms[dev] = n;
  return n;
}

fsdp_status_t check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size, const char *what) {
  if (ld < cols) return fail(FSDP_EINVAL, std::string(what) + ": row distance below the number of columns");
  if (rows > 0 && ld > INT64_MAX / 16 / rows) return fail(FSDP_EUNSUPPORTED, std::string(what) + " is too large");
  return check_ptr(p, rows * cols * size, size, what, -1);
}

cudaError_t launch_kernel(const void *fn, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t stream,
                          bool overlap, int cluster) {
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  if (overlap) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
    at[cfg.numAttrs].val.clusterDim.y = 1;
    at[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace fsdp

using namespace fsdp;

extern "C" fsdp_status_t fsdp_ops_sync_status(fsdp_stream_t stream) {
  static thread_local uint32_t seen[kMaxDevices][GAVE_UP_KINDS];
  uint32_t *at = nullptr, now[GAVE_UP_KINDS] = {}, kinds = 0;
  int dev = -1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = counts(&at, &dev);
  if (e == cudaSuccess) e = cudaMemcpyAsync(now, at, sizeof(now), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status read: ") + cudaGetErrorString(e));
  for (int k = 0; k < GAVE_UP_KINDS; ++k) {
    if (now[k] != seen[dev][k]) kinds |= 16u << k;
    seen[dev][k] = now[k];
  }
  if (kinds)
    return fail(FSDP_ETIMEOUT, "a bounded device wait gave up (status bits " + std::to_string(kinds) + ")");
  clear_error();
  return FSDP_OK;
}
