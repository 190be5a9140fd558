// Host side that the training operators (fsdp_ops.h) share: device queries,
// argument checks, launches, and the word that records waits that gave up.
#include "ops.h"

#include <mutex>

namespace fsdp {
namespace {
constexpr int kMaxDevices = 64;
__device__ uint32_t g_status;
}  // namespace

cudaError_t status_word(uint32_t **word) {
  static std::mutex lock;
  static uint32_t *at[kMaxDevices];
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> hold(lock);
  if (!at[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, g_status);
    if (e != cudaSuccess) return e;
    at[dev] = static_cast<uint32_t *>(p);
  }
  *word = at[dev];
  return cudaSuccess;
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
  uint32_t *at = nullptr, word = 0;
  cudaError_t e = status_word(&at);
  if (e == cudaSuccess) e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaMemcpy(&word, at, sizeof(word), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && word) e = cudaMemset(at, 0, sizeof(word));
  if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status read: ") + cudaGetErrorString(e));
  if (word)
    return fail(FSDP_ETIMEOUT, "a bounded device wait gave up (status bits " + std::to_string(word) + ")");
  clear_error();
  return FSDP_OK;
}
