// launch.cuh -- host-side helpers that every entry point shares: the device's
// limits, occupancy, and launches with programmatic stream serialisation.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/topk_b200.h"
#include "common.cuh"

namespace tk {

// Status word of the library's other translation unit (decode_api.cu).
__attribute__((visibility("hidden"))) int decode_take_device_status(int* out);

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxN = 2147483647LL;       // indices are int32
constexpr int64_t kMaxElems = 1LL << 50;      // keeps the partition arithmetic in int64
constexpr size_t kSmemPerSm = 228 * 1024;
constexpr size_t kSmemReservedPerCta = 1024;

struct DeviceInfo {
  bool init = false;
  int sms = 0;
  int max_smem_optin = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

int current_device_info(DeviceInfo* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TOPK_ECUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.init) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return TOPK_ECUDA;
    if (cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
        cudaSuccess)
      return TOPK_ECUDA;
    d.init = true;
  }
  *out = d;
  return TOPK_OK;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int host_next_pow2(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

// Resident CTAs per SM of (kernel, dynamic smem) on a device, cached: the
// attribute call and the occupancy query cost microseconds of host time.
struct OccKey {
  int dev;
  const void* fn;
  size_t smem;
  int blocks;
};
constexpr int kOccSlots = 1024;
OccKey g_occ[kOccSlots];
int g_occ_n = 0;
std::mutex g_occ_mu;

// Kernels whose dynamic shared-memory limit has been raised, per device.  The
// limit is raised once to the device's opt-in maximum, so any later launch of
// the kernel may use any size up to it (a per-size setting would be undone by
// the next call that asks for less).
struct AttrKey {
  int dev;
  const void* fn;
};
AttrKey g_attr[kOccSlots];
int g_attr_n = 0;

template <typename KernelT>
int raise_smem_limit_locked(KernelT kernel, int dev, int max_optin) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  for (int i = 0; i < g_attr_n; ++i)
    if (g_attr[i].dev == dev && g_attr[i].fn == fn) return TOPK_OK;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return TOPK_ECUDA;
  const int dyn_max = max_optin - static_cast<int>(fa.sharedSizeBytes);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn_max) !=
      cudaSuccess)
    return TOPK_ECUDA;
  if (g_attr_n >= kOccSlots) return TOPK_ECUDA;
  g_attr[g_attr_n++] = AttrKey{dev, fn};
  return TOPK_OK;
}

template <typename KernelT>
int prepare_kernel(KernelT kernel) {
  int dev = 0, max_optin = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ECUDA;
  if (cudaDeviceGetAttribute(&max_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
      cudaSuccess)
    return TOPK_ECUDA;
  std::lock_guard<std::mutex> lk(g_occ_mu);
  return raise_smem_limit_locked(kernel, dev, max_optin);
}

template <typename KernelT>
int occupancy(KernelT kernel, int block, size_t smem, int* blocks) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return TOPK_ECUDA;
  const void* fn = reinterpret_cast<const void*>(kernel);
  {
    std::lock_guard<std::mutex> lk(g_occ_mu);
    for (int i = 0; i < g_occ_n; ++i) {
      if (g_occ[i].dev == dev && g_occ[i].fn == fn && g_occ[i].smem == smem) {
        *blocks = g_occ[i].blocks;
        return TOPK_OK;
      }
    }
  }
  int rc = prepare_kernel(kernel);
  if (rc) return rc;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(blocks, kernel, block, smem) != cudaSuccess)
    return TOPK_ECUDA;
  if (*blocks < 1) return TOPK_EUNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_occ_mu);
  if (g_occ_n < kOccSlots) g_occ[g_occ_n++] = OccKey{dev, fn, smem, *blocks};
  return TOPK_OK;
}

// Launch errors are read right after the launch; a non-sticky error left by
// an earlier, unrelated runtime call is cleared first (clear_launch_error) so
// that it is not reported as this launch's failure.
void clear_launch_error() { (void)cudaGetLastError(); }

int launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? TOPK_OK : TOPK_ECUDA;
}

// Launch with programmatic stream serialisation: the kernel may begin while
// the previous kernel on the stream finishes; it waits on the device
// (griddepcontrol.wait) before reading or writing global memory.
template <typename... KArgs, typename... Args>
int launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
               Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  clear_launch_error();
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return TOPK_ECUDA;
  }
  return launch_status();
}

// launch_pdl for a kernel launched in clusters of cluster_x CTAs (along x).
template <typename... KArgs, typename... Args>
int launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       int cluster_x, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster_x);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  clear_launch_error();
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return TOPK_ECUDA;
  }
  return launch_status();
}

// Reads and clears this translation unit's device status word.
int take_device_status(int* out) {
  const int zero = 0;
  if (cudaMemcpyFromSymbol(out, g_device_status, sizeof(int)) != cudaSuccess) return TOPK_ECUDA;
  if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return TOPK_ECUDA;
  return TOPK_OK;
}

}  // namespace
}  // namespace tk
