// host.cuh -- what the C entry points of every source file share: the device
// table, the shared-memory opt-in and the launch with programmatic stream
// serialization.  Everything is local to the including file.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/fp8q.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kInt32Max = 2147483647;

// ------------------------------------------------------------ device info ---

struct DeviceInfo {
  int sms = 0;
  bool ready = false;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

fp8q_status current_device(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return FP8Q_ERR_CUDA;
  if (*dev < 0 || *dev >= kMaxDevices) return FP8Q_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[*dev];
  if (!d.ready) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) return FP8Q_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess) return FP8Q_ERR_CUDA;
    if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess) return FP8Q_ERR_CUDA;
    if (major != 10 || minor != 0) return FP8Q_ERR_UNSUPPORTED;   // built for sm_100a only
    d.ready = true;
  }
  *sms = d.sms;
  return FP8Q_OK;
}

// Opt a kernel in to large dynamic shared memory, once per (kernel, device).
struct SmemOptIn {
  const void* fn;
  int dev;
};
SmemOptIn g_optin[256];
int g_noptin = 0;
std::mutex g_optin_mu;

template <typename K>
fp8q_status ensure_smem(K kernel, int bytes, int dev) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  std::lock_guard<std::mutex> lk(g_optin_mu);
  for (int i = 0; i < g_noptin; ++i)
    if (g_optin[i].fn == fn && g_optin[i].dev == dev) return FP8Q_OK;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return FP8Q_ERR_CUDA;
  if (g_noptin < 256) g_optin[g_noptin++] = {fn, dev};
  return FP8Q_OK;
}

// cluster_x > 0: launched in clusters of cluster_x CTAs (for kernels without
// a compile-time cluster shape).
template <typename... KArgs, typename... Args>
fp8q_status launch_clustered(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, void* stream,
                             int cluster_x, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  // Programmatic dependent launch: the kernel may begin while its stream
  // predecessor finishes; every kernel here waits (griddepcontrol.wait)
  // before touching global memory.
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster_x > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster_x);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FP8Q_OK : FP8Q_ERR_CUDA;
}

template <typename... KArgs, typename... Args>
fp8q_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, void* stream, Args... args) {
  return launch_clustered(kernel, grid, block, smem, stream, 0, args...);
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
