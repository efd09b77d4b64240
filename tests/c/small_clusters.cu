// The norm's gradient as a device would run it that holds no cluster of 16 CTAs:
// norm.cu with a limit of our own on the clusters that can be resident and that
// are launched.
#include <cuda_runtime.h>

static unsigned g_most = 16;
extern "C" void set_largest_cluster(unsigned most) { g_most = most; }

static bool too_large(const cudaLaunchConfig_t* cfg) {
  for (unsigned i = 0; i < cfg->numAttrs; i++)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension && cfg->attrs[i].val.clusterDim.x > g_most) return true;
  return false;
}

template <typename Kernel>
static cudaError_t limited_clusters(int* n, Kernel kernel, const cudaLaunchConfig_t* cfg) {
  *n = 0;
  return too_large(cfg) ? cudaErrorInvalidClusterSize : cudaOccupancyMaxActiveClusters(n, kernel, cfg);
}

template <typename... Params, typename... Args>
static cudaError_t limited_launch(const cudaLaunchConfig_t* cfg, void (*kernel)(Params...), Args&&... args) {
  return too_large(cfg) ? cudaErrorInvalidClusterSize : cudaLaunchKernelEx(cfg, kernel, static_cast<Args&&>(args)...);
}

#define cudaOccupancyMaxActiveClusters limited_clusters
#define cudaLaunchKernelEx limited_launch
#include "norm.cu"
