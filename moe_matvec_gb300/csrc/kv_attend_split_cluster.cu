// Attention over the paged 8-bit cache: queries in two f16 parts, 8 rows a fragment,
// a cluster per item.
#include "kv_attend.cuh"

namespace qmv {

cudaError_t launch_attend_split_cluster(AttendParams& p, int D, cudaStream_t stream) {
  return launch_attend_as<false, true>(p, D, stream);
}

// Clusters of c CTAs, one an SM, that the GPU holds at once (0 if it cannot be
// told): every variant takes most of an SM, so one stands for all.
int attend_resident_clusters(int c) {
  static std::atomic<int> known[64][4];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev > 63) return 0;
  std::atomic<int>& k = known[dev][c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : 3];
  if ((n = k.load()) != 0) return n;
  const size_t smem = attend_smem<128, 64, 1, false>(0);
  const auto kernel = kv_attend_kernel<128, 64, 1, false, true>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, device_smem_optin() - 1024) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  make_config(cfg, attr, dim3(c), dim3(at_warps(128, 1, false) * 32), smem, nullptr, true);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
  k.store(n);
  return n;
}

}  // namespace qmv
