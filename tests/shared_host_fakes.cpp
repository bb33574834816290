// Stands in for what the host side of mla_shared_fwd calls, so that its calls can be counted and made to
// fail without a GPU: built with api_long.cu as one host library by the CPU tests.
#include <cstdint>

#include "kernels.h"
#include "ops.h"

extern "C" {
int fake_maps, fake_launches, fake_joins;  // calls so far
int fake_maps_fail, fake_launch_fail;      // set by the test
}

cudaError_t cudaGetDevice(int* device) {
  *device = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* value, cudaDeviceAttr, int) {
  *value = 152;
  return cudaSuccess;
}

namespace mla {
mla_status_t device_ready(int* device) {
  *device = 0;
  return MLA_OK;
}
bool cache_maps(const void*, int64_t, int, CUtensorMap*, CUtensorMap*) {
  ++fake_maps;
  return !fake_maps_fail;
}
cudaError_t launch_shared(const SharedParams&, const SharedMaps&, cudaStream_t) {
  ++fake_launches;
  return fake_launch_fail ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t launch_shared_join(const SharedParams&, int32_t, cudaStream_t) {
  ++fake_joins;
  return cudaSuccess;
}
cudaError_t launch_block_means(const BlockMeansParams&, bool, int32_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_block_scores(const BlockScoresParams&, int32_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_block_select(const BlockSelectParams&, cudaStream_t) { return cudaSuccess; }
}  // namespace mla
