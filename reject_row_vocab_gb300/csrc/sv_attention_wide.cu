// Attention for many query rows over a cache of bf16: the launch of the kernel that sv_attention_wide.cuh describes.
#include "sv_attention_wide.cuh"

namespace sv {

cudaError_t launch_attention_wide(const AttnParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int dim = p.c.head_dim;
  const KvMaps maps = kv_maps(p.c);
  return dim <= 64 ? launch_wide<1, 1, RowSource>(p, maps, dev, stream) : dim <= 128 ? launch_wide<2, 1, RowSource>(p, maps, dev, stream) : launch_wide<2, 2, RowSource>(p, maps, dev, stream);
}

}  // namespace sv
