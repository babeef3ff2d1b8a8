// Tile kernel of the attention: the instances with capped scores. See
// attention_tiles.cuh.
#include "attention_tiles.cuh"

namespace sai {

cudaError_t launch_attn_tiles_cap(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                                  cudaStream_t stream) {
  return p.slopes ? launch_tiles<kMasks | kCap | kBias>(p, max_keys, workspace, num_sms, stream)
                  : launch_tiles<kMasks | kCap>(p, max_keys, workspace, num_sms, stream);
}

}  // namespace sai
