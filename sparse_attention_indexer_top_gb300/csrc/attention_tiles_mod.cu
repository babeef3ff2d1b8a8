// Tile kernel of the attention: the instances with masks and a bias by distance.
// See attention_tiles.cuh.
#include "attention_tiles.cuh"

namespace sai {

cudaError_t launch_attn_tiles_mod(const AttnLaunch& p, long long max_keys, void* workspace, int num_sms,
                                  cudaStream_t stream) {
  if (p.cap_log2 > 0.f) return launch_attn_tiles_cap(p, max_keys, workspace, num_sms, stream);
  return p.slopes ? launch_tiles<kMasks | kBias>(p, max_keys, workspace, num_sms, stream)
                  : launch_tiles<kMasks>(p, max_keys, workspace, num_sms, stream);
}

}  // namespace sai
