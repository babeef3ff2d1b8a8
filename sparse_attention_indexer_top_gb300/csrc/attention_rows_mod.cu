// Row kernel of the attention: the instances with changed scores and masks. See
// attention_rows.cuh.
#include "attention_rows.cuh"

namespace sai {

cudaError_t launch_attn_rows_mod(const AttnLaunch& p, cudaStream_t stream) { return launch_rows<true>(p, stream); }

}  // namespace sai
