// block_norm_bwd_post.cu -- the block norm's backward with a branch norm, without a gate.
#include "block_norm_bwd.cuh"

namespace sbl {

cudaError_t block_norm_bwd_post(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                cudaStream_t stream, int num_sms) {
  return run_mode<true, false>(a, g, y_bf16, h_f32, blocks, stream, num_sms);
}

}  // namespace sbl
