// block_norm_bwd_plain.cu -- the block norm's backward without a branch norm or a gate.
#include "block_norm_bwd.cuh"

namespace sbl {

cudaError_t block_norm_bwd_plain(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                 cudaStream_t stream, int num_sms) {
  return run_mode<false, false>(a, g, y_bf16, h_f32, blocks, stream, num_sms);
}

}  // namespace sbl
