// block_norm_bwd_gate.cu -- the block norm's backward with a gate, without a branch norm.
#include "block_norm_bwd.cuh"

namespace sbl {

cudaError_t block_norm_bwd_gate(BwdArgs& a, const GradOut& g, bool y_bf16, bool h_f32, int& blocks,
                                cudaStream_t stream, int num_sms) {
  return run_mode<false, true>(a, g, y_bf16, h_f32, blocks, stream, num_sms);
}

}  // namespace sbl
