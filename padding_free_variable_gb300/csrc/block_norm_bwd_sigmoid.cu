// block_norm_bwd_sigmoid.cu -- backward pass of the norms around a block, gate sig(g).
#include "block_norm_bwd.cuh"

namespace lstm {

lstm_status norm_bwd_sigmoid(NormArgs& a, const BwdShape& s, cudaStream_t cs) { return run_gate<LSTM_GATE_SIGMOID>(a, s, cs); }

}  // namespace lstm
