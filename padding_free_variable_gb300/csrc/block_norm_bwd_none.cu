// block_norm_bwd_none.cu -- backward pass of the norms around a block, no gate.
#include "block_norm_bwd.cuh"

namespace lstm {

lstm_status norm_bwd_none(NormArgs& a, const BwdShape& s, cudaStream_t cs) { return run_gate<LSTM_GATE_NONE>(a, s, cs); }

}  // namespace lstm
