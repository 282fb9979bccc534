// block_norm_bwd_silu.cu -- backward pass of the norms around a block, gate g sig(g).
#include "block_norm_bwd.cuh"

namespace lstm {

lstm_status norm_bwd_silu(NormArgs& a, const BwdShape& s, cudaStream_t cs) { return run_gate<LSTM_GATE_SILU>(a, s, cs); }

}  // namespace lstm
