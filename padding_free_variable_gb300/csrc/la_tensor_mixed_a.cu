// la_tensor_mixed_a.cu -- the tensor-core walks of la_tensor.cuh for padded widths of 64 (queries, keys) and 128 (values).
#include "la_tensor.cuh"

namespace lstm {

lstm_status launch_la_64_128(const LaArgs& a, bool states, cudaStream_t cs)
{
    return launch_padded<64, 128>(a, states, cs);
}

}  // namespace lstm
