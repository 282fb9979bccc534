// la_tensor_64.cu -- the tensor-core walks of la_tensor.cuh for padded widths of 64 (queries, keys) and 64 (values).
#include "la_tensor.cuh"

namespace lstm {

lstm_status launch_la_64_64(const LaArgs& a, bool states, cudaStream_t cs)
{
    return launch_padded<64, 64>(a, states, cs);
}

}  // namespace lstm
