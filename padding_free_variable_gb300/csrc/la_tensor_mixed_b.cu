// la_tensor_mixed_b.cu -- the tensor-core walks of la_tensor.cuh for padded widths of 128 (queries, keys) and 64 (values).
#include "la_tensor.cuh"

namespace lstm {

lstm_status launch_la_128_64(const LaArgs& a, bool states, cudaStream_t cs)
{
    return launch_padded<128, 64>(a, states, cs);
}

}  // namespace lstm
