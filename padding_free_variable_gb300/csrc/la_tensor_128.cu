// la_tensor_128.cu -- the tensor-core walks of la_tensor.cuh for padded widths of 128 (queries, keys) and 128 (values).
#include "la_tensor.cuh"

namespace lstm {

lstm_status launch_la_128_128(const LaArgs& a, bool states, cudaStream_t cs)
{
    return launch_padded<128, 128>(a, states, cs);
}

}  // namespace lstm
