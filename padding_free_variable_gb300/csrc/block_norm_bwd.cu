// block_norm_bwd.cu -- backward pass of the norms around a block: choice of the row kernel, the column sums.
#include "block_norm_bwd.cuh"

namespace lstm {

namespace {

// The partial sums of one parameter's 32 columns: warp w adds every 32nd part in order, then the warps in order.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const NormArgs p)
{
    __shared__ float s_part[32][32];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane, which = blockIdx.y;
    if (!p.sums[which]) return;
    float s = 0.f;
    if (c < p.D)
        #pragma unroll 4
        for (int b = w; b < p.parts; b += 32) s += p.part[((int64_t)b * kSums + which) * p.D + c];
    s_part[w][lane] = s;
    __syncthreads();
    if (w > 0 || c >= p.D) return;
    for (int x = 1; x < 32; ++x) s += s_part[x][lane];
    p.sums[which][c] = s;
}

// Blocks with parts missing, other mixes of types, and the widest rows.
lstm_status run_any(NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    if (norm_whole(a)) {
        if (s.threads <= 128) return run<Any, Any, Any, 8, 1, 1, 128, 6, 0, 0>(a, s, cs);
        if (s.threads <= 256) return run<Any, Any, Any, 8, 1, 1, 256, 3, 0, 0>(a, s, cs);
        if (s.per == 1) return run<Any, Any, Any, 8, 1, 1, 512, 1, 0, 0>(a, s, cs);
        if (s.per == 2) return run<Any, Any, Any, 8, 2, 1, 512, 1, 0, 0>(a, s, cs);
        return run<Any, Any, Any, 8, 4, 1, 512, 1, 0, 0>(a, s, cs);
    }
    if (s.threads <= 128) return run<Any, Any, Any, 1, 8, 1, 128, 6, 0, 0>(a, s, cs);
    if (s.threads <= 256) return run<Any, Any, Any, 1, 8, 1, 256, 3, 0, 0>(a, s, cs);
    if (s.per == 1) return run<Any, Any, Any, 1, 8, 1, 512, 1, 0, 0>(a, s, cs);
    if (s.per == 2) return run<Any, Any, Any, 1, 16, 1, 512, 1, 0, 0>(a, s, cs);
    return run<Any, Any, Any, 1, 32, 1, 512, 1, 0, 0>(a, s, cs);
}

}  // namespace

int norm_parts(int64_t rows, int D)
{
    const BwdShape s = bwd_shape(D);
    const int64_t groups = s.threads / s.tpr;
    return (int)shifted_blocks(std::min<int64_t>((rows + groups - 1) / groups, (int64_t)kSMs * s.ctas));
}

lstm_status launch_norm_bwd(NormArgs a, cudaStream_t cs)
{
    const BwdShape s = bwd_shape(a.D);
    lstm_status st = LSTM_OK;
    if ((s.per == 1 || (s.per == 2 && norm_whole(a))) && norm_full(a) && a.dn && a.dx_out && a.sums[0] && a.sums[2] && a.sums[3] &&
        (a.post == LSTM_NORM_LAYER) == (a.sums[1] != nullptr) && (a.post == LSTM_NORM_LAYER) == (a.sums[4] != nullptr))
        st = a.gate == LSTM_GATE_SILU ? norm_bwd_silu(a, s, cs) : a.gate == LSTM_GATE_SIGMOID ? norm_bwd_sigmoid(a, s, cs) : norm_bwd_none(a, s, cs);
    else
        st = run_any(a, s, cs);
    if (st != LSTM_OK) return st;
    norm_sums_kernel<<<dim3(ceil_div(a.D, 32), kSums), 1024, 0, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

}  // namespace lstm
