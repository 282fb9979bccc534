// block_norm_fwd.cu -- forward pass of the norms around a block.
//
// x' = x + scale * (norm(y) w + b) * act(gate), n = norm(x') w + b, row by row.  A row's values
// stay in its threads' registers from the one read of x, y and gate to the one write of x' and n;
// its variances are taken around its mean in a second sweep over registers, so a mean far above
// the deviation costs no digits.  Bound by memory: 5 values of traffic against about 20 operations.
// A warp takes a row of up to 1024 values (no barrier; many rows an SM hide the latency), wider
// rows take a CTA; a call of few rows spreads each over as many threads as it has groups of
// eight, since there only the time of one row counts (8 rows of 1024: 2.5 us in a graph).
//
// Measured, cold L2: 40555 x 1024 bf16 70 us, 5.9 TB/s (88 % of the copy rate; 91 us with kinds and
// types looked up at run time); 200000 x 128 fp32 74 us, 6.9 TB/s.  Odd widths: 9564 x 517 fp32 centred
// 38 us, 2.6 TB/s, where the sums over three warps and the rows' ends cost more than the bytes (issue
// 52 %, memory 22 %); value by value the same rows take 64 us.  A warp a row with four groups a
// lane, and rows 8 apart sharing a CTA's parameters, were no faster (42 us).
#include <algorithm>

#include "block_norm.cuh"

namespace lstm {

namespace {

// KIND as in the backward pass: a whole block of one kind, or 0, whatever the arguments say.
template <typename TB, typename TS, int VEC, int PER, int KIND, int GATE, bool SHIFT>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormArgs p, const int tpr)
{
    const int post = KIND ? KIND : p.post, pre = KIND ? KIND : p.pre, gate = KIND ? GATE : p.gate;
    const bool has_y = KIND || p.y;
    constexpr bool GIVEN = KIND != 0, BIAS = KIND != LSTM_NORM_RMS;
    const bool S16 = std::is_same<TS, Any>::value ? p.stream16 : sizeof(TS) == 2;
    const bool B16 = std::is_same<TB, Any>::value ? p.branch16 : sizeof(TB) == 2;
    const bool N16 = KIND ? B16 : p.norm16;
    __shared__ float s_part[2 * 64];
    extern __shared__ __align__(16) float4 s_own[];     // shifted columns: w_post, scale, w_pre (1, b_post, b_pre)
    const int groups = blockDim.x / tpr;
    const float inv = 1.f / (float)p.D;
    RowSum sum{s_part, tpr, 0};
    Cols<VEC, PER> c{(int)threadIdx.x % tpr, tpr, p.D};
    const OwnParams<SHIFT ? VEC : 4, PER> own{s_own};
    if constexpr (SHIFT) {
        c.shift = (int)((blockIdx.x * (uint64_t)groups + threadIdx.x / tpr) * (unsigned)p.D & 7u);
        own.fill(0, c, [&](int i) { return p.w.w_post[i]; });
        own.fill(1, c, [&](int i) { return p.w.scale[i]; });
        own.fill(2, c, [&](int i) { return p.w.w_pre[i]; });
        if (BIAS) {
            own.fill(3, c, [](int) { return 1.f; });
            own.fill(4, c, [&](int i) { return p.w.b_post[i]; });
            own.fill(5, c, [&](int i) { return p.w.b_pre[i]; });
        }
    }
    auto params = [&](int k, int which, const float* from, bool ever, float none, float (&v)[VEC]) {
        if (SHIFT && ever) {
            if constexpr (SHIFT) own.get(which, k, 0, v);
        } else if (ever) {
            get_params<VEC, GIVEN>(from, c.at(k), none, v);
        } else {
            get_params<VEC, false, false>(from, 0, none, v);
        }
    };
    // 1 for the row's values, 0 for the places beyond its ends: what a centred norm's mean would otherwise make of them
    auto inside = [&](int k, float (&v)[VEC]) { params(k, 3, nullptr, SHIFT && BIAS, 1.f, v); };
    // shifted: every so-many-th row; else a row each, in a grid of all rows
    int64_t r = blockIdx.x * (int64_t)groups + threadIdx.x / tpr;
    for (int64_t first = blockIdx.x * (int64_t)groups;;) {
        c.row = r < p.rows;

        Group<TS, VEC> rx[PER];
        Group<TB, VEC> ry[PER], rg[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            rx[k].zero();
            ry[k].zero();
            rg[k].zero();
            if (!c.has(k)) continue;
            if constexpr (SHIFT) {
                const bool all = c.whole(k) || r < p.rows - 1;
                load_shifted(rx[k], p.x, r * p.D, c, k, all, true);
                load_shifted(ry[k], p.y, r * p.ldy, c, k, all);
                if (gate) load_shifted(rg[k], p.g, r * p.ldg, c, k, all);
                continue;
            }
            load_group(rx[k], p.x, r * p.D + c.at(k), S16, true);
            if (has_y) load_group(ry[k], p.y, r * p.ldy + c.at(k), B16);
            if (gate) load_group(rg[k], p.g, r * p.ldg + c.at(k), B16);
        }
        float my = 0.f, sy = 1.f, mx = 0.f, sx = 1.f;
        if (post) {
            float a = 0.f;
            if (post == LSTM_NORM_LAYER) {
#pragma unroll
                for (int k = 0; k < PER; ++k)
                    if (c.has(k))
#pragma unroll
                        for (int v = 0; v < VEC; ++v) a += get_value(ry[k], v, B16);
                my = sum(a) * inv;
                a = 0.f;
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (!c.has(k)) continue;
                float in[VEC];
                inside(k, in);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float d = (get_value(ry[k], v, B16) - my) * in[v];
                    a = fmaf(d, d, a);
                }
            }
            sy = 1.f / sqrtf(fmaf(sum(a), inv, p.eps));
        }
        float x1[PER][VEC];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) x1[k][v] = get_value(rx[k], v, S16);
            if (!has_y || !c.has(k)) continue;
            float w[VEC], b[VEC], s[VEC];
            params(k, 0, p.w.w_post, true, 1.f, w);
            params(k, 4, p.w.b_post, BIAS, 0.f, b);
            params(k, 1, p.w.scale, true, 1.f, s);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float u = fmaf((get_value(ry[k], v, B16) - my) * sy, w[v], b[v]);
                x1[k][v] = fmaf(s[v] * u, gate ? activation(gate, get_value(rg[k], v, B16)) : 1.f, x1[k][v]);
            }
            if constexpr (SHIFT) put_shifted((TS*)p.x_out, r * p.D, c, k, x1[k]);
            else put_group<VEC>(p.x_out, r * p.D + c.at(k), S16, x1[k]);
        }
        if (pre) {
            float a = 0.f;
            if (pre == LSTM_NORM_LAYER) {
#pragma unroll
                for (int k = 0; k < PER; ++k)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a += x1[k][v];
                mx = sum(a) * inv;
                a = 0.f;
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (!c.has(k)) continue;
                float in[VEC];
                inside(k, in);
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float d = (x1[k][v] - mx) * in[v];
                    a = fmaf(d, d, a);
                }
            }
            sx = 1.f / sqrtf(fmaf(sum(a), inv, p.eps));
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (!c.has(k)) continue;
                float w[VEC], b[VEC];
                params(k, 2, p.w.w_pre, true, 1.f, w);
                params(k, 5, p.w.b_pre, BIAS, 0.f, b);
#pragma unroll
                for (int v = 0; v < VEC; ++v) w[v] = fmaf((x1[k][v] - mx) * sx, w[v], b[v]);
                if constexpr (SHIFT) put_shifted((TB*)p.n, r * p.D, c, k, w);
                else put_group<VEC>(p.n, r * p.D + c.at(k), N16, w);
            }
        }
        if (p.stats && c.t == 0 && c.row) *(float4*)(p.stats + r * 4) = make_float4(my, sy, mx, sx);
        if (!SHIFT) break;
        first += (int64_t)gridDim.x * groups;
        r += (int64_t)gridDim.x * groups;
        if (first >= p.rows) break;
    }
}

template <typename TB, typename TS, int VEC, int PER, int KIND, int GATE, bool SHIFT = false> lstm_status run(const NormArgs& a, int tpr, cudaStream_t cs)
{
    const int threads = tpr <= 32 ? 128 : tpr, groups = threads / tpr;
    int64_t blocks = (a.rows + groups - 1) / groups;
    size_t smem = 0;
    if constexpr (SHIFT) {      // CTAs that stay, reading the parameters once
        smem = OwnParams<VEC, PER>::bytes(KIND == LSTM_NORM_LAYER ? 6 : 3, threads);
        blocks = shifted_blocks(std::min<int64_t>(blocks, 152 * std::max(1, 1024 / threads)));
        static std::atomic<uint64_t> ready{0};
        int dev = 0;
        LSTM_CUDA_TRY(cudaGetDevice(&dev));
        const uint64_t bit = 1ull << (dev & 63);
        if (!(ready.load(std::memory_order_acquire) & bit)) {
            LSTM_CUDA_TRY(cudaFuncSetAttribute((const void*)norm_fwd_kernel<TB, TS, VEC, PER, KIND, GATE, SHIFT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, OwnParams<VEC, PER>::bytes(6, 512)));
            if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
        }
    }
    norm_fwd_kernel<TB, TS, VEC, PER, KIND, GATE, SHIFT><<<(unsigned)blocks, threads, smem, cs>>>(a, tpr);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

template <typename TB, typename TS, int KIND, int GATE> lstm_status go(const NormArgs& a, cudaStream_t cs)
{
    // Values of a thread: 8, 16 or 32.  8 where a call's few rows leave SMs idle: RMS, bf16, in a graph, 8 rows
    // of 1024 2.7 / 3.3 / 4.1 us, 304 rows 3.2 / 3.8 / 4.6, 304 of 4096 4.5 / 4.6 / 5.5, 608 of 4096 7.5 / 5.6 / 6.2.
    // Where rows are many (4e7 values, cold L2), 16 up to 512 columns and 32 beyond, which keeps a row
    // within a warp: centred bf16 512 119 / 80 / 91 us, 520 171 / 146 / 136, 768 126 / 105 / 101, 1024 122 / 91 / 93;
    // centred fp32 512 148 / 130 / 154, 520 185 / 199 / 156, 4096 181 / 187 / 160.  Up to 256 columns 8: fp32 128
    // 122 / 124 / 128, bf16 78 / 68 / 72.  Value by value 255 columns (1e7 values, fp32) 48 / 56 / 95, 1003 52 / 64 / 107.
    auto threads = [&](int each) { return row_threads(ceil_div(a.D, each)); };
    const bool few = a.rows <= 304;
    if (norm_whole(a)) {
        if (a.D <= 256 || (few && threads(8) <= 512)) return run<TB, TS, 8, 1, KIND, GATE>(a, threads(8), cs);
        if (a.D <= 512 || (few && threads(16) <= 512)) return run<TB, TS, 8, 2, KIND, GATE>(a, threads(16), cs);
        return run<TB, TS, 8, 4, KIND, GATE>(a, threads(32), cs);
    }
    if constexpr (KIND != 0)
        if (const int n = ceil_div(a.D + 7, 8); norm_shifted(a) && n <= 1024) {      // groups of a row
            if (n <= 512) return run<TB, TS, 8, 1, KIND, GATE, true>(a, row_threads(n), cs);
            return run<TB, TS, 8, 2, KIND, GATE, true>(a, row_threads(ceil_div(n, 2)), cs);
        }
    if (a.D <= 256 || (few && threads(8) <= 512)) return run<TB, TS, 1, 8, KIND, GATE>(a, threads(8), cs);
    if (threads(16) <= 512) return run<TB, TS, 1, 16, KIND, GATE>(a, threads(16), cs);
    return run<TB, TS, 1, 32, KIND, GATE>(a, threads(32), cs);
}

template <typename TB, typename TS> lstm_status go(const NormArgs& a, cudaStream_t cs)
{
    constexpr int R = LSTM_NORM_RMS, L = LSTM_NORM_LAYER;
    if (a.post == R) {
        if (a.gate == LSTM_GATE_SILU) return go<TB, TS, R, LSTM_GATE_SILU>(a, cs);
        return a.gate ? go<TB, TS, R, LSTM_GATE_SIGMOID>(a, cs) : go<TB, TS, R, LSTM_GATE_NONE>(a, cs);
    }
    if (a.gate == LSTM_GATE_SILU) return go<TB, TS, L, LSTM_GATE_SILU>(a, cs);
    return a.gate ? go<TB, TS, L, LSTM_GATE_SIGMOID>(a, cs) : go<TB, TS, L, LSTM_GATE_NONE>(a, cs);
}

}  // namespace

lstm_status launch_norm_fwd(const NormArgs& a, cudaStream_t cs)
{
    typedef __nv_bfloat16 H;
    if (!norm_full(a)) return go<Any, Any, 0, 0>(a, cs);
    if (!a.branch16) return go<float, float>(a, cs);
    return a.stream16 ? go<H, H>(a, cs) : go<H, float>(a, cs);
}

}  // namespace lstm
