// block_norm_bwd.cuh -- backward pass of the norms around a block: the row kernel.
//
// With yh, xh the normalised rows (recomputed from x, y, gate and the statistics kept by the
// forward pass, so x' is not read), t = dn w_pre, and mean(.) over a row,
//     dx   = dx' + rx (t - mean(t) - xh mean(t xh))            mean(t) for centred norms only
//     du   = scale dx,  dv = du act(g),  q = dv w_post
//     dy   = ry (q - mean(q) - yh mean(q yh)),  dgate = du v act'(g)
// and the parameters' gradients are sums over rows: dw_post = dv yh, db_post = dv, dscale = dx v
// act, dw_pre = dn xh, db_pre = dn.  Bound by memory: five values read and three written.  CTAs
// stay and take every so-many-th row; a thread keeps its columns from row to row and adds the
// parameters' terms to its own places in shared memory (no atomics: no other thread has them), so
// they cost no traffic.  Each CTA then writes its partial sums once, and a second kernel adds
// them in order.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace lstm {

struct BwdShape {
    int per, tpr, threads, ctas;        // values of a thread / 8, threads of a row and of a CTA, CTAs an SM
};

// Eight values a thread while a row then fits a CTA of 512.
inline BwdShape bwd_shape(int D)
{
    BwdShape s;
    s.per = D <= 4096 ? 1 : D <= 8192 ? 2 : 4;
    s.tpr = (ceil_div(D, 8 * s.per) + 31) / 32 * 32;
    s.threads = s.tpr == 32 ? 128 : s.tpr;
    s.ctas = s.threads <= 128 ? 6 : s.threads <= 256 ? 3 : 1;
    return s;
}


namespace {

// One warp a row (four rows a CTA) up to 256 columns, one CTA a row beyond.
template <typename TB, typename TS, typename TN, int VEC, int PER, int THREADS, int CTAS, int KIND, int GATE>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs p, const int tpr)
{
    // KIND: LSTM_NORM_RMS (no biases) or LSTM_NORM_LAYER (biases), a whole block with everything
    // given and wanted, or 0: whatever the arguments say
    const int post = KIND ? KIND : p.post, pre = KIND ? KIND : p.pre, gate = KIND ? GATE : p.gate;
    const bool has_y = KIND || p.y, has_dn = KIND || p.dn, has_dxo = KIND || p.dx_out;
    constexpr bool GIVEN = KIND != 0, BIAS = KIND != LSTM_NORM_RMS;
    auto wants = [&](int which) { return KIND ? which % 3 != 1 || KIND == LSTM_NORM_LAYER : p.sums[which] != nullptr; };
    constexpr int Q = VEC == 1 ? 1 : 4, N = VEC / Q;        // values handled together, such pieces of a group
    constexpr bool FAR = PER * VEC > 16;                    // the widest rows' sums do not fit shared memory: in the CTA's part
    // known types at compile time
    const bool S16 = std::is_same<TS, Any>::value ? p.stream16 : sizeof(TS) == 2;
    const bool B16 = std::is_same<TB, Any>::value ? p.branch16 : sizeof(TB) == 2;
    const bool N16 = std::is_same<TN, Any>::value ? p.norm16 : sizeof(TN) == 2;
    __shared__ float2 s_part[2 * 32];
    extern __shared__ __align__(16) float s_sums[];         // [kSums][PER * N][THREADS][Q]
    const int groups = blockDim.x / tpr, group = threadIdx.x / tpr;
    const Cols<VEC, PER> c{(int)threadIdx.x % tpr, tpr, p.D};
    RowSum sum{s_part, tpr / 32, 0};
    const float inv = 1.f / (float)p.D;
    float* const part = p.part + (int64_t)blockIdx.x * kSums * p.D;
    auto place = [&](int which, int k, int n) {
        return FAR ? part + which * p.D + c.at(k) + n * Q : s_sums + ((which * PER * N + k * N + n) * THREADS + (int)threadIdx.x) * Q;
    };
    auto add = [&](int which, int k, int n, const float (&x)[Q]) {
        float* at = place(which, k, n);
        if constexpr (Q == 1) {
            *at += x[0];
        } else {
            float4 q = *(float4*)at;
            q.x += x[0]; q.y += x[1]; q.z += x[2]; q.w += x[3];
            *(float4*)at = q;
        }
    };
    for (int which = 0; which < kSums; ++which)
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (!FAR || c.has(k))
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < Q; ++i) place(which, k, n)[i] = 0.f;

    for (int64_t r = blockIdx.x * (int64_t)groups + group; r < p.rows; r += (int64_t)gridDim.x * groups) {
        Group<TS, VEC> rx[PER], rd[PER];
        Group<TB, VEC> ry[PER], rg[PER];
        Group<TN, VEC> rn[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            rx[k].zero();
            rd[k].zero();
            ry[k].zero();
            rg[k].zero();
            rn[k].zero();
            if (!c.has(k)) continue;
            load_group(rx[k], p.x, r * p.D + c.at(k), S16);
            if (has_y) load_group(ry[k], p.y, r * p.ldy + c.at(k), B16);
            if (gate) load_group(rg[k], p.g, r * p.ldg + c.at(k), B16);
            if (has_dn) load_group(rn[k], p.dn, r * p.D + c.at(k), N16);
            if (has_dxo) load_group(rd[k], p.dx_out, r * p.D + c.at(k), S16, true);
        }
        const float4 st = __ldg((const float4*)(p.stats + r * 4));
        const float my = KIND == LSTM_NORM_RMS ? 0.f : st.x, sy = st.y, mx = KIND == LSTM_NORM_RMS ? 0.f : st.z, sx = st.w;
        float xh[PER][VEC], t[PER][VEC];
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float wq[Q], bq[Q], s[Q], wp[Q];
#pragma unroll
                for (int i = 0; i < Q; ++i) xh[k][n * Q + i] = t[k][n * Q + i] = 0.f;
                if (!c.has(k)) continue;
                const int at = c.at(k) + n * Q;
                get_params<Q, GIVEN>(p.w.w_post, at, 1.f, wq);
                get_params<Q, GIVEN, BIAS>(p.w.b_post, at, 0.f, bq);
                get_params<Q, GIVEN>(p.w.scale, at, 1.f, s);
                get_params<Q, GIVEN>(p.w.w_pre, at, 1.f, wp);
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int v = n * Q + i;
                    float x1 = get_value(rx[k], v, S16);
                    if (has_y) {
                        const float u = fmaf((get_value(ry[k], v, B16) - my) * sy, wq[i], bq[i]);
                        x1 = fmaf(s[i] * u, gate ? activation(gate, get_value(rg[k], v, B16)) : 1.f, x1);
                    }
                    xh[k][v] = (x1 - mx) * sx;
                    t[k][v] = get_value(rn[k], v, N16) * wp[i];
                    a += t[k][v];
                    b = fmaf(t[k][v], xh[k][v], b);
                }
            }
        float m0 = 0.f, m1 = 0.f;
        if (has_dn) {
            const float2 q = sum(a, b);
            if (pre == LSTM_NORM_LAYER) m0 = q.x * inv;
            m1 = q.y * inv;
        }
        a = b = 0.f;
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (!c.has(k)) continue;
                float wq[Q], bq[Q], s[Q], dx[Q], dg[Q], e[Q], f[Q];
                const int at = c.at(k) + n * Q;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int v = n * Q + i;
                    dx[i] = get_value(rd[k], v, S16);
                    if (has_dn) dx[i] = fmaf(sx, t[k][v] - m0 - xh[k][v] * m1, dx[i]);
                    e[i] = get_value(rn[k], v, N16);
                    f[i] = e[i] * xh[k][v];
                }
                if (wants(3)) add(3, k, n, f);
                if (wants(4)) add(4, k, n, e);
                put_group<Q>(p.dx, r * p.D + at, S16, dx);
                if (!has_y) continue;
                get_params<Q, GIVEN>(p.w.w_post, at, 1.f, wq);
                get_params<Q, GIVEN, BIAS>(p.w.b_post, at, 0.f, bq);
                get_params<Q, GIVEN>(p.w.scale, at, 1.f, s);
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int v = n * Q + i;
                    const float yh = (get_value(ry[k], v, B16) - my) * sy, u = fmaf(yh, wq[i], bq[i]), du = dx[i] * s[i];
                    float act = 1.f, slope = 0.f;
                    if (gate) activation(gate, get_value(rg[k], v, B16), act, slope);
                    const float dv = du * act;
                    dg[i] = du * u * slope;
                    t[k][v] = dv * wq[i];
                    xh[k][v] = yh;
                    a += t[k][v];
                    b = fmaf(t[k][v], yh, b);
                    wq[i] = dv * yh;
                    bq[i] = dv;
                    s[i] = dx[i] * u * act;
                }
                if (wants(0)) add(0, k, n, wq);
                if (wants(1)) add(1, k, n, bq);
                if (wants(2)) add(2, k, n, s);
                if (gate) put_group<Q>(p.dg, r * p.lddg + at, B16, dg);
            }
        if (!has_y) continue;
        float k0 = 0.f, k1 = 0.f;
        if (post) {
            const float2 q = sum(a, b);
            if (post == LSTM_NORM_LAYER) k0 = q.x * inv;
            k1 = q.y * inv;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (!c.has(k)) continue;
            float dy[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) dy[v] = post ? sy * (t[k][v] - k0 - xh[k][v] * k1) : t[k][v];
            put_group<VEC>(p.dy, r * p.lddy + c.at(k), B16, dy);
        }
    }
    if (FAR) return;
    // this CTA's sums, its rows' groups added in order
    __syncthreads();
    if (group > 0) return;
    for (int which = 0; which < kSums; ++which) {
        if (!wants(which)) continue;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (c.has(k))
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        float s = 0.f;
                        for (int g = 0; g < groups; ++g) s += place(which, k, n)[g * tpr * Q + i];
                        part[which * p.D + c.at(k) + n * Q + i] = s;
                    }
    }
}

template <typename TB, typename TS, typename TN, int VEC, int PER, int THREADS, int CTAS, int KIND, int GATE>
lstm_status run(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    static std::atomic<uint64_t> ready{0};
    auto* fn = norm_bwd_kernel<TB, TS, TN, VEC, PER, THREADS, CTAS, KIND, GATE>;
    const size_t smem = PER * VEC > 16 ? 0 : sizeof(float) * kSums * PER * VEC * THREADS;
    int dev = 0;
    LSTM_CUDA_TRY(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        LSTM_CUDA_TRY(cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    }
    fn<<<a.parts, s.threads, smem, cs>>>(a, s.tpr);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

// A whole block of one kind and gate, by types: y's, x's (dn has y's).
template <int KIND, int GATE, typename TB, typename TS> lstm_status run_block(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    if (norm_whole(a)) {
        if (s.threads <= 128) return run<TB, TS, TB, 8, 1, 128, 6, KIND, GATE>(a, s, cs);
        if (s.threads <= 256) return run<TB, TS, TB, 8, 1, 256, 3, KIND, GATE>(a, s, cs);
        return run<TB, TS, TB, 8, 1, 512, 1, KIND, GATE>(a, s, cs);
    }
    if (s.threads <= 128) return run<TB, TS, TB, 1, 8, 128, 6, KIND, GATE>(a, s, cs);
    if (s.threads <= 256) return run<TB, TS, TB, 1, 8, 256, 3, KIND, GATE>(a, s, cs);
    return run<TB, TS, TB, 1, 8, 512, 1, KIND, GATE>(a, s, cs);
}

template <int GATE> lstm_status run_gate(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    typedef __nv_bfloat16 H;
    const bool rms = a.post == LSTM_NORM_RMS;
    if (!a.branch16) return rms ? run_block<LSTM_NORM_RMS, GATE, float, float>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, float, float>(a, s, cs);
    if (a.stream16) return rms ? run_block<LSTM_NORM_RMS, GATE, H, H>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, H, H>(a, s, cs);
    return rms ? run_block<LSTM_NORM_RMS, GATE, H, float>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, H, float>(a, s, cs);
}

}  // namespace

// One translation unit a gate.
lstm_status norm_bwd_none(const NormArgs& a, const BwdShape& s, cudaStream_t cs);
lstm_status norm_bwd_sigmoid(const NormArgs& a, const BwdShape& s, cudaStream_t cs);
lstm_status norm_bwd_silu(const NormArgs& a, const BwdShape& s, cudaStream_t cs);

}  // namespace lstm
