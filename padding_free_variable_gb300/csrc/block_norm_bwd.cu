// block_norm_bwd.cu -- backward pass of the norms around a block.
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
#include <algorithm>

#include "block_norm.cuh"

namespace lstm {

namespace {

// One warp a row (four rows a CTA) up to 256 columns, one CTA a row beyond.
template <typename TB, typename TS, typename TN, int VEC, int PER, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs p, const int tpr)
{
    constexpr int Q = VEC == 1 ? 1 : 4, N = VEC / Q;        // values handled together, such pieces of a group
    constexpr bool FAR = PER * VEC > 16;                    // the widest rows' sums do not fit shared memory: in the CTA's part
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
            load_group(rx[k], p.x, r * p.D + c.at(k), p.stream16);
            if (p.y) load_group(ry[k], p.y, r * p.ldy + c.at(k), p.branch16);
            if (p.g) load_group(rg[k], p.g, r * p.ldg + c.at(k), p.branch16);
            if (p.dn) load_group(rn[k], p.dn, r * p.D + c.at(k), p.norm16);
            if (p.dx_out) load_group(rd[k], p.dx_out, r * p.D + c.at(k), p.stream16, true);
        }
        const float4 st = __ldg((const float4*)(p.stats + r * 4));
        const float my = st.x, sy = st.y, mx = st.z, sx = st.w;
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
                get_params<Q>(p.w.w_post, at, 1.f, wq);
                get_params<Q>(p.w.b_post, at, 0.f, bq);
                get_params<Q>(p.w.scale, at, 1.f, s);
                get_params<Q>(p.w.w_pre, at, 1.f, wp);
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int v = n * Q + i;
                    float x1 = get_value(rx[k], v, p.stream16);
                    if (p.y) {
                        const float u = fmaf((get_value(ry[k], v, p.branch16) - my) * sy, wq[i], bq[i]);
                        x1 = fmaf(s[i] * u, activation(p.gate, get_value(rg[k], v, p.branch16)), x1);
                    }
                    xh[k][v] = (x1 - mx) * sx;
                    t[k][v] = get_value(rn[k], v, p.norm16) * wp[i];
                    a += t[k][v];
                    b = fmaf(t[k][v], xh[k][v], b);
                }
            }
        float m0 = 0.f, m1 = 0.f;
        if (p.dn) {
            const float2 q = sum(a, b);
            if (p.pre == LSTM_NORM_LAYER) m0 = q.x * inv;
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
                    dx[i] = get_value(rd[k], v, p.stream16);
                    if (p.dn) dx[i] = fmaf(sx, t[k][v] - m0 - xh[k][v] * m1, dx[i]);
                    e[i] = get_value(rn[k], v, p.norm16);
                    f[i] = e[i] * xh[k][v];
                }
                if (p.sums[3]) add(3, k, n, f);
                if (p.sums[4]) add(4, k, n, e);
                put_group<Q>(p.dx, r * p.D + at, p.stream16, dx);
                if (!p.y) continue;
                get_params<Q>(p.w.w_post, at, 1.f, wq);
                get_params<Q>(p.w.b_post, at, 0.f, bq);
                get_params<Q>(p.w.scale, at, 1.f, s);
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const int v = n * Q + i;
                    const float yh = (get_value(ry[k], v, p.branch16) - my) * sy, u = fmaf(yh, wq[i], bq[i]), du = dx[i] * s[i];
                    float act = 1.f, slope = 0.f;
                    if (p.gate) activation(p.gate, get_value(rg[k], v, p.branch16), act, slope);
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
                if (p.sums[0]) add(0, k, n, wq);
                if (p.sums[1]) add(1, k, n, bq);
                if (p.sums[2]) add(2, k, n, s);
                if (p.dg) put_group<Q>(p.dg, r * p.lddg + at, p.branch16, dg);
            }
        if (!p.y) continue;
        float k0 = 0.f, k1 = 0.f;
        if (p.post) {
            const float2 q = sum(a, b);
            if (p.post == LSTM_NORM_LAYER) k0 = q.x * inv;
            k1 = q.y * inv;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (!c.has(k)) continue;
            float dy[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) dy[v] = p.post ? sy * (t[k][v] - k0 - xh[k][v] * k1) : t[k][v];
            put_group<VEC>(p.dy, r * p.lddy + c.at(k), p.branch16, dy);
        }
    }
    if (FAR) return;
    // this CTA's sums, its rows' groups added in order
    __syncthreads();
    if (group > 0) return;
    for (int which = 0; which < kSums; ++which) {
        if (!p.sums[which]) continue;
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

// The partial sums of one parameter's 32 columns: warp w adds every 8th part in order, then the warps in order.
__global__ void __launch_bounds__(256) norm_sums_kernel(const NormArgs p)
{
    __shared__ float s_part[8][32];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane, which = blockIdx.y;
    if (!p.sums[which]) return;
    float s = 0.f;
    if (c < p.D)
        for (int b = w; b < p.parts; b += 8) s += p.part[((int64_t)b * kSums + which) * p.D + c];
    s_part[w][lane] = s;
    __syncthreads();
    if (w > 0 || c >= p.D) return;
    for (int x = 1; x < 8; ++x) s += s_part[x][lane];
    p.sums[which][c] = s;
}

struct BwdShape {
    int per, tpr, threads, ctas;        // values of a thread / 8, threads of a row and of a CTA, CTAs an SM
};

// Eight values a thread while a row then fits a CTA of 512.
BwdShape bwd_shape(int D)
{
    BwdShape s;
    s.per = D <= 4096 ? 1 : D <= 8192 ? 2 : 4;
    s.tpr = (ceil_div(D, 8 * s.per) + 31) / 32 * 32;
    s.threads = s.tpr == 32 ? 128 : s.tpr;
    s.ctas = s.threads <= 128 ? 6 : s.threads <= 256 ? 3 : 1;
    return s;
}

constexpr int kSMs = 152;

template <typename TB, typename TS, typename TN, int VEC, int PER, int THREADS, int CTAS>
lstm_status run(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    static std::atomic<uint64_t> ready{0};
    auto* fn = norm_bwd_kernel<TB, TS, TN, VEC, PER, THREADS, CTAS>;
    const size_t smem = PER * VEC > 16 ? 0 : sizeof(float) * kSums * PER * VEC * THREADS;
    int dev = 0;
    LSTM_CUDA_TRY(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        LSTM_CUDA_TRY(cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    }
    fn<<<a.parts, s.threads, smem, cs>>>(a, s.tpr);
    norm_sums_kernel<<<dim3(ceil_div(a.D, 32), kSums), 256, 0, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

template <typename TB, typename TS, typename TN> lstm_status go(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    if (s.threads <= 128) return run<TB, TS, TN, 8, 1, 128, 6>(a, s, cs);
    if (s.threads <= 256) return run<TB, TS, TN, 8, 1, 256, 3>(a, s, cs);
    return run<TB, TS, TN, 8, 1, 512, 1>(a, s, cs);
}

lstm_status go_any(const NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    if (norm_whole(a)) {
        if (s.per == 2) return run<Any, Any, Any, 8, 2, 512, 1>(a, s, cs);
        return run<Any, Any, Any, 8, 4, 512, 1>(a, s, cs);
    }
    if (s.threads <= 128) return run<Any, Any, Any, 1, 8, 128, 6>(a, s, cs);
    if (s.threads <= 256) return run<Any, Any, Any, 1, 8, 256, 3>(a, s, cs);
    if (s.per == 1) return run<Any, Any, Any, 1, 8, 512, 1>(a, s, cs);
    if (s.per == 2) return run<Any, Any, Any, 1, 16, 512, 1>(a, s, cs);
    return run<Any, Any, Any, 1, 32, 512, 1>(a, s, cs);
}

}  // namespace

int norm_parts(int64_t rows, int D)
{
    const BwdShape s = bwd_shape(D);
    const int64_t groups = s.threads / s.tpr;
    return (int)std::min<int64_t>((rows + groups - 1) / groups, (int64_t)kSMs * s.ctas);
}

lstm_status launch_norm_bwd(const NormArgs& a, cudaStream_t cs)
{
    typedef __nv_bfloat16 H;
    const BwdShape s = bwd_shape(a.D);
    if (s.per > 1 || !norm_whole(a)) return go_any(a, s, cs);
    if (a.branch16)
        return a.stream16 ? (a.norm16 ? go<H, H, H>(a, s, cs) : go<H, H, float>(a, s, cs))
                          : (a.norm16 ? go<H, float, H>(a, s, cs) : go<H, float, float>(a, s, cs));
    return a.stream16 ? (a.norm16 ? go<float, H, H>(a, s, cs) : go<float, H, float>(a, s, cs))
                      : (a.norm16 ? go<float, float, H>(a, s, cs) : go<float, float, float>(a, s, cs));
}

}  // namespace lstm
