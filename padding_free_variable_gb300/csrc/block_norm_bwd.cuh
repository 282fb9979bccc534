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
//
// Measured with the sums' kernel, cold L2: 40555 x 1024 bf16 with a silu gate 140 us, 4.7 TB/s (two
// rows at a time and values two by two; one and one took 169 us): 59 instructions a value keep the
// schedulers busy in 54 % of their cycles and 128 registers leave 16 warps an SM to hide the rest;
// 200000 x 128 fp32 137 us, 6.0 TB/s; 5000 x 8192 bf16 196 us (344 us with everything looked up at run
// time); odd, 9564 x 517 fp32 centred, 77 us, 2.1 TB/s, value by value 83 us; 30000 x 1001 bf16 beside
// an fp32 stream 191 us, 3.5 TB/s.
#pragma once

#include <algorithm>

#include "block_norm.cuh"

namespace lstm {

constexpr int kSMs = 152;

struct BwdShape {
    int per, tpr, threads, ctas;        // values of a thread / 8, threads of a row and of a CTA, CTAs an SM
};

// Eight values a thread while a row then fits a CTA of 512.  (7 columns more than a row has: shifted
// rows may need a group more.)
inline BwdShape bwd_shape(int D)
{
    BwdShape s;
    const int wide = D % 8 && D + 7 <= 4096 ? D + 7 : D;
    s.per = wide <= 4096 ? 1 : wide <= 8192 ? 2 : 4;
    s.tpr = row_threads(ceil_div(wide, 8 * s.per));
    s.threads = s.tpr <= 32 ? 128 : s.tpr;
    s.ctas = s.threads <= 64 ? 16 : s.threads <= 96 ? 10 : s.threads <= 128 ? 8 : s.threads <= 256 ? 4 : 2;       // at most
    return s;
}

namespace {

// Arithmetic on one value or on two at once.
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
template <typename X> __device__ __forceinline__ X both(float v);
template <> __device__ __forceinline__ float both<float>(float v) { return v; }
template <> __device__ __forceinline__ F2 both<F2>(float v) { return F2(v, v); }
template <typename X> __device__ __forceinline__ X minus(X a, X b) { return fma2(b, both<X>(-1.f), a); }
__device__ __forceinline__ float total(float v) { return v; }
__device__ __forceinline__ float total(F2 v) { return v.lo() + v.hi(); }
__device__ __forceinline__ void spread(float v, float* to) { to[0] = v; }
__device__ __forceinline__ void spread(F2 v, float* to) { to[0] = v.lo(); to[1] = v.hi(); }
__device__ __forceinline__ void gate_pair(float x, float& s, float& c) { sigmoid_pair(x, s, c); }
__device__ __forceinline__ void gate_pair(F2 x, F2& s, F2& c) { sigmoid_pair2(x, s, c); }
__device__ __forceinline__ float gate_value(float x) { return rcp_approx(1.f + ex2_approx(x * kNegLog2e)); }
__device__ __forceinline__ F2 gate_value(F2 x) { return sigmoid2(x); }

template <typename X, typename G> __device__ __forceinline__ X values(const G& g, int v, bool b16)
{
    if constexpr (std::is_same<X, float>::value) return get_value(g, v, b16);
    else return F2(get_value(g, v, b16), get_value(g, v + 1, b16));
}
template <typename X> __device__ __forceinline__ X pick(const float* v, int i)
{
    if constexpr (std::is_same<X, float>::value) return v[i];
    else return F2(v[i], v[i + 1]);
}

// Q neighbouring values of a shifted group.
template <typename T, int VEC, int PER, int Q>
__device__ __forceinline__ void put_piece(T* base, int64_t row, const Cols<VEC, PER>& c, int k, int n, const float (&x)[Q])
{
    if (c.whole(k)) {
        put_group<Q>(base, row + c.at(k) + n * Q, sizeof(T) == 2, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < Q; ++i)
        if (c.valid(k, n * Q + i)) base[row + c.at(k) + n * Q + i] = from_f32<T>(x[i]);
}

// Sums of a kind of block, and its parameters (with the mark of a row's own places).
__host__ __device__ constexpr int bwd_vectors(int kind) { return kind == LSTM_NORM_RMS ? 3 : kSums; }

// Means over a row of t xh (m1) and, for centred norms, of t (m0); sums: R of the one, R of the other.
template <int R> __device__ __forceinline__ void row_means(RowSum& sum, float (&sums)[2 * R], bool centred, float inv, float (&m0)[R], float (&m1)[R])
{
    if (centred) {
        sum(sums);
    } else {
        float v[R];
#pragma unroll
        for (int q = 0; q < R; ++q) v[q] = sums[q];
        sum(v);
#pragma unroll
        for (int q = 0; q < R; ++q) sums[q] = v[q];
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        m1[q] = sums[q] * inv;
        m0[q] = centred ? sums[R + q] * inv : 0.f;
    }
}

// 4, 8, 16 threads or a warp a row up to 256 columns (then several rows a CTA), one CTA a row beyond.
template <typename TB, typename TS, typename TN, int VEC, int PER, int R, int THREADS, int CTAS, int KIND, int GATE, bool SHIFT>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs p, const int tpr)
{
    // KIND: LSTM_NORM_RMS (no biases) or LSTM_NORM_LAYER (biases), a whole block with everything
    // given and wanted, or 0: whatever the arguments say
    const int post = KIND ? KIND : p.post, pre = KIND ? KIND : p.pre, gate = KIND ? GATE : p.gate;
    const bool has_y = KIND || p.y, has_dn = KIND || p.dn, has_dxo = KIND || p.dx_out;
    constexpr bool GIVEN = KIND != 0, BIAS = KIND != LSTM_NORM_RMS, CENTRED = BIAS;
    auto wants = [&](int which) { return KIND ? which % 3 != 1 || KIND == LSTM_NORM_LAYER : p.sums[which] != nullptr; };
    constexpr int Q = VEC == 1 ? 1 : 4, N = VEC / Q;        // values handled together, such pieces of a group
    typedef typename std::conditional<VEC == 1, float, F2>::type X;     // values taken at once: P of them
    constexpr int P = VEC == 1 ? 1 : 2;
    constexpr bool FAR = PER * VEC > 16;                    // the widest rows' sums do not fit shared memory: in the CTA's part
    // known types at compile time
    const bool S16 = std::is_same<TS, Any>::value ? p.stream16 : sizeof(TS) == 2;
    const bool B16 = std::is_same<TB, Any>::value ? p.branch16 : sizeof(TB) == 2;
    const bool N16 = std::is_same<TN, Any>::value ? p.norm16 : sizeof(TN) == 2;
    __shared__ float s_part[2 * 64];
    extern __shared__ __align__(16) float s_sums[];         // [kSums][PER * N][THREADS][Q]
    const int groups = blockDim.x / tpr, group = threadIdx.x / tpr;
    // R rows at a time: the parameters are read and their sums updated once for them
    Cols<VEC, PER> c{(int)threadIdx.x % tpr, tpr, p.D};
    RowSum sum{s_part, tpr, 0};
    const float inv = 1.f / (float)p.D;
    float* const out = p.part + (int64_t)blockIdx.x * kSums * p.D;
    // a kind without biases keeps three sums; shifted rows' CTAs are as large as their rows need
    auto slot = [](int which) { return KIND == LSTM_NORM_RMS ? (which + 1) / 2 : which; };
    const int threads = SHIFT ? (int)blockDim.x : THREADS;
    auto place = [&](int which, int k, int n) {
        return FAR ? out + which * p.D + c.at(k) + n * Q : s_sums + ((slot(which) * PER * N + k * N + n) * threads + (int)threadIdx.x) * Q;
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
    // shifted columns' parameters, after the sums: w_post, scale, w_pre (1, b_post)
    const OwnParams<SHIFT ? VEC : 4, PER> own{(float4*)(s_sums + bwd_vectors(KIND) * PER * VEC * threads)};
    if constexpr (SHIFT) {
        c.shift = (int)((blockIdx.x * (uint64_t)groups + group) * (unsigned)p.D & 7u);
        own.fill(0, c, [&](int i) { return p.w.w_post[i]; });
        own.fill(1, c, [&](int i) { return p.w.scale[i]; });
        own.fill(2, c, [&](int i) { return p.w.w_pre[i]; });
        if (BIAS) {
            own.fill(3, c, [](int) { return 1.f; });
            own.fill(4, c, [&](int i) { return p.w.b_post[i]; });
        }
    }
    for (int which = 0; which < kSums; ++which)
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (wants(which) && (!FAR || c.has(k)))
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int i = 0; i < Q; ++i) place(which, k, n)[i] = 0.f;
    auto params = [&](int k, int n, int which, const float* from, bool ever, float none, float (&v)[Q]) {
        if (SHIFT && ever) {
            if constexpr (SHIFT) own.get(which, k, n, v);
        } else if (ever) {
            get_params<Q, GIVEN>(from, c.at(k) + n * Q, none, v);
        } else {
            get_params<Q, false, false>(from, 0, none, v);
        }
    };

    const int64_t step = (int64_t)gridDim.x * groups;           // the R rows lie this far apart
    for (int64_t base = blockIdx.x * (int64_t)groups; base < p.rows; base += step * R) {
        const int64_t r0 = base + group;
        Group<TS, VEC> rx[R][PER], rd[R][PER];
        Group<TB, VEC> ry[R][PER], rg[R][PER];
        Group<TN, VEC> rn[R][PER];
        float my[R], sy[R], mx[R], sx[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            // past the last row: zeros, which add nothing and are not written
            const bool row = r0 + q * step < p.rows;
            const int64_t r = row ? r0 + q * step : p.rows - 1;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                rx[q][k].zero();
                rd[q][k].zero();
                ry[q][k].zero();
                rg[q][k].zero();
                rn[q][k].zero();
                if (!c.has(k) || !row) continue;
                if constexpr (SHIFT) {
                    const bool inside = c.whole(k) || r < p.rows - 1;
                    load_shifted(rx[q][k], p.x, r * p.D, c, k, inside);
                    load_shifted(ry[q][k], p.y, r * p.ldy, c, k, inside);
                    if (gate) load_shifted(rg[q][k], p.g, r * p.ldg, c, k, inside);
                    load_shifted(rn[q][k], p.dn, r * p.D, c, k, inside);
                    load_shifted(rd[q][k], p.dx_out, r * p.D, c, k, inside, true);
                    continue;
                }
                load_group(rx[q][k], p.x, r * p.D + c.at(k), S16);
                if (has_y) load_group(ry[q][k], p.y, r * p.ldy + c.at(k), B16);
                if (gate) load_group(rg[q][k], p.g, r * p.ldg + c.at(k), B16);
                if (has_dn) load_group(rn[q][k], p.dn, r * p.D + c.at(k), N16);
                if (has_dxo) load_group(rd[q][k], p.dx_out, r * p.D + c.at(k), S16, true);
            }
            const float4 st = __ldg((const float4*)(p.stats + r * 4));
            my[q] = KIND == LSTM_NORM_RMS ? 0.f : st.x;
            sy[q] = st.y;
            mx[q] = KIND == LSTM_NORM_RMS ? 0.f : st.z;
            sx[q] = st.w;
        }
        X xh[R][PER][VEC / P], t[R][PER][VEC / P];
        float sums[2 * R];              // of t xh, then (centred norms) of t
        X part[2 * R];
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) part[q] = both<X>(0.f);
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float wq[Q], bq[Q], s[Q], wp[Q], in[Q];
#pragma unroll
                for (int q = 0; q < R; ++q)
#pragma unroll
                    for (int i = n * Q / P; i < (n + 1) * Q / P; ++i) xh[q][k][i] = t[q][k][i] = both<X>(0.f);
                if (!c.has(k)) continue;
                params(k, n, 0, p.w.w_post, true, 1.f, wq);
                params(k, n, 4, p.w.b_post, BIAS, 0.f, bq);
                params(k, n, 3, nullptr, SHIFT && CENTRED, 1.f, in);
                params(k, n, 1, p.w.scale, true, 1.f, s);
                params(k, n, 2, p.w.w_pre, true, 1.f, wp);
#pragma unroll
                for (int q = 0; q < R; ++q)
#pragma unroll
                    for (int i = 0; i < Q; i += P) {
                        const int v = n * Q + i;
                        X x1 = values<X>(rx[q][k], v, S16);
                        if (has_y) {
                            X u = values<X>(ry[q][k], v, B16);
                            if (CENTRED) u = u + both<X>(-my[q]);
                            u = u * both<X>(sy[q]) * pick<X>(wq, i);
                            if (BIAS) u = u + pick<X>(bq, i);
                            u = u * pick<X>(s, i);
                            if (gate) {
                                const X g = values<X>(rg[q][k], v, B16), a = gate_value(g);
                                u = u * (gate == LSTM_GATE_SILU ? g * a : a);
                            }
                            x1 = x1 + u;
                        }
                        if (CENTRED) x1 = x1 + both<X>(-mx[q]);
                        X h = x1 * both<X>(sx[q]);
                        const X e = values<X>(rn[q][k], v, N16) * pick<X>(wp, i);
                        // (zeros beyond a row's ends stay zeros unless a mean is taken off)
                        if (SHIFT && CENTRED) h = h * pick<X>(in, i);
                        xh[q][k][v / P] = h;
                        t[q][k][v / P] = e;
                        part[q] = fma2(e, h, part[q]);
                        if (CENTRED) part[R + q] = part[R + q] + e;
                    }
            }
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) {
            sums[q] = total(part[q]);
            part[q] = both<X>(0.f);
        }
        float m0[R], m1[R];
        if (has_dn) row_means(sum, sums, pre == LSTM_NORM_LAYER, inv, m0, m1);
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                if (!c.has(k)) continue;
                float wq[Q], bq[Q], s[Q], in[Q];
                X a[kSums][Q / P];      // the parameters' gradients' terms of these rows
                params(k, n, 0, p.w.w_post, true, 1.f, wq);
                params(k, n, 4, p.w.b_post, BIAS, 0.f, bq);
                params(k, n, 3, nullptr, SHIFT && CENTRED, 1.f, in);
                params(k, n, 1, p.w.scale, true, 1.f, s);
#pragma unroll
                for (int which = 0; which < kSums; ++which)
#pragma unroll
                    for (int i = 0; i < Q / P; ++i) a[which][i] = both<X>(0.f);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const int64_t r = r0 + q * step;
                    const bool row = r < p.rows;
                    float dx[Q], dg[Q];
#pragma unroll
                    for (int i = 0; i < Q; i += P) {
                        const int v = n * Q + i;
                        const X h = xh[q][k][v / P], e = values<X>(rn[q][k], v, N16);
                        X d = values<X>(rd[q][k], v, S16);
                        if (has_dn) {
                            X x = fma2(h, both<X>(-m1[q]), t[q][k][v / P]);
                            if (CENTRED) x = x + both<X>(-m0[q]);
                            d = fma2(x, both<X>(sx[q]), d);
                        }
                        if (SHIFT && CENTRED) d = d * pick<X>(in, i);
                        a[3][i / P] = fma2(e, h, a[3][i / P]);
                        a[4][i / P] = a[4][i / P] + e;
                        spread(d, dx + i);
                        if (!has_y) continue;
                        X yh = values<X>(ry[q][k], v, B16);
                        if (CENTRED) yh = yh + both<X>(-my[q]);
                        yh = yh * both<X>(sy[q]);
                        X u = yh * pick<X>(wq, i);
                        if (BIAS) u = u + pick<X>(bq, i);
                        X du = d * pick<X>(s, i), dv = du, ua = u;
                        if (gate) {
                            const X g = values<X>(rg[q][k], v, B16);
                            X act, neg;
                            gate_pair(g, act, neg);
                            // act' = s (1 - s), or of the silu gate s (1 + g (1 - s))
                            const X slope = gate == LSTM_GATE_SILU ? act * fma2(g, neg, both<X>(1.f)) : act * neg;
                            if (gate == LSTM_GATE_SILU) act = g * act;
                            spread(du * u * slope, dg + i);
                            dv = du * act;
                            ua = u * act;
                        }
                        const X e2 = dv * pick<X>(wq, i);
                        t[q][k][v / P] = e2;
                        xh[q][k][v / P] = yh;
                        part[q] = fma2(e2, yh, part[q]);
                        if (CENTRED) part[R + q] = part[R + q] + e2;
                        a[0][i / P] = fma2(dv, yh, a[0][i / P]);
                        a[1][i / P] = a[1][i / P] + dv;
                        a[2][i / P] = fma2(d, ua, a[2][i / P]);
                    }
                    if (!row) continue;
                    if constexpr (SHIFT) {
                        put_piece((TS*)p.dx, r * p.D, c, k, n, dx);
                        if (gate) put_piece((TB*)p.dg, r * p.lddg, c, k, n, dg);
                    } else {
                        put_group<Q>(p.dx, r * p.D + c.at(k) + n * Q, S16, dx);
                        if (gate) put_group<Q>(p.dg, r * p.lddg + c.at(k) + n * Q, B16, dg);
                    }
                }
#pragma unroll
                for (int which = 0; which < kSums; ++which)
                    if (wants(which)) {
                        float f[Q];
#pragma unroll
                        for (int i = 0; i < Q; i += P) spread(a[which][i / P], f + i);
                        add(which, k, n, f);
                    }
            }
        if (!has_y) continue;
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) sums[q] = total(part[q]);
        if (post) row_means(sum, sums, post == LSTM_NORM_LAYER, inv, m0, m1);
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int64_t r = r0 + q * step;
            if (r >= p.rows) continue;
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (!c.has(k)) continue;
                float dy[VEC];
#pragma unroll
                for (int v = 0; v < VEC; v += P) {
                    X d = t[q][k][v / P];
                    if (post) {
                        d = fma2(xh[q][k][v / P], both<X>(-m1[q]), d);
                        if (CENTRED) d = d + both<X>(-m0[q]);
                        d = d * both<X>(sy[q]);
                    }
                    spread(d, dy + v);
                }
                if constexpr (SHIFT) put_shifted((TB*)p.dy, r * p.lddy, c, k, dy);
                else put_group<VEC>(p.dy, r * p.lddy + c.at(k), B16, dy);
            }
        }
    }
    if (FAR) return;
    // this CTA's sums, its rows' groups added in order
    __syncthreads();
    if constexpr (SHIFT) {      // the groups' columns are shifted differently: by column
        for (int which = 0; which < kSums; ++which)
            for (int i = threadIdx.x; wants(which) && i < p.D; i += blockDim.x) {
                float s = 0.f;
                for (int g = 0; g < groups; ++g) {
                    const int shift = (int)((blockIdx.x * (uint64_t)groups + g) * (unsigned)p.D & 7u), at = i + shift;
                    const int n = at % VEC / Q, t = at / VEC;
                    s += s_sums[((slot(which) * N + n) * threads + g * tpr + t) * Q + at % Q];
                }
                out[which * p.D + i] = s;
            }
        return;
    }
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
                        out[which * p.D + c.at(k) + n * Q + i] = s;
                    }
    }
}

template <typename TB, typename TS, typename TN, int VEC, int PER, int R, int THREADS, int CTAS, int KIND, int GATE, bool SHIFT = false>
lstm_status run(NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    static std::atomic<uint64_t> ready{0};
    auto* fn = norm_bwd_kernel<TB, TS, TN, VEC, PER, R, THREADS, CTAS, KIND, GATE, SHIFT>;
    const int64_t groups = s.threads / s.tpr;
    constexpr size_t VECTOR = sizeof(float) * PER * VEC;        // a thread's part of one sum or parameter
    const size_t smem = PER * VEC > 16 ? 0 : VECTOR * bwd_vectors(KIND) * (SHIFT ? 2 * s.threads : THREADS);
    int dev = 0;
    LSTM_CUDA_TRY(cudaGetDevice(&dev));
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        LSTM_CUDA_TRY(cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)(PER * VEC > 16 ? 0 : VECTOR * bwd_vectors(KIND) * (SHIFT ? 2 : 1) * THREADS)));
        if (dev < 64) ready.fetch_or(bit, std::memory_order_release);
    }
    // as many CTAs as stay resident, asked for once for each size of a CTA
    static std::atomic<int> resident[17];
    std::atomic<int>& known = resident[s.threads / 32];
    int fit = known.load(std::memory_order_relaxed);
    if (fit == 0) {
        LSTM_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, s.threads, smem));
        fit = std::max(fit, 1);
        known.store(fit, std::memory_order_relaxed);
    }
    const int64_t rows = (a.rows + R - 1) / R;
    a.parts = (int)std::min<int64_t>(a.parts, std::min<int64_t>((rows + groups - 1) / groups, (int64_t)kSMs * fit));
    if (SHIFT) a.parts = (int)shifted_blocks(a.parts);
    fn<<<a.parts, s.threads, smem, cs>>>(a, s.tpr);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

// A whole block of one kind and gate, by types: y's, x's (dn has y's).
template <int KIND, int GATE, typename TB, typename TS> lstm_status run_block(NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    // rows with 2-byte values two at a time (40000 x 1024 bf16 beside an fp32 stream 156 us, 183 one at a
    // time; centred 183 and 225 us); fp32 rows twice over do not fit the registers.  Four CTAs of 128 for
    // two rows and for the centred fp32 block (80000 x 512: 266 us, six CTAs of 80 registers 345), six for
    // the other (200000 x 320: 375 us, four 407).
    constexpr int R = sizeof(TB) == 2 ? 2 : 1;
    if (norm_whole(a)) {
        if (s.threads <= 128) return run<TB, TS, TB, 8, 1, R, 128, R == 2 || KIND == LSTM_NORM_LAYER ? 4 : 6, KIND, GATE>(a, s, cs);
        if (s.threads <= 256) return run<TB, TS, TB, 8, 1, R, 256, R == 2 ? 2 : 3, KIND, GATE>(a, s, cs);
        if (s.per == 2) return run<TB, TS, TB, 8, 2, 1, 512, 1, KIND, GATE>(a, s, cs);
        if (s.threads <= 384) return run<TB, TS, TB, 8, 1, 1, 384, 2, KIND, GATE>(a, s, cs);
        return run<TB, TS, TB, 8, 1, R, 512, 1, KIND, GATE>(a, s, cs);
    }
    if (norm_shifted(a) && a.D + 7 <= 4096) {
        // more warps gain more than more registers until these run out: seven CTAs of 128 threads an SM, five
        // for centred rows (60000 x 511 bf16: 244 us, five 308; centred, beside an fp32 stream, 355 us, seven
        // 402).  Rows of a CTA of 512, which leaves no second one, two at a time (9000 x 3501 bf16 269 and 308 us).
        if (s.threads <= 128) return run<TB, TS, TB, 8, 1, 1, 128, KIND == LSTM_NORM_RMS ? 7 : 5, KIND, GATE, true>(a, s, cs);
        if (s.threads <= 256) return run<TB, TS, TB, 8, 1, 1, 256, 3, KIND, GATE, true>(a, s, cs);
        if (s.threads <= 384) return run<TB, TS, TB, 8, 1, 1, 384, 2, KIND, GATE, true>(a, s, cs);
        return run<TB, TS, TB, 8, 1, R, 512, 1, KIND, GATE, true>(a, s, cs);
    }
    if (s.threads <= 128) return run<TB, TS, TB, 1, 8, 1, 128, 6, KIND, GATE>(a, s, cs);
    if (s.threads <= 256) return run<TB, TS, TB, 1, 8, 1, 256, 3, KIND, GATE>(a, s, cs);
    return run<TB, TS, TB, 1, 8, 1, 512, 1, KIND, GATE>(a, s, cs);
}

template <int GATE> lstm_status run_gate(NormArgs& a, const BwdShape& s, cudaStream_t cs)
{
    typedef __nv_bfloat16 H;
    const bool rms = a.post == LSTM_NORM_RMS;
    if (!a.branch16) return rms ? run_block<LSTM_NORM_RMS, GATE, float, float>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, float, float>(a, s, cs);
    if (a.stream16) return rms ? run_block<LSTM_NORM_RMS, GATE, H, H>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, H, H>(a, s, cs);
    return rms ? run_block<LSTM_NORM_RMS, GATE, H, float>(a, s, cs) : run_block<LSTM_NORM_LAYER, GATE, H, float>(a, s, cs);
}

}  // namespace

// One translation unit a gate.
lstm_status norm_bwd_none(NormArgs& a, const BwdShape& s, cudaStream_t cs);
lstm_status norm_bwd_sigmoid(NormArgs& a, const BwdShape& s, cudaStream_t cs);
lstm_status norm_bwd_silu(NormArgs& a, const BwdShape& s, cudaStream_t cs);

}  // namespace lstm
