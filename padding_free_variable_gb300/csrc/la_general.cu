// la_general.cu -- linear attention on CUDA cores: fp32, and bf16 rows that the tensor cores' loads cannot take.
//
// A CTA walks one head of one sequence (or a piece of it) 64 steps at a time, everything in shared memory in fp32: the
// products of the chunk's steps with each other (64 x 64), the outputs from them and from the state, then the state.
// Per step that is 4 a b products for the state and 64 (a + b) between steps.
#include <type_traits>

#include "la.cuh"

namespace lstm {

namespace {

constexpr int kSteps = 64, kThreads = 256, kLdP = kSteps + 4;

// Floats of a row in shared memory: an odd number of groups of four, so that eight rows next to each other read their
// groups from different banks.
__host__ __device__ constexpr int ld_of(int w) { return ((w + 3) / 4 | 1) * 4; }

size_t shared_bytes(int a, int b, bool states)
{
    const int a4 = (a + 3) / 4 * 4;
    return sizeof(float) * ((size_t)kSteps * (2 * ld_of(a) + ld_of(b)) + (states ? 0 : kSteps * kLdP) + (size_t)a4 * ld_of(b) + kSteps + 4);
}

// `n` rows of `w` values into shared memory, zeros behind them and behind the width's last value.
template <typename T, int V>
__device__ __forceinline__ void load_rows(float* dst, int ld, const LaRows& r, const LaArgs& p, const LaPart& c, int w, int u, int n, bool rev)
{
    const T* base = (const T*)r.p + c.d * r.dir + c.h * r.head;
    const int groups = (w + 3) / 4;
    for (int i = threadIdx.x; i < kSteps * groups; i += kThreads) {
        const int s = i / groups, g = (i - s * groups) * 4;
        float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < n) {
            const int t = rev ? c.len - 1 - (u + s) : u + s;
            const T* at = base + (int64_t)(__ldg(p.off + t) + c.slot) * r.row + g;
            if constexpr (V == 4 && sizeof(T) == 4) {
                q = __ldg((const float4*)at);
            } else if constexpr (V == 4) {
                const uint2 x = __ldg((const uint2*)at);
                q = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                                __uint_as_float(x.y & 0xffff0000u));
            } else {
                q.x = to_f32(at[0]);
                if (g + 1 < w) q.y = to_f32(at[1]);
                if (g + 2 < w) q.z = to_f32(at[2]);
                if (g + 3 < w) q.w = to_f32(at[3]);
            }
        }
        *(float4*)(dst + s * ld + g) = q;
    }
}

template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ void fma4(float4& s, float x, const float4& y)
{
    s.x = fmaf(x, y.x, s.x); s.y = fmaf(x, y.y, s.y); s.z = fmaf(x, y.z, s.z); s.w = fmaf(x, y.w, s.w);
}

// STATES: only what a piece adds to Y, into `starts` (pieces with one behind them).
template <typename T, int V, bool STATES>
__global__ void __launch_bounds__(kThreads) la_general_kernel(const LaArgs p)
{
    extern __shared__ __align__(16) float sm[];
    const LaPart c = la_part(p, blockIdx.x);
    const LaJob& j = p.job[c.job];
    if (STATES && c.last) return;
    const int tid = threadIdx.x, a = j.a, b = j.b, a4 = (a + 3) / 4, b4 = (b + 3) / 4, lda = ld_of(a), ldb = ld_of(b);
    float* const Q = sm;
    float* const K = Q + kSteps * lda;
    float* const W = K + kSteps * lda;
    float* const Vs = W + kSteps + 4;
    float* const Y = Vs + kSteps * ldb;
    float* const P = Y + a4 * 4 * ldb;
    const bool rev = (c.d == 1) != (j.back != 0);
    const float l2 = la_log2_decay(p, c.d, c.h);
    const int64_t state = la_state(p, j, c);

    if (!STATES) {
        la_past_end<T>(p, j, c);
        if (c.len == 0) return la_pass(j, state);
    }
    if (tid <= kSteps) W[tid] = exp2f(tid * l2);
    __syncthreads();
    {
        const float first = j.early ? W[1] : 1.f;
        const float* from = STATES ? nullptr : j.starts ? la_start(p, j, c) : j.init ? j.init + state : nullptr;
        for (int i = tid; i < a4 * 4 * ldb; i += kThreads) {
            const int x = i / ldb, y = i - x * ldb;
            float v = 0.f;
            if (from && x < a && y < b) v = j.starts ? from[x * b + y] : first * from[j.flip ? y * a + x : x * b + y];
            Y[i] = v;
        }
    }
    for (int u = c.begin; u < c.end; u += kSteps) {
        const int n = min(kSteps, c.end - u);
        const bool final = c.last && u + kSteps >= c.end;
        if (!STATES) load_rows<T, V>(Q, lda, j.q, p, c, a, u, n, rev);
        load_rows<T, V>(K, lda, j.k, p, c, a, u, n, rev);
        load_rows<T, V>(Vs, ldb, j.v, p, c, b, u, n, rev);
        __syncthreads();
        if (!STATES) {
            // steps against steps: rows ti + 16 m, columns tj + 16 n of a thread
            const int ti = tid / 16, tj = tid % 16;
            float s[4][4] = {};
            for (int x = 0; x < a4; ++x) {
                float4 q[4], k[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    q[m] = *(const float4*)(Q + (ti + 16 * m) * lda + 4 * x);
                    k[m] = *(const float4*)(K + (tj + 16 * m) * lda + 4 * x);
                }
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int o = 0; o < 4; ++o)
                        s[m][o] = fmaf(q[m].w, k[o].w, fmaf(q[m].z, k[o].z, fmaf(q[m].y, k[o].y, fmaf(q[m].x, k[o].x, s[m][o]))));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    const int near = ti + 16 * m - (tj + 16 * o);
                    P[(ti + 16 * m) * kLdP + tj + 16 * o] = near >= 0 ? s[m][o] * (j.sP * W[near]) : 0.f;
                }
            __syncthreads();
            T* out = (T*)j.out.p + c.d * j.out.dir + c.h * j.out.head;
            for (int i = tid; i < 16 * b4; i += kThreads) {
                const int r = i / b4, g = (i - r * b4) * 4;
                float4 o[4] = {};
                for (int x = 0; x < a4; ++x) {
                    float4 y[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) y[m] = *(const float4*)(Y + (4 * x + m) * ldb + g);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float4 q = *(const float4*)(Q + (r + 16 * m) * lda + 4 * x);
                        fma4(o[m], q.x, y[0]); fma4(o[m], q.y, y[1]); fma4(o[m], q.z, y[2]); fma4(o[m], q.w, y[3]);
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float f = j.sI * W[r + 16 * m];
                    o[m] = make_float4(o[m].x * f, o[m].y * f, o[m].z * f, o[m].w * f);
                }
                for (int x = 0; x < kSteps / 4; ++x) {
                    float4 v[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) v[m] = *(const float4*)(Vs + (4 * x + m) * ldb + g);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float4 q = *(const float4*)(P + (r + 16 * m) * kLdP + 4 * x);
                        fma4(o[m], q.x, v[0]); fma4(o[m], q.y, v[1]); fma4(o[m], q.z, v[2]); fma4(o[m], q.w, v[3]);
                    }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s1 = r + 16 * m;
                    if (s1 >= n) continue;
                    const int t = rev ? c.len - 1 - (u + s1) : u + s1;
                    T* at = out + (int64_t)(__ldg(p.off + t) + c.slot) * j.out.row + g;
                    if constexpr (V == 4 && sizeof(T) == 4) {
                        *(float4*)at = o[m];
                    } else {
                        const float v[4] = {o[m].x, o[m].y, o[m].z, o[m].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (g + e < b) at[e] = narrow<T>(v[e]);
                    }
                }
            }
            if (final && !j.fin) return;
        }
        // the state: keys weighted by what is left of the chunk behind them
        const int less = final ? j.early : 0;
        for (int i = tid; i < n * a4; i += kThreads) {
            const int s = i / a4, g = (i - s * a4) * 4;
            const float w = j.sK * W[n - less - s];
            float4* k = (float4*)(K + s * lda + g);
            const float4 q = *k;
            *k = make_float4(q.x * w, q.y * w, q.z * w, q.w * w);
        }
        __syncthreads();
        const float keep = W[n - less];
        for (int i = tid; i < a4 * b4; i += kThreads) {
            const int x = i / b4, g = (i - x * b4) * 4;
            float4 y[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                y[m] = *(const float4*)(Y + (4 * x + m) * ldb + g);
                y[m] = make_float4(y[m].x * keep, y[m].y * keep, y[m].z * keep, y[m].w * keep);
            }
            for (int s = 0; s < n; ++s) {
                const float4 k = *(const float4*)(K + s * lda + 4 * x), v = *(const float4*)(Vs + s * ldb + g);
                fma4(y[0], k.x, v); fma4(y[1], k.y, v); fma4(y[2], k.z, v); fma4(y[3], k.w, v);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) *(float4*)(Y + (4 * x + m) * ldb + g) = y[m];
        }
        __syncthreads();
    }
    float* const to = STATES ? la_start(p, j, c) : c.last && j.fin ? j.fin + state : nullptr;
    if (to)
        for (int i = tid; i < a * b; i += kThreads) to[i] = Y[i / b * ldb + i % b];
}

template <typename T, int V>
lstm_status launch(const LaArgs& a, bool states, cudaStream_t cs)
{
    size_t need = 0;
    for (int k = 0; k < a.jobs; ++k) {
        const size_t n = shared_bytes(a.job[k].a, a.job[k].b, states);
        need = n > need ? n : need;
    }
    const unsigned grid = (unsigned)((int64_t)a.count * a.ndir * a.heads * a.jobs);
    auto kernel = states ? la_general_kernel<T, V, true> : la_general_kernel<T, V, false>;
    LSTM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)need));
    kernel<<<grid, kThreads, need, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

}  // namespace

lstm_status launch_la_general(const LaArgs& a, bool bf16, bool states, cudaStream_t cs)
{
    bool whole = true;          // groups of four values line up everywhere
    const int e = bf16 ? 2 : 4;
    for (int k = 0; k < a.jobs; ++k) {
        const LaJob& j = a.job[k];
        whole = whole && j.a % 4 == 0 && j.b % 4 == 0;
        for (const LaRows* r : {&j.q, &j.k, &j.v, &j.out})
            whole = whole && (uintptr_t)r->p % (4 * e) == 0 && r->row % 4 == 0 && (a.ndir == 1 || r->dir % 4 == 0) && (a.heads == 1 || r->head % 4 == 0);
    }
    if (bf16) return whole ? launch<__nv_bfloat16, 4>(a, states, cs) : launch<__nv_bfloat16, 1>(a, states, cs);
    return whole ? launch<float, 4>(a, states, cs) : launch<float, 1>(a, states, cs);
}

}  // namespace lstm
