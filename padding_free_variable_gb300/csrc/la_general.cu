// la_general.cu -- linear attention on CUDA cores: fp32, and bf16 rows that la_tensor.cuh's loads cannot take.
//
// A CTA walks one head of one sequence (or a piece of it) 64 steps at a time, everything in shared memory in fp32: the
// products of the chunk's steps with each other (64 x 64, steps that no row sees left out), the outputs from them and from the
// state, then the state.  Per step that is 4 a b operations for the state and some 80 (a + b) between steps.  Bound by shared
// memory (three quarters of its wavefronts) and fp32 instructions: 29008 steps of 8 heads of 32 + 64 values, cut into pieces,
// 226 us, the three gradients 579 us; with registers for two CTAs an SM in place of three 241 and 611.  37 sequences of up to
// 700 steps of 2 x 3 heads of 37 + 53 values 123 us: the longest one's chunks.  Three tf32 products on mma.sync in place of
// each fp32 product took a tenth longer and six times the rounding error (tensor cores cut off sums).
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
    return sizeof(float) * ((size_t)kSteps * (2 * ld_of(a) + ld_of(b)) + (states ? 0 : kSteps * kLdP) + (size_t)a4 * ld_of(b) + 3 * kSteps + 4);
}

// `n` rows of `w` values into shared memory, zeros behind them and behind the width's last value.  rows: of the chunk's
// steps; log: of the threads of a row.
template <typename T, int V>
__device__ __forceinline__ void load_rows(float* dst, int ld, int log, const LaRows& r, const LaPart& c, const int* rows, int w, int n)
{
    const T* const base = (const T*)r.p + c.d * r.dir + c.h * r.head;
    const int g = (threadIdx.x & ((1 << log) - 1)) * 4;
    if (g >= w) return;
#pragma unroll 4
    for (int s = threadIdx.x >> log; s < kSteps; s += kThreads >> log) {
        const bool on = s < n;
        const T* const at = on ? base + rows[s] * r.row + g : base;
        float* const to = dst + s * ld + g;
        if constexpr (sizeof(T) == 4) {
            // asynchronous copies: the rows of all three operands are on their way together
#pragma unroll
            for (int e = 0; e < 4; e += V) {
                const int bytes = on && g + e < w ? 4 * V : 0;
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(to + e);
                if constexpr (V == 4) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(at), "r"(bytes) : "memory");
                else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(bytes ? at + e : at), "r"(bytes) : "memory");
            }
        } else {
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && V == 4) {
                const uint2 x = __ldg((const uint2*)at);
                q = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                                __uint_as_float(x.y & 0xffff0000u));
            } else if (on) {
                q.x = to_f32(at[0]);
                if (g + 1 < w) q.y = to_f32(at[1]);
                if (g + 2 < w) q.z = to_f32(at[2]);
                if (g + 3 < w) q.w = to_f32(at[3]);
            }
            *(float4*)to = q;
        }
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
__global__ void __launch_bounds__(kThreads, 3) la_general_kernel(const LaArgs p)
{
    extern __shared__ __align__(16) float sm[];
    const LaPart c = la_part(p, blockIdx.x);
    const LaJob& j = p.job[c.job];
    if (STATES && c.last) return;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, a = j.a, b = j.b, a4 = (a + 3) / 4, b4 = (b + 3) / 4, lda = ld_of(a), ldb = ld_of(b);
    float* const Q = sm;
    float* const K = Q + kSteps * lda;
    float* const W = K + kSteps * lda;
    int* rows = (int*)(W + kSteps + 4);         // [2][kSteps]: of this chunk's steps and the next one's
    float* const Vs = W + 3 * kSteps + 4;
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
    // the row of a chunk's step (the last one's where there is none)
    auto row_of = [&](int u) {
        const int s = min(u + tid, c.end - 1), t = rev ? c.len - 1 - s : s;
        return __ldg(p.off + t) + c.slot;
    };
    int ahead = 0, loga = 0, logb = 0;
    while (1 << loga < a4) ++loga;
    while (1 << logb < b4) ++logb;
    if (tid < kSteps) rows[tid] = row_of(c.begin);
    __syncthreads();
    {
        const float first = j.early && !j.starts ? W[1] : 1.f;
        const bool flip = j.starts ? j.flip_starts : j.flip;
        const float* from = STATES ? nullptr : j.starts ? la_start(p, j, c) : j.init ? j.init + state : nullptr;
        for (int x = warp; x < 4 * a4; x += kThreads / 32)
            for (int y = lane; y < 4 * b4; y += 32) {
                float v = 0.f;
                if (from && x < a && y < b) v = first * from[flip ? y * a + x : x * b + y];
                Y[x * ldb + y] = v;
            }
    }
    // a warp's places of Y, 4 x 4 values each: nx of a column, ng of a row, `share` threads each
    int share = 1, nx = 8, ng = 4;
    while (share < 8) {
        const int x = nx > ng ? nx / 2 : nx, y = nx > ng ? ng : ng / 2;
        if ((a4 + x - 1) / x * ((b4 + y - 1) / y) > kThreads / 32) break;
        share *= 2;
        nx = x;
        ng = y;
    }
    for (int u = c.begin; u < c.end; u += kSteps) {
        const int n = min(kSteps, c.end - u);
        const bool final = c.last && u + kSteps >= c.end;
        load_rows<T, V>(K, lda, loga, j.k, c, rows, a, n);
        if (!STATES) load_rows<T, V>(Q, lda, loga, j.q, c, rows, a, n);
        load_rows<T, V>(Vs, ldb, logb, j.v, c, rows, b, n);
        if (tid < kSteps && u + kSteps < c.end) ahead = row_of(u + kSteps);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        if (!STATES) {
            // steps against steps: rows ti + 16 m, columns tj + 16 n of a thread; a warp's lanes 8 x 4, so that either side's
            // rows come in one piece of 128 bytes or less
            const int ti = warp % 2 * 8 + lane / 4, tj = warp / 2 * 4 + lane % 4;
            float s[4][4] = {};
#pragma unroll 2
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
                    for (int o = 0; o <= m; ++o)        // what is later than all of its rows stays 0
                        s[m][o] = fmaf(q[m].w, k[o].w, fmaf(q[m].z, k[o].z, fmaf(q[m].y, k[o].y, fmaf(q[m].x, k[o].x, s[m][o]))));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int o = 0; o <= m; ++o) {
                    const int near = ti + 16 * m - (tj + 16 * o);
                    P[(ti + 16 * m) * kLdP + tj + 16 * o] = near >= 0 ? s[m][o] * (j.sP * W[near]) : 0.f;
                }
            __syncthreads();
            T* out = (T*)j.out.p + c.d * j.out.dir + c.h * j.out.head;
            const int r = ti;
            for (int g = 4 * tj; g < b; g += 64) {
                float4 o[4] = {};
#pragma unroll 2
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
#pragma unroll
                for (int first = 0; first < 4; ++first)     // rows of block m weigh the steps of blocks up to m
#pragma unroll 2
                    for (int x = 4 * first; x < 4 * first + 4; ++x) {
                        float4 v[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) v[m] = *(const float4*)(Vs + (4 * x + m) * ldb + g);
#pragma unroll
                        for (int m = first; m < 4; ++m) {
                            const float4 q = *(const float4*)(P + (r + 16 * m) * kLdP + 4 * x);
                            fma4(o[m], q.x, v[0]); fma4(o[m], q.y, v[1]); fma4(o[m], q.z, v[2]); fma4(o[m], q.w, v[3]);
                        }
                    }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int s1 = r + 16 * m;
                    if (s1 >= n) continue;
                    T* at = out + rows[s1] * j.out.row + g;
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
        rows = (int*)(W + kSteps + 4) + ((u - c.begin) / kSteps % 2 ? 0 : kSteps);
        if (tid < kSteps) rows[tid] = ahead;
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
        // few places: 2 to 8 threads next to each other share one, each a part of the steps
        const int each = (n + share - 1) / share, s0 = min(n, lane % share * each), s1 = min(n, s0 + each);
        const int wide = (b4 + ng - 1) / ng, blocks = (a4 + nx - 1) / nx * wide, at = lane / share;
        for (int i = warp; i < blocks; i += kThreads / 32) {
            const int x = i / wide * nx + at / ng, g = (i % wide * ng + at % ng) * 4;
            if (x >= a4 || g >= b) continue;
            float4 y[4] = {};
#pragma unroll 4
            for (int s = s0; s < s1; ++s) {
                const float4 k = *(const float4*)(K + s * lda + 4 * x), v = *(const float4*)(Vs + s * ldb + g);
                fma4(y[0], k.x, v); fma4(y[1], k.y, v); fma4(y[2], k.z, v); fma4(y[3], k.w, v);
            }
            for (int m = share / 2; m > 0; m /= 2) {
                const unsigned group = ((1u << share) - 1) << (lane & ~(share - 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e].x += __shfl_xor_sync(group, y[e].x, m); y[e].y += __shfl_xor_sync(group, y[e].y, m);
                    y[e].z += __shfl_xor_sync(group, y[e].z, m); y[e].w += __shfl_xor_sync(group, y[e].w, m);
                }
            }
            if (lane % share == 0) {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    float4* const at = (float4*)(Y + (4 * x + m) * ldb + g);
                    const float4 q = *at;
                    *at = make_float4(fmaf(q.x, keep, y[m].x), fmaf(q.y, keep, y[m].y), fmaf(q.z, keep, y[m].z), fmaf(q.w, keep, y[m].w));
                }
            }
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
    if (need > 48 * 1024) LSTM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)need));
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
            whole = whole && (uintptr_t)r->p % (4 * e) == 0 && (a.rows == 1 || r->row % 4 == 0) && (a.ndir == 1 || r->dir % 4 == 0) && (a.heads == 1 || r->head % 4 == 0);
    }
    if (bf16) return whole ? launch<__nv_bfloat16, 4>(a, states, cs) : launch<__nv_bfloat16, 1>(a, states, cs);
    return whole ? launch<float, 4>(a, states, cs) : launch<float, 1>(a, states, cs);
}

}  // namespace lstm
