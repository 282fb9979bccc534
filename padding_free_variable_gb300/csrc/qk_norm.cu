// qk_norm.cu -- norms of queries and keys for each head with the position rotation in the same pass, forward and backward.
//
// A head lies on 1 to 32 lanes, four pairs of values each: the pairs that are rotated together, so that a rotation needs
// no other lane, and a norm a few shuffles.  A warp takes a row (or, where rows are few, a part of one) and walks its
// heads 32 / lanes at a time, several loads ahead: sines and cosines are found once a row and pair and shared by the warp.
// Every value is read once and written once; bound by instructions and latency short of memory: 40555 rows of 32 heads of
// 64 bf16 values, half of each rotated, 79 us forward (62 % of the copy rate) and 147 us backward (50 %); 9564 rows of 7 heads of 74
// fp32 values, read one by one, 27 and 33 us.  Four lanes' sines each lane for itself, and selects between the layouts, took 125
// and 194 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "scan_plan.cuh"

namespace lstm {

namespace {

// kMaxParts: the CTAs of the backward pass, three an SM, as many as its registers let the GPU hold; four an SM in two rounds 201 us
// instead of 151.  A constant, so that the order of the weights' sums depends on the rows alone.
constexpr int kWarps = 8, kMaxParts = 456, kMaxHead = 256;

struct QkArgs {
    // 0: queries, 1: keys
    const void* x[2] = {};
    const void* dy[2] = {};
    void* out[2] = {};
    int64_t xr[2] = {}, xh[2] = {}, yr[2] = {}, yh[2] = {}, our[2] = {}, oh[2] = {};
    int heads[2] = {};
    const float* w[2] = {};
    const int64_t* turns = nullptr;
    const int32_t* positions = nullptr;
    int64_t first = 0, rows = 0;
    const int32_t* off = nullptr;       // of the plan, NULL without one
    const int32_t* len = nullptr;
    int T = 0, B = 0, padded = 0;
    int d = 0, rotary = 0, half = 0, kind = 0, lanes = 0, split = 1;
    float eps = 0.f, turn_scale = 1.f;
    float* part = nullptr;              // [parts][2][d]
    float* dw[2] = {};
    int parts = 0;
};

// The step of a packed row: the last one whose rows start at or before it.  32 candidates a round.
__device__ __forceinline__ int step_of(const QkArgs& p, int64_t row, int lane)
{
    int lo = 0, hi = p.T;               // off[lo] <= row < off[hi]
    while (hi - lo > 1) {
        const int by = (hi - lo + 31) / 32, at = lo + lane * by;
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && __ldg(p.off + at) <= row);
        const int k = 31 - __clz(below);                // lane 0 is below always
        const int next = lo + (k + 1) * by;
        lo += k * by;
        hi = min(hi, next);
    }
    return lo;
}

template <typename T> struct Four;
template <> struct Four<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *(const float4*)p; }
    __device__ __forceinline__ void store(float* p) const { *(float4*)p = v; }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
    __device__ __forceinline__ void set(const float (&f)[4]) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <> struct Four<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *(const uint2*)p; }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *(uint2*)p = v; }
    __device__ __forceinline__ void get(float (&f)[4]) const
    {
        f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float (&f)[4])
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        v = make_uint2(*(const unsigned*)&a, *(const unsigned*)&b);
    }
};

template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Where a lane's four pairs lie.  VEC: pairs 4 l to 4 l + 3, in two groups of four neighbours: with HALF the pairs' first and
// second values (what is not rotated has no pairs), else two pairs each.  Otherwise every value has a column of its own, and
// pairs next to each other belong to lanes next to each other, so that a warp's single values share their sectors.
template <bool VEC, bool HALF> struct Lane {
    int pair, by, d, turned;            // first pair, distance to the next; turned: pairs of halves, `turned` apart
    int at[VEC ? 1 : 8];                // each value's column, -1: none
    bool on;
    __device__ __forceinline__ void set(const QkArgs& p, int l)
    {
        pair = VEC ? 4 * l : l;
        by = VEC ? 1 : p.lanes;
        d = p.d;
        turned = HALF ? p.rotary / 2 : 0;
        on = 2 * pair < d;
        if (!VEC) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = pair_of(e / 2), c = HALF && k < turned ? k + e % 2 * turned : 2 * k + e % 2;
                at[VEC ? 0 : e] = c < d ? c : -1;
            }
        }
    }
    __device__ __forceinline__ int pair_of(int e) const { return pair + e * by; }
    __device__ __forceinline__ int col(int e, int which) const
    {
        if (!VEC) return at[VEC ? 0 : 2 * e + which];
        return HALF ? group(which) + e : 2 * (pair + e) + which;
    }
    __device__ __forceinline__ bool has(int e, int which) const { return VEC ? on : col(e, which) >= 0; }
    __device__ __forceinline__ int group(int which) const { return HALF && pair < turned ? pair + which * turned : 2 * pair + 4 * which; }
};

// A lane's values of one head as they were read: first[4] and second[4] of its pairs.
template <typename T, bool VEC> struct Pairs;
template <typename T> struct Pairs<T, true> {
    Four<T> a, b;
    __device__ __forceinline__ void zero() { const float z[4] = {}; a.set(z); b.set(z); }
    template <bool HALF> __device__ __forceinline__ void load(const T* p, const Lane<true, HALF>& w) { a.load(p + w.group(0)); b.load(p + w.group(1)); }
    template <bool HALF> __device__ __forceinline__ void get(float (&f)[4], float (&s)[4], const Lane<true, HALF>&) const
    {
        float x[4], y[4];
        a.get(x);
        b.get(y);
        if (HALF) {
#pragma unroll
            for (int e = 0; e < 4; ++e) { f[e] = x[e]; s[e] = y[e]; }
        } else {
            f[0] = x[0]; s[0] = x[1]; f[1] = x[2]; s[1] = x[3];
            f[2] = y[0]; s[2] = y[1]; f[3] = y[2]; s[3] = y[3];
        }
    }
    template <bool HALF> __device__ __forceinline__ static void put(T* p, const float (&f)[4], const float (&s)[4], const Lane<true, HALF>& w)
    {
        Four<T> a, b;
        if (HALF) {
            a.set(f);
            b.set(s);
        } else {
            const float x[4] = {f[0], s[0], f[1], s[1]}, y[4] = {f[2], s[2], f[3], s[3]};
            a.set(x);
            b.set(y);
        }
        a.store(p + w.group(0));
        b.store(p + w.group(1));
    }
};
template <typename T> struct Pairs<T, false> {
    float f[4], s[4];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = s[e] = 0.f;
    }
    template <typename L> __device__ __forceinline__ void load(const T* p, const L& w)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = w.has(e, 0) ? to_f32(p[w.col(e, 0)]) : 0.f;
            s[e] = w.has(e, 1) ? to_f32(p[w.col(e, 1)]) : 0.f;
        }
    }
    template <typename L> __device__ __forceinline__ void get(float (&a)[4], float (&b)[4], const L&) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) { a[e] = f[e]; b[e] = s[e]; }
    }
    template <typename L> __device__ __forceinline__ static void put(T* p, const float (&f)[4], const float (&s)[4], const L& w)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (w.has(e, 0)) p[w.col(e, 0)] = narrow<T>(f[e]);
            if (w.has(e, 1)) p[w.col(e, 1)] = narrow<T>(s[e]);
        }
    }
};

// Sum over a head's lanes, in all of them.
__device__ __forceinline__ float head_sum(float v, int lanes)
{
    for (int m = lanes / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Two values at once: one instruction of the fp32 pipe.
struct Two {
    unsigned long long v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ float sum() const { float a, b; asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); return a + b; }
    __device__ __forceinline__ void get(float* p) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(p[0]), "=f"(p[1]) : "l"(v)); }
};
__device__ __forceinline__ Two operator*(Two a, Two b) { Two r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ Two operator+(Two a, Two b) { Two r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v)); return r; }
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) { Two r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v)); return r; }
__device__ __forceinline__ Two both(float a) { return Two(a, a); }

// Four values.
struct Quad {
    Two a, b;
    __device__ __forceinline__ void set(const float (&f)[4]) { a = Two(f[0], f[1]); b = Two(f[2], f[3]); }
    __device__ __forceinline__ void get(float (&f)[4]) const { a.get(f); b.get(f + 2); }
};
__device__ __forceinline__ Quad operator*(Quad x, Quad y) { return {x.a * y.a, x.b * y.b}; }
__device__ __forceinline__ Quad operator*(Quad x, Two y) { return {x.a * y, x.b * y}; }
__device__ __forceinline__ Quad operator+(Quad x, Two y) { return {x.a + y, x.b + y}; }
__device__ __forceinline__ Quad fma2(Quad x, Quad y, Quad z) { return {fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ Quad fma2(Quad x, Two y, Quad z) { return {fma2(x.a, y, z.a), fma2(x.b, y, z.b)}; }
// x . x2 + y . y2
__device__ __forceinline__ float dot(Quad x, Quad x2, Quad y, Quad y2)
{
    const Quad s = fma2(x, x2, y * y2);
    return (s.a + s.b).sum();
}
__device__ __forceinline__ float total(Quad x, Quad y) { return ((x.a + y.a) + (x.b + y.b)).sum(); }

template <typename T, bool VEC, bool BACK, bool HALF>
__global__ void __launch_bounds__(kWarps * 32, 3) qk_norm_kernel(const QkArgs p)
{
    constexpr int AHEAD = BACK ? 1 : 4;                 // heads of a lane on their way at a time
    __shared__ float turns[kWarps][2][kMaxHead / 2];    // cosines and sines of the warp's row
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % p.lanes, sub = lane / p.lanes, at_once = 32 / p.lanes;
    Lane<VEC, HALF> w;
    w.set(p, l);
    Quad gf[2], gs[2];
    for (int k = 0; k < 2; ++k) gf[k].a = gf[k].b = gs[k].a = gs[k].b = Two(0.f, 0.f);
    const int passes0 = (p.heads[0] + at_once - 1) / at_once;
    const float per = 1.f / p.d;
    const int64_t units = p.rows * p.split;
    for (int64_t unit = blockIdx.x * (int64_t)kWarps + warp; unit < units; unit += (int64_t)gridDim.x * kWarps) {
        const int64_t row = p.split == 1 ? unit : unit / p.split;
        const int begin = p.split == 1 ? 0 : (int)(unit - row * p.split);
        bool live = true;
        int step = 0;
        if (p.off) {
            if (p.padded) {
                step = (int)(row / p.B);
                live = step < __ldg(p.len + (int)(row - (int64_t)step * p.B));
            } else if (!p.positions && p.rotary) {
                step = step_of(p, row, lane);
            }
        }
        float co[4] = {1.f, 1.f, 1.f, 1.f}, si[4] = {};
        if (p.rotary) {
            // a lane each pair, then every lane its own four; position * frequency modulo a turn, in half turns from -1 to 1
            const int64_t at = p.positions ? (int64_t)__ldg(p.positions + row) : p.first + step;
            __syncwarp();
            for (int i = lane; i < p.rotary / 2; i += 32) {
                const unsigned long long a = (unsigned long long)at * (unsigned long long)__ldg((const long long*)p.turns + i);
                float s, c;
                sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);
                turns[warp][0][i] = c * p.turn_scale;
                turns[warp][1][i] = s * p.turn_scale;
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (w.pair_of(e) < p.rotary / 2) {
                    co[e] = turns[warp][0][w.pair_of(e)];
                    si[e] = turns[warp][1][w.pair_of(e)];
                }
        }
        // the heads of one operand, `at_once` a pass; of a row's passes this warp takes every split-th
        auto heads = [&](auto which) {
            constexpr int k = decltype(which)::value;
            const int count = p.heads[k];
            int h = (k == 0 ? begin : (begin + passes0 * (p.split - 1)) % p.split) * at_once + sub;
            const int by = at_once * p.split;
            const T* x0 = (const T*)p.x[k] + row * p.xr[k] + h * p.xh[k];
            const T* y0 = BACK ? (const T*)p.dy[k] + row * p.yr[k] + h * p.yh[k] : nullptr;
            T* o0 = (T*)p.out[k] + row * p.our[k] + h * p.oh[k];
            const int64_t xs = by * p.xh[k], ys = by * p.yh[k], os = by * p.oh[k];
            // the weights, from L1 once a row: registers are what keeps warps off the SM
            float wf[4], ws[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                wf[e] = w.has(e, 0) ? p.w[k] ? __ldg(p.w[k] + w.col(e, 0)) : 1.f : 0.f;
                ws[e] = w.has(e, 1) ? p.w[k] ? __ldg(p.w[k] + w.col(e, 1)) : 1.f : 0.f;
            }
            // a rotated and weighted pair: first A + second B, first C + second D; backwards the weights come later
            Quad A, B, C, D, wq, wr;
            wq.set(wf);
            wr.set(ws);
            {
                const float ni[4] = {-si[0], -si[1], -si[2], -si[3]};
                A.set(co);
                C.set(si);
                D = A;
                B.set(ni);
                if (!BACK) { A = wq * A; C = wq * C; B = wr * B; D = wr * D; }
            }
            for (; h - sub < count; h += AHEAD * by) {
                Pairs<T, VEC> x[AHEAD], y[BACK ? AHEAD : 1];
#pragma unroll
                for (int n = 0; n < AHEAD; ++n) {
                    x[n].zero();
                    if (BACK) y[BACK ? n : 0].zero();
                    if (h + n * by < count && w.on && live) {
                        x[n].load(x0, w);
                        if (BACK) y[BACK ? n : 0].load(y0, w);
                    }
                    x0 += xs;
                    if (BACK) y0 += ys;
                }
#pragma unroll
                for (int n = 0; n < AHEAD; ++n) {
                    if (h - sub + n * by >= count) break;
                    float f[4], s[4], r = 1.f;
                    x[n].get(f, s, w);
                    if (p.kind == LSTM_NORM_LAYER) {
                        const float mean = head_sum(((f[0] + s[0]) + (f[1] + s[1])) + ((f[2] + s[2]) + (f[3] + s[3])), p.lanes) * per;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[e] = w.has(e, 0) ? f[e] - mean : 0.f;
                            s[e] = w.has(e, 1) ? s[e] - mean : 0.f;
                        }
                    }
                    Quad u, v;
                    u.set(f);
                    v.set(s);
                    if (p.kind != LSTM_NORM_NONE) r = rsqrtf(head_sum(dot(u, u, v, v), p.lanes) * per + p.eps);
                    if (!BACK) {
                        const Quad first = fma2(u, A, v * B), second = fma2(u, C, v * D);
                        u = first * both(r);
                        v = second * both(r);
                    } else {
                        // the error before the rotation, the weights' gradients, the weighted error through the norm
                        float df[4], ds[4];
                        y[BACK ? n : 0].get(df, ds, w);
                        Quad g, q;
                        g.set(df);
                        q.set(ds);
                        const Quad a = fma2(g, A, q * C), b = fma2(q, D, g * B);
                        u = u * both(r);
                        v = v * both(r);
                        gf[k] = fma2(a, u, gf[k]);
                        gs[k] = fma2(b, v, gs[k]);
                        g = a * wq;
                        q = b * wr;
                        if (p.kind != LSTM_NORM_NONE) {
                            const float along = head_sum(dot(g, u, q, v), p.lanes) * per;
                            const float mean = p.kind == LSTM_NORM_LAYER ? head_sum(total(g, q), p.lanes) * per : 0.f;
                            g = fma2(u, both(-along), g) + both(-mean);
                            q = fma2(v, both(-along), q) + both(-mean);
                            u = g * both(r);
                            v = q * both(r);
                        } else {
                            u = g;
                            v = q;
                        }
                    }
                    u.get(f);
                    v.get(s);
                    if (h + n * by < count && w.on) Pairs<T, VEC>::put(o0, f, s, w);
                    o0 += os;
                }
            }
        };
        heads(std::integral_constant<int, 0>());
        if (p.heads[1] > 0) heads(std::integral_constant<int, 1>());
    }
    if (BACK && p.part) {
        // the block's sums: lanes of a warp, then its warps in order
        __shared__ float sum[kWarps][2][kMaxHead];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float mf[4], ms[4];
            gf[k].get(mf);
            gs[k].get(ms);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a = mf[e], b = ms[e];
                for (int m = 16; m >= p.lanes; m /= 2) {
                    a += __shfl_xor_sync(0xffffffffu, a, m);
                    b += __shfl_xor_sync(0xffffffffu, b, m);
                }
                if (sub == 0) {
                    if (w.has(e, 0)) sum[warp][k][w.col(e, 0)] = a;
                    if (w.has(e, 1)) sum[warp][k][w.col(e, 1)] = b;
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.d; i += blockDim.x) {
            const int k = i >= p.d, c = i - k * p.d;
            float s = 0.f;
            for (int m = 0; m < kWarps; ++m) s += sum[m][k][c];
            p.part[((int64_t)blockIdx.x * 2 + k) * p.d + c] = s;
        }
    }
}

// The blocks' sums of one column, a warp each: a lane's every 32nd block in order, then the lanes.
__global__ void __launch_bounds__(256) qk_norm_sums_kernel(const QkArgs p)
{
    const int i = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (i >= 2 * p.d) return;
    const int k = i >= p.d, c = i - k * p.d;
    if (!p.dw[k]) return;
    float s = 0.f;
    for (int m = lane; m < p.parts; m += 32) s += p.part[((int64_t)m * 2 + k) * p.d + c];
    s = head_sum(s, 32);
    if (lane == 0) p.dw[k][c] = s;
}

int blocks_of(int64_t rows) { return (int)std::min<int64_t>((rows + kWarps - 1) / kWarps, kMaxParts); }

template <typename T, bool VEC, bool HALF>
lstm_status launch_layout(QkArgs p, bool back, cudaStream_t cs)
{
    if (!back) {
        // a warp a row; where that leaves warps without one, a row's heads are spread over several
        const int at_once = 32 / p.lanes, passes = ceil_div(p.heads[0], at_once) + ceil_div(p.heads[1], at_once);
        while (p.split < passes && p.rows * p.split < 152 * kWarps) p.split *= 2;
        if (p.split > passes) p.split = passes;
        const int64_t blocks = std::min<int64_t>((p.rows * p.split + kWarps - 1) / kWarps, 152 * 3);
        qk_norm_kernel<T, VEC, false, HALF><<<(unsigned)blocks, kWarps * 32, 0, cs>>>(p);
    } else {
        p.parts = blocks_of(p.rows);
        qk_norm_kernel<T, VEC, true, HALF><<<p.parts, kWarps * 32, 0, cs>>>(p);
        if (p.part) qk_norm_sums_kernel<<<ceil_div(2 * p.d, 8), 256, 0, cs>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

template <typename T, bool VEC>
lstm_status launch(const QkArgs& p, bool back, cudaStream_t cs)
{
    return p.half ? launch_layout<T, VEC, true>(p, back, cs) : launch_layout<T, VEC, false>(p, back, cs);
}

// ---------------------------------------------------------------- checks

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

lstm_status check_shape(const lstm_qk_norm_shape* s)
{
    if (!s || s->q_heads < 1 || s->k_heads < 0 || s->head_size < 1) return LSTM_ERR_INVALID_ARG;
    if (s->kind < LSTM_NORM_NONE || s->kind > LSTM_NORM_LAYER || s->rotary_size < 0 || s->rotary_size % 2 || s->rotary_size > s->head_size)
        return LSTM_ERR_INVALID_ARG;
    if (s->layout != LSTM_ROTARY_HALF && s->layout != LSTM_ROTARY_INTERLEAVED) return LSTM_ERR_INVALID_ARG;
    if ((s->dtype != LSTM_F32 && s->dtype != LSTM_BF16) || !(s->eps > 0.f) || !std::isfinite(s->eps) || !std::isfinite(s->rotary_scale))
        return LSTM_ERR_INVALID_ARG;
    if (s->head_size > kMaxHead || s->q_heads > 4096 || s->k_heads > 4096) return LSTM_ERR_UNSUPPORTED;
    return LSTM_OK;
}

constexpr int64_t kMaxStride = 1ll << 40;

// Rows of one operand: there, aligned to their element, strides in range; written ones without two values at a place.
bool good(const void* p, int64_t row, int64_t head, int64_t rows, int heads, int d, size_t e, bool written)
{
    if (heads == 0) return p == nullptr;
    if (!p || !aligned(p, e) || row < 0 || head < 0 || row > kMaxStride || head > kMaxStride) return false;
    if (!written) return true;
    // the finer stride steps over a head, the other over all of the finer ones
    const bool head_in = heads > 1 && (rows <= 1 || head <= row);
    int64_t span = d;
    if (head_in) {
        if (head < span) return false;
        span += (heads - 1) * head;
        return rows <= 1 || row >= span;
    }
    if (rows > 1) {
        if (row < span) return false;
        span += (rows - 1) * row;
    }
    return heads <= 1 || head >= span;
}

template <typename R>
bool good_rows(const lstm_qk_norm_shape& s, const R& r, int64_t rows, bool written)
{
    const size_t e = s.dtype == LSTM_BF16 ? 2 : 4;
    return good(r.q, r.q_row_stride, r.q_head_stride, rows, s.q_heads, s.head_size, e, written) &&
           good(r.k, r.k_row_stride, r.k_head_stride, rows, s.k_heads, s.head_size, e, written);
}

// What both passes check and set.
lstm_status common(const lstm_plan* plan, const lstm_qk_norm_shape* shape, const lstm_qk_norm_params* params, const lstm_qk_rows* in,
                   int64_t rows, QkArgs* a)
{
    const lstm_status st = check_shape(shape);
    if (st != LSTM_OK) return st;
    const lstm_qk_norm_shape& s = *shape;
    if (!params || !in || rows < 0 || rows > INT32_MAX || (plan && plan->p.rows != rows)) return LSTM_ERR_INVALID_ARG;
    if (s.kind == LSTM_NORM_NONE && (params->w_q || params->w_k)) return LSTM_ERR_INVALID_ARG;
    if (s.k_heads == 0 && params->w_k) return LSTM_ERR_INVALID_ARG;
    if (!aligned(params->w_q, 4) || !aligned(params->w_k, 4) || !aligned(params->positions, 4) || !aligned(params->turns, 8))
        return LSTM_ERR_INVALID_ARG;
    if (s.rotary_size > 0 && (!params->turns || (!params->positions && !plan))) return LSTM_ERR_INVALID_ARG;
    if (plan) {
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess || dev != plan->p.device) return LSTM_ERR_INVALID_ARG;
        a->off = plan->p.d_off; a->len = plan->p.d_len; a->T = plan->p.T; a->B = plan->p.B; a->padded = plan->p.padded ? 1 : 0;
    }
    if (rows == 0) return LSTM_OK;
    if (!good_rows(s, *in, rows, false)) return LSTM_ERR_INVALID_ARG;
    a->x[0] = in->q; a->x[1] = in->k;
    a->xr[0] = in->q_row_stride; a->xr[1] = in->k_row_stride; a->xh[0] = in->q_head_stride; a->xh[1] = in->k_head_stride;
    a->heads[0] = s.q_heads; a->heads[1] = s.k_heads;
    a->w[0] = params->w_q; a->w[1] = params->w_k;
    a->turns = params->turns; a->positions = params->positions; a->first = params->first_position;
    a->rows = rows; a->d = s.head_size; a->rotary = s.rotary_size; a->half = s.layout == LSTM_ROTARY_HALF; a->kind = s.kind;
    a->eps = s.eps; a->turn_scale = s.rotary_scale;
    a->lanes = 1;
    while (a->lanes * 8 < s.head_size) a->lanes *= 2;
    return LSTM_OK;
}

void out_rows(const lstm_qk_out_rows& o, QkArgs* a)
{
    a->out[0] = o.q; a->out[1] = o.k;
    a->our[0] = o.q_row_stride; a->our[1] = o.k_row_stride; a->oh[0] = o.q_head_stride; a->oh[1] = o.k_head_stride;
}

lstm_status run(const QkArgs& a, int dtype, bool back, cudaStream_t cs)
{
    // four values at a time where every head of every operand starts on a multiple of four
    const int64_t e = dtype == LSTM_BF16 ? 2 : 4;
    bool vec = a.d % 8 == 0 && (!a.half || a.rotary % 8 == 0);
    for (int k = 0; k < 2; ++k) {
        if (a.heads[k] == 0) continue;
        for (const void* p : {a.x[k], (const void*)a.out[k], a.dy[k]}) vec = vec && aligned(p, 4 * e);
        vec = vec && a.xr[k] % 4 == 0 && a.xh[k] % 4 == 0 && a.our[k] % 4 == 0 && a.oh[k] % 4 == 0 && a.yr[k] % 4 == 0 && a.yh[k] % 4 == 0;
    }
    if (dtype == LSTM_BF16) return vec ? launch<__nv_bfloat16, true>(a, back, cs) : launch<__nv_bfloat16, false>(a, back, cs);
    return vec ? launch<float, true>(a, back, cs) : launch<float, false>(a, back, cs);
}

}  // namespace

}  // namespace lstm

using namespace lstm;

extern "C" {

lstm_status lstm_qk_norm_fwd(const lstm_plan* plan, const lstm_qk_norm_shape* shape, const lstm_qk_norm_params* params,
                             const lstm_qk_rows* in, int64_t rows, const lstm_qk_out_rows* out, void* stream)
{
    QkArgs a;
    const lstm_status st = common(plan, shape, params, in, rows, &a);
    if (st != LSTM_OK) return st;
    if (!out) return LSTM_ERR_INVALID_ARG;
    if (rows == 0) return LSTM_OK;
    if (!good_rows(*shape, *out, rows, true)) return LSTM_ERR_INVALID_ARG;
    out_rows(*out, &a);
    return run(a, shape->dtype, false, (cudaStream_t)stream);
}

size_t lstm_qk_norm_scratch_bytes(const lstm_qk_norm_shape* shape, int64_t rows)
{
    if (check_shape(shape) != LSTM_OK || rows < 0 || rows > INT32_MAX) return 0;
    return std::max<size_t>(16, sizeof(float) * 2 * shape->head_size * blocks_of(rows));
}

lstm_status lstm_qk_norm_bwd(const lstm_plan* plan, const lstm_qk_norm_shape* shape, const lstm_qk_norm_params* params,
                             const lstm_qk_rows* in, int64_t rows, const lstm_qk_rows* dout, const lstm_qk_out_rows* din,
                             const lstm_qk_norm_grads* grads, void* scratch, void* stream)
{
    QkArgs a;
    const lstm_status st = common(plan, shape, params, in, rows, &a);
    if (st != LSTM_OK) return st;
    if (!dout || !din || !grads || !aligned(grads->w_q, 4) || !aligned(grads->w_k, 4) || !aligned(scratch, 16)) return LSTM_ERR_INVALID_ARG;
    if (shape->kind == LSTM_NORM_NONE && (grads->w_q || grads->w_k)) return LSTM_ERR_INVALID_ARG;
    if (shape->k_heads == 0 && grads->w_k) return LSTM_ERR_INVALID_ARG;
    const bool sums = grads->w_q || grads->w_k;
    cudaStream_t cs = (cudaStream_t)stream;
    if (rows == 0) {
        for (float* g : {grads->w_q, grads->w_k})
            if (g) LSTM_CUDA_TRY(cudaMemsetAsync(g, 0, sizeof(float) * shape->head_size, cs));
        return LSTM_OK;
    }
    if (!good_rows(*shape, *dout, rows, false) || !good_rows(*shape, *din, rows, true) || (sums && !scratch)) return LSTM_ERR_INVALID_ARG;
    a.dy[0] = dout->q; a.dy[1] = dout->k;
    a.yr[0] = dout->q_row_stride; a.yr[1] = dout->k_row_stride; a.yh[0] = dout->q_head_stride; a.yh[1] = dout->k_head_stride;
    out_rows(*din, &a);
    a.part = sums ? (float*)scratch : nullptr;
    a.dw[0] = grads->w_q; a.dw[1] = grads->w_k;
    return run(a, shape->dtype, true, cs);
}

}  // extern "C"
