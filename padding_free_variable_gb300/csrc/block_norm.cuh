// block_norm.cuh -- arguments of the block norms' kernels and the row access they share.
#pragma once

#include <type_traits>

#include "glr.cuh"

namespace lstm {

constexpr int kSums = 5;            // w_post, b_post, scale, w_pre, b_pre

struct NormArgs {
    int D = 0;
    int post = 0, pre = 0, gate = 0;
    bool branch16 = false, stream16 = false, norm16 = false;
    float eps = 0.f;
    int64_t rows = 0;
    lstm_block_norm_params w = {};
    const void* x = nullptr;
    const void* y = nullptr;
    const void* g = nullptr;
    int64_t ldy = 0, ldg = 0;
    void* x_out = nullptr;
    void* n = nullptr;
    float* stats = nullptr;         // [rows][4]: mean and 1/deviation, post then pre
    // backward
    const void* dx_out = nullptr;
    const void* dn = nullptr;
    void* dx = nullptr;
    void* dy = nullptr;
    void* dg = nullptr;
    int64_t lddy = 0, lddg = 0;
    float* part = nullptr;          // [parts][kSums][D]
    float* sums[kSums] = {};
    int parts = 0;
};


// Values of a thread: PER groups of VEC neighbours, the threads of a row next to each other in each
// group.  Rows of a width that no multiple of 8 divides start anywhere in memory: then a group is
// 8 values from a multiple of 8 in memory, `shift` before the columns that a row on such a boundary
// would give it, and its first and last group of a row reach into the neighbours.
template <int VEC, int PER> struct Cols {
    int t, n, D;            // thread of the row, threads of a row, width
    int shift = 0;
    bool row = true;        // is there a row at all?
    __device__ __forceinline__ int at(int k) const { return (k * n + t) * VEC - shift; }
    __device__ __forceinline__ bool has(int k) const { return row && at(k) < D; }
    __device__ __forceinline__ bool whole(int k) const { return at(k) >= 0 && at(k) + VEC <= D; }
    __device__ __forceinline__ bool valid(int k, int v) const { return (unsigned)(at(k) + v) < (unsigned)D; }
};

// VEC values of one group as they lie in memory.
template <typename T, int VEC> struct Group {
    static constexpr int N = VEC * (int)sizeof(T) / 16 > 0 ? VEC * (int)sizeof(T) / 16 : 1;
    uint4 w[VEC == 1 ? 1 : N];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 2) w[0].x = __ldg((const unsigned short*)p);
            else w[0].x = __ldg((const unsigned*)p);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __ldg((const uint4*)p + i);
        }
    }
    // x and dx' may be overwritten in place by the thread that reads them: no read-only path
    __device__ __forceinline__ void load_own(const T* p)
    {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 2) w[0].x = *(const unsigned short*)p;
            else w[0].x = *(const unsigned*)p;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = ((const uint4*)p)[i];
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (VEC == 1 ? 1 : N); ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ unsigned word(int i) const
    {
        const uint4 q = w[i / 4];
        return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
    }
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(word(v));
        else return __uint_as_float(v % 2 ? word(v / 2) & 0xffff0000u : word(v / 2) << 16);
    }
};

// The same with the type known at run time, for the kernels that are not worth a copy for each type.
struct Any {};
template <int VEC> struct Group<Any, VEC> {
    static constexpr int N = VEC == 1 ? 1 : VEC / 4;
    uint4 w[N];
    __device__ __forceinline__ void load_any(const void* base, int64_t at, bool b16, bool own)
    {
        if constexpr (VEC == 1) {
            if (b16) w[0].x = own ? ((const unsigned short*)base)[at] : __ldg((const unsigned short*)base + at);
            else w[0].x = own ? ((const unsigned*)base)[at] : __ldg((const unsigned*)base + at);
        } else {
            const uint4* p = (const uint4*)((const char*)base + at * (b16 ? 2 : 4));
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i < (b16 ? N / 2 : N)) w[i] = own ? p[i] : __ldg(p + i);
        }
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ unsigned word(int i) const
    {
        const uint4 q = w[i / 4];
        return i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
    }
    __device__ __forceinline__ float get(int v, bool b16) const
    {
        return __uint_as_float(!b16 ? word(v) : v % 2 ? word(v / 2) & 0xffff0000u : word(v / 2) << 16);
    }
};

template <typename T, int VEC>
__device__ __forceinline__ void load_group(Group<T, VEC>& g, const void* base, int64_t at, bool b16, bool own = false)
{
    if constexpr (std::is_same<T, Any>::value) g.load_any(base, at, b16, own);
    else if (own) g.load_own((const T*)base + at);
    else g.load((const T*)base + at);
}
// A group of shifted columns, the neighbours' values in it as 0 (whatever they are, NaN too, stays
// theirs).  `inside`: all of it lies in the tensor; else value by value.
template <typename T, int VEC, int PER>
__device__ __forceinline__ void load_shifted(Group<T, VEC>& g, const void* base, int64_t row, const Cols<VEC, PER>& c, int k, bool inside, bool own = false)
{
    if (inside) {
        load_group(g, base, row + c.at(k), sizeof(T) == 2, own);
        if (c.whole(k)) return;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            if (!c.valid(k, v)) ((unsigned*)g.w)[v * (int)sizeof(T) / 4] &= sizeof(T) == 4 ? 0u : v % 2 ? 0xffffu : 0xffff0000u;
        return;
    }
    const T* p = (const T*)base + row + c.at(k);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        unsigned x = 0;
        if (c.valid(k, v)) x = sizeof(T) == 2 ? (unsigned)*(const unsigned short*)(p + v) : *(const unsigned*)(p + v);
        unsigned& w = ((unsigned*)g.w)[v * (int)sizeof(T) / 4];
        w = sizeof(T) == 4 ? x : v % 2 ? w | x << 16 : x;
    }
}
template <typename T, int VEC> __device__ __forceinline__ float get_value(const Group<T, VEC>& g, int v, bool b16)
{
    if constexpr (std::is_same<T, Any>::value) return g.get(v, b16);
    else return g.get(v);
}

// Store VEC values as bf16 or fp32.
template <int VEC> __device__ __forceinline__ void put_group(void* base, int64_t at, bool b16, const float (&v)[VEC])
{
    if constexpr (VEC == 1) {
        if (b16) ((__nv_bfloat16*)base)[at] = __float2bfloat16_rn(v[0]);
        else ((float*)base)[at] = v[0];
    } else if (b16) {
        unsigned q[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
            q[i / 2] = *(const unsigned*)&h;
        }
        if constexpr (VEC == 8) *(uint4*)((__nv_bfloat16*)base + at) = make_uint4(q[0], q[1], q[2], q[3]);
        else *(uint2*)((__nv_bfloat16*)base + at) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *(float4*)((float*)base + at + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// The valid values of a shifted group, one by one at a row's ends.
template <typename T, int VEC, int PER>
__device__ __forceinline__ void put_shifted(T* base, int64_t row, const Cols<VEC, PER>& c, int k, const float (&x)[VEC])
{
    if (c.whole(k)) {
        put_group<VEC>(base, row + c.at(k), sizeof(T) == 2, x);
        return;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v)
        if (c.valid(k, v)) base[row + c.at(k) + v] = from_f32<T>(x[v]);
}

// A thread's own parameters in shared memory, four neighbours at a time, the threads' next to each
// other: for shifted columns, which no vector load of the parameters fits; 0 beyond a row's ends.
template <int VEC, int PER> struct OwnParams {
    float4* s;
    static constexpr int bytes(int count, int threads) { return count * PER * VEC * 4 * threads; }
    __device__ __forceinline__ float4* place(int which, int k, int n) const { return s + ((which * PER + k) * (VEC / 4) + n) * blockDim.x + threadIdx.x; }
    template <typename V> __device__ __forceinline__ void fill(int which, const Cols<VEC, PER>& c, V&& value) const
    {
#pragma unroll
        for (int k = 0; k < PER; ++k)
#pragma unroll
            for (int n = 0; n < VEC / 4; ++n) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = c.valid(k, n * 4 + i) ? value(c.at(k) + n * 4 + i) : 0.f;
                *place(which, k, n) = make_float4(x[0], x[1], x[2], x[3]);
            }
    }
    template <int Q> __device__ __forceinline__ void get(int which, int k, int n, float (&v)[Q]) const
    {
#pragma unroll
        for (int i = 0; i < Q; i += 4) {
            const float4 q = *place(which, k, n + i / 4);
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    }
};
// Rows that one thread takes one after another are a multiple of 8 apart, so that their columns are shifted alike.
inline int64_t shifted_blocks(int64_t blocks) { return (blocks + 7) / 8 * 8; }

// VEC parameters, or `none` where there are no such parameters.
// GIVEN: known to be there; EVER: such a kind has them at all.
template <int VEC, bool GIVEN = false, bool EVER = true>
__device__ __forceinline__ void get_params(const float* p, int at, float none, float (&v)[VEC])
{
    if (!EVER || (!GIVEN && !p)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = none;
    } else if constexpr (VEC == 1) {
        v[0] = __ldg(p + at);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 q = __ldg((const float4*)(p + at + i));
            v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
        }
    }
}

// Sums over the threads of a row: within a warp by shuffles, across the warps of a CTA (then one
// row a CTA) through shared memory, each use on the other half so that one barrier suffices.
struct RowSum {
    float* part;            // [2][16][4]
    int lanes, half;        // threads of a row: a power of two up to 32, or whole warps
    template <int N> __device__ __forceinline__ void operator()(float (&v)[N])
    {
        static_assert(N <= 4, "four sums at a time");
#pragma unroll
        for (int o = 16; o; o >>= 1)
            if (o < lanes)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lanes <= 32) return;
        const int warps = lanes / 32;
        float* s = part + half * 64;
        half ^= 1;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[threadIdx.x / 32 * 4 + i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = threadIdx.x % 32 < warps ? s[threadIdx.x % 32 * 4 + i] : 0.f;
#pragma unroll
        for (int o = 8; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
    __device__ __forceinline__ float operator()(float x)
    {
        float v[1] = {x};
        (*this)(v);
        return v[0];
    }
};

// act(q)
__device__ __forceinline__ float activation(int kind, float q)
{
    const float s = rcp_approx(1.f + ex2_approx(q * kNegLog2e));
    return kind == LSTM_GATE_SIGMOID ? s : kind == LSTM_GATE_SILU ? q * s : 1.f;
}

// A whole block: both norms of one kind with all that this kind has, types among those with kernels of their own.
bool norm_full(const NormArgs& a);
// Rows, pointers and widths allow groups of eight; the same for shifted ones (rows that all start
// equally far from a multiple of 8 values).
bool norm_whole(const NormArgs& a);
bool norm_shifted(const NormArgs& a);
// Threads of a row of `groups` groups: 4, 8, 16 or whole warps.
inline int row_threads(int groups) { return groups <= 4 ? 4 : groups <= 8 ? 8 : groups <= 16 ? 16 : (groups + 31) / 32 * 32; }
int norm_parts(int64_t rows, int D);
lstm_status launch_norm_fwd(const NormArgs& a, cudaStream_t cs);
lstm_status launch_norm_bwd(NormArgs a, cudaStream_t cs);

}  // namespace lstm
