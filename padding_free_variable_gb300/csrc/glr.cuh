// glr.cuh -- arguments of the gated linear recurrence's kernels and the gate arithmetic they share.
#pragma once

#include "common.cuh"

namespace lstm {

// Everything a launch reads; strides in elements.
struct GlrArgs {
    int T = 0, B = 0, H = 0, ndir = 1;
    int padded = 0;
    const int32_t* off = nullptr;       // [T+1]
    const int32_t* len = nullptr;       // [B] by slot
    const int32_t* perm = nullptr;      // [B]
    const int32_t* chunk = nullptr;     // [B+1]
    const void* f = nullptr;
    const void* z = nullptr;
    const void* i = nullptr;
    int64_t ld = 0, dstride = 0;
    const float* h0 = nullptr;          // [ndir][B][H] caller order
    void* y = nullptr;                  // [rows][ndir*H]
    float* h_n = nullptr;
    float* ws = nullptr;                // [chunks][ndir][H]
    // backward
    const void* dy = nullptr;
    const float* dh_n = nullptr;
    void* df = nullptr;
    void* dz = nullptr;
    void* di = nullptr;
    int64_t gld = 0, gdstride = 0;
    float* dh0 = nullptr;
};

__device__ __forceinline__ float ex2_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// min(sig(x), sig(-x)) = e / (1 + e) with e = exp(-|x|): the smaller of the gate and its
// complement, to a relative error near 2^-21 however close to 0 or 1 the gate is.  The larger
// one is 1 - m, exact to half an ulp; so neither sig(x) nor 1 - sig(x) loses its digits (with
// one of them subtracted from 1, a gate near 1 would leave 1 - a with few), and a product of
// many gates near 1 does not drift.
__device__ __forceinline__ float smaller_gate(float x)
{
    constexpr float kLog2e = 1.44269504088896341f;
    const float e = ex2_approx(-fabsf(x) * kLog2e);
    return e * rcp_approx(1.f + e);
}

// sig(x) and sig(-x)
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& c)
{
    const float m = smaller_gate(x), g = 1.f - m;
    const bool up = x >= 0.f;
    s = up ? g : m;
    c = up ? m : g;
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace lstm
