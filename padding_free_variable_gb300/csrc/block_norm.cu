// block_norm.cu -- the norms before and after a block with its gate and residual scale: entry points and kernels.
#include <algorithm>

#include "glr.cuh"

namespace lstm {

namespace {

constexpr int kSums = 5;            // w_post, b_post, scale, w_pre, b_pre
constexpr int kMaxParts = 304;      // row ranges of the backward pass's column sums

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

__device__ __forceinline__ float load1(const void* p, int64_t i, bool b16)
{
    return b16 ? __bfloat162float(((const __nv_bfloat16*)p)[i]) : ((const float*)p)[i];
}

__device__ __forceinline__ void store1(void* p, int64_t i, bool b16, float v)
{
    if (b16) ((__nv_bfloat16*)p)[i] = __float2bfloat16_rn(v);
    else ((float*)p)[i] = v;
}

__device__ float block_sum(float v)
{
    __shared__ float part[32];
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += part[w];
    return s;
}

// act(g) and act'(g)
__device__ __forceinline__ void activation(int kind, float q, float& act, float& slope)
{
    if (kind == LSTM_GATE_NONE) { act = 1.f; slope = 0.f; return; }
    float s, c;
    sigmoid_pair(q, s, c);
    if (kind == LSTM_GATE_SIGMOID) { act = s; slope = s * c; }
    else { act = q * s; slope = s * (1.f + q * c); }
}

__device__ __forceinline__ float x_out_of(const NormArgs& p, int64_t r, int c, float mean, float rstd)
{
    float x = load1(p.x, r * p.D + c, p.stream16);
    if (!p.y) return x;
    const float hat = (load1(p.y, r * p.ldy + c, p.branch16) - mean) * rstd;
    const float v = hat * (p.w.w_post ? p.w.w_post[c] : 1.f) + (p.w.b_post ? p.w.b_post[c] : 0.f);
    float act = 1.f, slope;
    if (p.gate) activation(p.gate, load1(p.g, r * p.ldg + c, p.branch16), act, slope);
    return x + (p.w.scale ? p.w.scale[c] : 1.f) * v * act;
}

__global__ void block_norm_fwd_kernel(const NormArgs p)
{
    const int64_t r = blockIdx.x;
    float my = 0.f, ry = 1.f, mx = 0.f, rx = 1.f;
    if (p.post) {
        float s = 0.f;
        if (p.post == LSTM_NORM_LAYER) {
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) s += load1(p.y, r * p.ldy + c, p.branch16);
            my = block_sum(s) / p.D;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = load1(p.y, r * p.ldy + c, p.branch16) - my;
            s += v * v;
        }
        ry = 1.f / sqrtf(block_sum(s) / p.D + p.eps);
    }
    if (p.pre) {
        float s = 0.f;
        if (p.pre == LSTM_NORM_LAYER) {
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) s += x_out_of(p, r, c, my, ry);
            mx = block_sum(s) / p.D;
        }
        s = 0.f;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float v = x_out_of(p, r, c, my, ry) - mx;
            s += v * v;
        }
        rx = 1.f / sqrtf(block_sum(s) / p.D + p.eps);
    }
    for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
        const float x1 = x_out_of(p, r, c, my, ry);
        if (p.n)
            store1(p.n, r * p.D + c, p.norm16,
                   (x1 - mx) * rx * (p.w.w_pre ? p.w.w_pre[c] : 1.f) + (p.w.b_pre ? p.w.b_pre[c] : 0.f));
        if (p.x_out) store1(p.x_out, r * p.D + c, p.stream16, x1);
    }
    if (p.stats && threadIdx.x == 0) {
        float* t = p.stats + r * 4;
        t[0] = my; t[1] = ry; t[2] = mx; t[3] = rx;
    }
}

__global__ void block_norm_bwd_kernel(const NormArgs p)
{
    float* part = p.part + (int64_t)blockIdx.x * kSums * p.D;
    for (int c = threadIdx.x; c < kSums * p.D; c += blockDim.x) part[c] = 0.f;
    __syncthreads();
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const float my = p.stats[r * 4], ry = p.stats[r * 4 + 1], mx = p.stats[r * 4 + 2], rx = p.stats[r * 4 + 3];
        // dx' = dx_out + rx (t - mean t - xh mean(t xh)), t = dn w_pre
        float s0 = 0.f, s1 = 0.f;
        if (p.dn)
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                const float t = load1(p.dn, r * p.D + c, p.norm16) * (p.w.w_pre ? p.w.w_pre[c] : 1.f);
                s0 += t;
                s1 += t * (x_out_of(p, r, c, my, ry) - mx) * rx;
            }
        const float m0 = p.pre == LSTM_NORM_LAYER ? block_sum(s0) / p.D : 0.f, m1 = block_sum(s1) / p.D;
        auto dx_of = [&](int c) {
            float dx = p.dx_out ? load1(p.dx_out, r * p.D + c, p.stream16) : 0.f;
            if (p.dn) {
                const float t = load1(p.dn, r * p.D + c, p.norm16) * (p.w.w_pre ? p.w.w_pre[c] : 1.f);
                dx += rx * (t - m0 - (x_out_of(p, r, c, my, ry) - mx) * rx * m1);
            }
            return dx;
        };
        auto sc = [&](int c) { return p.w.scale ? p.w.scale[c] : 1.f; };
        auto wp = [&](int c) { return p.w.w_post ? p.w.w_post[c] : 1.f; };
        float q0 = 0.f, q1 = 0.f;
        if (p.y && p.post)
            for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                float act = 1.f, slope;
                if (p.gate) activation(p.gate, load1(p.g, r * p.ldg + c, p.branch16), act, slope);
                const float t = dx_of(c) * sc(c) * act * wp(c);
                q0 += t;
                q1 += t * (load1(p.y, r * p.ldy + c, p.branch16) - my) * ry;
            }
        const float k0 = p.post == LSTM_NORM_LAYER ? block_sum(q0) / p.D : 0.f, k1 = block_sum(q1) / p.D;
        for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
            const float dx = dx_of(c);
            if (p.dn) {
                const float dn = load1(p.dn, r * p.D + c, p.norm16);
                part[3 * p.D + c] += dn * (x_out_of(p, r, c, my, ry) - mx) * rx;
                part[4 * p.D + c] += dn;
            }
            if (p.y) {
                const float hat = (load1(p.y, r * p.ldy + c, p.branch16) - my) * ry;
                const float v = hat * wp(c) + (p.w.b_post ? p.w.b_post[c] : 0.f);
                float act = 1.f, slope = 0.f;
                if (p.gate) activation(p.gate, load1(p.g, r * p.ldg + c, p.branch16), act, slope);
                const float du = dx * sc(c), dv = du * act, t = dv * wp(c);
                part[c] += dv * hat;
                part[p.D + c] += dv;
                part[2 * p.D + c] += dx * v * act;
                store1(p.dy, r * p.lddy + c, p.branch16, p.post ? ry * (t - k0 - hat * k1) : t);
                if (p.gate) store1(p.dg, r * p.lddg + c, p.branch16, du * v * slope);
            }
            store1(p.dx, r * p.D + c, p.stream16, dx);
        }
        __syncthreads();
    }
}

__global__ void block_norm_sums_kernel(const NormArgs p)
{
    const int c = blockIdx.x * blockDim.x + threadIdx.x, k = blockIdx.y;
    if (c >= p.D || !p.sums[k]) return;
    float s = 0.f;
    for (int b = 0; b < p.parts; ++b) s += p.part[((int64_t)b * kSums + k) * p.D + c];
    p.sums[k][c] = s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

size_t elem(int dtype) { return dtype == LSTM_BF16 ? 2 : 4; }

lstm_status check_norm_shape(const lstm_block_norm_shape* s)
{
    if (!s || s->width < 1 || !(s->eps > 0.f)) return LSTM_ERR_INVALID_ARG;
    for (int k : {s->post_kind, s->pre_kind})
        if (k < LSTM_NORM_NONE || k > LSTM_NORM_LAYER) return LSTM_ERR_INVALID_ARG;
    if (s->gate < LSTM_GATE_NONE || s->gate > LSTM_GATE_SILU) return LSTM_ERR_INVALID_ARG;
    for (int t : {s->branch_dtype, s->stream_dtype, s->norm_dtype})
        if (t != LSTM_F32 && t != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
    if (s->width > 16384) return LSTM_ERR_UNSUPPORTED;
    return LSTM_OK;
}

// What forward and backward have in common: shape, parameters, the rows that come in.
lstm_status norm_args(const lstm_block_norm_shape* shape, const lstm_block_norm_params* params,
                      const lstm_block_norm_inputs* in, int64_t rows, NormArgs* a)
{
    const lstm_status st = check_norm_shape(shape);
    if (st != LSTM_OK) return st;
    const lstm_block_norm_shape& s = *shape;
    if (!params || !in || rows < 0 || rows > INT32_MAX) return LSTM_ERR_INVALID_ARG;
    for (const float* w : {params->w_post, params->b_post, params->scale, params->w_pre, params->b_pre})
        if (!aligned(w, 4)) return LSTM_ERR_INVALID_ARG;
    if (s.post_kind == LSTM_NORM_NONE && (params->w_post || params->b_post)) return LSTM_ERR_INVALID_ARG;
    if (s.pre_kind == LSTM_NORM_NONE && (params->w_pre || params->b_pre)) return LSTM_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!in->x || !aligned(in->x, elem(s.stream_dtype))) return LSTM_ERR_INVALID_ARG;
        if (!in->y) {
            if (s.post_kind != LSTM_NORM_NONE || s.gate != LSTM_GATE_NONE || s.pre_kind == LSTM_NORM_NONE || params->scale)
                return LSTM_ERR_INVALID_ARG;
        } else if (!aligned(in->y, elem(s.branch_dtype)) || in->y_stride < s.width) {
            return LSTM_ERR_INVALID_ARG;
        }
        if ((s.gate != LSTM_GATE_NONE) != (in->gate != nullptr)) return LSTM_ERR_INVALID_ARG;
        if (in->gate && (!aligned(in->gate, elem(s.branch_dtype)) || in->gate_stride < s.width)) return LSTM_ERR_INVALID_ARG;
    }
    a->D = s.width;
    a->post = s.post_kind; a->pre = s.pre_kind; a->gate = s.gate;
    a->branch16 = s.branch_dtype == LSTM_BF16;
    a->stream16 = s.stream_dtype == LSTM_BF16;
    a->norm16 = s.norm_dtype == LSTM_BF16;
    a->eps = s.eps; a->rows = rows; a->w = *params;
    a->x = in->x; a->y = in->y; a->g = in->gate; a->ldy = in->y_stride; a->ldg = in->gate_stride;
    return LSTM_OK;
}

int norm_parts(int64_t rows) { return (int)std::min<int64_t>(rows, kMaxParts); }

lstm_status launched() { return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA; }

}  // namespace

}  // namespace lstm

using namespace lstm;

extern "C" {

lstm_status lstm_block_norm_fwd(const lstm_block_norm_shape* shape, const lstm_block_norm_params* params,
                                const lstm_block_norm_inputs* in, int64_t rows, void* x_out, void* n,
                                float* stats, void* stream)
{
    NormArgs a;
    const lstm_status st = norm_args(shape, params, in, rows, &a);
    if (st != LSTM_OK) return st;
    if (rows == 0) return LSTM_OK;
    if ((in->y != nullptr) != (x_out != nullptr) || (shape->pre_kind != LSTM_NORM_NONE) != (n != nullptr))
        return LSTM_ERR_INVALID_ARG;
    if (!aligned(x_out, elem(shape->stream_dtype)) || !aligned(n, elem(shape->norm_dtype)) || !aligned(stats, 16))
        return LSTM_ERR_INVALID_ARG;
    a.x_out = x_out; a.n = n; a.stats = stats;
    block_norm_fwd_kernel<<<(unsigned)rows, 256, 0, (cudaStream_t)stream>>>(a);
    return launched();
}

size_t lstm_block_norm_scratch_bytes(const lstm_block_norm_shape* shape, int64_t rows)
{
    if (check_norm_shape(shape) != LSTM_OK || rows < 0 || rows > INT32_MAX) return 0;
    return std::max<size_t>(16, (size_t)norm_parts(rows) * kSums * shape->width * sizeof(float));
}

lstm_status lstm_block_norm_bwd(const lstm_block_norm_shape* shape, const lstm_block_norm_params* params,
                                const lstm_block_norm_inputs* in, int64_t rows, const float* stats,
                                const void* dx_out, const void* dn, const lstm_block_norm_input_grads* din,
                                const lstm_block_norm_grads* grads, void* scratch, void* stream)
{
    NormArgs a;
    const lstm_status st = norm_args(shape, params, in, rows, &a);
    if (st != LSTM_OK) return st;
    if (!din || !grads) return LSTM_ERR_INVALID_ARG;
    cudaStream_t cs = (cudaStream_t)stream;
    float* const sums[kSums] = {grads->w_post, grads->b_post, grads->scale, grads->w_pre, grads->b_pre};
    for (float* g : sums)
        if (!aligned(g, 4)) return LSTM_ERR_INVALID_ARG;
    if (rows == 0) {
        for (float* g : sums)
            if (g) LSTM_CUDA_TRY(cudaMemsetAsync(g, 0, sizeof(float) * shape->width, cs));
        return LSTM_OK;
    }
    const size_t be = elem(shape->branch_dtype), se = elem(shape->stream_dtype);
    if (!stats || !aligned(stats, 16) || !scratch || !aligned(scratch, 16)) return LSTM_ERR_INVALID_ARG;
    if (!aligned(dx_out, se) || !aligned(dn, elem(shape->norm_dtype)) || (dn && shape->pre_kind == LSTM_NORM_NONE))
        return LSTM_ERR_INVALID_ARG;
    if (!din->dx || !aligned(din->dx, se)) return LSTM_ERR_INVALID_ARG;
    if ((din->dy != nullptr) != (in->y != nullptr) || (din->dgate != nullptr) != (in->gate != nullptr)) return LSTM_ERR_INVALID_ARG;
    if (din->dy && (!aligned(din->dy, be) || din->dy_stride < shape->width)) return LSTM_ERR_INVALID_ARG;
    if (din->dgate && (!aligned(din->dgate, be) || din->dgate_stride < shape->width)) return LSTM_ERR_INVALID_ARG;
    a.stats = const_cast<float*>(stats);
    a.dx_out = dx_out; a.dn = dn; a.dx = din->dx; a.dy = din->dy; a.dg = din->dgate;
    a.lddy = din->dy_stride; a.lddg = din->dgate_stride;
    a.part = (float*)scratch; a.parts = norm_parts(rows);
    for (int k = 0; k < kSums; ++k) a.sums[k] = sums[k];
    block_norm_bwd_kernel<<<a.parts, 256, 0, cs>>>(a);
    block_norm_sums_kernel<<<dim3(ceil_div(a.D, 128), kSums), 128, 0, cs>>>(a);
    return launched();
}

}  // extern "C"
