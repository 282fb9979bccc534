// block_norm.cu -- the norms before and after a block with its gate and residual scale: entry points.
#include <algorithm>

#include "block_norm.cuh"

namespace lstm {

namespace {

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

}  // namespace

bool norm_full(const NormArgs& a)
{
    const bool layer = a.post == LSTM_NORM_LAYER;
    return a.y && a.post && a.post == a.pre && a.w.w_post && a.w.scale && a.w.w_pre && layer == (a.w.b_post != nullptr) &&
           layer == (a.w.b_pre != nullptr) && a.norm16 == a.branch16 && (a.branch16 || !a.stream16);
}

static bool norm_aligned(const NormArgs& a)
{
    bool ok = true;
    for (const void* p : {a.x, a.y, a.g, (const void*)a.x_out, (const void*)a.n, a.dx_out, a.dn, (const void*)a.dx,
                          (const void*)a.dy, (const void*)a.dg, (const void*)a.w.w_post, (const void*)a.w.b_post,
                          (const void*)a.w.scale, (const void*)a.w.w_pre, (const void*)a.w.b_pre})
        ok = ok && aligned(p, 16);
    return ok;
}

bool norm_whole(const NormArgs& a)
{
    return a.D % 8 == 0 && a.ldy % 8 == 0 && a.ldg % 8 == 0 && a.lddy % 8 == 0 && a.lddg % 8 == 0 && norm_aligned(a);
}

bool norm_shifted(const NormArgs& a)
{
    // (a row but the last reads up to 7 values past its end, which the next row must have)
    const int64_t D = a.D;
    return norm_full(a) && D >= 7 && D % 8 != 0 && (a.ldy - D) % 8 == 0 && (!a.g || (a.ldg - D) % 8 == 0) && (!a.dy || (a.lddy - D) % 8 == 0) &&
           (!a.dg || (a.lddg - D) % 8 == 0) && norm_aligned(a);
}

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
    return launch_norm_fwd(a, (cudaStream_t)stream);
}

size_t lstm_block_norm_scratch_bytes(const lstm_block_norm_shape* shape, int64_t rows)
{
    if (check_norm_shape(shape) != LSTM_OK || rows < 0 || rows > INT32_MAX) return 0;
    return std::max<size_t>(16, (size_t)norm_parts(rows, shape->width) * kSums * shape->width * sizeof(float));
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
    a.part = (float*)scratch; a.parts = norm_parts(rows, shape->width);
    for (int k = 0; k < kSums; ++k) a.sums[k] = sums[k];
    return launch_norm_bwd(a, cs);
}

}  // extern "C"
