// glr.cu -- the gated linear recurrence over packed rows: entry points and kernels.
//
// h_t = a_t h_{t-1} + b_t per unit, a = sig(f), b = (1 - a) z (tied) or sig(i) z (gated).
#include <algorithm>
#include <type_traits>

#include "glr.cuh"

namespace lstm {

namespace {

template <typename T, bool GATED>
__global__ void glr_step_kernel(const GlrArgs p, const int32_t* slots, int rows, int num_slots, const float* state_in,
                                float* state_out)
{
    const int64_t n = (int64_t)rows * p.H;
    for (int64_t k = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; k < n; k += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = k / p.H;
        const int u = (int)(k - r * p.H);
        const int slot = slots ? slots[r] : (int)r;
        float h = 0.f;
        if (slot >= 0 && slot < num_slots) {
            const int64_t at = r * p.ld + u;
            float a, b;
            sigmoid_pair(to_f32(((const T*)p.f)[at]), a, b);
            if (GATED) {
                float c;
                sigmoid_pair(to_f32(((const T*)p.i)[at]), b, c);
            }
            h = fmaf(a, state_in[(int64_t)slot * p.H + u], b * to_f32(((const T*)p.z)[at]));
            state_out[(int64_t)slot * p.H + u] = h;
        }
        ((T*)p.y)[k] = from_f32<T>(h);
    }
}

lstm_status launched() { return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA; }

lstm_status check_glr_shape(const lstm_glr_shape* s)
{
    if (!s || s->hidden_size < 1) return LSTM_ERR_INVALID_ARG;
    if (s->num_directions != 1 && s->num_directions != 2) return LSTM_ERR_INVALID_ARG;
    if (s->dtype != LSTM_F32 && s->dtype != LSTM_BF16) return LSTM_ERR_INVALID_ARG;
    if (s->cell != LSTM_GLR_TIED && s->cell != LSTM_GLR_GATED) return LSTM_ERR_INVALID_ARG;
    if (s->hidden_size > 65536) return LSTM_ERR_UNSUPPORTED;
    return LSTM_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Gate pointers (read or written): all there, aligned to their element, rows that do not overlap themselves.
bool good_gates(const lstm_glr_shape& s, const void* f, const void* z, const void* i, int64_t ld, int64_t ds)
{
    const size_t e = s.dtype == LSTM_BF16 ? 2 : 4;
    if (!f || !z || !aligned(f, e) || !aligned(z, e)) return false;
    if ((s.cell == LSTM_GLR_GATED) != (i != nullptr) || !aligned(i, e)) return false;
    return ld >= s.hidden_size && (s.num_directions == 1 || ds >= s.hidden_size);
}

bool right_device(const Plan& p)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == p.device;
}

bool fits(const void* p, int64_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

GlrArgs plan_args(const Plan& p, const lstm_glr_shape& s, const lstm_glr_gates& g)
{
    GlrArgs a;
    a.T = p.T; a.B = p.B; a.H = s.hidden_size; a.ndir = s.num_directions;
    a.padded = p.padded ? 1 : 0;
    a.off = p.d_off; a.len = p.d_len; a.perm = p.d_perm; a.chunk = p.d_chunk;
    a.f = g.f; a.z = g.z; a.i = g.i; a.ld = g.row_stride; a.dstride = g.dir_stride;
    return a;
}

template <typename F>
void dispatch(const lstm_glr_shape& s, F&& go)
{
    const bool gated = s.cell == LSTM_GLR_GATED;
    if (s.dtype == LSTM_BF16) {
        if (gated) go((__nv_bfloat16*)nullptr, std::true_type());
        else go((__nv_bfloat16*)nullptr, std::false_type());
    } else {
        if (gated) go((float*)nullptr, std::true_type());
        else go((float*)nullptr, std::false_type());
    }
}

// Every sequence is empty: what comes in as the state (or its error) goes out unchanged.
lstm_status pass_through(const float* in, float* out, size_t bytes, cudaStream_t cs)
{
    if (!out) return LSTM_OK;
    LSTM_CUDA_TRY(in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, cs) : cudaMemsetAsync(out, 0, bytes, cs));
    return LSTM_OK;
}

}  // namespace

GlrRows glr_rows(const GlrArgs& a, int elem)
{
    // every row of every operand starts on a multiple of `bytes`, and so does its length
    auto whole = [&](int64_t bytes) {
        bool ok = true;
        for (int64_t n : {(int64_t)a.H, a.ld, a.ndir == 1 ? 0 : a.dstride, a.gld, a.ndir == 1 ? 0 : a.gdstride})
            ok = ok && n * elem % bytes == 0;
        for (const void* p : {a.f, a.z, a.i, (const void*)a.y, a.dy, (const void*)a.df, (const void*)a.dz, (const void*)a.di})
            ok = ok && fits(p, bytes);
        return ok;
    };
    // fp32 rows of at most 32 units fill a warp with one unit a lane
    if (whole(16) && (elem == 2 || a.H > 32)) return GLR_WIDE;
    return whole(4) ? GLR_NARROW : GLR_SINGLE;
}

void glr_cut(const Plan& p, int V, int ctas, void* scratch, GlrArgs* a)
{
    // An uncut sequence takes T/64 iterations one after another; all of them, spread evenly over
    // the CTAs that the GPU holds, `share`.  Where the longest sequence would run far past that, it
    // is cut (every piece's gates are then read twice), into pieces short enough to spread well and
    // long enough that starting them (about two iterations) does not show.
    const int64_t blocks = ceil_div(a->H, 32 * V), slots = (int64_t)p.num_sms * ctas;
    const int64_t share = p.chunks * blocks * a->ndir / slots, longest = ceil_div(p.T, kScanChunk);
    int l = p.levels - 1;
    if (scratch && longest > share * 3 / 2 + 12)
        for (l = 0; l < p.levels - 1 && ((int64_t)kScanPiece << l) < kScanChunk * share / 5; ++l) {}
    a->pieces = p.d_pieces + p.level_first[l];
    a->count = p.level_count[l];
    a->cut = l < p.levels - 1;
    a->piece = a->cut ? kScanPiece << l : INT32_MAX;
    a->maps = (float4*)scratch;
}

size_t glr_scratch(const Plan& p, const lstm_glr_shape& s)
{
    // the finest level's maps, 8 bytes a unit, in blocks of at most 64 units
    return p.levels < 2 ? 0 : (size_t)p.level_count[0] * s.num_directions * (size_t)ceil_div(s.hidden_size, 64) * 64 * 8;
}

}  // namespace lstm

using namespace lstm;

extern "C" {

size_t lstm_glr_workspace_bytes(const lstm_plan* plan, const lstm_glr_shape* shape)
{
    if (!plan || check_glr_shape(shape) != LSTM_OK) return 0;
    const size_t n = (size_t)plan->p.chunks * shape->num_directions * shape->hidden_size * sizeof(float);
    return n > 16 ? n : 16;
}

size_t lstm_glr_scratch_bytes(const lstm_plan* plan, const lstm_glr_shape* shape)
{
    if (!plan || check_glr_shape(shape) != LSTM_OK) return 0;
    return glr_scratch(plan->p, *shape);
}

lstm_status lstm_glr_fwd(const lstm_plan* plan, const lstm_glr_shape* shape, const lstm_glr_gates* gates,
                         const float* h0, void* y, float* h_n, void* workspace, void* scratch, void* stream)
{
    if (!plan || !gates) return LSTM_ERR_INVALID_ARG;
    lstm_status st = check_glr_shape(shape);
    if (st != LSTM_OK) return st;
    const Plan& p = plan->p;
    const lstm_glr_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!aligned(h0, 4) || !aligned(h_n, 4) || !aligned(workspace, 16) || !aligned(scratch, 16) || !right_device(p)) return LSTM_ERR_INVALID_ARG;
    if (p.rows == 0) return pass_through(h0, h_n, sizeof(float) * s.num_directions * p.B * s.hidden_size, cs);
    if (!y || !aligned(y, s.dtype == LSTM_BF16 ? 2 : 4) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    if (gates->row_stride > kGlrMaxStride) return LSTM_ERR_UNSUPPORTED;
    GlrArgs a = plan_args(p, s, *gates);
    a.h0 = h0; a.y = y; a.h_n = h_n; a.ws = (float*)workspace;
    return launch_glr_fwd(p, s, a, scratch, cs);
}

lstm_status lstm_glr_bwd(const lstm_plan* plan, const lstm_glr_shape* shape, const lstm_glr_gates* gates,
                         const void* workspace, const void* dy, const float* dh_n,
                         const lstm_glr_gate_grads* grads, float* dh0, void* scratch, void* stream)
{
    if (!plan || !gates || !grads) return LSTM_ERR_INVALID_ARG;
    lstm_status st = check_glr_shape(shape);
    if (st != LSTM_OK) return st;
    const Plan& p = plan->p;
    const lstm_glr_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!aligned(dh_n, 4) || !aligned(dh0, 4) || !aligned(workspace, 16) || !aligned(scratch, 16) || !right_device(p)) return LSTM_ERR_INVALID_ARG;
    if (p.rows == 0) return pass_through(dh_n, dh0, sizeof(float) * s.num_directions * p.B * s.hidden_size, cs);
    if (!workspace || !dy || !aligned(dy, s.dtype == LSTM_BF16 ? 2 : 4) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride) ||
        !good_gates(s, grads->f, grads->z, grads->i, grads->row_stride, grads->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    if (gates->row_stride > kGlrMaxStride || grads->row_stride > kGlrMaxStride) return LSTM_ERR_UNSUPPORTED;
    GlrArgs a = plan_args(p, s, *gates);
    a.ws = (float*)const_cast<void*>(workspace); a.dy = dy; a.dh_n = dh_n; a.dh0 = dh0;
    a.df = grads->f; a.dz = grads->z; a.di = grads->i; a.gld = grads->row_stride; a.gdstride = grads->dir_stride;
    return launch_glr_bwd(p, s, a, scratch, cs);
}

lstm_status lstm_glr_step(const lstm_glr_shape* shape, const lstm_glr_gates* gates, int32_t rows,
                          const int32_t* slots, int32_t num_slots, const float* state_in, float* state_out,
                          void* y, void* stream)
{
    lstm_status st = check_glr_shape(shape);
    if (st != LSTM_OK) return st;
    const lstm_glr_shape& s = *shape;
    if (!gates || rows < 0 || num_slots < 0 || s.num_directions != 1 || (!slots && num_slots < rows))
        return LSTM_ERR_INVALID_ARG;
    if (rows == 0) return LSTM_OK;
    if (!y || !aligned(y, s.dtype == LSTM_BF16 ? 2 : 4) || !aligned(slots, 4) || !aligned(state_in, 4) ||
        !aligned(state_out, 4) || (num_slots > 0 && (!state_in || !state_out)) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    GlrArgs a;
    a.H = s.hidden_size;
    a.f = gates->f; a.z = gates->z; a.i = gates->i; a.ld = gates->row_stride; a.y = y;
    const int64_t n = (int64_t)rows * s.hidden_size;
    const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 65535);
    dispatch(s, [&](auto* t, auto gated) {
        glr_step_kernel<std::remove_pointer_t<decltype(t)>, decltype(gated)::value>
            <<<grid, 256, 0, (cudaStream_t)stream>>>(a, slots, rows, num_slots, state_in, state_out);
    });
    return launched();
}

}  // extern "C"
