// glr.cu -- the gated linear recurrence over packed rows: entry points and kernels.
//
// h_t = a_t h_{t-1} + b_t per unit, a = sig(f), b = (1 - a) z (tied) or sig(i) z (gated).
#include <algorithm>
#include <type_traits>

#include "glr.cuh"

namespace lstm {

namespace {

// One frame of many streams: V units of a stream a thread; threads of a block: x along the units, y
// along the streams.  Bound by memory where streams are many (gates and states read once, states
// and outputs written once: 4096 streams of 1024 fp32 units 19 us with a cold L2, 5.2 TB/s; one unit
// a thread and a division for the stream took 35 us), by the launch where they are few (8 streams of
// 512 bf16 units 1.3 us in a graph, 6.8 us as a call).
template <typename T, bool GATED, int V>
__global__ void __launch_bounds__(128) glr_step_kernel(const GlrArgs p, const int32_t* slots, int rows, int num_slots, const float* state_in,
                                                       float* state_out)
{
    typedef typename std::conditional<V * sizeof(T) == 16, uint4, T>::type Bits;
    union G { Bits b; T e[V]; __device__ G() {} };
    const int u = (blockIdx.x * blockDim.x + threadIdx.x) * V;
    if (u >= p.H) return;
    for (int64_t r = blockIdx.y * (int64_t)blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.y * blockDim.y) {
        const int slot = slots ? __ldg(slots + r) : (int)r;
        G f, z, g, out;
        float h[V];
        const int64_t at = r * p.ld + u, state = (int64_t)slot * p.H + u;
        if (slot >= 0 && slot < num_slots) {
            f.b = *(const Bits*)((const T*)p.f + at);
            z.b = *(const Bits*)((const T*)p.z + at);
            if (GATED) g.b = *(const Bits*)((const T*)p.i + at);
            if constexpr (V % 4 == 0) {
#pragma unroll
                for (int v = 0; v < V; v += 4) {
                    const float4 q = *(const float4*)(state_in + state + v);
                    h[v] = q.x; h[v + 1] = q.y; h[v + 2] = q.z; h[v + 3] = q.w;
                }
            } else {
                h[0] = state_in[state];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float a, b;
                sigmoid_pair(to_f32(f.e[v]), a, b);
                if (GATED) b = rcp_approx(1.f + ex2_approx(to_f32(g.e[v]) * kNegLog2e));
                h[v] = fmaf(a, h[v], b * to_f32(z.e[v]));
            }
            if constexpr (V % 4 == 0) {
#pragma unroll
                for (int v = 0; v < V; v += 4) *(float4*)(state_out + state + v) = make_float4(h[v], h[v + 1], h[v + 2], h[v + 3]);
            } else {
                state_out[state] = h[0];
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) out.e[v] = from_f32<T>(h[v]);
        *(Bits*)((T*)p.y + r * p.H + u) = out.b;
    }
}

template <typename T, bool GATED, int V>
lstm_status step(const GlrArgs& a, const int32_t* slots, int rows, int num_slots, const float* in, float* out, cudaStream_t cs)
{
    const int along = ceil_div(a.H, V);
    int x = 1;
    while (x < 128 && x < along) x *= 2;
    const dim3 block(x, 128 / x), grid(ceil_div(along, x), (unsigned)std::min<int64_t>(((int64_t)rows + block.y - 1) / block.y, 65535));
    glr_step_kernel<T, GATED, V><<<grid, block, 0, cs>>>(a, slots, rows, num_slots, in, out);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

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

GlrArgs plan_args(const ScanPlan& sp, const lstm_glr_shape& s, const lstm_glr_gates& g)
{
    const Plan& p = sp.p;
    GlrArgs a;
    a.T = p.T; a.B = p.B; a.H = s.hidden_size; a.ndir = s.num_directions;
    a.padded = p.padded ? 1 : 0;
    a.off = p.d_off; a.len = p.d_len; a.perm = p.d_perm; a.chunk = sp.scan.d_chunk;
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

size_t state_bytes(const ScanPlan& p, int ndir, int H) { return sizeof(float) * ndir * p.p.B * H; }

// The state that comes in and the one that goes out: one array or two, but not parts of each other.
bool same_or_apart(const float* in, const float* out, size_t bytes)
{
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out;
    return !in || !out || in == out || a + bytes <= b || b + bytes <= a;
}

// Bytes of the finest level's maps, 8 a unit, in blocks of at most 64 units.
size_t map_bytes(const ScanPlan& p, int ndir, int H) { return (size_t)p.scan.level_count[0] * ndir * (size_t)ceil_div(H, 64) * 64 * 8; }

// Every sequence is empty: what comes in as the state (or its error) goes out unchanged.
lstm_status pass_through(const float* in, float* out, size_t bytes, cudaStream_t cs)
{
    if (!out || out == in) return LSTM_OK;
    LSTM_CUDA_TRY(in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, cs) : cudaMemsetAsync(out, 0, bytes, cs));
    return LSTM_OK;
}

}  // namespace

// Every row of every operand starts on a multiple of `bytes`, and so does its length.
static bool glr_whole(const GlrArgs& a, int elem, int64_t bytes)
{
    bool ok = true;
    for (int64_t n : {(int64_t)a.H, a.ld, a.ndir == 1 ? 0 : a.dstride, a.gld, a.ndir == 1 ? 0 : a.gdstride})
        ok = ok && n * elem % bytes == 0;
    for (const void* p : {a.f, a.z, a.i, (const void*)a.y, a.dy, (const void*)a.df, (const void*)a.dz, (const void*)a.di})
        ok = ok && fits(p, bytes);
    return ok;
}

GlrRows glr_rows(const GlrArgs& a, int elem)
{
    // 40555 frames of 2 x 512 bf16 units forward / backward: wide 52 / 89 us, narrow (rows 4 bytes
    // off) 64 / 105 us, single (2 bytes off) 85 / 154 us; 70 k frames of 2 x 256 fp32, three gates: wide
    // 91 / 158 us, narrow 107 / 206 us.  Grouped against wide: 74 sequences of 21099 frames of 8 bf16
    // units 113 / 168 against 326 / 480 us, 60 of 19 to 211 frames of 2 x 16 units 9 / 11 against 13 / 15.
    if (glr_whole(a, elem, 16)) return a.H > 32 ? GLR_WIDE : GLR_GROUPED;
    return glr_whole(a, elem, 4) ? GLR_NARROW : GLR_SINGLE;
}

void glr_cut(const ScanPlan& p, int V, int ctas, void* scratch, GlrArgs* a)
{
    // An uncut sequence takes T/64 iterations one after another; all of them, spread evenly over
    // the CTAs that the GPU holds, `share`.  Where the longest sequence would run far past that, it
    // is cut (every piece's gates are then read twice), into pieces short enough to spread well and
    // long enough that starting them (about two iterations) does not show.  One sequence of 65536
    // frames of 1024 bf16 units, tied, forward: 132 us cut, 752 us uncut; two of 20 to 30 thousand frames
    // of 512 fp32 units forward / backward 91 / 132 against 367 / 871 us; 32 of 200 to 2400 frames of 256
    // bf16 units, just past the rule's edge, 31 / 44 against 33 / 58 us.
    const int64_t blocks = ceil_div(a->H, 32 * V), slots = (int64_t)p.p.num_sms * ctas;
    const int64_t steps = (int64_t)kScanChunk * a->groups, share = p.scan.chunks / a->groups * blocks * a->ndir / slots;
    const int64_t longest = (p.p.T + steps - 1) / steps;
    int l = p.scan.levels - 1;
    if (scratch && longest > share * 3 / 2 + 12)
        for (l = 0; l < p.scan.levels - 1 && ((int64_t)kScanPiece << l) < steps * share / 5; ++l) {}
    a->pieces = p.scan.d_pieces + p.scan.level_first[l];
    a->count = p.scan.level_count[l];
    a->cut = l < p.scan.levels - 1;
    a->piece = a->cut ? kScanPiece << l : INT32_MAX;
    a->maps = (float4*)scratch;
}

bool glr_short(const ScanPlan& p, int V, int ctas, GlrArgs* a)
{
    // A warp takes 8 steps at a time, all warps that the GPU holds at once: the longest sequence's
    // tiles against an even share.  A CTA's 64 steps cost it as much for a sequence of 8.  512
    // directions of 70 frames of 1024 bf16 units forward / backward: 42 / 87 us, a CTA each 76 / 136 us.
    // Sequences of two tiles at most need no such share: 64 of 16 frames of 512 bf16 units 3.6 / 5.0 us in a graph, a
    // CTA each 6.2 / 8.6; few of them come out alike (8: 3.5 / 4.7 and 3.3 / 4.3), three tiles no more (8 of 24 frames:
    // 4.0 / 5.8 and 3.6 / 4.0).
    const int64_t items = (int64_t)ceil_div(a->H, 32 * V) * a->ndir * p.p.B, warps = (int64_t)p.p.num_sms * ctas * kGlrWarps;
    const int64_t longest = ceil_div(p.p.T, kGlrSteps), share = p.p.rows / kGlrSteps * (items / p.p.B) / warps;
    if (longest > 2 && (items * 2 < warps || longest > 2 * share + 8)) return false;
    const int l = p.scan.levels - 1;
    a->pieces = p.scan.d_pieces + p.scan.level_first[l];
    a->count = p.scan.level_count[l];
    a->cut = false;
    a->piece = INT32_MAX;
    return true;
}

size_t glr_scratch(const ScanPlan& p, const lstm_glr_shape& s)
{
    // the maps, and behind them a copy of the states (glr_carry)
    const int nd = s.num_directions, H = s.hidden_size;
    return p.scan.levels < 2 ? 0 : map_bytes(p, nd, H) + state_bytes(p, nd, H);
}

lstm_status glr_carry(const ScanPlan& p, const GlrArgs& a, const float** in, const float* out, void* scratch, cudaStream_t cs)
{
    if (!a.cut || *in != out || !out) return LSTM_OK;
    float* const copy = (float*)((char*)scratch + map_bytes(p, a.ndir, a.H));
    LSTM_CUDA_TRY(cudaMemcpyAsync(copy, out, state_bytes(p, a.ndir, a.H), cudaMemcpyDeviceToDevice, cs));
    *in = copy;
    return LSTM_OK;
}

}  // namespace lstm

using namespace lstm;

extern "C" {

size_t lstm_glr_workspace_bytes(const lstm_plan* plan, const lstm_glr_shape* shape)
{
    if (!plan || check_glr_shape(shape) != LSTM_OK) return 0;
    const size_t n = (size_t)static_cast<const ScanPlan*>(plan)->scan.chunks * shape->num_directions * shape->hidden_size * sizeof(float);
    return n > 16 ? n : 16;
}

size_t lstm_glr_scratch_bytes(const lstm_plan* plan, const lstm_glr_shape* shape)
{
    if (!plan || check_glr_shape(shape) != LSTM_OK) return 0;
    return glr_scratch(*static_cast<const ScanPlan*>(plan), *shape);
}

lstm_status lstm_glr_fwd(const lstm_plan* plan, const lstm_glr_shape* shape, const lstm_glr_gates* gates,
                         const float* h0, void* y, float* h_n, void* workspace, void* scratch, void* stream)
{
    if (!plan || !gates) return LSTM_ERR_INVALID_ARG;
    lstm_status st = check_glr_shape(shape);
    if (st != LSTM_OK) return st;
    const ScanPlan& sp = *static_cast<const ScanPlan*>(plan);
    const Plan& p = sp.p;
    const lstm_glr_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!aligned(h0, 4) || !aligned(h_n, 4) || !aligned(workspace, 16) || !aligned(scratch, 16) || !right_device(p)) return LSTM_ERR_INVALID_ARG;
    const size_t states = state_bytes(sp, s.num_directions, s.hidden_size);
    if (!same_or_apart(h0, h_n, states)) return LSTM_ERR_INVALID_ARG;
    if (p.rows == 0) return pass_through(h0, h_n, states, cs);
    if (!y || !aligned(y, s.dtype == LSTM_BF16 ? 2 : 4) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    if (gates->row_stride > kGlrMaxStride) return LSTM_ERR_UNSUPPORTED;
    GlrArgs a = plan_args(sp, s, *gates);
    a.h0 = h0; a.y = y; a.h_n = h_n; a.ws = (float*)workspace;
    return launch_glr_fwd(sp, s, a, scratch, cs);
}

lstm_status lstm_glr_bwd(const lstm_plan* plan, const lstm_glr_shape* shape, const lstm_glr_gates* gates,
                         const void* workspace, const void* dy, const float* dh_n,
                         const lstm_glr_gate_grads* grads, float* dh0, void* scratch, void* stream)
{
    if (!plan || !gates || !grads) return LSTM_ERR_INVALID_ARG;
    lstm_status st = check_glr_shape(shape);
    if (st != LSTM_OK) return st;
    const ScanPlan& sp = *static_cast<const ScanPlan*>(plan);
    const Plan& p = sp.p;
    const lstm_glr_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    if (!aligned(dh_n, 4) || !aligned(dh0, 4) || !aligned(workspace, 16) || !aligned(scratch, 16) || !right_device(p)) return LSTM_ERR_INVALID_ARG;
    const size_t states = state_bytes(sp, s.num_directions, s.hidden_size);
    if (!same_or_apart(dh_n, dh0, states)) return LSTM_ERR_INVALID_ARG;
    if (p.rows == 0) return pass_through(dh_n, dh0, states, cs);
    if (!workspace || !dy || !aligned(dy, s.dtype == LSTM_BF16 ? 2 : 4) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride) ||
        !good_gates(s, grads->f, grads->z, grads->i, grads->row_stride, grads->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    if (gates->row_stride > kGlrMaxStride || grads->row_stride > kGlrMaxStride) return LSTM_ERR_UNSUPPORTED;
    GlrArgs a = plan_args(sp, s, *gates);
    a.ws = (float*)const_cast<void*>(workspace); a.dy = dy; a.dh_n = dh_n; a.dh0 = dh0;
    a.df = grads->f; a.dz = grads->z; a.di = grads->i; a.gld = grads->row_stride; a.gdstride = grads->dir_stride;
    return launch_glr_bwd(sp, s, a, scratch, cs);
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
        !same_or_apart(state_in, state_out, sizeof(float) * num_slots * s.hidden_size) ||
        !good_gates(s, gates->f, gates->z, gates->i, gates->row_stride, gates->dir_stride))
        return LSTM_ERR_INVALID_ARG;
    GlrArgs a;
    a.H = s.hidden_size;
    a.f = gates->f; a.z = gates->z; a.i = gates->i; a.ld = gates->row_stride; a.y = y;
    const bool whole = fits(state_in, 16) && fits(state_out, 16) && glr_whole(a, s.dtype == LSTM_BF16 ? 2 : 4, 16);
    lstm_status st2 = LSTM_OK;
    dispatch(s, [&](auto* t, auto gated) {
        typedef std::remove_pointer_t<decltype(t)> T;
        constexpr bool G = decltype(gated)::value;
        cudaStream_t cs = (cudaStream_t)stream;
        st2 = whole ? step<T, G, 16 / (int)sizeof(T)>(a, slots, rows, num_slots, state_in, state_out, cs)
                    : step<T, G, 1>(a, slots, rows, num_slots, state_in, state_out, cs);
    });
    return st2;
}

}  // extern "C"
