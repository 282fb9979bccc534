// la.cu -- linear attention with a decay for each head: entry points, single frames, starts of cut sequences' pieces.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "la.cuh"

namespace lstm {

namespace {

// ---------------------------------------------------------------- single frames

struct StepArgs {
    LaRows q, k, v;
    const float* log_decay;
    const int32_t* slots;
    const float* in;
    float* out;
    void* y;
    float scale;
    int heads, a, b, rows, num_slots;
};

template <typename T, int V> struct StepValues { float e[V]; };

template <typename T, int V>
__device__ __forceinline__ StepValues<T, V> step_load(const T* p)
{
    StepValues<T, V> r;
    if constexpr (V == 1) {
        r.e[0] = to_f32(p[0]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 x = *(const float4*)p;
        r.e[0] = x.x; r.e[1] = x.y; r.e[2] = x.z; r.e[3] = x.w;
    } else {
        const uint2 x = *(const uint2*)p;
        r.e[0] = __uint_as_float(x.x << 16); r.e[1] = __uint_as_float(x.x & 0xffff0000u);
        r.e[2] = __uint_as_float(x.y << 16); r.e[3] = __uint_as_float(x.y & 0xffff0000u);
    }
    return r;
}

// A block takes one head of one stream: threads along the state's columns (V a thread) and, as many as are left, along
// its rows; each reads its part of the state once, writes it once and adds up its share of y; the shares meet in shared
// memory.  Bound by the states, 8 a b bytes a head: 997 streams of 8 heads of 128 x 128 201 us (5.3 TB/s, 78 % of the copy
// rate), 8 streams of 8 heads of 64 x 64 a launch.
template <typename T, int V>
__global__ void __launch_bounds__(256) la_step_kernel(const StepArgs p)
{
    extern __shared__ float sums[];                 // [row groups][b]
    const int64_t r = blockIdx.x / p.heads;
    const int h = blockIdx.x - (int)r * p.heads, b = p.b, a = p.a;
    const int cols = (b + V - 1) / V, col = threadIdx.x % cols, group = threadIdx.x / cols, groups = blockDim.x / cols;
    T* const y = (T*)p.y + (r * p.heads + h) * b;
    const int slot = p.slots ? __ldg(p.slots + r) : (int)r;
    if (slot < 0 || slot >= p.num_slots) {
        for (int i = threadIdx.x; i < b; i += blockDim.x) y[i] = (T)0.f;
        return;
    }
    float acc[V] = {};
    if (group < groups) {
        const float lam = exp2f(fminf(fmaxf(__ldg(p.log_decay + h), -138.f), 0.f) * 1.4426950408889634f);
        const T* const q = (const T*)p.q.p + r * p.q.row + h * p.q.head;
        const T* const k = (const T*)p.k.p + r * p.k.row + h * p.k.head;
        const StepValues<T, V> v = step_load<T, V>((const T*)p.v.p + r * p.v.row + h * p.v.head + col * V);
        const int64_t at = ((int64_t)slot * p.heads + h) * a * b + col * V;
        const float* const in = p.in + at;
        float* const out = p.out + at;
#pragma unroll 8
        for (int x = group; x < a; x += groups) {
            const StepValues<float, V> s = step_load<float, V>(in + (int64_t)x * b);
            const float kx = to_f32(k[x]), qx = to_f32(q[x]);
            float n[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                n[e] = fmaf(kx, v.e[e], lam * s.e[e]);
                acc[e] = fmaf(qx, n[e], acc[e]);
            }
            if constexpr (V == 4) {
                *(float4*)(out + (int64_t)x * b) = make_float4(n[0], n[1], n[2], n[3]);
            } else {
                out[(int64_t)x * b] = n[0];
            }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sums[group * b + col * V + e] = acc[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < b; i += blockDim.x) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += sums[g * b + i];
        s *= p.scale;
        if constexpr (sizeof(T) == 4) y[i] = s;
        else y[i] = __float2bfloat16_rn(s);
    }
}

template <typename T, int V>
lstm_status step(const StepArgs& a, cudaStream_t cs)
{
    const int cols = ceil_div(a.b, V), groups = std::max(1, std::min(256 / cols, a.a));
    const int threads = ceil_div(cols * groups, 32) * 32;
    const int64_t blocks = (int64_t)a.rows * a.heads;
    if (blocks > INT32_MAX) return LSTM_ERR_UNSUPPORTED;
    la_step_kernel<T, V><<<(unsigned)blocks, threads, sizeof(float) * (threads / cols) * a.b, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

// ---------------------------------------------------------------- starts of pieces

// Y in front of each piece of a cut sequence from what each piece adds to it, in place: a thread a value, 16 pieces' values on
// their way while 16 are written (128 pieces of 8 states of 128 x 128 29 us, 4.7 TB/s; 8 at a time without reading ahead 93 us).
__global__ void __launch_bounds__(256) la_starts_kernel(const LaArgs p)
{
    const LaJob& j = p.job[blockIdx.z];
    const int dhs = p.ndir * p.heads, dh = blockIdx.x % dhs, slot = blockIdx.x / dhs, d = dh / p.heads, h = dh - d * p.heads;
    const int4 e = __ldg(p.pieces + slot);
    const int pieces = max(1, (int)(((int64_t)e.z + p.piece - 1) / p.piece)), size = j.a * j.b;
    const int i = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= size) return;
    const float l2 = la_log2_decay(p, d, h), keep = exp2f(l2 * p.piece);
    float y = 0.f;
    if (j.init) {
        const int x = i / j.b, c = i - x * j.b;
        const float* s = j.init + (((int64_t)d * p.B + __ldg(p.perm + slot)) * p.heads + h) * size;
        y = (j.early ? exp2f(l2) : 1.f) * s[j.flip ? c * j.a + x : i];
    }
    float* at = j.starts + ((int64_t)e.w * dhs + dh) * size + i;
    const int64_t step = (int64_t)dhs * size;
    // 16 pieces at a time, the next 16 read before these are written
    float add[16], next[16];
#pragma unroll
    for (int o = 0; o < 16; ++o) add[o] = o < pieces - 1 ? at[o * step] : 0.f;
    for (int n = 0; n < pieces; n += 16) {
#pragma unroll
        for (int o = 0; o < 16; ++o) next[o] = n + 16 + o < pieces - 1 ? at[(n + 16 + o) * step] : 0.f;
#pragma unroll
        for (int o = 0; o < 16; ++o) {
            if (n + o < pieces) at[(n + o) * step] = y;
            y = fmaf(keep, y, add[o]);
            add[o] = next[o];
        }
    }
}

// ---------------------------------------------------------------- checks

lstm_status check_shape(const lstm_la_shape* s)
{
    if (!s || s->num_heads < 1 || s->key_size < 1 || s->value_size < 1) return LSTM_ERR_INVALID_ARG;
    if (s->num_directions != 1 && s->num_directions != 2) return LSTM_ERR_INVALID_ARG;
    if ((s->dtype != LSTM_F32 && s->dtype != LSTM_BF16) || !std::isfinite(s->scale)) return LSTM_ERR_INVALID_ARG;
    if (s->key_size > kLaMax || s->value_size > kLaMax || s->num_heads > 4096) return LSTM_ERR_UNSUPPORTED;
    return LSTM_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool good_rows(const lstm_la_rows& r, size_t e)
{
    return r.ptr && aligned(r.ptr, e) && r.row_stride >= 0 && r.dir_stride >= 0 && r.head_stride >= 0 && r.row_stride <= (1ll << 40) &&
           r.dir_stride <= (1ll << 40) && r.head_stride <= (1ll << 40);
}

bool good_inputs(const lstm_la_shape& s, const lstm_la_inputs& in)
{
    const size_t e = s.dtype == LSTM_BF16 ? 2 : 4;
    return good_rows(in.q, e) && good_rows(in.k, e) && good_rows(in.v, e);
}

// Written rows: no two values at one place.  Dimensions by their strides, each at least what the ones inside it span.
bool apart(const lstm_la_grad_rows& r, int64_t rows, int ndir, int heads, int width, size_t e)
{
    if (!r.ptr || !aligned(r.ptr, e)) return false;
    struct { int64_t n, step; } d[3] = {{rows, r.row_stride}, {ndir, r.dir_stride}, {heads, r.head_stride}};
    std::sort(d, d + 3, [](auto& x, auto& y) { return x.step < y.step; });
    int64_t span = width;
    for (auto& x : d) {
        if (x.n <= 1) continue;
        if (x.step < span || x.step > (1ll << 40)) return false;
        span += (x.n - 1) * x.step;
    }
    return true;
}

bool right_device(const Plan& p)
{
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == p.device;
}

bool same_or_apart(const float* in, const float* out, size_t bytes)
{
    const uintptr_t a = (uintptr_t)in, b = (uintptr_t)out;
    return !in || !out || in == out || a + bytes <= b || b + bytes <= a;
}

size_t state_bytes(const Plan& p, const lstm_la_shape& s)
{
    return sizeof(float) * s.num_directions * p.B * s.num_heads * s.key_size * s.value_size;
}

LaRows rows_of(const lstm_la_rows& r)
{
    LaRows o;
    o.p = r.ptr; o.row = r.row_stride; o.dir = r.dir_stride; o.head = r.head_stride;
    return o;
}

LaRows rows_of(const lstm_la_grad_rows& r)
{
    LaRows o;
    o.p = r.ptr; o.row = r.row_stride; o.dir = r.dir_stride; o.head = r.head_stride;
    return o;
}

// y and dy: [rows][ndir][heads][value_size]
LaRows dense_rows(const void* p, const lstm_la_shape& s)
{
    LaRows o;
    o.p = p; o.head = s.value_size; o.dir = o.head * s.num_heads; o.row = o.dir * s.num_directions;
    return o;
}

// The level of the plan's pieces that `jobs` walks of every sequence run over (the last one: uncut).  A sequence is walked
// chunk by chunk; where the longest one runs far past an even share of all steps for the CTAs that the GPU holds, sequences
// are cut, and every piece's keys and values are read once more for what it adds to the state.  One sequence of 65536 steps of 8
// heads of 128 bf16 values: pieces of an eighth of a share or more 401 us (390 by now), of a quarter 413, of a sixteenth 451, uncut 3424; two
// of 29008 steps together, 8 heads of 32 + 64 fp32 values, forward / backward 226 / 579 us, uncut 1880 / 1951.  Just past the rule's
// edge both are alike or cutting loses: 37 sequences of up to 700 steps, 2 x 3 heads of 37 + 53 fp32 values, 122 and 123 us; 24
// of 200 to 2400 steps, 8 heads of 64 bf16 values, 112 and 100 us.
int cut_level(const ScanPlan& sp, const lstm_la_shape& s, int jobs)
{
    const bool bf16 = s.dtype == LSTM_BF16, wide = s.key_size > 64 || s.value_size > 64;
    const int64_t slots = (int64_t)sp.p.num_sms * (bf16 ? wide ? 1 : 2 : wide ? 1 : 3), each = (int64_t)s.num_directions * s.num_heads * jobs;
    const int64_t share = (sp.p.padded ? sp.p.frames : sp.p.rows) * each / slots;
    const int whole = sp.scan.levels - 1;
    if (sp.p.T <= share * 2 + 3 * kScanPiece) return whole;
    for (int l = 0; l < whole; ++l)
        if (((int64_t)kScanPiece << l) * 8 >= share) return l;
    return whole;
}

size_t start_bytes(const ScanPlan& sp, const lstm_la_shape& s, int level)
{
    if (level >= sp.scan.levels - 1) return 0;
    return sizeof(float) * sp.scan.level_count[level] * s.num_directions * s.num_heads * s.key_size * s.value_size;
}

LaArgs plan_args(const ScanPlan& sp, const lstm_la_shape& s, const float* log_decay, int level)
{
    const Plan& p = sp.p;
    LaArgs a;
    a.heads = s.num_heads; a.ndir = s.num_directions; a.B = p.B; a.T = p.T; a.padded = p.padded ? 1 : 0;
    a.off = p.d_off; a.perm = p.d_perm; a.log_decay = log_decay;
    a.pieces = sp.scan.d_pieces + sp.scan.level_first[level];
    a.count = sp.scan.level_count[level];
    a.piece = level < sp.scan.levels - 1 ? kScanPiece << level : INT32_MAX;
    a.status = p.d_status; a.limit_ns = p.wait_limit_ns; a.sms = p.num_sms; a.rows = p.rows;
    return a;
}

// The walks of `a`; cut sequences' starts are found first, by those of its jobs that have starts of their own.
lstm_status run_jobs(const LaArgs& a, const lstm_la_shape& s, cudaStream_t cs)
{
    if ((int64_t)a.count * a.ndir * a.heads * a.jobs > INT32_MAX) return LSTM_ERR_UNSUPPORTED;
    const bool bf16 = s.dtype == LSTM_BF16, tensor = bf16 && la_tensor_fits(a);
    auto launch = [&](const LaArgs& b, bool states) { return tensor ? launch_la_tensor(b, states, cs) : launch_la_general(b, bf16, states, cs); };
    if (a.job[0].starts) {
        LaArgs first = a;
        first.jobs = 0;
        for (int k = 0; k < a.jobs; ++k)
            if (!a.job[k].flip_starts) first.job[first.jobs++] = a.job[k];
        const lstm_status st = launch(first, true);
        if (st != LSTM_OK) return st;
        const dim3 grid((unsigned)(a.B * a.ndir * a.heads), ceil_div(s.key_size * s.value_size, 256), first.jobs);
        la_starts_kernel<<<grid, 256, 0, cs>>>(first);
        if (cudaGetLastError() != cudaSuccess) return LSTM_ERR_CUDA;
    }
    return launch(a, false);
}

lstm_status pass_through(const float* in, float* out, size_t bytes, cudaStream_t cs)
{
    if (!out || out == in) return LSTM_OK;
    LSTM_CUDA_TRY(in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, cs) : cudaMemsetAsync(out, 0, bytes, cs));
    return LSTM_OK;
}

}  // namespace

}  // namespace lstm

using namespace lstm;

extern "C" {

size_t lstm_la_scratch_bytes(const lstm_plan* plan, const lstm_la_shape* shape)
{
    if (!plan || check_shape(shape) != LSTM_OK) return 0;
    const ScanPlan& sp = *static_cast<const ScanPlan*>(plan);
    return std::max(start_bytes(sp, *shape, cut_level(sp, *shape, 1)), 2 * start_bytes(sp, *shape, cut_level(sp, *shape, 3)));
}

lstm_status lstm_la_fwd(const lstm_plan* plan, const lstm_la_shape* shape, const lstm_la_inputs* in,
                        const float* log_decay, const float* s0, void* y, float* s_n, void* scratch, void* stream)
{
    if (!plan || !in) return LSTM_ERR_INVALID_ARG;
    const lstm_status st = check_shape(shape);
    if (st != LSTM_OK) return st;
    const ScanPlan& sp = *static_cast<const ScanPlan*>(plan);
    const lstm_la_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    const size_t states = state_bytes(sp.p, s);
    if (!aligned(s0, 4) || !aligned(s_n, 4) || !aligned(scratch, 16) || !right_device(sp.p) || !same_or_apart(s0, s_n, states))
        return LSTM_ERR_INVALID_ARG;
    if (sp.p.rows == 0) return pass_through(s0, s_n, states, cs);
    if (!y || !aligned(y, s.dtype == LSTM_BF16 ? 2 : 4) || !log_decay || !aligned(log_decay, 4) || !good_inputs(s, *in))
        return LSTM_ERR_INVALID_ARG;
    if (sp.p.T > kLaMaxSteps) return LSTM_ERR_UNSUPPORTED;
    const int level = scratch ? cut_level(sp, s, 1) : sp.scan.levels - 1;
    LaArgs a = plan_args(sp, s, log_decay, level);
    a.jobs = 1;
    LaJob& j = a.job[0];
    j.q = rows_of(in->q); j.k = rows_of(in->k); j.v = rows_of(in->v); j.out = dense_rows(y, s);
    j.a = s.key_size; j.b = s.value_size;
    j.init = s0; j.fin = s_n; j.early = 1;
    j.sP = j.sI = s.scale;
    j.starts = level < sp.scan.levels - 1 ? (float*)scratch : nullptr;
    return run_jobs(a, s, cs);
}

lstm_status lstm_la_bwd(const lstm_plan* plan, const lstm_la_shape* shape, const lstm_la_inputs* in,
                        const float* log_decay, const float* s0, const void* dy, const float* ds_n,
                        const lstm_la_grads* grads, float* ds0, void* scratch, void* stream)
{
    if (!plan || !in || !grads) return LSTM_ERR_INVALID_ARG;
    const lstm_status st = check_shape(shape);
    if (st != LSTM_OK) return st;
    const ScanPlan& sp = *static_cast<const ScanPlan*>(plan);
    const lstm_la_shape& s = *shape;
    cudaStream_t cs = (cudaStream_t)stream;
    const size_t states = state_bytes(sp.p, s), e = s.dtype == LSTM_BF16 ? 2 : 4;
    if (!aligned(s0, 4) || !aligned(ds_n, 4) || !aligned(ds0, 4) || !aligned(scratch, 16) || !right_device(sp.p) ||
        !same_or_apart(ds_n, ds0, states))
        return LSTM_ERR_INVALID_ARG;
    if (sp.p.rows == 0) return pass_through(ds_n, ds0, states, cs);
    if (!dy || !aligned(dy, e) || !log_decay || !aligned(log_decay, 4) || !good_inputs(s, *in) ||
        !apart(grads->dq, sp.p.rows, s.num_directions, s.num_heads, s.key_size, e) ||
        !apart(grads->dk, sp.p.rows, s.num_directions, s.num_heads, s.key_size, e) ||
        !apart(grads->dv, sp.p.rows, s.num_directions, s.num_heads, s.value_size, e))
        return LSTM_ERR_INVALID_ARG;
    if (sp.p.T > kLaMaxSteps) return LSTM_ERR_UNSUPPORTED;
    const int level = scratch ? cut_level(sp, s, 3) : sp.scan.levels - 1;
    LaArgs a = plan_args(sp, s, log_decay, level);
    const LaRows q = rows_of(in->q), k = rows_of(in->k), v = rows_of(in->v), g = dense_rows(dy, s);
    const size_t starts = start_bytes(sp, s, level);
    a.jobs = 3;
    LaJob &jv = a.job[0], &jk = a.job[1], &jq = a.job[2];
    jq.q = g; jq.k = v; jq.v = k; jq.out = rows_of(grads->dq);
    jq.a = s.value_size; jq.b = s.key_size; jq.init = s0; jq.flip = 1; jq.early = 1; jq.sP = jq.sI = s.scale; jq.pieces = 2;
    jk.q = v; jk.k = g; jk.v = q; jk.out = rows_of(grads->dk);
    jk.a = s.value_size; jk.b = s.key_size; jk.init = ds_n; jk.flip = 1; jk.back = 1; jk.sP = jk.sK = s.scale; jk.pieces = 2;
    jv.q = k; jv.k = q; jv.v = g; jv.out = rows_of(grads->dv);
    jv.a = s.key_size; jv.b = s.value_size; jv.init = ds_n; jv.back = 1; jv.sP = jv.sK = s.scale; jv.fin = ds0;
    if (starts) {
        // the errors in front of dk's pieces are dv's, transposed
        jv.starts = jk.starts = (float*)scratch;
        jk.flip_starts = 1;
        jq.starts = (float*)((char*)scratch + starts);
    }
    if (!starts && ds0 && ds0 == ds_n) {
        // dk reads the errors that dv's walk overwrites: it goes first (cut sequences read them before either walk)
        LaArgs first = a;
        first.jobs = 2;
        first.job[0] = jk;
        first.job[1] = jq;
        const lstm_status st1 = run_jobs(first, s, cs);
        if (st1 != LSTM_OK) return st1;
        a.jobs = 1;
    }
    return run_jobs(a, s, cs);
}

lstm_status lstm_la_step(const lstm_la_shape* shape, const lstm_la_inputs* in, const float* log_decay,
                         int32_t rows, const int32_t* slots, int32_t num_slots, const float* state_in,
                         float* state_out, void* y, void* stream)
{
    const lstm_status st = check_shape(shape);
    if (st != LSTM_OK) return st;
    const lstm_la_shape& s = *shape;
    if (!in || rows < 0 || num_slots < 0 || s.num_directions != 1 || (!slots && num_slots < rows)) return LSTM_ERR_INVALID_ARG;
    if (rows == 0) return LSTM_OK;
    const size_t e = s.dtype == LSTM_BF16 ? 2 : 4;
    if (!y || !aligned(y, e) || !log_decay || !aligned(log_decay, 4) || !aligned(slots, 4) || !aligned(state_in, 4) ||
        !aligned(state_out, 4) || (num_slots > 0 && (!state_in || !state_out)) ||
        !same_or_apart(state_in, state_out, sizeof(float) * num_slots * s.num_heads * s.key_size * s.value_size) || !good_inputs(s, *in))
        return LSTM_ERR_INVALID_ARG;
    StepArgs a;
    a.q = rows_of(in->q); a.k = rows_of(in->k); a.v = rows_of(in->v);
    a.log_decay = log_decay; a.slots = slots; a.in = state_in; a.out = state_out; a.y = y; a.scale = s.scale;
    a.heads = s.num_heads; a.a = s.key_size; a.b = s.value_size; a.rows = rows; a.num_slots = num_slots;
    const bool whole = s.value_size % 4 == 0 && aligned(state_in, 16) && aligned(state_out, 16) && aligned(a.v.p, 4 * e) &&
                       a.v.row % 4 == 0 && a.v.head % 4 == 0;
    cudaStream_t cs = (cudaStream_t)stream;
    if (s.dtype == LSTM_BF16) return whole ? step<__nv_bfloat16, 4>(a, cs) : step<__nv_bfloat16, 1>(a, cs);
    return whole ? step<float, 4>(a, cs) : step<float, 1>(a, cs);
}

}  // extern "C"
