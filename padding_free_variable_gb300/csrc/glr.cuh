// glr.cuh -- arguments of the gated linear recurrence's kernels and the gate arithmetic they share.
#pragma once

#include <atomic>

#include "scan_plan.cuh"

namespace lstm {

// Everything a launch reads; strides in elements.
struct GlrArgs {
    int T = 0, B = 0, H = 0, ndir = 1;
    int padded = 0;
    int groups = 1;                     // GLR_GROUPED: groups of lanes, each with steps of its own
    const int4* pieces = nullptr;       // this level's
    int piece = 0;                      // its pieces' steps
    int count = 0;                      // and their number
    bool cut = false;                   // do some sequences have several?
    float4* maps = nullptr;             // [piece by slot][ndir][blocks]: each piece's map (cut sequences only)
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

// Two fp32 values in one 64-bit register: add, multiply and multiply-add work on both at once.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ float lo() const { return __uint_as_float((unsigned)v); }
    __device__ __forceinline__ float hi() const { return __uint_as_float((unsigned)(v >> 32)); }
};
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Gates: with e = exp(-x), sig(x) = 1 / (1 + e) and 1 - sig(x) = e / (1 + e).  Both are formed
// from e, neither by subtracting the other from 1, so a gate near 1 keeps the digits of 1 - a and
// one near 0 those of a.  Long products of gates near 1 drift by the mean of the gates' errors:
// measured over a million gates each, 1.6e-8 of the value for x in 0 to 1, 0.9e-8 at most beyond (a
// rounding is up to 6e-8).  1 - a carries the exponential's error, which grows with its argument: mean
// 1.4e-7 for x in 12 to 16.  For the pair e is held below 2^126 (x above -87), where e / (1 + e) is
// still 1 and not inf * 0.
constexpr float kNegLog2e = -1.44269504088896341f;

__device__ __forceinline__ F2 sigmoid2(F2 x)
{
    const F2 t = x * F2(kNegLog2e, kNegLog2e);
    const F2 d = F2(ex2_approx(t.lo()), ex2_approx(t.hi())) + F2(1.f, 1.f);
    return F2(rcp_approx(d.lo()), rcp_approx(d.hi()));
}

// The gate of a state: sig(x), at least 2^-126, so that no gate makes a NaN of an infinite state.
__device__ __forceinline__ F2 forget2(F2 x)
{
    const F2 t = x * F2(kNegLog2e, kNegLog2e);
    const F2 d = F2(ex2_approx(min_nan(t.lo(), 126.f)), ex2_approx(min_nan(t.hi(), 126.f))) + F2(1.f, 1.f);
    return F2(rcp_approx(d.lo()), rcp_approx(d.hi()));
}

__device__ __forceinline__ void sigmoid_pair2(F2 x, F2& s, F2& c)
{
    const F2 t = x * F2(kNegLog2e, kNegLog2e);
    const F2 e = F2(ex2_approx(min_nan(t.lo(), 126.f)), ex2_approx(min_nan(t.hi(), 126.f)));
    const F2 d = e + F2(1.f, 1.f);
    s = F2(rcp_approx(d.lo()), rcp_approx(d.hi()));
    c = e * s;
}

// sig(x) and sig(-x)
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& c)
{
    const float e = ex2_approx(min_nan(x * kNegLog2e, 126.f));
    s = rcp_approx(1.f + e);
    c = e * s;
}

// ---------------------------------------------------------------- rows in and out

// A lane's V neighbouring elements as they lie in memory, in 32-bit words.
template <typename T, int V> struct Raw {
    static constexpr int BYTES = V * (int)sizeof(T), WORDS = BYTES < 4 ? 1 : BYTES / 4;
    unsigned w[WORDS];

    template <typename P> __device__ __forceinline__ void load(P&& word_at, const char* p)
    {
        if constexpr (BYTES == 2) {
            w[0] = word_at((const unsigned short*)p);
        } else if constexpr (BYTES == 4) {
            w[0] = word_at((const unsigned*)p);
        } else {
            const uint2 q = word_at((const uint2*)p);
            w[0] = q.x; w[1] = q.y;
        }
    }
    __device__ __forceinline__ void load_global(const char* p)
    {
        load([](auto* q) { return __ldg(q); }, p);
    }
    __device__ __forceinline__ void load_shared(const char* p)
    {
        load([](auto* q) { return *q; }, p);
    }
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[v]);
        return __uint_as_float(v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
    }
};

template <typename T, int V, typename X> __device__ __forceinline__ void store_values(char* p, const X& x)
{
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 1) *(float*)p = x.get(0);
        else *(float2*)p = make_float2(x.get(0), x.get(1));
    } else {
        if constexpr (V == 1) *(__nv_bfloat16*)p = __float2bfloat16_rn(x.get(0));
        else *(__nv_bfloat162*)p = __floats2bfloat162_rn(x.get(0), x.get(1));
    }
}

__device__ __forceinline__ void cp_async16(void* to, const char* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---------------------------------------------------------------- launch shape

// Largest row stride (elements): strides in bytes stay within 32 bits, their products with a row are 64 bits wide.
constexpr int64_t kGlrMaxStride = 1 << 29;
constexpr int kGlrWarps = 8;            // parts of a CTA's 64 steps, one a warp
constexpr int kGlrSteps = 8;            // consecutive steps of one thread
static_assert(kGlrWarps * kGlrSteps == kScanChunk, "a CTA's iteration is one kept state");

// ---------------------------------------------------------------- affine maps of V units

// Products of gates are held at the smallest normal number (`hold`, before a map is applied or
// passed on): one that underflowed to 0 would make NaN of an infinite state, which frame by frame
// stays infinite.  A finite state h gains at most 2^-126 |h| from it.
constexpr float kLeast = 1.17549435e-38f;

// V values of a lane, in pairs.
template <int V> struct Vals {
    F2 q[V / 2];
    __device__ __forceinline__ float get(int v) const { return v & 1 ? q[v / 2].hi() : q[v / 2].lo(); }
    __device__ __forceinline__ void fill(float x)
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = F2(x, x);
    }
    __device__ __forceinline__ void mad(const Vals& a, const Vals& b)       // a * this + b
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = fma2(a.q[v], q[v], b.q[v]);
    }
    __device__ __forceinline__ void mul(const Vals& a)
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = a.q[v] * q[v];
    }
    __device__ __forceinline__ void add(const Vals& a)
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = q[v] + a.q[v];
    }
    __device__ __forceinline__ void sub(const Vals& a)      // exact negation, one rounding
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = fma2(a.q[v], F2(-1.f, -1.f), q[v]);
    }
    __device__ __forceinline__ void sigmoid()
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = sigmoid2(q[v]);
    }
    __device__ __forceinline__ void forget()
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = forget2(q[v]);
    }
    __device__ __forceinline__ void hold()
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) q[v] = F2(max_nan(q[v].lo(), kLeast), max_nan(q[v].hi(), kLeast));
    }
    __device__ __forceinline__ void sigmoids(Vals& s, Vals& c) const
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) sigmoid_pair2(q[v], s.q[v], c.q[v]);
    }
    __device__ __forceinline__ Vals from(int lane) const
    {
        Vals r;
#pragma unroll
        for (int v = 0; v < V / 2; ++v) r.q[v].v = __shfl_sync(0xffffffffu, q[v].v, lane);
        return r;
    }
    template <typename G> __device__ __forceinline__ void each(G&& value)
    {
#pragma unroll
        for (int v = 0; v < V; v += 2) q[v / 2] = F2(value(v), value(v + 1));
    }
};
template <> struct Vals<1> {
    float q;
    __device__ __forceinline__ float get(int) const { return q; }
    __device__ __forceinline__ void fill(float x) { q = x; }
    __device__ __forceinline__ void mad(const Vals& a, const Vals& b) { q = fmaf(a.q, q, b.q); }
    __device__ __forceinline__ void mul(const Vals& a) { q *= a.q; }
    __device__ __forceinline__ void add(const Vals& a) { q += a.q; }
    __device__ __forceinline__ void sub(const Vals& a) { q -= a.q; }
    __device__ __forceinline__ void sigmoid() { q = rcp_approx(1.f + ex2_approx(q * kNegLog2e)); }
    __device__ __forceinline__ void forget() { q = rcp_approx(1.f + ex2_approx(min_nan(q * kNegLog2e, 126.f))); }
    __device__ __forceinline__ void hold() { q = max_nan(q, kLeast); }
    __device__ __forceinline__ void sigmoids(Vals& s, Vals& c) const { sigmoid_pair(q, s.q, c.q); }
    template <typename G> __device__ __forceinline__ void each(G&& value) { q = value(0); }
};

// h -> A h + U of a warp's 32 V units, in shared memory.
template <int V> struct WarpMap {
    float4 m[V / 2][32];
    __device__ __forceinline__ void put(int lane, const Vals<V>& A, const Vals<V>& U)
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) m[v][lane] = make_float4(A.q[v].lo(), A.q[v].hi(), U.q[v].lo(), U.q[v].hi());
    }
    __device__ __forceinline__ void get(int lane, Vals<V>& A, Vals<V>& U) const
    {
#pragma unroll
        for (int v = 0; v < V / 2; ++v) {
            const float4 x = m[v][lane];
            A.q[v] = F2(x.x, x.y);
            U.q[v] = F2(x.z, x.w);
        }
    }
    __device__ __forceinline__ void apply(int lane, Vals<V>& h) const
    {
        Vals<V> A, U;
        get(lane, A, U);
        h.mad(A, U);
    }
};
template <> struct WarpMap<1> {
    float2 m[32];
    __device__ __forceinline__ void put(int lane, const Vals<1>& A, const Vals<1>& U) { m[lane] = make_float2(A.q, U.q); }
    __device__ __forceinline__ void get(int lane, Vals<1>& A, Vals<1>& U) const { A.q = m[lane].x; U.q = m[lane].y; }
    __device__ __forceinline__ void apply(int lane, Vals<1>& h) const { h.q = fmaf(m[lane].x, h.q, m[lane].y); }
};

// How a kernel takes its rows.
enum GlrRows {
    GLR_WIDE = 0,       // 2 units a lane; rows through shared memory in 16-byte pieces
    GLR_NARROW = 1,     // 4 bytes a lane (2 bf16 units or 1 fp32 unit), each lane its own
    GLR_SINGLE = 2,     // bf16 rows that are not aligned to 4 bytes: 1 unit a lane
    GLR_GROUPED = 3      // as wide rows, of at most 32 units: groups of 16 or 8 lanes take 8 steps each
};

// A warp's rows: 32 V units of each.  Wide rows reach the warp's own part of shared memory by
// cp.async, eight (bf16) or sixteen (fp32) lanes a row, so an address is formed once for several
// rows and not by each lane of each row; the others are loaded by each lane into registers.
template <typename T, int ROWS, int G> struct RowTile {
    static constexpr int S = kGlrSteps;
    static constexpr bool GROUPED = ROWS == GLR_GROUPED;
    static constexpr int V = ROWS == GLR_WIDE || GROUPED ? 2 : ROWS == GLR_NARROW ? 4 / (int)sizeof(T) : 1;
    static constexpr int OWN = V * (int)sizeof(T);              // bytes of a lane's units
    static constexpr int RB = 32 * OWN;                         // bytes of a row
    static constexpr bool STAGED = ROWS == GLR_WIDE || GROUPED;
    // Loads past a piece's end are left out where that gains: they are wasted reads (two sequences of 20 to
    // 30 thousand frames x 512 fp32 backward 137 us with them, 132 us without), but the branch costs the
    // bf16 kernels their schedule (40555 frames x 2 x 512 backward 89 us with them, 101 us without).
    static constexpr bool BOUNDED = GROUPED || sizeof(T) == 4;
    static constexpr int WIDTH = STAGED ? 16 : OWN;             // bytes a lane moves at a time
    static constexpr int LR = RB / WIDTH, RI = 32 / LR;         // lanes of a row, rows of one instruction
    static constexpr int BYTES = G * S * RB;                    // a warp's rows of one stage: [operand][step][RB]

    const char* src[G];
    unsigned ld[G];             // bytes from row to row
    int at;                     // this lane's piece: byte in a staged row
    bool writes;                // is it a piece of the row?
    int lanes = 32;             // of a group
    char* in;                   // this warp's rows of stage 0
    Raw<T, V> raw[STAGED ? 1 : G][STAGED ? 1 : S];

    // lanes past the end of a row (of `end` bytes) read its last piece again: what they compute is not written
    __device__ __forceinline__ void place(int lane, int end, int groups)
    {
        at = lane % LR * WIDTH;
        if (GROUPED) lanes = 32 / groups;
        writes = col() < end;
        const int from = min(col(), end - WIDTH);
#pragma unroll
        for (int x = 0; x < G; ++x) src[x] += from;
    }
    __device__ __forceinline__ int unit_lane(int lane) const { return GROUPED ? lane & (lanes - 1) : lane; }
    __device__ __forceinline__ int group(int lane) const { return GROUPED ? lane / lanes : 0; }
    // the piece's byte in the row in memory (grouped: the groups' rows are staged next to each other)
    __device__ __forceinline__ int col() const { return GROUPED ? at & (lanes * OWN - 1) : at; }
    // the warp's step whose row the piece of staged row k + lane / LR is of
    __device__ __forceinline__ int step(int lane, int k) const { return (GROUPED ? at / (lanes * OWN) * S : 0) + k + lane / LR; }
    // `rows`: lane k holds the packed row of the warp's step k; `any`: is there one to load?
    __device__ __forceinline__ void load(int lane, unsigned rows, int stage, bool any = true)
    {
        if (STAGED && !any) {       // (a branch around loads into registers would wait for them)
            cp_async_commit();
            return;
        }
        char* to = in + stage + lane / LR * RB + at;
#pragma unroll
        for (int k = 0; k < S; k += RI) {
            const unsigned row = __shfl_sync(0xffffffffu, rows, step(lane, k));
#pragma unroll
            for (int x = 0; x < G; ++x) {
                const char* from = src[x] + (uint64_t)row * ld[x];
                if constexpr (STAGED) cp_async16(to + (x * S + k) * RB, from);
                else raw[x][k].load_global(from);
            }
        }
        if (STAGED) cp_async_commit();
    }
    __device__ __forceinline__ Raw<T, V> value(int lane, int x, int k, int stage) const
    {
        if constexpr (!STAGED) return raw[x][k];
        Raw<T, V> r;
        r.load_shared(in + stage + (x * S + k) * RB + lane * OWN);
        return r;
    }
    // The same through shared memory in either case; what `stash` puts there for rows loaded into registers.
    __device__ __forceinline__ char* slot(int lane, int x, int k, int stage) const { return in + stage + (x * S + k) * RB + lane * OWN; }
    __device__ __forceinline__ void stash(int lane) const
    {
        if constexpr (!STAGED) {
#pragma unroll
            for (int x = 0; x < G; ++x)
#pragma unroll
                for (int k = 0; k < S; ++k) {
                    if constexpr (OWN == 2) *(unsigned short*)slot(lane, x, k, 0) = (unsigned short)raw[x][k].w[0];
                    else *(unsigned*)slot(lane, x, k, 0) = raw[x][k].w[0];
                }
        }
    }
    __device__ __forceinline__ Vals<V> held(int lane, int x, int k, int stage) const
    {
        Raw<T, V> r;
        r.load_shared(slot(lane, x, k, stage));
        Vals<V> q;
        q.each([&](int v) { return r.get(v); });
        return q;
    }
    // operand x of two units of step k, or of one unit of steps k and k + 1
    __device__ __forceinline__ F2 two(int lane, int x, int k, int stage) const
    {
        const Raw<T, V> r = value(lane, x, k, stage);
        return F2(r.get(0), V == 1 ? value(lane, x, k + 1, stage).get(0) : r.get(V - 1));
    }
};

GlrRows glr_rows(const GlrArgs& a, int elem);
// Groups of a warp of grouped rows: 64 places by 16 or 32 units.
inline int glr_groups(int H) { return H > 16 ? 2 : 4; }
// Whether to cut sequences into pieces that run side by side, and how long: fills the pieces' fields.
// `ctas` is what an SM holds of the scan kernel, `scratch` the caller's (null: uncut).
void glr_cut(const ScanPlan& p, int V, int ctas, void* scratch, GlrArgs* a);      // (groups set)
size_t glr_scratch(const ScanPlan& p, const lstm_glr_shape& s);
// Every piece of a cut sequence reads the state that comes in, whichever piece writes the one that goes out: where both are
// one array, `in` becomes a copy of it in the scratch.
lstm_status glr_carry(const ScanPlan& p, const GlrArgs& a, const float** in, const float* out, void* scratch, cudaStream_t cs);
// Whether each warp takes a sequence of its own (uncut: fills the pieces' fields).
bool glr_short(const ScanPlan& p, int V, int ctas, GlrArgs* a);

lstm_status launch_glr_fwd(const ScanPlan& p, const lstm_glr_shape& s, GlrArgs a, void* scratch, cudaStream_t cs);
lstm_status launch_glr_bwd(const ScanPlan& p, const lstm_glr_shape& s, GlrArgs a, void* scratch, cudaStream_t cs);

// One launch of `fn` over all pieces, directions and blocks of units: an item a CTA, or (WARPS, the
// kernel then takes their number too) an item a warp.  `ready`: a bit for each device whose
// shared-memory limit is raised.
template <bool WARPS = false, typename F>
lstm_status glr_launch(const Plan& p, F* fn, const GlrArgs& a, int V, size_t smem, std::atomic<uint64_t>& ready, cudaStream_t cs)
{
    const int64_t items = (int64_t)ceil_div(a.H, 32 * V) * a.ndir * a.count;
    if (items > INT32_MAX - kGlrWarps) return LSTM_ERR_UNSUPPORTED;
    const uint64_t bit = 1ull << (p.device & 63);
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        LSTM_CUDA_TRY(cudaFuncSetAttribute((const void*)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (p.device < 64) ready.fetch_or(bit, std::memory_order_release);
    }
    if constexpr (WARPS) fn<<<(unsigned)((items + kGlrWarps - 1) / kGlrWarps), 32 * kGlrWarps, smem, cs>>>(a, (int)items);
    else fn<<<(unsigned)items, 32 * kGlrWarps, smem, cs>>>(a);
    trace_end(p, -1, cs, 1);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

// Where a CTA works: blocks of a row next to each other, then directions, then pieces.
struct Place {
    int u0, block, d, j, len, piece, first;     // first: the slot's first piece among the level's by slot
    __device__ __forceinline__ Place(const GlrArgs& p, int item, int units)
    {
        const int blocks = (p.H + units - 1) / units;
        block = item % blocks;
        u0 = block * units;
        item /= blocks;
        d = item % p.ndir;
        const int4 q = __ldg(p.pieces + item / p.ndir);
        j = q.x; piece = q.y; len = q.z; first = q.w;
    }
    // the map of this slot's piece k
    template <int V> __device__ __forceinline__ WarpMap<V>* map(const GlrArgs& p, int k) const
    {
        const int blocks = (p.H + 32 * V - 1) / (32 * V);
        return (WarpMap<V>*)p.maps + ((int64_t)(first + k) * p.ndir + d) * blocks + block;
    }
    // packed row of step s + lane % 8 of the direction's order (of the last step, past the end); the
    // next group of 8 is `gap` steps on
    __device__ __forceinline__ unsigned row_of(const GlrArgs& p, int s, int lane, int gap) const
    {
        s = max(0, min(s + lane % kGlrSteps + lane / kGlrSteps * gap, len - 1));
        return (unsigned)(__ldg(p.off + (d ? len - 1 - s : s)) + j);
    }
};

// Maps of a warp's groups of lanes (`lanes` each), composed over the groups up to (UP) or from each one's: what a group's
// own comes to behind (before) the others.  The total is the last (first) group's.
template <bool UP, int V> __device__ __forceinline__ void compose_groups(int lane, int lanes, Vals<V>& A, Vals<V>& U)
{
    for (int o = lanes; o < 32; o *= 2) {
        const Vals<V> a = A.from(UP ? lane - o : lane + o);
        Vals<V> u = U.from(UP ? lane - o : lane + o);
        if (UP ? lane < o : lane + o >= 32) continue;
        u.mad(A, U);
        U = u;
        A.mul(a);
        A.hold();
    }
}

template <int V> __device__ __forceinline__ void identity(Vals<V>& A, Vals<V>& U)
{
    A.fill(1.f);
    U.fill(0.f);
}

}  // namespace lstm
