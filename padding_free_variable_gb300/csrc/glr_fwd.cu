// glr_fwd.cu -- forward scan of the gated linear recurrence.
//
// h_t = a_t h_{t-1} + b_t is a composition of affine maps (A, U): h -> A h + U, and maps compose
// associatively, (A2, U2) after (A1, U1) = (A1 A2, A2 U1 + U2).  Each warp of a CTA holds 8
// consecutive steps of 32 V units (a lane V units) in registers, so every gate is read once and y
// written once.  A thread composes its 8 maps and puts the result in shared memory; the state
// before its next 8 steps is the one after its last 8, taken through the maps in between, so no
// thread carries more than its own state and an iteration needs one barrier.  Every order is
// fixed by the shape and the plan: the result does not depend on timing.
//
// Why so: about ten operations and two transcendentals a unit against 6 to 16 bytes, so memory is
// the bound once T steps do not run one after another (a thread a unit did: 40555 frames of 2 x 512
// bf16 units, three gates, 1084 us; here 66 us).  8 warps by 8 steps: 16 values of a thread fit the
// registers with three CTAs an SM.  Measured, forward, cold L2: 70 k frames of 2 x 256 fp32 units, three
// gates, 91 us, 6.3 TB/s (95 % of the copy rate); 40555 frames of 2 x 512 bf16 units three gates 66 us,
// 5.5 TB/s, two gates 52 us, 5.3 TB/s.  fp32 is at the memory's rate; bf16 halves the bytes but not the
// instructions, and the schedulers issue in 62 % of their cycles.
#include "glr.cuh"

namespace lstm {

namespace {

// Gates of 8 steps -> their maps a, b; the identity for steps past the end.
template <typename Tile, bool GATED>
__device__ __forceinline__ void step_maps(const Tile& t, int lane, int stage, int left, Vals<Tile::V> (&a)[kGlrSteps],
                                          Vals<Tile::V> (&b)[kGlrSteps])
{
    constexpr int S = kGlrSteps, V = Tile::V;
#pragma unroll
    for (int k = 0; k < S; k += V == 1 ? 2 : 1) {
        F2 s, c;
        if (GATED) {
            s = forget2(t.two(lane, 0, k, stage));
            c = sigmoid2(t.two(lane, 2, k, stage));
        } else {
            sigmoid_pair2(t.two(lane, 0, k, stage), s, c);
        }
        c = c * t.two(lane, 1, k, stage);
        if constexpr (V == 1) {
            a[k].q = s.lo(); a[k + 1].q = s.hi();
            b[k].q = c.lo(); b[k + 1].q = c.hi();
        } else {
            a[k].q[0] = s;
            b[k].q[0] = c;
        }
    }
    if (left < S) {
        Vals<V> one, zero;
        one.fill(1.f);
        zero.fill(0.f);
#pragma unroll
        for (int k = 0; k < S; ++k)
            if (k >= left) { a[k] = one; b[k] = zero; }
    }
}

template <int V> __device__ __forceinline__ void compose(const Vals<V> (&a)[kGlrSteps], const Vals<V> (&b)[kGlrSteps], Vals<V>& A, Vals<V>& U)
{
    A = a[0];
    U = b[0];
#pragma unroll
    for (int k = 1; k < kGlrSteps; ++k) {
        U.mad(a[k], b[k]);
        A.mul(a[k]);
    }
    A.hold();
}

// 8 rows of y that a warp has staged at `out` ([step][RB]), to memory in 16-byte pieces.
template <typename Tile> __device__ __forceinline__ void flush_rows(const Tile& t, const char* out, int lane, char* y, unsigned yld, unsigned rows, int n)
{
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kGlrSteps; k += Tile::RI) {
        const int s = t.step(lane, k);
        const unsigned row = __shfl_sync(0xffffffffu, rows, s);
        const uint4 q = *(const uint4*)(out + (k + lane / Tile::LR) * Tile::RB + t.at);
        if (s < n) *(uint4*)(y + (uint64_t)row * yld) = q;
    }
}

template <typename T, int ROWS, int G> __device__ __forceinline__ RowTile<T, ROWS, G> gate_rows(const GlrArgs& p, const Place& c, int lane)
{
    RowTile<T, ROWS, G> t;
    const int64_t from = (c.d * p.dstride + c.u0) * (int64_t)sizeof(T);
    t.src[0] = (const char*)p.f + from;
    t.src[1] = (const char*)p.z + from;
    if (G == 3) t.src[G - 1] = (const char*)p.i + from;
#pragma unroll
    for (int x = 0; x < G; ++x) t.ld[x] = (unsigned)p.ld * (unsigned)sizeof(T);
    t.place(lane, (p.H - c.u0) * (int)sizeof(T), p.groups);
    return t;
}

// Rows of y past a sequence's end in the padded comparator's layout.
template <typename T, int WIDTH> __device__ void zero_past_end(const GlrArgs& p, const Place& c, char* y, unsigned yld, int first, int step)
{
    for (int t = c.len + first; t < p.T; t += step)
        for (int x = 0; x < WIDTH; x += (int)sizeof(T)) *(T*)(y + (uint64_t)(p.off[t] + c.j) * yld + x) = from_f32<T>(0.f);
}

// ---------------------------------------------------------------- a CTA a sequence

template <typename T, bool GATED, int ROWS> struct FwdTile : RowTile<T, ROWS, GATED ? 3 : 2> {
    typedef RowTile<T, ROWS, GATED ? 3 : 2> R;
    static constexpr int W = kGlrWarps;
    static constexpr int OUT = R::STAGED ? W * R::S * R::RB : 0;
    static constexpr int MAPS = 3 * W * (int)sizeof(WarpMap<R::V>);
    // CTAs an SM holds: three within 80 registers a thread (bf16 measured 8 to 13 % faster than
    // with two); staged fp32 rows leave shared memory for two
    static constexpr int CTAS = R::STAGED && sizeof(T) == 4 ? 2 : 3;
    static constexpr int STAGE = R::STAGED ? W * R::BYTES : 0;
    static constexpr int FIT = (227 * 1024 / CTAS - 1024 - OUT - MAPS) / (STAGE + 1);
    static constexpr int NS = !R::STAGED || FIT < 1 ? 1 : FIT > 2 ? 2 : FIT;
    static constexpr int SMEM = NS * STAGE + OUT + MAPS;
};

template <typename T, bool GATED, int ROWS> struct MapTile : RowTile<T, ROWS, GATED ? 3 : 2> {
    typedef RowTile<T, ROWS, GATED ? 3 : 2> R;
    static constexpr int W = kGlrWarps;
    static constexpr int STAGE = R::STAGED ? W * R::BYTES : 0;
    static constexpr int FIT = 72 * 1024 / (STAGE + 1);
    static constexpr int NS = !R::STAGED ? 1 : FIT < 2 ? 2 : FIT > 4 ? 4 : FIT;
    static constexpr int SMEM = NS * STAGE;
};

template <typename T, bool GATED, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, FwdTile<T, GATED, ROWS>::CTAS) glr_fwd_kernel(const GlrArgs p)
{
    typedef FwdTile<T, GATED, ROWS> C;
    constexpr int S = C::S, W = C::W, V = C::V, NS = C::NS;
    extern __shared__ __align__(128) char smem[];
    WarpMap<V>* const s_map = (WarpMap<V>*)(smem + NS * C::STAGE + C::OUT);
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    // cut sequences: the pieces whose maps were formed last are the ones still in L2
    const Place c(p, p.cut ? gridDim.x - 1 - blockIdx.x : blockIdx.x, 32 * V);
    auto tile = gate_rows<T, ROWS, GATED ? 3 : 2>(p, c, lane);
    // (grouped: groups of lanes hold the same units, a group's 8 steps after the other's)
    constexpr int GAP = C::GROUPED ? S : 0;
    const int groups = C::GROUPED ? p.groups : 1, g = tile.group(lane), ul = tile.unit_lane(lane), chunk = groups * kScanChunk;
    const int u = c.u0 + ul * V, len = c.len;
    const bool live = u < p.H;
    const int64_t state = ((int64_t)c.d * p.B + p.perm[c.j]) * p.H + u;
    tile.in = smem + w * C::BYTES;
    char* const out = smem + NS * C::STAGE + w * (S * C::RB);
    const unsigned yld = (unsigned)(p.ndir * p.H) * (unsigned)sizeof(T);
    char* y = (char*)p.y + ((int64_t)c.d * p.H + c.u0) * (int64_t)sizeof(T) + tile.col();
    Vals<V> h;
    h.each([&](int v) { return live && p.h0 ? p.h0[state + v] : 0.f; });
    const int begin = c.piece * (p.cut ? p.piece : 0), end = p.cut ? min(len, begin + p.piece) : len;

    if (len > 0) {
        int s0 = begin + w * S * groups;
        unsigned rows[NS + 2];          // of the iterations from this one on
#pragma unroll
        for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, s0 + q * chunk, lane, GAP);
#pragma unroll
        for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::STAGE, !C::BOUNDED || begin + q * chunk < end);
        // maps of this iteration and of the one before (nothing, at first); a third set, as a warp
        // may write the next iteration's while another still reads these two
        WarpMap<V>*now = s_map, *before = s_map + 2 * W;
        Vals<V> A, U;
        if (c.piece > 0) {
            // the state before this piece: the earlier pieces' maps, an eighth of them composed by each warp
            identity(A, U);
            const int share = (c.piece + W - 1) / W, last = min(c.piece, (w + 1) * share);
#pragma unroll 4
            for (int k = w * share; k < last; ++k) {
                Vals<V> a, b;
                c.map<V>(p, k)->get(ul, a, b);
                U.mad(a, b);
                A.mul(a);
            }
            A.hold();
            now[w].put(ul, A, U);
            __syncthreads();
#pragma unroll
            for (int x = 0; x < W; ++x) now[x].apply(ul, h);
        }
        identity(A, U);
        before[w].put(ul, A, U);
        __syncthreads();
        int stage = 0;
        for (int base = begin; base < end; base += chunk, s0 += chunk) {
            const int mine = s0 + g * S;
            Vals<V> a[S], b[S];
            if (C::STAGED) {
                cp_async_wait<NS - 1>();
                __syncwarp();
            }
            step_maps<RowTile<T, ROWS, GATED ? 3 : 2>, GATED>(tile, lane, stage, len - mine, a, b);
            if (C::STAGED) __syncwarp();
            tile.load(lane, rows[NS], stage, !C::BOUNDED || base + NS * chunk < end);
            stage = stage == (NS - 1) * C::STAGE ? 0 : stage + C::STAGE;
            const unsigned rows_now = rows[0];
#pragma unroll
            for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
            rows[NS + 1] = c.row_of(p, s0 + (NS + 2) * chunk, lane, GAP);
            compose<V>(a, b, A, U);
            if constexpr (C::GROUPED) {
                compose_groups<true>(lane, tile.lanes, A, U);
                if (g == groups - 1) now[w].put(ul, A, U);
                A = A.from(lane - tile.lanes);      // of the groups before this one
                U = U.from(lane - tile.lanes);
                if (g == 0) identity(A, U);
            } else {
                now[w].put(lane, A, U);
            }
            __syncthreads();
#pragma unroll
            for (int x = 1; x < W; ++x) (w + x < W ? before + w + x : now + w + x - W)->apply(ul, h);
            if constexpr (C::GROUPED) h.mad(A, U);
            before = now;
            now = now == s_map + 2 * W ? s_map : now + W;
            if ((C::GROUPED ? mine % kScanChunk == 0 && mine < len : w == 0) && p.ws && live) {
                float* ws = p.ws + ((int64_t)(p.chunk[c.j] + mine / kScanChunk) * p.ndir + c.d) * p.H + u;
#pragma unroll
                for (int v = 0; v < V; ++v) ws[v] = h.get(v);
            }
            const int n = tile.writes ? len - s0 : 0;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                h.mad(a[k], b[k]);
                if constexpr (C::STAGED) {
                    store_values<T, V>(out + k * C::RB + lane * C::OWN, h);
                } else {
                    const unsigned row = __shfl_sync(0xffffffffu, rows_now, k);
                    if (k < n) store_values<T, V>(y + (uint64_t)row * yld, h);
                }
            }
            if constexpr (C::GROUPED) h = h.from((groups - 1) * tile.lanes + ul);
            if constexpr (C::STAGED) flush_rows(tile, out, lane, y, yld, rows_now, n);
        }
        if (C::STAGED) cp_async_wait<0>();
    }
    if (p.h_n && live && g == 0 && w == W - 1 && end == len)
#pragma unroll
        for (int v = 0; v < V; ++v) p.h_n[state + v] = h.get(v);
    if (p.padded && tile.writes && c.piece == 0) zero_past_end<T, C::WIDTH>(p, c, y, yld, w, W);
}

// ---------------------------------------------------------------- a warp a sequence

// Many sequences, or very short ones: a warp walks a sequence 8 steps at a time by itself, running
// the steps as they come.  No maps, no barriers, and no warp idles past a short sequence's end.
// 512 directions of 70 frames of 1024 bf16 units: 42 us, 5.4 TB/s.
template <typename T, bool GATED, int ROWS> struct ShortTile : RowTile<T, ROWS, GATED ? 3 : 2> {
    typedef RowTile<T, ROWS, GATED ? 3 : 2> R;
    static constexpr int W = kGlrWarps, CTAS = 3;
    static constexpr int OUT = R::STAGED ? R::S * R::RB : 0;                    // a warp's
    static constexpr int FIT = (72 * 1024 / W - OUT) / R::BYTES;
    static constexpr int NS = !R::STAGED || FIT < 2 ? 1 : FIT > 4 ? 4 : FIT;
    static constexpr int WARP = (R::STAGED ? NS * R::BYTES : 0) + OUT, SMEM = W * WARP;
};

template <typename T, bool GATED, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, 3) glr_fwd_short_kernel(const GlrArgs p, const int items)
{
    typedef ShortTile<T, GATED, ROWS> C;
    constexpr int S = C::S, V = C::V, NS = C::NS;
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, item = blockIdx.x * kGlrWarps + w;
    if (item >= items) return;
    const Place c(p, item, 32 * V);
    const int u = c.u0 + lane * V, len = c.len;
    const bool live = u < p.H;
    const int64_t state = ((int64_t)c.d * p.B + p.perm[c.j]) * p.H + u;
    auto tile = gate_rows<T, ROWS, GATED ? 3 : 2>(p, c, lane);
    tile.in = smem + w * C::WARP;
    char* const out = tile.in + (C::STAGED ? NS * C::BYTES : 0);
    const unsigned yld = (unsigned)(p.ndir * p.H) * (unsigned)sizeof(T);
    char* y = (char*)p.y + ((int64_t)c.d * p.H + c.u0) * (int64_t)sizeof(T) + tile.col();
    Vals<V> h;
    if (len > 0) {
        unsigned rows[NS + 2];          // of the tiles from this one on
#pragma unroll
        for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, q * S, lane, 0);
#pragma unroll
        for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::BYTES, q * S < len);
        h.each([&](int v) { return live && p.h0 ? p.h0[state + v] : 0.f; });
        int stage = 0;
        for (int s0 = 0; s0 < len; s0 += S) {
            Vals<V> a[S], b[S];
            if (C::STAGED) {
                cp_async_wait<NS - 1>();
                __syncwarp();
            }
            step_maps<RowTile<T, ROWS, GATED ? 3 : 2>, GATED>(tile, lane, stage, len - s0, a, b);
            if (C::STAGED) __syncwarp();
            tile.load(lane, rows[NS], stage, s0 + NS * S < len);
            stage = stage == (NS - 1) * C::BYTES ? 0 : stage + C::BYTES;
            const unsigned rows_now = rows[0];
#pragma unroll
            for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
            rows[NS + 1] = c.row_of(p, s0 + (NS + 2) * S, lane, 0);
            if (p.ws && live && s0 % kScanChunk == 0) {
                float* ws = p.ws + ((int64_t)(p.chunk[c.j] + s0 / kScanChunk) * p.ndir + c.d) * p.H + u;
#pragma unroll
                for (int v = 0; v < V; ++v) ws[v] = h.get(v);
            }
            const int n = tile.writes ? len - s0 : 0;
#pragma unroll
            for (int k = 0; k < S; ++k) {
                h.mad(a[k], b[k]);
                if constexpr (C::STAGED) {
                    store_values<T, V>(out + k * C::RB + lane * C::OWN, h);
                } else {
                    const unsigned row = __shfl_sync(0xffffffffu, rows_now, k);
                    if (k < n) store_values<T, V>(y + (uint64_t)row * yld, h);
                }
            }
            if constexpr (C::STAGED) flush_rows(tile, out, lane, y, yld, rows_now, n);
        }
        if (C::STAGED) cp_async_wait<0>();
    } else {
        h.each([&](int v) { return live && p.h0 ? p.h0[state + v] : 0.f; });
    }
    if (p.h_n && live)
#pragma unroll
        for (int v = 0; v < V; ++v) p.h_n[state + v] = h.get(v);
    if (p.padded && tile.writes) zero_past_end<T, C::WIDTH>(p, c, y, yld, 0, 1);
}

// ---------------------------------------------------------------- a piece's map

// Where sequences are cut, every piece but a sequence's last is first reduced to its map: warp w
// composes its eighth of the piece in order, its rows up to four loads ahead, with no barrier until
// the warps' maps meet.  Gates are so read twice, partly out of L2, which the memory's rate bounds: a
// 65536-frame sequence of 1024 bf16 units takes 55 us here (4.9 TB/s) of 132 us in all.  Passing the
// state on between CTAs that hold a piece each would read them once, but waits: clusters in lockstep,
// tried, lose 2 to 3 us every 64 steps a CTA and took 190 to 290 us.
template <typename T, bool GATED, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, 3) glr_fwd_map_kernel(const GlrArgs p)
{
    typedef MapTile<T, GATED, ROWS> C;
    constexpr int S = C::S, W = C::W, V = C::V, NS = C::NS;
    extern __shared__ __align__(128) char smem[];
    __shared__ WarpMap<V> s_map[W];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const Place c(p, blockIdx.x, 32 * V);
    if ((int64_t)(c.piece + 1) * p.piece >= c.len) return;
    auto tile = gate_rows<T, ROWS, GATED ? 3 : 2>(p, c, lane);
    tile.in = smem + w * C::BYTES;
    // (grouped: each group of lanes its own part of the warp's)
    const int groups = C::GROUPED ? p.groups : 1, part = p.piece / (W * groups), gap = C::GROUPED ? part : 0, ul = tile.unit_lane(lane);
    int s0 = c.piece * p.piece + w * groups * part;
    const int end = s0 + part;
    unsigned rows[NS + 2];
#pragma unroll
    for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, s0 + q * S, lane, gap);
#pragma unroll
    for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::STAGE, s0 + q * S < end);
    Vals<V> A, U;
    identity(A, U);
    int stage = 0;
    for (; s0 < end; s0 += S) {
        Vals<V> a[S], b[S];
        if (C::STAGED) {
            cp_async_wait<NS - 1>();
            __syncwarp();
        }
        step_maps<RowTile<T, ROWS, GATED ? 3 : 2>, GATED>(tile, lane, stage, S, a, b);
        if (C::STAGED) __syncwarp();
        tile.load(lane, rows[NS], stage, s0 + NS * S < end);
#pragma unroll
        for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
        rows[NS + 1] = c.row_of(p, s0 + (NS + 2) * S, lane, gap);
        stage = stage == (NS - 1) * C::STAGE ? 0 : stage + C::STAGE;
#pragma unroll
        for (int k = 0; k < S; ++k) {
            U.mad(a[k], b[k]);
            A.mul(a[k]);
        }
    }
    A.hold();
    if (C::STAGED) cp_async_wait<0>();
    if constexpr (C::GROUPED) compose_groups<true>(lane, tile.lanes, A, U);
    if (tile.group(lane) == groups - 1) s_map[w].put(ul, A, U);
    __syncthreads();
    if (w > 0) return;
    s_map[0].get(ul, A, U);
    for (int x = 1; x < W; ++x) {
        Vals<V> a, b;
        s_map[x].get(ul, a, b);
        U.mad(a, b);
        A.mul(a);
    }
    A.hold();
    c.map<V>(p, c.piece)->put(ul, A, U);
}

template <typename T, bool GATED, int ROWS>
lstm_status go(const ScanPlan& p, GlrArgs a, void* scratch, cudaStream_t cs)
{
    static std::atomic<uint64_t> ready{0}, ready_map{0}, ready_short{0};
    typedef FwdTile<T, GATED, ROWS> C;
    typedef MapTile<T, GATED, ROWS> M;
    constexpr int ALONE = ROWS == GLR_GROUPED ? GLR_WIDE : ROWS;     // a warp a sequence: one group
    typedef ShortTile<T, GATED, ALONE> Q;
    if (glr_short(p, C::V, Q::CTAS, &a)) return glr_launch<true>(p.p, glr_fwd_short_kernel<T, GATED, ALONE>, a, C::V, Q::SMEM, ready_short, cs);
    if (C::GROUPED) a.groups = glr_groups(a.H);
    glr_cut(p, C::V, C::CTAS, scratch, &a);
    if (a.cut) {
        lstm_status st = glr_carry(p, a, &a.h0, a.h_n, scratch, cs);
        if (st != LSTM_OK) return st;
        st = glr_launch(p.p, glr_fwd_map_kernel<T, GATED, ROWS>, a, C::V, M::SMEM, ready_map, cs);
        if (st != LSTM_OK) return st;
    }
    return glr_launch(p.p, glr_fwd_kernel<T, GATED, ROWS>, a, C::V, C::SMEM, ready, cs);
}

template <typename T, bool GATED>
lstm_status go(const ScanPlan& p, const GlrArgs& a, void* scratch, cudaStream_t cs)
{
    const GlrRows rows = glr_rows(a, (int)sizeof(T));
    if (rows == GLR_WIDE) return go<T, GATED, GLR_WIDE>(p, a, scratch, cs);
    if (rows == GLR_GROUPED) return go<T, GATED, GLR_GROUPED>(p, a, scratch, cs);
    if constexpr (sizeof(T) == 2)
        if (rows == GLR_SINGLE) return go<T, GATED, GLR_SINGLE>(p, a, scratch, cs);
    return go<T, GATED, GLR_NARROW>(p, a, scratch, cs);
}

}  // namespace

lstm_status launch_glr_fwd(const ScanPlan& p, const lstm_glr_shape& s, GlrArgs a, void* scratch, cudaStream_t cs)
{
    const bool gated = s.cell == LSTM_GLR_GATED;
    if (s.dtype == LSTM_BF16) return gated ? go<__nv_bfloat16, true>(p, a, scratch, cs) : go<__nv_bfloat16, false>(p, a, scratch, cs);
    return gated ? go<float, true>(p, a, scratch, cs) : go<float, false>(p, a, scratch, cs);
}

}  // namespace lstm
