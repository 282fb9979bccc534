// glr_bwd.cu -- backward scan of the gated linear recurrence.
//
// With G_t = dL/dh_t the total error of a state and e_t = a_t G_t what it passes to the one before,
//     G_t = dy_t + e_{t+1},   e_t = a_t (dy_t + e_{t+1})
// is the forward's recurrence run from the end, an affine map e -> A e + W of the same A, and
//     df = G (h_{t-1} - z) a (1 - a),  dz = G (1 - a)                                  (tied)
//     df = G h_{t-1} a (1 - a),  dz = G sig(i),  di = G z sig(i) (1 - sig(i))          (gated).
// The states are not read back (y may be bf16): each 64 steps start from the fp32 state that the
// forward pass kept and are run again.  A CTA walks 64 steps at a time from the end, its warps
// holding 8 steps each as in the forward pass; both maps, (A, U) of h within the 64 steps and
// (A, W) of e, meet in shared memory at one barrier.  Gates and errors stay where they arrived in
// shared memory for the second pass over a warp's steps, and the gradients leave from there.
//
// Bound by memory for fp32 (70 k frames of 2 x 256 units, three gates, 158 us, 6.4 TB/s, 95 % of the
// copy rate); bf16 by shared memory and issue at half the bytes (40555 frames of 2 x 512 units, two
// gates, 89 us, 5.1 TB/s).  Two CTAs an SM: a, 1 - a and b of 8 steps take 48 registers of 128.
#include "glr.cuh"

namespace lstm {

namespace {

template <typename T, bool GATED, int ROWS> struct BwdTile : RowTile<T, ROWS, GATED ? 4 : 3> {
    typedef RowTile<T, ROWS, GATED ? 4 : 3> R;
    static constexpr int W = kGlrWarps;
    static constexpr int STAGE = W * R::BYTES;
    static constexpr int MAPS = 2 * 3 * W * (int)sizeof(WarpMap<R::V>);
    static constexpr int CTAS = 2;
    static constexpr int FIT = (227 * 1024 / CTAS - 1024 - MAPS) / STAGE;
    static constexpr int NS = !R::STAGED || FIT < 2 ? 1 : 2;
    static constexpr int SMEM = NS * STAGE + MAPS;
};

template <typename T, int ROWS, int G> __device__ __forceinline__ RowTile<T, ROWS, G> error_rows(const GlrArgs& p, const Place& c, int lane)
{
    constexpr int64_t e = (int64_t)sizeof(T);
    RowTile<T, ROWS, G> t;
    const int64_t from = (c.d * p.dstride + c.u0) * e;
    t.src[0] = (const char*)p.f + from;
    t.src[1] = (const char*)p.z + from;
    if (G == 4) t.src[2] = (const char*)p.i + from;
#pragma unroll
    for (int x = 0; x < G - 1; ++x) t.ld[x] = (unsigned)p.ld * (unsigned)e;
    t.src[G - 1] = (const char*)p.dy + ((int64_t)c.d * p.H + c.u0) * e;
    t.ld[G - 1] = (unsigned)(p.ndir * p.H) * (unsigned)e;
    t.place(lane, (p.H - c.u0) * (int)e, p.groups);
    return t;
}

// a, 1 - a and b of 8 steps, the identity for those past the end.
template <bool GATED, typename Tile>
__device__ __forceinline__ void step_parts(const Tile& tile, int lane, int stage, int left, Vals<Tile::V> (&a)[kGlrSteps],
                                           Vals<Tile::V> (&n)[kGlrSteps], Vals<Tile::V> (&b)[kGlrSteps])
{
#pragma unroll
    for (int k = 0; k < kGlrSteps; ++k) {
        const Vals<Tile::V> z = tile.held(lane, 1, k, stage);
        tile.held(lane, 0, k, stage).sigmoids(a[k], n[k]);
        if (GATED) {
            b[k] = tile.held(lane, 2, k, stage);
            b[k].sigmoid();
        } else {
            b[k] = n[k];
        }
        b[k].mul(z);
    }
    if (left < kGlrSteps) {
#pragma unroll
        for (int k = 0; k < kGlrSteps; ++k)
            if (k >= left) {
                a[k].fill(1.f);
                b[k].fill(0.f);
            }
    }
}

// One step backwards: e comes in as the error from the step after and leaves as what this one passes on; `h` is the
// state before the step.
template <bool GATED, typename Tile, int V>
__device__ __forceinline__ void step_gradients(const Tile& tile, int lane, int k, int stage, const Vals<V>& a, Vals<V> n, Vals<V> h, Vals<V>& e,
                                               Vals<V>& df, Vals<V>& dz, Vals<V>& di)
{
    e.add(tile.held(lane, GATED ? 3 : 2, k, stage));        // G
    const Vals<V> z = tile.held(lane, 1, k, stage);
    n.mul(e);                                               // G (1 - a)
    dz = di = e;
    if (GATED) {
        Vals<V> g, ng;
        tile.held(lane, 2, k, stage).sigmoids(g, ng);
        df = n;
        dz.mul(g);
        di = dz;
        di.mul(ng);
        di.mul(z);
    } else {
        dz = n;
        df = n;
        h.sub(z);
    }
    df.mul(a);
    df.mul(h);
    e.mul(a);
}

template <typename T, bool GATED, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, BwdTile<T, GATED, ROWS>::CTAS) glr_bwd_kernel(const GlrArgs p)
{
    typedef BwdTile<T, GATED, ROWS> C;
    constexpr int S = C::S, W = C::W, V = C::V, NS = C::NS, G = GATED ? 4 : 3, DY = G - 1;
    extern __shared__ __align__(128) char smem[];
    WarpMap<V>* const s_map = (WarpMap<V>*)(smem + NS * C::STAGE);      // [3][W] of e, then [3][W] of h
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    // cut sequences: the pieces whose maps were formed last are the ones still in L2
    const Place c(p, p.cut ? gridDim.x - 1 - blockIdx.x : blockIdx.x, 32 * V);
    auto tile = error_rows<T, ROWS, G>(p, c, lane);
    // (grouped: groups of lanes hold the same units, a group's 8 steps after the other's)
    constexpr int GAP = C::GROUPED ? S : 0;
    const int groups = C::GROUPED ? p.groups : 1, g = tile.group(lane), ul = tile.unit_lane(lane), chunk = groups * kScanChunk;
    const int u = c.u0 + ul * V, len = c.len;
    const bool live = u < p.H;
    const int64_t state = ((int64_t)c.d * p.B + p.perm[c.j]) * p.H + u;
    tile.in = smem + w * C::BYTES;
    const unsigned gld = (unsigned)p.gld * (unsigned)sizeof(T);
    const int64_t to = (c.d * p.gdstride + c.u0) * (int64_t)sizeof(T) + tile.col();
    char* grad[G - 1];
    grad[0] = (char*)p.df + to;
    grad[1] = (char*)p.dz + to;
    if (GATED) grad[G - 2] = (char*)p.di + to;
    Vals<V> e;
    e.each([&](int v) { return live && p.dh_n ? p.dh_n[state + v] : 0.f; });
    const int begin = p.cut ? c.piece * p.piece : 0, end = p.cut ? min(len, begin + p.piece) : len;

    if (len > 0) {
        int base = (end - 1) / chunk * chunk;
        unsigned rows[NS + 2];          // of the iterations from this one on
#pragma unroll
        for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, base + w * S * groups - q * chunk, lane, GAP);
#pragma unroll
        for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::STAGE, !C::BOUNDED || base - q * chunk >= begin);
        // the states kept before each 64 steps
        const float* kept = p.ws + ((int64_t)(p.chunk[c.j] + base / kScanChunk) * p.ndir + c.d) * p.H + (live ? u : 0);
        Vals<V> start;
        start.each([&](int v) { return live ? __ldg(kept + v) : 0.f; });
        WarpMap<V>*now = s_map, *before = s_map + 2 * W;        // maps of e; those of h lie 3 W further
        Vals<V> A, U;
        if (end < len) {
            // the error from beyond this piece: the later pieces' maps, an eighth of them composed by each warp
            const int last = (len - 1) / p.piece, n = last - c.piece, share = (n + W - 1) / W;
            identity(A, U);
#pragma unroll 4
            for (int k = w * share; k < min(n, (w + 1) * share); ++k) {
                Vals<V> a, b;
                c.map<V>(p, last - k)->get(ul, a, b);
                U.mad(a, b);
                A.mul(a);
            }
            A.hold();
            now[w].put(ul, A, U);
            __syncthreads();
#pragma unroll
            for (int x = 0; x < W; ++x) now[x].apply(ul, e);
        }
        identity(A, U);
        before[w].put(ul, A, U);
        __syncthreads();
        int stage = 0;
        for (; base >= begin; base -= chunk) {
            const int s0 = base + w * S * groups, mine = s0 + g * S;
            if (C::STAGED) {
                cp_async_wait<NS - 1>();
                __syncwarp();
            } else {
                tile.stash(lane);
                tile.load(lane, rows[1], 0);
            }
            if (s0 + S * groups > len) {        // past the end no error enters
                for (int k = max(0, len - mine); k < S; ++k)
                    for (int x = 0; x < C::OWN; x += (int)sizeof(T)) *(T*)(tile.slot(lane, DY, k, stage) + x) = from_f32<T>(0.f);
                __syncwarp();
            }
            Vals<V> a[S], n[S], b[S];               // a, 1 - a, b
            step_parts<GATED>(tile, lane, stage, len - mine, a, n, b);
            A = a[0];
            U = b[0];
#pragma unroll
            for (int k = 1; k < S; ++k) {
                U.mad(a[k], b[k]);
                A.mul(a[k]);
            }
            A.hold();
            Vals<V> AH, UH, AE;     // grouped: of the steps before and after this group's
            if constexpr (C::GROUPED) {
                AH = AE = A;
                UH = U;
                compose_groups<true>(lane, tile.lanes, AH, UH);
                if (g == groups - 1) now[3 * W + w].put(ul, AH, UH);
                AH = AH.from(lane - tile.lanes);
                UH = UH.from(lane - tile.lanes);
                if (g == 0) identity(AH, UH);
            } else {
                now[3 * W + w].put(lane, A, U);
            }
            U = tile.held(lane, DY, S - 1, stage);
            U.mul(a[S - 1]);
#pragma unroll
            for (int k = S - 2; k >= 0; --k) {
                U.add(tile.held(lane, DY, k, stage));
                U.mul(a[k]);
            }
            if constexpr (C::GROUPED) {
                compose_groups<false>(lane, tile.lanes, AE, U);
                if (g == 0) now[w].put(ul, AE, U);
                AE = AE.from(lane + tile.lanes);
                U = U.from(lane + tile.lanes);
                if (g == groups - 1) identity(AE, U);
            } else {
                now[w].put(lane, A, U);
            }
            Vals<V> h = start;
            if (base > begin) {
                kept -= (int64_t)groups * p.ndir * p.H;
                start.each([&](int v) { return live ? __ldg(kept + v) : 0.f; });
            }
            __syncthreads();
#pragma unroll
            for (int x = 1; x < W; ++x) (w - x >= 0 ? before + w - x : now + w - x + W)->apply(ul, e);
#pragma unroll
            for (int x = 0; x < W - 1; ++x)
                if (x < w) now[3 * W + x].apply(ul, h);
            if constexpr (C::GROUPED) {
                h.mad(AH, UH);
                e.mad(AE, U);
            }
            before = now;
            now = now == s_map + 2 * W ? s_map : now + W;
#pragma unroll
            for (int k = 0; k < S; ++k) {           // b becomes the state before the step
                const Vals<V> was = h;
                h.mad(a[k], b[k]);
                b[k] = was;
            }
            const unsigned rows_now = rows[0];
            const int m = tile.writes ? len - s0 : 0;
#pragma unroll
            for (int k = S - 1; k >= 0; --k) {
                Vals<V> df, dz, di;
                step_gradients<GATED>(tile, lane, k, stage, a[k], n[k], b[k], e, df, dz, di);
                if constexpr (C::STAGED) {
                    store_values<T, V>(tile.slot(lane, 0, k, stage), df);
                    store_values<T, V>(tile.slot(lane, 1, k, stage), dz);
                    if (GATED) store_values<T, V>(tile.slot(lane, 2, k, stage), di);
                } else {
                    const uint64_t row = (uint64_t)__shfl_sync(0xffffffffu, rows_now, k) * gld;
                    if (k < m) {
                        store_values<T, V>(grad[0] + row, df);
                        store_values<T, V>(grad[1] + row, dz);
                        if (GATED) store_values<T, V>(grad[G - 2] + row, di);
                    }
                }
            }
            if constexpr (C::GROUPED) e = e.from(ul);
            if constexpr (C::STAGED) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < S; k += C::RI) {
                    const int s = tile.step(lane, k);
                    const uint64_t row = (uint64_t)__shfl_sync(0xffffffffu, rows_now, s) * gld;
#pragma unroll
                    for (int x = 0; x < G - 1; ++x) {
                        const uint4 q = *(const uint4*)(tile.in + stage + (x * S + k + lane / C::LR) * C::RB + tile.at);
                        if (s < m) *(uint4*)(grad[x] + row) = q;
                    }
                }
                __syncwarp();
                tile.load(lane, rows[NS], stage, !C::BOUNDED || base - NS * chunk >= begin);
                stage = stage == (NS - 1) * C::STAGE ? 0 : stage + C::STAGE;
            }
#pragma unroll
            for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
            rows[NS + 1] = c.row_of(p, s0 - (NS + 2) * chunk, lane, GAP);
        }
        if (C::STAGED) cp_async_wait<0>();
    }
    if (p.dh0 && live && g == 0 && w == 0 && c.piece == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.dh0[state + v] = e.get(v);
    if (p.padded && tile.writes && c.piece == 0)        // the padded comparator's rows past the end
        for (int t = len + w; t < p.T; t += W)
#pragma unroll
            for (int x = 0; x < G - 1; ++x)
                for (int y = 0; y < C::WIDTH; y += (int)sizeof(T))
                    *(T*)(grad[x] + (uint64_t)(p.off[t] + c.j) * gld + y) = from_f32<T>(0.f);
}

// A warp a sequence, as in the forward pass: each 64 steps from the end, their states run again 8
// steps at a time (a second reading, out of the caches, where there are more than 8), then their
// gradients 8 steps at a time.  512 directions of 70 frames of 1024 bf16 units: 87 us, 4.3 TB/s.
template <typename T, bool GATED, int ROWS> struct BwdShortTile : RowTile<T, ROWS, GATED ? 4 : 3> {
    typedef RowTile<T, ROWS, GATED ? 4 : 3> R;
    static constexpr int W = kGlrWarps, CTAS = 2;
    static constexpr int TILES = kScanChunk / kGlrSteps;
    static constexpr int STATES = TILES * 32 * R::V * 4;        // a warp's
    static constexpr int FIT = (112 * 1024 / W - STATES) / R::BYTES;
    static constexpr int NS = !R::STAGED || FIT < 2 ? 1 : FIT > 3 ? 3 : FIT;
    static constexpr int WARP = NS * R::BYTES + STATES, SMEM = W * WARP;
};

template <typename T, bool GATED, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, 2) glr_bwd_short_kernel(const GlrArgs p, const int items)
{
    typedef BwdShortTile<T, GATED, ROWS> C;
    constexpr int S = C::S, V = C::V, NS = C::NS, G = GATED ? 4 : 3;
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, item = blockIdx.x * kGlrWarps + w;
    if (item >= items) return;
    const Place c(p, item, 32 * V);
    const int u = c.u0 + lane * V, len = c.len;
    const bool live = u < p.H;
    const int64_t state = ((int64_t)c.d * p.B + p.perm[c.j]) * p.H + u;
    auto tile = error_rows<T, ROWS, G>(p, c, lane);
    tile.in = smem + w * C::WARP;
    Vals<V>* const before = (Vals<V>*)(tile.in + NS * C::BYTES) + lane;     // [tile][lane]: states before the tiles
    const unsigned gld = (unsigned)p.gld * (unsigned)sizeof(T);
    const int64_t to = (c.d * p.gdstride + c.u0) * (int64_t)sizeof(T) + tile.col();
    char* grad[G - 1];
    grad[0] = (char*)p.df + to;
    grad[1] = (char*)p.dz + to;
    if (GATED) grad[G - 2] = (char*)p.di + to;
    Vals<V> e;
    e.each([&](int v) { return live && p.dh_n ? p.dh_n[state + v] : 0.f; });
    for (int base = len > 0 ? (len - 1) / kScanChunk * kScanChunk : -1; base >= 0; base -= kScanChunk) {
        const float* kept = p.ws + ((int64_t)(p.chunk[c.j] + base / kScanChunk) * p.ndir + c.d) * p.H + (live ? u : 0);
        Vals<V> h;
        h.each([&](int v) { return live ? __ldg(kept + v) : 0.f; });
        const int tiles = min(C::TILES, (len - base + S - 1) / S);
        before[0] = h;
        // sweep 0: the tiles but the last, forwards, for the states before them; sweep 1: all of them, backwards
        for (int sweep = tiles > 1 ? 0 : 1; sweep < 2; ++sweep) {
            const int count = sweep == 0 ? tiles - 1 : tiles;
            auto first = [&](int x) { return base + (sweep == 0 ? x : tiles - 1 - x) * S; };     // step of the x-th tile
            unsigned rows[NS + 2];
#pragma unroll
            for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, first(q), lane, 0);
#pragma unroll
            for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::BYTES, q < count);
            int stage = 0;
            for (int x = 0; x < count; ++x) {
                const int s0 = first(x);
                if (C::STAGED) {
                    cp_async_wait<NS - 1>();
                    __syncwarp();
                } else {
                    tile.stash(lane);
                    tile.load(lane, rows[1], 0);
                }
                if (s0 + S > len) {     // past the end no error enters
                    for (int k = max(0, len - s0); k < S; ++k)
                        for (int y = 0; y < C::OWN; y += (int)sizeof(T)) *(T*)(tile.slot(lane, G - 1, k, stage) + y) = from_f32<T>(0.f);
                    __syncwarp();
                }
                Vals<V> a[S], n[S], b[S];
                step_parts<GATED>(tile, lane, stage, len - s0, a, n, b);
                if (sweep == 0) {
#pragma unroll
                    for (int k = 0; k < S; ++k) h.mad(a[k], b[k]);
                    before[(x + 1) * 32] = h;
                } else {
                    h = before[(tiles - 1 - x) * 32];
#pragma unroll
                    for (int k = 0; k < S; ++k) {       // b becomes the state before the step
                        const Vals<V> was = h;
                        h.mad(a[k], b[k]);
                        b[k] = was;
                    }
                    const int m = tile.writes ? len - s0 : 0;
#pragma unroll
                    for (int k = S - 1; k >= 0; --k) {
                        Vals<V> df, dz, di;
                        step_gradients<GATED>(tile, lane, k, stage, a[k], n[k], b[k], e, df, dz, di);
                        if constexpr (C::STAGED) {
                            store_values<T, V>(tile.slot(lane, 0, k, stage), df);
                            store_values<T, V>(tile.slot(lane, 1, k, stage), dz);
                            if (GATED) store_values<T, V>(tile.slot(lane, 2, k, stage), di);
                        } else {
                            const uint64_t row = (uint64_t)__shfl_sync(0xffffffffu, rows[0], k) * gld;
                            if (k < m) {
                                store_values<T, V>(grad[0] + row, df);
                                store_values<T, V>(grad[1] + row, dz);
                                if (GATED) store_values<T, V>(grad[G - 2] + row, di);
                            }
                        }
                    }
                    if constexpr (C::STAGED) {
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < S; k += C::RI) {
                            const int s = k + lane / C::LR;
                            const uint64_t row = (uint64_t)__shfl_sync(0xffffffffu, rows[0], s) * gld;
#pragma unroll
                            for (int q = 0; q < G - 1; ++q) {
                                const uint4 bits = *(const uint4*)(tile.in + stage + (q * S + s) * C::RB + tile.at);
                                if (s < m) *(uint4*)(grad[q] + row) = bits;
                            }
                        }
                    }
                }
                if (C::STAGED) {
                    __syncwarp();
                    tile.load(lane, rows[NS], stage, x + NS < count);
                    stage = stage == (NS - 1) * C::BYTES ? 0 : stage + C::BYTES;
                }
#pragma unroll
                for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
                rows[NS + 1] = c.row_of(p, first(x + NS + 2), lane, 0);
            }
            if (C::STAGED) cp_async_wait<0>();
        }
    }
    if (p.dh0 && live)
#pragma unroll
        for (int v = 0; v < V; ++v) p.dh0[state + v] = e.get(v);
    if (p.padded && tile.writes)        // the padded comparator's rows past the end
        for (int t = len; t < p.T; ++t)
#pragma unroll
            for (int x = 0; x < G - 1; ++x)
                for (int y = 0; y < C::WIDTH; y += (int)sizeof(T))
                    *(T*)(grad[x] + (uint64_t)(p.off[t] + c.j) * gld + y) = from_f32<T>(0.f);
}

// A piece's map of e, from f and dy alone: every piece but a sequence's first.
template <typename T, int ROWS> struct BwdMapTile : RowTile<T, ROWS, 2> {
    typedef RowTile<T, ROWS, 2> R;
    static constexpr int W = kGlrWarps;
    static constexpr int STAGE = R::STAGED ? W * R::BYTES : 0;
    static constexpr int FIT = 72 * 1024 / (STAGE + 1);
    static constexpr int NS = !R::STAGED ? 1 : FIT < 2 ? 2 : FIT > 4 ? 4 : FIT;
    static constexpr int SMEM = NS * STAGE;
};

template <typename T, int ROWS>
__global__ void __launch_bounds__(32 * kGlrWarps, 3) glr_bwd_map_kernel(const GlrArgs p)
{
    typedef BwdMapTile<T, ROWS> C;
    constexpr int S = C::S, W = C::W, V = C::V, NS = C::NS;
    extern __shared__ __align__(128) char smem[];
    __shared__ WarpMap<V> s_map[W];
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const Place c(p, blockIdx.x, 32 * V);
    if (c.piece == 0) return;
    RowTile<T, ROWS, 2> tile;
    constexpr int64_t el = (int64_t)sizeof(T);
    tile.src[0] = (const char*)p.f + (c.d * p.dstride + c.u0) * el;
    tile.ld[0] = (unsigned)p.ld * (unsigned)el;
    tile.src[1] = (const char*)p.dy + ((int64_t)c.d * p.H + c.u0) * el;
    tile.ld[1] = (unsigned)(p.ndir * p.H) * (unsigned)el;
    tile.place(lane, (p.H - c.u0) * (int)el, p.groups);
    tile.in = smem + w * C::BYTES;
    // (grouped: each group of lanes its own part of the warp's)
    const int groups = C::GROUPED ? p.groups : 1, part = p.piece / (W * groups), gap = C::GROUPED ? part : 0;
    const int g = tile.group(lane), ul = tile.unit_lane(lane), first = c.piece * p.piece + w * groups * part;
    int s0 = first + part - S;
    unsigned rows[NS + 2];
#pragma unroll
    for (int q = 0; q < NS + 2; ++q) rows[q] = c.row_of(p, s0 - q * S, lane, gap);
#pragma unroll
    for (int q = 0; q < NS; ++q) tile.load(lane, rows[q], q * C::STAGE, s0 - q * S >= first);
    Vals<V> A, U;
    identity(A, U);
    int stage = 0;
    for (; s0 >= first; s0 -= S) {
        if (C::STAGED) {
            cp_async_wait<NS - 1>();
            __syncwarp();
        }
        Vals<V> a[S], d[S];
#pragma unroll
        for (int k = 0; k < S; ++k) {
            const Raw<T, V> rf = tile.value(lane, 0, k, stage), rd = tile.value(lane, 1, k, stage);
            a[k].each([&](int v) { return rf.get(v); });
            a[k].forget();
            d[k].each([&](int v) { return rd.get(v); });
        }
        if (C::STAGED) __syncwarp();
        tile.load(lane, rows[NS], stage, s0 - NS * S >= first);
#pragma unroll
        for (int q = 0; q < NS + 1; ++q) rows[q] = rows[q + 1];
        rows[NS + 1] = c.row_of(p, s0 - (NS + 2) * S, lane, gap);
        stage = stage == (NS - 1) * C::STAGE ? 0 : stage + C::STAGE;
#pragma unroll
        for (int k = S - 1; k >= 0; --k) {
            if (s0 + g * gap + k >= c.len) continue;
            U.add(d[k]);
            U.mul(a[k]);
            A.mul(a[k]);
        }
    }
    A.hold();
    if (C::STAGED) cp_async_wait<0>();
    if constexpr (C::GROUPED) compose_groups<false>(lane, tile.lanes, A, U);
    if (g == 0) s_map[w].put(ul, A, U);
    __syncthreads();
    if (w < W - 1) return;
    s_map[w].get(ul, A, U);
    for (int x = W - 2; x >= 0; --x) {
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
    typedef BwdTile<T, GATED, ROWS> C;
    constexpr int ALONE = ROWS == GLR_GROUPED ? GLR_WIDE : ROWS;     // a warp a sequence: one group
    typedef BwdShortTile<T, GATED, ALONE> Q;
    if (glr_short(p, C::V, Q::CTAS, &a)) return glr_launch<true>(p.p, glr_bwd_short_kernel<T, GATED, ALONE>, a, C::V, Q::SMEM, ready_short, cs);
    if (C::GROUPED) a.groups = glr_groups(a.H);
    glr_cut(p, C::V, C::CTAS, scratch, &a);
    if (a.cut) {
        lstm_status st = glr_carry(p, a, &a.dh_n, a.dh0, scratch, cs);
        if (st != LSTM_OK) return st;
        st = glr_launch(p.p, glr_bwd_map_kernel<T, ROWS>, a, C::V, BwdMapTile<T, ROWS>::SMEM, ready_map, cs);
        if (st != LSTM_OK) return st;
    }
    return glr_launch(p.p, glr_bwd_kernel<T, GATED, ROWS>, a, C::V, C::SMEM, ready, cs);
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

lstm_status launch_glr_bwd(const ScanPlan& p, const lstm_glr_shape& s, GlrArgs a, void* scratch, cudaStream_t cs)
{
    const bool gated = s.cell == LSTM_GLR_GATED;
    if (s.dtype == LSTM_BF16) return gated ? go<__nv_bfloat16, true>(p, a, scratch, cs) : go<__nv_bfloat16, false>(p, a, scratch, cs);
    return gated ? go<float, true>(p, a, scratch, cs) : go<float, false>(p, a, scratch, cs);
}

}  // namespace lstm
