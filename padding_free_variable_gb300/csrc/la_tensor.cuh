// la_tensor.cuh -- linear attention of bf16 rows on the tensor cores (tcgen05, accumulators in tensor memory).
//
// A CTA walks one head of one sequence (or a piece of it) 128 steps at a time.  Per chunk, with M = 128 rows of a product:
//     S = Q K^T                  128 x 128     O = Q Y           128 x B    (Y in two bf16 pieces)
//     P = S lambda^(i-j), i >= j, rounded to bf16, back into tensor memory as the next product's left operand
//     O' = P V                   128 x B       out = sP O' + sI lambda^i O
//     Y = lambda^n Y + K^T (sK lambda^(n-j) V) A x B            (the weighted values in bf16 pieces)
// Tensor cores cut off what does not fit behind a sum, so a chunk's products are added up from zero, the smallest pieces
// first, and Y, in registers, takes their sum with a rounding: a long memory does not shrink chunk by chunk.
// The weighted values enter in three pieces (24 bits) where Y may be asked for in the end, in two (16 bits) where it
// only serves outputs that are rounded to bf16.  Rows come by cp.async into the 128-byte swizzled layout, one image of 64 columns a panel: read along a row it is the
// K-major operand of S, read along a column the MN-major operand of the other products, so nothing is transposed.
//
// Bound by neither memory nor the tensor cores alone but by the chain S, P, O', Y of a chunk: 40555 steps of 2 x 8 heads of
// 64 values 148 us (38 % of the copy rate; the tensor cores 20 %, issue 45 %), 65536 steps of 8 heads of 128 as one sequence
// 130 us for the pieces' sums, 28 us for their starts and 232 us for the outputs.  Rows by TMA gathers of four rows took 75 to
// 84 cycles an instruction, 218 us instead of 158; the sums for Y in front of S's pass instead of behind it, 179 us.
//
// CTAs stay on the GPU and take every so-many-th walk; the next chunk's rows, of the same walk or the next, are on their way
// as soon as the products that read the last ones are done.
#pragma once

#include <type_traits>

#include "la.cuh"
#include "tc_ptx.cuh"

namespace lstm {

namespace {

constexpr int kC = 128, kPanel = kC * 128;      // steps of a chunk, bytes of 64 columns of all of them

// A: width of queries and keys, B: of values, padded to 64 or 128.
template <int A, int B> struct Layout {
    // two CTAs an SM where their shared and tensor memory allow it, else one of twice the threads
    static constexpr int T = A == 64 && B == 64 ? 256 : 512, CTAS = A == 64 && B == 64 ? 2 : 1, PARTS = T / 128;
    static constexpr int Q = 0, K = Q + kC * A * 2, V = K + kC * A * 2, V1 = V + kC * B * 2, V2 = V1 + kC * B * 2;
    static constexpr bool in_q = A == 128 && B == 128;          // no room: the third piece takes the queries' place
    static constexpr int V3 = in_q ? Q : V2 + kC * B * 2;
    static constexpr int Y1 = (in_q ? V2 : V3) + kC * B * 2, Y2 = Y1 + A * B * 2;
    static constexpr int POWERS = Y2 + A * B * 2;               // [2][64]: lambda^n and lambda^(31-n), of two walks
    static constexpr int BARS = POWERS + 512, WALKS = BARS + 64, BYTES = WALKS + 128;       // WALKS: of this walk, the next and the last one
    // tensor memory, columns
    static constexpr uint32_t S = 0, O = 128, Y = O + B, COLUMNS = B == 64 ? 256 : 512;
    static constexpr int OC = B / PARTS, YC = A == 128 ? B / PARTS : B / (2 * PARTS);       // columns of a thread
};

__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// Where 8 columns from 8 * chunk on of a row lie, panels of `rows` rows.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk, int panel) { return (chunk >> 3) * panel + swizzled(row, chunk & 7); }

// Descriptor of an MN-major operand in the 128-byte swizzled layout: 64 values of the M or N dimension a 128-byte row, a row
// a step of K, groups of 8 rows 1024 bytes apart, the next 64 values `panel` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t panel)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(panel >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

constexpr uint32_t kAmn = 1u << 15, kBmn = 1u << 16;            // instruction descriptor: A, B are MN-major

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two values at once: one instruction of the fp32 pipe.
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b)
{
    asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mul.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b)
{
    asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}" : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
// x = s x + a
__device__ __forceinline__ void fma2(float& x, float& y, float s, float a, float b)
{
    asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n mov.b64 r, {%4, %4};\n fma.rn.f32x2 p, p, r, q;\n mov.b64 {%0, %1}, p;\n}"
        : "+f"(x), "+f"(y) : "f"(a), "f"(b), "f"(s));
}

// Two values less what their first piece holds (the piece's sign is turned, so that it can be added).
__device__ __forceinline__ uint32_t cut(float& x, float& y)
{
    const uint32_t w = pack2(x, y), v = w ^ 0x80008000u;
    add2(x, y, low(v), high(v));
    return w;
}

// STATES: only what a piece adds to Y, into `starts`.
template <int A, int B, bool STATES>
__global__ void __launch_bounds__(Layout<A, B>::T, Layout<A, B>::CTAS) la_tensor_kernel(const __grid_constant__ LaArgs p, int total)
{
    typedef Layout<A, B> L;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, quad = warp % 4, part = warp / 4;
    const uint32_t base = tc::smem_u32(sm);
    float* const powers = (float*)(sm + L::POWERS);
    // S and O, O', the sum for Y are done; everything is, after a wait that ran out
    uint64_t* const bar = (uint64_t*)(sm + L::BARS);
    enum { DONE_S = 0, DONE_O, DONE_Y, DRAINED, BARRIERS };
    uint32_t* const slot_of_tmem = (uint32_t*)(bar + BARRIERS);
    int* const stop = (int*)(slot_of_tmem + 1);
    if (tid == 0) {
        for (int i = 0; i < BARRIERS; ++i) tc::mbar_init(bar + i, 1);
        *stop = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(slot_of_tmem, L::COLUMNS);
        tc::tmem_relinquish();
    }

    // the next walk of this CTA that has a step: there and back along the CTAs, as walks get shorter
    int round = -1;
    auto next_walk = [&](LaPart* to) {
        for (;;) {
            ++round;
            const int64_t id = (int64_t)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (id >= total) return false;
            const LaPart c = la_part(p, (unsigned)id);
            if (STATES) {
                if (c.last) continue;
            } else {
                const LaJob& j = p.job[c.job];
                la_past_end<__nv_bfloat16>(p, j, c);
                if (c.len == 0) {
                    la_pass(j, la_state(p, j, c));
                    continue;
                }
            }
            if (tid == 0) *to = c;
            return true;
        }
    };
    // first row of a step (the walk's own lies `slot` behind it); steps past the chunk's end count as its last
    auto row_of = [&](const LaPart& c, int u, int back, int step, int n) {
        const int v = u + min(step, n - 1), t = (c.d == 1) != (back != 0) ? c.len - 1 - v : v;
        return __ldg(p.off + t);
    };
    auto steps_of = [&](const LaPart& c, int u) { return min(kC, c.end - u); };
    // steps that a chunk's state decays by: one less behind the last step of a walk whose final state holds one lambda less
    auto decay_of = [&](const LaPart& c, int u) { return steps_of(c, u) - (c.last && u + kC >= c.end ? p.job[c.job].early : 0); };
    auto set_powers = [&](int which, float l2) {
        if (tid < 64) powers[which * 64 + tid] = exp2f((tid < 32 ? tid : 63 - tid) * l2);
    };

    // a chunk's rows: 16 bytes a thread and copy, zeros past the end.  Where they lie is looked up a chunk ahead.
    constexpr int CHA = A / 8, EACHA = L::T / CHA, ITA = kC / EACHA, CHB = B / 8, EACHB = L::T / CHB, ITB = kC / EACHB;
    int rows_a[ITA], rows_b[A == B ? 1 : ITB];
    auto find_rows = [&](const LaPart& c, int u) {
        const int n = steps_of(c, u), back = p.job[c.job].back;
#pragma unroll
        for (int i = 0; i < ITA; ++i) rows_a[i] = row_of(c, u, back, i * EACHA + tid / CHA, n);
        if (A != B) {
#pragma unroll
            for (int i = 0; i < ITB; ++i) rows_b[A == B ? 0 : i] = row_of(c, u, back, i * EACHB + tid / CHB, n);
        }
    };
    auto copy = [&](const LaRows& r, const LaPart& c, int u, int to, int w, const auto& rows, auto width) {
        constexpr int CH = decltype(width)::value / 8, EACH = L::T / CH;
        const int ch = tid % CH, n = ch * 8 < w ? steps_of(c, u) : 0;
        const __nv_bfloat16* const from = (const __nv_bfloat16*)r.p + c.d * r.dir + c.h * r.head + c.slot * r.row + (n > 0 ? ch * 8 : 0);
        const uint32_t at0 = base + to + tile_at(tid / CH, ch, kPanel);     // EACH rows on: the same swizzle, EACH a multiple of 8
#pragma unroll
        for (int i = 0; i < kC / EACH; ++i) cp_async16(at0 + i * EACH * 128, from + rows[i] * r.row, i * EACH + tid / CH < n);
    };
    auto load_q = [&](const LaPart& c, int u) {
        const LaJob& j = p.job[c.job];
        if (!STATES) copy(j.q, c, u, L::Q, j.a, rows_a, std::integral_constant<int, A>());
    };
    auto load_kv = [&](const LaPart& c, int u) {
        const LaJob& j = p.job[c.job];
        copy(j.k, c, u, L::K, j.a, rows_a, std::integral_constant<int, A>());
        if constexpr (A == B) copy(j.v, c, u, L::V, j.b, rows_a, std::integral_constant<int, B>());
        else copy(j.v, c, u, L::V, j.b, rows_b, std::integral_constant<int, B>());
    };

    LaPart* const walks = (LaPart*)(sm + L::WALKS);
    int now = 0, u = 0;                                 // this walk's place, and the chunk's first step
    bool more = next_walk(walks);
    tc::tc_fence_before_sync();
    __syncthreads();
    tc::tc_fence_after_sync();
    const uint32_t tmem = *slot_of_tmem, mine = tmem + ((uint32_t)(quad * 32) << 16);
    const int row = quad * 32 + lane;                   // of S and O
    // of Y: with A = 64 the second 64 lanes hold the rows once more, for other columns
    const int x = row % A, y0 = (A == 128 ? part : (quad >> 1) * L::PARTS + part) * L::YC, o0 = part * L::OC;
    auto waited = [&](int which, uint32_t phase) {
        if (!tc::mbar_wait(bar + which, phase, p.limit_ns)) {
            *(volatile int*)stop = 1;
            record_failure(p.status, LSTM_ERR_TIMEOUT, 0x90000u | which);
        }
        __syncwarp();
    };
    float y[L::YC];                                     // Y, this thread's columns of row x
    auto put_pieces = [&] {
#pragma unroll
        for (int k = 0; k < L::YC; k += 8) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = y[k + e];
            const uint32_t to = tile_at(x, (y0 + k) / 8, A * 128);
            uint4 w;
            w.x = cut(f[0], f[1]); w.y = cut(f[2], f[3]); w.z = cut(f[4], f[5]); w.w = cut(f[6], f[7]);
            *(uint4*)(sm + L::Y1 + to) = w;
            *(uint4*)(sm + L::Y2 + to) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        }
    };
    auto load_columns = [&](uint32_t column, auto& v) {
        constexpr int N = sizeof(v) / sizeof(v[0]);
        uint32_t r[N / 16][16];
#pragma unroll
        for (int k = 0; k < N / 16; ++k) tc::tmem_ld_32x32b_x16(mine + column + 16 * k, r[k]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = __uint_as_float(r[k / 16][k % 16]);
    };
    // a state on its way in or out, in the place of Y's pieces: 16 bytes next to each other for threads next to each other
    auto whole_at = [&](int r, int f) { return L::Y1 + r * B * 4 + ((f ^ (r & 7)) << 4); };
    // Y in front of a walk; false: nothing
    auto first_state = [&](const LaPart& c, float l2) {
        const LaJob& j = p.job[c.job];
        const float* from = STATES ? nullptr : j.starts ? la_start(p, j, c) : j.init ? j.init + la_state(p, j, c) : nullptr;
        if (!from) {
#pragma unroll
            for (int k = 0; k < L::YC; ++k) y[k] = 0.f;
            return false;
        }
        const bool flip = j.starts ? j.flip_starts : j.flip;
        const float first = j.early && !j.starts ? exp2f(l2) : 1.f;
        if (!flip && ((uintptr_t)from & 15) == 0) {
            float4 in[A * B / 4 / L::T];        // all reads on their way before the first is stored
#pragma unroll
            for (int k = 0; k < A * B / 4 / L::T; ++k) {
                const int i = k * L::T + tid, r = i / (B / 4), f = i % (B / 4);
                in[k] = r < j.a && 4 * f < j.b ? *(const float4*)(from + r * j.b + 4 * f) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < A * B / 4 / L::T; ++k) {
                const int i = k * L::T + tid;
                *(float4*)(sm + whole_at(i / (B / 4), i % (B / 4))) = in[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < L::YC; k += 4) {
                const float4 q = *(const float4*)(sm + whole_at(x, (y0 + k) / 4));
                y[k] = first * q.x; y[k + 1] = first * q.y; y[k + 2] = first * q.z; y[k + 3] = first * q.w;
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int k = 0; k < L::YC; ++k) {
                const int col = y0 + k;
                y[k] = x < j.a && col < j.b ? first * from[flip ? col * j.a + x : x * j.b + col] : 0.f;
            }
        }
        if (!STATES) put_pieces();
        return true;
    };

    float l2 = 0.f;
    bool carry = false;                                 // is there anything in Y?
    int table = 0, sums = 0;                            // the walk's powers; sums for Y so far
    if (more) {
        u = walks[0].begin;
        find_rows(walks[0], u);
        load_q(walks[0], u);
        load_kv(walks[0], u);
        l2 = la_log2_decay(p, walks[0].d, walks[0].h);
        set_powers(0, l2);
        carry = first_state(walks[0], l2);
    }
    for (uint32_t phase = 0; more; phase ^= 1) {
        const LaPart& at = walks[now];
        const LaJob& j = p.job[at.job];
        const int n = steps_of(at, u), steps = (n + 15) / 16, pieces = j.pieces;
        const bool final = u + kC >= at.end, sum = STATES || !final || (at.last && j.fin);
        const int then = final ? (now + 1) % 3 : now;
        const LaPart& to = walks[then];
        const bool next = !final || next_walk(walks + then);
        cp_async_wait();
        tc::fence_async_smem();
        tc::tc_fence_before_sync();
        __syncthreads();
        if (*(volatile int*)stop) break;
        const int then_u = final ? to.begin : u + kC;
        float next_l2 = l2;
        if (final && next) {
            next_l2 = la_log2_decay(p, to.d, to.h);
            set_powers(table ^ 1, next_l2);
        }
        if (next) find_rows(to, then_u);
        if (!STATES && tid == 0) {
            tc::tc_fence_after_sync();
            for (int k = 0; k < A / 16; ++k) {
                const uint32_t k0 = (k / 4) * kPanel + (k % 4) * 32;
                tc::mma_bf16_ss(tmem + L::S, tc::sdesc_sw128(base + L::Q + k0), tc::sdesc_sw128(base + L::K + k0),
                                tc::idesc_bf16_f32(128, 128), k > 0);
            }
            if (carry)
                for (int k = 0; k < 2 * (A / 16); ++k) {
                    const int s = k % (A / 16);
                    tc::mma_bf16_ss(tmem + L::O, tc::sdesc_sw128(base + L::Q + (s / 4) * kPanel + (s % 4) * 32),
                                    sdesc_mn(base + (k < A / 16 ? L::Y1 : L::Y2) + s * 2048, A * 128), tc::idesc_bf16_f32(128, B) | kBmn,
                                    k > 0);
                }
            tc::mma_commit(bar + DONE_S);
        }
        __syncwarp();
        // the weighted values in pieces
        constexpr int CH = B / 8, EACH = L::T / CH, IT = kC / EACH;
        uint4 third[L::in_q ? IT : 1];
        if (sum) {
            const int behind = decay_of(at, u);
            uint4 in[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) in[i] = *(const uint4*)(sm + L::V + tile_at(i * EACH + tid / CH, tid % CH, kPanel));
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int s = i * EACH + tid / CH;
                const uint32_t v0 = tile_at(s, tid % CH, kPanel);
                uint4 v = in[i];
                if (s >= n) v = make_uint4(0, 0, 0, 0);
                const float w = j.sK * exp2f(max(behind - s, 0) * l2);
                float f[8] = {low(v.x), high(v.x), low(v.y), high(v.y), low(v.z), high(v.z), low(v.w), high(v.w)};
#pragma unroll
                for (int e = 0; e < 8; e += 2) mul2(f[e], f[e + 1], w, w);
                uint4 a, b;
                a.x = cut(f[0], f[1]); a.y = cut(f[2], f[3]); a.z = cut(f[4], f[5]); a.w = cut(f[6], f[7]);
                *(uint4*)(sm + L::V1 + v0) = a;
                b.x = cut(f[0], f[1]); b.y = cut(f[2], f[3]); b.z = cut(f[4], f[5]); b.w = cut(f[6], f[7]);
                *(uint4*)(sm + L::V2 + v0) = b;
                if (pieces > 2) {
                    const uint4 last = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                    if (L::in_q) third[L::in_q ? i : 0] = last;
                    else *(uint4*)(sm + L::V3 + v0) = last;
                }
            }
        }
        float o[L::OC];
        constexpr int CPR = L::OC / 8, RPT = 32 / CPR;
        int rows_out[CPR];
        if (!STATES && L::in_q) {
            waited(DONE_S, phase);
            tc::tc_fence_after_sync();
        }
        if (L::in_q && sum && pieces > 2) {
#pragma unroll
            for (int i = 0; i < IT; ++i) *(uint4*)(sm + L::V3 + tile_at(i * EACH + tid / CH, tid % CH, kPanel)) = third[L::in_q ? i : 0];
        }
        if (!STATES) {
#pragma unroll
            for (int k = 0; k < CPR; ++k) rows_out[k] = row_of(at, u, j.back, quad * 32 + k * RPT + lane / CPR, n);
            if (!L::in_q) {
                waited(DONE_S, phase);
                tc::tc_fence_after_sync();
                if (next) load_q(to, then_u);
            }
        }
        if (!STATES) {
            const float* const power = powers + table * 64;
            // S to P, 32 columns at a time; each piece of P lies where its columns of S lay
#pragma unroll
            for (int b = part; b < 4; b += L::PARTS) {
                uint32_t w[16];
                if (b > quad) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0;
                } else {
                    float s[32];
                    load_columns(L::S + 32 * b, s);
                    if (b == quad && l2 < -3.f) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            w[e] = pack2(s[2 * e] * power[max(lane - 2 * e, 0)], s[2 * e + 1] * power[max(lane - 2 * e - 1, 0)]);
                    } else {
                        // lambda^(i-j) in two factors: from the block's last column on, and up to it; within the diagonal block the
                        // first is above 1, at most 2^93
                        const float f = exp2f((row - 32 * b - 31) * l2);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float4 g = *(const float4*)(power + 32 + 2 * e);
                            mul2(g.x, g.y, f, f);
                            mul2(g.z, g.w, f, f);
                            mul2(s[2 * e], s[2 * e + 1], g.x, g.y);
                            mul2(s[2 * e + 2], s[2 * e + 3], g.z, g.w);
                            w[e] = pack2(s[2 * e], s[2 * e + 1]);
                            w[e + 1] = pack2(s[2 * e + 2], s[2 * e + 3]);
                        }
                    }
                    if (b == quad) {                    // what is later than the row: bits, whatever they say, to zero
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] &= lane > 2 * e ? 0xffffffffu : lane == 2 * e ? 0xffffu : 0u;
                    }
                }
                tc::tmem_st_32x32b_x16(mine + L::S + 32 * b, w);
            }
            if (carry) {
                const float f = j.sI * exp2f(row * l2);
                load_columns(L::O + o0, o);
#pragma unroll
                for (int k = 0; k < L::OC; k += 2) mul2(o[k], o[k + 1], f, f);
            } else {
#pragma unroll
                for (int k = 0; k < L::OC; ++k) o[k] = 0.f;
            }
            tc::tmem_wait_st();
        }
        tc::fence_async_smem();
        tc::tc_fence_before_sync();
        __syncthreads();
        if (*(volatile int*)stop) break;
        if (tid == 0) {
            tc::tc_fence_after_sync();
            if (!STATES) {
                for (int k = 0; k < steps; ++k)
                    tc::mma_bf16_ts(tmem + L::O, tmem + L::S + 32 * (k / 2) + 8 * (k % 2), sdesc_mn(base + L::V + k * 2048, kPanel),
                                    tc::idesc_bf16_f32(128, B) | kBmn, k > 0);
                tc::mma_commit(bar + DONE_O);
            }
            if (sum) {
                for (int e = pieces - 1; e >= 0; --e)
                    for (int k = 0; k < steps; ++k)
                        // keys of 64 columns: the same panel again for the second 64 rows of the product
                        tc::mma_bf16_ss(tmem + L::Y, sdesc_mn(base + L::K + k * 2048, A == 128 ? kPanel : 0),
                                        sdesc_mn(base + (e == 0 ? L::V1 : e == 1 ? L::V2 : L::V3) + k * 2048, kPanel),
                                        tc::idesc_bf16_f32(128, B) | kAmn | kBmn, e < pieces - 1 || k > 0);
                tc::mma_commit(bar + DONE_Y);
            }
        }
        __syncwarp();
        if (!STATES) {
            // rows out: 16 bytes a thread and CPR threads a row, by way of the warp's part of the pieces of Y, which S and O have read
            unsigned char* const stage = sm + L::Y1 + warp * 64 * L::OC;
            __nv_bfloat16* const out = (__nv_bfloat16*)j.out.p + at.d * j.out.dir + at.h * j.out.head + at.slot * j.out.row + o0;
            waited(DONE_O, phase);
            tc::tc_fence_after_sync();
            float v[L::OC];
            load_columns(L::O + o0, v);
#pragma unroll
            for (int k = 0; k < L::OC; k += 2) fma2(v[k], v[k + 1], j.sP, o[k], o[k + 1]);
#pragma unroll
            for (int k = 0; k < CPR; ++k)
                *(uint4*)(stage + lane * 2 * L::OC + ((k ^ ((lane >> 1) & (CPR - 1))) << 4)) =
                    make_uint4(pack2(v[8 * k], v[8 * k + 1]), pack2(v[8 * k + 2], v[8 * k + 3]), pack2(v[8 * k + 4], v[8 * k + 5]),
                               pack2(v[8 * k + 6], v[8 * k + 7]));
            __syncwarp();
            uint4 w[CPR];
#pragma unroll
            for (int k = 0; k < CPR; ++k) {
                const int r = k * RPT + lane / CPR, ch = lane % CPR;
                w[k] = *(const uint4*)(stage + r * 2 * L::OC + ((ch ^ ((r >> 1) & (CPR - 1))) << 4));
            }
#pragma unroll
            for (int k = 0; k < CPR; ++k) {
                const int r = k * RPT + lane / CPR, ch = lane % CPR;
                if (quad * 32 + r < n && o0 + ch * 8 < j.b) *(uint4*)(out + rows_out[k] * j.out.row + ch * 8) = w[k];
            }
        }
        if (sum) {
            waited(DONE_Y, sums & 1);
            tc::tc_fence_after_sync();
            ++sums;
        }
        if (next) {
            if (L::in_q) load_q(to, then_u);
            load_kv(to, then_u);
        }
        if (sum) {
            float v[L::YC];
            const float keep = exp2f(decay_of(at, u) * l2);
            load_columns(L::Y + y0, v);
#pragma unroll
            for (int k = 0; k < L::YC; k += 2) fma2(y[k], y[k + 1], keep, v[k], v[k + 1]);
        }
        if (!STATES) __syncthreads();                   // the rows have left the pieces' place
        if (!final) {
            if (!STATES) put_pieces();
            carry = true;
        } else {
            if (sum) {
                float* const fin = STATES ? la_start(p, j, at) : j.fin + la_state(p, j, at);
                if (((uintptr_t)fin & 15) == 0) {       // widths are multiples of 8
#pragma unroll
                    for (int k = 0; k < L::YC; k += 4)
                        *(float4*)(sm + whole_at(x, (y0 + k) / 4)) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    __syncthreads();
#pragma unroll
                    for (int k = 0; k < A * B / 4 / L::T; ++k) {
                        const int i = k * L::T + tid, r = i / (B / 4), f = i % (B / 4);
                        if (r < j.a && 4 * f < j.b) *(float4*)(fin + r * j.b + 4 * f) = *(const float4*)(sm + whole_at(r, f));
                    }
                    __syncthreads();
                } else {
#pragma unroll
                    for (int k = 0; k < L::YC; ++k)
                        if (x < j.a && y0 + k < j.b) fin[x * j.b + y0 + k] = y[k];
                }
            }
            carry = next ? first_state(to, next_l2) : false;
            table ^= 1;
            l2 = next_l2;
        }
        now = then;
        u = then_u;
        more = next;
    }
    if (*(volatile int*)stop && tid == 0) {             // products still on their way read shared memory and write tensor memory
        tc::mma_commit(bar + DRAINED);
        tc::mbar_wait(bar + DRAINED, 0, 100000000ull);
    }
    __syncwarp();
    cp_async_wait();
    tc::tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after_sync();
        tc::tmem_dealloc(tmem, L::COLUMNS);
    }
}

template <int A, int B, bool STATES>
lstm_status launch(const LaArgs& a, cudaStream_t cs)
{
    typedef Layout<A, B> L;
    auto kernel = la_tensor_kernel<A, B, STATES>;
    LSTM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES));
    const int total = a.count * a.ndir * a.heads * a.jobs, ctas = a.sms * L::CTAS;
    kernel<<<total < ctas ? total : ctas, L::T, L::BYTES, cs>>>(a, total);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

template <int A, int B>
lstm_status launch_padded(const LaArgs& a, bool states, cudaStream_t cs)
{
    return states ? launch<A, B, true>(a, cs) : launch<A, B, false>(a, cs);
}

}  // namespace

// One translation unit each (la_tensor_*.cu).
lstm_status launch_la_64_64(const LaArgs& a, bool states, cudaStream_t cs);
lstm_status launch_la_64_128(const LaArgs& a, bool states, cudaStream_t cs);
lstm_status launch_la_128_64(const LaArgs& a, bool states, cudaStream_t cs);
lstm_status launch_la_128_128(const LaArgs& a, bool states, cudaStream_t cs);

}  // namespace lstm
