// la_tensor.cu -- linear attention of bf16 rows on the tensor cores (tcgen05, accumulators in tensor memory).
//
// A CTA walks one head of one sequence (or a piece of it) 128 steps at a time.  Per chunk, with M = 128 rows of a product:
//     S = Q K^T                  128 x 128     O = Q Y           128 x B    (Y in two bf16 pieces)
//     P = S lambda^(i-j), i >= j, rounded to bf16, back into tensor memory as the next product's left operand
//     O' = P V                   128 x B       out = sP O' + sI lambda^i O
//     Y = lambda^n Y + K^T (sK lambda^(n-j) V) A x B            (the weighted values in three bf16 pieces: fp32 accuracy)
// Rows come by cp.async into the 128-byte swizzled layout, one image of 64 columns a panel: read along a row it is the
// K-major operand of S, read along a column the MN-major operand of the other products, so nothing is transposed.  Y stays in
// tensor memory; once a chunk it is read, cut into pieces for the next chunk and decayed.
#include <type_traits>

#include "la.cuh"
#include "tc_ptx.cuh"

namespace lstm {

namespace {

constexpr int kC = 128, kThreads = 256, kPanel = kC * 128;      // steps, threads, bytes of 64 columns of all steps

// A: width of queries and keys, B: of values, padded to 64 or 128.
template <int A, int B> struct Layout {
    static constexpr int Q = 0, K = Q + kC * A * 2, V = K + kC * A * 2, V1 = V + kC * B * 2, V2 = V1 + kC * B * 2;
    static constexpr bool in_q = A >= B;                        // the third piece takes the queries' place
    static constexpr int V3 = in_q ? Q : V2 + kC * B * 2;
    static constexpr int Y1 = (in_q ? V2 : V3) + kC * B * 2, Y2 = Y1 + A * B * 2;
    static constexpr int W = Y2 + A * B * 2, G = W + (kC + 4) * 4, BARS = G + 32 * 4, BYTES = BARS + 32;
    // tensor memory, columns
    static constexpr uint32_t S = 0, O = 128, Y = O + B, COLUMNS = B == 64 ? 256 : 512;
    static constexpr int YC = A == 128 ? B / 2 : B / 4, OC = B / 2;     // columns of a thread
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

// Two values less what their first piece holds.
__device__ __forceinline__ uint32_t cut(float& x, float& y)
{
    const uint32_t w = pack2(x, y);
    x -= low(w);
    y -= high(w);
    return w;
}

// STATES: only what a piece adds to Y, into `starts`.
template <int A, int B, bool STATES>
__global__ void __launch_bounds__(kThreads, A == 64 && B == 64 ? 2 : 1) la_tensor_kernel(const __grid_constant__ LaArgs p)
{
    typedef Layout<A, B> L;
    extern __shared__ __align__(1024) unsigned char sm[];
    const LaPart c = la_part(p, blockIdx.x);
    const LaJob& j = p.job[c.job];
    if (STATES && c.last) return;
    const int64_t state = la_state(p, j, c);
    if (!STATES) {
        la_past_end<__nv_bfloat16>(p, j, c);
        if (c.len == 0) return la_pass(j, state);
    }
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, quad = warp % 4, half = warp / 4;
    const uint32_t base = tc::smem_u32(sm);
    float* const W = (float*)(sm + L::W);               // lambda^n
    float* const G = (float*)(sm + L::G);               // lambda^(31-n)
    uint64_t* const bar = (uint64_t*)(sm + L::BARS);    // [0] queries read, [1] chunk done
    uint32_t* const slot_of_tmem = (uint32_t*)(bar + 2);
    int* const stop = (int*)(slot_of_tmem + 1);
    const bool rev = (c.d == 1) != (j.back != 0);
    const float l2 = la_log2_decay(p, c.d, c.h);
    if (tid == 0) {
        tc::mbar_init(bar, 1);
        tc::mbar_init(bar + 1, 1);
        *stop = 0;
        tc::fence_mbar_init();
    }
    if (warp == 0) {
        tc::tmem_alloc(slot_of_tmem, L::COLUMNS);
        tc::tmem_relinquish();
    }
    if (tid <= kC) W[tid] = exp2f(tid * l2);
    if (tid < 32) G[tid] = exp2f((31 - tid) * l2);

    // rows of one operand: 16 bytes a thread, rows next to each other in the panels
    auto load = [&](const LaRows& r, int to, int w, auto width, int u, int n) {
        constexpr int CH = decltype(width)::value / 8, EACH = kThreads / CH;
        const int ch = tid % CH;
        const __nv_bfloat16* from = (const __nv_bfloat16*)r.p + c.d * r.dir + c.h * r.head;
#pragma unroll
        for (int i = 0; i < kC / EACH; ++i) {
            const int s = i * EACH + tid / CH;
            const bool on = s < n && ch * 8 < w;
            const int t = rev ? c.len - 1 - (u + s) : u + s;
            const __nv_bfloat16* at = on ? from + (int64_t)(__ldg(p.off + t) + c.slot) * r.row + ch * 8 : from;
            cp_async16(base + to + tile_at(s, ch, kPanel), at, on);
        }
    };
    auto load_chunk = [&](int u) {
        const int n = min(kC, c.end - u);
        if (!STATES) load(j.q, L::Q, j.a, std::integral_constant<int, A>(), u, n);
        load(j.k, L::K, j.a, std::integral_constant<int, A>(), u, n);
        load(j.v, L::V, j.b, std::integral_constant<int, B>(), u, n);
    };
    load_chunk(c.begin);
    tc::tc_fence_before_sync();
    __syncthreads();
    tc::tc_fence_after_sync();
    const uint32_t tmem = *slot_of_tmem, mine = tmem + ((uint32_t)(quad * 32) << 16);
    const int row = quad * 32 + lane;                   // of S and O
    // of Y: with A = 64 the second 64 lanes hold the rows once more, for other columns
    const int x = row % A, y0 = A == 128 ? half * L::YC : ((quad >> 1) * 2 + half) * L::YC;
    const int o0 = half * L::OC;

    auto failed = [&](bool ok, unsigned where) {
        if (!ok) {
            *(volatile int*)stop = 1;
            record_failure(p.status, LSTM_ERR_TIMEOUT, 0x90000u | where);
        }
    };
    // Y in front of a chunk of n steps: its pieces for the outputs, decayed by the chunk for the sum of its products.
    auto put_state = [&](float (&y)[L::YC], float keep) {
#pragma unroll
        for (int k = 0; k < L::YC; k += 16) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(y[k + e] * keep);
            tc::tmem_st_32x32b_x16(mine + L::Y + y0 + k, r);
            if (!STATES) {
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint4 hi, lo;
                    hi.x = cut(y[k + e], y[k + e + 1]); hi.y = cut(y[k + e + 2], y[k + e + 3]);
                    hi.z = cut(y[k + e + 4], y[k + e + 5]); hi.w = cut(y[k + e + 6], y[k + e + 7]);
                    lo.x = pack2(y[k + e], y[k + e + 1]); lo.y = pack2(y[k + e + 2], y[k + e + 3]);
                    lo.z = pack2(y[k + e + 4], y[k + e + 5]); lo.w = pack2(y[k + e + 6], y[k + e + 7]);
                    const uint32_t at = tile_at(x, (y0 + k + e) / 8, A * 128);
                    *(uint4*)(sm + L::Y1 + at) = hi;
                    *(uint4*)(sm + L::Y2 + at) = lo;
                }
            }
        }
        tc::tmem_wait_st();
    };
    auto get_state = [&](float (&y)[L::YC]) {
#pragma unroll
        for (int k = 0; k < L::YC; k += 16) {
            uint32_t r[16];
            tc::tmem_ld_32x32b_x16(mine + L::Y + y0 + k, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) y[k + e] = __uint_as_float(r[e]);
        }
    };
    // steps that a chunk's state decays by: one less behind the last step of a walk whose final state holds one lambda less
    auto powers = [&](int u) { return min(kC, c.end - u) - (c.last && u + kC >= c.end ? j.early : 0); };

    const float* from = STATES ? nullptr : j.starts ? la_start(p, j, c) : j.init ? j.init + state : nullptr;
    bool carry = from != nullptr;                       // is there anything in Y?
    if (carry) {
        float y[L::YC];
        const float first = j.early && !j.starts ? W[1] : 1.f;
#pragma unroll
        for (int k = 0; k < L::YC; ++k) {
            const int col = y0 + k;
            y[k] = x < j.a && col < j.b ? first * from[j.flip && !j.starts ? col * j.a + x : x * j.b + col] : 0.f;
        }
        put_state(y, W[powers(c.begin)]);
    }
    uint32_t phase = 0;
    for (int u = c.begin; u < c.end; u += kC, phase ^= 1) {
        const int n = min(kC, c.end - u), steps = (n + 15) / 16;
        const bool final = u + kC >= c.end, sum = STATES || !final || (c.last && j.fin);
        cp_async_wait();
        tc::fence_async_smem();
        tc::tc_fence_before_sync();
        __syncthreads();
        if (*(volatile int*)stop) break;
        if (!STATES && tid == 0) {
            tc::tc_fence_after_sync();
            for (int k = 0; k < A / 16; ++k) {
                const uint32_t at = (k / 4) * kPanel + (k % 4) * 32;
                tc::mma_bf16_ss(tmem + L::S, tc::sdesc_sw128(base + L::Q + at), tc::sdesc_sw128(base + L::K + at),
                                tc::idesc_bf16_f32(128, 128), k > 0);
            }
            if (carry)
                for (int k = 0; k < 2 * (A / 16); ++k) {
                    const int s = k % (A / 16);
                    tc::mma_bf16_ss(tmem + L::O, tc::sdesc_sw128(base + L::Q + (s / 4) * kPanel + (s % 4) * 32),
                                    sdesc_mn(base + (k < A / 16 ? L::Y1 : L::Y2) + s * 2048, A * 128), tc::idesc_bf16_f32(128, B) | kBmn,
                                    k > 0);
                }
            tc::mma_commit(bar);
        }
        __syncwarp();
        // the weighted values in pieces
        constexpr int CH = B / 8, EACH = kThreads / CH, IT = kC / EACH;
        uint4 third[IT];
        if (sum) {
            const int behind = powers(u);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int s = i * EACH + tid / CH;
                const uint32_t at = tile_at(s, tid % CH, kPanel);
                const uint4 v = *(const uint4*)(sm + L::V + at);
                const float w = s < n ? j.sK * W[behind - s] : 0.f;
                float f[8] = {low(v.x) * w, high(v.x) * w, low(v.y) * w, high(v.y) * w, low(v.z) * w, high(v.z) * w, low(v.w) * w, high(v.w) * w};
                uint4 a, b;
                a.x = cut(f[0], f[1]); a.y = cut(f[2], f[3]); a.z = cut(f[4], f[5]); a.w = cut(f[6], f[7]);
                b.x = cut(f[0], f[1]); b.y = cut(f[2], f[3]); b.z = cut(f[4], f[5]); b.w = cut(f[6], f[7]);
                third[i] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                *(uint4*)(sm + L::V1 + at) = a;
                *(uint4*)(sm + L::V2 + at) = b;
            }
        }
        float o[L::OC];
        if (!STATES) {
            failed(tc::mbar_wait(bar, phase, p.limit_ns), 1);
            __syncwarp();
            tc::tc_fence_after_sync();
        }
        if (sum) {
#pragma unroll
            for (int i = 0; i < IT; ++i) *(uint4*)(sm + L::V3 + tile_at(i * EACH + tid / CH, tid % CH, kPanel)) = third[i];
        }
        if (!STATES) {
            // S to P, 32 columns at a time; each piece of P lies where its columns of S lay
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int b = half + 2 * k;
                uint32_t w[16];
                if (b > quad) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0;
                } else {
                    uint32_t r0[16], r1[16];
                    tc::tmem_ld_32x32b_x16(mine + L::S + 32 * b, r0);
                    tc::tmem_ld_32x32b_x16(mine + L::S + 32 * b + 16, r1);
                    tc::tmem_wait_ld();
                    if (b == quad) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float s0 = __uint_as_float(e < 8 ? r0[2 * e % 16] : r1[2 * e % 16]);
                            float s1 = __uint_as_float(e < 8 ? r0[(2 * e + 1) % 16] : r1[(2 * e + 1) % 16]);
                            s0 = lane >= 2 * e ? s0 * W[max(lane - 2 * e, 0)] : 0.f;
                            s1 = lane >= 2 * e + 1 ? s1 * W[max(lane - 2 * e - 1, 0)] : 0.f;
                            w[e] = pack2(s0, s1);
                        }
                    } else {
                        const float f = W[row - 32 * b - 31];
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 g = *(const float4*)(G + 2 * e);
                            const float s0 = __uint_as_float(e < 8 ? r0[2 * e % 16] : r1[2 * e % 16]);
                            const float s1 = __uint_as_float(e < 8 ? r0[(2 * e + 1) % 16] : r1[(2 * e + 1) % 16]);
                            const float s2 = __uint_as_float(e < 8 ? r0[(2 * e + 2) % 16] : r1[(2 * e + 2) % 16]);
                            const float s3 = __uint_as_float(e < 8 ? r0[(2 * e + 3) % 16] : r1[(2 * e + 3) % 16]);
                            w[e] = pack2(s0 * (f * g.x), s1 * (f * g.y));
                            w[e + 1] = pack2(s2 * (f * g.z), s3 * (f * g.w));
                        }
                    }
                }
                tc::tmem_st_32x32b_x16(mine + L::S + 32 * b, w);
            }
            if (carry) {
                const float f = j.sI * W[row];
#pragma unroll
                for (int k = 0; k < L::OC; k += 16) {
                    uint32_t r[16];
                    tc::tmem_ld_32x32b_x16(mine + L::O + o0 + k, r);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[k + e] = f * __uint_as_float(r[e]);
                }
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
            if (!STATES)
                for (int k = 0; k < steps; ++k)
                    tc::mma_bf16_ts(tmem + L::O, tmem + L::S + 32 * (k / 2) + 8 * (k % 2), sdesc_mn(base + L::V + k * 2048, kPanel),
                                    tc::idesc_bf16_f32(128, B) | kBmn, k > 0);
            if (sum)
                for (int e = 0; e < 3; ++e)
                    for (int k = 0; k < steps; ++k)
                        // keys of 64 columns: the same panel again for the second 64 rows of the product
                        tc::mma_bf16_ss(tmem + L::Y, sdesc_mn(base + L::K + k * 2048, A == 128 ? kPanel : 0),
                                        sdesc_mn(base + (e == 0 ? L::V1 : e == 1 ? L::V2 : L::V3) + k * 2048, kPanel),
                                        tc::idesc_bf16_f32(128, B) | kAmn | kBmn, carry || e > 0 || k > 0);
            tc::mma_commit(bar + 1);
        }
        __syncwarp();
        failed(tc::mbar_wait(bar + 1, phase, p.limit_ns), 2);
        __syncwarp();
        tc::tc_fence_after_sync();
        if (!final) load_chunk(u + kC);
        if (!STATES) {
            const int t = rev ? c.len - 1 - (u + row) : u + row;
            __nv_bfloat16* const to = row < n ? (__nv_bfloat16*)j.out.p + (int64_t)(__ldg(p.off + t) + c.slot) * j.out.row + c.d * j.out.dir +
                                                    c.h * j.out.head + o0
                                              : nullptr;
#pragma unroll
            for (int k = 0; k < L::OC; k += 16) {
                uint32_t r[16];
                tc::tmem_ld_32x32b_x16(mine + L::O + o0 + k, r);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    float v[8];
#pragma unroll
                    for (int m = 0; m < 8; ++m) v[m] = fmaf(j.sP, __uint_as_float(r[e + m]), o[k + e + m]);
                    if (to && o0 + k + e < j.b)
                        *(uint4*)(to + k + e) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                }
            }
        }
        if (sum) {
            float y[L::YC];
            get_state(y);
            if (!final) {
                carry = true;
                put_state(y, W[powers(u + kC)]);
            } else {
                float* const to = STATES ? la_start(p, j, c) : j.fin + state;
#pragma unroll
                for (int k = 0; k < L::YC; ++k)
                    if (x < j.a && y0 + k < j.b) to[x * j.b + y0 + k] = y[k];
            }
        }
    }
    cp_async_wait();
    tc::tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::tc_fence_after_sync();
        tc::tmem_dealloc(tmem, L::COLUMNS);
    }
}

template <int A, int B>
lstm_status launch(const LaArgs& a, bool states, cudaStream_t cs)
{
    auto kernel = states ? la_tensor_kernel<A, B, true> : la_tensor_kernel<A, B, false>;
    LSTM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<A, B>::BYTES));
    kernel<<<(unsigned)((int64_t)a.count * a.ndir * a.heads * a.jobs), kThreads, Layout<A, B>::BYTES, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? LSTM_OK : LSTM_ERR_CUDA;
}

}  // namespace

bool la_tensor_fits(const LaArgs& a)
{
    for (int k = 0; k < a.jobs; ++k) {
        const LaJob& j = a.job[k];
        if (j.a % 8 || j.b % 8) return false;
        for (const LaRows* r : {&j.q, &j.k, &j.v, &j.out})
            if ((uintptr_t)r->p % 16 || r->row % 8 || (a.ndir > 1 && r->dir % 8) || (a.heads > 1 && r->head % 8)) return false;
    }
    return true;
}

lstm_status launch_la_tensor(const LaArgs& a, bool states, cudaStream_t cs)
{
    // jobs of one pair of padded widths to a launch
    for (int wide = 0; wide < 4; ++wide) {
        LaArgs some = a;
        some.jobs = 0;
        for (int k = 0; k < a.jobs; ++k)
            if ((a.job[k].a > 64) * 2 + (a.job[k].b > 64) == wide) some.job[some.jobs++] = a.job[k];
        if (some.jobs == 0) continue;
        const lstm_status st = wide == 0 ? launch<64, 64>(some, states, cs) : wide == 1 ? launch<64, 128>(some, states, cs)
                             : wide == 2 ? launch<128, 64>(some, states, cs) : launch<128, 128>(some, states, cs);
        if (st != LSTM_OK) return st;
    }
    return LSTM_OK;
}

}  // namespace lstm
