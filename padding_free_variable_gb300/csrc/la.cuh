// la.cuh -- linear attention with a decay for each head: arguments shared by its kernels.
//
// One operator serves the forward pass and all three gradients.  In the order of its own time u = 0, 1, ...
//     out_u = sum_{w <= u} sP lambda^(u-w) (q_u . k_w) v_w + sI lambda^u q_u^T Y
// where Y [a x b] is what came before; behind c steps Y becomes lambda^c Y + sK sum_w lambda^(c-w) k_w v_w^T.
//     forward  q, k, v as they are      Y = lambda S_0     sP = sI = scale, sK = 1
//     dq       dy, v, k                 Y = lambda S_0^T   the same
//     dk       v, dy, q, time reversed  Y = dS_n^T         sP = sK = scale, sI = 1
//     dv       k, q, dy, time reversed  Y = dS_n           the same
// Y holds one factor lambda more than S behind the same steps, and as many as dS in front of them: the final state
// of the forward pass takes one factor less at its last step (`early`), dS_0 is Y itself.
#pragma once

#include "scan_plan.cuh"

namespace lstm {

constexpr int kLaMax = 128;             // largest key or value size
constexpr int kLaMaxSteps = 1 << 30;    // longest sequence: a step and a chunk more stay within 32 bits

struct LaRows {
    const void* p = nullptr;
    int64_t row = 0, dir = 0, head = 0;
};

struct LaJob {
    LaRows q, k, v, out;                // out is written
    int a = 0, b = 0;                   // widths of q and k, of v and out
    const float* init = nullptr;        // [ndir][B][heads][a][b], or [b][a] with `flip`
    float* fin = nullptr;               // [ndir][B][heads][a][b]
    float* starts = nullptr;            // cut sequences: Y in front of each piece, [entry][ndir * heads][a][b] ([b][a] with `flip_starts`)
    float sP = 1.f, sI = 1.f, sK = 1.f;
    int flip = 0, flip_starts = 0, back = 0, early = 0;
    int pieces = 3;                     // bf16 pieces of a weighted value in Y's products (tensor cores)
};

struct LaArgs {
    int heads = 0, ndir = 0, B = 0, T = 0, padded = 0;
    const int32_t* off = nullptr;
    const int32_t* perm = nullptr;
    const float* log_decay = nullptr;
    const int4* pieces = nullptr;       // (slot, piece, length of the sequence, entry of the slot's first piece)
    int count = 0, piece = 0;           // pieces and their steps
    int jobs = 0, sms = 0;
    int64_t rows = 0;
    LaJob job[3];
    DeviceStatus* status = nullptr;
    unsigned long long limit_ns = 0;
};

// What a block works on: a piece of a sequence, a direction and head, and one of the jobs (the jobs of one piece
// next to each other, as they read the same rows).
struct LaPart {
    int job, d, h, slot, piece, entry, begin, end, len;
    bool last;
};

__device__ __forceinline__ LaPart la_part(const LaArgs& p, unsigned id)
{
    LaPart c;
    c.job = id % p.jobs;
    id /= p.jobs;
    const int dh = id % (p.ndir * p.heads);
    const int4 e = __ldg(p.pieces + id / (p.ndir * p.heads));
    c.d = dh / p.heads;
    c.h = dh - c.d * p.heads;
    c.slot = e.x; c.piece = e.y; c.len = e.z; c.entry = e.w + e.y;
    c.begin = (int)min((int64_t)e.y * p.piece, (int64_t)e.z);
    c.end = (int)min((int64_t)c.begin + p.piece, (int64_t)e.z);
    c.last = c.end == e.z;
    return c;
}

// log2 of a head's decay: at most 0, and low enough that any power but the 0th is 0 in fp32.
__device__ __forceinline__ float la_log2_decay(const LaArgs& p, int d, int h)
{
    return fminf(fmaxf(__ldg(p.log_decay + d * p.heads + h), -138.f), 0.f) * 1.4426950408889634f;
}

// The padded comparator's rows past a sequence's end: zeros, written by the block of its first piece.
template <typename T>
__device__ __forceinline__ void la_past_end(const LaArgs& p, const LaJob& j, const LaPart& c)
{
    if (!p.padded || c.piece != 0) return;
    T* const out = (T*)j.out.p + c.d * j.out.dir + c.h * j.out.head;
    for (int64_t i = threadIdx.x; i < (int64_t)(p.T - c.len) * j.b; i += blockDim.x)
        out[(int64_t)(__ldg(p.off + c.len + (int)(i / j.b)) + c.slot) * j.out.row + (int)(i % j.b)] = (T)0.f;
}

// Where a sequence's state lies, and Y's start for a piece.
__device__ __forceinline__ int64_t la_state(const LaArgs& p, const LaJob& j, const LaPart& c)
{
    return (((int64_t)c.d * p.B + __ldg(p.perm + c.slot)) * p.heads + c.h) * j.a * j.b;
}

__device__ __forceinline__ float* la_start(const LaArgs& p, const LaJob& j, const LaPart& c)
{
    return j.starts + ((int64_t)c.entry * p.ndir * p.heads + c.d * p.heads + c.h) * j.a * j.b;
}

// No step: the state that came in goes out.
__device__ __forceinline__ void la_pass(const LaJob& j, int64_t state)
{
    if (!j.fin || j.fin == j.init) return;
    for (int i = threadIdx.x; i < j.a * j.b; i += blockDim.x) j.fin[state + i] = j.init ? j.init[state + i] : 0.f;
}

lstm_status launch_la_general(const LaArgs& a, bool bf16, bool states, cudaStream_t cs);
lstm_status launch_la_tensor(const LaArgs& a, bool states, cudaStream_t cs);
bool la_tensor_fits(const LaArgs& a);     // bf16 rows that its 16-byte loads can take

}  // namespace lstm
