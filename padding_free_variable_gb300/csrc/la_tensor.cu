// la_tensor.cu -- linear attention on the tensor cores: which rows they take, launches by padded widths.
#include "la_tensor.cuh"

namespace lstm {

bool la_tensor_fits(const LaArgs& a)
{
    for (int k = 0; k < a.jobs; ++k) {
        const LaJob& j = a.job[k];
        if (j.a % 8 || j.b % 8) return false;
        for (const LaRows* r : {&j.q, &j.k, &j.v, &j.out})
            if ((uintptr_t)r->p % 16 || (a.rows > 1 && r->row % 8) || (a.ndir > 1 && r->dir % 8) || (a.heads > 1 && r->head % 8)) return false;
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
        const lstm_status st = wide == 0 ? launch_la_64_64(some, states, cs) : wide == 1 ? launch_la_64_128(some, states, cs)
                             : wide == 2 ? launch_la_128_64(some, states, cs) : launch_la_128_128(some, states, cs);
        if (st != LSTM_OK) return st;
    }
    return LSTM_OK;
}

}  // namespace lstm
