// The plan, the checks and the commit of a compaction, for both caches (internal header; apart from
// kara_common.cuh, whose kernels' recorded profiles hold for that header as it was).
#pragma once

#include "kara_tokens.cuh"

namespace kara {

// Releases the old tail of sequence s, installs the fresh ids and sets the new length, unless an error was
// recorded; `lanes` threads together.
__device__ __forceinline__ void commit_sequence(const Geo &g, const SeqPlan &p, int32_t error, const int32_t *fresh,
                                                int32_t *freed, int32_t *new_len, int32_t *bt, int s, int lane, int lanes)
{
    if (error != 0 || p.p0 < 0) {
        if (lane == 0) new_len[s] = g.len[s];
        return;
    }
    int32_t *row = bt + (int64_t)s * g.bt_stride + p.p0;
    for (int t = lane; t < p.n_old; t += lanes) {
        const int32_t old = row[t];
        freed[p.off_old + t] = old;
        row[t] = t < p.n_new ? fresh[p.off_new + t] : -1;
    }
    if (lane == 0) new_len[s] = p.Lnew;
}

// Launchers of kara_common.cuh, and of the parts of theirs, with a choice (dependent: as a programmatic dependent of
// what precedes it on the stream).
cudaError_t launch_plan(const Geo &g, int64_t n_fresh, SeqPlan *plan, int32_t *err, cudaStream_t st, bool dependent);
cudaError_t launch_fresh_check(const Geo &g, const SeqPlan *plan, const int32_t *fresh, int64_t n_fresh,
                               int32_t *err, cudaStream_t st, bool dependent);
cudaError_t launch_kept_check(const Geo &g, const int32_t *kept, int32_t *err, cudaStream_t st, bool dependent);
cudaError_t launch_commit(const Geo &g, const SeqPlan *plan, const int32_t *fresh, int32_t *freed,
                          int32_t *new_len, int32_t *bt, const int32_t *err, cudaStream_t st, bool dependent);
cudaError_t launch_prepare(const Geo &g, const int32_t *kept, const int32_t *fresh, int64_t n_fresh, SeqPlan *plan,
                           int32_t *done, int32_t *err, cudaStream_t st);

}  // namespace kara
