// Launchers of the new-token entry points (internal header).
#pragma once

#include "kara_common.cuh"

namespace kara {

// Limit of the bounded waits of a call that stages its copies as usual, for tests: KARA_DEBUG_WAIT_NS
// nanoseconds if that is in the environment.
inline uint64_t debug_wait(uint64_t normal_ns)
{
    const char *v = getenv("KARA_DEBUG_WAIT_NS");
    return v ? strtoull(v, nullptr, 10) : normal_ns;
}

// Launches `kern` as a programmatic dependent of what precedes it on the stream: its launch overlaps
// that grid's end, and it reads nothing global before its griddepcontrol.wait.
template <class... A>
cudaError_t launch_dependent(void (*kern)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

cudaError_t launch_extend(int32_t num_blocks, const int32_t *len, const int32_t *n_new, int32_t *bt, int32_t bt_stride,
                          const int32_t *fresh, int64_t n_fresh, const kara_tokens *t,
                          int32_t *used, int32_t *err, cudaStream_t st);
cudaError_t launch_append(const kara_cache *c, int32_t layer, const kara_tokens *t, const kara_rope *r, const void *q,
                          int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          void *q_out, void *ring, int32_t W, int32_t *err, cudaStream_t st);
size_t chunk_workspace_bytes(const kara_cache *c);
cudaError_t launch_chunk(const kara_cache *c, int32_t layer, const kara_tokens *t, const int32_t *bt,
                         int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st);

}  // namespace kara
