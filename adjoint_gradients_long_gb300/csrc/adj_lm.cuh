// adj_lm.cuh -- launchers of the log-probability and gradient-clipping kernels.
#pragma once
#include "adj_internal.cuh"

namespace adj {

struct LogprobArgs {
    int64_t N, V, ld, ldd;
    int top;
    const void *logits;
    const int64_t *targets;
    float *logp, *entropy, *lse;
    int32_t *top_id;
    float *top_logp;
    const float *glp, *gent;
    void *dlogits;
    int blocks, log_blocks;     // of a row, set by the launcher
};

cudaError_t launch_logprob(const LogprobArgs &a, bool bf16, cudaStream_t st);

size_t clip_ws_bytes();
cudaError_t launch_grad_clip(const adj_grad_seg *segs, int64_t nseg, float max_norm, float *out, char *ws,
                             cudaStream_t st);

}  // namespace adj
