// Token log probabilities and their gradient (lora_logprob.cu): what the host
// ABI hands to the kernels.
#pragma once
#include "lora_internal.cuh"

namespace rd {

struct LogprobParams {
    const void *logits;    // M rows of V, row stride in elements
    int64_t stride;
    int M, V;
    const int32_t *tokens; // [M], or nullptr
    float inv_t;
    int top_k;
    float *logprob;        // [M], or nullptr
    float *entropy;        // [M], or nullptr
    float *stats;          // [M][2], or nullptr
    int32_t *top_ids;      // [M][top_k]
    float *top_logprobs;   // [M][top_k]
    uint32_t *status;
};

struct LogprobGradParams {
    const void *logits;
    int64_t stride;
    int M, V;
    const int32_t *tokens;     // [M], or nullptr
    float inv_t;
    const float *stats;        // [M][2]
    const float *entropy;      // [M] (with g_entropy)
    const float *g_logprob;    // [M], or nullptr
    const float *g_entropy;    // [M], or nullptr
    void *dlogits;
    int64_t d_stride;
};

cudaError_t launch_logprob(const LogprobParams &p, int dtype, int num_sms, cudaStream_t st);
cudaError_t launch_logprob_grad(const LogprobGradParams &p, int dtype, cudaStream_t st);

} // namespace rd
