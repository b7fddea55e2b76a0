// Distillation from a teacher's best tokens (lora_distill.cu): what the host
// ABI hands to the kernels.
#pragma once
#include "lora_internal.cuh"

namespace rd {

struct DistillParams {
    const void *logits; // M rows of V, row stride in elements
    int64_t stride;
    int M, V;
    float inv_t;
    const int32_t *ids;   // [M][n]
    const float *teacher; // [M][n]
    int n;
    int rest;             // the rest of the vocabulary is one more class
    float *loss;          // [M]; not the gradient by itself
    float *stats;         // [M][LORA_DISTILL_STATS], or nullptr; read by the gradient by itself
    const float *g;       // [M]
    void *dlogits;        // or nullptr
    int64_t d_stride;
    uint32_t *status;
};

cudaError_t launch_distill(const DistillParams &p, int dtype, int num_sms, cudaStream_t st);
cudaError_t launch_distill_grad(const DistillParams &p, int dtype, cudaStream_t st);

} // namespace rd
