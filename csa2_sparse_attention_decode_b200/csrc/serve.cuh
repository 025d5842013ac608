// Launchers of the calls a serving program makes around the CSA2 layers of a
// step: the token plan, the head norm with rotation, the prompt's attention
// and the verification of drafted tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/csa2.h"

namespace csa2 {

struct PlanArgs {
    int32_t batch, max_pages, n_pages, max_new;
    const int32_t *n_tokens, *n_new, *m;
    int32_t *page_table, *free_pages;
    const int32_t *n_free;
    int32_t *n_free_out, *cu_new, *token_req, *token_pos, *token_slot, *error;
};
cudaError_t launch_plan(const PlanArgs &a, cudaStream_t st);

struct NormRopeArgs {
    int32_t n, heads, kv_heads, rot_dim;
    const uint16_t *q, *k;
    int64_t q_stride, k_stride;                // elements from token to token
    const float *q_weight, *k_weight;
    uint16_t *q_out, *k_out;
    float *k_out_f32;
    const int32_t *pos, *n_valid;
    const float *inv_freq;
    float eps;
    uint32_t flags;
};
cudaError_t launch_norm_rope(const NormRopeArgs &a, int dim, cudaStream_t st);

struct VerifyArgs {
    int32_t batch, max_draft, vocab;
    const float *target, *probs;
    const int32_t *draft, *n_draft;
    const float *u;
    int32_t *n_accepted, *tokens, *error;
};
cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st);

struct PromptArgs {
    int32_t batch;
    const int32_t *cu_q, *cu_k;
    int32_t n_q, n_k, heads;
    const uint16_t *q, *lat;
    int64_t lat_stride;                        // elements from latent to latent
    int32_t window;
    float scale;
    void *out;
    int32_t out_is_fp32;
    float *lse;
    int32_t *error;
    void *ws;
};
size_t prompt_workspace_bytes(int64_t n_q, int heads, int64_t n_k);
cudaError_t launch_prompt_attend(const PromptArgs &a, cudaStream_t st);

}  // namespace csa2
