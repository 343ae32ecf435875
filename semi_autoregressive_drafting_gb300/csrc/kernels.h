// kernels.h -- host launchers of the libdspark kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dspark {

// dst[c][r] = src[r][c] for a rows x cols matrix of 2- or 4-byte elements (es), both row-major.
cudaError_t launch_transpose(const void* src, void* dst, int rows, int cols, int es, cudaStream_t stream);
cudaError_t launch_confidence(int B, int G, int V, int r, int d, int w_bf16, const void* W1,
                              const void* w, int u_bf16, const void* h, const int32_t* x0,
                              const int32_t* tokens, float* c, float* S, cudaStream_t stream);
cudaError_t launch_tv_label(int N, int V, float T, const float* d, const float* t, float* cstar,
                            float* l1, cudaStream_t stream);
size_t verify_workspace_bytes(int B, int G, int V);
cudaError_t launch_verify(int B, int G, int V, float T, uint64_t seed, const float* zd,
                          const float* zt, const int32_t* tok, int32_t* n_acc, int32_t* out,
                          void* workspace, cudaStream_t stream);
size_t loss_workspace_bytes(int B, int G, int V);
cudaError_t launch_loss(int B, int G, int V, float T, const float* zd, const float* zt,
                        const int32_t* lab, const float* conf, float a_ce, float a_tv, float a_conf,
                        float* loss, float* parts, float* grad_z, float* grad_c, void* workspace,
                        cudaStream_t stream);
size_t sts_workspace_bytes(int N, int G, int ng, int bins);
cudaError_t launch_sts(int N, int G, const float* conf, const int32_t* acc, int ng, const float* grid,
                       int bins, float* tau, float* ece, float* ece_grid, void* workspace,
                       cudaStream_t stream);
cudaError_t launch_prefix_schedule(int B, int G, const float* S, const double* sps, int32_t* len,
                                   double* theta, cudaStream_t stream);
size_t logprobs_workspace_bytes(int N, int V, int top);
cudaError_t launch_logprobs(int N, int V, float T, int bf16, const void* logits, long long ld,
                            const int32_t* tokens, int top, float* logp, float* norm, float* entropy,
                            int32_t* rank, int32_t* top_ids, float* top_logp, void* workspace,
                            cudaStream_t stream);
cudaError_t launch_logprobs_grad(int N, int V, float T, int bf16, const void* logits, long long ld,
                                 const int32_t* tokens, const float* norm, const float* entropy,
                                 const float* gl, const float* gh, void* grad, long long gld,
                                 cudaStream_t stream);
cudaError_t launch_embedding(int N, int V, int D, float scale, int w_bf16, const void* W,
                             const int32_t* tokens, int o_bf16, void* out, cudaStream_t stream);
size_t embedding_grad_workspace_bytes(int N, int V, int D);
cudaError_t launch_embedding_grad(int N, int V, int D, float scale, int g_bf16, const void* grad,
                                  const int32_t* tokens, int o_bf16, void* gW, int accumulate,
                                  void* workspace, cudaStream_t stream);
size_t bias_grad_workspace_bytes(int N, int V, int r, int w_bf16, int nsm);
cudaError_t launch_bias_grad(int N, int V, int r, int g_bf16, const void* G, int w_bf16, const void* a,
                             const void* W2, int w2_rv, float* grad_a, float* grad_W2, int accumulate,
                             int stuck, void* workspace, int nsm, cudaStream_t stream);
// grad: `in` is the gradient with respect to the processed logits and `raw` the logits (of out's type);
// otherwise `in` is the logits and `raw` is not used.
cudaError_t launch_process(int grad, int B, int R, int V, int i_bf16, const void* in, long long in_ld, int o_bf16,
                           void* out, long long out_ld, const void* raw, long long raw_ld, const int32_t* history,
                           long long history_ld, int H, const int32_t* lengths, const int32_t* prompts,
                           const int32_t* drafted, const float* repetition, const float* presence,
                           const float* frequency, int nb, const int32_t* bias_tokens, const float* bias,
                           const uint32_t* mask, long long mask_ld, int M, const int32_t* mask_rows,
                           int nsm, cudaStream_t stream);
size_t distill_workspace_bytes(int N, int V, int K);
// norm_in: the gradient alone, from an earlier call's normalisers (then loss, parts and norm are NULL).
cudaError_t launch_distill(int N, int V, float T, int bf16, const void* logits, long long ld, int K,
                           const int32_t* ids, const float* logq, const float* weight, float a_kl, float a_l1,
                           int rest, const float* norm_in, float* loss, float* parts, float* norm, void* grad,
                           long long gld, int stuck, void* workspace, int nsm, cudaStream_t stream);

}  // namespace dspark
