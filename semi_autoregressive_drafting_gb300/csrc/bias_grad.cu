// bias_grad.cu -- the gradients of the low-rank bias product B_k = a W2 (Eq 5; Eq 6 with
// a = tanh(o)), "DSpark -- paper verification", section 1.
//
// For gradients G [N][V] of the logits, conditioning rows a [N][r] and W2 as [V][r] or [r][V]:
//   grad_a[n][j] = sum_v G[n][v] W2[v][j],   grad_W2[v][j] = sum_n G[n][v] a[n][j].
#include "common.cuh"
#include "kernels.h"

namespace dspark {
namespace {

// C[m][n] (+)= sum_k A(m, k) B(k, n) over 32 x 32 tiles; A and B by row and column strides.
template <typename TA, typename TB>
__global__ void __launch_bounds__(256) gemm_plain_kernel(int M, int Nn, int K, const TA* __restrict__ A,
                                                         long long am, long long ak,
                                                         const TB* __restrict__ B, long long bk,
                                                         long long bn, float* __restrict__ C, long long cm,
                                                         long long cn, int accumulate) {
  __shared__ float sa[32][33], sb[32][33];
  const int m0 = blockIdx.x * 32, n0 = blockIdx.y * 32;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < K; k0 += 32) {
    for (int i = ty; i < 32; i += 8) {
      // the tile index with unit stride goes along the lanes
      const int ma = ak == 1 ? i : tx, ka = ak == 1 ? tx : i;
      const bool oka = m0 + ma < M && k0 + ka < K;
      sa[ka][ma] = oka ? to_f<TA>(A[(m0 + ma) * am + (k0 + ka) * ak]) : 0.f;
      const int kb = bn == 1 ? i : tx, nb = bn == 1 ? tx : i;
      const bool okb = k0 + kb < K && n0 + nb < Nn;
      sb[kb][nb] = okb ? to_f<TB>(B[(k0 + kb) * bk + (n0 + nb) * bn]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[u] = fmaf(sa[k][ty + 8 * u], sb[k][tx], acc[u]);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int m = m0 + ty + 8 * u, n = n0 + tx;
    if (m < M && n < Nn) {
      float* c = C + m * cm + n * cn;
      *c = accumulate ? *c + acc[u] : acc[u];
    }
  }
}

template <typename TG, typename TW>
cudaError_t run(int N, int V, int r, const TG* G, const TW* a, const TW* W2, int rv, float* ga, float* gW,
                int accumulate, cudaStream_t stream) {
  const long long wv = rv ? 1 : r, wj = rv ? V : 1;
  if (N > 0 && ga) {
    gemm_plain_kernel<TG, TW><<<dim3((N + 31) / 32, (r + 31) / 32), 256, 0, stream>>>(
        N, r, V, G, V, 1, W2, wv, wj, ga, r, 1, 0);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (gW)
    gemm_plain_kernel<TG, TW><<<dim3((V + 31) / 32, (r + 31) / 32), 256, 0, stream>>>(
        V, r, N, G, 1, V, a, r, 1, gW, wv, wj, accumulate);
  return cudaGetLastError();
}

}  // namespace

size_t bias_grad_workspace_bytes(int, int, int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_bias_grad(int N, int V, int r, int g_bf16, const void* G, int w_bf16, const void* a,
                             const void* W2, int w2_rv, float* grad_a, float* grad_W2, int accumulate,
                             void*, int, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (g_bf16 && w_bf16)
    return run(N, V, r, (const bf*)G, (const bf*)a, (const bf*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
  if (g_bf16)
    return run(N, V, r, (const bf*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
  if (w_bf16)
    return run(N, V, r, (const float*)G, (const bf*)a, (const bf*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
  return run(N, V, r, (const float*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
}

}  // namespace dspark
