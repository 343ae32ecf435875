// embedding.cu -- rows of a table for given tokens, scaled, and the table's gradient.
//
//   out[i] = scale W[t_i]  (zero for t_i = -1: padding);
//   grad_W[v] = scale sum_{i : t_i = v} grad[i], the sum in the order of i.
#include "common.cuh"
#include "kernels.h"

namespace dspark {
namespace {

constexpr int kEThr = 256;

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename TW, typename TO>
__global__ void __launch_bounds__(kEThr) embed_kernel(int V, int D, float scale, const TW* __restrict__ W,
                                                      const int32_t* __restrict__ tokens,
                                                      TO* __restrict__ out) {
  const long long i = blockIdx.x;
  const int t = tokens[i];
  for (int j = threadIdx.x; j < D; j += kEThr) {
    float x = 0.f;
    if (t < -1 || t >= V)
      x = NAN;
    else if (t >= 0)
      x = scale * to_f<TW>(W[(long long)t * D + j]);
    put(out + i * D + j, x);
  }
}

// One block per table row: it looks through all tokens for its own.
template <typename TG, typename TO>
__global__ void __launch_bounds__(kEThr) embed_grad_kernel(int N, int D, float scale,
                                                           const TG* __restrict__ grad,
                                                           const int32_t* __restrict__ tokens,
                                                           TO* __restrict__ gW, int accumulate) {
  const int v = blockIdx.x;
  for (int j0 = 0; j0 < D; j0 += kEThr) {
    const int j = j0 + (int)threadIdx.x;
    float s = 0.f;
    bool any = false;
    for (int i = 0; i < N; ++i)
      if (tokens[i] == v) {
        any = true;
        if (j < D) s += to_f<TG>(grad[(long long)i * D + j]);
      }
    if (j < D && (any || !accumulate)) {
      TO* o = gW + (long long)v * D + j;
      put(o, accumulate ? to_f<TO>(*o) + scale * s : scale * s);
    }
  }
}

__global__ void embed_check_kernel(int N, int V, const int32_t* __restrict__ tokens, unsigned* status) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < N && (tokens[i] < -1 || tokens[i] >= V)) atomicMax(status, kErrInvalid);
}

}  // namespace

cudaError_t launch_embedding(int N, int V, int D, float scale, int w_bf16, const void* W,
                             const int32_t* tokens, int o_bf16, void* out, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (w_bf16 && o_bf16)
    embed_kernel<bf, bf><<<N, kEThr, 0, stream>>>(V, D, scale, (const bf*)W, tokens, (bf*)out);
  else if (w_bf16)
    embed_kernel<bf, float><<<N, kEThr, 0, stream>>>(V, D, scale, (const bf*)W, tokens, (float*)out);
  else if (o_bf16)
    embed_kernel<float, bf><<<N, kEThr, 0, stream>>>(V, D, scale, (const float*)W, tokens, (bf*)out);
  else
    embed_kernel<float, float><<<N, kEThr, 0, stream>>>(V, D, scale, (const float*)W, tokens, (float*)out);
  return cudaGetLastError();
}

size_t embedding_grad_workspace_bytes(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_embedding_grad(int N, int V, int D, float scale, int g_bf16, const void* grad,
                                  const int32_t* tokens, int o_bf16, void* gW, int accumulate,
                                  void* workspace, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (N > 0) {
    embed_check_kernel<<<(N + 255) / 256, 256, 0, stream>>>(N, V, tokens, &((WsHeader*)workspace)->status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (g_bf16 && o_bf16)
    embed_grad_kernel<bf, bf><<<V, kEThr, 0, stream>>>(N, D, scale, (const bf*)grad, tokens, (bf*)gW, accumulate);
  else if (g_bf16)
    embed_grad_kernel<bf, float><<<V, kEThr, 0, stream>>>(N, D, scale, (const bf*)grad, tokens, (float*)gW, accumulate);
  else if (o_bf16)
    embed_grad_kernel<float, bf><<<V, kEThr, 0, stream>>>(N, D, scale, (const float*)grad, tokens, (bf*)gW, accumulate);
  else
    embed_grad_kernel<float, float><<<V, kEThr, 0, stream>>>(N, D, scale, (const float*)grad, tokens, (float*)gW, accumulate);
  return cudaGetLastError();
}

}  // namespace dspark
