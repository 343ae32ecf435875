// logprobs.cu -- log probabilities of given tokens, with entropy, rank and top alternatives, and
// the gradient of the first two.
//
// For a row z of V logits, a token x and a temperature T, with m = max_v z_v, d_v = (z_v - m) / T
// and S = sum_v exp d_v:
//   norm = (m, ln S);  ln p_v = d_v - ln S;  logp = ln p_x;
//   H = -sum_v p_v ln p_v = ln S - (1 / S) sum_v d_v exp d_v;   rank = 1 + #{v : z_v > z_x};
//   the K alternatives are the K largest z_v above -inf, the lower index first among equal ones.
//   dL/dz_v = (1 / T) (g ([v == x] - p_v) - h p_v (ln p_v + H)) for g = dL/dlogp, h = dL/dH.
// The maximum is subtracted before the scale is applied: a row whose entries are all the type's
// lowest number is a uniform row, not an overflow.
#include "common.cuh"
#include "kernels.h"

namespace dspark {
namespace {

constexpr int kPThr = 256;

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kPThr / 32; ++w) v = fmaxf(v, red[w]);
  return v;
}
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kPThr / 32; ++w) v += red[w];
  return v;
}

// One block per row: a pass for the maximum, one for the sums, one per alternative.
template <typename T>
__global__ void __launch_bounds__(kPThr) logprob_kernel(
    int V, float invT, const T* __restrict__ logits, long long ld, const int32_t* __restrict__ tokens,
    int top, float* __restrict__ logp, float2* __restrict__ norm, float* __restrict__ entropy,
    int32_t* __restrict__ rank, int32_t* __restrict__ top_ids, float* __restrict__ top_logp,
    unsigned* status) {
  __shared__ float red[kPThr / 32];
  __shared__ double dred[kPThr / 32];
  __shared__ unsigned long long kred[kPThr / 32];
  const long long row = blockIdx.x;
  const T* z = logits + row * ld;
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += kPThr) m = fmaxf(m, to_f<T>(z[v]));
  m = block_max(m, red);
  const int x = tokens ? tokens[row] : -1;
  const bool bad = x < -1 || x >= V;
  const float zx = x >= 0 && !bad ? to_f<T>(z[x]) : 0.f;
  double s = 0.0, t = 0.0, c = 0.0;
  for (int v = threadIdx.x; v < V; v += kPThr) {
    const float f = to_f<T>(z[v]);
    const float d = f == -INFINITY ? -INFINITY : (f - m) * invT, e = expf(d);
    s += e;
    t += e == 0.f ? 0.0 : (double)e * d;
    c += f > zx ? 1.0 : 0.0;
  }
  s = block_sum(s, dred);
  t = block_sum(t, dred);
  c = block_sum(c, dred);
  const bool none = s == 0.0;  // every entry -inf
  const float ls = none ? 0.f : (float)log(s);
  if (threadIdx.x == 0) {
    if (norm) norm[row] = make_float2(m, ls);
    if (entropy) entropy[row] = none ? 0.f : (float)(log(s) - t / s);
    float lp = x < 0 ? 0.f : zx == -INFINITY ? -INFINITY : (zx - m) * invT - ls;
    if (bad) {
      lp = NAN;
      atomicMax(status, kErrInvalid);
    }
    if (isnan(s)) lp = x == -1 ? 0.f : NAN;
    if (logp) logp[row] = lp;
    if (rank) rank[row] = bad ? -1 : x < 0 ? 0 : (int)c + 1;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < top; ++k) {
    unsigned long long best = 0ull;
    for (int v = threadIdx.x; v < V; v += kPThr) {
      const float f = to_f<T>(z[v]) + 0.f;
      const unsigned long long key = f > -INFINITY ? make_key(f, (uint32_t)v) : 0ull;
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long q = __shfl_xor_sync(0xffffffffu, best, o);
      best = q > best ? q : best;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) kred[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kPThr / 32; ++w) best = kred[w] > best ? kred[w] : best;
    if (threadIdx.x == 0) {
      top_ids[row * top + k] = best ? (int32_t)key_token(best) : -1;
      top_logp[row * top + k] = best ? (key_score(best) - m) * invT - ls : -INFINITY;
    }
    last = best ? best : 1ull;
  }
}

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T>
__global__ void __launch_bounds__(kPThr) logprob_grad_kernel(
    int V, float invT, const T* __restrict__ logits, long long ld, const int32_t* __restrict__ tokens,
    const float2* __restrict__ norm, const float* __restrict__ entropy, const float* __restrict__ gl,
    const float* __restrict__ gh, T* grad, long long gld) {
  const long long row = blockIdx.y;
  const int x = tokens ? tokens[row] : -1;
  const float2 n = norm[row];
  const float g = gl && x >= 0 ? gl[row] : 0.f;
  const float h = gh ? gh[row] : 0.f, H = gh ? entropy[row] : 0.f;
  const bool bad = x < -1 || x >= V;
  const int v = blockIdx.x * kPThr + (int)threadIdx.x;
  if (v >= V) return;
  const float f = to_f<T>(logits[row * ld + v]);
  const float lp = f == -INFINITY ? -INFINITY : (f - n.x) * invT - n.y;
  const float p = expf(lp);
  float d = -p * (g + (p == 0.f ? 0.f : h * (lp + H)));
  if (v == x) d += g;
  grad[row * gld + v] = from_f<T>(bad ? NAN : d * invT);
}

}  // namespace

size_t logprobs_workspace_bytes(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_logprobs(int N, int V, float T, int bf16, const void* logits, long long ld,
                            const int32_t* tokens, int top, float* logp, float* norm, float* entropy,
                            int32_t* rank, int32_t* top_ids, float* top_logp, void* workspace,
                            cudaStream_t stream) {
  if (bf16)
    logprob_kernel<__nv_bfloat16><<<N, kPThr, 0, stream>>>(
        V, 1.f / T, (const __nv_bfloat16*)logits, ld, tokens, top, logp, (float2*)norm, entropy, rank,
        top_ids, top_logp, &((WsHeader*)workspace)->status);
  else
    logprob_kernel<float><<<N, kPThr, 0, stream>>>(V, 1.f / T, (const float*)logits, ld, tokens, top, logp,
                                                   (float2*)norm, entropy, rank, top_ids, top_logp,
                                                   &((WsHeader*)workspace)->status);
  return cudaGetLastError();
}

cudaError_t launch_logprobs_grad(int N, int V, float T, int bf16, const void* logits, long long ld,
                                 const int32_t* tokens, const float* norm, const float* entropy,
                                 const float* gl, const float* gh, void* grad, long long gld,
                                 cudaStream_t stream) {
  for (int r0 = 0; r0 < N; r0 += 65535) {
    const int n = N - r0 < 65535 ? N - r0 : 65535;
    const dim3 grid((V + kPThr - 1) / kPThr, n);
    const int32_t* tk = tokens ? tokens + r0 : nullptr;
    const float2* nm = (const float2*)norm + r0;
    const float *en = entropy ? entropy + r0 : nullptr, *a = gl ? gl + r0 : nullptr, *b = gh ? gh + r0 : nullptr;
    if (bf16)
      logprob_grad_kernel<__nv_bfloat16><<<grid, kPThr, 0, stream>>>(
          V, 1.f / T, (const __nv_bfloat16*)logits + r0 * ld, ld, tk, nm, en, a, b,
          (__nv_bfloat16*)grad + r0 * gld, gld);
    else
      logprob_grad_kernel<float><<<grid, kPThr, 0, stream>>>(V, 1.f / T, (const float*)logits + r0 * ld, ld,
                                                             tk, nm, en, a, b, (float*)grad + r0 * gld, gld);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dspark
