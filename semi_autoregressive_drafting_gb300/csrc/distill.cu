// distill.cu -- the loss of rows of logits against a teacher's K largest log probabilities, and its gradient.
//
// A row has K + 1 outcomes: the teacher's tokens S = {id_j}, and the rest.  q_j = exp(logq_j), q_r = 1 - sum q_j;
// p = softmax(z / T), p_r = sum of p outside S.  With (a, b) the weights of the two parts and w the row's:
//   KL = sum_j q_j (ln q_j - ln p_j),  L1 = sum_j |p_j - q_j|  (over the rest too, or over S alone),
//   loss = w (a KL + b L1);
//   t_j = -a q_j + b p_j sign(p_j - q_j)  (p times the loss's derivative by p),  M = sum_j t_j,
//   dL/dz_v = (w / T) (t_j - p_j M) for v = id_j, else (w / T) P_v (t_r - p_r M), P_v = p_v / p_r.
// The rest has a maximum and a sum of its own, P_v = exp((z_v - m_r) / T - ln S_r): no difference of two sums
// near one is formed, and a rest that is far below the row's maximum keeps its digits.
//
// Forward: a warp takes a 4 KB segment of a row, puts -inf in place of the row's own tokens, and leaves the
// segment's maximum and sum; a second launch, one block per row, joins them, fetches the K logits and forms
// the outcomes in 64 bits (K + 1 exponentials and logarithms a row).  The gradient is a third pass.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

namespace dspark {
namespace {

constexpr int kThr = 256;
constexpr int kWarps = kThr / 32;
constexpr int kMaxK = 128;
constexpr int kIdLane = kMaxK / 32;   // a row's tokens per lane
constexpr int kSegment = 8;           // 16-byte loads per lane of a segment (4 KB)
constexpr float kL2e = 1.4426950408889634f;

// What a row's gradient needs beside the logits.
struct RowCoef {
  float nm, ls, c;  // P_v = exp((z_v + nm) / T - ls), dL/dz_v = c P_v
  float pad;
};

struct DsArgs {
  int V, K, nchunk, rest;
  float T, a_kl, a_l1;
  long long ld, gld;
  const int32_t* ids;
  const float* logq;
  const float* weight;
  float *loss, *parts, *norm;
  const float* norm_in;
  WsHeader* hdr;
  float2* part;    // [N][nchunk][kWarps] the segments' (maximum, sum) outside S
  RowCoef* coef;   // [N]
  float* at;       // [N][K] gradient at the row's tokens
};

// The row's tokens, four per lane (-1: none).
__device__ __forceinline__ void load_ids(int (&id)[kIdLane], const int32_t* ids, int K) {
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    const int j = i * 32 + (int)(threadIdx.x & 31);
    id[i] = j < K ? __ldg(ids + j) : -1;
  }
}

template <typename T>
__device__ __forceinline__ void put(uint4& q, int e, uint32_t fill) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      w[i] = e == i ? fill : w[i];
    } else {
      w[i] = e == 2 * i ? (w[i] & 0xFFFF0000u) | (fill & 0xFFFFu) : w[i];
      w[i] = e == 2 * i + 1 ? (w[i] & 0xFFFFu) | (fill & 0xFFFF0000u) : w[i];
    }
  }
  q = make_uint4(w[0], w[1], w[2], w[3]);
}

// One warp's segment: its maximum and sum of 2^((z - m) log2(e) / T) outside S.
template <typename T>
__global__ void __launch_bounds__(kThr) distill_part_kernel(const T* __restrict__ logits, const DsArgs a) {
  constexpr int E = Lg<T>::E;
  const long long row = blockIdx.x / (unsigned)a.nchunk;
  const int ch = (int)(blockIdx.x % (unsigned)a.nchunk), lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  if (a.weight && a.weight[row] == 0.f) return;
  const T* z = logits + row * a.ld;
  const int head = row_head(z);
  const int g0 = (ch * kWarps + warp) * (32 * kSegment);   // the segment's first group
  const int first = g0 * E - head, last = first + 32 * kSegment * E;
  if (first >= a.V) return;
  uint4 q[kSegment];
#pragma unroll
  for (int u = 0; u < kSegment; ++u) q[u] = load16<T>(z, (g0 + u * 32 + lane) * E - head, a.V);
  int id[kIdLane];
  load_ids(id, a.ids + row * a.K, a.K);
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    uint32_t here = __ballot_sync(0xffffffffu, id[i] >= 0 && id[i] >= first && id[i] < last);
    while (here) {
      const int src = __ffs(here) - 1;
      here &= here - 1;
      const int at = __shfl_sync(0xffffffffu, id[i], src) - first;
      const int g = at / E, e = at % E;
      if ((g & 31) == lane) {
#pragma unroll
        for (int u = 0; u < kSegment; ++u)
          if (u == g >> 5) put<T>(q[u], e, Lg<T>::kFill);
      }
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kSegment; ++u) m = Lg<T>::max16(m, q[u]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float s2 = kL2e / a.T, nm = m == -INFINITY ? 0.f : -m;
  float S = 0.f;
#pragma unroll
  for (int u = 0; u < kSegment; ++u) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 f = un2(Lg<T>::pair(q[u], e));
      S += ex2p((f.x + nm) * s2) + ex2p((f.y + nm) * s2);
    }
  }
  S = warp_sum(S);
  if (lane == 0) a.part[(row * a.nchunk + ch) * kWarps + warp] = make_float2(m, S);
}

// Sum over the block's 128 threads in a fixed order; every thread has it.
__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  return (sm[0] + sm[1]) + (sm[2] + sm[3]);
}

// One block per row joins the segments (FWD) or takes the normalisers of an earlier call, forms the
// outcomes, and leaves the loss and what the gradient needs.
template <typename T, bool FWD>
__global__ void __launch_bounds__(kMaxK) distill_rows_kernel(const T* __restrict__ logits, const DsArgs a) {
  __shared__ double s_sum[4];
  __shared__ float s_m[4];
  __shared__ int s_id[kMaxK];
  const long long row = blockIdx.x;
  const int tid = (int)threadIdx.x;
  const float w = a.weight ? a.weight[row] : 1.f;
  if (w == 0.f) {  // a padding row: not read
    if (tid == 0) {
      if (a.loss) a.loss[row] = 0.f;
      if (a.parts) ((float2*)a.parts)[row] = make_float2(0.f, 0.f);
      if (a.norm) ((float4*)a.norm)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.coef) a.coef[row] = RowCoef{0.f, 0.f, 0.f, 0.f};
    }
    if (a.at && tid < a.K) a.at[row * a.K + tid] = 0.f;
    return;
  }
  const T* z = logits + row * a.ld;
  const int id = tid < a.K ? a.ids[row * a.K + tid] : -1;
  const float lq = id >= 0 && id < a.V ? a.logq[row * a.K + tid] : -INFINITY;
  const float zj = id >= 0 && id < a.V ? to_f<T>(z[id]) : -INFINITY;
  s_id[tid] = id;
  __syncthreads();
  bool bad = id < -1 || id >= a.V;
  if (id >= 0)
    for (int j = 0; j < tid; ++j) bad |= s_id[j] == id;
  bad = __syncthreads_or(bad);

  const double invT = 1.0 / (double)a.T;
  float mr, mall;
  double lsr, ls;   // ln of the sums relative to mr, mall
  double dj;        // (z_j - mall) / T
  bool none;        // the row is -inf everywhere
  if (FWD) {
    pdl_wait();
    // the rest: the segments' maximum, then their sums relative to it
    const int head = row_head(z), nseg = (a.V + head + 32 * kSegment * Lg<T>::E - 1) / (32 * kSegment * Lg<T>::E);
    const float2* part = a.part + row * a.nchunk * kWarps;
    float m = -INFINITY;
    for (int i = tid; i < nseg; i += kMaxK) m = fmaxf(m, __ldcg(&part[i].x));
    float mz = zj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
    }
    __shared__ float s_z[4];
    if ((tid & 31) == 0) {
      s_m[tid >> 5] = m;
      s_z[tid >> 5] = mz;
    }
    __syncthreads();
    mr = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    mall = fmaxf(mr, fmaxf(fmaxf(s_z[0], s_z[1]), fmaxf(s_z[2], s_z[3])));
    const float s2 = kL2e / a.T;
    double S = 0.0;
    for (int i = tid; i < nseg; i += kMaxK) {
      const float2 p = __ldcg(part + i);
      // (an empty segment is left out; NaN stays)
      if (p.x != -INFINITY || isnan(p.y)) S += (double)p.y * (double)ex2p((p.x - mr) * s2);
    }
    S = block_sum(S, s_sum);
    none = mall == -INFINITY;
    lsr = mr == -INFINITY && !isnan(S) ? 0.0 : log(S);
    dj = id >= 0 && zj != -INFINITY ? ((double)zj - (double)mall) * invT : -INFINITY;
    const double e = id >= 0 && zj != -INFINITY ? exp(dj) : 0.0;
    const double Sr = mr == -INFINITY && !isnan(S) ? 0.0 : S * exp(((double)mr - (double)mall) * invT);
    const double all = Sr + block_sum(e, s_sum);
    ls = none && !isnan(all) ? 0.0 : log(all);
  } else {
    const float4 n = ((const float4*)a.norm_in)[row];
    mall = n.x;
    ls = n.y;
    mr = n.z;
    lsr = n.w;
    none = mall == -INFINITY;
    dj = id >= 0 && zj != -INFINITY ? ((double)zj - (double)mall) * invT : -INFINITY;
  }
  // the outcomes; thread j holds the j-th, all hold the rest
  const double lp = dj - ls, p = exp(lp);
  const double lpr = mr == -INFINITY ? -INFINITY : ((double)mr - (double)mall) * invT + lsr - ls, pr = exp(lpr);
  const double q = id >= 0 ? exp((double)lq) : 0.0;
  const double Q = block_sum(q, s_sum);
  const double qr = Q < 1.0 ? 1.0 - Q : Q >= 1.0 ? 0.0 : Q;   // (NaN stays)
  const double sgn = p > q ? 1.0 : p < q ? -1.0 : p - q, sgnr = pr > qr ? 1.0 : pr < qr ? -1.0 : pr - qr;
  const double a_kl = a.a_kl, a_l1 = a.a_l1;
  const double t = id >= 0 ? -a_kl * q + a_l1 * (p * sgn) : 0.0;
  const double tr = a.rest ? -a_kl * qr + a_l1 * (pr * sgnr) : 0.0;
  const double M = block_sum(t, s_sum) + tr;
  if (FWD && (a.loss || a.parts)) {
    double kl = id >= 0 && q != 0.0 ? q * ((double)lq - lp) : 0.0, l1 = id >= 0 ? fabs(p - q) : 0.0;
    kl = block_sum(kl, s_sum);
    l1 = block_sum(l1, s_sum);
    if (a.rest) {
      if (qr != 0.0) kl += qr * (log(qr) - lpr);
      l1 += fabs(pr - qr);
    }
    if (tid == 0) {
      const double k = a_kl != 0.0 ? a_kl * kl : 0.0, l = a_l1 != 0.0 ? a_l1 * l1 : 0.0;
      // NaN anywhere in the row is in its sum, and so in lp_r or ls
      if (a.loss) a.loss[row] = bad || isnan(ls) ? NAN : (float)((double)w * (k + l));
      if (a.parts) ((float2*)a.parts)[row] = bad || isnan(ls) ? make_float2(NAN, NAN) : make_float2((float)kl, (float)l1);
    }
  }
  const bool nan = bad || isnan(ls) || isnan(lsr);
  const double scale = (double)w * invT;
  if (a.at && tid < a.K) a.at[row * a.K + tid] = nan ? NAN : (float)(scale * (t - (id >= 0 ? p * M : 0.0)));
  if (tid == 0) {
    if (FWD && a.norm)
      ((float4*)a.norm)[row] = bad ? make_float4(NAN, NAN, NAN, NAN) : make_float4(mall, (float)ls, mr, (float)lsr);
    if (a.coef) {
      const double c = mr == -INFINITY ? 0.0 : scale * (tr - pr * M);
      a.coef[row] = RowCoef{mr == -INFINITY ? 0.f : -mr, (float)lsr, nan ? NAN : (float)c, 0.f};
    }
    if (bad && a.hdr) atomicMax(&a.hdr->status, kErrInvalid);
  }
}

constexpr int kGPer = 4;  // 16-byte groups per thread

// dL/dz = c P_v outside S, `at` at the row's tokens.
template <typename T>
__global__ void __launch_bounds__(kThr) distill_grad_kernel(const T* logits, T* grad, const DsArgs a) {
  constexpr int E = Lg<T>::E;
  const long long row = blockIdx.x / (unsigned)a.nchunk;
  const int ch = (int)(blockIdx.x % (unsigned)a.nchunk), lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const T* z = logits + row * a.ld;
  T* o = grad + row * a.gld;
  const int head = row_head(z);
  const int g0 = (ch * kWarps + warp) * (32 * kGPer);
  const int first = g0 * E - head, last = first + 32 * kGPer * E;
  uint4 q[kGPer];
#pragma unroll
  for (int u = 0; u < kGPer; ++u) {
    const int v0 = (g0 + u * 32 + lane) * E - head;
    q[u] = v0 >= 0 && v0 + E <= a.V ? __ldcs((const uint4*)(z + v0)) : load16<T>(z, v0, a.V);
  }
  int id[kIdLane];
  load_ids(id, a.ids + row * a.K, a.K);
  pdl_wait();
  const float4 cf = __ldcg((const float4*)(a.coef + row));
  const float invT = 1.f / a.T, nm = cf.x, ls = cf.y, c = cf.z;
  const bool same = row_head((const T*)o) == head;
#pragma unroll
  for (int u = 0; u < kGPer; ++u) {
    const int v0 = (g0 + u * 32 + lane) * E - head;
    if (v0 >= a.V) break;
    float f[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 zz = un2(Lg<T>::pair(q[u], e));
      f[2 * e] = c == 0.f ? 0.f : c * ex2p(fmaf(zz.x + nm, invT, -ls) * kL2e);
      f[2 * e + 1] = c == 0.f ? 0.f : c * ex2p(fmaf(zz.y + nm, invT, -ls) * kL2e);
    }
    if (same && v0 >= 0 && v0 + E <= a.V) {
      __stcs((uint4*)(o + v0), pack16<T>(f));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v0 + e >= 0 && v0 + e < a.V) o[v0 + e] = from_f<T>(f[e]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kIdLane; ++i)
    if (id[i] >= first && id[i] < last && id[i] >= 0 && id[i] < a.V)
      o[id[i]] = from_f<T>(__ldcg(a.at + row * a.K + i * 32 + lane));
}

constexpr size_t al(size_t x) { return (x + 255) / 256 * 256; }

// chunks of a row of kWarps segments of `per` 16-byte groups per lane; a group more when rows may start off a
// 16-byte boundary
int chunks(int V, int E, int per, bool aligned_rows) {
  const int groups = (V + (aligned_rows ? 0 : E - 1) + E - 1) / E;
  return (groups + kThr * per - 1) / (kThr * per);
}
size_t part_bytes(int N, int V) { return al((size_t)N * chunks(V, 4, kSegment, false) * kWarps * sizeof(float2)); }

struct Ws {
  WsHeader* hdr;
  RowCoef* coef;
  float* at;
  float2* part;
};
Ws layout(void* workspace, int N, int V, int K) {
  uint8_t* w = (uint8_t*)workspace;
  Ws s;
  s.hdr = (WsHeader*)w;
  w += sizeof(WsHeader);
  s.coef = (RowCoef*)w;
  w += al((size_t)N * sizeof(RowCoef));
  s.at = (float*)w;
  w += al((size_t)N * K * sizeof(float));
  s.part = (float2*)w;
  return s;
}

template <typename T>
cudaError_t forward(int N, const T* logits, DsArgs a, bool al_rows, cudaStream_t stream) {
  a.nchunk = chunks(a.V, Lg<T>::E, kSegment, al_rows);
  distill_part_kernel<T><<<(unsigned)N * (unsigned)a.nchunk, kThr, 0, stream>>>(logits, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(distill_rows_kernel<T, true>, (unsigned)N, kMaxK, 0, stream, logits, a);
}

template <typename T>
cudaError_t gradient(int N, const T* logits, T* grad, DsArgs a, bool al_rows, cudaStream_t stream) {
  a.nchunk = chunks(a.V, Lg<T>::E, kGPer, al_rows);
  return launch_pdl(distill_grad_kernel<T>, (unsigned)N * (unsigned)a.nchunk, kThr, 0, stream, logits, grad, a);
}

template <typename T>
cudaError_t run(int N, const T* logits, T* grad, const DsArgs& a, cudaStream_t stream) {
  const bool al_rows = ((uintptr_t)logits % 16) == 0 && (a.ld * (long long)sizeof(T)) % 16 == 0;
  cudaError_t e;
  if (a.norm_in) {
    distill_rows_kernel<T, false><<<(unsigned)N, kMaxK, 0, stream>>>(logits, a);
    e = cudaGetLastError();
  } else {
    e = forward(N, logits, a, al_rows, stream);
  }
  if (e != cudaSuccess || !grad) return e;
  return gradient(N, logits, grad, a, al_rows, stream);
}

}  // namespace

size_t distill_workspace_bytes(int N, int V, int K) {
  return sizeof(WsHeader) + al((size_t)N * sizeof(RowCoef)) + al((size_t)N * K * sizeof(float)) + part_bytes(N, V);
}

cudaError_t launch_distill(int N, int V, float T, int bf16, const void* logits, long long ld, int K,
                           const int32_t* ids, const float* logq, const float* weight, float a_kl, float a_l1,
                           int rest, const float* norm_in, float* loss, float* parts, float* norm, void* grad,
                           long long gld, void* workspace, cudaStream_t stream) {
  const Ws s = layout(workspace, N, V, K);
  DsArgs a;
  a.V = V;
  a.K = K;
  a.nchunk = 0;
  a.rest = rest;
  a.T = T;
  a.a_kl = a_kl;
  a.a_l1 = a_l1;
  a.ld = ld;
  a.gld = gld;
  a.ids = ids;
  a.logq = logq;
  a.weight = weight;
  a.loss = loss;
  a.parts = parts;
  a.norm = norm;
  a.norm_in = norm_in;
  a.hdr = s.hdr;
  a.part = s.part;
  a.coef = grad ? s.coef : nullptr;
  a.at = grad ? s.at : nullptr;
  using H = __nv_bfloat16;
  return bf16 ? run<H>(N, (const H*)logits, (H*)grad, a, stream) : run<float>(N, (const float*)logits, (float*)grad, a, stream);
}

}  // namespace dspark
