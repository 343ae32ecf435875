// bias_grad.cu -- the gradients of the low-rank bias product B_k = a W2 (Eq 5; Eq 6 with
// a = tanh(o)), "DSpark -- paper verification", section 1.
//
// For gradients G [N][V] of the logits, conditioning rows a [N][r] and W2 as [V][r] or [r][V]:
//   grad_a[n][j] = sum_v G[n][v] W2[v][j],   grad_W2[v][j] = sum_n G[n][v] a[n][j].
//
// bf16 weights: two tensor-core products (tcgen05, kind::f16, fp32 accumulation in TMEM), each with
// G as the M-side operand in tiles of up to 256 x 64, so that the 256-column operand that passes by
// (W2 or a) is read once per 256 rows of M:
//   grad_W2: M = 256 vocabulary entries (G as it lies is M-major), K = N; one tile per work item;
//   grad_a:  M = 256 rows, K = a share of the vocabulary (G as it lies is K-major); the shares'
//            fp32 results are added in order by a second launch.
// A block per SM walks over its work items: a TMA thread, one thread that issues the MMAs, four
// warps that read the accumulators out of TMEM.  An fp32 G enters as two bf16 parts, G = hi + lo with
// hi = bf16(G), lo = bf16(G - hi) (16 significant bits or more, an error of at most 2^-18 |G|,
// below that of an fp32 sum of these lengths); eight warps split it on its way from global to
// shared memory.  The same warps bring a G whose rows TMA cannot address.
// fp32 weights (small heads): CUDA-core tiles.
#include <cuda.h>

#include "draft.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ fp32 weights: CUDA cores
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
cudaError_t plain(int N, int V, int r, const TG* G, const TW* a, const TW* W2, int rv, float* ga, float* gW,
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

// ------------------------------------------------------------------ bf16 weights: tensor cores
constexpr int kBox = 64 * 128;        // bytes of one shared-memory box: 64 rows of 64 bf16
constexpr int kTileA = 2 * kBox;      // 128 (M) x 64 (K) of G
constexpr int kBytesB = 4 * kBox;     // 64 (K) x 256 of W2 or a
constexpr int kBN = 256;              // columns per work item
constexpr int kMaxItems = 2;          // work items per SM at most when the vocabulary is shared out

struct BgArgs {
  int N, V, r;
  int items, nrb;       // work items; blocks of 256 columns of r
  int nmb;              // grad_a: blocks of 256 rows
  int per_split;        // grad_a: K stages per share of the vocabulary
  int nstage_k;         // K stages in all
  int b_kmajor;         // grad_a: W2 is [r][V]
  int out_rv;           // grad_W2 is [r][V]
  int accumulate;
  float* out;           // grad_W2, or grad_a's shares [split][N][r]
  const void* G;
  unsigned* status;
};

// A bounded wait of one thread that also ends when another role of the block gave up.
// (limit: for the accumulators, whose K stages all come first)
__device__ __forceinline__ bool wait_or(uint64_t* bar, uint32_t parity, volatile int* stop,
                                        unsigned long long limit = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) {
    if (*stop) return false;
    if (globaltimer() - t0 > limit) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// One work item: M tiles of 128 (1 or 2), their first row, the first and last K stage, the first column.
struct Item {
  int m0, tiles, k0, k1, c0, cols, split;
};
template <bool WANT_A>
__device__ __forceinline__ Item item_of(const BgArgs& a, int i) {
  Item t;
  const int rb = i % a.nrb;
  i /= a.nrb;
  t.c0 = rb * kBN;
  t.cols = min(kBN, a.r - t.c0);
  if (WANT_A) {
    t.m0 = (i % a.nmb) * 256;
    t.split = i / a.nmb;
    t.k0 = t.split * a.per_split;
    t.k1 = min(a.nstage_k, t.k0 + a.per_split);
    t.tiles = a.N - t.m0 > 128 ? 2 : 1;
  } else {
    t.m0 = i * 256;
    t.split = 0;
    t.k0 = 0;
    t.k1 = a.nstage_k;
    t.tiles = a.V - t.m0 > 128 ? 2 : 1;
  }
  return t;
}

// Four consecutive elements of a row of G, zero from `n` on.
template <typename TG, bool VEC>
__device__ __forceinline__ float4 load_quad(const TG* p, int n) {
  if (n <= 0) return make_float4(0.f, 0.f, 0.f, 0.f);
  if (VEC) return __ldcg((const float4*)p);  // (fp32 only; V is a multiple of 4)
  return make_float4(to_f<TG>(p[0]), n > 1 ? to_f<TG>(p[1]) : 0.f, n > 2 ? to_f<TG>(p[2]) : 0.f,
                     n > 3 ? to_f<TG>(p[3]) : 0.f);
}
__device__ __forceinline__ uint2 pack_hi(const float4& f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
  uint2 w;
  memcpy(&w.x, &a, 4);
  memcpy(&w.y, &b, 4);
  return w;
}
__device__ __forceinline__ uint2 pack_lo(const float4& f, const uint2& hi) {
  return pack_hi(make_float4(f.x - __uint_as_float(hi.x << 16), f.y - __uint_as_float(hi.x & 0xFFFF0000u),
                             f.z - __uint_as_float(hi.y << 16), f.w - __uint_as_float(hi.y & 0xFFFF0000u)));
}

// MODE 0: bf16 G by TMA.  1: fp32 G by 16-byte loads, two parts.  2: fp32 G element by element.
// 3: bf16 G element by element (one part).
template <int MODE>
struct Src {
  static constexpr bool kTma = MODE == 0, kVec = MODE == 1;
  static constexpr int kParts = MODE == 1 || MODE == 2 ? 2 : 1;
  static constexpr int kStages = kParts == 2 ? 2 : 3;
  static constexpr int kStage = kParts * 2 * kTileA + kBytesB;
  static constexpr int kThreads = kTma ? 256 : 512;
  using T = typename std::conditional<MODE == 3, bf16, float>::type;
};

template <bool WANT_A, int MODE>
__global__ void __launch_bounds__(Src<MODE>::kThreads, 1)
    bias_grad_kernel(const BgArgs a, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmB) {
  using S = Src<MODE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(smem + S::kStages * S::kStage);
  uint64_t* empty = full + S::kStages;
  uint64_t* done = empty + S::kStages;
  uint64_t* tfree = done + 1;
  uint32_t* tbase = (uint32_t*)(tfree + 1);
  volatile int* stop = (volatile int*)(tbase + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kOffB = S::kParts * 2 * kTileA;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1 + (S::kTma ? 0 : 8));
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    mbar_init(tfree, 4);
    *stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tbase, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tbase;

  if (warp == 0) {
    if (lane == 0) {  // ---- TMA
      const uint64_t once = policy_evict_first(), keep = policy_evict_last();
      int g = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
        const Item t = item_of<WANT_A>(a, i);
        const int nb = (t.cols + 63) / 64;
        const uint32_t bytes = (uint32_t)(nb * kBox + (S::kTma ? t.tiles * kTileA : 0));
        for (int s = t.k0; s < t.k1; ++s, ++g) {
          const int slot = g % S::kStages;
          if (g >= S::kStages && !wait_or(&empty[slot], (uint32_t)((g / S::kStages - 1) & 1), stop)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + slot * S::kStage;
          mbar_expect_tx(&full[slot], bytes);
          if (S::kTma) {
            for (int b = 0; b < 2 * t.tiles; ++b)
              if (WANT_A)
                tc::tma_load_2d(st + b * kBox, &tmG, s * 64, t.m0 + 64 * b, &full[slot], once);
              else
                tc::tma_load_2d(st + b * kBox, &tmG, t.m0 + 64 * b, s * 64, &full[slot], once);
          }
          for (int b = 0; b < nb; ++b)
            if (WANT_A && a.b_kmajor)
              tc::tma_load_2d(st + kOffB + b * kBox, &tmB, s * 64, t.c0 + 64 * b, &full[slot], keep);
            else
              tc::tma_load_2d(st + kOffB + b * kBox, &tmB, t.c0 + 64 * b, s * 64, &full[slot], keep);
        }
      }
      if (!ok) atomicMax(a.status, kErrTimeout);
      // every copy lands before the block ends (the phase of each slot's last use)
      for (int j = max(0, g - S::kStages); j < g; ++j) mbar_wait(&full[j % S::kStages], (uint32_t)((j / S::kStages) & 1));
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ---- MMA
      int g = 0, n = 0;
      bool ok = true;
      for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x, ++n) {
        const Item t = item_of<WANT_A>(a, i);
        const uint32_t idesc = tc::idesc_bf16_f32(128, (t.cols + 15) / 16 * 16) |
                               (WANT_A ? 0u : tc::kIdescAMajorMN) |
                               (WANT_A && a.b_kmajor ? 0u : tc::kIdescBMajorMN);
        if (n > 0 && !wait_or(tfree, (uint32_t)((n - 1) & 1), stop)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        for (int s = t.k0; s < t.k1; ++s, ++g) {
          const int slot = g % S::kStages;
          if (!wait_or(&full[slot], (uint32_t)((g / S::kStages) & 1), stop)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t sa = smem_u32(smem + slot * S::kStage), sb = sa + kOffB;
          // K-major: 16 elements of K are 32 bytes along the rows; M- or N-major: 16 rows of 128 bytes
          const uint64_t bd = WANT_A && a.b_kmajor ? tc::sdesc_sw128(sb) : tc::sdesc_sw128_mn(sb, kBox);
          const uint64_t bstep = WANT_A && a.b_kmajor ? 2 : 128;
          for (int m = 0; m < t.tiles; ++m) {
#pragma unroll
            for (int h = 0; h < S::kParts; ++h) {
              const uint32_t at = sa + (uint32_t)(h * 2 + m) * kTileA;
              const uint64_t ad = WANT_A ? tc::sdesc_sw128(at) : tc::sdesc_sw128_mn(at, kBox);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_bf16(tmem + m * kBN, ad + (WANT_A ? 2 : 128) * kk, bd + bstep * kk, idesc,
                             (s - t.k0) | h | kk);
            }
          }
          tc::mma_commit(&empty[slot]);
        }
        if (ok) tc::mma_commit(done);
      }
      if (!ok) {
        atomicMax(a.status, kErrTimeout);
        // what was issued completes before TMEM is freed
        tc::mma_commit(done);
        mbar_wait(done, (uint32_t)(n & 1));
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {  // ---- accumulators to global memory
    const int q = warp & 3;
    int n = 0;
    for (int i = blockIdx.x; i < a.items; i += gridDim.x, ++n) {
      const Item t = item_of<WANT_A>(a, i);
      bool ok = true;
      if (lane == 0) ok = wait_or(done, (uint32_t)(n & 1), stop, kWaitLimitNs + 20000ull * (unsigned)(t.k1 - t.k0));
      if (!__shfl_sync(0xffffffffu, ok, 0)) {
        if (lane == 0) atomicMax(a.status, kErrTimeout);
        break;
      }
      tc::fence_after_sync();
      for (int m = 0; m < t.tiles; ++m) {
        const int row = t.m0 + 128 * m + 32 * q + lane;
        const bool live = row < (WANT_A ? a.N : a.V);
        for (int c = 0; c < t.cols; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tc::tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + m * kBN + c, v);
          tc::tmem_ld_wait();
          if (!live) continue;
          if (!WANT_A && a.out_rv) {
            float* o = a.out + (size_t)(t.c0 + c) * a.V + row;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < t.cols) {
                float x = __uint_as_float(v[j]);
                if (a.accumulate) x += o[(size_t)j * a.V];
                __stcs(o + (size_t)j * a.V, x);
              }
          } else {
            float* o = a.out + (WANT_A ? ((size_t)t.split * a.N + row) : (size_t)row) * a.r + t.c0 + c;
#pragma unroll
            for (int j = 0; j < 32; j += 8)  // (r is a multiple of 8)
              if (c + j < t.cols) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[j + e]);
                if (!WANT_A && a.accumulate) {
                  const float4 x = *(const float4*)(o + j), y = *(const float4*)(o + j + 4);
                  f[0] += x.x; f[1] += x.y; f[2] += x.z; f[3] += x.w;
                  f[4] += y.x; f[5] += y.y; f[6] += y.z; f[7] += y.w;
                }
                if (WANT_A) {
                  *(float4*)(o + j) = make_float4(f[0], f[1], f[2], f[3]);
                  *(float4*)(o + j + 4) = make_float4(f[4], f[5], f[6], f[7]);
                } else {
                  __stcs((float4*)(o + j), make_float4(f[0], f[1], f[2], f[3]));
                  __stcs((float4*)(o + j + 4), make_float4(f[4], f[5], f[6], f[7]));
                }
              }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(tfree);
    }
  } else if (!S::kTma && warp >= 8) {  // ---- G from global memory, split into its parts
    using TG = typename S::T;
    const TG* G = (const TG*)a.G;
    const int pt = tid - 256;
    // a thread's sixteen quads of a stage: grad_a: row (16 i + pt / 16) of 256, quad pt % 16 of the
    // 64 entries; grad_W2: row (4 i + pt / 64) of 64, quad pt % 64 of the 256 entries
    const int prow = WANT_A ? pt >> 4 : pt >> 6, pq = WANT_A ? pt & 15 : pt & 63;
    constexpr int kRowStep = WANT_A ? 16 : 4;
    float4 r[2][8];
    auto fetch = [&](const Item& t, int s, int half) {
      const int row0 = (WANT_A ? t.m0 : s * 64) + prow + half * 8 * kRowStep;
      const int col = (WANT_A ? s * 64 : t.m0) + 4 * pq;
      const int n = (WANT_A || pq < 32 * t.tiles) ? a.V - col : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = row0 + u * kRowStep;
        const bool in = row < a.N && (!WANT_A || half == 0 || t.tiles == 2);
        r[half][u] = load_quad<TG, S::kVec>(G + (long long)row * a.V + col, in ? n : 0);
      }
    };
    auto put = [&](uint8_t* st, const Item& t, int half) {
      if (WANT_A ? (half == 1 && t.tiles == 1) : pq >= 32 * t.tiles) return;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = prow + (half * 8 + u) * kRowStep;
        const int box = WANT_A ? row >> 6 : pq >> 4, y = row & 63, x = pq & 15;
        const uint32_t at = (uint32_t)(box * kBox + y * 128 + (((x >> 1) ^ (y & 7)) << 4) + (x & 1) * 8);
        const uint2 hi = pack_hi(r[half][u]);
        *(uint2*)(st + at) = hi;
        if (S::kParts == 2) *(uint2*)(st + 2 * kTileA + at) = pack_lo(r[half][u], hi);
      }
    };
    int i = blockIdx.x, g = 0;
    if (i < a.items) {
      Item t = item_of<WANT_A>(a, i);
      int s = t.k0;
      fetch(t, s, 0);
      for (;;) {
        fetch(t, s, 1);
        Item nt = t;
        int ns = s + 1, ni = i;
        if (ns == t.k1) {
          ni = i + gridDim.x;
          if (ni < a.items) {
            nt = item_of<WANT_A>(a, ni);
            ns = nt.k0;
          }
        }
        const int slot = g % S::kStages;
        bool ok = true;
        if (g >= S::kStages && lane == 0) ok = wait_or(&empty[slot], (uint32_t)((g / S::kStages - 1) & 1), stop);
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          if (lane == 0) atomicMax(a.status, kErrTimeout);
          break;
        }
        uint8_t* st = smem + slot * S::kStage;
        put(st, t, 0);
        if (ni < a.items) fetch(nt, ns, 0);
        put(st, t, 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        ++g;
        if (ni >= a.items) break;
        t = nt;
        s = ns;
        i = ni;
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// grad_a from the shares, in their order: four threads per 16 bytes, each a contiguous quarter.
__global__ void __launch_bounds__(256) share_sum_kernel(long long quads, int splits,
                                                        const float4* __restrict__ part,
                                                        float4* __restrict__ out) {
  __shared__ float4 sh[4][64];
  const long long i = (long long)blockIdx.x * 64 + (threadIdx.x & 63);
  const int h = (int)threadIdx.x >> 6;
  const int per = (splits + 3) / 4, s1 = min(splits, (h + 1) * per);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < quads) {
#pragma unroll 8
    for (int s = h * per; s < s1; ++s) {
      const float4 v = part[(long long)s * quads + i];
      x.x += v.x;
      x.y += v.y;
      x.z += v.z;
      x.w += v.w;
    }
  }
  sh[h][threadIdx.x & 63] = x;
  __syncthreads();
  if (h == 0 && i < quads) {
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      const float4 v = sh[k][threadIdx.x];
      x.x += v.x;
      x.y += v.y;
      x.z += v.z;
      x.w += v.w;
    }
    out[i] = x;
  }
}

size_t bg_align(size_t x) { return (x + 255) / 256 * 256; }

// floats of shared-out results at most: kMaxItems work items of 256 x 256 per SM, and no more shares
// than that many work items
size_t share_floats(int N, int r, int nsm) {
  const size_t cap = (size_t)kMaxItems * nsm, all = cap * N * r, tiles = cap * 65536;
  return all < tiles ? all : tiles;
}

template <bool WANT_A, int MODE>
cudaError_t bg_launch(const BgArgs& a, const CUtensorMap& tg, const CUtensorMap& tb, int nsm, cudaStream_t stream) {
  using S = Src<MODE>;
  const size_t smem = (size_t)S::kStages * S::kStage + 1024 + 256;
  cudaError_t e = cudaFuncSetAttribute(bias_grad_kernel<WANT_A, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  bias_grad_kernel<WANT_A, MODE><<<a.items < nsm ? a.items : nsm, S::kThreads, smem, stream>>>(a, tg, tb);
  return cudaGetLastError();
}
template <bool WANT_A>
cudaError_t bg_mode(int mode, const BgArgs& a, const CUtensorMap& tg, const CUtensorMap& tb, int nsm,
                    cudaStream_t stream) {
  switch (mode) {
    case 0: return bg_launch<WANT_A, 0>(a, tg, tb, nsm, stream);
    case 1: return bg_launch<WANT_A, 1>(a, tg, tb, nsm, stream);
    case 2: return bg_launch<WANT_A, 2>(a, tg, tb, nsm, stream);
    default: return bg_launch<WANT_A, 3>(a, tg, tb, nsm, stream);
  }
}

cudaError_t tensor(int N, int V, int r, int g_bf16, const void* G, const bf16* a, const bf16* W2, int rv,
                   float* ga, float* gW, int accumulate, uint8_t* ws, int nsm, cudaStream_t stream) {
  const int mode = g_bf16 ? (V % 8 == 0 ? 0 : 3) : (V % 4 == 0 ? 1 : 2);
  float* part = (float*)(ws + sizeof(WsHeader));
  BgArgs p;
  p.N = N;
  p.V = V;
  p.r = r;
  p.nrb = (r + kBN - 1) / kBN;
  p.accumulate = accumulate;
  p.out_rv = rv;
  p.G = G;
  p.status = &((WsHeader*)ws)->status;
  p.nmb = p.per_split = p.b_kmajor = 0;
  CUtensorMap tg, tb;
  if (mode == 0) {
    if (!encode_bf16_2d(&tg, G, N, V, V, 64)) return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaSuccess;
  if (gW) {
    if (!encode_bf16_2d(&tb, a, N, r, r, 64)) return cudaErrorInvalidValue;
    if (mode != 0) tg = tb;  // (not used)
    p.items = (V + 255) / 256 * p.nrb;
    p.nstage_k = (N + 63) / 64;
    p.out = gW;
    if ((e = bg_mode<false>(mode, p, tg, tb, nsm, stream)) != cudaSuccess) return e;
  }
  if (ga) {
    p.b_kmajor = rv;
    const bf16* W = W2;
    if (rv && V % 8 != 0) {  // rows that TMA cannot address: a [V][r] copy in the workspace
      bf16* t = (bf16*)(ws + sizeof(WsHeader) + bg_align(share_floats(N, r, nsm) * 4));
      if ((e = launch_transpose(W2, t, r, V, 2, stream)) != cudaSuccess) return e;
      W = t;
      p.b_kmajor = 0;
    }
    if (!(p.b_kmajor ? encode_bf16_2d(&tb, W, r, V, V, 64) : encode_bf16_2d(&tb, W, V, r, r, 64)))
      return cudaErrorInvalidValue;
    if (mode != 0) tg = tb;
    p.nmb = (N + 255) / 256;
    p.nstage_k = (V + 63) / 64;
    // Shares of the vocabulary: the rounds of work items times the stages of one, against writing and
    // reading the shares' results (microseconds: a stage of 256 x 64 at the memory's rate per SM)
    const int base = p.nmb * p.nrb;
    const double stage = (g_bf16 ? 0.75 : 1.5), io = (double)N * r * 8 / 6.7e6;
    int splits = 1;
    double best = 1e300;
    for (int s = 1; s <= p.nstage_k && (long long)base * s <= (long long)kMaxItems * nsm; ++s) {
      const int per = (p.nstage_k + s - 1) / s;
      const double t = (double)((base * s + nsm - 1) / nsm) * per * stage + (s > 1 ? s * io + 2.0 : 0.0);
      if (t < best) {
        best = t;
        splits = s;
      }
    }
    p.per_split = (p.nstage_k + splits - 1) / splits;
    splits = (p.nstage_k + p.per_split - 1) / p.per_split;
    p.items = base * splits;
    p.out = splits > 1 ? part : ga;
    if ((e = bg_mode<true>(mode, p, tg, tb, nsm, stream)) != cudaSuccess) return e;
    if (splits > 1) {
      const long long quads = (long long)N * r / 4;
      share_sum_kernel<<<(unsigned)((quads + 63) / 64), 256, 0, stream>>>(quads, splits, (const float4*)part,
                                                                          (float4*)ga);
      e = cudaGetLastError();
    }
  }
  return e;
}

__global__ void __launch_bounds__(256) zero_kernel(long long n4, float4* __restrict__ p) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n4; i += (long long)gridDim.x * 256)
    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

}  // namespace

size_t bias_grad_workspace_bytes(int N, int V, int r, int w_bf16, int nsm) {
  size_t o = sizeof(WsHeader);
  if (w_bf16) o += bg_align(share_floats(N, r, nsm) * 4) + (V % 8 ? (size_t)V * r * 2 : 0);
  return o;
}

cudaError_t launch_bias_grad(int N, int V, int r, int g_bf16, const void* G, int w_bf16, const void* a,
                             const void* W2, int w2_rv, float* grad_a, float* grad_W2, int accumulate,
                             void* workspace, int nsm, cudaStream_t stream) {
  if (N == 0) {  // no rows: grad_a is empty and grad_W2 zero
    if (!grad_W2 || accumulate) return cudaSuccess;
    zero_kernel<<<4 * nsm, 256, 0, stream>>>((long long)V * r / 4, (float4*)grad_W2);
    return cudaGetLastError();
  }
  if (w_bf16)
    return tensor(N, V, r, g_bf16, G, (const bf16*)a, (const bf16*)W2, w2_rv, grad_a, grad_W2, accumulate,
                  (uint8_t*)workspace, nsm, stream);
  if (g_bf16)
    return plain(N, V, r, (const bf16*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
  return plain(N, V, r, (const float*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, stream);
}

}  // namespace dspark
