// bias_grad.cu -- the gradients of the low-rank bias product B_k = a W2 (Eq 5; Eq 6 with
// a = tanh(o)), "DSpark -- paper verification", section 1.
//
// For gradients G [N][V] of the logits, conditioning rows a [N][r] and W2 as [V][r] or [r][V]:
//   grad_a[n][j] = sum_v G[n][v] W2[v][j],   grad_W2[v][j] = sum_n G[n][v] a[n][j].
//
// bf16 weights: two tensor-core products (tcgen05, kind::f16, fp32 accumulation in TMEM), each with
// G as the M-side operand and 256 columns of the other one:
//   grad_W2: M = 128 vocabulary entries (G as it lies is M-major), K = N; one tile per work item;
//   grad_a:  M = 128 rows, K = a share of the vocabulary (G as it lies is K-major); the shares'
//            fp32 results are added in order by a second launch.
// A block per SM walks over its work items: a TMA thread, one thread that issues the MMAs, eight
// warps that read the accumulators out of TMEM.  An fp32 G enters as two bf16 parts, G = hi + lo with
// hi = bf16(G), lo = bf16(G - hi) (16 significant bits or more, an error of at most 2^-18 |G|,
// below that of an fp32 sum of these lengths); eight warps split it on its way from global to
// shared memory.  The same warps bring a G whose rows TMA cannot address.
//
// The tensor cores add into fp32 accumulators with truncation: over a long K the sums shrink by about
// 2e-8 of themselves per MMA (measured: 1.5e-5 after 784).  So after every 32 MMAs of a tile the
// accumulators are added, rounded to nearest, to a second set of 256 TMEM columns and start anew.
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
constexpr int kRun = 32;              // MMAs of K = 16 into one set of accumulators

struct BgArgs {
  int N, V, r;
  int items, nrb;       // work items; blocks of 256 columns of r
  int nmb;              // grad_a: blocks of 128 rows
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

// One work item: the tile's first row, its first and last K stage, its columns.
struct Item {
  int m0, k0, k1, c0, cols, split;
};
template <bool WANT_A>
__device__ __forceinline__ Item item_of(const BgArgs& a, int i) {
  Item t;
  const int rb = i % a.nrb;
  i /= a.nrb;
  t.c0 = rb * kBN;
  t.cols = min(kBN, a.r - t.c0);
  if (WANT_A) {
    t.m0 = (i % a.nmb) * 128;
    t.split = i / a.nmb;
    t.k0 = t.split * a.per_split;
    t.k1 = min(a.nstage_k, t.k0 + a.per_split);
  } else {
    t.m0 = i * 128;
    t.split = 0;
    t.k0 = 0;
    t.k1 = a.nstage_k;
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
  static constexpr int kStages = kParts == 2 ? 3 : 4;
  static constexpr int kStage = kParts * kTileA + kBytesB;
  static constexpr int kRunStages = kRun / 4 / kParts;
  static constexpr int kThreads = kTma ? 384 : 640;
  using T = typename std::conditional<MODE == 3, bf16, float>::type;
};

// Uses of registers that a TMEM load writes come after the wait for it.
__device__ __forceinline__ void loaded(uint32_t (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(v[j]));
}

// 32 columns of one row of a tile, from column c of the item's on.
template <bool WANT_A>
__device__ __forceinline__ void write_out(const BgArgs& a, const Item& t, int row, int c, const uint32_t (&v)[32]) {
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
    for (int j = 0; j < 32; j += 4)  // (r is a multiple of 8)
      if (c + j < t.cols) {
        float4 f = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                               __uint_as_float(v[j + 3]));
        if (!WANT_A && a.accumulate) {
          const float4 x = *(const float4*)(o + j);
          f.x += x.x;
          f.y += x.y;
          f.z += x.z;
          f.w += x.w;
        }
        if (WANT_A)
          *(float4*)(o + j) = f;
        else
          __stcs((float4*)(o + j), f);
      }
  }
}

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
  constexpr int kOffB = S::kParts * kTileA;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1 + (S::kTma ? 0 : 8));
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    mbar_init(tfree, 8);
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
        const uint32_t bytes = (uint32_t)(nb * kBox + (S::kTma ? kTileA : 0));
        for (int s = t.k0; s < t.k1; ++s, ++g) {
          const int slot = g % S::kStages;
          if (g >= S::kStages && !wait_or(&empty[slot], (uint32_t)((g / S::kStages - 1) & 1), stop)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + slot * S::kStage;
          mbar_expect_tx(&full[slot], bytes);
          if (S::kTma) {
            for (int b = 0; b < 2; ++b)
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
      int g = 0, n = 0;  // stages and runs so far
      bool ok = true;
      for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
        const Item t = item_of<WANT_A>(a, i);
        const uint32_t idesc = tc::idesc_bf16_f32(128, (t.cols + 15) / 16 * 16) |
                               (WANT_A ? 0u : tc::kIdescAMajorMN) |
                               (WANT_A && a.b_kmajor ? 0u : tc::kIdescBMajorMN);
        for (int s0 = t.k0; ok && s0 < t.k1; s0 += S::kRunStages) {
          if (n > 0 && !wait_or(tfree, (uint32_t)((n - 1) & 1), stop)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const int s1 = min(t.k1, s0 + S::kRunStages);
          for (int s = s0; s < s1; ++s, ++g) {
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
#pragma unroll
            for (int h = 0; h < S::kParts; ++h) {
              const uint32_t at = sa + (uint32_t)h * kTileA;
              const uint64_t ad = WANT_A ? tc::sdesc_sw128(at) : tc::sdesc_sw128_mn(at, kBox);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc::mma_bf16(tmem, ad + (WANT_A ? 2 : 128) * kk, bd + bstep * kk, idesc, (s - s0) | h | kk);
            }
            tc::mma_commit(&empty[slot]);
          }
          if (ok) {
            tc::mma_commit(done);
            ++n;
          }
        }
      }
      if (!ok) {
        atomicMax(a.status, kErrTimeout);
        // what was issued completes before TMEM is freed
        tc::mma_commit(done);
        mbar_wait(done, (uint32_t)(n & 1));
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {  // ---- accumulators: to the sums, or to global memory
    const int q = warp & 3, c_lo = warp < 8 ? 0 : kBN / 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    int n = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
      const Item t = item_of<WANT_A>(a, i);
      const int row = t.m0 + 32 * q + lane, c_hi = min(t.cols, c_lo + kBN / 2);
      const bool live = row < (WANT_A ? a.N : a.V);
      for (int s0 = t.k0; s0 < t.k1; s0 += S::kRunStages, ++n) {
        const bool first = s0 == t.k0, last = s0 + S::kRunStages >= t.k1;
        if (lane == 0) ok = wait_or(done, (uint32_t)(n & 1), stop);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) atomicMax(a.status, kErrTimeout);
          break;
        }
        tc::fence_after_sync();
        for (int c = c_lo; c < c_hi; c += 32) {
          uint32_t v[32];
          __syncwarp();
          tc::tmem_ld32(lanes + c, v);
          if (!first) {
            uint32_t w[32];
            tc::tmem_ld32(lanes + kBN + c, w);
            tc::tmem_ld_wait();
            loaded(v);
            loaded(w);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + __uint_as_float(w[j]));
          } else {
            tc::tmem_ld_wait();
            loaded(v);
          }
          if (!last) {
            tc::tmem_st32(lanes + kBN + c, v);
          } else if (live) {
            write_out<WANT_A>(a, t, row, c, v);
          }
        }
        tc::tmem_st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(tfree);
      }
    }
  } else if (!S::kTma && warp >= 12) {  // ---- G from global memory, split into its parts
    using TG = typename S::T;
    const TG* G = (const TG*)a.G;
    const int pt = tid - 384;
    // a thread's eight quads of a stage: grad_a: row (16 u + pt / 16) of 128, quad pt % 16 of the 64
    // entries; grad_W2: row (8 u + pt / 32) of 64, quad pt % 32 of the 128 entries
    const int prow = WANT_A ? pt >> 4 : pt >> 5, pq = WANT_A ? pt & 15 : pt & 31;
    constexpr int kRowStep = WANT_A ? 16 : 8;
    float4 r[2][8];
    auto fetch = [&](const Item& t, int s, float4 (&x)[8]) {
      const int row0 = (WANT_A ? t.m0 : s * 64) + prow;
      const int col = (WANT_A ? s * 64 : t.m0) + 4 * pq, n = a.V - col;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int row = row0 + u * kRowStep;
        x[u] = load_quad<TG, S::kVec>(G + (long long)row * a.V + col, row < a.N ? n : 0);
      }
    };
    // the stage after (i, s); i past the last item: none
    auto step = [&](int& i, Item& t, int& s) {
      if (++s == t.k1) {
        i += gridDim.x;
        if (i < a.items) {
          t = item_of<WANT_A>(a, i);
          s = t.k0;
        }
      }
    };
    int i = blockIdx.x, g = 0, s = 0;
    Item t = {};
    if (i < a.items) {
      t = item_of<WANT_A>(a, i);
      s = t.k0;
      fetch(t, s, r[0]);
      step(i, t, s);
      for (bool more = true; more;) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {  // stage g is in r[p]; the next goes to the other half
          if (!more) break;
          more = i < a.items;
          if (more) {
            fetch(t, s, r[p ^ 1]);
            step(i, t, s);
          }
          const int slot = g % S::kStages;
          bool ok = true;
          if (g >= S::kStages && lane == 0) ok = wait_or(&empty[slot], (uint32_t)((g / S::kStages - 1) & 1), stop);
          if (!__shfl_sync(0xffffffffu, ok, 0)) {
            if (lane == 0) atomicMax(a.status, kErrTimeout);
            more = false;
            break;
          }
          uint8_t* st = smem + slot * S::kStage;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int row = prow + u * kRowStep;
            const int box = WANT_A ? row >> 6 : pq >> 4, y = row & 63, x = pq & 15;
            const uint32_t at = (uint32_t)(box * kBox + y * 128 + (((x >> 1) ^ (y & 7)) << 4) + (x & 1) * 8);
            const uint2 hi = pack_hi(r[p][u]);
            *(uint2*)(st + at) = hi;
            if (S::kParts == 2) *(uint2*)(st + kTileA + at) = pack_lo(r[p][u], hi);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]);
          ++g;
        }
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

// floats of shared-out results at most: kMaxItems work items of 128 x 256 per SM, and no more shares
// than that many work items
size_t share_floats(int N, int r, int nsm) {
  const size_t cap = (size_t)kMaxItems * nsm, all = cap * N * r, tiles = cap * 128 * kBN;
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
    p.items = (V + 127) / 128 * p.nrb;
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
    p.nmb = (N + 127) / 128;
    p.nstage_k = (V + 63) / 64;
    // Shares of the vocabulary: the rounds of work items times the stages of one, against writing and
    // reading the shares' results (microseconds: a stage of 128 x 64 at the memory's rate per SM)
    const int base = p.nmb * p.nrb;
    const double stage = (g_bf16 ? 0.38 : 0.75), io = (double)N * r * 8 / 6.7e6;
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
