// bias_grad.cu -- the gradients of the low-rank bias product B_k = a W2 (Eq 5; Eq 6 with
// a = tanh(o)), "DSpark -- paper verification", section 1.
//
// For gradients G [N][V] of the logits, conditioning rows a [N][r] and W2 as [V][r] or [r][V]:
//   grad_a[n][j] = sum_v G[n][v] W2[v][j],   grad_W2[v][j] = sum_n G[n][v] a[n][j].
//
// bf16 weights: two tensor-core products (tcgen05, kind::f16, fp32 accumulation in TMEM), each with
// G as the M-side operand and 256 columns of the other one:
//   grad_W2: M = vocabulary entries (G as it lies is M-major), K = N; one tile per work item;
//   grad_a:  M = rows, K = a share of the vocabulary (G as it lies is K-major); the shares' fp32 results
//            are added in order by a second launch.
// One block per SM walks over work items: TMA threads, one thread that issues the MMAs, eight warps that
// read the accumulators out of TMEM.
// A bf16 G comes by TMA, and a pair of CTAs (cta_group::2) takes an item of 256 rows: each holds 128 of
// them and half the columns, so that W2 or a reaches each SM's shared memory once per 256 rows of G.
// An fp32 G enters as three bf16 parts, hi = bf16(G), mid = bf16(G - hi), lo = bf16(G - hi - mid): all
// 24 bits (two parts measured 2.5e-6 of the result off, an fp32 product 1e-6); where |G| is above bf16's
// largest number, as parts cut off and not rounded, so that they are finite.  TMA brings it as it
// lies, and eight warps split it from one shared-memory buffer into another.  A G whose rows TMA
// cannot address is brought by the same warps: fp32 element by element, bf16 by copied words (3584 x 262143
// x 256 2.7 ms, three and a half times the aligned size).  These
// paths take items of 128 rows, one CTA each (a pair gained nothing there: the signals between its CTAs
// cost what the halved operand saved).
//
// The tensor cores add into fp32 accumulators with truncation: over a long K the sums shrink by about
// 2e-8 of themselves per MMA (measured: 1.5e-5 after 784).  So a run of 24 or 32 MMAs goes to one half
// of TMEM, and while the next run goes to the other half, the eight warps add the first to sums in
// their registers (128 columns of a row per thread), rounded to nearest.
//
// 3584 x 262144 x 256 from bf16: 820 us in a row of calls (370 us per product alone; a library bf16
// product of the same operands 357 and 313; one CTA per item 385 and 400).  G's stream bounds it: with 16
// columns in place of 256 a product still takes 335 us (5.6 TB/s).  448 x 151936 x 256 from fp32: 207 us,
// 95 and 105 per product.  Copies with a step taken out took, of the 95 of grad_a: the split 82, two
// thirds of the MMAs 88, W2 88, reading the accumulators 89, all of them 50: the chain of the steps bounds
// it, through shared memory that moves 288 KB per 64-deep stage (2250 cycles of about 2430).  Fences at
// cluster scope in a pair's signals had cost 60 us.
// fp32 weights (small heads): CUDA-core tiles, 22 to 26 TFLOP/s (256 x 8192 x 128 50 us, 448 x 151936 x 256
// 2.7 ms, twice a library fp32 product).
#include <cuda.h>

#include "draft.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dspark {
namespace {

using bf16 = __nv_bfloat16;

// ------------------------------------------------------------------ fp32 weights: CUDA cores
// C[share][m][n] (+)= sum over the share's k of A(m, k) B(k, n): 64 x 64 tiles, 16 products per thread
// and step of K, the next 32 steps' elements in registers meanwhile.  A and B by row and column strides
// (the index with unit stride goes along the lanes).
constexpr int kFT = 64, kFK = 32, kFE = kFT * kFK / 256;  // kFE: elements of a tile per thread

template <typename TA, typename TB>
__global__ void __launch_bounds__(256) gemm_f32_kernel(int M, int Nn, int K, int per, const TA* __restrict__ A,
                                                       long long am, long long ak, const TB* __restrict__ B,
                                                       long long bk, long long bn, float* __restrict__ C,
                                                       long long cm, long long cn, long long cshare,
                                                       int accumulate) {
  __shared__ float sa[2][kFK][kFT + 4], sb[2][kFK][kFT + 4];
  pdl_trigger();
  const int m0 = blockIdx.x * kFT, n0 = blockIdx.y * kFT, tid = threadIdx.x;
  const int ka = blockIdx.z * per, kb = min(K, ka + per);
  const int tx = tid & 15, ty = tid >> 4;
  float ra[kFE], rb[kFE], acc[4][4] = {};
  // element e of a thread: (k, m) by 256 e + tid, with k or m along the lanes
  auto at_a = [&](int e, int& k, int& m) {
    const int i = e * 256 + tid;
    k = ak == 1 ? i % kFK : i / kFT;
    m = ak == 1 ? i / kFK : i % kFT;
  };
  auto at_b = [&](int e, int& k, int& n) {
    const int i = e * 256 + tid;
    k = bn == 1 ? i / kFT : i % kFK;
    n = bn == 1 ? i % kFT : i / kFK;
  };
  auto fetch = [&](int k0) {
#pragma unroll
    for (int e = 0; e < kFE; ++e) {
      int k, m;
      at_a(e, k, m);
      ra[e] = k0 + k < kb && m0 + m < M ? to_f<TA>(A[(m0 + m) * am + (k0 + k) * ak]) : 0.f;
      at_b(e, k, m);
      rb[e] = k0 + k < kb && n0 + m < Nn ? to_f<TB>(B[(k0 + k) * bk + (n0 + m) * bn]) : 0.f;
    }
  };
  fetch(ka);
  int p = 0;
  for (int k0 = ka; k0 < kb; k0 += kFK, p ^= 1) {
#pragma unroll
    for (int e = 0; e < kFE; ++e) {
      int k, m;
      at_a(e, k, m);
      sa[p][k][m] = ra[e];
      at_b(e, k, m);
      sb[p][k][m] = rb[e];
    }
    __syncthreads();  // (the other buffer's readers passed this barrier's predecessor)
    if (k0 + kFK < kb) fetch(k0 + kFK);
#pragma unroll
    for (int k = 0; k < kFK; ++k) {
      const float4 x = *(const float4*)&sa[p][k][ty * 4], y = *(const float4*)&sb[p][k][tx * 4];
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
    }
  }
  C += blockIdx.z * cshare;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < Nn) {
        float* c = C + m * cm + n * cn;
        *c = accumulate ? *c + acc[i][j] : acc[i][j];
      }
    }
  // grad_a's launch runs beside grad_W2's (neither reads what the other writes) but does not end before
  // it, so that whatever waits for this launch finds both done.
  pdl_wait();
}

// ------------------------------------------------------------------ bf16 weights: tensor cores
constexpr int kBox = 64 * 128;        // bytes of one shared-memory box: 64 rows of 64 bf16
constexpr int kTileA = 2 * kBox;      // 128 (M) x 64 (K) of G
constexpr int kBN = 256;              // columns of a work item
constexpr int kMaxItems = 2;          // work items per CTA or pair at most when the vocabulary is shared out
constexpr int kRawBytes = 128 * 32 * 4;  // half a stage of an fp32 G as it lies
constexpr int kWordBytes = 2 * 16 * 128 * 4;  // a half stage's words of G, those of unaligned rows twice
constexpr unsigned long long kStuckNs = 20000, kSettleNs = 1000000;
constexpr int kDeep = 4;              // half stages of words in flight per group of four warps
// Registers per thread where eight more warps bring G (640 threads, launched with 96 each): the
// three shares, 128 x (48 + 2 x 160 + 2 x 56), are the launch's 640 x 96.
constexpr int kRegsIssue = 48, kRegsSums = 160, kRegsBring = 56;

struct BgArgs {
  int N, V, r;
  int items, nrb;       // work items; blocks of 256 columns of r
  int nmb;              // grad_a: blocks of 128 rows (a pair: 256)
  int per_split;        // grad_a: K stages per share of the vocabulary
  int nstage_k;         // K stages in all
  int b_kmajor;         // grad_a: W2 is [r][V]
  int out_rv;           // grad_W2 is [r][V]
  int accumulate;
  int wide;             // out is 32-byte aligned
  int stuck;            // failure-path test hook: a wait of the sums (1) or of the MMA thread (2) runs out
  float* out;           // grad_W2, or grad_a's shares [split][N][r]
  const void* G;
  unsigned* status;
};

// How a block gives up: a flag that its roles look at while they wait, and in a pair the other CTA's flag.
struct Stop {
  volatile int* mine;
  uint32_t other;  // shared::cluster address, 0 without a pair
};
__device__ __forceinline__ void give_up(Stop stop) {
  *stop.mine = 1;
  if (stop.other) asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(stop.other), "r"(1) : "memory");
}
// A bounded wait of one thread that also ends when another role of the block, or of the pair, gave up.
__device__ __forceinline__ bool wait_or(uint64_t* bar, uint32_t parity, Stop stop,
                                        unsigned long long limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) {
    if (*stop.mine) return false;
    if (globaltimer() - t0 > limit_ns) {
      give_up(stop);
      return false;
    }
  }
  return true;
}

// One work item as a CTA sees it: its 128 rows, the K stages, the columns; the columns that the MMA takes
// (a multiple of 16, in a pair of 32: the MMA of two CTAs takes no others), and those of them that this
// CTA brings (half of them in a pair): first, number.
struct Item {
  int m0, k0, k1, c0, cols, split, n, b0, nb;
};
template <bool WANT_A, bool PAIR>
__device__ __forceinline__ Item item_of(const BgArgs& a, int i, int rank) {
  Item t;
  const int rb = i % a.nrb;
  i /= a.nrb;
  t.c0 = rb * kBN;
  t.cols = min(kBN, a.r - t.c0);
  t.n = PAIR ? (t.cols + 31) / 32 * 32 : (t.cols + 15) / 16 * 16;  // (the columns past r are zeros)
  t.nb = PAIR ? t.n / 2 : t.n;
  t.b0 = t.c0 + rank * t.nb;
  if (WANT_A) {
    t.m0 = (i % a.nmb) * (PAIR ? 256 : 128) + rank * 128;
    t.split = i / a.nmb;
    t.k0 = t.split * a.per_split;
    t.k1 = min(a.nstage_k, t.k0 + a.per_split);
  } else {
    t.m0 = i * (PAIR ? 256 : 128) + rank * 128;
    t.split = 0;
    t.k0 = 0;
    t.k1 = a.nstage_k;
  }
  return t;
}

// Four consecutive elements of a row of G, zero from `n` on.
__device__ __forceinline__ float4 load_quad(const float* p, int n) {
  if (n <= 0) return make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}
// bf16 of four values, and what it leaves of them (exactly): numbers up to bf16's largest, NaN
__device__ __forceinline__ uint2 take_bf16(float4& f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
  uint2 w;
  memcpy(&w.x, &a, 4);
  memcpy(&w.y, &b, 4);
  f.x -= __uint_as_float(w.x << 16);
  f.y -= __uint_as_float(w.x & 0xFFFF0000u);
  f.z -= __uint_as_float(w.y << 16);
  f.w -= __uint_as_float(w.y & 0xFFFF0000u);
  return w;
}
// The same of any numbers, by cutting off and not rounding, so that the part of a finite number is finite.
// An infinity leaves nothing.
__device__ __forceinline__ float left_of(float x) {
  const float part = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
  return x == part ? 0.f : x - part;
}
__device__ __forceinline__ uint2 cut_bf16(float4& f) {
  const uint2 w = make_uint2(__byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632),
                             __byte_perm(__float_as_uint(f.z), __float_as_uint(f.w), 0x7632));
  f = make_float4(left_of(f.x), left_of(f.y), left_of(f.z), left_of(f.w));
  return w;
}
__device__ __forceinline__ float abs_max(const float4& f) {
  return fmaxf(fmaxf(fabsf(f.x), fabsf(f.y)), fmaxf(fabsf(f.z), fabsf(f.w)));
}
constexpr float kBf16Most = 3.3895313892515355e38f;  // bf16's largest finite number

// MODE 0: bf16 G by TMA.  1: fp32 G by TMA, split into three parts.  2: fp32 G element by element.
// 3: bf16 G element by element (one part).
template <int MODE>
struct Src {
  static constexpr bool kTma = MODE == 0, kTmaRaw = MODE == 1;
  static constexpr bool kPair = kTma;
  static constexpr int kBM = kPair ? 256 : 128;
  static constexpr int kTileB = (kPair ? 2 : 4) * kBox;  // 64 (K) x 128 or 256 of W2 or a
  static constexpr int kParts = MODE == 1 || MODE == 2 ? 3 : 1;
  static constexpr int kStagesA = kTma ? 6 : 2;  // of G's parts
  static constexpr int kStagesB = kTma ? 6 : 2;  // of W2 or a
  // Where warps bring G, a stage is filled, multiplied and freed in halves of 32 of its K: twice the
  // steps in flight in the same memory (the chain of fill, MMAs and signals bounds this path).
  static constexpr int kHalves = kTma ? 1 : 2;
  static constexpr int kSlotsA = kStagesA * kHalves;
  static constexpr int kRaw = kTmaRaw ? 4 : 0;          // half stages of an fp32 G as it lies
  static constexpr int kStageA = kParts * kTileA;
  static constexpr int kRunStages = kParts == 3 ? 2 : 8;  // 24 or 32 MMAs into one set of accumulators
  static constexpr int kThreads = kTma ? 384 : 640;
  static constexpr int kOffB = kStagesA * kStageA, kOffRaw = kOffB + kStagesB * kTileB,
                       kOffBar = kOffRaw + (MODE == 3 ? 2 * kDeep * kWordBytes : kRaw * kRawBytes);
  static constexpr int kSmem = kOffBar + 512 + 1024;
  // The two groups of warps take alternate half stages: with an even number of slots a slot is always
  // the same group's, which has then seen every phase of its barriers before the one it waits for.
  static_assert(kTma || (kSlotsA % 2 == 0 && kRaw % 2 == 0), "a slot belongs to one group");
};

// A thread's part of a finished tile: columns c0 .. c0 + 127 of the item's, of one row.
template <bool WANT_A>
__device__ __forceinline__ void write_out(const BgArgs& a, const Item& t, int row, int c0, const float (&x)[kBN / 2]) {
  if (!WANT_A && a.out_rv) {
    float* o = a.out + (size_t)(t.c0 + c0) * a.V + row;
#pragma unroll
    for (int j = 0; j < kBN / 2; ++j)
      if (c0 + j < t.cols) {
        float f = x[j];
        if (a.accumulate) f += *o;
        __stcs(o, f);
        o += a.V;
      }
  } else {
    float* o = a.out + (WANT_A ? ((size_t)t.split * a.N + row) : (size_t)row) * a.r + t.c0 + c0;
#pragma unroll
    for (int j = 0; j < kBN / 2; j += 8)  // (r is a multiple of 8)
      if (c0 + j < t.cols) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = !WANT_A && a.accumulate ? x[j + e] + o[j + e] : x[j + e];
        if (a.wide) {  // whole sectors
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + j), "f"(f[0]), "f"(f[1]),
                       "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
                       : "memory");
        } else {
          *(float4*)(o + j) = make_float4(f[0], f[1], f[2], f[3]);
          *(float4*)(o + j + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
  }
}

template <bool WANT_A, int MODE>
__global__ void __cluster_dims__(Src<MODE>::kPair ? 2 : 1, 1, 1) __launch_bounds__(Src<MODE>::kThreads, 1)
    bias_grad_kernel(const BgArgs a, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmB) {
  using S = Src<MODE>;
  constexpr bool kPair = S::kPair;
  constexpr int kTileB = S::kTileB, kSA = S::kSlotsA, kSB = S::kStagesB, kRaw = S::kRaw > 0 ? S::kRaw : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* raw = smem + S::kOffRaw;
  // Of a pair's two copies, rank 0's count: G's parts in place (afull), W2 or a in place (bfull),
  // accumulators read (tfree).  Both ranks' own: MMAs have read a stage (aempty, bempty), a run's MMAs
  // are complete (done), an fp32 G has arrived or been split (rfull, rempty).
  uint64_t* afull = (uint64_t*)(smem + S::kOffBar);
  uint64_t* aempty = afull + kSA;
  uint64_t* bfull = aempty + kSA;
  uint64_t* bempty = bfull + kSB;
  uint64_t* done = bempty + kSB;
  uint64_t* tfree = done + 2;
  uint64_t* rfull = tfree + 2;
  uint64_t* rempty = rfull + kRaw;
  uint32_t* tbase = (uint32_t*)(rempty + kRaw);
  uint64_t* never = (uint64_t*)(tbase + 2);  // nothing arrives here
  static_assert((2 * kSA + 2 * kSB + 4 + 2 * kRaw) * 8 + 16 <= 512, "barriers fit");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kPair ? (int)cluster_rank() : 0;
  const Stop stop{(volatile int*)(tbase + 1), kPair ? cluster_addr(tbase + 1, rank ^ 1) : 0u};
  const int pair = (int)blockIdx.x >> (kPair ? 1 : 0), pairs = (int)gridDim.x >> (kPair ? 1 : 0);

  if (tid == 0) {
    for (int i = 0; i < kSA; ++i) {
      mbar_init(&afull[i], S::kTma ? 1 : 4);
      mbar_init(&aempty[i], 1);
    }
    for (int i = 0; i < kSB; ++i) {
      mbar_init(&bfull[i], 1);
      mbar_init(&bempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&done[i], 1);
      mbar_init(&tfree[i], kPair ? 16 : 8);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], 4);
    }
    mbar_init(never, 1);
    *stop.mine = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (kPair) cluster_sync_all();  // both CTAs are there
  pdl_trigger();  // (grad_a's launch, or the sum of its shares, may follow)
  if (warp == 1) {
    if (kPair) {
      tc::tmem_alloc_pair(tbase, 512);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(tbase, 512);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (kPair) cluster_sync_all();  // both CTAs' barriers and TMEM are ready
  tc::fence_after_sync();
  const uint32_t tmem = *tbase;

  if (warp < 4) {
    if (!S::kTma) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && lane == 0) {  // ---- TMA: W2 or a
      const uint64_t keep = policy_evict_last();
      int g = 0;
      bool ok = true;
      for (int i = pair; ok && i < a.items; i += pairs) {
        const Item t = item_of<WANT_A, kPair>(a, i, rank);
        const int nb = (t.nb + 63) / 64;
        for (int s = t.k0; s < t.k1; ++s, ++g) {
          const int slot = g % kSB;
          if (g >= kSB && !wait_or(&bempty[slot], (uint32_t)((g / kSB - 1) & 1), stop)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + S::kOffB + slot * kTileB;
          if (rank == 0) mbar_expect_tx(&bfull[slot], (uint32_t)((kPair ? 2 : 1) * nb * kBox));  // both CTAs' boxes
          for (int b = 0; b < nb; ++b) {
            const int c = t.b0 + 64 * b;
            const bool km = WANT_A && a.b_kmajor;
            if (kPair)
              tc::tma_load_2d_pair(st + b * kBox, &tmB, km ? s * 64 : c, km ? c : s * 64, cluster_addr(&bfull[slot], 0),
                                   keep);
            else
              tc::tma_load_2d(st + b * kBox, &tmB, km ? s * 64 : c, km ? c : s * 64, &bfull[slot], keep);
          }
        }
      }
      if (!ok) atomicMax(a.status, kErrTimeout);
      // every copy lands before the pair ends (the phase of each slot's last use)
      if (rank == 0)
        for (int j = max(0, g - kSB); j < g && mbar_wait(&bfull[j % kSB], (uint32_t)((j / kSB) & 1)); ++j) {}
    } else if ((S::kTma || S::kTmaRaw) && warp == 2 && lane == 0) {  // ---- TMA: G
      const uint64_t once = policy_evict_first();
      constexpr int kS = S::kTma ? kSA : kRaw;
      int g = 0;
      bool ok = true;
      for (int i = pair; ok && i < a.items; i += pairs) {
        const Item t = item_of<WANT_A, kPair>(a, i, rank);
        for (int s = t.k0 * S::kHalves; s < t.k1 * S::kHalves; ++s, ++g) {
          const int slot = g % kS;
          if (g >= kS && !wait_or(S::kTma ? &aempty[slot] : &rempty[slot], (uint32_t)((g / kS - 1) & 1), stop)) {
            ok = false;
            break;
          }
          if (S::kTma) {
            if (rank == 0) mbar_expect_tx(&afull[slot], 2 * kTileA);
            const uint32_t bar = cluster_addr(&afull[slot], 0);
            uint8_t* st = smem + slot * S::kStageA;
            for (int b = 0; b < 2; ++b)
              if (WANT_A)
                tc::tma_load_2d_pair(st + b * kBox, &tmG, s * 64, t.m0 + 64 * b, bar, once);
              else
                tc::tma_load_2d_pair(st + b * kBox, &tmG, t.m0 + 64 * b, s * 64, bar, once);
          } else {
            mbar_expect_tx(&rfull[slot], kRawBytes);
            tc::tma_load_2d(raw + slot * kRawBytes, &tmG, WANT_A ? s * 32 : t.m0, WANT_A ? t.m0 : s * 32,
                            &rfull[slot], once);
          }
        }
      }
      if (!ok) atomicMax(a.status, kErrTimeout);
      if (!S::kTma || rank == 0)
        for (int j = max(0, g - kS);
             j < g && mbar_wait(S::kTma ? &afull[j % kS] : &rfull[j % kS], (uint32_t)((j / kS) & 1)); ++j) {}
    } else if (warp == 1 && lane == 0 && rank == 0) {  // ---- MMA, for both CTAs
      auto commit = [](uint64_t* bar) {
        if (kPair)
          tc::mma_commit_pair(bar);
        else
          tc::mma_commit(bar);
      };
      int g = 0, n = 0;  // stages and runs so far
      bool ok = a.stuck != 2 || wait_or(never, 0, stop, kStuckNs);
      for (int i = pair; ok && i < a.items; i += pairs) {
        const Item t = item_of<WANT_A, kPair>(a, i, 0);
        const uint32_t idesc = tc::idesc_bf16_f32(S::kBM, t.n) | (WANT_A ? 0u : tc::kIdescAMajorMN) |
                               (WANT_A && a.b_kmajor ? 0u : tc::kIdescBMajorMN);
        for (int s0 = t.k0; ok && s0 < t.k1; s0 += S::kRunStages) {
          const int buf = n & 1;
          if (n > 1 && !wait_or(&tfree[buf], (uint32_t)((n / 2 - 1) & 1), stop)) {
            ok = false;
            break;
          }
          const int s1 = min(t.k1, s0 + S::kRunStages);
          for (int s = s0; s < s1; ++s, ++g) {
            const int slb = g % kSB;
            if (!wait_or(&bfull[slb], (uint32_t)((g / kSB) & 1), stop)) {
              ok = false;
              break;
            }
            const uint32_t sa = smem_u32(smem + (g % S::kStagesA) * S::kStageA);
            const uint32_t sb = smem_u32(smem + S::kOffB + slb * kTileB);
            // K-major: 16 elements of K are 32 bytes along the rows; M- or N-major: 16 rows of 128 bytes
            const uint64_t bd = WANT_A && a.b_kmajor ? tc::sdesc_sw128(sb) : tc::sdesc_sw128_mn(sb, kBox);
            const uint64_t bstep = WANT_A && a.b_kmajor ? 2 : 128;
#pragma unroll
            for (int half = 0; half < S::kHalves; ++half) {
              const int ga = g * S::kHalves + half, sla = ga % kSA;
              if (!wait_or(&afull[sla], (uint32_t)((ga / kSA) & 1), stop)) {
                ok = false;
                break;
              }
              tc::fence_after_sync();
#pragma unroll
              for (int h = 0; h < S::kParts; ++h) {
                const uint32_t at = sa + (uint32_t)h * kTileA;
                const uint64_t ad = WANT_A ? tc::sdesc_sw128(at) : tc::sdesc_sw128_mn(at, kBox);
#pragma unroll
                for (int j = 0; j < 4 / S::kHalves; ++j) {
                  const int kk = half * (4 / S::kHalves) + j;
                  if (kPair)
                    tc::mma_bf16_pair(tmem + buf * kBN, ad + (WANT_A ? 2 : 128) * kk, bd + bstep * kk, idesc,
                                      (s - s0) | half | h | j);
                  else
                    tc::mma_bf16(tmem + buf * kBN, ad + (WANT_A ? 2 : 128) * kk, bd + bstep * kk, idesc,
                                 (s - s0) | half | h | j);
                }
              }
              commit(&aempty[sla]);
            }
            if (!ok) break;
            commit(&bempty[slb]);
          }
          if (ok) {
            commit(&done[buf]);
            ++n;
          }
        }
      }
      if (!ok) {
        atomicMax(a.status, kErrTimeout);
        commit(&done[n & 1]);
        ++n;
      }
      // what was issued completes before TMEM is freed, whether or not anything else waits for it
      if (n > 0) mbar_wait(&done[(n - 1) & 1], (uint32_t)(((n - 1) / 2) & 1));
    }
    __syncwarp();
  } else if (warp < 12) {  // ---- accumulators to the sums, sums to global memory
    if (!S::kTma) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums));
    const int q = warp & 3, c_lo = warp < 8 ? 0 : kBN / 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + c_lo;
    int n = 0;
    bool ok = true;
    if (a.stuck == 1) {
      if (lane == 0 && !wait_or(never, 0, stop, kStuckNs)) atomicMax(a.status, kErrTimeout);
      __syncwarp();
      ok = false;
    }
    for (int i = pair; ok && i < a.items; i += pairs) {
      const Item t = item_of<WANT_A, kPair>(a, i, rank);
      float x[kBN / 2];
#pragma unroll
      for (int j = 0; j < kBN / 2; ++j) x[j] = 0.f;
      for (int s0 = t.k0; s0 < t.k1; s0 += S::kRunStages, ++n) {
        const int buf = n & 1;
        if (lane == 0) ok = wait_or(&done[buf], (uint32_t)((n / 2) & 1), stop);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) atomicMax(a.status, kErrTimeout);
          break;
        }
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < kBN / 2; c += 16)
          if (c_lo + c < t.cols) {
            uint32_t v[16];
            tc::tmem_ld16_wait(lanes + buf * kBN + c, v);
#pragma unroll
            for (int j = 0; j < 16; ++j) x[c + j] += __uint_as_float(v[j]);
          }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (kPair)
            tc::mbar_arrive_cluster_relaxed(cluster_addr(&tfree[buf], 0));
          else
            mbar_arrive(&tfree[buf]);
        }
      }
      const int row = t.m0 + 32 * q + lane;
      if (ok && row < (WANT_A ? a.N : a.V)) write_out<WANT_A>(a, t, row, c_lo, x);
      __syncwarp();
    }
  } else if (!S::kTma) {  // ---- G into its parts
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsBring));
    // Two groups of four warps take alternate half stages, so that one group's waits and fences pass
    // beside the other's work.  A thread's eight quads of a half: grad_a: 128 rows of 8 quads (the rows
    // of a warp are four apart in pairs: their swizzled stores meet all banks); grad_W2: 32 rows of 32.
    const int half = (warp - 12) >> 2, pt = (tid - 384) & 127, j8 = pt >> 3;
    const int prow = WANT_A ? (j8 & 1) * 4 + ((j8 >> 1) & 3) + (j8 & 8) : pt >> 5, pq = WANT_A ? pt & 7 : pt & 31;
    constexpr int kRowStep = WANT_A ? 16 : 4, kRowQuads = WANT_A ? 8 : 32;
    int g = 0;  // stages so far
    bool ok = true;
    if constexpr (MODE == 3) {
      // bf16 rows that start at any element: pairs of entries, consecutive along the lanes (half a warp
      // per row of 32 in grad_a, two warps per row of 128 in grad_W2), from one 32-bit word, or from two
      // where the row starts in the middle of one.  Every thread copies its own words ahead
      // (asynchronously, kDeep half stages) and puts them in place when their turn comes.
      const int row_of = WANT_A ? pt >> 4 : pt >> 6, x2 = WANT_A ? (pt & 15) * 2 : (pt & 63) * 2;
      constexpr int kRows = WANT_A ? 8 : 2;  // rows per round (even: a thread's rows are all odd or all even)
      const bool odd = (row_of & a.V & 1) != 0;
      const long long words = ((long long)a.N * a.V) >> 1;  // (then perhaps half of one)
      uint32_t* mine = (uint32_t*)(raw + half * kDeep * kWordBytes) + pt;
      const long long dk = (long long)kRows * a.V / 2;  // words from one of a thread's rows to its next
      auto copy = [&](const Item& t, int s, int slot) {
        const int row0 = (WANT_A ? t.m0 : s * 64 + 32 * half) + row_of;
        const int col = (WANT_A ? s * 64 + 32 * half : t.m0) + x2, left = a.V - col;
        const int rows = left > 0 && row0 < a.N ? min(16, (a.N - row0 + kRows - 1) / kRows) : 0;
        const long long k0 = ((long long)row0 * a.V + col) >> 1;
        const uint32_t* src = (const uint32_t*)a.G + k0;
        uint32_t dst = smem_u32(mine + slot * (kWordBytes / 4));
        // the word that only half exists, if it is one of these: a thread's last row's first or second
        const int half0 = k0 + (rows - 1) * dk == words ? rows - 1 : -1;
        const int half1 = k0 + 1 + (rows - 1) * dk == words ? rows - 1 : -1;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const bool in = u < rows;  // zeros where there is nothing to copy
          const uint32_t* p = in ? src : (const uint32_t*)a.G;
          const uint32_t n0 = !in ? 0u : u == half0 ? 2u : 4u;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(p), "r"(n0) : "memory");
          if (odd) {
            const bool in1 = in && left > 1;
            const uint32_t n1 = !in1 ? 0u : u == half1 ? 2u : 4u;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 16 * 512), "l"(in1 ? p + 1 : p),
                         "r"(n1)
                         : "memory");
          }
          src += dk;
          dst += 512;
        }
      };
      auto step = [&](int& i, Item& t, int& s) {
        if (++s == t.k1) {
          i += pairs;
          if (i < a.items) {
            t = item_of<WANT_A, kPair>(a, i, rank);
            s = t.k0;
          }
        }
      };
      int i = pair, s = 0;
      Item t = {};
      if (i < a.items) {
        t = item_of<WANT_A, kPair>(a, i, rank);
        s = t.k0;
      }
      int ni = i, ns = s;  // the half stage to copy next
      Item nt = t;
      for (int d = 0; d < kDeep; ++d) {
        if (ni < a.items) {
          copy(nt, ns, d);
          step(ni, nt, ns);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
      while (i < a.items) {
        const int ga = 2 * g + half, slot = ga % kSA;
        asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
        if (lane == 0 && ga >= kSA) ok = wait_or(&aempty[slot], (uint32_t)((ga / kSA - 1) & 1), stop);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) atomicMax(a.status, kErrTimeout);
          break;
        }
        const uint32_t* w = mine + (g % kDeep) * (kWordBytes / 4);
        const int left = a.V - ((WANT_A ? s * 64 + 32 * half : t.m0) + x2);
        uint8_t* st = smem + (g % S::kStagesA) * S::kStageA;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int row = row_of + u * kRows + (WANT_A ? 0 : 32 * half), col = x2 + (WANT_A ? 32 * half : 0);
          const int box = WANT_A ? row >> 6 : col >> 6, y = row & 63, x = col & 63;
          uint32_t v = w[u * 128];
          if (odd) v = (v >> 16) | (w[(16 + u) * 128] << 16);
          if (left < 2) v = left < 1 ? 0u : v & 0xFFFFu;
          *(uint32_t*)(st + box * kBox + y * 128 + (((x >> 3) ^ (y & 7)) << 4) + (x & 7) * 2) = v;
        }
        if (ni < a.items) {
          copy(nt, ns, g % kDeep);
          step(ni, nt, ns);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        step(i, t, s);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[slot]);
        ++g;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
      for (int i = pair; ok && i < a.items; i += pairs) {
        const Item t = item_of<WANT_A, kPair>(a, i, rank);
        for (int s = t.k0; s < t.k1; ++s, ++g) {
          const int ga = 2 * g + half, slot = ga % kSA;
          if (lane == 0) {
            if (S::kTmaRaw) ok = wait_or(&rfull[ga % kRaw], (uint32_t)((ga / kRaw) & 1), stop);
            if (ok && ga >= kSA) ok = wait_or(&aempty[slot], (uint32_t)((ga / kSA - 1) & 1), stop);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) {
            if (lane == 0) atomicMax(a.status, kErrTimeout);
            break;
          }
          float4 r[8];
          if (S::kTmaRaw) {
            const float4* in = (const float4*)(raw + (ga % kRaw) * kRawBytes) + prow * kRowQuads + pq;
#pragma unroll
            for (int u = 0; u < 8; ++u) r[u] = in[u * kRowStep * kRowQuads];
          } else {
            const int row0 = (WANT_A ? t.m0 : s * 64 + 32 * half) + prow;
            const int col = (WANT_A ? s * 64 + 32 * half : t.m0) + 4 * pq, n = a.V - col;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int row = row0 + u * kRowStep;
              r[u] = load_quad((const float*)a.G + (long long)row * a.V + col, row < a.N ? n : 0);
            }
          }
          uint8_t* st = smem + (g % S::kStagesA) * S::kStageA;
          auto split = [&](auto take) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int row = prow + u * kRowStep + (WANT_A ? 0 : 32 * half);
              const int box = WANT_A ? row >> 6 : pq >> 4, y = row & 63, x = WANT_A ? pq + 8 * half : pq & 15;
              const uint32_t at = (uint32_t)(box * kBox + y * 128 + (((x >> 1) ^ (y & 7)) << 4) + (x & 1) * 8);
#pragma unroll
              for (int h = 0; h < S::kParts; ++h) *(uint2*)(st + h * kTileA + at) = take(r[u]);
            }
          };
          float most = abs_max(r[0]);
#pragma unroll
          for (int u = 1; u < 8; ++u) most = fmaxf(most, abs_max(r[u]));
          if (most <= kBf16Most)
            split([](float4& f) { return take_bf16(f); });
          else
            split([](float4& f) { return cut_bf16(f); });
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (S::kTmaRaw) mbar_arrive(&rempty[ga % kRaw]);
            mbar_arrive(&afull[slot]);
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && !*stop.mine) {
    // The MMAs' signals that the last stages have been read are not waited for above, and in a pair come
    // from the other CTA too: they arrive before this block ends, or they would find another's shared
    // memory in its place.  (The phases before each slot's last use were waited for.)
    int g = 0;
    for (int i = pair; i < a.items; i += pairs) {
      const Item t = item_of<WANT_A, kPair>(a, i, rank);
      g += t.k1 - t.k0;
    }
    for (int j = max(0, g - kSB); j < g && mbar_wait(&bempty[j % kSB], (uint32_t)((j / kSB) & 1)); ++j) {}
    g *= S::kHalves;
    for (int j = max(0, g - kSA); j < g && mbar_wait(&aempty[j % kSA], (uint32_t)((j / kSA) & 1)); ++j) {}
  }
  if (kPair) cluster_sync_all();  // the other CTA no longer reads this one's shared memory or arrives here
  if (tid == 0 && *stop.mine) {
    // Given up: the roles have stopped at different stages, and copies and signals of stages that only
    // some of them reached are waited for by none.  They arrive within microseconds.
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < kSettleNs) __nanosleep(1000);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    if (kPair)
      tc::tmem_dealloc_pair(tmem, 512);
    else
      tc::tmem_dealloc(tmem, 512);
  }
  if (kPair) cluster_sync_all();  // neither CTA ends before both have freed
  // grad_a's launch starts on the SMs that grad_W2's has left (neither reads what the other writes) but
  // does not end before it, so that whatever waits for this launch finds both done.
  if (WANT_A) pdl_wait();
}

// grad_a from the shares, in their order: four threads per 16 bytes, each a contiguous quarter.
__global__ void __launch_bounds__(256) share_sum_kernel(long long quads, int splits,
                                                        const float4* __restrict__ part,
                                                        float4* __restrict__ out) {
  __shared__ float4 sh[4][64];
  pdl_wait();
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

// fp32 weights: most blocks of a launch that shares the vocabulary out, and the floats of their results
size_t plain_blocks(int nsm) { return 2 * (size_t)nsm; }
size_t plain_floats(int N, int r, int nsm) {
  const size_t all = plain_blocks(nsm) * N * r, tiles = plain_blocks(nsm) * kFT * kFT;
  return all < tiles ? all : tiles;
}

template <typename TG, typename TW>
cudaError_t plain(int N, int V, int r, const TG* G, const TW* a, const TW* W2, int rv, float* ga, float* gW,
                  int accumulate, float* part, int nsm, cudaStream_t stream) {
  const long long wv = rv ? 1 : r, wj = rv ? V : 1;
  const unsigned nb = (unsigned)((r + kFT - 1) / kFT);
  cudaError_t e = cudaSuccess;
  if (gW) {
    gemm_f32_kernel<TG, TW><<<dim3((unsigned)((V + kFT - 1) / kFT), nb), 256, 0, stream>>>(
        V, r, N, (N + kFK - 1) / kFK * kFK, G, 1, V, a, r, 1, gW, wv, wj, 0, accumulate);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (ga) {
    // shares of at least 64 entries, as many as fill the machine
    const unsigned mb = (unsigned)((N + kFT - 1) / kFT);
    int splits = (int)(plain_blocks(nsm) / ((size_t)mb * nb));
    splits = splits > (V + 63) / 64 ? (V + 63) / 64 : splits < 1 ? 1 : splits;
    const int per = ((V + splits - 1) / splits + kFK - 1) / kFK * kFK;
    splits = (V + per - 1) / per;
    float* out = splits > 1 ? part : ga;
    const dim3 grid(mb, nb, splits);
    if (gW)
      e = launch_pdl(gemm_f32_kernel<TG, TW>, grid, 256, 0, stream, N, r, V, per, G, V, 1, W2, wv, wj, out, r, 1,
                     (long long)N * r, 0);
    else
      gemm_f32_kernel<TG, TW><<<grid, 256, 0, stream>>>(N, r, V, per, G, V, 1, W2, wv, wj, out, r, 1,
                                                        (long long)N * r, 0);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (splits > 1) {
      const long long quads = (long long)N * r / 4;
      e = launch_pdl(share_sum_kernel, (unsigned)((quads + 63) / 64), 256, 0, stream, quads, splits,
                     (const float4*)part, (float4*)ga);
    }
  }
  return e;
}

size_t bg_align(size_t x) { return (x + 255) / 256 * 256; }

// floats of shared-out results at most: kMaxItems work items of 128 x 256 per SM (of 256 x 256 per pair),
// and no more shares than that many work items
size_t share_floats(int N, int r, int nsm) {
  const size_t cap = (size_t)kMaxItems * nsm, all = cap * N * r, tiles = cap * 128 * kBN;
  return all < tiles ? all : tiles;
}

template <bool WANT_A, int MODE>
cudaError_t bg_launch(const BgArgs& a, const CUtensorMap& tg, const CUtensorMap& tb, int nsm, bool behind,
                      cudaStream_t stream) {
  using S = Src<MODE>;
  cudaError_t e = cudaFuncSetAttribute(bias_grad_kernel<WANT_A, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       S::kSmem);
  if (e != cudaSuccess) return e;
  constexpr int kCtas = S::kPair ? 2 : 1;
  const int units = a.items < nsm / kCtas ? a.items : nsm / kCtas;
  if (behind)
    return launch_pdl(bias_grad_kernel<WANT_A, MODE>, kCtas * units, S::kThreads, S::kSmem, stream, a, tg, tb);
  bias_grad_kernel<WANT_A, MODE><<<kCtas * units, S::kThreads, S::kSmem, stream>>>(a, tg, tb);
  return cudaGetLastError();
}
template <bool WANT_A>
cudaError_t bg_mode(int mode, const BgArgs& a, const CUtensorMap& tg, const CUtensorMap& tb, int nsm, bool behind,
                    cudaStream_t stream) {
  switch (mode) {
    case 0: return bg_launch<WANT_A, 0>(a, tg, tb, nsm, behind, stream);
    case 1: return bg_launch<WANT_A, 1>(a, tg, tb, nsm, behind, stream);
    case 2: return bg_launch<WANT_A, 2>(a, tg, tb, nsm, behind, stream);
    default: return bg_launch<WANT_A, 3>(a, tg, tb, nsm, behind, stream);
  }
}

cudaError_t tensor(int N, int V, int r, int g_bf16, const void* G, const bf16* a, const bf16* W2, int rv,
                   float* ga, float* gW, int accumulate, int stuck, uint8_t* ws, int nsm,
                   cudaStream_t stream) {
  const int mode = g_bf16 ? (V % 8 == 0 ? 0 : 3) : (V % 4 == 0 ? 1 : 2);
  const int bm = mode == 0 ? 256 : 128;  // rows of a work item: a pair's or a CTA's
  float* part = (float*)(ws + sizeof(WsHeader));
  BgArgs p;
  p.N = N;
  p.V = V;
  p.r = r;
  p.nrb = (r + kBN - 1) / kBN;
  p.accumulate = accumulate;
  p.out_rv = rv;
  p.stuck = stuck;
  p.G = G;
  p.status = &((WsHeader*)ws)->status;
  p.nmb = p.per_split = p.b_kmajor = 0;
  CUtensorMap tg, tb;
  if (mode == 0 && !encode_bf16_2d(&tg, G, N, V, V, 64)) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  const bf16* W = W2;
  if (ga && rv && V % 8 != 0) {  // rows that TMA cannot address: a [V][r] copy in the workspace
    bf16* t = (bf16*)(ws + sizeof(WsHeader) + bg_align(share_floats(N, r, nsm) * 4));
    if ((e = launch_transpose(W2, t, r, V, 2, stream)) != cudaSuccess) return e;
    W = t;
  }
  if (gW) {
    if (!encode_bf16_2d(&tb, a, N, r, r, 64)) return cudaErrorInvalidValue;
    if (mode == 1 && !encode_f32_2d(&tg, G, N, V, 128, 32)) return cudaErrorInvalidValue;
    if (mode > 1) tg = tb;  // (not used)
    p.items = (V + bm - 1) / bm * p.nrb;
    p.nstage_k = (N + 63) / 64;
    p.out = gW;
    p.wide = ((uintptr_t)gW % 32) == 0;
    if ((e = bg_mode<false>(mode, p, tg, tb, nsm, false, stream)) != cudaSuccess) return e;
  }
  if (ga) {
    p.b_kmajor = rv && W == W2;
    if (!(p.b_kmajor ? encode_bf16_2d(&tb, W, r, V, V, 64) : encode_bf16_2d(&tb, W, V, r, r, 64)))
      return cudaErrorInvalidValue;
    if (mode == 1 && !encode_f32_2d(&tg, G, N, V, 32, 128)) return cudaErrorInvalidValue;
    if (mode > 1) tg = tb;
    p.nmb = (N + bm - 1) / bm;
    p.nstage_k = (V + 63) / 64;
    // Shares of the vocabulary: the rounds of work items times the stages of one, against writing and
    // reading the shares' results (microseconds: a stage of 128 x 64 at the memory's rate per SM)
    const int base = p.nmb * p.nrb, units = mode == 0 ? nsm / 2 : nsm;
    const double stage = (g_bf16 ? 0.38 : 0.75), io = (double)N * r * 8 / 6.7e6;
    int splits = 1;
    double best = 1e300;
    for (int s = 1; s <= p.nstage_k && (long long)base * s <= (long long)kMaxItems * units; ++s) {
      const int per = (p.nstage_k + s - 1) / s;
      const double t = (double)((base * s + units - 1) / units) * per * stage + (s > 1 ? s * io + 2.0 : 0.0);
      if (t < best) {
        best = t;
        splits = s;
      }
    }
    p.per_split = (p.nstage_k + splits - 1) / splits;
    splits = (p.nstage_k + p.per_split - 1) / p.per_split;
    p.items = base * splits;
    p.out = splits > 1 ? part : ga;
    p.wide = ((uintptr_t)p.out % 32) == 0;
    if ((e = bg_mode<true>(mode, p, tg, tb, nsm, gW != nullptr, stream)) != cudaSuccess) return e;
    if (splits > 1) {
      const long long quads = (long long)N * r / 4;
      e = launch_pdl(share_sum_kernel, (unsigned)((quads + 63) / 64), 256, 0, stream, quads, splits,
                     (const float4*)part, (float4*)ga);
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
  o += w_bf16 ? bg_align(share_floats(N, r, nsm) * 4) + (V % 8 ? (size_t)V * r * 2 : 0)
              : plain_floats(N, r, nsm) * 4;
  return o;
}

cudaError_t launch_bias_grad(int N, int V, int r, int g_bf16, const void* G, int w_bf16, const void* a,
                             const void* W2, int w2_rv, float* grad_a, float* grad_W2, int accumulate,
                             int stuck, void* workspace, int nsm, cudaStream_t stream) {
  if (N == 0) {  // no rows: grad_a is empty and grad_W2 zero
    if (!grad_W2 || accumulate) return cudaSuccess;
    zero_kernel<<<4 * nsm, 256, 0, stream>>>((long long)V * r / 4, (float4*)grad_W2);
    return cudaGetLastError();
  }
  if (w_bf16)
    return tensor(N, V, r, g_bf16, G, (const bf16*)a, (const bf16*)W2, w2_rv, grad_a, grad_W2, accumulate,
                  stuck, (uint8_t*)workspace, nsm, stream);
  float* part = (float*)((uint8_t*)workspace + sizeof(WsHeader));
  if (g_bf16)
    return plain(N, V, r, (const bf16*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, part,
                 nsm, stream);
  return plain(N, V, r, (const float*)G, (const float*)a, (const float*)W2, w2_rv, grad_a, grad_W2, accumulate, part,
               nsm, stream);
}

}  // namespace dspark
