// process.cu -- what a request asks of its logits: penalties for the tokens that its text holds, biases
// and a grammar's mask; and the gradient with respect to the raw logits.
//
// Row (b, k) is position k of request b's block; its text is the request's history and the k tokens drafted
// before it.  With c = how often the text's generated part holds v, and seen = whether the text does:
//   y = z / rho if z > 0 else z rho, where seen;  y -= f c + p [c > 0];  y += the biases of v;
//   -inf where the mask's bit of v is clear.
//   dL/dz = dL/dy (1 / rho if z > 0 else rho, where seen), 0 where masked.
//
// A block takes a slice of the vocabulary for all rows of a request.  Its warps count the text's tokens of the slice in
// shared memory (each block reads the whole text, from L2; nothing waits for an atomic's answer) and set a bit for
// each entry that the text or a bias touches.  Then they copy units of 64 bytes per lane, masked, in 16- and 32-byte
// pieces; entries that a mask rules out are not read.  A warp lists its unit's touched entries, and a lane takes one
// of them, whose line is still in the L1: the entries that no text touches cost a copy.  (Patching them in the lane
// that copies them, where a warp waits for each other's branches, took 3 times as long.)  The gradient writes its
// touched entries after the whole slice, in (entry, row) pairs, since they also wait for the raw logits.
//
// HBM bounds the copy: 64 x 8 x 151936 bf16 rows to fp32 take 77 us (6.1 TB/s) without a text, and 85 with texts of
// 4096 tokens on average (5.5 TB/s): the counting, the lists and the entries written twice are instructions (50 % of
// the issue slots) and latency.  512 x 151936 fp32 rows, three quarters of them masked, 113 us (4.5 TB/s); without
// text and mask 96 (6.5 TB/s).  Roles for warps in resident blocks (some copy, some count ahead) reached 97 and 139.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

#include <type_traits>

namespace dspark {
namespace {

constexpr int kThr = 256;                  // threads of a block
// Blocks per SM and entries of a slice: a block's life is a chain of latencies (the request's numbers, its text, the
// logits, the touched ones), which the other blocks' copies and a larger slice hide; slices much larger leave few
// blocks, and five blocks leave a thread too few registers to copy and list.  512 x 1 rows: 128 us with slices of
// 8192, 117 with 16384; 64 x 8 rows: 98 with 4096, 93 with 8192, 114 with 12288, 151 with five blocks.  The gradient,
// 512 x 7 rows of 262144 bf16: 690 us with four blocks, 631 with five, 727 with six.
constexpr int kBlocks = 4, kBlocksGrad = 5;
constexpr int kSlice = 8192, kSliceOne = 16384;   // with several rows, with one
// Where a text may have this many tokens for each entry that a block copies, its blocks have more threads and larger
// slices, which read it fewer times (8 requests of 262144 bf16 with texts of up to 131072: 25 us, with small blocks 51).
constexpr int kLong = 3, kThrLong = 1024, kSliceLong = 16384;
constexpr int kLeast = 512;                // slices are multiples of this
constexpr int kRound = 8192;               // what a block takes besides its copies, in entries
constexpr int kChunk = 256;                // entries that a warp looks through for touched ones, in the gradient
constexpr int kListed = 128;               // touched entries of a unit that a warp lists at a time
constexpr int kMaxRows = 32;               // rows of a block at most
struct PrArgs {
  int R, V, S, nslice, H, nb, M;
  long long in_ld, out_ld, raw_ld, history_ld, mask_ld;
  const int32_t *history, *lengths, *prompts, *drafted;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_tokens;
  const float* bias;
  const uint32_t* mask;
  const int32_t* mask_rows;
};

// Eight entries of a row as they lie in memory: four words of bf16 or eight of fp32.
template <typename T>
struct Raw {
  static constexpr int N = sizeof(T) * 2;
  uint32_t w[N];
};

__device__ __forceinline__ void ld32(uint32_t* w, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void ld16(uint32_t* w, const void* p) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p)
               : "memory");
}
// Eight entries, if `on`, from a boundary of their size.  (A predicate: the loads of a unit are on their way together.)
__device__ __forceinline__ void load8_if(Raw<float>& x, const float* p, bool on) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %9, 0;\n"
               "@q ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n}"
               : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]),
                 "=r"(x.w[7])
               : "l"(p), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void load8_if(Raw<__nv_bfloat16>& x, const __nv_bfloat16* p, bool on) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %5, 0;\n@q ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n}"
               : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3])
               : "l"(p), "r"((uint32_t)on)
               : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Raw<__nv_bfloat16>& x) {
  __stcs((uint4*)p, make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]));
}
__device__ __forceinline__ void store8(float* p, const Raw<float>& x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x.w[0]), "r"(x.w[1]),
               "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7])
               : "memory");
}

// Eight entries from any address: from the 16-byte pieces that hold them, `off` entries into the first
// (off = 0: the pieces are the entries).  The pieces lie inside the row.
__device__ __forceinline__ Raw<__nv_bfloat16> load8(const __nv_bfloat16* p, int off) {
  Raw<__nv_bfloat16> x;
  if (off == 0) {
    ld16(x.w, p);
    return x;
  }
  uint32_t w[8];
  ld16(w, p - off);
  ld16(w + 4, p - off + 8);
  const int words = off >> 1;
#pragma unroll
  for (int i = 0; i < 7; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) x.w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (off & 1));
  return x;
}
__device__ __forceinline__ Raw<float> load8(const float* p, int off) {
  Raw<float> x;
  if (off == 0) {
    if (((uintptr_t)p & 31) == 0) {
      ld32(x.w, p);
    } else {
      ld16(x.w, p);
      ld16(x.w + 4, p + 4);
    }
    return x;
  }
  uint32_t w[12];
#pragma unroll
  for (int i = 0; i < 3; ++i) ld16(w + 4 * i, p - off + 4 * i);
#pragma unroll
  for (int i = 0; i < 11; ++i) w[i] = off & 1 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 8; ++i) x.w[i] = off & 2 ? w[i + 2] : w[i];
  return x;
}
// entries past the eight that load8's pieces hold
template <typename T>
__device__ __forceinline__ int beyond(int off) {
  return off == 0 ? 0 : sizeof(T) == 2 ? 8 - off : 4 - off;
}

__device__ __forceinline__ void convert8(Raw<float>& o, const Raw<float>& x) { o = x; }
__device__ __forceinline__ void convert8(Raw<__nv_bfloat16>& o, const Raw<__nv_bfloat16>& x) { o = x; }
__device__ __forceinline__ void convert8(Raw<float>& o, const Raw<__nv_bfloat16>& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.w[2 * i] = x.w[i] << 16;
    o.w[2 * i + 1] = x.w[i] & 0xFFFF0000u;
  }
}
__device__ __forceinline__ void convert8(Raw<__nv_bfloat16>& o, const Raw<float>& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1]));
    memcpy(&o.w[i], &b, 4);
  }
}
// `fill` (of the output's type, in every half of a word of bf16) where the bit is clear
__device__ __forceinline__ void mask8(Raw<float>& o, uint32_t bits, uint32_t fill) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o.w[i] = (bits >> i) & 1u ? o.w[i] : fill;
}
__device__ __forceinline__ void mask8(Raw<__nv_bfloat16>& o, uint32_t bits, uint32_t fill) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t keep = ((bits >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((bits >> (2 * i)) & 2u ? 0xFFFF0000u : 0u);
    o.w[i] = (o.w[i] & keep) | (fill & ~keep);
  }
}

__device__ __forceinline__ bool allowed(const uint32_t* mask, int v) {
  return !mask || ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u);
}
// the mask's bits of entries v .. v + 7, all inside the vocabulary
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int v) {
  const int w = v >> 5, sh = v & 31;
  const uint32_t lo = __ldg(mask + w), hi = sh > 24 ? __ldg(mask + w + 1) : 0u;
  return __funnelshift_r(lo, hi, sh) & 0xFFu;
}

// What the tools of a request make of one raw logit (or of its gradient).
template <bool GRAD>
__device__ __forceinline__ float one_entry(float x, float raw, bool seen, int c, float rho, float pres, float freq,
                                           bool biased, float bias) {
  // (divided, not multiplied by a rounded 1 / rho: what the formula says, to half a step)
  float y = seen ? (raw > 0.f ? __fdiv_rn(x, rho) : x * rho) : x;
  if (GRAD) return y;
  if (c > 0) y = y - freq * (float)c - pres;
  return biased ? y + bias : y;
}

// How often a text generates each token is counted in 16 bits where no text is longer than that, else in 32; the
// gradient needs no counts.  (What shared memory the blocks of an SM take is missing in its L1, where the loads on
// their way have their places: with 205 KB of it taken a copy of 77 us took 97.)
enum Count { kNoCount, kCount16, kCount32 };

// A block's slice [s0, s0 + n) of the vocabulary, in shared memory.
template <int COUNT>
struct Slice {
  uint32_t* touched;  // [S / 32] bits: what a text touches
  uint32_t* text;     // [S / 32] tokens of the prompt (without counts: of the history)
  uint32_t* drafted;  // [S / 32] tokens that are drafted
  uint32_t* biased;   // [S / 32]
  uint32_t* count;    // [S / 2] or [S]
  uint16_t* before;   // [S / 32] 1 + the place in `bias` of the first of a word's biased tokens
  float* bias;        // [nb] their sums
  int s0, n;
  static constexpr int kPer32 = 4 * 4 + (COUNT == kCount16 ? 64 : COUNT == kCount32 ? 128 : 0);   // bytes for 32 entries
  __device__ __forceinline__ Slice(uint8_t* smem, int S, int nb, int V, int slice) {
    const int words = S / 32;
    touched = (uint32_t*)smem;
    text = touched + words;
    drafted = text + words;
    biased = drafted + words;
    count = biased + words;
    before = (uint16_t*)(smem + (size_t)words * kPer32);
    bias = (float*)(before + words);
    s0 = slice * S;
    n = min(S, V - s0);
  }
  static __device__ __forceinline__ bool is(const uint32_t* bits, int u) { return (bits[u >> 5] >> (u & 31)) & 1u; }
  // (nothing waits for the old values)
  static __device__ __forceinline__ void set(uint32_t* bits, int u) { atomicOr(&bits[u >> 5], 1u << (u & 31)); }
  __device__ __forceinline__ void add(int u, bool prompt) const {
    if (COUNT == kNoCount || prompt)
      set(text, u);
    else if (COUNT == kCount16)
      atomicAdd(&count[u >> 1], 1u << (16 * (u & 1)));
    else
      atomicAdd(&count[u], 1u);
    set(touched, u);
  }
  __device__ __forceinline__ int place(int u) const {
    return before[u >> 5] - 1 + __popc(biased[u >> 5] & ((1u << (u & 31)) - 1u));
  }
  __device__ __forceinline__ int times(int u) const {
    return COUNT == kNoCount ? 0 : COUNT == kCount16 ? (int)((const uint16_t*)count)[u] : (int)count[u];
  }
};

// Counts a text of L tokens, the first P of them the prompt, by the block's threads.  Returns the largest token + 1 as
// an unsigned number, of this thread's share: above V when a token is outside [-1, V).
template <int COUNT>
__device__ __forceinline__ uint32_t count_text(const Slice<COUNT>& sl, const int32_t* h, int L, int P) {
  uint32_t most = 0u;
  const int tid = (int)threadIdx.x, nthr = (int)blockDim.x;
  auto one = [&](int i, int t) {
    most = max(most, (uint32_t)t + 1u);   // (unsigned: any token is defined)
    const uint32_t u = (uint32_t)t - (uint32_t)sl.s0;
    if (u < (uint32_t)sl.n) sl.add((int)u, i < P);
  };
  const int head = min(L, (int)((16 - ((uintptr_t)h & 15)) & 15) >> 2);   // up to a 16-byte boundary
  const int n4 = (L - head) >> 2;
  if (tid < head) one(tid, __ldg(h + tid));
  for (int i = head + 4 * n4 + tid; i < L; i += nthr) one(i, __ldg(h + i));
  const int4* h4 = (const int4*)(h + head);
  constexpr int kDeep = 4;   // 16-byte loads per thread in flight
  for (int i0 = tid; i0 < n4; i0 += kDeep * nthr) {
    int4 q[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) q[j] = i0 + j * nthr < n4 ? __ldg(h4 + i0 + j * nthr) : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = head + 4 * (i0 + j * nthr);
      one(i, q[j].x);
      one(i + 1, q[j].y);
      one(i + 2, q[j].z);
      one(i + 3, q[j].w);
    }
  }
  return most;
}

// The bits of the slice's biased tokens, by the block's threads; t: entry tid.  in: bits of the entries of the slice.
// Returns the largest token + 1.
template <int COUNT>
__device__ __forceinline__ uint32_t list_biases(const Slice<COUNT>& sl, const int32_t* tokens, int nb, int t,
                                                uint32_t* in) {
  uint32_t most = 0u;
  for (int i = (int)threadIdx.x;;) {
    const uint32_t u = (uint32_t)t - (uint32_t)sl.s0;
    const bool mine = u < (uint32_t)sl.n;
    most = max(most, (uint32_t)t + 1u);
    if (mine) {
      sl.set(sl.biased, (int)u);
      sl.set(sl.touched, (int)u);
    }
    if (i < nb) sl.bias[i] = 0.f;
    const uint32_t some = __ballot_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) in[i >> 5] = some;
    i += (int)blockDim.x;
    if (i - (int)(threadIdx.x & 31) >= nb) return most;
    t = i < nb ? __ldg(tokens + i) : -1;
  }
}

// One warp: their sums.  Step by step of 32 entries, each word of bits that is met gets places for its tokens, and the
// biases are added, those of one token in the list's order: the entries of a token in one step by the first of them.
template <int COUNT>
__device__ __forceinline__ void add_biases(const Slice<COUNT>& sl, const int32_t* tokens, const float* bias, int nb,
                                           const uint32_t* in) {
  const int lane = (int)(threadIdx.x & 31);
  const uint32_t bits = lane * 32 < nb ? in[lane] : 0u;
  int places = 0;
  for (uint32_t steps = __ballot_sync(0xffffffffu, bits != 0u); steps; steps &= steps - 1) {
    const int step = __ffs(steps) - 1, i = step * 32 + lane;
    const bool mine = (__shfl_sync(0xffffffffu, bits, step) >> lane) & 1u;
    const int u = mine ? __ldg(tokens + i) - sl.s0 : -1 - lane;
    const float x = mine ? __ldg(bias + i) : 0.f;
    const uint32_t word = __match_any_sync(0xffffffffu, mine ? u >> 5 : u);
    const bool opens = mine && lane == __ffs(word) - 1 && sl.before[u >> 5] == 0;
    const int n = opens ? __popc(sl.biased[u >> 5]) : 0;
    int at = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += y;
    }
    if (opens) sl.before[u >> 5] = (uint16_t)(places + at - n + 1);
    places += __shfl_sync(0xffffffffu, at, 31);
    __syncwarp();
    const uint32_t peers = __match_any_sync(0xffffffffu, u);
    const bool first = mine && lane == __ffs(peers) - 1;
    float sum = first ? sl.bias[sl.place(u)] + x : 0.f;
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine && !first); todo; todo &= todo - 1) {
      const int j = __ffs(todo) - 1;
      const float y = __shfl_sync(0xffffffffu, x, j);
      if ((peers >> j) & 1u) sum += y;
    }
    if (first) sl.bias[sl.place(u)] = sum;
    __syncwarp();
  }
}

// TI: the input's type; TO: the output's; GRAD: the input is dL/dy and the raw logits have the output's type.
// units: what a warp copies at a time (64 bytes per lane of one row), per row of the slice.  A warp counts its
// share of the text, then takes units until none is left.
template <typename TI, typename TO, bool GRAD, int COUNT, int THR>
__global__ void __launch_bounds__(THR, THR != kThr ? 1 : GRAD ? kBlocksGrad : kBlocks)
    process_kernel(const TI* in, TO* out, const TO* raw, const PrArgs a, const int units, const bool same) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_next, s_bad;
  __shared__ uint32_t s_in[32];      // which biases are of the slice's tokens (nb <= 1024)
  __shared__ uint64_t s_counted;
  __shared__ int s_drafted[kMaxRows];
  __shared__ uint16_t s_list[THR / 32][GRAD ? kChunk / 2 : kListed];
  __shared__ int s_mask[kMaxRows];   // the rows' masks (-1: none, -2: not a row of the mask)
  const int b = (int)(blockIdx.x / (unsigned)a.nslice);
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Slice<COUNT> sl(smem, a.S, a.nb, a.V, (int)(blockIdx.x % (unsigned)a.nslice));
  const int s0 = sl.s0, s1 = sl.s0 + sl.n;
  const float rho = a.repetition ? __ldg(a.repetition + b) : 1.f;
  const float pres = !GRAD && a.presence ? __ldg(a.presence + b) : 0.f;
  const float freq = !GRAD && a.frequency ? __ldg(a.frequency + b) : 0.f;
  const int L = a.lengths ? __ldg(a.lengths + b) : a.H, P = a.prompts ? __ldg(a.prompts + b) : 0;
  if (tid < a.R) {
    const long long row = (long long)b * a.R + tid;
    const int m = !a.mask ? -1 : a.mask_rows ? __ldg(a.mask_rows + row) : (int)row;
    s_mask[tid] = m < -1 || (m >= a.M && a.mask) ? -2 : m;
    s_drafted[tid] = a.drafted && tid < a.R - 1 ? __ldg(a.drafted + (long long)b * (a.R - 1) + tid) : -1;
  }
  const bool biased = !GRAD && a.nb > 0;
  const int32_t* bias_tokens = biased ? a.bias_tokens + (long long)b * a.nb : nullptr;
  const int t0 = biased && tid < a.nb ? __ldg(bias_tokens + tid) : -1;
  for (int i = tid; i < a.S / 32 * (sl.kPer32 / 16) + (biased ? a.S / 256 : 0); i += THR)
    ((uint4*)smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) {
    s_next = s_bad = 0;
    mbar_init(&s_counted, THR / 32);
    fence_mbar_init();
  }
  const bool penalised = rho != 1.f || pres != 0.f || freq != 0.f, any = penalised || biased;
  __syncthreads();

  uint32_t most = 0u;   // the largest token + 1
  if (biased) {
    most = list_biases(sl, bias_tokens, a.nb, t0, s_in);
    __syncthreads();
  }
  if (any) {
    if (biased && warp == 0) add_biases(sl, bias_tokens, a.bias + (long long)b * a.nb, a.nb, s_in);
    if (penalised) {
      if (L < 0 || L > a.H || P < 0 || P > L)
        most = 0xFFFFFFFFu;
      else
        most = max(most, count_text(sl, a.history + (long long)b * a.history_ld, L, P));
      if (tid < a.R - 1) {   // (R <= 32: the first warp)
        const uint32_t t = (uint32_t)s_drafted[tid], u = t - (uint32_t)s0;
        most = max(most, t + 1u);
        if (u < (uint32_t)sl.n) {
          sl.set(sl.drafted, (int)u);
          sl.set(sl.touched, (int)u);
        }
      }
    }
  }

  if (!GRAD && any) {
    if (most > (uint32_t)a.V) s_bad = 1;
    __syncwarp();
    if (lane == 0) mbar_arrive(&s_counted);
  }

  // the copy, masked
  bool counted = false, wrong = false;
  using W = typename std::conditional<sizeof(TO) == 2, uint16_t, uint32_t>::type;
  const uint32_t fill = GRAD ? 0u : sizeof(TO) == 2 ? 0xFF80FF80u : 0xFF800000u;
  const uint32_t nan = sizeof(TO) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
  constexpr int kDepth = 64 / (int)sizeof(Raw<TI>), A = 8 * sizeof(TO);
  for (;;) {
    int unit = 0;
    if (lane == 0) unit = atomicAdd(&s_next, 1);
    unit = __shfl_sync(0xffffffffu, unit, 0);
    const int r = unit / units;
    if (r >= a.R) break;
    const int m = s_mask[r];
    if (same && m == -1 && (GRAD || !any)) continue;
    const long long row = (long long)b * a.R + r;
    const TI* z = in + row * a.in_ld;
    TO* o = out + row * a.out_ld;
    const uint32_t* mask = m >= 0 ? a.mask + (long long)m * a.mask_ld : nullptr;
    // groups of eight entries on the output's boundaries; those that reach out of the slice by entries
    const int head = (int)(((uintptr_t)o & (A - 1)) / sizeof(TO));
    const int off = (int)(((uintptr_t)(z - head) & 15) / sizeof(TI));
    const int lo = max(s0, off), hi = min(s1, a.V - beyond<TI>(off));   // whole groups are inside these
    const int v00 = ((s0 + head) >> 3) * 8 - head + ((unit - r * units) * (32 * kDepth) + lane) * 8;
    Raw<TI> x[kDepth];
    uint32_t bits[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int v0 = v00 + i * 256;
      bits[i] = m != -2 && v0 >= lo && v0 + 8 <= hi ? 0xFFu : 0u;
      if (mask && bits[i]) bits[i] = mask_bits(mask, v0);
    }
    // (entries that the mask rules out are not needed)
    if (((uintptr_t)(z + v00) & (sizeof(Raw<TI>) - 1)) == 0) {
#pragma unroll
      for (int i = 0; i < kDepth; ++i) load8_if(x[i], z + v00 + i * 256, bits[i] && !(same && bits[i] == 0xFFu));
    } else {
#pragma unroll
      for (int i = 0; i < kDepth; ++i)
        if (bits[i] && !(same && bits[i] == 0xFFu)) x[i] = load8(z + v00 + i * 256, off);
    }
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int v0 = v00 + i * 256;
      if (v0 >= lo && v0 + 8 <= hi) {
        if (same && bits[i] == 0xFFu) continue;
        Raw<TO> y;
        convert8(y, x[i]);
        if (mask || m == -2) mask8(y, bits[i], m == -2 ? nan : fill);
        store8(o + v0, y);
      } else {
#pragma unroll 1
        for (int v = max(v0, s0); v < min(v0 + 8, s1); ++v) {
          if (m == -2 || !allowed(mask, v))
            ((W*)o)[v] = (W)(m == -2 ? nan : fill);
          else if (std::is_same<TI, TO>::value && !same)
            ((W*)o)[v] = ((const W*)z)[v];   // (bits: through fp32 every bf16 NaN would become one)
          else if (!same)
            o[v] = from_f<TO>(to_f<TI>(z[v]));
        }
      }
    }
    if constexpr (!GRAD) {
      if (!any || m == -2) continue;
      __syncwarp();   // (the warp's stores before those below)
      if (!counted) {
        // (the wait ends: no warp waits before it has arrived; one that ran out would be told by NaN)
        wrong = !mbar_wait_warp(&s_counted, 0u) || s_bad;
        counted = true;
      }
      const int u00 = v00 - lane * 8, va = max(u00, s0), vb = min(u00 + 256 * kDepth, s1);   // the unit's entries
      if (wrong) {
        for (int v = va + lane; v < vb; v += 32) o[v] = from_f<TO>(NAN);
        continue;
      }
      // the unit's touched entries, kListed at a time: 32 entries' bits per lane make a list, a lane takes one of it
      uint16_t* list = s_list[warp];
      for (int w0 = (va - s0) >> 5; w0 * 32 < vb - s0; w0 += 32) {
        const int e0 = (w0 + lane) * 32 + s0;   // the lane's first entry
        uint32_t t = e0 < vb ? sl.touched[w0 + lane] : 0u;
        if (e0 < va) t &= 0xFFFFFFFFu << (va - e0);
        if (t && vb - e0 < 32) t &= (1u << (vb - e0)) - 1u;
        if (mask && t) t &= __ldg(mask + (e0 >> 5));   // (slices begin at whole words)
        if (!__any_sync(0xffffffffu, t != 0u)) continue;
        const int mine = __popc(t);
        int at = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, at, d);
          if (lane >= d) at += y;
        }
        const int all = __shfl_sync(0xffffffffu, at, 31);
        at -= mine;
        for (int base = 0; base < all; base += kListed) {
          int k = at - base;
          for (uint32_t bits = t; bits; bits &= bits - 1u, ++k)
            if ((unsigned)k < (unsigned)kListed) list[k] = (uint16_t)(e0 - s0 + __ffs(bits) - 1);
          __syncwarp();
#pragma unroll 1
          for (int i = lane; i < min(all - base, kListed); i += 32) {
            const int u = list[i], v = s0 + u;
            const float f = to_f<TI>(z[v]);
            int n = sl.times(u);
            bool seen = n > 0 || sl.is(sl.text, u);
            if (r > 0 && sl.is(sl.drafted, u))
              for (int d = 0; d < r; ++d)
                if (s_drafted[d] == v) {
                  ++n;
                  seen = true;
                }
            const bool has = biased && sl.is(sl.biased, u);
            if (seen || has)
              o[v] = from_f<TO>(one_entry<GRAD>(f, f, seen, n, rho, pres, freq, has, has ? sl.bias[sl.place(u)] : 0.f));
          }
          __syncwarp();
        }
      }
    }
  }
  if constexpr (GRAD) {
    const bool bad = __syncthreads_or(most > (uint32_t)a.V);
    if (bad) {
      for (int r = 0; r < a.R; ++r)
        for (int v = s0 + tid; v < s1; v += THR) out[((long long)b * a.R + r) * a.out_ld + v] = from_f<TO>(NAN);
      return;
    }
    if (!any) return;
    // a warp lists the touched entries of kChunk, then takes them in (entry, row) pairs, kDeep per lane
    constexpr int kDeep = 4;
    uint8_t* list = (uint8_t*)s_list[warp];
    for (int c = warp; c * kChunk < sl.n; c += THR / 32) {
      uint32_t w = ((const uint8_t*)sl.touched)[c * 32 + lane];
      int all = __popc(w), at = all;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += y;
      }
      at -= all;
      all = __shfl_sync(0xffffffffu, at + all, 31);
      for (; w; w &= w - 1) list[at++] = (uint8_t)(lane * 8 + __ffs(w) - 1);
      __syncwarp();
      const int pairs = all * a.R;
      for (int i0 = lane; i0 - lane < pairs; i0 += 32 * kDeep) {
        float f[kDeep], g[kDeep];
        long long to[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
          const int i = i0 + j * 32, slot = i / a.R, r = i - slot * a.R;
          to[j] = -1;
          if (i >= pairs) continue;
          const int u = c * kChunk + list[slot], v = s0 + u, m = s_mask[r];
          bool seen = sl.is(sl.text, u);
          for (int d = 0; d < r && !seen; ++d) seen = s_drafted[d] == v;
          if (!seen || m == -2 || !allowed(m >= 0 ? a.mask + (long long)m * a.mask_ld : nullptr, v)) continue;
          const long long row = (long long)b * a.R + r;
          f[j] = to_f<TI>(in[row * a.in_ld + v]);
          g[j] = to_f<TO>(raw[row * a.raw_ld + v]);
          to[j] = row * a.out_ld + v;
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j)
          if (to[j] >= 0) out[to[j]] = from_f<TO>(one_entry<GRAD>(f[j], g[j], true, 0, rho, 0.f, 0.f, false, 0.f));
      }
      __syncwarp();
    }
  }
}

// Slices of at most S entries, smaller ones where that gives every SM its blocks.
int slice_of(int B, int V, int S, int blocks) {
  const long long even = ((long long)B * V + blocks - 1) / blocks;
  return even < S ? (int)((even + kLeast - 1) / kLeast) * kLeast : S;
}

// Up to twice as many slices where the blocks then fill what the device holds of them at a time more evenly: a round of
// blocks counted as its copies and as much again as kRound entries' (the gradient of 77 x 7 x 50021: 51 us, then 45; 72 x 8 x
// 68171: 75 and 66).
int even_slice(int B, int V, int S, int resident) {
  const int least = (V + S - 1) / S;
  long long best = 0;
  int chosen = S;
  for (int n = least, step = (least + 15) / 16; n <= 2 * least; n += step) {   // (17 tries at most)
    const int each = ((V + n - 1) / n + kLeast - 1) / kLeast * kLeast;
    const long long cost = ((long long)B * n + resident - 1) / resident * (each + kRound);
    if (best == 0 || cost < best) {
      best = cost;
      chosen = each;
    }
    if (each == kLeast) break;
  }
  return chosen;
}

template <typename TI, typename TO, bool GRAD, int COUNT, int THR>
cudaError_t launch(int B, const TI* in, TO* out, const TO* raw, PrArgs a, int S, cudaStream_t stream) {
  a.S = S;
  a.nslice = (a.V + S - 1) / S;
  constexpr int unit = 32 * (64 / (int)sizeof(Raw<TI>));   // groups
  const bool al = ((uintptr_t)out % (8 * sizeof(TO))) == 0 && (a.out_ld * sizeof(TO)) % (8 * sizeof(TO)) == 0;
  const int units = (S / 8 + (al ? 0 : 1) + unit - 1) / unit;
  const size_t smem = (size_t)S / 32 * Slice<COUNT>::kPer32 + (a.nb > 0 ? (size_t)a.nb * 4 + S / 16 : 0);
  auto kernel = process_kernel<TI, TO, GRAD, COUNT, THR>;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)B * (unsigned)a.nslice, THR, smem, stream>>>(in, out, raw, a, units,
                                                                  (const void*)in == (const void*)out);
  return cudaGetLastError();
}

template <typename TI, typename TO, bool GRAD, int COUNT>
cudaError_t run_count(int B, const TI* in, TO* out, const TO* raw, const PrArgs& a, int nsm, cudaStream_t stream) {
  const int S = slice_of(B, a.V, !GRAD && a.R == 1 ? kSliceOne : kSlice, 2 * nsm);
  if (a.H / a.R >= kLong * (long long)(S < a.V ? S : a.V))
    return launch<TI, TO, GRAD, COUNT, kThrLong>(B, in, out, raw, a, slice_of(B, a.V, kSliceLong, nsm), stream);
  return launch<TI, TO, GRAD, COUNT, kThr>(B, in, out, raw, a,
                                           even_slice(B, a.V, S, nsm * (GRAD ? kBlocksGrad : kBlocks)), stream);
}

template <typename TI, typename TO, bool GRAD>
cudaError_t run(int B, const TI* in, TO* out, const TO* raw, PrArgs a, int nsm, cudaStream_t stream) {
  if constexpr (GRAD) {
    a.nb = 0;
    return run_count<TI, TO, GRAD, kNoCount>(B, in, out, raw, a, nsm, stream);
  } else {
    return a.H + a.R <= 65535 ? run_count<TI, TO, GRAD, kCount16>(B, in, out, raw, a, nsm, stream)
                              : run_count<TI, TO, GRAD, kCount32>(B, in, out, raw, a, nsm, stream);
  }
}

template <bool GRAD>
cudaError_t run_types(int B, int i_bf16, const void* in, int o_bf16, void* out, const void* raw, const PrArgs& a,
                      int nsm, cudaStream_t stream) {
  using H = __nv_bfloat16;
  if (i_bf16)
    return o_bf16 ? run<H, H, GRAD>(B, (const H*)in, (H*)out, (const H*)raw, a, nsm, stream)
                  : run<H, float, GRAD>(B, (const H*)in, (float*)out, (const float*)raw, a, nsm, stream);
  return o_bf16 ? run<float, H, GRAD>(B, (const float*)in, (H*)out, (const H*)raw, a, nsm, stream)
                : run<float, float, GRAD>(B, (const float*)in, (float*)out, (const float*)raw, a, nsm, stream);
}

}  // namespace

cudaError_t launch_process(int grad, int B, int R, int V, int i_bf16, const void* in, long long in_ld, int o_bf16,
                           void* out, long long out_ld, const void* raw, long long raw_ld, const int32_t* history,
                           long long history_ld, int H, const int32_t* lengths, const int32_t* prompts,
                           const int32_t* drafted, const float* repetition, const float* presence,
                           const float* frequency, int nb, const int32_t* bias_tokens, const float* bias,
                           const uint32_t* mask, long long mask_ld, int M, const int32_t* mask_rows,
                           int nsm, cudaStream_t stream) {
  PrArgs a;
  a.R = R;
  a.V = V;
  a.S = a.nslice = 0;
  a.H = H;
  a.nb = nb;
  a.M = mask ? M : 0;
  a.in_ld = in_ld;
  a.out_ld = out_ld;
  a.raw_ld = raw_ld;
  a.history_ld = history_ld;
  a.mask_ld = mask_ld;
  a.history = history;
  a.lengths = lengths;
  a.prompts = prompts;
  a.drafted = drafted;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_tokens = bias_tokens;
  a.bias = bias;
  a.mask = mask;
  a.mask_rows = mask_rows;
  return grad ? run_types<true>(B, i_bf16, in, o_bf16, out, raw, a, nsm, stream)
              : run_types<false>(B, i_bf16, in, o_bf16, out, raw, a, nsm, stream);
}

}  // namespace dspark
