// process.cu -- what a request asks of its logits: penalties for the tokens that its text holds, biases
// and a grammar's mask; and the gradient with respect to the raw logits.
//
// Row (b, k) is position k of request b's block; its text is the request's history and the k tokens drafted
// before it.  With c = how often the text's generated part holds v, and seen = whether the text does:
//   y = z / rho if z > 0 else z rho, where seen;  y -= f c + p [c > 0];  y += the biases of v;
//   -inf where the mask's bit of v is clear.
//   dL/dz = dL/dy (1 / rho if z > 0 else rho, where seen), 0 where masked.
//
// A block takes a slice of the vocabulary for all rows of a request.  It counts the text's tokens of its slice in
// shared memory (each block reads the whole text, from L2; nothing waits for an atomic's answer), copies its
// entries of every row, masked, in 16- and 32-byte pieces, and then writes the touched entries again: a bit for
// each entry says which, warps list those bits, and a lane takes an (entry, row) pair, so that the entries that no
// text and no bias touches cost a copy.  Patching them in the copying lanes instead, where a warp waits for each
// other's branches, took 2 to 3 times as long (64 x 8 x 151936: 268 us against 97).
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

#include <type_traits>

namespace dspark {
namespace {

constexpr int kThr = 256, kBlocks = 5;     // threads of a block, blocks per SM
constexpr int kSlice = 4096;               // entries of a block's slice, with several rows
constexpr int kSliceOne = 8192;            // with one
constexpr int kLong = 24576, kThrLong = 1024, kSliceLong = 16384;   // texts of this many tokens per row
constexpr int kChunk = 512;                // entries that a warp looks through for touched ones; slices are multiples
constexpr int kMostBias = 1024;
constexpr int kMostSmem = kSliceLong * 4 + kSliceLong / 8 + kMostBias * 6;
constexpr int kMaxRows = 32;               // rows of a block at most
constexpr uint32_t kSeen = 1u << 31;       // the prompt holds the token
constexpr uint32_t kDrafted = 1u << 30;    // one of the drafted tokens
constexpr uint32_t kBiased = 1u << 29;
constexpr uint32_t kCount = kBiased - 1u;  // how often the generated part of the history holds it

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

// A block's slice [s0, s0 + n) of the vocabulary, in shared memory: how often the text holds each token, and
// the bits of those that a text or a bias touches.
struct Slice {
  uint32_t* count;    // [S]
  uint32_t* touched;  // [S / 32]
  float* bias;        // [nb] the sums of the slice's biased tokens
  uint16_t* bias_u;   // [nb] those tokens, each once
  int s0, n;
  // (nothing waits for the old values; a flag stays once set, and a count cannot reach it)
  __device__ __forceinline__ void add(int u, uint32_t flag) const {
    if (flag)
      atomicOr(&count[u], flag);
    else
      atomicAdd(&count[u], 1u);
    atomicOr(&touched[u >> 5], 1u << (u & 31));
  }
};

// Counts a text of L tokens, the first P of them the prompt, by the block's threads.  Returns the largest token + 1 as
// an unsigned number, of this thread's share: above V when a token is outside [-1, V).
__device__ __forceinline__ uint32_t count_text(const Slice& sl, const int32_t* h, int L, int P) {
  uint32_t most = 0u;
  const int tid = (int)threadIdx.x, nthr = (int)blockDim.x;
  auto one = [&](int i, int t) {
    most = max(most, (uint32_t)(t + 1));
    const int u = t - sl.s0;
    if ((unsigned)u < (unsigned)sl.n) sl.add(u, i < P ? kSeen : 0u);
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

// One warp: the slice's biases, those of one token in the list's order: a step of 32 entries at a time, the
// entries of a token in one step added by the first of them.  n: how many tokens have some.
__device__ __forceinline__ uint32_t add_biases(const Slice& sl, const int32_t* tokens, const float* bias, int nb,
                                               int* n) {
  uint32_t most = 0u;
  const int lane = (int)(threadIdx.x & 31);
  int t = lane < nb ? __ldg(tokens + lane) : -1, have = 0;
  for (int i0 = 0; i0 < nb; i0 += 32) {
    const int i = i0 + lane, next = i + 32 < nb ? __ldg(tokens + i + 32) : -1, u = t - sl.s0;
    most = max(most, (uint32_t)(t + 1));
    const bool mine = (unsigned)u < (unsigned)sl.n;
    t = next;
    uint32_t todo = __ballot_sync(0xffffffffu, mine);
    if (!todo) continue;
    const float x = mine ? __ldg(bias + i) : 0.f;
    const uint32_t peers = __match_any_sync(0xffffffffu, mine ? u : -1 - lane);
    const bool first = mine && lane == __ffs(peers) - 1;
    int slot = -1;   // of an earlier step
    if (first && (sl.count[u] & kBiased))
      for (slot = 0; sl.bias_u[slot] != u;) ++slot;
    float sum = slot >= 0 ? sl.bias[slot] : 0.f;
    for (; todo; todo &= todo - 1) {
      const int j = __ffs(todo) - 1;
      const float y = __shfl_sync(0xffffffffu, x, j);
      if ((peers >> j) & 1u) sum += y;
    }
    const uint32_t fresh = __ballot_sync(0xffffffffu, first && slot < 0);
    if (first && slot < 0) {
      slot = have + __popc(fresh & ((1u << lane) - 1u));
      sl.bias_u[slot] = (uint16_t)u;
      atomicOr(&sl.count[u], kBiased);
    }
    if (first) sl.bias[slot] = sum;
    have += __popc(fresh);
    __syncwarp();
  }
  if (lane == 0) *n = have;
  return most;
}

// TI: the input's type; TO: the output's; GRAD: the input is dL/dy and the raw logits have the output's type.
// units: what a warp copies at a time (64 bytes per lane of one row), per row of the slice.  A warp counts its
// share of the text, then takes units until none is left.
template <typename TI, typename TO, bool GRAD, int THR>
__global__ void __launch_bounds__(THR, THR == kThr ? kBlocks : 1)
    process_kernel(const TI* in, TO* out, const TO* raw, const PrArgs a, const int units, const bool same) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_next, s_biased;
  __shared__ int s_drafted[kMaxRows];
  __shared__ uint16_t s_list[THR / 32][kChunk];
  __shared__ int s_mask[kMaxRows];   // the rows' masks (-1: none, -2: not a row of the mask)
  const int b = (int)(blockIdx.x / (unsigned)a.nslice);
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Slice sl;
  sl.count = (uint32_t*)smem;
  sl.touched = sl.count + a.S;
  sl.bias = (float*)(sl.touched + a.S / 32);
  sl.bias_u = (uint16_t*)(sl.bias + a.nb);
  sl.s0 = (int)(blockIdx.x % (unsigned)a.nslice) * a.S;
  sl.n = min(a.S, a.V - sl.s0);
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
  for (int i = tid; i < (a.S + a.S / 32) / 4; i += THR) ((uint4*)smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) s_next = s_biased = 0;
  const bool penalised = rho != 1.f || pres != 0.f || freq != 0.f, any = penalised || biased;
  __syncthreads();

  uint32_t most = 0u;   // the largest token + 1
  if (any) {
    if (biased && warp == 0) most = add_biases(sl, a.bias_tokens + (long long)b * a.nb, a.bias + (long long)b * a.nb, a.nb,
                                                &s_biased);
    if (penalised) {
      if (L < 0 || L > a.H || P < 0 || P > L)
        most = 0xFFFFFFFFu;
      else
        most = max(most, count_text(sl, a.history + (long long)b * a.history_ld, L, P));
      if (tid < a.R - 1) {   // (R <= 32: the first warp)
        const int t = s_drafted[tid], u = t - s0;
        most = max(most, (uint32_t)(t + 1));
        if ((unsigned)u < (unsigned)sl.n) sl.add(u, kDrafted);
      }
    }
  }

  // the copy, masked; touched entries are written again below
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
    if (same && m == -1) continue;
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
#pragma unroll
    for (int i = 0; i < kDepth; ++i)   // (entries that the mask rules out are not needed)
      if (bits[i] && !(same && bits[i] == 0xFFu)) x[i] = load8(z + v00 + i * 256, off);
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      const int v0 = v00 + i * 256;
      if (v0 >= lo && v0 + 8 <= hi) {
        if (same && bits[i] == 0xFFu) continue;
        Raw<TO> y;
        convert8(y, x[i]);
        mask8(y, bits[i], m == -2 ? nan : fill);
        store8(o + v0, y);
      } else {
#pragma unroll 1
        for (int v = max(v0, s0); v < min(v0 + 8, s1); ++v) {
          if (m == -2 || !allowed(mask, v))
            ((W*)o)[v] = (W)(m == -2 ? nan : fill);
          else if (!same)
            o[v] = from_f<TO>(to_f<TI>(z[v]));
        }
      }
    }
  }
  const bool bad = __syncthreads_or(most > (uint32_t)a.V);
  if (bad) {
    for (int r = 0; r < a.R; ++r)
      for (int v = s0 + tid; v < s1; v += THR) out[((long long)b * a.R + r) * a.out_ld + v] = from_f<TO>(NAN);
    return;
  }
  if (!any) return;

  // kDeep touched entries per lane, in rows r (v < 0: none): their logits are fetched, then written anew
  constexpr int kDeep = 4;
  auto again = [&](const int (&v)[kDeep], const int (&r)[kDeep], const float (&bias)[kDeep], bool mine) {
    float f[kDeep], g[kDeep];
    bool on[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      on[j] = false;
      if (v[j] < 0) continue;
      const int m = s_mask[r[j]];
      if (m == -2 || !allowed(m >= 0 ? a.mask + (long long)m * a.mask_ld : nullptr, v[j])) continue;
      const long long row = (long long)b * a.R + r[j];
      f[j] = to_f<TI>(in[row * a.in_ld + v[j]]);
      g[j] = GRAD ? to_f<TO>(raw[row * a.raw_ld + v[j]]) : f[j];
      on[j] = true;
    }
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      if (!on[j]) continue;
      const uint32_t w = sl.count[v[j] - s0];
      int n = (int)(w & kCount);
      bool seen = (w & (kSeen | kCount)) != 0u;
      if (w & kDrafted)
        for (int d = 0; d < r[j]; ++d)
          if (s_drafted[d] == v[j]) {
            ++n;
            seen = true;
          }
      if ((seen || mine) && mine == ((w & kBiased) != 0u))
        out[((long long)b * a.R + r[j]) * a.out_ld + v[j]] =
            from_f<TO>(one_entry<GRAD>(f[j], g[j], seen, n, rho, pres, freq, mine, bias[j]));
    }
  };
  // a warp lists the entries of kChunk that the text touches, then takes them in (entry, row) pairs
  uint16_t* list = s_list[warp];
  for (int c = warp; c * kChunk < sl.n; c += THR / 32) {
    uint32_t w = ((const uint16_t*)sl.touched)[c * 32 + lane];
    int all = __popc(w), at = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += y;
    }
    at -= all;
    all = __shfl_sync(0xffffffffu, at + all, 31);
    for (; w; w &= w - 1) list[at++] = (uint16_t)(lane * 16 + __ffs(w) - 1);
    __syncwarp();
    const int pairs = all * a.R;
    for (int i0 = lane; i0 - lane < pairs; i0 += 32 * kDeep) {
      const float none[kDeep] = {};
      int v[kDeep], r[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        const int i = i0 + j * 32, slot = i / a.R;
        r[j] = i - slot * a.R;
        v[j] = i < pairs ? s0 + c * kChunk + list[slot] : -1;
      }
      again(v, r, none, false);
    }
    __syncwarp();
  }
  // the biased ones
  const int pairs = biased ? s_biased * a.R : 0;
  for (int i0 = tid; i0 < pairs; i0 += THR * kDeep) {
    float bias[kDeep];
    int v[kDeep], r[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) {
      const int i = i0 + j * THR, slot = i / a.R;
      r[j] = i - slot * a.R;
      v[j] = i < pairs ? s0 + sl.bias_u[slot] : -1;
      bias[j] = i < pairs ? sl.bias[slot] : 0.f;
    }
    again(v, r, bias, true);
  }
}

// Slices of at most S entries, smaller ones where that gives every SM its blocks.
template <typename TI, typename TO, bool GRAD, int THR>
cudaError_t launch(int B, const TI* in, TO* out, const TO* raw, PrArgs a, int S, int blocks, cudaStream_t stream) {
  const long long even = ((long long)B * a.V + blocks - 1) / blocks;
  if (even < S) S = (int)((even + kChunk - 1) / kChunk) * kChunk;
  a.S = S;
  a.nslice = (a.V + S - 1) / S;
  constexpr int unit = 32 * (64 / (int)sizeof(Raw<TI>));   // groups
  const bool al = ((uintptr_t)out % (8 * sizeof(TO))) == 0 && (a.out_ld * sizeof(TO)) % (8 * sizeof(TO)) == 0;
  const int units = (S / 8 + (al ? 0 : 1) + unit - 1) / unit;
  const size_t smem = (size_t)S * 4 + S / 8 + (size_t)a.nb * 6;
  auto kernel = process_kernel<TI, TO, GRAD, THR>;
  // (beside the lists: 48 KB are exceeded by long slices, and by the larger blocks)
  if (S > kSlice || THR > kThr) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)B * (unsigned)a.nslice, THR, smem, stream>>>(in, out, raw, a, units,
                                                                  (const void*)in == (const void*)out);
  return cudaGetLastError();
}

// Long texts of few rows: large slices read them fewer times, by blocks of more threads.
template <typename TI, typename TO, bool GRAD>
cudaError_t run(int B, const TI* in, TO* out, const TO* raw, PrArgs a, cudaStream_t stream) {
  if (GRAD) a.nb = 0;
  if (a.H / a.R >= kLong) return launch<TI, TO, GRAD, kThrLong>(B, in, out, raw, a, kSliceLong, 152, stream);
  return launch<TI, TO, GRAD, kThr>(B, in, out, raw, a, a.R > 1 ? kSlice : kSliceOne, 304, stream);
}

template <bool GRAD>
cudaError_t run_types(int B, int i_bf16, const void* in, int o_bf16, void* out, const void* raw, const PrArgs& a,
                      cudaStream_t stream) {
  using H = __nv_bfloat16;
  if (i_bf16)
    return o_bf16 ? run<H, H, GRAD>(B, (const H*)in, (H*)out, (const H*)raw, a, stream)
                  : run<H, float, GRAD>(B, (const H*)in, (float*)out, (const float*)raw, a, stream);
  return o_bf16 ? run<float, H, GRAD>(B, (const float*)in, (H*)out, (const H*)raw, a, stream)
                : run<float, float, GRAD>(B, (const float*)in, (float*)out, (const float*)raw, a, stream);
}

}  // namespace

cudaError_t launch_process(int grad, int B, int R, int V, int i_bf16, const void* in, long long in_ld, int o_bf16,
                           void* out, long long out_ld, const void* raw, long long raw_ld, const int32_t* history,
                           long long history_ld, int H, const int32_t* lengths, const int32_t* prompts,
                           const int32_t* drafted, const float* repetition, const float* presence,
                           const float* frequency, int nb, const int32_t* bias_tokens, const float* bias,
                           const uint32_t* mask, long long mask_ld, int M, const int32_t* mask_rows,
                           cudaStream_t stream) {
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
  return grad ? run_types<true>(B, i_bf16, in, o_bf16, out, raw, a, stream)
              : run_types<false>(B, i_bf16, in, o_bf16, out, raw, a, stream);
}

}  // namespace dspark
