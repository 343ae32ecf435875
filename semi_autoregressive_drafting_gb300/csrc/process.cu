// process.cu -- what a request asks of its logits: penalties for the tokens that its text holds, biases
// and a grammar's mask; and the gradient with respect to the raw logits.
//
// Row (b, k) is position k of request b's block; its text is the request's history and the k tokens drafted
// before it.  With c = how often the text's generated part holds v, and seen = whether the text does:
//   y = z / rho if z > 0 else z rho, where seen;  y -= f c + p [c > 0];  y += the biases of v;
//   -inf where the mask's bit of v is clear.
//   dL/dz = dL/dy (1 / rho if z > 0 else rho, where seen), 0 where masked.
//
// A block takes a slice of the vocabulary for all rows of a request.  It counts the history's tokens in its
// slice in shared memory and lists those it meets (each block reads the whole history: from L2, at once),
// copies its entries of every row, masked, in 16- and 32-byte pieces, and then goes over the listed tokens
// alone: the entries that no text and no bias touches cost a copy.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

#include <type_traits>

namespace dspark {
namespace {

constexpr int kThr = 256;
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

// The list of a block's touched tokens, in shared memory behind the counts.
struct Slice {
  uint32_t* count;  // [S]
  uint16_t* list;   // [S]
  float* bias;      // [S] with biases
};

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

// TI: the input's type; TO: the output's; GRAD: the input is dL/dy and the raw logits have the output's type.
template <typename TI, typename TO, bool GRAD>
__global__ void __launch_bounds__(kThr) process_kernel(const TI* in, TO* out, const TO* raw, const PrArgs a,
                                                       const bool same) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_n;
  __shared__ int s_drafted[kMaxRows];
  const int b = (int)(blockIdx.x / (unsigned)a.nslice), tid = (int)threadIdx.x;
  const int s0 = (int)(blockIdx.x % (unsigned)a.nslice) * a.S, s1 = min(s0 + a.S, a.V), n = s1 - s0;
  Slice sl;
  sl.count = (uint32_t*)smem;
  sl.list = (uint16_t*)(sl.count + a.S);
  sl.bias = (float*)(sl.list + a.S);
  const float rho = a.repetition ? a.repetition[b] : 1.f;
  const float pres = !GRAD && a.presence ? a.presence[b] : 0.f;
  const float freq = !GRAD && a.frequency ? a.frequency[b] : 0.f;
  const bool penalised = rho != 1.f || pres != 0.f || freq != 0.f;
  const bool biased = !GRAD && a.nb > 0;
  bool bad = false;
  if (penalised || biased) {
    for (int i = tid; i < a.S; i += kThr) {
      sl.count[i] = 0u;
      if (biased) sl.bias[i] = 0.f;
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
  }
  if (penalised) {
    const int L = a.lengths ? a.lengths[b] : a.H, P = a.prompts ? a.prompts[b] : 0;
    bad = L < 0 || L > a.H || P < 0 || P > L;
    const int32_t* h = a.history + (long long)b * a.history_ld;
    const int nh = bad ? 0 : L;
#pragma unroll 4
    for (int i = tid; i < nh; i += kThr) {
      const int t = __ldg(h + i), u = t - s0;
      if ((unsigned)u < (unsigned)n) {
        const uint32_t old = i < P ? atomicOr(&sl.count[u], kSeen) : atomicAdd(&sl.count[u], 1u);
        if (old == 0u) sl.list[atomicAdd(&s_n, 1)] = (uint16_t)u;
      } else if (t < -1 || t >= a.V) {
        bad = true;
      }
    }
    if (tid < a.R - 1) {
      const int t = a.drafted ? a.drafted[(long long)b * (a.R - 1) + tid] : -1, u = t - s0;
      s_drafted[tid] = t;
      if ((unsigned)u < (unsigned)n) {
        if (atomicOr(&sl.count[u], kDrafted) == 0u) sl.list[atomicAdd(&s_n, 1)] = (uint16_t)u;
      } else if (t < -1 || t >= a.V) {
        bad = true;
      }
    }
  }
  if (biased && tid < 32) {
    // one warp, in the list's order: entries of the same token in one step are added by the first of them
    for (int i0 = 0; i0 < a.nb; i0 += 32) {
      const int i = i0 + tid;
      const int t = i < a.nb ? __ldg(a.bias_tokens + (long long)b * a.nb + i) : -1, u = t - s0;
      const bool mine = (unsigned)u < (unsigned)n;
      if (!mine && (t < -1 || t >= a.V)) bad = true;
      const float x = mine ? __ldg(a.bias + (long long)b * a.nb + i) : 0.f;
      if (!__any_sync(0xffffffffu, mine)) continue;
      const uint32_t peers = __match_any_sync(0xffffffffu, mine ? u : -1 - tid);
      float sum = mine ? sl.bias[u] : 0.f;
      for (int j = 0; j < 32; ++j) {
        const float y = __shfl_sync(0xffffffffu, x, j);
        if ((peers >> j) & 1u) sum += y;
      }
      if (mine && tid == __ffs(peers) - 1) {
        sl.bias[u] = sum;
        if (atomicOr(&sl.count[u], kBiased) == 0u) sl.list[atomicAdd(&s_n, 1)] = (uint16_t)u;
      }
      __syncwarp();
    }
  }
  bad = __syncthreads_or(bad);

  using W = typename std::conditional<sizeof(TO) == 2, uint16_t, uint32_t>::type;
  const uint32_t fill = GRAD ? 0u : sizeof(TO) == 2 ? 0xFF80FF80u : 0xFF800000u;
  for (int r = 0; r < a.R; ++r) {
    const long long row = (long long)b * a.R + r;
    const TI* z = in + row * a.in_ld;
    TO* o = out + row * a.out_ld;
    const int mr = !a.mask ? -1 : a.mask_rows ? a.mask_rows[row] : (int)row;
    if (bad || mr < -1 || mr >= a.M) {  // (M = 0 without a mask, and mr is -1)
      if (bad || a.mask)
        for (int v = s0 + tid; v < s1; v += kThr) o[v] = from_f<TO>(NAN);
      continue;
    }
    const uint32_t* mask = mr >= 0 ? a.mask + (long long)mr * a.mask_ld : nullptr;
    if (same && !mask) continue;
    // groups of eight entries on the output's boundaries; those that reach out of the slice by entries
    constexpr int A = 8 * sizeof(TO);
    const int head = (int)(((uintptr_t)o & (A - 1)) / sizeof(TO));
    const int off = (int)(((uintptr_t)(z - head) & 15) / sizeof(TI));
    const int g1 = (s1 + head + 7) >> 3;
    for (int g = ((s0 + head) >> 3) + tid; g < g1; g += kThr) {
      const int v0 = g * 8 - head;
      if (v0 >= s0 && v0 + 8 <= s1 && v0 - off >= 0 && v0 + 8 + beyond<TI>(off) <= a.V) {
        const uint32_t bits = mask ? mask_bits(mask, v0) : 0xFFu;
        if (same && bits == 0xFFu) continue;
        Raw<TO> y;
        convert8(y, load8(z + v0, off));
        mask8(y, bits, fill);
        store8(o + v0, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int v = v0 + e;
          if (v < s0 || v >= s1) continue;
          if (!allowed(mask, v))
            ((W*)o)[v] = (W)fill;
          else if (!same)
            o[v] = from_f<TO>(to_f<TI>(z[v]));
        }
      }
    }
  }
  if (bad || !(penalised || biased)) return;
  __syncthreads();

  const int touched = s_n;
  for (int i = tid; i < touched; i += kThr) {
    const int u = sl.list[i], v = s0 + u;
    const uint32_t w = sl.count[u];
    const bool mine = (w & kBiased) != 0u;
    const float bias = mine ? sl.bias[u] : 0.f;
    const int c0 = (int)(w & kCount);
    int c = c0;
    bool seen = (w & (kSeen | kCount)) != 0u;
    for (int r = 0; r < a.R; ++r) {
      if (r > 0 && (w & kDrafted) && s_drafted[r - 1] == v) {
        ++c;
        seen = true;
      }
      if (!seen && !mine) continue;
      const long long row = (long long)b * a.R + r;
      const int mr = !a.mask ? -1 : a.mask_rows ? a.mask_rows[row] : (int)row;
      if (mr < -1 || mr >= a.M) {
        if (a.mask) continue;
      }
      if (!allowed(mr >= 0 ? a.mask + (long long)mr * a.mask_ld : nullptr, v)) continue;
      const float x = to_f<TI>(in[row * a.in_ld + v]);
      const float z = GRAD ? to_f<TO>(raw[row * a.raw_ld + v]) : x;
      out[row * a.out_ld + v] = from_f<TO>(one_entry<GRAD>(x, z, seen, c, rho, pres, freq, mine, bias));
    }
  }
}

template <typename TI, typename TO, bool GRAD>
cudaError_t run(int B, const TI* in, TO* out, const TO* raw, PrArgs a, cudaStream_t stream) {
  a.S = 4096;
  a.nslice = (a.V + a.S - 1) / a.S;
  const size_t smem = (size_t)a.S * (a.nb > 0 && !GRAD ? 10 : 6);
  const bool same = (const void*)in == (const void*)out;
  process_kernel<TI, TO, GRAD><<<(unsigned)B * (unsigned)a.nslice, kThr, smem, stream>>>(in, out, raw, a, same);
  return cudaGetLastError();
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
