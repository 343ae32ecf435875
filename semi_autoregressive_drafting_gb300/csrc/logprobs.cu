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
//
// Forward, one read of the logits: a warp (two in small calls) takes a 16-byte-aligned segment of a row
// (4 KB), holds it in registers (all loads issued at once), forms the maximum, then the sums relative to
// it, and leaves them as one partial result.  A block per row merges the row's partial results in their
// order: in large calls a second launch, so that a segment's warp ends with its store; in small ones the
// row's last block to finish (a counter per row, no waits).  One warp or two add a segment's halves in the
// same order: a row has the same bits in calls of any number of rows.
// Alternatives: the warps also leave the largest entry of each quarter of their segments.  The K-th
// largest entry is no less than the K-th largest of these maxima.  So the block that merges the row
// finds a bound just below that (of groups of quarters in long rows), re-reads the quarters that reach
// it, mostly from L2, and sorts the entries that do; no lists are kept during the pass.  A row of fewer
// than 2 K quarters, whose maxima say little, is read whole, with the threads' own maxima in their place.
//
// Bound by HBM once the rows are many: 3584 x 262144 bf16 rows take 287 us (6.5 TB/s, 0.97 of a copy's
// rate), the fp32 gradient of 448 x 151936 rows 82 us (6.7 TB/s).  With the merge in the pass itself
// the first took 340 us: a block that waits for its fence and counter holds registers that loads could
// use.  512 x 151936 fp32 rows with 20 alternatives take 60 us, 50 of them the pass; ranking the segments
// by all pairs instead of the counted bound cost 13 us more.  Small calls are a chain of latencies (launch,
// loads, fence and counter, bound, quarters, sort): 8 x 151936 bf16 rows with 5 alternatives 10.2 us in a
// row of calls; in a graph 8.2, and 4.3 without alternatives.
#include "common.cuh"
#include "kernels.h"

#include <type_traits>

namespace dspark {
namespace {

constexpr int kPThr = 256;
constexpr int kPWarps = kPThr / 32;
constexpr float kPL2e = 1.4426950408889634f;
constexpr float kPLn2 = 0.6931471805599453f;
constexpr int kPGroups = 2 * kPThr;  // groups of quarter segments ranked at most (two per thread)
constexpr int kSegment = 8;     // 16-byte loads per lane of a segment (4 KB)
constexpr int kPKeep = 256;     // candidates kept before a cut to the K best
constexpr int kPBuf = kPKeep + kPThr * 8;
static_assert(kPBuf % kPThr == 0 && kPBuf / kPThr * 32 <= 2 * kPThr, "what a first cut leaves: two per thread");

__device__ __forceinline__ float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one 64-bit register pair: one instruction per pair on sm_100 and later.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// What a type needs: E entries per 16 bytes, the 32-bit word of fill entries (-inf), the largest
// entry of 16 bytes, and the number of entries above a threshold.
template <typename T>
struct Lg;
template <>
struct Lg<float> {
  static constexpr int E = 4;
  static constexpr uint32_t kFill = 0xFF800000u;
  struct Thr {
    float x;
  };
  struct Cnt {
    int n;
  };
  __device__ __forceinline__ static float max16(float m, const uint4& q) {
    return fmaxf(m, fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
                          fmaxf(__uint_as_float(q.z), __uint_as_float(q.w))));
  }
  __device__ __forceinline__ static F2 pair(const uint4& q, int i) {
    return i == 0 ? f2(__uint_as_float(q.x), __uint_as_float(q.y)) : f2(__uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ __forceinline__ static Thr thr(float x) { return Thr{x}; }
  __device__ __forceinline__ static void above(Cnt& c, const uint4& q, const Thr& t) {
    c.n += (__uint_as_float(q.x) > t.x ? 1 : 0) + (__uint_as_float(q.y) > t.x ? 1 : 0) +
           (__uint_as_float(q.z) > t.x ? 1 : 0) + (__uint_as_float(q.w) > t.x ? 1 : 0);
  }
  __device__ __forceinline__ static Cnt zero() { return Cnt{0}; }
  __device__ __forceinline__ static int total(const Cnt& c) { return c.n; }
};
template <>
struct Lg<__nv_bfloat16> {
  static constexpr int E = 8;
  static constexpr uint32_t kFill = 0xFF80FF80u;
  struct Thr {
    __nv_bfloat162 x;
  };
  struct Cnt {
    __nv_bfloat162 n;  // counts of up to 2 x 256 entries are exact
  };
  __device__ __forceinline__ static __nv_bfloat162 b2(uint32_t w) {
    __nv_bfloat162 r;
    memcpy(&r, &w, 4);
    return r;
  }
  __device__ __forceinline__ static float max16(float m, const uint4& q) {
    const __nv_bfloat162 a = __hmax2(__hmax2(b2(q.x), b2(q.y)), __hmax2(b2(q.z), b2(q.w)));
    return fmaxf(m, fmaxf(__low2float(a), __high2float(a)));
  }
  __device__ __forceinline__ static F2 pair(const uint4& q, int i) {
    const uint32_t w = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static Thr thr(float x) { return Thr{__float2bfloat162_rn(x)}; }
  __device__ __forceinline__ static void above(Cnt& c, const uint4& q, const Thr& t) {
    c.n = __hadd2(c.n, __hadd2(__hadd2(__hgt2(b2(q.x), t.x), __hgt2(b2(q.y), t.x)),
                               __hadd2(__hgt2(b2(q.z), t.x), __hgt2(b2(q.w), t.x))));
  }
  __device__ __forceinline__ static Cnt zero() { return Cnt{__float2bfloat162_rn(0.f)}; }
  __device__ __forceinline__ static int total(const Cnt& c) {
    return (int)(__low2float(c.n) + __high2float(c.n));
  }
};

// The 16 bytes of a row whose first entry is v0 (16-byte aligned; v0 < 0 in front of a row that
// starts inside them): entries outside [0, V) are not read, and are -inf.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* z, int v0, int V) {
  constexpr int E = Lg<T>::E;
  if (v0 >= 0 && v0 + E <= V) return __ldg((const uint4*)(z + v0));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (E == 4) {
      w[i] = v0 + i >= 0 && v0 + i < V ? ((const uint32_t*)z)[v0 + i] : Lg<T>::kFill;
    } else {
      const int a = v0 + 2 * i;
      const uint32_t lo = a >= 0 && a < V ? ((const uint16_t*)z)[a] : (Lg<T>::kFill & 0xFFFFu);
      const uint32_t hi = a + 1 >= 0 && a + 1 < V ? ((const uint16_t*)z)[a + 1] : (Lg<T>::kFill & 0xFFFFu);
      w[i] = lo | (hi << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// entries between the 16-byte boundary at or below a row's start and the start
template <typename T>
__device__ __forceinline__ int row_head(const T* z) {
  return (int)(((uintptr_t)z & 15) / sizeof(T));
}

// A set of entries: maximum, S = sum 2^y and A = sum y 2^y with y = (z - m) log2(e) / T, and the
// number of entries above the token's.
struct Part {
  float m, S, A;
  int c;
};
__device__ __forceinline__ void part_merge(Part& a, const Part& b, float s2) {
  const float m = fmaxf(a.m, b.m);
  // shifts in the same units; an empty side (maximum -inf) is left out, so is one that underflows
  const float da = a.m == -INFINITY ? -256.f : fmaxf((a.m - m) * s2, -256.f);
  const float db = b.m == -INFINITY ? -256.f : fmaxf((b.m - m) * s2, -256.f);
  const float wa = ex2p(da), wb = ex2p(db);
  // (fused as written, so that every kernel rounds alike; an empty side changes nothing)
  a.A = fmaf(fmaf(a.S, da, a.A), wa, __fmul_rn(fmaf(b.S, db, b.A), wb));
  a.S = fmaf(a.S, wa, __fmul_rn(b.S, wb));
  a.m = m;
  a.c += b.c;
}
__device__ __forceinline__ Part part_shfl(const Part& p, int o) {
  Part q;
  q.m = __shfl_xor_sync(0xffffffffu, p.m, o);
  q.S = __shfl_xor_sync(0xffffffffu, p.S, o);
  q.A = __shfl_xor_sync(0xffffffffu, p.A, o);
  q.c = __shfl_xor_sync(0xffffffffu, p.c, o);
  return q;
}

// What the warps that share a segment tell one another: maxima and counts, the second one's sums.
struct PairSm {
  float m[kPWarps];
  int c[kPWarps];
  float S[kPWarps / 2][32], A[kPWarps / 2][32];
};

struct LpWs {
  WsHeader* hdr;
  unsigned* count;  // [kCountRows] blocks of the row done; zero between calls
  float4* part;     // [N][nchunk][segments of a chunk] each segment's Part
  uint4* quart;     // [N][nchunk][8] the largest entries of a warp's quarters, orderable (with alternatives)
};

struct LpArgs {
  int V, nchunk, top;
  float invT;
  long long ld;
  const int32_t* tokens;
  float* logp;
  float2* norm;
  float* entropy;
  int32_t* rank;
  int32_t* top_ids;
  float* top_logp;
  LpWs ws;
};

// Shared memory of the alternatives' search.
struct TopSm {
  int list[kPGroups];                      // the groups to read, in any order
  int pieces;
  unsigned long long buf[kPBuf];
  unsigned long long most[kPThr];          // each thread's largest candidate
  unsigned long long cut;                  // candidates below this are out
  int n;                                   // candidates (all that passed: over kPBuf, not all are kept)
};

// Keeps the K largest of the candidates, sorted, and raises the cut to the K-th.  The candidates
// differ, so their ranks do.  More than one per thread are first cut down: any of the K largest is no
// less than the K-th largest of the threads' own maxima.
__device__ __forceinline__ void top_prune(TopSm& t, int K) {
  const int tid = (int)threadIdx.x;
  int n = t.n;
  if (n > kPThr) {
    constexpr int kPer = kPBuf / kPThr;
    unsigned long long k[kPer], m = 0ull;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = tid + u * kPThr;
      k[u] = i < n ? t.buf[i] : 0ull;
      m = k[u] > m ? k[u] : m;
    }
    t.most[tid] = m;
    __syncthreads();
    if (tid == 0) t.n = 0;
    int r = 0;
    for (int j = 0; j < kPThr; ++j) r += t.most[j] > m ? 1 : 0;
    if (r == K - 1) t.cut = m;
    __syncthreads();
    const unsigned long long cut = t.cut;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (k[u] >= cut) t.buf[atomicAdd(&t.n, 1)] = k[u];  // at most kPer K of them
    __syncthreads();
    n = t.n;
  }
  unsigned long long k[2];
  int r[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = tid + u * kPThr;
    k[u] = i < n ? t.buf[i] : 0ull;
    r[u] = i < n ? 0 : K;
    if (u * kPThr < n)
      for (int j = 0; j < n; ++j) r[u] += t.buf[j] > k[u] ? 1 : 0;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (r[u] < K) {
      t.buf[r[u]] = k[u];
      if (r[u] == K - 1) t.cut = k[u];
    }
  if (tid == 0) t.n = min(n, K);
  __syncthreads();
}

constexpr uint32_t kNone = 0x007FFFFFu;  // orderable(-inf)

// the logit of a cut
__device__ __forceinline__ float cut_score(unsigned long long cut) {
  return (uint32_t)(cut >> 32) > kNone ? key_score(cut) : -INFINITY;
}

// The candidates among 16 bytes of a row whose first entry is v0 (few have one: their maximum is looked
// at first).
template <typename T>
__device__ __forceinline__ void top_filter(TopSm& t, const uint4& q, int v0, unsigned long long cut) {
  if (!(Lg<T>::max16(-INFINITY, q) >= cut_score(cut))) return;
#pragma unroll
  for (int e = 0; e < Lg<T>::E / 2; ++e) {
    const float2 f = un2(Lg<T>::pair(q, e));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = (h ? f.y : f.x) + 0.f;
      if (x > -INFINITY) {
        const unsigned long long k = make_key(x, (uint32_t)(v0 + 2 * e + h));
        if (k >= cut) {
          const int at = atomicAdd(&t.n, 1);
          if (at < kPBuf) t.buf[at] = k;
        }
      }
    }
  }
}

// The groups of a row's quarter segments: g quarters each, ng of them, at most two per thread.
struct Groups {
  int g, ng;
  uint32_t key[2];  // the largest entries of the thread's groups, orderable
};
__device__ __forceinline__ Groups load_groups(const LpArgs& a, long long row) {
  Groups q;
  const int nq = 4 * a.nchunk * kPWarps;
  q.g = (nq + kPGroups - 1) / kPGroups;
  q.ng = (nq + q.g - 1) / q.g;
  const uint32_t* quart = (const uint32_t*)(a.ws.quart + row * a.nchunk * kPWarps);
  const int id = (int)threadIdx.x;
  if (q.g == 1) {
    q.key[0] = id < nq ? __ldcg(quart + id) : kNone;
    q.key[1] = id + kPThr < nq ? __ldcg(quart + id + kPThr) : kNone;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int first = (id + h * kPThr) * q.g;
      q.key[h] = kNone;
      for (int i = first; i < min(nq, first + q.g); ++i) q.key[h] = max(q.key[h], __ldcg(quart + i));
    }
  }
  return q;
}

// The K largest entries of a row, sorted, into t.buf (t.n of them), by a whole block.  `beside` is run
// by the last warp while the others read.
template <typename T, int PER, typename F>
__device__ __forceinline__ void top_search(TopSm& t, const LpArgs& a, const T* z, int head, const Groups& q4, F beside) {
  constexpr int E = Lg<T>::E;
  constexpr int kQuart = 8 * PER;  // 16-byte vectors per quarter segment
  const int K = a.top, tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = q4.g, ng = q4.ng;
  uint32_t key[2] = {q4.key[0], q4.key[1]};
  if (tid == 0) t.n = t.pieces = 0;
  const bool whole = ng < 2 * K;
  const int len = whole ? (a.V + head + E - 1) / E : g * kQuart;  // vectors per piece of the row
  auto vec = [&](int i) {
    const int v0 = i * E - head;
    return v0 < a.V ? load16<T>(z, v0, a.V) : make_uint4(Lg<T>::kFill, Lg<T>::kFill, Lg<T>::kFill, Lg<T>::kFill);
  };
  if (whole) {
    float m = -INFINITY;
#pragma unroll 8
    for (int i = tid; i < len; i += kPThr) m = Lg<T>::max16(m, vec(i));
    key[0] = orderable(m + 0.f);
    key[1] = kNone;
  }
  // the largest bound, to 15 bits (sign, exponent, six of the mantissa), that K threads' maxima reach
  const uint32_t most = max(key[0], key[1]);
  uint32_t bound = 0u;
  for (int bit = 31; bit >= 17; --bit) {
    const uint32_t c = bound | (1u << bit);
    if (__syncthreads_count(most >= c) >= K) bound = c;
  }
  if (whole) {
    if (tid == 0) t.list[t.pieces++] = 0;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (key[h] > kNone && key[h] >= bound) t.list[atomicAdd(&t.pieces, 1)] = tid + h * kPThr;
  }
  if (tid == 0) t.cut = max(1ull, (unsigned long long)bound << 32);
  __syncthreads();
  const unsigned long long cut = t.cut;
  // The pieces (few entries but the K pass the cut) in runs of 32 vectors, eight in flight per warp.
  const int runs = (len + 31) / 32, pieces = t.pieces;
  const uint32_t inv = 0xFFFFFFFFu / (uint32_t)runs + 1u;  // c / runs = high half of c inv (c runs < 2^32)
  for (int c0 = warp; c0 < pieces * runs; c0 += 8 * kPWarps) {
    uint4 q[8];
    int at[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * kPWarps, r = runs == 1 ? c : (int)__umulhi((uint32_t)c, inv), i = (c - r * runs) * 32 + lane;
      const bool in = r < pieces && i < len;
      at[u] = in ? t.list[r] * len + i : 0;
      q[u] = in ? vec(at[u]) : make_uint4(Lg<T>::kFill, Lg<T>::kFill, Lg<T>::kFill, Lg<T>::kFill);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) top_filter<T>(t, q[u], at[u] * E - head, cut);
  }
  if (warp == kPWarps - 1) beside();
  __syncthreads();
  if (t.n > kPBuf) {  // (in every thread or none: the count changes next behind a barrier)
    __syncthreads();
    // Too many at once (sorted or constant rows): step by step, cutting to the K best whenever kPKeep are
    // exceeded, which raises the cut.
    if (tid == 0) t.n = 0;
    __syncthreads();
    for (int r = 0; r < pieces; ++r) {
      const int first = t.list[r] * len;
      for (int i0 = 0; i0 < len; i0 += kPThr) {
        const int i = i0 + tid;
        if (i < len) top_filter<T>(t, vec(first + i), (first + i) * E - head, t.cut);
        __syncthreads();
        const bool full = t.n > kPKeep;
        __syncthreads();  // (every thread has read the count before the next candidates add to it)
        if (full) top_prune(t, K);
      }
    }
  }
  top_prune(t, K);
}

// Shared memory of a row's merge.
template <bool TOP>
struct RowSm {
  TopSm top;
  Part red[kPWarps];
  float m, ls;
};
template <>
struct RowSm<false> {
  Part red[kPWarps];
  float m, ls;
};


// A row's outputs from its segments' partial results, by a whole block.
template <typename T, int PER, bool TOP>
__device__ __forceinline__ void finish_row(RowSm<TOP>& sm, const LpArgs& a, const T* z, int head, long long row,
                                           int x, float zx, float s2) {
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nseg = a.nchunk * (kPWarps * PER / kSegment);
  Groups q4;
  if constexpr (TOP) q4 = load_groups(a, row);  // (in flight beside the partial results)
  Part p{-INFINITY, 0.f, 0.f, 0};
  const float4* part = a.ws.part + row * nseg;
  for (int i = tid; i < nseg; i += kPThr) {
    const float4 v = __ldcg(part + i);
    part_merge(p, Part{v.x, v.y, v.z, __float_as_int(v.w)}, s2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part_merge(p, part_shfl(p, o), s2);
  if (lane == 0) sm.red[warp] = p;
  auto outputs = [&]() {  // (one warp, after a barrier)
    p = sm.red[lane & (kPWarps - 1)];
#pragma unroll
    for (int o = kPWarps / 2; o > 0; o >>= 1) part_merge(p, part_shfl(p, o), s2);
    if (lane == 0) {
      const bool bad = x < -1 || x >= a.V;
      const bool none = p.S == 0.f;  // every entry -inf
      const float ls = none ? 0.f : logf(p.S);
      if (a.norm) a.norm[row] = make_float2(p.m, ls);
      if (a.entropy) a.entropy[row] = none ? 0.f : fmaf(-kPLn2, p.A / p.S, ls);
      if (a.logp)
        a.logp[row] = x == -1 ? 0.f
                      : bad || isnan(p.S) ? NAN
                      : zx == -INFINITY   ? -INFINITY
                                          : fmaf(zx - p.m, a.invT, -ls);
      if (a.rank) a.rank[row] = bad ? -1 : x < 0 ? 0 : p.c + 1;
      if (bad) atomicMax(&a.ws.hdr->status, kErrInvalid);
      sm.m = p.m;
      sm.ls = ls;
    }
  };
  if constexpr (TOP) {
    TopSm& t = sm.top;
    top_search<T, PER>(t, a, z, head, q4, outputs);
    if (tid < a.top) {
      const bool has = tid < t.n;
      a.top_ids[row * a.top + tid] = has ? (int32_t)key_token(t.buf[tid]) : -1;
      a.top_logp[row * a.top + tid] = has ? fmaf(key_score(t.buf[tid]) - sm.m, a.invT, -sm.ls) : -INFINITY;
    }
  } else {
    __syncthreads();
    if (warp == 0) outputs();
  }
}

// a row's token (-1: none) and its logit, +inf without one: nothing is above it
template <typename T>
__device__ __forceinline__ float token_logit(const LpArgs& a, const T* z, int x) {
  return x >= 0 && x < a.V ? to_f<T>(z[x]) : INFINITY;
}

// ONE: the row's last block also merges it (small calls).  Large calls keep five blocks per SM: with four,
// at 52 registers, the largest call took 294 us, against 287.
template <typename T, int PER, bool TOP, bool ONE>
__global__ void __launch_bounds__(kPThr, ONE ? 0 : 5) logprob_kernel(const T* __restrict__ logits, const LpArgs a) {
  constexpr int E = Lg<T>::E;
  if constexpr (!ONE) pdl_trigger();
  const long long row = blockIdx.x / (unsigned)a.nchunk;
  const int ch = (int)(blockIdx.x % (unsigned)a.nchunk);
  const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const T* z = logits + row * a.ld;
  const int head = row_head(z), V = a.V;
  const int g0 = (ch * kPWarps + warp) * (32 * PER);  // this warp's first 16-byte group
  const int x = a.tokens ? a.tokens[row] : -1;
  uint4 q[PER];
  if (g0 * E >= head && (g0 + 32 * PER) * E - head <= V) {
#pragma unroll
    for (int u = 0; u < PER; ++u) q[u] = __ldg((const uint4*)(z + ((g0 + u * 32 + lane) * E - head)));
  } else {
#pragma unroll
    for (int u = 0; u < PER; ++u) q[u] = load16<T>(z, (g0 + u * 32 + lane) * E - head, V);
  }
  const float zx = token_logit<T>(a, z, x);
  const float s2 = a.invT * kPL2e;
  Part p;
  p.m = -INFINITY;
  if constexpr (TOP) {
    uint32_t k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float m = -INFINITY;
#pragma unroll
      for (int u = j * (PER / 4); u < (j + 1) * (PER / 4); ++u) m = Lg<T>::max16(m, q[u]);
      k[j] = __reduce_max_sync(0xffffffffu, orderable(m + 0.f));
    }
    if (lane == 0) a.ws.quart[(row * a.nchunk + ch) * kPWarps + warp] = make_uint4(k[0], k[1], k[2], k[3]);
    p.m = key_score((unsigned long long)max(max(k[0], k[1]), max(k[2], k[3])) << 32);
  } else {
#pragma unroll
    for (int u = 0; u < PER; ++u) p.m = Lg<T>::max16(p.m, q[u]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) p.m = fmaxf(p.m, __shfl_xor_sync(0xffffffffu, p.m, o));
  }
  typename Lg<T>::Cnt cnt = Lg<T>::zero();
  const typename Lg<T>::Thr thr = Lg<T>::thr(zx);
  constexpr bool kPaired = PER < kSegment;  // two warps share a segment
  __shared__ typename std::conditional<kPaired, PairSm, int>::type pair;
  if constexpr (kPaired) {
#pragma unroll
    for (int u = 0; u < PER; ++u) Lg<T>::above(cnt, q[u], thr);
    p.c = __reduce_add_sync(0xffffffffu, Lg<T>::total(cnt));
    if (lane == 0) {
      pair.m[warp] = p.m;
      pair.c[warp] = p.c;
    }
    __syncthreads();
    p.m = fmaxf(p.m, pair.m[warp ^ 1]);
    p.c += pair.c[warp ^ 1];
  }
  const float mu = p.m == -INFINITY ? 0.f : p.m;
  const F2 nm = f2(-mu, -mu), ss = f2(s2, s2);
  // S and A of vectors u0 to u0 + 3
  auto sums = [&](int u0, float& s, float& a1) {
    F2 S = f2(0.f, 0.f), A = S;
#pragma unroll
    for (int u = 0; u < kSegment / 2; ++u)
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        float2 y = un2(mul2(add2(Lg<T>::pair(q[u0 + u], e), nm), ss));
        // 2^y is zero from -150 down: -inf becomes a finite factor of a zero.  (A NaN passes through
        // the exponential, not through this maximum.)
        const F2 ex = f2(ex2p(y.x), ex2p(y.y));
        S = add2(S, ex);
        A = fma2(ex, f2(fmaxf(y.x, -256.f), fmaxf(y.y, -256.f)), A);
      }
    const float2 S1 = un2(S), A1 = un2(A);
    s = S1.x + S1.y;
    a1 = A1.x + A1.y;
  };
  sums(0, p.S, p.A);
  if constexpr (kPaired) {
    if (warp & 1) {
      pair.S[warp >> 1][lane] = p.S;
      pair.A[warp >> 1][lane] = p.A;
    }
    __syncthreads();
    if (!(warp & 1)) {
      p.S += pair.S[warp >> 1][lane];
      p.A += pair.A[warp >> 1][lane];
    }
  } else {
    float S, A;
    sums(kSegment / 2, S, A);
    p.S += S;
    p.A += A;
  }
  if (!kPaired || !(warp & 1)) {
    p.S = warp_sum(p.S);
    p.A = warp_sum(p.A);
    if constexpr (!kPaired) {
#pragma unroll
      for (int u = 0; u < PER; ++u) Lg<T>::above(cnt, q[u], thr);
      p.c = __reduce_add_sync(0xffffffffu, Lg<T>::total(cnt));
    }
    if (lane == 0)
      a.ws.part[(row * a.nchunk + ch) * (kPWarps * PER / kSegment) + warp * PER / kSegment] =
          make_float4(p.m, p.S, p.A, __int_as_float(p.c));
  }
  if constexpr (ONE) {
    __shared__ __align__(16) RowSm<TOP> sm;
    __shared__ int s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
      s_last = 1;
      if (a.nchunk > 1) {
        __threadfence();
        s_last = atomicAdd(&a.ws.count[row], 1u) == (unsigned)a.nchunk - 1u;
        if (s_last) {
          __threadfence();
          a.ws.count[row] = 0u;
        }
      }
    }
    __syncthreads();
    if (s_last) finish_row<T, PER, TOP>(sm, a, z, head, row, x, zx, s2);
  }
}

template <typename T, int PER, bool TOP>
__global__ void __launch_bounds__(kPThr) logprob_rows_kernel(const T* __restrict__ logits, const LpArgs a) {
  __shared__ __align__(16) RowSm<TOP> sm;
  const long long row = blockIdx.x;
  const T* z = logits + row * a.ld;
  const int x = a.tokens ? a.tokens[row] : -1;
  const float zx = token_logit<T>(a, z, x);
  pdl_wait();  // (above: only what the caller gave)
  finish_row<T, PER, TOP>(sm, a, z, row_head(z), row, x, zx, a.invT * kPL2e);
}

// ------------------------------------------------------------------ gradient
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    memcpy(&w[i], &b, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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

constexpr int kGPer = 4;  // 16-byte groups per thread

// With lp = ln p_v: dz = p (c0 + c1 lp), c0 = -(g + h H) / T, c1 = -h / T, plus g / T at the token.
template <typename T>
__global__ void __launch_bounds__(kPThr) logprob_grad_kernel(
    int V, int nchunk, float invT, const T* logits, long long ld, const int32_t* __restrict__ tokens,
    const float2* __restrict__ norm, const float* __restrict__ entropy, const float* __restrict__ gl,
    const float* __restrict__ gh, T* grad, long long gld) {
  constexpr int E = Lg<T>::E;
  const long long row = blockIdx.x / (unsigned)nchunk;
  const int ch = (int)(blockIdx.x % (unsigned)nchunk);
  const T* z = logits + row * ld;
  T* o = grad + row * gld;
  const int head = row_head(z);
  const int g0 = ch * (kPThr * kGPer) + (int)threadIdx.x;
  uint4 q[kGPer];
#pragma unroll
  for (int u = 0; u < kGPer; ++u) {
    const int v0 = (g0 + u * kPThr) * E - head;
    q[u] = v0 >= 0 && v0 + E <= V ? __ldcs((const uint4*)(z + v0)) : load16<T>(z, v0, V);
  }
  const int x = tokens ? tokens[row] : -1;
  const float2 n = norm[row];
  const float g = gl && x >= 0 ? gl[row] : 0.f;
  const float h = gh ? gh[row] : 0.f, H = gh ? entropy[row] : 0.f;
  const bool bad = x < -1 || x >= V || isnan(n.y);  // (a row with NaN or +inf: NaN throughout)
  const float nm = n.x == -INFINITY ? 0.f : -n.x;  // (then every entry is -inf and every p is zero)
  const float c1 = bad ? NAN : -h * invT, c0 = bad ? NAN : -(g + h * H) * invT;
  const bool same = row_head((const T*)o) == head;
#pragma unroll
  for (int u = 0; u < kGPer; ++u) {
    const int v0 = (g0 + u * kPThr) * E - head;
    if (v0 >= V) break;
    float f[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 zz = un2(Lg<T>::pair(q[u], e));
      // -inf becomes a finite factor of a p that is zero
      const float la = fmaxf(fmaf(zz.x + nm, invT, -n.y), -1000.f);
      const float lb = fmaxf(fmaf(zz.y + nm, invT, -n.y), -1000.f);
      f[2 * e] = ex2p(la * kPL2e) * fmaf(c1, la, c0);
      f[2 * e + 1] = ex2p(lb * kPL2e) * fmaf(c1, lb, c0);
    }
    if (x >= v0 && x < v0 + E) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v0 + e == x) f[e] = fmaf(g, invT, f[e]);
    }
    if (same && v0 >= 0 && v0 + E <= V) {
      __stcs((uint4*)(o + v0), pack16<T>(f));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v0 + e >= 0 && v0 + e < V) o[v0 + e] = from_f<T>(f[e]);
    }
  }
}

constexpr size_t lp_align(size_t x) { return (x + 255) / 256 * 256; }

// chunks of a row for 16-byte groups of E entries, PER per thread; one more group when rows may
// start off a 16-byte boundary
int lp_chunks(int V, int E, int per, bool aligned_rows) {
  const int groups = (V + (aligned_rows ? 0 : E - 1) + E - 1) / E;
  return (groups + kPThr * per - 1) / (kPThr * per);
}

// Sixteen-byte loads per thread.  Small calls take one launch (measured: 16 MB of fp32 rows 8.4 us this way
// and 10.4 us the other, 64 MB with 20 alternatives the other way round).  They give a segment to two warps
// where whole chunks would be fewer than the SMs (8 x 151936 bf16 rows 4.3 us, against 5.1 with one warp)
// or a row fits in half a chunk; else to one (77 x 50021 fp32 rows, 8 alternatives: 11.6 us against 12.7).
constexpr int kPerMany = kSegment, kPerFew = kSegment / 2;
constexpr int kFill = 152;  // chunks for every SM
constexpr long long kFewBytes = 16ll << 20;
// Rows that are counted at most: only small calls count, and only rows of more than one chunk, that is of
// more than kPThr kPerFew - 1 whole groups.  The counters have this room in every workspace, whatever N:
// what a call of other sizes leaves in the workspace is never in their place.
constexpr int kCountRows = (int)(kFewBytes / ((kPThr * kPerFew - 1) * 16)) + 1;

template <typename T, bool TOP>
cudaError_t lp_run(int N, const T* logits, LpArgs a, cudaStream_t stream) {
  constexpr int E = Lg<T>::E;
  const bool al = ((uintptr_t)logits % 16) == 0 && (a.ld * (long long)sizeof(T)) % 16 == 0;
  if ((long long)N * a.V * (long long)sizeof(T) <= kFewBytes) {
    a.nchunk = lp_chunks(a.V, E, kPerMany, al);
    if (lp_chunks(a.V, E, kPerFew, al) > 1 && (long long)N * a.nchunk >= kFill) {
      logprob_kernel<T, kPerMany, TOP, true><<<(unsigned)N * (unsigned)a.nchunk, kPThr, 0, stream>>>(logits, a);
      return cudaGetLastError();
    }
    a.nchunk = lp_chunks(a.V, E, kPerFew, al);
    logprob_kernel<T, kPerFew, TOP, true><<<(unsigned)N * (unsigned)a.nchunk, kPThr, 0, stream>>>(logits, a);
    return cudaGetLastError();
  }
  a.nchunk = lp_chunks(a.V, E, kPerMany, al);
  logprob_kernel<T, kPerMany, TOP, false><<<(unsigned)N * (unsigned)a.nchunk, kPThr, 0, stream>>>(logits, a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(logprob_rows_kernel<T, kPerMany, TOP>, (unsigned)N, kPThr, 0, stream, logits, a);
}

// Room for the chunks of N rows of at most V entries, whatever their type and alignment.  Short
// chunks (problems of at most kFewBytes, of kPThr kPerFew 16 bytes per chunk) are bounded by their
// total: the room never shrinks as N or V grows, so a workspace serves smaller problems too.
size_t lp_slots(int N, int V) {
  const size_t many = (size_t)N * lp_chunks(V, 4, kPerMany, false);
  const size_t few = (size_t)N * lp_chunks(V, 4, kPerFew, false), cap = (size_t)kFewBytes / (kPThr * kPerFew * 16) + 2 * (size_t)N;
  return many > (few < cap ? few : cap) ? many : few < cap ? few : cap;
}

}  // namespace

size_t logprobs_workspace_bytes(int N, int V, int top) {
  const size_t part = lp_align(lp_slots(N, V) * kPWarps * sizeof(float4));
  return sizeof(WsHeader) + lp_align(kCountRows * sizeof(unsigned)) + (top ? 2 : 1) * part;
}

cudaError_t launch_logprobs(int N, int V, float T, int bf16, const void* logits, long long ld,
                            const int32_t* tokens, int top, float* logp, float* norm, float* entropy,
                            int32_t* rank, int32_t* top_ids, float* top_logp, void* workspace,
                            cudaStream_t stream) {
  LpArgs a;
  a.V = V;
  a.top = top;
  a.invT = 1.f / T;
  a.ld = ld;
  a.tokens = tokens;
  a.logp = logp;
  a.norm = (float2*)norm;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  uint8_t* w = (uint8_t*)workspace;
  a.ws.hdr = (WsHeader*)w;
  w += sizeof(WsHeader);
  a.ws.count = (unsigned*)w;
  w += lp_align(kCountRows * sizeof(unsigned));
  a.ws.part = (float4*)w;
  a.ws.quart = (uint4*)(w + lp_align(lp_slots(N, V) * kPWarps * sizeof(float4)));
  const __nv_bfloat16* zb = (const __nv_bfloat16*)logits;
  const float* zf = (const float*)logits;
  if (bf16) return top ? lp_run<__nv_bfloat16, true>(N, zb, a, stream) : lp_run<__nv_bfloat16, false>(N, zb, a, stream);
  return top ? lp_run<float, true>(N, zf, a, stream) : lp_run<float, false>(N, zf, a, stream);
}

cudaError_t launch_logprobs_grad(int N, int V, float T, int bf16, const void* logits, long long ld,
                                 const int32_t* tokens, const float* norm, const float* entropy,
                                 const float* gl, const float* gh, void* grad, long long gld,
                                 cudaStream_t stream) {
  const bool al = ((uintptr_t)logits % 16) == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0;
  const int nchunk = lp_chunks(V, bf16 ? 8 : 4, kGPer, al);
  const unsigned grid = (unsigned)N * (unsigned)nchunk;
  if (bf16)
    logprob_grad_kernel<__nv_bfloat16><<<grid, kPThr, 0, stream>>>(
        V, nchunk, 1.f / T, (const __nv_bfloat16*)logits, ld, tokens, (const float2*)norm, entropy, gl, gh,
        (__nv_bfloat16*)grad, gld);
  else
    logprob_grad_kernel<float><<<grid, kPThr, 0, stream>>>(V, nchunk, 1.f / T, (const float*)logits, ld, tokens,
                                                           (const float2*)norm, entropy, gl, gh, (float*)grad,
                                                           gld);
  return cudaGetLastError();
}

}  // namespace dspark
