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
// Loss with gradient: a cluster of blocks reads a row once into their shared memory (bulk copies), puts -inf in place
// of the row's own tokens, forms the maximum and sum of each 4 KB segment, exchanges them (distributed shared
// memory), forms the outcomes and writes the gradient: each logit crosses HBM once each way.  The loss alone of few
// rows goes this way too.  Rows that no cluster holds (above 3.2 MB), and the loss alone of many: a warp takes a
// segment in registers, a second launch with one block per row joins the segments and forms the outcomes, and a
// third, for the gradient, reads the row again.  Both form the same sums in the same order.  The gradient of given
// normalisers is the last two of these.
//
// 3584 x 262144 bf16, 64 tokens: 740 us (5.1 TB/s; three passes would be 850), bound by what is resident: 24 of 28 MB
// of shared memory hold rows, for 11 us each, of which the loads take 3, the sums 2, the exchange and the outcomes
// 4 and the gradient 2.5 (resident clusters that load the next row behind the gradient: 838; blocks of half the
// size, twice as many: 1010).  448 x 151936 fp32: 116 us (4.7 TB/s).  The gradient alone: 540 and 84 us (6.95 and 6.5
// TB/s); the loss alone, 499 x 50021 fp32: 29 us, two launches.  The teacher's part is hidden behind the loads.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"

#include <mutex>

namespace dspark {
namespace {

constexpr int kThr = 256;
constexpr int kWarps = kThr / 32;
constexpr int kMaxK = 128;
constexpr int kIdLane = kMaxK / 32;   // a row's tokens per lane
constexpr int kSegment = 8;           // 16-byte loads per lane of a segment (4 KB)
constexpr float kL2e = 1.4426950408889634f;
template <typename T>
constexpr int kSegEntries = 32 * kSegment * Lg<T>::E;

// What a row's gradient needs beside the logits.
struct RowCoef {
  float nm, ls, c;  // P_v = exp((z_v + nm) / T - ls), dL/dz_v = c P_v
  float pad;
};

struct DsArgs {
  int V, K, nchunk, rest, stuck;
  float T, invT, invT_lo, a_kl, a_l1;
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

// -inf in place of the entries whose bits are set
template <typename T>
__device__ __forceinline__ uint4 without(const uint4& q, uint32_t bits) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      w[i] = (bits >> i) & 1u ? Lg<T>::kFill : w[i];
    } else {
      const uint32_t m = ((bits >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((bits >> (2 * i)) & 2u ? 0xFFFF0000u : 0u);
      w[i] = (w[i] & ~m) | (Lg<T>::kFill & m);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The maximum and the sum of 2^((z - m) log2(e) / T) of a warp's segment, whose 16-byte groups q gives by number:
// registers, or shared memory read twice.
template <typename T, typename Q>
__device__ __forceinline__ float2 segment_sum(const Q& q, float s2) {
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < kSegment; ++u) m = Lg<T>::max16(m, q(u));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const F2 nm = f2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m), s22 = f2(s2, s2);
  F2 S = f2(0.f, 0.f);
#pragma unroll
  for (int u = 0; u < kSegment; ++u) {
    const uint4 g = q(u);
#pragma unroll
    for (int e = 0; e < Lg<T>::E / 2; ++e) {
      const float2 y = un2(mul2(add2(Lg<T>::pair(g, e), nm), s22));
      S = add2(S, f2(ex2p(y.x), ex2p(y.y)));
    }
  }
  const float2 two = un2(S);
  return make_float2(m, warp_sum(two.x + two.y));
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
  unsigned long long mine = 0ull;   // E bits for each of the lane's groups: the row's own tokens
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    uint32_t here = __ballot_sync(0xffffffffu, id[i] >= 0 && id[i] >= first && id[i] < last);
    while (here) {
      const int src = __ffs(here) - 1;
      here &= here - 1;
      const int at = __shfl_sync(0xffffffffu, id[i], src) - first, g = at / E;
      if ((g & 31) == lane) mine |= 1ull << ((g >> 5) * E + at % E);
    }
  }
  if (__any_sync(0xffffffffu, mine != 0ull)) {
#pragma unroll
    for (int u = 0; u < kSegment; ++u) q[u] = without<T>(q[u], (uint32_t)(mine >> (u * E)) & ((1u << E) - 1u));
  }
  const float2 p = segment_sum<T>([&](int u) { return q[u]; }, kL2e / a.T);
  if (lane == 0) a.part[(row * a.nchunk + ch) * kWarps + warp] = p;
}

// ------------------------------------------------------------------ the outcomes of a row
// In fp32, with numbers as sums of two where one would round away what they hold (ln S is up to 17, half a step
// of that 1e-6; 1 - Q is what Q's last digits make it).  64-bit arithmetic for these few numbers took 11 us of a
// row's 18.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add_two(float a, float b) {
  const float s = a + b, t = s - a;
  return Two{s, isinf(s) ? 0.f : (a - (s - t)) + (b - t)};
}
// (x - m) / T, with 1 / T in two parts
__device__ __forceinline__ Two scaled(float x, float m, const Two& invT) {
  const Two d = add_two(x, -m);
  const float y = d.hi * invT.hi;
  return Two{y, isinf(y) ? 0.f : fmaf(d.hi, invT.hi, -y) + fmaf(d.lo, invT.hi, d.hi * invT.lo)};
}
__device__ __forceinline__ Two minus(const Two& a, const Two& b) {
  const Two s = add_two(a.hi, -b.hi);
  return Two{s.hi, s.lo + (a.lo - b.lo)};
}
__device__ __forceinline__ Two plus(const Two& a, const Two& b) {
  const Two s = add_two(a.hi, b.hi);
  return Two{s.hi, s.lo + (a.lo + b.lo)};
}
// ln 2 in two parts: nine bits, so that its multiples are exact, and the rest (to 2e-12)
constexpr float kLn2a = 0.693359375f, kLn2b = -2.12194440e-4f;
// exp x to some 2^-26 of itself: 2^k e^r with |r| <= 0.35, and e^r = 1 + r + r^2 (1/2 + r/6 + ...) by its series, of
// which only what is small is rounded
__device__ __forceinline__ Two exp_two(const Two& x) {
  if (!(x.hi > -87.f && x.hi < 88.f)) return Two{x.hi >= 88.f ? INFINITY : isnan(x.hi) ? x.hi : 0.f, 0.f};
  const float k = rintf(x.hi * kL2e);
  const Two r0 = add_two(fmaf(-k, kLn2a, x.hi), -k * kLn2b);
  const Two r = add_two(r0.hi, r0.lo + (x.lo - fmaf(k, kLn2b, -(k * kLn2b))));
  float s = 1.f / 40320.f;
  s = fmaf(s, r.hi, 1.f / 5040.f);
  s = fmaf(s, r.hi, 1.f / 720.f);
  s = fmaf(s, r.hi, 1.f / 120.f);
  s = fmaf(s, r.hi, 1.f / 24.f);
  s = fmaf(s, r.hi, 1.f / 6.f);
  s = fmaf(s, r.hi, 0.5f);
  const Two e = add_two(1.f, r.hi);
  const Two y = add_two(e.hi, fmaf(r.hi * r.hi, s, fmaf(r.hi, r.lo, r.lo)) + e.lo);
  const float p = __int_as_float((127 + (int)k) << 23);   // (k from -126 to 127)
  return Two{y.hi * p, y.lo * p};
}
// exp x to 2^-22 of itself (the instruction's), however long x is; of -inf and NaN too
__device__ __forceinline__ float exp_of(const Two& x) {
  const float y = x.hi * kL2e;
  const float lo = fmaf(x.hi, kL2e, -y) + fmaf(x.hi, 1.925963033e-8f, x.lo * kL2e);   // (log2 e's own rest)
  const float e = ex2p(y);
  return isinf(y) ? e : fmaf(e, lo * 0.69314718f, e);
}
// ln S of a sum: the power of two split off, its multiple of ln 2 in parts
__device__ __forceinline__ Two ln_two(float S) {
  if (!(S > 0.f) || isinf(S)) return Two{S == 0.f ? -INFINITY : S > 0.f ? S : NAN, 0.f};
  const int b = __float_as_int(S);
  int k = (b >> 23) - 127;   // (a sum that counts is at least 2^-126)
  float f = __int_as_float((b & 0x7FFFFF) | 0x3F800000);
  if (f > 1.41421356f) {
    f *= 0.5f;
    ++k;
  }
  const Two s = add_two((float)k * kLn2a, log1pf(f - 1.f));
  return Two{s.hi, fmaf((float)k, kLn2b, s.lo)};
}

__device__ __forceinline__ Two warp_sum(Two v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = plus(v, Two{__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  return v;
}

// A row's K tokens in shared memory.
struct RowSm {
  int id[kMaxK], bad;   // a token outside [-1, V), or one that is there twice
  float lq[kMaxK];
  Two q[kMaxK];
  float z[kMaxK];       // the row's logits there
  float mass, rest;     // the teacher's: of the tokens, and what is left
};
constexpr int kSeen = 2048;
struct SeenSm {
  uint8_t by[kSeen];    // who was the last with an id of these low bits
};
__device__ __forceinline__ bool in_vocabulary(int id, int V) { return id >= 0 && id < V; }
// kMaxK threads, a token each (barrier 1 among them).
__device__ __forceinline__ void load_teacher(RowSm& sm, SeenSm& seen, const DsArgs& a, long long row, int tid) {
  const int id = tid < a.K ? __ldg(a.ids + row * a.K + tid) : -1;
  const float lq = tid < a.K ? __ldg(a.logq + row * a.K + tid) : -INFINITY;
  if (tid == 0) sm.bad = 0;
  sm.id[tid] = id;
  const bool have = in_vocabulary(id, a.V);
  if (have) seen.by[id % kSeen] = (uint8_t)tid;
  sm.lq[tid] = have ? lq : -INFINITY;
  sm.q[tid] = exp_two(Two{have ? lq : -INFINITY, 0.f});
  asm volatile("bar.sync 1, 128;" ::: "memory");
  bool bad = id < -1 || id >= a.V;
  if (have && seen.by[id % kSeen] != tid) {   // (another one: of two equal ids one finds the other here)
    int n = 0;
    for (int j = 0; j < a.K; ++j) n += sm.id[j] == id ? 1 : 0;
    bad = n > 1;
  }
  if (bad) sm.bad = 1;
  if (tid < 32) {
    Two Q{0.f, 0.f};   // with its roundings
#pragma unroll
    for (int i = 0; i < kIdLane; ++i)
      if (i * 32 < a.K) Q = plus(Q, sm.q[i * 32 + tid]);
    Q = warp_sum(Q);
    const Two left = add_two(1.f - Q.hi, -Q.lo);   // (1 - Q.hi is exact where it matters)
    if (tid == 0) {
      sm.mass = Q.hi;
      sm.rest = left.hi > 0.f ? left.hi : left.hi <= 0.f ? 0.f : left.hi;   // (NaN stays)
    }
  }
}

// One warp's work on a row, up to four tokens per lane (its reductions need no barriers), in two parts: what the
// gradient needs, which the other blocks wait for and which takes no logarithm, then the loss.
struct Outcomes {
  float mr, mall;     // the largest logit of the rest, of the row
  float S, all;       // the sums relative to them (of this call's segments)
  float p[kIdLane], pr;
  bool nan;
};
__device__ __forceinline__ float sign(float x) { return x > 0.f ? 1.f : x < 0.f ? -1.f : x; }

// The maxima, the sums and the student's probabilities, FWD: from the segments, part; otherwise from the normalisers
// of an earlier call.
template <bool FWD>
__device__ __forceinline__ void row_sums(Outcomes& y, const RowSm& sm, const DsArgs& a, long long row,
                                         const float2* part, int nseg) {
  const int lane = (int)(threadIdx.x & 31);
  const Two inv{a.invT, a.invT_lo};
  Two ls{0.f, 0.f}, lsr{0.f, 0.f};
  if (!FWD) {
    const float4 n = __ldg((const float4*)a.norm_in + row);
    y.mall = n.x;
    ls.hi = n.y;
    y.mr = n.z;
    lsr.hi = n.w;
  }
  float z[kIdLane], e = 0.f;
#pragma unroll
  for (int i = 0; i < kIdLane; ++i)
    z[i] = i * 32 < a.K && in_vocabulary(sm.id[i * 32 + lane], a.V) ? sm.z[i * 32 + lane] : -INFINITY;
  if (FWD) {
    float m = -INFINITY, mz = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    for (int i = lane; i < nseg; i += 32) m = fmaxf(m, part[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      mz = fmaxf(mz, __shfl_xor_sync(0xffffffffu, mz, o));
    }
    y.mr = m;
    y.mall = fmaxf(m, mz);
  }
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    y.p[i] = 0.f;
    if (i * 32 >= a.K || z[i] == -INFINITY) continue;
    const Two d = scaled(z[i], y.mall, inv);
    y.p[i] = exp_of(FWD ? d : minus(d, ls));
    e += y.p[i];
  }
  const Two d = y.mr == -INFINITY ? Two{-INFINITY, 0.f} : scaled(y.mr, y.mall, inv);
  if (FWD) {
    const float s2 = kL2e * a.invT;
    float S = 0.f;
    for (int i = lane; i < nseg; i += 32) {
      const float2 p = part[i];
      // (an empty segment is left out; NaN stays)
      if (p.x != -INFINITY || isnan(p.y)) S = fmaf(p.y, ex2p((p.x - y.mr) * s2), S);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      e += __shfl_xor_sync(0xffffffffu, e, o);
    }
    const float r = y.mr == -INFINITY && !isnan(S) ? 0.f : S * exp_of(d);
    y.S = S;
    y.all = r + e;
    const float one = y.all > 0.f ? __fdividef(1.f, y.all) : y.all == 0.f ? 0.f : NAN;   // (a row without entries: p = 0)
    y.pr = r * one;
#pragma unroll
    for (int i = 0; i < kIdLane; ++i) y.p[i] *= one;
    y.nan = isnan(y.all);
  } else {
    y.pr = exp_of(plus(d, minus(lsr, ls)));
    y.S = lsr.hi;   // (its logarithm)
    y.nan = isnan(ls.hi) || isnan(lsr.hi);
  }
  y.nan |= sm.bad != 0 || isnan(sm.rest);
}

// What the gradient needs: for the rest, and at, for the lane's tokens.
template <bool FWD>
__device__ __forceinline__ RowCoef row_gradient(const Outcomes& y, const RowSm& sm, const DsArgs& a, float w,
                                                float (&at)[kIdLane]) {
  const int lane = (int)(threadIdx.x & 31);
  // t_j = p_j times the loss's derivative by p_j
  const float qr = sm.rest, tr = a.rest ? fmaf(-a.a_kl, qr, a.a_l1 * (y.pr * sign(y.pr - qr))) : 0.f;
  float t[kIdLane], M = 0.f;
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    t[i] = 0.f;
    if (i * 32 >= a.K) continue;
    const Two q = sm.q[i * 32 + lane];
    t[i] = fmaf(-a.a_kl, q.hi, a.a_l1 * (y.p[i] * sign((y.p[i] - q.hi) - q.lo)));
    M += t[i];
  }
  M = a.a_l1 == 0.f ? -a.a_kl * (a.rest ? fmaxf(sm.mass, 1.f) : sm.mass) : dspark::warp_sum(M) + tr;
  const float scale = w * a.invT;
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) at[i] = y.nan ? NAN : scale * fmaf(-y.p[i], M, t[i]);
  if (y.nan) return RowCoef{0.f, 0.f, NAN, 0.f};
  if (y.mr == -INFINITY) return RowCoef{0.f, 0.f, 0.f, 0.f};
  const float c = scale * fmaf(-y.pr, M, tr);
  return RowCoef{-y.mr, FWD ? 0.f : y.S, FWD ? __fdividef(c, y.S) : c, 0.f};
}

__device__ __forceinline__ void row_loss(const Outcomes& y, const RowSm& sm, const DsArgs& a, long long row, float w) {
  const int lane = (int)(threadIdx.x & 31);
  const Two inv{a.invT, a.invT_lo}, never{-INFINITY, 0.f};
  const Two lsr = y.mr == -INFINITY && !isnan(y.S) ? Two{0.f, 0.f} : ln_two(y.S);
  const Two ls = y.mall == -INFINITY && !isnan(y.all) ? Two{0.f, 0.f} : ln_two(y.all);
  float kl = 0.f, l1 = 0.f;
#pragma unroll
  for (int i = 0; i < kIdLane; ++i) {
    const int j = i * 32 + lane;
    if (j >= a.K || !in_vocabulary(sm.id[j], a.V)) continue;
    const Two q = sm.q[j], lp = sm.z[j] == -INFINITY ? never : minus(scaled(sm.z[j], y.mall, inv), ls);
    // (below e^-87 q counts as 0, but a token that the student rules out is no less ruled out for that)
    kl += q.hi != 0.f ? q.hi * ((sm.lq[j] - lp.hi) - lp.lo) : sm.lq[j] > -INFINITY && lp.hi == -INFINITY ? INFINITY : 0.f;
    l1 += fabsf((y.p[i] - q.hi) - q.lo);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    kl += __shfl_xor_sync(0xffffffffu, kl, o);
    l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  }
  if (lane != 0) return;
  if (a.rest) {
    const float qr = sm.rest;
    const Two lpr = y.mr == -INFINITY ? never : plus(scaled(y.mr, y.mall, inv), minus(lsr, ls));
    kl = qr != 0.f ? fmaf(qr, (logf(qr) - lpr.hi) - lpr.lo, kl) : kl;
    l1 += fabsf(y.pr - qr);
  }
  const float k = a.a_kl != 0.f ? a.a_kl * kl : 0.f, l = a.a_l1 != 0.f ? a.a_l1 * l1 : 0.f;
  if (a.loss) a.loss[row] = y.nan ? NAN : w * (k + l);
  if (a.parts) ((float2*)a.parts)[row] = y.nan ? make_float2(NAN, NAN) : make_float2(kl, l1);
  if (a.norm)
    ((float4*)a.norm)[row] = sm.bad ? make_float4(NAN, NAN, NAN, NAN)
                                    : make_float4(y.mall, ls.hi + ls.lo, y.mr, lsr.hi + lsr.lo);
}
// A padding row's outputs.
__device__ __forceinline__ void row_zero(const DsArgs& a, long long row) {
  if (a.loss) a.loss[row] = 0.f;
  if (a.parts) ((float2*)a.parts)[row] = make_float2(0.f, 0.f);
  if (a.norm) ((float4*)a.norm)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// One block per row.
template <typename T, bool FWD>
__global__ void __launch_bounds__(kMaxK) distill_rows_kernel(const T* __restrict__ logits, const DsArgs a) {
  __shared__ RowSm sm;
  __shared__ SeenSm seen;
  const long long row = blockIdx.x;
  const int tid = (int)threadIdx.x;
  const float w = a.weight ? a.weight[row] : 1.f;
  if (w == 0.f) {  // a padding row: whatever it holds
    if (tid == 0) {
      row_zero(a, row);
      if (a.coef) a.coef[row] = RowCoef{0.f, 0.f, 0.f, 0.f};
    }
    if (a.at && tid < a.K) a.at[row * a.K + tid] = 0.f;
    return;
  }
  const T* z = logits + row * a.ld;
  load_teacher(sm, seen, a, row, tid);
  if (in_vocabulary(sm.id[tid], a.V)) sm.z[tid] = to_f<T>(z[sm.id[tid]]);
  __syncthreads();
  if (tid >= 32) return;
  if (FWD) pdl_wait();
  const int nseg = (a.V + row_head(z) + kSegEntries<T> - 1) / kSegEntries<T>;
  const float2* part = a.part + row * a.nchunk * kWarps;
  Outcomes y;
  float at[kIdLane];
  row_sums<FWD>(y, sm, a, row, part, nseg);
  const RowCoef c = row_gradient<FWD>(y, sm, a, w, at);
  if (FWD) row_loss(y, sm, a, row, w);
  if (tid == 0 && sm.bad) atomicMax(&a.hdr->status, kErrInvalid);
  if (a.at) {
#pragma unroll
    for (int i = 0; i < kIdLane; ++i)
      if (i * 32 + tid < a.K) a.at[row * a.K + i * 32 + tid] = at[i];
  }
  if (a.coef && tid == 0) a.coef[row] = c;
}

// ------------------------------------------------------------------ loss and gradient of a row on the chip
// A cluster of blocks takes a row, each block a whole number of segments: the row is read once and stays in their
// shared memory.  Every block gets the segments' partial results and the row's logits at the teacher's tokens, and a
// warp of it forms what its gradient needs (sending that from one block takes another barrier); in the first block
// another warp forms the loss, which nobody waits for.
template <typename T>
__device__ __forceinline__ uint4 grad16(const uint4& q, const RowCoef& c, float s2) {
  constexpr int E = Lg<T>::E;
  float f[E];
  const F2 nm = f2(c.nm, c.nm), s22 = f2(s2, s2), ls = f2(-c.ls * kL2e, -c.ls * kL2e), cc = f2(c.c, c.c);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    const float2 y = un2(fma2(add2(Lg<T>::pair(q, e), nm), s22, ls));
    const float2 g = un2(mul2(f2(ex2p(y.x), ex2p(y.y)), cc));
    f[2 * e] = g.x;
    f[2 * e + 1] = g.y;
  }
  return pack16<T>(f);
}

__device__ __forceinline__ void st_cluster_f(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// (a load each time it is asked for, so that a segment takes no 32 registers)
__device__ __forceinline__ uint4 lds16(const uint4* p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p)));
  return v;
}

constexpr int kChipBlocks = 4;   // per SM, that registers leave room for (shared memory: three of 64 KB)
struct ChipSm {
  RowSm row;
  SeenSm seen;
  uint64_t full;
  RowCoef coef;
  float at[kMaxK];    // the gradient at the row's tokens
};

// A block's share of a row: 16-byte groups [ga, gb) of the row's, of which [wa, wb) lie whole inside it; its entries
// are [va, vb) (va < 0 in front of a row that starts inside a group).
struct Share {
  int head, ngroups, ga, gb, wa, wb, va, vb;
};
template <typename T>
__device__ __forceinline__ Share share_of(const T* z, int V, int groups, uint32_t rank) {
  constexpr int E = Lg<T>::E;
  Share s;
  s.head = row_head(z);
  s.ngroups = (V + s.head + E - 1) / E;
  s.ga = min((int)rank * groups, s.ngroups);
  s.gb = min(s.ga + groups, s.ngroups);
  s.va = s.ga * E - s.head;
  s.vb = min(s.gb * E - s.head, V);
  s.wa = s.ga + (s.va < 0 ? 1 : 0);
  s.wb = s.gb * E - s.head > V ? s.gb - 1 : s.gb;
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThr, kChipBlocks)
    distill_chip_kernel(const T* logits, T* grad, const DsArgs a, int C, int segs) {
  constexpr int E = Lg<T>::E, kGroups = 32 * kSegment;   // 16-byte groups of a segment
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ChipSm sm;
  uint4* buf = (uint4*)smem;                              // [segs][kGroups]
  float2* part = (float2*)(buf + segs * kGroups);         // [C segs]
  const uint32_t rank = cluster_rank();
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = segs * kGroups;
  const long long row = blockIdx.x / (unsigned)C;
  const T* z = logits + row * a.ld;
  T* o = grad + row * a.gld;
  const Share s = share_of(z, a.V, groups, rank);
  // whole groups by bulk copies, those at the ends of the row by entries
  if (tid == 0) {
    mbar_init(&sm.full, 1u);
    fence_mbar_init();
    const uint32_t bytes = s.wb > s.wa ? (uint32_t)(s.wb - s.wa) * 16u : 0u;
    mbar_expect_tx(&sm.full, bytes);
    const uint64_t pol = policy_evict_first();
    for (uint32_t at = 0; at < bytes; at += 16384u)
      bulk_g2s((uint8_t*)(buf + (s.wa - s.ga)) + at, (const uint8_t*)(z + (long long)s.wa * E - s.head) + at,
               min(16384u, bytes - at), &sm.full, pol);
  }
  // (no block writes to another's shared memory before that one has started)
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const float w = a.weight ? __ldg(a.weight + row) : 1.f;
  if (tid < kMaxK) load_teacher(sm.row, sm.seen, a, row, tid);
  if (tid == kThr - 32 && s.ga < s.wa) buf[0] = load16<T>(z, s.va, a.V);
  if (tid == kThr - 64 && s.wb < s.gb && s.wb >= s.wa) buf[s.wb - s.ga] = load16<T>(z, s.wb * E - s.head, a.V);
  for (int i = (s.gb - s.ga) + tid; i < groups; i += kThr) {   // behind the row
    const uint32_t f = Lg<T>::kFill;
    buf[i] = make_uint4(f, f, f, f);
  }
  __syncthreads();
  // (a wait that runs out: once more, so that nothing is in flight at the end)
  bool ok = !a.stuck && mbar_wait(&sm.full, 0u);
  if (!ok) ok = mbar_wait(&sm.full, 0u) && false;
  asm volatile("barrier.cluster.wait;" ::: "memory");
  // the row's own tokens out of the rest
  const int id = tid < kMaxK ? sm.row.id[tid] : -1;
  const bool here = id >= max(s.va, 0) && id < s.vb;
  if (here) {
    T* p = (T*)buf + (id + s.head - s.ga * E);
    const float x = ok ? to_f<T>(*p) : NAN;
    for (int c = 0; c < C; ++c) st_cluster_f(cluster_addr(&sm.row.z[tid], (uint32_t)c), x);
    *p = from_f<T>(-INFINITY);
  }
  __syncthreads();
  const float s2 = kL2e / a.T;
  for (int sg = warp; sg < segs; sg += kWarps) {
    const uint4* at = buf + sg * kGroups + lane;
    float2 p = segment_sum<T>([&](int u) { return lds16(at + u * 32); }, s2);
    if (!ok) p.y = NAN;
    if (lane < C) st_cluster_f2(cluster_addr(&part[(int)rank * segs + sg], (uint32_t)lane), p);
  }
  cluster_sync_all();
  const int nseg = (s.ngroups + kGroups - 1) / kGroups;
  if (!ok && tid == 0) atomicMax(&a.hdr->status, kErrTimeout);
  if (!grad && !(warp == 1 && rank == 0)) return;   // (the loss alone)
  if (warp == 0 || (warp == 1 && rank == 0)) {
    Outcomes y;
    if (w != 0.f) row_sums<true>(y, sm.row, a, row, part, nseg);
    if (warp == 0) {
      float at[kIdLane] = {};
      RowCoef c{0.f, 0.f, 0.f, 0.f};   // a padding row: zeros, whatever was read
      if (w != 0.f) c = row_gradient<true>(y, sm.row, a, w, at);
#pragma unroll
      for (int i = 0; i < kIdLane; ++i)
        if (i * 32 < a.K) sm.at[i * 32 + lane] = at[i];
      if (lane == 0) sm.coef = c;
    } else if (w != 0.f) {
      row_loss(y, sm.row, a, row, w);
      if (lane == 0 && sm.row.bad) atomicMax(&a.hdr->status, kErrInvalid);
    } else if (lane == 0) {
      row_zero(a, row);
    }
  }
  if (!grad) return;
  __syncthreads();
  const RowCoef c = sm.coef;
  // 16-byte groups on the output's boundaries: the buffer's own, or entries from any place of it
  const T* entries = (const T*)buf + (s.head - s.ga * E);   // entry v at [v]
  const int ohead = row_head((const T*)o), e0 = max(s.va, 0), e1 = s.vb;
  const bool same = ohead == s.head, none = c.c == 0.f;   // (zeros, whatever the entries are)
  for (int v0 = (e0 + ohead) / E * E - ohead + tid * E; v0 < e1; v0 += kThr * E) {
    const bool whole = v0 >= e0 && v0 + E <= e1;
    uint4 q;
    if (same) {
      q = *(const uint4*)(entries + v0);
    } else {
      T f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = whole || (v0 + e >= e0 && v0 + e < e1) ? entries[v0 + e] : from_f<T>(0.f);
      memcpy(&q, f, 16);
    }
    q = none ? make_uint4(0u, 0u, 0u, 0u) : grad16<T>(q, c, s2);
    if (whole) {
      __stcs((uint4*)(o + v0), q);
    } else {
      T f[E];
      memcpy(f, &q, 16);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v0 + e >= e0 && v0 + e < e1) o[v0 + e] = f[e];
    }
  }
  __syncthreads();
  if (here) o[id] = from_f<T>(sm.at[tid]);
}

constexpr int kGPer = 4;  // 16-byte groups per thread

__device__ __forceinline__ uint4 shuffle16(const uint4& q, int lane) {
  return make_uint4(__shfl_sync(0xffffffffu, q.x, lane), __shfl_sync(0xffffffffu, q.y, lane),
                    __shfl_sync(0xffffffffu, q.z, lane), __shfl_sync(0xffffffffu, q.w, lane));
}
// the 16 bytes that begin k entries into those of a, which b follows
template <typename T>
__device__ __forceinline__ uint4 shift16(const uint4& a, const uint4& b, int k) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const int words = k * (int)sizeof(T) / 4;
#pragma unroll
  for (int i = 0; i < 7; ++i) w[i] = words & 1 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = words & 2 ? w[i + 2] : w[i];
  if (sizeof(T) == 2)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (k & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// entries va .. vb - 1 of those that y holds from entry v0 on
template <typename T>
__device__ __forceinline__ void store_some(T* o, int v0, const uint4& y, int va, int vb) {
  T f[Lg<T>::E];
  memcpy(f, &y, 16);
#pragma unroll
  for (int e = 0; e < Lg<T>::E; ++e)
    if (v0 + e >= va && v0 + e < vb) o[v0 + e] = f[e];
}

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
  const RowCoef c{cf.x, cf.y, cf.z, 0.f};
  const bool none = c.c == 0.f;   // (zeros, whatever the entries are)
  const float s2 = kL2e / a.T;
#pragma unroll
  for (int u = 0; u < kGPer; ++u) q[u] = none ? make_uint4(0u, 0u, 0u, 0u) : grad16<T>(q[u], c, s2);
  // entries past a group's first at which the output's 16-byte groups begin: a lane stores from there on, with what it
  // lacks from the next lane; the ends of the warp's entries are its own (1758 x 128892 bf16 into rows of another
  // alignment: 163 us, entry by entry 500)
  const int k = (head - row_head((const T*)o)) & (E - 1);
#pragma unroll
  for (int u = 0; u < kGPer; ++u) {
    const int v0 = (g0 + u * 32 + lane) * E - head, v = v0 + k;
    uint4 y = q[u];
    bool more = true;   // whether the next lane's are there
    if (k) {
      uint4 next = shuffle16(q[u], (lane + 1) & 31);
      if (u + 1 < kGPer) {
        const uint4 x = shuffle16(q[u + 1], 0);
        if (lane == 31) next = x;
      } else {
        more = lane < 31;
      }
      y = shift16<T>(q[u], next, k);
      if (u == 0 && lane == 0) store_some(o, v0, q[0], max(v0, 0), min(v, a.V));
    }
    if (more && v >= 0 && v + E <= a.V)
      __stcs((uint4*)(o + v), y);
    else
      store_some(o, v, y, max(v, 0), min(more ? v + E : v0 + E, a.V));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kIdLane; ++i)
    if (id[i] >= first && id[i] < last && id[i] >= 0 && id[i] < a.V)
      o[id[i]] = from_f<T>(__ldcg(a.at + row * a.K + i * 32 + lane));
}

// The loss alone: one launch on the chip for up to 64 MB of logits, else two (64 x 47358 fp32 rows 7.0 us and 11.9,
// 2000 x 8000 bf16 20 and 25, 448 x 151936 fp32 63 and 50).
constexpr int kFewSegs = 16384;
// Segments of a block's share of a row: 64 KB, three blocks per SM, and as many as its shared memory holds; blocks
// of a cluster at most.
constexpr int kSegs = 16, kMostSegs = 50, kMostC = 16;
constexpr int kMostSmem = kMostSegs * 4096 + kMostC * kMostSegs * (int)sizeof(float2);

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

// How rows of nseg segments go to the chip: in clusters of C blocks of `segs` segments, of which the device holds
// `clusters` at once (0: no cluster holds them).  Bit c of `fits`: it holds clusters of c blocks too.
struct ChipShape {
  int C, segs, clusters;
  uint32_t fits;
  bool asked;
};
int segments_each(int nseg, int C) { return (nseg + C - 1) / C; }
size_t chip_smem(int C, int segs) { return (size_t)segs * 4096 + (size_t)C * segs * sizeof(float2); }
cudaLaunchConfig_t chip_config(const ChipShape& h, int clusters, cudaLaunchAttribute* at, cudaStream_t stream) {
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = (unsigned)h.C;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * h.C));
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = chip_smem(h.C, h.segs);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}
// The cluster size of which the most fit, of blocks of at most kSegs segments where 16 blocks hold the row so (a
// cluster lies inside a GPC, so the smallest size is not always it).  Asked for once for each length of row, and kept.
template <typename T>
cudaError_t chip_shape(int nseg, ChipShape* shape) {
  constexpr int kDevices = 16;   // beyond these: asked at each call
  static std::mutex mu;
  static ChipShape known[kDevices][kMostC * kMostSegs + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  ChipShape best{};
  if (dev < kDevices) best = known[dev][nseg];
  if (!best.asked) {
    auto kernel = distill_chip_kernel<T>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int least = segments_each(nseg, kSegs);
    for (int C = least < kMostC ? least : kMostC; C <= kMostC && C <= nseg; ++C) {
      ChipShape h{C, segments_each(nseg, C), 0, best.fits, false};
      cudaLaunchAttribute at{};
      const cudaLaunchConfig_t cfg = chip_config(h, 1, &at, nullptr);
      if (cudaOccupancyMaxActiveClusters(&h.clusters, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();   // a size that the device does not take
        h.clusters = 0;
      }
      if (h.clusters > 0) best.fits = h.fits |= 1u << C;
      if (h.clusters > best.clusters) best = h;
    }
    best.asked = true;
    if (dev < kDevices) known[dev][nseg] = best;
  }
  *shape = best;
  return cudaSuccess;
}

template <typename T>
cudaError_t on_chip(int N, int nseg, const T* logits, T* grad, const DsArgs& a, ChipShape h, int nsm,
                    cudaStream_t stream) {
  // few rows: blocks for every SM (a row's results do not depend on how many share it)
  for (int C = kMostC; C > h.C; --C) {
    if ((long long)C * N > nsm || !((h.fits >> C) & 1u)) continue;
    h.C = C;
    h.segs = segments_each(nseg, C);
  }
  cudaLaunchAttribute at{};
  const cudaLaunchConfig_t cfg = chip_config(h, N, &at, stream);
  return cudaLaunchKernelEx(&cfg, distill_chip_kernel<T>, logits, grad, a, h.C, h.segs);
}

template <typename T>
cudaError_t run(int N, const T* logits, T* grad, const DsArgs& a, int nsm, cudaStream_t stream) {
  const bool al_rows = ((uintptr_t)logits % 16) == 0 && (a.ld * (long long)sizeof(T)) % 16 == 0;
  cudaError_t e;
  if (a.norm_in) {
    distill_rows_kernel<T, false><<<(unsigned)N, kMaxK, 0, stream>>>(logits, a);
    e = cudaGetLastError();
  } else {
    const int nseg = (a.V + (al_rows ? 0 : Lg<T>::E - 1) + kSegEntries<T> - 1) / kSegEntries<T>;
    if ((grad || (long long)N * nseg <= kFewSegs) && nseg <= kMostC * kMostSegs) {
      ChipShape shape;
      e = chip_shape<T>(nseg, &shape);
      if (e != cudaSuccess) return e;
      if (shape.clusters > 0) return on_chip(N, nseg, logits, grad, a, shape, nsm, stream);
    }
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
                           long long gld, int stuck, void* workspace, int nsm, cudaStream_t stream) {
  const Ws s = layout(workspace, N, V, K);
  DsArgs a;
  a.V = V;
  a.K = K;
  a.nchunk = 0;
  a.rest = rest;
  a.stuck = stuck;
  a.T = T;
  a.invT = 1.f / T;
  a.invT_lo = (float)(1.0 / (double)T - (double)a.invT);
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
  return bf16 ? run<H>(N, (const H*)logits, (H*)grad, a, nsm, stream)
              : run<float>(N, (const float*)logits, (float*)grad, a, nsm, stream);
}

}  // namespace dspark
