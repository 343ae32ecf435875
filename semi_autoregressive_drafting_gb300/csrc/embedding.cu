// embedding.cu -- rows of a table for given tokens, scaled, and the table's gradient.
//
//   out[i] = scale W[t_i]  (zero for t_i = -1: padding);
//   grad_W[v] = scale sum_{i : t_i = v} grad[i].
//
// The gradient sums every token's rows in an order that the tokens alone decide.  The positions are
// sorted by token first (stable), so that a token's rows are a run of consecutive positions:
//   - up to 4096 tokens, one launch counts for every position how many precede it (all pairs);
//   - more, a stable radix sort with digits of at most 9 bits: two or three scatter launches.
// Then one launch sums slices of the sorted positions (a warp per slice and 512 bytes of columns,
// eight rows in flight) and, in other blocks, zeroes the rows of tokens that do not occur, which a
// bitmap names.  A run inside one slice is written at once; of a longer one every slice's warp leaves
// an fp32 partial sum, and the last of them to arrive (a counter per run and columns, no waits) adds
// those up in their order.
//
// Bound by HBM once the table is large: 448 tokens x 256 over 151936 rows of fp32 take 26.4 us (the 156 MB
// written, 0.87 of a copy's rate; about 5 us are the sort), 32768 bf16 rows of 2560 into 1.56 GB 272 us (0.94).
// The join in the sum launch replaced a launch of its own that took 27 us in the second case; 16-byte
// stores two apart, half a sector each, had made the zeroing take 390 us.  Over a small table the launches
// of the sort and the chain behind them bound it: 8192 x 256 fp32 over 10000 rows 26 us, of which the bytes
// need 3.  The lookup of 32768 rows of 4096 bf16 takes 64 us (5.8 TB/s), of 4095, element by element, 171.
#include "common.cuh"
#include "kernels.h"

namespace dspark {
namespace {

constexpr int kEThr = 256;
using bf16 = __nv_bfloat16;

// E consecutive elements as floats, from a 16-byte (or, for E = 1, a single-element) load
template <typename T, int E>
struct Row;
template <>
struct Row<float, 4> {
  uint4 q;
  __device__ __forceinline__ void load(const float* p) { q = __ldg((const uint4*)p); }
  __device__ __forceinline__ void get(float* f) const { Vec<float>::unpack(q, f); }
};
template <>
struct Row<bf16, 8> {
  uint4 q;
  __device__ __forceinline__ void load(const bf16* p) { q = __ldg((const uint4*)p); }
  __device__ __forceinline__ void get(float* f) const { Vec<bf16>::unpack(q, f); }
};
template <typename T>
struct Row<T, 1> {
  T x;
  __device__ __forceinline__ void load(const T* p) { x = *p; }
  __device__ __forceinline__ void get(float* f) const { f[0] = to_f<T>(x); }
};

// E floats to consecutive elements (aligned to E elements), rounded once
template <int E>
__device__ __forceinline__ void store(float* p, const float* f) {
  if (E == 1) {
    *p = f[0];
  } else if (E == 8) {  // one 32-byte store: whole sectors
    asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1 % E]),
                 "f"(f[2 % E]), "f"(f[3 % E]), "f"(f[4 % E]), "f"(f[5 % E]), "f"(f[6 % E]), "f"(f[7 % E])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) __stcs((float4*)(p + i), make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]));
  }
}
template <int E>
__device__ __forceinline__ void store(bf16* p, const float* f) {
  if (E == 1) {
    *p = __float2bfloat16_rn(f[0]);
  } else {
    uint32_t w[E / 2 > 0 ? E / 2 : 1];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      memcpy(&w[i], &b, 4);
    }
    if (E == 4) __stcs((uint2*)p, make_uint2(w[0], w[1]));
    if (E == 8) __stcs((uint4*)p, make_uint4(w[0], w[1], w[2 % (E / 2 > 0 ? E / 2 : 1)], w[3 % (E / 2 > 0 ? E / 2 : 1)]));
  }
}
template <int E>
__device__ __forceinline__ void load_out(const bf16* p, float* f) {
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = __bfloat162float(p[i]);
}

// partial sums that other blocks have written
template <int E>
__device__ __forceinline__ void load_part(const float* p, float* f) {
  if (E == 1) {
    f[0] = __ldcg(p);
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 v = __ldcg((const float4*)(p + i));
      f[i] = v.x;
      f[(i + 1) % E] = v.y;
      f[(i + 2) % E] = v.z;
      f[(i + 3) % E] = v.w;
    }
  }
}

// ------------------------------------------------------------------ lookup
constexpr int kLook = 2;  // pieces of E elements per thread (measured, 32768 x 4096 bf16: 1, 2, 4, 8: 87, 64, 68, 81 us)

template <typename TW, typename TO, int E>
__global__ void __launch_bounds__(kEThr) embed_kernel(int N, int V, int D, float scale,
                                                      const TW* __restrict__ W,
                                                      const int32_t* __restrict__ tokens,
                                                      TO* __restrict__ out) {
  const unsigned per = (unsigned)D / E;  // pieces of a row
  const unsigned long long first = (unsigned long long)blockIdx.x * (kEThr * kLook);
  const unsigned long long row0 = first / per;
  const unsigned off = (unsigned)(first - row0 * per) + threadIdx.x;
  int t[kLook];
  unsigned c[kLook];
  long long row[kLook];
#pragma unroll
  for (int u = 0; u < kLook; ++u) {
    const unsigned p = off + u * kEThr;
    row[u] = (long long)row0 + p / per;
    c[u] = (p % per) * E;
    t[u] = row[u] < N ? tokens[row[u]] : -1;
  }
  Row<TW, E> r[kLook];
#pragma unroll
  for (int u = 0; u < kLook; ++u)
    if (t[u] >= 0 && t[u] < V) r[u].load(W + (long long)t[u] * D + c[u]);
#pragma unroll
  for (int u = 0; u < kLook; ++u) {
    if (row[u] >= N) break;
    float f[E];
    if (t[u] >= 0 && t[u] < V) {
      r[u].get(f);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] *= scale;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = t[u] == -1 ? 0.f : NAN;
    }
    store<E>(out + row[u] * D + c[u], f);
  }
}

// Rows of any length and alignment: a warp per 256 elements of a row, consecutive along the lanes.
template <typename TW, typename TO>
__global__ void __launch_bounds__(kEThr) embed_any_kernel(int N, int V, int D, float scale, unsigned tiles,
                                                          const TW* __restrict__ W,
                                                          const int32_t* __restrict__ tokens,
                                                          TO* __restrict__ out) {
  const long long item = (long long)blockIdx.x * (kEThr / 32) + (threadIdx.x >> 5);
  const long long row = item / tiles;
  if (row >= N) return;
  const int c0 = (int)(item - row * tiles) * 256 + (int)(threadIdx.x & 31);
  const int t = tokens[row];
  const bool in = t >= 0 && t < V;
  const TW* w = W + (in ? (long long)t * D : 0);
  TO* o = out + row * D;
  float f[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int c = c0 + 32 * u;
    f[u] = in ? (c < D ? to_f<TW>(w[c]) : 0.f) : t == -1 ? 0.f : NAN;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int c = c0 + 32 * u;
    const float x = in ? f[u] * scale : f[u];
    if (c < D) store<1>(o + c, &x);
  }
}

template <typename TW, typename TO>
cudaError_t embed_run(int N, int V, int D, float scale, const TW* W, const int32_t* tokens, TO* out,
                      cudaStream_t stream) {
  constexpr int E = 16 / (int)sizeof(TW);
  const bool vec = D % E == 0 && ((uintptr_t)W % 16) == 0 && ((uintptr_t)out % (E * sizeof(TO))) == 0;
  if (vec) {
    const long long pieces = (long long)N * (D / E);
    const unsigned grid = (unsigned)((pieces + kEThr * kLook - 1) / (kEThr * kLook));
    embed_kernel<TW, TO, E><<<grid, kEThr, 0, stream>>>(N, V, D, scale, W, tokens, out);
  } else {
    const unsigned tiles = ((unsigned)D + 255) / 256;
    const unsigned grid = (unsigned)(((long long)N * tiles + kEThr / 32 - 1) / (kEThr / 32));
    embed_any_kernel<TW, TO><<<grid, kEThr, 0, stream>>>(N, V, D, scale, tiles, W, tokens, out);
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------ gradient: workspace
// Most tokens that are sorted by counting all pairs: measured, the whole gradient of 4000 tokens takes
// 28.8 us this way, of 8192 39.0, and 31.8 with the radix sort.
constexpr int kPairs = 4096;
constexpr int kBinBits = 9, kBins = 1 << kBinBits;
constexpr int kSortThr = 512, kSortWarps = kSortThr / 32;
constexpr int kTile = 1024;       // keys per tile of a sort block
constexpr int kSortBlocks = 64;   // most blocks of a sort launch
constexpr int kMaxSlices = 2048;
constexpr size_t kMapBytes = (1u << 24) / 8;

struct EgWs {
  WsHeader* hdr;
  unsigned* count;     // [slices][column tiles] arrivals at the run that begins in the slice
  uint32_t* map;       // bit v: token v occurs; zero between calls
  uint32_t* key[2];    // [N] sorted tokens
  uint32_t* pos[2];    // [N] their positions
  unsigned* hist[2];   // [kSortBlocks][kBins]
  float* part;         // [slices][2][D]
};

constexpr size_t eg_align(size_t x) { return (x + 255) / 256 * 256; }

// positions per slice: 32, more once there would be over kMaxSlices of them
int slice_len(int N) { return 32 * ((N + 32 * kMaxSlices - 1) / (32 * kMaxSlices)); }
size_t slice_room(int N) {
  const size_t s = ((size_t)N + 31) / 32;
  return s < (size_t)kMaxSlices ? s : (size_t)kMaxSlices;
}

size_t eg_layout(int N, int D, uint8_t* base, EgWs* ws) {
  size_t o = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += eg_align(bytes);
    return base + at;
  };
  EgWs w;
  w.hdr = (WsHeader*)base;
  w.map = (uint32_t*)take(kMapBytes);  // (one size and place for every V: it stays clear)
  w.count = (unsigned*)take(slice_room(N) * (((size_t)D + 31) / 32) * 4);
  for (int i = 0; i < 2; ++i) {
    w.key[i] = (uint32_t*)take((size_t)N * 4);
    w.pos[i] = (uint32_t*)take((size_t)N * 4);
    w.hist[i] = (unsigned*)take((size_t)kSortBlocks * kBins * 4);
  }
  w.part = (float*)take(slice_room(N) * 2 * (size_t)D * 4);
  if (ws) *ws = w;
  return o;
}

// the sort key of a position: its token, or V (after every token) for padding and invalid tokens
__device__ __forceinline__ uint32_t key_of(int t, int V, unsigned* status) {
  if (t >= 0 && t < V) return (uint32_t)t;
  if (t != -1) atomicMax(status, kErrInvalid);
  return (uint32_t)V;
}

// ------------------------------------------------------------------ sort, few tokens
// A block ranks 32 positions, one per lane; its warps share out the positions compared with.
__global__ void __launch_bounds__(kEThr) pairs_kernel(int N, int V, const int32_t* __restrict__ tokens,
                                                      int mark, int ncount, EgWs ws) {
  __shared__ __align__(16) uint32_t key[kPairs];
  __shared__ int cnt[kEThr / 32][32];
  pdl_trigger();
  const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
  const int n4 = (N + 3) & ~3;
  for (int i = threadIdx.x; i < n4; i += kEThr)
    key[i] = i < N ? key_of(tokens[i], V, &ws.hdr->status) : 0xFFFFFFFFu;  // (larger than any)
  for (int i = (int)(blockIdx.x * kEThr + threadIdx.x); i < ncount; i += (int)gridDim.x * kEThr) ws.count[i] = 0u;
  __syncthreads();
  const int i0 = (int)blockIdx.x * 32, i = i0 + lane;
  const uint32_t k = i < N ? key[i] : 0u;
  const int per = ((n4 / 4 + kEThr / 32 - 1) / (kEThr / 32)) * 4;
  const int ja = min(n4, warp * per), jb = min(n4, ja + per);
  int c = 0;
  // before the block's own positions an equal token precedes, after them it does not
  const int je = min(jb, max(ja, i0)), jl = min(jb, max(ja, i0 + 32));
  for (int j = ja; j < je; j += 4) {
    const uint4 q = *(const uint4*)(key + j);
    c += (q.x <= k) + (q.y <= k) + (q.z <= k) + (q.w <= k);
  }
  for (int j = je; j < jl; ++j) c += key[j] < k || (key[j] == k && j < i);
  for (int j = jl; j < jb; j += 4) {
    const uint4 q = *(const uint4*)(key + j);
    c += (q.x < k) + (q.y < k) + (q.z < k) + (q.w < k);
  }
  cnt[warp][lane] = c;
  __syncthreads();
  if (warp == 0 && i < N) {
    for (int w = 1; w < kEThr / 32; ++w) c += cnt[w][lane];
    ws.key[0][c] = k;
    ws.pos[0][c] = (uint32_t)i;
    if (mark && k < (uint32_t)V) atomicOr(&ws.map[k >> 5], 1u << (k & 31));
  }
}

// ------------------------------------------------------------------ sort, many tokens
// Digit counts of every block's share of the tokens (the first pass; later passes' counts are made
// by the scatter before them).
__global__ void __launch_bounds__(kSortThr) count_kernel(int N, int V, int per_block, int bits,
                                                         const int32_t* __restrict__ tokens, int mark,
                                                         int ncount, EgWs ws) {
  __shared__ unsigned h[kBins];
  pdl_trigger();
  for (int b = threadIdx.x; b < kBins; b += kSortThr) {
    h[b] = 0u;
    ws.hist[1][blockIdx.x * kBins + b] = 0u;
  }
  for (int i = (int)(blockIdx.x * kSortThr + threadIdx.x); i < ncount; i += (int)gridDim.x * kSortThr) ws.count[i] = 0u;
  __syncthreads();
  const int i1 = min((long long)N, (long long)(blockIdx.x + 1) * per_block);
  for (int i = (int)blockIdx.x * per_block + (int)threadIdx.x; i < i1; i += kSortThr) {
    const uint32_t k = key_of(tokens[i], V, &ws.hdr->status);
    atomicAdd(&h[k & ((1u << bits) - 1u)], 1u);
    if (mark && k < (uint32_t)V) atomicOr(&ws.map[k >> 5], 1u << (k & 31));
  }
  __syncthreads();
  for (int b = threadIdx.x; b < kBins; b += kSortThr) ws.hist[0][blockIdx.x * kBins + b] = h[b];
}

// One stable pass: block b moves its share of the keys to where their digit's keys go, after those
// of the blocks before it.  The first pass reads the tokens (key_in null); every pass but the last
// counts the next digit of the keys at their new places.
__global__ void __launch_bounds__(kSortThr) scatter_kernel(int N, int V, int per_block, int shift, int bits,
                                                           int last, const int32_t* __restrict__ tokens,
                                                           const uint32_t* __restrict__ key_in,
                                                           const uint32_t* __restrict__ pos_in,
                                                           const unsigned* __restrict__ hist,
                                                           unsigned* __restrict__ next,
                                                           uint32_t* __restrict__ key_out,
                                                           uint32_t* __restrict__ pos_out) {
  __shared__ unsigned cnt[kSortWarps][kBins];
  __shared__ unsigned base[kBins];
  __shared__ unsigned wsum[kSortWarps];
  const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = (int)gridDim.x;
  pdl_trigger();
  pdl_wait();
  {  // base[d]: keys of lower digits, and of this digit in the blocks before
    unsigned below = 0u, all = 0u;
#pragma unroll 8
    for (int b = 0; b < nb; ++b) {
      const unsigned h = hist[b * kBins + tid];
      all += h;
      below += b < (int)blockIdx.x ? h : 0u;
    }
    unsigned inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned w0 = 0u;
    for (int w = 0; w < warp; ++w) w0 += wsum[w];
    base[tid] = w0 + inc - all + below;
  }
  const uint32_t mask = (1u << bits) - 1u;
  const long long i1 = min((long long)N, (long long)(blockIdx.x + 1) * per_block);
  for (long long t0 = (long long)blockIdx.x * per_block; t0 < i1; t0 += kTile) {
    for (int j = tid; j < kSortWarps * kBins; j += kSortThr) (&cnt[0][0])[j] = 0u;
    __syncthreads();
    uint32_t k[kTile / kSortThr], r[kTile / kSortThr];
#pragma unroll
    for (int u = 0; u < kTile / kSortThr; ++u) {  // the warp's 128 keys, 32 consecutive ones at a time
      const long long i = t0 + warp * (kTile / kSortWarps) + u * 32 + lane;
      const bool in = i < i1;
      k[u] = !in ? 0xFFFFFFFFu : tokens ? (tokens[i] >= 0 && tokens[i] < V ? (uint32_t)tokens[i] : (uint32_t)V) : key_in[i];
      const uint32_t d = in ? (k[u] >> shift) & mask : kBins;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const unsigned before = __popc(same & ((1u << lane) - 1u));
      r[u] = in ? cnt[warp][d] + before : 0u;
      __syncwarp();
      if (in && before == 0u) cnt[warp][d] += (unsigned)__popc(same);
      __syncwarp();
    }
    __syncthreads();
    {
      unsigned b = base[tid];
      for (int w = 0; w < kSortWarps; ++w) {
        const unsigned c = cnt[w][tid];
        cnt[w][tid] = b;
        b += c;
      }
      base[tid] = b;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTile / kSortThr; ++u) {
      const long long i = t0 + warp * (kTile / kSortWarps) + u * 32 + lane;
      if (i < i1) {
        const unsigned p = cnt[warp][(k[u] >> shift) & mask] + r[u];
        key_out[p] = k[u];
        pos_out[p] = pos_in ? pos_in[i] : (uint32_t)i;
        if (!last) atomicAdd(&next[(p / (unsigned)per_block) * kBins + ((k[u] >> (shift + bits)) & mask)], 1u);
      }
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kSortThr) clear_kernel(unsigned* __restrict__ h) {
  pdl_trigger();
  pdl_wait();
  h[blockIdx.x * kBins + threadIdx.x] = 0u;
}

// ------------------------------------------------------------------ sums
constexpr int kAhead = 8;  // rows in flight per warp

struct SumArgs {
  int N, V, D, plen, nslice, ntile;  // positions per slice, slices, column tiles of 32 E
  float scale;
  int accumulate;
  int fill_blocks;                   // blocks that zero absent rows (they come after the others)
  const uint32_t *key, *pos;
  EgWs ws;
};

// A finished row.  Added to the output, it is added by the memory (fp32), so that no warp waits for what
// is there (448 tokens x 64: 12.4 us, 18.6 by load and store); each element gets one addition, so its order
// is not in question.  The memory's additions take subnormal numbers, and leave them, as zero.
template <int E>
__device__ __forceinline__ void add_out(float* o, const float* f) {
  if (E == 1) {
    asm volatile("red.global.add.f32 [%0], %1;" ::"l"(o), "f"(f[0]) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(o + i), "f"(f[i]), "f"(f[(i + 1) % E]),
                   "f"(f[(i + 2) % E]), "f"(f[(i + 3) % E])
                   : "memory");
  }
}
template <int E>
__device__ __forceinline__ void add_out(bf16* o, const float* f) {
  float g[E];
  load_out<E>(o, g);
#pragma unroll
  for (int e = 0; e < E; ++e) g[e] += f[e];
  store<E>(o, g);
}

template <typename TO, int E>
__device__ __forceinline__ void put_row(TO* o, const float* s, float scale, int accumulate) {
  float f[E];
#pragma unroll
  for (int e = 0; e < E; ++e) f[e] = scale * s[e];
  if (accumulate)
    add_out<E>(o, f);
  else
    store<E>(o, f);
}

// One slice's part of a run that crosses slices has been stored (part 1 of the slice in which it
// begins, part 0 of the others).  The last warp to arrive adds the parts up in their order.
template <typename TO, int E>
__device__ __noinline__ void join(const SumArgs& a, TO* gW, uint32_t k, int slice, bool begun, int tile,
                                  int lane, int col, bool live) {
  int s0 = slice, s1 = slice;  // the slices in which the run begins and ends
  if (!begun) {
    for (s0 = slice - 1;; s0 -= 32) {
      const int t = s0 - lane;  // does the run go on from slice t - 1 into t?
      const unsigned in = __ballot_sync(0xffffffffu, t >= 1 && a.key[(long long)t * a.plen - 1] == k);
      if (in != 0xffffffffu) {
        s0 -= __ffs(~in) - 1;
        break;
      }
    }
  }
  for (;; s1 += 32) {
    const int t = s1 + 1 + lane;
    const unsigned in = __ballot_sync(0xffffffffu, t < a.nslice && a.key[(long long)t * a.plen] == k);
    if (in != 0xffffffffu) {
      s1 += __ffs(~in) - 1;
      break;
    }
  }
  __threadfence();
  __syncwarp();
  unsigned last = 0u;
  if (lane == 0) last = atomicAdd(&a.ws.count[(long long)s0 * a.ntile + tile], 1u) == (unsigned)(s1 - s0);
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  if (!live) return;
  float s[E] = {};
  for (int c = s0; c <= s1; c += kAhead) {
    float f[kAhead][E];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (c + j <= s1) load_part<E>(a.ws.part + ((long long)(c + j) * 2 + (c + j == s0 ? 1 : 0)) * a.D + col, f[j]);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (c + j <= s1) {
#pragma unroll
        for (int e = 0; e < E; ++e) s[e] += f[j][e];
      }
  }
  put_row<TO, E>(gW + (long long)k * a.D + col, s, a.scale, a.accumulate);
}

template <typename TG, typename TO, int E>
__global__ void __launch_bounds__(kEThr) sum_kernel(const SumArgs a, const TG* __restrict__ grad,
                                                    TO* __restrict__ gW) {
  const int lane = (int)(threadIdx.x & 31);
  const int sum_blocks = (int)gridDim.x - a.fill_blocks;
  pdl_wait();
  if ((int)blockIdx.x >= sum_blocks) {  // zero the rows of absent tokens, 32 rows at a time
    const int words = (a.V + 31) / 32;
    const unsigned per = (unsigned)a.D / E;
    for (int w = (int)blockIdx.x - sum_blocks; w < words; w += a.fill_blocks) {
      const uint32_t m = a.ws.map[w];
      const unsigned rows = (unsigned)min(32, a.V - 32 * w);
      TO* o = gW + (long long)w * 32 * a.D;
      const float zero[E] = {};
      unsigned r = threadIdx.x / per, c = threadIdx.x % per;
      const unsigned dr = kEThr / per, dc = kEThr % per;
      while (r < rows) {
        if (!((m >> r) & 1u)) store<E>(o + (long long)r * a.D + (long long)c * E, zero);
        r += dr;
        c += dc;
        if (c >= per) {
          c -= per;
          ++r;
        }
      }
      __syncthreads();
      if (threadIdx.x == 0 && m) a.ws.map[w] = 0u;
    }
    return;
  }
  const long long unit = (long long)blockIdx.x * (kEThr / 32) + (threadIdx.x >> 5);
  const int slice = (int)(unit / a.ntile), tile = (int)(unit % a.ntile);
  if (slice >= a.nslice) return;
  const long long p0 = (long long)slice * a.plen, p1 = min((long long)a.N, p0 + a.plen);
  const int col = (tile * 32 + lane) * E;
  const bool live = col < a.D;
  const uint32_t none = (uint32_t)a.V;
  const uint32_t before = p0 > 0 ? a.key[p0 - 1] : 0xFFFFFFFFu;
  const uint32_t after = p1 < a.N ? a.key[p1] : 0xFFFFFFFFu;
  uint32_t cur = a.key[p0];
  bool begun = cur != before;  // the current run begins in this slice
  uint32_t crossed = none;     // the run that came from the slice before, once it has ended
  float s[E] = {};
  for (long long b = p0; b < p1; b += 32) {
    const int n = (int)min(32ll, p1 - b);
    const uint32_t kl = lane < n ? a.key[b + lane] : none, pl = lane < n ? a.pos[b + lane] : 0u;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      Row<TG, E> r[kAhead];
      uint32_t k[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        k[j] = __shfl_sync(0xffffffffu, kl, (i0 + j) & 31);
        const uint32_t p = __shfl_sync(0xffffffffu, pl, (i0 + j) & 31);
        if (i0 + j >= n) k[j] = none;
        if (k[j] != none && live) r[j].load(grad + (long long)p * a.D + col);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (k[j] == none) continue;  // padding sorts last
        if (k[j] != cur) {
          if (live) {
            if (begun)
              put_row<TO, E>(gW + (long long)cur * a.D + col, s, a.scale, a.accumulate);
            else
              store<E>(a.ws.part + (long long)slice * 2 * a.D + col, s);
          }
          if (!begun) crossed = cur;
          cur = k[j];
          begun = true;
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] = 0.f;
        }
        if (live) {
          float f[E];
          r[j].get(f);
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] += f[e];
        }
      }
    }
  }
  if (crossed != none) join<TO, E>(a, gW, crossed, slice, false, tile, lane, col, live);
  if (cur == none) return;
  if (begun && cur != after) {
    if (live) put_row<TO, E>(gW + (long long)cur * a.D + col, s, a.scale, a.accumulate);
    return;
  }
  if (live) store<E>(a.ws.part + ((long long)slice * 2 + (begun ? 1 : 0)) * a.D + col, s);
  join<TO, E>(a, gW, cur, slice, begun, tile, lane, col, live);
}

template <typename TG, typename TO, int E>
cudaError_t sums(SumArgs a, const TG* grad, TO* gW, cudaStream_t stream) {
  const int words = (a.V + 31) / 32;
  a.fill_blocks = a.accumulate ? 0 : words < 16384 ? words : 16384;
  const long long warps = (long long)a.nslice * a.ntile;
  const unsigned grid = (unsigned)((warps + kEThr / 32 - 1) / (kEThr / 32)) + (unsigned)a.fill_blocks;
  if (grid == 0) return cudaSuccess;
  return launch_pdl(sum_kernel<TG, TO, E>, grid, kEThr, 0, stream, a, grad, gW);
}

template <typename TG, typename TO>
cudaError_t sums_by_shape(const SumArgs& a, bool vec, const TG* grad, TO* gW, cudaStream_t stream) {
  return vec ? sums<TG, TO, 16 / (int)sizeof(TG)>(a, grad, gW, stream) : sums<TG, TO, 1>(a, grad, gW, stream);
}

}  // namespace

cudaError_t launch_embedding(int N, int V, int D, float scale, int w_bf16, const void* W,
                             const int32_t* tokens, int o_bf16, void* out, cudaStream_t stream) {
  if (w_bf16 && o_bf16) return embed_run(N, V, D, scale, (const bf16*)W, tokens, (bf16*)out, stream);
  if (w_bf16) return embed_run(N, V, D, scale, (const bf16*)W, tokens, (float*)out, stream);
  if (o_bf16) return embed_run(N, V, D, scale, (const float*)W, tokens, (bf16*)out, stream);
  return embed_run(N, V, D, scale, (const float*)W, tokens, (float*)out, stream);
}

size_t embedding_grad_workspace_bytes(int N, int, int D) { return eg_layout(N, D, nullptr, nullptr); }

cudaError_t launch_embedding_grad(int N, int V, int D, float scale, int g_bf16, const void* grad,
                                  const int32_t* tokens, int o_bf16, void* gW, int accumulate,
                                  void* workspace, cudaStream_t stream) {
  SumArgs a;
  eg_layout(N, D, (uint8_t*)workspace, &a.ws);
  a.N = N;
  a.V = V;
  a.D = D;
  a.scale = scale;
  a.accumulate = accumulate;
  a.plen = N > 0 ? slice_len(N) : 32;
  a.nslice = (int)(((long long)N + a.plen - 1) / a.plen);
  const int E = g_bf16 ? 8 : 4;
  const bool vec = D % E == 0 && ((uintptr_t)grad % 16) == 0 && ((uintptr_t)gW % 32) == 0;
  a.ntile = vec ? (D / E + 31) / 32 : (D + 31) / 32;
  const int mark = !accumulate, ncount = a.nslice * a.ntile;
  cudaError_t e = cudaSuccess;
  int at = 0;
  if (N > 0 && N <= kPairs) {
    pairs_kernel<<<(N + 31) / 32, kEThr, 0, stream>>>(N, V, tokens, mark, ncount, a.ws);
    e = cudaGetLastError();
  } else if (N > 0) {
    int bits = 1;  // keys are 0 .. V
    while ((1 << bits) <= V) ++bits;
    const int passes = (bits + kBinBits - 1) / kBinBits, digit = (bits + passes - 1) / passes;
    const int tiles = (N + kTile - 1) / kTile;
    const int nb0 = tiles < kSortBlocks ? tiles : kSortBlocks;
    const int per_block = (tiles + nb0 - 1) / nb0 * kTile;
    const int nb = (N + per_block - 1) / per_block;
    count_kernel<<<nb, kSortThr, 0, stream>>>(N, V, per_block, digit, tokens, mark, ncount, a.ws);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    for (int p = 0; p < passes; ++p) {
      const int last = p == passes - 1;
      if (p >= 1 && !last) {  // (three passes: the counts of the first digit make room for the third's)
        if ((e = launch_pdl(clear_kernel, nb, kSortThr, 0, stream, a.ws.hist[(p + 1) & 1])) != cudaSuccess) return e;
      }
      if ((e = launch_pdl(scatter_kernel, nb, kSortThr, 0, stream, N, V, per_block, p * digit, digit, last,
                          p == 0 ? tokens : nullptr, p ? a.ws.key[(p + 1) & 1] : nullptr,
                          p ? a.ws.pos[(p + 1) & 1] : nullptr, a.ws.hist[p & 1], a.ws.hist[(p + 1) & 1],
                          a.ws.key[p & 1], a.ws.pos[p & 1])) != cudaSuccess)
        return e;
      at = p & 1;
    }
  }
  if (e != cudaSuccess) return e;
  a.key = a.ws.key[at];
  a.pos = a.ws.pos[at];
  if (g_bf16 && o_bf16) return sums_by_shape(a, vec, (const bf16*)grad, (bf16*)gW, stream);
  if (g_bf16) return sums_by_shape(a, vec, (const bf16*)grad, (float*)gW, stream);
  if (o_bf16) return sums_by_shape(a, vec, (const float*)grad, (bf16*)gW, stream);
  return sums_by_shape(a, vec, (const float*)grad, (float*)gW, stream);
}

}  // namespace dspark
