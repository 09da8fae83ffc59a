// Blocks of a cache (include/blocks.h): bounds of their keys and the selection of
// blocks for each query.  The attention over them is the decode kernels' (decode.cu,
// decode_e2m1.cu).
//
// Bounds: one warp per (full block, KV head) reads the block's keys, 16 bytes per
// lane, and keeps the minimum and maximum of 8 components in registers.  Bound by HBM.
//
// Selection, with the group's heads h and a block's bounds lo, hi:
//   score = sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d M_d lo_d + P_d hi_d,
//   M_d = sum_h min(q_hd, 0), P_d = sum_h max(q_hd, 0):
// one dot product of 2 D terms per block and KV head, however many heads the group
// has, and it is bound by reading the bounds (4 D bytes).  A list must not depend on the
// order of fp32 sums, so a kernel takes the scores in fp32 with a bound on
// their error, and a second one decides: a threshold t with K scores above it, E the largest
// bound; a score above t + 2 E belongs to the K largest whatever the errors
// are, one below t - 2 E does not, and only those between are summed again in fp64.
// (At least K exact scores are >= t - E and fewer than K of the others exceed t + E.)
#include "kernels.cuh"
#include "kv_read.cuh"
#include "../../include/blocks.h"

namespace gb300 {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // NaN if either is
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

struct BlocksPar {
  uint16_t* bounds;          // [num_rows, Hkv, 2, D]
  int64_t num_rows;
  const int64_t* row_base;   // contiguous cache
  int32_t log2_bs;
  int32_t Hkv, B;
  const int32_t* cu_seqlens; // NULL: one token per request
  KvIndex kv;
  int32_t* status;
  // bounds
  const int32_t* start;      // NULL: cache_lens
  const void* k_cache;
  const uint8_t* k_block_scale;
  float k_scale;
  int32_t ctas_per_request;
  // selection
  const uint16_t* q;         // [N, Hq, D]
  int32_t q_f16, N, G, first, last, keep, max_blocks, chunk, chunks;
  float2* scores;            // [N, Hkv, max_blocks]: score, bound on its error
  int32_t* list;             // [N, Hkv, keep]
};

// Row of the bounds of block i of a request, or -1 (a page outside the cache, a row
// outside the bounds).
__device__ __forceinline__ int64_t bounds_row(const BlocksPar& p, const ReqInfo& r, int b, int i) {
  int64_t row;
  if (r.pages) {
    const int64_t slot = cache_slot(p.kv, r, i << p.log2_bs);
    row = slot < 0 ? -1 : slot >> p.log2_bs;
  } else {
    row = __ldg(p.row_base + b) + i;
  }
  return row < p.num_rows ? row : -1;
}

// ---------------------------------------------------------------- bounds
template <int D, int KV>
__global__ void __launch_bounds__(kThreads) block_bounds_kernel(const BlocksPar p) {
  constexpr int L = D / 8, KPW = 32 / L;  // lanes per key, keys per warp and step
  const int b = blockIdx.x / p.ctas_per_request, part = blockIdx.x % p.ctas_per_request;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launch_dependents();
  grid_dependency_wait();  // the appended entries, the lengths
  int n = 1;
  if (p.cu_seqlens) n = __ldg(p.cu_seqlens + b + 1) - __ldg(p.cu_seqlens + b);
  const ReqInfo r = load_request(p.kv, b, n);
  if (!r.valid) {
    if (part == 0 && threadIdx.x == 0) set_status(p.status, n < 0 ? ATTN_STATUS_SEQLENS : ATTN_STATUS_CAPACITY);
    return;
  }
  const int from = max(p.start ? __ldg(p.start + b) : r.cached, 0) >> p.log2_bs;
  const int64_t items = (int64_t)(((r.cached + n) >> p.log2_bs) - from) * p.Hkv;
  const int li = lane % L, sub = lane / L;
  for (int64_t it = (int64_t)part * kWarps + warp; it < items; it += (int64_t)p.ctas_per_request * kWarps) {
    const int i = from + (int)(it / p.Hkv), kh = (int)(it % p.Hkv);
    const int64_t slot = cache_slot(p.kv, r, i << p.log2_bs);
    const int64_t row = bounds_row(p, r, b, i);
    if ((slot < 0 || row < 0) && lane == 0) set_status(p.status, ATTN_STATUS_CAPACITY);
    if (row < 0) continue;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (slot >= 0) {
      auto key = [&](int k) {
        return read8<KV>(p.k_cache, p.k_block_scale, p.k_scale, p.kv.num_slots, slot + k, p.Hkv, kh, li, D == 128 ? 4 : 3);
      };
      lo = hi = key(sub);
      const int bs = 1 << p.log2_bs;
#pragma unroll 8
      for (int k = sub + KPW; k < bs; k += KPW) {
        const uint4 x = key(k);
        lo = make_uint4(min2(lo.x, x.x), min2(lo.y, x.y), min2(lo.z, x.z), min2(lo.w, x.w));
        hi = make_uint4(max2(hi.x, x.x), max2(hi.y, x.y), max2(hi.z, x.z), max2(hi.w, x.w));
      }
#pragma unroll
      for (int off = L; off < 32; off <<= 1) {
        auto other = [&](uint32_t v) { return __shfl_xor_sync(0xffffffffu, v, off); };
        lo = make_uint4(min2(lo.x, other(lo.x)), min2(lo.y, other(lo.y)), min2(lo.z, other(lo.z)), min2(lo.w, other(lo.w)));
        hi = make_uint4(max2(hi.x, other(hi.x)), max2(hi.y, other(hi.y)), max2(hi.z, other(hi.z)), max2(hi.w, other(hi.w)));
      }
    }
    if (lane < 2 * L) {
      uint4* dst = reinterpret_cast<uint4*>(p.bounds + (row * p.Hkv + kh) * (2 * D));
      dst[lane] = lane < L ? lo : hi;  // lanes L .. 2 L - 1: component run lane - L, as in lane % L
    }
  }
}

// ---------------------------------------------------------------- scores
__device__ __forceinline__ float q_value(uint32_t bits, int f16) {
  return f16 ? __half2float(__ushort_as_half((uint16_t)bits)) : __uint_as_float(bits << 16);
}

// How many blocks a query sees, 0 if it gets no list; `report`: this thread sets the status.
__device__ __forceinline__ int query_blocks(const BlocksPar& p, int t, ReqInfo* r, int* b, bool report) {
  int n, j;
  if (!find_token(p.cu_seqlens, p.B, t, b, &n, &j)) {
    if (report) set_status(p.status, ATTN_STATUS_SEQLENS);
    return 0;
  }
  *r = load_request(p.kv, *b, n);
  if (!r->valid) {
    if (report) set_status(p.status, ATTN_STATUS_CAPACITY);
    return 0;
  }
  const int blocks = ((r->cached + j) >> p.log2_bs) + 1;
  if (blocks > p.max_blocks) {
    if (report) set_status(p.status, ATTN_STATUS_BOUNDS);
    return 0;
  }
  return blocks;
}

// Rounding of a score: each term goes through at most 7 additions in M or P, 8 in its
// lane's chain and 5 between lanes, 20 half steps of its magnitude; the sum of magnitudes is
// rounded likewise.  What products below the normal range lose is less than the constant.
constexpr float kErrorOfMagnitude = 24.f * 5.9604645e-8f;
constexpr float kErrorFloor = 1e-40f;

// A warp takes 8 blocks at a time: lane l of the D / 4 lanes of a block holds 8
// components of lo (the first half of the lanes) or hi.
template <int D>
__global__ void __launch_bounds__(kThreads) block_score_kernel(const BlocksPar p) {
  constexpr int L = D / 4, BPW = 32 / L;  // lanes per block, blocks per warp and load
  __shared__ float coef[2 * D];           // M, P
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kh = blockIdx.x / p.chunks % p.Hkv, t = blockIdx.x / p.chunks / p.Hkv, c = blockIdx.x % p.chunks;
  launch_dependents();
  grid_dependency_wait();
  ReqInfo r;
  int b;
  const int n = query_blocks(p, t, &r, &b, c == 0 && kh == 0 && threadIdx.x == 0);
  const int i0 = p.first + c * p.chunk, i1 = min(i0 + p.chunk, n - p.last);
  if (n <= p.keep || i0 >= i1) return;
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float m = 0.f, q = 0.f;
    for (int h = 0; h < p.G; ++h) {
      const float x = q_value(__ldg(p.q + ((int64_t)t * p.Hkv * p.G + kh * p.G + h) * D + d), p.q_f16);
      // a NaN enters both
      m += x > 0.f ? 0.f : x;
      q += x < 0.f ? 0.f : x;
    }
    coef[d] = m;
    coef[D + d] = q;
  }
  __syncthreads();
  const int li = lane % L, sub = lane / L;
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = coef[8 * li + e];
  float2* out = p.scores + ((int64_t)t * p.Hkv + kh) * p.max_blocks;
  bool outside = false;
  for (int i = i0 + warp * 8 * BPW; i < i1; i += kWarps * 8 * BPW) {
    // rows of the warp's 8 * BPW blocks, one per lane
    int64_t row = -1;
    if (lane < 8 * BPW && i + lane < i1) {
      row = bounds_row(p, r, b, i + lane);
      outside |= row < 0;
    }
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t rk = __shfl_sync(0xffffffffu, row, k * BPW + sub);
      x[k] = rk < 0 ? make_uint4(0, 0, 0, 0)
                    : __ldg(reinterpret_cast<const uint4*>(p.bounds + (rk * p.Hkv + kh) * (2 * D)) + li);
    }
    float s[8], a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float y[8];
      unpack_bf16x8(x[k], y);
      s[k] = w[0] * y[0];
      a[k] = fabsf(s[k]);
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        s[k] = fmaf(w[e], y[e], s[k]);
        a[k] = fmaf(fabsf(w[e]), fabsf(y[e]), a[k]);
      }
    }
    // sums over the block's lanes; of the 8 values each lane keeps the one of its bits 0 .. 2
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
      const bool up = lane & half;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        const float give_s = up ? s[k] : s[k + half], give_a = up ? a[k] : a[k + half];
        s[k] = (up ? s[k + half] : s[k]) + __shfl_xor_sync(0xffffffffu, give_s, half);
        a[k] = (up ? a[k + half] : a[k]) + __shfl_xor_sync(0xffffffffu, give_a, half);
      }
    }
#pragma unroll
    for (int off = 8; off < L; off <<= 1) {
      s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], off);
    }
    const int at = i + (lane & 7) * BPW + sub;
    if (li < 8 && at < i1) out[at] = make_float2(s[0], fmaf(a[0], kErrorOfMagnitude, kErrorFloor));
  }
  if (outside) set_status(p.status, ATTN_STATUS_CAPACITY);
}

// ---------------------------------------------------------------- selection
// Larger float -> larger key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The same in 64 bits; -0 as 0, and NaN above all.
__device__ __forceinline__ unsigned long long order_key64(double x) {
  if (!(x == x)) return ~0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr int kHeld = 8;       // scores held in registers per thread: up to 2048 candidates
constexpr int kMaxOpen = 256;  // candidates summed again and ranked in shared memory

// The sum over the CTA of one count per thread: alternating buffers, one barrier.
struct Counter {
  int (*part)[kWarps];  // [2][kWarps]
  int turn = 0;
  __device__ __forceinline__ int operator()(int mine) {
    const int s = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = s;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += part[turn][w];
    turn ^= 1;
    return sum;
  }
};

// Score of a block in fp64, summed by one warp in the same order for every block.
template <int D>
__device__ __forceinline__ double exact_score(const BlocksPar& p, const ReqInfo& r, int b, int kh, int i,
                                              const double* coef, int lane) {
  const int64_t row = bounds_row(p, r, b, i);
  double s = 0.0;
  if (row >= 0 && lane < D / 4) {
    float y[8];
    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p.bounds + (row * p.Hkv + kh) * (2 * D)) + lane), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma(coef[8 * lane + e], (double)y[e], s);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// One CTA per list.
template <int D>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const BlocksPar p) {
  extern __shared__ uint32_t bits[];  // candidate i is selected: bit i % 32 of word i / 32
  __shared__ int part[2][kWarps];
  __shared__ double coef[2 * D];
  __shared__ int open_idx[kMaxOpen];
  __shared__ unsigned long long open_key[kMaxOpen];
  __shared__ int open_n, odd;
  __shared__ float red[3][kWarps];
  const int t = blockIdx.x / p.Hkv, kh = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  grid_dependency_wait();
  ReqInfo r;
  int b;
  const int n = query_blocks(p, t, &r, &b, false);
  if (n == 0) return;
  int32_t* list = p.list + ((int64_t)t * p.Hkv + kh) * p.keep;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kThreads) list[i] = i < n ? i : -1;
    return;
  }
  const int m = n - p.first - p.last, K = p.keep - p.first - p.last;
  for (int i = tid; i < p.first; i += kThreads) list[i] = i;
  for (int i = tid; i < p.last; i += kThreads) list[p.keep - p.last + i] = n - p.last + i;
  if (K == 0) return;
  float2* scores = p.scores + ((int64_t)t * p.Hkv + kh) * p.max_blocks + p.first;

  // the largest error bound, the range of the keys, and whether anything is not finite
  uint32_t key[kHeld];
  const bool held = m <= kHeld * kThreads;
  float err = 0.f;
  uint32_t kmin = ~0u, kmax = 0u;
  bool bad = false;
  auto look = [&](float2 v) {
    bad |= !(fabsf(v.x) <= 3.4028235e38f && v.y <= 3.4028235e38f);
    err = fmaxf(err, v.y);
    const uint32_t k = order_key(v.x);
    kmin = min(kmin, k);
    kmax = max(kmax, k);
    return k;
  };
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const int i = e * kThreads + tid;
    key[e] = 0u;  // below every finite score's key
    if (i < m) key[e] = look(__ldcg(scores + i));
  }
  if (!held)
    for (int i = kHeld * kThreads + tid; i < m; i += kThreads) look(__ldcg(scores + i));
  err = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(err)));
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    red[0][warp] = err;
    red[1][warp] = __uint_as_float(kmin);
    red[2][warp] = __uint_as_float(kmax);
  }
  if (tid == 0) open_n = 0;
  odd = 0;
  __syncthreads();
  if (bad) odd = 1;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    err = fmaxf(err, red[0][w]);
    kmin = min(kmin, __float_as_uint(red[1][w]));
    kmax = max(kmax, __float_as_uint(red[2][w]));
  }
  __syncthreads();
  const bool all_exact = odd;
  Counter count{part};

  // f(i, key of candidate i) for this thread's candidates, i = tid, tid + 256, ...; the
  // lanes of a warp are at 32 consecutive candidates, and all of them call f
  auto each = [&](auto&& f) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e)
      if (e * kThreads + warp * 32 < m) f(e * kThreads + tid, key[e]);
    for (int i = kHeld * kThreads + tid; i - lane < m; i += kThreads)
      f(i, i < m ? order_key(__ldcg(&scores[i].x)) : 0u);
  };

  int sure = 0, open = m;
  float low = 0.f, high = 0.f;  // scores above high are in, those below low are out
  if (!all_exact) {
    // the largest threshold with at least K keys at or above it, from the first bit in
    // which keys differ; it is enough that exactly K are
    const int top = 31 - __clz((int)(kmin ^ kmax));  // -1: all the same
    uint32_t thr = top >= 31 ? 0u : kmax & ~((2u << max(top, 0)) - 1u);
    if (top < 0) thr = kmax;
    for (int bit = top; bit >= 0; --bit) {
      const uint32_t cand = thr | (1u << bit);
      int mine = 0;
#pragma unroll
      for (int e = 0; e < kHeld; ++e) mine += key[e] >= cand;
      if (!held)
        for (int i = kHeld * kThreads + tid; i < m; i += kThreads) mine += order_key(__ldcg(&scores[i].x)) >= cand;
      const int c = count(mine);
      if (c >= K) thr = cand;
      if (c == K) break;
    }
    const float tau = key_value(thr), width = 2.02f * err;
    low = tau - width;
    high = tau + width;
    int s = 0, o = 0;
    each([&](int i, uint32_t k) {
      if (i >= m) return;
      const float x = key_value(k);
      s += x > high;
      o += x >= low && !(x > high);
    });
    sure = count(s);
    open = count(o);
  }
  const int need = K - sure;  // of the open ones
  const int words = (m + 31) >> 5;
  if (!all_exact && open == need) {
    each([&](int i, uint32_t k) {
      const uint32_t v = __ballot_sync(0xffffffffu, i < m && key_value(k) >= low);
      if (lane == 0) bits[i >> 5] = v;
    });
    __syncthreads();
  } else {
    for (int d = tid; d < D; d += kThreads) {
      double lo = 0.0, hi = 0.0;
      for (int h = 0; h < p.G; ++h) {
        const float x = q_value(__ldg(p.q + ((int64_t)t * p.Hkv * p.G + kh * p.G + h) * D + d), p.q_f16);
        lo += x > 0.f ? 0.0 : (double)x;
        hi += x < 0.f ? 0.0 : (double)x;
      }
      coef[d] = lo;
      coef[D + d] = hi;
    }
    __syncthreads();
    if (!all_exact && open <= kMaxOpen) {
      each([&](int i, uint32_t k) {
        const float x = key_value(k);
        const uint32_t v = __ballot_sync(0xffffffffu, i < m && x > high);
        if (lane == 0) bits[i >> 5] = v;
        if (i < m && x >= low && !(x > high)) open_idx[atomicAdd(&open_n, 1)] = i;  // the order does not matter
      });
      __syncthreads();
      for (int o = warp; o < open; o += kWarps) {
        const double s = exact_score<D>(p, r, b, kh, p.first + open_idx[o], coef, lane);
        if (lane == 0) open_key[o] = order_key64(s);
      }
      __syncthreads();
      if (tid < open) {
        const unsigned long long mine = open_key[tid];
        const int idx = open_idx[tid];
        int better = 0;
        for (int o = 0; o < open; ++o) better += open_key[o] > mine || (open_key[o] == mine && open_idx[o] < idx);
        if (better < need) atomicOr(&bits[idx >> 5], 1u << (idx & 31));
      }
      __syncthreads();
    } else {
      // many equal scores, or some that are not finite: every candidate's key in 64 bits, in
      // place of its score, and a search by bits
      unsigned long long* keys = reinterpret_cast<unsigned long long*>(scores);
      __syncthreads();
      for (int i = warp; i < m; i += kWarps) {
        const double s = exact_score<D>(p, r, b, kh, p.first + i, coef, lane);
        if (lane == 0) __stcg(keys + i, order_key64(s));
      }
      __syncthreads();
      unsigned long long thr = 0ull;
      for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long cand = thr | (1ull << bit);
        int mine = 0;
        for (int i = tid; i < m; i += kThreads) mine += __ldcg(keys + i) >= cand;
        if (count(mine) >= K) thr = cand;
      }
      int above = 0;
      for (int i = tid; i < m; i += kThreads) above += __ldcg(keys + i) > thr;
      int ties = K - count(above);  // of those at the threshold the lowest
      if (warp == 0) {
        for (int w = 0; w < words; ++w) {
          const int i = 32 * w + lane;
          const unsigned long long k = i < m ? __ldcg(keys + i) : 0ull;
          const uint32_t more = __ballot_sync(0xffffffffu, i < m && k > thr);
          const uint32_t same = __ballot_sync(0xffffffffu, i < m && k == thr);
          const bool take = (same >> lane & 1u) && __popc(same & ((1u << lane) - 1u)) < ties;
          const uint32_t some = __ballot_sync(0xffffffffu, take);
          ties -= __popc(some);
          if (lane == 0) bits[w] = more | some;
        }
      }
      __syncthreads();
    }
  }

  // the selected candidates in ascending order: each thread writes out a run of words
  const int per = (words + kThreads - 1) / kThreads;
  const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  int* sums = &part[0][0];
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int at = p.first + incl - mine;
  for (int w = 0; w < warp; ++w) at += sums[w];
  for (int w = w0; w < w1; ++w)
    for (uint32_t v = bits[w]; v; v &= v - 1) list[at++] = p.first + 32 * w + __ffs((int)v) - 1;
}

// ---------------------------------------------------------------- host
int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

bool block_size_ok(int bs) { return bs == 64 || bs == 128 || bs == 256; }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool ws_fits(const void* ws, size_t bytes, size_t need) { return ws && aligned(ws, 256) && bytes >= need; }

int check_blocks(const attn_kv_t* kv, const attn_blocks_t* blocks) {
  if (!blocks || !blocks->bounds || !aligned(blocks->bounds, 16) || blocks->num_rows <= 0) return ATTN_EINVAL;
  if (!block_size_ok(blocks->block_size)) return ATTN_EINVAL;
  if (kv->page_table) {
    if (blocks->block_size > kv->page_size || blocks->num_rows < kv->num_slots / blocks->block_size) return ATTN_EINVAL;
  } else if (!blocks->row_base || !aligned(blocks->row_base, 8)) {
    return ATTN_EINVAL;
  }
  return ATTN_OK;
}

BlocksPar blocks_par(const attn_config_t* cfg, const attn_kv_t& kv, const attn_blocks_t* blocks,
                     const int32_t* cu_seqlens, int32_t B, void* workspace) {
  BlocksPar p = {};
  p.bounds = static_cast<uint16_t*>(blocks->bounds);
  p.num_rows = blocks->num_rows;
  p.row_base = blocks->row_base;
  p.log2_bs = log2_of(blocks->block_size);
  p.Hkv = cfg->num_kv_heads;
  p.G = cfg->num_q_heads / cfg->num_kv_heads;
  p.B = B;
  p.cu_seqlens = cu_seqlens;
  p.kv = kv_index(kv);
  p.status = static_cast<int32_t*>(workspace);
  return p;
}

int blocks_of(int32_t max_kv_len, int32_t block_size) { return (int)(((int64_t)max_kv_len + block_size - 1) / block_size); }

size_t scores_bytes(const attn_config_t* cfg, int64_t N, int32_t max_blocks) {
  return (size_t)N * cfg->num_kv_heads * max_blocks * sizeof(float2);
}

template <int D, int KV>
int launch_bounds_t(const BlocksPar& p, cudaStream_t s) {
  return launch_dependent(block_bounds_kernel<D, KV>, dim3((unsigned)((int64_t)p.B * p.ctas_per_request)),
                          dim3(kThreads), 0, s, p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}
template <int D>
int launch_bounds_d(const BlocksPar& p, int kv_dtype, cudaStream_t s) {
  switch (kv_dtype) {
    case ATTN_KV_E4M3: return launch_bounds_t<D, ATTN_KV_E4M3>(p, s);
    case ATTN_KV_E2M1: return launch_bounds_t<D, ATTN_KV_E2M1>(p, s);
    default: return launch_bounds_t<D, ATTN_KV_BF16>(p, s);
  }
}

template <int D>
int launch_select_t(const BlocksPar& p, cudaStream_t s) {
  const int64_t lists = (int64_t)p.N * p.Hkv;
  if (lists * p.chunks > 0x7fffffff) return ATTN_EINVAL;
  if (launch_dependent(block_score_kernel<D>, dim3((unsigned)(lists * p.chunks)), dim3(kThreads), 0, s, p) != cudaSuccess)
    return ATTN_ELAUNCH;
  const size_t smem = (size_t)((p.max_blocks + 31) / 32) * 4;  // at most 32 KB
  return launch_dependent(block_select_kernel<D>, dim3((unsigned)lists), dim3(kThreads), smem, s, p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

size_t attn_block_workspace_size(const attn_config_t* cfg, int32_t max_tokens, int32_t max_kv_len,
                                 int32_t block_size, int32_t keep) {
  if (abi_check_config(cfg) != ATTN_OK || max_tokens < 0 || max_kv_len < 1 || max_kv_len > (1 << 24)) return 0;
  if (!block_size_ok(block_size) || keep < 1 || keep > kMaxListed) return 0;
  const size_t scores = scores_bytes(cfg, max_tokens, blocks_of(max_kv_len, block_size));
  return kWsHeader + align_up(scores, 256);
}

int attn_block_bounds(const attn_config_t* cfg, const attn_kv_t* kv, const attn_blocks_t* blocks,
                      const int32_t* start, const int32_t* cu_seqlens, int32_t B, void* workspace,
                      size_t ws_bytes, void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = abi_check_kv(kv))) return rc;
  if ((rc = check_blocks(kv, blocks))) return rc;
  if (B < 0 || B > (1 << 24) || !aligned(start, 4) || !aligned(cu_seqlens, 4)) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, kWsHeader)) return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (B == 0) return ATTN_OK;
  const attn_kv_t c = load_kv(kv);
  BlocksPar p = blocks_par(cfg, c, blocks, cu_seqlens, B, workspace);
  p.start = start;
  p.k_cache = c.k_cache;
  p.k_block_scale = static_cast<const uint8_t*>(c.k_block_scale);
  p.k_scale = c.k_scale;
  // how many blocks become full is on the device: a grid that fills the card walks them
  p.ctas_per_request = std::max(1, std::min(4096, 1216 / B));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cfg->head_dim == 128 ? launch_bounds_d<128>(p, c.kv_dtype, s) : launch_bounds_d<64>(p, c.kv_dtype, s);
}

int attn_block_select(const attn_config_t* cfg, const void* q, const int32_t* cu_seqlens, int32_t B, int32_t N,
                      int32_t max_kv_len, const attn_kv_t* kv, const attn_blocks_t* blocks, int32_t first,
                      int32_t last, int32_t keep, int32_t* list, void* workspace, size_t ws_bytes, void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = abi_check_kv(kv))) return rc;
  if ((rc = check_blocks(kv, blocks))) return rc;
  if (!q || !list || !aligned(q, 16) || !aligned(list, 4) || !aligned(cu_seqlens, 4)) return ATTN_EINVAL;
  if (B < 0 || N < 0 || (!cu_seqlens && N != B) || max_kv_len < 1 || max_kv_len > (1 << 24)) return ATTN_EINVAL;
  if (keep < 1 || keep > kMaxListed || first < 0 || last < 1 || last > keep || first > keep - last) return ATTN_EINVAL;
  const int max_blocks = blocks_of(max_kv_len, blocks->block_size);
  if (!ws_fits(workspace, ws_bytes, kWsHeader + scores_bytes(cfg, N, max_blocks))) return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (N == 0 || B == 0) return ATTN_OK;
  const attn_kv_t c = load_kv(kv);
  BlocksPar p = blocks_par(cfg, c, blocks, cu_seqlens, B, workspace);
  p.q = static_cast<const uint16_t*>(q);
  p.q_f16 = c.kv_dtype != ATTN_KV_BF16;
  p.N = N;
  p.first = first;
  p.last = last;
  p.keep = keep;
  p.max_blocks = max_blocks;
  p.scores = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kWsHeader);
  p.list = list;
  p.chunk = 64;
  p.chunks = (max_blocks + p.chunk - 1) / p.chunk;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cfg->head_dim == 128 ? launch_select_t<128>(p, s) : launch_select_t<64>(p, s);
}

int attn_block_attend(const attn_config_t* cfg, const void* q, const int32_t* cu_seqlens, int32_t B, int32_t N,
                      const attn_kv_t* kv, int32_t block_size, const int32_t* list, int32_t keep, void* out,
                      void* workspace, size_t ws_bytes, void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = abi_check_kv(kv))) return rc;
  if (!block_size_ok(block_size) || (kv->page_table && block_size > kv->page_size)) return ATTN_EINVAL;
  if (!q || !list || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(list, 4) || !aligned(cu_seqlens, 4))
    return ATTN_EINVAL;
  if (B < 0 || N < 0 || (!cu_seqlens && N != B) || keep < 1 || keep > kMaxListed) return ATTN_EINVAL;
  DecodeArgs a = {};
  block_splits((int64_t)std::max(N, 1) * cfg->num_kv_heads, keep, block_size, &a.max_splits, &a.split_len);
  if ((int64_t)N * a.max_splits > 0x7fffffff) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, kWsHeader)) return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (N == 0 || B == 0) return ATTN_OK;
  a.cfg = *cfg;
  a.B = B;
  a.kv = load_kv(kv);
  a.q = q;
  a.cu_seqlens = cu_seqlens;
  a.N = N;
  a.list = list;
  a.keep = keep;
  a.log2_bs = log2_of(block_size);
  a.out = out;
  a.status = static_cast<int32_t*>(workspace);
  return launch_block_attend(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
