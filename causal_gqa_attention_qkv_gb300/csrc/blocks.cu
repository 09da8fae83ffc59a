// Blocks of a cache (include/blocks.h): bounds of their keys and the selection of
// blocks for each query.  The attention over them is the decode kernels' (decode.cu,
// decode_e2m1.cu).
//
// Bounds: one warp per (full block, KV head) reads the block's keys, 16 bytes per
// lane, and keeps the minima and maxima of its components in registers.  Bound by HBM.
//
// Selection, with the group's heads h and a block's bounds lo, hi:
//   score = sum_h sum_d max(q_hd lo_d, q_hd hi_d) = sum_d M_d lo_d + P_d hi_d,
//   M_d = sum_h min(q_hd, 0), P_d = sum_h max(q_hd, 0):
// one dot product of 2 D terms per block and KV head, however many heads the group
// has, and it is bound by reading the bounds (4 D bytes).  A list must not depend on the
// order of fp32 sums, so a kernel takes the scores in fp32 with a bound on
// their error E, and a second one decides: t the K-th score, u the one after it; a score above
// u + 2 E belongs to the K largest whatever the errors are, one below t - 2 E does not, and
// only those between, if any, are summed again in fp64.  (Of the others only K - 1 can exceed
// u + E, and at least K exact scores are >= t - E.  A threshold between t and u will do for both.)
//
// The kernels let dependents start only behind their own wait: a decode kernel reads the
// requests' lengths before its wait, and a call that writes them may come before these.
#include "cluster.cuh"
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

// The larger of magnitudes a >= 0 and those of x.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t x) {
  const __nv_bfloat162 y = __habs2(*reinterpret_cast<__nv_bfloat162*>(&x));
  return max2(a, *reinterpret_cast<const uint32_t*>(&y));
}
__device__ __forceinline__ uint4 larger(const uint4& a, const uint4& x) {
  return make_uint4(larger(a.x, x.x), larger(a.y, x.y), larger(a.z, x.z), larger(a.w, x.w));
}

struct Range;

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
  int32_t q_f16, N, G, first, last, keep, max_kv_len, max_blocks, chunk, chunks;
  float* scores;             // [N, Hkv, max_blocks]
  Range* ranges;             // [N, Hkv, chunks]
  unsigned long long* keys;  // [N, Hkv, max_blocks] exact scores, where they are needed
  int32_t* list;             // [N, Hkv, keep]
};

// Row of the bounds of block i of a request, or -1 (a page outside the cache, a row
// outside the bounds).
__device__ __forceinline__ int64_t bounds_row(const BlocksPar& p, const ReqInfo& r, int b, int i) {
  int64_t row;
  if (r.pages) {
    const int64_t slot = block_slot(p.kv, r, i << p.log2_bs);
    row = slot < 0 ? -1 : slot >> p.log2_bs;
  } else {
    row = __ldg(p.row_base + b) + i;
  }
  return row >= 0 && row < p.num_rows ? row : -1;
}

// The same from the arguments alone; any i >= 0.
__device__ __forceinline__ int64_t bounds_row_at(const BlocksPar& p, int b, int i) {
  int64_t row;
  if (p.kv.page_table) {
    const int64_t pos = (int64_t)i << p.log2_bs;
    const int64_t pg = pos >> p.kv.log2_page;
    if (pg >= p.kv.pages_per_req) return -1;
    const int64_t page = __ldg(p.kv.page_table + (int64_t)b * p.kv.pages_per_req + pg);
    if (page < 0 || page >= p.kv.num_slots >> p.kv.log2_page) return -1;
    row = ((page << p.kv.log2_page) + (pos & ((1 << p.kv.log2_page) - 1))) >> p.log2_bs;
  } else {
    row = __ldg(p.row_base + b) + i;
  }
  return row >= 0 && row < p.num_rows ? row : -1;
}

// ---------------------------------------------------------------- bounds
// 16 bytes of a head's vector as pairs in which minimum and maximum are taken: bf16 entries as
// they are; codes as f16 pairs, exact (code, or code times block scale).  The product with the
// tensor's scale and the rounding to bf16 keep the order and are left to the end.
template <int KV>
struct Chunk {
  static constexpr int kPairs = KV == ATTN_KV_BF16 ? 4 : KV == ATTN_KV_E4M3 ? 8 : 16;
  uint32_t v[kPairs];
};
template <int KV>
__device__ __forceinline__ void unpack_chunk(const uint4& x, uint32_t scales, Chunk<KV>& c) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (KV == ATTN_KV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.v[i] = w[i];
  } else if constexpr (KV == ATTN_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_to_f16(w[i], c.v[2 * i], c.v[2 * i + 1]);
  } else {
    const uint32_t s = e4m3x2_to_f16(scales);  // the two blocks of 16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t* h = c.v + 4 * i;
      e2m1x8_to_f16(w[i], h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = i < 2 ? mul_f16x2_lo(h[e], s) : mul_f16x2_hi(h[e], s);
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t lower(uint32_t a, uint32_t b) {
  if constexpr (!F16) return min2(a, b);
  const __half2 r = __hmin2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool F16>
__device__ __forceinline__ uint32_t higher(uint32_t a, uint32_t b) {
  if constexpr (!F16) return max2(a, b);
  const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// One warp per (block, KV head), a lane 16 bytes of a key, 16 loads (or those of 64 keys) in
// flight: 32768 bf16 tokens (Hkv 8, D 128) 13.8 us, 5.0 TB/s (8 loads 14.8, 32 loads 17.3).
template <int D, int KV>
__global__ void __launch_bounds__(kThreads, 2) block_bounds_kernel(const BlocksPar p) {
  constexpr bool F16 = KV != ATTN_KV_BF16;
  constexpr int kBytes = KV == ATTN_KV_BF16 ? 2 * D : KV == ATTN_KV_E4M3 ? D : D / 2;  // of a key
  constexpr int L = kBytes / 16, KPW = 32 / L;   // lanes per key, keys per warp and load
  constexpr int U = 64 / KPW < 16 ? 64 / KPW : 16;
  constexpr int P = Chunk<KV>::kPairs;
  const int b = blockIdx.x / p.ctas_per_request, part = blockIdx.x % p.ctas_per_request;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();  // the appended entries, the lengths
  launch_dependents();
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
    const int64_t slot = block_slot(p.kv, r, i << p.log2_bs);
    const int64_t row = bounds_row(p, r, b, i);
    if ((slot < 0 || row < 0) && lane == 0) set_status(p.status, ATTN_STATUS_CAPACITY);
    if (row < 0) continue;
    Chunk<KV> lo = {}, hi = {};
    if (slot >= 0) {
      const uint4* keys = static_cast<const uint4*>(p.k_cache) + ((slot + sub) * p.Hkv + kh) * L + li;
      const uint16_t* scales = nullptr;  // of this lane's 32 codes
      if constexpr (KV == ATTN_KV_E2M1)
        scales = reinterpret_cast<const uint16_t*>(p.k_block_scale + ((int64_t)kh * p.kv.num_slots + slot + sub) * (D / 16)) + li;
      const int bs = 1 << p.log2_bs;
#pragma unroll 1
      for (int k0 = 0; k0 < bs; k0 += U * KPW) {
        uint4 x[U];
        uint32_t s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u] = __ldg(keys + (int64_t)(k0 + u * KPW) * (p.Hkv * L));
          s[u] = KV == ATTN_KV_E2M1 ? __ldg(scales + (k0 + u * KPW) * (D / 32)) : 0u;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Chunk<KV> c;
          unpack_chunk<KV>(x[u], s[u], c);
          if (u == 0 && k0 == 0) {
            lo = hi = c;
          } else {
#pragma unroll
            for (int e = 0; e < P; ++e) {
              lo.v[e] = lower<F16>(lo.v[e], c.v[e]);
              hi.v[e] = higher<F16>(hi.v[e], c.v[e]);
            }
          }
        }
      }
#pragma unroll
      for (int off = L; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          lo.v[e] = lower<F16>(lo.v[e], __shfl_xor_sync(0xffffffffu, lo.v[e], off));
          hi.v[e] = higher<F16>(hi.v[e], __shfl_xor_sync(0xffffffffu, hi.v[e], off));
        }
      if constexpr (F16) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo.v[e]));
          const float2 c = __half22float2(*reinterpret_cast<__half2*>(&hi.v[e]));
          lo.v[e] = pack_bf16(__fmul_rn(a.x, p.k_scale), __fmul_rn(a.y, p.k_scale));
          hi.v[e] = pack_bf16(__fmul_rn(c.x, p.k_scale), __fmul_rn(c.y, p.k_scale));
        }
      }
    }
    if (sub < 2) {  // the first group of lanes writes the minima, the second the maxima
      uint4* dst = reinterpret_cast<uint4*>(p.bounds + ((row * p.Hkv + kh) * 2 + sub) * D) + li * (P / 4);
#pragma unroll
      for (int e = 0; e < P; e += 4)
        dst[e / 4] = sub == 0 ? make_uint4(lo.v[e], lo.v[e + 1], lo.v[e + 2], lo.v[e + 3])
                              : make_uint4(hi.v[e], hi.v[e + 1], hi.v[e + 2], hi.v[e + 3]);
    }
  }
}

// ---------------------------------------------------------------- scores
__device__ __forceinline__ float q_value(uint32_t bits, int f16) {
  return f16 ? __half2float(__ushort_as_half((uint16_t)bits)) : __uint_as_float(bits << 16);
}

// How many blocks the query at place j of a request sees, 0 if it gets no list; `report`:
// this thread sets the status.
__device__ __forceinline__ int visible_blocks(const BlocksPar& p, const ReqInfo& r, int j, bool report) {
  if (!r.valid) {
    if (report) set_status(p.status, ATTN_STATUS_CAPACITY);
    return 0;
  }
  if (r.cached + r.n_new > p.max_kv_len) {
    if (report) set_status(p.status, ATTN_STATUS_BOUNDS);
    return 0;
  }
  return ((r.cached + j) >> p.log2_bs) + 1;  // at most max_blocks
}
__device__ __forceinline__ int query_blocks(const BlocksPar& p, int t, ReqInfo* r, int* b, bool report) {
  int n, j;
  if (!find_token(p.cu_seqlens, p.B, t, b, &n, &j)) {
    if (report) set_status(p.status, ATTN_STATUS_SEQLENS);
    return 0;
  }
  *r = load_request(p.kv, *b, n);
  return visible_blocks(p, *r, j, report);
}

constexpr int kMaxGroup = 8;

// f(component d of each head of token t in KV head kh's group): all loads go out together,
// whatever the group's size (absent heads count as 0; one after another they took 2400 cycles).
template <typename F>
__device__ __forceinline__ void each_head(const BlocksPar& p, int t, int kh, int D, int d, F&& f) {
  const uint16_t* row = p.q + ((int64_t)t * p.Hkv + kh) * p.G * D + d;
  uint16_t v[kMaxGroup];
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) v[h] = h < p.G ? __ldg(row + h * D) : (uint16_t)0;
#pragma unroll
  for (int h = 0; h < kMaxGroup; ++h) f(q_value(v[h], p.q_f16));
}

// M and P of token t and KV head kh, for component d; a NaN enters both.
__device__ __forceinline__ void coefficients(const BlocksPar& p, int t, int kh, int D, int d, float* m, float* q) {
  float lo = 0.f, hi = 0.f;
  each_head(p, t, kh, D, d, [&](float x) {
    lo += x > 0.f ? 0.f : x;
    hi += x < 0.f ? 0.f : x;
  });
  *m = lo;
  *q = hi;
}

// s + x = the new s + what is added to rest, exactly where nothing overflows (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float& s, float& rest, float x) {
  const float u = s + x, v = u - s;
  rest += (s - (u - v)) + (x - v);
  s = u;
}
// The same in 64 bits.  fp64 units are few (a list's 2 D G additions took 1500 cycles there): two fp32
// words hold the sums, exactly if the entries' magnitudes are within 2^36 of each other, to
// 2^-47 of them otherwise; fp64 takes those that are huge or not finite.
__device__ __forceinline__ void coefficients(const BlocksPar& p, int t, int kh, int D, int d, double* m, double* q) {
  float lo = 0.f, lo_rest = 0.f, hi = 0.f, hi_rest = 0.f;
  each_head(p, t, kh, D, d, [&](float x) {
    two_sum(lo, lo_rest, x > 0.f ? 0.f : x);
    two_sum(hi, hi_rest, x < 0.f ? 0.f : x);
  });
  if (hi - lo < 1e38f) {
    *m = (double)lo + (double)lo_rest;
    *q = (double)hi + (double)hi_rest;
    return;
  }
  double a = 0.0, b = 0.0;
  each_head(p, t, kh, D, d, [&](float x) {
    a += x > 0.f ? 0.0 : (double)x;
    b += x < 0.f ? 0.0 : (double)x;
  });
  *m = a;
  *q = b;
}

// Two fp32 operations in one instruction, each rounded to nearest even.
__device__ __forceinline__ uint64_t bf16x2_to_f32x2(uint32_t v) {
  return (uint64_t)(v & 0xFFFF0000u) << 32 | (uint64_t)(v << 16);
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Larger float -> larger key.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// What a warp (a CTA) knows of its scores: a bound on their errors, the range of their keys.
struct Range {
  float err;
  uint32_t kmin, kmax;
};
__device__ __forceinline__ Range join(const Range& a, const Range& b) {
  return {max_nan(a.err, b.err), min(a.kmin, b.kmin), max(a.kmax, b.kmax)};
}
__device__ __forceinline__ Range no_scores() { return {0.f, ~0u, 0u}; }

// The bound on the rounding of scores is a multiple of A = sum_d |w_d| max_i |y_id|, the largest
// magnitude that a component has among the blocks times that of its coefficient (half an
// instruction per component, the same for every token; each block's own sums of magnitudes
// cost a third of the call), and of what products below the normal range can lose.
//
// Sums in fp32: a term goes through at most 7 additions in M or P, 5 in its lane's two chains
// and 5 between lanes, 17 half steps of 2^-24.
constexpr float kFp32Error = 24.f * 5.9604645e-8f;
// On the tensor cores: a coefficient is the sum of two bf16 to within 2^-16; products are
// exact and added with at least fp32's precision in two chains of 128, and with any rounding,
// 2^-23 each; then the chains, the two parts, and the 7 additions in M or P.  The sums of
// magnitudes come the same way, 1.001 for their own rounding.
constexpr float kMmaError = 1.52587891e-5f + 144.f * 1.1920929e-7f;
constexpr float kErrorFloor = 1e-37f;
// There subnormal factors may be flushed, 2^-126 of the other factor each: a magnitude counts as
// 2^-110 at least (times kMmaError, 2^-125), and what parts of coefficients lose is taken with the
// largest magnitude.
constexpr uint32_t kLeast = 0x08800880u;  // a pair of bf16 2^-110
constexpr float kSubnormals = 2.4e-38f;

// Scores of the blocks [i0, i1) of a request for one token, by the CTA: a warp takes 8 blocks
// (D = 64: 16) at a time, lane l of the D / 4 lanes of a block holds 8 components of lo (the
// first half of the lanes) or hi.  Three CTAs per SM are bound by issue slots (240 instructions for 8
// blocks; as a product on the tensor cores, whose 16 rows one token leaves nearly empty, the
// registers leave room for two CTAs per SM instead of three: 16.4 us against 13.9).  coef: M, P; row_of(i): the row of block i; put(block, score);
// tell(range of this warp's scores), by one lane.  Returns whether a row lay outside.
template <int D, typename Row, typename Put, typename Tell>
__device__ __forceinline__ bool score_blocks(const BlocksPar& p, int kh, int i0, int i1, const float* coef, Row&& row_of,
                                             Put&& put, Tell&& tell) {
  constexpr int L = D / 4, BPW = 32 / L;  // lanes per block, blocks per warp and load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, li = lane % L, sub = lane / L;
  bool outside = false;
  uint4 big = make_uint4(0, 0, 0, 0);  // largest magnitudes
  float lowest = -kNegInf, highest = kNegInf;  // (a NaN shows in the error bound)
  const uint4* rows = reinterpret_cast<const uint4*>(p.bounds) + kh * (D / 4) + li;
  uint64_t w[4];  // pairs of coefficients
  *reinterpret_cast<ulonglong2*>(w) = *reinterpret_cast<const ulonglong2*>(coef + 8 * li);
  *reinterpret_cast<ulonglong2*>(w + 2) = *reinterpret_cast<const ulonglong2*>(coef + 8 * li + 4);
  // rows of the warp's blocks, one per lane; those of the next pass are looked up a pass ahead.
  // Lanes past the last block repeat it; a block of no row reads the first row and counts as 0.
  auto look_up = [&](int i) {
    int row = 0;
    if (lane < 8 * BPW && i < i1) {
      row = (int)row_of(min(i + lane, i1 - 1));
      outside |= row < 0;
    }
    return row;
  };
  int next = look_up(i0 + warp * 8 * BPW);
  for (int i = i0 + warp * 8 * BPW; i < i1; i += kWarps * 8 * BPW) {
    const int row = next, there = max(row, 0);
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = __ldg(rows + (int64_t)__shfl_sync(0xffffffffu, there, k * BPW + sub) * (p.Hkv * (D / 4)));
    next = look_up(i + kWarps * 8 * BPW);
    float s[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      big = larger(big, x[k]);
      uint64_t acc = mul_f32x2(w[0], bf16x2_to_f32x2(x[k].x));
      acc = fma_f32x2(w[1], bf16x2_to_f32x2(x[k].y), acc);
      acc = fma_f32x2(w[2], bf16x2_to_f32x2(x[k].z), acc);
      acc = fma_f32x2(w[3], bf16x2_to_f32x2(x[k].w), acc);
      s[k] = __uint_as_float((uint32_t)acc) + __uint_as_float((uint32_t)(acc >> 32));
    }
    // sums over the block's lanes; of the 8 values each lane keeps the one of its bits 0 .. 2
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
      const bool up = lane & half;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        const float give = up ? s[k] : s[k + half];
        s[k] = (up ? s[k + half] : s[k]) + __shfl_xor_sync(0xffffffffu, give, half);
      }
    }
#pragma unroll
    for (int off = 8; off < L; off <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
    const int at = i + (lane & 7) * BPW + sub;
    if (__shfl_sync(0xffffffffu, row, (lane & 7) * BPW + sub) < 0) s[0] = 0.f;
    if (li < 8 && at < i1) {
      put(at, s[0]);
      lowest = fminf(lowest, s[0]);
      highest = fmaxf(highest, s[0]);
    }
  }
  const uint32_t kmin = __reduce_min_sync(0xffffffffu, order_key(lowest));
  const uint32_t kmax = __reduce_max_sync(0xffffffffu, order_key(highest));
  float y[8], a = 0.f;
  unpack_bf16x8(big, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaf(fabsf(__uint_as_float((uint32_t)(w[e >> 1] >> (32 * (e & 1))))), y[e], a);
#pragma unroll
  for (int off = 1; off < L; off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
  if (BPW > 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, L & 31));
  if (lane == 0) tell(Range{fmaf(a, kFp32Error, kErrorFloor), kmin, kmax});
  return outside;
}

// Scores for the two-kernel selection: a CTA takes a run of blocks for up to kTokens tokens of a
// request, so that the bounds are read once for all of them, as a product on the tensor cores.
constexpr int kTokens = 8;

// The g-th group of up to kTokens tokens: request *b, its tokens from place *j on.  False past
// the last one.  All threads of the CTA call this.  cu_seqlens that are not in order may give
// any request and place (sums may even pass 32 bits then), but no request outside [0, B).
__device__ __forceinline__ bool find_group(const BlocksPar& p, int g, int* b, int* j) {
  if (!p.cu_seqlens) {
    *b = g;
    *j = 0;
    return g < p.B;
  }
  __shared__ int sums[kWarps], found[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) found[0] = -1;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int i = b0 + threadIdx.x;
    const int n = i < p.B ? __ldg(p.cu_seqlens + i + 1) - __ldg(p.cu_seqlens + i) : 0;
    const int mine = (min(max(n, 0), p.N) + kTokens - 1) / kTokens;
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += sums[w];
      total += sums[w];
    }
    if (g < total) {
      if (g >= incl - mine && g < incl) {
        found[0] = i;
        found[1] = (g - (incl - mine)) * kTokens;
      }
      __syncthreads();
      *b = found[0];
      *j = found[1];
      return *b >= 0;
    }
    g -= total;
    __syncthreads();
  }
  return false;
}

// m16n8k16: row g of A holds the upper, row g + 8 the lower bf16 part of token g's coefficients,
// a column of B a block.  Which component a k slot holds is free as long as A and B agree: quad
// member q takes the 16-byte chunks q, q + 4, ... of its block's row, each good for two products.
// A comes from shared memory, so a warp takes two tiles of 8 blocks for each of its reads (one tile
// was bound by them).  The sums of magnitudes are a product too: M <= 0 <= P, so they are those of
// the blocks' largest magnitudes, negated for lo.  55 tokens of 12 requests over up to 100000
// keys: 25.5 us with the selection (fp32 units took 48 where a first form of this took 33.6).
template <int D>
__global__ void __launch_bounds__(kThreads, 2) block_score_kernel(const BlocksPar p) {
  constexpr int C = D / 16;      // 16-byte chunks of a block's row per lane
  __shared__ __align__(16) float coef[kTokens][2 * D];  // M, P
  __shared__ __align__(16) uint4 frag[2 * C * 32];
  __shared__ uint32_t kmin[kTokens], kmax[kTokens], magnitude[kTokens], huge;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int kh = blockIdx.x / p.chunks % p.Hkv, c = blockIdx.x % p.chunks;
  grid_dependency_wait();
  launch_dependents();
  int b, j, n = 1, t = 0;
  if (!find_group(p, blockIdx.x / p.chunks / p.Hkv, &b, &j)) return;
  if (p.cu_seqlens) {
    t = __ldg(p.cu_seqlens + b);
    n = __ldg(p.cu_seqlens + b + 1) - t;
    t += j;
  } else {
    t = b;
  }
  const int run = min(min(n - j, kTokens), p.N - t);  // tokens past N have no list
  if (t < 0 || run <= 0) return;
  if (threadIdx.x < kTokens) {
    kmin[threadIdx.x] = ~0u;
    kmax[threadIdx.x] = magnitude[threadIdx.x] = 0u;
    huge = 0u;
  }
  const ReqInfo r = load_request(p.kv, b, n);
  const int most = r.valid ? ((r.cached + j + run - 1) >> p.log2_bs) + 1 : 0;  // blocks that the last token sees
  const int i0 = p.first + c * p.chunk, i1 = min(min(i0 + p.chunk, most - p.last), p.max_blocks);
  if (most <= p.keep || i0 >= i1) return;
  for (int i = threadIdx.x; i < kTokens * (D / 8); i += kThreads) {  // eight components of a token
    const int k = i / (D / 8), d = i % (D / 8) * 8;
    float m[8] = {}, x[8] = {};
    if (k < run) {
      const uint16_t* row = p.q + ((int64_t)(t + k) * p.Hkv + kh) * p.G * D + d;
      uint4 v[kMaxGroup];
#pragma unroll
      for (int h = 0; h < kMaxGroup; ++h)
        v[h] = h < p.G ? __ldg(reinterpret_cast<const uint4*>(row + h * D)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int h = 0; h < kMaxGroup; ++h) {
        const uint32_t w[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // as in coefficients()
          const float y = q_value((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu, p.q_f16);
          m[e] += y > 0.f ? 0.f : y;
          x[e] += y < 0.f ? 0.f : y;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      coef[k][d + e] = m[e];
      coef[k][D + d + e] = x[e];
    }
  }
  __syncthreads();
  // the A operand of each product, as the lanes want it
  for (int i = threadIdx.x; i < 2 * C * 32; i += kThreads) {
    const int s = i >> 5, tok = (i & 31) >> 2;
    const float4 w = *reinterpret_cast<const float4*>(&coef[tok][8 * (4 * (s >> 1) + (i & 3)) + 4 * (s & 1)]);
    const uint32_t u = pack_bf16(w.x, w.y), v = pack_bf16(w.z, w.w);
    frag[i] = make_uint4(u, bf16_rest(w.x, w.y, u), v, bf16_rest(w.z, w.w, v));
    // bf16 may round a larger one to infinity: then there is no bound
    if (!(fmaxf(fmaxf(fabsf(w.x), fabsf(w.y)), fmaxf(fabsf(w.z), fabsf(w.w))) < 3e38f)) huge = 1u;
  }
  __syncthreads();
  const int64_t list = (int64_t)t * p.Hkv + kh;
  // token g's scores; some past what the token sees are written too
  float* to = p.scores + (list + (int64_t)min(g, run - 1) * p.Hkv) * p.max_blocks;
  const uint4* rows = reinterpret_cast<const uint4*>(p.bounds) + kh * (D / 4) + q;
  uint4 big[C];
#pragma unroll
  for (int k = 0; k < C; ++k) big[k] = make_uint4(kLeast, kLeast, kLeast, kLeast);
  float lowest = -kNegInf, highest = kNegInf;
  bool outside = false;
  // columns past the last block repeat it; a block of no row counts as 0
  auto row_at = [&](int i) {
    const int row = (int)bounds_row(p, r, b, min(i, i1 - 1));
    outside |= row < 0;
    return row;
  };
  // columns 2 q, 2 q + 1 of token g: four chains, the upper and the lower part
  auto total = [](const float (&d)[2][4], int e) { return (d[0][e] + d[1][e]) + (d[0][2 + e] + d[1][2 + e]); };
  for (int i = i0 + warp * 16; i < i1; i += kWarps * 16) {
    const int row[2] = {row_at(i + g), row_at(i + 8 + g)};
    uint4 x[2][C];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < C; ++k)
        x[u][k] = __ldg(rows + (int64_t)max(row[u], 0) * (p.Hkv * (D / 4)) + 4 * k);
    if (__any_sync(0xffffffffu, min(row[0], row[1]) < 0)) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < C; ++k)
          if (row[u] < 0) x[u][k] = make_uint4(0, 0, 0, 0);
    }
    float d[2][2][4] = {};  // [tile][chain]
#pragma unroll
    for (int k = 0; k < C; ++k) {
      big[k] = larger(larger(big[k], x[0][k]), x[1][k]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 f = frag[(2 * k + h) * 32 + lane];
        const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          mma_bf16_16816(d[u][h], a, h ? x[u][k].z : x[u][k].x, h ? x[u][k].w : x[u][k].y);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float s = total(d[u], e);
        const int at = i + 8 * u + 2 * q + e;
        if (g < run && at < i1) {
          to[at] = s;
          lowest = fminf(lowest, s);
          highest = fmaxf(highest, s);
        }
      }
  }
  if (outside) set_status(p.status, ATTN_STATUS_CAPACITY);
  float d[2][4] = {};
  uint32_t top2 = 0u;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const uint32_t sign = k < C / 2 ? 0x80008000u : 0u;
    const uint32_t y[4] = {big[k].x | sign, big[k].y | sign, big[k].z | sign, big[k].w | sign};
#pragma unroll
    for (int e = 0; e < 4; ++e) top2 = max2(top2, y[e] & 0x7FFF7FFFu);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 f = frag[(2 * k + h) * 32 + lane];
      const uint32_t a[4] = {f.x, f.y, f.z, f.w};
      mma_bf16_16816(d[h], a, y[2 * h], y[2 * h + 1]);
    }
  }
  float top = max_nan(bf16_lo(top2), bf16_hi(top2));  // of the lane's column
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (g < run) {
    const float sum = max_nan(total(d, 0), total(d, 1));
    // NaN and infinity are the largest as words, and a sum of magnitudes has no sign
    atomicMax(&magnitude[g], __float_as_uint(fabsf(fmaf(top, 2 * D * kSubnormals / kMmaError, sum))));
    atomicMin(&kmin[g], order_key(lowest));
    atomicMax(&kmax[g], order_key(highest));
  }
  __syncthreads();
  if ((int)threadIdx.x < run) {
    const float a = __uint_as_float(magnitude[threadIdx.x]);
    const float err = huge ? -kNegInf : fmaf(a, kMmaError * 1.001f, kErrorFloor);
    p.ranges[(list + (int64_t)threadIdx.x * p.Hkv) * p.chunks + c] = Range{err, kmin[threadIdx.x], kmax[threadIdx.x]};
  }
}

// ---------------------------------------------------------------- selection
// order_key() in 64 bits; -0 as 0, and NaN above all.
__device__ __forceinline__ unsigned long long order_key64(double x) {
  if (!(x == x)) return ~0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

constexpr int kHeld = 8;                     // keys held in registers per thread
constexpr int kHeldAll = kHeld * kThreads;   // candidates that are all held
constexpr int kMaxOpen = 256;                // candidates summed again and ranked in shared memory
constexpr int kBins = 1024;

template <int D>
struct SelectSmem {
  int part[2][3][kWarps];
  double coef[2 * D];
  int open_idx[kMaxOpen];
  unsigned long long open_key[kMaxOpen];
  int bins[kBins];
  uint32_t bin_key[kMaxOpen];
  int open_n, bin_n;
  int bin, above, inside;  // the bin with the K-th key: keys above it, keys in it
  uint32_t thr, next;  // the K-th key, the one after it
  int sums[kWarps];
};

// Sums over the CTA of up to three counts per thread: one barrier a call, alternating buffers.
struct Counter {
  int (*part)[3][kWarps];  // [2]
  int turn = 0;
  template <int N>
  __device__ __forceinline__ void operator()(int (&c)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      c[k] = __reduce_add_sync(0xffffffffu, c[k]);
      if ((threadIdx.x & 31) == 0) part[turn][k][threadIdx.x >> 5] = c[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      c[k] = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) c[k] += part[turn][k][w];
    }
    turn ^= 1;
  }
};

// This lane's entries of a block's bounds, and the block's score in fp64, summed by one warp in the
// same order for every block.
template <int D>
__device__ __forceinline__ uint4 bounds_entries(const BlocksPar& p, const ReqInfo& r, int b, int kh, int i, int lane) {
  const int64_t row = lane < D / 4 ? bounds_row(p, r, b, i) : -1;
  if (row < 0) return make_uint4(0, 0, 0, 0);
  return __ldg(reinterpret_cast<const uint4*>(p.bounds + (row * p.Hkv + kh) * (2 * D)) + lane);
}
template <int D>
__device__ __forceinline__ double exact_score(const uint4& entries, const double* coef, int lane) {
  double s = 0.0;
  if (lane < D / 4) {
    float y[8];
    unpack_bf16x8(entries, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma(coef[8 * lane + e], (double)y[e], s);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// One CTA chooses the K largest of the m = n - first - last candidates of token t and KV head
// kh and writes the list.  at(i): candidate i's score (read once for the first kHeldAll, again
// and again for others), range: of them all; bits: ceil(m / 32) words; keys: m words of 64
// bits.  sm.bins, sm.open_n and sm.bin_n are zero; Coef: sm.coef is there already.
template <int D, bool Coef, typename At>
__device__ void select_blocks(const BlocksPar& p, const ReqInfo& r, int b, int t, int kh, int n, At&& at, const Range& range,
                              uint32_t* bits, unsigned long long* keys, SelectSmem<D>& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* list = p.list + ((int64_t)t * p.Hkv + kh) * p.keep;
  const int m = n - p.first - p.last, K = p.keep - p.first - p.last;
  for (int i = tid; i < p.first; i += kThreads) list[i] = i;
  for (int i = tid; i < p.last; i += kThreads) list[p.keep - p.last + i] = n - p.last + i;
  if (K == 0) return;

  uint32_t key[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e)
    if (e * kThreads < m) key[e] = __float_as_uint(at(min(e * kThreads + tid, m - 1)));  // all loads first
#pragma unroll
  for (int e = 0; e < kHeld; ++e) key[e] = e * kThreads + tid < m ? order_key(__uint_as_float(key[e])) : 0u;
  const uint32_t kmin = range.kmin, kmax = range.kmax;
  // Magnitudes whose sum is finite give finite scores, or ones that just overflow.
  const bool all_exact = !(range.err <= 3.4028235e38f && fabsf(key_value(kmin)) <= 3.4028235e38f &&
                           fabsf(key_value(kmax)) <= 3.4028235e38f);
  Counter count{sm.part};

  // f(i, key of candidate i) for this thread's candidates, i = tid, tid + 256, ...; the
  // lanes of a warp are at 32 consecutive candidates, and all of them call f
  auto each = [&](auto&& f) {
#pragma unroll
    for (int e = 0; e < kHeld; ++e)
      if (e * kThreads + warp * 32 < m) f(e * kThreads + tid, key[e]);
    for (int i = kHeldAll + tid; i - lane < m; i += kThreads) f(i, i < m ? order_key(at(i)) : 0u);
  };

  int sure = 0, open = m;
  float low = 0.f, high = 0.f;  // scores above high are in, those below low are out
  if (!all_exact) {
    // A threshold with exactly K keys at or above it, or else the K-th key: the keys in bins of
    // equal width, then those of the K-th's bin (one or two of 1000) by their ranks.
    const int shift = max(0, 22 - __clz((int)(kmax - kmin)));  // the range in fewer than kBins steps
    // (cu_seqlens that are not in order can leave scores unwritten: nothing may index past its array)
    auto bin_of = [&](uint32_t k) { return min((k - kmin) >> shift, (uint32_t)kBins - 1u); };
    each([&](int i, uint32_t k) {
      if (i < m) atomicAdd(&sm.bins[bin_of(k)], 1);
    });
    __syncthreads();
    constexpr int R = kBins / kThreads;  // bins per thread, the highest first
    int c[R], mine = 0;
#pragma unroll
    for (int e = 0; e < R; ++e) mine += c[e] = sm.bins[kBins - 1 - (tid * R + e)];
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) sm.sums[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) incl += sm.sums[w];
    int before = incl - mine;
    if (before < K && incl >= K) {
#pragma unroll
      for (int e = 0; e < R; ++e) {
        if (before < K && before + c[e] >= K) {
          sm.bin = kBins - 1 - (tid * R + e);
          sm.above = before;
          sm.inside = c[e];
        }
        before += c[e];
      }
    }
    __syncthreads();
    const int inside = sm.inside, want = K - sm.above;
    uint32_t thr = kmin + ((uint32_t)sm.bin << shift), next = thr;  // next: K + 1 keys there, or no more than thr
    if (inside > want && inside <= kMaxOpen) {
      const uint32_t bin = sm.bin;
      each([&](int i, uint32_t k) {
        if (i < m && bin_of(k) == bin) sm.bin_key[atomicAdd(&sm.bin_n, 1)] = k;  // in any order
      });
      __syncthreads();
      if (tid < inside) {
        const uint32_t k = sm.bin_key[tid];
        int larger = 0, same = 0;
        for (int o = 0; o < inside; ++o) {
          larger += sm.bin_key[o] > k;
          same += sm.bin_key[o] == k;
        }
        if (larger < want && larger + same >= want) sm.thr = k;  // equal keys write the same
        if (larger <= want && larger + same > want) sm.next = k;
      }
      __syncthreads();
      thr = sm.thr;
      next = sm.next;
    } else if (inside > want) {
      // a crowded bin (a few scores far from all others): bit by bit below the bin's edge, two
      // at a time; it is enough that exactly K keys are at or above
      for (int bit = shift - 1; bit >= 0; bit -= 2) {
        const uint32_t hi = 1u << bit, lo = bit > 0 ? hi >> 1 : 0u;
        int n3[3] = {0, 0, 0};
        each([&](int i, uint32_t k) {
          if (i >= m) return;
          n3[0] += k >= thr + lo;
          n3[1] += k >= thr + hi;
          n3[2] += k >= thr + hi + lo;
        });
        count(n3);
        const int take = n3[2] >= K ? 3 : n3[1] >= K ? 2 : n3[0] >= K ? 1 : 0;
        if (take & 2) thr += hi;
        if (take & 1) thr += lo;
        if (take != 0 && n3[take - 1] == K) break;
      }
      next = thr;
    }
    const float width = 2.02f * range.err;
    low = key_value(thr) - width;
    high = key_value(next) + width;
    int so[2] = {0, 0};  // per warp
    each([&](int i, uint32_t k) {
      const float x = key_value(k);
      const uint32_t in = __ballot_sync(0xffffffffu, i < m && x >= low);
      const int s = __popc(__ballot_sync(0xffffffffu, i < m && x > high));
      if (lane == 0) {
        bits[i >> 5] = in;
        so[0] += s;
        so[1] += __popc(in) - s;
      }
    });
    count(so);
    sure = so[0];
    open = so[1];
  }
  const int need = K - sure;  // of the open ones
  const int words = (m + 31) >> 5;
  if (all_exact || open != need) {
    auto make_coef = [&] {
      if constexpr (!Coef)
        for (int d = tid; d < D; d += kThreads) coefficients(p, t, kh, D, d, &sm.coef[d], &sm.coef[D + d]);
      __syncthreads();
    };
    __syncthreads();
    if (!all_exact && open <= kMaxOpen) {
      each([&](int i, uint32_t k) {
        const float x = key_value(k);
        const uint32_t v = __ballot_sync(0xffffffffu, i < m && x > high);
        if (lane == 0) bits[i >> 5] = v;
        if (i < m && x >= low && !(x > high)) sm.open_idx[atomicAdd(&sm.open_n, 1)] = i;  // in any order
      });
      __syncthreads();
      if (need > 0 && open > 0) {  // (K are sure, or scores were left unwritten)
        auto entries = [&](int o) {
          return bounds_entries<D>(p, r, b, kh, p.first + sm.open_idx[min(o, open - 1)], lane);
        };
        uint4 y = entries(warp);  // on their way while the coefficients are made
        make_coef();
        for (int o = warp; o < open; o += kWarps) {
          const double s = exact_score<D>(y, sm.coef, lane);
          if (lane == 0) sm.open_key[o] = order_key64(s);
          if (o + kWarps < open) y = entries(o + kWarps);
        }
      }
      __syncthreads();
      if (tid < open && need > 0) {
        const unsigned long long mine = sm.open_key[tid];
        const int idx = sm.open_idx[tid];
        int better = 0;
        for (int o = 0; o < open; ++o)
          better += sm.open_key[o] > mine || (sm.open_key[o] == mine && sm.open_idx[o] < idx);
        if (better < need) atomicOr(&bits[idx >> 5], 1u << (idx & 31));
      }
      __syncthreads();
    } else {
      // many equal scores, or some that are not finite: every candidate's key in 64 bits and a
      // search by bits
      make_coef();
      for (int i = warp; i < m; i += kWarps) {
        const double s = exact_score<D>(bounds_entries<D>(p, r, b, kh, p.first + i, lane), sm.coef, lane);
        if (lane == 0) keys[i] = order_key64(s);
      }
      __syncthreads();
      unsigned long long thr = 0ull;
      for (int bit = 63; bit >= 0; --bit) {
        const unsigned long long cand = thr | (1ull << bit);
        int c[1] = {0};
        for (int i = tid; i < m; i += kThreads) c[0] += keys[i] >= cand;
        count(c);
        if (c[0] >= K) thr = cand;
      }
      int above[1] = {0};
      for (int i = tid; i < m; i += kThreads) above[0] += keys[i] > thr;
      count(above);
      int ties = K - above[0];  // of those at the threshold the lowest
      if (warp == 0) {
        for (int w = 0; w < words; ++w) {
          const int i = 32 * w + lane;
          const unsigned long long k = i < m ? keys[i] : 0ull;
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

  // the selected candidates in ascending order
  if (m <= kHeldAll) {  // every warp sums the words up for itself
    const uint32_t w0 = lane < words ? bits[lane] : 0u, w1 = 32 + lane < words ? bits[32 + lane] : 0u;
    int s0 = __popc(w0), s1 = __popc(w1);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v0 = __shfl_up_sync(0xffffffffu, s0, off), v1 = __shfl_up_sync(0xffffffffu, s1, off);
      if (lane >= off) {
        s0 += v0;
        s1 += v1;
      }
    }
    s1 += __shfl_sync(0xffffffffu, s0, 31) - __popc(w1);
    s0 -= __popc(w0);
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int w = e * kWarps + warp;  // this warp's word
      if (w >= words) break;
      const uint32_t v = __shfl_sync(0xffffffffu, w < 32 ? w0 : w1, w & 31);
      const int to = p.first + __shfl_sync(0xffffffffu, w < 32 ? s0 : s1, w & 31) + __popc(v & ((1u << lane) - 1u));
      if ((v >> lane & 1u) && to < p.first + K) list[to] = p.first + 32 * w + lane;
    }
    return;
  }
  // each thread writes out a run of words
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
  __syncthreads();  // sums is read again
  if (lane == 31) sm.sums[warp] = incl;
  __syncthreads();
  int to = p.first + incl - mine;
  for (int w = 0; w < warp; ++w) to += sm.sums[w];
  for (int w = w0; w < w1; ++w)
    for (uint32_t v = bits[w]; v && to < p.first + K; v &= v - 1) list[to++] = p.first + 32 * w + __ffs((int)v) - 1;
}

template <int D>
__device__ __forceinline__ void clear_select(SelectSmem<D>& sm) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.bins[i] = 0;
  if (threadIdx.x == 0) sm.open_n = sm.bin_n = 0;
}
__device__ __forceinline__ Range join_lanes(Range v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v.err = max_nan(v.err, __shfl_xor_sync(0xffffffffu, v.err, off));
  v.kmin = __reduce_min_sync(0xffffffffu, v.kmin);
  v.kmax = __reduce_max_sync(0xffffffffu, v.kmax);
  return v;
}

__device__ __forceinline__ void whole_list(const BlocksPar& p, int t, int kh, int n) {
  int32_t* list = p.list + ((int64_t)t * p.Hkv + kh) * p.keep;
  for (int i = threadIdx.x; i < p.keep; i += kThreads) list[i] = i < n ? i : -1;
}

// The second of the two kernels: one CTA per list, scores in the workspace.
template <int D>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const BlocksPar p) {
  extern __shared__ uint32_t bits[];
  __shared__ SelectSmem<D> sm;
  const int t = blockIdx.x / p.Hkv, kh = blockIdx.x % p.Hkv;
  // Before the wait: q, the lengths and the page table, which were there when the kernel of the scores
  // passed its own wait.  Most lists have a few scores to sum again and need the coefficients.
  for (int d = threadIdx.x; d < D; d += kThreads) coefficients(p, t, kh, D, d, &sm.coef[d], &sm.coef[D + d]);
  clear_select(sm);
  ReqInfo r;
  int b;
  const int n = query_blocks(p, t, &r, &b, kh == 0 && threadIdx.x == 0);
  grid_dependency_wait();
  launch_dependents();
  if (n == 0) return;
  if (n <= p.keep) {
    whole_list(p, t, kh, n);
    return;
  }
  const int64_t list = (int64_t)t * p.Hkv + kh;
  const float* scores = p.scores + list * p.max_blocks + p.first;
  Range range = no_scores();
  const int lane = threadIdx.x & 31;
  for (int c = lane; p.first + c * p.chunk < n - p.last; c += 32) range = join(range, p.ranges[list * p.chunks + c]);
  range = join_lanes(range);
  __syncthreads();
  select_blocks<D, true>(p, r, b, t, kh, n, [&](int i) { return __ldcg(scores + i); }, range, bits,
                   p.keys + list * p.max_blocks, sm);
}

// Both in one kernel for lists of up to kHeldAll candidates: a cluster of p.chunks CTAs scores
// runs of p.chunk candidates into the shared memory of its first CTA, which selects.  One
// token's call is a chain of latencies, so the loads that do not wait for each other go out
// together (lengths, q, page numbers, then the bounds), scores are pushed rather than fetched,
// and the other CTAs leave when theirs have arrived.
template <int D>
__global__ void __launch_bounds__(kThreads) block_pick_kernel(const BlocksPar p) {
  __shared__ SelectSmem<D> sm;
  __shared__ __align__(16) float coef[2 * D];
  __shared__ uint32_t bits[kHeldAll / 32];
  __shared__ float scores[kHeldAll];  // of the first CTA
  __shared__ Range told[16 * kWarps];
  __shared__ unsigned long long keys[kHeldAll];
  const int rank = blockIdx.x % p.chunks, list = blockIdx.x / p.chunks, t = list / p.Hkv, kh = list % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.chunks > 1) cluster_arrive();  // this CTA has started
  clear_select(sm);
  grid_dependency_wait();
  launch_dependents();
  int b, nn, j;
  const bool report = rank == 0 && kh == 0 && threadIdx.x == 0;
  const bool found = find_token(p.cu_seqlens, p.B, t, &b, &nn, &j);
  if (!found) {  // the whole cluster
    if (p.chunks > 1) cluster_wait();
    if (report) set_status(p.status, ATTN_STATUS_SEQLENS);
    return;
  }
  for (int d = threadIdx.x; d < D; d += kThreads) coefficients(p, t, kh, D, d, &coef[d], &coef[D + d]);
  const int i0 = p.first + rank * p.chunk;
  // the row of the first block that this lane will look up, before it is known to be there
  constexpr int PER = 8 * 32 / (D / 4);  // blocks per warp and pass
  const int ahead = i0 + warp * PER + lane;
  const int64_t row0 = lane < PER ? bounds_row_at(p, b, ahead) : -1;
  const ReqInfo r = load_request(p.kv, b, nn);
  const int n = visible_blocks(p, r, j, report);
  if (p.chunks > 1) cluster_wait();  // every CTA has started: its shared memory is there
  if (n == 0) return;
  if (n <= p.keep) {
    if (rank == 0) whole_list(p, t, kh, n);
    return;
  }
  const int i1 = min(i0 + p.chunk, n - p.last);
  __syncthreads();
  const uint32_t to = peer_addr(smem_u32(scores), 0), to_range = peer_addr(smem_u32(told + rank * kWarps + warp), 0);
  auto tell = [&](const Range& v) {
    peer_store(to_range, v.err);
    peer_store(to_range + 4, __uint_as_float(v.kmin));
    peer_store(to_range + 8, __uint_as_float(v.kmax));
  };
  if (i0 < i1) {
    if (score_blocks<D>(
            p, kh, i0, i1, coef, [&](int i) { return i == ahead ? row0 : bounds_row(p, r, b, i); },
            [&](int i, float v) { peer_store(to + (uint32_t)(i - p.first) * 4u, v); }, tell))
      set_status(p.status, ATTN_STATUS_CAPACITY);
  } else if (lane == 0) {
    tell(no_scores());
  }
  if (p.chunks > 1) {
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
  } else {
    __syncthreads();
  }
  Range range = no_scores();
  for (int w = lane; w < p.chunks * kWarps; w += 32) range = join(range, told[w]);
  range = join_lanes(range);
  select_blocks<D, false>(p, r, b, t, kh, n, [&](int i) { return scores[i]; }, range, bits, keys, sm);
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
  if (!blocks || !blocks->bounds || !aligned(blocks->bounds, 16) || blocks->num_rows <= 0 || blocks->num_rows > 0x7fffffff) return ATTN_EINVAL;
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

// Blocks per CTA of the two-kernel selection: 55 tokens of 12 requests over up to 100000 keys take
// 28.3, 25.9, 28.3, 32.0 us with 256, 512, 768, 1024 (each CTA has its coefficients to make first).
constexpr int kChunk = 512;

// Behind the header: exact scores, scores, ranges.
size_t scores_bytes(const attn_config_t* cfg, int64_t N, int32_t max_blocks) {
  const size_t lists = (size_t)N * cfg->num_kv_heads;
  return align_up(lists * max_blocks * (sizeof(float) + 8) + lists * ((max_blocks + kChunk - 1) / kChunk) * sizeof(Range), 256);
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

// One kernel or two: tokens of one request next to each other share the reading of the bounds
// in the two, and the one spares a launch and the scores' way through memory.  16 requests of
// up to 30000 keys: 14.3 us (one kernel), 17.7 (two) with a token each, 15.1 and 19.1 with 24
// tokens, 18.8 and 21.4 with 40, 27.6 and 25.3 with 80; 30 tokens of 12 requests of up to 100000
// keys 34.1 and 26.6; few lists: 8 tokens of one request of 30000 keys 9.3 and 16.0, of 100000
// 18.5 and 16.8.
// Clusters where there are few lists (us with 1, 4, 8, 16 CTAs each; two were not the best at any of these
// sizes).  A CTA's share is a power of two, 64 blocks at least, so some of a cluster may have none: of the
// two CTAs for 33 to 64 blocks one, just above a power of two of blocks nearly half.
// 8 lists of 128 blocks 5.9, 5.4, 5.5, 6.1; 8 of 1016 17.5, 8.4, 6.8, 6.6; 32 of 256 8.3, 8.0, 7.7, 10.0;
// 64 of 470 12.1, 11.5, 12.6, 16.9; 96 of 313 9.9, 9.7, 12.7, 21.9; 96 of 940 22.9, 15.5, 18.1, 26.1;
// 128 of 470 13.6, 13.2, 16.3, -; 160 of 470 15.8, 17.0, 21.7, -.
template <int D>
int launch_select_t(BlocksPar& p, cudaStream_t s) {
  const int64_t lists = (int64_t)p.N * p.Hkv;
  const bool few = lists <= 96;
  if (p.max_blocks <= kHeldAll && (few || p.N < (p.max_blocks <= 1024 ? 3 : 2) * (int64_t)p.B)) {
    int c = 1;
    while (few && c < 16 && lists * c <= 192 && p.max_blocks > 32 * c) c *= 2;
    p.chunks = c;
    p.chunk = 64;
    while (p.chunk * c < p.max_blocks) p.chunk *= 2;
    if (lists * c > 0x7fffffff) return ATTN_EINVAL;
    return launch_cluster_dependent(block_pick_kernel<D>, dim3((unsigned)(lists * c)), dim3(kThreads), 0, c, s, p) ==
                   cudaSuccess
               ? ATTN_OK
               : ATTN_ELAUNCH;
  }
  const int64_t groups = std::min<int64_t>(p.N, p.N / kTokens + (int64_t)p.B);
  p.chunk = kChunk;
  p.chunks = (p.max_blocks + p.chunk - 1) / p.chunk;
  const int64_t ctas = groups * p.Hkv * p.chunks;
  if (ctas > 0x7fffffff || lists > 0x7fffffff) return ATTN_EINVAL;
  if (launch_dependent(block_score_kernel<D>, dim3((unsigned)ctas), dim3(kThreads), 0, s, p) != cudaSuccess)
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
  return kWsHeader + scores;
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
  p.ctas_per_request = std::max(1, 608 / B);
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
  p.max_kv_len = max_kv_len;
  p.max_blocks = max_blocks;
  const size_t slots = (size_t)N * p.Hkv * max_blocks;
  p.keys = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + kWsHeader);
  p.scores = reinterpret_cast<float*>(p.keys + slots);
  p.ranges = reinterpret_cast<Range*>(p.scores + slots);
  p.list = list;
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
