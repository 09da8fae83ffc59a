// Cached entries of any type read as bf16, and the request of a packed token.
#pragma once

#include "common.cuh"

namespace gb300 {

namespace {

// Eight entries at chunk c of head kh's vector in a slot, as bf16 pairs.
template <int KV>
__device__ __forceinline__ uint4 read8(const void* cache, const uint8_t* bscale, float scale, int64_t num_slots,
                                       int64_t slot, int Hkv, int kh, int c, int log2_chunks) {
  const int64_t row = ((slot * Hkv + kh) << log2_chunks) + c;  // in chunks
  if constexpr (KV == ATTN_KV_BF16) return __ldg(static_cast<const uint4*>(cache) + row);
  uint32_t h[4];
  float s = 1.f;
  if constexpr (KV == ATTN_KV_E4M3) {
    const uint2 w = __ldg(static_cast<const uint2*>(cache) + row);
    e4m3x4_to_f16(w.x, h[0], h[1]);
    e4m3x4_to_f16(w.y, h[2], h[3]);
  } else {
    const int64_t blk = (((int64_t)kh * num_slots + slot) << (log2_chunks - 1)) + (c >> 1);
    s = f16_lo(e4m3x2_to_f16(__ldg(bscale + blk)));
    e2m1x8_to_f16(__ldg(static_cast<const uint32_t*>(cache) + row), h[0], h[1], h[2], h[3]);
  }
  uint32_t r[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
    r[e] = pack_bf16(__fmul_rn(__fmul_rn(f.x, s), scale), __fmul_rn(__fmul_rn(f.y, s), scale));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Slot of the first entry of a block (64 positions or more within a page) at position pos of a
// request, -1 where its page is not one of the cache's: unlike cache_slot(), whose callers read
// entry by entry or by tiles that end with the cache, a page that the cache's end cuts is none.
__device__ __forceinline__ int64_t block_slot(const KvIndex& kv, const ReqInfo& r, int pos) {
  if (!r.pages) return r.slot0 + pos;
  const int64_t pg = __ldg(r.pages + (pos >> kv.log2_page));
  if (pg < 0 || pg >= kv.num_slots >> kv.log2_page) return -1;
  return (pg << kv.log2_page) + (pos & ((1 << kv.log2_page) - 1));
}

// The request of packed token t, the number of its new tokens and the token's place j
// among them; cu == NULL: one token per request.  False for a token of no request.  The lanes
// of a warp search together, 32 requests a step: all of them call this with the same t.
__device__ __forceinline__ bool find_token(const int32_t* cu, int B, int t, int* b, int* n, int* j) {
  if (!cu) {
    *b = t;
    *n = 1;
    *j = 0;
    return true;
  }
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;  // largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5, probe = lo + (lane + 1) * step;
    const int below = __popc(__ballot_sync(0xffffffffu, probe < hi && __ldg(cu + probe) <= t));
    lo += below * step;
    hi = min(hi, lo + step);
  }
  const int c0 = __ldg(cu + lo);
  *b = lo;
  *n = __ldg(cu + lo + 1) - c0;
  *j = t - c0;
  return *j >= 0 && *j < *n;
}

}  // namespace

}  // namespace gb300
