// attn_kv_gather: cached entries of ranges of positions read back as packed
// bf16 rows (the transformer-basics page's cache read, past_key_values, for a
// cache that may hold codes).  One warp per token: 8 entries per lane and
// step, K then V.  Bound by HBM: every entry is read once and written once (131072
// positions, Hkv 8, D 128, 64-slot pages: bf16 155 us, 6.9 TB/s; E4M3 121 us, 6.7;
// E2M1 116 us, 5.9); a decode step's 64 new entries by the launch, 3.9 us.
#include "kernels.cuh"

namespace gb300 {

namespace {

constexpr int kWarps = 8;

struct GatherPar {
  const void* k_cache;
  const void* v_cache;
  const uint8_t* k_block_scale;
  const uint8_t* v_block_scale;
  float k_scale, v_scale;
  KvIndex kv;
  const int32_t* cu_seqlens;
  int32_t B, N, Hkv, log2_chunks;  // 8-entry chunks per head vector: D / 8
  uint4* k_out;
  uint4* v_out;
  int32_t* status;
};

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

template <int KV>
__global__ void __launch_bounds__(kWarps * 32) kv_gather_kernel(const GatherPar p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();  // the entries of the call before this one
  if (t >= p.N) return;
  int lo = 0, hi = p.B;  // largest b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
  }
  const int c0 = __ldg(p.cu_seqlens + lo), n = __ldg(p.cu_seqlens + lo + 1) - c0, j = t - c0;
  if (t == 0 && lane == 0 && __ldg(p.cu_seqlens + p.B) != p.N) set_status(p.status, ATTN_STATUS_SEQLENS);
  if (j < 0 || j >= n) {
    if (lane == 0) set_status(p.status, ATTN_STATUS_SEQLENS);
    return;
  }
  const ReqInfo r = load_request(p.kv, lo, n);
  const int64_t slot = r.valid ? cache_slot(p.kv, r, r.cached + j) : -1;
  if (slot < 0 && lane == 0) set_status(p.status, ATTN_STATUS_CAPACITY);
  if (!r.valid) return;
  const int chunks = p.Hkv << p.log2_chunks;
  const int64_t out = (int64_t)t * chunks;
  for (int i = lane; i < chunks; i += 32) {
    const int kh = i >> p.log2_chunks, c = i & ((1 << p.log2_chunks) - 1);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (slot >= 0) {
      k = read8<KV>(p.k_cache, p.k_block_scale, p.k_scale, p.kv.num_slots, slot, p.Hkv, kh, c, p.log2_chunks);
      v = read8<KV>(p.v_cache, p.v_block_scale, p.v_scale, p.kv.num_slots, slot, p.Hkv, kh, c, p.log2_chunks);
    }
    p.k_out[out + i] = k;
    p.v_out[out + i] = v;
  }
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream) {
  GatherPar p;
  p.k_cache = a.kv.k_cache;
  p.v_cache = a.kv.v_cache;
  p.k_block_scale = static_cast<const uint8_t*>(a.kv.k_block_scale);
  p.v_block_scale = static_cast<const uint8_t*>(a.kv.v_block_scale);
  p.k_scale = a.kv.k_scale;
  p.v_scale = a.kv.v_scale;
  p.kv = kv_index(a.kv);
  p.cu_seqlens = a.cu_seqlens;
  p.B = a.B;
  p.N = a.N;
  p.Hkv = a.Hkv;
  p.log2_chunks = a.D == 128 ? 4 : 3;
  p.k_out = static_cast<uint4*>(a.k_out);
  p.v_out = static_cast<uint4*>(a.v_out);
  p.status = a.status;
  const dim3 grid((unsigned)(((int64_t)a.N + kWarps - 1) / kWarps)), block(kWarps * 32);
  switch (a.kv.kv_dtype) {
    case ATTN_KV_E4M3: return launch_dependent(kv_gather_kernel<ATTN_KV_E4M3>, grid, block, 0, stream, p);
    case ATTN_KV_E2M1: return launch_dependent(kv_gather_kernel<ATTN_KV_E2M1>, grid, block, 0, stream, p);
    default: return launch_dependent(kv_gather_kernel<ATTN_KV_BF16>, grid, block, 0, stream, p);
  }
}

}  // namespace gb300
