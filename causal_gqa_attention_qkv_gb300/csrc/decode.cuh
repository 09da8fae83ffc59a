// What the decode kernels share: their parameters, the append of the new token
// and the split of a request's keys.
#pragma once

#include "cluster.cuh"
#include "kernels.cuh"
#include "kv_read.cuh"

namespace gb300 {

namespace {

constexpr int kKeysPerTile = 64;
constexpr int kConsumerWarps = 4;
constexpr int kThreads = (kConsumerWarps + 1) * 32;

struct DecodePar {
  const uint16_t* qkv;       // [B, W]
  const uint16_t* q_norm_w;  // [D]
  const uint16_t* k_norm_w;  // [D], or NULL: the cache already holds the new K/V
  void* k_cache;             // written only with k_norm_w
  void* v_cache;
  uint8_t* k_block_scale;    // E2M1: [Hkv, num_slots, D / 16]
  uint8_t* v_block_scale;
  float inv_k, inv_v;        // E4M3, E2M1: fp32(1 / scale), rounded on the host
  RopeFreqs freqs;
  RopeAxes axes;
  float eps;
  int32_t W;
  uint16_t* out;
  float* part_o;
  float* part_ml;
  KvIndex kv;
  int32_t* status;
  int32_t Hq, Hkv, G, split_len, max_splits;
  float scale_log2;  // log2(e) / sqrt(D), times k_scale for a cache of codes
  float v_scale;     // 1, or v_scale for a cache of codes
  // attention over listed blocks
  const uint16_t* q;          // [N, Hq, D] prepared
  const int32_t* cu_seqlens;  // NULL: one token per request
  const int32_t* list;        // [N, Hkv, keep]
  int32_t B, keep, log2_bs;
};

constexpr int kMaxSplitBlocks = 512;  // entries of a list that one split may take (4096 in at most 16 splits)

// What a split over listed blocks keeps of them in shared memory: the blocks that hold a
// visible key and their first slots.
template <bool Blocks>
struct SplitBlocks {};
template <>
struct SplitBlocks<true> {
  int block[kMaxSplitBlocks], slot[kMaxSplitBlocks], count;
};

// The tiles of 64 keys of a split: consecutive from k0 ...
template <bool Blocks>
struct Tiles {
  int k0, n;
  // First position of tile i.
  __device__ __forceinline__ int pos(int i, int) const { return k0 + i * kKeysPerTile; }
};
// ... or those of listed blocks.
template <>
struct Tiles<true> {
  const SplitBlocks<true>& list;
  int sh;  // log2 of the tiles per block
  int n;
  // First position of tile i; of a tile past the last (one that was not loaded) `past`.
  __device__ __forceinline__ int pos(int i, int past) const {
    if (i >= n) return past;
    return (list.block[i >> sh] << (sh + 6)) + ((i & ((1 << sh) - 1)) << 6);
  }
  // First slot of tile i < n, -64 for a page outside the cache.
  __device__ __forceinline__ int slot(int i) const {
    const int s = list.slot[i >> sh];
    return s < 0 ? -kKeysPerTile : s + ((i & ((1 << sh) - 1)) << 6);
  }
};

__device__ __forceinline__ void named_sync_consumers() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumerWarps * 32) : "memory");
}

// The new token of request b (position c_b): its K and V of KV head kh
// written to the cache by one warp in the prologue kernel's pair layout and
// arithmetic (lanes [0, D/16) K, lanes [D/16, D/8) V).  Each writer then
// orders its stores before later async-proxy (TMA) reads, and the
// __syncwarp hands that order to the lane that issues the tile loads.
template <int D, int KV, bool Axes>
__device__ __forceinline__ void append_new_kv(const DecodePar& p, const ReqInfo& r, int b, int kh, int lane) {
  constexpr int L = D / 16, H2 = D / 2;
  const int li = lane % L, which = lane / L;  // 0: K, 1: V, else idle
  const int64_t slot = cache_slot(p.kv, r, r.cached);
  uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
  if (which < 2) {
    const uint16_t* src = p.qkv + (int64_t)b * p.W + (int64_t)(p.Hq + which * p.Hkv + kh) * D + li * 8;
    xa = __ldg(reinterpret_cast<const uint4*>(src));
    xb = __ldg(reinterpret_cast<const uint4*>(src + H2));
  }
  const uint4 wa = __ldg(reinterpret_cast<const uint4*>(p.k_norm_w + li * 8));
  const uint4 wb = __ldg(reinterpret_cast<const uint4*>(p.k_norm_w + li * 8 + H2));
  float ra[8], rb[8];
  if constexpr (KV == ATTN_KV_E2M1) {
    F2 cs[8], sn[8];
    if constexpr (Axes) pair_angles_fine<D>(AxisPos{p.axes, b}, p.freqs, lane, cs, sn);
    else pair_angles_fine<D>(OnePos{(float)r.cached}, p.freqs, lane, cs, sn);
    norm_rope_pair_fine<D>(xa, xb, wa, wb, cs, sn, p.eps, ra, rb);
  } else {
    float cs[8], sn[8];
    if constexpr (Axes) pair_angles<D>(AxisPos{p.axes, b}, p.freqs, lane, cs, sn);
    else pair_angles<D>(OnePos{(float)r.cached}, p.freqs, lane, cs, sn);
    norm_rope_pair<D>(xa, xb, wa, wb, cs, sn, p.eps, ra, rb);
  }
  if constexpr (KV == ATTN_KV_E2M1) {
    if (which != 0) {
      unpack_bf16x8(xa, ra);
      unpack_bf16x8(xb, rb);
    }
    store_e2m1_pair<D>(ra, rb, which == 0 ? p.inv_k : p.inv_v, which < 2 && slot >= 0, li,
                       static_cast<uint8_t*>(which == 0 ? p.k_cache : p.v_cache) + (slot * p.Hkv + kh) * (D / 2),
                       (which == 0 ? p.k_block_scale : p.v_block_scale) +
                           ((int64_t)kh * p.kv.num_slots + slot) * (D / 16));
    asm volatile("fence.proxy.async.global;" ::: "memory");
  } else if (which < 2 && slot >= 0) {
    const int64_t e0 = (slot * p.Hkv + kh) * D + li * 8;
    if constexpr (KV == ATTN_KV_E4M3) {
      uint8_t* dst = static_cast<uint8_t*>(which == 0 ? p.k_cache : p.v_cache) + e0;
      if (which == 0) {
        *reinterpret_cast<uint2*>(dst) = e4m3x8(ra, p.inv_k);
        *reinterpret_cast<uint2*>(dst + H2) = e4m3x8(rb, p.inv_k);
      } else {
        float y[8];
        unpack_bf16x8(xa, y);
        *reinterpret_cast<uint2*>(dst) = e4m3x8(y, p.inv_v);
        unpack_bf16x8(xb, y);
        *reinterpret_cast<uint2*>(dst + H2) = e4m3x8(y, p.inv_v);
      }
    } else {
      uint16_t* dst = static_cast<uint16_t*>(which == 0 ? p.k_cache : p.v_cache) + e0;
      if (which == 0) {
        xa = make_uint4(pack_bf16(ra[0], ra[1]), pack_bf16(ra[2], ra[3]), pack_bf16(ra[4], ra[5]),
                        pack_bf16(ra[6], ra[7]));
        xb = make_uint4(pack_bf16(rb[0], rb[1]), pack_bf16(rb[2], rb[3]), pack_bf16(rb[4], rb[5]),
                        pack_bf16(rb[6], rb[7]));
      }
      *reinterpret_cast<uint4*>(dst) = xa;
      *reinterpret_cast<uint4*>(dst + H2) = xb;
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");
  }
  if (lane == 0 && slot < 0) set_status(p.status, ATTN_STATUS_CAPACITY);
  __syncwarp();
}

// The tiles of a split, which decode_begin() or blocks_begin() has set out.
template <bool Blocks>
__device__ __forceinline__ Tiles<Blocks> split_tiles(const DecodePar& p, const SplitBlocks<Blocks>& list, int k0, int k1) {
  if constexpr (Blocks) return Tiles<true>{list, p.log2_bs - 6, list.count << (p.log2_bs - 6)};
  else return Tiles<false>{k0, (k1 - k0 + kKeysPerTile - 1) / kKeysPerTile};
}

// The part of request b's keys that split `split` takes, [k0, k1), and how many
// splits the request spans; false: nothing to do (a request that is skipped, or
// past the host bound, whose new K/V are still appended).
template <int D, int KV, bool Axes>
__device__ __forceinline__ bool decode_begin(const DecodePar& p, int split, int kh, int b, ReqInfo* req, int* k0,
                                             int* k1, int* splits) {
  // Request facts: written by the caller, or by a page call, whose last kernel lets
  // no dependent start before it has completed.
  const ReqInfo r = load_request(p.kv, b, 1);
  const bool append = p.k_norm_w != nullptr;
  if (!r.valid) {  // nothing written (with the append kernel before this one: flagged there)
    if (append && split == 0 && kh == 0 && threadIdx.x == 0) set_status(p.status, ATTN_STATUS_CAPACITY);
    return false;
  }
  if (Axes && !axes_in_range(p.axes, b)) {  // nothing appended, no output
    if (split == 0 && kh == 0 && threadIdx.x == 0) set_status(p.status, ATTN_STATUS_POSITION);
    return false;
  }
  const int kv_len = r.cached + 1;
  const int n_splits = (kv_len + p.split_len - 1) / p.split_len;
  if (n_splits > p.max_splits) {  // max_cache_len below this request's length
    if (split == 0 && kh == 0 && threadIdx.x == 0) set_status(p.status, ATTN_STATUS_BOUNDS);
    if (append && split == p.max_splits - 1 && threadIdx.x < 32) {  // the new K/V are still appended
      grid_dependency_wait();
      append_new_kv<D, KV, Axes>(p, r, b, kh, threadIdx.x);
    }
    return false;
  }
  if (split >= n_splits) return false;
  *req = r;
  *k0 = split * p.split_len;
  *k1 = min(*k0 + p.split_len, kv_len);
  *splits = n_splits;
  return true;
}

// The same for token t over its listed blocks: the entries of the split that hold a
// visible key go to `mine` with their first slots (no page-table read stands before a tile's load
// then: one token over 65000 keys 9.0 -> 8.6 us); k1 is the end of the visible positions.
// False: a token without output.
__device__ __forceinline__ bool blocks_begin(const DecodePar& p, int split, int kh, int t, SplitBlocks<true>& mine,
                                             ReqInfo* req, int* k1) {
  const int lane = threadIdx.x & 31;
  const int32_t* list = p.list + ((int64_t)t * p.Hkv + kh) * p.keep;
  const int first = split * p.split_len, e1 = min(first + p.split_len, p.keep);
  int entry = threadIdx.x < 32 && first + lane < e1 ? __ldcg(list + first + lane) : -1;  // on its way with the lengths
  int b, n, j;
  const bool report = split == 0 && kh == 0 && threadIdx.x == 0;
  if (!find_token(p.cu_seqlens, p.B, t, &b, &n, &j)) {
    if (report) set_status(p.status, ATTN_STATUS_SEQLENS);
    return false;
  }
  const ReqInfo r = load_request(p.kv, b, n);
  if (!r.valid) {
    if (report) set_status(p.status, ATTN_STATUS_CAPACITY);
    return false;
  }
  const int end = r.cached + j + 1;
  if (threadIdx.x < 32) {
    int at = 0;
    for (int e0 = first; e0 < e1; e0 += 32) {
      const bool live = entry >= 0 && ((int64_t)entry << p.log2_bs) < end;
      const uint32_t all = __ballot_sync(0xffffffffu, live);
      if (live) {
        const int to = at + __popc(all & ((1u << lane) - 1u));
        const int slot = (int)block_slot(p.kv, r, entry << p.log2_bs);
        mine.block[to] = entry;
        mine.slot[to] = slot;
        if (slot < 0) set_status(p.status, ATTN_STATUS_CAPACITY);
      }
      at += __popc(all);
      entry = e0 + 32 + lane < e1 ? __ldcg(list + e0 + 32 + lane) : -1;
    }
    if (lane == 0) mine.count = at;
  }
  __syncthreads();
  *req = r;
  *k1 = end;
  return true;
}

// ---------------------------------------------------------------- merge of listed blocks
// The splits of a list are one cluster and merge through distributed shared memory: no
// partial results in memory and no second launch.
constexpr int kMaxSplits = 16;  // of a list: the largest cluster

// A split's maxima and sums, for its peers: at the same place in every CTA, and not among the
// stage buffers, where copies may still land when a wait has run out.
template <bool Blocks>
struct SplitSums {};
template <>
struct SplitSums<true> {
  float max[8], sum[8];  // a sum below 0: this split gave up
};

// The output rows of token t's group from the warps' partial results mo [warps][G][D], mm
// and ml [warps][G] (maximum, sum) of every split.  All consumer threads call this;
// the producer warp calls block_merge_rest().  A list may leave a warp, a split or the token
// without a key: their maxima are -inf, and no key at all gives zeros.  Where a split gave up
// (block_merge_none()) none of them stores.
template <int D>
__device__ __forceinline__ void block_merge(const DecodePar& p, float* mo, const float* mm, const float* ml,
                                            SplitSums<true>& mine, int kh, int t) {
  const int G = p.G, splits = p.max_splits;
  uint16_t* out = p.out + ((int64_t)t * p.Hq + kh * G) * D;
  auto store = [&](int idx, float acc, float L) {
    const __nv_bfloat16 v = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L);
    out[idx] = *reinterpret_cast<const uint16_t*>(&v);
  };
  for (int idx = threadIdx.x; idx < G * D; idx += kConsumerWarps * 32) {
    const int row = idx / D;
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, mm[w * G + row]);
    float L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) {
      const float sw = M == kNegInf ? 0.f : fast_exp2(mm[w * G + row] - M);
      L += sw * ml[w * G + row];
      acc += sw * mo[w * G * D + idx];
    }
    if (splits == 1) {
      store(idx, acc, L);
    } else {
      mo[idx] = acc;  // read by this thread only
      if (idx % D == 0) {
        mine.max[row] = M;
        mine.sum[row] = L;
      }
    }
  }
  if (splits == 1) return;
  cluster_sync();
  // a warp's 32 components are of one head: lane s looks at split s for the weights
  const int lane = threadIdx.x & 31;
  for (int i0 = (cluster_rank() * kConsumerWarps + (threadIdx.x >> 5)) * 32; i0 < G * D;
       i0 += splits * kConsumerWarps * 32) {
    const int idx = i0 + lane, row = i0 / D;
    float v[kMaxSplits];
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) v[s] = s < splits ? peer_f32(smem_u32(mo + idx), s) : 0.f;
    const bool there = lane < splits;
    const float ms = there ? peer_f32(smem_u32(mine.max + row), lane) : kNegInf;
    float L = there ? peer_f32(smem_u32(mine.sum + row), lane) : 0.f, M = ms;
    const bool gone = __any_sync(0xffffffffu, L < 0.f);
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float w = M == kNegInf ? 0.f : fast_exp2(ms - M);
    L *= w;
    float acc = 0.f;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < splits) acc += __shfl_sync(0xffffffffu, w, s) * v[s];
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    L = __shfl_sync(0xffffffffu, L, 0);
    if (!gone) store(idx, acc, L);
  }
  cluster_sync();  // no CTA leaves while another reads from it
}
__device__ __forceinline__ void block_merge_rest(const DecodePar& p) {
  if (p.max_splits == 1) return;
  cluster_sync();
  cluster_sync();
}
// The consumer threads of a split whose wait ran out call this instead of block_merge().
__device__ __forceinline__ void block_merge_none(const DecodePar& p, SplitSums<true>& mine) {
  if (threadIdx.x < 8) mine.sum[threadIdx.x] = -1.f;
  block_merge_rest(p);
}

// The kernels' form of a call's arguments.
inline DecodePar decode_par(const DecodeArgs& a) {
  const int D = a.cfg.head_dim;
  const bool codes = a.kv.kv_dtype != ATTN_KV_BF16;
  DecodePar p;
  p.qkv = static_cast<const uint16_t*>(a.qkv);
  p.q_norm_w = static_cast<const uint16_t*>(a.q_norm_w);
  p.k_norm_w = static_cast<const uint16_t*>(a.k_norm_w);
  p.k_cache = a.kv.k_cache;
  p.v_cache = a.kv.v_cache;
  p.k_block_scale = static_cast<uint8_t*>(a.kv.k_block_scale);
  p.v_block_scale = static_cast<uint8_t*>(a.kv.v_block_scale);
  p.inv_k = inv_scale(a.kv, a.kv.k_scale);
  p.inv_v = inv_scale(a.kv, a.kv.v_scale);
  p.freqs = a.freqs;
  p.axes = a.axes;
  p.eps = a.cfg.rms_eps;
  p.W = (a.cfg.num_q_heads + 2 * a.cfg.num_kv_heads) * D;
  p.out = static_cast<uint16_t*>(a.out);
  p.part_o = a.part_o;
  p.part_ml = a.part_ml;
  p.kv = kv_index(a.kv);
  p.status = a.status;
  p.Hq = a.cfg.num_q_heads;
  p.Hkv = a.cfg.num_kv_heads;
  p.G = a.cfg.num_q_heads / a.cfg.num_kv_heads;
  p.split_len = a.split_len;
  p.max_splits = a.max_splits;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)D) * (codes ? a.kv.k_scale : 1.0f);
  p.v_scale = codes ? a.kv.v_scale : 1.0f;
  p.q = static_cast<const uint16_t*>(a.q);
  p.cu_seqlens = a.cu_seqlens;
  p.list = a.list;
  p.B = a.B;
  p.keep = a.keep;
  p.log2_bs = a.log2_bs;
  return p;
}

// Launch of a split kernel over listed blocks: the splits of a (token, KV head) form a cluster.
template <typename Kernel>
int launch_block_splits(Kernel kernel, size_t smem, const DecodeArgs& a, const CacheMaps& maps, cudaStream_t stream) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATTN_ELAUNCH;
  return launch_cluster_dependent(kernel, dim3((unsigned)(a.N * a.max_splits), a.cfg.num_kv_heads), dim3(kThreads), smem,
                                  a.max_splits, stream, maps.k, maps.v, decode_par(a)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // namespace

}  // namespace gb300
