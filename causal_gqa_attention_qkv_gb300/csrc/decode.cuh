// What the decode kernels share: their parameters, the append of the new token
// and the split of a request's keys.
#pragma once

#include "kernels.cuh"

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
  return p;
}

}  // namespace

}  // namespace gb300
