// Prologue of the attention step: split qkv, RMSNorm + RoPE on K (and on Q
// when a Q output is given), write K and V to the cache (and the prepared Q).
//
// Zero-to-sglang Ch.3 code walkthrough, section 3.3: AttentionLayer.forward
// splits the merged projection into Q, K and V, applies RMSNorm to each Q/K
// head's last dimension and RoPE at each token's position (V is not rotated);
// transformer-basics "Prefill vs Decode": the new K/V are appended to the
// per-layer cache (past_key_values.update).  One pass: every (token, head)
// vector of D bf16 values is read once with 16-byte loads by a group of D/16
// lanes, reduced with warp shuffles, and written once.
#include "kernels.cuh"

namespace gb300 {

namespace {

constexpr int kWarpsPerBlock = 8;  // each warp takes one run of (token, step) units
constexpr int kThreads = kWarpsPerBlock * 32;
#ifndef PROLOGUE_BATCH
#define PROLOGUE_BATCH 6
#endif
#ifndef PROLOGUE_BATCH_F8
#define PROLOGUE_BATCH_F8 4
#endif
#ifndef PROLOGUE_BATCH_F4
#define PROLOGUE_BATCH_F4 2
#endif
#ifndef PROLOGUE_MIN_BLOCKS
#define PROLOGUE_MIN_BLOCKS 2
#endif
// steps whose loads are issued before processing (bf16 cache, E4M3 cache):
// as many as fit in the registers two blocks per SM allow
constexpr int kBatchBf16 = PROLOGUE_BATCH;
constexpr int kBatchF8 = PROLOGUE_BATCH_F8;
constexpr int kBatchF4 = PROLOGUE_BATCH_F4;
constexpr int kMinBlocks = PROLOGUE_MIN_BLOCKS;  // resident blocks per SM the registers allow

struct ProloguePar {
  const uint16_t* __restrict__ qkv;        // [N, W] bf16
  const uint16_t* __restrict__ q_norm_w;   // [D] bf16 (used when q_out != NULL)
  const uint16_t* __restrict__ k_norm_w;   // [D] bf16
  uint16_t* __restrict__ q_out;            // [N, Hq, D] bf16 or NULL
  const int32_t* cu_seqlens;  // [B+1] or NULL: token b is request b (decode)
  void* __restrict__ k_cache;  // bf16, or codes (E4M3: one byte per entry, E2M1: half a byte)
  void* __restrict__ v_cache;
  uint8_t* __restrict__ k_block_scale;  // E2M1: [Hkv, num_slots, D/16]
  uint8_t* __restrict__ v_block_scale;
  float inv_k, inv_v;          // E4M3, E2M1: fp32(1 / scale), rounded on the host
  KvIndex kv;
  int32_t* status;
  int32_t B, N, Hq, Hkv;
  int64_t steps_per_warp;  // each warp takes this many consecutive (token, step) units
  float eps;
  RopeFreqs freqs;
  RopeAxes axes;
};

// One warp per token.  A head vector (D bf16) is held by L = D/16 lanes, lane
// li taking the 8 values at 8*li and the 8 values at D/2 + 8*li: the two
// members of each rotation pair (i, i + D/2) sit in the same lane, so RoPE
// needs no data exchange and the norm's sum of squares needs log2(L) shuffles.
// HPI = 32 / L head vectors are taken per step; each load instruction reads
// HPI runs of 128 contiguous bytes and each store writes whole runs.  cos/sin
// of the token's D/2 rotation angles are computed once (D/64 per lane) and
// handed to the lanes that need them with shuffles.  KV: the cache's element
// type (ATTN_KV_*).  Axes: rotary positions with several axes; a lane holds the
// positions of its own D/64 pairs, read one token ahead (32768 tokens, Hq 32, Hkv 8,
// D 128, three axes: 132 us, 6.1 TB/s, the same as without axes; read where they are
// used: 143).  E2M1: the fine K and the codes bound the 9942-token Qwen3-4B prologue
// at 69 us, where a bf16 cache takes 43.4.
template <int D, int KV, bool Axes>
__global__ void __launch_bounds__(kThreads, kMinBlocks) kv_append_kernel(const ProloguePar p) {
  constexpr int L = D / 16;     // lanes per head vector
  constexpr int HPI = 32 / L;   // head vectors per warp-wide step
  constexpr int H2 = D / 2;     // offset of the second member of a rotation pair
  constexpr bool F8 = KV == ATTN_KV_E4M3, F4 = KV == ATTN_KV_E2M1;
  constexpr int kBatch = F4 ? kBatchF4 : F8 ? kBatchF8 : kBatchBf16;
  const int lane = threadIdx.x & 31;
  launch_dependents();  // the attention kernel after this one may be scheduled as CTAs finish

  const bool with_q = p.q_out != nullptr;
  const int hd0 = with_q ? 0 : p.Hq;               // first head handled (Q heads only with q_out)
  const int nhead = p.Hq + 2 * p.Hkv - hd0;
  const int nstep = (nhead + HPI - 1) / HPI;
  const int64_t W = (int64_t)(p.Hq + 2 * p.Hkv) * D;
  const int li = lane % L;
  const int sub = lane / L;                        // head slot within a step

  uint4 qw[2], kw[2];  // norm weights of this lane's 16 values, bf16 pairs
  {
    const uint16_t* wk = p.k_norm_w + li * 8;
    const uint16_t* wq = with_q ? p.q_norm_w + li * 8 : wk;
    kw[0] = __ldg(reinterpret_cast<const uint4*>(wk));
    kw[1] = __ldg(reinterpret_cast<const uint4*>(wk + H2));
    qw[0] = __ldg(reinterpret_cast<const uint4*>(wq));
    qw[1] = __ldg(reinterpret_cast<const uint4*>(wq + H2));
  }

  // this warp's units: steps [u0, u_end) of the N x nstep (token, step) grid,
  // the same count for every warp so that all of them finish together
  int64_t u0 = ((int64_t)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5)) * p.steps_per_warp;
  const int64_t u_end = min((int64_t)p.N * nstep, u0 + p.steps_per_warp);
  if (u0 >= u_end) return;
  int t = (int)(u0 / nstep);
  int s_begin = (int)(u0 - (int64_t)t * nstep);
  constexpr int PPL = D / 64;
  int32_t next_pos[PPL];  // Axes: positions of the coming token
  auto load_positions = [&](int token) {
#pragma unroll
    for (int e = 0; e < PPL; ++e) {
      const int pair = lane * PPL + e;
      const uint32_t a = (p.axes.axis[pair >> 4] >> (2 * (pair & 15))) & 3u;
      next_pos[e] = __ldg(p.axes.positions + (int64_t)a * p.axes.ld + token);
    }
  };
  if constexpr (Axes) load_positions(t);
  for (;;) {
    const int s_end = (int)min((int64_t)nstep, s_begin + (u_end - u0));
    const uint16_t* row = p.qkv + (int64_t)t * W + (int64_t)hd0 * D + li * 8;

    // first batch of loads before anything that depends on the request lookup
    uint4 raw_a[kBatch], raw_b[kBatch];  // values 8*li.. and D/2 + 8*li.. of a head
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int hd = (s_begin + k) * HPI + sub;
      const bool in = s_begin + k < s_end && hd < nhead;
      const uint16_t* src = row + (int64_t)hd * D;
      raw_a[k] = in ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      raw_b[k] = in ? __ldg(reinterpret_cast<const uint4*>(src + H2)) : make_uint4(0, 0, 0, 0);
    }

    // request of this token: 0 = none, 1 = Q only (region too small), 2 = Q and cache
    int ok = 0;
    int64_t slot = 0;
    float pos = 0.f;
    {
      int b = t, j = 0, n = 1;
      bool seq_ok = true;
      if (p.cu_seqlens) {
        int lo = 0, hi = p.B;  // largest b with cu[b] <= t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
        }
        b = lo;
        const int c0 = __ldg(p.cu_seqlens + b);
        j = t - c0;
        n = __ldg(p.cu_seqlens + b + 1) - c0;
        seq_ok = j >= 0 && j < n;
        if (!seq_ok && lane == 0) set_status(p.status, ATTN_STATUS_SEQLENS);
        if (t == 0 && lane == 0 && __ldg(p.cu_seqlens + p.B) != p.N) set_status(p.status, ATTN_STATUS_SEQLENS);
      }
      if (seq_ok) {
        const ReqInfo r = load_request(p.kv, b, n);
        ok = 1;
        pos = (float)(r.cached + j);
        slot = r.valid ? cache_slot(p.kv, r, r.cached + j) : -1;
        if (slot >= 0)
          ok = 2;
        else if (lane == 0)
          set_status(p.status, ATTN_STATUS_CAPACITY);
      }
    }
    LanePos<PPL> own;
    if constexpr (Axes) {
      bool in_range = true;
#pragma unroll
      for (int e = 0; e < PPL; ++e) {
        own.pos[e] = (float)next_pos[e];
        in_range = in_range && (uint32_t)next_pos[e] <= kMaxPosition;
      }
      if (u_end - u0 > s_end - s_begin) load_positions(t + 1);
      if (!__all_sync(0xffffffffu, in_range) && ok != 0) {
        ok = 0;
        if (lane == 0) set_status(p.status, ATTN_STATUS_POSITION);
      }
    }
    if (ok != 0) {  // warp-uniform

      // cos/sin of the 8 rotation pairs 8*li .. 8*li + 7 this lane's values belong to
      float cs[8], sn[8];
      F2 cs2[F4 ? 8 : 1], sn2[F4 ? 8 : 1];  // E2M1: K is rotated to the last bit of fp32
      auto angles = [&](const auto& at) {
        if constexpr (F4) {
          pair_angles_fine<D>(at, p.freqs, lane, cs2, sn2);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            cs[e] = cs2[e].hi;
            sn[e] = sn2[e].hi;
          }
        } else {
          pair_angles<D>(at, p.freqs, lane, cs, sn);
        }
      };
      if constexpr (Axes) angles(own);
      else angles(OnePos{pos});
      uint16_t* q_row = with_q ? p.q_out + (int64_t)t * p.Hq * D + li * 8 : nullptr;
      const int64_t cache_row = slot * p.Hkv * D + li * 8;

      for (int base = s_begin; base < s_end; base += kBatch) {
        if (base > s_begin) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int hd = (base + k) * HPI + sub;
            const bool in = base + k < s_end && hd < nhead;
            const uint16_t* src = row + (int64_t)hd * D;
            raw_a[k] = in ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            raw_b[k] = in ? __ldg(reinterpret_cast<const uint4*>(src + H2)) : make_uint4(0, 0, 0, 0);
          }
        }
        // step base + k, whose values are xa and xb
        auto step = [&](int k, const uint4& xa, const uint4& xb) {
          const int hd = hd0 + (base + k) * HPI + sub;  // head index in the qkv row
          const bool live = hd < p.Hq + 2 * p.Hkv;
          const bool is_q = hd < p.Hq;
          const bool is_v = hd >= p.Hq + p.Hkv;
          // steps made only of V heads: bit copies into the cache
          const bool step_all_v = hd0 + (base + k) * HPI >= p.Hq + p.Hkv;
          if (F4 && step_all_v) {
            const int kvh = live ? hd - p.Hq - p.Hkv : 0;
            float fa[8], fb[8];
            unpack_bf16x8(xa, fa);
            unpack_bf16x8(xb, fb);
            store_e2m1_pair<D>(fa, fb, p.inv_v, live && ok == 2, li,
                               static_cast<uint8_t*>(p.v_cache) + (slot * p.Hkv + kvh) * (D / 2),
                               p.v_block_scale + (kvh * p.kv.num_slots + slot) * (D / 16));
            return;
          }
          if (step_all_v) {
            if (live && ok == 2) {
              const int64_t e0 = cache_row + (int64_t)(hd - p.Hq - p.Hkv) * D;
              if constexpr (F8) {
                float y[8];
                uint8_t* dst = static_cast<uint8_t*>(p.v_cache) + e0;
                unpack_bf16x8(xa, y);
                *reinterpret_cast<uint2*>(dst) = e4m3x8(y, p.inv_v);
                unpack_bf16x8(xb, y);
                *reinterpret_cast<uint2*>(dst + H2) = e4m3x8(y, p.inv_v);
              } else {
                uint16_t* dst = static_cast<uint16_t*>(p.v_cache) + e0;
                *reinterpret_cast<uint4*>(dst) = xa;
                *reinterpret_cast<uint4*>(dst + H2) = xb;
              }
            }
            return;
          }
          float ra[8], rb[8];
          const bool with_k = hd0 + (base + k) * HPI + HPI > p.Hq;  // step-uniform
          if constexpr (F4) {
            if (with_k)
              norm_rope_pair_fine<D>(xa, xb, is_q ? qw[0] : kw[0], is_q ? qw[1] : kw[1], cs2, sn2, p.eps, ra, rb);
            else
              norm_rope_pair<D>(xa, xb, qw[0], qw[1], cs, sn, p.eps, ra, rb);
          } else {
            norm_rope_pair<D>(xa, xb, is_q ? qw[0] : kw[0], is_q ? qw[1] : kw[1], cs, sn, p.eps, ra, rb);
          }
          if constexpr (F4) {  // K heads, and V heads in a step that they share (all lanes: it shuffles)
            if (with_k) {
              const int kvh = live ? hd - (is_v ? p.Hq + p.Hkv : p.Hq) : 0;
              const int64_t at = kvh > 0 ? kvh : 0;
              float fa[8], fb[8];
              if (is_v) {
                unpack_bf16x8(xa, fa);
                unpack_bf16x8(xb, fb);
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  fa[e] = ra[e];
                  fb[e] = rb[e];
                }
              }
              store_e2m1_pair<D>(fa, fb, is_v ? p.inv_v : p.inv_k, live && !is_q && ok == 2, li,
                                 static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + (slot * p.Hkv + at) * (D / 2),
                                 (is_v ? p.v_block_scale : p.k_block_scale) + (at * p.kv.num_slots + slot) * (D / 16));
            }
            if (!is_q) return;
          }
          if (!live) return;
          const int64_t e0 = cache_row + (int64_t)(hd - (is_v ? p.Hq + p.Hkv : p.Hq)) * D;
          if (F8 && !is_q) {
            if (ok == 2) {
              uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + e0;
              const float r = is_v ? p.inv_v : p.inv_k;
              float ya[8], yb[8];
              if (is_v) {
                unpack_bf16x8(xa, ya);
                unpack_bf16x8(xb, yb);
              }
              *reinterpret_cast<uint2*>(dst) = e4m3x8(is_v ? ya : ra, r);
              *reinterpret_cast<uint2*>(dst + H2) = e4m3x8(is_v ? yb : rb, r);
            }
            return;
          }
          // the prepared Q is f16 next to a cache of codes (the prefill kernel's operand type), else bf16
          uint4 va, vb;
          if (is_v) {
            va = xa;
            vb = xb;
          } else if (F8 || F4) {
            va = make_uint4(pack_f16(ra[0], ra[1]), pack_f16(ra[2], ra[3]), pack_f16(ra[4], ra[5]), pack_f16(ra[6], ra[7]));
            vb = make_uint4(pack_f16(rb[0], rb[1]), pack_f16(rb[2], rb[3]), pack_f16(rb[4], rb[5]), pack_f16(rb[6], rb[7]));
          } else {
            va = make_uint4(pack_bf16(ra[0], ra[1]), pack_bf16(ra[2], ra[3]), pack_bf16(ra[4], ra[5]),
                            pack_bf16(ra[6], ra[7]));
            vb = make_uint4(pack_bf16(rb[0], rb[1]), pack_bf16(rb[2], rb[3]), pack_bf16(rb[4], rb[5]),
                            pack_bf16(rb[6], rb[7]));
          }
          uint16_t* dst = is_q ? q_row + (int64_t)hd * D
                               : static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + e0;
          if (is_q || ok == 2) {
            *reinterpret_cast<uint4*>(dst) = va;
            *reinterpret_cast<uint4*>(dst + H2) = vb;
          }
        };
        if constexpr (F4) {
          // One copy of the (long) body, the batch shifted through its first place:
          // unrolled it overflows the instruction cache (prepare of the Qwen3-4B
          // prefill: 83 us with two copies, 115 us with four, 70 us so).
#pragma unroll 1
          for (int k = 0; k < kBatch && base + k < s_end; ++k) {
            step(k, raw_a[0], raw_b[0]);
#pragma unroll
            for (int e = 0; e + 1 < kBatch; ++e) {
              raw_a[e] = raw_a[e + 1];
              raw_b[e] = raw_b[e + 1];
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (base + k >= s_end) break;  // warp-uniform
            step(k, raw_a[k], raw_b[k]);
          }
        }
      }
    }  // ok != 0
    u0 += s_end - s_begin;
    if (u0 >= u_end) break;
    ++t;
    s_begin = 0;
  }
}

template <bool Axes>
void launch_kv(int kv_dtype, int head_dim, const ProloguePar& p, dim3 grid, cudaStream_t stream) {
  switch (kv_dtype * 2 + (head_dim == 128)) {
    case ATTN_KV_BF16 * 2: kv_append_kernel<64, ATTN_KV_BF16, Axes><<<grid, kThreads, 0, stream>>>(p); break;
    case ATTN_KV_BF16 * 2 + 1: kv_append_kernel<128, ATTN_KV_BF16, Axes><<<grid, kThreads, 0, stream>>>(p); break;
    case ATTN_KV_E4M3 * 2: kv_append_kernel<64, ATTN_KV_E4M3, Axes><<<grid, kThreads, 0, stream>>>(p); break;
    case ATTN_KV_E4M3 * 2 + 1: kv_append_kernel<128, ATTN_KV_E4M3, Axes><<<grid, kThreads, 0, stream>>>(p); break;
    case ATTN_KV_E2M1 * 2: kv_append_kernel<64, ATTN_KV_E2M1, Axes><<<grid, kThreads, 0, stream>>>(p); break;
    default: kv_append_kernel<128, ATTN_KV_E2M1, Axes><<<grid, kThreads, 0, stream>>>(p); break;
  }
}

}  // namespace

cudaError_t launch_prologue(const PrologueArgs& a, cudaStream_t stream) {
  if (a.N <= 0) return cudaSuccess;
  ProloguePar p;
  p.qkv = static_cast<const uint16_t*>(a.qkv);
  p.q_norm_w = static_cast<const uint16_t*>(a.q_norm_w);
  p.k_norm_w = static_cast<const uint16_t*>(a.k_norm_w);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.cu_seqlens = a.cu_seqlens;
  p.k_cache = a.kv.k_cache;
  p.v_cache = a.kv.v_cache;
  p.k_block_scale = static_cast<uint8_t*>(a.kv.k_block_scale);
  p.v_block_scale = static_cast<uint8_t*>(a.kv.v_block_scale);
  p.inv_k = inv_scale(a.kv, a.kv.k_scale);
  p.inv_v = inv_scale(a.kv, a.kv.v_scale);
  p.kv = kv_index(a.kv);
  p.status = a.status;
  p.B = a.B;
  p.N = a.N;
  p.Hq = a.cfg.num_q_heads;
  p.Hkv = a.cfg.num_kv_heads;
  p.eps = a.cfg.rms_eps;
  p.freqs = a.freqs;
  p.axes = a.axes;
  // (token, step) units: a step covers 32 / (D/16) head vectors of a token.
  // Warps take equal runs of consecutive units, cut across token boundaries:
  // with more units than the resident warps (kMinBlocks blocks per SM) every
  // resident warp takes one run, else every unit gets a warp of its own (a
  // decode append is latency-bound: its steps run side by side).
  const int hpi = 512 / a.cfg.head_dim;
  const int nstep = (a.cfg.num_q_heads * (a.q_out ? 1 : 0) + 2 * a.cfg.num_kv_heads + hpi - 1) / hpi;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return cudaErrorInvalidDevice;
  const int64_t units = (int64_t)a.N * nstep;
  const int64_t resident = (int64_t)sms * kMinBlocks * kWarpsPerBlock;
  p.steps_per_warp = (units + resident - 1) / resident;
  const int64_t warps = (units + p.steps_per_warp - 1) / p.steps_per_warp;
  const dim3 grid((unsigned)((warps + kWarpsPerBlock - 1) / kWarpsPerBlock));
  if (a.axes.positions) launch_kv<true>(a.kv.kv_dtype, a.cfg.head_dim, p, grid, stream);
  else launch_kv<false>(a.kv.kv_dtype, a.cfg.head_dim, p, grid, stream);
  return cudaGetLastError();
}

}  // namespace gb300
