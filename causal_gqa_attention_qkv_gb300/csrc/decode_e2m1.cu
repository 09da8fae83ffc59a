// Decode over an E2M1 cache: the split kernel of decode.cu for four-bit codes
// with block scales.
//
// out = softmax(q K^T / sqrt(D)) V for one new token per request, K and V
// entries code * s_block * scale.  A decode step reads every cached byte once:
// D/2 + D/16 bytes per entry vector, a quarter (and an eighth of a byte per
// entry) of what the bf16 kernel reads.  What bounds the kernel is therefore as
// much the work per byte: every code has to become an f16 operand (one
// conversion and one product with its block scale for two codes), so the layout
// below is chosen to need nothing else per code.  64 requests of 512 .. 8192 keys
// (Hkv 8, D 128, 322 MB): 79 us on the device, 4.1 TB/s; the loads by themselves
// take 65 us, the products 74.  16 requests of 30001 .. 65000 keys with groups of 8
// (876 MB): 188 us with the gather of the new entries, 4.7 TB/s; 152 and 161.
//
// Same grid as decode.cu: (split, KV head, request).  A producer warp brings stages
// of 2 x 64 keys, codes by TMA, block scales by untiled bulk copies (a head's scales
// of consecutive slots are contiguous); four consumer warps take 16 keys of each half.
//   S^T = K Q^T: keys are the M dimension of m16n8k16, heads the N dimension.
//     Quad member q takes the columns [q D/4, (q+1) D/4) of its key rows (16
//     contiguous bytes), so an A register is one converted byte: columns 2j and
//     2j + 1 of one key, scaled by one pair (s, s).
//   O^T = V^T P^T with groups of up to 4 heads: the k slots are (key, parity): slots
//     2q and 2q + 1 hold the entries 2j and 2j + 1 of one key, again one converted
//     byte, and the N dimension holds the 4 heads for the even and the same 4 for
//     the odd entries: column (head, parity) of P^T is p at its own parity's slots,
//     0 at the others.  V needs no interleaving of two keys' codes, and O takes D/8
//     registers per lane.
//   With 8 heads that would double the products.  A legacy m16n8k16 holds the
//     issue port for 8 cycles here, as much as 8 conversions, so there the codes of
//     two keys are interleaved instead (k slots = keys, one pair (s, s') of scales).
//   The softmax reference moves only when a score passes it by 2^8 (a vote over
//     the warp): P stays below 256, exact in f16's range, and the reductions
//     over keys and the rescaling of O are left out of most passes.
#include "decode.cuh"

namespace gb300 {

namespace {

#ifndef DECODE_F4_STAGES
#define DECODE_F4_STAGES 3
#endif
#ifndef DECODE_F4_MIN_BLOCKS
#define DECODE_F4_MIN_BLOCKS 3
#endif

constexpr float kRescaleThreshold = 8.f;  // log2 units

// A stage: two halves of 64 keys.  Per half one box of 64 rows x D / 2 bytes of K
// and of V codes (64-byte swizzled when D = 128) and the keys' block scales, D / 16
// bytes per key.  A bulk copy starts on 16 bytes, a key's scales on D / 16: the
// copy starts up to 12 bytes early, the same for every tile of a CTA.
template <int D>
struct E2m1Layout {
  static constexpr int kTileBytes = kKeysPerTile * (D / 2);         // codes of a half
  static constexpr int kScaleBytes = kKeysPerTile * (D / 16) + 16;  // block scales of a half
  static constexpr int kV = 2 * kTileBytes;                         // offsets in a stage: K codes, V codes,
  static constexpr int kKs = 4 * kTileBytes;                        // K scales, V scales (two halves each)
  static constexpr int kVs = kKs + 2 * kScaleBytes;
  static constexpr int kStageBytes = (kVs + 2 * kScaleBytes + 511) / 512 * 512;
  static constexpr int kStages = DECODE_F4_STAGES * 128 / D;
  static constexpr int kQOffset = kStages * kStageBytes;            // prepared Q: 8 heads x D f16
  static constexpr int kBarOffset = kQOffset + 8 * D * 2;
  static constexpr int kSmemBytes = kBarOffset + 2 * kStages * 8 + 1024;  // + alignment slack
  static_assert(kQOffset >= kConsumerWarps * 8 * D * 4 + 2 * kConsumerWarps * 8 * 4, "the warps' partial results fit the stages");
};

// Byte offset of `byte` of key row `key` in a tile of codes (D = 128: the 16-byte
// chunk index XORed with the row index / 2 modulo 4).
template <int D>
__device__ __forceinline__ uint32_t code_off(uint32_t key, uint32_t byte) {
  return D == 128 ? key * 64u + (byte ^ (((key >> 1) & 3u) << 4)) : key * (uint32_t)(D / 2) + byte;
}

// Which of its 8 keys row r of an S fragment holds.  With these the rows that one
// shared-memory access touches fall into different banks, for the K reads (8
// lanes: rows r, r + 1) and the V reads (16 lanes: rows 0, 2, 4, 6 or 1, 3, 5, 7)
// alike.
__device__ __forceinline__ int key_of_row(int r) { return (int)((0x65742130u >> (4 * r)) & 7u); }

// Untiled copy global -> shared (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The group's query heads normed and rotated (the prologue kernel's arithmetic)
// as f16 rows in shared memory, heads [G, 4 or 8) zero.  A warp takes 512 / D heads.
template <int D, bool Wide, bool Axes>
__device__ __forceinline__ void stage_q(const DecodePar& p, const ReqInfo& r, int b, int kh, int warp, int lane,
                                        uint8_t* q_smem) {
  constexpr int L = D / 16, HPW = 32 / L, H2 = D / 2, NH = Wide ? 8 : 4;
  if (warp * HPW >= NH) return;
  const int li = lane % L, head = warp * HPW + lane / L;
  const bool live = head < p.G;
  uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
  if (live) {
    const uint16_t* src = p.qkv + (int64_t)b * p.W + (int64_t)(kh * p.G + head) * D + li * 8;
    xa = __ldg(reinterpret_cast<const uint4*>(src));
    xb = __ldg(reinterpret_cast<const uint4*>(src + H2));
  }
  const uint4 wa = __ldg(reinterpret_cast<const uint4*>(p.q_norm_w + li * 8));
  const uint4 wb = __ldg(reinterpret_cast<const uint4*>(p.q_norm_w + li * 8 + H2));
  float cs[8], sn[8], ra[8], rb[8];
  if constexpr (Axes) pair_angles<D>(AxisPos{p.axes, b}, p.freqs, lane, cs, sn);
  else pair_angles<D>(OnePos{(float)r.cached}, p.freqs, lane, cs, sn);
  norm_rope_pair<D>(xa, xb, wa, wb, cs, sn, p.eps, ra, rb);
  if (head >= NH) return;
  uint4 va = make_uint4(0, 0, 0, 0), vb = va;
  if (live) {
    va = make_uint4(pack_f16(ra[0], ra[1]), pack_f16(ra[2], ra[3]), pack_f16(ra[4], ra[5]), pack_f16(ra[6], ra[7]));
    vb = make_uint4(pack_f16(rb[0], rb[1]), pack_f16(rb[2], rb[3]), pack_f16(rb[4], rb[5]), pack_f16(rb[6], rb[7]));
  }
  uint8_t* dst = q_smem + head * (D * 2) + li * 16;
  *reinterpret_cast<uint4*>(dst) = va;
  *reinterpret_cast<uint4*>(dst + D) = vb;
}

// The same from prepared rows [Hq, D] f16.
template <int D, bool Wide>
__device__ __forceinline__ void copy_q(const uint16_t* q, int G, int thread, uint8_t* q_smem) {
  constexpr int NH = Wide ? 8 : 4, C = D / 8;  // 16-byte chunks per head
  for (int i = thread; i < NH * C; i += kConsumerWarps * 32) {
    const uint4 v = i / C < G ? __ldg(reinterpret_cast<const uint4*>(q) + i) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(q_smem + i * 16) = v;
  }
}

// Wide: groups of more than 4 query heads.  Blocks: the keys of listed blocks, as in decode.cu.
template <int D, bool Wide, bool Axes, bool Blocks>
__global__ void __launch_bounds__(kThreads, DECODE_F4_MIN_BLOCKS)
    decode_split_e2m1_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                             const DecodePar p) {
  using Lay = E2m1Layout<D>;
  constexpr int S = Lay::kStages, NH = Wide ? 8 : 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Lay::kBarOffset);
  uint64_t* empty = full + S;
  __shared__ int s_cons_abort;  // written by consumers only, read after their barrier

  __shared__ SplitBlocks<Blocks> s_list;
  __shared__ SplitSums<Blocks> s_sums;

  // b: the request, or the token (Blocks)
  const int split = Blocks ? blockIdx.x % p.max_splits : blockIdx.x, kh = blockIdx.y;
  const int b = Blocks ? blockIdx.x / p.max_splits : blockIdx.z;
  if (!Blocks) launch_dependents();  // the merge kernel may be scheduled as CTAs finish
  ReqInfo r;
  int k0 = 0, k1, n_splits;
  if constexpr (Blocks) {
    grid_dependency_wait();  // the list
    launch_dependents();  // behind the wait: a decode kernel reads the lengths before its own
    if (!blocks_begin(p, split, kh, b, s_list, &r, &k1)) return;
    n_splits = p.max_splits;
  } else {
    if (!decode_begin<D, ATTN_KV_E2M1, Axes>(p, split, kh, b, &r, &k0, &k1, &n_splits)) return;
  }
  const Tiles<Blocks> tiles = split_tiles<Blocks>(p, s_list, k0, k1);
  const int npass = Blocks ? (tiles.n + 1) / 2 : (k1 - k0 + 2 * kKeysPerTile - 1) / (2 * kKeysPerTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kConsumerWarps);
    }
    s_cons_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (!Blocks) grid_dependency_wait();  // the append kernel's cache entries, earlier kernels' reads of the outputs

  if (warp == kConsumerWarps) {  // ---------------- producer warp
    const bool append = !Blocks && p.k_norm_w && split == n_splits - 1;  // the new token's key is in the last stage
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&vmap);
    }
    constexpr uint32_t SB = D / 16;  // bytes of block scales per key
    const int64_t row0 = (int64_t)kh * p.kv.num_slots;
    const int64_t end = (int64_t)p.Hkv * p.kv.num_slots * SB;
    // First slots of the tiles [w0, w0 + 32) (slot_now, one per lane) and of the 32 after
    // them, read ahead: no page-table read stands between a free stage and its refill.
    const int ntiles = tiles.n;
    // A page outside the cache reads as zeros; its scales are not read.
    auto tile_slot = [&](int t) -> int64_t {
      if constexpr (Blocks) return t < ntiles ? tiles.slot(t) : 0;
      else return t < ntiles ? cache_slot(p.kv, r, tiles.pos(t, 0), -kKeysPerTile) : 0;
    };
    int w0 = 0;
    int64_t slot_now = tile_slot(lane), slot_next = tile_slot(32 + lane);
    int issued = 0, st = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < npass; ++i) {
      if (2 * i >= w0 + 32) {
        w0 += 32;
        slot_now = slot_next;
        slot_next = tile_slot(w0 + 32 + lane);
      }
      if (i >= S) ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1));
      if (!ok) break;
      if constexpr (!Blocks)
        if (append && i == npass - 1) append_new_kv<D, ATTN_KV_E2M1, Axes>(p, r, b, kh, lane);
      const int halves = min(2, ntiles - 2 * i);
      const uint32_t stage = smem_u32(smem) + st * Lay::kStageBytes;
      // Lanes 0 .. 3 issue the copies of K and V (bit 0) of the halves (bit 1): one
      // lane issuing all eight in turn cost 4 % of the call.
      const int which = lane & 1, half = (lane >> 1) & 1;
      const bool issues = lane < 2 * halves;
      const int64_t slot = __shfl_sync(0xffffffffu, slot_now, 2 * i - w0 + half);
      // the same for every half of the CTA (a half past the end has no slot)
      const uint32_t shift = (uint32_t)((row0 + __shfl_sync(0xffffffffu, slot, 0)) * SB) & 15u;
      const uint32_t sbytes = kKeysPerTile * SB + (shift ? 16u : 0u);
      const int64_t at = (row0 + slot) * SB - shift;
      // else past the arrays, or a page outside the cache: key by key
      const bool bulk = __all_sync(0xffffffffu, !issues || (slot >= 0 && at + sbytes <= end));
      if (!bulk) {
        if (issues && slot < 0) set_status(p.status, ATTN_STATUS_CAPACITY);
        for (int h = 0; h < halves; ++h) {
          const int64_t from = __shfl_sync(0xffffffffu, at, 2 * h) + shift;
          const bool none = __shfl_sync(0xffffffffu, slot, 2 * h) < 0;
          for (int key = lane; key < kKeysPerTile; key += 32) {
            const int64_t a = from + key * SB;
            const bool in = !none && a + SB <= end;
            const uint32_t dst = stage + h * Lay::kScaleBytes + shift + key * SB;
            for (uint32_t w = 0; w < SB; w += 4) {
              const uint32_t x = in ? __ldcg(reinterpret_cast<const uint32_t*>(p.k_block_scale + a + w)) : 0u;
              const uint32_t y = in ? __ldcg(reinterpret_cast<const uint32_t*>(p.v_block_scale + a + w)) : 0u;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + Lay::kKs + w), "r"(x) : "memory");
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + Lay::kVs + w), "r"(y) : "memory");
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later bulk copy to the same place
        __syncwarp();  // before the arrival below
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[st], halves * 2 * (Lay::kTileBytes + (bulk ? sbytes : 0)));
      __syncwarp();
      if (issues) {
        tma_load_3d(smem + st * Lay::kStageBytes + (which ? Lay::kV : 0) + half * Lay::kTileBytes,
                    which ? &vmap : &kmap, &full[st], 0, kh, (int)slot);
        if (bulk)
          bulk_load(stage + (which ? Lay::kVs : Lay::kKs) + half * Lay::kScaleBytes,
                    (which ? p.v_block_scale : p.k_block_scale) + at, sbytes, &full[st]);
      }
      __syncwarp();
      issued = i + 1;
      if (++st == S) { st = 0; ph ^= 1; }
    }
    if (Blocks || !ok) {  // let the copies still in flight land before exit (as in decode.cu)
      for (int i = max(0, issued - S); i < issued; ++i) (void)mbar_wait(&full[i % S], (i / S) & 1);
      if (!ok && lane == 0) set_status(p.status, ATTN_STATUS_TIMEOUT);
    }
    if constexpr (Blocks) {
      __syncwarp();
      block_merge_rest(p);
    }
    return;
  }

  // ---------------- consumer warps: warp w owns keys [16w, 16w + 16) of each half
  const int G = p.G;
  const int g = lane >> 2, q = lane & 3;  // fragment row and quad member
  if constexpr (Blocks) copy_q<D, Wide>(p.q + ((int64_t)b * p.Hq + kh * G) * D, G, threadIdx.x, smem + Lay::kQOffset);
  else stage_q<D, Wide, Axes>(p, r, b, kh, warp, lane, smem + Lay::kQOffset);
  named_sync_consumers();
  uint32_t qb[D / 16][2];  // Q of S column g (head g mod NH): columns q D/4 + 4 ks + {0, 1} and {2, 3}
  {
    const uint32_t row = smem_u32(smem + Lay::kQOffset) + (g & (NH - 1)) * (D * 2) + q * (D / 2);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint4 v = lds128(row + 16 * c);
      qb[2 * c][0] = v.x;
      qb[2 * c][1] = v.y;
      qb[2 * c + 1][0] = v.z;
      qb[2 * c + 1][1] = v.w;
    }
  }
  // keys (of the warp's 16) of S row g and of the k slots 2q, 2q + 1; + 8 for the others
  const int key_g = key_of_row(g), key_a = key_of_row(2 * q), key_b = key_of_row(2 * q + 1);
  // p of a key as a B register: at this column's parity (g >> 2), the other half 0
  const uint32_t sel_a = g < 4 ? 0x4410u : 0x1044u, sel_b = g < 4 ? 0x4432u : 0x3244u;
  // O^T.  Wide: rows g, g + 8: d = g D/8 + 2 mt and + 1; columns 2q, 2q + 1 are heads.
  // Else: rows g, g + 8: bytes 2 mt, 2 mt + 1 of this lane's D/16; columns (head, parity).
  constexpr int MT = Wide ? D / 16 : D / 32;
  float o[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};  // S columns 2q, 2q + 1
  bool ok = true;

  // this lane's offsets in a stage: codes of its K keys and V keys, their block scales
  const uint32_t shift =
      (uint32_t)(((int64_t)kh * p.kv.num_slots + (r.pages ? 0 : r.slot0 + k0)) * (D / 16)) & 15u;
  const uint32_t off_k = code_off<D>(warp * 16 + key_g, q * (D / 8));
  const uint32_t off_ks = Lay::kKs + shift + (warp * 16 + key_g) * (D / 16) + q * (D / 64);
  const uint32_t off_va = Lay::kV + code_off<D>(warp * 16 + key_a, g * (D / 16));
  const uint32_t off_vb = Lay::kV + code_off<D>(warp * 16 + key_b, g * (D / 16));
  const uint32_t blk = (uint32_t)g * (D / 8) / 16;
  const uint32_t off_vsa = Lay::kVs + shift + (warp * 16 + key_a) * (D / 16) + blk;
  const uint32_t off_vsb = Lay::kVs + shift + (warp * 16 + key_b) * (D / 16) + blk;
  constexpr uint32_t kNext8 = 8 * (D / 2), kNextS8 = 8 * (D / 16);  // 8 keys on (the swizzle repeats every 8 rows)
  constexpr uint32_t kTile = Lay::kTileBytes, kTileS = Lay::kScaleBytes;  // the other half
  int st = 0;
  uint32_t ph = 0;
  for (int i = 0; i < npass; ++i) {
    if (!mbar_wait(&full[st], ph)) {
      ok = false;
      break;
    }
    // A half past k1 was not copied: it holds older keys or nothing, all masked.
    const uint32_t stage = smem_u32(smem) + st * Lay::kStageBytes;
    float s[2][4];  // key_g: columns 2q, 2q + 1; key_g + 8: the same
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t kw[2][D / 32], sc[2];  // eight codes per word; the columns' one or two block scales
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = stage + t * kTile + h * kNext8 + off_k;
        const uint32_t sa = stage + t * kTileS + h * kNextS8 + off_ks;
        if constexpr (D == 128) {
          const uint4 raw = lds128(at);
          kw[h][0] = raw.x; kw[h][1] = raw.y; kw[h][2] = raw.z; kw[h][3] = raw.w;
          sc[h] = e4m3x2_to_f16(lds16(sa));
        } else {
          const uint2 raw = lds64(at);
          kw[h][0] = raw.x; kw[h][1] = raw.y;
          sc[h] = e4m3x2_to_f16(lds8(sa));
        }
      }
      s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16(kw[0][w], x[0], x[1], x[2], x[3]);
        e2m1x8_to_f16(kw[1][w], y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[4];
          if (w < 2) {
            a[0] = mul_f16x2_lo(x[2 * h], sc[0]);
            a[1] = mul_f16x2_lo(y[2 * h], sc[1]);
            a[2] = mul_f16x2_lo(x[2 * h + 1], sc[0]);
            a[3] = mul_f16x2_lo(y[2 * h + 1], sc[1]);
          } else {
            a[0] = mul_f16x2_hi(x[2 * h], sc[0]);
            a[1] = mul_f16x2_hi(y[2 * h], sc[1]);
            a[2] = mul_f16x2_hi(x[2 * h + 1], sc[0]);
            a[3] = mul_f16x2_hi(y[2 * h + 1], sc[1]);
          }
          mma_f16_16816(s[t], a, qb[2 * w + h][0], qb[2 * w + h][1]);
        }
      }
    }
    // the warp's first key of the first half, and in either half
    const int kt0 = Blocks ? tiles.pos(2 * i, k1) + warp * 16 : k0 + i * 2 * kKeysPerTile + warp * 16;
    const int kt1 = Blocks ? tiles.pos(2 * i + 1, k1) + warp * 16 : kt0 + kKeysPerTile;
    auto first_key = [&](int t) { return Blocks && t == 1 ? kt1 : kt0 + t * kKeysPerTile; };
    const bool partial = Blocks ? max(kt0, kt1) + 16 > k1 : kt0 + kKeysPerTile + 16 > k1;
    if (partial) {  // keys past the end: arbitrary bits, no part in the softmax
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = first_key(t) + key_g;
        if (key >= k1) s[t][0] = s[t][1] = kNegInf;
        if (key + 8 >= k1) s[t][2] = s[t][3] = kNegInf;
      }
    }
    float mx[2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
      mx[e] = fmaxf(max3f(s[0][e], s[0][2 + e], s[1][e]), s[1][2 + e]) * p.scale_log2;
    const bool grow = mx[0] > m[0] + kRescaleThreshold || mx[1] > m[1] + kRescaleThreshold;
    if (__any_sync(0xffffffffu, grow)) {  // move the reference to the maximum over the warp's keys so far
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = mx[e];
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        const float m_new = fmaxf(m[e], v);
        alpha[e] = m_new == kNegInf ? 1.f : fast_exp2(m[e] - m_new);
        m[e] = m_new;
        l[e] *= alpha[e];
      }
      // O column 2q + e is of the head of S column 2q + e (mod 4 when not Wide: the same values)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= alpha[0];
        o[mt][1] *= alpha[1];
        o[mt][2] *= alpha[0];
        o[mt][3] *= alpha[1];
      }
    }
    const float neg_m[2] = {m[0] == kNegInf ? 0.f : -m[0], m[1] == kNegInf ? 0.f : -m[1]};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[t][e] = fast_exp2(fmaf(s[t][e], p.scale_log2, neg_m[e & 1]));
        l[e & 1] += s[t][e];
      }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // P of S column g's keys 2q, 2q + 1 (+ 8): the B registers, or those of each parity
      const uint32_t pt0 = movmatrix_trans(pack_f16(s[t][0], s[t][1]));
      const uint32_t pt1 = movmatrix_trans(pack_f16(s[t][2], s[t][3]));
      // V: bytes [g D/16, (g+1) D/16) of the keys a, b, a + 8, b + 8 and their block's scale
      uint32_t vw[4][D / 64], sc[4];  // sc: the scale in the low half
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = stage + t * kTile + h * kNext8, sa = stage + t * kTileS + h * kNextS8;
        if constexpr (D == 128) {
          const uint2 x = lds64(at + off_va), y = lds64(at + off_vb);
          vw[2 * h][0] = x.x; vw[2 * h][1] = x.y;
          vw[2 * h + 1][0] = y.x; vw[2 * h + 1][1] = y.y;
        } else {
          vw[2 * h][0] = lds32(at + off_va);
          vw[2 * h + 1][0] = lds32(at + off_vb);
        }
        if constexpr (Wide) {
          sc[2 * h] = lds8(sa + off_vsa) | (lds8(sa + off_vsb) << 8);
        } else {
          sc[2 * h] = lds8(sa + off_vsa);
          sc[2 * h + 1] = lds8(sa + off_vsb);
        }
      }
      if (partial) {  // keys past the end hold arbitrary bits: a scale of 0 makes their entries 0 (codes are finite)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ka = first_key(t) + key_a + 8 * h, kc = first_key(t) + key_b + 8 * h;
          if constexpr (Wide) {
            sc[2 * h] &= (ka < k1 ? 0xFFu : 0u) | (kc < k1 ? 0xFF00u : 0u);
          } else {
            if (ka >= k1) sc[2 * h] = 0u;
            if (kc >= k1) sc[2 * h + 1] = 0u;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; k += Wide ? 2 : 1) sc[k] = e4m3x2_to_f16(sc[k]);
      if constexpr (Wide) {
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t x[2][2][4];  // [keys a, b | a + 8, b + 8][even, odd column][byte]: pairs of keys
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = vw[2 * h][w], c = vw[2 * h + 1][w];
            const uint32_t ev = (a & 0x0F0F0F0Fu) | ((c << 4) & 0xF0F0F0F0u);
            const uint32_t od = ((a >> 4) & 0x0F0F0F0Fu) | (c & 0xF0F0F0F0u);
            e2m1x8_to_f16(ev, x[h][0][0], x[h][0][1], x[h][0][2], x[h][0][3]);
            e2m1x8_to_f16(od, x[h][1][0], x[h][1][1], x[h][1][2], x[h][1][3]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t a[4] = {mul_f16x2(x[0][0][c], sc[0]), mul_f16x2(x[0][1][c], sc[0]),
                                   mul_f16x2(x[1][0][c], sc[2]), mul_f16x2(x[1][1][c], sc[2])};
            mma_f16_16816(o[4 * w + c], a, pt0, pt1);
          }
        }
      } else {
        const uint32_t pb[4] = {prmt(pt0, 0u, sel_a), prmt(pt0, 0u, sel_b), prmt(pt1, 0u, sel_a), prmt(pt1, 0u, sel_b)};
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t x[4][4];  // [key a, b, a + 8, b + 8][byte]: columns 2j, 2j + 1
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e2m1x8_to_f16(vw[k][w], x[k][0], x[k][1], x[k][2], x[k][3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[k][c] = mul_f16x2_lo(x[k][c], sc[k]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {x[2 * h][2 * c], x[2 * h][2 * c + 1], x[2 * h + 1][2 * c], x[2 * h + 1][2 * c + 1]};
              mma_f16_16816(o[2 * w + c], a, pb[2 * h], pb[2 * h + 1]);
            }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (++st == S) { st = 0; ph ^= 1; }
  }
  if (!ok) {
    s_cons_abort = 1;
    set_status(p.status, ATTN_STATUS_TIMEOUT);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {  // the column's sum over the warp's keys
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
  }

  // ---------------- merge the warps' partial softmax states
  named_sync_consumers();  // every consumer is done with the stage buffers
  if (s_cons_abort) {  // same value for every consumer thread
    if constexpr (Blocks) block_merge_none(p, s_sums);
    return;
  }
  float* mo = reinterpret_cast<float*>(smem);  // [warps][G][D]
  float* mm = mo + kConsumerWarps * G * D;         // [warps][G]
  float* ml = mm + kConsumerWarps * G;                 // [warps][G]
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int head = Wide ? 2 * q + e : 2 * (q & 1) + e;
    if (head < G) {
      float* dst = mo + (warp * G + head) * D + g * (D / 8) + (Wide ? 0 : q >> 1);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        dst[(Wide ? 2 : 4) * mt] = o[mt][e] * p.v_scale;
        dst[(Wide ? 2 : 4) * mt + (Wide ? 1 : 2)] = o[mt][2 + e] * p.v_scale;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (g == 0 && 2 * q + e < G) {
      mm[warp * G + 2 * q + e] = m[e];
      ml[warp * G + 2 * q + e] = l[e];
    }
  named_sync_consumers();
  if constexpr (Blocks) {
    block_merge<D>(p, mo, mm, ml, s_sums, kh, b);
    return;
  }
  const bool direct = n_splits == 1;
  for (int idx = threadIdx.x; idx < G * D; idx += kConsumerWarps * 32) {
    const int row = idx / D, d = idx % D;
    float M = kNegInf;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, mm[w * G + row]);
    float L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumerWarps; ++w) {
      const float sw = fast_exp2(mm[w * G + row] - M);
      L += sw * ml[w * G + row];
      acc += sw * mo[(w * G + row) * D + d];
    }
    const int64_t hrow = (int64_t)b * p.Hq + kh * G + row;
    if (direct) {
      const __nv_bfloat16 v = __float2bfloat16_rn(acc / L);
      p.out[hrow * D + d] = *reinterpret_cast<const uint16_t*>(&v);
    } else {
      const int64_t prow = hrow * p.max_splits + split;
      p.part_o[prow * D + d] = acc;
      if (d == 0) {
        p.part_ml[prow * 2] = M;
        p.part_ml[prow * 2 + 1] = L;
      }
    }
  }
}

template <int D, bool Wide, bool Axes, bool Blocks>
int launch_t(const DecodeArgs& a, cudaStream_t stream) {
  using Lay = E2m1Layout<D>;
  CacheMaps maps;
  if (make_cache_maps(a.kv, a.cfg.num_kv_heads, D, kKeysPerTile, &maps) != 0) return ATTN_ELAUNCH;
  if constexpr (Blocks) {
    return launch_block_splits(decode_split_e2m1_kernel<D, Wide, Axes, true>, Lay::kSmemBytes, a, maps, stream);
  } else {
    if (cudaFuncSetAttribute(decode_split_e2m1_kernel<D, Wide, Axes, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Lay::kSmemBytes) != cudaSuccess)
      return ATTN_ELAUNCH;
    const dim3 grid(a.max_splits, a.cfg.num_kv_heads, a.B);
    return launch_dependent(decode_split_e2m1_kernel<D, Wide, Axes, false>, grid, dim3(kThreads), Lay::kSmemBytes,
                            stream, maps.k, maps.v, decode_par(a)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ELAUNCH;
  }
}

template <int D, bool Wide>
int launch_n(const DecodeArgs& a, cudaStream_t stream) {
  return a.axes.positions ? launch_t<D, Wide, true, false>(a, stream) : launch_t<D, Wide, false, false>(a, stream);
}

}  // namespace

int launch_decode_e2m1(const DecodeArgs& a, cudaStream_t stream) {
  const bool wide = a.cfg.num_q_heads / a.cfg.num_kv_heads > 4;
  if (a.cfg.head_dim == 128) return wide ? launch_n<128, true>(a, stream) : launch_n<128, false>(a, stream);
  return wide ? launch_n<64, true>(a, stream) : launch_n<64, false>(a, stream);
}

int launch_block_attend_e2m1(const DecodeArgs& a, cudaStream_t stream) {
  const bool wide = a.cfg.num_q_heads / a.cfg.num_kv_heads > 4;
  if (a.cfg.head_dim == 128)
    return wide ? launch_t<128, true, false, true>(a, stream) : launch_t<128, false, false, true>(a, stream);
  return wide ? launch_t<64, true, false, true>(a, stream) : launch_t<64, false, false, true>(a, stream);
}

}  // namespace gb300
