// Device helpers shared by the attention kernels: bf16 packing, mbarriers,
// TMA tile loads, ldmatrix / mma.sync fragments, bounded pipeline waits.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/attn.h"

namespace gb300 {

// Layout of the caller's workspace: a 256-byte header (status word first),
// then the per-call scratch areas, each 256-byte aligned.
constexpr size_t kWsHeader = 256;

constexpr float kNegInf = -__builtin_huge_valf();

__host__ __device__ constexpr size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ---------------------------------------------------------------- bf16
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// What rounding (lo, hi) to the bf16 pair h left of them, as a bf16 pair.
__device__ __forceinline__ uint32_t bf16_rest(float lo, float hi, uint32_t h) {
  return pack_bf16(lo - bf16_lo(h), hi - bf16_hi(h));
}

// ---------------------------------------------------------------- f16 and E4M3
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Four E4M3 codes (byte i = element i) -> two f16 pairs: lo = elements 0, 1,
// hi = elements 2, 3 (first element in the low half).  Exact: every E4M3
// value is an f16 value.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// E4M3 codes of two fp32 values, first in the low byte: round to nearest
// even, magnitudes beyond 448 clamped to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- E2M1 with block scales
// Eight E2M1 codes (nibble i = element i) -> four f16 pairs (elements 2i and
// 2i + 1).  Exact: every E2M1 value is an f16 value.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1, uint32_t& h2, uint32_t& h3) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
}

// E2M1 codes of eight fp32 values, nibble i = element i: round to nearest
// even, magnitudes beyond 6 clamped to 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&z)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  return r;
}

// Two E4M3 codes (bits 0-7 and 8-15) -> an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  return h;
}
__device__ __forceinline__ float f16_lo(uint32_t h) { return __half2float(__ushort_as_half((uint16_t)h)); }

// Product of two f16 pairs.  An E2M1 value (2 significant bits) times an E4M3
// scale (4) needs 6 and lies in [2^-10, 2688]: the product of an entry and its
// block scale is exact in f16.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The same with the low (high) half of s for both.
__device__ __forceinline__ uint32_t mul_f16x2_lo(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), __low2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2_hi(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), __high2half2(*reinterpret_cast<__half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Largest magnitude of eight values (NaN if one is NaN).
__device__ __forceinline__ float amax8(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = max_nan(m, fabsf(y[e]));
  return m;
}

// The E4M3 scale (its code) of a block with largest magnitude amax, by an IEEE
// division: 16-bit inputs meet the rounding boundaries exactly, and a product with
// a rounded reciprocal would decide those ties by the reciprocal's error.
__device__ __forceinline__ uint32_t e2m1_block_scale(float amax) { return e4m3x2(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu; }

// Codes of eight values of a block with scale s (the value of its code): those of
// the quotients y / s rounded to fp32, for less than eight divisions.  Every
// boundary between codes is a multiple m of 1/4.  With m the multiple nearest to an
// approximate quotient, y - m s rounds to zero only if it is zero (m s is exact: 4
// and 5 bits) and m + (y - m s) / s, rounded once, lies on the side of m that y / s
// does: a nonzero y - m s is at least an ulp of y, and (ulp of y) / s exceeds half
// an ulp of m since s is below twice the power of two in it.  All on |y|; the sign is
// put back at the end, so that a zero keeps its own.
__device__ __forceinline__ uint32_t e2m1_codes8(const float (&y)[8], float s) {
  if (!(s > 0.f)) {  // an empty block, or a NaN one (whose codes do not matter)
    return 0u;
  }
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));  // s is in [2^-9, 448]
  constexpr float kQuarters = 3145728.f;  // 1.5 * 2^21: its ulp is 1/4
  float z[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fabsf(y[e]);
    const float q = fminf(__fmul_rn(a, inv), 8.f);
    const float m = __fsub_rn(__fadd_rn(q, kQuarters), kQuarters);
    z[e] = copysignf(fmaf(fmaf(-m, s, a), inv, m), y[e]);
  }
  return e2m1x8(z);
}

// Byte permute: result byte i = byte sel_i of the pair (a = bytes 0-3, b = 4-7).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// ---------------------------------------------------------------- dependent launches
// A kernel launched with programmatic stream serialisation may start while
// the kernel before it in the stream is still running; it waits here before
// it touches memory that kernel (or any earlier one) writes.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets such a kernel after this one be scheduled once every CTA of this
// kernel has started (its CTAs then fill SMs as this kernel's CTAs exit).
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- status
__device__ __forceinline__ void set_status(int32_t* status, int32_t bit) {
  if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------- shared memory addresses
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Non-suspending check of the same condition (mbarrier.try_wait may suspend
// the thread for a while before it returns false; test_wait never does).
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Wait for the phase with the given parity to complete.  Gives up after about
// two seconds (a pipeline that never completes is an internal error): returns
// false and the caller records ATTN_STATUS_TIMEOUT and leaves its loop.  The
// first check is inline; the bounded polling loop is out of line, which keeps
// the common case (the phase is already complete) short.
constexpr uint32_t kWaitSpinLimit = 1u << 22;
static __device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kWaitSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (i > 64) __nanosleep(i < 4096 ? 64 : 512);
  }
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_slow(bar, parity);
}

// ---------------------------------------------------------------- TMA
// 3-D tiled load global -> shared, completion counted on `bar` (bytes).
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3)
      : "memory");
}

// 3-D tiled store shared -> global, tracked as a bulk group of this thread.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t c0,
                                             int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit_group() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The shared-memory sources of this thread's bulk groups have been read.
__device__ __forceinline__ void bulk_wait_read_all() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// This thread's bulk groups have completed (writes performed).
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` inside a tile
// written by TMA with CU_TENSOR_MAP_SWIZZLE_128B (rows of 128 bytes; the
// chunk index is XORed with the row index modulo 8; tile base 1024-aligned).
__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

// ---------------------------------------------------------------- mma.sync fragments
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// D = A * B + D, m16n8k16, bf16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_bf16_16816(float* d, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A * B + D, m16n8k16, f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- RoPE
// Rotation frequencies theta^(-2i/D) for i < D/2 as float-float pairs
// (hi = nearest float, lo = remainder), and 2*pi as a float-float pair for
// the range reduction.  Computed on the host in double for every call.
struct RopeFreqs {
  float hi[64];
  float lo[64];
  float two_pi_hi, two_pi_lo, inv_two_pi;
};

// cos and sin of pos * f for f = hi + lo: float-float product (pos is an
// exact integer below 2^24, so one fma recovers the rounding error of pos*hi
// exactly), then Cody-Waite additive range reduction modulo 2*pi with 2*pi
// split into two floats, then the hardware sin/cos on |r| <= pi.  The angle
// keeps about 1e-7 rad absolute error at any position; cos/sin about 4e-7.
__device__ __forceinline__ void rope_angle(float pos, float f_hi, float f_lo, const RopeFreqs& fr,
                                           float* c, float* s) {
  const float a_hi = pos * f_hi;
  const float a_err = fmaf(pos, f_hi, -a_hi);
  const float a_lo = fmaf(pos, f_lo, a_err);
  const float k = rintf(a_hi * fr.inv_two_pi);
  float r = fmaf(-k, fr.two_pi_hi, a_hi);
  r = fmaf(-k, fr.two_pi_lo, r);
  r += a_lo;
  __sincosf(r, s, c);  // |r| <= pi + 1e-6: hardware sin/cos, absolute error ~4e-7
}

// ---------------------------------------------------------------- head vectors, pair layout
// A head vector of D bf16 values is held by L = D/16 consecutive lanes: lane
// li of the group takes the 8 values at 8 li and the 8 values at D/2 + 8 li
// (two 16-byte loads), so both members of every rotate-half pair (i, i + D/2)
// sit in one lane.  The prologue kernel and the decode kernel's append both
// use these, so they write the same cache entries bit for bit.

// Eight bf16 values (16 bytes) as fp32, element i from bytes 2i, 2i + 1.
__device__ __forceinline__ void unpack_bf16x8(const uint4& raw, float (&y)[8]) {
  const uint32_t* rw = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[2 * e] = bf16_lo(rw[e]);
    y[2 * e + 1] = bf16_hi(rw[e]);
  }
}

// E4M3 codes of eight fp32 values times an fp32 factor (the product rounded
// to fp32 first, as the cache format states), element i in byte i.
__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8], float r) {
  uint2 v;
  v.x = e4m3x2(__fmul_rn(y[0], r), __fmul_rn(y[1], r)) | (e4m3x2(__fmul_rn(y[2], r), __fmul_rn(y[3], r)) << 16);
  v.y = e4m3x2(__fmul_rn(y[4], r), __fmul_rn(y[5], r)) | (e4m3x2(__fmul_rn(y[6], r), __fmul_rn(y[7], r)) << 16);
  return v;
}

// Position of every rotation pair of a token: the same one ...
struct OnePos {
  float pos;
  __device__ __forceinline__ float operator()(int) const { return pos; }
};
// ... or that of the pair's axis (attn_rope_axes_t): two bits per pair.
struct RopeAxes {
  const int32_t* positions;  // [A, ld]; nullptr: no axes
  int64_t ld;
  uint32_t axis[4];          // axis of pair i: bits 2 (i % 16), 2 (i % 16) + 1 of word i / 16
  int32_t num_axes;
  uint32_t used;             // bit a: some pair takes axis a
};
struct AxisPos {
  const RopeAxes& ax;
  int64_t token;
  __device__ __forceinline__ float operator()(int pair) const {
    const uint32_t a = (ax.axis[pair >> 4] >> (2 * (pair & 15))) & 3u;
    return (float)__ldg(ax.positions + (int64_t)a * ax.ld + token);
  }
};
// Positions that a lane of a warp holds for its own pairs N lane .. N lane + N - 1.
template <int N>
struct LanePos {
  float pos[N];
  __device__ __forceinline__ float operator()(int pair) const { return pos[pair & (N - 1)]; }
};
constexpr uint32_t kMaxPosition = 1u << 24;  // exact in fp32
// Every position of the token, on the axes that have pairs, lies in [0, 2^24].
__device__ __forceinline__ bool axes_in_range(const RopeAxes& ax, int64_t token) {
  bool ok = true;
  for (int a = 0; a < ax.num_axes; ++a)
    if (ax.used >> a & 1) ok = ok && (uint32_t)__ldg(ax.positions + a * ax.ld + token) <= kMaxPosition;
  return ok;
}

// cos/sin of the rotation pairs 8 li .. 8 li + 7 (li = lane % (D/16)) at
// position(s) pos: each lane computes D/64 of the D/2 angles, the lanes that
// need them read them by shuffle.  All 32 lanes must call this.
template <int D, class Pos>
__device__ __forceinline__ void pair_angles(const Pos& pos, const RopeFreqs& fr, int lane, float (&cs)[8],
                                            float (&sn)[8]) {
  constexpr int PPL = D / 64;
  const int li = lane % (D / 16);
  float c_own[PPL], s_own[PPL];
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    const int pr = lane * PPL + e;
    rope_angle(pos(pr), fr.hi[pr], fr.lo[pr], fr, &c_own[e], &s_own[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int pr = li * 8 + e;
    cs[e] = __shfl_sync(0xffffffffu, c_own[e % PPL], pr / PPL);
    sn[e] = __shfl_sync(0xffffffffu, s_own[e % PPL], pr / PPL);
  }
}

// E2M1 entries of one head vector in the pair layout, at cache row e (slot *
// Hkv + head) of the codes and block row sb of the block scales: this lane's
// 8 values at 8 li (ya) and at D/2 + 8 li (yb) as they are before the division
// by the tensor's scale (r = its fp32 reciprocal).  A block of 16 sits in two
// neighbouring lanes; the even one stores its scale.  All 32 lanes must call
// this; lanes with live == false store nothing.
template <int D>
__device__ __forceinline__ void store_e2m1_pair(const float (&xa)[8], const float (&xb)[8], float r, bool live,
                                                int li, uint8_t* codes, uint8_t* scales) {
  float ya[8], yb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ya[e] = __fmul_rn(xa[e], r);
    yb[e] = __fmul_rn(xb[e], r);
  }
  float ma = amax8(ya), mb = amax8(yb);
  ma = max_nan(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
  mb = max_nan(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
  const uint32_t sa = e2m1_block_scale(ma), sb = e2m1_block_scale(mb);
  const uint32_t ca = e2m1_codes8(ya, f16_lo(e4m3x2_to_f16(sa)));
  const uint32_t cb = e2m1_codes8(yb, f16_lo(e4m3x2_to_f16(sb)));
  if (!live) return;
  *reinterpret_cast<uint32_t*>(codes + 4 * li) = ca;
  *reinterpret_cast<uint32_t*>(codes + D / 4 + 4 * li) = cb;
  if ((li & 1) == 0) {
    scales[li >> 1] = (uint8_t)sa;
    scales[D / 32 + (li >> 1)] = (uint8_t)sb;
  }
}

// ---------------------------------------------------------------- K to the last bit of fp32
// A four-bit code moves by up to a third of its value when its input crosses a
// rounding boundary, so the prologue and the decode kernels bring K to within an
// fp32 ulp of the exact value before it is coded: of the 10.2 M codes of K of the
// Qwen3-4B prefill none differs from the exact value's, with plain fp32 steps 5 do
// (its prepare then takes 56 us in place of 68, back to back).  The fused projection
// (proj.cu) codes K from its plain fp32 steps: its accumulators are off by more.
// Values are pairs hi + lo of floats: the
// error-free sum and product are Knuth's and Dekker's (by fma).
struct F2 {
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ F2 two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, fmaf(a, b, -p)};
}

// cos and sin of pos * f as pairs: the angle reduced by multiples of pi / 2 to a
// pair |r| <= pi / 4, then the Taylor series with the leading terms (r, and 1 - r^2 /
// 2) kept exactly.  Far out one rounded quotient is off by up to one multiple (the
// quotient at 2^24 has steps of 1), so the reduction (Cody and Waite's, on pairs) is
// done twice; the second quotient is small.  Absolute error about 2e-8 up to
// positions of 2^22, 8e-8 at 2^24 (the roundings of the low part, which grows with
// the position).
__device__ __forceinline__ void rope_angle_fine(float pos, float f_hi, float f_lo, const RopeFreqs& fr, F2* c, F2* s) {
  const F2 a = two_prod(pos, f_hi);
  const float h_hi = 0.25f * fr.two_pi_hi, h_lo = 0.25f * fr.two_pi_lo;  // pi / 2
  const float k1 = rintf(a.hi * (4.f * fr.inv_two_pi));
  const F2 p = two_prod(-k1, h_hi), q = two_prod(-k1, h_lo);
  const F2 u = two_sum(a.hi, p.hi);
  const F2 t = two_sum(u.hi, q.hi);
  const F2 v = two_sum(t.hi, fmaf(pos, f_lo, a.lo));
  const F2 z = two_sum(v.hi, ((t.lo + v.lo) + (p.lo + u.lo)) + q.lo);
  const float k2 = rintf(z.hi * (4.f * fr.inv_two_pi));
  const F2 r = two_sum(fmaf(-k2, h_hi, z.hi), fmaf(-k2, h_lo, z.lo));
  const F2 r2 = two_prod(r.hi, r.hi);
  const float x = r2.hi;
  const float ps = fmaf(fmaf(fmaf(fmaf(-1.f / 39916800, x, 1.f / 362880), x, -1.f / 5040), x, 1.f / 120), x, -1.f / 6);
  const float pc = fmaf(fmaf(fmaf(fmaf(1.f / 479001600, x, -1.f / 3628800), x, 1.f / 40320), x, -1.f / 720), x, 1.f / 24);
  F2 sn = two_sum(r.hi, r.hi * x * ps);
  sn = two_sum(sn.hi, fmaf(r.lo, fmaf(-0.5f, x, 1.f), sn.lo));
  F2 cs = two_sum(1.f, -0.5f * x);
  cs = two_sum(cs.hi, cs.lo + (fmaf(x * x, pc, -0.5f * r2.lo) - r.hi * r.lo));  // hi alone is the nearest float
  const int quarter = (int)(k1 + k2) & 3;
  const bool swap = quarter & 1, neg_c = quarter == 1 || quarter == 2, neg_s = quarter >= 2;
  *c = swap ? sn : cs;
  *s = swap ? cs : sn;
  if (neg_c) *c = {-c->hi, -c->lo};
  if (neg_s) *s = {-s->hi, -s->lo};
}

// pair_angles() with pairs hi + lo.
template <int D, class Pos>
__device__ __forceinline__ void pair_angles_fine(const Pos& pos, const RopeFreqs& fr, int lane, F2 (&cs)[8], F2 (&sn)[8]) {
  constexpr int PPL = D / 64;
  const int li = lane % (D / 16);
  F2 c_own[PPL], s_own[PPL];
#pragma unroll
  for (int e = 0; e < PPL; ++e) {
    const int pr = lane * PPL + e;
    rope_angle_fine(pos(pr), fr.hi[pr], fr.lo[pr], fr, &c_own[e], &s_own[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int from = (li * 8 + e) / PPL;
    cs[e].hi = __shfl_sync(0xffffffffu, c_own[e % PPL].hi, from);
    cs[e].lo = __shfl_sync(0xffffffffu, c_own[e % PPL].lo, from);
    sn[e].hi = __shfl_sync(0xffffffffu, s_own[e % PPL].hi, from);
    sn[e].lo = __shfl_sync(0xffffffffu, s_own[e % PPL].lo, from);
  }
}

// y c - z s rounded once (s negated by the caller for the sum).
__device__ __forceinline__ float rotate_fine(const F2& y, const F2& c, const F2& z, const F2& s) {
  const F2 m = two_prod(y.hi, c.hi), n = two_prod(-z.hi, s.hi);
  const F2 d = two_sum(m.hi, n.hi);
  const float e = fmaf(y.hi, c.lo, fmaf(y.lo, c.hi, m.lo)) - fmaf(z.hi, s.lo, fmaf(z.lo, s.hi, -n.lo));
  return d.hi + (d.lo + e);
}

// norm_rope_pair() with one rounding to fp32 at the end.  x and w are bf16: x^2
// and w x are exact in fp32.
template <int D>
__device__ __forceinline__ void norm_rope_pair_fine(const uint4& raw_a, const uint4& raw_b, const uint4& w_a,
                                                    const uint4& w_b, const F2 (&cs)[8], const F2 (&sn)[8], float eps,
                                                    float (&ra)[8], float (&rb)[8]) {
  constexpr int L = D / 16;
  float xa[8], xb[8];
  unpack_bf16x8(raw_a, xa);
  unpack_bf16x8(raw_b, xb);
  F2 ss = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const F2 t = two_sum(xa[e] * xa[e], xb[e] * xb[e]);
    const F2 u = two_sum(ss.hi, t.hi);
    ss = {u.hi, ss.lo + (u.lo + t.lo)};
  }
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) {
    const F2 u = two_sum(ss.hi, __shfl_xor_sync(0xffffffffu, ss.hi, off));
    ss = {u.hi, ss.lo + __shfl_xor_sync(0xffffffffu, ss.lo, off) + u.lo};
  }
  F2 v = two_sum(ss.hi * (1.0f / D), eps);
  v.lo += ss.lo * (1.0f / D);
  // 1 / sqrt(v): one Newton step on rsqrtf's value g, its correction kept apart
  const float g = rsqrtf(v.hi);
  const F2 g2 = two_prod(g, g);
  const float res = fmaf(-v.hi, g2.hi, 1.f) - fmaf(v.hi, g2.lo, v.lo * g2.hi);
  // (past the range of fp32 squares g is 0 and its correction no number: then none)
  const float g_lo = fabsf(res) < 1.f ? 0.5f * g * res : 0.f;
  float wa[8], wb[8];
  unpack_bf16x8(w_a, wa);
  unpack_bf16x8(w_b, wb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float pa = wa[e] * xa[e], pb = wb[e] * xb[e];
    F2 ya = two_prod(pa, g), yb = two_prod(pb, g);
    ya.lo = fmaf(pa, g_lo, ya.lo);
    yb.lo = fmaf(pb, g_lo, yb.lo);
    ra[e] = rotate_fine(ya, cs[e], yb, sn[e]);
    rb[e] = rotate_fine(yb, cs[e], ya, F2{-sn[e].hi, -sn[e].lo});
  }
}

// RMSNorm and rotate-half of one head vector in the pair layout: raw_a /
// raw_b are this lane's values at 8 li and D/2 + 8 li, w_a / w_b the norm
// weights there (bf16).  Sum of squares: two chains of 8 fused multiply-adds,
// their sum, log2(D/16) shuffle adds over the head's lanes; then
// y = w * (x * rsqrt(ss / D + eps)) and (y_i, y_j) -> (y_i c - y_j s,
// y_j c + y_i s) for j = i + D/2.  All 32 lanes must call this.
template <int D>
__device__ __forceinline__ void norm_rope_pair(const uint4& raw_a, const uint4& raw_b, const uint4& w_a,
                                               const uint4& w_b, const float (&cs)[8], const float (&sn)[8],
                                               float eps, float (&ra)[8], float (&rb)[8]) {
  constexpr int L = D / 16;
  float xa[8], xb[8];
  unpack_bf16x8(raw_a, xa);
  unpack_bf16x8(raw_b, xb);
  float sa = 0.f, sb = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sa = fmaf(xa[e], xa[e], sa);
    sb = fmaf(xb[e], xb[e], sb);
  }
  float ss = sa + sb;
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float inv = rsqrtf(ss * (1.0f / D) + eps);
  float wa[8], wb[8];
  unpack_bf16x8(w_a, wa);
  unpack_bf16x8(w_b, wb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    xa[e] = wa[e] * (xa[e] * inv);
    xb[e] = wb[e] * (xb[e] * inv);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ra[e] = fmaf(xb[e], -sn[e], xa[e] * cs[e]);
    rb[e] = fmaf(xa[e], sn[e], xb[e] * cs[e]);
  }
}

// One query row (D bf16 values at `row`) normalised and rotated, delivered in
// the m16n8k16 A-fragment distribution: this thread (quad member q = lane & 3)
// holds columns 16ks + 2q + {0,1} in frag[ks][0] and 16ks + 8 + 2q + {0,1} in
// frag[ks][1].  The four threads of a quad hold the whole row, so the RMSNorm
// sum is a quad reduction, and RoPE's partner column c + D/2 sits in the same
// thread at ks + D/32.  All 32 lanes must call this (it shuffles); rows with
// valid == false yield zeros.  Rest: rest holds what the rounding to bf16 left.
template <int D, bool Rest, class Pos>
__device__ __forceinline__ void q_row_frags(const uint16_t* row, bool valid, const uint16_t* w,
                                            float eps, const Pos& pos, const RopeFreqs& fr,
                                            uint32_t (&frag)[D / 16][2], uint32_t (&rest)[D / 16][2]) {
  const int q = threadIdx.x & 3;
  float x[D / 16][4];
  float ss = 0.f;
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t a = valid ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * ks + 2 * q)) : 0u;
    const uint32_t b = valid ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * ks + 8 + 2 * q)) : 0u;
    x[ks][0] = bf16_lo(a);
    x[ks][1] = bf16_hi(a);
    x[ks][2] = bf16_lo(b);
    x[ks][3] = bf16_hi(b);
#pragma unroll
    for (int j = 0; j < 4; ++j) ss = fmaf(x[ks][j], x[ks][j], ss);
  }
  ss += __shfl_xor_sync(0xffffffffu, ss, 1);
  ss += __shfl_xor_sync(0xffffffffu, ss, 2);
  const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t wa = __ldg(reinterpret_cast<const uint32_t*>(w + 16 * ks + 2 * q));
    const uint32_t wb = __ldg(reinterpret_cast<const uint32_t*>(w + 16 * ks + 8 + 2 * q));
    x[ks][0] = bf16_lo(wa) * (x[ks][0] * inv);
    x[ks][1] = bf16_hi(wa) * (x[ks][1] * inv);
    x[ks][2] = bf16_lo(wb) * (x[ks][2] * inv);
    x[ks][3] = bf16_hi(wb) * (x[ks][3] * inv);
  }
#pragma unroll
  for (int ks = 0; ks < D / 32; ++ks) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 16 * ks + (j >> 1) * 8 + 2 * q + (j & 1);  // rotation pair index < D/2
      float c, s;
      rope_angle(pos(i), fr.hi[i], fr.lo[i], fr, &c, &s);
      const float x1 = x[ks][j], x2 = x[ks + D / 32][j];
      x[ks][j] = x1 * c - x2 * s;
      x[ks + D / 32][j] = x2 * c + x1 * s;
    }
  }
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    frag[ks][0] = pack_bf16(x[ks][0], x[ks][1]);
    frag[ks][1] = pack_bf16(x[ks][2], x[ks][3]);
    if constexpr (Rest) {
      rest[ks][0] = bf16_rest(x[ks][0], x[ks][1], frag[ks][0]);
      rest[ks][1] = bf16_rest(x[ks][2], x[ks][3], frag[ks][1]);
    }
  }
}

// One query row normalised and rotated, as f16 A fragments in the layout
// the E4M3 decode kernel reads keys in: quad member c = lane & 3 holds the
// columns [c D/4, (c+1) D/4), frag[ks][0] = columns c D/4 + 4ks + {0,1} and
// frag[ks][1] = c D/4 + 4ks + {2,3} (the dot product does not depend on
// which k slot a column occupies, as long as query and key agree).  The
// RMSNorm sum is a quad reduction; the RoPE partner column (D/2 away) sits
// in quad member c ^ 2.  All 32 lanes must call this; rows with
// valid == false yield zeros.
template <int D, class Pos>
__device__ __forceinline__ void q_row_frags_quarters(const uint16_t* row, bool valid,
                                                     const uint16_t* w, float eps, const Pos& pos,
                                                     const RopeFreqs& fr,
                                                     uint32_t (&frag)[D / 16][2]) {
  constexpr int Q = D / 4;  // columns per quad member
  const int c = threadIdx.x & 3;
  float x[Q];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < Q / 8; ++v) {
    const uint4 u = valid ? __ldg(reinterpret_cast<const uint4*>(row + c * Q + 8 * v)) : make_uint4(0, 0, 0, 0);
    const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * v + 2 * j] = bf16_lo(uw[j]);
      x[8 * v + 2 * j + 1] = bf16_hi(uw[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) ss = fmaf(x[i], x[i], ss);
  ss += __shfl_xor_sync(0xffffffffu, ss, 1);
  ss += __shfl_xor_sync(0xffffffffu, ss, 2);
  const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
  for (int v = 0; v < Q / 8; ++v) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(w + c * Q + 8 * v));
    const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * v + 2 * j] = bf16_lo(uw[j]) * (x[8 * v + 2 * j] * inv);
      x[8 * v + 2 * j + 1] = bf16_hi(uw[j]) * (x[8 * v + 2 * j + 1] * inv);
    }
  }
  const bool first_half = c < 2;
#pragma unroll
  for (int e = 0; e < Q; ++e) {
    const int i = (c & 1) * Q + e;  // rotation pair index < D/2
    float cs, sn;
    rope_angle(pos(i), fr.hi[i], fr.lo[i], fr, &cs, &sn);
    const float other = __shfl_xor_sync(0xffffffffu, x[e], 2);
    // first half: x_i c - x_{i+D/2} s; second half: x_{i+D/2} c + x_i s
    x[e] = first_half ? x[e] * cs - other * sn : x[e] * cs + other * sn;
  }
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    frag[ks][0] = pack_f16(x[4 * ks], x[4 * ks + 1]);
    frag[ks][1] = pack_f16(x[4 * ks + 2], x[4 * ks + 3]);
  }
}

// ---------------------------------------------------------------- requests
// How kernels find cache entries (the attn_kv_t indexing fields).
struct KvIndex {
  const int64_t* slot_base;      // contiguous layout
  const int32_t* cache_lens;
  const int32_t* slot_capacity;
  const int32_t* page_table;     // nullptr: contiguous layout
  int64_t num_slots;
  int32_t log2_page;             // log2(page_size) (paged layout)
  int32_t pages_per_req;
};

// Per-request facts every kernel derives the same way from the arguments.
struct ReqInfo {
  int64_t slot0;         // contiguous layout: slot of position 0
  const int32_t* pages;  // paged layout: the request's page-table row, else nullptr
  int32_t cached;        // c_b
  int32_t n_new;         // n_b
  bool valid;            // the request can hold c_b + n_b entries and cu_seqlens is sane
};

__device__ __forceinline__ ReqInfo load_request(const KvIndex& kv, int b, int32_t n_new) {
  ReqInfo r;
  r.cached = kv.cache_lens[b];
  r.n_new = n_new;
  const int64_t end = (int64_t)r.cached + (int64_t)n_new;
  const bool sizes = n_new >= 0 && r.cached >= 0 && end <= (int64_t)kv.slot_capacity[b] && end <= (1 << 24);
  if (kv.page_table) {
    r.pages = kv.page_table + (int64_t)b * kv.pages_per_req;
    r.slot0 = 0;
    r.valid = sizes && end <= ((int64_t)kv.pages_per_req << kv.log2_page);
  } else {
    r.pages = nullptr;
    r.slot0 = kv.slot_base[b];
    r.valid = sizes && r.slot0 >= 0 && r.slot0 + end <= kv.num_slots;
  }
  return r;
}

// Slot of the entry at position pos of a request, or `none` (negative) when its
// page number is outside the cache (paged layout; pos < pages_per_req * page_size).
// A tile of n keys read from slot -n is all zeros: TMA fills them in.
__device__ __forceinline__ int64_t cache_slot(const KvIndex& kv, const ReqInfo& r, int pos, int none = -1) {
  if (!r.pages) return r.slot0 + pos;
  const int64_t pg = __ldg(r.pages + (pos >> kv.log2_page));
  const int64_t slot = (pg << kv.log2_page) + (pos & ((1 << kv.log2_page) - 1));
  return (pg >= 0 && slot < kv.num_slots) ? slot : none;
}

}  // namespace gb300
