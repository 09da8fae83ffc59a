// Rules on rows of logits and the table of seen tokens (include/logits.h).
//
// Each logit goes through x + bias, the repetition penalty, the frequency and
// presence penalties and the mask, each operation rounded to fp32.  Bound by memory:
// 4 bytes read and 4 written per logit, 2 of the table, an eighth of a byte of the mask.
// A CTA takes a run of one row; the row's biases, few and in any order, are filtered for the
// run first and summed in shared memory, each token's by one thread in list order (no
// atomics: the order decides the rounding).
#include "kernels.cuh"
#include "../../include/logits.h"

namespace gb300 {

namespace {

constexpr int kThreads = 256;

struct AdjustPar {
  const float* logits;
  float* out;
  int64_t ld, ld_out;
  int32_t V, runs;
  attn_logits_rules_t r;
};

// One logit through the rules after the bias.
__device__ __forceinline__ float apply_rules(float x, uint32_t word, float rep, float freq, float pres, bool allowed) {
  if (word) {
    if (rep > 0.f) x = x > 0.f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
    const uint32_t n = word & 0x7FFFu;
    if (n) {
      x = __fsub_rn(x, __fmul_rn(freq, (float)n));
      x = __fsub_rn(x, pres);
    }
  }
  return allowed ? x : kNegInf;
}

// Four logits per thread and step, Q steps: all loads of a run go out before its biases are
// looked at.  Vec: rows of logits and out are 16-byte aligned, a thread's four are neighbours;
// else they are 256 apart (a row's start may lie anywhere).
template <int Q, bool Vec>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const AdjustPar p) {
  constexpr int kRun = Q * 4 * kThreads;
  __shared__ __align__(16) float bias[kRun];
  __shared__ int tok[kThreads];
  __shared__ float val[kThreads];
  __shared__ int cnt[kThreads / 32];
  const int b = blockIdx.x / p.runs, v0 = blockIdx.x % p.runs * kRun;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  grid_dependency_wait();
  const int n = min(kRun, p.V - v0);  // logits of this run
  const float* in = p.logits + b * p.ld + v0;
  float* out = p.out + b * p.ld_out + v0;
  const uint16_t* seen = nullptr;
  if (p.r.seen) {
    const int row = p.r.seen_row ? __ldg(p.r.seen_row + b) : b;
    if (row >= 0 && row < p.r.seen_rows) seen = p.r.seen + row * p.r.seen_ld + v0;
  }
  const uint32_t* mask = nullptr;
  if (p.r.mask) {
    const int row = p.r.mask_row ? __ldg(p.r.mask_row + b) : b;
    if (row >= 0 && row < p.r.mask_rows) mask = p.r.mask + row * p.r.mask_ld + (v0 >> 5);
  }
  auto place = [&](int q, int e) { return Vec ? (q * kThreads + tid) * 4 + e : (q * 4 + e) * kThreads + tid; };
  float x[Q][4];
  uint32_t word[Q][4], allow[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int i0 = place(q, 0);
    if (Vec && i0 + 4 <= n) {
      *reinterpret_cast<float4*>(x[q]) = *reinterpret_cast<const float4*>(in + i0);
      const uint2 w = seen ? *reinterpret_cast<const uint2*>(seen + i0) : make_uint2(0u, 0u);
      const uint32_t m = mask ? __ldg(mask + (i0 >> 5)) >> (i0 & 31) : 15u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        word[q][e] = ((e < 2 ? w.x : w.y) >> (16 * (e & 1))) & 0xFFFFu;
        allow[q][e] = m >> e & 1u;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = place(q, e);
        const bool there = i < n;
        x[q][e] = there ? in[i] : 0.f;
        word[q][e] = there && seen ? seen[i] : 0u;
        allow[q][e] = there && mask ? __ldg(mask + (i >> 5)) >> (i & 31) & 1u : 1u;
      }
    }
  }
  const float rep = p.r.repetition ? __ldg(p.r.repetition + b) : 0.f;
  const float freq = p.r.frequency ? __ldg(p.r.frequency + b) : 0.f;
  const float pres = p.r.presence ? __ldg(p.r.presence + b) : 0.f;
  bool biased = false;
  if (p.r.bias_start) {
    const int e0 = __ldg(p.r.bias_start + b), e1 = __ldg(p.r.bias_start + b + 1);
    for (int e = e0; e < e1; e += kThreads) {
      const int i = e + tid;
      const int t = i < e1 ? __ldg(p.r.bias_token + i) : -1;
      const bool mine = t >= v0 && t < v0 + n;
      const uint32_t all = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) cnt[warp] = __popc(all);
      __syncthreads();
      int at = 0, m = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += cnt[w];
        m += cnt[w];
      }
      if (m > 0 && !biased) {
        for (int k = tid; k < kRun; k += kThreads) bias[k] = 0.f;
        biased = true;
      }
      if (mine) {
        at += __popc(all & ((1u << lane) - 1u));
        tok[at] = t - v0;
        val[at] = __ldg(p.r.bias_value + i);
      }
      __syncthreads();
      for (int k = 0; k < m; ++k)
        if ((tok[k] & (kThreads - 1)) == tid) bias[tok[k]] += val[k];
      __syncthreads();
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y = x[q][e];
      if (biased) y = __fadd_rn(y, bias[place(q, e)]);
      x[q][e] = apply_rules(y, word[q][e], rep, freq, pres, allow[q][e] != 0u);
    }
    const int i0 = place(q, 0);
    if (Vec && i0 + 4 <= n) {
      *reinterpret_cast<float4*>(out + i0) = *reinterpret_cast<const float4*>(x[q]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (place(q, e) < n) out[place(q, e)] = x[q][e];
    }
  }
}

// ---------------------------------------------------------------- seen tokens
struct SeenPar {
  uint16_t* seen;
  int64_t ld;
  int32_t num_rows, V;
  const int32_t* rows;
  const int32_t* cu_seqlens;
  const int32_t* tokens;
  int32_t B, N, prompt, parts;  // parts: CTAs per row that starts anew
};

__device__ __forceinline__ int64_t seen_row_of(const SeenPar& p, int b) {
  const int row = p.rows ? __ldg(p.rows + b) : b;
  return row >= 0 && row < p.num_rows ? row : -1;
}

// Rows that start anew: a CTA owns kSegment words of a row, counts the row's tokens that fall
// there in shared memory and writes the words out, the row's only trip through memory.
// Emptying the rows and marking in a second kernel took 13.4 us for 64 prompts of up to 8192
// tokens (V 151936).  Where a row is named more than once its first entry's CTAs take the tokens
// of all.
constexpr int kSegment = 8192;
__global__ void __launch_bounds__(kThreads) seen_fill_kernel(const SeenPar p) {
  __shared__ __align__(16) uint32_t count[kSegment];
  const int b = blockIdx.x / p.parts, v0 = blockIdx.x % p.parts * kSegment;
  const int tid = threadIdx.x;
  launch_dependents();
  grid_dependency_wait();
  const int64_t row = seen_row_of(p, b);
  if (row < 0) return;
  bool before = false;
  if (p.rows)
    for (int i = tid; i < b; i += kThreads) before |= __ldg(p.rows + i) == row;
  for (int i = tid; i < kSegment / 4; i += kThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
  if (__syncthreads_or(before)) return;
  for (int i = b; i < p.B; ++i) {
    if (i > b) {  // the next entry with this row
      if (!p.rows) break;
      int next = p.B;
      for (int k0 = i; k0 < p.B && next == p.B; k0 += kThreads) {
        const bool same = k0 + tid < p.B && __ldg(p.rows + k0 + tid) == row;
        __shared__ int first;
        if (tid == 0) first = p.B;
        __syncthreads();
        if (same) atomicMin(&first, k0 + tid);
        __syncthreads();
        next = first;
        __syncthreads();
      }
      i = next;
      if (i >= p.B) break;
    }
    int t0 = i, t1 = min(i + 1, p.N);
    if (p.cu_seqlens) {
      t0 = max(__ldg(p.cu_seqlens + i), 0);
      t1 = min(__ldg(p.cu_seqlens + i + 1), p.N);
    }
#pragma unroll 8
    for (int t = t0 + tid; t < t1; t += kThreads) {
      const int v = __ldg(p.tokens + t);
      if (v >= 0 && v < p.V && v >= v0 && v < v0 + kSegment) atomicAdd(&count[v - v0], 1u);
    }
  }
  __syncthreads();
  const int n = (int)min((int64_t)kSegment, p.ld - v0);  // a multiple of 8
  uint4* dst = reinterpret_cast<uint4*>(p.seen + row * p.ld + v0);
  for (int i = tid; i < n / 8; i += kThreads) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 c = *reinterpret_cast<const uint2*>(&count[8 * i + 2 * e]);
      const uint32_t a = p.prompt ? (c.x ? 0x8000u : 0u) : min(c.x, 0x7FFFu);
      const uint32_t d = p.prompt ? (c.y ? 0x8000u : 0u) : min(c.y, 0x7FFFu);
      w[e] = a | (d << 16);
    }
    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(kThreads) seen_mark_kernel(const SeenPar p) {
  launch_dependents();
  grid_dependency_wait();
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t >= p.N) return;
  int b = t;
  if (p.cu_seqlens) {
    int lo = 0, hi = p.B;  // largest b with cu[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
    }
    if (t < __ldg(p.cu_seqlens + lo) || t >= __ldg(p.cu_seqlens + lo + 1)) return;
    b = lo;
  }
  const int64_t row = seen_row_of(p, b);
  const int v = __ldg(p.tokens + t);
  if (row < 0 || v < 0 || v >= p.V) return;
  unsigned short* at = p.seen + row * p.ld + v;
  unsigned short old = *reinterpret_cast<volatile unsigned short*>(at);
  for (;;) {  // ends: each failure is another thread's success, of which there are at most N
    unsigned short now = old;
    if (p.prompt) now |= 0x8000u;
    else if ((old & 0x7FFFu) != 0x7FFFu) now = old + 1;
    if (now == old) return;
    const unsigned short was = atomicCAS(at, old, now);
    if (was == old) return;
    old = was;
  }
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_rules(const attn_logits_rules_t* r, int32_t V) {
  if (r->seen) {
    if (!aligned(r->seen, 16) || r->seen_rows < 1 || r->seen_ld < V || r->seen_ld % 8 != 0) return ATTN_EINVAL;
  }
  if (r->bias_start && (!r->bias_token || !r->bias_value)) return ATTN_EINVAL;
  if (r->mask && (r->mask_rows < 1 || r->mask_ld < (V + 31) / 32)) return ATTN_EINVAL;
  for (const void* p : {(const void*)r->seen_row, (const void*)r->repetition, (const void*)r->presence,
                        (const void*)r->frequency, (const void*)r->bias_start, (const void*)r->bias_token,
                        (const void*)r->bias_value, (const void*)r->mask, (const void*)r->mask_row})
    if (!aligned(p, 4)) return ATTN_EINVAL;
  return ATTN_OK;
}

}  // namespace
}  // namespace gb300

using namespace gb300;

extern "C" {

int attn_logits_adjust(const float* logits, int32_t B, int32_t V, int64_t ld, const attn_logits_rules_t* rules,
                       float* out, int64_t ld_out, void* stream) {
  if (!logits || !rules || !out || !aligned(logits, 4) || !aligned(out, 4)) return ATTN_EINVAL;
  if (B < 0 || V < 1 || V > (1 << 23) || ld < V || ld_out < V || (logits == out && ld != ld_out)) return ATTN_EINVAL;
  int rc = check_rules(rules, V);
  if (rc) return rc;
  AdjustPar p;
  // runs of 4096 logits, of 1024 where that leaves SMs without any
  const bool small = (int64_t)B * ((V + 4095) / 4096) < 304;
  p.runs = small ? (V + 1023) / 1024 : (V + 4095) / 4096;
  if ((int64_t)B * p.runs > 0x7fffffff) return ATTN_EINVAL;
  if ((rc = abi_check_device())) return rc;
  if (B == 0) return ATTN_OK;
  p.logits = logits;
  p.out = out;
  p.ld = ld;
  p.ld_out = ld_out;
  p.V = V;
  p.r = *rules;
  const bool vec = aligned(logits, 16) && aligned(out, 16) && (B == 1 || (ld % 4 == 0 && ld_out % 4 == 0));
  auto kernel = small ? (vec ? logits_adjust_kernel<1, true> : logits_adjust_kernel<1, false>)
                      : (vec ? logits_adjust_kernel<4, true> : logits_adjust_kernel<4, false>);
  return launch_dependent(kernel, dim3((unsigned)(B * p.runs)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), p) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

int attn_tokens_seen(uint16_t* seen, int64_t ld, int32_t num_rows, int32_t V, const int32_t* rows,
                     const int32_t* cu_seqlens, const int32_t* tokens, int32_t B, int32_t N, int32_t flags,
                     void* stream) {
  if (!seen || !aligned(seen, 16) || !aligned(rows, 4) || !aligned(cu_seqlens, 4) || !aligned(tokens, 4)) return ATTN_EINVAL;
  if (B < 0 || N < 0 || (N > 0 && !tokens) || (!cu_seqlens && N != B)) return ATTN_EINVAL;
  if (V < 1 || V > (1 << 23) || ld < V || ld % 8 != 0 || num_rows < 1) return ATTN_EINVAL;
  if (flags & ~(ATTN_SEEN_PROMPT | ATTN_SEEN_CLEAR)) return ATTN_EINVAL;
  SeenPar p;
  const int64_t parts = (ld + kSegment - 1) / kSegment;
  if (B * parts > 0x7fffffff) return ATTN_EINVAL;
  p.parts = (int)parts;
  int rc = abi_check_device();
  if (rc) return rc;
  if (B == 0) return ATTN_OK;
  p.seen = seen;
  p.ld = ld;
  p.num_rows = num_rows;
  p.V = V;
  p.rows = rows;
  p.cu_seqlens = cu_seqlens;
  p.tokens = tokens;
  p.B = B;
  p.N = N;
  p.prompt = flags & ATTN_SEEN_PROMPT;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (flags & ATTN_SEEN_CLEAR)
    return launch_dependent(seen_fill_kernel, dim3((unsigned)(B * p.parts)), dim3(kThreads), 0, s, p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ELAUNCH;
  if (N == 0) return ATTN_OK;
  return launch_dependent(seen_mark_kernel, dim3((unsigned)(((int64_t)N + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                          s, p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // extern "C"
