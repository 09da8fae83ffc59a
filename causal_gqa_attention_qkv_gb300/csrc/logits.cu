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
constexpr int kRun = 4096;  // logits per CTA

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

__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const AdjustPar p) {
  __shared__ float bias[kRun];
  __shared__ int tok[kThreads];
  __shared__ float val[kThreads];
  __shared__ int cnt[kThreads / 32];
  const int b = blockIdx.x / p.runs, v0 = blockIdx.x % p.runs * kRun;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  grid_dependency_wait();
  const int v1 = min(v0 + kRun, p.V);
  bool biased = false;
  if (p.r.bias_start) {
    const int e0 = __ldg(p.r.bias_start + b), e1 = __ldg(p.r.bias_start + b + 1);
    for (int e = e0; e < e1; e += kThreads) {
      const int i = e + tid;
      const int t = i < e1 ? __ldg(p.r.bias_token + i) : -1;
      const bool mine = t >= v0 && t < v1;
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
  const uint16_t* seen = nullptr;
  if (p.r.seen) {
    const int row = p.r.seen_row ? __ldg(p.r.seen_row + b) : b;
    if (row >= 0 && row < p.r.seen_rows) seen = p.r.seen + row * p.r.seen_ld;
  }
  const uint32_t* mask = nullptr;
  if (p.r.mask) {
    const int row = p.r.mask_row ? __ldg(p.r.mask_row + b) : b;
    if (row >= 0 && row < p.r.mask_rows) mask = p.r.mask + row * p.r.mask_ld;
  }
  const float rep = p.r.repetition ? __ldg(p.r.repetition + b) : 0.f;
  const float freq = p.r.frequency ? __ldg(p.r.frequency + b) : 0.f;
  const float pres = p.r.presence ? __ldg(p.r.presence + b) : 0.f;
  const float* in = p.logits + b * p.ld;
  float* out = p.out + b * p.ld_out;
  for (int v = v0 + tid; v < v1; v += kThreads) {
    float x = in[v];
    if (biased) x = __fadd_rn(x, bias[v - v0]);
    const uint32_t word = seen ? seen[v] : 0u;
    const bool allowed = !mask || (__ldg(mask + (v >> 5)) >> (v & 31) & 1u);
    out[v] = apply_rules(x, word, rep, freq, pres, allowed);
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
  int32_t B, N, prompt, parts;  // parts: CTAs per row that is emptied
};

__device__ __forceinline__ int64_t seen_row_of(const SeenPar& p, int b) {
  const int row = p.rows ? __ldg(p.rows + b) : b;
  return row >= 0 && row < p.num_rows ? row : -1;
}

__global__ void __launch_bounds__(kThreads) seen_clear_kernel(const SeenPar p) {
  launch_dependents();
  grid_dependency_wait();
  const int64_t row = seen_row_of(p, blockIdx.x / p.parts);
  if (row < 0) return;
  uint4* dst = reinterpret_cast<uint4*>(p.seen + row * p.ld);
  for (int64_t i = (int64_t)(blockIdx.x % p.parts) * kThreads + threadIdx.x; i < p.ld / 8; i += (int64_t)p.parts * kThreads)
    dst[i] = make_uint4(0, 0, 0, 0);
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
  p.runs = (V + kRun - 1) / kRun;
  if ((int64_t)B * p.runs > 0x7fffffff) return ATTN_EINVAL;
  if ((rc = abi_check_device())) return rc;
  if (B == 0) return ATTN_OK;
  p.logits = logits;
  p.out = out;
  p.ld = ld;
  p.ld_out = ld_out;
  p.V = V;
  p.r = *rules;
  return launch_dependent(logits_adjust_kernel, dim3((unsigned)(B * p.runs)), dim3(kThreads), 0,
                          static_cast<cudaStream_t>(stream), p) == cudaSuccess
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
  p.parts = (int)std::min<int64_t>((ld / 8 + kThreads - 1) / kThreads, 1024);
  if ((int64_t)B * p.parts > 0x7fffffff) return ATTN_EINVAL;
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
  if ((flags & ATTN_SEEN_CLEAR) &&
      launch_dependent(seen_clear_kernel, dim3((unsigned)(B * p.parts)), dim3(kThreads), 0, s, p) != cudaSuccess)
    return ATTN_ELAUNCH;
  if (N == 0) return ATTN_OK;
  return launch_dependent(seen_mark_kernel, dim3((unsigned)(((int64_t)N + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                          s, p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // extern "C"
