// Rules on rows of logits and the table of seen tokens (include/logits.h).
//
// Each logit goes through x + bias, the repetition penalty, the frequency and
// presence penalties and the mask, each operation rounded to fp32.  Bound by memory:
// 4 bytes read and 4 written per logit, 2 of the table, an eighth of a byte of the mask.
// A CTA takes a run of one row and filters the row's biases, few and in any order, for it;
// those of one token are summed by one thread in list order (the order decides the rounding).
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

struct Penalties {
  float repetition, frequency, presence;
};
// A logit of a seen token, after the bias.
__device__ __forceinline__ float penalised(float x, uint32_t word, const Penalties& c) {
  if (c.repetition > 0.f) x = x > 0.f ? __fdiv_rn(x, c.repetition) : __fmul_rn(x, c.repetition);
  const uint32_t n = word & 0x7FFFu;
  if (n) {
    x = __fsub_rn(x, __fmul_rn(c.frequency, (float)n));
    x = __fsub_rn(x, c.presence);
  }
  return x;
}

constexpr int kListed = 1024;

// The row's biases for the tokens of a run in list order, summed into bias[] (kRun floats): each
// token's by one thread.  For rows with many of them.
__device__ void sum_biases(const attn_logits_rules_t& r, int e0, int e1, int v0, int n, int run, float* bias, int* tok,
                           float* val, int* cnt) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int k = tid; k < run; k += kThreads) bias[k] = 0.f;
  for (int e = e0; e < e1; e += kThreads) {
    const int i = e + tid;
    const int t = i < e1 ? __ldg(r.bias_token + i) : -1;
    const bool mine = t >= v0 && t < v0 + n;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) cnt[warp] = __popc(all);
    __syncthreads();
    int at = 0, m = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += cnt[w];
      m += cnt[w];
    }
    if (mine) {
      at += __popc(all & ((1u << lane) - 1u));
      tok[at] = t - v0;
      val[at] = __ldg(r.bias_value + i);
    }
    __syncthreads();
    for (int k = 0; k < m; ++k)
      if ((tok[k] & (kThreads - 1)) == tid) bias[tok[k]] += val[k];
    __syncthreads();
  }
}

// Four logits per thread and step, Q steps: all loads of a run go out before its biases are
// looked at.  Vec: rows of logits and out are 16-byte aligned, a thread's four are neighbours;
// else they are 256 apart (a row's start may lie anywhere).  Seen and biased tokens are few and
// scattered (a division in place would keep most warps for one lane): they go to lists in shared
// memory that the threads share out, and are stored after the others.  A list of seen
// tokens that is full leaves the rest in place; a run with more than kThreads biases takes
// sum_biases().
template <int Q, bool Vec>
__global__ void __launch_bounds__(kThreads) logits_adjust_kernel(const AdjustPar p) {
  constexpr int kRun = Q * 4 * kThreads;
  __shared__ __align__(16) float bias[kRun];
  __shared__ int tok[kThreads], idx[kThreads];
  __shared__ float val[kThreads];
  __shared__ int cnt[kThreads / 32], listed, biases;
  __shared__ float list_x[kListed];
  __shared__ uint32_t list_at[kListed];  // place in the run, word << 16
  const int b = blockIdx.x / p.runs, v0 = blockIdx.x % p.runs * kRun;
  const int tid = threadIdx.x;
  launch_dependents();
  if (tid == 0) listed = biases = 0;
  __syncthreads();
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
  auto allowed = [&](int i) { return !mask || (__ldg(mask + (i >> 5)) >> (i & 31) & 1u); };
  float x[Q][4];
  uint2 words[Q];     // of the four logits
  uint32_t allow[Q];  // bit e
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int i0 = place(q, 0);
    allow[q] = 15u;
    if (Vec && i0 + 4 <= n) {
      *reinterpret_cast<float4*>(x[q]) = *reinterpret_cast<const float4*>(in + i0);
      words[q] = seen ? *reinterpret_cast<const uint2*>(seen + i0) : make_uint2(0u, 0u);
      if (mask) allow[q] = __ldg(mask + (i0 >> 5)) >> (i0 & 31);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = place(q, e);
        const bool there = i < n;
        x[q][e] = there ? in[i] : 0.f;
        w[e] = there && seen ? seen[i] : 0u;
        if (mask && there && !allowed(i)) allow[q] &= ~(1u << e);
      }
      words[q] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
  const Penalties c = {p.r.repetition ? __ldg(p.r.repetition + b) : 0.f, p.r.frequency ? __ldg(p.r.frequency + b) : 0.f,
                       p.r.presence ? __ldg(p.r.presence + b) : 0.f};
  int few = 0;  // biases in the run, if they fit the list
  if (p.r.bias_start) {
    const int e0 = __ldg(p.r.bias_start + b), e1 = __ldg(p.r.bias_start + b + 1);
    for (int i = e0 + tid; i < e1; i += kThreads) {
      const int t = __ldg(p.r.bias_token + i) - v0;
      if (t >= 0 && t < n) {
        const int at = atomicAdd(&biases, 1);  // in any order
        if (at < kThreads) {
          tok[at] = t;
          val[at] = __ldg(p.r.bias_value + i);
          idx[at] = i;
        }
      }
    }
    __syncthreads();
    few = biases;
    if (few > kThreads) {
      sum_biases(p.r, e0, e1, v0, n, kRun, bias, tok, val, cnt);
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[q][e] = __fadd_rn(x[q][e], bias[place(q, e)]);
      few = 0;
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (mask) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[q][e] = allow[q] >> e & 1u ? x[q][e] : kNegInf;
    }
    if (words[q].x | words[q].y) {
      uint32_t w[4] = {words[q].x & 0xFFFFu, words[q].x >> 16, words[q].y & 0xFFFFu, words[q].y >> 16};
      int mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(allow[q] >> e & 1u)) w[e] = 0u;
        mine += w[e] != 0u;
      }
      if (mine > 0) {
        int at = atomicAdd(&listed, mine);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (w[e] == 0u) continue;
          if (at < kListed) {
            list_x[at] = x[q][e];
            list_at[at] = (uint32_t)place(q, e) | (w[e] << 16);
          } else {
            x[q][e] = penalised(x[q][e], w[e], c);
          }
          ++at;
        }
      }
    }
  }
  float special = 0.f;
  bool owner = false;  // of a biased token: the first of its entries in list order
  if (few > 0) {
    if (tid < few) {
      const int t = tok[tid], me = idx[tid];
      owner = true;
      float sum = 0.f;
      // its entries in list order: the next one is that with the smallest index above the last
      for (int last = -1;;) {
        int next = 0x7fffffff, at = 0;
        for (int k = 0; k < few; ++k)
          if (tok[k] == t && idx[k] > last && idx[k] < next) {
            next = idx[k];
            at = k;
          }
        if (next == 0x7fffffff) break;
        if (last < 0 && next != me) {  // another thread's token
          owner = false;
          break;
        }
        sum = __fadd_rn(sum, val[at]);
        last = next;
      }
      if (owner) {
        special = kNegInf;
        if (allowed(t)) {
          special = __fadd_rn(in[t], sum);
          const uint32_t w = seen ? seen[t] : 0u;
          if (w) special = penalised(special, w, c);
        }
      }
    }
    __syncthreads();  // in[] has been read where out is the same
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int i0 = place(q, 0);
    if (Vec && i0 + 4 <= n) {
      *reinterpret_cast<float4*>(out + i0) = *reinterpret_cast<const float4*>(x[q]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (place(q, e) < n) out[place(q, e)] = x[q][e];
    }
  }
  __syncthreads();  // the list is complete, and its logits are stored as they were before
  for (int k = tid; k < min(listed, kListed); k += kThreads)
    out[list_at[k] & 0xFFFFu] = penalised(list_x[k], list_at[k] >> 16, c);
  if (few > 0) {
    __syncthreads();
    if (owner) out[tok[tid]] = special;
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
