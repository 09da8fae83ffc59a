// Rules on rows of logits and the table of seen tokens (include/logits.h).
//
// Each logit goes through x + bias, the repetition penalty, the frequency and
// presence penalties and the mask, each operation rounded to fp32.  Bound by memory:
// 4 bytes read and 4 written per logit, 2 of the table, an eighth of a byte of the mask.
// A CTA takes a run of one row and filters the row's biases, few and in any order, for it;
// those of one token are summed by one thread in list order (the order decides the rounding).
//
// Dependents start only behind these kernels' own wait (see blocks.cu).
#include <algorithm>
#include <type_traits>

#include "kernels.cuh"
#include "../../include/logits.h"

namespace gb300 {

namespace {

constexpr int kThreads = 256;  // of the kernels for seen tokens
constexpr int kAdjust = 128;   // of a run of logits
constexpr int kSteps = 2;      // of four logits per thread
constexpr int kFew = kAdjust;  // biases of a run that are handled one per thread

struct AdjustPar {
  const float* logits;
  float* out;
  int64_t ld, ld_out;
  int32_t V;
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

// The row's biases for the tokens of a run in list order, summed into bias[] (kRun floats): each
// token's by one thread.  For rows with many of them.
__device__ void sum_biases(const attn_logits_rules_t& r, int e0, int e1, int v0, int n, int run, float* bias, int* tok,
                           float* val, int* cnt) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int k = tid; k < run; k += kAdjust) bias[k] = 0.f;
  for (int64_t e = e0; e < e1; e += kAdjust) {
    const int64_t i = e + tid;
    const int t = i < e1 ? __ldg(r.bias_token + i) : -1;
    const bool mine = t >= v0 && t < v0 + n;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) cnt[warp] = __popc(all);
    __syncthreads();
    int at = 0, m = 0;
    for (int w = 0; w < kAdjust / 32; ++w) {
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
      if ((tok[k] & (kAdjust - 1)) == tid) bias[tok[k]] += val[k];
    __syncthreads();
  }
}

// Four logits per thread and step, Q steps: all loads of a run go out before its biases are
// looked at.  Vec: rows of logits and out are 16-byte aligned, a thread's four are neighbours;
// else they are kAdjust apart (a row's start may lie anywhere).  Seen and biased tokens are few
// and scattered (a division in place would keep most warps for one lane: 42.7 us for 64 rows
// of 151936): they go to lists in shared memory that the threads share out, and are stored
// after the others.  A run with more than kFew biases takes sum_biases().  A run is a chain
// of latencies, so runs are short and sixteen CTAs share an SM: 23.9 us, 4.1 TB/s (16 logits per
// thread and ten CTAs 26.1, 256 threads and five 28.2; without any rule the same rows take 8 us
// from L2).
template <int Q, bool Vec>
__global__ void __launch_bounds__(kAdjust, 16) logits_adjust_kernel(const AdjustPar p) {
  constexpr int kRun = Q * 4 * kAdjust;
  __shared__ __align__(16) float bias[kRun];  // where they are many
  __shared__ uint16_t list_at[kRun];
  __shared__ uint32_t is_biased[kRun / 32];
  __shared__ int tok[kFew], idx[kFew];
  __shared__ float val[kFew];
  __shared__ int cnt[kAdjust / 32], listed, biases;
  const int b = blockIdx.x, v0 = blockIdx.y * kRun;  // low tokens first: vocabularies mostly list the frequent ones there
  const int tid = threadIdx.x;
  if (tid == 0) listed = biases = 0;
  if (tid < kRun / 32) is_biased[tid] = 0u;
  __syncthreads();
  grid_dependency_wait();
  launch_dependents();
  const int n = min(kRun, p.V - v0);  // logits of this run
  const float* in = p.logits + b * p.ld + v0;
  float* out = p.out + b * p.ld_out + v0;
  // what is known of the row, in one round of loads
  const int seen_at = p.r.seen && p.r.seen_row ? __ldg(p.r.seen_row + b) : b;
  const int mask_at = p.r.mask && p.r.mask_row ? __ldg(p.r.mask_row + b) : b;
  const int e0 = p.r.bias_start ? max(__ldg(p.r.bias_start + b), 0) : 0;
  const int e1 = p.r.bias_start ? min(__ldg(p.r.bias_start + b + 1), p.r.num_biases) : 0;
  const Penalties c = {p.r.repetition ? __ldg(p.r.repetition + b) : 0.f, p.r.frequency ? __ldg(p.r.frequency + b) : 0.f,
                       p.r.presence ? __ldg(p.r.presence + b) : 0.f};
  auto place = [&](int q, int e) { return Vec ? (q * kAdjust + tid) * 4 + e : (q * 4 + e) * kAdjust + tid; };
  float x[Q][4];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (Vec && place(q, 0) + 4 <= n) {
      *reinterpret_cast<float4*>(x[q]) = *reinterpret_cast<const float4*>(in + place(q, 0));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[q][e] = place(q, e) < n ? in[place(q, e)] : 0.f;
    }
  }
  const uint16_t* seen =
      p.r.seen && seen_at >= 0 && seen_at < p.r.seen_rows ? p.r.seen + seen_at * p.r.seen_ld + v0 : nullptr;
  const uint32_t* mask =
      p.r.mask && mask_at >= 0 && mask_at < p.r.mask_rows ? p.r.mask + mask_at * p.r.mask_ld + (v0 >> 5) : nullptr;
  auto allowed = [&](int i) { return !mask || (__ldg(mask + (i >> 5)) >> (i & 31) & 1u); };
  uint2 words[Q];     // of the four logits
  uint32_t allow[Q];  // bit e
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int i0 = place(q, 0);
    allow[q] = 15u;
    words[q] = make_uint2(0u, 0u);
    if (Vec && i0 + 4 <= n) {
      if (seen) words[q] = *reinterpret_cast<const uint2*>(seen + i0);
      if (mask) allow[q] = __ldg(mask + (i0 >> 5)) >> (i0 & 31);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = place(q, e);
        w[e] = i < n && seen ? seen[i] : 0u;
        if (mask && i < n && !allowed(i)) allow[q] &= ~(1u << e);
      }
      words[q] = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
  int few = 0;  // biases in the run, if they fit the list
  if (e1 > e0) {
    for (int64_t i0 = e0; i0 < e1; i0 += 4 * kAdjust) {
      int t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t i = i0 + k * kAdjust + tid;
        t[k] = i < e1 ? __ldg(p.r.bias_token + i) - v0 : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (t[k] < 0 || t[k] >= n) continue;
        const int i = (int)i0 + k * kAdjust + tid;  // an entry: below e1
        const int at = atomicAdd(&biases, 1);  // in any order
        atomicOr(&is_biased[t[k] >> 5], 1u << (t[k] & 31));
        if (at < kFew) {
          tok[at] = t[k];
          val[at] = __ldg(p.r.bias_value + i);
          idx[at] = i;
        }
      }
    }
    __syncthreads();
    few = biases;
    if (few > kFew) {
      sum_biases(p.r, e0, e1, v0, n, kRun, bias, tok, val, cnt);
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = place(q, e);  // a logit without a bias stays as it is: -0 + 0 would be 0
          if (is_biased[i >> 5] >> (i & 31) & 1u) x[q][e] = __fadd_rn(x[q][e], bias[i]);
        }
      few = 0;
      __syncthreads();
    }
  }
  // a biased token's own logit, word and bit, on their way while the others are looked at
  float special = 0.f;
  uint32_t special_word = 0u;
  bool special_allowed = false;
  if (tid < few) {
    const int t = tok[tid];
    special = in[t];
    if (seen) special_word = seen[t];
    special_allowed = allowed(t);
  }
  uint32_t marks = 0u;  // bit 4 q + e: seen, allowed
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (mask) {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[q][e] = allow[q] >> e & 1u ? x[q][e] : kNegInf;
    }
    // bits 15 and 31 of a word pair: that word is not 0
    const uint32_t u = (((words[q].x & 0x7FFF7FFFu) + 0x7FFF7FFFu) | words[q].x) & 0x80008000u;
    const uint32_t v = (((words[q].y & 0x7FFF7FFFu) + 0x7FFF7FFFu) | words[q].y) & 0x80008000u;
    marks |= (((u >> 15 | u >> 30) | (v >> 13 | v >> 28)) & allow[q] & 15u) << (4 * q);
  }
  if (marks) {
    int at = atomicAdd(&listed, __popc(marks));  // in any order
    for (; marks; marks &= marks - 1u) {
      const int k = __ffs((int)marks) - 1;
      list_at[at++] = (uint16_t)place(k >> 2, k & 3);
    }
  }
  bool owner = tid < few;  // of a biased token: the first of its entries in list order
  if (owner) {
    const int t = tok[tid], me = idx[tid];
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
    if (special_allowed) {
      special = __fadd_rn(special, sum);
      if (special_word) special = penalised(special, special_word, c);
    } else {
      special = kNegInf;
    }
  }
  if (p.logits == p.out && few > 0) __syncthreads();  // the biased logits have been read
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
  __syncthreads();  // the list is complete, and its logits are stored without penalties
  for (int k = tid; k < listed; k += kAdjust) {
    const int i = list_at[k];
    if (few == 0 || !(is_biased[i >> 5] >> (i & 31) & 1u)) out[i] = penalised(out[i], seen[i], c);
  }
  if (owner) out[tok[tid]] = special;
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
// there in shared memory and writes the words out, the row's only trip through memory: 7.4 us
// for 64 prompts of up to 8192 tokens (V 151936; with counts 10), and 14.2 with the rows emptied
// first and marked by a second kernel.  Where a row is named more than once its first entry's CTAs take the tokens
// of all.
constexpr int kSegment = 8192;
template <bool Prompt>
__global__ void __launch_bounds__(kThreads) seen_fill_kernel(const SeenPar p) {
  using Mark = std::conditional_t<Prompt, uint8_t, uint32_t>;  // there or not; how often
  __shared__ __align__(16) Mark mark[kSegment];
  const int b = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  launch_dependents();
  const int64_t row = seen_row_of(p, b);
  int t0 = b, t1 = min(b + 1, p.N);
  if (p.cu_seqlens) {
    t0 = max(__ldg(p.cu_seqlens + b), 0);
    t1 = min(__ldg(p.cu_seqlens + b + 1), p.N);
  }
  if (row < 0) return;
  bool before = false, after = false;  // other entries with this row
  if (p.rows)
    for (int i = tid; i < p.B; i += kThreads) {
      const bool same = __ldg(p.rows + i) == row;
      before |= same && i < b;
      after |= same && i > b;
    }
  for (int i = tid; i < (int)sizeof(mark) / 16; i += kThreads) reinterpret_cast<uint4*>(mark)[i] = make_uint4(0, 0, 0, 0);
  if (__syncthreads_or(before)) return;
  const bool again = __syncthreads_or(after);
  for (int i = b;;) {
#pragma unroll 8
    for (int64_t t = t0 + tid; t < t1; t += kThreads) {
      const uint32_t v = (uint32_t)__ldg(p.tokens + t);
      if (v < (uint32_t)p.V && v / kSegment == (uint32_t)part) {
        if constexpr (Prompt) mark[v % kSegment] = 1;
        else atomicAdd(&mark[v % kSegment], 1u);
      }
    }
    if (!again) break;
    do ++i; while (i < p.B && __ldg(p.rows + i) != row);  // the next one, the same for every thread
    if (i >= p.B) break;
    t0 = i;
    t1 = min(i + 1, p.N);
    if (p.cu_seqlens) {
      t0 = max(__ldg(p.cu_seqlens + i), 0);
      t1 = min(__ldg(p.cu_seqlens + i + 1), p.N);
    }
  }
  __syncthreads();
  const int64_t v0 = (int64_t)part * kSegment;  // rows may be longer than 2^31 words
  const int n = (int)min((int64_t)kSegment, p.ld - v0);  // a multiple of 8
  uint4* dst = reinterpret_cast<uint4*>(p.seen + row * p.ld + v0);
  for (int i = tid; i < n / 8; i += kThreads) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = mark[8 * i + 2 * e], v = mark[8 * i + 2 * e + 1];
      w[e] = Prompt ? (u << 15) | (v << 31) : min(u, 0x7FFFu) | (min(v, 0x7FFFu) << 16);
    }
    dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__global__ void __launch_bounds__(kThreads) seen_mark_kernel(const SeenPar p) {
  grid_dependency_wait();
  launch_dependents();
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= p.N) return;
  int b = (int)t;
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
  if (r->bias_start && (r->num_biases < 0 || (r->num_biases > 0 && (!r->bias_token || !r->bias_value)))) return ATTN_EINVAL;
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
  if (!rules || (B != 0 && (!logits || !out)) || !aligned(logits, 4) || !aligned(out, 4)) return ATTN_EINVAL;
  if (B < 0 || V < 1 || V > (1 << 23) || ld < V || ld_out < V || (logits == out && ld != ld_out)) return ATTN_EINVAL;
  int rc = check_rules(rules, V);
  if (rc) return rc;
  // Runs of 1024 logits, of 512 where those are few: 1 x 151936 3.7 and 3.2 us, 8 x 32003 5.4 and 3.8,
  // 32 x 32003 6.9 and 6.4, 64 x 151936 23.9 and 30.0.
  constexpr int kBig = kSteps * 4 * kAdjust, kSmall = 4 * kAdjust;
  const bool small = (int64_t)B * ((V + kBig - 1) / kBig) < 1216;
  const int runs = small ? (V + kSmall - 1) / kSmall : (V + kBig - 1) / kBig;  // at most 2^14
  if ((rc = abi_check_device())) return rc;
  if (B == 0) return ATTN_OK;
  AdjustPar p;
  p.logits = logits;
  p.out = out;
  p.ld = ld;
  p.ld_out = ld_out;
  p.V = V;
  p.r = *rules;
  const bool vec = aligned(logits, 16) && aligned(out, 16) && (B == 1 || (ld % 4 == 0 && ld_out % 4 == 0));
  auto kernel = small ? (vec ? logits_adjust_kernel<1, true> : logits_adjust_kernel<1, false>)
                      : (vec ? logits_adjust_kernel<kSteps, true> : logits_adjust_kernel<kSteps, false>);
  return launch_dependent(kernel, dim3((unsigned)B, (unsigned)runs), dim3(kAdjust), 0, static_cast<cudaStream_t>(stream), p) ==
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
  const int64_t parts = ld / kSegment + (ld % kSegment != 0);
  if ((flags & ATTN_SEEN_CLEAR) && parts > 0x7fffffff / std::max(B, 1)) return ATTN_EINVAL;  // CTAs of the call
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
    return launch_dependent(p.prompt ? seen_fill_kernel<true> : seen_fill_kernel<false>, dim3((unsigned)(B * p.parts)), dim3(kThreads), 0, s, p) == cudaSuccess
               ? ATTN_OK
               : ATTN_ELAUNCH;
  if (N == 0) return ATTN_OK;
  return launch_dependent(seen_mark_kernel, dim3((unsigned)(((int64_t)N + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                          s, p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // extern "C"
