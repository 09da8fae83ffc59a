// block_merge() of csrc/decode.cuh by itself: partial results and flags come from arrays.
// tests/test_gpu_block_merge.py compiles and runs it.
#include "../causal_gqa_attention_qkv_gb300/csrc/decode.cuh"

namespace gb300 {
namespace {

// mo [lists, splits, warps, G, D], mm and ml [lists, splits, warps, G], gave_up [lists, splits];
// a list is a (token, KV head).
template <int D>
__global__ void __launch_bounds__(kThreads) merge_kernel(const DecodePar p, const float* mo, const float* mm,
                                                         const float* ml, const int* gave_up) {
  extern __shared__ float smem[];
  __shared__ SplitSums<true> s_sums;
  const int split = blockIdx.x % p.max_splits, t = blockIdx.x / p.max_splits, kh = blockIdx.y;
  const int64_t at = ((int64_t)t * gridDim.y + kh) * p.max_splits + split;
  if (threadIdx.x >> 5 == kConsumerWarps) {
    block_merge_rest(p);
    return;
  }
  if (gave_up[at]) {
    block_merge_none(p, s_sums);
    return;
  }
  const int n = kConsumerWarps * p.G, tid = threadIdx.x;
  float *so = smem, *sm = so + n * D, *sl = sm + n;
  for (int i = tid; i < n * D; i += kConsumerWarps * 32) so[i] = mo[at * n * D + i];
  for (int i = tid; i < n; i += kConsumerWarps * 32) {
    sm[i] = mm[at * n + i];
    sl[i] = ml[at * n + i];
  }
  named_sync_consumers();
  block_merge<D>(p, so, sm, sl, s_sums, kh, t);
}

template <int D>
int run(const DecodePar& p, int N, int Hkv, const float* mo, const float* mm, const float* ml, const int* gave_up,
        cudaStream_t s) {
  const size_t smem = (size_t)kConsumerWarps * p.G * (D + 2) * 4;
  return launch_cluster_dependent(merge_kernel<D>, dim3(N * p.max_splits, Hkv), dim3(kThreads), smem, p.max_splits, s, p,
                                  mo, mm, ml, gave_up);
}

}  // namespace
}  // namespace gb300

// out: bf16 [N, Hkv * G * D]; G <= 8, 1 <= splits <= 16.
extern "C" __attribute__((visibility("default"))) int test_block_merge(int N, int Hkv, int G, int D, int splits,
                                                                       const float* mo, const float* mm, const float* ml,
                                                                       const int* gave_up, void* out, void* stream) {
  gb300::DecodePar p = {};
  p.Hq = Hkv * G;
  p.Hkv = Hkv;
  p.G = G;
  p.max_splits = splits;
  p.out = static_cast<uint16_t*>(out);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 128 ? gb300::run<128>(p, N, Hkv, mo, mm, ml, gave_up, s) : gb300::run<64>(p, N, Hkv, mo, mm, ml, gave_up, s);
}
