// The keys that any query token of a sequence sees under modified scores, and
// the length a plan has to cover (see mj_score_spans_device): one CTA a
// sequence takes the extremes of its tokens' ranges.

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "score_mod.cuh"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kSpanThreads = 128;

__global__ void __launch_bounds__(kSpanThreads)
    score_spans_kernel(const ScoreModDev m, const int32_t* seq_lens, int q_len, int causal, int64_t max_len, int4* spans,
                       int32_t* plan_lens) {
  __shared__ int first, last;
  if (threadIdx.x == 0) {
    first = INT32_MAX;
    last = -1;
  }
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.x;
  int L = seq_lens[b];
  L = L < 0 ? 0 : (L > max_len ? static_cast<int>(max_len) : L);
  RowRange r{0, -1, 0};
  int lo = INT32_MAX, hi = -1;
  for (int qi = threadIdx.x; qi < q_len; qi += kSpanThreads) {
    r = row_range(m, causal, q_len, b, L, qi);
    if (r.lo <= r.hi) {
      lo = r.lo < lo ? r.lo : lo;
      hi = r.hi > hi ? r.hi : hi;
    }
  }
  atomicMin(&first, lo);
  atomicMax(&last, hi);
  __syncthreads();
  if (threadIdx.x == 0) spans[b] = make_span(first, last, r.pfx, &plan_lens[b]);
}

}  // namespace

cudaError_t launch_score_spans(const ScoreModDev& m, const int32_t* seq_lens, int num_seqs, int q_len, int causal,
                               int64_t max_len, int4* spans, int32_t* plan_lens, cudaStream_t stream) {
  return launch_pdl(score_spans_kernel, dim3(static_cast<unsigned>(num_seqs), 1, 1), dim3(kSpanThreads, 1, 1), 0, stream,
                    m, seq_lens, q_len, causal, max_len, spans, plan_lens);
}

}  // namespace mj
