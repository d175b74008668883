// Pages handed out for new tokens and taken back (see mj_pages_reserve,
// mj_pages_release).
//
// What a call reads and writes is a few words a sequence, page and token (under
// 0.2 us at HBM's rate for 65000 tokens): it is bound by the launch and a chain
// of cold loads, lengths -> table entry -> store.  One launch therefore does it
// all: a cluster of CTAs each of which makes the prefix sums over all sequences
// for itself (a thousand threads, one sequence each in a decode batch) and then
// takes its share of the tokens and pages, finding each one's sequence by a
// binary search in shared memory.  The lengths and the list's size may be
// written where they were read: the cluster's barrier is between.  Numbers that
// are no page of the pool are neither given nor taken back: every CTA looks at
// all pages to be given (a round of loads that the stores repeat from L1: 0.2 us
// of the smallest call; looked at when the sums are done 0.1 more, loaded ahead
// of the sums no less); what comes back is written as it is read, and once more
// by one CTA if a number among it was none.
//
// Measured: one token for each of 256 sequences 4.9 us a call (4.6 in a graph),
// 33 prompts of 65000 tokens in all 11.5 (10.4; two tokens a thread in flight for
// four made no difference beyond the noise), a trim 4.4 (4.0).

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;  // CTAs of a call with many tokens or pages
constexpr int kStatusInvalid = 1;   // MJ_ERR_INVALID_ARG
constexpr int kStatusCapacity = 3;  // MJ_ERR_CAPACITY

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// *flag = 1 in the cluster's first CTA
__device__ __forceinline__ void set_in_first(int* flag) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"(ptx::smem_u32(flag)));
  asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(at) : "memory");
}

__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

struct Pair {
  int64_t a, b;
};

// Inclusive prefix sums of two values over the block, and the block's totals.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* red, Pair* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair inc{warp_scan(v.a, lane), warp_scan(v.b, lane)};
  __syncthreads();  // red is free
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const Pair x = red[lane];
    red[lane] = Pair{warp_scan(x.a, lane), warp_scan(x.b, lane)};
  }
  __syncthreads();
  *total = red[kWarps - 1];
  if (warp > 0) {
    inc.a += red[warp - 1].a;
    inc.b += red[warp - 1].b;
  }
  return inc;
}

// The last b with off[b] <= x (off[0] = 0; sequences without an element share
// the offset of the one behind them).
__device__ __forceinline__ int find(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp32(int64_t x) {
  return x > INT32_MAX ? INT32_MAX : static_cast<int32_t>(x);
}

__device__ __forceinline__ void report(int32_t* status, int what) {
  if (status) atomicExch(status, what);
}

__global__ void __launch_bounds__(kThreads, 1) reserve_kernel(const PagesDev a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ int32_t smem[];
  int32_t* const tok = smem;                       // [num_seqs + 1] tokens before b
  int32_t* const need = tok + a.num_seqs + 1;      // [num_seqs + 1] pages before b
  int32_t* const held = need + a.num_seqs + 1;     // [num_seqs] tokens held; -1: gets no slots
  __shared__ Pair red[kWarps];
  __shared__ int wrong, taken;  // bit 0: an invalid length or page, bit 1: too few pages
  __shared__ int bad_page;      // the first of the list's pages, from its end, that is none
  const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
  const int shift = a.page_shift, row_mask = (1 << shift) - 1;
  if (tid == 0) {
    wrong = taken = 0;
    tok[0] = need[0] = 0;
    bad_page = INT32_MAX;
  }
  int n_free = a.num_free[0];
  if (n_free < 0 || n_free > a.num_pages) {
    n_free = 0;
    if (tid == 0) wrong = 1;
  }
  auto free_page = [&](int x) { return __ldg(a.free_pages + n_free - 1 - x); };
  auto is_page = [&](int64_t page) { return page >= 0 && page < a.num_pages; };
  __syncthreads();
  for (int avail = n_free;;) {  // pages that may be given
    Pair base{0, 0};
    for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
      const int b = b0 + tid;
      Pair v{0, 0};
      int old = -1;
      if (b < a.num_seqs) {
        const int L = a.seq_lens[b], n = a.new_tokens ? a.new_tokens[b] : a.q_len;
        if (L < 0 || n < 0) {
          atomicOr(&wrong, 1);
        } else {
          v.a = n;
          if (static_cast<int64_t>(L) + n > a.max_len) {
            atomicOr(&wrong, 1);
          } else {
            old = L;
            v.b = ((static_cast<int64_t>(L) + n + row_mask) >> shift) - ((static_cast<int64_t>(L) + row_mask) >> shift);
          }
        }
      }
      Pair total;
      const Pair inc = block_scan(v, red, &total);
      if (b < a.num_seqs) {
        const int64_t end = base.b + inc.b;
        if (v.b > 0 && end > avail) {  // its pages are no longer in the list
          old = -1;
          atomicOr(&wrong, 2);
        } else if (v.b > 0) {
          atomicMax(&taken, static_cast<int>(end));
        }
        tok[b + 1] = clamp32(base.a + inc.a);
        need[b + 1] = clamp32(end);
        held[b] = old;
      }
      base.a += total.a;
      base.b += total.b;
    }
    // The pages to give, all of them looked at by every CTA, a thousand before the
    // sums are done: the list ends at one that is no page of the pool, and what its
    // sequence and those behind it wanted is left out.
    if (tid < n_free && !is_page(free_page(tid))) atomicMin(&bad_page, tid);
    __syncthreads();
    if (taken > kThreads) {
      for (int x = kThreads + tid; x < taken; x += kThreads)
        if (!is_page(free_page(x))) atomicMin(&bad_page, x);
      __syncthreads();
    }
    if (bad_page >= taken) break;  // (the second time at the latest: no more than bad_page are taken then)
    avail = bad_page;
    __syncthreads();  // both are read
    if (tid == 0) {
      wrong |= 1;
      taken = 0;
    }
    __syncthreads();
  }
  const int tokens = tok[a.num_seqs];
  if (tid == 0 && rank == 0) {
    if ((wrong & 1) || ((a.positions || a.slots) && tokens > a.num_tokens))
      report(a.status, kStatusInvalid);
    else if (wrong && a.status)
      atomicCAS(a.status, 0, kStatusCapacity);  // (what is wrong may be reported meanwhile)
  }
  // the new tokens' positions and slots
  bool bad_held = false;  // a page that a sequence holds is none
  if (a.positions || a.slots) {
    // four a thread at a time, so that their loads are in flight together
    constexpr int kBatch = 4;
    constexpr int64_t kNone = INT64_MIN;
    const int step = ctas * kThreads;
    for (int t0 = rank * kThreads + tid; t0 < a.num_tokens; t0 += kBatch * step) {
      int pos[kBatch];
      int64_t slot[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i * step;
        pos[i] = 0;
        slot[i] = kNone;
        if (t < a.num_tokens && t < tokens) {
          const int b = find(tok, a.num_seqs, t);
          const int old = held[b];
          if (old >= 0) {
            pos[i] = old + t - tok[b];
            const int blk = pos[i] >> shift, have = (old + row_mask) >> shift;
            // (the old pages' entries are not written here, the new ones' not read)
            if (a.slots)
              slot[i] = blk < have ? __ldg(a.block_table + static_cast<int64_t>(b) * a.max_blocks + blk)
                                   : free_page(need[b] + blk - have);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i * step;
        if (t >= a.num_tokens) continue;
        if (a.positions) a.positions[t] = pos[i];
        if (a.slots) a.slots[t] = is_page(slot[i]) ? (slot[i] << shift) + (pos[i] & row_mask) : -1;
        bad_held |= slot[i] != kNone && !is_page(slot[i]);
      }
    }
  }
  if (bad_held) report(a.status, kStatusInvalid);
  // the new pages' entries
  for (int x = rank * kThreads + tid; x < taken; x += ctas * kThreads) {
    const int b = find(need, a.num_seqs, x);
    const int blk = ((held[b] + row_mask) >> shift) + x - need[b];
    a.block_table_out[static_cast<int64_t>(b) * a.max_blocks + blk] = free_page(x);
  }
  // every CTA of the cluster has read the lengths and the list's size
  if (ctas > 1) cluster_sync();
  for (int b = rank * kThreads + tid; b < a.num_seqs; b += ctas * kThreads) {
    const int old = held[b];
    // (the sums of tokens may have been clamped)
    const int n = old < 0 ? 0 : (a.new_tokens ? a.new_tokens[b] : a.q_len);
    a.seq_lens_out[b] = old >= 0 ? old + n : a.seq_lens[b];
    if (a.granted) a.granted[b] = n;
  }
  if (a.cu_tokens)
    for (int b = rank * kThreads + tid; b <= a.num_seqs; b += ctas * kThreads) a.cu_tokens[b] = tok[b];
  if (rank == 0 && tid == 0) a.num_free_out[0] = n_free - taken;
}

__global__ void __launch_bounds__(kThreads, 1) release_kernel(const PagesDev a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ int32_t smem[];
  int32_t* const gone = smem;                   // [num_seqs + 1] pages before b
  int32_t* const kept = gone + a.num_seqs + 1;  // [num_seqs] pages that stay
  __shared__ Pair red[kWarps];
  __shared__ int wrong, bad_page;  // bad_page: of the first CTA, one that is no page is among those given back
  const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
  const int shift = a.page_shift, row_mask = (1 << shift) - 1;
  if (tid == 0) {
    wrong = bad_page = 0;
    gone[0] = 0;
  }
  if (ctas > 1) cluster_arrive();  // bad_page may be set from here on
  int n_free = a.num_free[0];
  if (n_free < 0 || n_free > a.num_pages) {
    n_free = 0;
    if (tid == 0) wrong = kStatusInvalid;
  }
  __syncthreads();
  int64_t base = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
    const int b = b0 + tid;
    Pair v{0, 0};
    if (b < a.num_seqs) {
      const int L = a.seq_lens[b], keep = a.new_tokens[b];
      if (keep < 0 || keep > L || L > a.max_len) {
        wrong = kStatusInvalid;
      } else {
        kept[b] = (keep + row_mask) >> shift;
        v.a = ((L + row_mask) >> shift) - kept[b];
      }
    }
    Pair total;
    const Pair inc = block_scan(v, red, &total);
    if (b < a.num_seqs) gone[b + 1] = clamp32(base + inc.a);
    base += total.a;
  }
  __syncthreads();
  int pages = gone[a.num_seqs];
  if (pages > a.num_pages - n_free) {  // more than the pool has: some were given back before
    pages = a.num_pages - n_free;
    if (tid == 0 && rank == 0) report(a.status, kStatusCapacity);
  } else if (wrong && tid == 0 && rank == 0) {
    report(a.status, wrong);
  }
  if (ctas > 1) cluster_wait();
  auto is_page = [&](int page) { return page >= 0 && page < a.num_pages; };
  for (int x = rank * kThreads + tid; x < pages; x += ctas * kThreads) {
    const int b = find(gone, a.num_seqs, x);
    const int page = a.block_table[static_cast<int64_t>(b) * a.max_blocks + kept[b] + x - gone[b]];
    a.free_pages_out[n_free + x] = page;
    if (!is_page(page)) set_in_first(&bad_page);
  }
  if (ctas > 1)  // every CTA has read the list's size
    cluster_sync();
  else
    __syncthreads();
  if (rank != 0) return;
  if (bad_page) {
    // An entry is no page of the pool: the first CTA writes the others' once more
    // without it, a thread a sequence.
    int at = n_free, full = 0;
    for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
      const int b = b0 + tid;
      const int64_t row = static_cast<int64_t>(b) * a.max_blocks;
      const int first = b < a.num_seqs ? kept[b] : 0, n = b < a.num_seqs ? gone[b + 1] - gone[b] : 0;
      Pair v{0, 0};
      for (int i = 0; i < n; ++i) v.a += is_page(a.block_table[row + first + i]);
      Pair total;
      const Pair inc = block_scan(v, red, &total);
      int64_t to = at + inc.a - v.a;
      for (int i = 0; i < n; ++i) {
        const int page = a.block_table[row + first + i];
        if (is_page(page) && to++ < a.num_pages) a.free_pages_out[to - 1] = page;
      }
      if (at + total.a > a.num_pages) full = 1;
      at = full ? a.num_pages : static_cast<int>(at + total.a);
    }
    pages = at - n_free;
    if (tid == 0) report(a.status, full ? kStatusCapacity : kStatusInvalid);
  }
  if (tid == 0) a.num_free_out[0] = n_free + pages;
}

cudaError_t launch(void (*kern)(PagesDev), const PagesDev& a, size_t smem, int64_t elements, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const unsigned ctas = elements > 4 * kThreads ? kCluster : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_pages_reserve(const PagesDev& a, cudaStream_t stream) {
  const int64_t tokens = a.positions || a.slots ? a.num_tokens : 0;
  return launch(reserve_kernel, a, (3 * static_cast<size_t>(a.num_seqs) + 2) * 4, tokens, stream);
}

cudaError_t launch_pages_release(const PagesDev& a, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(a.num_seqs) * a.max_blocks;  // pages, at most
  return launch(release_kernel, a, (2 * static_cast<size_t>(a.num_seqs) + 1) * 4, most < a.num_pages ? most : a.num_pages,
                stream);
}

}  // namespace mj
