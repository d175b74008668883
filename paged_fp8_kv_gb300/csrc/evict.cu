// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence b, kv head g): with new = min(L, budget), the `new` slots that
// rank first by (protected, weight descending, slot ascending) are kept.  A
// kept slot below `new` stays where it is; the i-th kept slot at or past
// `new` moves into the i-th slot below `new` that is not kept.  Those two sets
// are disjoint from each other and of equal size, so the moves need no order,
// no buffer and no row is read after it was written; keeping the rows' order
// instead would shift nearly the whole cache behind the first evicted slot.
// Attention does not depend on the order of the keys it sees (K is cached
// rotated); what needs a token's position carries it in key_pos.
//
// Ranks are 32-bit keys: protected slots the largest, then the weights in
// order (sign-folded bits, -0 as 0), NaN the smallest.  The threshold comes
// from four 8-bit histogram passes (most significant digit first); slots equal
// to the threshold are kept in slot order until `new` is reached, by counting.
//
// Kernel 1 finds the threshold and writes the moves and the kept weights;
// kernel 2 copies the rows: eight lanes a row of 128 bytes, K and V, a CTA
// kMovesPerCta moves of one (b, g).

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMovesPerCta = 64;
constexpr int kStatusInvalidArg = 1;  // MJ_ERR_INVALID_ARG

__device__ __forceinline__ uint32_t rank_key(float w, bool held) {
  if (held) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the CTA (in thread order) and its total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int before = (warp > 0 ? warp_sums[warp - 1] : 0) + x - v;
  total = warp_sums[31];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictDev a) {
  // a programmatic dependent: no global access before the grid ahead is done
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int bg = blockIdx.x;
  const int b = bg / a.h_k, g = bg - b * a.h_k;
  const int tid = threadIdx.x;
  const int64_t max_len = static_cast<int64_t>(a.max_blocks) * a.page_size;
  int L = a.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (tid == 0 && a.status) atomicExch(a.status, kStatusInvalidArg);
    L = L < 0 ? 0 : static_cast<int>(max_len);
  }
  const int fresh = L < a.budget ? L : a.budget;  // the new length
  const int64_t off = b * a.acc_seq + g * a.acc_head;
  const float* acc = a.acc + off;
  const int32_t* pos = a.key_pos ? a.key_pos + off : nullptr;
  const int64_t end = (pos ? a.next_pos[b] : L) - static_cast<int64_t>(a.keep_last);
  auto key_of = [&](int j) {
    const int p = pos ? pos[j] : j;
    return rank_key(acc[j], p < a.keep_first || p >= end);
  };
  int32_t* const moves = a.moves + static_cast<int64_t>(bg) * a.moves_cap * 2;  // [dst | src]
  if (g == 0 && tid == 0) a.new_lens[b] = fresh;

  if (L <= a.budget) {  // nothing leaves
    if (tid == 0) a.counts[bg] = 0;
    for (int j = tid; j < L; j += kSelThreads) {
      if (a.acc_out != a.acc) a.acc_out[off + j] = acc[j];
      if (pos && a.key_pos_out != a.key_pos) a.key_pos_out[off + j] = pos[j];
    }
    return;
  }

  // ---- the threshold: the fresh-th largest key
  uint32_t prefix = 0;
  int need = fresh;  // how many of the keys with this prefix are kept
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < L; j += kSelThreads) {
      const uint32_t k = key_of(j);
      const uint32_t above = shift == 24 ? 0u : k >> (shift + 8);
      if (above == (shift == 24 ? 0u : prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // keys above the threshold are kept, and the first `need` equal to it

  // ---- keep flags, the ranks of holes and movers, in slot order
  int ties = 0, holes = 0, movers = 0;
  for (int j0 = 0; j0 < L; j0 += kSelThreads) {
    const int j = j0 + tid;
    const bool in = j < L;
    const uint32_t k = in ? key_of(j) : 0u;
    const bool tie = in && k == prefix;
    int total;
    const int before = block_scan(tie, warp_sums, total);
    const bool keep = in && (k > prefix || (tie && ties + before < need));
    ties += total;
    const bool hole = in && j < fresh && !keep, mover = keep && j >= fresh;
    const int rank = block_scan(static_cast<int>(hole) | (static_cast<int>(mover) << 16), warp_sums, total);
    if (hole) moves[holes + (rank & 0xFFFF)] = j;
    if (mover) moves[a.moves_cap + movers + (rank >> 16)] = j;
    holes += total & 0xFFFF;
    movers += total >> 16;
    if (keep && !mover) {
      if (a.acc_out != a.acc) a.acc_out[off + j] = acc[j];
      if (pos && a.key_pos_out != a.key_pos) a.key_pos_out[off + j] = pos[j];
    }
  }
  __syncthreads();
  for (int i = tid; i < holes; i += kSelThreads) {
    const int dst = moves[i], src = moves[a.moves_cap + i];
    a.acc_out[off + dst] = acc[src];
    if (pos) a.key_pos_out[off + dst] = pos[src];
  }
  if (tid == 0) a.counts[bg] = holes;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictDev a, int chunks) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int bg = blockIdx.x / chunks;
  const int b = bg / a.h_k, g = bg - b * a.h_k;
  const int n = a.counts[bg];
  const int first = (blockIdx.x - bg * chunks) * kMovesPerCta;
  if (first >= n) return;
  const int last = first + kMovesPerCta < n ? first + kMovesPerCta : n;
  const int32_t* moves = a.moves + static_cast<int64_t>(bg) * a.moves_cap * 2;
  const int32_t* table = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
  const int vecs = a.row_bytes / 16;  // 8, 6 or 4 of eight lanes
  const int lane8 = threadIdx.x & 7;
  // eight lanes a move: its K row and its V row
  for (int i = first + (threadIdx.x >> 3); i < last; i += kMoveThreads / 8) {
    const int dst = moves[i], src = moves[a.moves_cap + i];
    const int dp = table[dst / a.page_size], sp = table[src / a.page_size];
    if (dp < 0 || dp >= a.num_pages || sp < 0 || sp >= a.num_pages) {
      if (lane8 == 0 && a.status) atomicExch(a.status, kStatusInvalidArg);
      continue;
    }
    const int dr = dst % a.page_size, sr = src % a.page_size;
    if (lane8 < vecs) {
      const uint4 kv = *reinterpret_cast<const uint4*>(a.k + sp * a.k_page + sr * a.k_row + g * a.k_head + lane8 * 16);
      const uint4 vv = *reinterpret_cast<const uint4*>(a.v + sp * a.v_page + sr * a.v_row + g * a.v_head + lane8 * 16);
      *reinterpret_cast<uint4*>(a.k + dp * a.k_page + dr * a.k_row + g * a.k_head + lane8 * 16) = kv;
      *reinterpret_cast<uint4*>(a.v + dp * a.v_page + dr * a.v_row + g * a.v_head + lane8 * 16) = vv;
    }
    if (a.ks && lane8 < 2) {  // nvfp4: the row's eight scales, K on lane 0, V on lane 1
      uint8_t* const base = lane8 == 0 ? a.ks : a.vs;
      const int64_t page = lane8 == 0 ? a.ks_page : a.vs_page, head = lane8 == 0 ? a.ks_head : a.vs_head;
      *reinterpret_cast<uint2*>(base + dp * page + g * head + dr * 8) =
          *reinterpret_cast<const uint2*>(base + sp * page + g * head + sr * 8);
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictDev& a, cudaStream_t stream) {
  const unsigned groups = static_cast<unsigned>(a.num_seqs) * a.h_k;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(groups, 1, 1), dim3(kSelThreads, 1, 1), 0, stream, a);
  if (e != cudaSuccess || a.moves_cap == 0) return e;
  const int chunks = (a.moves_cap + kMovesPerCta - 1) / kMovesPerCta;
  return launch_pdl(evict_move_kernel, dim3(static_cast<unsigned>(chunks) * groups, 1, 1), dim3(kMoveThreads, 1, 1), 0,
                    stream, a, chunks);
}

}  // namespace mj
