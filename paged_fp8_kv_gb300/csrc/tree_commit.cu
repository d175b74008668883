// The accepted branch of a drafted tree moved to the front of it (see
// mj_tree_commit): slot ctx + i <- slot ctx + accepted[i], in place.
//
// One CTA a sequence.  A thread owns a 16-byte column of the rows (of one kv
// head, of K or V; 8 bytes of a scale plane; a position) and takes the branch in
// order, eight rows read before they are written: a node's index is at least
// its place in the branch, and both rise, so what is written never lies ahead
// of what is still to be read, and no two threads share a byte.  The (page, row)
// of 64 moves at a time come from shared memory.  Bound by the chain of cold
// loads (branch, table, row) and the launch; the rows of a batch are a few MB:
// branches of up to 13 nodes of 250 sequences 3.8 us in a graph (floor 0.9),
// small trees' 2.5.

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kChunk = 64;  // moves looked up at a time
constexpr int kBatch = 8;   // rows in flight a thread
constexpr int kStatusInvalid = 1;  // MJ_ERR_INVALID_ARG

__global__ void __launch_bounds__(kMaxThreads) tree_commit_kernel(const CommitDev a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  // of each move: destination and source slot, and their pages (-1: not moved)
  __shared__ int4 moves[kChunk];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int shift = a.page_shift, row_mask = (1 << shift) - 1;
  const int32_t* const path = a.accepted + static_cast<int64_t>(b) * a.max_accept;
  // one round of loads: the branch beside the numbers that say how much of it counts
  const int mine = tid < a.max_accept ? path[tid] : 0;
  const int ahead = tid > 0 && tid < a.max_accept ? path[tid - 1] : -1;
  const int L = a.seq_lens[b], count = a.num_accepted[b];
  int nodes = a.tree_lens ? a.tree_lens[b] : a.q_len;
  nodes = nodes < 0 ? 0 : (nodes > a.q_len ? a.q_len : nodes);
  int bad = L < 0 || L > a.max_len || count < 0 || count > a.max_accept;
  if (!bad) {
    nodes = nodes > L ? L : nodes;
    if (tid < count) bad |= mine < 0 || mine >= nodes || mine <= ahead;
    for (int i = tid + blockDim.x; i < count; i += blockDim.x) {
      const int m = path[i];
      bad |= m < 0 || m >= nodes || m <= path[i - 1];
    }
  }
  bad = __syncthreads_or(bad);  // also: every thread has read the length
  if (bad) {
    if (tid == 0) {
      if (a.status) atomicExch(a.status, kStatusInvalid);
      a.new_lens[b] = L;
    }
    return;
  }
  const int ctx = L - nodes;
  if (tid == 0) a.new_lens[b] = ctx + count;

  const int chunks = a.row_bytes / 16;
  const int kv_cols = 2 * a.h_k * chunks;
  const int scale_cols = a.ks ? 2 * a.h_k : 0;
  // one plane of positions for all heads is moved once
  const int pos_cols = a.key_pos ? (a.kp_head == 0 ? 1 : a.h_k) : 0;
  const int cols = kv_cols + scale_cols + pos_cols;

  for (int c0 = 0; c0 < count; c0 += kChunk) {
    const int n = count - c0 < kChunk ? count - c0 : kChunk;
    if (tid < n) {
      const int to = ctx + c0 + tid, of = ctx + (c0 == 0 ? mine : path[c0 + tid]);
      int pt = -1, pf = -1;
      if (to != of) {
        const int64_t row = static_cast<int64_t>(b) * a.max_blocks;
        pt = a.block_table[row + (to >> shift)];
        pf = a.block_table[row + (of >> shift)];
        if (pt < 0 || pt >= a.num_pages || pf < 0 || pf >= a.num_pages) {
          if (a.status) atomicExch(a.status, kStatusInvalid);
          pt = -1;
        }
      }
      moves[tid] = make_int4(to, of, pt, pf);
    }
    __syncthreads();
    for (int c = tid; c < cols; c += blockDim.x) {
      if (c < kv_cols) {
        const bool v = c >= a.h_k * chunks;
        const int g = (v ? c - a.h_k * chunks : c) / chunks, piece = c % chunks;
        uint8_t* const base = (v ? a.v + g * a.v_head : a.k + g * a.k_head) + piece * 16;
        const int64_t page = v ? a.v_page : a.k_page, row = v ? a.v_row : a.k_row;
        for (int i0 = 0; i0 < n; i0 += kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= n) continue;
            const int4 m = moves[i0 + i];
            if (m.z >= 0) x[i] = *reinterpret_cast<const uint4*>(base + m.w * page + (m.y & row_mask) * row);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= n) continue;
            const int4 m = moves[i0 + i];
            if (m.z >= 0) *reinterpret_cast<uint4*>(base + m.z * page + (m.x & row_mask) * row) = x[i];
          }
        }
      } else if (c < kv_cols + scale_cols) {
        const int s = c - kv_cols;
        const bool v = s >= a.h_k;
        const int g = v ? s - a.h_k : s;
        uint8_t* const base = v ? a.vs + g * a.vs_head : a.ks + g * a.ks_head;
        const int64_t page = v ? a.vs_page : a.ks_page;
        for (int i = 0; i < n; ++i) {
          const int4 m = moves[i];
          if (m.z >= 0)
            *reinterpret_cast<uint2*>(base + m.z * page + (m.x & row_mask) * 8) =
                *reinterpret_cast<const uint2*>(base + m.w * page + (m.y & row_mask) * 8);
        }
      } else {
        int32_t* const plane = a.key_pos + b * a.kp_seq + (c - kv_cols - scale_cols) * a.kp_head;
        for (int i = 0; i < n; ++i) {
          const int4 m = moves[i];
          if (m.z >= 0) plane[m.x] = plane[m.y];
        }
      }
    }
    __syncthreads();  // moves are read
  }
}

}  // namespace

cudaError_t launch_tree_commit(const CommitDev& a, cudaStream_t stream) {
  const int cols = 2 * a.h_k * (a.row_bytes / 16) + (a.ks ? 2 * a.h_k : 0) + (a.key_pos ? a.h_k : 0);
  int threads = (cols + 31) / 32 * 32;
  threads = threads < kChunk ? kChunk : (threads > kMaxThreads ? kMaxThreads : threads);
  return launch_pdl(tree_commit_kernel, dim3(static_cast<unsigned>(a.num_seqs), 1, 1),
                    dim3(static_cast<unsigned>(threads), 1, 1), 0, stream, a);
}

}  // namespace mj
