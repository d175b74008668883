// The work list of attention over whole prompts (see mj_prompt_plan).
//
// A sequence's packed rows go in row tiles of 256; a row tile's keys are those
// its tokens see between them, in tiles of 128.  With T tiles in all and S CTAs
// a head (152 / h_k), a row tile of more than chunk = max(4, ceil(T / S)) tiles
// is cut into equal pieces of at most that many: a long prompt has row tiles
// enough and is not cut, a few rows before a long cache are.  At most S row
// tiles are longer than T / S, and their pieces are at most T / chunk plus one
// each, so 2 S parts hold all partial results whatever the lengths.
//
// Items are ordered by their cost in tiles, longest first (up to 8192; beyond that order
// hardly matters): the attention's CTAs take them in turns, forth and back.  (A
// list that gives each unit to the CTA with the least so far ended a step of a
// long chunk among decode tokens 1 % sooner and took 130 us to make.)
//
// One CTA of 1024 threads, latency-bound: a prefix sum over the sequences, one
// pass over the row tiles for T, one with prefix sums over batches of 1024 row
// tiles that writes the items, and a bitonic sort of (length, index) keys.

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "prompt.cuh"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kStatusInvalid = 1;   // MJ_ERR_INVALID_ARG
constexpr int kStatusCapacity = 3;  // MJ_ERR_CAPACITY

__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// Inclusive prefix sum over the block; *total receives the block's sum.
__device__ __forceinline__ int block_scan(int v, int* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inc = warp_scan(v, lane);
  __syncthreads();  // red is free
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  if (warp == 0) red[lane] = warp_scan(red[lane], lane);
  __syncthreads();
  *total = red[kWarps - 1];
  return inc + (warp > 0 ? red[warp - 1] : 0);
}

__global__ void __launch_bounds__(kThreads) prompt_plan_kernel(const PromptPlanDev a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  uint64_t* const keys = reinterpret_cast<uint64_t*>(smem);                  // [kPromptSortMax]
  int32_t* const off = reinterpret_cast<int32_t*>(keys + kPromptSortMax);    // [num_seqs + 1] row tiles before b
  __shared__ int red[kWarps];
  __shared__ unsigned long long sum;
  __shared__ int bad, bad_cu;
  const int tid = threadIdx.x;
  if (tid == 0) {
    sum = 0;
    bad = bad_cu = 0;
  }
  __syncthreads();

  // a sequence's tokens and length (a length out of range is clamped; tokens
  // out of order or range leave the whole list empty)
  auto shape = [&](int b, int* tok0, int* n, int* len) {
    const int L = a.seq_lens[b];
    *tok0 = a.cu_tokens[b];
    *n = a.cu_tokens[b + 1] - *tok0;
    *len = L < 0 ? 0 : (L > a.max_len ? static_cast<int>(a.max_len) : L);
  };

  int base = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += kThreads) {
    const int b = b0 + tid;
    int tiles = 0;
    if (b < a.num_seqs) {
      const int c0 = a.cu_tokens[b], c1 = a.cu_tokens[b + 1], L = a.seq_lens[b];
      if (c0 < 0 || c1 < c0 || c1 > a.num_tokens)
        bad_cu = 1;
      else
        tiles = ((c1 - c0) * a.h_r + kPromptRows - 1) / kPromptRows;
      if (L < 0 || L > a.max_len) bad = 1;
    }
    int total;
    const int inc = block_scan(tiles, red, &total);
    if (b < a.num_seqs) off[b + 1] = base + inc;
    base += total;
  }
  if (tid == 0) off[0] = 0;
  __syncthreads();
  const int row_tiles = base;
  const bool fits = bad_cu == 0 && row_tiles <= a.items_cap - 2 * a.slots;

  // the item that holds the whole of row tile x
  auto whole = [&](int x) {
    int lo = 0, hi = a.num_seqs - 1;  // the last b with off[b] <= x (empty sequences before it share its offset)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    PromptItem it;
    it.b = lo;
    shape(lo, &it.tok0, &it.n_tok, &it.len);
    it.row0 = (x - off[lo]) * kPromptRows;
    it.part = -1;
    prompt_tiles(it.len, it.n_tok, a.h_r, it.row0, kPromptRows, a.causal, a.window, &it.t0, &it.t1);
    return it;
  };

  if (fits) {
    unsigned long long mine = 0;
    for (int x = tid; x < row_tiles; x += kThreads) {
      const PromptItem it = whole(x);
      mine += it.t1 - it.t0;
    }
    atomicAdd(&sum, mine);  // whole numbers: any order gives the same sum
  }
  __syncthreads();
  long long chunk = (static_cast<long long>(sum) + a.slots - 1) / a.slots;
  if (chunk < kPromptMinChunk) chunk = kPromptMinChunk;

  int n_items = 0, n_parts = 0, n_merges = 0;
  if (fits) {
    for (int x0 = 0; x0 < row_tiles; x0 += kThreads) {
      const int x = x0 + tid;
      PromptItem it;
      int pieces = 0, kt = 0;
      if (x < row_tiles) {
        it = whole(x);
        kt = it.t1 - it.t0;
        pieces = kt <= chunk ? 1 : static_cast<int>((kt + chunk - 1) / chunk);
        if (pieces > a.max_splits) pieces = a.max_splits;
      }
      const int cut = pieces > 1;
      int t_items, t_parts, t_merges;
      const int i_end = block_scan(pieces, red, &t_items);
      const int p_end = block_scan(cut ? pieces : 0, red, &t_parts);
      const int m_end = block_scan(cut, red, &t_merges);
      if (pieces > 0) {
        const int at = n_items + i_end - pieces;
        const int p0 = n_parts + p_end - pieces;
        if (cut) {
          PromptMerge m;
          m.b = it.b;
          m.row0 = it.row0;
          m.part0 = p0;
          m.n_parts = pieces;
          m.tok0 = it.tok0;
          m.n_tok = it.n_tok;
          m.pad0 = m.pad1 = 0;
          a.merges[n_merges + m_end - 1] = m;
        }
        const int t0 = it.t0;
        for (int s = 0; s < pieces; ++s) {
          it.t0 = t0 + static_cast<int>(static_cast<long long>(kt) * s / pieces);
          it.t1 = t0 + static_cast<int>(static_cast<long long>(kt) * (s + 1) / pieces);
          it.part = cut ? p0 + s : -1;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            int g0, g1;
            prompt_tiles(it.len, it.n_tok, a.h_r, it.row0 + w * kPromptRows / 2, kPromptRows / 2, a.causal, a.window, &g0, &g1);
            it.g0[w] = max(g0, it.t0);
            it.g1[w] = max(min(g1, it.t1), it.g0[w]);
          }
          if (it.n_tok * a.h_r - it.row0 <= kPromptRows / 2 && it.t1 - it.t0 >= 2) {
            it.g0[0] = it.g0[1] = it.t0;
            it.g1[0] = it.t1;
            it.g1[1] = -1;
          }
          a.scratch[at + s] = it;
          // (a tile that the row groups take in turn costs about 5/8 of one they share)
          const int cost = (it.t1 - it.t0) * (it.g1[1] < 0 ? 5 : 8);
          if (at + s < kPromptSortMax)
            keys[at + s] = (static_cast<uint64_t>(0x7FFFFFFF - cost) << 32) | static_cast<uint32_t>(at + s);
        }
      }
      n_items += t_items;
      n_parts += t_parts;
      n_merges += t_merges;
    }
  }
  const bool sorted = n_items <= kPromptSortMax;
  int n = 1;
  while (n < n_items) n <<= 1;
  if (sorted)
    for (int i = n_items + tid; i < n; i += kThreads) keys[i] = ~0ull;
  __syncthreads();  // also: the scratch items are written (this block reads them back)
  if (sorted) {
    for (int k = 2; k <= n; k <<= 1) {
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = tid; i < n; i += kThreads) {
          const int q = i ^ j;
          if (q > i) {
            const uint64_t x = keys[i], y = keys[q];
            if ((x > y) == ((i & k) == 0)) {
              keys[i] = y;
              keys[q] = x;
            }
          }
        }
        __syncthreads();
      }
    }
  }
  for (int i = tid; i < n_items; i += kThreads) a.items[i] = a.scratch[sorted ? static_cast<uint32_t>(keys[i]) : i];
  if (tid == 0) {
    a.head->n_items = n_items;
    a.head->n_merges = n_merges;
    a.head->n_parts = n_parts;
    a.head->chunk = static_cast<int32_t>(chunk);
    a.head->num_seqs = a.num_seqs;
    a.head->num_tokens = a.num_tokens;
    a.head->h_k = a.h_k;
    a.head->h_r = a.h_r;
    a.head->causal = a.causal;
    a.head->window = a.window;
    a.head->max_splits = a.max_splits;
    a.head->page_size = a.page_size;
    a.head->max_blocks = a.max_blocks;
    a.head->magic = kPromptMagic;
    if (a.status && (bad || bad_cu)) atomicExch(a.status, kStatusInvalid);
    else if (a.status && !fits) atomicExch(a.status, kStatusCapacity);
  }
}

}  // namespace

cudaError_t launch_prompt_plan(const PromptPlanDev& a, cudaStream_t stream) {
  const size_t smem = kPromptSortMax * 8 + (static_cast<size_t>(a.num_seqs) + 1) * 4;
  const cudaError_t e =
      cudaFuncSetAttribute(prompt_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_plan_kernel, dim3(1, 1, 1), dim3(kThreads, 1, 1), smem, stream, a);
}

}  // namespace mj
