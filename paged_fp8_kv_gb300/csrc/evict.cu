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
// from three histogram passes over the key's digits (11, 11 and 10 bits, most
// significant first); slots equal to the threshold are kept in slot order
// until `new` is reached, by counting.
//
// One cluster of 1 to 16 CTAs serves a (b, g), its slots cut into that many
// runs: a CTA reads its run once, keeps the keys in shared memory for the
// later passes, and the cluster's histograms and counts are summed over
// distributed shared memory.  The move lists meet in the workspace (L2) and
// the cluster's CTAs then copy the rows between them: eight lanes a row of 128
// bytes, K and V, two moves in flight a lane.  One launch; long caches of few
// heads get their CTAs from the cluster, short ones of many heads from the
// grid, four 512-thread CTAs an SM.

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 16;
constexpr int kStatusInvalidArg = 1;  // MJ_ERR_INVALID_ARG

__device__ __forceinline__ uint32_t rank_key(float w, bool held) {
  if (held) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Address of this CTA's shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Barrier over the cluster's threads; orders their shared and global accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int warp_sum_before(int v, int lane, int& total) {
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  total = __shfl_sync(0xffffffffu, x, 31);
  return x - v;
}

struct Shared {
  int hist[2][kBins];
  int warp_sums[kWarps];
  int totals[4];  // holes, movers of this CTA
  uint32_t bin;
  int need;
  int bin_count;
};

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictDev a, int cluster, int key_cap) {
  // a programmatic dependent: no global access before the grid ahead is done
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ __align__(16) Shared s;
  extern __shared__ uint32_t keys[];  // [key_cap] of this CTA's run
  const int bg = blockIdx.x / cluster, rank = blockIdx.x - bg * cluster;
  const int b = bg / a.h_k, g = bg - b * a.h_k;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t max_len = static_cast<int64_t>(a.max_blocks) * a.page_size;
  int L = a.seq_lens[b];
  if (L < 0 || L > max_len) {
    if (tid == 0 && a.status) atomicExch(a.status, kStatusInvalidArg);
    L = L < 0 ? 0 : static_cast<int>(max_len);
  }
  const int fresh = L < a.budget ? L : a.budget;  // the new length
  const int64_t off = b * a.acc_seq + g * a.acc_head;
  const float* const acc = a.acc + off;
  const int32_t* const pos = a.key_pos ? a.key_pos + off : nullptr;
  const bool copy_acc = a.acc_out != a.acc, copy_pos = pos && a.key_pos_out != a.key_pos;
  if (g == 0 && rank == 0 && tid == 0) a.new_lens[b] = fresh;
  // this CTA's run of slots, whole rows of 32
  const int per_cta = (((L + cluster - 1) / cluster) + 31) / 32 * 32;
  const int begin = rank * per_cta < L ? rank * per_cta : L;
  const int n = L - begin < per_cta ? L - begin : per_cta;

  if (L <= a.budget) {  // nothing leaves (uniform over the cluster)
    for (int i = tid; i < n; i += kThreads) {
      const int j = begin + i;
      if (copy_acc) a.acc_out[off + j] = acc[j];
      if (copy_pos) a.key_pos_out[off + j] = pos[j];
    }
    return;
  }

  const int64_t end = (pos ? a.next_pos[b] : L) - static_cast<int64_t>(a.keep_last);
  auto make_key = [&](int j) {
    const int p = pos ? pos[j] : j;
    return rank_key(acc[j], p < a.keep_first || p >= end);
  };
  const bool cached = n <= key_cap;
  auto key_of = [&](int i) { return cached ? keys[i] : make_key(begin + i); };

  // ---- the threshold: the fresh-th largest key.  need: how many keys of the
  // prefix found so far are kept
  uint32_t prefix = 0;
  int need = fresh;
  for (int i = tid; i < 2 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    int* const hist = s.hist[pass & 1];
    if (pass == 2) {  // every CTA has read pass 0's counts (it passed pass 1's barrier)
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
    }
    if (pass == 0) {
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = make_key(begin + i);
        if (cached) keys[i] = k;
        atomicAdd(&hist[k >> 21], 1);
      }
    } else {
      const int above = pass == 1 ? 21 : 10;
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t k = key_of(i);
        if ((k >> above) == (prefix >> above)) atomicAdd(&hist[(k >> shift) & digits], 1);
      }
    }
    cluster_sync();
    // every CTA sums the cluster's counts: thread t bins 4 t' .. 4 t' + 3 from
    // the top, so that a prefix sum over the threads counts the larger keys
    const int q = kThreads - 1 - tid;
    int4 c = make_int4(0, 0, 0, 0);
    const uint32_t mine = ptx::smem_u32(hist + 4 * q);
    for (int r = 0; r < cluster; ++r) {
      const int4 v = ld_cluster_v4(map_rank(mine, r));
      c.x += v.x;
      c.y += v.y;
      c.z += v.z;
      c.w += v.w;
    }
    const int sum = c.x + c.y + c.z + c.w;
    int total;
    int before = warp_sum_before(sum, lane, total);
    if (lane == 31) s.warp_sums[warp] = total;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += s.warp_sums[w];
    if (before < need && need <= before + sum) {  // one thread: the threshold's digit is among its bins
      const int cnt[4] = {c.w, c.z, c.y, c.x};
      int left = need - before, e = 0;
      while (e < 3 && cnt[e] < left) left -= cnt[e++];
      s.bin = 4 * q + 3 - e;
      s.need = left;
      s.bin_count = cnt[e];
    }
    __syncthreads();
    prefix |= s.bin << shift;
    need = s.need;
  }
  static_assert(kThreads * 4 == kBins, "four bins a thread");
  // keys above the threshold are kept, and of the ties (equal to it) the
  // first `need`; those of lower runs are in the last histogram
  const bool all_ties = s.bin_count == need;
  int tie_rank = 0;  // ties before this warp's rows
  const int rows = (n + 31) / 32;
  const int rows_per_warp = (rows + kWarps - 1) / kWarps;
  const int row0 = warp * rows_per_warp < rows ? warp * rows_per_warp : rows;
  const int row1 = row0 + rows_per_warp < rows ? row0 + rows_per_warp : rows;
  if (!all_ties) {
    for (int r = 0; r < rank; ++r) tie_rank += ld_cluster(map_rank(ptx::smem_u32(&s.hist[0][prefix & 1023u]), r));
    int mine = 0;
    for (int r = row0; r < row1; ++r) {
      const int i = r * 32 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, i < n && key_of(i) == prefix));
    }
    __syncthreads();
    if (lane == 0) s.warp_sums[warp] = mine;
    __syncthreads();
    for (int w = 0; w < warp; ++w) tie_rank += s.warp_sums[w];
  }
  // keep flags of a row of 32 slots, as ballots: holes and movers
  auto flags = [&](int r, int& ties, uint32_t& holes, uint32_t& movers) {
    const int i = r * 32 + lane;
    const bool in = i < n;
    const uint32_t k = in ? key_of(i) : 0u;
    bool keep = in && k >= prefix;
    if (!all_ties) {
      const uint32_t tie = __ballot_sync(0xffffffffu, in && k == prefix);
      if (in && k == prefix) keep = ties + __popc(tie & ((1u << lane) - 1u)) < need;
      ties += __popc(tie);
    }
    const int j = begin + i;
    holes = __ballot_sync(0xffffffffu, in && j < fresh && !keep);
    movers = __ballot_sync(0xffffffffu, keep && j >= fresh);
  };
  int n_holes = 0, n_movers = 0, ties = tie_rank;
  for (int r = row0; r < row1; ++r) {
    uint32_t h, m;
    flags(r, ties, h, m);
    n_holes += __popc(h);
    n_movers += __popc(m);
  }
  __syncthreads();
  if (lane == 0) s.warp_sums[warp] = n_holes | (n_movers << 16);
  __syncthreads();
  int hole_at = 0, mover_at = 0, cta_holes = 0, cta_movers = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int v = s.warp_sums[w], h = v & 0xFFFF, m = v >> 16;
    if (w < warp) {
      hole_at += h;
      mover_at += m;
    }
    cta_holes += h;
    cta_movers += m;
  }
  if (tid == 0) {
    s.totals[0] = cta_holes;
    s.totals[1] = cta_movers;
  }
  cluster_sync();
  int moves_n = 0;
  for (int r = 0; r < cluster; ++r) {
    const int h = ld_cluster(map_rank(ptx::smem_u32(&s.totals[0]), r));
    const int m = ld_cluster(map_rank(ptx::smem_u32(&s.totals[1]), r));
    if (r < rank) {
      hole_at += h;
      mover_at += m;
    }
    moves_n += h;
  }
  int32_t* const moves = a.moves + static_cast<int64_t>(bg) * a.moves_cap * 2;  // [dst | src]
  ties = tie_rank;
  const uint32_t below = (1u << lane) - 1u;
  for (int r = row0; r < row1; ++r) {
    uint32_t h, m;
    flags(r, ties, h, m);
    const int j = begin + r * 32 + lane;
    if ((h >> lane) & 1u) moves[hole_at + __popc(h & below)] = j;
    if ((m >> lane) & 1u) moves[a.moves_cap + mover_at + __popc(m & below)] = j;
    hole_at += __popc(h);
    mover_at += __popc(m);
    if (j < fresh && j < begin + n && !((h >> lane) & 1u)) {
      if (copy_acc) a.acc_out[off + j] = acc[j];
      if (copy_pos) a.key_pos_out[off + j] = pos[j];
    }
  }
  cluster_sync();  // the lists are whole (and no CTA's shared memory is read any more)

  // ---- the moves: eight lanes one, CTAs of the cluster in turn
  const int32_t* const table = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
  const int vecs = a.row_bytes / 16;  // 8, 6 or 4 of the eight lanes
  const int lane8 = tid & 7;
  constexpr int kUnroll = 2;
  const int step = cluster * (kThreads / 8);
  for (int i0 = rank * (kThreads / 8) + (tid >> 3); i0 < moves_n; i0 += step * kUnroll) {
    int dst[kUnroll], src[kUnroll], dp[kUnroll], sp[kUnroll];
    bool ok[kUnroll];
    uint4 kv[kUnroll], vv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * step;
      ok[u] = i < moves_n;
      dst[u] = ok[u] ? moves[i] : 0;
      src[u] = ok[u] ? moves[a.moves_cap + i] : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      dp[u] = table[dst[u] / a.page_size];
      sp[u] = table[src[u] / a.page_size];
      if (ok[u] && lane8 == 0) {
        a.acc_out[off + dst[u]] = acc[src[u]];
        if (pos) a.key_pos_out[off + dst[u]] = pos[src[u]];
      }
      if (ok[u] && (dp[u] < 0 || dp[u] >= a.num_pages || sp[u] < 0 || sp[u] >= a.num_pages)) {
        if (lane8 == 0 && a.status) atomicExch(a.status, kStatusInvalidArg);
        ok[u] = false;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (ok[u] && lane8 < vecs) {
        const int sr = src[u] % a.page_size;
        kv[u] = *reinterpret_cast<const uint4*>(a.k + sp[u] * a.k_page + sr * a.k_row + g * a.k_head + lane8 * 16);
        vv[u] = *reinterpret_cast<const uint4*>(a.v + sp[u] * a.v_page + sr * a.v_row + g * a.v_head + lane8 * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int dr = dst[u] % a.page_size;
      if (ok[u] && lane8 < vecs) {
        *reinterpret_cast<uint4*>(a.k + dp[u] * a.k_page + dr * a.k_row + g * a.k_head + lane8 * 16) = kv[u];
        *reinterpret_cast<uint4*>(a.v + dp[u] * a.v_page + dr * a.v_row + g * a.v_head + lane8 * 16) = vv[u];
      }
      if (a.ks && ok[u] && lane8 < 2) {  // nvfp4: the row's eight scales, K on lane 0, V on lane 1
        const int sr = src[u] % a.page_size;
        uint8_t* const base = lane8 == 0 ? a.ks : a.vs;
        const int64_t page = lane8 == 0 ? a.ks_page : a.vs_page, head = lane8 == 0 ? a.ks_head : a.vs_head;
        *reinterpret_cast<uint2*>(base + dp[u] * page + g * head + dr * 8) =
            *reinterpret_cast<const uint2*>(base + sp[u] * page + g * head + sr * 8);
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictDev& a, cudaStream_t stream) {
  const int64_t groups = static_cast<int64_t>(a.num_seqs) * a.h_k;
  const int64_t max_len = static_cast<int64_t>(a.max_blocks) * a.page_size;
  // CTAs a group: enough to fill about one wave (four an SM), each with 2048
  // slots or more
  int cluster = 1;
  while (cluster < kMaxCluster && groups * cluster * 2 <= 152 * 4 && max_len / (cluster * 2) >= 2048) cluster *= 2;
  // keys in shared memory when a run fits beside the histograms (else they
  // are made again from the weights, in L2, by every pass)
  const int64_t run = (max_len + cluster - 1) / cluster + 32;
  const int key_cap = run <= 49152 ? static_cast<int>(run) : 0;
  const size_t smem = static_cast<size_t>(key_cap) * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 49152 * 4);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel, a, cluster, key_cap);
}

}  // namespace mj
