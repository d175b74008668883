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
// from histogram passes of 11 bits, most significant first, over the keys'
// offsets from the smallest one: weights lie within a few binades, so without
// the offset the first pass would count nearly all of them in a few dozen
// bins, whose shared-memory atomics then wait on one another.  Slots equal to
// the threshold are kept in slot order until `new` is reached, by counting.
//
// Kernel 1: one cluster of 1 to 8 CTAs serves a (b, g), its slots cut into that
// many runs.  A CTA reads its run's weights and positions once, keeps the keys
// in shared memory for the later passes, and the cluster's histograms and
// counts are summed over distributed shared memory.  It writes the kept slots'
// weights, and the move lists with their pages looked up.  Long caches of few
// heads get their CTAs from the cluster, short ones of many heads from the
// grid, two CTAs an SM; when those do not all fit, the longest sequences start
// first, so that the last ones to run are short (64 sequences of 8 heads and
// 512 to 8192 keys, cut to 2048: the call 82 us, in batch order 86).
// The host knows the block table's width, not the lengths, and sizes the key
// buffer by the longest run the table allows: one CTA an SM from about 24000
// slots a CTA on, and past kMaxKeys no buffer, the keys made again from the
// weights by every pass (the same batch under tables of 8192 and 20000 slots
// 86 us, of 32768 95, of 49152 to 131072 105 to 109).
// Bound: on that batch, instructions (57 % of the issue slots while a CTA is
// there; each of its threads pays for the bins and scans whatever its keys)
// and the second wave of CTAs: 33 us, with 256 threads 50, with 1024 43; on a
// few long caches, the chain of cluster barriers between the passes (29 us).
// Kernel 2 moves the rows: the moves of all groups are one list, cut evenly
// over the CTAs (a group's share differs by its length and its luck), sixteen
// lanes a move, two in flight a thread (the same batch, before the order by
// length: 86 us; one in flight 95, four 90, eight 87).  Bound: DRAM, at rows of
// 64 to 128 bytes in random places (that batch: 221 MB in 48 us, 4.6 TB/s);
// more of them in flight, or other cache hints, are no faster.

#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kThreads = 256;     // of the move kernel
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxKeys = 49152;  // keys of a run in shared memory
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
template <int N>
__device__ __forceinline__ void ld_cluster_n(uint32_t addr, int* v) {
  static_assert(N == 2 || N == 4, "vector width");
  if constexpr (N == 4) {
    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
  } else {
    asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
  }
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

// Sum of the warps' values before `warp`, and of all N (N <= 32).
template <int N>
__device__ __forceinline__ int warps_before(const int* sums, int warp, int lane, int& total) {
  const int before = warp_sum_before(lane < N ? sums[lane] : 0, lane, total);
  return __shfl_sync(0xffffffffu, before, warp);
}

struct Shared {
  int hist[2][kBins];
  int warp_sums[32];
  int warp_holes[32];
  int totals[4];  // holes, movers of this CTA
  uint32_t range[2];  // smallest key, largest unprotected key of this CTA
  uint32_t bin;
  int need;
  int bin_count;
};

// T threads: 512, two CTAs an SM, or 1024 when the groups do not fill the GPU
template <int T>
__global__ void __launch_bounds__(T, 1024 / T)
    evict_select_kernel(const EvictDev a, int cluster, int key_cap, bool by_length) {
  // a programmatic dependent: no global access before the grid ahead is done
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  constexpr int kSelWarps = T / 32;
  constexpr int kPer = kBins / T;  // bins a thread
  __shared__ __align__(16) Shared s;
  extern __shared__ uint32_t keys[];  // [key_cap] of this CTA's run
  int bg = blockIdx.x / cluster;
  const int rank = blockIdx.x - bg * cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t max_len = static_cast<int64_t>(a.max_blocks) * a.page_size;
  int b = bg / a.h_k;
  const int g = bg - b * a.h_k;
  if (by_length) {  // the b-th longest sequence (at most T of them); ties by index
    int* const lens = s.hist[0];
    if (tid < a.num_seqs) lens[tid] = a.seq_lens[tid];
    __syncthreads();
    if (tid < a.num_seqs) {
      int rank_of = 0;
      for (int j = 0; j < a.num_seqs; ++j) rank_of += lens[j] > lens[tid] || (lens[j] == lens[tid] && j < tid);
      if (rank_of == b) s.need = tid;
    }
    __syncthreads();
    b = s.need;
    bg = b * a.h_k + g;
    __syncthreads();
  }
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
    if (rank == 0 && tid == 0) a.counts[bg] = 0;
    for (int i = tid; i < n; i += T) {
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
  // 16-byte accesses where the planes allow them (runs start at multiples of 32)
  const bool wide =
      ((reinterpret_cast<uintptr_t>(acc) | reinterpret_cast<uintptr_t>(a.acc_out + off) |
        (pos ? reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(a.key_pos_out + off) : 0u)) & 15u) == 0;
  auto key_of = [&](int i) { return cached ? keys[i] : make_key(begin + i); };

  // ---- the one read of the weights (and positions): keys and their range,
  // and the copy of every slot below the new length (the holes among them are
  // written again by the moves)
  uint32_t k_min = 0xFFFFFFFFu, k_max = 0u;
  {
    auto take = [&](int i, float w, int p) {
      const uint32_t k = rank_key(w, p < a.keep_first || p >= end);
      if (cached) keys[i] = k;
      k_min = k < k_min ? k : k_min;
      k_max = k > k_max && k != 0xFFFFFFFFu ? k : k_max;
    };
    const int quads = wide ? n / 4 : 0;
    constexpr int kBatch = 2;  // loads in flight a thread, before any of their stores
    for (int v0 = tid; v0 < quads; v0 += kBatch * T) {
      float4 w[kBatch];
      int4 p[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int v = v0 + u * T, j = begin + 4 * v;
        if (v < quads) w[u] = *reinterpret_cast<const float4*>(acc + j);
        p[u] = pos && v < quads ? *reinterpret_cast<const int4*>(pos + j) : make_int4(j, j + 1, j + 2, j + 3);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int v = v0 + u * T, j = begin + 4 * v;
        if (v >= quads) break;
        take(4 * v, w[u].x, p[u].x);
        take(4 * v + 1, w[u].y, p[u].y);
        take(4 * v + 2, w[u].z, p[u].z);
        take(4 * v + 3, w[u].w, p[u].w);
        if (j + 3 < fresh) {
          if (copy_acc) *reinterpret_cast<float4*>(a.acc_out + off + j) = w[u];
          if (copy_pos) *reinterpret_cast<int4*>(a.key_pos_out + off + j) = p[u];
        } else {
          const float ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          const int ps[4] = {p[u].x, p[u].y, p[u].z, p[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (j + e >= fresh) break;
            if (copy_acc) a.acc_out[off + j + e] = ws[e];
            if (copy_pos) a.key_pos_out[off + j + e] = ps[e];
          }
        }
      }
    }
    for (int i = 4 * quads + tid; i < n; i += T) {
      const int j = begin + i;
      const float w = acc[j];
      const int p = pos ? pos[j] : j;
      take(i, w, p);
      if (j < fresh) {
        if (copy_acc) a.acc_out[off + j] = w;
        if (copy_pos) a.key_pos_out[off + j] = p;
      }
    }
  }
  for (int i = tid; i < 2 * kBins; i += T) (&s.hist[0][0])[i] = 0;
  if (tid < 2) s.range[tid] = tid == 0 ? 0xFFFFFFFFu : 0u;
  __syncthreads();
  k_min = __reduce_min_sync(0xffffffffu, k_min);
  k_max = __reduce_max_sync(0xffffffffu, k_max);
  if (lane == 0) {
    atomicMin(&s.range[0], k_min);
    atomicMax(&s.range[1], k_max);
  }
  if (cluster > 1) {
    cluster_sync();
    const uint32_t r = lane < cluster ? lane : rank;
    k_min = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(ld_cluster(map_rank(ptx::smem_u32(&s.range[0]), r))));
    k_max = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(ld_cluster(map_rank(ptx::smem_u32(&s.range[1]), r))));
  } else {
    __syncthreads();
    k_min = s.range[0];
    k_max = s.range[1];
  }
  // protected slots rank just above the largest other key; all as offsets
  // (all protected: one value)
  const uint32_t k_top = k_max >= k_min ? k_max + 1 : k_min;
  auto digits_of = [&](uint32_t k) { return (k < k_top ? k : k_top) - k_min; };
  const int bits = 32 - __clz(k_top - k_min);  // 0: all keys equal
  const int passes = bits <= 11 ? 1 : (bits <= 22 ? 2 : 3);

  // ---- the threshold: the fresh-th largest.  need: how many keys of the
  // prefix found so far are kept
  uint32_t prefix = 0;
  int need = fresh;
  int left_bits = bits, last_pass = 0;
  for (int pass = 0; pass < passes; ++pass) {
    const int width = left_bits < 11 ? left_bits : 11, above = left_bits;
    left_bits -= width;
    const int shift = left_bits;
    int* const hist = s.hist[pass & 1];
    if (pass == 2) {  // every CTA has read pass 0's counts (it passed pass 1's barrier)
      for (int i = tid; i < kBins; i += T) hist[i] = 0;
      __syncthreads();
    }
    const uint32_t mask = (1u << width) - 1u;
    // (above = 32 only when every bit is left: then all keys match)
#pragma unroll 8
    for (int i = tid; i < n; i += T) {
      const uint32_t k = digits_of(key_of(i));
      if (pass == 0 || (k >> above) == (prefix >> above)) atomicAdd(&hist[(k >> shift) & mask], 1);
    }
    if (cluster > 1)
      cluster_sync();
    else
      __syncthreads();
    // every CTA sums the cluster's counts: thread t a few bins, the highest
    // first, so that a prefix sum over the threads counts the larger keys
    const int q = T - 1 - tid;
    int c[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) c[e] = hist[kPer * q + kPer - 1 - e];
    if (cluster > 1) {
      // (three other CTAs' counts in flight, each CTA going round from its own
      // neighbour: all reading one at a time would queue on that one's SM)
      const uint32_t mine = ptx::smem_u32(hist + kPer * q);
      for (int r0 = 1; r0 < cluster; r0 += 3) {
        int o[3][kPer];
#pragma unroll
        for (int u = 0; u < 3; ++u)
          if (r0 + u < cluster) ld_cluster_n<kPer>(map_rank(mine, (rank + r0 + u) & (cluster - 1)), o[u]);
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          if (r0 + u >= cluster) break;
#pragma unroll
          for (int e = 0; e < kPer; ++e) c[e] += o[u][kPer - 1 - e];
        }
      }
    }
    int sum = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) sum += c[e];
    int total;
    int before = warp_sum_before(sum, lane, total);
    if (lane == 31) s.warp_sums[warp] = total;
    __syncthreads();
    before += warps_before<kSelWarps>(s.warp_sums, warp, lane, total);
    if (before < need && need <= before + sum) {  // one thread: the threshold's digit is among its bins
      int left = need - before;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (left > 0 && left <= c[e]) {
          s.bin = kPer * q + kPer - 1 - e;
          s.need = left;
          s.bin_count = c[e];
        }
        left -= c[e];
      }
    }
    __syncthreads();
    prefix |= s.bin << shift;
    need = s.need;
    last_pass = pass;
    if (s.bin_count == need) break;  // the whole bin is kept: the lower digits do not matter
  }
  const int* const last_hist = s.hist[last_pass & 1];
  const uint32_t last_bin = s.bin;
  // keys above the threshold are kept, and of the ties (equal to it) the
  // first `need`; those of lower runs are in the last histogram
  const bool all_ties = s.bin_count == need;
  int tie_rank = 0;  // ties before this warp's rows
  const int rows = (n + 31) / 32;
  const int rows_per_warp = (rows + kSelWarps - 1) / kSelWarps;
  const int row0 = warp * rows_per_warp < rows ? warp * rows_per_warp : rows;
  const int row1 = row0 + rows_per_warp < rows ? row0 + rows_per_warp : rows;
  if (!all_ties) {
    const int theirs = ld_cluster(map_rank(ptx::smem_u32(last_hist + last_bin), lane < cluster ? lane : rank));
    int all;
    const int before = warp_sum_before(lane < cluster ? theirs : 0, lane, all);
    tie_rank = __shfl_sync(0xffffffffu, before, rank);
    int mine = 0;
    for (int r = row0; r < row1; ++r) {
      const int i = r * 32 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, i < n && digits_of(key_of(i)) == prefix));
    }
    __syncthreads();
    if (lane == 0) s.warp_sums[warp] = mine;
    __syncthreads();
    for (int w = 0; w < warp; ++w) tie_rank += s.warp_sums[w];
  }
  // keep flags of a row of 32 slots (key offsets k), as ballots: holes and movers
  auto flags = [&](int r, uint32_t k, int& ties, uint32_t& holes, uint32_t& movers) {
    const int i = r * 32 + lane;
    const bool in = i < n;
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
  auto row_key = [&](int r) {
    const int i = r * 32 + lane;
    return r < row1 && i < n ? digits_of(key_of(i)) : 0u;
  };
  int n_holes = 0, n_movers = 0, ties = tie_rank;
  constexpr int kRows = 4;  // rows' keys read before any of their flags is stored
  for (int r0 = row0; r0 < row1; r0 += kRows) {
    uint32_t k[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) k[u] = row_key(r0 + u);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = r0 + u;
      if (r >= row1) break;
      uint32_t h, m;
      flags(r, k[u], ties, h, m);
      n_holes += __popc(h);
      n_movers += __popc(m);
      if (cached && lane < 2) keys[r * 32 + lane] = lane == 0 ? h : m;  // over the row's keys, done with
    }
  }
  __syncthreads();
  if (lane == 0) {
    s.warp_holes[warp] = n_holes;
    s.warp_sums[warp] = n_movers;
  }
  __syncthreads();
  int cta_holes, cta_movers;
  int hole_at = warps_before<kSelWarps>(s.warp_holes, warp, lane, cta_holes);
  int mover_at = warps_before<kSelWarps>(s.warp_sums, warp, lane, cta_movers);
  if (tid == 0) {
    s.totals[0] = cta_holes;
    s.totals[1] = cta_movers;
  }
  cluster_sync();
  int moves_n = 0;
  {  // lane r: CTA r's counts
    const uint32_t r = lane < cluster ? lane : rank;
    const int h = ld_cluster(map_rank(ptx::smem_u32(&s.totals[0]), r));
    const int m = ld_cluster(map_rank(ptx::smem_u32(&s.totals[1]), r));
    int all;
    int before = warp_sum_before(lane < cluster ? h : 0, lane, all);
    hole_at += __shfl_sync(0xffffffffu, before, rank);
    moves_n = all;
    before = warp_sum_before(lane < cluster ? m : 0, lane, all);
    mover_at += __shfl_sync(0xffffffffu, before, rank);
  }
  // (slot, page) of every destination, then of every source
  int2* const to = reinterpret_cast<int2*>(a.moves) + static_cast<int64_t>(bg) * a.moves_cap * 2;
  int2* const from = to + a.moves_cap;
  const int32_t* const table = a.block_table + static_cast<int64_t>(b) * a.max_blocks;
  const int page_shift = 31 - __clz(a.page_size);
  ties = tie_rank;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int r = row0; r < row1; ++r) {
    uint32_t h, m;
    if (cached) {
      h = keys[r * 32];
      m = keys[r * 32 + 1];
    } else {
      flags(r, row_key(r), ties, h, m);
    }
    const int j = begin + r * 32 + lane;
    const bool is_hole = (h >> lane) & 1u, is_mover = (m >> lane) & 1u;
    if (is_hole || is_mover) {
      const int2 e = make_int2(j, __ldg(table + (j >> page_shift)));
      if (is_hole) to[hole_at + __popc(h & below)] = e;
      if (is_mover) from[mover_at + __popc(m & below)] = e;
    }
    hole_at += __popc(h);
    mover_at += __popc(m);
  }
  if (rank == 0 && tid == 0) a.counts[bg] = moves_n;
  if (cluster > 1) cluster_sync();  // no CTA leaves while its shared memory may be read
}

__global__ void __launch_bounds__(kThreads, 4) evict_move_kernel(const EvictDev a, int groups) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int s_group;
  __shared__ int64_t s_before;  // moves of the groups before s_group
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // all moves are one list, in group order; this CTA's share of it
  const int per = (groups + kThreads - 1) / kThreads;
  const int g0 = tid * per < groups ? tid * per : groups;
  const int g1 = g0 + per < groups ? g0 + per : groups;
  int64_t mine = 0;
  for (int q = g0; q < g1; ++q) mine += a.counts[q];
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    total += warp_sums[w];
  }
  const int64_t first = total * blockIdx.x / gridDim.x, last = total * (blockIdx.x + 1) / gridDim.x;
  if (first == last) return;  // uniform over the CTA
  if (before <= first && first < before + mine) {  // one thread: the first move's group
    int q = g0;
    while (first >= before + a.counts[q]) before += a.counts[q++];
    s_group = q;
    s_before = before;
  }
  __syncthreads();

  // sixteen lanes a move (eight vectors of its K row and eight of its V row;
  // lane 0 its weight and lane 1 its position), kUnroll of them in flight,
  // every load before any store
  const int l16 = tid & 15, l8 = tid & 7;
  const bool is_v = l16 >= 8;
  const bool has_vec = l8 < a.row_bytes / 16;  // 8, 6 or 4 of the eight
  const int page_mask = a.page_size - 1;       // 16, 32, 64 or 128 rows
  const int64_t page_step = is_v ? a.v_page : a.k_page, row_step = is_v ? a.v_row : a.k_row;
  const bool has_word = l16 == 0 || (l16 == 1 && a.key_pos);
  constexpr int kUnroll = 2;
  constexpr int step = kThreads / 16;
  int64_t at = first, group_begin = s_before;
  for (int bg = s_group; at < last; ++bg) {
    const int count = a.counts[bg];
    const int64_t group_end = group_begin + count;
    const int stop = static_cast<int>((group_end < last ? group_end : last) - group_begin);  // moves of this group
    const int b = bg / a.h_k, g = bg - b * a.h_k;
    const int64_t off = b * a.acc_seq + g * a.acc_head;
    const int2* const to = reinterpret_cast<const int2*>(a.moves) + static_cast<int64_t>(bg) * a.moves_cap * 2;
    const int2* const from = to + a.moves_cap;
    uint8_t* const pool = (is_v ? a.v + g * a.v_head : a.k + g * a.k_head) + l8 * 16;
    const uint32_t* const word_in = l16 == 0 ? reinterpret_cast<const uint32_t*>(a.acc + off)
                                             : reinterpret_cast<const uint32_t*>(a.key_pos + off);
    uint32_t* const word_out = l16 == 0 ? reinterpret_cast<uint32_t*>(a.acc_out + off)
                                        : reinterpret_cast<uint32_t*>(a.key_pos_out + off);
    const int start = static_cast<int>(at - group_begin) + (tid >> 4);
    int2 dst[kUnroll], src[kUnroll];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = i0 + u * step;
        dst[u] = i < stop ? to[i] : make_int2(-1, 0);  // slot -1: no move
        src[u] = i < stop ? from[i] : make_int2(0, 0);
      }
    };
    if (start < stop) fetch(start);
    for (int i0 = start; i0 < stop; i0 += step * kUnroll) {
      uint4 row[kUnroll];
      uint32_t word[kUnroll];
      int2 to_now[kUnroll];
      bool ok[kUnroll];  // both pages are pages
      int sp[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        to_now[u] = dst[u];
        sp[u] = src[u].y;
        ok[u] = static_cast<uint32_t>(dst[u].y) < static_cast<uint32_t>(a.num_pages) &&
                static_cast<uint32_t>(sp[u]) < static_cast<uint32_t>(a.num_pages);
        if (dst[u].x >= 0 && ok[u] && has_vec)
          row[u] = *reinterpret_cast<const uint4*>(pool + sp[u] * page_step + (src[u].x & page_mask) * row_step);
        if (dst[u].x >= 0 && has_word) word[u] = word_in[src[u].x];
      }
      if (a.ks && l8 == 0) {  // nvfp4: the rows' eight scales, K's and V's
        uint8_t* const plane = is_v ? a.vs + g * a.vs_head : a.ks + g * a.ks_head;
        const int64_t step_s = is_v ? a.vs_page : a.ks_page;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (to_now[u].x >= 0 && ok[u])
            *reinterpret_cast<uint2*>(plane + to_now[u].y * step_s + (to_now[u].x & page_mask) * 8) =
                *reinterpret_cast<const uint2*>(plane + sp[u] * step_s + (src[u].x & page_mask) * 8);
      }
      if (i0 + step * kUnroll < stop) fetch(i0 + step * kUnroll);  // the next round's list entries
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (to_now[u].x < 0) continue;
        if (ok[u] && has_vec)
          *reinterpret_cast<uint4*>(pool + to_now[u].y * page_step + (to_now[u].x & page_mask) * row_step) = row[u];
        if (has_word) word_out[to_now[u].x] = word[u];
        if (!ok[u] && l16 == 0 && a.status) atomicExch(a.status, kStatusInvalidArg);
      }
    }
    group_begin = group_end;
    at = group_end < last ? group_end : last;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictDev& a, int sm_count, cudaStream_t stream) {
  const int64_t groups = static_cast<int64_t>(a.num_seqs) * a.h_k;
  const int64_t max_len = static_cast<int64_t>(a.max_blocks) * a.page_size;
  // CTAs a group: enough to fill about one wave (two an SM), each with 2048
  // slots or more
  int cluster = 1;
  while (cluster < kMaxCluster && groups * cluster * 2 <= sm_count * 2 && max_len / (cluster * 2) >= 2048) cluster *= 2;
  // keys in shared memory when a run fits beside the histograms (else they
  // are made again from the weights, in L2, by every pass)
  const int64_t run = (max_len + cluster - 1) / cluster + 32;
  const int key_cap = run <= kMaxKeys ? static_cast<int>(run) : 0;
  // (four caches of two heads and up to 131072 keys: the call 54 us with 512
  // threads, 48 with 1024)
  const bool large = groups * cluster <= sm_count;
  auto kern = large ? evict_select_kernel<1024> : evict_select_kernel<512>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * cluster), 1, 1);
  cfg.blockDim = dim3(large ? 1024 : 512, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(key_cap) * 4;
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
  // more CTAs than one wave: by length, where a thread can rank a sequence
  const bool by_length = groups > 2 * sm_count && a.num_seqs <= 512;
  e = cudaLaunchKernelEx(&cfg, kern, a, cluster, key_cap, by_length);
  if (e != cudaSuccess || a.moves_cap == 0) return e;
  const int64_t most = (groups * a.moves_cap + 15) / 16;  // CTAs with one move a half warp
  const int64_t ctas = most < sm_count * 4 ? most : sm_count * 4;
  return launch_pdl(evict_move_kernel, dim3(static_cast<unsigned>(ctas), 1, 1), dim3(kThreads, 1, 1), 0, stream, a,
                    static_cast<int>(groups));
}

}  // namespace mj
