// Accumulated attention weight of every cached key (see mj_key_weights):
//   acc[j] <- (fresh ? 0 : decay acc[j]) + sum_n exp(z_nj - lse_n)
// over the rows n of one kv head that see key j.
//
// One pass over K (V is not read): per 128-key tile, S[key, row] = K Q^T with
// the keys on the MMA's M (the K tile as it lands from the TMA is operand A,
// the rows' e4m3 parts operand B), so a TMEM lane is a key, its row sum is
// thread-local, and one coalesced 4-byte store a key is all that leaves.  The
// logits and the row sums are fp32; bf16 Q is split into hi + lo e4m3 parts
// as in the decode kernels (exact down to 2^-10 of the scaled row maximum),
// up to 16 rows side by side in one MMA a K step with their products added in
// registers (half the MMA issues, 70 to 100 cycles each: 4 rows 65 -> 61 us;
// at 32 rows the additions cost as much as they save: 126 -> 130), else into
// one accumulator.
// With lse known there is no running maximum and nothing to merge, so the
// plan's items are only a list of tiles: it is cut evenly, whatever the items'
// lengths, into shares for which every kv head has a resident CTA, and a CTA
// walks its share as segments of one item each, the K ring running on across
// them.  The heads' CTAs of a share go over the same pages side by side: their
// rows of a token are neighbours, and the loads' 256-byte L2 sectors serve two
// of them (shares cut across the heads read a quarter more from HBM).
//
// Bound: 128 bytes of K a key and head against one exponential per row and
// key: HBM up to about 64 rows, the exponential units and the MMA above.  64
// sequences of 512 to 8192 keys, 8 heads, 4 rows: 55 us, 5.6 TB/s; 32 of 2048
// to 32768, 32 rows under a soft cap: 116 us, 5.4 TB/s, the cap's polynomial
// taking the issue slots (58 %, of which two CTAs can use little more).  A
// launch takes 256 packed rows of e4m3 Q or 128 of bf16 Q (two segments'
// operand rows beside a ring of seven K tiles); more rows are further launches
// that add on, in order.
//
// Roles (320 threads): warp 0 issues the K tiles into a ring, warp 1 (TMEM
// allocator) the MMAs, warps 2-5 and 6-9 take alternate tiles.  Up to 64 rows
// two CTAs fit an SM, one's segment starts under the other's stream.  Q parts
// and row constants are double-buffered over segments, the next segment's Q
// rows and scalars fetched during one.  Tiles that no row sees
// (a window, documents) are neither loaded nor multiplied; their weights only
// decay.

#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mj_kernels.h"
#include "score_mod.cuh"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kKeys = 128;                   // keys per tile = MMA M
constexpr int kTileBytes = kKeys * 128;      // 16 KB
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far above any legal wait
constexpr int kStatusTimeout = 5;            // MJ_ERR_TIMEOUT
constexpr int kStatusInvalidArg = 1;         // MJ_ERR_INVALID_ARG
constexpr int kThreads = 64 + 256;
constexpr int kMaxStages = 8;
constexpr int kBarCons = 1;  // named barrier of the 256 consumer threads
constexpr int kStackRows = 16;   // bf16 rows up to which both parts go into one MMA
constexpr int kItemCost = 3;     // tiles that a segment takes to start (0: 62 us for 55 on a decode batch; 2, 4 the same)
constexpr int kTwoCtaRows = 64;  // rows up to which two CTAs share an SM

struct KwArgs {
  DecodeModDev d;
  const float* lse;
  float* acc;
  int64_t acc_seq, acc_head;
  float decay;
  int32_t fresh;
  int32_t n0, n_rows;  // packed rows of this launch
  int32_t rows;        // n_rows rounded up: 8, or a multiple of 16
  int32_t n_mma;       // the MMA's N: rows (at least 16), or both parts of them
  int32_t stacked;     // bf16 Q: hi and lo rows side by side in one MMA
  int32_t stages;
  int32_t tmem_cols;
  int32_t s_bufs;      // S buffers of each group: 1 or 2
  int32_t off_q, off_stage, off_row, off_bar;  // shared memory, from the 1 KB boundary
};

__device__ __forceinline__ void set_abort(volatile int* abort, int32_t* status) {
  *abort = 1;
  if (status) atomicExch(status, kStatusTimeout);
}

// 128-byte-swizzled K-major row: 16-byte chunk cc of row r at cc ^ (r % 8)
__device__ __forceinline__ uint8_t* swz(uint8_t* part, int r, int cc) { return part + r * 128 + ((cc ^ (r & 7)) << 4); }

// The CTA's share as segments: tiles [t0, t1) of sequence b, of the CTA's head.
struct Segment {
  int t0, t1, b;
};
struct Walk {
  const int4* work;
  int w, t;          // where the next segment starts
  int w_end, t_end;  // the share ends before tile t_end of item w_end
  __device__ __forceinline__ bool next(Segment& s) {
    while (w < w_end || (w == w_end && t < t_end)) {
      const int4 item = work[w];
      const int tiles = w == w_end ? t_end : item.z - item.y;
      const int t0 = t;
      if (w == w_end) {
        t = t_end;
      } else {
        ++w;
        t = 0;
      }
      if (t0 < tiles) {
        s = Segment{item.y + t0, item.y + tiles, item.x};
        return true;
      }
    }
    return false;
  }
};

// Ranges of the launch's rows of one sequence, over a warp (identical in every
// warp): the smallest and largest first and last keys, and the prefix.
struct Limits {
  int lo_min, lo_max, hi_min, hi_max, pfx;
  // some row sees a key of the tile
  __device__ __forceinline__ bool seen(int key0) const {
    return key0 < pfx || (key0 <= hi_max && key0 + kKeys - 1 >= lo_min);
  }
  // one of the tiles [t0, t1) is seen
  __device__ __forceinline__ bool any(int t0, int t1) const {
    if (t0 * kKeys < pfx) return true;
    if (hi_max < 0) return false;
    const int from = lo_min / kKeys > t0 ? lo_min / kKeys : t0, to = hi_max / kKeys < t1 - 1 ? hi_max / kKeys : t1 - 1;
    return from <= to;
  }
  // every row sees every key of the tile
  __device__ __forceinline__ bool whole(int key0) const {
    return key0 + kKeys <= pfx || (key0 >= lo_max && key0 + kKeys - 1 <= hi_min);
  }
};
template <bool kMod>
__device__ __forceinline__ Limits warp_limits(const KwArgs& p, int b, int L, int lane) {
  const DecodeModDev& a = p.d;
  const int q0 = p.n0 / a.h_r, q1 = (p.n0 + p.n_rows - 1) / a.h_r;
  Limits m;
  if constexpr (!kMod) {
    const int first = L - a.q_len + q0, last = L - a.q_len + q1;
    m.lo_min = m.lo_max = 0;
    m.hi_min = a.causal && first < L - 1 ? first : L - 1;
    m.hi_max = a.causal && last < L - 1 ? last : L - 1;
    m.pfx = 0;
  } else {
    int lo_min = INT32_MAX, lo_max = -1, hi_min = INT32_MAX, hi_max = -1;
    m.pfx = 0;
    for (int qi = q0 + lane; qi <= q1; qi += 32) {
      const RowRange r = row_range(a.mod, a.causal, a.q_len, b, L, qi);
      m.pfx = r.pfx;
      lo_max = r.lo > lo_max ? r.lo : lo_max;
      hi_min = r.hi < hi_min ? r.hi : hi_min;
      if (r.lo <= r.hi) {
        lo_min = r.lo < lo_min ? r.lo : lo_min;
        hi_max = r.hi > hi_max ? r.hi : hi_max;
      }
    }
    m.lo_min = __reduce_min_sync(0xffffffffu, lo_min);
    m.lo_max = __reduce_max_sync(0xffffffffu, lo_max);
    m.hi_min = __reduce_min_sync(0xffffffffu, hi_min);
    m.hi_max = __reduce_max_sync(0xffffffffu, hi_max);
    m.pfx = __reduce_max_sync(0xffffffffu, m.pfx);
  }
  return m;
}

template <bool kQe4m3, bool kMod>
__global__ void __launch_bounds__(kThreads, 2)
    key_weights_kernel(const __grid_constant__ KwArgs p, const __grid_constant__ CUtensorMap tmap_k) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const DecodeModDev& a = p.d;
  constexpr int kParts = kQe4m3 ? 1 : 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(sm);
  // per-row constants of a segment, two buffers of [5][n_mma]
  float* const row_base = reinterpret_cast<float*>(sm + p.off_row);
  uint8_t* const misc = sm + p.off_bar + 8 * (2 * kMaxStages + 12);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  float* const amax_red = reinterpret_cast<float*>(misc + 32);      // [8]
  int64_t* const scan_red = reinterpret_cast<int64_t*>(misc + 64);  // [10]
  int* const walk_s = reinterpret_cast<int*>(misc + 160);           // (w, t) of the share's start and end
  int64_t* const need_red = reinterpret_cast<int64_t*>(misc + 176);  // [10]

  const uint32_t bar0 = sbase + p.off_bar;
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto sfull = [&](int buf) { return bar0 + 8u * (2 * kMaxStages + buf); };  // buf: group * 2 + its buffer
  auto sfree = [&](int buf) { return bar0 + 8u * (2 * kMaxStages + 4 + buf); };
  auto qready = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 8 + s); };
  const uint32_t drain = bar0 + 8u * (2 * kMaxStages + 10);
  // a group's n-th seen tile: its buffer, and that barrier's phase
  const int two = p.s_bufs - 1;
  const int buf_cols = p.tmem_cols >> (1 + two);
  auto buf_of = [&](int wg, int n) { return wg * 2 + (n & two); };
  auto phase_of = [&](int n) { return static_cast<uint32_t>((n >> two) & 1); };
  auto s_cols = [&](int wg, int n) { return static_cast<uint32_t>((wg * p.s_bufs + (n & two)) * buf_cols); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stages = p.stages;
  const int4* const work = reinterpret_cast<const int4*>(a.work);

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(kfull(s), 1);
      ptx::mbar_init(kempty(s), 1);
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(sfull(i), 1);
      ptx::mbar_init(sfree(i), 4);
    }
    for (int i = 0; i < 2; ++i) ptx::mbar_init(qready(i), 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), p.tmem_cols);
    ptx::tmem_relinquish();
  }
  const int max_len = a.max_blocks * a.page_size;  // acc has no more slots
  auto length_of = [&](int b) {
    const int L = a.seq_lens[b];
    return L < 0 ? 0 : (L < max_len ? L : max_len);
  };
  // ---- this CTA's share of the items' tiles in order, for one kv head; the
  // CTAs of the other heads' shares run beside it.  An item costs its tiles
  // and kItemCost more (the start of a segment); a cut inside that start falls
  // on the item's first tile.
  const int g = blockIdx.x % a.h_k;
  {
    const int per = (a.num_work + kThreads - 1) / kThreads;
    const int w0 = tid * per < a.num_work ? tid * per : a.num_work;
    const int w1 = w0 + per < a.num_work ? w0 + per : a.num_work;
    auto cost = [&](int w) -> int64_t {
      const int4 item = work[w];
      return item.z > item.y ? item.z - item.y + kItemCost : 0;
    };
    int64_t mine = 0;
    for (int w = w0; w < w1; ++w) mine += cost(w);
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan_red[warp] = x;
    // (one CTA) tiles that the sequences have and the items do not: a plan of
    // other lengths, such as the spans', whose other keys would go unnoticed
    const bool counts = blockIdx.x == 0 && a.status;
    if (counts) {
      int64_t need = 0;
      for (int b = tid; b < a.num_seqs; b += kThreads) {
        const int L = length_of(b);
        need += L > 0 ? (L + kKeys - 1) / kKeys : 1;  // a plan has a tile of an empty one too
      }
      for (int w = w0; w < w1; ++w) need -= work[w].z - work[w].y;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) need += __shfl_xor_sync(0xffffffffu, need, o);
      if (lane == 0) need_red[warp] = need;
    }
    if (tid < 2) {  // a cut past every item (the last share's end)
      walk_s[2 * tid] = a.num_work;
      walk_s[2 * tid + 1] = 0;
    }
    __syncthreads();
    int64_t before = x - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? scan_red[w] : 0;
      total += scan_red[w];
    }
    if (counts && tid == 0) {
      int64_t need = 0;
      for (int w = 0; w < kThreads / 32; ++w) need += need_red[w];
      if (need > 0) atomicExch(a.status, kStatusInvalidArg);
    }
    const int shares = gridDim.x / a.h_k, share = blockIdx.x / a.h_k;
    for (int cut = 0; cut < 2; ++cut) {
      const int64_t at = total * (share + cut) / shares;
      if (before <= at && at < before + mine) {  // one thread
        int64_t c = before;
        int w = w0;
        while (at >= c + cost(w)) c += cost(w++);
        walk_s[2 * cut] = w;
        walk_s[2 * cut + 1] = at - c > kItemCost ? static_cast<int>(at - c) - kItemCost : 0;
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk{work, walk_s[0], walk_s[1], walk_s[2], walk_s[3]};
  Segment sg;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    const int PS = a.page_size;
    const int box_rows = PS < kKeys ? PS : kKeys;
    const int nbox = kKeys / box_rows;
    const bool active = lane < nbox;
    if (lane == 0) ptx::prefetch_tmap(&tmap_k);
    const bool evict_first = a.kv_evict_first != 0;
    const uint64_t policy = ptx::policy_evict_first();
    const uint32_t tile_tx = kv_box_bytes(a.kv_format, kKeys);
    int u = 0;  // tiles issued
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int L = length_of(sg.b);
      const Limits lim = warp_limits<kMod>(p, sg.b, L, lane);
      const int64_t bt_row = static_cast<int64_t>(sg.b) * a.max_blocks;
      int valid_pages = (L + PS - 1) / PS;
      valid_pages = valid_pages < a.max_blocks ? valid_pages : a.max_blocks;
      // block-table entries from a register window (lane l: block wbase + l),
      // the next 32 one refill ahead
      auto load_win = [&](int base) -> int {
        const int blk = base + lane;
        return blk < valid_pages ? a.block_table[bt_row + blk] : a.num_pages;
      };
      int wbase = sg.t0 * kKeys / PS;
      int win = load_win(wbase), win_next = load_win(wbase + 32);
      for (int t = sg.t0; t < sg.t1; ++t) {
        const int key0 = t * kKeys;
        if (key0 / PS >= wbase + 32) {
          wbase += 32;
          win = win_next;
          win_next = load_win(wbase + 32);
        }
        if (!lim.seen(key0)) continue;
        const int st = u % stages;
        if (u >= stages) {
          const bool freed = ptx::mbar_wait_bounded(kempty(st), ((u / stages) - 1) & 1, abort_flag, kWaitNs);
          if (__any_sync(0xffffffffu, !freed)) {
            if (lane == 0) set_abort(abort_flag, a.status);
            ok = false;
            break;
          }
        }
        const int key = key0 + lane * box_rows;
        const int pg = __shfl_sync(0xffffffffu, win, (key / PS - wbase) & 31);
        const int page = (active && key < L) ? pg : a.num_pages;  // out of bounds: zeros
        if (lane == 0) ptx::mbar_arrive_expect_tx(kfull(st), tile_tx);
        __syncwarp();
        if (active)
          ptx::tma_load_kv(sbase + st * kTileBytes + lane * box_rows * 128, &tmap_k, kfull(st), 0, key % PS, g, page,
                           evict_first, policy);
        ++u;
      }
    }
    if (*abort_flag && lane == 0) {  // leave no copy in flight
      volatile int never = 0;
      for (int i = (u > stages ? u - stages : 0); i < u; ++i)
        ptx::mbar_wait_bounded(kfull(i % stages), (i / stages) & 1, &never, kWaitNs / 4);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA
    // (the whole warp walks and takes the limits; lane 0 waits and issues)
    const uint32_t idesc = ptx::idesc_f8f6f4(kKeys, p.n_mma, false, false, kv_mma_format(a.kv_format), 0);
    const uint64_t kdesc0 = ptx::smem_desc(sbase, 16, 1024, ptx::kSwizzle128B);
    const uint64_t part_step = static_cast<uint64_t>(p.rows * 128) >> 4;
    const int parts = kParts == 2 && !p.stacked ? 2 : 1;  // MMAs a K step
    const int q_bytes = (kParts == 2 ? 2 * p.rows : p.n_mma) * 128;  // of one segment's operand rows
    int u = 0, s = 0;  // tiles, segments with a seen tile (only those have a Q buffer)
    bool ok = true;
    while (ok && walk.next(sg)) {
      const Limits lim = warp_limits<kMod>(p, sg.b, length_of(sg.b), lane);
      if (!lim.any(sg.t0, sg.t1)) continue;
      const uint64_t qdesc =
          ptx::smem_desc(sbase + p.off_q + (s & 1) * q_bytes, 16, 1024, ptx::kSwizzle128B);
      if (lane == 0) {
        ok = ptx::mbar_wait_bounded(qready(s & 1), (s >> 1) & 1, abort_flag, kWaitNs);
        for (int t = sg.t0; ok && t < sg.t1; ++t) {
          if (!lim.seen(t * kKeys)) continue;
          const int st = u % stages, wg = u & 1, n = u >> 1;
          if (!ptx::mbar_wait_bounded(kfull(st), (u / stages) & 1, abort_flag, kWaitNs) ||
              (n > two &&
               !ptx::mbar_wait_bounded(sfree(buf_of(wg, n)), phase_of(n - 1 - two), abort_flag, kWaitNs))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint64_t kdesc = kdesc0 + static_cast<uint64_t>((st * kTileBytes) >> 4);
          const uint32_t d = tmem + s_cols(wg, n);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            ptx::mma_e4m3(d, kdesc + 2 * kk, qdesc + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            if (parts == 2) ptx::mma_e4m3(d, kdesc + 2 * kk, qdesc + part_step + 2 * kk, idesc, 1u);
          }
          ptx::mma_commit(sfull(buf_of(wg, n)));
          ptx::mma_commit(kempty(st));
          ++u;
        }
      }
      ++s;
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      if (!ok) set_abort(abort_flag, a.status);
      ptx::mma_commit(drain);
      volatile int never = 0;
      ptx::mbar_wait_bounded(drain, 0, &never, kWaitNs);
    }
  } else {
    // ----------------------------------------------------------- weights
    const int ct = tid - 64;  // consumer thread
    const int wg = ct >> 7, quarter = warp & 3;
    const int key_in_tile = quarter * 32 + lane;
    const uint32_t tmem_w = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool far = false;  // the last capped tile held scores past the polynomial's range
    const float cap2 = kMod ? a.mod.softcap * kLog2e : 0.f;
    const float2 cap22 = make_float2(cap2, cap2);
    const TanhRatio ratio(cap2);
    int u = 0, s = 0;
    // the next segment's raw Q rows (this thread's 16-element chunks, by
    // asynchronous copies) and scalars are on their way during a segment
    constexpr int kChunkBytes = kQe4m3 ? 16 : 32;
    uint8_t* const stage = sm + p.off_stage;
    int L_next = 0;
    float kd_next = 0.f, qd_next = 0.f, lse_next = 0.f;
    auto fetch = [&](int b) {
      const uint8_t* src = static_cast<const uint8_t*>(a.q) +
                           (b * a.q_seq + (static_cast<int64_t>(g) * a.n_q + p.n0) * kHeadDimDev) * (kQe4m3 ? 1 : 2);
      for (int id = ct; id < p.n_rows * 8; id += 256) {
        cp_async16(stage + id * kChunkBytes, src + id * kChunkBytes, true);
        if (!kQe4m3) cp_async16(stage + id * kChunkBytes + 16, src + id * kChunkBytes + 16, true);
      }
      cp_async_commit();
      L_next = length_of(b);
      kd_next = a.kd[b * a.kd_seq + g * a.kd_head];
      qd_next = a.qd[b * a.qd_seq + g * a.qd_head];
      if (ct < p.n_rows) lse_next = p.lse[(static_cast<int64_t>(b) * a.h_k + g) * a.n_q + p.n0 + ct];
    };
    Segment upcoming;
    bool more = walk.next(upcoming);
    if (more) fetch(upcoming.b);
    while (more) {
      sg = upcoming;
      const int b = sg.b, L = L_next;
      const float kd = kd_next, qd = qd_next;
      const Limits lim = warp_limits<kMod>(p, b, L, lane);
      cp_async_wait<0>();
      float* const row_nlse2 = row_base + (s & 1) * 5 * p.rows;  // -lse in log2 units
      float* const row_slope2 = row_nlse2 + p.rows;
      float* const row_pos = row_slope2 + p.rows;
      int* const row_lo = reinterpret_cast<int*>(row_pos + p.rows);
      int* const row_hi = row_lo + p.rows;
      uint8_t* const qbase = sm + p.off_q + (s & 1) * (kParts == 2 ? 2 * p.rows : p.n_mma) * 128;

      int shift = 0;
      // ---- Q rows -> one (e4m3) or two (bf16: hi + lo) operand rows, a
      // 16-element chunk a thread and round
      if (lim.any(sg.t0, sg.t1)) {
        const int chunks = p.rows * 8;
        if constexpr (!kQe4m3) {
          uint32_t mbits = 0;  // bf16 |q| maximum: integer maximum of the magnitude bits
          for (int id = ct; id < p.n_rows * 8; id += 256) {
            const uint4* src = reinterpret_cast<const uint4*>(stage + id * kChunkBytes);
            const uint4 r0 = src[0], r1 = src[1];
            const uint32_t v8[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) mbits = max(mbits, max(v8[e] & 0x7FFFu, (v8[e] >> 16) & 0x7FFFu));
          }
          mbits = __reduce_max_sync(0xffffffffu, mbits);
          if (lane == 0) amax_red[warp - 2] = __uint_as_float(mbits << 16);
        }
        // (also: both groups are done with the segment before, so this one's
        // buffers, used two segments ago, are free)
        ptx::named_bar_sync(kBarCons, 256);
        if constexpr (!kQe4m3) {
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax_red[i]);
          if (amax > 0.f) {
            const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 127;
            shift = 7 - e;  // max |q| 2^shift in [128, 256)
            shift = shift > 126 ? 126 : (shift < -126 ? -126 : shift);
          }
        }
        const float qscale = ldexpf(1.f, shift);
        for (int id = ct; id < chunks; id += 256) {
          const int r = id >> 3, cc = id & 7;
          const bool live = r < p.n_rows;
          if constexpr (kQe4m3) {
            const uint4* src = reinterpret_cast<const uint4*>(stage + id * kChunkBytes);
            *reinterpret_cast<uint4*>(swz(qbase, r, cc)) = live ? *src : make_uint4(0u, 0u, 0u, 0u);
          } else {
            const uint4* src = reinterpret_cast<const uint4*>(stage + id * kChunkBytes);
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            const uint4 r0 = live ? src[0] : z, r1 = live ? src[1] : z;
            const uint32_t w8[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int wi = 0; wi < 4; ++wi) {
              float x[4], hf[4];
              x[0] = __uint_as_float(w8[2 * wi] << 16) * qscale;
              x[1] = __uint_as_float(w8[2 * wi] & 0xFFFF0000u) * qscale;
              x[2] = __uint_as_float(w8[2 * wi + 1] << 16) * qscale;
              x[3] = __uint_as_float(w8[2 * wi + 1] & 0xFFFF0000u) * qscale;
              const uint16_t h01 = ptx::f32x2_to_e4m3x2(x[0], x[1]);
              const uint16_t h23 = ptx::f32x2_to_e4m3x2(x[2], x[3]);
              hw[wi] = static_cast<uint32_t>(h01) | (static_cast<uint32_t>(h23) << 16);
              e4m3x4_to_f32(hw[wi], hf);
              const uint16_t l01 = ptx::f32x2_to_e4m3x2(x[0] - hf[0], x[1] - hf[1]);
              const uint16_t l23 = ptx::f32x2_to_e4m3x2(x[2] - hf[2], x[3] - hf[3]);
              lw[wi] = static_cast<uint32_t>(l01) | (static_cast<uint32_t>(l23) << 16);
            }
            *reinterpret_cast<uint4*>(swz(qbase, r, cc)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(swz(qbase + p.rows * 128, r, cc)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
          }
        }
        // ---- the rows' constants; a row past n_rows or without keys adds
        // 2^-inf (its scores are finite: Q's rows are zeros or data)
        if (ct < p.rows) {
          const int n = p.n0 + ct;
          float nlse2 = -INFINITY, slope2 = 0.f;
          int lo = 0, hi = -1, from_first = 0;
          if (ct < p.n_rows) {
            const int qi = n / a.h_r;
            from_first = qi - p.n0 / a.h_r;
            if constexpr (kMod) {
              const RowRange r = row_range(a.mod, a.causal, a.q_len, b, L, qi);
              lo = r.lo;
              hi = r.hi;
              if (a.mod.slopes) slope2 = a.mod.slopes[g * a.h_r + n % a.h_r] * kLog2e;
            } else {
              const int pos = L - a.q_len + qi;
              hi = a.causal && pos < L - 1 ? pos : L - 1;
            }
            nlse2 = lse_next == -INFINITY ? -INFINITY : -lse_next * kLog2e;
          }
          row_nlse2[ct] = nlse2;
          row_slope2[ct] = slope2;
          row_pos[ct] = static_cast<float>(from_first);
          row_lo[ct] = lo;
          row_hi[ct] = hi;
        }
        ptx::fence_proxy_async_smem();
        ptx::named_bar_sync(kBarCons, 256);
        if (ct == 0) ptx::mbar_arrive(qready(s & 1));
        ++s;
      }
      more = walk.next(upcoming);
      if (more) fetch(upcoming.b);  // (this thread has read its staged chunks)

      const float to_logit = a.softmax_scale * qd * kd * ldexpf(1.f, -shift);
      const float c1 = cap2 > 0.f ? to_logit / a.mod.softcap : to_logit * kLog2e;
      const float2 c12 = make_float2(c1, c1);
      const int pos_min = L - a.q_len + p.n0 / a.h_r;  // of the launch's rows
      float* const acc = p.acc + b * p.acc_seq + g * p.acc_head;
      // this group's tiles: every second one that is seen (the MMA's order),
      // and every second of the others; the accumulators of its next tile are
      // on their way while it works on one
      auto reads = [&](int key) { return key < L - p.fresh && p.decay > 0.f; };
      auto own = [&](int t) {  // its first tile from t on, counting the other group's in u
        for (; t < sg.t1; ++t) {
          if (lim.seen(t * kKeys)) {
            if ((u & 1) == wg) break;
            ++u;
          } else if ((t & 1) == wg) {
            break;
          }
        }
        return t;
      };
      int t = own(sg.t0);
      float old = t < sg.t1 && reads(t * kKeys + key_in_tile) ? acc[t * kKeys + key_in_tile] : 0.f;
      while (t < sg.t1) {
        const int key0 = t * kKeys;
        const int key = key0 + key_in_tile;
        const bool is_seen = lim.seen(key0);
        const int n = u >> 1;  // its place among the group's seen tiles
        u += is_seen;
        const int t_next = own(t + 1);
        const float old_next =
            t_next < sg.t1 && reads(t_next * kKeys + key_in_tile) ? acc[t_next * kKeys + key_in_tile] : 0.f;
        float2 sum2 = make_float2(0.f, 0.f);
        if (is_seen) {
          const int sb = buf_of(wg, n);
          const uint32_t tmem_s = tmem_w + s_cols(wg, n);
          if (!ptx::mbar_wait_bounded(sfull(sb), phase_of(n), abort_flag, kWaitNs)) set_abort(abort_flag, a.status);
          ptx::tc_fence_after();
          const bool whole = lim.whole(key0);  // uniform
          // positions from the launch's first row's: exact to 2^24 of distance anywhere
          const float fkey = static_cast<float>(key - pos_min);
          const float2 nkey2 = make_float2(-fkey, -fkey);
          const bool ahead = key0 + kKeys - 1 > pos_min;  // some distance may be negative
          // the tile's row sums; capped scores by the polynomial (near) or by
          // the exponential form; returns whether all lay in its range
          auto sums_of = [&](auto width, bool near) {
            constexpr int W = decltype(width)::value;  // columns at a time
            float top = 0.f;  // largest square of a score over the cap
            sum2 = make_float2(0.f, 0.f);
            for (int c0 = 0; c0 < p.rows; c0 += W) {
              uint32_t r[W];
              if constexpr (W == 8)
                MJ_TMEM_LD8(tmem_s + c0, r);
              else
                MJ_TMEM_LD16(tmem_s + c0, r);
              if (!kQe4m3 && p.stacked) {  // the lo rows' products
                uint32_t lo[W];
                if constexpr (W == 8)
                  MJ_TMEM_LD8(tmem_s + p.rows + c0, lo);
                else
                  MJ_TMEM_LD16(tmem_s + p.rows + c0, lo);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < W; e += 2) {
                  const float2 x = add2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])),
                                        make_float2(__uint_as_float(lo[e]), __uint_as_float(lo[e + 1])));
                  r[e] = __float_as_uint(x.x);
                  r[e + 1] = __float_as_uint(x.y);
                }
              } else {
                ptx::tmem_ld_wait();
              }
              float2 y[W / 2];
              if (kMod && cap2 > 0.f) {
                if (near) {
#pragma unroll
                  for (int e = 0; e < W / 2; ++e) {
                    const float2 t = mul2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), c12);
                    const float2 sq = mul2(t, t);
                    top = fmax3(top, sq.x, sq.y);
                    y[e] = fma2(t, ratio(sq), *reinterpret_cast<const float2*>(row_nlse2 + c0 + 2 * e));
                  }
                } else {
#pragma unroll
                  for (int e = 0; e < W / 2; ++e) {
                    const float2 t = mul2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), c12);
                    const float2 sq = mul2(t, t);
                    top = fmax3(top, sq.x, sq.y);
                    y[e] = fma2(make_float2(tanh_any(t.x), tanh_any(t.y)), cap22,
                                *reinterpret_cast<const float2*>(row_nlse2 + c0 + 2 * e));
                  }
                }
              } else {
#pragma unroll
                for (int e = 0; e < W / 2; ++e)
                  y[e] = fma2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), c12,
                              *reinterpret_cast<const float2*>(row_nlse2 + c0 + 2 * e));
              }
              if (kMod && a.mod.slopes) {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                  const float2 sl = *reinterpret_cast<const float2*>(row_slope2 + c0 + 2 * e);
                  float2 d = add2(*reinterpret_cast<const float2*>(row_pos + c0 + 2 * e), nkey2);
                  if (ahead) d = make_float2(fabsf(d.x), fabsf(d.y));
                  y[e] = fma2(make_float2(-sl.x, -sl.y), d, y[e]);
                }
              }
              if (whole) {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) sum2 = add2(sum2, make_float2(fast_exp2(y[e].x), fast_exp2(y[e].y)));
              } else {
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                  const int c = c0 + 2 * e;
                  const bool v0 = key < lim.pfx || (key >= row_lo[c] && key <= row_hi[c]);
                  const bool v1 = key < lim.pfx || (key >= row_lo[c + 1] && key <= row_hi[c + 1]);
                  sum2.x += v0 ? fast_exp2(y[e].x) : 0.f;
                  sum2.y += v1 ? fast_exp2(y[e].y) : 0.f;
                }
              }
            }
            return __all_sync(0xffffffffu, top < kTanhSmall * kTanhSmall);
          };
          auto tile_sums = [&](bool near) {
            return p.rows == 8 ? sums_of(std::integral_constant<int, 8>{}, near)
                               : sums_of(std::integral_constant<int, 16>{}, near);
          };
          if (kMod && cap2 > 0.f) {
            // most scores are small against a cap; a tile that holds others is
            // done again, and the next one starts with the exponential form
            if (!far && !tile_sums(true)) far = true;
            if (far) far = !tile_sums(false);
          } else {
            tile_sums(true);
          }
          ptx::tc_fence_before();  // the buffer is read
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(sfree(sb));
        }
        if (key < L && !*abort_flag) acc[key] = (reads(key) ? p.decay * old : 0.f) + (sum2.x + sum2.y);
        t = t_next;
        old = old_next;
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, p.tmem_cols);
}

template <bool kQe4m3, bool kMod>
cudaError_t launch_kw(const KwArgs& p, const CUtensorMap& mk, int ctas, size_t smem, cudaStream_t stream) {
  auto kern = key_weights_kernel<kQe4m3, kMod>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas), 1, 1), dim3(kThreads, 1, 1), smem, stream, p, mk);
}

}  // namespace

cudaError_t launch_key_weights(const DecodeModDev& a, bool q_e4m3, bool has_mod, int n0, int n_rows, const float* lse,
                               float* acc, int64_t acc_seq, int64_t acc_head, float decay, int fresh, int sm_count,
                               cudaStream_t stream) {
  KwArgs p{};
  p.d = a;
  p.lse = lse;
  p.acc = acc;
  p.acc_seq = acc_seq;
  p.acc_head = acc_head;
  p.decay = decay;
  p.fresh = fresh;
  p.n0 = n0;
  p.n_rows = n_rows;
  p.rows = n_rows <= 8 ? 8 : (n_rows + 15) / 16 * 16;
  p.stacked = !q_e4m3 && p.rows <= kStackRows;
  p.n_mma = p.stacked ? 2 * p.rows : (p.rows < 16 ? 16 : p.rows);
  const int per_sm = n_rows <= kTwoCtaRows ? 2 : 1;
  // S buffers: two of each group (the MMA runs a tile ahead) where TMEM has
  // the columns
  p.s_bufs = 4 * p.n_mma <= 512 / per_sm ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.s_bufs * p.n_mma) p.tmem_cols *= 2;
  const int part_bytes = (q_e4m3 ? p.n_mma : 2 * p.rows) * 128;  // a segment's operand rows
  const int q_bytes = 2 * part_bytes;                            // two segments'
  const int row_bytes = 2 * 5 * p.rows * 4;
  const int stage_bytes = p.rows * 128 * (q_e4m3 ? 1 : 2);
  const int tail = stage_bytes + row_bytes + 8 * (2 * kMaxStages + 12) + 256;
  const int limit = (per_sm == 2 ? 112 : 224) * 1024;
  p.stages = (limit - 1024 - q_bytes - tail) / kTileBytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.off_q = p.stages * kTileBytes;
  p.off_stage = p.off_q + q_bytes;
  p.off_row = p.off_stage + stage_bytes;
  p.off_bar = p.off_row + row_bytes;
  const size_t smem = 1024 + static_cast<size_t>(p.off_q) + q_bytes + tail;
  const int box_rows = a.page_size < kKeys ? a.page_size : kKeys;
  CUtensorMap mk;
  if (!make_kv_map(&mk, a.k, a.page_size, a.h_k, a.num_pages, a.k_row, a.k_head, a.k_page, box_rows, 1, a.kv_format))
    return cudaErrorInvalidValue;
  // one share a resident CTA, the same cuts for every head; never more shares
  // than tiles could be (an item holds at most all of a sequence's)
  const int64_t tiles = static_cast<int64_t>(a.num_work) * ((a.max_blocks * a.page_size + kKeys - 1) / kKeys);
  int64_t shares = sm_count * per_sm / a.h_k;
  shares = shares < 1 ? 1 : (shares > tiles ? tiles : shares);
  const int ctas = static_cast<int>(shares) * a.h_k;
  if (q_e4m3)
    return has_mod ? launch_kw<true, true>(p, mk, ctas, smem, stream) : launch_kw<true, false>(p, mk, ctas, smem, stream);
  return has_mod ? launch_kw<false, true>(p, mk, ctas, smem, stream) : launch_kw<false, false>(p, mk, ctas, smem, stream);
}

}  // namespace mj
