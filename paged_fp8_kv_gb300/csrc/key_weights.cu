// Accumulated attention weight of every cached key (see mj_key_weights):
//   acc[j] <- (fresh ? 0 : decay acc[j]) + sum_n exp(z_nj - lse_n)
// over the rows n of one kv head that see key j.
//
// One pass over K (V is not read): per 128-key tile, S[key, row] = K Q^T with
// the keys on the MMA's M (the K tile as it lands from the TMA is operand A,
// the rows' e4m3 parts operand B), so a TMEM lane is a key, its row sum is
// thread-local, and one coalesced 4-byte store a key is all that leaves.  The
// logits and the row sums are fp32; bf16 Q is split into hi + lo e4m3 parts
// as in the decode kernels (exact down to 2^-10 of the scaled row maximum).
// With lse known there is no running maximum and nothing to merge between the
// plan's items.
//
// Bound: 128 bytes of K a key and head against one exponential per row and
// key: HBM up to about 80 rows, the exponential units above.  256 packed rows
// a launch (TMEM holds two buffers of 256 columns); more rows are further
// launches that add on, in order.
//
// Roles (320 threads): warp 0 issues the K tiles into a ring, warp 1 (TMEM
// allocator) the MMAs, warps 2-5 and 6-9 take alternate tiles.  Up to 128
// rows two CTAs fit an SM, one's start and end under the other's stream.
// Tiles that no row sees (a window, documents) are neither loaded nor
// multiplied; their weights only decay.

#include <cuda.h>
#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "score_mod.cuh"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kKeys = 128;                   // keys per tile = MMA M
constexpr int kTileBytes = kKeys * 128;      // 16 KB
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far above any legal wait
constexpr int kStatusTimeout = 5;            // MJ_ERR_TIMEOUT
constexpr int kThreads = 64 + 256;
constexpr int kMaxRows = 256;
constexpr int kMaxStages = 8;
constexpr int kBarCons = 1;  // named barrier of the 256 consumer threads

struct KwArgs {
  DecodeModDev d;
  const float* lse;
  float* acc;
  int64_t acc_seq, acc_head;
  float decay;
  int32_t fresh;
  int32_t n0, n_rows;   // packed rows of this launch
  int32_t n_mma;        // n_rows rounded up to 16: the MMA's N
  int32_t stages;
  int32_t tmem_cols;
  int32_t off_q, off_row, off_bar;  // shared memory, from the 1 KB boundary
};

__device__ __forceinline__ void set_abort(volatile int* abort, int32_t* status) {
  *abort = 1;
  if (status) atomicExch(status, kStatusTimeout);
}

// 128-byte-swizzled K-major row: 16-byte chunk cc of row r at cc ^ (r % 8)
__device__ __forceinline__ uint8_t* swz(uint8_t* part, int r, int cc) { return part + r * 128 + ((cc ^ (r & 7)) << 4); }

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
  // per-row constants, [kMaxRows] each
  float* const row_lse2 = reinterpret_cast<float*>(sm + p.off_row);
  int* const row_hi = reinterpret_cast<int*>(row_lse2 + kMaxRows);
  int* const row_lo = row_hi + kMaxRows;
  float* const row_slope2 = reinterpret_cast<float*>(row_lo + kMaxRows);
  float* const row_pos = row_slope2 + kMaxRows;
  uint8_t* const misc = sm + p.off_bar + 8 * (2 * kMaxStages + 8);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 4);
  int* const lim = reinterpret_cast<int*>(misc + 8);  // lo_min, lo_max, hi_min, hi_max over the rows
  float* const amax_red = reinterpret_cast<float*>(misc + 32);  // [8]

  const uint32_t bar0 = sbase + p.off_bar;
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto sfull = [&](int wg) { return bar0 + 8u * (2 * kMaxStages + wg); };
  auto sfree = [&](int wg) { return bar0 + 8u * (2 * kMaxStages + 2 + wg); };
  const uint32_t qready = bar0 + 8u * (2 * kMaxStages + 4);
  const uint32_t drain = qready + 8u;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.h_k;
  const int4 item = reinterpret_cast<const int4*>(a.work)[blockIdx.x / a.h_k];
  const int b = item.x, t_begin = item.y, t_end = item.z;
  if (t_end <= t_begin) return;  // padding item
  int L = a.seq_lens[b];
  L = L < a.max_blocks * a.page_size ? L : a.max_blocks * a.page_size;  // acc has no more slots
  const int T = t_end - t_begin;
  const int stages = p.stages;

  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(kfull(s), 1);
      ptx::mbar_init(kempty(s), 1);
    }
    for (int wg = 0; wg < 2; ++wg) {
      ptx::mbar_init(sfull(wg), 1);
      ptx::mbar_init(sfree(wg), 4);
    }
    ptx::mbar_init(qready, 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    lim[0] = INT32_MAX;
    lim[1] = -1;
    lim[2] = INT32_MAX;
    lim[3] = -1;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), p.tmem_cols);
    ptx::tmem_relinquish();
  }
  // the rows' ranges: thread r is row r
  int pfx = 0;
  if (kMod && a.mod.prefix) {
    pfx = a.mod.prefix[b];
    pfx = pfx < 0 ? 0 : (pfx > L ? L : pfx);
  }
  if (tid < kMaxRows) {
    const int n = p.n0 + tid;
    const bool live = tid < p.n_rows;
    float lse2 = INFINITY, slope2 = 0.f;
    int lo = 0, hi = -1, pos = 0;
    if (live) {
      const int qi = n / a.h_r;
      pos = L - a.q_len + qi;
      if constexpr (kMod) {
        const RowRange r = row_range(a.mod, a.causal, a.q_len, b, L, qi);
        lo = r.lo;
        hi = r.hi;
        if (a.mod.slopes) slope2 = a.mod.slopes[g * a.h_r + n % a.h_r] * kLog2e;
      } else {
        hi = a.causal && pos < L - 1 ? pos : L - 1;
      }
      const float lse = p.lse[(static_cast<int64_t>(b) * a.h_k + g) * a.n_q + n];
      lse2 = lse == -INFINITY ? INFINITY : lse * kLog2e;  // a row without keys adds nothing
      atomicMin(&lim[0], lo <= hi ? lo : INT32_MAX);
      atomicMax(&lim[1], lo);
      atomicMin(&lim[2], hi);
      atomicMax(&lim[3], lo <= hi ? hi : -1);
    }
    row_lse2[tid] = lse2;
    row_hi[tid] = hi;
    row_lo[tid] = lo;
    row_slope2[tid] = slope2;
    row_pos[tid] = static_cast<float>(pos);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int lo_min = lim[0], lo_max = lim[1], hi_min = lim[2], hi_max = lim[3];
  auto key_of_tile = [&](int i) { return (t_begin + i) * kKeys; };
  // a tile some row sees (every role walks the same list)
  auto seen = [&](int i) {
    const int k0 = key_of_tile(i);
    return k0 < pfx || (k0 <= hi_max && k0 + kKeys - 1 >= lo_min);
  };

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    const int PS = a.page_size;
    const int box_rows = PS < kKeys ? PS : kKeys;
    const int nbox = kKeys / box_rows;
    const bool active = lane < nbox;
    const int64_t bt_row = static_cast<int64_t>(b) * a.max_blocks;
    int valid_pages = (L + PS - 1) / PS;
    valid_pages = valid_pages < a.max_blocks ? valid_pages : a.max_blocks;
    if (lane == 0) ptx::prefetch_tmap(&tmap_k);
    const bool evict_first = a.kv_evict_first != 0;
    const uint64_t policy = ptx::policy_evict_first();
    const uint32_t tile_tx = kv_box_bytes(a.kv_format, kKeys);
    // block-table entries from a register window (lane l: block wbase + l),
    // the next 32 one refill ahead
    auto load_win = [&](int base) -> int {
      const int blk = base + lane;
      return blk < valid_pages ? a.block_table[bt_row + blk] : a.num_pages;
    };
    int wbase = key_of_tile(0) / PS;
    int win = load_win(wbase), win_next = load_win(wbase + 32);
    int u = 0;
    for (int i = 0; i < T; ++i) {
      const int key0 = key_of_tile(i);
      if (key0 / PS >= wbase + 32) {
        wbase += 32;
        win = win_next;
        win_next = load_win(wbase + 32);
      }
      if (!seen(i)) continue;
      const int st = u % stages;
      if (u >= stages) {
        const bool freed = ptx::mbar_wait_bounded(kempty(st), ((u / stages) - 1) & 1, abort_flag, kWaitNs);
        if (__any_sync(0xffffffffu, !freed)) {
          if (lane == 0) set_abort(abort_flag, a.status);
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
    if (*abort_flag && lane == 0) {  // leave no copy in flight
      volatile int never = 0;
      for (int i = (u > stages ? u - stages : 0); i < u; ++i)
        ptx::mbar_wait_bounded(kfull(i % stages), (i / stages) & 1, &never, kWaitNs / 4);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- MMA
    if (lane == 0) {
      bool ok = ptx::mbar_wait_bounded(qready, 0, abort_flag, kWaitNs);
      const uint32_t idesc = ptx::idesc_f8f6f4(kKeys, p.n_mma, false, false, kv_mma_format(a.kv_format), 0);
      const uint64_t kdesc0 = ptx::smem_desc(sbase, 16, 1024, ptx::kSwizzle128B);
      const uint64_t qdesc = ptx::smem_desc(sbase + p.off_q, 16, 1024, ptx::kSwizzle128B);
      const uint64_t part_step = static_cast<uint64_t>(p.n_mma * 128) >> 4;
      int u = 0;
      for (int i = 0; ok && i < T; ++i) {
        if (!seen(i)) continue;
        const int st = u % stages, wg = u & 1, t = u >> 1;
        if (!ptx::mbar_wait_bounded(kfull(st), (u / stages) & 1, abort_flag, kWaitNs) ||
            (t >= 1 && !ptx::mbar_wait_bounded(sfree(wg), (t - 1) & 1, abort_flag, kWaitNs))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t kdesc = kdesc0 + static_cast<uint64_t>((st * kTileBytes) >> 4);
        const uint32_t d = tmem + wg * (p.tmem_cols >> 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            ptx::mma_e4m3(d, kdesc + 2 * kk, qdesc + part * part_step + 2 * kk, idesc, (kk > 0 || part > 0) ? 1u : 0u);
        }
        ptx::mma_commit(sfull(wg));
        ptx::mma_commit(kempty(st));
        ++u;
      }
      if (!ok) set_abort(abort_flag, a.status);
      ptx::mma_commit(drain);
      volatile int never = 0;
      ptx::mbar_wait_bounded(drain, 0, &never, kWaitNs);
    }
  } else {
    // ----------------------------------------------------------- weights
    const int ct = tid - 64;  // consumer thread = Q row to lay out
    const int wg = ct >> 7, quarter = warp & 3;
    const int key_in_tile = quarter * 32 + lane;
    const float kd = a.kd[b * a.kd_seq + g * a.kd_head];
    const float qd = a.qd[b * a.qd_seq + g * a.qd_head];

    // ---- Q row -> one (e4m3) or two (bf16: hi + lo) operand rows
    uint8_t* const qbase = sm + p.off_q;
    const bool live = ct < p.n_rows;
    const int64_t qoff = b * a.q_seq + (static_cast<int64_t>(g) * a.n_q + p.n0 + (live ? ct : 0)) * kHeadDimDev;
    int shift = 0;
    if constexpr (kQe4m3) {
      if (ct < p.n_mma) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + qoff);
#pragma unroll
        for (int cc = 0; cc < 8; ++cc)
          *reinterpret_cast<uint4*>(swz(qbase, ct, cc)) = live ? src[cc] : make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + qoff);
      uint4 raw[16];
      uint32_t mbits = 0;
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        raw[w] = live ? src[w] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t v4[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) mbits = max(mbits, max(v4[e] & 0x7FFFu, (v4[e] >> 16) & 0x7FFFu));
      }
      float amax = __uint_as_float(mbits << 16);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (lane == 0) amax_red[warp - 2] = amax;
      ptx::named_bar_sync(kBarCons, 256);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, amax_red[i]);
      if (amax > 0.f) {
        const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFF) - 127;
        shift = 7 - e;  // max |q| 2^shift in [128, 256)
        shift = shift > 126 ? 126 : (shift < -126 ? -126 : shift);
      }
      const float qscale = ldexpf(1.f, shift);
      if (ct < p.n_mma) {
#pragma unroll
        for (int cc = 0; cc < 8; ++cc) {
          uint32_t hw[4], lw[4];
          const uint32_t w8[8] = {raw[2 * cc].x,     raw[2 * cc].y,     raw[2 * cc].z,     raw[2 * cc].w,
                                  raw[2 * cc + 1].x, raw[2 * cc + 1].y, raw[2 * cc + 1].z, raw[2 * cc + 1].w};
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
          *reinterpret_cast<uint4*>(swz(qbase, ct, cc)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          *reinterpret_cast<uint4*>(swz(qbase + p.n_mma * 128, ct, cc)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
      }
    }
    ptx::fence_proxy_async_smem();
    ptx::named_bar_sync(kBarCons, 256);
    if (ct == 0) ptx::mbar_arrive(qready);

    const float to_logit = a.softmax_scale * qd * kd * ldexpf(1.f, -shift);
    const float cap2 = kMod ? a.mod.softcap * kLog2e : 0.f;
    const float c1 = kMod && a.mod.softcap > 0.f ? to_logit / a.mod.softcap : to_logit * kLog2e;
    const uint32_t tmem_s = tmem + wg * (p.tmem_cols >> 1) + (static_cast<uint32_t>(quarter * 32) << 16);
    float* const acc = p.acc + b * p.acc_seq + g * p.acc_head;
    int u = 0;
    for (int i = 0; i < T; ++i) {
      const int key0 = key_of_tile(i);
      const int key = key0 + key_in_tile;
      const bool is_seen = seen(i);
      if (is_seen ? (u & 1) != wg : (i & 1) != wg) {  // the other group's tile
        u += is_seen;
        continue;
      }
      const bool reads = key < L - p.fresh && p.decay > 0.f;
      float sum = 0.f;
      const float old = reads ? acc[key] : 0.f;
      if (is_seen) {
        const int t = u >> 1;
        ++u;
        if (!ptx::mbar_wait_bounded(sfull(wg), t & 1, abort_flag, kWaitNs)) set_abort(abort_flag, a.status);
        ptx::tc_fence_after();
        const bool unmasked =
            key0 + kKeys <= pfx || (key0 >= lo_max && key0 + kKeys - 1 <= hi_min);  // uniform over the CTA
        const float fkey = static_cast<float>(key);
        for (int c0 = 0; c0 < p.n_mma; c0 += 16) {
          uint32_t r[16];
          MJ_TMEM_LD16(tmem_s + c0, r);
          ptx::tmem_ld_wait();
          if (c0 + 16 >= p.n_mma) {  // read whole: the next MMA may overwrite it
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sfree(wg));
          }
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(r[e]) * c1;
          if constexpr (kMod) {
            if (cap2 > 0.f) {
              float top = 0.f;
#pragma unroll
              for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[e]));
              if (__all_sync(0xffffffffu, top < kTanhSmall)) {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = cap2 * tanh_small(y[e]);
              } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = cap2 * tanh_any(y[e]);
              }
            }
            if (a.mod.slopes) {
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = fmaf(-row_slope2[c0 + e], fabsf(row_pos[c0 + e] - fkey), y[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float w = fast_exp2(y[e] - row_lse2[c0 + e]);
            if (unmasked) {
              sum += c0 + e < p.n_rows ? w : 0.f;
            } else {
              const bool vis = (key < pfx || (key >= row_lo[c0 + e] && key <= row_hi[c0 + e])) && c0 + e < p.n_rows;
              sum += vis ? w : 0.f;
            }
          }
        }
      }
      if (key < L && !*abort_flag) acc[key] = (reads ? p.decay * old : 0.f) + sum;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc(tmem, p.tmem_cols);
}

template <bool kQe4m3, bool kMod>
cudaError_t launch_kw(const KwArgs& p, const CUtensorMap& mk, size_t smem, cudaStream_t stream) {
  auto kern = key_weights_kernel<kQe4m3, kMod>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(p.d.num_work) * p.d.h_k, 1, 1), dim3(kThreads, 1, 1), smem, stream,
                    p, mk);
}

}  // namespace

cudaError_t launch_key_weights(const DecodeModDev& a, bool q_e4m3, bool has_mod, int n0, int n_rows, const float* lse,
                               float* acc, int64_t acc_seq, int64_t acc_head, float decay, int fresh,
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
  p.n_mma = (n_rows + 15) / 16 * 16;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * p.n_mma) p.tmem_cols *= 2;
  const int q_bytes = p.n_mma * 128 * (q_e4m3 ? 1 : 2);
  const int tail = 5 * kMaxRows * 4 + 8 * (2 * kMaxStages + 8) + 128;
  // two CTAs an SM when their shared memory and TMEM allow it
  const int limit = n_rows <= 128 ? 112 * 1024 : 224 * 1024;
  p.stages = (limit - 1024 - q_bytes - tail) / kTileBytes;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.off_q = p.stages * kTileBytes;
  p.off_row = p.off_q + q_bytes;
  p.off_bar = p.off_row + 5 * kMaxRows * 4;
  const size_t smem = 1024 + static_cast<size_t>(p.off_q) + q_bytes + tail;
  const int box_rows = a.page_size < kKeys ? a.page_size : kKeys;
  CUtensorMap mk;
  if (!make_kv_map(&mk, a.k, a.page_size, a.h_k, a.num_pages, a.k_row, a.k_head, a.k_page, box_rows, 1, a.kv_format))
    return cudaErrorInvalidValue;
  if (q_e4m3) return has_mod ? launch_kw<true, true>(p, mk, smem, stream) : launch_kw<true, false>(p, mk, smem, stream);
  return has_mod ? launch_kw<false, true>(p, mk, smem, stream) : launch_kw<false, false>(p, mk, smem, stream);
}

}  // namespace mj
