// Attention of whole prompts over the paged e4m3 cache (see mj_prompt_attn):
// many query rows a sequence, sequences of different lengths packed one behind
// the other, each against its own pages.
//
//   S[row, key] = Q[row] . K[key]         O[row, d] += P[row, key] V[key, d]
//
// A work item is 256 packed rows (token, head of the group) of one sequence
// and one kv head against its keys, 128 at a time: one read of a K and V tile
// serves two groups of 128 rows, a softmax warpgroup each.  Operands:
//   S   Q as hi + lo e4m3 parts (q 2^s = hi + lo, s by row) against the K codes
//       as they lie in the cache, kind::f8f6f4: K is never converted, and the
//       two parts cost what one bf16 product would
//   O   P in half precision from TMEM against V in half precision (every e4m3
//       value is one), kind::f16.  A converter warpgroup turns each V tile once
//       for both groups.  Splitting P into e4m3 parts instead would cost the
//       softmax threads four conversions a pair of scores for one, and keep 8
//       bits of P for 11 (trees of 244 rows by the query-rows kernel, which does
//       that: 593 us for 424 to 437 here).
//
// TMEM has room for both O (2 x 128 columns), both P (2 x 64) and one S of 128
// keys, which the groups use in turn: the softmax threads read a row of scores
// whole (128 registers of 184), after which the other group's scores take its
// place, while their exponentials run and the last tile's O product fills the
// gap.  Measured on a prompt of 20001 tokens, 32 heads: S, P and the next S of
// a group in the same 128 columns 3123 us (every product waits for the one
// before); two S of 64 keys a group 2611 (a product of 64 keys reads its Q
// operand from shared memory for half the work: 48 cycles for 32); this 2180
// to 2290, 1.43 to 1.50 PFLOP/s, 0.75 to 0.79 of what cuBLAS reaches.
//
// Up to 128 rows (decode tokens, a prompt's end) both groups hold the same rows
// and take the tiles in turn, each with a maximum, sum and O of its own, joined
// at the end: 1.05 us a tile for 1.65 of both groups' rows, 4.7 TB/s over 19
// tokens of 32769 keys, 8 heads.
//
// Bound, 256 rows: the tensor core needs 2048 cycles a tile, a tile takes about
// 2900.  The rest is the chain score product -> read -> maximum -> exponentials
// -> P -> O product, each step of it near 200 cycles of waits and arrivals
// (without the exponentials, the maximum or the conversions: 3 to 4 % less
// each).  Between items Q's conversion (about 5500 cycles a group, from its last
// score product on) and O's way out (5500) are hidden in part: about 12 thousand
// cycles an item of a prompt of 3000 tokens (384 to 400 us for five such, floor
// 218).  Measured and not kept: the first V tile ahead of Q 407 us; half of the
// next Q ahead of the last V tile 442; all of O read before any of it is written
// 412.  Changes of a few hundred instructions anywhere move each case by 3 % one
// way or the other: the loops are as large as the instruction caches.
//
// Roles (512 threads, one CTA an SM): warps 0-3 and 4-7 softmax of the two row
// groups (thread = row = TMEM lane) and O's way out; 8-11 Q and V conversion; 12
// issues the MMAs; 14 and 15 load K and V tiles by TMA, one box a page (13 idles).
// The CTA takes items in turns, forth and back through a list ordered by cost;
// the loads and conversions of an item run under the end of the one before it.
//
// Every wait is bounded: a role that gives up sets the abort flag and the
// status word, the others stop at their next wait, copies and MMAs in flight
// are drained and TMEM is freed.
//
// kTree: the same over a decode plan's work items (mj_decode_attn_tree): packed
// rows, context keys by a range and a prefix, the last keys a tree's nodes by
// the row's bits of the mask, spans.  Rows without a node compute too and are
// written as rows without a key.

#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mj_kernels.h"
#include "prompt.cuh"
#include "score_mod.cuh"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kRows = 128;               // rows of a group = MMA M; keys of a tile = MMA N
constexpr int kTile = 128 * 128;         // bytes of a K tile, a raw V tile, an e4m3 part of a group's Q
constexpr int kVfTile = 2 * kTile;       // a V tile in half precision
constexpr int kThreads = 512;
constexpr int kConvWarp = 8, kMmaWarp = 12, kKWarp = 14;
constexpr int kVf = 2;                   // converted V tiles held
constexpr int kTries = 1 << 22;          // of a wait: seconds, far above any legal one
constexpr uint64_t kDrainNs = 500000000ull;
constexpr int kStatusTimeout = 5;        // MJ_ERR_TIMEOUT
constexpr int kStatusInvalid = 1;        // MJ_ERR_INVALID_ARG
// P is 2^kPBias 2^(s - m): the reference m of a row moves only when a score
// passes it by kTau (log2 units), so P stays below 2^15, and an entry keeps
// half precision's 11 bits down to 2^-21 of the reference.
constexpr float kPBias = 7.f;
constexpr float kTau = 8.f;
// The least factor from scores to log2 units: one that had become 0 would turn a
// masked key's -inf into NaN.  A score of at most 2^25 is below 2^-100 by it, which
// adds nothing to a sum of exponentials.
constexpr float kLeastScale = 0x1p-126f;

template <bool kQe4m3>
struct Cfg {
  static constexpr int kParts = kQe4m3 ? 1 : 2;
  static constexpr int kSK = kQe4m3 ? 4 : 3, kSV = kQe4m3 ? 3 : 2;  // K and raw V rings
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kSK * kTile;
  static constexpr int kOffVf = kOffV + kSV * kTile;
  static constexpr int kOffQ = kOffVf + kVf * kVfTile;           // [group][part]
  static constexpr int kOffOut = kOffQ + 2 * kParts * kTile;     // [softmax warp] 32 rows x 64 bytes of O on their way out
  static constexpr int kOffShift = kOffOut + 8 * 2048;           // [group][2][128] s of each row
  static constexpr int kOffStat = kOffShift + 2 * 256;           // maximum and sum of the second group's rows
  static constexpr int kOffBar = kOffStat + 128 * 8;
  static constexpr int kBars = 2 * (kSK + kSV + kVf) + 1 + 6 * 2 + 2;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kBytes = kOffMisc + 16 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

__device__ __forceinline__ void give_up(volatile int* abort, int32_t* status) {
  *abort = 1;
  if (status) atomicExch(status, kStatusTimeout);
}

// chunk cc (16 bytes) of row r in a 128-byte-swizzled tile
__device__ __forceinline__ uint32_t swz(int r, int cc) { return r * 128 + ((cc ^ (r & 7)) << 4); }

// D (fp32, TMEM) += A (half precision, TMEM) B (half precision, shared memory)
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {  // of the magnitudes
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A row's scores of a tile over the cap: t = s c1 -> cap2 tanh(t), the cap in
// log2 units.  Where a warp's |t| are all below 0.45 (22 of a cap of 50) by an odd
// polynomial of degree 7 (fitted for this file; 1.3e-7 of the cap off, in fp32),
// two scores at a time; else tanh to fp32 precision for all of them.  One vote a
// tile, and nothing kept between the look at the magnitudes and the polynomial:
// a row's scores are 128 registers of 184.  (Prompts of 13500 tokens, 32 heads, a
// window of 1024 keys: 351 us, 250 without a cap, 418 by cap_scores, whose
// polynomial holds to 0.6 with two degrees more; 15 us an operation a pair of
// scores.)
__device__ __forceinline__ void cap_row(uint32_t (&s)[kRows], float c1, float cap2) {
  float top[4] = {};
#pragma unroll
  for (int e = 0; e < kRows; e += 2)
    top[(e >> 1) & 3] = fmax3_abs(top[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
  const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  if (__all_sync(0xffffffffu, fabsf(most * c1) < 0.45f)) {
    const float2 c12 = make_float2(c1, c1);
    const float c[4] = {9.999997550e-01f * cap2, -3.332945200e-01f * cap2, 1.323617008e-01f * cap2, -4.602166407e-02f * cap2};
#pragma unroll
    for (int e = 0; e < kRows; e += 2) {
      const float2 t = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c12);
      const float2 u = mul2(t, t);
      float2 p = make_float2(c[3], c[3]);
#pragma unroll
      for (int i = 2; i >= 0; --i) p = fma2(p, u, make_float2(c[i], c[i]));
      p = mul2(p, t);
      s[e] = __float_as_uint(p.x);
      s[e + 1] = __float_as_uint(p.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kRows; ++e) s[e] = __float_as_uint(tanh_any(__uint_as_float(s[e]) * c1) * cap2);
  }
}

// An item with, for a tree, the keys its sequence's rows see (score_mod.cuh):
// tile v of the plan's list is the sequence's tile v below the span's prefix
// tiles, then v + jump.
struct TreeItem : PromptItem {
  int4 span;
  int prefix_tiles, jump;
};

template <bool kTree>
__device__ __forceinline__ int tile_key(const std::conditional_t<kTree, TreeItem, PromptItem>& it, int t) {
  if constexpr (kTree)
    return (t < it.prefix_tiles ? t : t + it.jump) * kRows;
  else
    return t * kRows;
}

template <bool kQe4m3, bool kCap, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const std::conditional_t<kTree, PromptTreeDev, PromptDev> a, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v) {
  using C = Cfg<kQe4m3>;
  constexpr int SK = C::kSK, SV = C::kSV;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  using Item = std::conditional_t<kTree, TreeItem, PromptItem>;
  int units;
  if constexpr (kTree) {
    units = a.t.num_work * a.n_q_tiles * a.h_k;
  } else {
    if (!prompt_plan_fits(a)) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && a.status) atomicExch(a.status, kStatusInvalid);
      return;
    }
    units = a.head->n_items * a.h_k;
  }
  if (static_cast<int>(blockIdx.x) >= units) return;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(sm);
  int8_t* const q_shift = reinterpret_cast<int8_t*>(sm + C::kOffShift);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const uint32_t bar0 = sbase + C::kOffBar;
  auto kfull = [&](int s) { return bar0 + 8u * s; };
  auto kempty = [&](int s) { return bar0 + 8u * (SK + s); };
  auto vfull = [&](int s) { return bar0 + 8u * (2 * SK + s); };
  auto vempty = [&](int s) { return bar0 + 8u * (2 * SK + SV + s); };
  auto ffull = [&](int s) { return bar0 + 8u * (2 * SK + 2 * SV + s); };   // converted V
  auto fempty = [&](int s) { return bar0 + 8u * (2 * SK + 2 * SV + kVf + s); };
  constexpr int kB = 2 * (SK + SV + kVf);
  const uint32_t sread = bar0 + 8u * kB;  // either group's scores read
  // of each group: 0 scores written, 1 P written, 2 a tile's product done, 3 O
  // read out, 4 Q laid out, 5 Q read
  auto gbar = [&](int w, int k) { return bar0 + 8u * (kB + 1 + 6 * w + k); };
  const uint32_t drain = bar0 + 8u * (kB + 13), stats = drain + 8u;  // stats: the second group's row statistics written

  if (tid == 0) {
    for (int s = 0; s < SK; ++s) {
      ptx::mbar_init(kfull(s), 1);
      ptx::mbar_init(kempty(s), 1);
    }
    for (int s = 0; s < SV; ++s) {
      ptx::mbar_init(vfull(s), 1);
      ptx::mbar_init(vempty(s), 4);
    }
    for (int s = 0; s < kVf; ++s) {
      ptx::mbar_init(ffull(s), 4);
      ptx::mbar_init(fempty(s), 1);
    }
    ptx::mbar_init(sread, 4);
    for (int w = 0; w < 2; ++w) {
      for (int k = 0; k < 6; ++k) ptx::mbar_init(gbar(w, k), k == 1 || k == 3 || k == 4 ? 4 : 1);
    }
    ptx::mbar_init(drain, 1);
    ptx::mbar_init(stats, 4);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(sbase + C::kOffMisc, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // columns: the scores of either group (128), each group's P (64), each group's O (128)
  const uint32_t tmem = *tmem_slot;
  auto p_col = [&](int w) { return 128u + 64u * w; };
  auto o_col = [&](int w) { return 256u + 128u * w; };

  auto wait = [&](uint32_t bar, uint32_t parity) { return ptx::mbar_wait_tries(bar, parity, abort_flag, kTries); };
  // the CTA's k-th unit: forth and back through the list (longest first)
  const int G = gridDim.x, me = blockIdx.x;
  auto unit_at = [&](int k) { return k * G + ((k & 1) ? G - 1 - me : me); };
  auto load_item = [&](int u) {
    Item it;
    if constexpr (kTree) {
      const int rest = u / a.h_k;
      const int4 w = reinterpret_cast<const int4*>(a.t.work)[rest / a.n_q_tiles];
      it.b = w.x;
      it.t0 = w.y;
      it.t1 = w.z;
      it.row0 = rest % a.n_q_tiles * kPromptRows;
      it.len = a.t.seq_lens[w.x];
      it.part = a.t.n_splits[w.x] > 1 ? w.w : -1;
      it.tok0 = 0;
      it.n_tok = a.t.q_len;
#pragma unroll
      for (int w2 = 0; w2 < 2; ++w2) {
        it.g0[w2] = it.t0;
        it.g1[w2] = it.row0 + w2 * kRows < a.t.n_q ? it.t1 : it.t0;
      }
      if (it.row0 + kRows >= a.t.n_q && it.t1 - it.t0 >= 2) it.g1[1] = -1;
      it.span = make_int4(it.len, 0, it.len, 0);
      it.prefix_tiles = it.jump = 0;
      if (a.t.mod.spans) {
        it.span = a.t.mod.spans[w.x];
        it.span.z = min(it.span.z, it.len);
        it.prefix_tiles = (it.span.x + kRows - 1) / kRows;
        it.jump = max(it.span.y / kRows - it.prefix_tiles, 0);
      }
    } else {
      const int4* src = reinterpret_cast<const int4*>(a.items + u / a.h_k);
#pragma unroll
      for (int i = 0; i < 3; ++i) reinterpret_cast<int4*>(&it)[i] = src[i];
    }
    return it;
  };
  // A warpgroup's share of the launch's 512 x 128 registers: 2 x 184 + 88 + 56
  // = 4 x 128 (the softmax threads hold 128 scores).  All four warps of a
  // warpgroup execute the same instruction.
  if (warp >= kMmaWarp)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  else if (warp >= kConvWarp)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");

  if (warp >= kKWarp) {
    // ------------------------------------------------------------- TMA loads
    const bool is_k = warp == kKWarp;
    const int NS = is_k ? SK : SV;
    const uint32_t ring = sbase + (is_k ? C::kOffK : C::kOffV);
    const CUtensorMap* const tmap = is_k ? &tmap_k : &tmap_v;
    auto full = [&](int s) { return is_k ? kfull(s) : vfull(s); };
    auto empty = [&](int s) { return is_k ? kempty(s) : vempty(s); };
    const int PS = a.page_size;
    const int nbox = kRows / PS;  // pages of a tile
    if (lane == 0) ptx::prefetch_tmap(tmap);
    const bool evict_first = a.kv_evict_first != 0;
    const uint64_t policy = ptx::policy_evict_first();
    int n = 0;  // tiles issued
    bool ok = true;
    for (int k = 0; ok && unit_at(k) < units; ++k) {
      const int u = unit_at(k), g = u % a.h_k;
      const Item it = load_item(u);
      const int64_t table = static_cast<int64_t>(it.b) * a.max_blocks;
      // lane l loads the tile's l-th page; its table entry comes a tile ahead (a
      // tree's length is the device's, which may pass its table: the plan reports that)
      auto page_of = [&](int t) {
        const int key = tile_key<kTree>(it, t) + lane * PS;
        bool there = t < it.t1 && lane < nbox && key < it.len;
        if constexpr (kTree) there = there && key / PS < a.max_blocks;
        return there ? a.block_table[table + key / PS] : a.num_pages;
      };
      int page = page_of(it.t0);
      for (int t = it.t0; t < it.t1; ++t, ++n) {
        const int st = n % NS;
        const int next = page_of(t + 1);
        if (n >= NS && !wait(empty(st), ((n / NS) - 1) & 1)) ok = false;
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(full(st), kTile);
        __syncwarp();
        if (lane < nbox)
          ptx::tma_load_kv(ring + st * kTile + lane * PS * 128, tmap, full(st), 0, 0, g, page, evict_first, policy);
        page = next;
      }
    }
    if (!ok) {
      if (lane == 0) {
        give_up(abort_flag, a.status);
        volatile int never = 0;
        for (int i = n > NS ? n - NS : 0; i < n; ++i)
          ptx::mbar_wait_bounded(full(i % NS), (i / NS) & 1, &never, kDrainNs);
      }
    } else if (*abort_flag && lane == 0) {
      volatile int never = 0;
      for (int i = n > NS ? n - NS : 0; i < n; ++i)
        ptx::mbar_wait_bounded(full(i % NS), (i / NS) & 1, &never, kDrainNs);
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------------- MMA
    // One warp issues everything, in the order S_0(t), O_0(t - 1), S_1(t),
    // O_1(t - 1): a group's O product runs while its new scores are read, after
    // which the other group's scores take their place.  The whole warp goes
    // through the loop and computes descriptors, addresses and phases, so that
    // they lie in uniform registers; one lane waits and issues (with the
    // arithmetic in its branch each MMA took 118 cycles to issue, with all
    // lanes waiting a wait took 200).
    if (warp == kMmaWarp) {
      const bool leader = ptx::elect_one() != 0;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t idesc_s = ptx::idesc_e4m3(kRows, kRows, false, false);
      const uint32_t idesc_o = ptx::idesc_e4m3(kRows, kRows, false, true);  // formats 0: half precision in kind::f16
      const uint64_t qdesc = ptx::smem_desc(sbase + C::kOffQ, 16, 1024, ptx::kSwizzle128B);
      const uint64_t kdesc = ptx::smem_desc(sbase + C::kOffK, 16, 1024, ptx::kSwizzle128B);
      // V, d-major: 64 elements of d a 128-byte row, the other 64 a tile half further
      const uint64_t vdesc = ptx::smem_desc(sbase + C::kOffVf, kTile, 1024, ptx::kSwizzle128B);
      auto scores = [&](int w, uint64_t kd) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int part = 0; part < C::kParts; ++part)
            ptx::mma_e4m3(tm, qdesc + static_cast<uint32_t>((w * C::kParts + part) * (kTile >> 4) + 2 * kk), kd + 2 * kk, idesc_s,
                          kk > 0 || part > 0);
      };
      auto output = [&](int w, uint64_t vd, uint32_t more) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // 16 keys: 8 columns of P, 16 rows of V
          mma_f16_ts(tm + o_col(w), tm + p_col(w) + 8 * kk, vd + 128 * kk, idesc_o, kk > 0 ? 1u : more);
      };
      uint32_t ks = 0, kph = 0, vs = 0, vph = 0;  // stage and phase of the next K and converted V tile
      uint32_t sph = 1;                           // of the scores read (none to wait for at first)
      uint32_t qph = 0, pph = 0, oph = 3;         // bit w: of group w's Q, its P, and its O read out (likewise)
      for (int k = 0; unit_at(k) < units; ++k) {
        const Item it = load_item(unit_at(k));
        const int t0 = __shfl_sync(0xffffffffu, it.t0, 0), t1 = __shfl_sync(0xffffffffu, it.t1, 0);
        if (t1 <= t0) continue;
        int g0[2], g1[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          g0[w] = __shfl_sync(0xffffffffu, it.g0[w], 0);
          g1[w] = __shfl_sync(0xffffffffu, it.g1[w], 0);
        }
        bool ok = true;
        if (g1[1] < 0) {
          // both groups hold the same rows and take the tiles in turn: scores of
          // tile t, O of tile t - 2 (of the same group, whose next scores these are)
          for (int t = t0; t < t1 + 2; ++t) {
            const int w = (t - t0) & 1;
            const uint32_t sc = gbar(w, 0), pf = gbar(w, 1), pd = gbar(w, 2);
            if (t < t1) {
              const uint64_t kd = kdesc + ks * (kTile >> 4);
              if (leader) {
                ok &= wait(kfull(ks), kph);
                if (t < t0 + 2) ok &= wait(gbar(w, 4), (qph >> w) & 1);
                ok &= wait(sread, sph);
                ptx::tc_fence_after();
                scores(w, kd);
                ptx::mma_commit(sc);
                ptx::mma_commit(kempty(ks));
                if (t + 2 >= t1) ptx::mma_commit(gbar(w, 5));
              }
              __syncwarp();
              sph ^= 1;
              if (t < t0 + 2) qph ^= 1u << w;
              if (++ks == SK) {
                ks = 0;
                kph ^= 1;
              }
            }
            if (t >= t0 + 2) {
              const uint64_t vd = vdesc + vs * (kVfTile >> 4);
              const uint32_t more = t >= t0 + 4;
              if (leader) {
                ok &= wait(ffull(vs), vph);
                ok &= wait(pf, (pph >> w) & 1);
                if (!more) ok &= wait(gbar(w, 3), (oph >> w) & 1);
                ptx::tc_fence_after();
                output(w, vd, more);
                ptx::mma_commit(pd);
                ptx::mma_commit(fempty(vs));
              }
              __syncwarp();
              pph ^= 1u << w;
              if (!more) oph ^= 1u << w;
              if (++vs == kVf) {
                vs = 0;
                vph ^= 1;
              }
            }
          }
          if (leader && !ok) give_up(abort_flag, a.status);
          if (__any_sync(0xffffffffu, !ok)) break;
          continue;
        }
        const int t_all = (g0[0] > g0[1] ? g0[0] : g0[1]) + 1, t_end = (g1[0] < g1[1] ? g1[0] : g1[1]) - 1;
        for (int t = t0; t <= t1; ++t) {  // scores of tile t, O of tile t - 1
          const uint64_t kd = kdesc + ks * (kTile >> 4), vd = vdesc + vs * (kVfTile >> 4);
          // Most tiles: all four products, none of them an item's first or last.
          // (The instructions between two products are on the critical path.)
          if (t > t_all && t < t_end) {
            const uint32_t kf = kfull(ks), ke = kempty(ks), vf = ffull(vs), ve = fempty(vs);
            const uint32_t p0 = pph & 1, p1 = pph >> 1;
            const uint32_t ks_next = ks + 1 == SK ? 0 : ks + 1, vs_next = vs + 1 == kVf ? 0 : vs + 1;
            if (leader) {
              ok &= wait(kf, kph) & wait(sread, sph);
              ptx::tc_fence_after();
              scores(0, kd);
              ptx::mma_commit(gbar(0, 0));
              ok &= wait(vf, vph) & wait(gbar(0, 1), p0);
              ptx::tc_fence_after();
              output(0, vd, 1u);
              ptx::mma_commit(gbar(0, 2));
              ok &= wait(sread, sph ^ 1);
              ptx::tc_fence_after();
              scores(1, kd);
              ptx::mma_commit(gbar(1, 0));
              ptx::mma_commit(ke);
              ok &= wait(gbar(1, 1), p1);
              ptx::tc_fence_after();
              output(1, vd, 1u);
              ptx::mma_commit(gbar(1, 2));
              ptx::mma_commit(ve);
            }
            __syncwarp();
            pph ^= 3;
            kph ^= ks_next == 0;
            vph ^= vs_next == 0;
            ks = ks_next;
            vs = vs_next;
            continue;
          }
          const bool load_k = t < t1, load_v = t > t0;
          if (load_k && leader) ok &= wait(kfull(ks), kph);
          __syncwarp();
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (t >= g0[w] && t < g1[w]) {
              if (leader) {
                if (t == g0[w]) ok &= wait(gbar(w, 4), (qph >> w) & 1);
                ok &= wait(sread, sph);
                ptx::tc_fence_after();
                scores(w, kd);
                ptx::mma_commit(gbar(w, 0));
                if (t + 1 == g1[w]) ptx::mma_commit(gbar(w, 5));  // the item's Q is read
              }
              __syncwarp();
              sph ^= 1;
              if (t == g0[w]) qph ^= 1u << w;
            }
            if (w == 1 && load_k && leader) ptx::mma_commit(kempty(ks));
            __syncwarp();
            if (t > g0[w] && t <= g1[w]) {
              const uint32_t more = t > g0[w] + 1;
              if (leader) {
                ok &= wait(ffull(vs), vph);  // (the same phase for both groups)
                ok &= wait(gbar(w, 1), (pph >> w) & 1);
                if (!more) ok &= wait(gbar(w, 3), (oph >> w) & 1);  // O read out
                ptx::tc_fence_after();
                output(w, vd, more);
                ptx::mma_commit(gbar(w, 2));
              }
              __syncwarp();
              pph ^= 1u << w;
              if (!more) oph ^= 1u << w;
            }
          }
          if (load_v && leader) {
            ok &= wait(ffull(vs), vph);  // (also where no group's rows see the tile)
            ptx::mma_commit(fempty(vs));
          }
          __syncwarp();
          if (load_k && ++ks == SK) {
            ks = 0;
            kph ^= 1;
          }
          if (load_v && ++vs == kVf) {
            vs = 0;
            vph ^= 1;
          }
        }
        if (leader && !ok) give_up(abort_flag, a.status);
        if (__any_sync(0xffffffffu, !ok)) break;
      }
      if (leader) {
        ptx::mma_commit(drain);
        volatile int never = 0;
        ptx::mbar_wait_bounded(drain, 0, &never, kDrainNs);
      }
      __syncwarp();
    }
  } else if (warp >= kConvWarp) {
    // ------------------------------------------------ Q and V conversion
    const int cw = warp - kConvWarp;
    int n = 0;
    uint32_t q_items[2] = {0, 0};  // items of each group
    bool ok = true;
    for (int k = 0; ok && unit_at(k) < units; ++k) {
      const int u = unit_at(k), g = u % a.h_k;
      const Item it = load_item(u);
      if (it.t1 <= it.t0) continue;
      // ---- a V tile: this warp turns 32 keys, four rows a load, 16 codes a lane
      auto convert = [&](int t) {
        const int st = n % SV, vf = n % kVf;
        if (!wait(vfull(st), (n / SV) & 1) || (n >= kVf && !wait(fempty(vf), ((n / kVf) - 1) & 1))) ok = false;
        if (__any_sync(0xffffffffu, !ok)) return false;
        const uint8_t* const src = sm + C::kOffV + st * kTile;
        const int key0 = tile_key<kTree>(it, t);
        uint8_t* const dst = sm + C::kOffVf + vf * kVfTile;
        const int cc = lane & 7;
        // (the roles' code contends for the instruction caches: unrolled whole, five
        // prompts take 397 us, so 384)
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          const int r = cw * 32 + i * 4 + (lane >> 3);
          uint4 x = *reinterpret_cast<const uint4*>(src + swz(r, cc));
          const int key = key0 + r;
          bool dead = key >= it.len;
          if constexpr (kTree) dead = key >= it.span.z || (key >= it.span.x && key < it.span.y);
          if (dead) x = make_uint4(0u, 0u, 0u, 0u);  // 0 x what lies there must not reach O
          const uint32_t v4[4] = {x.x, x.y, x.z, x.w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h[2 * e] = e4m3x2_to_f16x2(static_cast<uint16_t>(v4[e] & 0xFFFFu));
            h[2 * e + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(v4[e] >> 16));
          }
          // codes 16 cc ..: chunks 2 (cc % 4) and the next of half cc / 4; the
          // halves' lanes take theirs in opposite order (they share banks)
          uint8_t* const half = dst + (cc >> 2) * kTile;
          const int c0 = 2 * (cc & 3), flip = cc >> 2;
          *reinterpret_cast<uint4*>(half + swz(r, c0 + flip)) =
              flip ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(half + swz(r, c0 + 1 - flip)) =
              flip ? make_uint4(h[0], h[1], h[2], h[3]) : make_uint4(h[4], h[5], h[6], h[7]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(ffull(vf));
          ptx::mbar_arrive(vempty(st));
        }
        ++n;
        return true;
      };
      // ---- Q: this warp lays out 32 of a group's 128 rows, eight lanes a row
      // (a lane 16 elements: one 16-byte chunk of each part), four rows a turn
      constexpr int kVecs = kQe4m3 ? 1 : 2;  // 16-byte loads a lane and row
      constexpr int kBatch = 4;              // turns in flight
      const int piece = lane & 7;
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        const bool dual = it.g1[1] < 0;
        if (!dual && (w ? it.g1[1] : it.g1[0]) <= (w ? it.g0[1] : it.g0[0])) continue;
        const int r0 = cw * 32 + (lane >> 3);  // this lane's rows of the group: r0, r0 + 4, ..
        const int first = it.row0 + (dual ? 0 : w * kRows) + r0;
        int left = it.n_tok * a.h_r - first;  // rows there are from this one on
        const int tok = first / a.h_r;
        int hr = first - tok * a.h_r;
        constexpr int kEl = kQe4m3 ? 1 : 2;
        // (a lane without a row of its own reads the item's first one)
        const uint8_t* const valid = static_cast<const uint8_t*>(a.q) + piece * 16 * kEl +
                                     prompt_at(a.q_rows, it.b, it.tok0 + it.row0 / a.h_r, g, it.row0 % a.h_r) * kEl;
        const uint8_t* at = static_cast<const uint8_t*>(a.q) + piece * 16 * kEl + prompt_at(a.q_rows, it.b, it.tok0 + tok, g, hr) * kEl;
        const int64_t step_h = 4 * a.q_rows.s_h * kEl, step_t = (a.q_rows.s_tok - a.h_r * a.q_rows.s_h) * kEl;
        const uint32_t turn = w ? q_items[1]++ : q_items[0]++;
        int8_t* const shifts = q_shift + (2 * w + (turn & 1)) * 128;
        uint8_t* const part = sm + C::kOffQ + w * C::kParts * kTile;
#pragma unroll 1
        for (int l0 = 0; l0 < 8; l0 += kBatch) {
          uint4 raw[kBatch][kVecs];
          uint32_t there = 0;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const uint4* const src = reinterpret_cast<const uint4*>(left > 0 ? at : valid);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) raw[i][v] = __ldg(src + v);
            there |= (left > 0 ? 1u : 0u) << i;
            left -= 4;
            at += step_h;
            for (hr += 4; hr >= a.h_r; hr -= a.h_r) at += step_t;
          }
          if (l0 == 0) {
            if (turn > 0 && !wait(gbar(w, 5), (turn - 1) & 1)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
              ok = false;
              break;
            }
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + (l0 + i) * 4;
            const uint32_t keep = (there >> i) & 1u ? 0xFFFFFFFFu : 0u;
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
              raw[i][v] = make_uint4(raw[i][v].x & keep, raw[i][v].y & keep, raw[i][v].z & keep, raw[i][v].w & keep);
            if constexpr (kQe4m3) {
              *reinterpret_cast<uint4*>(part + swz(r, piece)) = raw[i][0];
            } else {
              // the row's largest |q| goes to [128, 256).  Half precision then
              // holds every element's 8 bits down to 2^-22 of it; hi = e4m3(x),
              // lo = e4m3(x - hi), the difference exact: hi + lo is within 2^-10
              const uint32_t v8[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                                      raw[i][kVecs - 1].x, raw[i][kVecs - 1].y, raw[i][kVecs - 1].z, raw[i][kVecs - 1].w};
              uint32_t m2[8];  // pairs of magnitudes
#pragma unroll
              for (int e = 0; e < 8; ++e) m2[e] = v8[e] & 0x7FFF7FFFu;
#pragma unroll
              for (int o = 4; o >= 1; o >>= 1)
#pragma unroll
                for (int e = 0; e < o; ++e) m2[e] = __vmaxu2(m2[e], m2[e + o]);
#pragma unroll
              for (int o = 4; o >= 1; o >>= 1) m2[0] = __vmaxu2(m2[0], __shfl_xor_sync(0xffffffffu, m2[0], o));
              const uint32_t top = max(m2[0] & 0xFFFFu, m2[0] >> 16);
              int shift = 134 - static_cast<int>(top >> 7);  // 7 - exponent
              shift = top == 0 ? 0 : (shift > 126 ? 126 : (shift < -126 ? -126 : shift));
              const float qs = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
              uint32_t hw[4], lw[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                uint32_t e2[2], l2[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t z = v8[2 * h + y];
                  const float2 x = mul2(make_float2(__uint_as_float(z << 16), __uint_as_float(z & 0xFFFF0000u)), make_float2(qs, qs));
                  const uint32_t x2 = f32x2_to_f16x2(x.x, x.y);
                  const uint16_t hi = f16x2_to_e4m3x2(x2);
                  e2[y] = hi;
                  l2[y] = f16x2_to_e4m3x2(sub_f16x2(x2, e4m3x2_to_f16x2(hi)));
                }
                hw[h] = e2[0] | (e2[1] << 16);
                lw[h] = l2[0] | (l2[1] << 16);
              }
              *reinterpret_cast<uint4*>(part + swz(r, piece)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
              *reinterpret_cast<uint4*>(part + kTile + swz(r, piece)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
              if (piece == 0) shifts[r] = static_cast<int8_t>(shift);
            }
          }
        }
        if (!ok) break;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(gbar(w, 4));
      }
      if (!ok) break;
      ok = convert(it.t0);
      if (!ok) break;
      // the next item's Q is on its way to L2 meanwhile
      if (unit_at(k + 1) < units) {
        const int u2 = unit_at(k + 1);
        const Item nx = load_item(u2);
        constexpr int kLines = kQe4m3 ? 1 : 2;  // of 128 bytes a row
#pragma unroll 1
        for (int i = cw * 32 + lane; i < kPromptRows * kLines; i += 128) {
          const int row = nx.row0 + i / kLines, tok = row / a.h_r;
          if (row < nx.n_tok * a.h_r) {
            const int64_t at = prompt_at(a.q_rows, nx.b, nx.tok0 + tok, u2 % a.h_k, row - tok * a.h_r);
            const uint8_t* const line = static_cast<const uint8_t*>(a.q) + at * (kQe4m3 ? 1 : 2) + (i % kLines) * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
          }
        }
      }
      for (int t = it.t0 + 1; ok && t < it.t1; ++t) ok = convert(t);
    }
    if (!ok && lane == 0) give_up(abort_flag, a.status);
  } else {
    // --------------------------------------------------------------- softmax
    const int w = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row of the group = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off, tp = ts + p_col(w), to = ts + o_col(w);
    int q = 0, items = 0, duals = 0;  // the group's tiles and items, and those it shares
    // a wait that gives up sets the abort flag and the loop runs on (later waits
    // return at once), so that a warp's lanes stay together
    for (int k = 0; unit_at(k) < units; ++k) {
      // the threads hold 128 scores: what only an item's ends need is looked up
      // again there, so that it takes no register in between
      auto unit = [&] {
        int u = unit_at(k);
        asm volatile("" : "+r"(u));
        return u;
      };
      int g0 = 0, g1 = 0, lo = 0, lim = INT32_MAX;  // the group's tiles; the row sees keys lo .. lim
      bool dual;                                    // both groups hold these rows and take turns
      int pfx = 0, prefix_tiles = 0, jump = 0;      // kTree: and those below pfx, and nodes by its mask
      // reference maximum (in units of the scores as read), sum of 2^kPBias p,
      // score -> log2 units, or over the cap (less the shift of the row's Q, which
      // is not known yet)
      float m_run = -INFINITY, l_run = 0.f, c2 = 1.f, cap_c1 = 0.f;
      {
        const int u = unit(), g = u % a.h_k;
        const Item it = load_item(u);
        const float raw_l = a.softmax_scale * a.qd[it.b * a.qd_seq + g * a.qd_head] * a.kd[it.b * a.kd_seq + g * a.kd_head];
        if constexpr (kCap)  // scores become logits in log2 units as they are read
          cap_c1 = raw_l / a.softcap;
        else
          c2 = kQe4m3 ? fmaxf(raw_l * kLog2e, kLeastScale) : raw_l * kLog2e;
        dual = it.g1[1] < 0;
        g0 = dual ? it.t0 + w : (w ? it.g0[1] : it.g0[0]);
        g1 = dual ? it.t1 : (w ? it.g1[1] : it.g1[0]);
        if constexpr (kTree) {
          if (it.t1 <= it.t0) continue;  // padding of the work list
          prefix_tiles = it.prefix_tiles;
          jump = it.jump;
        }
        const int row = it.row0 + (dual ? 0 : w * kRows) + r;  // (rows past the last compute what nobody reads)
        if (row < it.n_tok * a.h_r) {
          const int tok = row / a.h_r;
          if constexpr (kTree) {
            const TreeShape tree = tree_shape(a.t, it.b, it.len);
            if (tok < tree.nodes) {  // (rows without a node compute too, and are written as rows without a key)
              const RowRange rr = tree_range(a.t, it.b, tok, tree.ctx);
              if (!tree_span_holds(it.span, rr, tree) && a.status) atomicExch(a.status, kStatusInvalid);
              lim = min(rr.hi, it.span.z - 1);
              lo = max(rr.lo, it.span.y);
              pfx = min(rr.pfx, it.span.x);
            }
          } else {
            prompt_range(it.len, it.n_tok, tok, tok, a.causal, a.window, &lo, &lim);
          }
        }
      }
      for (int t = g0; t < g1; t += dual ? 2 : 1, ++q) {
        const int key0 = kTree ? (t < prefix_tiles ? t : t + jump) * kRows : t * kRows;
        if (!wait(gbar(w, 0), q & 1)) give_up(abort_flag, a.status);
        ptx::tc_fence_after();
        if (!kQe4m3 && t == g0) {  // the row's shift is there since its Q was laid out
          const float f = __uint_as_float(static_cast<uint32_t>(127 - q_shift[(2 * w + (items & 1)) * 128 + r]) << 23);
          if constexpr (kCap)
            cap_c1 *= f;
          else
            c2 = fmaxf(c2 * f, kLeastScale);
        }
        const bool unmasked = __all_sync(0xffffffffu, (key0 >= lo && key0 + kRows - 1 <= lim) || (kTree && key0 + kRows <= pfx));
        uint32_t s[kRows];
#pragma unroll
        for (int c = 0; c < kRows; c += 16) MJ_TMEM_LD16(ts + c, (s + c));
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(sread);  // the other group's scores may come
        if constexpr (kCap) cap_row(s, cap_c1, a.softcap * kLog2e);
        if (!unmasked) {
          const int e0 = lo - key0, e1 = lim - key0;
          if constexpr (kTree) {  // (few tiles: the row's node is looked up again)
            uint32_t bits[4] = {};
            const Item it = load_item(unit());
            const int row = it.row0 + (dual ? 0 : w * kRows) + r;
            if (row < it.n_tok * a.h_r) {
              const int tok = row / a.h_r;
              const TreeShape tree = tree_shape(a.t, it.b, it.len);
              if (tok < tree.nodes) {
                const uint32_t* const mask = a.t.mask + (static_cast<int64_t>(it.b) * a.t.q_len + tok) * a.t.mask_words;
#pragma unroll
                for (int i = 0; i < 4; ++i) bits[i] = tree_bits(mask, tree.nodes, key0 + 32 * i - tree.ctx);
              }
            }
            const int e2 = pfx - key0;
#pragma unroll
            for (int e = 0; e < kRows; ++e)
              s[e] = (e >= e0 && e <= e1) || e < e2 || ((bits[e >> 5] >> (e & 31)) & 1u) != 0 ? s[e] : 0xFF800000u;
          } else {
#pragma unroll
            for (int e = 0; e < kRows; ++e) s[e] = e >= e0 && e <= e1 ? s[e] : 0xFF800000u;  // -inf
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kRows; e += 2)
          m4[(e >> 1) & 3] = fmax3(m4[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const bool moved = (mt - m_run) * c2 > kTau;  // from -inf too; -inf after -inf is NaN: no
        // the tile before is added up: its P and O are free
        if (q > 0 && !wait(gbar(w, 2), (q - 1) & 1)) give_up(abort_flag, a.status);
        ptx::tc_fence_after();
        if (__any_sync(0xffffffffu, moved)) {
          const float m_new = moved ? mt : m_run;
          const float corr = moved ? fast_exp2((m_run - m_new) * c2) : 1.f;  // 0 for a row that had seen no key
          l_run *= corr;
          m_run = m_new;
          if (t > g0) {  // a warp corrects O when any of its rows moved
#pragma unroll 1
            for (int h0 = 0; h0 < kRows; h0 += 16) {
              uint32_t o[16];
              MJ_TMEM_LD16(to + h0, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              MJ_TMEM_ST16(to + h0, o);
            }
          }
        }
        // P, two keys a column
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        const float bias = fmaf(-mu, c2, kPBias);
        const float2 c22 = make_float2(c2, c2), bias2 = make_float2(bias, bias);
        float2 sum2[4] = {};
#pragma unroll
        for (int p0 = 0; p0 < 64; p0 += 16) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int e = 2 * (p0 + i);
            const float2 y = fma2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c22, bias2);
            const float2 x = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum2[i & 3] = add2(sum2[i & 3], x);
            p[i] = f32x2_to_f16x2(x.x, x.y);
          }
          MJ_TMEM_ST16(tp + p0, p);
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(gbar(w, 1));
        const float2 all = add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3]));
        l_run += all.x + all.y;
      }
      if (g1 > g0) ++items;
      // ---- epilogue: O, or its part, of this group's rows
      const bool any = g1 > g0;
      // (what does not depend on O is looked up while the last product runs)
      const int u = unit(), g = u % a.h_k;
      const Item it = load_item(u);
      const int row = it.row0 + (dual ? 0 : w * kRows) + r;
      const bool live = row < it.n_tok * a.h_r;
      const int tok = live ? row / a.h_r : 0;
      const int hr = live ? row - tok * a.h_r : 0;
      const bool final_out = it.part < 0;
      const float vd = a.vd[it.b * a.vd_seq + g * a.vd_head];
      int64_t part_row;
      if constexpr (kTree)
        part_row = mj::part_row(a.t, it.b, g, it.part, live ? row : 0);
      else
        part_row = (static_cast<int64_t>(it.part) * a.h_k + g) * kPromptRows + w * kRows + r;
      const int64_t orow = final_out ? prompt_at(a.o_rows, it.b, it.tok0 + tok, g, hr) : part_row * kHeadDimDev;
      uint8_t* dst[4];
      bool on[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 8 * j + (lane >> 2);
        const int64_t at = __shfl_sync(0xffffffffu, orow, i);
        on[j] = __shfl_sync(0xffffffffu, static_cast<int>(live), i) != 0;
        dst[j] = (final_out ? reinterpret_cast<uint8_t*>(a.o + at) : reinterpret_cast<uint8_t*>(a.o_part + at)) + (lane & 3) * 16;
      }
      if (any && !wait(gbar(w, 2), (q - 1) & 1)) give_up(abort_flag, a.status);
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;  // nothing is written out after that
      // The second group's row statistics go to the first one, which reads both O
      // (and gives them free with O, without which no later item's are written;
      // the second group may be writing out an item without keys by then).
      float* const stat = reinterpret_cast<float*>(sm + C::kOffStat) + 2 * r;
      float m1 = -INFINITY, l1 = 0.f;
      if (dual) {
        if (w == 1) {
          *reinterpret_cast<float2*>(stat) = make_float2(m_run, l_run);
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(stats);
          continue;
        }
        if (!wait(stats, duals & 1)) give_up(abort_flag, a.status);
        if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        ++duals;
        const float2 x = *reinterpret_cast<const float2*>(stat);
        m1 = x.x;
        l1 = x.y;
      }
      ptx::tc_fence_after();
      const float mx = fmaxf(m_run, m1);
      const float f0 = m_run == -INFINITY ? 0.f : fast_exp2((m_run - mx) * c2), f1 = m1 == -INFINITY ? 0.f : fast_exp2((m1 - mx) * c2);
      m_run = mx;
      float l = (l_run * f0 + l1 * f1) * (1.f / 128.f);  // 2^-kPBias
      bool seen = m_run > -INFINITY;
      if constexpr (kTree) seen = seen && tok < tree_shape(a.t, it.b, it.len).nodes;
      float f = vd * (1.f / 128.f) * (final_out ? a.scale_o / (seen ? l : 1.f) : 1.f);
      if (kTree && !seen) l = f = 0.f;
      const float fa = f * f0, fb = f * f1;  // of this group's O and, where rows are shared, of the other's
      // A lane holds a row; the rows leave through shared memory, 64 bytes of each
      // at a time, as pieces of four lanes (16 bytes a lane and row would be 32
      // half-used sectors an instruction): 16-byte chunk c of row i at chunk
      // c ^ (i / 2 % 4) of its 64 bytes
      uint8_t* const out = sm + C::kOffOut + warp * 2048;
      uint8_t* const mine = out + lane * 64;
      auto emit = [&](const uint4 (&v)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(mine + ((c ^ ((lane >> 1) & 3)) << 4)) = v[c];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 8 * j + (lane >> 2);
          const uint4 y = *reinterpret_cast<const uint4*>(out + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
          if (on[j]) *reinterpret_cast<uint4*>(dst[j]) = y;
          dst[j] += 64;
        }
        __syncwarp();
      };
      // (a row that saw no key of the group's tiles has O = 0 there; a group
      // without tiles has nothing in its columns)
#pragma unroll 1
      for (int h0 = 0; h0 < kRows; h0 += 32) {
        uint32_t o[32];
        if (any) {
          MJ_TMEM_LD16(to + h0, o);
          MJ_TMEM_LD16(to + h0 + 16, (o + 16));
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fa);
        if (dual) {
          uint32_t o1[32];
          MJ_TMEM_LD16(ts + o_col(1) + h0, o1);
          MJ_TMEM_LD16(ts + o_col(1) + h0 + 16, (o1 + 16));
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), fb, __uint_as_float(o[e])));
        }
        if constexpr (kTree) {  // a row without a node may have added up anything
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = seen ? o[e] : 0u;
        }
        uint4 v[4];
        if (final_out) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t b4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[8 * c + 2 * i]), __uint_as_float(o[8 * c + 2 * i + 1]));
              b4[i] = *reinterpret_cast<const uint32_t*>(&y);
            }
            v[c] = make_uint4(b4[0], b4[1], b4[2], b4[3]);
          }
          emit(v);
        } else {
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t b4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) b4[i] = o[c0 + 4 * c + i];
              v[c] = make_uint4(b4[0], b4[1], b4[2], b4[3]);
            }
            emit(v);
          }
        }
      }
      if (any) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(gbar(w, 3));
          if (dual) ptx::mbar_arrive(gbar(1, 3));
        }
      }
      if (live) {
        const float top = kTree && !seen ? -INFINITY : m_run * c2 * (1.f / kLog2e);
        if (!final_out) {
          a.m_part[part_row] = top;
          a.l_part[part_row] = l;
        } else if (a.lse) {
          a.lse[prompt_at(a.lse_rows, it.b, it.tok0 + tok, g, hr)] = seen ? top + logf(l) : -INFINITY;
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
}

// Row tiles whose keys were cut: parts rescaled to their common maximum and
// added in order, O and LSE of every row.  Eight warps take eight rows of few
// parts, or one row's parts in turn; each lane holds 4 of the 128 elements.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const PromptDev a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ float s_m[kMergeWarps], s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!prompt_plan_fits(a)) return;
  const int groups = a.head->n_merges * a.h_k * (kPromptRows / kMergeWarps);  // of eight rows
  for (int x = blockIdx.x; x < groups; x += gridDim.x) {
    const int r0 = x % (kPromptRows / kMergeWarps) * kMergeWarps;
    const int g = x / (kPromptRows / kMergeWarps) % a.h_k;
    const PromptMerge m = a.merges[x / (kPromptRows / kMergeWarps) / a.h_k];
    const int rows = m.n_tok * a.h_r - m.row0;
    const bool together = m.n_parts > 8;  // the warps share a row
    const int64_t stride = static_cast<int64_t>(a.h_k) * kPromptRows;  // rows between a row's parts
    const int64_t base = static_cast<int64_t>(m.part0) * stride + g * kPromptRows;
    for (int i = 0; i < (together ? kMergeWarps : 1); ++i) {
      const int r = r0 + (together ? i : warp);
      if (r >= rows) break;  // uniform over the CTA (together) or the warp
      const int p0 = together ? warp : 0, step = together ? kMergeWarps : 1;
      float mx = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = p0 + lane * step; p < m.n_parts; p += 32 * step) mx = fmaxf(mx, a.m_part[base + r + p * stride]);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll 4
      for (int p = p0; p < m.n_parts; p += step) {
        const int64_t at = base + r + p * stride;
        const float mp = a.m_part[at];
        const float wt = mp == -INFINITY ? 0.f : __expf(mp - mx);
        const float4 v = *reinterpret_cast<const float4*>(a.o_part + at * kHeadDimDev + lane * 4);
        l = fmaf(wt, a.l_part[at], l);
        o.x = fmaf(wt, v.x, o.x);
        o.y = fmaf(wt, v.y, o.y);
        o.z = fmaf(wt, v.z, o.z);
        o.w = fmaf(wt, v.w, o.w);
      }
      if (together) {
        if (lane == 0) {
          s_m[warp] = mx;
          s_l[warp] = l;
        }
        s_o[warp][lane] = o;
        __syncthreads();
        if (warp == 0) {
          mx = -INFINITY;
          for (int v = 0; v < kMergeWarps; ++v) mx = fmaxf(mx, s_m[v]);
          l = 0.f;
          o = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int v = 0; v < kMergeWarps; ++v) {
            const float f = s_m[v] == -INFINITY ? 0.f : __expf(s_m[v] - mx);
            const float4 ov = s_o[v][lane];
            l = fmaf(f, s_l[v], l);
            o.x = fmaf(f, ov.x, o.x);
            o.y = fmaf(f, ov.y, o.y);
            o.z = fmaf(f, ov.z, o.z);
            o.w = fmaf(f, ov.w, o.w);
          }
        }
      }
      if (!together || warp == 0) {
        const int row = m.row0 + r, tok = row / a.h_r, hr = row - tok * a.h_r;
        const float inv = l > 0.f ? a.scale_o / l : 0.f;
        const __nv_bfloat162 lo2 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        const __nv_bfloat162 hi2 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2*>(a.o + prompt_at(a.o_rows, m.b, m.tok0 + tok, g, hr) + lane * 4) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
        if (lane == 0 && a.lse)
          a.lse[prompt_at(a.lse_rows, m.b, m.tok0 + tok, g, hr)] = l > 0.f ? mx + logf(l) : -INFINITY;
      }
      if (together) __syncthreads();  // s_o is read
    }
  }
}

template <bool kQe4m3, bool kCap, bool kTree>
cudaError_t launch(const std::conditional_t<kTree, PromptTreeDev, PromptDev>& a, int sm_count, const CUtensorMap& mk,
                   const CUtensorMap& mv, cudaStream_t stream) {
  constexpr int smem = Cfg<kQe4m3>::kBytes;
  auto kern = prompt_attn_kernel<kQe4m3, kCap, kTree>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(sm_count), 1, 1), dim3(kThreads, 1, 1), smem, stream, a, mk, mv);
}

template <bool kTree>
cudaError_t launch_maps(const std::conditional_t<kTree, PromptTreeDev, PromptDev>& a, bool q_e4m3, int sm_count,
                        cudaStream_t stream) {
  CUtensorMap mk, mv;
  if (!make_kv_map(&mk, a.k, a.page_size, a.h_k, a.num_pages, a.k_row, a.k_head, a.k_page, a.page_size, 1, 0) ||
      !make_kv_map(&mv, a.v, a.page_size, a.h_k, a.num_pages, a.v_row, a.v_head, a.v_page, a.page_size, 1, 0))
    return cudaErrorInvalidValue;
  if (a.softcap > 0.f)
    return q_e4m3 ? launch<true, true, kTree>(a, sm_count, mk, mv, stream) : launch<false, true, kTree>(a, sm_count, mk, mv, stream);
  return q_e4m3 ? launch<true, false, kTree>(a, sm_count, mk, mv, stream) : launch<false, false, kTree>(a, sm_count, mk, mv, stream);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptDev& a, bool q_e4m3, bool merge, int sm_count, cudaStream_t stream) {
  const cudaError_t e = launch_maps<false>(a, q_e4m3, sm_count, stream);
  if (e != cudaSuccess || !merge) return e;
  return launch_pdl(prompt_merge_kernel, dim3(static_cast<unsigned>(4 * sm_count), 1, 1), dim3(kMergeWarps * 32, 1, 1), 0,
                    stream, a);
}

cudaError_t launch_prompt_tree(const DecodeTreeDev& a, int n_q_tiles, bool q_e4m3, int sm_count, cudaStream_t stream) {
  PromptTreeDev d{};
  d.t = a;
  d.n_q_tiles = n_q_tiles;
  d.q = a.q;
  d.q_rows = {a.q_seq, static_cast<int64_t>(a.h_r) * kHeadDimDev, static_cast<int64_t>(a.n_q) * kHeadDimDev, kHeadDimDev};
  d.o = a.o;
  d.o_rows = {a.o_seq, static_cast<int64_t>(a.h_r) * kHeadDimDev, static_cast<int64_t>(a.n_q) * kHeadDimDev, kHeadDimDev};
  d.lse = a.lse;
  d.lse_rows = {static_cast<int64_t>(a.h_k) * a.n_q, a.h_r, a.n_q, 1};
  d.k = a.k;
  d.v = a.v;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.v_page = a.v_page;
  d.v_row = a.v_row;
  d.v_head = a.v_head;
  d.block_table = a.block_table;
  d.qd = a.qd;
  d.kd = a.kd;
  d.vd = a.vd;
  d.qd_seq = a.qd_seq;
  d.qd_head = a.qd_head;
  d.kd_seq = a.kd_seq;
  d.kd_head = a.kd_head;
  d.vd_seq = a.vd_seq;
  d.vd_head = a.vd_head;
  d.softmax_scale = a.softmax_scale;
  d.scale_o = a.scale_o;
  d.softcap = a.mod.softcap;
  d.o_part = a.o_part;
  d.m_part = a.m_part;
  d.l_part = a.l_part;
  d.status = a.status;
  d.num_seqs = a.num_seqs;
  d.h_k = a.h_k;
  d.h_r = a.h_r;
  d.page_size = a.page_size;
  d.max_blocks = a.max_blocks;
  d.num_pages = a.num_pages;
  d.kv_evict_first = a.kv_evict_first && n_q_tiles == 1;  // several q tiles share the pages
  d.max_splits = a.max_splits;
  const int64_t units = static_cast<int64_t>(a.num_work) * n_q_tiles * a.h_k;
  return launch_maps<true>(d, q_e4m3, static_cast<int>(units < sm_count ? units : sm_count), stream);
}

}  // namespace mj
