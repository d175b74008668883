// Rotary positions with one to four axes, the Q pack and the new tokens' rows
// in the paged e4m3 cache, in one pass over the projection's output.
//
// For pair i of a head (elements (i, i + rot/2), or (2i, 2i + 1)) and the
// position p of the axis that turns frequency i:
//   (x_a, x_b) -> (x_a cos - x_b sin, x_b cos + x_a sin),  cos, sin from row p
// of the caller's table.  Q rows leave as bf16 (packed or in the token
// layout), K rows as e4m3(y / k_descale) and V rows as e4m3(v / v_descale) in
// the slot the block table gives.  Everything between the bf16 inputs and
// those roundings is fp32, each operation rounded by itself: K is not rounded
// to bf16 on the way, so a code differs from the exact one's only next to a
// rounding border.
//
// Every byte is touched once (128 (4 h_r + 6) of them a token and kv head), so the
// bound is HBM for prompts (15005 tokens of 48 heads, 341 MB: 65 us, 5.2 TB/s,
// 59 % of the issue slots) and one chain of dependent loads (position ->
// table row; sequence length -> block table) plus the launch for decode
// batches: 64 tokens take 2.9 us a call back to back in a graph, everything in
// L2, but 6.4 us of kernel with cold inputs, and about 9 a call so from the host.
// One CTA takes one or more whole tokens: the token's cos and sin are fetched
// once into shared memory, by frequency, whatever the axes' map, and serve
// all of its heads; the tokens' slots are looked up at the same time, and the
// first heads' rows are already in flight before the barrier.  Eight lanes
// hold a head: lane t the pairs of frequencies 8t .. 8t+7 (two 16-byte
// vectors), or, past rot_dim, two vectors that pass unchanged.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mj_kernels.h"
#include "sm100_ptx.cuh"

namespace mj {
namespace {

constexpr int kMaxTokens = 8;      // tokens per CTA
constexpr int kLongCtas = 1024;    // CTAs from which they take more tokens instead
constexpr int kRopeThreads = 384;  // 48 heads at a time
constexpr int kStatusInvalidArg = 1;  // MJ_ERR_INVALID_ARG

struct TokenInfo {
  int32_t seq;    // its sequence, or -1: padding, nothing is done
  int32_t qi;     // index among the sequence's new tokens
  int32_t slot;   // cache slot, or -1: no K / V row
  int32_t page;   // its page
  int32_t pos0;   // position on axis 0
  int32_t bad;    // a position outside the table
};

__device__ __forceinline__ void unpack8(const uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint2 to_codes8(const float* q) {
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo = ptx::f32x2_to_e4m3x2(q[4 * i], q[4 * i + 1]);
    const uint16_t hi = ptx::f32x2_to_e4m3x2(q[4 * i + 2], q[4 * i + 3]);
    u[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint2(u[0], u[1]);
}

// x[i] / d for sixteen values, each as the IEEE division gives it, at three
// operations a value: with r = 1/d and q = x r rounded, x - q d is exact in an
// fma and q + (x - q d) r rounds to the quotient (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990, theorem
// 7).  The steps run on -q and -r, so that a zero keeps its sign: for x = -0
// the remainder is +0, and +0 (-r) - (-0) is +0, the quotient's negative.
// It needs r, q and the remainder clear of overflow and underflow: d
// outside [2^-60, 2^60] or a quotient past 2^40 takes the division itself; a
// remainder that underflows then belongs to a quotient below 2^-18, which
// every e4m3 rounding makes zero.  (The divisions were most of the kernel's
// instructions: on the prompt above 95 us with them, 77 so.)
__device__ __forceinline__ void divide16(float* x, float d) {
  const float r = __frcp_rn(d);
  const float2 nr2 = make_float2(-r, -r), d2 = make_float2(d, d);
  float2 q[8];  // negative quotients
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = mul2(make_float2(x[2 * i], x[2 * i + 1]), nr2);
    top = fmax3(top, fabsf(q[i].x), fabsf(q[i].y));
  }
  if (d >= 0x1p-60f && d <= 0x1p60f && top <= 0x1p40f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = fma2(fma2(q[i], d2, make_float2(x[2 * i], x[2 * i + 1])), nr2, q[i]);
      x[2 * i] = -q[i].x;
      x[2 * i + 1] = -q[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], d);
  }
}

// kPairs: neighbouring elements are a pair
template <bool kPairs>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeDev a, int tokens_per_cta) {
  __shared__ TokenInfo info[kMaxTokens];
  __shared__ int bad_pos[kMaxTokens];
  if (threadIdx.x < kMaxTokens) bad_pos[threadIdx.x] = 0;
  __syncthreads();
  // a programmatic dependent: no global load or store before the grid ahead
  // of this one has completed; the next kernel may launch now
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ __align__(16) float cs[];  // [token][cos: half | sin: half]

  const int half = a.rot_dim >> 1;
  const int t0 = blockIdx.x * tokens_per_cta;
  const int nt = a.num_tokens - t0 < tokens_per_cta ? a.num_tokens - t0 : tokens_per_cta;
  const int h_q = a.h_k * a.h_r;
  const int heads = h_q + 2 * a.h_k;
  const int lane8 = threadIdx.x & 7;
  const int groups = blockDim.x >> 3;

  // elements of this lane: two vectors of eight
  const bool turned = kPairs ? 16 * lane8 < a.rot_dim : 8 * lane8 < half;
  int c0, c1;  // their chunks of eight
  if (kPairs) {
    c0 = 2 * lane8;
    c1 = c0 + 1;
  } else if (turned) {
    c0 = lane8;
    c1 = lane8 + half / 8;
  } else {
    c0 = a.rot_dim / 8 + 2 * (lane8 - half / 8);
    c1 = c0 + 1;
  }

  auto source = [&](int item, int& tl, int& head) -> const uint4* {
    tl = item / heads;
    head = item - tl * heads;
    const int64_t t = t0 + tl;
    const __nv_bfloat16* src;
    if (head < h_q)
      src = a.q + t * a.q_tok + head * a.q_head;
    else if (head < h_q + a.h_k)
      src = a.k + t * a.k_tok + (head - h_q) * a.k_head_in;
    else
      src = a.v + t * a.v_tok + (head - h_q - a.h_k) * a.v_head_in;
    return reinterpret_cast<const uint4*>(src);
  };

  // where each token belongs (one thread each, from the CTA's end, so that
  // the table's loads below start at the same time in other warps)
  const int back = blockDim.x - 1 - threadIdx.x;
  if (back < nt) {
    const int t = t0 + back;
    TokenInfo f{-1, 0, -1, 0, a.positions[t], 0};
    int n = a.q_len;
    if (a.cu_tokens == nullptr) {
      f.seq = t / a.q_len;
      f.qi = t - f.seq * a.q_len;
    } else if (t >= a.cu_tokens[0] && t < a.cu_tokens[a.num_seqs]) {
      int lo = 0, hi = a.num_seqs - 1;  // the last sequence that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_tokens[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      f.seq = lo;
      f.qi = t - a.cu_tokens[lo];
      n = a.cu_tokens[lo + 1] - a.cu_tokens[lo];
    }
    if (f.seq >= 0) {
      const int64_t slot = static_cast<int64_t>(a.seq_lens[f.seq]) - n + f.qi;
      // (a sequence left out by the reservation: these slots are its last keys')
      const int granted = a.granted ? a.granted[f.seq] : n;
      if (slot >= 0 && granted != 0) {
        bool ok = granted == n && slot < a.max_blocks * a.page_size;
        if (ok) {
          f.page = a.block_table[static_cast<int64_t>(f.seq) * a.max_blocks + slot / a.page_size];
          ok = f.page >= 0 && f.page < a.num_pages;
        }
        if (ok)
          f.slot = static_cast<int>(slot);
        else if (a.status)
          atomicExch(a.status, kStatusInvalidArg);
      }
    }
    info[back] = f;
  }
  // the first heads' rows, in flight across the barrier (padding rows are
  // inside the input: reading them is harmless, they are not written); one
  // head in flight a group of eight lanes (with two, their registers cost a
  // CTA an SM: 77 us for 64 on a prompt of 15005 tokens and 48 heads)
  const int items = nt * heads;
  int item = threadIdx.x >> 3;
  int tl = 0, head = 0;
  uint4 w0 = make_uint4(0u, 0u, 0u, 0u), w1 = w0;
  if (item < items) {
    const uint4* src = source(item, tl, head);
    w0 = src[c0];
    w1 = src[c1];
  }
  // each token's cos and sin by frequency
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int t = i / half, f = i - t * half;
    int p = a.positions[a.axis_of[f] * a.pos_axis + t0 + t];
    if (p < 0 || p >= a.max_pos) {
      p = 0;
      bad_pos[t] = 1;
    }
    const float* row = a.cos_sin + static_cast<int64_t>(p) * a.rot_dim;
    cs[t * a.rot_dim + f] = row[f];
    cs[t * a.rot_dim + half + f] = row[half + f];
  }
  __syncthreads();
  if (threadIdx.x < nt && bad_pos[threadIdx.x] && info[threadIdx.x].seq >= 0 && a.status)
    atomicExch(a.status, kStatusInvalidArg);

  while (item < items) {
    const int cur_tl = tl, cur_head = head;
    float x[16];
    unpack8(w0, x);
    unpack8(w1, x + 8);
    item += groups;
    if (item < items) {  // the next head's rows
      const uint4* src = source(item, tl, head);
      w0 = src[c0];
      w1 = src[c1];
    }
    const TokenInfo f = info[cur_tl];
    if (f.seq < 0 || bad_pos[cur_tl]) continue;
    const bool is_v = cur_head >= h_q + a.h_k;
    if (turned && !is_v) {
      const float4* cv = reinterpret_cast<const float4*>(cs + cur_tl * a.rot_dim + 8 * lane8);
      const float4* sv = reinterpret_cast<const float4*>(cs + cur_tl * a.rot_dim + half + 8 * lane8);
      const float4 cc[2] = {cv[0], cv[1]}, ss[2] = {sv[0], sv[1]};
      const float c[8] = {cc[0].x, cc[0].y, cc[0].z, cc[0].w, cc[1].x, cc[1].y, cc[1].z, cc[1].w};
      const float s[8] = {ss[0].x, ss[0].y, ss[0].z, ss[0].w, ss[1].x, ss[1].y, ss[1].z, ss[1].w};
      // products and sums rounded one by one, as the formula stands: with a
      // product fused, about one code in a million next to a rounding border
      // would differ from a plain evaluation's (the prompt above: 65.3 for 64.7 us)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int ia = kPairs ? 2 * i : i, ib = kPairs ? 2 * i + 1 : i + 8;
        const float xa = x[ia], xb = x[ib];
        x[ia] = __fsub_rn(__fmul_rn(xa, c[i]), __fmul_rn(xb, s[i]));
        x[ib] = __fadd_rn(__fmul_rn(xb, c[i]), __fmul_rn(xa, s[i]));
      }
    }
    if (cur_head < h_q) {
      const int g = cur_head / a.h_r;
      const int64_t row =
          a.q_packed ? f.seq * a.q_out_stride +
                           ((static_cast<int64_t>(g) * a.q_len + f.qi) * a.h_r + (cur_head - g * a.h_r)) * kHeadDimDev
                     : static_cast<int64_t>(t0 + cur_tl) * a.q_out_stride + static_cast<int64_t>(cur_head) * kHeadDimDev;
      uint4* dst = reinterpret_cast<uint4*>(a.q_out + row);
      dst[c0] = pack8(x);
      dst[c1] = pack8(x + 8);
    } else if (f.slot >= 0) {
      const int g = cur_head - h_q - (is_v ? a.h_k : 0);
      const int r = f.slot % a.page_size;
      uint8_t* row;
      float descale;
      if (is_v) {
        row = a.v_cache + f.page * a.v_page + r * a.v_row + g * a.v_head;
        descale = a.vd[f.seq * a.vd_seq + g * a.vd_head];
      } else {
        row = a.k_cache + f.page * a.k_page + r * a.k_row + g * a.k_head;
        descale = a.kd[f.seq * a.kd_seq + g * a.kd_head];
        if (a.key_pos && lane8 == 0) a.key_pos[f.seq * a.kp_seq + g * a.kp_head + f.slot] = f.pos0;
      }
      uint2* dst = reinterpret_cast<uint2*>(row);
      divide16(x, descale);
      dst[c0] = to_codes8(x);
      dst[c1] = to_codes8(x + 8);
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeDev& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  const int heads = a.h_k * (a.h_r + 2);
  // whole tokens: about one head per group of eight lanes, and more of them
  // once the CTAs fill the GPU several times over (they share one
  // chain of dependent loads: one token a CTA took 152 us where eight take 64)
  int per_cta = (kRopeThreads / 8) / heads;
  per_cta = per_cta < 1 ? 1 : (per_cta > kMaxTokens ? kMaxTokens : per_cta);
  while (per_cta * 2 <= kMaxTokens && a.num_tokens >= kLongCtas * per_cta * 2) per_cta *= 2;
  int threads = per_cta * heads * 8;
  threads = (threads + 31) / 32 * 32;
  if (threads > kRopeThreads) threads = kRopeThreads;
  const unsigned grid = static_cast<unsigned>((a.num_tokens + per_cta - 1) / per_cta);
  const size_t smem = static_cast<size_t>(per_cta) * a.rot_dim * sizeof(float);
  return launch_pdl(a.interleaved ? rope_append_kernel<true> : rope_append_kernel<false>, dim3(grid, 1, 1),
                    dim3(static_cast<unsigned>(threads), 1, 1), smem, stream, a, per_cta);
}

}  // namespace mj
