// C ABI entry points of the cache's own operators: rotary append, spans of
// modified scores, key weights, eviction.  Argument checks and launches.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "mj.h"
#include "mj_checks.h"
#include "mj_internal.h"
#include "mj_kernels.h"
#include "score_mod.cuh"

namespace mj {

mj_status score_mod_dev(const mj_decode_params& p, const mj_score_mod& mod, const int32_t* spans, ScoreModDev* out) {
  // a cap for which neither 1 / softcap nor a score over it leaves fp32's range
  if (mod.softcap != 0.f && !(mod.softcap >= 0x1p-20f && mod.softcap <= 0x1p60f)) return MJ_ERR_INVALID_ARG;
  if (mod.window < 0 || (mod.window > 0 && p.causal == 0)) return MJ_ERR_INVALID_ARG;
  if (!aligned4(mod.alibi_slopes) || !aligned4(mod.key_begin) || !aligned4(mod.key_end) || !aligned4(mod.prefix) ||
      !aligned16(spans))
    return MJ_ERR_INVALID_ARG;
  out->softcap = mod.softcap;
  out->window = std::min(mod.window, 1 << 30);  // no length is longer
  out->slopes = mod.alibi_slopes;
  out->key_begin = mod.key_begin;
  out->key_end = mod.key_end;
  out->prefix = mod.prefix;
  out->spans = reinterpret_cast<const int4*>(spans);
  return MJ_OK;
}

mj_status tree_mod_dev(const mj_decode_params& p, const mj_score_mod* mod, const int32_t* spans, ScoreModDev* out) {
  // these take positions for slots, which a tree's are not
  if (mod && (mod->window != 0 || mod->alibi_slopes || mod->key_end)) return MJ_ERR_UNSUPPORTED;
  const mj_score_mod none{};
  return score_mod_dev(p, mod ? *mod : none, spans, out);
}

}  // namespace mj

using namespace mj;

extern "C" mj_status mj_rope_append(const mj_rope_params* params, const mj_rope_args* args, mj_stream_t stream) {
  if (!params || !args) return MJ_ERR_INVALID_ARG;
  const mj_rope_params& p = *params;
  const mj_rope_args& a = *args;
  if (p.num_seqs < 1 || p.q_len < 1 || p.h_k < 1 || p.h_r < 1 || p.max_blocks < 1 || p.num_pages < 1 || p.max_pos < 1)
    return MJ_ERR_INVALID_ARG;
  if (p.interleaved != 0 && p.interleaved != 1) return MJ_ERR_INVALID_ARG;
  if (p.head_dim != kHeadDim || !page_size_ok(p.page_size)) return MJ_ERR_UNSUPPORTED;
  if (p.rot_dim < 16 || p.rot_dim > kHeadDim || p.rot_dim % 16 != 0) return MJ_ERR_UNSUPPORTED;
  if (p.n_axes < 1 || p.n_axes > 4) return MJ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p.max_blocks) * p.page_size > (int64_t{1} << 30)) return MJ_ERR_UNSUPPORTED;
  const int64_t h_q = static_cast<int64_t>(p.h_k) * p.h_r;
  if (h_q + 2 * static_cast<int64_t>(p.h_k) > 4096) return MJ_ERR_UNSUPPORTED;
  if (!a.cos_sin || !a.k_cache || !a.v_cache || !a.block_table || !a.seq_lens || !a.k_descale || !a.v_descale)
    return MJ_ERR_INVALID_ARG;
  // (a batch without tokens has none of these)
  if (a.num_tokens != 0 && (!a.q || !a.k || !a.v || !a.positions || !a.q_out)) return MJ_ERR_INVALID_ARG;
  if (a.num_tokens < 0 || (a.q_packed != 0 && a.q_packed != 1)) return MJ_ERR_INVALID_ARG;
  if (!a.cu_tokens && static_cast<int64_t>(p.num_seqs) * p.q_len != a.num_tokens) return MJ_ERR_INVALID_ARG;
  if (a.cu_tokens && a.q_packed) return MJ_ERR_INVALID_ARG;  // packed rows need one q_len
  for (const void* x : {a.q, a.k, a.v, static_cast<const void*>(a.cos_sin), static_cast<const void*>(a.q_out),
                        static_cast<const void*>(a.k_cache), static_cast<const void*>(a.v_cache)})
    if (!aligned16(x)) return MJ_ERR_INVALID_ARG;
  for (const void* x :
       {static_cast<const void*>(a.positions), static_cast<const void*>(a.cu_tokens),
        static_cast<const void*>(a.block_table), static_cast<const void*>(a.seq_lens),
        static_cast<const void*>(a.k_descale), static_cast<const void*>(a.v_descale),
        static_cast<const void*>(a.key_pos), static_cast<const void*>(a.status), static_cast<const void*>(a.granted)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  const int64_t in_strides[6] = {a.q_tok, a.q_head, a.k_tok, a.k_head_in, a.v_tok, a.v_head_in};
  for (int64_t s : in_strides)
    if (s < 0 || s % 8 != 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  for (int64_t s : {a.k_page, a.k_row, a.k_head, a.v_page, a.v_row, a.v_head})
    if (s <= 0 || s % 16 != 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  for (int64_t s : {a.kd_seq, a.kd_head, a.vd_seq, a.vd_head, a.kp_seq, a.kp_head, a.pos_axis})
    if (s < 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  const int64_t row_elems = h_q * kHeadDim * (a.q_packed ? p.q_len : 1);
  const int64_t rows = a.q_packed ? p.num_seqs : a.num_tokens;
  if (too_far(a.num_tokens, a.q_tok) || too_far(a.num_tokens, a.k_tok) || too_far(a.num_tokens, a.v_tok) ||
      too_far(h_q, a.q_head) || too_far(p.h_k, a.k_head_in) || too_far(p.h_k, a.v_head_in) ||
      too_far(rows, a.q_out_stride))
    return MJ_ERR_INVALID_ARG;
  if (pool_too_far(p.num_pages, p.page_size, p.h_k, a.k_page, a.k_row, a.k_head) ||
      pool_too_far(p.num_pages, p.page_size, p.h_k, a.v_page, a.v_row, a.v_head) ||
      heads_too_far(p.num_seqs, p.h_k, a.kd_seq, a.kd_head) || heads_too_far(p.num_seqs, p.h_k, a.vd_seq, a.vd_head) ||
      (a.key_pos && heads_too_far(p.num_seqs, p.h_k, a.kp_seq, a.kp_head)))
    return MJ_ERR_INVALID_ARG;
  if (a.q_out_stride % 8 != 0 || a.q_out_stride < 0 || a.q_out_stride >= kMaxStride) return MJ_ERR_INVALID_ARG;
  if (rows > 1 && a.q_out_stride < row_elems) return MJ_ERR_INVALID_ARG;
  RopeDev d{};
  uint8_t axes_used = 0;
  for (int i = 0; i < p.rot_dim / 2; ++i) {
    d.axis_of[i] = a.freq_axis ? a.freq_axis[i] : 0;
    if (d.axis_of[i] >= p.n_axes) return MJ_ERR_INVALID_ARG;
    axes_used = std::max(axes_used, d.axis_of[i]);
  }
  if (axes_used > 0 && a.pos_axis < a.num_tokens) return MJ_ERR_INVALID_ARG;
  if (a.num_tokens == 0) return MJ_OK;
  // an output over an input is refused, but for Q rotated where it lies
  const int64_t out_bytes = ((rows - 1) * a.q_out_stride + row_elems) * 2;
  auto in_bytes = [&](int64_t tok, int64_t head, int64_t heads) {
    return ((a.num_tokens - 1) * tok + (heads - 1) * head + kHeadDim) * 2;
  };
  const bool in_place = a.q_out == a.q && !a.q_packed && a.q_tok == a.q_out_stride && (h_q == 1 || a.q_head == kHeadDim);
  if (!in_place && overlap(a.q_out, out_bytes, a.q, in_bytes(a.q_tok, a.q_head, h_q))) return MJ_ERR_INVALID_ARG;
  // (in place, Q's rows may lie between K's and V's of the same projection:
  // a token's rows of x then fall behind its Q rows and before the next's)
  auto beside = [&](const void* x, int64_t tok, int64_t head) {
    if (!in_place || tok != a.q_tok || tok == 0) return false;
    int64_t at = (static_cast<const char*>(x) - static_cast<const char*>(a.q)) / 2 % tok;
    if (at < 0) at += tok;
    return at >= h_q * kHeadDim && at + (p.h_k - 1) * head + kHeadDim <= tok;
  };
  if ((overlap(a.q_out, out_bytes, a.k, in_bytes(a.k_tok, a.k_head_in, p.h_k)) && !beside(a.k, a.k_tok, a.k_head_in)) ||
      (overlap(a.q_out, out_bytes, a.v, in_bytes(a.v_tok, a.v_head_in, p.h_k)) && !beside(a.v, a.v_tok, a.v_head_in)))
    return MJ_ERR_INVALID_ARG;

  d.q = static_cast<const __nv_bfloat16*>(a.q);
  d.k = static_cast<const __nv_bfloat16*>(a.k);
  d.v = static_cast<const __nv_bfloat16*>(a.v);
  d.q_tok = a.q_tok;
  d.q_head = a.q_head;
  d.k_tok = a.k_tok;
  d.k_head_in = a.k_head_in;
  d.v_tok = a.v_tok;
  d.v_head_in = a.v_head_in;
  d.positions = a.positions;
  d.pos_axis = a.pos_axis;
  d.cos_sin = a.cos_sin;
  d.cu_tokens = a.cu_tokens;
  d.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  d.q_out_stride = a.q_out_stride;
  d.k_cache = a.k_cache;
  d.v_cache = a.v_cache;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.v_page = a.v_page;
  d.v_row = a.v_row;
  d.v_head = a.v_head;
  d.block_table = a.block_table;
  d.seq_lens = a.seq_lens;
  d.kd = a.k_descale;
  d.vd = a.v_descale;
  d.kd_seq = a.kd_seq;
  d.kd_head = a.kd_head;
  d.vd_seq = a.vd_seq;
  d.vd_head = a.vd_head;
  d.key_pos = a.key_pos;
  d.kp_seq = a.kp_seq;
  d.kp_head = a.kp_head;
  d.status = a.status;
  d.granted = a.granted;
  d.num_tokens = a.num_tokens;
  d.num_seqs = p.num_seqs;
  d.q_len = p.q_len;
  d.h_k = p.h_k;
  d.h_r = p.h_r;
  d.page_size = p.page_size;
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  d.rot_dim = p.rot_dim;
  d.max_pos = p.max_pos;
  d.q_packed = a.q_packed;
  d.interleaved = p.interleaved;
  const NvtxRange range("mj_rope_append");
  return launch_rope_append(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_score_spans(const mj_decode_params* params, const mj_score_mod* mod,
                                    const int32_t* seq_lens_host, int32_t* spans_host, int32_t* plan_lens_host) {
  mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!mod || !seq_lens_host || !spans_host || !plan_lens_host) return MJ_ERR_INVALID_ARG;
  const mj_decode_params& p = *params;
  ScoreModDev m{};
  st = score_mod_dev(p, *mod, nullptr, &m);
  if (st != MJ_OK) return st;
  for (int b = 0; b < p.num_seqs; ++b) {
    const int L = seq_lens_host[b];
    if (L < 0 || L > static_cast<int64_t>(p.max_blocks) * p.page_size) return MJ_ERR_INVALID_ARG;
    int first = INT32_MAX, last = -1, pfx = 0;
    for (int qi = 0; qi < p.q_len; ++qi) {
      const RowRange r = row_range(m, p.causal, p.q_len, b, L, qi);
      pfx = r.pfx;
      if (r.lo <= r.hi) {
        first = std::min(first, r.lo);
        last = std::max(last, r.hi);
      }
    }
    const int4 s = make_span(first, last, pfx, &plan_lens_host[b]);
    const int32_t four[4] = {s.x, s.y, s.z, s.w};
    std::memcpy(spans_host + 4 * static_cast<int64_t>(b), four, sizeof(four));
  }
  return MJ_OK;
}

extern "C" mj_status mj_score_spans_device(const mj_decode_params* params, const mj_score_mod* mod,
                                           const int32_t* seq_lens, int32_t* spans, int32_t* plan_lens,
                                           mj_stream_t stream) {
  mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!mod || !seq_lens || !spans || !plan_lens || !aligned4(seq_lens) || !aligned4(plan_lens)) return MJ_ERR_INVALID_ARG;
  ScoreModDev m{};
  st = score_mod_dev(*params, *mod, spans, &m);
  if (st != MJ_OK) return st;
  const int64_t max_len = static_cast<int64_t>(params->max_blocks) * params->page_size;
  const cudaError_t e = launch_score_spans(m, seq_lens, params->num_seqs, params->q_len, params->causal, max_len,
                                           reinterpret_cast<int4*>(spans), plan_lens,
                                           reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_tree_spans(const mj_decode_params* params, const mj_tree* tree, const mj_score_mod* mod,
                                   const int32_t* seq_lens_host, int32_t* spans_host, int32_t* plan_lens_host) {
  mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!tree || !seq_lens_host || !spans_host || !plan_lens_host || !aligned4(tree->tree_lens)) return MJ_ERR_INVALID_ARG;
  const mj_decode_params& p = *params;
  ScoreModDev m{};
  st = tree_mod_dev(p, mod, nullptr, &m);
  if (st != MJ_OK) return st;
  for (int b = 0; b < p.num_seqs; ++b) {
    const int L = seq_lens_host[b];
    if (L < 0 || L > static_cast<int64_t>(p.max_blocks) * p.page_size) return MJ_ERR_INVALID_ARG;
    const TreeShape t = tree_shape(tree->tree_lens, p.q_len, b, L);
    int first = INT32_MAX, pfx = 0;
    for (int qi = 0; qi < t.nodes; ++qi) {
      const RowRange r = tree_range(m, p.q_len, b, qi, t.ctx);
      pfx = r.pfx;
      first = std::min(first, r.lo);
    }
    const int4 s = make_tree_span(t, first, pfx, &plan_lens_host[b]);
    const int32_t four[4] = {s.x, s.y, s.z, s.w};
    std::memcpy(spans_host + 4 * static_cast<int64_t>(b), four, sizeof(four));
  }
  return MJ_OK;
}

extern "C" mj_status mj_tree_spans_device(const mj_decode_params* params, const mj_tree* tree, const mj_score_mod* mod,
                                          const int32_t* seq_lens, int32_t* spans, int32_t* plan_lens, mj_stream_t stream) {
  mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!tree || !seq_lens || !spans || !plan_lens || !aligned4(tree->tree_lens) || !aligned4(seq_lens) || !aligned4(plan_lens))
    return MJ_ERR_INVALID_ARG;
  ScoreModDev m{};
  st = tree_mod_dev(*params, mod, spans, &m);
  if (st != MJ_OK) return st;
  const int64_t max_len = static_cast<int64_t>(params->max_blocks) * params->page_size;
  const cudaError_t e = launch_tree_spans(m, tree->tree_lens, seq_lens, params->num_seqs, params->q_len, max_len,
                                          reinterpret_cast<int4*>(spans), plan_lens, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_key_weights(const mj_decode_params* params, const mj_score_mod* mod,
                                    const mj_decode_args* args, float* acc, int64_t acc_seq, int64_t acc_head,
                                    float decay, int32_t fresh, mj_stream_t stream) {
  mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!args || !acc) return MJ_ERR_INVALID_ARG;
  const mj_decode_params& p = *params;
  const mj_decode_args& a = *args;
  if (p.kv_format == MJ_KV_NVFP4) return MJ_ERR_UNSUPPORTED;
  if (!a.q || !a.k || !a.block_table || !a.seq_lens || !a.work || !a.q_descale || !a.k_descale || !a.lse)
    return MJ_ERR_INVALID_ARG;
  if (a.num_work < 1 || static_cast<int64_t>(a.num_work) * p.h_k > INT32_MAX) return MJ_ERR_INVALID_ARG;
  const int64_t kv_strides[6] = {a.k_page, a.k_row, a.k_head, a.k_page, a.k_row, a.k_head};
  if (!kv_layout_ok(p, a.k, a.k, kv_strides)) return MJ_ERR_INVALID_ARG;
  const int q_bytes = p.q_dtype == MJ_E4M3 ? 1 : 2;
  const int n_q = p.q_len * p.h_r;
  if (!aligned16(a.q) || !aligned16(a.work) || !aligned4(acc) || !aligned4(a.lse)) return MJ_ERR_INVALID_ARG;
  if (a.q_seq_stride < 0 || ((a.q_seq_stride * q_bytes) & 15) != 0) return MJ_ERR_INVALID_ARG;
  if (p.num_seqs > 1 && a.q_seq_stride < static_cast<int64_t>(p.h_k) * n_q * kHeadDim) return MJ_ERR_INVALID_ARG;
  for (int64_t s : {a.qd_seq, a.qd_head, a.kd_seq, a.kd_head, acc_seq, acc_head})
    if (s < 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  const int64_t max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  if (too_far(p.num_seqs, a.q_seq_stride) || heads_too_far(p.num_seqs, p.h_k, a.qd_seq, a.qd_head) ||
      heads_too_far(p.num_seqs, p.h_k, a.kd_seq, a.kd_head) || heads_too_far(p.num_seqs, p.h_k, acc_seq, acc_head))
    return MJ_ERR_INVALID_ARG;
  if (!planes_apart(p.num_seqs, p.h_k, acc_seq, acc_head, max_len)) return MJ_ERR_INVALID_ARG;
  if (!(a.softmax_scale > 0.f) || !(decay >= 0.f && decay <= 1.f) || fresh < 0) return MJ_ERR_INVALID_ARG;

  DecodeModDev d{};
  if (mod) {
    st = score_mod_dev(p, *mod, nullptr, &d.mod);
    if (st != MJ_OK) return st;
  }
  d.q = a.q;
  d.q_seq = a.q_seq_stride;
  d.k = a.k;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.block_table = a.block_table;
  d.seq_lens = a.seq_lens;
  d.work = a.work;
  d.num_work = a.num_work;
  d.qd = a.q_descale;
  d.kd = a.k_descale;
  d.qd_seq = a.qd_seq;
  d.qd_head = a.qd_head;
  d.kd_seq = a.kd_seq;
  d.kd_head = a.kd_head;
  d.softmax_scale = a.softmax_scale;
  d.status = a.status;
  d.num_seqs = p.num_seqs;
  d.h_k = p.h_k;
  d.n_q = n_q;
  d.q_len = p.q_len;
  d.h_r = p.h_r;
  d.page_size = p.page_size;
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  d.causal = p.causal;
  d.kv_evict_first = kv_evict_first(p);
  d.kv_format = p.kv_format;
  const int sms = device_sm_count();
  if (sms < 1) return MJ_ERR_CUDA;
  const NvtxRange range("mj_key_weights");
  const int step = p.q_dtype == MJ_E4M3 ? 256 : 128;  // rows a launch takes
  for (int n0 = 0; n0 < n_q; n0 += step) {
    const int rows = std::min(step, n_q - n0);
    // later row groups add onto what the first one wrote
    const cudaError_t e =
        launch_key_weights(d, p.q_dtype == MJ_E4M3, mod != nullptr, n0, rows, a.lse, acc, acc_seq, acc_head,
                           n0 == 0 ? decay : 1.f, n0 == 0 ? fresh : 0, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return MJ_ERR_CUDA;
  }
  return MJ_OK;
}

namespace {

struct EvictLayout {
  int64_t cap;  // moves of one (b, g) at most
  size_t counts_off, total;
};

EvictLayout evict_layout(const mj_decode_params& p, int32_t budget) {
  EvictLayout w{};
  const int64_t max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  w.cap = std::max<int64_t>(0, std::min<int64_t>(budget, max_len - budget));
  const size_t groups = static_cast<size_t>(p.num_seqs) * p.h_k;
  // (slot, page) of a destination and a source a move, and the moves' number
  w.counts_off = groups * static_cast<size_t>(w.cap) * 16;
  w.total = w.counts_off + groups * 4;
  return w;
}

}  // namespace

extern "C" size_t mj_evict_workspace_bytes(const mj_decode_params* params, int32_t budget) {
  if (check_params(params) != MJ_OK || budget < 1) return 0;
  return evict_layout(*params, budget).total;
}

extern "C" mj_status mj_evict(const mj_decode_params* params, const mj_evict_args* args, mj_stream_t stream) {
  const mj_status st = check_params(params);
  if (st != MJ_OK) return st;
  if (!args) return MJ_ERR_INVALID_ARG;
  const mj_decode_params& p = *params;
  const mj_evict_args& a = *args;
  if (!a.k || !a.v || !a.block_table || !a.seq_lens || !a.acc || !a.acc_out || !a.new_lens) return MJ_ERR_INVALID_ARG;
  if (a.key_pos && (!a.key_pos_out || !a.next_pos)) return MJ_ERR_INVALID_ARG;
  if (a.budget < 1 || a.keep_first < 0 || a.keep_last < 0 ||
      static_cast<int64_t>(a.keep_first) + a.keep_last > a.budget)
    return MJ_ERR_INVALID_ARG;
  const int64_t kv_strides[6] = {a.k_page, a.k_row, a.k_head, a.v_page, a.v_row, a.v_head};
  if (!kv_layout_ok(p, a.k, a.v, kv_strides)) return MJ_ERR_INVALID_ARG;
  mj_decode_args scales{};
  scales.k_scales = a.k_scales;
  scales.v_scales = a.v_scales;
  scales.ks_page = a.ks_page;
  scales.ks_head = a.ks_head;
  scales.vs_page = a.vs_page;
  scales.vs_head = a.vs_head;
  if (!scales_ok(p, scales)) return MJ_ERR_INVALID_ARG;
  for (const void* x :
       {static_cast<const void*>(a.block_table), static_cast<const void*>(a.seq_lens), static_cast<const void*>(a.acc),
        static_cast<const void*>(a.acc_out), static_cast<const void*>(a.key_pos),
        static_cast<const void*>(a.key_pos_out), static_cast<const void*>(a.next_pos),
        static_cast<const void*>(a.new_lens), static_cast<const void*>(a.status)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  for (int64_t s : {a.acc_seq, a.acc_head})
    if (s < 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  if (heads_too_far(p.num_seqs, p.h_k, a.acc_seq, a.acc_head) ||
      pool_too_far(p.num_pages, p.page_size, p.h_k, a.k_page, a.k_row, a.k_head) ||
      pool_too_far(p.num_pages, p.page_size, p.h_k, a.v_page, a.v_row, a.v_head) ||
      (p.kv_format == MJ_KV_NVFP4 && (pool_too_far(p.num_pages, 1, p.h_k, a.ks_page, 0, a.ks_head) ||
                                      pool_too_far(p.num_pages, 1, p.h_k, a.vs_page, 0, a.vs_head))))
    return MJ_ERR_INVALID_ARG;
  const int64_t lens_bytes = static_cast<int64_t>(p.num_seqs) * 4;
  if (overlap(a.new_lens, lens_bytes, a.seq_lens, lens_bytes)) return MJ_ERR_INVALID_ARG;
  if (a.key_pos && overlap(a.new_lens, lens_bytes, a.next_pos, lens_bytes)) return MJ_ERR_INVALID_ARG;
  // an output plane is its input or apart from it
  const int64_t max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  const int64_t plane = ((p.num_seqs - 1) * a.acc_seq + (p.h_k - 1) * a.acc_head + max_len) * 4;
  if (a.acc_out != a.acc && overlap(a.acc_out, plane, a.acc, plane)) return MJ_ERR_INVALID_ARG;
  if (a.key_pos && a.key_pos_out != a.key_pos && overlap(a.key_pos_out, plane, a.key_pos, plane))
    return MJ_ERR_INVALID_ARG;
  // and the heads' slots are their own
  if (!planes_apart(p.num_seqs, p.h_k, a.acc_seq, a.acc_head, max_len)) return MJ_ERR_INVALID_ARG;
  const EvictLayout w = evict_layout(p, a.budget);
  if (!a.workspace || !aligned16(a.workspace)) return MJ_ERR_INVALID_ARG;
  if (a.workspace_bytes < w.total) return MJ_ERR_CAPACITY;
  if (static_cast<int64_t>(p.num_seqs) * p.h_k > (int64_t{1} << 27)) return MJ_ERR_UNSUPPORTED;  // the grid's range

  EvictDev d{};
  d.k = a.k;
  d.v = a.v;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.v_page = a.v_page;
  d.v_row = a.v_row;
  d.v_head = a.v_head;
  d.block_table = a.block_table;
  d.seq_lens = a.seq_lens;
  d.acc = a.acc;
  d.acc_out = a.acc_out;
  d.acc_seq = a.acc_seq;
  d.acc_head = a.acc_head;
  d.key_pos = a.key_pos;
  d.key_pos_out = a.key_pos_out;
  d.next_pos = a.next_pos;
  d.new_lens = a.new_lens;
  d.moves = static_cast<int32_t*>(a.workspace);
  d.counts = reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + w.counts_off);
  d.moves_cap = static_cast<int32_t>(w.cap);
  d.budget = a.budget;
  d.keep_first = a.keep_first;
  d.keep_last = a.keep_last;
  d.num_seqs = p.num_seqs;
  d.h_k = p.h_k;
  d.page_size = p.page_size;
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  d.row_bytes = 16 * kv_bits(p.kv_format);
  d.status = a.status;
  if (p.kv_format == MJ_KV_NVFP4) {
    d.ks = a.k_scales;
    d.vs = a.v_scales;
    d.ks_page = a.ks_page;
    d.ks_head = a.ks_head;
    d.vs_page = a.vs_page;
    d.vs_head = a.vs_head;
  }
  const int sms = device_sm_count();
  if (sms < 1) return MJ_ERR_CUDA;
  const NvtxRange range("mj_evict");
  return launch_evict(d, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}
