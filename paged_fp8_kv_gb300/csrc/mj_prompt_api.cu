// C ABI entry points of attention over whole prompts: sizes, argument checks
// and launches.

#include <cuda_runtime.h>

#include <algorithm>

#include "mj.h"
#include "mj_checks.h"
#include "mj_internal.h"
#include "mj_kernels.h"
#include "prompt.cuh"

namespace mj {
namespace {

mj_status check_prompt(const mj_decode_params* params, int32_t num_tokens) {
  if (!params) return MJ_ERR_INVALID_ARG;
  mj_decode_params p = *params;
  p.q_len = 1;  // not looked at here
  p.kernel = MJ_KERNEL_AUTO;
  p.l2_prefetch = 0;
  const mj_status st = check_params(&p);
  if (st != MJ_OK) return st;
  if (p.kv_format != MJ_KV_E4M3) return MJ_ERR_UNSUPPORTED;
  if (num_tokens < 0) return MJ_ERR_INVALID_ARG;
  const int64_t h_q = static_cast<int64_t>(p.h_k) * p.h_r;
  if (h_q > 4096 || p.num_seqs > kMaxDevicePlanSeqs) return MJ_ERR_UNSUPPORTED;
  if (num_tokens * h_q > (int64_t{1} << 30)) return MJ_ERR_UNSUPPORTED;
  return MJ_OK;
}

int slots_of(const mj_decode_params& p) { return std::max(1, kPromptSlots / p.h_k); }

// every row tile, and the parts that cutting adds (at most two a slot)
int64_t items_cap(const mj_decode_params& p, int32_t num_tokens) {
  return static_cast<int64_t>(num_tokens) * p.h_r / kPromptRows + p.num_seqs + 2 * slots_of(p);
}

struct PlanLayout {
  size_t items, scratch, merges, total;
};
PlanLayout plan_layout(const mj_decode_params& p, int32_t num_tokens) {
  const size_t n = static_cast<size_t>(items_cap(p, num_tokens));
  PlanLayout l{};
  l.items = sizeof(PromptHeader);
  l.scratch = l.items + n * sizeof(PromptItem);
  l.merges = l.scratch + n * sizeof(PromptItem);
  l.total = l.merges + static_cast<size_t>(slots_of(p)) * sizeof(PromptMerge);
  return l;
}

int64_t part_rows(const mj_decode_params& p) { return static_cast<int64_t>(2) * slots_of(p) * p.h_k * kPromptRows; }

}  // namespace
}  // namespace mj

using namespace mj;

extern "C" size_t mj_prompt_plan_bytes(const mj_decode_params* params, int32_t num_tokens) {
  if (check_prompt(params, num_tokens) != MJ_OK) return 0;
  return plan_layout(*params, num_tokens).total;
}

extern "C" size_t mj_prompt_workspace_bytes(const mj_decode_params* params) {
  if (check_prompt(params, 0) != MJ_OK || params->max_splits == 1) return 0;
  return static_cast<size_t>(part_rows(*params)) * (kHeadDim + 2) * sizeof(float);
}

extern "C" mj_status mj_prompt_plan(const mj_decode_params* params, const int32_t* cu_tokens, const int32_t* seq_lens,
                                    int32_t num_tokens, int32_t window, void* plan, size_t plan_bytes, int32_t* status,
                                    mj_stream_t stream) {
  const mj_status st = check_prompt(params, num_tokens);
  if (st != MJ_OK) return st;
  const mj_decode_params& p = *params;
  if (!cu_tokens || !seq_lens || !plan || !aligned16(plan)) return MJ_ERR_INVALID_ARG;
  if (!aligned4(cu_tokens) || !aligned4(seq_lens) || !aligned4(status)) return MJ_ERR_INVALID_ARG;
  if (window < 0 || (window > 0 && p.causal == 0)) return MJ_ERR_INVALID_ARG;
  const PlanLayout l = plan_layout(p, num_tokens);
  if (plan_bytes < l.total) return MJ_ERR_CAPACITY;
  char* const base = static_cast<char*>(plan);
  PromptPlanDev d{};
  d.cu_tokens = cu_tokens;
  d.seq_lens = seq_lens;
  d.num_seqs = p.num_seqs;
  d.num_tokens = num_tokens;
  d.h_k = p.h_k;
  d.h_r = p.h_r;
  d.causal = p.causal;
  d.window = std::min(window, 1 << 30);  // no length is longer
  d.max_splits = p.max_splits;
  d.page_size = p.page_size;
  d.max_blocks = p.max_blocks;
  d.max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  d.head = reinterpret_cast<PromptHeader*>(base);
  d.items = reinterpret_cast<PromptItem*>(base + l.items);
  d.scratch = reinterpret_cast<PromptItem*>(base + l.scratch);
  d.merges = reinterpret_cast<PromptMerge*>(base + l.merges);
  d.items_cap = static_cast<int32_t>(items_cap(p, num_tokens));
  d.slots = slots_of(p);
  d.status = status;
  const NvtxRange range("mj_prompt_plan");
  return launch_prompt_plan(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_prompt_attn(const mj_decode_params* params, const mj_prompt_args* args, mj_stream_t stream) {
  if (!args) return MJ_ERR_INVALID_ARG;
  const mj_prompt_args& a = *args;
  const mj_status st = check_prompt(params, a.num_tokens);
  if (st != MJ_OK) return st;
  const mj_decode_params& p = *params;
  if (!a.k || !a.v || !a.block_table || !a.plan || !a.q_descale || !a.k_descale || !a.v_descale) return MJ_ERR_INVALID_ARG;
  if (a.num_tokens != 0 && (!a.q || !a.o)) return MJ_ERR_INVALID_ARG;
  const int64_t kv_strides[6] = {a.k_page, a.k_row, a.k_head, a.v_page, a.v_row, a.v_head};
  if (!kv_layout_ok(p, a.k, a.v, kv_strides)) return MJ_ERR_INVALID_ARG;
  if (pool_too_far(p.num_pages, p.page_size, p.h_k, a.k_page, a.k_row, a.k_head) ||
      pool_too_far(p.num_pages, p.page_size, p.h_k, a.v_page, a.v_row, a.v_head))
    return MJ_ERR_INVALID_ARG;
  for (const void* x : {a.q, static_cast<const void*>(a.o), a.plan, static_cast<const void*>(a.workspace)})
    if (!aligned16(x)) return MJ_ERR_INVALID_ARG;
  for (const void* x :
       {static_cast<const void*>(a.block_table), static_cast<const void*>(a.q_descale),
        static_cast<const void*>(a.k_descale), static_cast<const void*>(a.v_descale), static_cast<const void*>(a.lse),
        static_cast<const void*>(a.status)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  const int64_t h_q = static_cast<int64_t>(p.h_k) * p.h_r;
  const int q_bytes = p.q_dtype == MJ_E4M3 ? 1 : 2;
  for (int64_t s : {a.q_tok, a.q_head})
    if (s < 0 || (s * q_bytes) % 16 != 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  if (a.o_tok < 0 || a.o_tok % 8 != 0 || a.o_tok >= kMaxStride) return MJ_ERR_INVALID_ARG;
  if (a.num_tokens > 1 && a.o_tok < h_q * kHeadDim) return MJ_ERR_INVALID_ARG;
  if (too_far(a.num_tokens, a.q_tok) || too_far(h_q, a.q_head) || too_far(a.num_tokens, a.o_tok)) return MJ_ERR_INVALID_ARG;
  for (int64_t s : {a.qd_seq, a.qd_head, a.kd_seq, a.kd_head, a.vd_seq, a.vd_head})
    if (s < 0 || s >= kMaxStride) return MJ_ERR_INVALID_ARG;
  if (heads_too_far(p.num_seqs, p.h_k, a.qd_seq, a.qd_head) || heads_too_far(p.num_seqs, p.h_k, a.kd_seq, a.kd_head) ||
      heads_too_far(p.num_seqs, p.h_k, a.vd_seq, a.vd_head))
    return MJ_ERR_INVALID_ARG;
  if (!(a.softmax_scale > 0.f) || !(a.scale_o == a.scale_o)) return MJ_ERR_INVALID_ARG;
  if (a.softcap != 0.f && !(a.softcap >= 0x1p-20f && a.softcap <= 0x1p60f)) return MJ_ERR_INVALID_ARG;
  if (a.window < 0 || (a.window > 0 && p.causal == 0)) return MJ_ERR_INVALID_ARG;
  const PlanLayout l = plan_layout(p, a.num_tokens);
  if (a.plan_bytes < l.total) return MJ_ERR_CAPACITY;
  const size_t ws = mj_prompt_workspace_bytes(params);
  if (ws > 0 && !a.workspace) return MJ_ERR_INVALID_ARG;
  if (a.workspace_bytes < ws) return MJ_ERR_CAPACITY;
  if (a.num_tokens == 0) return MJ_OK;
  const int64_t q_end = ((a.num_tokens - 1) * a.q_tok + (h_q - 1) * a.q_head + kHeadDim) * q_bytes;
  const int64_t o_end = ((a.num_tokens - 1) * a.o_tok + h_q * kHeadDim) * 2;
  const int64_t lse_end = a.num_tokens * h_q * 4;
  if (overlap(a.o, o_end, a.q, q_end)) return MJ_ERR_INVALID_ARG;
  if (a.lse && (overlap(a.lse, lse_end, a.q, q_end) || overlap(a.lse, lse_end, a.o, o_end))) return MJ_ERR_INVALID_ARG;

  PromptDev d{};
  d.q = a.q;
  d.q_rows = {0, a.q_tok, p.h_r * a.q_head, a.q_head};
  d.o = static_cast<__nv_bfloat16*>(a.o);
  d.o_rows = {0, a.o_tok, static_cast<int64_t>(p.h_r) * kHeadDim, kHeadDim};
  d.lse = a.lse;
  d.lse_rows = {0, h_q, p.h_r, 1};
  d.k = a.k;
  d.v = a.v;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.v_page = a.v_page;
  d.v_row = a.v_row;
  d.v_head = a.v_head;
  d.block_table = a.block_table;
  d.qd = a.q_descale;
  d.kd = a.k_descale;
  d.vd = a.v_descale;
  d.qd_seq = a.qd_seq;
  d.qd_head = a.qd_head;
  d.kd_seq = a.kd_seq;
  d.kd_head = a.kd_head;
  d.vd_seq = a.vd_seq;
  d.vd_head = a.vd_head;
  d.softmax_scale = a.softmax_scale;
  d.scale_o = a.scale_o;
  d.softcap = a.softcap;
  const char* const base = static_cast<const char*>(a.plan);
  d.head = reinterpret_cast<const PromptHeader*>(base);
  d.items = reinterpret_cast<const PromptItem*>(base + l.items);
  d.merges = reinterpret_cast<const PromptMerge*>(base + l.merges);
  if (ws > 0) {
    d.o_part = static_cast<float*>(a.workspace);
    d.m_part = d.o_part + part_rows(p) * kHeadDim;
    d.l_part = d.m_part + part_rows(p);
  }
  d.status = a.status;
  d.num_seqs = p.num_seqs;
  d.num_tokens = a.num_tokens;
  d.h_k = p.h_k;
  d.h_r = p.h_r;
  d.page_size = p.page_size;
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  d.causal = p.causal;
  d.window = std::min(a.window, 1 << 30);
  d.kv_evict_first = p.kv_evict_first == 1;
  d.max_splits = p.max_splits;
  // keys are cut only into parts of kPromptMinChunk tiles or more
  const bool merge = p.max_splits > 1 && static_cast<int64_t>(p.max_blocks) * p.page_size > kPromptMinChunk * 128;
  const int sms = device_sm_count();  // a CTA each: they share the items out among themselves
  if (sms < 1) return MJ_ERR_CUDA;
  const NvtxRange range("mj_prompt_attn");
  const cudaError_t e = launch_prompt_attn(d, p.q_dtype == MJ_E4M3, merge, sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}
