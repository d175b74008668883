// C ABI entry points of the cache's pages and of a drafted tree's accepted
// branch: argument checks and launches.

#include <cuda_runtime.h>

#include <utility>

#include "mj.h"
#include "mj_checks.h"
#include "mj_internal.h"
#include "mj_kernels.h"

namespace mj {
namespace {

// entries of the free list, and tokens of a call: the kernels' threads count past
// them in int32 by a few thousand
constexpr int32_t kMaxEntries = 1 << 30;

mj_status check_pages(const mj_page_params* p) {
  if (!p) return MJ_ERR_INVALID_ARG;
  if (p->num_seqs < 1 || p->max_blocks < 1 || p->num_pages < 1) return MJ_ERR_INVALID_ARG;
  if (!page_size_ok(p->page_size) || p->num_seqs > kMaxDevicePlanSeqs) return MJ_ERR_UNSUPPORTED;
  if (p->num_pages > kMaxEntries || static_cast<int64_t>(p->max_blocks) * p->page_size > (int64_t{1} << 30)) return MJ_ERR_UNSUPPORTED;
  return MJ_OK;
}

int shift_of(int page_size) {
  int s = 4;
  while ((1 << s) < page_size) ++s;
  return s;
}

PagesDev pages_dev(const mj_page_params& p) {
  PagesDev d{};
  d.num_seqs = p.num_seqs;
  d.page_shift = shift_of(p.page_size);
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  d.max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  return d;
}

}  // namespace
}  // namespace mj

using namespace mj;

extern "C" mj_status mj_pages_reserve(const mj_page_params* params, const mj_reserve_args* args, mj_stream_t stream) {
  const mj_status st = check_pages(params);
  if (st != MJ_OK) return st;
  if (!args) return MJ_ERR_INVALID_ARG;
  const mj_page_params& p = *params;
  const mj_reserve_args& a = *args;
  if (!a.seq_lens || !a.free_pages || !a.num_free || !a.num_free_out || !a.block_table || !a.seq_lens_out)
    return MJ_ERR_INVALID_ARG;
  if ((!a.new_tokens && a.q_len < 1) || a.num_tokens < 0) return MJ_ERR_INVALID_ARG;
  if (a.num_tokens > kMaxEntries) return MJ_ERR_UNSUPPORTED;
  for (const void* x :
       {static_cast<const void*>(a.seq_lens), static_cast<const void*>(a.new_tokens),
        static_cast<const void*>(a.free_pages), static_cast<const void*>(a.num_free),
        static_cast<const void*>(a.num_free_out), static_cast<const void*>(a.block_table),
        static_cast<const void*>(a.seq_lens_out), static_cast<const void*>(a.cu_tokens),
        static_cast<const void*>(a.positions), static_cast<const void*>(a.status), static_cast<const void*>(a.granted)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a.slots) & 7) != 0) return MJ_ERR_INVALID_ARG;
  // an output over an input is refused, but for the lengths and the list's size (the first two outputs) in place
  const int64_t lens = static_cast<int64_t>(p.num_seqs) * 4, list = static_cast<int64_t>(p.num_pages) * 4;
  const int64_t table = static_cast<int64_t>(p.num_seqs) * p.max_blocks * 4, tokens = a.num_tokens;
  const struct {
    const void* at;
    int64_t bytes;
  } ins[] = {{a.seq_lens, lens}, {a.new_tokens, lens}, {a.free_pages, list}, {a.num_free, 4}},
    outs[] = {{a.seq_lens_out, lens}, {a.num_free_out, 4},           {a.block_table, table},
              {a.cu_tokens, lens + 4}, {a.positions, tokens * 4}, {a.slots, tokens * 8}, {a.granted, lens}};
  for (const auto& o : outs) {
    if (!o.at) continue;
    for (const auto& i : ins) {
      const bool same = o.at == i.at && ((&o == &outs[0] && &i == &ins[0]) || (&o == &outs[1] && &i == &ins[3]));
      if (i.at && !same && overlap(o.at, o.bytes, i.at, i.bytes)) return MJ_ERR_INVALID_ARG;
    }
    for (const auto& q : outs)
      if (&q != &o && q.at && overlap(o.at, o.bytes, q.at, q.bytes)) return MJ_ERR_INVALID_ARG;
  }
  PagesDev d = pages_dev(p);
  d.seq_lens = a.seq_lens;
  d.new_tokens = a.new_tokens;
  d.q_len = a.q_len;
  d.free_pages = a.free_pages;
  d.num_free = a.num_free;
  d.num_free_out = a.num_free_out;
  d.block_table = a.block_table;
  d.block_table_out = a.block_table;
  d.seq_lens_out = a.seq_lens_out;
  d.cu_tokens = a.cu_tokens;
  d.positions = a.positions;
  d.slots = a.slots;
  d.granted = a.granted;
  d.num_tokens = a.num_tokens;
  d.status = a.status;
  const NvtxRange range("mj_pages_reserve");
  return launch_pages_reserve(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_pages_release(const mj_page_params* params, const mj_release_args* args, mj_stream_t stream) {
  const mj_status st = check_pages(params);
  if (st != MJ_OK) return st;
  if (!args) return MJ_ERR_INVALID_ARG;
  const mj_page_params& p = *params;
  const mj_release_args& a = *args;
  if (!a.seq_lens || !a.keep_lens || !a.free_pages || !a.num_free || !a.num_free_out || !a.block_table)
    return MJ_ERR_INVALID_ARG;
  for (const void* x :
       {static_cast<const void*>(a.seq_lens), static_cast<const void*>(a.keep_lens),
        static_cast<const void*>(a.free_pages), static_cast<const void*>(a.num_free),
        static_cast<const void*>(a.num_free_out), static_cast<const void*>(a.block_table),
        static_cast<const void*>(a.status)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  const int64_t lens = static_cast<int64_t>(p.num_seqs) * 4, list = static_cast<int64_t>(p.num_pages) * 4;
  const int64_t table = static_cast<int64_t>(p.num_seqs) * p.max_blocks * 4;
  for (const auto& [at, bytes] : {std::pair<const void*, int64_t>{a.seq_lens, lens}, {a.keep_lens, lens}, {a.block_table, table}})
    if (overlap(a.free_pages, list, at, bytes) || overlap(a.num_free_out, 4, at, bytes)) return MJ_ERR_INVALID_ARG;
  if (overlap(a.free_pages, list, a.num_free, 4) || overlap(a.free_pages, list, a.num_free_out, 4))
    return MJ_ERR_INVALID_ARG;
  PagesDev d = pages_dev(p);
  d.seq_lens = a.seq_lens;
  d.new_tokens = a.keep_lens;
  d.free_pages = a.free_pages;
  d.free_pages_out = a.free_pages;
  d.num_free = a.num_free;
  d.num_free_out = a.num_free_out;
  d.block_table = a.block_table;
  d.status = a.status;
  const NvtxRange range("mj_pages_release");
  return launch_pages_release(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}

extern "C" mj_status mj_tree_commit(const mj_decode_params* params, const mj_commit_args* args, mj_stream_t stream) {
  if (!params || !args) return MJ_ERR_INVALID_ARG;
  mj_decode_params p = *params;
  p.h_r = 1;  // not looked at
  p.kernel = MJ_KERNEL_AUTO;
  if (p.kv_format == MJ_KV_NVFP4) {  // its limits are the decode kernels'
    p.q_dtype = MJ_E4M3;
    p.q_len = 1;
  }
  const mj_status st = check_params(&p);
  if (st != MJ_OK) return st;
  p.q_len = params->q_len;
  const mj_commit_args& a = *args;
  if (!a.k || !a.v || !a.block_table || !a.seq_lens || !a.accepted || !a.num_accepted || !a.new_lens)
    return MJ_ERR_INVALID_ARG;
  if (p.q_len < 1 || a.max_accept < 1) return MJ_ERR_INVALID_ARG;
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
       {static_cast<const void*>(a.block_table), static_cast<const void*>(a.seq_lens),
        static_cast<const void*>(a.tree_lens), static_cast<const void*>(a.accepted),
        static_cast<const void*>(a.num_accepted), static_cast<const void*>(a.new_lens),
        static_cast<const void*>(a.key_pos), static_cast<const void*>(a.status)})
    if (!aligned4(x)) return MJ_ERR_INVALID_ARG;
  if (pool_too_far(p.num_pages, p.page_size, p.h_k, a.k_page, a.k_row, a.k_head) ||
      pool_too_far(p.num_pages, p.page_size, p.h_k, a.v_page, a.v_row, a.v_head) ||
      (p.kv_format == MJ_KV_NVFP4 && (pool_too_far(p.num_pages, 1, p.h_k, a.ks_page, 0, a.ks_head) ||
                                      pool_too_far(p.num_pages, 1, p.h_k, a.vs_page, 0, a.vs_head))))
    return MJ_ERR_INVALID_ARG;
  const int64_t max_len = static_cast<int64_t>(p.max_blocks) * p.page_size;
  if (a.key_pos) {
    if (a.kp_seq < 0 || a.kp_head < 0 || a.kp_seq >= kMaxStride || a.kp_head >= kMaxStride) return MJ_ERR_INVALID_ARG;
    if (heads_too_far(p.num_seqs, p.h_k, a.kp_seq, a.kp_head)) return MJ_ERR_INVALID_ARG;
    // planes of their own, or one a sequence for all heads
    if (!planes_apart(p.num_seqs, a.kp_head == 0 ? 1 : p.h_k, a.kp_seq, a.kp_head, max_len)) return MJ_ERR_INVALID_ARG;
  }
  const int64_t lens = static_cast<int64_t>(p.num_seqs) * 4;
  const bool in_place = a.new_lens == a.seq_lens;
  if ((!in_place && overlap(a.new_lens, lens, a.seq_lens, lens)) || overlap(a.new_lens, lens, a.num_accepted, lens) ||
      overlap(a.new_lens, lens, a.accepted, lens * a.max_accept) ||
      (a.tree_lens && overlap(a.new_lens, lens, a.tree_lens, lens)) ||
      overlap(a.new_lens, lens, a.block_table, lens * p.max_blocks))
    return MJ_ERR_INVALID_ARG;
  CommitDev d{};
  d.k = a.k;
  d.v = a.v;
  d.k_page = a.k_page;
  d.k_row = a.k_row;
  d.k_head = a.k_head;
  d.v_page = a.v_page;
  d.v_row = a.v_row;
  d.v_head = a.v_head;
  if (p.kv_format == MJ_KV_NVFP4) {
    d.ks = a.k_scales;
    d.vs = a.v_scales;
    d.ks_page = a.ks_page;
    d.ks_head = a.ks_head;
    d.vs_page = a.vs_page;
    d.vs_head = a.vs_head;
  }
  d.block_table = a.block_table;
  d.seq_lens = a.seq_lens;
  d.tree_lens = a.tree_lens;
  d.accepted = a.accepted;
  d.num_accepted = a.num_accepted;
  d.new_lens = a.new_lens;
  d.key_pos = a.key_pos;
  d.kp_seq = a.kp_seq;
  d.kp_head = a.kp_head;
  d.status = a.status;
  d.max_len = max_len;
  d.num_seqs = p.num_seqs;
  d.q_len = p.q_len;
  d.max_accept = a.max_accept;
  d.h_k = p.h_k;
  d.row_bytes = 16 * kv_bits(p.kv_format);
  d.page_shift = shift_of(p.page_size);
  d.max_blocks = p.max_blocks;
  d.num_pages = p.num_pages;
  const NvtxRange range("mj_tree_commit");
  return launch_tree_commit(d, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MJ_OK : MJ_ERR_CUDA;
}
