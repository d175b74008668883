// Attention over whole prompts: the plan's records, shared by the kernel that
// makes them (prompt_plan.cu), the attention (prompt_attn.cu) and its merge.
#pragma once

#include <cstdint>

#include "mj_device.cuh"

namespace mj {

constexpr int kPromptRows = 256;  // packed query rows of a work item
constexpr int kPromptSlots = 152; // CTAs the plan cuts for (a GB300's SMs; sizes of plans and workspaces follow from it)
constexpr int kPromptMinChunk = 4;   // tiles of the shortest piece a row tile is cut into
constexpr int kPromptSortMax = 8192; // items ordered by cost in shared memory

// 256 packed rows (row n of a sequence: token n / h_r, head n % h_r of the
// group) of one sequence, from row0 on, against the keys of tiles [t0, t1).
// part < 0: the item holds all the keys its rows see and writes O and LSE;
// else its partial results go to part `part`.
// (g0, g1): of those tiles, the ones that the first and the second 128 rows see
// any key of; g1[1] < 0: there are 128 rows at most and two tiles at least, and
// both row groups hold those rows and take the tiles in turn.
struct __align__(16) PromptItem {
  int32_t b, row0, t0, t1;
  int32_t part, tok0, n_tok, len;  // tok0: the sequence's first token in Q and O
  int32_t g0[2], g1[2];
};
// The row tile that parts part0 .. part0 + n_parts - 1 make up.
struct __align__(16) PromptMerge {
  int32_t b, row0, part0, n_parts;
  int32_t tok0, n_tok, pad0, pad1;
};
struct __align__(16) PromptHeader {
  int32_t n_items, n_merges, n_parts, chunk;
  // what it was made for: another shape's attention refuses it
  int32_t num_seqs, num_tokens, h_k, h_r, causal, window, max_splits, magic;
  int32_t page_size, max_blocks;  // (items' lengths are within these tables)
};
constexpr int32_t kPromptMagic = 0x6d6a7071;

struct PromptPlanDev {
  const int32_t* cu_tokens;
  const int32_t* seq_lens;
  int32_t num_seqs, num_tokens, h_k, h_r, causal, window, max_splits, page_size, max_blocks;
  int64_t max_len;
  PromptHeader* head;
  PromptItem* items;    // [items_cap]
  PromptItem* scratch;  // [items_cap], before they are ordered
  PromptMerge* merges;  // [slots]
  int32_t items_cap, slots;  // slots: CTAs a head's items are cut for
  int32_t* status;
};

// Rows of Q, O and LSE: token t (of all), head g * h_r + hr of sequence b at
// b * s_b + t * s_tok + g * s_g + hr * s_h (elements).
struct PromptRows {
  int64_t s_b, s_tok, s_g, s_h;
};
__device__ __forceinline__ int64_t prompt_at(const PromptRows& s, int b, int tok, int g, int hr) {
  return b * s.s_b + tok * s.s_tok + g * s.s_g + hr * s.s_h;
}

struct PromptDev {
  const void* q;
  PromptRows q_rows, o_rows, lse_rows;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;
  const int32_t* block_table;
  const float* qd;
  const float* kd;
  const float* vd;
  int64_t qd_seq, qd_head, kd_seq, kd_head, vd_seq, vd_head;
  float softmax_scale, scale_o, softcap;
  __nv_bfloat16* o;
  float* lse;  // or null
  const PromptHeader* head;
  const PromptItem* items;
  const PromptMerge* merges;
  float* o_part;  // [part][g][256][128]
  float* m_part;  // [part][g][256]
  float* l_part;
  int32_t* status;
  int32_t num_seqs, num_tokens, h_k, h_r, page_size, max_blocks, num_pages, causal, window, kv_evict_first, max_splits;
};

// The plan was made for this call's shape.
__device__ __forceinline__ bool prompt_plan_fits(const PromptDev& a) {
  const PromptHeader& h = *a.head;
  return h.magic == kPromptMagic && h.num_seqs == a.num_seqs && h.num_tokens == a.num_tokens && h.h_k == a.h_k &&
         h.h_r == a.h_r && h.causal == a.causal && h.window == a.window && h.max_splits == a.max_splits && h.page_size == a.page_size &&
         h.max_blocks == a.max_blocks;
}

// The same kernel over a decode plan's work items (mj_decode_attn_tree above 128
// rows): packed rows, context keys by ranges, the last keys a drafted tree's.
// Q, O and LSE rows as above (b, token of q_len, kv head, head of the group);
// parts as the decode merge reads them.
struct PromptTreeDev : PromptDev {
  DecodeTreeDev t;
  int32_t n_q_tiles;  // of 256 rows
};

// Keys [first, last] that tokens [i0, i1] of a sequence (n_tok new ones at the
// end of len keys) see between them; last < first: none.
__host__ __device__ __forceinline__ void prompt_range(int len, int n_tok, int i0, int i1, int causal, int window,
                                                      int* first, int* last) {
  const int p0 = len - n_tok + i0, p1 = len - n_tok + i1;
  *last = causal && p1 < len - 1 ? p1 : len - 1;
  *first = 0;
  if (window > 0) {
    const int w = p0 - window + 1;  // window <= 2^30: no overflow
    *first = w > 0 ? w : 0;
  }
}

// The tiles of 128 keys that rows [row0, row0 + rows) see any key of (t1 == t0:
// none).
__host__ __device__ __forceinline__ void prompt_tiles(int len, int n_tok, int h_r, int row0, int rows, int causal,
                                                      int window, int* t0, int* t1) {
  const int end = n_tok * h_r;  // checked to fit
  *t0 = *t1 = 0;
  if (row0 >= end) return;
  const int last_row = (row0 + rows < end ? row0 + rows : end) - 1;
  int first, last;
  prompt_range(len, n_tok, row0 / h_r, last_row / h_r, causal, window, &first, &last);
  if (last < first) return;
  *t0 = first / 128;
  *t1 = last / 128 + 1;
}

}  // namespace mj
