// Argument checks and the profiler range shared by the operators' entry points.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <cstdint>

namespace mj {

inline constexpr int64_t kMaxStride = int64_t{1} << 40;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// n elements `stride` apart reach past any memory (the offsets below and in
// the kernels are 64-bit)
inline bool too_far(int64_t n, int64_t stride) { return n > 1 && stride > (int64_t{1} << 44) / (n - 1); }

// [a, a + an) and [b, b + bn) share a byte
inline bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

// the same of a pool's pages, rows and heads, or of a (sequence, head) array
inline bool pool_too_far(int num_pages, int page_size, int h_k, int64_t page, int64_t row, int64_t head) {
  return too_far(num_pages, page) || too_far(page_size, row) || too_far(h_k, head);
}
inline bool heads_too_far(int num_seqs, int h_k, int64_t seq, int64_t head) {
  return too_far(num_seqs, seq) || too_far(h_k, head);
}

// The planes of `len` slots at b*seq + g*head (b < num_seqs, g < h_k) have no
// slot in common: each index's step passes all that the other one reaches.
inline bool planes_apart(int num_seqs, int h_k, int64_t seq, int64_t head, int64_t len) {
  if (num_seqs == 1) return h_k == 1 || head >= len;
  if (h_k == 1) return seq >= len;
  return (head >= len && seq >= (h_k - 1) * head + len) || (seq >= len && head >= (num_seqs - 1) * seq + len);
}

inline bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }

// An NVTX range around a call's launches, so a profiler's timeline names them.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

}  // namespace mj
