// What the paged cache's translation units share (tp_kv_append.cu, tp_paged_attention.cu): checks
// of the caller's structures, and their reading on the device.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "tp_internal.h"

namespace tp {

// A batch as the kernels read it.  The three arrays are device memory that only the kernels see:
// every value is taken within bounds, and one that is not is recorded in the status word.
struct BatchView {
  const int32_t* seq_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int64_t ld_table;
  int n_seqs, max_new, T;
  int max_keys;    // max_pages * page_size
  int n_pages;
  int page_size, page_shift;
  unsigned int* status;
};

// Checks of the structures and sizes that both calls take; *empty: nothing to do.
tp_status check_paged(const tp_paged_cache* c, const tp_paged_batch* b, int64_t T, int n_heads, bool* empty);
BatchView batch_view(const tp_paged_cache& c, const tp_paged_batch& b, int64_t T, unsigned int* status);

#ifdef __CUDACC__
// Sequence s: rows [a, a + n) of the call, `len` keys in its pages, first row at position pos0
// (negative where the sequence claims fewer tokens than it has rows).
struct SeqView {
  int a, n, len, pos0;
};

__device__ __forceinline__ void bad_index(const BatchView& b) { atomicOr(b.status, TP_DEVSTATUS_INDEX); }

__device__ __forceinline__ SeqView seq_view(const BatchView& b, int s) {
  const int a = b.seq_start[s], e = b.seq_start[s + 1], len = b.kv_len[s];
  SeqView v{0, 0, 0, 0};
  if (a < 0 || e < a || e > b.T || len < 0 || len > (1 << 30)) {
    bad_index(b);
    return v;
  }
  v.a = a;
  v.n = e - a;
  v.len = len;
  v.pos0 = len - v.n;
  if (v.n > b.max_new) {
    v.n = b.max_new;
    bad_index(b);
  }
  if (v.len > b.max_keys) {
    v.len = b.max_keys;
    bad_index(b);
  }
  return v;
}

// The sequence that owns slot u of a numbering in which sequence s has the slots from
// base(s) = seq_start[s] / per + gap * s on: rows are cut into blocks of `per` (P rows of
// sequence s never need more than base(s + 1) - base(s) blocks for gap large enough), and
// no prefix sum over the sequences is needed.  Warp-collective: 32 sequences are probed at once.
// Returns -1 where u lies before the first sequence; a u behind the last belongs to the last.
__device__ __forceinline__ int find_sequence(const BatchView& b, int64_t u, int per, int gap, int lane) {
  int lo = -1, hi = b.n_seqs;   // base(lo) <= u (or lo = -1), base(hi) > u or hi = n_seqs
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;   // probes lo + step, lo + 2 step, ... below hi
    const int64_t s = static_cast<int64_t>(lo) + static_cast<int64_t>(step) * (lane + 1);
    bool below = false;
    if (s < hi) below = static_cast<int64_t>(max(b.seq_start[s], 0)) / per + static_cast<int64_t>(gap) * s <= u;
    const int n = __popc(__ballot_sync(0xffffffffu, below));   // starts ascend: the lanes below form a prefix
    hi = static_cast<int>(min(static_cast<int64_t>(hi), static_cast<int64_t>(lo) + static_cast<int64_t>(step) * (n + 1)));
    lo += step * n;
  }
  return lo;
}
#endif

}  // namespace tp
