// Sliding-window attention with sinks (the first n_sink tokens stay visible):
// what its kernels share, dense and over a paged cache.
#pragma once
#include "paged_index.h"
#include "ptx.cuh"

namespace ttcd {

// K and V of dense sequences [B, T, Hkv, HD] and of a paged cache
// [n_pages, Hkv, page_size, HD] through a table [n_seq, max_pages].
struct PagedCache {
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int* table;
  int max_pages, n_pages, page_log2, Hkv;
};

// The ragged batch of a paged call.
struct Ragged {
  const int* q_start;  // [n_seq + 1]
  const int* kv_len;   // [n_seq], the new tokens included
  int n_seq, total_q;
};

__device__ __forceinline__ SeqSpan load_span(const Ragged& r, int s, long long capacity) {
  return seq_span(r.q_start[s], r.q_start[s + 1], r.kv_len[s], r.total_q, capacity);
}

// Sequence whose first tile slot is the last one not beyond `slot` (one warp,
// every lane gets the answer; -1: none).
__device__ __forceinline__ int find_seq(const Ragged& r, long long slot, int tpt) {
  const int lane = threadIdx.x & 31;
  int last = -1;
  for (int s0 = 0; s0 < r.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < r.n_seq && tile_slot(r.q_start[s], s, tpt) <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (m) last = s0 + 31 - __clz(m);
    if (m != 0xffffffffu) break;
  }
  return last;
}

// Sequence of a slot of the further units (those after a sequence's first): the
// last one whose first such slot is not beyond it.
__device__ __forceinline__ int find_extra_seq(const Ragged& r, int slot, int tpt) {
  const int lane = threadIdx.x & 31;
  int last = -1;
  for (int s0 = 0; s0 < r.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, s < r.n_seq && extra_slot(r.q_start[s], tpt) <= slot);
    if (m) last = s0 + 31 - __clz(m);
    if (m != 0xffffffffu) break;
  }
  return last;
}

// Sequence of a row of the packed queries: the last one that begins at or before
// it (one warp, every lane gets the answer; -1: none).
__device__ __forceinline__ int seq_of_row(const Ragged& r, int row) {
  const int lane = threadIdx.x & 31;
  int last = -1;
  for (int s0 = 0; s0 < r.n_seq; s0 += 32) {
    const int s = s0 + lane;
    const unsigned m = __ballot_sync(0xffffffffu, s < r.n_seq && r.q_start[s] <= row);
    if (m) last = s0 + 31 - __clz(m);
    if (m != 0xffffffffu) break;
  }
  return last;
}

}  // namespace ttcd
