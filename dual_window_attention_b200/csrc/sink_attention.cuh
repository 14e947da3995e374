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

// The last s of [0, n) that holds(s) is true of, for a condition that is true up to
// some s and false from there on (-1: of none).  One warp, every lane gets the answer:
// 32 probes at a time, so 1024 sequences take two loads one after the other (one
// by one in steps of 32 they took 32: 10.5 us for a write of 1024 tokens).  For lengths that
// cannot be, which break the order, any answer in range will do.
template <class Holds>
__device__ __forceinline__ int last_where(int n, Holds holds) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  for (;;) {
    const int step = (len + 31) >> 5, x = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, x < len && holds(lo + x));
    if (!m) return -1;
    const int at = (31 - __clz(m)) * step;
    lo += at;
    if (step == 1) return lo;
    len = min(step, len - at);
  }
}

// Sequence whose first tile slot is the last one not beyond `slot`.
__device__ __forceinline__ int find_seq(const Ragged& r, long long slot, int tpt) {
  return last_where(r.n_seq, [&](int s) { return tile_slot(r.q_start[s], s, tpt) <= slot; });
}

// Sequence of a slot of the further units (those after a sequence's first): the
// last one whose first such slot is not beyond it.
__device__ __forceinline__ int find_extra_seq(const Ragged& r, int slot, int tpt) {
  return last_where(r.n_seq, [&](int s) { return extra_slot(r.q_start[s], tpt) <= slot; });
}

// Sequence of a row of the packed queries: the last one that begins at or before it.
__device__ __forceinline__ int seq_of_row(const Ragged& r, int row) {
  return last_where(r.n_seq, [&](int s) { return r.q_start[s] <= row; });
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// Keeps the scores of N columns (a multiple of 32) whose bit is set, the others
// become -inf; word(k) has the bits of the columns 32 k ...: two instructions per
// score, where the comparisons themselves would be six.
template <int N, class Word>
__device__ __forceinline__ void mask_scores(float (&s)[N], Word word) {
#pragma unroll
  for (int k = 0; k < N / 32; ++k) {
    const uint32_t w = word(k);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[32 * k + i] = (w >> i) & 1u ? s[32 * k + i] : -INFINITY;
  }
}
// What the rounding of a pair to `hi` leaves, as bf16.
__device__ __forceinline__ uint32_t rest2(float a, float b, uint32_t hi) {
  return pack_bf16x2(a - bf16lo_to_f32(hi), b - bf16hi_to_f32(hi));
}
// The columns of keys k0 .. k0 + 31 that the query at t sees.
__device__ __forceinline__ uint32_t seen_bits(int t, int k0, int window, int n_sink) {
  return low_bits(t + 1 - k0) & (~low_bits(t - window + 1 - k0) | low_bits(n_sink - k0));
}

}  // namespace ttcd
