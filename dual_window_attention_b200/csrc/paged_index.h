// Index arithmetic of the sink-window and paged attention: which rows a tile of
// queries holds, which keys it sees, and where a key lies in a paged cache.
// Plain C++ for host and device, so that it is checked on the CPU.
//
// Mask: the query at position t sees key j iff j <= t and (j > t - window or
// j < n_sink).
#pragma once

#ifdef __CUDACC__
#define TTCD_HD __host__ __device__ __forceinline__
#else
#define TTCD_HD inline
#endif

namespace ttcd {

// One sequence of a ragged batch: its rows [q0, q0 + n) of the packed queries
// and L keys in the cache, the new tokens included, so that its token i has
// position L - n + i.  n = 0 for a sequence that is skipped (none of its rows
// or keys is touched): no new tokens, or inconsistent numbers (bad = true).
struct SeqSpan {
  int q0, n, L;
  bool bad;
};
TTCD_HD SeqSpan seq_span(int begin, int end, int kv_len, int total_q, long long capacity) {
  SeqSpan s{begin, 0, 0, false};
  if (begin < 0 || end < begin || end > total_q) {
    s.bad = true;
  } else if (end > begin) {
    if (kv_len < end - begin || kv_len > capacity) {
      s.bad = true;
    } else {
      s.n = end - begin;
      s.L = kv_len;
    }
  }
  return s;
}

// Which token of its sequence the row `row` >= 0 of the packed queries is; -1 for
// padding and for the rows of a sequence that is skipped, whose q0 may be any number
// (row - q0 is formed only where it cannot overflow).
TTCD_HD int row_token(const SeqSpan& s, int row) {
  return s.n > 0 && row >= s.q0 && row - s.q0 < s.n ? row - s.q0 : -1;
}

// Query tiles of tpt tokens.  Sequence s's tiles have the slots
// tile_slot(q_start[s], s) .. + ceil(n / tpt) - 1; the slots of two sequences
// never meet, because floor((a + n) / tpt) + 1 >= floor(a / tpt) + ceil(n / tpt),
// and they all lie below tile_slots(total_q, n_seq), so that a grid can be sized
// without the lengths.  A slot belongs to the last sequence whose first slot is
// not beyond it (and to none if that sequence has fewer tiles).
TTCD_HD long long tile_slot(int q_start, int s, int tpt) {
  return static_cast<long long>(q_start / tpt) + s;
}
TTCD_HD long long tile_slots(int total_q, int n_seq, int tpt) {
  return static_cast<long long>(total_q / tpt) + n_seq;
}

// Units of tpt tokens, another numbering: the first unit of sequence s has slot s,
// and its unit i >= 1 slot n_seq + extra_slot(q_start[s]) + i - 1.  These do not
// meet either, because floor((a + n) / tpt) >= floor(a / tpt) + ceil(n / tpt) - 1,
// and lie below n_seq + total_q / tpt; such a slot belongs to the last sequence
// whose first one is not beyond it (and to none if that has fewer units).
TTCD_HD int extra_slot(int q_start, int tpt) { return q_start / tpt; }
// First token of the unit at extra slot x of a sequence that begins at q_start.
TTCD_HD int extra_token(int x, int q_start, int tpt) {
  const long long t = (static_cast<long long>(x) - extra_slot(q_start, tpt) + 1) * tpt;
  return t < (1 << 30) ? static_cast<int>(t) : (1 << 30);
}

// Keys that a tile with the positions [t_lo, t_hi] sees: [lo, t_hi] and the
// sinks [0, sink_end) before lo.
struct KeyRange {
  int lo, hi, sink_end;
};
TTCD_HD KeyRange key_range(int t_lo, int t_hi, int window, int n_sink) {
  KeyRange r;
  r.lo = t_lo - window + 1 > 0 ? t_lo - window + 1 : 0;  // window <= 2^30: no overflow
  r.hi = t_hi;
  r.sink_end = n_sink < r.lo ? n_sink : r.lo;
  return r;
}
TTCD_HD bool in_range(const KeyRange& r, int j) {
  return (j >= r.lo && j <= r.hi) || (j >= 0 && j < r.sink_end);
}
// Whether any key of [a, b] is seen.
TTCD_HD bool touches(const KeyRange& r, int a, int b) {
  return (b >= r.lo && a <= r.hi) || (b >= 0 && a < r.sink_end);
}

// Row of key 0 of (page, head) in the cache seen as rows of head_dim elements
// ([n_pages, Hkv, page_size] rows), or -1 for a page that does not exist.
TTCD_HD long long page_row(int page, int n_pages, int Hkv, int head, int page_size) {
  if (page < 0 || page >= n_pages) return -1;
  return (static_cast<long long>(page) * Hkv + head) * page_size;
}

}  // namespace ttcd
