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

template <int HD>
__device__ __forceinline__ void ld_lane(const __nv_bfloat16* row, int lane, float (&x)[HD / 32]) {
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) x[i] = __bfloat162float(row[lane * (HD / 32) + i]);
}
template <int HD>
__device__ __forceinline__ float warp_dot(const float (&a)[HD / 32], const float (&b)[HD / 32]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Backward, one warp per (query row, head): dq.
template <int HD>
__global__ void sink_attn_dq_simple_kernel(const __nv_bfloat16* q, const __nv_bfloat16* k,
                                           const __nv_bfloat16* v, const __nv_bfloat16* o,
                                           const float* lse, const __nv_bfloat16* d_o,
                                           __nv_bfloat16* dq, int B, int T, int Hq, int Hkv,
                                           int window, int n_sink, float scale) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (item >= static_cast<long long>(B) * T * Hq) return;
  const long long row = item / Hq;
  const int h = static_cast<int>(item % Hq), g = h / (Hq / Hkv);
  const int b = static_cast<int>(row / T), t = static_cast<int>(row % T);
  float qf[E], of[E], gf[E], acc[E] = {};
  ld_lane<HD>(q + item * HD, lane, qf);
  ld_lane<HD>(o + item * HD, lane, of);
  ld_lane<HD>(d_o + item * HD, lane, gf);
  const float delta = warp_dot<HD>(of, gf);
  const float ls = lse[(static_cast<long long>(b) * Hq + h) * T + t];
  const KeyRange kr = key_range(t, t, window, n_sink);
  for (int j = 0; j <= kr.hi; ++j) {
    if (j == kr.sink_end && j < kr.lo) j = kr.lo;
    const long long off = ((static_cast<long long>(b) * T + j) * Hkv + g) * HD;
    float kf[E], vf[E];
    ld_lane<HD>(k + off, lane, kf);
    ld_lane<HD>(v + off, lane, vf);
    const float p = __expf(warp_dot<HD>(qf, kf) * scale - ls);
    const float ds = p * (warp_dot<HD>(gf, vf) - delta) * scale;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(ds, kf[i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) dq[item * HD + lane * E + i] = __float2bfloat16_rn(acc[i]);
}

// Backward, one warp per (key row, KV head): dk and dv.
template <int HD>
__global__ void sink_attn_dkv_simple_kernel(const __nv_bfloat16* q, const __nv_bfloat16* k,
                                            const __nv_bfloat16* v, const __nv_bfloat16* o,
                                            const float* lse, const __nv_bfloat16* d_o,
                                            __nv_bfloat16* dk, __nv_bfloat16* dv, int B, int T,
                                            int Hq, int Hkv, int window, int n_sink, float scale) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (item >= static_cast<long long>(B) * T * Hkv) return;
  const long long row = item / Hkv;
  const int g = static_cast<int>(item % Hkv), G = Hq / Hkv;
  const int b = static_cast<int>(row / T), j = static_cast<int>(row % T);
  float kf[E], vf[E], ak[E] = {}, av[E] = {};
  ld_lane<HD>(k + item * HD, lane, kf);
  ld_lane<HD>(v + item * HD, lane, vf);
  const int t_end = j < n_sink || window > T - j ? T : j + window;
  for (int h = g * G; h < (g + 1) * G; ++h)
    for (int t = j; t < t_end; ++t) {
      const long long off = ((static_cast<long long>(b) * T + t) * Hq + h) * HD;
      float qf[E], of[E], gf[E];
      ld_lane<HD>(q + off, lane, qf);
      ld_lane<HD>(o + off, lane, of);
      ld_lane<HD>(d_o + off, lane, gf);
      const float ls = lse[(static_cast<long long>(b) * Hq + h) * T + t];
      const float p = __expf(warp_dot<HD>(qf, kf) * scale - ls);
      const float ds = p * (warp_dot<HD>(gf, vf) - warp_dot<HD>(of, gf)) * scale;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        ak[i] = fmaf(ds, qf[i], ak[i]);
        av[i] = fmaf(p, gf[i], av[i]);
      }
    }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    dk[item * HD + lane * E + i] = __float2bfloat16_rn(ak[i]);
    dv[item * HD + lane * E + i] = __float2bfloat16_rn(av[i]);
  }
}

}  // namespace ttcd
