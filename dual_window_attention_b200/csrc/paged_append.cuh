// New tokens into a paged cache: rotary positions on q and k, K and V rows into
// their pages, one pass over the projected rows.
//
// Row r of qkv (Hq + 2 Hkv heads of hd) is token i = r - q_start[s] of sequence
// s, at position p = kv_len[s] - n + i.  Rotate-half rotary embedding: the pair
// (x_i, x_{i + hd/2}) turns by the angle p theta^(-2i/hd).  q goes to q_out
// [rows, Hq, hd]; k and v go to row p % page_size of page table[s][p / page_size]
// in [n_pages, Hkv, page_size, hd].
//
// Angles: theta^(-2i/hd) / 2 pi and its product with p in 64 bits, reduced to a
// fraction of a turn there, then sincospi in 32 bits: at p = 10^6 a 32-bit
// product alone would be off by 0.06 radians.
//
// Bound by DRAM: each row is read once and written once (16 bytes per thread
// and access); the angles of a token are formed once for all its heads.
#pragma once
#include "sink_attention.cuh"

namespace ttcd {

constexpr int APPEND_THREADS = 256;

struct AppendArgs {
  const __nv_bfloat16* qkv;  // [total_q, (Hq + 2 Hkv) hd]
  __nv_bfloat16* q_out;      // [total_q, Hq, hd]
  __nv_bfloat16* k_pages;    // [n_pages, Hkv, page_size, hd]
  __nv_bfloat16* v_pages;
  const int* table;          // [n_seq, max_pages]
  Ragged rg;
  int max_pages, n_pages, page_log2, Hq, Hkv, hd;
  double log2_theta;  // log2 of the base
  bool rotate;
};

// TOK tokens per block and turn of its loop.
template <int TOK>
__global__ void __launch_bounds__(APPEND_THREADS) paged_append_kernel(const AppendArgs a,
                                                                      uint32_t* err) {
  __shared__ double freq[64];       // turns per position
  __shared__ float2 cs[TOK][64];    // cos, sin
  __shared__ int pos[TOK];          // -1: no token here
  __shared__ long long kv_row[TOK]; // row of (page, head 0), -1: no page
  const int half = a.hd / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page_size = 1 << a.page_log2;
  if (threadIdx.x < half)
    freq[threadIdx.x] =
        exp2(-2.0 * threadIdx.x / a.hd * a.log2_theta) * 0.15915494309189533577;  // 1 / 2 pi
  if (blockIdx.x == 0) {  // every sequence's numbers are consistent, or this call says so
    const long long cap = static_cast<long long>(a.max_pages) << a.page_log2;
    for (int s = threadIdx.x; s < a.rg.n_seq; s += APPEND_THREADS)
      if (load_span(a.rg, s, cap).bad) atomicOr(err, DEV_ERR_BAD_INDEX);
  }
  const int rope_units = (a.Hq + a.Hkv) * (half / 8), units = rope_units + a.Hkv * (a.hd / 8);
  for (int row0 = blockIdx.x * TOK; row0 < a.rg.total_q; row0 += gridDim.x * TOK) {
    if (warp < TOK) {  // whose token, where
      const int row = row0 + warp;
      const int s = seq_of_row(a.rg, row);
      int p = -1;
      long long r = -1;
      if (s >= 0 && row < a.rg.total_q) {
        const SeqSpan sp = load_span(a.rg, s, static_cast<long long>(a.max_pages) << a.page_log2);
        if (row - sp.q0 < sp.n) {
          p = sp.L - sp.n + row - sp.q0;
          const int id = a.table[static_cast<long long>(s) * a.max_pages + (p >> a.page_log2)];
          r = page_row(id, a.n_pages, a.Hkv, 0, page_size);
          if (r < 0 && lane == 0) atomicOr(err, DEV_ERR_BAD_INDEX);
        }
      }
      if (lane == 0) {
        pos[warp] = p;
        kv_row[warp] = r;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < TOK * half; e += APPEND_THREADS) {
      const int tk = e / half, i = e % half;
      float2 c = make_float2(1.f, 0.f);
      if (a.rotate && pos[tk] >= 0) {
        const double turns = pos[tk] * freq[i];
        sincospif(2.f * static_cast<float>(turns - rint(turns)), &c.y, &c.x);
      }
      cs[tk][i] = c;
    }
    __syncthreads();
    for (int u = threadIdx.x; u < TOK * units; u += APPEND_THREADS) {
      const int tk = u / units, w = u % units;
      const int p = pos[tk];
      if (p < 0) continue;
      const long long row = row0 + tk;
      const __nv_bfloat16* src = a.qkv + row * (a.Hq + 2 * a.Hkv) * a.hd;
      const long long in_page = p & (page_size - 1);
      if (w < rope_units) {
        const int head = w / (half / 8), i = (w % (half / 8)) * 8;
        float x[8], y[8];
        ld8f(src + head * a.hd + i, x);
        ld8f(src + head * a.hd + half + i, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 c = cs[tk][i + e];
          const float x0 = x[e];
          x[e] = x0 * c.x - y[e] * c.y;
          y[e] = y[e] * c.x + x0 * c.y;
        }
        __nv_bfloat16* dst;
        if (head < a.Hq) {
          dst = a.q_out + (row * a.Hq + head) * a.hd;
        } else {
          if (kv_row[tk] < 0) continue;
          dst = a.k_pages +
                (kv_row[tk] + static_cast<long long>(head - a.Hq) * page_size + in_page) * a.hd;
        }
        st8f(dst + i, x);
        st8f(dst + half + i, y);
      } else if (kv_row[tk] >= 0) {
        const int head = (w - rope_units) / (a.hd / 8), i = ((w - rope_units) % (a.hd / 8)) * 8;
        *reinterpret_cast<uint4*>(
            a.v_pages + (kv_row[tk] + static_cast<long long>(head) * page_size + in_page) * a.hd + i) =
            *reinterpret_cast<const uint4*>(src + (a.Hq + a.Hkv + head) * a.hd + i);
      }
    }
    __syncthreads();  // the tables are free for the next tokens
  }
}

}  // namespace ttcd
