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
// Bound by DRAM: each row is read once and written once (16 bytes per thread and
// access).  One warp per token and no barrier of the block: lane l forms
// the angles l and l + 32 and hands them on through shared memory of its warp; then each
// lane keeps the 8 angles of its chunk for all the heads, whose loads go out four
// at a time before the first is used.  17416 tokens of 32 heads of 128: 47 us, 6.0
// TB/s (one block per token with its barriers: 94); 8 tokens: 3.5 us captured, a chain of
// four loads.
#pragma once
#include "sink_attention.cuh"

namespace ttcd {

constexpr int APPEND_WARPS = 4;
constexpr int APPEND_THREADS = 32 * APPEND_WARPS;

struct AppendArgs {
  const __nv_bfloat16* qkv;  // [total_q, (Hq + 2 Hkv) hd]
  __nv_bfloat16* q_out;      // [total_q, Hq, hd]
  __nv_bfloat16* k_pages;    // [n_pages, Hkv, page_size, hd]
  __nv_bfloat16* v_pages;
  const int* table;          // [n_seq, max_pages]
  Ragged rg;
  int max_pages, n_pages, page_log2, Hq, Hkv;
  double log2_theta;  // log2 of the base
  bool rotate;
};

template <int HD>
__global__ void __launch_bounds__(APPEND_THREADS) paged_append_kernel(const AppendArgs a,
                                                                      uint32_t* err) {
  constexpr int HALF = HD / 2;
  constexpr int LPH = HALF / 8;         // lanes per rotated head: a chunk of 8 pairs each
  constexpr int HPW = 32 / LPH;         // rotated heads per pass of the warp
  constexpr int VPL = HD / 8;           // chunks of a v head
  __shared__ float2 cs_all[APPEND_WARPS][HALF];  // cos, sin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float2* cs = cs_all[warp];
  const int page_size = 1 << a.page_log2;
  const long long cap = static_cast<long long>(a.max_pages) << a.page_log2;
  if (blockIdx.x == 0) {  // every sequence's numbers are consistent, or this call says so
    for (int s = threadIdx.x; s < a.rg.n_seq; s += APPEND_THREADS)
      if (load_span(a.rg, s, cap).bad) atomicOr(err, DEV_ERR_BAD_INDEX);
  }
  // turns per position of this lane's angles
  double freq[(HALF + 31) / 32];
#pragma unroll
  for (int i = 0; i < (HALF + 31) / 32; ++i)
    freq[i] = exp2(-2.0 * (lane + 32 * i) / HD * a.log2_theta) * 0.15915494309189533577;  // 1 / 2 pi
  const int c = lane % LPH, h0 = lane / LPH;
  const int n_rot = a.Hq + a.Hkv;
  for (int row = blockIdx.x * APPEND_WARPS + warp; row < a.rg.total_q;
       row += gridDim.x * APPEND_WARPS) {
    const __nv_bfloat16* src = a.qkv + static_cast<long long>(row) * (a.Hq + 2 * a.Hkv) * HD;
    // the first rotated heads' loads go out before the token's place is known
    uint4 lo[4], hi[4];
    auto load = [&](int first) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int head = first + u * HPW + h0;
        if (head < n_rot) {
          lo[u] = *reinterpret_cast<const uint4*>(src + head * HD + c * 8);
          hi[u] = *reinterpret_cast<const uint4*>(src + head * HD + HALF + c * 8);
        }
      }
    };
    load(0);
    const int s = seq_of_row(a.rg, row);
    if (s < 0) continue;
    const SeqSpan sp = load_span(a.rg, s, cap);
    const int tok = row_token(sp, row);
    if (tok < 0) continue;  // padding, or a sequence that cannot be
    const int p = sp.L - sp.n + tok;
    const int id = a.table[static_cast<long long>(s) * a.max_pages + (p >> a.page_log2)];
    const long long kv_row = page_row(id, a.n_pages, a.Hkv, 0, page_size);
    if (kv_row < 0 && lane == 0) atomicOr(err, DEV_ERR_BAD_INDEX);
    const long long kv_at = (kv_row + (p & (page_size - 1))) * HD;  // of head 0
    __syncwarp();  // the previous token's angles have been read
#pragma unroll
    for (int i = 0; i < (HALF + 31) / 32; ++i)
      if (lane + 32 * i < HALF) {
        float2 x = make_float2(1.f, 0.f);
        if (a.rotate) {
          const double turns = p * freq[i];
          sincospif(2.f * static_cast<float>(turns - rint(turns)), &x.y, &x.x);
        }
        cs[lane + 32 * i] = x;
      }
    __syncwarp();
    float2 rot[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rot[e] = cs[c * 8 + e];
    for (int first = 0; first < n_rot; first += 4 * HPW) {
      if (first > 0) load(first);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int head = first + u * HPW + h0;
        if (head >= n_rot || (head >= a.Hq && kv_row < 0)) continue;
        const uint32_t xw[4] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w};
        const uint32_t yw[4] = {hi[u].x, hi[u].y, hi[u].z, hi[u].w};
        uint32_t xo[4], yo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = bf16lo_to_f32(xw[e]), x1 = bf16hi_to_f32(xw[e]);
          const float y0 = bf16lo_to_f32(yw[e]), y1 = bf16hi_to_f32(yw[e]);
          const float2 r0 = rot[2 * e], r1 = rot[2 * e + 1];
          xo[e] = pack_bf16x2(x0 * r0.x - y0 * r0.y, x1 * r1.x - y1 * r1.y);
          yo[e] = pack_bf16x2(y0 * r0.x + x0 * r0.y, y1 * r1.x + x1 * r1.y);
        }
        __nv_bfloat16* dst =
            head < a.Hq ? a.q_out + (static_cast<long long>(row) * a.Hq + head) * HD
                        : a.k_pages + kv_at + static_cast<long long>(head - a.Hq) * page_size * HD;
        *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(xo[0], xo[1], xo[2], xo[3]);
        *reinterpret_cast<uint4*>(dst + HALF + c * 8) = make_uint4(yo[0], yo[1], yo[2], yo[3]);
      }
    }
    if (kv_row >= 0) {
      const __nv_bfloat16* vs = src + n_rot * HD;
      for (int u0 = lane; u0 < a.Hkv * VPL; u0 += 4 * 32) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u0 + 32 * u < a.Hkv * VPL) w[u] = *reinterpret_cast<const uint4*>(vs + (u0 + 32 * u) * 8);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int x = u0 + 32 * u;
          if (x < a.Hkv * VPL)
            *reinterpret_cast<uint4*>(a.v_pages + kv_at +
                                      static_cast<long long>(x / VPL) * page_size * HD +
                                      (x % VPL) * 8) = w[u];
        }
      }
    }
  }
}

}  // namespace ttcd
