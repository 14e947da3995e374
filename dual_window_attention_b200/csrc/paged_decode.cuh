// Attention of a few query rows over a paged cache with the mask of the sink
// windows: single tokens of a batch of sequences, or a handful of them.
//
// All rows of a unit (up to 16 rows: tokens x heads of one KV head's group) read
// the same keys once, so the work is bound by DRAM: 4 hd bytes per key for at most
// 16 x 4 hd operations.  Each warp takes a run of 16-key tiles, and K and V go from
// global memory straight into the operands of mma.sync, with no shared memory
// between: a contraction does not care for the order of its index, so each lane
// loads 16 contiguous bytes and Q is loaded in the same order.
//   S = Q K^T (m16n8k16): lane (n = lane / 4, p = lane % 4) holds key n's chunks p,
//     p + 4, ... of 8 elements; chunk i makes the steps 2i and 2i + 1.
//   O += P V: the accumulator of S is the operand P; lane (n, p) loads VE elements at
//     VE n of the keys 2p, 2p + 1, 2p + 8, 2p + 9 and pairs them by byte permutes, so
//     that output tile i holds the columns VE n + i.  Up to 8 rows: O^T += V^T P^T.
// The next tile's K is requested as soon as S is formed, its V after P V, and the
// page numbers two tiles ahead: at head_dim 128 about 6 KB in flight per warp and 12
// warps per SM, or, with two tiles in turn, 14 KB and 8 warps.
//
// The 4 warps of a CTA and the CTAs of a cluster share a unit's tiles and merge
// their (m, l, O) through shared memory, then distributed shared memory.
//
// 64 sequences that see 498721 keys together, 8 heads of 128: 332 us, 6.2 TB/s.  One of
// 8196 keys: 16.4 us a call, 13.7 captured, its K and V in L2; its 8 units in clusters of
// 16 are 128 CTAs of 4 warps, so 20 SMs stay empty and a warp walks 8 tiles, two in
// flight.  Those four rounds of memory latency are half of the time, the rest the chain
// lengths -> page -> keys and the merge.
//
// Softmax as in the tiled kernel: base-2 units, the reference maximum of a row is
// moved only when a score exceeds it by 2^8.  P becomes a bf16 operand, and the rounding
// of a key with most of a row's weight (a sink often has it) would show in the result,
// up to 2^-8 of it, with few rows to average over.  head_dim 128: a warp scales its O by
// sum p / sum round(p), in which the rounding of such a key falls out (registers are
// short: what the rounding leaves as a second operand costs 13 % there).  Up to 64: that
// second operand, at no cost (the scaling 10 %).  lse is that of the unrounded p.
#pragma once
#include "sink_attention_fwd.cuh"

namespace ttcd {

constexpr int PDEC_WARPS = 4;
constexpr int PDEC_THREADS = 32 * PDEC_WARPS;
// CTAs per SM (register bound) of a variant.
template <int HD, int ROWS, int DEPTH>
constexpr int PDEC_CTAS = ROWS * HD > 1024 ? 2 : HD == 32 ? 4 : (HD == 64 ? 5 : 4) - DEPTH;

struct PagedDecodeArgs {
  const __nv_bfloat16* q;  // [total_q, Hq, HD]
  PagedCache pc;
  Ragged rg;
  __nv_bfloat16* o;
  float* lse;  // [Hq, total_q], nullable
  int Hq, G, tpt;  // tpt: tokens per unit
  int window, n_sink;
  float scale_log2;
  int splits;       // CTAs per cluster
  int only_small;   // sequences with more than tpt new tokens are another kernel's
};

__device__ __forceinline__ void mma_16816(float& c0, float& c1, float& c2, float& c3, uint32_t a0,
                                          uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Streamed reads: each line is used by one warp, once.
__device__ __forceinline__ void ld_stream(uint32_t (&r)[4], const void* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p));
}
__device__ __forceinline__ void ld_stream(uint32_t (&r)[2], const void* p) {
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "l"(p));
}

// ROWS: 8 or 16 query rows of a unit (the tensor instruction has 16 either way;
// with 8 the registers of the others are free).
// DEPTH: tiles of K and V in registers or on their way to them.
template <int HD, int ROWS, int DEPTH>
__global__ void __launch_bounds__(PDEC_THREADS, (PDEC_CTAS<HD, ROWS, DEPTH>))
    paged_decode_kernel(const PagedDecodeArgs a, uint32_t* err) {
  constexpr int NR = ROWS / 8;                  // rows per lane
  constexpr int KC = HD / 32;                   // K chunks per lane and key
  constexpr int VE = HD >= 64 ? 8 : HD / 8;     // V elements per load
  constexpr int VC = HD / (8 * VE);             // V chunks per lane and key
  constexpr int VW = VE / 2;                    // words of a V chunk
  constexpr bool REST = HD <= 64;               // P as two operands
  __shared__ __align__(16) float part[PDEC_WARPS][ROWS][HD + 4];  // accessed 16 bytes at a time
  __shared__ float2 ml[PDEC_WARPS][ROWS];       // reference maximum, sum
  __shared__ float2 ml_cta[ROWS];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = lane >> 2, p = lane & 3;
  const int rank = a.splits > 1 ? static_cast<int>(blockIdx.x) % a.splits : 0;
  const int item = static_cast<int>(blockIdx.x) / a.splits;
  const int hk = item % a.pc.Hkv, slot = item / a.pc.Hkv;
  const int page = 1 << a.pc.page_log2;
  const long long capacity = static_cast<long long>(a.pc.max_pages) << a.pc.page_log2;
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < a.rg.n_seq; s += PDEC_THREADS)
      if (load_span(a.rg, s, capacity).bad) atomicOr(err, DEV_ERR_BAD_INDEX);
  grid_dep_launch();  // the tiled kernel of the same call may start beside the last of these
  // the first n_seq slots: the first unit of each sequence; then the further ones
  int seq = slot, tok0 = 0;
  if (slot >= a.rg.n_seq) {
    seq = find_extra_seq(a.rg, slot - a.rg.n_seq, a.tpt);
    if (seq >= 0) tok0 = extra_token(slot - a.rg.n_seq, a.rg.q_start[seq], a.tpt);
  }
  if (seq < 0) return;
  const SeqSpan sp = load_span(a.rg, seq, capacity);
  if (tok0 >= sp.n || (a.only_small && sp.n > a.tpt)) return;  // the whole cluster
  const int n_tok = min(a.tpt, sp.n - tok0), n_rows = n_tok * a.G;
  const int pos0 = sp.L - sp.n + tok0;
  const KeyRange kr = key_range(pos0, pos0 + n_tok - 1, a.window, a.n_sink);
  // 16-key tiles: the window's, then the sinks' before it
  const int lo16 = kr.lo >> 4, n_win = (kr.hi >> 4) - lo16 + 1;
  const int total = n_win + min((kr.sink_end + 15) >> 4, lo16);
  const int share = rank * PDEC_WARPS + warp, shares = a.splits * PDEC_WARPS;
  const int v0 = static_cast<int>(static_cast<long long>(total) * share / shares);
  const int v1 = static_cast<int>(static_cast<long long>(total) * (share + 1) / shares);
  auto key_of = [&](int v) { return (v < n_win ? lo16 + v : v - n_win) << 4; };
  const int* table = a.pc.table + static_cast<long long>(seq) * a.pc.max_pages;
  auto page_of = [&](int v) { return v < v1 ? table[key_of(v) >> a.pc.page_log2] : 0; };
  // element offset of the tile's first row, -1: no such page (it counts as zeros)
  auto row_of = [&](int v, int id) {
    const long long r = page_row(id, a.pc.n_pages, a.pc.Hkv, hk, page);
    return r < 0 ? -1ll : (r + (key_of(v) & (page - 1))) * HD;
  };
  uint32_t Ks[DEPTH][2][KC][4], Vs[DEPTH][4][VC][VW];
  auto load_k = [&](long long at, uint32_t (&K)[2][KC][4]) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        if (at >= 0) {
          ld_stream(K[nt][i], a.pc.k + at + (nt * 8 + n) * HD + (p + 4 * i) * 8);
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) K[nt][i][w] = 0;
        }
      }
  };
  auto load_v = [&](long long at, uint32_t (&V)[4][VC][VW]) {
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int j = 0; j < VC; ++j) {
        if (at >= 0) {
          ld_stream(V[y][j], a.pc.v + at + (2 * p + (y & 1) + (y >> 1) * 8) * HD + j * 8 * VE + n * VE);
        } else {
#pragma unroll
          for (int w = 0; w < VW; ++w) V[y][j][w] = 0;
        }
      }
  };
  int ids[DEPTH], next_ids[DEPTH];
#pragma unroll
  for (int x = 0; x < DEPTH; ++x) ids[x] = page_of(v0 + x);
#pragma unroll
  for (int x = 0; x < DEPTH; ++x) next_ids[x] = page_of(v0 + DEPTH + x);
  bool bad = false;
#pragma unroll
  for (int x = 0; x < DEPTH; ++x)
    if (v0 + x < v1) {
      const long long at = row_of(v0 + x, ids[x]);
      bad = bad || at < 0;
      load_k(at, Ks[x]);
      load_v(at, Vs[x]);
    }
  // Q in the order of K's chunks; rows that are not there are zeros
  uint32_t Q[NR][KC][4];
  int t[NR];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    const int r = n + 8 * x;
    t[x] = pos0 + min(r / a.G, n_tok - 1);
    const long long row = (static_cast<long long>(sp.q0) + tok0 + r / a.G) * a.Hq + hk * a.G + r % a.G;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r < n_rows) w = *reinterpret_cast<const uint4*>(a.q + row * HD + (p + 4 * i) * 8);
      Q[x][i][0] = w.x; Q[x][i][1] = w.y; Q[x][i][2] = w.z; Q[x][i][3] = w.w;
    }
  }
  // 16 rows: [column 2p + e of output tile i][row n + 8 x]; 8 rows: see below
  float O[VC][NR * VE / 2][4] = {};
  float m[NR], l[NR], lr[NR];  // reference maximum, sum of p, of p as rounded
#pragma unroll
  for (int x = 0; x < NR; ++x) { m[x] = -INFINITY; l[x] = lr[x] = 0.f; }
  // O times a factor of each row n + 8 x
  auto scale_rows = [&](const float (&f)[NR]) {
    float g[4];
    if (NR > 1) {
      g[0] = g[1] = f[0];
      g[2] = g[3] = f[NR - 1];
    } else {  // rows 2p and 2p + 1
      g[0] = g[2] = __shfl_sync(0xffffffffu, f[0], 8 * p);
      g[1] = g[3] = __shfl_sync(0xffffffffu, f[0], 8 * p + 4);
    }
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int i = 0; i < NR * VE / 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[c][i][e] *= g[e];
  };
  auto step = [&](int v, uint32_t (&K)[2][KC][4], uint32_t (&V)[4][VC][VW], int& next_id) {
    const int k0 = key_of(v);
    const bool more = v + DEPTH < v1;
    const long long next = more ? row_of(v + DEPTH, next_id) : -1;
    next_id = page_of(v + 2 * DEPTH);
    bad = bad || (more && next < 0);
    float s[NR][4];  // keys 2p, 2p + 1, 2p + 8, 2p + 9
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          mma_16816(c[0], c[1], c[2], c[3], Q[0][i][2 * half], NR > 1 ? Q[NR - 1][i][2 * half] : 0u,
                    Q[0][i][2 * half + 1], NR > 1 ? Q[NR - 1][i][2 * half + 1] : 0u,
                    K[nt][i][2 * half], K[nt][i][2 * half + 1]);
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        s[x][2 * nt] = c[2 * x];
        s[x][2 * nt + 1] = c[2 * x + 1];
      }
    }
    if (more) load_k(next, K);
    const bool all = k0 + 15 <= pos0 && (k0 > pos0 + n_tok - 1 - a.window || k0 + 16 <= a.n_sink);
    if (!all) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int j = k0 + 2 * p + (y & 1) + (y >> 1) * 8;
#pragma unroll
        for (int x = 0; x < NR; ++x)
          if (j > t[x] || (j <= t[x] - a.window && j >= a.n_sink)) s[x][y] = -INFINITY;
        // rows that no query of the unit sees may hold anything: 0 times NaN is NaN
        if (!in_range(kr, j)) {
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int w = 0; w < VW; ++w) V[y][c][w] = 0;
        }
      }
    }
    bool grow = false;
    float mx[NR];
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      mx[x] = fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3])) * a.scale_log2;
      grow = grow || mx[x] > m[x] + ATT_RESCALE_THRESHOLD;  // m = -inf: any key
    }
    if (__any_sync(0xffffffffu, grow)) {
      float f[NR];
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        f[x] = 1.f;
        float g = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if (g > m[x] + ATT_RESCALE_THRESHOLD) {
          const float al = ex2_approx(m[x] - g);
          m[x] = g;
          l[x] *= al;
          lr[x] *= al;
          f[x] = al;
        }
      }
      scale_rows(f);
    }
    uint32_t P[NR][2], R[NR][2];  // P, and (REST) what its rounding leaves
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const float nm = m[x] == -INFINITY ? 0.f : -m[x];
      float e[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) e[y] = ex2_approx(fmaf(s[x][y], a.scale_log2, nm));
      l[x] += (e[0] + e[1]) + (e[2] + e[3]);
      P[x][0] = pack_bf16x2(e[0], e[1]);
      P[x][1] = pack_bf16x2(e[2], e[3]);
      if constexpr (REST) {
        R[x][0] = rest2(e[0], e[1], P[x][0]);
        R[x][1] = rest2(e[2], e[3], P[x][1]);
      } else {
        lr[x] += (bf16lo_to_f32(P[x][0]) + bf16hi_to_f32(P[x][0])) +
                 (bf16lo_to_f32(P[x][1]) + bf16hi_to_f32(P[x][1]));
      }
    }
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        // pairs of keys: elements 2w and 2w + 1, keys 2p .. and 2p + 8 ..
        const uint32_t e0 = __byte_perm(V[0][c][w], V[1][c][w], 0x5410);
        const uint32_t o0 = __byte_perm(V[0][c][w], V[1][c][w], 0x7632);
        const uint32_t e1 = __byte_perm(V[2][c][w], V[3][c][w], 0x5410);
        const uint32_t o1 = __byte_perm(V[2][c][w], V[3][c][w], 0x7632);
        if constexpr (NR > 1) {
          float(&x)[4] = O[c][2 * w], (&y)[4] = O[c][2 * w + 1];
          mma_16816(x[0], x[1], x[2], x[3], P[0][0], P[1][0], P[0][1], P[1][1], e0, e1);
          mma_16816(y[0], y[1], y[2], y[3], P[0][0], P[1][0], P[0][1], P[1][1], o0, o1);
          if constexpr (REST) {
            mma_16816(x[0], x[1], x[2], x[3], R[0][0], R[1][0], R[0][1], R[1][1], e0, e1);
            mma_16816(y[0], y[1], y[2], y[3], R[0][0], R[1][0], R[0][1], R[1][1], o0, o1);
          }
        } else {
          // O^T = V^T P^T: columns of V as the 16 rows of the instruction, so that
          // 8 queries leave no accumulator unused
          float(&x)[4] = O[c][w];
          mma_16816(x[0], x[1], x[2], x[3], e0, o0, e1, o1, P[0][0], P[0][1]);
          if constexpr (REST) mma_16816(x[0], x[1], x[2], x[3], e0, o0, e1, o1, R[0][0], R[0][1]);
        }
      }
    if (more) load_v(next, V);
  };
  for (int v = v0; v < v1; v += DEPTH) {
#pragma unroll
    for (int x = 0; x < DEPTH; ++x)
      if (v + x < v1) step(v + x, Ks[x], Vs[x], next_ids[x]);
  }
  if (bad && lane == 0) atomicOr(err, DEV_ERR_BAD_INDEX);
  // ------------------------------------------------------------------- merge
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    const int r = n + 8 * x;
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if (p == 0) ml[warp][r] = make_float2(m[x], l[x]);
    if constexpr (!REST) {
      lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 1);
      lr[x] += __shfl_xor_sync(0xffffffffu, lr[x], 2);
      lr[x] = lr[x] > 0.f ? l[x] / lr[x] : 1.f;
    }
  }
  if constexpr (!REST) scale_rows(lr);
#pragma unroll
  for (int c = 0; c < VC; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < VE; i += 4) {
        if constexpr (NR > 1) {
#pragma unroll
          for (int x = 0; x < NR; ++x)
            *reinterpret_cast<float4*>(&part[warp][n + 8 * x][c * 8 * VE + VE * (2 * p + e) + i]) =
                make_float4(O[c][i][2 * x + e], O[c][i + 1][2 * x + e], O[c][i + 2][2 * x + e],
                            O[c][i + 3][2 * x + e]);
        } else {
          *reinterpret_cast<float4*>(&part[warp][2 * p + e][c * 8 * VE + VE * n + i]) =
              make_float4(O[c][i / 2][e], O[c][i / 2][2 + e], O[c][i / 2 + 1][e],
                          O[c][i / 2 + 1][2 + e]);
        }
      }
  __syncthreads();
  constexpr int QV = HD / 4;  // float4 of a row
  auto store = [&](int r, int c, float4 x, float top, float sum) {
    const int tok = r / a.G, head = hk * a.G + r % a.G;
    const long long row = static_cast<long long>(sp.q0) + tok0 + tok;
    const float inv = 1.f / sum;
    *reinterpret_cast<uint2*>(a.o + (row * a.Hq + head) * HD + 4 * c) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (c == 0 && a.lse)
      a.lse[static_cast<long long>(head) * a.rg.total_q + row] =
          (top + __log2f(sum)) * 0.6931471805599453f;
  };
  for (int it = threadIdx.x; it < n_rows * QV; it += PDEC_THREADS) {
    const int r = it / QV, c = it % QV;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < PDEC_WARPS; ++w) top = fmaxf(top, ml[w][r].x);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < PDEC_WARPS; ++w) {
      const float2 s = ml[w][r];
      const float f = s.x == -INFINITY ? 0.f : ex2_approx(s.x - top);
      const float4 y = *reinterpret_cast<const float4*>(&part[w][r][4 * c]);
      sum = fmaf(f, s.y, sum);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    if (a.splits == 1) {
      store(r, c, x, top, sum);
    } else {
      *reinterpret_cast<float4*>(&part[0][r][4 * c]) = x;  // read by this thread alone
      if (c == 0) ml_cta[r] = make_float2(top, sum);
    }
  }
  if (a.splits > 1) {
    __syncwarp();
    cluster_sync_all();
    const uint32_t ml_addr = smem_u32(ml_cta), part_addr = smem_u32(part);
    for (int it = rank * PDEC_THREADS + threadIdx.x; it < n_rows * QV; it += a.splits * PDEC_THREADS) {
      const int r = it / QV, c = it % QV;
      float4 x;
      float top, sum;
      merge_parts(ml_addr + 8 * r, part_addr + (r * (HD + 4) + 4 * c) * 4, a.splits, x, top, sum);
      store(r, c, x, top, sum);
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its part is read
  }
}

}  // namespace ttcd
