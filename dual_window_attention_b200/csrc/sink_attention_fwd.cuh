// Forward of the sliding-window attention with sinks on the tensor cores, over
// dense sequences and over a paged cache.
//
//   o_t = sum_j p_j v_j,  p = softmax_j(scale q_t . k_j)  over the visible keys,
// online in log2 units: m running reference, l = sum 2^(s - m), O = sum 2^(s - m) v.
//
// Work unit: one CTA owns two tiles of packed query rows (A, B) of one KV head,
// and every K/V tile it loads serves both.  A row is (token, query head of the
// group): a tile holds floor(128 / G) consecutive tokens of all G heads, so a
// group of any size fills the 128 rows (G = 3: 126), and short chunks of a
// prompt fill them with heads.  Where pairs of tiles would leave half of the SMs
// idle, a CTA has tile A alone.  Key tiles of 128 are visited from the newest
// backwards, and last the sinks' tile if the window does not reach it; a tile
// that only one of A and B sees is computed for that one.
//
// splits > 1 (few query tiles and many keys: a chunk of one prompt): the CTAs of a
// cluster take contiguous shares of the visits of one work unit and merge their
// partial (m, l, O) through distributed shared memory, every CTA a part of the rows.
//
// Pipeline (384 threads), TMEM (512 columns: S_A, S_B, O_A, O_B; P over its S),
// lazy rescaling and register split are those of dual_window_attn_kernel:
//   warp 0      TMA producer: Q of both tiles, then K and V of each visit.  Paged:
//               one box per page and panel, issued by as many lanes; a page
//               that no query of the CTA sees is not read (a box outside the
//               pool: zeros)
//   warp 1      TMEM owner and MMA issuer; zeroes V rows that no query of the CTA
//               sees (behind the sequence, before the window), which may hold
//               anything: 0 times NaN is NaN
//   warps 4..7  softmax of tile A (thread = row), warps 8..11 tile B
//
// P is rounded to bf16 as an operand.  The sinks' tile is the last visit, and there what
// that rounding leaves is a second operand, over the scores beside P: ceil(n_sink / 16) more
// steps.  Relative error of o where queries lean on the sinks 0.0021 -> 0.0017 (its last
// rounding alone: 0.0017), for 0-2 % of the time.
//
// Exponentials: one pair in four on the FMA pipe, by a quartic in the fractional part
// (relative error 2.8e-6, so that l and the log-sum-exp keep 32-bit quality; the
// dual kernel's cubic has 1.0e-4).
//
// What bounds it, from clock marks in one CTA (cycles of a visit of both tiles):
//   head_dim 128  3270: S to P 1740 of one tile, then its 16 + 8 steps of P V and the next
//                 Q K^T (1024, 1100-1200 with the loads' share of shared memory) and 300
//                 of hand-overs; the tensor cores work 2048 of them
//   head_dim 64   2860: S to P 1850 (the two tiles' softmax overlap), products and
//                 hand-overs 1010; P V with 64 columns takes as long as with 128
// 65536 tokens, 16 / 8 heads of 128, window 8192: 3.36 ms after idling, 3.9-4.0 one call
// after another under the power cap (2.5 ms at the measured cuBLAS rate); 16384, 15 / 5 of
// 64, window 4096: 0.36 and 0.37 ms.
// Measured and not kept (0.37 ms as the base): two threads per row (16 softmax
// warps) 0.44; visits of 64 or 96 keys with two score buffers and one or two issuing
// warps 0.40-0.48; a third score buffer at head_dim 64 0.38; turns at the exponentials
// 0.42; P in two halves 0.36 (the same), and that with the maximum beside the exponentials
// 0.41; the share of the FMA pipe 0, 1/4, 3/8: 0.38, 0.37, 0.38.
#pragma once
#include <type_traits>

#include "attention.cuh"
#include "sink_attention.cuh"

namespace ttcd {

struct SinkArgs {
  __nv_bfloat16* o;  // [rows, Hq, HD]
  float* lse;        // dense [B, Hq, T], paged [Hq, total_q]; nullable
  Ragged rg;         // paged
  const int* table;  // paged
  int max_pages, n_pages, page_log2;
  int oob_row;       // paged: first row past the pool
  int B, T;          // dense
  int n_units;       // dense: work units per sequence; paged: slots of them
  int Hq, Hkv, G, tpt;  // tpt = 128 / G tokens per tile
  int tpu;           // tokens per work unit: tpt or 2 tpt
  int window, n_sink;
  float scale_log2;
  int splits;        // CTAs per cluster
  int min_q;         // paged: sequences with fewer new tokens are another kernel's
};

template <int HD>
struct SinkCfg {
  using A = AttnCfg<HD>;
  static constexpr int ML_OFF = A::BAR_OFF + 512;  // (m, l) of 256 rows
  static constexpr int PITCH = HD * 4 + 16;        // fp32 partial row, over the tiles
  static_assert(256 * PITCH <= A::BAR_OFF, "partial rows fit over the operand tiles");
  static constexpr int SMEM_RAW = 1024 + ML_OFF + 256 * 8;
  // at least 120 KB: one CTA per SM (it takes all 512 TMEM columns)
  static constexpr int SMEM = SMEM_RAW > 122880 ? SMEM_RAW : 122880;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The largest number, or NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// exp2_poly2 with a quartic (relative error 2.8e-6; the same fit): inputs are
// clamped at -127, where the polynomial is 1 and its exponent becomes that of 0, so that
// a masked score weighs exactly 0 (2^-126 of a large hidden value would show); between
// -127 and -126 results are some number below 2^-126.  NaN gives 0, unless KEEP_NAN: then
// the maximum keeps it, and a last step, x 0 + y, puts it back after the exponent was
// added to its bits.
template <bool KEEP_NAN = false>
__device__ __forceinline__ uint64_t exp2_poly2_fine(uint64_t x) {
  constexpr float SHIFT = 12582912.0f;  // 1.5 * 2^23
  constexpr float C1 = 0.6931241934163351f, C2 = 0.24024098610072953f,
                  C3 = 0.0559064246048171f, C4 = 0.00958285308972204f;
  float x0, x1;
  f2unpack(x, x0, x1);
  x0 = KEEP_NAN ? max_nan(x0, -127.0f) : fmaxf(x0, -127.0f);
  x1 = KEEP_NAN ? max_nan(x1, -127.0f) : fmaxf(x1, -127.0f);
  const uint64_t xc = f2pack(x0, x1);
  const uint64_t t = add2(xc, f2pack(SHIFT, SHIFT));
  const uint64_t n = add2(t, f2pack(-SHIFT, -SHIFT));
  const uint64_t fr = fma2(n, f2pack(-1.0f, -1.0f), xc);
  uint64_t p = fma2(fr, f2pack(C4, C4), f2pack(C3, C3));
  p = fma2(p, fr, f2pack(C2, C2));
  p = fma2(p, fr, f2pack(C1, C1));
  p = fma2(p, fr, f2pack(1.0f, 1.0f));
  float p0, p1, t0, t1;
  f2unpack(p, p0, p1);
  f2unpack(t, t0, t1);
  const float r0 = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  const float r1 = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
  const uint64_t r = f2pack(r0, r1);
  return KEEP_NAN ? fma2(xc, f2pack(0.f, 0.f), r) : r;
}

// Four columns of a row merged over the parts of a cluster's CTAs (four parts in
// flight): its reference maximum and sum at ml, its fp32 columns at x4, the same
// offsets in every CTA.  A part without keys has -inf and finite columns.
__device__ __forceinline__ void merge_parts(uint32_t ml, uint32_t x4, int parts, float4& x,
                                            float& top, float& sum) {
  x = make_float4(0.f, 0.f, 0.f, 0.f);
  top = -INFINITY;
  sum = 0.f;
  for (int c0 = 0; c0 < parts; c0 += 4) {
    float2 s[4];
    float4 y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int from = min(c0 + u, parts - 1);
      s[u] = ld_cluster_f32x2(mapa_shared(ml, from));
      y[u] = ld_cluster_f32x4(mapa_shared(x4, from));
      if (c0 + u >= parts) s[u].x = -INFINITY;
    }
    const float g = fmaxf(fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x)), top);
    const float al = top == -INFINITY ? 0.f : ex2_approx(top - g);
    sum *= al;
    x.x *= al;
    x.y *= al;
    x.z *= al;
    x.w *= al;
    top = g;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = s[u].x == -INFINITY ? 0.f : ex2_approx(s[u].x - top);
      sum = fmaf(f, s[u].y, sum);
      x.x = fmaf(f, y[u].x, x.x);
      x.y = fmaf(f, y[u].y, x.y);
      x.z = fmaf(f, y[u].z, x.z);
      x.w = fmaf(f, y[u].w, x.w);
    }
  }
}

// mbar_wait for a converged warp, the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const DevStatus& st,
                                          volatile int* abort) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort));
  tc_fence_after();
  return ok;
}

__device__ __forceinline__ uint32_t pack2(uint64_t x) {
  float a, b;
  f2unpack(x, a, b);
  return pack_bf16x2(a, b);
}

// Visits first .. first + run - 1, then (n = run + 1) `extra`.
struct TileRange {
  int first, run, extra, n;
};

// The positions and visits of one work unit; identical for every role.
struct SinkVisits {
  int pos_lo[2], pos_hi[2], n[2];  // per tile; n = 0: no tile
  int j_lo[2], j_hi[2];            // its key tiles of the window
  KeyRange all;
  int jhi, n_win, total, n_sink;
  __device__ SinkVisits(int pos0, int left, int tpt, int window, int n_sink_) : n_sink(n_sink_) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      n[h] = max(0, min(tpt, left - h * tpt));
      pos_lo[h] = pos0 + h * tpt;
      pos_hi[h] = pos_lo[h] + n[h] - 1;
      j_lo[h] = key_range(pos_lo[h], pos_hi[h], window, 0).lo / ATT_BN;
      j_hi[h] = pos_hi[h] / ATT_BN;
    }
    all = key_range(pos0, n[1] > 0 ? pos_hi[1] : pos_hi[0], window, n_sink);
    jhi = all.hi / ATT_BN;
    n_win = jhi - all.lo / ATT_BN + 1;
    total = n_win + (all.sink_end > 0 && all.lo >= ATT_BN ? 1 : 0);
  }
  __device__ int tile(int v) const { return v < n_win ? jhi - v : 0; }
  // the visits of [v0, v1) that tile h needs
  __device__ TileRange range(int h, int v0, int v1) const {
    TileRange r;
    r.first = max(v0, jhi - j_hi[h]);
    r.run = n[h] > 0 ? max(0, min(v1, jhi - j_lo[h] + 1) - r.first) : 0;
    r.extra = total - 1;  // the sinks' tile
    const bool sinks = n[h] > 0 && n_sink > 0 && j_lo[h] > 0 && tile(r.extra) == 0;
    r.n = r.run + (sinks && r.extra >= v0 && r.extra < v1 ? 1 : 0);
    return r;
  }
  // whether any row of tile h sees a key of key tile j
  __device__ bool need(int h, int j) const {
    return n[h] > 0 && ((j >= j_lo[h] && j <= j_hi[h]) || (j == 0 && n_sink > 0));
  }
};

// 2^(s scale + offset) of a pair of scores.
__device__ __forceinline__ uint64_t prob2(float s0, float s1, uint64_t scale2, uint64_t offset2,
                                          int column) {
  const uint64_t x = fma2(f2pack(s0, s1), scale2, offset2);
  // one pair in four on the FMA pipe
  if (((column >> 1) & 3) == 3) return exp2_poly2_fine(x);
  float x0, x1;
  f2unpack(x, x0, x1);
  return f2pack(ex2_approx(x0), ex2_approx(x1));
}

template <int HD, bool PAGED>
__global__ void __launch_bounds__(ATT_THREADS, 1)
    sink_window_attn_kernel(const __grid_constant__ CUtensorMap mapQ,
                            const __grid_constant__ CUtensorMap mapK,
                            const __grid_constant__ CUtensorMap mapV, const SinkArgs a,
                            const DevStatus st) {
  using Cfg = AttnCfg<HD>;
  using SC = SinkCfg<HD>;
  constexpr uint32_t IDESC_QK = idesc_bf16_f32(ATT_BM, ATT_BN, false, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(ATT_BM, HD, false, true);
  constexpr int PANEL = ATT_BM * 128;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  uint64_t* q_full = bars;                  // 1
  uint64_t* k_full = bars + 1;              // KS
  uint64_t* k_empty = k_full + ATT_KS;      // KS
  uint64_t* v_full = k_empty + ATT_KS;      // VS
  uint64_t* v_empty = v_full + ATT_VS;      // VS
  uint64_t* s_full = v_empty + ATT_VS;      // 2 (per tile)
  uint64_t* p_full = s_full + 2;            // 2 (per tile, 128 arrivals)
  uint64_t* o_done = p_full + 2;            // 2 (per tile)
  uint64_t* drain = o_done + 2;             // 1
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = a.splits > 1 ? static_cast<int>(blockIdx.x) % a.splits : 0;
  const int item = static_cast<int>(blockIdx.x) / a.splits;
  const int hk = item % a.Hkv;
  const int tpu = a.tpu;

  // The work unit, found by every warp for itself.  A slot without work leaves before the
  // CTA takes its tensor memory: a batch of many single tokens has mostly such slots.
  int seq, tok0, q0, n, L;
  if (PAGED) {
    const long long capacity = static_cast<long long>(a.max_pages) << a.page_log2;
    if (blockIdx.x == 0)
      for (int s = threadIdx.x; s < a.rg.n_seq; s += ATT_THREADS)
        if (load_span(a.rg, s, capacity).bad) atomicOr(st.err, DEV_ERR_BAD_INDEX);
    const long long slot = item / a.Hkv;
    seq = find_seq(a.rg, slot, tpu);
    SeqSpan sp{0, 0, 0, false};
    long long t0 = 0;
    if (seq >= 0) {
      sp = load_span(a.rg, seq, capacity);
      t0 = (slot - tile_slot(sp.q0, seq, tpu)) * tpu;
      if (t0 >= sp.n || sp.n < a.min_q) sp.n = 0;
    }
    tok0 = static_cast<int>(t0);
    q0 = sp.q0;
    n = sp.n;
    L = sp.L;
  } else {  // longest (latest) units first
    const int u = a.n_units - 1 - item / (a.B * a.Hkv);
    seq = item / a.Hkv % a.B;
    tok0 = u * tpu;
    q0 = seq * a.T;
    n = L = a.T;
  }
  // after the kernel of few rows in the same call, this grid may end only when that
  // one has
  auto leave = [&]() {
    if (PAGED && blockIdx.x == 0) grid_dep_wait();
  };
  if (n == 0) {  // no tile here; the same for every CTA of the cluster
    leave();
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < ATT_KS; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int s = 0; s < ATT_VS; ++s) { mbar_init(&v_full[s], 1); mbar_init(&v_empty[s], 1); }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const SinkVisits vis(L - n + tok0, min(n - tok0, tpu), a.tpt, a.window, a.n_sink);
  const int v0 = static_cast<int>(static_cast<long long>(vis.total) * rank / a.splits);
  const int v1 = static_cast<int>(static_cast<long long>(vis.total) * (rank + 1) / a.splits);
  // The register split of dual_window_attn_kernel: 128 x 56 + 256 x 224 = 384 x 168.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
    if (warp == 0) {
      // ------------------------------------------------------------- TMA producer
      const int boxes = PAGED ? Cfg::PANELS << (7 - a.page_log2) : Cfg::PANELS;
      const int panel = lane % Cfg::PANELS, part = lane / Cfg::PANELS;
      // paged: this lane's page of visit v (-1: not seen by this CTA)
      auto page_of = [&](int v) {
        const int key = vis.tile(v) * ATT_BN + (part << a.page_log2);
        if (lane >= boxes || !touches(vis.all, key, key + (1 << a.page_log2) - 1)) return -1;
        const int id = a.table[static_cast<long long>(seq) * a.max_pages + (key >> a.page_log2)];
        return id == -1 ? -2 : id;
      };
      auto load = [&](int off, const CUtensorMap* map, uint64_t* bar, int v, int id) {
        if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::LOAD_BYTES);
        __syncwarp();
        if (lane < boxes) {
          if (PAGED) {
            const long long row = page_row(id, a.n_pages, a.Hkv, hk, 1 << a.page_log2);
            tma_load_2d(smem + off + panel * PANEL + (part << (a.page_log2 + 7)), map, bar,
                        64 * panel, row < 0 ? a.oob_row : static_cast<int>(row));
          } else {
            tma_load_4d(smem + off + panel * PANEL, map, bar, 64 * panel, hk,
                        vis.tile(v) * ATT_BN, seq);
          }
        }
      };
      if (v0 < v1) {
        const uint32_t q_bytes = Cfg::PANELS * 128 * a.G * a.tpt;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, vis.n[1] > 0 ? 2 * q_bytes : q_bytes);
#pragma unroll
          for (int p = 0; p < Cfg::PANELS; ++p) {
            tma_load_3d(smem + Cfg::QA_OFF + p * PANEL, &mapQ, q_full, 64 * p, hk * a.G, q0 + tok0);
            if (vis.n[1] > 0)
              tma_load_3d(smem + Cfg::QB_OFF + p * PANEL, &mapQ, q_full, 64 * p, hk * a.G,
                          q0 + tok0 + a.tpt);
          }
        }
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort));
        };
        int issued_k = 0, issued_v = 0;
        int id = PAGED ? page_of(v0) : 0;
        bool bad = false;
        for (int v = v0; v < v1; ++v) {
          const int i = v - v0, ks = i % ATT_KS, vs = i % ATT_VS;
          const int next = PAGED && v + 1 < v1 ? page_of(v + 1) : 0;  // in flight behind the waits
          if (!wait(&k_empty[ks], ((i / ATT_KS) & 1) ^ 1)) break;
          load(Cfg::K_OFF + ks * Cfg::TILE_BYTES, &mapK, &k_full[ks], v, id);
          ++issued_k;
          if (!wait(&v_empty[vs], ((i / ATT_VS) & 1) ^ 1)) break;
          load(Cfg::V_OFF + vs * Cfg::TILE_BYTES, &mapV, &v_full[vs], v, id);
          ++issued_v;
          bad = bad || id < -1 || id >= a.n_pages;
          id = next;
        }
        if (PAGED && bad) atomicOr(st.err, DEV_ERR_BAD_INDEX);
        volatile int no_abort = 0;
        mbar_wait(q_full, 0, st, &no_abort);
        for (int j = max(0, issued_k - ATT_KS); j < issued_k; ++j)
          mbar_wait(&k_full[j % ATT_KS], (j / ATT_KS) & 1, st, &no_abort);
        for (int j = max(0, issued_v - ATT_VS); j < issued_v; ++j)
          mbar_wait(&v_full[j % ATT_VS], (j / ATT_VS) & 1, st, &no_abort);
      }
    } else if (warp == 1 && v0 < v1) {
      // ------------------------------------------------------------- MMA issuer
      // The whole warp walks the loop and one elected lane issues, from descriptor
      // halves built once (as dual_window_attn_kernel).
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      const uint32_t q_lo[2] = {sdesc_lo(smem_u32(smem + Cfg::QA_OFF), 16),
                                sdesc_lo(smem_u32(smem + Cfg::QB_OFF), 16)};
      const uint32_t k_lo0 = sdesc_lo(smem_u32(smem + Cfg::K_OFF), 16);
      const uint32_t v_lo0 = sdesc_lo(smem_u32(smem + Cfg::V_OFF), PANEL);
      int done[2] = {0, 0};  // PV products issued per tile
      auto issue_qk = [&](int h, int i) {
        const uint32_t k_lo = k_lo0 + (((i % ATT_KS) * Cfg::TILE_BYTES) >> 4);
        const uint32_t qh = h ? q_lo[1] : q_lo[0];
        const uint32_t d = tmem + h * 128;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * PANEL + (kk & 3) * 32) >> 4;
            mma_bf16_ss_lh(d, qh + off, HI, k_lo + off, HI, IDESC_QK, kk > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[h]);
        }
        __syncwarp();
      };
      // rest: steps of 16 keys whose P is two operands
      auto issue_pv = [&](int h, int i, int rest) {
        const uint32_t v_lo = v_lo0 + (((i % ATT_VS) * Cfg::TILE_BYTES) >> 4);
        const uint32_t d = tmem + 256 + h * 128, pa = tmem + h * 128;
        const uint32_t acc0 = done[h] > 0 ? 1u : 0u;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < ATT_BN / 16; ++kk)
            mma_bf16_ts_lh(d, pa + kk * 8, v_lo + ((kk * 2048) >> 4), HI, IDESC_PV,
                           kk > 0 ? 1u : acc0);
          for (int kk = 0; kk < rest; ++kk)
            mma_bf16_ts_lh(d, pa + 64 + kk * 8, v_lo + ((kk * 2048) >> 4), HI, IDESC_PV, 1u);
          mma_commit(&o_done[h]);
        }
        __syncwarp();
        ++done[h];
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort));
      };
      const int nv = v1 - v0;
      bool ok = wait(q_full, 0) && wait(&k_full[0], 0);
      if (ok) {
        tc_fence_after();
        for (int h = 0; h < 2; ++h)
          if (vis.need(h, vis.tile(v0))) issue_qk(h, 0);
        if (elect_one()) mma_commit(&k_empty[0]);
        __syncwarp();
      }
      for (int i = 0; i < nv && ok; ++i) {
        const bool more = i + 1 < nv;
        const int j = vis.tile(v0 + i), j_next = more ? vis.tile(v0 + i + 1) : 0;
        const int k0 = j * ATT_BN;
        if (!wait(&v_full[i % ATT_VS], (i / ATT_VS) & 1)) break;
        if (k0 < vis.all.lo || k0 + ATT_BN - 1 > vis.all.hi) {
          uint8_t* vt = smem + Cfg::V_OFF + (i % ATT_VS) * Cfg::TILE_BYTES;
          for (int r = lane; r < ATT_BN; r += 32)
            if (!in_range(vis.all, k0 + r)) {
#pragma unroll
              for (int c = 0; c < Cfg::PANELS * 8; ++c)
                *reinterpret_cast<uint4*>(vt + (c >> 3) * PANEL + r * 128 + (c & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
          fence_async_smem();
          __syncwarp();
        }
        if (more && !wait(&k_full[(i + 1) % ATT_KS], ((i + 1) / ATT_KS) & 1)) break;
        for (int h = 0; h < 2; ++h) {
          if (vis.need(h, j)) {
            if (!wait(&p_full[h], done[h] & 1)) { ok = false; break; }
            tc_fence_after();
            issue_pv(h, i, j == 0 ? (a.n_sink + 15) >> 4 : 0);
          }
          if (more && vis.need(h, j_next)) issue_qk(h, i + 1);
        }
        if (!ok) break;
        if (elect_one()) {
          if (more) mma_commit(&k_empty[(i + 1) % ATT_KS]);
          mma_commit(&v_empty[i % ATT_VS]);
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(drain, 0, st, &no_abort);
    }
    __syncwarp();
    if (a.splits > 1) {  // the partial rows are written; they have been read
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory");
    // --------------------------------------------------------------- softmax rows
    const int h = (warp - 4) >> 2;  // 0: tile A, 1: tile B
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int tok = r / a.G, head = hk * a.G + r % a.G;
    const int t = (h ? vis.pos_lo[1] : vis.pos_lo[0]) + tok;  // position of the query
    const int n_tok = h ? vis.n[1] : vis.n[0];
    const bool row_ok = tok < n_tok;
    const int p_lo = h ? vis.pos_lo[1] : vis.pos_lo[0], p_hi = h ? vis.pos_hi[1] : vis.pos_hi[0];
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + h * 128;
    const uint32_t o_addr = tmem + lane_off + 256 + h * 128;
    const int row = q0 + tok0 + h * a.tpt + tok;
    const float sl2 = a.scale_log2;
    // m_ref = -inf: nothing visible yet; O is zero for such a row
    float m_ref = -INFINITY, l = 0.f;
    int cnt = 0;
    bool ok = true;
    const TileRange rg = h ? vis.range(1, v0, v1) : vis.range(0, v0, v1);
    // One visit; false: a wait gave up.  HAS_SINKS: the sinks' tile, always the last
    // (code of its own, because a branch here costs the others 3 to 9 %).
    auto visit = [&](int k0, auto has_sinks) -> bool {
      constexpr bool HAS_SINKS = decltype(has_sinks)::value;
      ok = mbar_wait(&s_full[h], cnt & 1, st, abort);
      ++cnt;
      tc_fence_after();
      float s[128];
      tmem_ld_cols<128>(s_addr, s);
      // every row of the tile sees the whole key tile
      const bool unmasked = k0 + ATT_BN - 1 <= p_lo &&
                            (k0 > p_hi - a.window || k0 + ATT_BN <= a.n_sink);
      if (!unmasked)
        mask_scores(s, [&](int k) { return seen_bits(t, k0 + 32 * k, a.window, a.n_sink); });
      // row maximum as four independent chains (short dependency latency); a visible
      // score of NaN or +inf makes it NaN and with it the row, as the softmax does (the
      // exponentials alone would lose it in the columns of the FMA pipe)
      float mx4[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float m = max_nan(s[32 * q], s[32 * q + 1], s[32 * q + 2]);
#pragma unroll
        for (int c = 3; c < 31; c += 2) m = max_nan(m, s[32 * q + c], s[32 * q + c + 1]);
        mx4[q] = max_nan(m, s[32 * q + 31]);
      }
      const float mx = max_nan(max_nan(mx4[0], mx4[1]), max_nan(mx4[2], mx4[3]));
      const float m_tile = mx < INFINITY ? mx * sl2 : __int_as_float(0x7fffffff);
      const bool fresh = m_ref == -INFINITY;
      const bool grow = !fresh && !(m_tile <= m_ref + ATT_RESCALE_THRESHOLD);
      if (__any_sync(0xffffffffu, grow || !ok)) {
        if (!__all_sync(0xffffffffu, ok)) { ok = false; return false; }
        const float m_new = grow ? m_tile : m_ref;
        const float al = grow ? ex2_approx(m_ref - m_new) : 1.f;
        tmem_scale_row<HD>(o_addr, al);
        l *= al;
        m_ref = m_new;
      }
      if (fresh) m_ref = m_tile;  // may stay -inf: no visible key in this tile
      // exponentials, row sum, bf16 pack (a row still at -inf has only masked scores)
      const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
      const uint64_t sc2 = f2pack(sl2, sl2);
      const uint64_t nm2 = f2pack(nm, nm);
      uint64_t acc4[4] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f),
                          f2pack(0.f, 0.f)};
      uint32_t P[64];
#pragma unroll
      for (int c = 0; c < 128; c += 2) {
        const uint64_t e = prob2(s[c], s[c + 1], sc2, nm2, c);
        acc4[(c >> 1) & 3] = add2(acc4[(c >> 1) & 3], e);
        P[c >> 1] = pack2(e);
      }
      const uint64_t acc = add2(add2(acc4[0], acc4[1]), add2(acc4[2], acc4[3]));
      float a0, a1;
      f2unpack(acc, a0, a1);
      l += a0 + a1;
      if constexpr (HAS_SINKS) {
        // A sink often has most of a row's weight, and then the rounding of its P shows
        // in the result: what it leaves becomes a second operand, beside the first
        // (the last columns first: a chunk lies over scores that are done with).
#pragma unroll 1
        for (int c0 = (a.n_sink - 1) & ~31; c0 >= 0; c0 -= 32) {
          float x[32];
          uint32_t w[16];
          tmem_ld32f(s_addr + c0, x);
          mask_scores(x, [&](int) { return seen_bits(t, c0, a.window, a.n_sink); });
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            f2unpack(prob2(x[c], x[c + 1], sc2, nm2, c), x0, x1);
            w[c >> 1] = rest2(x0, x1, pack_bf16x2(x0, x1));
          }
          tmem_st16(s_addr + 64 + (c0 >> 1), w);
        }
      }
      tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&P[0]));
      tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&P[32]));
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[h]);
      return true;
    };
    auto key_of = [&](int i) { return vis.tile(i < rg.run ? rg.first + i : rg.extra) * ATT_BN; };
    const bool sinks = a.n_sink > 0 && rg.n > 0 && key_of(rg.n - 1) == 0;
    const int plain = rg.n - (sinks ? 1 : 0);
    for (int i = 0; i < plain; ++i)
      if (!visit(key_of(i), std::false_type{})) break;
    if (ok && sinks) visit(0, std::true_type{});
    if (ok && cnt > 0) {
      ok = warp_wait(&o_done[h], (cnt - 1) & 1, st, abort);
    }
    auto lse_at = [&](int rw, int hd_, int tt) {
      return PAGED ? static_cast<long long>(hd_) * a.rg.total_q + rw
                   : (static_cast<long long>(seq) * a.Hq + hd_) * a.T + tt;
    };
    if (a.splits == 1) {
      // ---------------------------------------------------------------- epilogue
      if (ok && cnt > 0) {
        __nv_bfloat16* dst = a.o + (static_cast<long long>(row) * a.Hq + head) * HD;
        // (a row whose visible scores are all -inf has no softmax: l and O are 0, their quotient NaN)
        tmem_store_row<HD, __nv_bfloat16>(o_addr, 1.f / l, dst, row_ok);
        if (row_ok && a.lse) a.lse[lse_at(row, head, t)] = (m_ref + __log2f(l)) * 0.6931471805599453f;
      }
    } else {
      // ------------------------------------------------- merge over the cluster
      // All products and copies of this CTA have ended once both tiles' warps
      // are here: the operand tiles become the partial rows.
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int R = h * 128 + r;
      float2* ml = reinterpret_cast<float2*>(smem + SC::ML_OFF);
      // a row with no visible key here has -inf, and then only a NaN of its l counts
      ml[R] = ok && cnt > 0 ? make_float2(m_ref, l) : make_float2(-INFINITY, 0.f);
      float* mine = reinterpret_cast<float*>(smem + R * SC::PITCH);
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        float x[32];
        if (cnt > 0) {  // the same for a whole tile; a tile without visits here: zeros
          tmem_ld32f(o_addr + c, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        store_f32x32(mine + c, x);
      }
      cluster_sync_all();
      const uint32_t ml_addr = smem_u32(ml), rows_addr = smem_u32(smem);
      constexpr int QV = HD / 4;  // float4 of a row
      for (int it = rank * 256 + (threadIdx.x - 128); it < 256 * QV; it += a.splits * 256) {
        const int R_ = it / QV, c = it % QV;
        const int hh = R_ >> 7, rr = R_ & 127;
        const int tk = rr / a.G, hd_ = hk * a.G + rr % a.G;
        if (tk >= (hh ? vis.n[1] : vis.n[0])) continue;
        float4 x;
        float top, sum;
        merge_parts(ml_addr + 8 * R_, rows_addr + R_ * SC::PITCH + 16 * c, a.splits, x, top, sum);
        const float inv = 1.f / sum;
        const int rw = q0 + tok0 + hh * a.tpt + tk;
        *reinterpret_cast<uint2*>(a.o + (static_cast<long long>(rw) * a.Hq + hd_) * HD + 4 * c) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
        if (c == 0 && a.lse)
          a.lse[lse_at(rw, hd_, (hh ? vis.pos_lo[1] : vis.pos_lo[0]) + tk)] =
              (top + __log2f(sum)) * 0.6931471805599453f;
      }
      __syncwarp();
      cluster_sync_all();
    }
  }
  leave();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace ttcd
