// Backward of the sliding-window attention with sinks on the tensor cores.
//
//   P = exp(scale Q K^T - lse),  dP = dO V^T,  dS = P (dP - delta),  delta_t = dO_t . O_t
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// Two kernels, each with its result in TMEM until it is stored once: dQ with the
// queries standing, then dK and dV with the keys standing.  S and dP are formed in
// both (7 products of a tile pair instead of 5), and in exchange nothing is added
// into global memory: no fp32 dq buffer, no reductions through L2, and two
// runs give the same bits.
//
// A tile of queries is floor(128 / G) tokens of the G heads of one KV head, as in
// the forward, so a group of any size fills the 128 rows and shares K and V.
//
// Both kernels run 640 threads: warp 0 the TMA producer, warp 1 the MMA issuer
// (one elected lane), warps 4..19 the element work on 128 x 128 scores, thread =
// (TMEM lane, quarter of the columns).  p stays in registers in 32 bits between the
// exponential and dS; P and dS are rounded to bf16 as operands of products.  In the sinks'
// key tile, whose few keys carry a large part of many rows' weight, what that rounding
// leaves is a second operand, in the columns beside the first: the last visit of a row
// in the dQ kernel (without sinks too, where it covers windows of one or two tiles), the
// items of the first key tile in the other.  With it the error of dq,
// dk and dv is that of their last rounding (0.0017, relative, instead of 0.0021-0.0028).  S and
// dP have one buffer each, and what alternates is the work: while the element warps
// form P from S, the tensor cores run the products of dS and the next dP, and while
// they form dS from dP the products of P and the next S.
//
// dQ kernel.  Q and dO stand in TMEM as A operands (put there by the threads of
// their rows, which also form delta), so that shared memory is read for K and V
// alone: 128 x 128 x 16 steps with both operands in shared memory take all of its
// 128 bytes per cycle.  Per key tile v: S(v+1), dQ(v) += dS K, dP(v+1), with dS
// over its dP.  It also writes -lse / scale and -delta of its rows, packed as the
// tiles are, for the second kernel.
//
// dK/dV kernel.  Per query tile v: dV += P^T dO, S^T(v+1) = K Q^T, dK += dS^T Q,
// dP^T(v+1) = V dO^T; P^T lies over its S^T and dS^T over its dP^T as A operands.
// There the numbers of a query belong to a column, the same for every thread: read
// from shared memory they cost 700 cycles of a visit's 3200, beside the products'
// operands.  So they ride along as one more step of 16 of the two score products: the
// key side holds 1, 1, 1, 0 ..., the query side the number as a sum of three bf16
// (24 bits), and the scores arrive with -lse / scale and -delta in them.
// The first key tile is seen by every query through its sinks: the query tiles
// past its window are cut into items of their own, which write fp32 partial rows of the
// sinks, and a last kernel adds them in a fixed order.  Where the key tiles are too few
// for the SMs, their own queries are cut into `parts` the same way.
//
// What bounds them, from clock marks in one CTA (cycles of a visit, 128 x 128 scores):
//   dQ     head_dim 128: 2030, of them 1536 of products; 64: 1650, of them 1000 from S to P
//          (the exponentials: 768 at the least), 310 of dS, the rest waits
//   dK/dV  128: 2910 (P 1090, then dV and the next S^T 1100 and 270 of hand-overs beside
//          dS; 2176 of products); 64: 2200 (products with 64 columns take as long as
//          with 128: 1664)
// 32768 tokens, 16 / 8 heads of 128, window 8192: 2.30 and 2.93 ms after idling (the
// forward 1.57), 2.55 and 3.21 (1.83) one step after another under the power cap; 16384,
// 15 / 5 of 64, window 4096: 0.48 and 0.49 (0.36) ms, a whole step 1.44 among others.
// Measured and not kept: 8 element warps 2-3 % slower; two issuing warps at head_dim
// 128 2.41 and 3.36 ms (the products interleave and each takes twice as long).
#pragma once
#include "attention_bwd.cuh"
#include "sink_attention_fwd.cuh"

namespace ttcd {

constexpr int SINKB_THREADS = 640;
constexpr int SINKB_ROWS = 512;  // element threads: (TMEM lane, quarter of the columns)

struct SinkBwdArgs {
  const __nv_bfloat16* q;    // [B, T, Hq, HD]
  const __nv_bfloat16* o;
  const __nv_bfloat16* d_o;
  const float* lse;          // [B, Hq, T]
  __nv_bfloat16* dq;         // [B, T, Hq, HD]
  __nv_bfloat16* dk;         // [B, T, Hkv, HD]
  __nv_bfloat16* dv;
  uint4* rows;     // [B, Hkv, n_qt, 2, 128]: -lse / scale and -delta, three bf16 each
  // dk and dv (fp32) of a key tile's items, summed by the last kernel:
  float* partial;    // the sinks' rows [n_far + 1, B, Hkv, 2, n_sink, HD]; the last are those of
                     // the first tile's near item where it is one (parts0 = 1)
  float* near0;      // parts0 > 1: [parts0, B, Hkv, 2, 128, HD]
  float* near_rows;  // parts > 1: [parts, B, Hkv, 2, n_kt 128, HD]
  int parts0, parts;  // near items of the first key tile, of each other one
  int B, T, Hq, Hkv, G, tpt, n_qt, n_kt;
  int window, n_sink;
  int n_far, far_tiles;  // items of the far queries of the sinks, query tiles each
  int far0;              // the first of these query tiles
  float scale, scale_log2, inv_scale;
};

template <int HD>
struct SinkDqCfg {
  static constexpr int PANELS = HD / 64;
  static constexpr int TILE = PANELS * 128 * 128;
  static constexpr int KS = 3, VS = 3;
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = KS * TILE;
  static constexpr int DEL_OFF = V_OFF + VS * TILE;  // (2 + 4) x 128 floats
  static constexpr int BAR_OFF = DEL_OFF + 6 * 512;
  static constexpr int SMEM_RAW = 1024 + BAR_OFF + 256;
  // at least 120 KB: one CTA per SM (it takes all 512 TMEM columns)
  static constexpr int SMEM = SMEM_RAW > 122880 ? SMEM_RAW : 122880;
};

template <int HD>
struct SinkDkvCfg {
  static constexpr int PANELS = HD / 64;
  static constexpr int TILE = PANELS * 128 * 128;
  // Buffers of S^T in TMEM: two fit at head_dim 64, and the next scores form a
  // visit ahead.
  static constexpr int NBS = HD == 64 ? 2 : 1;
  static constexpr int QS = NBS + 1;  // Q stages
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = TILE;
  static constexpr int Q_OFF = 2 * TILE;
  static constexpr int DO_OFF = Q_OFF + QS * TILE;  // two stages
  // query side of the extra step: per Q stage 128 rows of 16 bytes for S, then for dP
  static constexpr int EXT_OFF = DO_OFF + 2 * TILE;
  static constexpr int ONE_OFF = EXT_OFF + QS * 4096;  // its key side
  static constexpr int ZERO_OFF = ONE_OFF + 2048;      // elements 8 .. 15 of every row
  static constexpr int BAR_OFF = ZERO_OFF + 2048;
  static constexpr int SMEM_RAW = 1024 + BAR_OFF + 256;
  static constexpr int SMEM = SMEM_RAW > 122880 ? SMEM_RAW : 122880;
};

// x as hi + mid + lo in bf16, then zeros: 16 bytes.
__device__ __forceinline__ uint4 split3(float x) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  const float r = x - __bfloat162float(h);
  const __nv_bfloat16 m = __float2bfloat16_rn(r);
  const __nv_bfloat16 l = __float2bfloat16_rn(r - __bfloat162float(m));
  return make_uint4(__bfloat16_as_ushort(h) | static_cast<uint32_t>(__bfloat16_as_ushort(m)) << 16,
                    __bfloat16_as_ushort(l), 0, 0);
}

// p = 2^(s scale_log2 + nl) of 32 scores; nl per pair of columns.  One pair in
// four on the FMA pipe, as the forward.  KEEP_NAN: there too NaN stays NaN, for columns that are queries, whose log-sum-exp may be NaN
// (where rows are, the other columns of such a row show it).
template <bool KEEP_NAN, class NL>
__device__ __forceinline__ void probs32(float (&s)[32], float scale_log2, NL nl) {
  const uint64_t sc2 = f2pack(scale_log2, scale_log2);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const uint64_t x = fma2(f2pack(s[c], s[c + 1]), sc2, nl(c));
    if (((c >> 1) & 3) == 3) {
      f2unpack(exp2_poly2_fine<KEEP_NAN>(x), s[c], s[c + 1]);
    } else {
      float x0, x1;
      f2unpack(x, x0, x1);
      s[c] = ex2_approx(x0);
      s[c + 1] = ex2_approx(x1);
    }
  }
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// dS of 32 columns, p (dp + nd), in place of dp.
__device__ __forceinline__ void ds32(const float (&p)[32], float (&dp)[32], uint64_t nd2) {
#pragma unroll
  for (int i = 0; i < 32; i += 2)
    f2unpack(mul2(f2pack(p[i], p[i + 1]), add2(f2pack(dp[i], dp[i + 1]), nd2)), dp[i], dp[i + 1]);
}

// 32 columns as bf16 over the first half of their own columns, and, where `split`,
// what that leaves over the second half.
__device__ __forceinline__ void store_operand(uint32_t taddr, const float (&x)[32], bool split) {
  uint32_t w[16];
#pragma unroll
  for (int c = 0; c < 32; c += 2) w[c >> 1] = pack_bf16x2(x[c], x[c + 1]);
  tmem_st16(taddr, w);
  if (split) {
#pragma unroll
    for (int c = 0; c < 32; c += 2) w[c >> 1] = rest2(x[c], x[c + 1], w[c >> 1]);
    tmem_st16(taddr + 16, w);
  }
  tmem_st_wait();
  tc_fence_before();
}

template <int HD>
__global__ void __launch_bounds__(SINKB_THREADS, 1)
    sink_attn_dq_kernel(const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV, const SinkBwdArgs a,
                        const DevStatus st) {
  using Cfg = SinkDqCfg<HD>;
  grid_dep_launch();  // the dK/dV kernel's CTAs may set up beside the last of these
  constexpr int KS = Cfg::KS, VS = Cfg::VS, PANEL = 128 * 128;
  constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);  // S, dP
  constexpr uint32_t ID_DQ = idesc_bf16_f32(128, HD, false, true);
  constexpr uint32_t C_S = 0, C_DP = 128, C_DQ = 256, C_Q = 384, C_DO = 448;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  uint64_t* k_full = bars;             // KS
  uint64_t* k_empty = k_full + KS;     // KS
  uint64_t* v_full = k_empty + KS;     // VS
  uint64_t* v_empty = v_full + VS;     // VS
  uint64_t* a_ready = v_empty + VS;    // Q and dO are in TMEM (every element thread arrives)
  uint64_t* s_full = a_ready + 1;
  uint64_t* s_free = s_full + 1;       // every element thread arrives
  uint64_t* dp_full = s_free + 1;
  uint64_t* ds_ready = dp_full + 1;    // every element thread arrives
  uint64_t* sum_ready = ds_ready + 1;  // every element thread arrives
  uint64_t* done = sum_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* del = reinterpret_cast<float*>(smem + Cfg::DEL_OFF);
  float* sums = del + 256;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int hk = static_cast<int>(blockIdx.x) % a.Hkv;
  const int b = static_cast<int>(blockIdx.x) / a.Hkv % a.B;
  // longest (latest) tiles first
  const int qt = a.n_qt - 1 - static_cast<int>(blockIdx.x) / (a.Hkv * a.B);
  const int t0 = qt * a.tpt, t1 = min(t0 + a.tpt, a.T) - 1;
  const KeyRange kr = key_range(t0, t1, a.window, a.n_sink);
  const int jhi = kr.hi / 128, n_win = jhi - kr.lo / 128 + 1;
  const int nv = n_win + (kr.sink_end > 0 && kr.lo >= 128 ? 1 : 0);
  auto key_tile = [&](int v) { return v < n_win ? jhi - v : 0; };

  if (threadIdx.x == 0) {
    for (uint64_t* p = bars; p <= done; ++p)
      mbar_init(p, p == a_ready || p == s_free || p == ds_ready || p == sum_ready ? SINKB_ROWS : 1);
    *abort = 0;
    fence_mbar_init();
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
  // 128 x 64 + 512 x 104 = 640 x 96 registers
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------- TMA producer
      int issued_k = 0, issued_v = 0;
      auto load = [&](int off, const CUtensorMap* map, uint64_t* bar, int v) {
        mbar_arrive_expect_tx(bar, Cfg::TILE);
#pragma unroll
        for (int p = 0; p < Cfg::PANELS; ++p)
          tma_load_4d(smem + off + p * PANEL, map, bar, 64 * p, hk, key_tile(v) * 128, b);
      };
      for (int v = 0; v < nv; ++v) {
        const int ks = v % KS, vs = v % VS;
        if (!mbar_wait(&k_empty[ks], ((v / KS) & 1) ^ 1, st, abort)) break;
        load(Cfg::K_OFF + ks * Cfg::TILE, &mapK, &k_full[ks], v);
        ++issued_k;
        if (!mbar_wait(&v_empty[vs], ((v / VS) & 1) ^ 1, st, abort)) break;
        load(Cfg::V_OFF + vs * Cfg::TILE, &mapV, &v_full[vs], v);
        ++issued_v;
      }
      // every load issued lands before the CTA can exit
      volatile int no_abort = 0;
      for (int j = max(0, issued_k - KS); j < issued_k; ++j)
        mbar_wait(&k_full[j % KS], (j / KS) & 1, st, &no_abort);
      for (int j = max(0, issued_v - VS); j < issued_v; ++j)
        mbar_wait(&v_full[j % VS], (j / VS) & 1, st, &no_abort);
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      const uint32_t k_lo = sdesc_lo(smem_u32(smem + Cfg::K_OFF), 16);
      const uint32_t v_lo = sdesc_lo(smem_u32(smem + Cfg::V_OFF), 16);
      const uint32_t k_mn = sdesc_lo(smem_u32(smem + Cfg::K_OFF), PANEL);
      auto koff = [](int kk) { return static_cast<uint32_t>(((kk >> 2) * PANEL + (kk & 3) * 32) >> 4); };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, st, abort); };
      auto issue_s = [&](int v) {  // S = Q K^T
        const uint32_t kb = k_lo + (((v % KS) * Cfg::TILE) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_bf16_ts_lh(tmem + C_S, tmem + C_Q + kk * 8, kb + koff(kk), HI, ID_S, kk > 0 ? 1u : 0u);
          mma_commit(s_full);
        }
        __syncwarp();
      };
      auto issue_dp = [&](int v) {  // dP = dO V^T
        const uint32_t vb = v_lo + (((v % VS) * Cfg::TILE) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_bf16_ts_lh(tmem + C_DP, tmem + C_DO + kk * 8, vb + koff(kk), HI, ID_S, kk > 0 ? 1u : 0u);
          mma_commit(dp_full);
          mma_commit(&v_empty[v % VS]);
        }
        __syncwarp();
      };
      bool ok = wait(a_ready, 0) && wait(&k_full[0], 0);
      if (ok) {
        issue_s(0);
        ok = wait(&v_full[0], 0);
        if (ok) issue_dp(0);
      }
      for (int v = 0; v < nv && ok; ++v) {
        const bool more = v + 1 < nv;
        if (more) {
          if (!wait(s_free, v & 1) || !wait(&k_full[(v + 1) % KS], ((v + 1) / KS) & 1)) break;
          issue_s(v + 1);
        }
        if (!wait(ds_ready, v & 1)) break;
        const uint32_t kb = k_mn + (((v % KS) * Cfg::TILE) >> 4);
        if (elect_one()) {  // dQ += dS K; the quarters of dS over those of dP
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts_lh(tmem + C_DQ, tmem + C_DP + (kk >> 1) * 32 + (kk & 1) * 8,
                           kb + ((kk * 2048) >> 4), HI, ID_DQ, (v > 0 || kk > 0) ? 1u : 0u);
          if (v == nv - 1) {  // and what its rounding left
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts_lh(tmem + C_DQ, tmem + C_DP + (kk >> 1) * 32 + 16 + (kk & 1) * 8,
                             kb + ((kk * 2048) >> 4), HI, ID_DQ, 1u);
          }
          mma_commit(&k_empty[v % KS]);
        }
        __syncwarp();
        if (more) {
          if (!wait(&v_full[(v + 1) % VS], ((v + 1) / VS) & 1)) break;
          issue_dp(v + 1);
        }
      }
      if (elect_one()) mma_commit(done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(done, 0, st, &no_abort);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;" ::: "memory");
    // --------------------------------------------------------------- query rows
    const int qd = (warp - 4) >> 2;  // quarter of the columns
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int tok = r / a.G, head = hk * a.G + r % a.G;
    const int t = t0 + tok;
    const bool row_ok = tok < a.tpt && t < a.T;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const long long row = (static_cast<long long>(b) * a.T + t) * a.Hq + head;
    uint4* rows = a.rows + ((static_cast<long long>(b) * a.Hkv + hk) * a.n_qt + qt) * 256;
    const float lse = row_ok ? a.lse[(static_cast<long long>(b) * a.Hq + head) * a.T + t] : 0.f;
    const float nl = -lse * 1.4426950408889634f;
    {  // half a row of Q (quarters 0, 1) or dO (2, 3) into TMEM; rows that are not there: zeros
      constexpr int W = HD / 4;  // words
      const int half = qd & 1;
      uint32_t w[W];
      const uint4* src = reinterpret_cast<const uint4*>((qd >= 2 ? a.d_o : a.q) + row * HD + half * (HD / 2));
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 x = row_ok ? src[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
      }
      const uint32_t at = tmem + lane_off + (qd >= 2 ? C_DO : C_Q) + half * W;
      if constexpr (W == 32)
        tmem_st32(at, w);
      else
        tmem_st16(at, w);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(a_ready);
      if (qd >= 2) {
        const uint4* os = reinterpret_cast<const uint4*>(a.o + row * HD + half * (HD / 2));
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const uint4 x = row_ok ? os[i] : make_uint4(0, 0, 0, 0);
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d = fmaf(bf16lo_to_f32(u[e]), bf16lo_to_f32(w[4 * i + e]), d);
            d = fmaf(bf16hi_to_f32(u[e]), bf16hi_to_f32(w[4 * i + e]), d);
          }
        }
        del[half * 128 + r] = -d;
      }
    }
    asm volatile("bar.sync 1, 512;" ::: "memory");
    const float nd = del[r] + del[128 + r];
    // a row that is not there: its P is 0
    if (qd == 0) rows[r] = split3(row_ok ? -lse * a.inv_scale : -3e38f);
    uint64_t nd2 = f2pack(nd, nd);
    const uint64_t nl2 = f2pack(nl, nl);
    const uint32_t s_addr = tmem + lane_off + C_S + 32 * qd, dp_addr = tmem + lane_off + C_DP + 32 * qd;
    uint64_t sum2 = f2pack(0.f, 0.f);  // of p dp
    bool ok = true;
    for (int v = 0; v < nv; ++v) {
      const int k0 = key_tile(v) * 128;
      if (!warp_wait(s_full, v & 1, st, abort)) { ok = false; break; }
      float p[32];
      tmem_ld32f(s_addr, p);
      tc_fence_before();
      mbar_arrive(s_free);
      const bool unmasked =
          k0 + 127 <= t0 && (k0 > t1 - a.window || k0 + 128 <= a.n_sink);
      if (!unmasked)
        mask_scores(p, [&](int) { return seen_bits(t, k0 + 32 * qd, a.window, a.n_sink); });
      probs32<false>(p, a.scale_log2, [&](int) { return nl2; });
      if (!warp_wait(dp_full, v & 1, st, abort)) { ok = false; break; }
      float dp[32];
      tmem_ld32f(dp_addr, dp);
#pragma unroll
      for (int c = 0; c < 32; c += 2) sum2 = fma2(f2pack(p[c], p[c + 1]), f2pack(dp[c], dp[c + 1]), sum2);
      if (v == nv - 1) {
        // Now delta is known as sum_j p_j dp_j in 32 bits.  The one from dO and o carries
        // o's rounding to bf16, an error e that all keys of a row share: it puts
        // e sum p k into dQ, and that is a sum without cancellation over the sinks, which
        // many queries lean on.  They are in this last visit, so it takes the better
        // delta, and the second kernel takes it for all keys.
        float s0, s1;
        f2unpack(sum2, s0, s1);
        sums[qd * 128 + r] = s0 + s1;
        mbar_arrive(sum_ready);
        if (!warp_wait(sum_ready, 0, st, abort)) { ok = false; break; }
        const float exact = -((sums[r] + sums[128 + r]) + (sums[256 + r] + sums[384 + r]));
        nd2 = f2pack(exact, exact);
        if (qd == 0) rows[128 + r] = split3(row_ok ? exact : 0.f);
      }
      ds32(p, dp, nd2);
      store_operand(dp_addr, dp, v == nv - 1);
      mbar_arrive(ds_ready);
    }
    if (ok && warp_wait(done, 0, st, abort)) {
      // a quarter of the row's columns each
      __nv_bfloat16* dst = a.dq + row * HD + qd * (HD / 4);
#pragma unroll
      for (int c = 0; c < HD / 4; c += 16) {
        uint32_t x[16];
        tmem_ld16(tmem + lane_off + C_DQ + qd * (HD / 4) + c, x);
        tmem_ld_wait();
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(x[i]) * a.scale;
        if (row_ok) {
          st8f(dst + c, *reinterpret_cast<float(*)[8]>(&y[0]));
          st8f(dst + c + 8, *reinterpret_cast<float(*)[8]>(&y[8]));
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
__global__ void __launch_bounds__(SINKB_THREADS, 1)
    sink_attn_dkv_kernel(const __grid_constant__ CUtensorMap mapQ,
                         const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV,
                         const __grid_constant__ CUtensorMap mapDO, const SinkBwdArgs a,
                         const DevStatus st) {
  using Cfg = SinkDkvCfg<HD>;
  grid_dep_launch();
  constexpr int PANEL = 128 * 128, NBS = Cfg::NBS, QS = Cfg::QS;
  constexpr uint32_t ID_S = idesc_bf16_f32(128, 128, false, false);  // S^T, dP^T
  constexpr uint32_t ID_KV = idesc_bf16_f32(128, HD, false, true);   // dK, dV
  constexpr uint32_t C_S = 0, C_DP = NBS * 128, C_DK = C_DP + 128, C_DV = C_DK + HD;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::BAR_OFF);
  uint64_t* kv_full = bars;
  uint64_t* q_full = bars + 1;         // QS (Q and the extra step's rows)
  uint64_t* q_empty = q_full + QS;     // QS
  uint64_t* do_full = q_empty + QS;    // 2
  uint64_t* do_empty = do_full + 2;    // 2
  uint64_t* s_full = do_empty + 2;     // NBS
  uint64_t* p_ready = s_full + NBS;    // NBS, every element thread arrives
  uint64_t* dp_full = p_ready + NBS;
  uint64_t* ds_ready = dp_full + 1;    // every element thread arrives
  uint64_t* done = ds_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int hk = static_cast<int>(blockIdx.x) % a.Hkv;
  const int b = static_cast<int>(blockIdx.x) / a.Hkv % a.B;
  const int item = static_cast<int>(blockIdx.x) / (a.Hkv * a.B);
  const bool far = item < a.n_far;
  const int near = item - a.n_far, other = near - a.parts0;
  const int kt = other < 0 ? 0 : 1 + other / a.parts;
  const int parts = other < 0 ? a.parts0 : a.parts;
  const int part = far ? 0 : other < 0 ? near : other % a.parts;
  const int k0 = kt * 128;
  // query tiles [qt0, qt0 + nv)
  const int first = far ? a.far0 + item * a.far_tiles : k0 / a.tpt;
  const int all = (far ? min(first + a.far_tiles, a.n_qt)
                       : min(a.T - 1, k0 + 127 + a.window - 1) / a.tpt + 1) - first;
  const int cut = far ? 0 : static_cast<int>(static_cast<long long>(all) * part / parts);
  const int qt0 = first + cut;
  // may be 0: a part without visits
  const int nv = (far ? all : static_cast<int>(static_cast<long long>(all) * (part + 1) / parts)) - cut;
  const int rows_used = a.G * a.tpt;
  // the sinks' tile, or the only one (few rows, which average little)
  const bool split = kt == 0 && (a.n_sink > 0 || a.n_kt == 1);

  if (threadIdx.x == 0) {
    for (uint64_t* p = bars; p <= done; ++p) mbar_init(p, (p >= p_ready && p < dp_full) || p == ds_ready ? SINKB_ROWS : 1);
    *abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
    tma_prefetch_map(&mapDO);
  }
  // rows of the Q and dO stages that no load writes: zeros (their P is 0, and 0
  // times what lies there must be 0)
  constexpr int PANELS_IN = Cfg::PANELS * (QS + 2);
  for (int i = threadIdx.x; i < (128 - rows_used) * 8 * PANELS_IN; i += SINKB_THREADS) {
    const int c = i & 7, x = i >> 3, panel = x % PANELS_IN, r = rows_used + x / PANELS_IN;
    *reinterpret_cast<uint4*>(smem + Cfg::Q_OFF + panel * PANEL + r * 128 + c * 16) =
        make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x < 128) {
    *reinterpret_cast<uint4*>(smem + Cfg::ZERO_OFF + threadIdx.x * 16) = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(smem + Cfg::ONE_OFF + threadIdx.x * 16) =
        make_uint4(0x3f803f80u, 0x3f80u, 0, 0);  // 1, 1, 1, 0 ...
  }
  fence_async_smem();
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------- TMA producer
      const uint32_t bytes = Cfg::PANELS * 128 * rows_used;
      const uint4* rows = a.rows + (static_cast<long long>(b) * a.Hkv + hk) * a.n_qt * 256;
      mbar_arrive_expect_tx(kv_full, 2 * Cfg::TILE);
#pragma unroll
      for (int p = 0; p < Cfg::PANELS; ++p) {
        tma_load_4d(smem + Cfg::K_OFF + p * PANEL, &mapK, kv_full, 64 * p, hk, k0, b);
        tma_load_4d(smem + Cfg::V_OFF + p * PANEL, &mapV, kv_full, 64 * p, hk, k0, b);
      }
      grid_dep_wait();  // the rows' numbers are the dQ kernel's
      int issued_q = 0, issued_do = 0;
      for (int v = 0; v < nv; ++v) {
        const int sg = v % QS, so = v & 1, qt = qt0 + v;
        if (!mbar_wait(&q_empty[sg], ((v / QS) & 1) ^ 1, st, abort)) break;
        mbar_arrive_expect_tx(&q_full[sg], bytes + 4096);
#pragma unroll
        for (int p = 0; p < Cfg::PANELS; ++p)
          tma_load_4d(smem + Cfg::Q_OFF + sg * Cfg::TILE + p * PANEL, &mapQ, &q_full[sg], 64 * p,
                      hk * a.G, qt * a.tpt, b);
        bulk_load(smem + Cfg::EXT_OFF + sg * 4096, rows + qt * 256ll, 4096, &q_full[sg]);
        ++issued_q;
        if (!mbar_wait(&do_empty[so], ((v >> 1) & 1) ^ 1, st, abort)) break;
        mbar_arrive_expect_tx(&do_full[so], bytes);
#pragma unroll
        for (int p = 0; p < Cfg::PANELS; ++p)
          tma_load_4d(smem + Cfg::DO_OFF + so * Cfg::TILE + p * PANEL, &mapDO, &do_full[so], 64 * p,
                      hk * a.G, qt * a.tpt, b);
        ++issued_do;
      }
      volatile int no_abort = 0;
      mbar_wait(kv_full, 0, st, &no_abort);
      for (int j = max(0, issued_q - QS); j < issued_q; ++j)
        mbar_wait(&q_full[j % QS], (j / QS) & 1, st, &no_abort);
      for (int j = max(0, issued_do - 2); j < issued_do; ++j)
        mbar_wait(&do_full[j & 1], (j >> 1) & 1, st, &no_abort);
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      constexpr uint32_t HI = sdesc_hi_sw128(1024);
      constexpr uint32_t STAGE = Cfg::TILE >> 4;
      const uint32_t k_lo = sdesc_lo(smem_u32(smem + Cfg::K_OFF), 16);
      const uint32_t v_lo = sdesc_lo(smem_u32(smem + Cfg::V_OFF), 16);
      const uint32_t q_lo = sdesc_lo(smem_u32(smem + Cfg::Q_OFF), 16);
      const uint32_t do_lo = sdesc_lo(smem_u32(smem + Cfg::DO_OFF), 16);
      const uint32_t q_mn = sdesc_lo(smem_u32(smem + Cfg::Q_OFF), PANEL);
      const uint32_t do_mn = sdesc_lo(smem_u32(smem + Cfg::DO_OFF), PANEL);
      auto koff = [](int kk) { return static_cast<uint32_t>(((kk >> 2) * PANEL + (kk & 3) * 32) >> 4); };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity, st, abort); };
      // the extra step: 16-byte rows, 8 rows to 128 bytes, no swizzle; elements 8 .. 15
      // lie in the zeros
      constexpr uint32_t HI0 = (128u >> 4) | (1u << 14);
      const uint32_t one_lo = sdesc_lo(smem_u32(smem + Cfg::ONE_OFF), Cfg::ZERO_OFF - Cfg::ONE_OFF);
      auto issue_scores = [&](uint32_t d, uint32_t a_lo, uint32_t b_lo, int ext, uint64_t* bar) {
        const uint32_t e_lo = sdesc_lo(smem_u32(smem + ext), Cfg::ZERO_OFF - ext);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            mma_bf16_ss_lh(tmem + d, a_lo + koff(kk), HI, b_lo + koff(kk), HI, ID_S, kk > 0 ? 1u : 0u);
          mma_bf16_ss_lh(tmem + d, one_lo, HI0, e_lo, HI0, ID_S, 1u);
          mma_commit(bar);
        }
        __syncwarp();
      };
      auto issue_s = [&](int v) {
        const int sg = v % QS;
        issue_scores(C_S + (v % NBS) * 128, k_lo, q_lo + sg * STAGE, Cfg::EXT_OFF + sg * 4096,
                     &s_full[v % NBS]);
      };
      auto issue_dp = [&](int v) {
        issue_scores(C_DP, v_lo, do_lo + (v & 1) * STAGE, Cfg::EXT_OFF + (v % QS) * 4096 + 2048, dp_full);
      };
      // += P^T dO or dS^T Q; the quarters of the A operand over those of its scores
      auto issue_acc = [&](uint32_t d, uint32_t at, uint32_t b_mn, bool first, uint64_t* bar) {
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ts_lh(tmem + d, tmem + at + (kk >> 1) * 32 + (kk & 1) * 8,
                           b_mn + ((kk * 2048) >> 4), HI, ID_KV, (!first || kk > 0) ? 1u : 0u);
          if (split) {  // and what its rounding left
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ts_lh(tmem + d, tmem + at + (kk >> 1) * 32 + 16 + (kk & 1) * 8,
                             b_mn + ((kk * 2048) >> 4), HI, ID_KV, 1u);
          }
          mma_commit(bar);
        }
        __syncwarp();
      };
      bool ok = nv > 0 && wait(kv_full, 0) && wait(&q_full[0], 0);
      if (ok) {
        issue_s(0);
        ok = wait(&do_full[0], 0);
        if (ok) issue_dp(0);
      }
      if (ok && NBS == 2 && nv > 1) {
        ok = wait(&q_full[1], 0);
        if (ok) issue_s(1);
      }
      for (int v = 0; v < nv && ok; ++v) {
        const uint32_t so = v & 1;
        if (!wait(&p_ready[v % NBS], (v / NBS) & 1)) break;
        issue_acc(C_DV, C_S + (v % NBS) * 128, do_mn + so * STAGE, v == 0, &do_empty[so]);
        if (v + NBS < nv) {  // over the P^T that dV has just read
          if (!wait(&q_full[(v + NBS) % QS], ((v + NBS) / QS) & 1)) break;
          issue_s(v + NBS);
        }
        if (!wait(ds_ready, v & 1)) break;
        issue_acc(C_DK, C_DP, q_mn + (v % QS) * STAGE, v == 0, &q_empty[v % QS]);
        if (v + 1 < nv) {
          if (!wait(&do_full[so ^ 1], ((v + 1) >> 1) & 1)) break;
          issue_dp(v + 1);
        }
      }
      if (elect_one()) mma_commit(done);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(done, 0, st, &no_abort);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;" ::: "memory");
    // ----------------------------------------------------------------- key rows
    const int qd = (warp - 4) >> 2;  // quarter of the columns
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int j = k0 + r;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + C_S + 32 * qd, dp_addr = tmem + lane_off + C_DP + 32 * qd;
    bool ok = true;
    for (int v = 0; v < nv; ++v) {
      const int t0 = (qt0 + v) * a.tpt, t1 = t0 + a.tpt - 1;
      const uint32_t s_at = s_addr + (v % NBS) * 128;
      if (!warp_wait(&s_full[v % NBS], (v / NBS) & 1, st, abort)) { ok = false; break; }
      float p[32];
      tmem_ld32f(s_at, p);
      const bool unmasked =
          k0 + 127 <= t0 && (t1 - a.window < k0 || k0 + 128 <= a.n_sink);
      if (!unmasked) {
        // columns (token, head) of the tokens from j to the last that sees it
        const int lo = max(j - t0, 0) * a.G - 32 * qd;
        const int last = j < a.n_sink ? 128 : min(max(j + a.window - t0, 0), 128);
        const int hi = last * a.G - 32 * qd;
        mask_scores(p, [&](int) { return low_bits(hi) & ~low_bits(lo); });
      }
      probs32<true>(p, a.scale_log2, [](int) { return 0ull; });
      store_operand(s_at, p, split);
      mbar_arrive(&p_ready[v % NBS]);
      if (!warp_wait(dp_full, v & 1, st, abort)) { ok = false; break; }
      float dp[32];
      tmem_ld32f(dp_addr, dp);
#pragma unroll
      for (int c = 0; c < 32; c += 2)
        f2unpack(mul2(f2pack(p[c], p[c + 1]), f2pack(dp[c], dp[c + 1])), dp[c], dp[c + 1]);
      store_operand(dp_addr, dp, split);
      mbar_arrive(ds_ready);
    }
    // ------------------------------------ halves of the dK (quarters 0, 1) and dV rows
    if (ok && warp_wait(done, 0, st, abort)) {
      const int which = qd >> 1, col = (qd & 1) * (HD / 2);
      const float f = which ? 1.f : a.scale;
      const long long bh = static_cast<long long>(b) * a.Hkv + hk, heads = static_cast<long long>(a.B) * a.Hkv;
      // a sum of several items goes to its partial row
      float* ps = nullptr;
      if (!far && parts > 1)
        ps = kt == 0 ? a.near0 + (((part * heads + bh) * 2 + which) * 128 + r) * HD
                     : a.near_rows + (((part * heads + bh) * 2 + which) * a.n_kt * 128 + j) * HD;
      else if (a.n_far > 0 && kt == 0 && r < a.n_sink)
        ps = a.partial + ((((far ? item : a.n_far) * heads + bh) * 2 + which) * a.n_sink + r) * HD;
      __nv_bfloat16* dst = (which ? a.dv : a.dk) + ((static_cast<long long>(b) * a.T + j) * a.Hkv + hk) * HD + col;
#pragma unroll
      for (int c = 0; c < HD / 2; c += 32) {
        float x[32];
        if (nv > 0) {
          tmem_ld32f(tmem + lane_off + (which ? C_DV : C_DK) + col + c, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= f;
        if (ps && j < a.T)
          store_f32x32(ps + col + c, x);
        else if (!far && j < a.T)
          store_x32(dst + c, x);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums of partial rows, in the items' order: dk and dv of the sinks, of the first key
// tile (parts0 > 1) or of every key (parts > 1).  One thread per four elements.
__host__ __device__ __forceinline__ int join_rows(const SinkBwdArgs& a) {
  return a.parts > 1 ? a.T : a.parts0 > 1 ? (a.T < 128 ? a.T : 128) : a.n_sink;
}
template <int HD>
__global__ void sink_attn_join_kernel(const SinkBwdArgs a) {
  grid_dep_wait();
  const int rows = join_rows(a);
  const long long heads = static_cast<long long>(a.B) * a.Hkv;
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= heads * 2 * rows * (HD / 4)) return;
  const int c = static_cast<int>(i % (HD / 4)) * 4;
  long long y = i / (HD / 4);
  const int r = static_cast<int>(y % rows);
  y /= rows;
  const int which = static_cast<int>(y & 1);
  const long long bh = y >> 1;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float* p) {
    const float4 z = *reinterpret_cast<const float4*>(p);
    x.x += z.x;
    x.y += z.y;
    x.z += z.z;
    x.w += z.w;
  };
  if (r >= 128) {
    for (int f = 0; f < a.parts; ++f)
      add(a.near_rows + (((f * heads + bh) * 2 + which) * a.n_kt * 128 + r) * HD + c);
  } else if (a.parts0 > 1) {
    for (int f = 0; f < a.parts0; ++f)
      add(a.near0 + (((f * heads + bh) * 2 + which) * 128 + r) * HD + c);
  }
  if (r < a.n_sink && a.n_far > 0)
    for (int f = 0; f < a.n_far + (a.parts0 > 1 ? 0 : 1); ++f)
      add(a.partial + (((f * heads + bh) * 2 + which) * a.n_sink + r) * HD + c);
  const long long b = bh / a.Hkv, hk = bh % a.Hkv;
  *reinterpret_cast<uint2*>((which ? a.dv : a.dk) + ((b * a.T + r) * a.Hkv + hk) * HD + c) =
      make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

}  // namespace ttcd
