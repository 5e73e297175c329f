// Paged attention with up to 128 query rows per item; see paged.cuh for the method.
#pragma once
#include "paged.cuh"

namespace attn {

// ------------------------------------------------------------------ one query tile per CTA
// Warps 0-15 softmax: four groups of 32 keys of each tile, thread = tile row = TMEM lane.
// (Two groups of 64 keys: a tile took 3.9k cycles, chains of TMEM reads and exponentials that
// two warps per scheduler cannot hide.)  Warps 16 and 18 producers of K (and Q) and of V,
// warp 17 MMA issuer and, for an e4m3 cache, warps 19-26 that widen raw tiles to bf16 ones.
// TMEM: S in two buffers, so S of the next tile is computed while the softmax works on this
// one (P is written over S: keys [32k, 32k + 32) in columns [32k, 32k + 16)), and O.
template <int D_, bool KV8_>
struct RowsCfg {
  static constexpr int D = D_;
  static constexpr bool KV8 = KV8_;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kTeams = 1;
  static constexpr int kBox = 128 * 128;
  static constexpr int NB = D / 64;                // 64-column boxes of a bf16 tile
  static constexpr int QST = (KV8 && D == 128) ? 1 : 2;
  static constexpr bool K8 = false;
  static constexpr int KSK = 2, KSV = 2;           // stages of K and of V
  static constexpr int kKTile = kTile;
  static constexpr int kQTile = kTile, kQBox = kBox;
  static constexpr int kWiden = KV8 ? 8 : 0;       // widening warps
  static constexpr int kThreads = 608 + 32 * kWiden;
  static constexpr int kRawTile = 128 * D;         // e4m3 codes of a tile
  // Raw stages, K and V tiles alternating.  An even number: the two producers run on their
  // own, so each needs its own stages (with 3, K could take one that V had yet to fill).
  static constexpr int RST = KV8 ? (D == 128 ? 2 : 6) : 0;
  static_assert(RST % 2 == 0, "K and V must not share a raw stage");
  static constexpr int kRawMod = KV8 ? RST : 1;
  static constexpr int kS0 = 0, kS1 = 128, kO = 256;
  static constexpr int kTmemCols = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = QST * kTile;
  static constexpr int kOffV = kOffK + KSK * kTile;
  static constexpr int kOffRaw = kOffV + KSK * kTile;
  static constexpr int kOffScale = kOffRaw + RST * kRawTile;  // 128 scale bytes per raw stage
  static constexpr int kOffSh = kOffScale + RST * 128;
  static constexpr int kLayout = kOffSh + 8192;
  static constexpr int kSmem = kLayout + 1024;
  static_assert(kSmem <= 232448, "shared memory layout exceeds 227 KB");
};

struct RowsShared : PagedPipe {
  float xmax[2][4][128];      // [parity of the quadrant's steps][group][row] partial row maxima
  float xsum[4][128];
  uint64_t p_ready[2];
  uint64_t xbar[2][4];        // [parity][quadrant]: the four groups' warps posted their maxima
  uint64_t sbar[4];
  uint64_t o_free;
};
static_assert(sizeof(RowsShared) <= 8192, "RowsShared does not fit its slot");

template <int D, bool KV8>
__global__ void __launch_bounds__(RowsCfg<D, KV8>::kThreads, 1)
    attn_paged_rows_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const PagedParams p) {
  using C = RowsCfg<D, KV8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RowsShared& sh = *reinterpret_cast<RowsShared*>(smem + C::kOffSh);
  const PagedSmem m = {smem + C::kOffQ, smem + C::kOffK, smem + C::kOffV, smem + C::kOffRaw, smem + C::kOffScale, nullptr};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    paged_pipe_init<C>(sh, 18 + C::kWiden, 19 + C::kWiden);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.p_ready[i], 16);
      for (int q = 0; q < 4; ++q) mbar_init(&sh.xbar[i][q], 4);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&sh.sbar[q], 4);
    mbar_init(&sh.o_free, 16);
    fence_barrier_init();
  }
  if (warp == 0) { tmem_alloc(&sh.tmem_base, C::kTmemCols); tmem_relinquish(); }
  grid_dependency_wait();
  grid_dependency_launch();
  paged_plan(p, sh.plan, cta, warp == 16, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 16) {
    paged_produce_k<C>(p, sh, &tmq, &tmk, m, cta, lane);
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
    // Per piece: S(0), S(1); then per step j: PV(j), S(j + 2) into the buffer PV(j) just
    // read (MMAs of one thread run in issue order, so PV(j) reads P(j) first).
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
    constexpr uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t q_lo0 = sdesc_lo(smem_u32(m.q), 16);
    const uint32_t k_lo0 = sdesc_lo(smem_u32(m.k), 16);
    const uint32_t v_lo0 = sdesc_lo(smem_u32(m.v), C::kBox);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity));
    };
    int kc = 0, vc = 0, gs = 0, uq = 0;
    bool ok = true;
    auto issue_s = [&](int g, int qs) -> bool {     // S(g) = Q K(kc)^T into buffer g % 2
      const int st = kc & 1;
      if (!wait(&sh.k_full[st], (kc >> 1) & 1)) return false;
      tc_fence_after();
      if (leader) {
        const uint32_t q_lo = q_lo0 + qs * (C::kTile >> 4);
        const uint32_t k_lo = k_lo0 + st * (C::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::kBox + (k & 3) * 32) >> 4;
          umma_ss_lo(tmem + ((g & 1) ? C::kS1 : C::kS0), q_lo + off, k_lo + off, hi, idS, k > 0);
        }
        umma_commit(&sh.k_done[kc & 7]);
      }
      __syncwarp();
      ++kc;
      return true;
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      const int qs = uq % C::QST;
      ok = wait(&sh.q_full[qs], (uq / C::QST) & 1);
      for (int t = 0; t < 2 && t < w.n && ok; ++t) {
        ok = issue_s(gs + t, qs);
        if (ok && t == w.n - 1 && leader) umma_commit(&sh.q_empty[qs]);
        __syncwarp();
      }
      for (int j = 0; j < w.n && ok; ++j, ++vc) {
        const int g = gs + j, vst = vc & 1;
        ok = wait(&sh.v_full[vst], (vc >> 1) & 1);
        if (!KV8 && ok) paged_zero_v<C>(w, j, m.v + vst * C::kTile, lane);
        if (ok) ok = wait(&sh.p_ready[g & 1], (g >> 1) & 1);
        if (ok && j == 0 && uq >= 1) ok = wait(&sh.o_free, (uq - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t v_lo = v_lo0 + vst * (C::kTile >> 4);
          const uint32_t sbase = tmem + ((g & 1) ? C::kS1 : C::kS0);
#pragma unroll
          for (int k2 = 0; k2 < 8; ++k2)
            umma_ts_lo(tmem + C::kO, sbase + (k2 >> 1) * 32 + (k2 & 1) * 8, v_lo + ((k2 * 2048) >> 4), hi, idO,
                       !(j == 0 && k2 == 0));
          umma_commit(&sh.v_done[vc & 7]);
        }
        __syncwarp();
        if (j + 2 < w.n) {
          ok = issue_s(g + 2, qs);
          if (ok && j + 2 == w.n - 1 && leader) umma_commit(&sh.q_empty[qs]);
          __syncwarp();
        }
      }
      gs += w.n;
      ++uq;
    }
    if (leader) {
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp == 18) {
    paged_produce_v<C>(p, sh, &tmv, m, lane);
  } else if (warp >= 19) {
    if constexpr (KV8) paged_widen<C>(sh, m, threadIdx.x - 608, lane, [](int, int) {});
  } else {
    // ------------------------------------------------------------ softmax warps 0-15
    const int grp = warp >> 2;                                  // keys [32 grp, 32 grp + 32)
    const int quad = warp & 3;
    const int row = quad * 32 + lane;                           // tile row = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    constexpr int OH = D / 4;
    const uint32_t o_base = lane_base + C::kO + grp * OH;
    const float c = p.cs;
    const uint64_t c2 = f2pack(c, c);
    const int i = row / p.G, h = row - i * p.G;                 // token of the tile, head of the group
    int gs = 0, uq = 0;
    int xs = 0;                 // steps in which this quadrant had rows: its maxima barriers' count
    bool ok = true;
    auto mask16 = [&](uint32_t (&r)[16], int col0, int lo, int lim) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (col0 + k < lo || col0 + k > lim) r[k] = 0xff800000u;
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      const bool valid = i < w.ntok && row < p.G * p.R;
      const bool active = __any_sync(0xffffffffu, valid);       // a warp without rows only keeps step
      const int pos = w.pos0 + i;
      const int lastk = p.causal ? min(w.len - 1, pos) : w.len - 1;
      const int firstk = p.wl >= 0 ? pos - p.wl : 0;
      float m_used = -INFINITY;
      uint64_t lsum = f2pack(0.f, 0.f);
      for (int j = 0; j < w.n && ok; ++j) {
        const int g2 = gs + j, xp = xs & 1;
        const uint32_t s_base = lane_base + ((g2 & 1) ? C::kS1 : C::kS0) + grp * 32;
        ok = __all_sync(0xffffffffu, tile_done_wait(sh.k_done, g2));
        if (!ok) break;
        if (!active) {
          if (lane == 0) mbar_arrive(&sh.p_ready[g2 & 1]);
          __syncwarp();
          continue;
        }
        tc_fence_after();
        const int kbase = (w.j0 + j) * 128 + grp * 32;
        const int lo = firstk - kbase, lim = lastk - kbase;        // visible columns [lo, lim]
        const bool msk = __any_sync(0xffffffffu, valid && (lo > 0 || lim < 31));
        uint32_t r[2][16];
        tmem_ld16(s_base, r[0]);
        tmem_ld16(s_base + 16, r[1]);
        tmem_wait_ld();
        reg_fence(r[0]);
        reg_fence(r[1]);
        if (msk) { mask16(r[0], 0, lo, lim); mask16(r[1], 16, lo, lim); }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int cc = 0; cc < 2; ++cc)
#pragma unroll
          for (int kk = 0; kk < 16; kk += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx4[e] = max3f(mx4[e], __uint_as_float(r[cc][kk + e]), __uint_as_float(r[cc][kk + e + 4]));
        sh.xmax[xp][grp][row] = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.xbar[xp][quad]);
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.xbar[xp][quad], (xs >> 1) & 1));
        if (!ok) break;
        ++xs;
        const float mx = fmaxf(fmaxf(sh.xmax[xp][0][row], sh.xmax[xp][1][row]),
                               fmaxf(sh.xmax[xp][2][row], sh.xmax[xp][3][row]));
        const float m_tile = mx == -INFINITY ? -INFINITY : mx * c;
        float alpha = 1.f;
        // a row that has seen no key keeps m_used = -inf (and p = 0) until it sees one
        const bool need = valid && m_tile > m_used + kRescaleTau;
        if (need) {
          alpha = (m_used == -INFINITY) ? 0.f : ex2_approx(m_used - m_tile);
          float l0, l1;
          f2unpack(lsum, l0, l1);
          lsum = f2pack(l0 * alpha, l1 * alpha);
          m_used = m_tile;
        }
        // S(j) was issued before PV(j - 1) (and after PV(j - 2), which its commit covers):
        // wait for PV(j - 1) before rescaling O
        if (__any_sync(0xffffffffu, need && j > 0)) {
          ok = __all_sync(0xffffffffu, tile_done_wait(sh.v_done, g2 - 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int q4 = 0; q4 < OH / 16; ++q4) {
            uint32_t o[16];
            tmem_ld16(o_base + q4 * 16, o);
            tmem_wait_ld();
            reg_fence(o);
#pragma unroll
            for (int kk = 0; kk < 16; ++kk)
              o[kk] = alpha == 0.f ? 0u : __float_as_uint(__uint_as_float(o[kk]) * alpha);
            tmem_st16(o_base + q4 * 16, o);
          }
        }
        const float mb = m_used == -INFINITY ? 0.f : m_used;
        const uint64_t nm2 = f2pack(-mb, -mb);
        // the scores are still in registers; P goes over this group's own columns of S
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t pk[8];
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t xx =
                ffma2(f2pack(__uint_as_float(r[cc][2 * kk]), __uint_as_float(r[cc][2 * kk + 1])), c2, nm2);
            float x0, x1;
            f2unpack(xx, x0, x1);
            const float a0 = ex2_approx(x0), a1 = ex2_approx(x1);
            lsum = fadd2(lsum, f2pack(a0, a1));
            pk[kk] = pack_bf16x2(a0, a1);
          }
          tmem_st8(s_base + cc * 8, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[g2 & 1]);
      }
      if (!ok) break;
      // epilogue: the four groups' sums, the last PV, O / l and the LSE of this piece
      const int glast = gs + w.n - 1;
      float l = 0.f;
      if (active) {
        float l0, l1;
        f2unpack(lsum, l0, l1);
        sh.xsum[grp][row] = l0 + l1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sbar[quad]);
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.sbar[quad], uq & 1));
      if (!ok) break;
      if (active) l = (sh.xsum[0][row] + sh.xsum[1][row]) + (sh.xsum[2][row] + sh.xsum[3][row]);
      ok = __all_sync(0xffffffffu, tile_done_wait(sh.v_done, glast));
      if (!ok) break;
      if (active) {
        tc_fence_after();
        const bool none = l == 0.f;                               // no key seen
        const float inv_l = none ? 0.f : 1.f / l;
        const float lse_s = none ? -INFINITY : (m_used + __log2f(l)) * 0.69314718055994531f;
        const size_t orow = static_cast<size_t>(w.tok0 + i) * p.Hq + w.g * p.G + h;
        const bool store = valid && in_range(w.tok0 + i, p.T) && in_range(row, w.slot < 0 ? 128 : p.slot_rows);
#pragma unroll 1
        for (int q4 = 0; q4 < OH / 16; ++q4) {
          uint32_t o[16];
          tmem_ld16(o_base + q4 * 16, o);
          tmem_wait_ld();
          reg_fence(o);
          if (!store) continue;
          float f[16];
#pragma unroll
          for (int kk = 0; kk < 16; ++kk) f[kk] = none ? 0.f : __uint_as_float(o[kk]) * inv_l;
          if (w.slot < 0) {
            uint32_t pk[8];
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) pk[kk] = pack_bf16x2(f[2 * kk], f[2 * kk + 1]);
            uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D + grp * OH + q4 * 16);
            dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          } else {
            float4* dst = reinterpret_cast<float4*>(
                p.opart + (static_cast<size_t>(w.slot) * p.slot_rows + row) * D + grp * OH + q4 * 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              dst[kk] = make_float4(f[4 * kk], f[4 * kk + 1], f[4 * kk + 2], f[4 * kk + 3]);
          }
        }
        if (store && grp == 0) {
          if (w.slot < 0) p.lse[orow] = lse_s;
          else p.lpart[static_cast<size_t>(w.slot) * p.slot_rows + row] = lse_s;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free);
      gs += w.n;
      ++uq;
    }
  }

  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.teardown);
  if (warp == 0) {
    mbar_wait(&sh.teardown, 0);
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace attn
