// Paged attention with many query rows per sequence (chunks of a prompt), bf16 cache: two
// query tiles per CTA; see paged.cuh for the method and the sharing of work.
//
// An item is two adjacent 128-row query tiles A and B of one KV head, 2R tokens, which see
// the same keys but for the last tile or so: each K/V tile is read once for both.  Team A
// (warps 0-7) owns tile A, team B (warps 8-15) tile B, and the MMA warp interleaves their
// products as the dense forward does (fwd_pp.cuh): while one team exponentiates, the tensor
// cores work on the other team's S or PV.  One query tile per CTA reaches 930 TFLOP/s on a
// 4K chunk over 28K cached keys, its softmax and products taking turns.
//
//   warps 0-7, 8-15  softmax teams; inside a team, group k = (warp % 8) / 4 owns keys
//                    [64k, 64k + 64) of each S tile and O columns [kD/2, (k+1)D/2); thread =
//                    query row = TMEM lane
//   warps 16, 18     producers of K (and Q) and of V
//   warp 17          MMA issuer: per key tile PV_A(j), S_A(j+1), PV_B(j), S_B(j+1), each PV in
//                    two halves (p_half: the first 32 keys of each group's P are there)
// TMEM: S_A at 0, S_B at 128 (P written over S), O_A at 256, O_B at 256 + D.
#pragma once
#include "paged.cuh"

namespace attn {

template <int D_>
struct PairCfg {
  static constexpr int D = D_;
  static constexpr bool KV8 = false, K8 = false;
  static constexpr int kTeams = 2;
  static constexpr int kTile = 128 * D * 2, kKTile = kTile;
  static constexpr int kBox = 128 * 128;
  static constexpr int NB = D / 64;
  static constexpr int kQBox = kBox, kQTeam = kTile;      // Q of one team
  static constexpr int kQTile = 2 * kTile;
  static constexpr int QST = D == 64 ? 2 : 1;
  static constexpr int KSK = 2, KSV = 2;
  static constexpr int RST = 0, kRawMod = 1, kRawTile = 0, kWiden = 0;
  static constexpr int kFmaPairs = D == 64 ? 2 : 1;       // of 8 score pairs, on the FMA pipe (fwd_pp.cuh)
  static constexpr int kThreads = 608;
  static constexpr int kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 256 + D;
  static constexpr int kTmemCols = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = QST * kQTile;
  static constexpr int kOffV = kOffK + KSK * kTile;
  static constexpr int kOffSh = kOffV + KSV * kTile;
  static constexpr int kShared = 8192;
  static constexpr int kSmem = kOffSh + kShared + 1024;
  static_assert(kSmem <= 232448, "shared memory layout exceeds 227 KB");
};

struct PairShared : PagedPipe {
  float xmax[2][2][2][128];   // [team][parity of the quadrant's steps][group][row]
  float xsum[2][2][128];      // [team][group][row]
  uint64_t s_full[2], p_half[2], p_ready[2], pv_done[2];      // per team
  uint64_t xbar[2][2][4];     // [team][parity][quadrant]: both groups' warps posted their maxima
  uint64_t sbar[2][4];        // [team][quadrant]
  uint64_t o_free[2];
};
static_assert(sizeof(PairShared) <= PairCfg<64>::kShared, "PairShared does not fit its slot");

template <int D>
__global__ void __launch_bounds__(PairCfg<D>::kThreads, 1)
    attn_paged_pair_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv, const PagedParams p) {
  using C = PairCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PairShared& sh = *reinterpret_cast<PairShared*>(smem + C::kOffSh);
  const PagedSmem m = {smem + C::kOffQ, smem + C::kOffK, smem + C::kOffV, nullptr, nullptr, nullptr};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    paged_pipe_init<C>(sh, 18, 19);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh.s_full[x], 1);
      mbar_init(&sh.p_half[x], 8);
      mbar_init(&sh.p_ready[x], 8);
      mbar_init(&sh.pv_done[x], 1);
      for (int q = 0; q < 4; ++q) {
        mbar_init(&sh.xbar[x][0][q], 2);
        mbar_init(&sh.xbar[x][1][q], 2);
        mbar_init(&sh.sbar[x][q], 2);
      }
      mbar_init(&sh.o_free[x], 8);
    }
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
  } else if (warp == 18) {
    paged_produce_v<C>(p, sh, &tmv, m, lane);
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
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
    int c0 = 0;                      // key tiles before the piece
    int gs[2] = {0, 0}, uu[2] = {0, 0};      // steps and pieces per team
    bool ok = true;
    auto issue_s = [&](int x, int qs, int c) {              // S_X = Q_X K(c)^T
      if (leader) {
        const uint32_t q_lo = q_lo0 + ((qs * C::kQTile + x * C::kQTeam) >> 4);
        const uint32_t k_lo = k_lo0 + (c % C::KSK) * (C::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::kBox + (k & 3) * 32) >> 4;
          umma_ss_lo(tmem + (x ? C::kS1 : C::kS0), q_lo + off, k_lo + off, hi, idS, k > 0);
        }
        umma_commit(&sh.s_full[x]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, int c, bool first, int half) {     // O_X (+)= P_X V(c)
      if (leader) {
        const uint32_t v_lo = v_lo0 + (c % C::KSV) * (C::kTile >> 4);
        const uint32_t sbase = tmem + (x ? C::kS1 : C::kS0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int k = (kk >> 1) * 4 + half * 2 + (kk & 1);      // half 0: keys 0-31 and 64-95
          umma_ts_lo(tmem + (x ? C::kO1 : C::kO0), sbase + (k >> 2) * 64 + (k & 3) * 8, v_lo + ((k * 2048) >> 4), hi,
                     idO, !(first && k == 0));
        }
        if (half) umma_commit(&sh.pv_done[x]);
      }
      __syncwarp();
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      const int qs = k % C::QST;
      const int teams = w.ntok > p.R ? 2 : 1;
      ok = wait(&sh.q_full[qs], (k / C::QST) & 1);
      if (ok) ok = wait(&sh.k_full[c0 % C::KSK], (c0 / C::KSK) & 1);
      if (!ok) break;
      tc_fence_after();
      for (int x = 0; x < teams; ++x) issue_s(x, qs, c0);
      if (leader) {
        umma_commit(&sh.k_done[c0 & 7]);
        if (w.n == 1) umma_commit(&sh.q_empty[qs]);
      }
      __syncwarp();
      for (int j = 0; j < w.n && ok; ++j) {
        const int c = c0 + j;
        const bool next = j + 1 < w.n;
        ok = wait(&sh.v_full[c % C::KSV], (c / C::KSV) & 1);
        if (ok) paged_zero_v<C>(w, j, m.v + (c % C::KSV) * C::kTile, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || x >= teams) continue;
          const int g = gs[x] + j;
          ok = wait(&sh.p_half[x], g & 1);
          if (ok && j == 0 && uu[x] >= 1) ok = wait(&sh.o_free[x], (uu[x] - 1) & 1);
          if (!ok) continue;
          tc_fence_after();
          issue_pv(x, c, j == 0, 0);
          ok = wait(&sh.p_ready[x], g & 1);
          if (!ok) continue;
          tc_fence_after();
          issue_pv(x, c, j == 0, 1);
          if (next) {
            if (x == 0) ok = wait(&sh.k_full[(c + 1) % C::KSK], ((c + 1) / C::KSK) & 1);
            if (!ok) continue;
            tc_fence_after();
            issue_s(x, qs, c + 1);                         // in issue order behind PV_X(j)
          }
        }
        if (!ok) break;
        if (leader) {
          umma_commit(&sh.v_done[c & 7]);
          if (next) umma_commit(&sh.k_done[(c + 1) & 7]);
          if (j + 2 == w.n) umma_commit(&sh.q_empty[qs]);
        }
        __syncwarp();
      }
      c0 += w.n;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x < teams) { gs[x] += w.n; ++uu[x]; }
    }
    if (leader) {
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax teams
    const int x = warp >> 3;                                    // team
    const int grp = (warp >> 2) & 1;                            // keys [64 grp, 64 grp + 64)
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_base = lane_base + (x ? C::kS1 : C::kS0) + grp * 64;
    constexpr int OH = D / 2;
    const uint32_t o_base = lane_base + (x ? C::kO1 : C::kO0) + grp * OH;
    const float c = p.cs;
    const uint64_t c2 = f2pack(c, c);
    const int it = row / p.G + x * p.R, h = row % p.G;          // token of the item, head of the group
    int gs = 0, uu = 0;
    int xs = 0;                 // steps in which this quadrant had rows
    bool ok = true;
    auto mask16 = [&](uint32_t (&r)[16], int col0, int lo, int lim) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (col0 + k < lo || col0 + k > lim) r[k] = 0xff800000u;
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      if (x == 1 && w.ntok <= p.R) continue;
      const bool valid = it < w.ntok && row < p.G * p.R;
      const bool active = __any_sync(0xffffffffu, valid);       // a warp without rows only keeps step
      const int pos = w.pos0 + it;
      const int lastk = p.causal ? min(w.len - 1, pos) : w.len - 1;
      const int firstk = p.wl >= 0 ? pos - p.wl : 0;
      float m_used = -INFINITY;
      uint64_t lsum = f2pack(0.f, 0.f);
      for (int j = 0; j < w.n && ok; ++j) {
        const int g = gs + j;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.s_full[x], g & 1));
        if (!ok) break;
        if (!active) {
          if (lane == 0) { mbar_arrive(&sh.p_half[x]); mbar_arrive(&sh.p_ready[x]); }
          __syncwarp();
          continue;
        }
        const int xp = xs & 1;
        tc_fence_after();
        const int kbase = (w.j0 + j) * 128 + grp * 64;
        const int lo = firstk - kbase, lim = lastk - kbase;     // visible columns [lo, lim]
        const bool msk = __any_sync(0xffffffffu, valid && (lo > 0 || lim < 63));
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        {
          uint32_t r0[16], r1[16], r2[16], r3[16];
          tmem_ld16(s_base, r0);
          tmem_ld16(s_base + 16, r1);
          tmem_ld16(s_base + 32, r2);
          tmem_ld16(s_base + 48, r3);
          tmem_wait_ld();
          reg_fence(r0);
          reg_fence(r1);
          reg_fence(r2);
          reg_fence(r3);
          if (msk) {
            // Masked columns become -inf here and go back to TMEM, so the exponent pass
            // below reads them already masked.
            mask16(r0, 0, lo, lim);
            mask16(r1, 16, lo, lim);
            mask16(r2, 32, lo, lim);
            mask16(r3, 48, lo, lim);
            tmem_st16(s_base, r0);
            tmem_st16(s_base + 16, r1);
            tmem_st16(s_base + 32, r2);
            tmem_st16(s_base + 48, r3);
            tmem_wait_st();
          }
#pragma unroll
          for (int kk = 0; kk < 16; kk += 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              mx4[e] = max3f_nan(mx4[e], __uint_as_float(r0[kk + e]), __uint_as_float(r0[kk + e + 4]));
              mx4[e] = max3f_nan(mx4[e], __uint_as_float(r1[kk + e]), __uint_as_float(r1[kk + e + 4]));
              mx4[e] = max3f_nan(mx4[e], __uint_as_float(r2[kk + e]), __uint_as_float(r2[kk + e + 4]));
              mx4[e] = max3f_nan(mx4[e], __uint_as_float(r3[kk + e]), __uint_as_float(r3[kk + e + 4]));
            }
          }
        }
        sh.xmax[x][xp][grp][row] = max3f_nan(max3f_nan(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.xbar[x][xp][quad]);
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.xbar[x][xp][quad], (xs >> 1) & 1));
        if (!ok) break;
        ++xs;
        const float mx = max3f_nan(sh.xmax[x][xp][0][row], sh.xmax[x][xp][1][row], -INFINITY);
        const float m_tile = mx == -INFINITY ? -INFINITY : mx * c;
        // A row that sees a NaN or an infinite score is NaN.  It has to say so by its base: the
        // polynomial would turn the one NaN into a small weight, on its columns and no others.
        if (!(m_tile < INFINITY)) m_used = NAN;
        float alpha = 1.f;
        const bool need = valid && m_tile > m_used + kRescaleTau;
        if (need) {
          alpha = (m_used == -INFINITY) ? 0.f : ex2_approx(m_used - m_tile);
          float l0, l1;
          f2unpack(lsum, l0, l1);
          lsum = f2pack(l0 * alpha, l1 * alpha);
          m_used = m_tile;
        }
        // The commit that signalled S_X(j) also covers PV_X(j-1), so O holds every step
        // before j; the wait below is then immediate.
        if (__any_sync(0xffffffffu, need && j > 0)) {
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.pv_done[x], (g - 1) & 1));
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
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t r[16];
          tmem_ld16(s_base + cc * 16, r);
          tmem_wait_ld();
          reg_fence(r);
          uint32_t pk[8];
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t xx = ffma2(f2pack(__uint_as_float(r[2 * kk]), __uint_as_float(r[2 * kk + 1])), c2, nm2);
            float x0, x1, a, b;
            f2unpack(xx, x0, x1);
            if (kk >= 8 - C::kFmaPairs) {
              exp2_fma_pair(x0, x1, a, b);
              // it ends at 2^-127, which is something beside a masked value of 2^127: 0 as below
              a = x0 < -126.f ? 0.f : a;
              b = x1 < -126.f ? 0.f : b;
            } else {
              a = ex2_approx(x0);
              b = ex2_approx(x1);
            }
            lsum = fadd2(lsum, f2pack(a, b));
            pk[kk] = pack_bf16x2(a, b);
          }
          if (cc == 2) {
            // chunks 0 and 1 were stored a chunk ago: half of P is in
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_half[x]);
          }
          tmem_st8(s_base + cc * 8, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[x]);
      }
      if (!ok) break;
      // epilogue: the two groups' sums, the last PV, O / l and the LSE of this piece
      const int glast = gs + w.n - 1;
      if (active) {
        float l0, l1;
        f2unpack(lsum, l0, l1);
        sh.xsum[x][grp][row] = l0 + l1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sbar[x][quad]);
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.sbar[x][quad], uu & 1));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&sh.pv_done[x], glast & 1));
      if (!ok) break;
      if (active) {
        tc_fence_after();
        const float l = sh.xsum[x][0][row] + sh.xsum[x][1][row];
        const bool none = l == 0.f;                             // no key seen
        const float inv_l = none ? 0.f : 1.f / l;
        const bool okrow = valid && in_range(w.tok0 + it, p.T) && in_range(x * p.G * p.R + row, w.slot < 0 ? 256 : p.slot_rows);
        if (w.slot < 0) {
          // 4 lanes exchange 16-byte chunks of their rows, so that a store instruction writes
          // 64 contiguous bytes of each of 8 rows (fwd_pp.cuh)
          const int row4 = quad * 32 + (lane & ~3);
          size_t dst[4];
          bool st[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int i4 = (row4 + t) / p.G, h4 = row4 + t - i4 * p.G, tok = x * p.R + i4;
            st[t] = tok < w.ntok && row4 + t < p.G * p.R && in_range(w.tok0 + tok, p.T);
            dst[t] = (static_cast<size_t>(w.tok0 + tok) * p.Hq + w.g * p.G + h4) * D + grp * OH + (lane & 3) * 8;
          }
#pragma unroll 1
          for (int hh = 0; hh < OH / 32; ++hh) {
            uint32_t o[2][16];
            tmem_ld16(o_base + hh * 32, o[0]);
            tmem_ld16(o_base + hh * 32 + 16, o[1]);
            tmem_wait_ld();
            reg_fence(o[0]);
            reg_fence(o[1]);
            uint32_t ch[4][4];
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) {
              const float a = none ? 0.f : __uint_as_float(o[kk >> 3][2 * (kk & 7)]) * inv_l;
              const float b = none ? 0.f : __uint_as_float(o[kk >> 3][2 * (kk & 7) + 1]) * inv_l;
              ch[kk >> 2][kk & 3] = pack_bf16x2(a, b);
            }
            transpose_row_chunks<4>(ch, lane);
#pragma unroll
            for (int t = 0; t < 4; ++t)
              if (st[t])
                *reinterpret_cast<uint4*>(p.o + dst[t] + hh * 32) = make_uint4(ch[t][0], ch[t][1], ch[t][2], ch[t][3]);
          }
        } else {
#pragma unroll 1
          for (int q4 = 0; q4 < OH / 16; ++q4) {
            uint32_t o[16];
            tmem_ld16(o_base + q4 * 16, o);
            tmem_wait_ld();
            reg_fence(o);
            if (!okrow) continue;
            float4* dst = reinterpret_cast<float4*>(
                p.opart + (static_cast<size_t>(w.slot) * p.slot_rows + x * p.G * p.R + row) * D + grp * OH + q4 * 16);
            float f[16];
#pragma unroll
            for (int kk = 0; kk < 16; ++kk) f[kk] = none ? 0.f : __uint_as_float(o[kk]) * inv_l;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              dst[kk] = make_float4(f[4 * kk], f[4 * kk + 1], f[4 * kk + 2], f[4 * kk + 3]);
          }
        }
        if (okrow && grp == 0) {
          const float lse_s = none ? -INFINITY : (m_used + __log2f(l)) * 0.69314718055994531f;
          if (w.slot < 0) p.lse[static_cast<size_t>(w.tok0 + it) * p.Hq + w.g * p.G + h] = lse_s;
          else p.lpart[static_cast<size_t>(w.slot) * p.slot_rows + x * p.G * p.R + row] = lse_s;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[x]);
      gs += w.n;
      ++uu;
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
