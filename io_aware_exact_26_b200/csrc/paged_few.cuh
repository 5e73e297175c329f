// Paged attention with few query rows per item (decoding: the query heads of a group times
// one token, or a handful of them); see paged.cuh for the method and the sharing of work.
//
// A 128-row query tile would leave most softmax lanes idle here, and its two warps with
// rows would take 1.3 us per key tile, more than a tile's bytes need from HBM at d = 64
// (0.75 us) or with 8-bit keys.  So the products are turned around: keys fill the 128 rows
// of the tensor-core tile and the NQ (16 or 32) query rows its columns,
//     S^T = K Q^T   [128 keys x NQ],      O^T += V^T P^T   [d x NQ],
// and a softmax thread owns a key, with NQ scores of its own: a tile takes 128 threads x
// the rows there really are.  What crosses lanes is the maximum over keys, and softmax
// needs no exact one: the exponent base of a row may be any number as long as O and the
// sum use the same.  A tile's threads vote whether any score passes its row's base by
// 2^kRescaleTau; only then (the first tiles of an item) are the maxima reduced, the base
// raised and O and the sums rescaled.  The sums stay per thread until the item ends.
//
//   warps 0-3   softmax (thread = key of the tile = TMEM lane; in the epilogue = column of O)
//   warp 4      producer (paged_produce)
//   warp 5      MMA issuer: S up to 3 tiles ahead (4 buffers of NQ columns), P double-buffered
//   warps 6-13  widening warps (e4m3 cache)
// P goes through shared memory (K-major, 128B swizzle) as the second operand of O^T; V is
// read column-major as the first.  At d = 64 the 128 rows of O^T hold d in the first 64;
// the others come from the 16 KB behind the V tile and are never read.
#pragma once
#include "paged.cuh"

namespace attn {

template <int D_, bool KV8_, int NQ>
struct FewCfg {
  static constexpr int D = D_;
  static constexpr bool KV8 = KV8_;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kBox = 128 * 128;
  static constexpr int NB = D / 64;                // 64-column boxes of a bf16 tile
  static constexpr int kQBox = NQ * 128;
  static constexpr int kQTile = NB * kQBox;
  static constexpr int kPTile = 2 * kQBox;         // P^T: NQ rows of 128 keys
  static constexpr int QST = (NQ == 32 && D == 128 && !KV8) ? 1 : 2;
  static constexpr int KST = KV8 ? (D == 128 ? 2 : 3) : (D == 128 ? 3 : 6);   // stages of K, and of V
  static constexpr int SA = KST < 3 ? KST : 3;     // tiles that S runs ahead
  static constexpr int kWiden = KV8 ? 8 : 0;
  static constexpr int kThreads = 192 + 32 * kWiden;
  static constexpr int kRawTile = 128 * D;
  static constexpr int kRoom = 232448 - 1024 - 2 * KST * kTile - QST * kQTile - 2 * kPTile - 3072;
  static constexpr int kRawFit = kRoom / (kRawTile + 128);
  static constexpr int RST = KV8 ? (kRawFit < 8 ? kRawFit : 8) : 0;   // as many raw stages as fit: bytes in flight
  static constexpr int kO = 4 * NQ;                // TMEM: S buffers at 0, NQ, 2 NQ, 3 NQ, then O
  static constexpr int kTmemCols = NQ == 16 ? 128 : 256;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = KST * kTile;
  static constexpr int kOffRaw = kOffV + KST * kTile;
  static constexpr int kOffQ = kOffRaw + RST * kRawTile;
  static constexpr int kOffP = kOffQ + QST * kQTile;
  static constexpr int kOffScale = kOffP + 2 * kPTile;
  static constexpr int kOffSh = kOffScale + RST * 128;
  static constexpr int kEnd = kOffSh + 3072;
  static constexpr int kLayout = kEnd > kOffRaw + kBox ? kEnd : kOffRaw + kBox;   // d = 64 reads 16 KB behind V
  static constexpr int kSmem = kLayout + 1024;
  static_assert(kSmem <= 232448, "shared memory layout exceeds 227 KB");
  static_assert(!KV8 || RST >= 3, "too few raw stages");
};

template <int NQ>
struct FewShared : PagedPipe {
  float wmax[4][NQ], wsum[4][NQ];      // per softmax warp
  int vote[2][4];                      // [step parity][warp]
  uint64_t s_full[4];
  uint64_t p_ready[2], pv_done[2];     // [step parity]
  uint64_t vbar[2];                    // [step parity]: the four warps voted
  uint64_t xbar, sbar;                 // the four warps posted their maxima / their sums
  uint64_t o_free;
};

// Reduction over the 32 lanes of NQ values per lane: each halving step exchanges half of
// the values still held, so it takes NQ - 1 (+ 1) shuffles instead of 5 NQ.  Afterwards
// v[0] holds the result of value `few_owner`.
template <int NQ, typename Op>
__device__ __forceinline__ float few_reduce(float (&v)[NQ], int lane, Op op) {
#pragma unroll
  for (int s = 0; s < 5; ++s) {
    const int off = 16 >> s;
    const int half = NQ >> (s + 1);
    if (half >= 1) {
      const bool up = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float send = up ? v[i] : v[i + half];
        const float keep = up ? v[i + half] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
    }
  }
  return v[0];
}
template <int NQ>
__device__ __forceinline__ int few_owner(int lane) {       // NQ = 32: the lane's bits; 16: without the last
  return NQ == 32 ? lane : lane >> 1;
}

template <int NQ>
__device__ __forceinline__ void few_tmem_ld(uint32_t addr, float (&f)[NQ]) {
#pragma unroll
  for (int b = 0; b < NQ / 16; ++b) {
    uint32_t r[16];
    tmem_ld16(addr + b * 16, r);
    tmem_wait_ld();
    reg_fence(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[b * 16 + i] = __uint_as_float(r[i]);
  }
}

template <int D, bool KV8, int NQ>
__global__ void __launch_bounds__(FewCfg<D, KV8, NQ>::kThreads, 1)
    attn_paged_few_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const PagedParams p) {
  using C = FewCfg<D, KV8, NQ>;
  static_assert(sizeof(FewShared<NQ>) <= 3072, "FewShared does not fit its slot");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewShared<NQ>& sh = *reinterpret_cast<FewShared<NQ>*>(smem + C::kOffSh);
  const PagedSmem m = {smem + C::kOffQ, smem + C::kOffK, smem + C::kOffV, smem + C::kOffRaw, smem + C::kOffScale};
  uint8_t* sP = smem + C::kOffP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    paged_pipe_init<C>(sh, 5 + C::kWiden, 6 + C::kWiden);
    for (int i = 0; i < 4; ++i) mbar_init(&sh.s_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.p_ready[i], 4);
      mbar_init(&sh.pv_done[i], 1);
      mbar_init(&sh.vbar[i], 4);
    }
    mbar_init(&sh.xbar, 4);
    mbar_init(&sh.sbar, 4);
    mbar_init(&sh.o_free, 4);
    fence_barrier_init();
  }
  if (warp == 0) { tmem_alloc(&sh.tmem_base, C::kTmemCols); tmem_relinquish(); }
  grid_dependency_wait();
  grid_dependency_launch();
  paged_plan(p, sh.plan, cta);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 4) {
    paged_produce<C>(p, sh, &tmq, &tmk, &tmv, m, cta, lane);
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(128, NQ, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(128, NQ, true, false);
    constexpr uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t q_lo0 = sdesc_lo(smem_u32(m.q), 16);
    const uint32_t k_lo0 = sdesc_lo(smem_u32(m.k), 16);
    const uint32_t v_lo0 = sdesc_lo(smem_u32(m.v), C::kBox);
    const uint32_t p_lo0 = sdesc_lo(smem_u32(sP), 16);
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, pipe_wait(bar, parity));
    };
    int kc = 0, vc = 0, gs = 0, uq = 0;
    bool ok = true;
    // S^T(g) = K(kc) Q^T into buffer g % 4.  Its last reader arrived on p_ready(g - 4),
    // which PV(g - 4), issued before, waited for.
    auto issue_s = [&](int g, int qs, bool last) -> bool {
      const int st = kc % C::KST;
      if (!wait(&sh.k_full[st], (kc / C::KST) & 1)) return false;
      tc_fence_after();
      if (leader) {
        const uint32_t q_lo = q_lo0 + qs * (C::kQTile >> 4);
        const uint32_t k_lo = k_lo0 + st * (C::kTile >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          umma_ss_lo(tmem + (g & 3) * NQ, k_lo + (((k >> 2) * C::kBox + (k & 3) * 32) >> 4),
                     q_lo + (((k >> 2) * C::kQBox + (k & 3) * 32) >> 4), hi, idS, k > 0);
        umma_commit(&sh.s_full[g & 3]);
        umma_commit(&sh.k_empty[st]);
        if (last) umma_commit(&sh.q_empty[qs]);
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
      for (int t = 0; t < C::SA && t < w.n && ok; ++t) ok = issue_s(gs + t, qs, t == w.n - 1);
      for (int j = 0; j < w.n && ok; ++j, ++vc) {
        const int g = gs + j, vst = vc % C::KST;
        ok = wait(&sh.v_full[vst], (vc / C::KST) & 1);
        if (!KV8 && ok) paged_zero_v<C>(w, j, m.v + vst * C::kTile, lane);
        if (ok) ok = wait(&sh.p_ready[g & 1], (g >> 1) & 1);
        if (ok && j == 0 && uq >= 1) ok = wait(&sh.o_free, (uq - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint32_t v_lo = v_lo0 + vst * (C::kTile >> 4);
          const uint32_t p_lo = p_lo0 + (g & 1) * (C::kPTile >> 4);
#pragma unroll
          for (int k2 = 0; k2 < 8; ++k2)
            umma_ss_lo(tmem + C::kO, v_lo + ((k2 * 2048) >> 4), p_lo + (((k2 >> 2) * C::kQBox + (k2 & 3) * 32) >> 4),
                       hi, idO, !(j == 0 && k2 == 0));
          umma_commit(&sh.pv_done[g & 1]);
          umma_commit(&sh.v_empty[vst]);
        }
        __syncwarp();
        if (j + C::SA < w.n) ok = issue_s(g + C::SA, qs, j + C::SA == w.n - 1);
      }
      gs += w.n;
      ++uq;
    }
    if (leader) {
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 6) {
    if constexpr (KV8) paged_widen<C>(sh, m, threadIdx.x - 192, lane);
  } else {
    // ------------------------------------------------------------ softmax warps 0-3
    const int row = warp * 32 + lane;                           // key of the tile, column of O
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const bool has_o = warp * 32 < D;                           // d = 64: warps 0 and 1 hold O
    const float c = p.cs;
    uint8_t* prow = sP + (row >> 6) * C::kQBox + (row & 7) * 2;
    const int chunk = ((row & 63) >> 3) << 4;
    int gs = 0, uq = 0, fs = 0;                                 // steps, pieces, raised bases
    bool ok = true;
    auto all_warps = [&](uint64_t* bar, uint32_t parity) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      return __all_sync(0xffffffffu, pipe_wait(bar, parity));
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      const int nrows = w.ntok * p.G;                           // rows 0 .. nrows - 1 are real
      const int pos_last = w.pos0 + w.ntok - 1;
      // keys [all_lo, all_hi] are visible to every row
      const int all_hi = p.causal ? min(w.len - 1, w.pos0) : w.len - 1;
      const int all_lo = p.wl >= 0 ? pos_last - p.wl : 0;
      float mu[NQ], ls[NQ];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        mu[q] = -INFINITY;
        ls[q] = 0.f;
      }
      for (int j = 0; j < w.n; ++j) {
        const int g = gs + j, par = g & 1;
        ok = __all_sync(0xffffffffu, pipe_wait(&sh.s_full[g & 3], (g >> 2) & 1));
        if (!ok) break;
        tc_fence_after();
        float x[NQ];
        few_tmem_ld<NQ>(lane_base + (g & 3) * NQ, x);
        const int k0 = (w.j0 + j) * 128, key = k0 + row;
        bool up = false;
        if (k0 >= all_lo && k0 + 127 <= all_hi) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            x[q] *= c;
            up |= q < nrows && x[q] > mu[q] + kRescaleTau;
          }
        } else {
          int i = 0, h = 0;                                     // token and head of row q
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const int pos = w.pos0 + i;
            const bool see = key < w.len && (!p.causal || key <= pos) && (p.wl < 0 || key >= pos - p.wl);
            x[q] = see ? x[q] * c : -INFINITY;
            up |= q < nrows && x[q] > mu[q] + kRescaleTau;
            if (++h == p.G) { h = 0; ++i; }
          }
        }
        up = __any_sync(0xffffffffu, up);
        if (lane == 0) sh.vote[par][warp] = up;
        ok = all_warps(&sh.vbar[par], (g >> 1) & 1);
        if (!ok) break;
        const volatile int* votes = sh.vote[par];
        if (votes[0] | votes[1] | votes[2] | votes[3]) {
          float t[NQ];
#pragma unroll
          for (int q = 0; q < NQ; ++q) t[q] = x[q];
          sh.wmax[warp][few_owner<NQ>(lane)] = few_reduce<NQ>(t, lane, [](float a, float b) { return fmaxf(a, b); });
          ok = all_warps(&sh.xbar, fs & 1);
          if (!ok) break;
          ++fs;
          float alpha[NQ];
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const float top = fmaxf(fmaxf(sh.wmax[0][q], sh.wmax[1][q]), fmaxf(sh.wmax[2][q], sh.wmax[3][q]));
            alpha[q] = 1.f;
            if (top > mu[q]) {
              alpha[q] = mu[q] == -INFINITY ? 0.f : ex2_approx(mu[q] - top);
              mu[q] = top;
              ls[q] *= alpha[q];
            }
          }
          if (j > 0 && has_o) {                                 // O holds the steps before this one
            ok = __all_sync(0xffffffffu, pipe_wait(&sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            float o[NQ];
            few_tmem_ld<NQ>(lane_base + C::kO, o);
#pragma unroll
            for (int b = 0; b < NQ / 16; ++b) {
              uint32_t r[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                r[i] = alpha[b * 16 + i] == 0.f ? 0u : __float_as_uint(o[b * 16 + i] * alpha[b * 16 + i]);
              tmem_st16(lane_base + C::kO + b * 16, r);
            }
            tmem_wait_st();
          }
        }
        // P(g) goes where P(g - 2) was: PV(g - 2) has to be done
        if (g >= 2) {
          ok = __all_sync(0xffffffffu, pipe_wait(&sh.pv_done[par], ((g >> 1) - 1) & 1));
          if (!ok) break;
        }
        uint8_t* dst = prow + par * C::kPTile;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (q < nrows) {
            const float e = ex2_approx(x[q] - (mu[q] == -INFINITY ? 0.f : mu[q]));
            ls[q] += e;
            *reinterpret_cast<__nv_bfloat16*>(dst + q * 128 + (chunk ^ ((q & 7) << 4))) = __float2bfloat16_rn(e);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[par]);
      }
      if (!ok) break;
      // epilogue: sums over the keys, the last PV, O / l and the LSE of this piece
      const int glast = gs + w.n - 1;
      {
        float t[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) t[q] = ls[q];
        sh.wsum[warp][few_owner<NQ>(lane)] = few_reduce<NQ>(t, lane, [](float a, float b) { return a + b; });
      }
      ok = all_warps(&sh.sbar, uq & 1);
      if (ok) ok = __all_sync(0xffffffffu, pipe_wait(&sh.pv_done[glast & 1], (glast >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      float o[NQ];
      few_tmem_ld<NQ>(lane_base + C::kO, o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free);
      int i = 0, h = 0;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q < nrows) {
          const float l = (sh.wsum[0][q] + sh.wsum[1][q]) + (sh.wsum[2][q] + sh.wsum[3][q]);
          const bool none = l == 0.f;                           // no key seen
          const float val = none ? 0.f : o[q] * (1.f / l);
          const size_t orow = static_cast<size_t>(w.tok0 + i) * p.Hq + w.g * p.G + h;
          const bool store = in_range(w.tok0 + i, p.T) && in_range(q, w.slot < 0 ? NQ : p.slot_rows);
          const size_t prow_ = static_cast<size_t>(w.slot < 0 ? 0 : w.slot) * p.slot_rows + q;
          if (store && has_o) {
            if (w.slot < 0) p.o[orow * D + row] = __float2bfloat16_rn(val);
            else p.opart[prow_ * D + row] = val;
          }
          if (store && row == q) {
            const float lse = none ? -INFINITY : (mu[q] + __log2f(l)) * 0.69314718055994531f;
            if (w.slot < 0) p.lse[orow] = lse;
            else p.lpart[prow_] = lse;
          }
          if (++h == p.G) { h = 0; ++i; }
        }
      }
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
