// Paged attention with few query rows per item (decoding: the query heads of a group times
// one token, or a handful of them); see paged.cuh for the method and the sharing of work.
//
// A 128-row query tile would leave most softmax lanes idle here, and its two warps with
// rows would take 1.3 us per key tile, more than a tile's bytes need from HBM at d = 64
// (0.75 us) or with 8-bit keys.  So the products are turned around: keys fill the 128 rows
// of the tensor-core tile and the query rows its NQ columns,
//     S^T = K Q^T   [128 keys x NQ],      O^T += V^T P^T   [d x NQ],
// and a softmax thread owns a key, with the scores of NR rows: the kernel is built for NR = 4,
// 8 and 16 rows per item (NQ = 16 is the least the tensor cores take), because a thread's
// work, registers and code follow NR (one build for all: 410 us, 64 x 8K over e4m3, pages
// of 16; a build per row count: 395).  From there on the 128-row kernel is faster.  What crosses lanes is the maximum over keys, and softmax
// needs no exact one: the exponent base of a row may be any number as long as O and the
// sum use the same.  A tile's threads vote whether any score passes its row's base by
// 2^kRescaleTau; only then (the first tiles of an item) are the maxima reduced, the base
// raised and O and the sums rescaled.  The sums stay per thread until the item ends.
//
// A tile's chain (scores, vote, exponentials, P, fence) is latency, not work: two groups of
// softmax warps take alternate tiles, each with its own bases, sums and O, joined like two
// shares of the keys when the item ends.
//
//   warps 0-3, 4-7  softmax groups 0, 1: group g % 2 takes step g (thread = key of the tile =
//                   TMEM lane); the epilogue is group 0's (thread = column of O)
//   warps 8, 9      producers of K (and Q) and of V
//   warp 10         MMA issuer: S runs SA steps ahead of P V, in 4 buffers of NQ columns.  (A
//                   warp for each product measured 17% slower with an e4m3 cache.)
//   warps 11-       widening warps (e4m3 cache)
// P goes through shared memory (K-major, 128B swizzle) as the second operand of O^T; V is
// read column-major as the first.  At d = 64 the 128 rows of O^T hold d in the first 64;
// the others come from the 16 KB behind the V tile and are never read.
//
// e4m3 cache.  K goes to the tensor cores as it lies (no widening: half of that work and of
// its shared-memory traffic), so Q has to be 8-bit too, without losing anything.  A bf16 value
// has 8 significant bits, e4m3 has 4, and e4m3 ends at 2^-9 where a query row may have any
// range, so q 2^-e (e from the row's largest magnitude, at most 448 2^e) goes as four parts:
//     q 2^-e = p0 + 2^-4 (p1 + 2^-18 (p2 + 2^-4 p3)),
// each the nearest e4m3 of what the parts before it left.  p0 takes 4 bits, p1 the 4 below them:
// exact down to 2^-6, from where what is left (at most 2^-10 in units of p1) starts again at
// p2's 256.  So a value is exact down to 2^-35 of its row's largest magnitude and off by at
// most 2^-43 of it below.  (Two parts, p1 unscaled, lose bits from 2^-10 of it on.)  The parts are
// columns of the same product (the MMA thread, which issues 8 small instructions per P V,
// bounds an e4m3 tile, so S should take few), and the softmax thread adds them up, the last two
// (at d = 64) only where a row of the piece has a value that the first two do not hold: they
// hold all down to 2^-13 of the largest magnitude.  The scales 2^e of a query row and of its key
// multiply the sum.  V is widened to bf16, as its products with P need.
#pragma once
#include "paged.cuh"

namespace attn {

template <int D_, bool KV8_, int NR_>
struct FewCfg {
  static constexpr int D = D_, NR = NR_;
  static constexpr int NQ = 16;                    // columns of S^T and O^T
  static_assert(NR == 4 || NR == 8 || NR == 16, "rows per item");
  static constexpr bool KV8 = KV8_, K8 = KV8_;
  static constexpr int kTile = 128 * D * 2;        // bf16 tile
  static constexpr int kTeams = 1;
  static constexpr int kBox = 128 * 128;
  static constexpr int NB = D / 64;                // 64-column boxes of a bf16 tile
  static constexpr int kKTile = K8 ? 128 * 128 : kTile;
  static constexpr int kQBox = (K8 ? (NR < 8 ? 8 : NR) : NQ) * 128;    // K8: read by the split only
  static constexpr int kQTile = NB * kQBox;
  static constexpr int kPBox = NQ * 128;
  static constexpr int kPTile = 2 * kPBox;         // P^T: NQ rows of 128 keys
  static constexpr int QST = 2;
  static constexpr int NS = K8 ? 4 * NR : NQ;      // columns of S^T; K8: part i of row r in column i NR + r
  static constexpr int kQ8 = K8 ? NS * 128 : 0;    // the parts, 128-byte rows
  // Columns of the last two parts are read only where a row needs them.  64 x 4K, pages of 64, one
  // head: 170 -> 150 us at d = 64; else the branch costs more than the columns (d = 128: 183 ->
  // 187; 8 rows of d = 64, 64 x 8K: 182 -> 185; 12 of d = 128, 16 x 8K: 86 -> 93).
  static constexpr bool kSkipParts = K8 && NR == 4 && D == 64;
  static constexpr int KSK = K8 ? 4 : D == 128 ? 3 : 6;
  static constexpr int KSV = KV8 ? (D == 128 ? 2 : 3) : KSK;
  // S(g) completes behind PV(g - SA), so P(g) may take the buffer of P(g - NP) for NP >= SA
  static constexpr int SA = 3;
  static constexpr int NP = 4;
  // K8: the scale bytes of the last 8 K tiles are kept: a tile is filled in KSK tiles ahead of
  // S, S runs SA ahead of the softmax
  static_assert(SA <= KSK && SA <= KSV + 1 && NP >= SA && KSK <= 8 && KSV <= 8 && (!K8 || KSK + SA + 1 <= 8), "stages");
  static constexpr int kWiden = KV8 ? 8 : 0;
  static constexpr int kThreads = 352 + 32 * kWiden;
  static constexpr int kRawTile = 128 * D;
  static constexpr int kShared = 4096;
  static constexpr int kRoom = 232448 - 1024 - KSK * kKTile - KSV * kTile - QST * (kQTile + kQ8) - NP * kPTile -
                               1024 - kShared;
  static constexpr int kRawFit = kRoom / (kRawTile + 128);
  static constexpr int RST = KV8 ? (kRawFit < 8 ? kRawFit : 8) : 0;   // as many raw stages as fit: bytes in flight
  static constexpr int kRawMod = KV8 ? RST : 1;
  static constexpr int kO = 4 * NS;                // TMEM: S buffers at 0, NS, 2 NS, 3 NS, then O of each group
  static constexpr int kTmemUsed = kO + 2 * NQ;
  static constexpr int kTmemCols = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = KSK * kKTile;
  static constexpr int kOffRaw = kOffV + KSV * kTile;
  static constexpr int kOffQ = kOffRaw + RST * kRawTile;
  static constexpr int kOffQ8 = kOffQ + QST * kQTile;
  static constexpr int kOffP = kOffQ8 + QST * kQ8;
  static constexpr int kOffScale = kOffP + NP * kPTile;
  static constexpr int kOffKScale = kOffScale + RST * 128;
  static constexpr int kOffSh = kOffKScale + 1024;
  static constexpr int kEnd = kOffSh + kShared;
  static constexpr int kLayout = kEnd > kOffRaw + kBox ? kEnd : kOffRaw + kBox;   // d = 64 reads 16 KB behind V
  static constexpr int kSmem = kLayout + 1024;
  static_assert(kSmem <= 232448, "shared memory layout exceeds 227 KB");
  static_assert(!KV8 || RST >= 3, "too few raw stages");
};

template <int NR>
struct FewShared : PagedPipe {
  float wmax[2][4][NR];                // [group][warp]
  float wsum[2][2][4][NR];             // [piece parity][group][warp]
  float base[2][2][NR];                // [piece parity][group] exponent bases
  alignas(16) float cq[4][NR];                    // K8: 2^e of the query rows, by piece % 4
  alignas(8) uint8_t wide[4][8];                  // K8: whether the rows of a widening warp need four parts, likewise
  int vote[2][2][4];                   // [group][parity of its steps][warp]
  // By step % 4: S runs up to 3 steps ahead of P V, so a group may finish two of its steps
  // before the MMA warp looks at the first (a parity wait tells two successive phases apart).
  uint64_t p_ready[4];
  uint64_t vbar[2][2];                 // [group][parity of its steps]: its four warps voted
  uint64_t xbar[2];                    // [group]: its four warps posted their maxima
  uint64_t done[2];                    // [piece parity]: all eight warps posted sums and bases
  uint64_t o_free;
};

// Exponent base of a row that has seen no key: below every score, and 2^(it - score) is 0.
constexpr float kNoBase = -3.0e38f;

// Reduction over the 32 lanes of NR values per lane: each halving step exchanges half of
// the values still held, so it takes fewer than NR + 5 shuffles instead of 5 NR.
// Afterwards the returned value is that of row few_owner(lane).
template <int NR, typename Op>
__device__ __forceinline__ float few_reduce(float (&v)[NR], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < 5; ++s) {
    const int off = 16 >> s;
    const int half = NR >> (s + 1);
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
template <int NR>
__device__ __forceinline__ int few_owner(int lane) {       // the lane's upper log2(NR) bits
  return lane / (32 / NR);
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// NR columns of this thread's TMEM lane.
template <int NR>
__device__ __forceinline__ void few_tmem_ld(uint32_t addr, float (&f)[NR]) {
  uint32_t r[NR];
  if constexpr (NR == 4) tmem_ld4(addr, r);
  else if constexpr (NR == 8) tmem_ld8(addr, r);
  else tmem_ld16(addr, r);
  tmem_wait_ld();
  reg_fence(r);
#pragma unroll
  for (int i = 0; i < NR; ++i) f[i] = __uint_as_float(r[i]);
}
template <int NR>
__device__ __forceinline__ void few_tmem_st(uint32_t addr, const float (&f)[NR]) {
  uint32_t r[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) r[i] = __float_as_uint(f[i]);
  if constexpr (NR == 4) tmem_st4(addr, r);
  else if constexpr (NR == 8) tmem_st8(addr, r);
  else tmem_st16(addr, r);
}

// Scale between part i of Q and part i + 1 (see the head of this file).
__host__ __device__ constexpr float few_part_step(int i) { return i == 1 ? 262144.f : 16.f; }

// Scores of this thread's key from the first PARTS parts of Q, smallest first: up to 16 columns per
// trip to TMEM.
template <int NR, int PARTS>
__device__ __forceinline__ void few_scores(uint32_t addr, float (&x)[NR]) {
  constexpr int PER = PARTS * NR <= 16 ? PARTS : 16 / NR;      // parts per trip
#pragma unroll
  for (int part = PARTS - PER; part >= 0; part -= PER) {
    float t[PER * NR];
    few_tmem_ld<PER * NR>(addr + part * NR, t);
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
#pragma unroll
      for (int q = 0; q < NR; ++q)
        x[q] = part + i == PARTS - 1 ? t[i * NR + q] : fmaf(x[q], 1.f / few_part_step(part + i), t[i * NR + q]);
  }
}

// 2^(byte - 127), also for byte 0 (subnormal).
__device__ __forceinline__ float e8m0_value(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// Q of a piece in four e4m3 parts (see the head of this file), row scales to cq, and to wide whether
// the first two leave anything.
template <class C>
__device__ __forceinline__ void few_split_q(const uint8_t* q, uint8_t* q8, float* cq, uint8_t* wide, int wt) {
  constexpr int CPR = C::D / 8;                      // 8-value chunks per row, one per lane
  static_assert(C::kWiden == 8, "a byte of `wide` per warp");
  bool more = false;
  for (int x = wt; x < C::NR * CPR; x += 32 * C::kWiden) {
    const int r = x / CPR, c = x % CPR;
    const uint4 raw = *reinterpret_cast<const uint4*>(q + (c >> 3) * C::kQBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    float f[8];
    Vec16<__nv_bfloat16>::load(raw, f);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(f[i]);
      amax = fmaxf(amax, a < INFINITY ? a : 0.f);
    }
#pragma unroll
    for (int m = CPR / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
    const int e = e4m3_exponent(amax);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] *= inv;
      if (!(fabsf(f[i]) < INFINITY)) f[i] = NAN;     // an infinite query value gives no finite score
    }
#pragma unroll
    for (int part = 0; part < 4; ++part) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t two = pack_e4m3x2(f[i], f[i + 1]);
        const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&back));
        f[i] = (f[i] - g.x) * few_part_step(part);
        f[i + 1] = (f[i + 1] - g.y) * few_part_step(part);
        w[i >> 1] = two;
        if (part == 1) more |= f[i] != 0.f || f[i + 1] != 0.f;
      }
      const int pr = part * C::NR + r;
      *reinterpret_cast<uint2*>(q8 + pr * 128 + (((c >> 1) ^ (pr & 7)) << 4) + (c & 1) * 8) =
          make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
    if (c == 0) cq[r] = e8m0_value(static_cast<uint32_t>(e + 127));
  }
  if constexpr (C::kSkipParts) {
    more = __any_sync(0xffffffffu, more);
    if ((wt & 31) == 0) wide[wt >> 5] = more;
  }
}

template <int D, bool KV8, int NR>
__global__ void __launch_bounds__(FewCfg<D, KV8, NR>::kThreads, 1)
    attn_paged_few_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const PagedParams p) {
  using C = FewCfg<D, KV8, NR>;
  constexpr int NQ = C::NQ;
  static_assert(sizeof(FewShared<NR>) <= C::kShared, "FewShared does not fit its slot");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  FewShared<NR>& sh = *reinterpret_cast<FewShared<NR>*>(smem + C::kOffSh);
  const PagedSmem m = {smem + C::kOffQ,   smem + C::kOffK,     smem + C::kOffV,
                       smem + C::kOffRaw, smem + C::kOffScale, smem + C::kOffKScale};
  uint8_t* sQ8 = smem + C::kOffQ8;
  uint8_t* sP = smem + C::kOffP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    paged_pipe_init<C>(sh, 10 + C::kWiden, 11 + C::kWiden);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.p_ready[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.vbar[i][0], 4);
      mbar_init(&sh.vbar[i][1], 4);
      mbar_init(&sh.xbar[i], 4);
      mbar_init(&sh.done[i], 8);
    }
    mbar_init(&sh.o_free, 4);
    fence_barrier_init();
  }
  if (warp == 0) { tmem_alloc(&sh.tmem_base, C::kTmemCols); tmem_relinquish(); }
  grid_dependency_wait();
  grid_dependency_launch();
  paged_plan(p, sh.plan, cta, warp == 8, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;

  if (warp == 8) {
    paged_produce_k<C>(p, sh, &tmq, &tmk, m, cta, lane);
  } else if (warp == 9) {
    paged_produce_v<C>(p, sh, &tmv, m, lane);
  } else if (warp == 10) {
    // ------------------------------------------------------------ MMA issuer (one thread)
    const bool leader = elect_one();
    constexpr uint32_t idS = KV8 ? idesc_e4m3_f32(128, C::NS, false, false) : idesc_bf16_f32(128, NQ, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(128, NQ, true, false);
    constexpr uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t q_lo0 = sdesc_lo(smem_u32(KV8 ? sQ8 : m.q), 16);
    const uint32_t k_lo0 = sdesc_lo(smem_u32(m.k), 16);
    const uint32_t v_lo0 = sdesc_lo(smem_u32(m.v), C::kBox);
    const uint32_t p_lo0 = sdesc_lo(smem_u32(sP), 16);
    int gs = 0;                                     // steps before the piece
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      if (leader) {
        const int qs = k % C::QST;
        ok = mbar_wait(KV8 ? &sh.q8_full[qs] : &sh.q_full[qs], (k / C::QST) & 1);
        const uint32_t q_lo = q_lo0 + qs * ((KV8 ? C::kQ8 : C::kQTile) >> 4);
        // S^T(g) = K Q^T into buffer g % 4.  Its last reader arrived on p_ready for step g - 4,
        // which PV(g - 4), issued before, waited for.
        auto issue_s = [&](int g) {
          const int st = g % C::KSK;
          if (!mbar_wait(&sh.k_full[st], (g / C::KSK) & 1)) return false;
          tc_fence_after();
          const uint32_t k_lo = k_lo0 + st * (C::kKTile >> 4), d = tmem + (g & 3) * C::NS;
          if constexpr (KV8) {
#pragma unroll
            for (int k2 = 0; k2 < D / 32; ++k2)
              umma_ss_f8_lo(d, k_lo + ((k2 * 32) >> 4), q_lo + ((k2 * 32) >> 4), hi, idS, k2 > 0);
          } else {
#pragma unroll
            for (int k2 = 0; k2 < D / 16; ++k2)
              umma_ss_lo(d, k_lo + (((k2 >> 2) * C::kBox + (k2 & 3) * 32) >> 4),
                         q_lo + (((k2 >> 2) * C::kQBox + (k2 & 3) * 32) >> 4), hi, idS, k2 > 0);
          }
          umma_commit(&sh.k_done[g & 7]);
          if (g == gs + w.n - 1) umma_commit(&sh.q_empty[qs]);
          return true;
        };
        for (int t = 0; t < C::SA && t < w.n && ok; ++t) ok = issue_s(gs + t);
        if (ok && k >= 1) ok = mbar_wait(&sh.o_free, (k - 1) & 1);
        for (int j = 0; j < w.n && ok; ++j) {
          // O^T of group g % 2 (+)= V^T P^T(g); the group's first step of a piece starts it
          const int g = gs + j, st = g % C::KSV;
          ok = mbar_wait(&sh.v_full[st], (g / C::KSV) & 1);
          if (ok) ok = mbar_wait(&sh.p_ready[g & 3], (g >> 2) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v_lo = v_lo0 + st * (C::kTile >> 4), p_lo = p_lo0 + (g % C::NP) * (C::kPTile >> 4);
          const uint32_t d = tmem + C::kO + (g & 1) * NQ;
#pragma unroll
          for (int k2 = 0; k2 < 8; ++k2)
            umma_ss_lo(d, v_lo + ((k2 * 2048) >> 4), p_lo + (((k2 >> 2) * C::kPBox + (k2 & 3) * 32) >> 4), hi, idO,
                       !(j < 2 && k2 == 0));
          umma_commit(&sh.v_done[g & 7]);
          if (j + C::SA < w.n) ok = issue_s(g + C::SA);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      gs += w.n;
    }
    if (leader) {
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 11) {
    if constexpr (KV8) {
      const int wt = threadIdx.x - 352;
      paged_widen<C>(sh, m, wt, lane, [&](int k, int qs) {
        few_split_q<C>(m.q + qs * C::kQTile, sQ8 + qs * C::kQ8, sh.cq[k & 3], sh.wide[k & 3], wt);
      });
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    const int x2 = warp >> 2, wq = warp & 3;                    // group, warp of the group
    const int row = wq * 32 + lane;                             // key of the tile, column of O
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const bool has_o = wq * 32 < D;                             // d = 64: the first two warps hold O
    uint8_t* prow = sP + (row >> 6) * C::kPBox + (row & 7) * 2;
    const int chunk = ((row & 63) >> 3) << 4;
    int gs = 0, uq = 0, fs = 0;                                 // steps, pieces, raised bases
    bool ok = true;
    auto group_sync = [&](uint64_t* bar, uint32_t parity) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      return __all_sync(0xffffffffu, mbar_wait(bar, parity));
    };
    for (int k = 0; ok; ++k) {
      const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
      if (w.n == 0) break;
      const int nrows = w.ntok * p.G;                           // rows 0 .. nrows - 1 are real
      // keys [all_lo, all_hi] are visible to every row
      const int all_hi = p.causal ? min(w.len - 1, w.pos0) : w.len - 1;
      const int all_lo = p.wl >= 0 ? w.pos0 + w.ntok - 1 - p.wl : 0;
      float mu[NR], ls[NR];                                     // exponent bases, sums
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        mu[q] = q < nrows ? kNoBase : INFINITY;                 // rows that are not there never vote
        ls[q] = 0.f;
      }
      const int g_end = gs + w.n;
      [[maybe_unused]] bool wide = !C::kSkipParts;              // K8: Q takes four parts
      for (int g = gs + ((gs ^ x2) & 1); g < g_end; g += 2) {
        const int par = (g >> 1) & 1;                           // parity of the group's steps
        ok = __all_sync(0xffffffffu, tile_done_wait(sh.k_done, g));
        if (!ok) break;
        tc_fence_after();
        float x[NR];
        // Scores in the exponent's units.  They are masked afterwards: no factor meets a -inf.
        if constexpr (!KV8) {
          few_tmem_ld<NR>(lane_base + (g & 3) * C::NS, x);
#pragma unroll
          for (int q = 0; q < NR; ++q) x[q] *= p.cs;
        } else {
          if (C::kSkipParts && g < gs + 2) {                    // the group's first step of the piece
            const uint2 f = *reinterpret_cast<const uint2*>(sh.wide[uq & 3]);
            wide = (f.x | f.y) != 0;
          }
          if (wide) few_scores<NR, 4>(lane_base + (g & 3) * C::NS, x);
          else few_scores<NR, 2>(lane_base + (g & 3) * C::NS, x);
          // The scales of key and row are multiplied first: a large one and a small one cancel
          // before either meets the sum, which alone can pass fp32 with the row's.
          const float c = p.cs * e8m0_value(m.kscale[(g & 7) * 128 + row]);
#pragma unroll
          for (int q = 0; q < NR; q += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sh.cq[uq & 3][q]);
            x[q] *= f.x * c; x[q + 1] *= f.y * c; x[q + 2] *= f.z * c; x[q + 3] *= f.w * c;
          }
        }
        const int k0 = (w.j0 + g - gs) * 128, key = k0 + row;
        bool up = false;
        if (!(k0 >= all_lo && k0 + 127 <= all_hi)) {
          int i = 0, h = 0;                                     // token and head of row q
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            const int pos = w.pos0 + i;
            const bool see = key < w.len && (!p.causal || key <= pos) && (p.wl < 0 || key >= pos - p.wl);
            if (!see) x[q] = -INFINITY;
            if (++h == p.G) { h = 0; ++i; }
          }
        }
#pragma unroll
        for (int q = 0; q < NR; ++q) up |= x[q] > mu[q] + kRescaleTau;
        up = __any_sync(0xffffffffu, up);
        if (lane == 0) sh.vote[x2][par][wq] = up;
        ok = group_sync(&sh.vbar[x2][par], (g >> 2) & 1);
        if (!ok) break;
        const volatile int* votes = sh.vote[x2][par];
        if (votes[0] | votes[1] | votes[2] | votes[3]) {
          {
            float t[NR];
#pragma unroll
            for (int q = 0; q < NR; ++q) t[q] = x[q];
            sh.wmax[x2][wq][few_owner<NR>(lane)] = few_reduce<NR>(t, [](float a, float b) { return fmaxf(a, b); });
          }
          ok = group_sync(&sh.xbar[x2], fs & 1);
          if (!ok) break;
          ++fs;
          float alpha[NR];
#pragma unroll
          for (int q = 0; q < NR; ++q) {
            const float (&wm)[4][NR] = sh.wmax[x2];
            const float top = fmaxf(fmaxf(wm[0][q], wm[1][q]), fmaxf(wm[2][q], wm[3][q]));
            alpha[q] = 1.f;
            if (top > mu[q]) {
              alpha[q] = ex2_approx(mu[q] - top);
              mu[q] = top;
              ls[q] *= alpha[q];
            }
          }
          if (g - 2 >= gs && has_o) {                           // O holds the group's steps before this one
            ok = __all_sync(0xffffffffu, tile_done_wait(sh.v_done, g - 2));
            if (!ok) break;
            tc_fence_after();
            float o[NR];
            few_tmem_ld<NR>(lane_base + C::kO + x2 * NQ, o);
#pragma unroll
            for (int q = 0; q < NR; ++q) o[q] = alpha[q] == 0.f ? 0.f : o[q] * alpha[q];
            few_tmem_st<NR>(lane_base + C::kO + x2 * NQ, o);
            tmem_wait_st();
          }
        }
        if (!KV8 && (k0 < w.kmin || k0 + 128 > w.len)) {
          // This thread's row of V, if its key is one that nobody sees (behind the sequence,
          // before the window, in a page that was not loaded), becomes zeros: its P is 0, and 0
          // times whatever lies there has to be 0.  (e4m3: the widening warps do it.)
          const int vst = g % C::KSV;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.v_full[vst], (g / C::KSV) & 1));
          if (!ok) break;
          if (key < w.kmin || key >= w.len) {
            uint4* v = reinterpret_cast<uint4*>(m.v + vst * C::kTile + row * 128);
#pragma unroll
            for (int b = 0; b < C::NB; ++b)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[b * (C::kBox / 16) + i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        // P(g) takes the buffer of P(g - NP): PV(g - NP) is done, S(g) came behind it
        uint8_t* dst = prow + (g % C::NP) * C::kPTile;
#pragma unroll
        for (int q = 0; q < NR; ++q) {
          const float e = ex2_approx(x[q] - mu[q]);
          ls[q] += e;
          *reinterpret_cast<__nv_bfloat16*>(dst + q * 128 + (chunk ^ ((q & 7) << 4))) = __float2bfloat16_rn(e);
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_ready[g & 3]);
      }
      if (!ok) break;
      // the group's sums over the keys and its bases.  Group 1 posts them only when group 0 has
      // read O of the piece before: a group without a step in a piece would else run ahead of
      // the buffers (and of the barrier) here.
      const int pp = uq & 1;
      if (x2 == 1 && uq >= 1) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.o_free, (uq - 1) & 1));
        if (!ok) break;
      }
      if (wq == 0 && lane == 0) {
#pragma unroll
        for (int q = 0; q < NR; ++q) sh.base[pp][x2][q] = mu[q];
      }
      sh.wsum[pp][x2][wq][few_owner<NR>(lane)] = few_reduce<NR>(ls, [](float a, float b) { return a + b; });
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.done[pp]);
      gs = g_end;
      if (x2 == 1) { ++uq; continue; }
      // epilogue (group 0): both groups' sums, the last PV, then O / l and the LSE of the piece
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.done[pp], (uq >> 1) & 1));
      const int glast = g_end - 1;
      if (ok) ok = __all_sync(0xffffffffu, tile_done_wait(sh.v_done, glast));
      if (!ok) break;
      tc_fence_after();
      float o0[NR], o1[NR];
      if (has_o) {
        few_tmem_ld<NR>(lane_base + C::kO, o0);
        few_tmem_ld<NR>(lane_base + C::kO + NQ, o1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free);
      int i = 0, h = 0;
#pragma unroll
      for (int q = 0; q < NR; ++q) {
        if (q >= nrows) break;
        const float m0 = sh.base[pp][0][q], m1 = sh.base[pp][1][q], top = fmaxf(m0, m1);
        const float f0 = ex2_approx(m0 - top), f1 = ex2_approx(m1 - top);
        const float (&s0)[4][NR] = sh.wsum[pp][0], (&s1)[4][NR] = sh.wsum[pp][1];
        const float l0 = (s0[0][q] + s0[1][q]) + (s0[2][q] + s0[3][q]);
        const float l1 = (s1[0][q] + s1[1][q]) + (s1[2][q] + s1[3][q]);
        const float l = l0 * f0 + l1 * f1;
        const bool none = l == 0.f;                             // no key seen
        // a group that saw nothing has l = 0, and anything in its columns of O
        const float val = none ? 0.f : ((l0 == 0.f ? 0.f : o0[q] * f0) + (l1 == 0.f ? 0.f : o1[q] * f1)) * (1.f / l);
        const size_t orow = static_cast<size_t>(w.tok0 + i) * p.Hq + w.g * p.G + h;
        const bool store = in_range(w.tok0 + i, p.T) && in_range(q, w.slot < 0 ? NR : p.slot_rows);
        const size_t part = static_cast<size_t>(w.slot < 0 ? 0 : w.slot) * p.slot_rows + q;
        if (store && has_o) {
          if (w.slot < 0) p.o[orow * D + row] = __float2bfloat16_rn(val);
          else p.opart[part * D + row] = val;
        }
        if (store && row == q) {
          const float lse = none ? -INFINITY : (top + __log2f(l)) * 0.69314718055994531f;
          if (w.slot < 0) p.lse[orow] = lse;
          else p.lpart[part] = lse;
        }
        if (++h == p.G) { h = 0; ++i; }
      }
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
