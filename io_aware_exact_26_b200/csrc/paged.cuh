// Attention of new tokens over a paged K/V cache for sm_100a.
//
// Method (page "attn-efficient", online-softmax section; page "attention 的显存线性化",
// reading list: FlashDecoding): the tiled online softmax of the forward, with K and V
// tiles gathered from pages, and the keys of a query tile shared out over several CTAs
// where there are few tiles.  With m = max_s LSE_s and w_s = exp(LSE_s - m) over the
// shares s of a row: O = sum_s w_s O_s / sum_s w_s, LSE = m + ln sum_s w_s.
//
// Work.  An item is (sequence b, KV head g, block of R tokens): the G query heads of the
// group times R = 128 / G tokens fill the 128 rows of a tensor-core tile (row = i * G + h),
// so K and V of a group are read once for all its heads.  Its work is the number of
// 128-key tiles that any of its rows sees.  All items' tiles, in the order (b, g, block),
// form one line of W tiles, and CTA c takes the tiles [W c / C, W (c+1) / C): every SM
// streams the same number of tiles whatever the lengths are.  Each CTA finds its place
// from cu_q and kv_len alone (no plan from the host, no counter), so a captured launch
// follows the lengths.  A CTA's share cuts at most two items; a cut item's parts go to
// the workspace (two slots per CTA, independent of lengths) and the merge kernel joins
// them in key order, so results do not depend on timing.  Items of few tiles are not cut but
// go to the CTA in whose share they begin, where writing and merging parts of many rows
// would cost more than the imbalance (p.whole).
#pragma once
#include "cache.cuh"
#include "fwd.cuh"

namespace attn {

struct PagedParams {
  CacheView c;
  __nv_bfloat16* o;           // [T][Hq][D]
  float* lse;                 // [T][Hq]
  const int* cu_q;
  const int* kv_len;
  const int* table;
  int B, T, max_pages;
  int Hq, Hkv, G, R;          // R tokens per tile, G * R <= 128
  int RI;                     // tokens per item: R * teams
  int causal, wl;             // wl < 0: no window
  int whole;                  // items of up to this many tiles are not cut (see PagedPlan)
  float cs;                   // scale * log2(e), floored (folded_scale)
  int ctas;                   // CTAs of the launch
  int slot_rows;              // rows of a workspace slot
  float* opart;               // [2 * ctas][slot_rows][D], normalised by the part's own sum
  float* lpart;               // [2 * ctas][slot_rows], natural log; -inf: no key seen
  struct PagedCut* cuts;      // [ctas]
};

// A cut item, written by the CTA that holds its first part.
struct PagedCut {
  int tok0, ntok, g;          // rows: tokens tok0 .. tok0 + ntok - 1 of KV head g; ntok = 0: nothing cut here
  int parts;                  // part 0 in slot 2c + 1, part i in slot 2 (c + i)
};

// One piece of work of a CTA, posted to its consumer warps.
struct PagedSeg {
  int b, g;
  int tok0, ntok;             // packed row of the first token, tokens of the item
  int pos0;                   // position of the first token
  int len;                    // keys of the sequence
  int kmin;                   // first key that a row of the item sees
  int j0, n;                  // key tiles [j0, j0 + n); n = 0 ends the sequence of pieces
  int slot;                   // -1: write o and lse; else the workspace slot
};

// sum of floor(max(0, a + r i) / 128) over 0 <= i < x, for r >= 1, in a few steps: the
// part of a and r that 128 divides is summed in closed form, the rest counts the lattice
// points under a line, with the axes exchanged until nothing is left.
__device__ __forceinline__ long long stair_sum(long long a, long long r, long long x) {
  if (a < 0) {
    const long long skip = (-a + r - 1) / r;
    if (skip >= x) return 0;
    a += r * skip;
    x -= skip;
  }
  long long m = 128, sum = 0;
  while (true) {
    if (r >= m) { sum += x * (x - 1) / 2 * (r / m); r %= m; }
    if (a >= m) { sum += x * (a / m); a %= m; }
    const long long top = r * x + a;
    if (top < m) return sum;
    x = top / m;
    a = top % m;
    const long long t = m;
    m = r;
    r = t;
  }
}

// The items of one (sequence, KV head).
struct PagedSeq {
  int nq, len, tok0;
  int nblk;                   // items
  __device__ __forceinline__ void load(const PagedParams& p, int b) {
    tok0 = p.cu_q[b];
    const int end = min(p.cu_q[b + 1], p.T);
    nq = tok0 >= 0 ? max(0, end - tok0) : 0;
    // no further than the table leads: what lies behind is not followed and, where rows would see
    // it, reported (a slot without new tokens may hold any length)
    const long long room = static_cast<long long>(p.max_pages) << p.c.page_shift;
    len = max(0, p.kv_len[b]);
    if (len > room) {
      if (nq > 0) record_bad_page();
      len = static_cast<int>(room);
    }
    // positions follow from the sequence's own count of tokens, also where T cuts it short
    pos0 = len - max(nq, p.cu_q[b + 1] - tok0);
    nblk = (nq + p.RI - 1) / p.RI;
  }
  int pos0;
  // first and last key tile of item i
  __device__ __forceinline__ void range(const PagedParams& p, int i, int& kmin, int& j0, int& n) const {
    const int p0 = pos0 + i * p.RI, p1 = pos0 + min(nq, (i + 1) * p.RI) - 1;
    kmin = p.wl >= 0 ? max(0, p0 - p.wl) : 0;
    const int kmax = p.causal ? min(p1, len - 1) : len - 1;
    j0 = kmin >> 7;
    n = max(1, (max(kmax, 0) >> 7) - j0 + 1);
  }
  // key tiles of the items before item i
  __device__ __forceinline__ long long before(const PagedParams& p, int i) const {
    if (i <= 0) return 0;
    long long last = 0;
    if (i == nblk) {          // the last item may have fewer tokens
      int kmin, j0, n;
      range(p, i - 1, kmin, j0, n);
      last = n;
      if (--i == 0) return last;
    }
    const long long hi = p.causal ? stair_sum(pos0 + p.RI - 1, p.RI, i) : static_cast<long long>(max(len - 1, 0) >> 7) * i;
    const long long lo = p.wl >= 0 ? stair_sum(static_cast<long long>(pos0) - p.wl, p.RI, i) : 0;
    return last + hi - lo + i;
  }
  __device__ __forceinline__ long long tiles(const PagedParams& p) const { return before(p, nblk); }
};

// Where a CTA's share begins.
struct PagedPlan {
  long long warp_sum[32];
  long long total;            // W
  long long begin, end;       // this CTA's tiles
  long long rest;             // begin, counted from the first tile of sequence b
  long long head_tiles;       // tiles of one (b, g)
  int parts;                  // C: CTAs that have a share
  int whole;                  // p.whole, but 4 at most where a share is under 2 tiles: there CTAs are left over
  int b;
};

__device__ __forceinline__ long long paged_tiles(const PagedParams& p, int b) {
  if (b >= p.B) return 0;
  PagedSeq s;
  s.load(p, b);
  return s.tiles(p) * p.Hkv;
}

// 64-bit quotient; most are of small numbers, for which 32-bit division is several times
// faster.
__device__ __forceinline__ long long small_div(long long a, long long b) {
  if ((static_cast<unsigned long long>(a) | static_cast<unsigned long long>(b)) >> 32) return a / b;
  return static_cast<unsigned>(a) / static_cast<unsigned>(b);
}

// The CTA's range of W tiles.
__device__ __forceinline__ void paged_share(const PagedParams& p, int cta, long long total, int& parts, long long& begin,
                                            long long& end) {
  parts = static_cast<int>(total < 1 ? 1 : total < p.ctas ? total : p.ctas);
  begin = cta < parts ? small_div(total * cta, parts) : total;
  end = cta < parts ? small_div(total * (cta + 1), parts) : total;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// The plan by one warp, for at most 32 sequences.
__device__ __forceinline__ void paged_plan_warp(const PagedParams& p, PagedPlan& pl, int cta, int lane) {
  const long long mine = paged_tiles(p, lane);
  const long long incl = warp_scan(mine, lane);
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  int parts;
  long long begin, end;
  paged_share(p, cta, total, parts, begin, end);
  if (lane == 0) {
    pl.total = total;
    pl.parts = parts;
    pl.whole = total < 2LL * p.ctas ? min(p.whole, 4) : p.whole;
    pl.begin = begin;
    pl.end = end;
    pl.b = p.B;
  }
  __syncwarp();
  const long long from = incl - mine;
  if (begin < end && from <= begin && begin < from + mine) {
    pl.b = lane;
    pl.rest = begin - from;
    pl.head_tiles = small_div(mine, p.Hkv);
  }
  __syncwarp();
}

// Block-wide inclusive scan of v; returns this thread's prefix, total in all threads.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sum, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  v = warp_scan(v, lane);
  __syncthreads();                            // warp_sum is free again
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int i = 0; i < nw; ++i) {
    const long long s = warp_sum[i];
    if (i < warp) before += s;
    total += s;
  }
  return before + v;
}

// The plan by all threads of the CTA, for any number of sequences.
__device__ __forceinline__ void paged_plan_block(const PagedParams& p, PagedPlan& pl, int cta) {
  const int nt = blockDim.x;
  long long mine = 0, incl = 0, total = 0, sum = 0;
  if (threadIdx.x == 0) pl.b = p.B;           // nothing found yet; the scan's barriers order this first
  for (int b0 = 0; b0 < p.B; b0 += nt) {
    mine = paged_tiles(p, b0 + threadIdx.x);
    incl = block_scan(mine, pl.warp_sum, sum);
    total += sum;
  }
  int parts;
  long long begin, end, base = 0;
  paged_share(p, cta, total, parts, begin, end);
  if (threadIdx.x == 0) {
    pl.total = total;
    pl.parts = parts;
    pl.whole = total < 2LL * p.ctas ? min(p.whole, 4) : p.whole;
    pl.begin = begin;
    pl.end = end;
  }
  for (int b0 = 0; b0 < p.B; b0 += nt) {      // find the sequence that holds tile `begin`
    const int b = b0 + threadIdx.x;
    if (p.B > nt) {
      mine = paged_tiles(p, b);
      incl = block_scan(mine, pl.warp_sum, sum);
    }
    const long long from = base + incl - mine;
    if (b < p.B && begin < end && from <= begin && begin < from + mine) {
      pl.b = b;
      pl.rest = begin - from;
      pl.head_tiles = small_div(mine, p.Hkv);
    }
    base += sum;
  }
  __syncthreads();
}

// W, the CTA's range and the sequence it begins in.  Up to 32 sequences, `planner` (the warp
// that walks through the share) finds them alone while the others set up barriers and TMEM;
// beyond, all threads do.
__device__ __forceinline__ void paged_plan(const PagedParams& p, PagedPlan& pl, int cta, bool planner, int lane) {
  if (p.B > 32) paged_plan_block(p, pl, cta);
  else if (planner) paged_plan_warp(p, pl, cta, lane);
}

// The pieces of a CTA's share, in order.  Used by one whole warp (the first place needs
// its lanes); afterwards every lane holds the same state.
struct PagedWalk {
  PagedSeq s;
  int b, g, i;                // sequence, KV head, item
  int skip;                   // tiles of the item that lie before the share
  long long left;             // tiles still to hand out
  long long cut_end = 0;      // of the item cut at the end of the share: the tile behind its last one
  __device__ __forceinline__ void begin(const PagedParams& p, const PagedPlan& pl, int lane) {
    left = pl.end - pl.begin;
    b = pl.b;
    g = i = skip = 0;
    if (left <= 0 || b >= p.B) { left = 0; return; }
    s.load(p, b);
    g = static_cast<int>(small_div(pl.rest, pl.head_tiles));
    const long long rest = pl.rest - g * pl.head_tiles;
    int lo = 0, hi = s.nblk;                  // before(lo) <= rest < before(hi)
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + (lane + 1) * step, hi);
      const unsigned m = __ballot_sync(0xffffffffu, at < hi && s.before(p, at) <= rest);
      lo += __popc(m) * step;
      hi = min(lo + step, hi);
    }
    i = lo;
    skip = static_cast<int>(rest - s.before(p, i));
  }
  // next piece; n = 0 when the share is used up
  __device__ __forceinline__ PagedSeg next(const PagedParams& p, const PagedPlan& pl, int cta) {
    PagedSeg w;
    w.n = 0;
    w.slot = -1;
    while (left > 0) {
      if (i >= s.nblk) {                      // next head, or next sequence that has tokens
        i = 0;
        if (++g >= p.Hkv) {
          g = 0;
          const int lane = threadIdx.x & 31;  // 32 sequences at a look: a padded batch may have many empty ones
          unsigned some = 0;
          for (++b; b < p.B; b += 32) {
            const int c = b + lane;
            some = __ballot_sync(0xffffffffu, c < p.B && min(p.cu_q[c + 1], p.T) > max(p.cu_q[c], 0));
            if (some) break;
          }
          if (!some) { left = 0; return w; }
          b += __ffs(some) - 1;
          s.load(p, b);
        }
      }
      int n;
      s.range(p, i, w.kmin, w.j0, n);
      if (n <= pl.whole && skip > 0) {         // begun in the share before: all of it went there
        left -= n - skip;
        skip = 0;
        ++i;
        continue;
      }
      w.b = b;
      w.g = g;
      w.tok0 = s.tok0 + i * p.RI;
      w.ntok = min(p.RI, s.nq - i * p.RI);
      w.pos0 = s.pos0 + i * p.RI;
      w.len = s.len;
      w.j0 += skip;
      const int have = n - skip;
      w.n = n <= pl.whole || left >= have ? have : static_cast<int>(left);
      if (skip > 0) w.slot = 2 * cta;
      else if (w.n < n) w.slot = 2 * cta + 1;
      if (skip == 0 && w.n < n) cut_end = pl.end - left + n;   // the first part of a cut item
      left -= w.n;
      skip = 0;
      ++i;
      return w;
    }
    return w;
  }
};

// Descriptor of the item that the CTA's share cuts (one thread, once the share is walked
// through): w is the last piece, which holds the item's first part if `walk` says so.
__device__ __forceinline__ void paged_post_cut(const PagedParams& p, const PagedPlan& pl, const PagedWalk& walk,
                                               const PagedSeg& w, int cta) {
  PagedCut cut = {0, 0, 0, 0};
  if (walk.cut_end > 0) {
    // CTA c holds the tiles [W c / C, W (c+1) / C): the one with tile x is ((x + 1) C - 1) / W
    const int c1 = static_cast<int>(small_div(walk.cut_end * pl.parts - 1, pl.total));
    cut = {w.tok0, w.ntok, w.g, c1 - cta + 1};
  }
  p.cuts[cta] = cut;
}

// Pieces passed from the producer warp to the consumer warps, in order.
struct SegRing {
  uint64_t full[4];           // count 1
  uint64_t empty[4];          // count = number of consumer warps
  PagedSeg seg[4];
};
__device__ __forceinline__ void seg_ring_init(SegRing& r, uint32_t consumers) {
  for (int i = 0; i < 4; ++i) {
    mbar_init(&r.full[i], 1);
    mbar_init(&r.empty[i], consumers);
  }
}
// Producer (one thread): post the k-th piece; false if a wait failed.
__device__ __forceinline__ bool seg_ring_post(SegRing& r, int k, const PagedSeg& w) {
  const int i = k & 3;
  if (k >= 4 && !mbar_wait(&r.empty[i], ((k >> 2) - 1) & 1)) return false;
  r.seg[i] = w;
  mbar_arrive(&r.full[i]);
  return true;
}
// Consumer (whole warp): the k-th piece; n = 0 at the end or if a wait failed (ok = false).
__device__ __forceinline__ PagedSeg seg_ring_take(SegRing& r, int k, int lane, bool& ok) {
  const int i = k & 3;
  PagedSeg w;
  w.n = 0;
  ok = __all_sync(0xffffffffu, mbar_wait(&r.full[i], (k >> 2) & 1));
  if (!ok) return w;
  w = r.seg[i];
  __syncwarp();
  if (lane == 0) mbar_arrive(&r.empty[i]);
  return w;
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const void* tmap, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// ------------------------------------------------------------------ pipeline shared by the kernels
// Barriers between the producer warp, the widening warps (e4m3 cache) and the MMA warp.
struct PagedPipe {
  uint64_t q_full[2], q_empty[2], q8_full[2];
  uint64_t k_full[8], v_full[8];       // by stage: the tile is there
  uint64_t k_done[8], v_done[8];       // by tile % 8: S, and P V, of that tile complete
  uint64_t raw_full[8], raw_empty[8];
  SegRing ring;
  uint64_t drain, teardown;
  PagedPlan plan;
  uint32_t tmem_base;
};
// C::KV8: the cache is e4m3.  C::K8: K tiles go to the tensor cores as e4m3 (Q then does as
// well, in two parts); else the widening warps turn them into bf16 tiles like those of V.
template <class C>
__device__ __forceinline__ void paged_pipe_init(PagedPipe& sh, int ring_consumers, int warps) {
  for (int i = 0; i < 2; ++i) {
    mbar_init(&sh.q_full[i], 1);
    mbar_init(&sh.q_empty[i], 1);
    mbar_init(&sh.q8_full[i], C::K8 ? C::kWiden : 1);
  }
  for (int i = 0; i < C::KSK; ++i) {
    mbar_init(&sh.k_full[i], C::K8 ? 33 : C::KV8 ? 4 : 1);     // 33: the copies, and each lane's scales
  }
  for (int i = 0; i < C::KSV; ++i) {
    mbar_init(&sh.v_full[i], C::KV8 ? 4 : 1);
  }
  for (int i = 0; i < 8; ++i) {
    mbar_init(&sh.k_done[i], 1);
    mbar_init(&sh.v_done[i], 1);
  }
  for (int i = 0; i < C::RST; ++i) {
    mbar_init(&sh.raw_full[i], 33);
    mbar_init(&sh.raw_empty[i], 4);
  }
  seg_ring_init(sh.ring, ring_consumers);
  mbar_init(&sh.drain, 1);
  mbar_init(&sh.teardown, warps);
}

// Wait until S (P V) of tile c, counted over the CTA's share, is complete: its K (V) stage
// may be filled again.
__device__ __forceinline__ bool tile_done_wait(uint64_t (&done)[8], int c) {
  return mbar_wait(&done[c & 7], (c >> 3) & 1);
}

// Shared-memory regions of a kernel.
struct PagedSmem {
  uint8_t *q, *k, *v;         // tiles as the tensor cores read them (q: bf16)
  uint8_t *raw, *scale;       // e4m3 tiles before widening, 128 scale bytes per stage
  uint8_t* kscale;            // K8: scale bytes of the last 8 K tiles
};

// Pages of a key tile that hold keys in [kmin, len): local indices.
struct PageTile {
  int first, count;
};
__device__ __forceinline__ PageTile page_tile(const PagedParams& p, const PagedSeg& w, int j) {
  const int lo = max(w.kmin, j * 128), hi = min(w.len, j * 128 + 128);
  PageTile t;
  t.first = 0;
  t.count = 0;
  if (hi <= lo) return t;
  const int sh = p.c.page_shift < 7 ? p.c.page_shift : 7;      // pages larger than a tile count as one box
  t.first = (lo - j * 128) >> sh;
  t.count = ((hi - 1 - j * 128) >> sh) - t.first + 1;
  return t;
}

// 128 successive entries of a sequence's row of the block table, 4 to a lane: the pages of
// the next 16 or more key tiles.  Looking entries up one by one cost the producer a trip to
// memory per tile (B = 64 requests of 8K, d = 64 bf16: 180 us; from here 143).
struct PageWindow {
  int e[4];
  int base;                   // page index of the first one
  __device__ __forceinline__ void load(const PagedParams& p, int b, int first, int lane) {
    base = first;
    const int* row = p.table + static_cast<long long>(b) * p.max_pages;
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = first + 32 * i + lane < p.max_pages ? row[first + 32 * i + lane] : -1;
  }
  // entry of page index pi (whole warp; any lane asks for its own, all within the window)
  __device__ __forceinline__ int get(int pi) const {
    const int off = pi - base;
    int v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = __shfl_sync(0xffffffffu, e[i], off & 31);
      if ((off >> 5) == i) v = x;
    }
    return v;
  }
};

// Four bytes, of which the first `bytes` come from src (nothing is read for 0) and the rest are 0.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}
// Arrive on the barrier once this thread's cp.async so far have landed (one of its count).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Copies of one tensor's key tiles of a piece: kv = 0 K, 1 V; kc counts the tiles before it.
// Lane 0 arms a stage's barrier, then lane i issues the copy of the tile's i-th (page,
// 64-column box).  A copy takes the copy engine some 60 ns however small it is, so the scale
// bytes of an e4m3 tile, 16 to a page, do not go by copies of their own: every lane fetches
// four of them by cp.async, which arrives on the same barrier.
template <class C, int kv>
__device__ __forceinline__ bool paged_load_tiles(const PagedParams& p, PagedPipe& sh, const CUtensorMap* tm,
                                                 const PagedSmem& m, const PagedSeg& w, int& kc, int lane) {
  constexpr bool kRaw = C::KV8 && !(C::K8 && kv == 0);         // e4m3 tiles on their way to be widened
  // bytes per key that the copies bring in: a padded e4m3 row of 128 bytes for K8
  constexpr int kRowBytes = kv == 0 && C::K8 ? 128 : C::KV8 ? C::D : 2 * C::D;
  constexpr int kStages = kRaw ? C::kRawMod : kv == 0 ? C::KSK : C::KSV;
  constexpr int NX = C::KV8 ? 1 : C::NB;                       // column boxes per page
  const int shift = p.c.page_shift, psh = shift < 7 ? shift : 7;
  const int rows = 1 << psh, per_tile = 128 >> psh;            // rows of a box, pages of a tile
  const int bx = lane / NX, bc = lane % NX;
  PageWindow win;
  int p0 = shift <= 7 ? w.j0 << (7 - shift) : w.j0 >> (shift - 7);
  win.load(p, w.b, p0, lane);
  for (int j = 0; j < w.n; ++j, ++kc) {
    const int jt = w.j0 + j;
    const PageTile t = page_tile(p, w, jt);
    p0 = shift <= 7 ? jt << (7 - shift) : jt >> (shift - 7);
    if (p0 + per_tile > win.base + 128) win.load(p, w.b, p0, lane);
    int page = win.get(p0 + min(t.first + bx, per_tile - 1));
    if (bx < t.count && (page < 0 || page >= p.c.num_pages)) {
      record_bad_page();
      page = -1;
    }
    const int y = shift > 7 ? (jt & ((1 << (shift - 7)) - 1)) * 128 : 0;      // row of the tile in its page
    // a stage and which use of it this is (K8 = false: K and V share the raw stages in turn)
    const int c = kRaw && !C::K8 ? 2 * kc + kv : kc;
    const int st = c % kStages, round = c / kStages;
    uint64_t* full = kRaw ? &sh.raw_full[st] : kv == 0 ? &sh.k_full[st] : &sh.v_full[st];
    uint8_t* dst = kRaw ? m.raw + st * C::kRawTile : kv == 0 ? m.k + st * C::kKTile : m.v + st * C::kTile;
    // Scale bytes of rows 4 lane .. 4 lane + 3.  Rows that are not followed get 0 like their codes,
    // not what the slot held: 0 times a stale factor of infinity would be NaN.
    const uint8_t* scale_src = kv ? p.c.vs : p.c.ks;
    int scale_bytes = 0;
    if constexpr (C::KV8) {
      const int r = 4 * lane, box = (r >> psh) - t.first;
      const int pg = __shfl_sync(0xffffffffu, page, box & 31);                // lane i holds the page of box i
      if (box >= 0 && box < t.count && pg >= 0) {
        scale_src += ((static_cast<long long>(pg) * p.Hkv + w.g) << shift) + y + (r & (rows - 1));
        scale_bytes = 4;
      }
    }
    if (round > 0) {
      const bool free = kRaw ? mbar_wait(&sh.raw_empty[st], (round - 1) & 1)
                             : tile_done_wait(kv ? sh.v_done : sh.k_done, kc - kStages);
      if (!__all_sync(0xffffffffu, free)) return false;
    }
    if (lane == 0) {
      if (t.count > 0) mbar_arrive_expect_tx(full, t.count * rows * kRowBytes);
      else mbar_arrive(full);
    }
    __syncwarp();
    if (bx < t.count) {
      const int r0 = (t.first + bx) << psh;         // row of the box in the tile
      in_range(r0 + rows - 1, 128);
      const int z = page < 0 ? p.c.num_pages : page;           // outside the pool: zeros
      tma_load_4d(dst + (C::KV8 ? r0 * kRowBytes : bc * C::kBox + r0 * 128), tm, full, C::KV8 ? 0 : bc * 64, y, w.g, z);
    }
    if constexpr (C::KV8) {
      uint8_t* scale = kRaw ? m.scale + st * 128 : m.kscale + (kc & 7) * 128;
      cp_async4(scale + 4 * lane, scale_src, scale_bytes);
      cp_async_arrive(full);
    }
  }
  return true;
}

// On an error: let the copies in flight of one tensor land (bounded); kc tiles were begun.
template <class C, int kv>
__device__ __forceinline__ void paged_drain_tiles(PagedPipe& sh, int kc, int lane) {
  constexpr bool kRaw = C::KV8 && !(C::K8 && kv == 0);
  constexpr int kStages = kRaw ? C::kRawMod : kv == 0 ? C::KSK : C::KSV;
  if constexpr (C::KV8) asm volatile("cp.async.wait_all;" ::: "memory");
  if (lane != 0) return;
  for (int t = max(0, kc - kStages); t <= kc; ++t) {
    const int c = kRaw && !C::K8 ? 2 * t + kv : t;
    uint64_t* full = kRaw ? &sh.raw_full[c % kStages] : kv == 0 ? &sh.k_full[c % kStages] : &sh.v_full[c % kStages];
    mbar_drain_wait(full, (c / kStages) & 1);
  }
}

// K producer warp: walks through the CTA's share, posts its pieces and brings in Q and K.
template <class C>
__device__ __forceinline__ void paged_produce_k(const PagedParams& p, PagedPipe& sh, const CUtensorMap* tmq,
                                                const CUtensorMap* tmk, const PagedSmem& m, int cta, int lane) {
  if (lane == 0) { tma_prefetch_desc(tmq); tma_prefetch_desc(tmk); }
  PagedWalk walk;
  walk.begin(p, sh.plan, lane);
  int kc = 0, uq = 0;                               // key tiles, pieces
  bool ok = true;
  PagedSeg last;
  for (int k = 0; ok; ++k) {
    const PagedSeg w = walk.next(p, sh.plan, cta);
    if (w.n > 0) last = w;
    if (lane == 0) {
      ok = seg_ring_post(sh.ring, k, w);
      if (ok && w.n > 0) {
        const int qs = uq % C::QST;
        if (uq >= C::QST) ok = mbar_wait(&sh.q_empty[qs], ((uq / C::QST) - 1) & 1);
        if (ok) {
          const int teams = C::kTeams > 1 && w.ntok > p.R ? 2 : 1;    // query tiles of the item
          mbar_arrive_expect_tx(&sh.q_full[qs], teams * p.G * p.R * C::D * 2);
          for (int c = 0; c < teams * C::NB; ++c)
            tma_load_3d(m.q + qs * C::kQTile + c * C::kQBox, tmq, &sh.q_full[qs], (c % C::NB) * 64, w.g * p.G,
                        w.tok0 + (c / C::NB) * p.R);
          ++uq;
        }
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (!ok || w.n == 0) break;
    ok = paged_load_tiles<C, 0>(p, sh, tmk, m, w, kc, lane);
  }
  if (lane == 0) paged_post_cut(p, sh.plan, walk, last, cta);
  if (!ok) {
    paged_drain_tiles<C, 0>(sh, kc, lane);
    if (lane == 0)
      for (int r = max(0, uq - C::QST); r < uq; ++r) mbar_drain_wait(&sh.q_full[r % C::QST], (r / C::QST) & 1);
  }
  if constexpr (C::KV8) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// V producer warp: follows the posted pieces (one warp for both tensors took 1.9k cycles
// per tile at work of its own, more than an e4m3 tile's 1.4k at HBM's rate).
template <class C>
__device__ __forceinline__ void paged_produce_v(const PagedParams& p, PagedPipe& sh, const CUtensorMap* tmv,
                                                const PagedSmem& m, int lane) {
  if (lane == 0) tma_prefetch_desc(tmv);
  int kc = 0;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
    if (w.n == 0) break;
    ok = paged_load_tiles<C, 1>(p, sh, tmv, m, w, kc, lane);
  }
  if (!ok) paged_drain_tiles<C, 1>(sh, kc, lane);
  if constexpr (C::KV8) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// Widening warps (e4m3 cache), wt = 0 .. 32 kWiden - 1, in groups of four: each group takes
// whole tiles in turn (K8: the V tiles; else group 0 those of K, group 1 those of V), so
// that a tile's waits and fences overlap the other group's work.  split_q(k, qs) readies Q
// of the k-th piece in buffer qs (K8).  A lane takes 16 codes of a row,
// widens them with the row's scale and stores two 16-byte chunks of the bf16 tile in the
// 128B-swizzled layout the TMA would write.  Eight lanes (one shared-memory wavefront)
// take 4 chunks of each of 2 rows: their stores then fall on 8 different chunk positions.
// At d = 128 the raw tile is swizzled too, and lanes 0-7 take the chunks {0, 5, 2, 7},
// lanes 8-15 {1, 4, 3, 6} of their rows, for which the loads of both rows are disjoint as
// well (without this, 30% more time per tile).
template <class C, typename SplitQ>
__device__ __forceinline__ void paged_widen(PagedPipe& sh, const PagedSmem& m, int wt, int lane, SplitQ split_q) {
  constexpr int D = C::D;
  constexpr int CPR = D / 16;                       // 16-code chunks per row
  constexpr int RPP = 128 / CPR;                    // rows per pass of a group
  constexpr int kGroups = C::kWiden / 4;
  const int grp = wt >> 7;
  wt &= 127;
  const int e = wt & 3, half = (wt >> 3) & 1;       // chunk inside its set, which set (d = 128)
  const int c = D == 128 ? (e ^ ((e & 1) << 2) ^ half) : e;
  const int r_in = D == 128 ? ((wt >> 4) << 1) + ((wt >> 2) & 1) : wt >> 2;
  int kc = 0;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const PagedSeg w = seg_ring_take(sh.ring, k, lane, ok);
    if (w.n == 0) break;
    if constexpr (C::K8) {
      const int qs = k % C::QST;
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_full[qs], (k / C::QST) & 1));
      if (!ok) break;
      split_q(k, qs);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q8_full[qs]);
    }
    for (int j = 0; j < w.n && ok; ++j, ++kc) {
      const int lo = w.kmin - (w.j0 + j) * 128, hi_row = w.len - (w.j0 + j) * 128;
      static_assert(C::K8 || C::KSK == C::KSV, "K and V tiles are widened in turn");
      const int st = kc % C::KSV;
#pragma unroll 1
      for (int kv = C::K8 ? 1 : 0; kv < 2; ++kv) {
        if ((C::K8 ? kc : kv) % kGroups != grp) continue;
        const int rc = C::K8 ? kc : 2 * kc + kv, rs = rc % C::RST;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.raw_full[rs], (rc / C::RST) & 1));
        if (ok && kc >= C::KSV)
          ok = __all_sync(0xffffffffu, tile_done_wait(kv ? sh.v_done : sh.k_done, kc - C::KSV));
        if (!ok) break;
        const uint8_t* raw = m.raw + rs * C::kRawTile;
        uint8_t* out = (kv ? m.v : m.k) + st * C::kTile;
        constexpr int NP = 128 / RPP;               // passes
        auto at = [&](int i) { return i * RPP + r_in; };
        auto load = [&](int i, uint32_t (&codes)[4], int& byte) {
          const int r = at(i), rawc = D == 128 ? c ^ (r & 7) : c;
          const uint4 x = *reinterpret_cast<const uint4*>(raw + r * D + rawc * 16);
          codes[0] = x.x; codes[1] = x.y; codes[2] = x.z; codes[3] = x.w;
          byte = m.scale[rs * 128 + r];
          if (kv && (r < lo || r >= hi_row)) {      // keys that nobody sees
            codes[0] = codes[1] = codes[2] = codes[3] = 0u;
            byte = 0;
          }
        };
        auto put = [&](int i, const uint32_t (&y)[8]) {
          // chunks 2c and 2c + 1 of the row, 8 to a 64-column box
          const int r = at(i), box = c >> 2, cc = (2 * c) & 7;
          uint8_t* row = out + box * C::kBox + r * 128;
          *reinterpret_cast<uint4*>(row + ((cc ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(row + (((cc + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
        };
        // Passes whose loads are in flight together.  Few: shorter loops measured
        // faster (4 passes: 182-201 us, 2: 170-184, 64 x 8K at d = 128); why was not isolated (missing
        // instructions are 0.9 of the 8.8 cycles between a warp's issues now).
        constexpr int NB = NP < 2 ? NP : 2;
#pragma unroll 1
        for (int i0 = 0; i0 < NP; i0 += NB) {
          uint32_t codes[NB][4];
          int byte[NB];
          bool rare = false;
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            load(i0 + i, codes[i], byte[i]);
            rare |= byte[i] > kE4m3FastByte || e4m3_any_nan<4>(codes[i]) != 0;
          }
          if (!__any_sync(0xffffffffu, rare)) {     // one branch for the warp
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              uint32_t y[8];
              e4m3_widen<4>(codes[i], byte[i], false, y);
              put(i0 + i, y);
            }
          } else {
#pragma unroll 1
            for (int i = 0; i < NB; ++i) {
              uint32_t again[4], y[8];
              int b;
              load(i0 + i, again, b);
              e4m3_widen<4>(again, b, true, y);
              put(i0 + i, y);
            }
          }
        }
        fence_proxy_async_smem();                   // generic-proxy writes -> tensor-core reads
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv ? &sh.v_full[st] : &sh.k_full[st]);
          mbar_arrive(&sh.raw_empty[rs]);
        }
      }
    }
  }
}

// Rows of a bf16 V tile at keys that nobody sees (behind the sequence, before the window,
// in pages that were not loaded) are zeroed by the MMA warp: their P is 0, and 0 times
// whatever lies there has to be 0.
template <class C>
__device__ __forceinline__ void paged_zero_v(const PagedSeg& w, int j, uint8_t* v, int lane) {
  const int lo = w.kmin - (w.j0 + j) * 128, hi_row = w.len - (w.j0 + j) * 128;
  if (lo <= 0 && hi_row >= 128) return;
  for (int x = lane; x < 128 * 8; x += 32) {
    const int r = x >> 3;
    if (r >= lo && r < hi_row) continue;
    for (int c = 0; c < C::NB; ++c) *reinterpret_cast<uint4*>(v + c * C::kBox + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Merge of cut items: the blocks of column x look after the item whose first part CTA x
// holds; one warp per row, D / 32 columns per lane.  The lanes first take the row's LSEs, one
// part each, then all read the parts' O in turn, 8 of them in flight.
template <int D>
__global__ void __launch_bounds__(256) attn_paged_merge_kernel(const PagedParams p) {
  grid_dependency_wait();
  constexpr int PER = D / 32;
  const int c = blockIdx.x, lane = threadIdx.x & 31;
  const PagedCut cut = p.cuts[c];
  const int rows = cut.ntok * p.G;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < rows; r += gridDim.y * 8) {
    auto at = [&](int s) { return static_cast<size_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)) * p.slot_rows + r; };
    float m = -INFINITY;
    for (int s = lane; s < cut.parts; s += 32) m = fmaxf(m, p.lpart[at(s)]);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    float acc[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) acc[x] = 0.f;
    float wsum = 0.f;
    for (int s0 = 0; s0 < cut.parts; s0 += 32) {
      const float ls = s0 + lane < cut.parts ? p.lpart[at(s0 + lane)] : -INFINITY;
      const float mine = ls == -INFINITY ? 0.f : ex2_approx((ls - m) * 1.4426950408889634f);
      const int n = min(32, cut.parts - s0);
      for (int t0 = 0; t0 < n; t0 += 8) {
        float o[8][PER];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
#pragma unroll
          for (int x = 0; x < PER; ++x) o[t][x] = 0.f;
          if (t0 + t < n) {
            const float* src = p.opart + at(s0 + t0 + t) * D + lane * PER;
            if constexpr (PER == 4) {
              const float4 v = *reinterpret_cast<const float4*>(src);
              o[t][0] = v.x; o[t][1] = v.y; o[t][2] = v.z; o[t][3] = v.w;
            } else {
              const float2 v = *reinterpret_cast<const float2*>(src);
              o[t][0] = v.x; o[t][1] = v.y;
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const float w = __shfl_sync(0xffffffffu, mine, (t0 + t) & 31);
          if (t0 + t < n) {
            wsum += w;
#pragma unroll
            for (int x = 0; x < PER; ++x) acc[x] = fmaf(w, o[t][x], acc[x]);
          }
        }
      }
    }
    const int i = r / p.G, h = r - i * p.G;
    const size_t orow = static_cast<size_t>(cut.tok0 + i) * p.Hq + cut.g * p.G + h;
    const bool none = wsum == 0.f;
    const float inv = none ? 0.f : 1.f / wsum;
    __nv_bfloat16* dst = p.o + orow * D + lane * PER;
#pragma unroll
    for (int x = 0; x < PER; x += 2)
      *reinterpret_cast<uint32_t*>(dst + x) = pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
    if (lane == 0) p.lse[orow] = none ? -INFINITY : m + __logf(wsum);
  }
}

}  // namespace attn
