// Rotary positions, and the paged K/V cache's write and read-back, for sm_100a.
//
// All three are streams: every input element is read once and every output element
// written once, with a few operations in between, so HBM bounds them at large sizes and
// the chain launch -> dependent loads -> store at small ones.
//
// Rotation.  Pair i of a row is turned by pos * f_i.  The angle of a far position needs
// more bits than fp32 has (pos = 10^6: an fp32 product is off by 0.03 rad), so a thread
// forms it in turns, r = pos * (f_i / 2 pi), in fp64, subtracts the nearest integer
// (exact) and hands |r| <= 1/2 to sincospif in fp32.  Sine and cosine depend on the token
// and the pair only: a thread owns one 16-byte unit of a token's rows -- for the half
// layout the chunk of first elements and the chunk of its partners -- and applies the
// same registers to every head it visits.
#pragma once
#include "sm100.cuh"

namespace attn {

// Set when a block table entry or a position lies outside the page pool.  Apart from
// g_attn_status on purpose: the kernels go on (the access is skipped), so nothing that
// waits has to give up.
__device__ int g_attn_bad_page = 0;
__device__ __forceinline__ void record_bad_page() { atomicExch(&g_attn_bad_page, 1); }

// Programmatic dependent launch: wait until the kernels before this one have finished and
// their writes are visible / let the next kernel's blocks start early.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct RowView {              // [batch][head][token][d], strides in elements
  char* p;
  long long sb, sh, st;
};

struct RopeParams {
  RowView q, qo, k, ko;       // k.p may be null with Hk = 0
  int Hq, Hk, B, N;
  const int* pos;
  long long pos_sb;
  const double* inv_freq;
  int rot, inverse;
  float mscale;
  int heads_per_block;        // heads that one block walks through
};

// 16 bytes of T as floats and back; bf16 rounds to nearest even.
template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec16<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void load(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// How a row of D elements of T is cut into the units that threads own.
//   half layout: unit u < rot / 2n holds chunks u and u + rot / 2n (n pairs); the copied
//     rest is cut the same way, into pairs of chunks
//   interleaved: unit u is chunk u, n / 2 pairs (or n copied elements)
// Chunks are 16 bytes (n elements), so a warp's accesses are contiguous in both layouts.
template <typename T, int D, bool INTER>
struct RopeUnit {
  static constexpr int n = Vec16<T>::n;
  static constexpr int kChunks = D / n;                    // per row
  static constexpr int kUnits = INTER ? kChunks : kChunks / 2;
  static constexpr int kPairs = INTER ? n / 2 : n;
  static constexpr int NC = INTER ? 1 : 2;                 // chunks per unit
  int c0, c1, pair0;
  bool turned;
  __device__ __forceinline__ RopeUnit(int u, int rot) {
    if constexpr (INTER) {
      c0 = c1 = u;
      turned = u * n < rot;
      pair0 = u * kPairs;
    } else {
      const int ru = rot / (2 * n);                        // turned units
      turned = u < ru;
      const int tail = (kChunks - 2 * ru) / 2;             // copied units
      c0 = turned ? u : 2 * ru + (u - ru);
      c1 = turned ? u + ru : c0 + tail;
      pair0 = u * n;
    }
  }
};

template <int P>
__device__ __forceinline__ void rope_sincos(const double* __restrict__ inv_freq, int pair0, int pos, float m,
                                            int inverse, float (&cs)[P], float (&sn)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const double r = static_cast<double>(pos) * (inv_freq[pair0 + i] * 0.15915494309189533577);   // turns
    const float x = static_cast<float>(r - rint(r));
    float s, c;
    sincospif(2.f * x, &s, &c);
    cs[i] = c * m;
    sn[i] = inverse ? -s * m : s * m;
  }
}

// y = m R x on one unit's registers: a[] is the first chunk, b[] its partner chunk (half
// layout) or unused (interleaved).
template <typename T, bool INTER, int P, int n>
__device__ __forceinline__ void rope_turn(float (&a)[n], float (&b)[n], const float (&cs)[P], const float (&sn)[P]) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * cs[i] - y * sn[i];
      a[2 * i + 1] = y * cs[i] + x * sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i] - y * sn[i];
      b[i] = y * cs[i] + x * sn[i];
    }
  }
}

// Grid: x over blocks of tokens (256 / kUnits tokens each), y over blocks of heads.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(256) attn_rope_kernel(const RopeParams p) {
  using U = RopeUnit<T, D, INTER>;
  constexpr int n = U::n;
  grid_dependency_wait();
  grid_dependency_launch();
  const int u = threadIdx.x % U::kUnits;
  const long long tok = static_cast<long long>(blockIdx.x) * (256 / U::kUnits) + threadIdx.x / U::kUnits;
  if (tok >= static_cast<long long>(p.B) * p.N) return;
  const int b = static_cast<int>(tok / p.N), t = static_cast<int>(tok - static_cast<long long>(b) * p.N);
  const U unit(u, p.rot);
  float cs[U::kPairs], sn[U::kPairs];
  if (unit.turned)
    rope_sincos<U::kPairs>(p.inv_freq, unit.pair0, p.pos[b * p.pos_sb + t], p.mscale, p.inverse, cs, sn);
  const int h0 = blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.Hq + p.Hk);
  auto src = [&](int h, int c) -> const uint4* {
    const RowView& v = h < p.Hq ? p.q : p.k;
    const int hh = h < p.Hq ? h : h - p.Hq;
    return reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(v.p) + b * v.sb + hh * v.sh + t * v.st + c * n);
  };
  auto dst = [&](int h, int c) -> uint4* {
    const RowView& v = h < p.Hq ? p.qo : p.ko;
    const int hh = h < p.Hq ? h : h - p.Hq;
    return reinterpret_cast<uint4*>(reinterpret_cast<T*>(v.p) + b * v.sb + hh * v.sh + t * v.st + c * n);
  };
  constexpr int UN = 4;                       // heads in flight: 64 or 128 bytes per thread
  for (int h = h0; h < h1; h += UN) {
    uint4 x[UN][U::NC];
#pragma unroll
    for (int i = 0; i < UN; ++i)
      if (h + i < h1) {
        x[i][0] = *src(h + i, unit.c0);
        if constexpr (U::NC == 2) x[i][1] = *src(h + i, unit.c1);
      }
#pragma unroll
    for (int i = 0; i < UN; ++i)
      if (h + i < h1) {
        if (unit.turned) {
          float a[n], bb[n];
          Vec16<T>::load(x[i][0], a);
          if constexpr (U::NC == 2) Vec16<T>::load(x[i][1], bb);
          rope_turn<T, INTER, U::kPairs, n>(a, bb, cs, sn);
          x[i][0] = Vec16<T>::store(a);
          if constexpr (U::NC == 2) x[i][1] = Vec16<T>::store(bb);
        }
        *dst(h + i, unit.c0) = x[i][0];
        if constexpr (U::NC == 2) *dst(h + i, unit.c1) = x[i][1];
      }
  }
}

// ------------------------------------------------------------------ cache write
struct CacheView {
  char* k;
  char* v;
  uint8_t* ks;
  uint8_t* vs;
  long long page_bytes;       // between pages of k and of v
  int num_pages, page_shift, Hkv;
};

struct WriteParams {
  CacheView c;
  RowView k, v, q, qo;        // packed rows, bf16
  int Hq;                     // 0: no queries
  const int* cu_q;
  const int* kv_len;
  const int* table;
  int B, T, max_pages;
  const double* inv_freq;     // null: no rotation
  int rot;
  float mscale;
  int heads_per_block;
};

// Sequence of packed row t: the number of boundaries cu_q[1..B] at or below it (B: padding
// behind the last sequence).  The warp counts 32 boundaries per step, for the tokens of
// all its lanes at once: loads that do not depend on one another, where a binary search
// would wait for one after the other.
template <int LANES>          // lanes per token, consecutive
__device__ __forceinline__ int find_sequence(const int* __restrict__ cu_q, int B, int t, int lane) {
  int cnt = 0;
  for (int j0 = 0; j0 < B; j0 += 32) {
    const int e = j0 + lane < B ? cu_q[1 + j0 + lane] : 0x7fffffff;
#pragma unroll
    for (int g = 0; g < 32 / LANES; ++g) {
      const int tg = __shfl_sync(0xffffffffu, t, g * LANES);
      const unsigned m = __ballot_sync(0xffffffffu, e <= tg);
      if (lane / LANES == g) cnt += __popc(m);
    }
    if (__all_sync(0xffffffffu, __shfl_sync(0xffffffffu, e, 31) > t)) break;
  }
  return cnt;
}

// Exponent of an e4m3 row's power-of-two scale: the smallest e with amax <= 448 * 2^e
// (448 = 1.75 * 2^8), at least -127.
__device__ __forceinline__ int e4m3_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// Grid: x over blocks of tokens, y over blocks of heads; heads 0 .. Hq-1 are queries, then
// Hkv of K, then Hkv of V.  Lanes of one row are consecutive, so a row's maximum is a few
// shuffles.  Rows of one warp differ in their heads only by the loop, never by the lane.
template <int D, bool E4M3, bool INTER>
__global__ void __launch_bounds__(256) attn_cache_write_kernel(const WriteParams p) {
  using T = __nv_bfloat16;
  using U = RopeUnit<T, D, INTER>;
  constexpr int n = U::n;
  grid_dependency_wait();
  grid_dependency_launch();
  const int lane = threadIdx.x & 31;
  const int u = threadIdx.x % U::kUnits;
  const long long tok = static_cast<long long>(blockIdx.x) * (256 / U::kUnits) + threadIdx.x / U::kUnits;
  const int t = static_cast<int>(tok < p.T ? tok : p.T);       // p.T: no token (cu_q[B] <= T)
  const int b = find_sequence<U::kUnits>(p.cu_q, p.B, t, lane);
  bool live = tok < p.T && b < p.B;
  int pos = 0;
  if (live) {
    pos = max(0, p.kv_len[b]) - p.cu_q[b + 1] + t;      // a negative length counts as 0
    live = pos >= 0 && t >= p.cu_q[b];          // (rows before cu_q[0] belong to nobody)
  }
  const RopeUnit<T, D, INTER> unit(u, p.inv_freq ? p.rot : 0);
  const int h0 = blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.Hq + 2 * p.c.Hkv);
  // page and row of the token, needed for K and V heads only
  int page = -1, in_row = 0;    // -1: nowhere
  if (live && h1 > p.Hq) {
    const int pi = pos >> p.c.page_shift;
    in_row = pos & ((1 << p.c.page_shift) - 1);
    if (pi < p.max_pages) page = p.table[static_cast<long long>(b) * p.max_pages + pi];
    if (page < 0 || page >= p.c.num_pages) {
      if (u == 0) record_bad_page();
      page = -1;
    }
  }
  float cs[U::kPairs], sn[U::kPairs];
  if (live && unit.turned) rope_sincos<U::kPairs>(p.inv_freq, unit.pair0, pos, p.mscale, 0, cs, sn);
  constexpr int UN = U::NC == 2 ? 2 : 4;        // heads in flight: 64 bytes per thread
  for (int hb = h0; hb < h1; hb += UN) {
    uint4 x[UN][U::NC];
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int h = hb + k;
#pragma unroll
      for (int c = 0; c < U::NC; ++c) x[k][c] = make_uint4(0u, 0u, 0u, 0u);
      if (!live || h >= h1) continue;
      const RowView& v = h < p.Hq ? p.q : h < p.Hq + p.c.Hkv ? p.k : p.v;
      const int hh = h < p.Hq ? h : h < p.Hq + p.c.Hkv ? h - p.Hq : h - p.Hq - p.c.Hkv;
      const T* row = reinterpret_cast<const T*>(v.p) + t * v.st + hh * v.sh;
      x[k][0] = *reinterpret_cast<const uint4*>(row + unit.c0 * n);
      if constexpr (U::NC == 2) x[k][1] = *reinterpret_cast<const uint4*>(row + unit.c1 * n);
    }
#pragma unroll
    for (int k = 0; k < UN; ++k) {
      const int h = hb + k;
      if (h >= h1) break;                       // the whole block alike
      const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.c.Hkv;
      const int hh = isq ? h : isk ? h - p.Hq : h - p.Hq - p.c.Hkv;
      const bool turn = live && unit.turned && (isq || isk);
      float a[n], bb[n];
      if (E4M3 || turn) {
        Vec16<T>::load(x[k][0], a);
        if constexpr (U::NC == 2) Vec16<T>::load(x[k][1], bb);
      }
      if (turn) rope_turn<T, INTER, U::kPairs, n>(a, bb, cs, sn);
      const long long in_page = (static_cast<long long>(hh) << p.c.page_shift) + in_row;
      if (isq || !E4M3) {
        if (turn) {
          x[k][0] = Vec16<T>::store(a);
          if constexpr (U::NC == 2) x[k][1] = Vec16<T>::store(bb);
        }
        T* row = nullptr;
        if (isq && live) row = reinterpret_cast<T*>(p.qo.p) + t * p.qo.st + hh * p.qo.sh;
        else if (!isq && page >= 0) row = reinterpret_cast<T*>((isk ? p.c.k : p.c.v) + page * p.c.page_bytes) + in_page * D;
        if (row) {
          *reinterpret_cast<uint4*>(row + unit.c0 * n) = x[k][0];
          if constexpr (U::NC == 2) *reinterpret_cast<uint4*>(row + unit.c1 * n) = x[k][1];
        }
      } else {
        // the row's largest finite magnitude, over the lanes that share the row
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float m0 = fabsf(a[i]);
          amax = fmaxf(amax, m0 < INFINITY ? m0 : 0.f);
          if constexpr (U::NC == 2) {
            const float m1 = fabsf(bb[i]);
            amax = fmaxf(amax, m1 < INFINITY ? m1 : 0.f);
          }
        }
#pragma unroll
        for (int m = U::kUnits / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const int e = e4m3_exponent(amax);
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);    // 2^-e
        auto codes = [&](const float (&y)[n]) {
          return make_uint2(pack_e4m3x2(y[0] * f, y[1] * f) | (pack_e4m3x2(y[2] * f, y[3] * f) << 16),
                            pack_e4m3x2(y[4] * f, y[5] * f) | (pack_e4m3x2(y[6] * f, y[7] * f) << 16));
        };
        if (page >= 0) {
          char* row = (isk ? p.c.k : p.c.v) + page * p.c.page_bytes + in_page * D;
          *reinterpret_cast<uint2*>(row + unit.c0 * n) = codes(a);
          if constexpr (U::NC == 2) *reinterpret_cast<uint2*>(row + unit.c1 * n) = codes(bb);
          if (u == 0)
            (isk ? p.c.ks : p.c.vs)[((static_cast<long long>(page) * p.c.Hkv) << p.c.page_shift) + in_page] =
                static_cast<uint8_t>(e + 127);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ cache read
struct ReadParams {
  CacheView c;
  __nv_bfloat16* ko;
  __nv_bfloat16* vo;
  const int* kv_len;
  const int* table;
  int max_pages, N;
};

// e4m3 codes times 2^(byte - 127) as bf16, exact.  A code's exponent and mantissa fields,
// shifted to where bf16 has its own, read as a bf16 of 2^-120 times the code's value
// (subnormal codes too); the product with 2^(byte - 127 + 120) puts that right.  Two rare
// things leave this path: the NaN codes, and scales whose factor passes bf16's largest
// power (byte > 134), which takes two products.
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t prmt_b32(uint32_t a, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(a), "r"(sel));
  return r;
}
constexpr int kE4m3FastByte = 134;                         // factor 2^(byte - 7) up to 2^127
__device__ __forceinline__ uint32_t e4m3_factor(int byte) { return static_cast<uint32_t>(byte + 120) * 0x00800080u; }
// Two codes, each sign-extended to 16 bits, to those fields (sign in bit 15, the rest from
// bit 4 up).  prmt's selectors 8 + i replicate the sign of byte i.
__device__ __forceinline__ uint32_t e4m3_fields(uint32_t x) { return (x << 4) & 0x87f087f0u; }
// High bit of each byte that is a NaN code (all ones but the sign).
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t codes) { return ((codes & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// Four codes with a factor, no NaN among them.
__device__ __forceinline__ void e4m3x4_widen_fast(uint32_t codes, uint32_t f, uint32_t& w0, uint32_t& w1) {
  w0 = bf16x2_mul(e4m3_fields(prmt_b32(codes, 0x9180)), f);      // codes 0 and 1
  w1 = bf16x2_mul(e4m3_fields(prmt_b32(codes, 0xb3a2)), f);      // codes 2 and 3
}
// Any four codes under any scale byte.
__device__ __forceinline__ uint2 e4m3x4_widen_any(uint32_t codes, int byte) {
  const int more = byte > kE4m3FastByte ? byte - kE4m3FastByte : 0;
  uint32_t w[2];
  e4m3x4_widen_fast(codes, e4m3_factor(byte - more), w[0], w[1]);
  const uint32_t f2 = static_cast<uint32_t>(more + 127) * 0x00800080u, nan = e4m3_nans(codes);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (more) w[i] = bf16x2_mul(w[i], f2);
    if (nan & (0x80u << (16 * i))) w[i] |= 0x00007fc0u;
    if (nan & (0x8000u << (16 * i))) w[i] |= 0x7fc00000u;
  }
  return make_uint2(w[0], w[1]);
}
// Nonzero where one of the words has a NaN code.
template <int N>
__device__ __forceinline__ uint32_t e4m3_any_nan(const uint32_t (&codes)[N]) {
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) nan |= (codes[i] & 0x7f7f7f7fu) + 0x01010101u;
  return nan & 0x80808080u;
}
// N words of codes of one row; `rare`: a NaN code or a scale beyond kE4m3FastByte among them.
template <int N>
__device__ __forceinline__ void e4m3_widen(const uint32_t (&codes)[N], int byte, bool rare, uint32_t (&out)[2 * N]) {
  if (!rare) {
    const uint32_t f = e4m3_factor(byte);
#pragma unroll
    for (int i = 0; i < N; ++i) e4m3x4_widen_fast(codes[i], f, out[2 * i], out[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint2 w = e4m3x4_widen_any(codes[i], byte);
      out[2 * i] = w.x;
      out[2 * i + 1] = w.y;
    }
  }
}

// Grid: x over blocks of positions, y over (sequence, head).  A thread moves 16 output
// bytes of K and of V at a position, ROWS positions per pass.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) attn_cache_read_kernel(const ReadParams p) {
  constexpr int CPR = D / 8;                 // 16-byte output chunks per row
  constexpr int RPB = 256 / CPR;             // rows per pass
  constexpr int PASSES = 2;                  // e4m3, 98K positions: 105 us; 1: 114, 4: 122, 8: 209
  grid_dependency_wait();
  grid_dependency_launch();
  const int bg = blockIdx.y, b = bg / p.c.Hkv, g = bg - b * p.c.Hkv;
  const int len = min(p.kv_len[b], p.N);
  const int first = blockIdx.x * (RPB * PASSES);
  if (first >= len) return;
  const int c = threadIdx.x % CPR;
  uint4 kx[PASSES], vx[PASSES];              // e4m3: codes in x and y, the scale byte in z, at first
  int pos[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {         // all loads first
    pos[i] = first + i * RPB + threadIdx.x / CPR;
    kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
    if (pos[i] >= len) continue;
    const int pi = pos[i] >> p.c.page_shift;
    const int page = pi < p.max_pages ? p.table[static_cast<long long>(b) * p.max_pages + pi] : -1;
    if (page < 0 || page >= p.c.num_pages) {
      if (c == 0) record_bad_page();
      continue;
    }
    const long long in_page = (static_cast<long long>(g) << p.c.page_shift) + (pos[i] & ((1 << p.c.page_shift) - 1));
    const long long src = page * p.c.page_bytes + in_page * (E4M3 ? D : 2 * D);
    if constexpr (E4M3) {
      const long long at = ((static_cast<long long>(page) * p.c.Hkv) << p.c.page_shift) + in_page;
      const uint2 kc = *reinterpret_cast<const uint2*>(p.c.k + src + c * 8);
      const uint2 vc = *reinterpret_cast<const uint2*>(p.c.v + src + c * 8);
      kx[i] = make_uint4(kc.x, kc.y, p.c.ks[at], 0u);
      vx[i] = make_uint4(vc.x, vc.y, p.c.vs[at], 0u);
    } else {
      kx[i] = *reinterpret_cast<const uint4*>(p.c.k + src + c * 16);
      vx[i] = *reinterpret_cast<const uint4*>(p.c.v + src + c * 16);
    }
  }
  if constexpr (E4M3) {
    auto widen = [](uint4& x) {
      const uint32_t codes[2] = {x.x, x.y};
      const int byte = static_cast<int>(x.z);
      uint32_t y[4];
      e4m3_widen<2>(codes, byte, byte > kE4m3FastByte || e4m3_any_nan<2>(codes), y);
      x = make_uint4(y[0], y[1], y[2], y[3]);
    };
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      widen(kx[i]);
      widen(vx[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (pos[i] >= len) continue;
    const long long o = (static_cast<long long>(bg) * p.N + pos[i]) * D + c * 8;
    *reinterpret_cast<uint4*>(p.ko + o) = kx[i];
    *reinterpret_cast<uint4*>(p.vo + o) = vx[i];
  }
}

}  // namespace attn
