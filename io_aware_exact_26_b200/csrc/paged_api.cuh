// Host side of include/attn_paged.h: validation, tensor maps and launches of the serving
// operators.  Included by api.cu, whose device query, alignment test and encoder it uses.
#pragma once
#include "attn_paged.h"
#include "paged_few.cuh"
#include "paged_pair.cuh"
#include "paged_rows.cuh"

namespace {

bool stride_ok(const attn_strides_t* s, int elem, bool batch) {
  auto ok = [&](long long x) { return x >= 0 && (x * elem) % 16 == 0 && x < (1ll << 38); };
  return s && ok(s->head) && ok(s->token) && (!batch || ok(s->batch));
}

attn::RowView row_view(const void* p, const attn_strides_t* s) {
  return {static_cast<char*>(const_cast<void*>(p)), s ? s->batch : 0, s ? s->head : 0, s ? s->token : 0};
}

int check_rope(const attn_rope_t* r, int d) {
  if (!r->inv_freq || r->rot < 16 || r->rot > d || r->rot % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if ((r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->mscale)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(r->inv_freq)) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

int check_cache(const attn_cache_t* c) {
  if (!c) return ATTN_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->dtype != ATTN_BF16 && c->dtype != ATTN_E4M3) return ATTN_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->Hkv > 65535) return ATTN_ERR_INVALID_ARG;
  const long long page = static_cast<long long>(c->Hkv) * c->page_size * c->d;
  const int elem = c->dtype == ATTN_BF16 ? 2 : 1;
  if (c->page_stride < page || c->page_stride >= (1ll << 38) || (c->page_stride * elem) % 16 != 0)
    return ATTN_ERR_INVALID_ARG;
  if (!c->k || !c->v || (c->dtype == ATTN_E4M3 && (!c->k_scale || !c->v_scale))) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return ATTN_ERR_ALIGNMENT;
  if (c->dtype == ATTN_E4M3 && (!aligned16(c->k_scale) || !aligned16(c->v_scale))) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

// int32 arrays: any 4-byte alignment will do (they are read word by word)
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_batch(const attn_batch_t* b, bool packed) {
  if (!b || b->B < 1 || b->max_pages < 1 || !b->kv_len || !b->block_table) return ATTN_ERR_INVALID_ARG;
  if (packed && (b->T < 0 || !b->cu_q)) return ATTN_ERR_INVALID_ARG;
  if (!aligned4(b->kv_len) || !aligned4(b->block_table) || (packed && !aligned4(b->cu_q))) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

attn::CacheView cache_view(const attn_cache_t* c) {
  attn::CacheView v;
  v.k = static_cast<char*>(c->k);
  v.v = static_cast<char*>(c->v);
  v.ks = static_cast<uint8_t*>(c->k_scale);
  v.vs = static_cast<uint8_t*>(c->v_scale);
  v.page_bytes = c->page_stride * (c->dtype == ATTN_BF16 ? 2 : 1);
  v.num_pages = c->num_pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  v.Hkv = c->Hkv;
  return v;
}

// Launch with programmatic stream serialisation: the kernel may be set up while the one
// before it runs, and waits for it on the device (griddepcontrol.wait).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Heads that one block walks through: all of them where the tokens alone fill the GPU
// (sine and cosine are then formed once per token), else few enough that the blocks do.
int heads_per_block(long long token_blocks, int heads, int sms) {
  const long long want = 8LL * sms;                       // blocks of 256 threads
  long long split = (want + token_blocks - 1) / token_blocks;
  if (split > heads) split = heads;
  return static_cast<int>((heads + split - 1) / split);
}

template <typename T, int D, bool INTER>
cudaError_t launch_rope(const attn::RopeParams& p0, int sms, cudaStream_t s) {
  attn::RopeParams p = p0;
  constexpr int tpb = 256 / attn::RopeUnit<T, D, INTER>::kUnits;
  const long long tb = (static_cast<long long>(p.B) * p.N + tpb - 1) / tpb;
  p.heads_per_block = heads_per_block(tb, p.Hq + p.Hk, sms);
  const dim3 grid(static_cast<unsigned>(tb), (p.Hq + p.Hk + p.heads_per_block - 1) / p.heads_per_block);
  return launch_pdl(attn::attn_rope_kernel<T, D, INTER>, grid, 256, 0, s, p);
}

template <int D, bool E4M3, bool INTER>
cudaError_t launch_cache_write(const attn::WriteParams& p0, int sms, cudaStream_t s) {
  attn::WriteParams p = p0;
  constexpr int tpb = 256 / attn::RopeUnit<__nv_bfloat16, D, INTER>::kUnits;
  const long long tb = (static_cast<long long>(p.T) + tpb - 1) / tpb;
  const int heads = p.Hq + 2 * p.c.Hkv;
  p.heads_per_block = heads_per_block(tb, heads, sms);
  const dim3 grid(static_cast<unsigned>(tb), (heads + p.heads_per_block - 1) / p.heads_per_block);
  return launch_pdl(attn::attn_cache_write_kernel<D, E4M3, INTER>, grid, 256, 0, s, p);
}

template <int D, bool E4M3>
cudaError_t launch_cache_read(const attn::ReadParams& p, int B, cudaStream_t s) {
  constexpr int rows = 256 / (D / 8) * 2;
  const dim3 grid((p.N + rows - 1) / rows, static_cast<unsigned>(B * p.c.Hkv));
  return launch_pdl(attn::attn_cache_read_kernel<D, E4M3>, grid, 256, 0, s, p);
}

// [num_pages][Hkv][page_size][d] as a 4-D map; one box is a page's (or 128 rows of it)
// 64 bf16 columns, swizzled as the MMAs read them, or all e4m3 columns (swizzled at d = 128,
// where a row is one 128-byte line, so that the widening warps read without conflicts).
// `pad`: e4m3 boxes of 128 columns whatever d is (zeros behind the row), swizzled, as the
// tensor cores read 8-bit tiles.
bool make_cache_map(CUtensorMap* m, const void* ptr, const attn_cache_t* c, bool pad = false) {
  auto enc = encode_fn();
  if (!enc) return false;
  const int elem = c->dtype == ATTN_BF16 ? 2 : 1;
  const cuuint64_t row = static_cast<cuuint64_t>(c->d) * elem;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                        static_cast<cuuint64_t>(c->Hkv), static_cast<cuuint64_t>(c->num_pages)};
  cuuint64_t strides[3] = {row, row * c->page_size, static_cast<cuuint64_t>(c->page_stride) * elem};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(elem == 2 ? 64 : pad ? 128 : c->d),
                       static_cast<cuuint32_t>(c->page_size < 128 ? c->page_size : 128), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
             const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             row >= 128 || pad ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T][Hq][d] as a 3-D map; a box is 64 columns of G heads of R tokens: rows i * G + h of a tile.
bool make_q_map(CUtensorMap* m, const void* q, const attn_strides_t* st, int T, int Hq, int d, int G, int R) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T)};
  // a stride that no element uses (one head, one token) may be anything: give a plain one
  const long long head = Hq > 1 ? st->head : d, token = T > 1 ? st->token : static_cast<long long>(Hq) * d;
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(R)};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows up to which the kernel for few rows is taken.  Its softmax grows with the rows, that
// of the 128-row kernel does not; but the latter takes longer per tile than a tile's bytes
// where those are few (d = 64), and longer still where it has to widen K (e4m3).  Few rows
// against the 128-row kernel, us, 16 sequences of 8K at 4 heads to 8, and 32 of 512:
//   bf16, d = 128:  8 rows 77 : 73, 24 : 21;  32 rows 143 : 75, 71 : 25;  4 rows 20 : 25 at 32 of 512
//   bf16, d = 64:   8 rows 52 : 64, 24 : 20;  16 rows 69 : 64, 35 : 22
//   e4m3, d = 64:   8 rows 57 : 78, 33 : 24;  16 rows 93 : 77, 51 : 28
//   e4m3, d = 128:  16 rows 92 : 119, 48 : 34;  32 rows 147 : 121, 79 : 37
// The other side is the faster one past these limits on long caches of one query head to
// a cache head (d = 64, 16 tokens on 65K: bf16 176 : 238; e4m3, d = 128, 32 tokens: 338 : 455).
constexpr int few_rows_limit(int d, bool kv8) { return d == 64 ? 8 : kv8 ? 16 : 4; }

// Query rows per item, by the batch's mean: the smallest build of the kernel for few rows
// that takes a sequence's rows, else 128, or 256 (two tiles, bf16 cache) where a sequence has
// more than one tile's.  Any form is right for any lengths.
int paged_form(int T, int B, int G, int d, int dtype) {
  const long long rows = static_cast<long long>(G) * ((T + B - 1) / B);
  if (rows <= few_rows_limit(d, dtype == ATTN_E4M3)) return rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  return rows <= 128 || dtype == ATTN_E4M3 ? 128 : 256;
}

// Workspace of the cut items: descriptors, LSE of the parts, then their O (fp32).
struct PagedWs {
  int slot_rows;
  size_t l_off, o_off, total;
};
PagedWs paged_ws(int T, int G, int form, int d, int sms) {
  PagedWs w;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const long long R = form == 256 ? 2 * (128 / G) : form / G;      // tokens of an item
  w.slot_rows = static_cast<int>((T < R ? T : R) * G);
  w.l_off = up(sizeof(attn::PagedCut) * sms);
  w.o_off = up(w.l_off + static_cast<size_t>(2) * sms * w.slot_rows * 4);
  w.total = up(w.o_off + static_cast<size_t>(2) * sms * w.slot_rows * d * 4);
  return w;
}

int check_paged_heads(int T, int B, int Hq, int Hkv, int d) {
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (T < 0 || B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 128) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * Hq >= (1ll << 38)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// C: the kernel's configuration.
template <class C, typename Kernel>
int launch_paged(Kernel kernel, const void* q, const attn_strides_t* q_strides, const attn_cache_t* cache,
                 const attn::PagedParams& p, cudaStream_t stream) {
  static std::once_flag attr_once[64];
  static bool attr_ok[64];
  int dev = 0;
  cudaGetDevice(&dev);
  std::call_once(attr_once[dev], [&] {
    attr_ok[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) == cudaSuccess;
  });
  if (!attr_ok[dev]) return ATTN_ERR_LAUNCH;
  CUtensorMap tq, tk, tv;
  if (!make_q_map(&tq, q, q_strides, p.T, p.Hq, cache->d, p.G, p.R) || !make_cache_map(&tk, cache->k, cache, C::K8) ||
      !make_cache_map(&tv, cache->v, cache))
    return ATTN_ERR_LAUNCH;
  if (launch_pdl(kernel, dim3(p.ctas), C::kThreads, C::kSmem, stream, tq, tk, tv, p) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  const dim3 grid(p.ctas, (p.slot_rows + 15) / 16);       // two rows to a warp at most
  if (launch_pdl(attn::attn_paged_merge_kernel<C::D>, grid, 256, 0, stream, p) != cudaSuccess) return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

template <int D, bool KV8>
int launch_paged_form(int form, const void* q, const attn_strides_t* q_strides, const attn_cache_t* cache,
                      const attn::PagedParams& p, cudaStream_t s) {
#define ATTN_FEW(NR) \
  if constexpr (NR <= few_rows_limit(D, KV8)) { \
    if (form == NR) \
      return launch_paged<attn::FewCfg<D, KV8, NR>>(attn::attn_paged_few_kernel<D, KV8, NR>, q, q_strides, cache, p, s); \
  }
  ATTN_FEW(4)
  ATTN_FEW(8)
  ATTN_FEW(16)
#undef ATTN_FEW
  if constexpr (!KV8) {
    if (form == 256)
      return launch_paged<attn::PairCfg<D>>(attn::attn_paged_pair_kernel<D>, q, q_strides, cache, p, s);
  }
  return launch_paged<attn::RowsCfg<D, KV8>>(attn::attn_paged_rows_kernel<D, KV8>, q, q_strides, cache, p, s);
}

}  // namespace

extern "C" {

int attn_rope(const void* q, const attn_strides_t* q_strides, void* q_out, const attn_strides_t* q_out_strides, int Hq,
              const void* k, const attn_strides_t* k_strides, void* k_out, const attn_strides_t* k_out_strides, int Hkv,
              int dtype, int B, int N, int d, const int* positions, long long pos_batch_stride,
              const attn_rope_t* rope, int inverse, void* stream) {
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (dtype != ATTN_BF16 && dtype != ATTN_F32) return ATTN_ERR_INVALID_ARG;
  if (!rope || Hq < 1 || B < 0 || N < 0 || (k && Hkv < 1)) return ATTN_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return ATTN_ERR_INVALID_ARG;
  if (pos_batch_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  const int elem = dtype == ATTN_BF16 ? 2 : 4;
  if (!stride_ok(q_strides, elem, true) || !stride_ok(q_out_strides, elem, true)) return ATTN_ERR_INVALID_ARG;
  if (k && (!stride_ok(k_strides, elem, true) || !stride_ok(k_out_strides, elem, true))) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(Hq) + (k ? Hkv : 0) > 65535) return ATTN_ERR_INVALID_ARG;
  const int st = check_rope(rope, d);
  if (st != ATTN_OK) return st;
  if (B == 0 || N == 0) return ATTN_OK;
  if (!q || !q_out || !positions || (k && !k_out)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || (k && (!aligned16(k) || !aligned16(k_out))) || !aligned4(positions))
    return ATTN_ERR_ALIGNMENT;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != 0) return ATTN_ERR_UNSUPPORTED;
  attn::RopeParams p;
  p.q = row_view(q, q_strides);
  p.qo = row_view(q_out, q_out_strides);
  p.k = row_view(k, k ? k_strides : nullptr);
  p.ko = row_view(k ? k_out : nullptr, k ? k_out_strides : nullptr);
  p.Hq = Hq;
  p.Hk = k ? Hkv : 0;
  p.B = B;
  p.N = N;
  p.pos = positions;
  p.pos_sb = pos_batch_stride;
  p.inv_freq = rope->inv_freq;
  p.rot = rope->rot;
  p.inverse = inverse;
  p.mscale = rope->mscale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](auto tag, auto dim) {
    using T = decltype(tag);
    constexpr int D = decltype(dim)::value;
    return rope->interleaved ? launch_rope<T, D, true>(p, di->sms, s) : launch_rope<T, D, false>(p, di->sms, s);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const cudaError_t e = dtype == ATTN_BF16 ? (d == 64 ? go(__nv_bfloat16(), D64()) : go(__nv_bfloat16(), D128()))
                                           : (d == 64 ? go(0.f, D64()) : go(0.f, D128()));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int attn_cache_write(const attn_cache_t* cache, const attn_batch_t* batch, const void* k,
                     const attn_strides_t* k_strides, const void* v, const attn_strides_t* v_strides,
                     const attn_rope_t* rope, const void* q, const attn_strides_t* q_strides, void* q_out,
                     const attn_strides_t* q_out_strides, int Hq, void* stream) {
  int st = check_cache(cache);
  if (st == ATTN_OK) st = check_batch(batch, true);
  if (st == ATTN_OK && rope) st = check_rope(rope, cache->d);
  if (st != ATTN_OK) return st;
  if (batch->T == 0) return ATTN_OK;
  if (!k || !v || !stride_ok(k_strides, 2, false) || !stride_ok(v_strides, 2, false)) return ATTN_ERR_INVALID_ARG;
  if (q && (!rope || !q_out || Hq < 1 || !stride_ok(q_strides, 2, false) || !stride_ok(q_out_strides, 2, false)))
    return ATTN_ERR_INVALID_ARG;
  const long long heads = (q ? static_cast<long long>(Hq) : 0) + 2LL * cache->Hkv;
  if (heads > 65535) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out)))) return ATTN_ERR_ALIGNMENT;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != 0) return ATTN_ERR_UNSUPPORTED;
  attn::WriteParams p;
  p.c = cache_view(cache);
  p.k = row_view(k, k_strides);
  p.v = row_view(v, v_strides);
  p.q = row_view(q, q ? q_strides : nullptr);
  p.qo = row_view(q ? q_out : nullptr, q ? q_out_strides : nullptr);
  p.Hq = q ? Hq : 0;
  p.cu_q = batch->cu_q;
  p.kv_len = batch->kv_len;
  p.table = batch->block_table;
  p.B = batch->B;
  p.T = batch->T;
  p.max_pages = batch->max_pages;
  p.inv_freq = rope ? rope->inv_freq : nullptr;
  p.rot = rope ? rope->rot : 0;
  p.mscale = rope ? rope->mscale : 1.f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = rope && rope->interleaved, e4m3 = cache->dtype == ATTN_E4M3;
  auto go = [&](auto dim, auto eight) {
    constexpr int D = decltype(dim)::value;
    constexpr bool E = decltype(eight)::value;
    return inter ? launch_cache_write<D, E, true>(p, di->sms, s) : launch_cache_write<D, E, false>(p, di->sms, s);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const cudaError_t e = cache->d == 64 ? (e4m3 ? go(D64(), std::true_type()) : go(D64(), std::false_type()))
                                       : (e4m3 ? go(D128(), std::true_type()) : go(D128(), std::false_type()));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

int attn_cache_read(const attn_cache_t* cache, const attn_batch_t* batch, void* k_out, void* v_out, int N,
                    void* stream) {
  int st = check_cache(cache);
  if (st == ATTN_OK) st = check_batch(batch, false);
  if (st != ATTN_OK) return st;
  if (N < 0 || N > (1 << 30)) return ATTN_ERR_INVALID_ARG;
  if (N == 0) return ATTN_OK;
  if (!k_out || !v_out) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(batch->B) * cache->Hkv > 65535) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return ATTN_ERR_ALIGNMENT;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != 0) return ATTN_ERR_UNSUPPORTED;
  attn::ReadParams p;
  p.c = cache_view(cache);
  p.ko = static_cast<__nv_bfloat16*>(k_out);
  p.vo = static_cast<__nv_bfloat16*>(v_out);
  p.kv_len = batch->kv_len;
  p.table = batch->block_table;
  p.max_pages = batch->max_pages;
  p.N = N;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == ATTN_E4M3;
  const cudaError_t e =
      cache->d == 64
          ? (e4m3 ? launch_cache_read<64, true>(p, batch->B, s) : launch_cache_read<64, false>(p, batch->B, s))
          : (e4m3 ? launch_cache_read<128, true>(p, batch->B, s) : launch_cache_read<128, false>(p, batch->B, s));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

size_t attn_paged_workspace_size(int T, int B, int Hq, int Hkv, int d) {
  if (check_paged_heads(T, B, Hq, Hkv, d) != ATTN_OK || T == 0) return 0;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != 0) return 0;
  // enough for either cache type
  const int G = Hq / Hkv;
  const size_t a = paged_ws(T, G, paged_form(T, B, G, d, ATTN_BF16), d, di->sms).total;
  const size_t b = paged_ws(T, G, paged_form(T, B, G, d, ATTN_E4M3), d, di->sms).total;
  return a > b ? a : b;
}

int attn_paged(const void* q, const attn_strides_t* q_strides, const attn_cache_t* cache, const attn_batch_t* batch,
               void* o, float* lse, int Hq, float scale, int causal, int window_left, void* workspace,
               size_t workspace_bytes, void* stream) {
  int st = check_cache(cache);
  if (st == ATTN_OK) st = check_batch(batch, true);
  if (st == ATTN_OK) st = check_paged_heads(batch->T, batch->B, Hq, cache->Hkv, cache->d);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale) || scale < 0.f || (causal != 0 && causal != 1)) return ATTN_ERR_INVALID_ARG;
  if (batch->T == 0) return ATTN_OK;
  if (!q || !o || !lse || !stride_ok(q_strides, 2, false)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse)) return ATTN_ERR_ALIGNMENT;
  if (workspace && !aligned16(workspace)) return ATTN_ERR_ALIGNMENT;
  DeviceInfo* di = nullptr;
  if (device_info(&di) != 0) return ATTN_ERR_UNSUPPORTED;
  const int d = cache->d, G = Hq / cache->Hkv;
  const int form = paged_form(batch->T, batch->B, G, d, cache->dtype);
  const PagedWs W = paged_ws(batch->T, G, form, d, di->sms);
  if (workspace && workspace_bytes < W.total) return ATTN_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = workspace;
  if (!ws && cudaMallocAsync(&ws, W.total, s) != cudaSuccess) {
    (void)cudaGetLastError();
    return ATTN_ERR_ALLOC;
  }
  attn::PagedParams p;
  p.c = cache_view(cache);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cu_q = batch->cu_q;
  p.kv_len = batch->kv_len;
  p.table = batch->block_table;
  p.B = batch->B;
  p.T = batch->T;
  p.max_pages = batch->max_pages;
  p.Hq = Hq;
  p.Hkv = cache->Hkv;
  p.G = G;
  p.R = (form == 256 ? 128 : form) / G;
  p.RI = form == 256 ? 2 * p.R : p.R;
  p.causal = causal;
  p.wl = window_left < 0 ? -1 : window_left < (1 << 30) ? window_left : 1 << 30;
  // A part of a few rows costs little; parts of a whole tile's rows are worth it from 13 key
  // tiles on (a 1000-token prompt: 51 us with every item cut where the shares meet, 33 so).
  p.whole = form <= 16 ? 0 : 12;
  p.cs = attn::folded_scale(scale);
  p.ctas = di->sms;
  p.slot_rows = W.slot_rows;
  p.cuts = static_cast<attn::PagedCut*>(ws);
  p.lpart = reinterpret_cast<float*>(static_cast<char*>(ws) + W.l_off);
  p.opart = reinterpret_cast<float*>(static_cast<char*>(ws) + W.o_off);
  int st2;
  if (cache->dtype == ATTN_E4M3)
    st2 = d == 64 ? launch_paged_form<64, true>(form, q, q_strides, cache, p, s)
                  : launch_paged_form<128, true>(form, q, q_strides, cache, p, s);
  else
    st2 = d == 64 ? launch_paged_form<64, false>(form, q, q_strides, cache, p, s)
                  : launch_paged_form<128, false>(form, q, q_strides, cache, p, s);
  if (!workspace && cudaFreeAsync(ws, s) != cudaSuccess) {
    (void)cudaGetLastError();
    return st2 != ATTN_OK ? st2 : ATTN_ERR_ALLOC;
  }
  return st2;
}

}  // extern "C"
