/* attn_paged.h -- C ABI of the serving operators of libattn_b200.so: rotary positions,
 * a paged K/V cache (write, read back) and attention of new tokens over that cache.
 *
 * The conventions of attn.h hold: device pointers on the current CUDA device, 16-byte
 * aligned, owned by the caller; work is enqueued on `stream` and the call returns
 * without waiting; arguments are checked on the host before any launch and a rejected
 * call launches nothing and returns a negative attn_status_t; nothing aborts, traps or
 * throws.  d is 64 or 128 throughout.  None of these calls keeps state between calls,
 * so they may run at once on any streams, as long as each has its own workspace.
 *
 * Sequences and tokens.  A call handles B sequences.  The new tokens of all of them are
 * packed: T rows, sequence b owning rows cu_q[b] .. cu_q[b+1] - 1 (int32, B + 1 entries,
 * not decreasing, cu_q[B] <= T).  kv_len[b] (int32) counts the sequence's tokens in the
 * cache, the new ones included, so the new token in row t of sequence b has position
 *     pos = kv_len[b] - cu_q[b+1] + t.
 * A sequence may have no new token, or one (decoding), or many (a prompt's chunk), in
 * the same call.  Rows before cu_q[0] and from cu_q[B] on (padding) are left alone.
 *
 * Pages.  The cache is a pool of num_pages pages of page_size positions (16, 32, 64, 128
 * or 256), shared by all sequences: position p of sequence b lies in row p % page_size of
 * page block_table[b * max_pages + p / page_size] (int32).  Only the table entries that
 * cover positions below kv_len[b] (attn_paged: that some row sees) are followed; the others
 * may hold anything.  An entry outside [0, num_pages), or a position beyond max_pages pages,
 * is never followed: the write of that token is skipped, reads see zeros there, attention
 * takes the sequence as max_pages pages long, and attn_get_device_status() reports
 * ATTN_ERR_DEVICE_PAGE once the work has run (not for a sequence without new tokens, which
 * the write and the attention pass over).  kv_len is below 2^30; a negative one counts as 0.
 */
#ifndef ATTN_B200_PAGED_H
#define ATTN_B200_PAGED_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ERR_DEVICE_PAGE (-10) /* a block table entry or a position was outside the page pool */

typedef enum { ATTN_BF16 = 0, ATTN_F32 = 1, ATTN_E4M3 = 2 } attn_dtype_t;

/* A paged K/V cache.
 *   k, v : bf16 or e4m3 [num_pages][Hkv][page_size][d]; consecutive pages lie page_stride
 *          elements apart (>= Hkv * page_size * d, a multiple of 16 bytes), so k and v may
 *          be interleaved page by page in one buffer.
 *   k_scale, v_scale : e4m3 only (NULL for bf16): uint8 [num_pages][Hkv][page_size], one
 *          power of two per token and head in E8M0 form: the cached row stands for
 *          code * 2^(byte - 127). */
typedef struct {
  void* k;
  void* v;
  void* k_scale;
  void* v_scale;
  long long page_stride;
  int num_pages, page_size, Hkv, d;
  int dtype;                     /* ATTN_BF16 or ATTN_E4M3 */
} attn_cache_t;

/* The sequences of a call; see the head of this file. */
typedef struct {
  const int* cu_q;               /* [B + 1] */
  const int* kv_len;             /* [B] */
  const int* block_table;        /* [B][max_pages] */
  int B, T, max_pages;
} attn_batch_t;

/* Rotary positions.  Of each row of d values the first `rot` are rot / 2 pairs; pair i is
 * turned by the angle pos * inv_freq[i] and multiplied by mscale, the rest is copied:
 *     a' = m (a cos - b sin),  b' = m (b cos + a sin),
 * with (a, b) = (x[i], x[i + rot/2]), or (x[2i], x[2i+1]) if interleaved.  The angle is
 * formed and reduced in fp64, so that it is off by at most 2^-26 of a turn and
 * 3 * 2^-53 of its own size (together 2^-24 of a turn up to 2^27 turns: 1 radian per
 * position up to position 8.4e8); sine, cosine and the rotation are fp32, rounded once at
 * the end.
 *   inv_freq : fp64 [rot / 2], radians per position (scaled for long contexts as the
 *              caller likes: any frequencies are taken)
 *   rot      : a multiple of 16, 16 <= rot <= d
 *   mscale   : finite */
typedef struct {
  const double* inv_freq;
  int rot;
  int interleaved;
  float mscale;
} attn_rope_t;

/* Strides of a [batch][head][token][d] tensor, in elements (d is contiguous); each a
 * multiple of 16 bytes.  A packed [T][H][d] tensor has one batch entry. */
typedef struct {
  long long batch, head, token;
} attn_strides_t;

/* q_out = rope(q) and, unless k is NULL, k_out = rope(k), for B batch entries of N tokens.
 *   dtype     : ATTN_BF16 or ATTN_F32, of all four tensors
 *   positions : int32; token n of batch entry b has positions[b * pos_batch_stride + n]
 *               (pos_batch_stride 0: one row for all)
 *   inverse   : 0 = the rotation; 1 = its transpose, which maps the gradient of the
 *               outputs to the gradient of the inputs (mscale applies to both)
 * q_out may be q and k_out may be k (same strides); otherwise inputs and outputs must not
 * overlap.  B * N is below 2^31, Hq + Hkv at most 65535.  One kernel. */
int attn_rope(const void* q, const attn_strides_t* q_strides, void* q_out, const attn_strides_t* q_out_strides, int Hq,
              const void* k, const attn_strides_t* k_strides, void* k_out, const attn_strides_t* k_out_strides, int Hkv,
              int dtype, int B, int N, int d, const int* positions, long long pos_batch_stride,
              const attn_rope_t* rope, int inverse, void* stream);

/* Write the new tokens' K and V rows into the cache: row t of sequence b goes to position
 * kv_len[b] - cu_q[b+1] + t (rows whose position is negative are skipped).
 *   k, v : bf16, packed: row t, head h starts at t * token + h * head (`batch` is ignored)
 *   rope : NULL, or the rotation applied to K on its way, by each token's position
 *   q, q_out : with rope only, and optional (NULL): bf16 queries [T][Hq][d] rotated by the
 *          same positions into q_out (q_out may be q)
 * A bf16 cache takes the rows as they are (rotated rows rounded once).  An e4m3 cache
 * takes code = round-to-nearest-even(x * 2^-e) with e the smallest exponent that brings
 * the row's largest finite magnitude to at most 448 (-127 <= e <= 120) and e + 127 as the
 * scale byte; rotated rows are quantised from fp32.  Infinities become +-448, NaN stays.
 * Two tokens of one call must not share a cache row.  Rows of the pages that no token
 * maps to keep their contents.  Hq + 2 Hkv is at most 65535.  One kernel. */
int attn_cache_write(const attn_cache_t* cache, const attn_batch_t* batch,
                     const void* k, const attn_strides_t* k_strides, const void* v, const attn_strides_t* v_strides,
                     const attn_rope_t* rope, const void* q, const attn_strides_t* q_strides,
                     void* q_out, const attn_strides_t* q_out_strides, int Hq, void* stream);

/* Read the cache back: for every sequence the positions [0, min(kv_len[b], N)) of K and V
 * to k_out, v_out : bf16 [B][Hkv][N][d] -- the layout of attn_fwd and attn_decode.  Rows
 * behind a sequence's length keep their contents.  e4m3 rows become code * 2^(byte - 127),
 * which bf16 holds exactly (down to its subnormals).  batch->cu_q is not used and may be
 * NULL.  B * Hkv is at most 65535 and N at most 2^30.  One kernel. */
int attn_cache_read(const attn_cache_t* cache, const attn_batch_t* batch, void* k_out, void* v_out, int N, void* stream);

/* Attention of the new tokens over the cache (which holds their own K and V too):
 *   o[t][h] = softmax(scale * q[t][h] K^T) V over the keys j of the token's sequence with
 *     j < kv_len[b],  j <= pos if causal,  j >= pos - window_left if window_left >= 0
 *   lse[t][h] = natural log of the sum of exp(scale * q . k_j) over those keys
 * A row that sees no key gets o = 0 and lse = -inf.
 *   q : bf16, row t, head h at t * token + h * head;  o : bf16 [T][Hq][d] and
 *   lse : fp32 [T][Hq], contiguous.  Hq is a multiple of Hkv with Hq / Hkv <= 128; query
 *   head h reads KV head h / (Hq / Hkv).
 * Both products run on the tensor cores with bf16 operands (e4m3 rows are widened on
 * chip, which is exact), but for few query rows over an e4m3 cache: there K is multiplied
 * as it lies, by Q in four e4m3 parts, which hold a query value exactly down to 2^-35 of
 * its row's largest magnitude and to 2^-43 of that magnitude below.  Sums and softmax
 * statistics are fp32; P is rounded to bf16.
 * Masked scores never reach the sums, whatever the cache holds there; values of V at
 * positions below kv_len[b] have to be finite in every 128-key tile that some row of the
 * sequence sees.  A row that sees a NaN score or one of +infinity is NaN; so may be a row
 * with an infinite query value.
 * The cache rows of this call's tokens must have been written before, on this stream or
 * ordered before it.
 * The keys are shared out evenly over the SMs by each CTA from cu_q and kv_len on the
 * device, so one captured launch serves any lengths; results do not depend on which SM
 * runs first, and equal calls give equal bits.
 * Lengths being on the device, the host picks one of three kernels by the mean of query
 * rows per sequence, Hq / Hkv * T / B, with T counting padding and B counting sequences
 * without new tokens.  Any of them is right for any batch, but one for few rows takes a long
 * chunk a few rows at a time: 256 sequences of which one has 256 new tokens over 4096 (32
 * query heads to 8, d = 128, bf16) take 263 us, that one alone 47.  Where long chunks meet
 * mostly empty or padded slots, leave those slots out or give the chunks their own call.
 * Workspace: attn_paged_workspace_size(...) bytes (queried with the same device current;
 * it does not depend on lengths), or NULL: the library takes it with cudaMallocAsync /
 * cudaFreeAsync on `stream`.  It is overwritten; calls that may overlap need one each.
 * Two kernels: the attention, and the merge of rows whose keys were shared out. */
size_t attn_paged_workspace_size(int T, int B, int Hq, int Hkv, int d);
int attn_paged(const void* q, const attn_strides_t* q_strides, const attn_cache_t* cache, const attn_batch_t* batch,
               void* o, float* lse, int Hq, float scale, int causal, int window_left,
               void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_B200_PAGED_H */
