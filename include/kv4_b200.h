/*
 * kv4_b200.h - C ABI of the 4-bit key/value cache and the attention over it, of
 * the same library (libattn_b200.so), for NVIDIA B200.
 *
 * For serving, next to the dense calls of attn_b200.h: the keys and values of
 * running sequences are kept in pages at 4.5 bits a value, new tokens are
 * quantised as they are written, and queries (one token of each sequence, a
 * few, or a long chunk) attend over the cache without it ever being expanded in
 * memory. (The pages the library follows define 4-bit weights and the block
 * formats; the cache applies the same block idea to keys and values.)
 *
 * Format. Each row (one token of one key/value head, d values) is cut into blocks
 * of 16 consecutive values. With e one integer per tensor (k_exp, v_exp):
 *     y    = x * 2^-e
 *     s    = E4M3 round-to-nearest-even of max|y| / 6, clamped to [2^-9, 448]
 *     code = E2M1 round-to-nearest-even, saturating, of y / s
 *     value read back = code * s * 2^e
 * (quotients in fp32, correctly rounded). E2M1 holds 0, 0.5, 1, 1.5, 2, 3, 4, 6
 * and their negatives: code bit 3 is the sign (that of x, for zeros too), bits 0-2 the index in that list.
 * An infinite value saturates; a block that holds a NaN gets scale byte 0x7F
 * (NaN) and reads back as NaN.
 *
 * Cache tensors (device memory owned by the caller, 16-byte aligned, dense):
 *   k_codes, v_codes : [num_pages, Hkv, page_size, d / 2] bytes; byte j of a row holds
 *                      the codes of values 2 j (low nibble) and 2 j + 1.
 *   k_sf, v_sf       : [num_pages, Hkv, page_size, d / 16] E4M3 scale bytes.
 *   block_table      : [B, max_pages] int32; position p of sequence b lies in page
 *                      block_table[b, p / page_size], slot p % page_size.
 *   seq_lens         : [B] int32 tokens of each sequence in the cache, 0 or more.
 * page_size is a power of two from 16 to 65536 (else ATTN_ERR_UNSUPPORTED); max_pages * page_size <= 2^30;
 * num_pages * Hkv * page_size < 2^32; d is 64 or 128 (else ATTN_ERR_UNSUPPORTED);
 * |k_exp|, |v_exp| <= 32. dtype (of k, v, q, o) is ATTN_BF16 or ATTN_FP16.
 *
 * The contents of block_table, seq_lens, new_lens, starts and q_lens cannot be
 * checked on the host. The kernels check them: a page number outside
 * [0, num_pages), a length that is negative or beyond its limit (max_pages *
 * page_size, or N) skips the access, counts as length clamped to that range, and
 * records ATTN_ERR_BOUNDS in the device status word (in release builds too),
 * read by attn_get_device_status(). The outputs of such a call are undefined
 * where they depend on the skipped entries.
 * Slots that no position of a sequence maps to are never interpreted: they may
 * hold anything, NaN patterns included.
 * The int32 arrays need 4-byte alignment only (they may be slices of larger ones).
 * Asynchronous on `stream`; nothing is allocated; other conventions and errors
 * as in attn_b200.h.
 */
#ifndef KV4_B200_H
#define KV4_B200_H

#include "attn_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache: its tensors and sizes, as every call takes them (a host struct, read during the call). */
typedef struct {
  void* k_codes;             /* device pointers */
  void* k_sf;
  void* v_codes;
  void* v_sf;
  int num_pages, page_size, Hkv, d;
  int k_exp, v_exp;
} attn_kv4_cache;

/*
 * attn_kv4_append - quantises new keys and values into the cache.
 *   k, v     : [B, Hkv, N, d] new tokens of each sequence.
 *   seq_lens : lengths AFTER this call (the array attn_fwd_kv4 takes next): token
 *              i < new_lens[b] is written at position seq_lens[b] - new_lens[b] + i.
 *   new_lens : [B] int32, 0 <= new_lens[b] <= min(N, seq_lens[b]), or NULL for N new
 *              tokens each; rows behind new_lens[b] are ignored.
 * Two sequences must not append to the same page slot in one call.
 */
ATTN_API attn_status attn_kv4_append(const attn_kv4_cache* cache, const void* k, const void* v, const int* block_table,
                                     const int* seq_lens, const int* new_lens, int B, int N, int max_pages,
                                     attn_dtype dtype, void* stream);

/*
 * attn_kv4_read - reads positions back.
 *   k, v   : [B, Hkv, N, d] outputs that do not overlap (else ATTN_ERR_INVALID_ARG): row
 *            i holds position starts[b] + i, rounded once to dtype (exact where the format
 *            holds it: 6 significant bits); rows at or behind seq_lens[b] are written as zeros.
 *   starts : [B] int32, 0 or more, or NULL for 0.
 */
ATTN_API attn_status attn_kv4_read(const attn_kv4_cache* cache, const int* block_table, const int* seq_lens,
                                   const int* starts, void* k, void* v, int B, int N, int max_pages,
                                   attn_dtype dtype, void* stream);

/*
 * attn_fwd_kv4 - attention of queries over the cache.
 *   q    : [B, Hq, N, d]; query head h reads key/value head h / (Hq / Hkv) (Hq is a
 *          multiple of Hkv).
 *   q_lens : [B] int32, 0 <= q_lens[b] <= N, or NULL for N. Query i < q_lens[b] is the
 *          token at position seq_lens[b] - q_lens[b] + i; it sees the keys at positions
 *          j < seq_lens[b], and with causal = 1 only j <= its own.
 *   o    : [B, Hq, N, d] output softmax(scale q K^T) V over the values as read back
 *          (must not overlap q: ATTN_ERR_INVALID_ARG).
 *   lse  : [B, Hq, N] fp32 (natural log, scale included), or NULL.
 *          Rows i >= q_lens[b] of o and lse are left as they were. A row that sees no
 *          key gets o = 0 and lse = -infinity; a row whose query holds an infinity or NaN and that
 *          sees a key gets o = NaN. A NaN key makes o and lse NaN in the rows
 *          that see it, a NaN value the 16 channels of its block in o; all else is unaffected.
 *   workspace : at least attn_fwd_kv4_workspace_bytes(...) bytes, 16-byte aligned,
 *          overwritten; needs no initialisation. Calls that overlap on the GPU, or that
 *          two host threads make at the same time, on one stream even (a call is two
 *          launches), need separate workspaces.
 *   scale: 0 selects 1/sqrt(d).
 *   Size: with R = Hq / Hkv * N <= 32 rows of a cached head, fewer than 2^31 tiles of 256 keys:
 *          B * Hkv * ceil(R / b) * (ceil(max_pages * page_size / 256) + 2) < 2^31 with b = 8
 *          (R <= 8 and 17 to 24) or 16, else ATTN_ERR_INVALID_ARG.
 * Arithmetic: scores and P V on f16 tensor-core products with fp32 accumulation
 * (every cached value is exact in f16; a query row is scaled by a power of two to
 * f16; P is rounded to f16, a row's largest between 2^7 and 2^15, so that probabilities
 * keep 11 bits down to 2^-21 of the row's largest, and none above 2^-32 of it is lost);
 * softmax statistics in fp32. Repeated calls give
 * bit-identical results.
 */
ATTN_API attn_status attn_fwd_kv4(const attn_kv4_cache* cache, const void* q, const int* block_table,
                                  const int* seq_lens, const int* q_lens, void* o, float* lse, void* workspace,
                                  size_t workspace_bytes, int B, int Hq, int N, int max_pages, float scale, int causal,
                                  attn_dtype dtype, void* stream);

/* attn_fwd_kv4_workspace_bytes - workspace attn_fwd_kv4 needs for this shape (0 also for
 * an invalid or unsupported one). Host only; launches nothing. */
ATTN_API size_t attn_fwd_kv4_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int page_size, int max_pages);

#ifdef __cplusplus
}
#endif

#endif /* KV4_B200_H */
