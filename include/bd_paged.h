/*
 * bd_paged.h -- C ABI of libbd, second part: a paged K/V cache and the
 * attention of new rows over it, for continuing the documents bd_attn.h's
 * operations train on or prefill, on sm_103a (GB300).
 *
 * What the operations are:
 *   - the K/V rows of a sequence live in fixed-size pages of a pool shared by
 *     all sequences; a page list per sequence says where: cache position j of
 *     sequence b is row j % page_size of page pages_b[j / page_size];
 *   - a step gives sequence b q_len[b] new rows, after which kv_len[b] rows of it
 *     are cached: new row i has cache position kv_len[b] - q_len[b] + i. That is
 *     the asymmetric segment with more keys than queries and bottom-right causal
 *     alignment that bd_segment cuts (bd_segment_t: diag_off = k_len - q_len);
 *   - new rows of all sequences are packed back to back, sequence by sequence;
 *   - bd_cache_write stores new K/V rows, bd_cache_read gets a batch's cached
 *     rows back as packed bf16 rows (the K/V bd_attn_fwd takes, sequences as
 *     documents), bd_paged_attn computes O and LSE of the new rows over the cache.
 *
 * Conventions are those of bd_attn.h (status returns, caller-owned buffers,
 * stream ordering, scale 1/sqrt(d), natural-log LSE, GQA head mapping). In
 * addition:
 *   - a plan (host blob, validated and balanced once per step, copied to the
 *     device by the caller) carries the lengths, the pages and the work lists;
 *     it serves every layer of a step. Kernels only read it (but for the failure
 *     status), so calls sharing one device copy may overlap on the GPU; each
 *     overlapping bd_paged_attn needs a workspace of its own.
 *   - launches have fixed shapes and read their counts from the device plan: a
 *     captured call may be replayed after the device copy has been overwritten
 *     with another step's plan of the same bd_paged_plan_key.
 *   - new rows are rows [0, T) of the packed tensors, T = sum of q_len; rows past
 *     T have no influence and are not written.
 */
#ifndef BD_PAGED_H
#define BD_PAGED_H

#include "bd_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element format of a cache. */
typedef enum {
  BD_CACHE_BF16 = 0, /* bf16 values                                                       */
  /* e4m3 codes and one exponent byte per (row, head): value = code * 2^(byte - 127).
   * bd_cache_write takes, per row and head, the smallest e in [-60, 60] with
   * max|x| <= 448 * 2^e (60 if there is none) and stores code = x * 2^-e rounded to
   * nearest even, saturating at +-448, and byte e + 127. A row with an infinity or a
   * NaN is stored as NaN codes with byte 255 and reads back as NaN. Values read back
   * are exact in bf16. Caches filled by other means may use bytes 67..187 and 255, and
   * the NaN codes 0x7f and 0xff in rows of byte 255 only; their V rows take the exponent
   * bd_cache_write would, or one near it: bd_paged_attn may hold a key's weight p * 2^e (p: its
   * probability, e: its V row's exponent) to no more than 2^-32 of the row's largest, so that
   * zeros of a high byte, say, would hide the keys that matter (bd_cache_write's zeros, of
   * byte 67, hide nothing above 2^-83 of a key's p * v). */
  BD_CACHE_E4M3 = 1
} bd_cache_fmt;

/* A paged K/V cache of one layer. k and v: stride_b is the stride from page to
 * page, stride_row and stride_head those of the rows of a page and of the
 * K/V heads (elements, any order of the dimensions; bytes must be multiples of 16,
 * as must the base pointers), rows = page_size, stride_c is unused, and the d
 * elements of a head are contiguous. k_exp, v_exp: exponent bytes of a
 * BD_CACHE_E4M3 cache with their common strides (ignored otherwise); bd_paged_attn
 * reads them by the aligned 4-byte words they lie in. */
typedef struct {
  bd_tensor k, v;
  uint8_t* k_exp;
  uint8_t* v_exp;
  int64_t exp_stride_page, exp_stride_row, exp_stride_head;
  int32_t fmt;       /* bd_cache_fmt            */
  int32_t num_pages; /* extent of the page dim  */
} bd_paged_cache;

/* A step's work over a paged cache. */
typedef struct {
  int32_t B;                   /* sequences, >= 1                                     */
  int32_t H, Hkv, d;           /* d in {64, 128, 256}; H % Hkv == 0; H / Hkv <= 128   */
  int32_t page_size;           /* rows of a page: a power of two, 16..1024            */
  int32_t num_pages;           /* pages of the pool; num_pages * page_size < 2^31     */
  int32_t fmt;                 /* bd_cache_fmt                                        */
  int32_t causal;              /* 1: new row i sees positions j <= kv_len - q_len + i;
                                  0: every new row sees all kv_len rows (a slice of a
                                  context held elsewhere as well; join by LSE)        */
  const int32_t* q_len;        /* host int32[B]: new rows, >= 0                       */
  const int32_t* kv_len;       /* host int32[B]: cached rows with the new ones, >= 0.
                                  With kv_len < q_len the first q_len - kv_len new
                                  rows have no position: they are not written and
                                  see nothing (O = 0, LSE = -inf)                     */
  const int32_t* pages;        /* host: all sequences' page lists back to back        */
  const int32_t* page_offsets; /* host int32[B+1]: sequence b's list is
                                  pages[page_offsets[b] .. page_offsets[b+1]), at
                                  least ceil(kv_len / page_size) entries, the used
                                  ones in [0, num_pages). Sequences may share pages.  */
} bd_paged_desc;

/* Bytes that hold the plan blob for `desc`, which is validated in full (lengths, head
 * counts, every page index used). A bound: the plan itself may be shorter (its third
 * 32-bit word is the number of words in use, all that has to be copied to the device).
 * Errors: BD_ERR_ARG, BD_ERR_UNSUPPORTED (head dim, head ratio, page size),
 * BD_ERR_CAPACITY (sizes past 2^31; pages in use times page_size past 2^34). */
BD_API int32_t bd_paged_plan_bytes(const bd_paged_desc* desc, size_t* bytes);

/* Build the plan blob into caller-owned host memory (16-byte aligned, blob_bytes
 * >= bd_paged_plan_bytes). The caller copies the same bytes to device memory
 * (16-byte aligned) and passes both copies to the calls below. The blob does not
 * refer to desc's arrays afterwards. Pure host function. */
BD_API int32_t bd_paged_plan_build(const bd_paged_desc* desc, void* blob, size_t blob_bytes);

/* A number that two plans share if a call captured with one may be replayed with
 * the other's bytes in the device copy: same heads, page size, pool size, format
 * and mask, and the same kernels launched. (The captured tensors must hold the new
 * plan's rows and its device buffer its bytes.) */
BD_API int32_t bd_paged_plan_key(const void* plan_host, uint64_t* key);

/* bd_cache_write -- store the new rows' K and V (bf16, row t = packed new row t, rows
 * >= T, stride_b and stride_c unused) at their cache positions, quantised for a
 * BD_CACHE_E4M3 cache; nothing else in the pool is touched. BD_ERR_PLAN if two new
 * rows of the batch share a cache row (sequences sharing the page they write to), if
 * the plan is not causal (its rows have no positions), or if the cache differs from
 * the plan's format or sizes. */
BD_API int32_t bd_cache_write(const void* plan_host, const void* plan_dev, const bd_tensor* k, const bd_tensor* v,
                              const bd_paged_cache* cache, void* stream);

/* bd_cache_read -- rows [0, kv_len) of every sequence of the plan as bf16, packed back
 * to back in batch order into rows [0, sum of kv_len) of k and v; rows past that are
 * left alone. */
BD_API int32_t bd_cache_read(const void* plan_host, const void* plan_dev, const bd_paged_cache* cache, bd_tensor* k,
                             bd_tensor* v, void* stream);

/* Workspace bytes of bd_paged_attn: partial results of rows whose keys are split
 * over several blocks. A function of the plan's key and d only: for the most there can be
 * (5 to 20 MB for few rows, 20 to 40 MB for more of them), however few are cut. */
BD_API int32_t bd_paged_attn_workspace(const void* plan_host, size_t* bytes);

/* bd_paged_attn -- O (bf16) and LSE (fp32, may be NULL) of the new rows over their
 * sequences' cached rows; q, out: rows >= T, stride_b and stride_c unused; lse
 * [H, rows], stride_head between heads, stride_b and stride_c unused. K/V rows past
 * kv_len, and pages past the last one used, may hold anything; so may cached rows that
 * a new row does not see: an infinity or a NaN there reaches the rows that see it only.
 * O's error is that of probabilities rounded to bf16 (2^-8 of each) and of its own rounding; few
 * rows over a BD_CACHE_E4M3 cache (up to 48 (new row, query head) pairs of a K/V head) have
 * weights p * 2^e in fp16 instead: 2^-11 of each, and 2^-32 of the row's largest where that is more.
 * out must not alias q or the cache. workspace: bd_paged_attn_workspace bytes, 256-byte aligned;
 * it needs no clearing and holds nothing between calls. */
BD_API int32_t bd_paged_attn(const void* plan_host, const void* plan_dev, const bd_tensor* q,
                             const bd_paged_cache* cache, bd_tensor* out, bd_rowstat* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BD_PAGED_H */
