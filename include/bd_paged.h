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
 *     documents), bd_paged_attn computes O and LSE of the new rows over the cache;
 *   - bd_cache_append writes new rows turned by their positions;
 *   - bd_block_bounds, bd_block_select and bd_sparse_attn let each new row attend the blocks
 *     (pages) of its sequence that a cheap score picks.
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
 *     with another step's plan of the same bd_paged_plan_key. The calls that write, append,
 *     read back, take bounds and select launch the CTAs that the captured plan's rows or
 *     pages fill (a few an SM at most), and these take all that the next plan has: right
 *     for every plan of the key, slow for one of many times the rows. Capture the largest step.
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
  BD_CACHE_E4M3 = 1,
  /* e2m1 codes, two a byte (the even element's in the low half; magnitudes 0, 0.5, 1, 1.5, 2, 3,
   * 4, 6 and a sign), and a scale byte for every 16 elements of a (row, head): value = code * s,
   * s = (1 + m / 8) * 2^(e - 15) for byte 8 e + m (m / 8 * 2^-14 for e = 0). bd_cache_write
   * takes, for every 16 values, the smallest byte of [8, 226] with max|x| <= 6 s (226, that is
   * 10240, if there is none) and stores x / s rounded to the nearest code (ties to the even one),
   * saturating at +-6. 16 values with an infinity or a NaN among them are stored as byte 255 and
   * read back as NaN. Values read back are exact in bf16 (and in fp16). Caches filled by other
   * means may use bytes 0..226 and 255. */
  BD_CACHE_E2M1 = 4
} bd_cache_fmt;

/* A paged K/V cache of one layer. k and v: stride_b is the stride from page to
 * page, stride_row and stride_head those of the rows of a page and of the
 * K/V heads (elements, any order of the dimensions; bytes must be multiples of 16,
 * as must the base pointers), rows = page_size, stride_c is unused, and the d
 * elements of a head are contiguous. k_exp, v_exp: exponent bytes of a
 * BD_CACHE_E4M3 cache with their common strides (ignored for bf16); bd_paged_attn
 * reads them by the aligned 4-byte words they lie in. Of a BD_CACHE_E2M1 cache k and v are bytes
 * (strides in bytes, d / 2 of them a head) and k_exp, v_exp the scale bytes, d / 16 contiguous
 * ones of a (row, head): pointers and strides are multiples of 8 bytes (4 at d = 64). */
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

/* Frequencies of a position rotation as the kernels take them: out[i] = turns a position
 * advances pair i by, modulo 1, in units of 2^-64 (host, n values; inv_freq in radians a
 * position, any finite number), off by at most 2^-63 + |inv_freq[i]| 2^-106 of a turn. A position's angle
 * is its product with out[i], modulo 2^64: exact, so positions up to 2^31 are off by no more than 2^-31 of
 * a turn (|inv_freq| up to 2^42). BD_ERR_ARG for an infinity or a NaN. Pure host function. */
BD_API int32_t bd_rope_phases(const double* inv_freq, int32_t n, uint64_t* out);

/* A rotation of pairs of elements of a head by angles p * inv_freq[i] at position p. */
typedef struct {
  const uint64_t* phase; /* device uint64[dim / 2], from bd_rope_phases, 8-byte aligned         */
  int32_t dim;           /* elements that take part, the first ones of a head: a multiple of 16,
                            0 < dim <= d                                                        */
  int32_t interleaved;   /* 1: pairs (2 i, 2 i + 1), 0: pairs (i, i + dim / 2)                  */
  float scale;           /* factor of the turned elements (1: none)                             */
  int32_t reserved;
} bd_rope;

/* bd_cache_append -- bd_cache_write with a rotation on the way: the new rows' K are turned by
 * their cache positions, (x, y) -> scale (x cos a - y sin a, y cos a + x sin a), rounded to bf16
 * and stored as bd_cache_write stores them; V is stored as it is. q (may be NULL, with q_out) is
 * turned the same way into q_out, both bf16 [rows, H, d] as in bd_paged_attn; q_out may be q itself and
 * overlaps nothing else. q rows without a position are copied. The turned values are off by at
 * most 2^-21 of the pair's length times scale before they are rounded. Errors as bd_cache_write;
 * BD_ERR_ARG for a rope's fields. */
BD_API int32_t bd_cache_append(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_tensor* k,
                               const bd_tensor* v, const bd_rope* rope, const bd_paged_cache* cache, bd_tensor* q_out,
                               void* stream);

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
 * weights p * 2^e in fp16 instead: 2^-11 of each, and 2^-32 of the row's largest where that is more. So do
 * rows over a BD_CACHE_E2M1 cache, few or many, with weights p.
 * out must not alias q or the cache. workspace: bd_paged_attn_workspace bytes, 256-byte aligned;
 * it needs no clearing and holds nothing between calls. */
BD_API int32_t bd_paged_attn(const void* plan_host, const void* plan_dev, const bd_tensor* q,
                             const bd_paged_cache* cache, bd_tensor* out, bd_rowstat* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ---- attention over selected blocks
 *
 * A block is a page of a sequence: block j holds its rows [j * page_size, (j + 1) * page_size).
 * Every new row attends, for every K/V head, a list of at most `blocks` of the blocks up to its
 * own; the heads of a group share the list. A block is chosen by the least and the greatest value
 * of each element of its keys, held in 8 bits beside the cache (2 d + 1 bytes a block and K/V head):
 *   bd_block_bounds   brings the bounds of the blocks up to date that new rows entered,
 *   bd_block_select   scores the blocks of every new row and lists the best,
 *   bd_sparse_attn    attends over the listed blocks.
 * That pays for few new rows over long contexts: every row reads its own blocks, where
 * bd_paged_attn reads a key once for all rows of a tile (661 rows of two prompts over 6000 to 16000 keys, 24
 * blocks of 32: 112 us, bd_paged_attn 79). A sparse plan takes 48 bytes and some 0.2 us of the host a row and
 * K/V head.
 * A sparse plan serves these, bd_cache_write and bd_cache_append of a step (bd_block_bounds takes
 * the other causal plans too); its bd_paged_plan_key covers the sparse description. */
typedef struct {
  int32_t blocks; /* blocks of a list, 1..4096, at least first + recent                      */
  int32_t first;  /* the first blocks of a sequence are always listed, >= 0                  */
  int32_t recent; /* as are the last ones up to the row's own, which counts as one, >= 1     */
  int32_t reserved;
} bd_sparse_desc;

/* Like bd_paged_plan_bytes / bd_paged_plan_build, for a step whose rows attend over selected
 * blocks. desc->causal must be 1. BD_ERR_UNSUPPORTED: a sequence of more than 16384 blocks. */
BD_API int32_t bd_sparse_plan_bytes(const bd_paged_desc* desc, const bd_sparse_desc* sparse, size_t* bytes);
BD_API int32_t bd_sparse_plan_build(const bd_paged_desc* desc, const bd_sparse_desc* sparse, void* blob, size_t blob_bytes);

/* The bounds of a pool's blocks: code[page][head][0][c] the lower, [1][c] the upper bound of
 * element c, value = code * 2^(exp[page][head] - 127). bd_block_bounds takes the smallest e in
 * [-50, 50] with max|k| <= 127 * 2^e (50 if there is none) and stores floor(min k * 2^-e) and
 * ceil(max k * 2^-e), saturating at +-127, and byte e + 127; a block with an infinity or a NaN among
 * its keys gets byte 255, which outscores every other (and is what a block's byte is to be set to before its
 * bounds are made; other bytes count as the nearest of 77..177). Base pointers and strides of code are
 * multiples of 16 bytes; strides of exp positive. */
typedef struct {
  int8_t* code;
  int64_t stride_page, stride_head, stride_bound; /* of code, in bytes; d contiguous         */
  uint8_t* exp;
  int64_t exp_stride_page, exp_stride_head;
  int32_t num_pages, reserved;
} bd_bounds;

/* bd_block_bounds -- bounds of the blocks that hold new rows, from their cached rows below kv_len
 * (all blocks of a sequence whose rows are all new). BD_ERR_PLAN if two sequences have new rows
 * in the same page, or the plan is not causal. (bd_paged_plan_key does not tell such a page: under a
 * captured call it gets the bounds of the most rows that a sequence with new rows in it uses.) */
BD_API int32_t bd_block_bounds(const void* plan_host, const void* plan_dev, const bd_paged_cache* cache,
                               const bd_bounds* bounds, void* stream);

/* The lists of the new rows: row t's blocks for K/V head g are entries [0, blocks) at
 * ptr + t * stride_row + g * stride_head, ascending, -1 past the last one. */
typedef struct {
  int32_t* ptr;
  int64_t stride_row, stride_head; /* elements */
  int32_t rows, reserved;
} bd_blocks;

/* bd_block_select -- the lists of the new rows (q [rows, H, d] as bd_paged_attn takes it). q is held
 * in 8 bits for this, codes rn(q * 2^-e) with the smallest e in [-50, 50] that has max|q| <= 127 * 2^e
 * (50 if there is none) for every row and head (codes saturate; a head with an infinity or a NaN
 * counts as zeros). A block's score for a head is sum_c max(q_c lo_c, q_c hi_c), for the group the largest of its
 * heads'. Listed are the first and the recent blocks and those of the largest scores, of equal ones the
 * lowest; all blocks up to the row's own if they are no more than `blocks`. Scores are exact: equal
 * inputs give equal lists. Rows without a position get -1 throughout. */
BD_API int32_t bd_block_select(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_bounds* bounds,
                               bd_blocks* blocks, void* stream);

/* bd_sparse_attn -- O and LSE of the new rows over the listed blocks of their sequences, as
 * bd_paged_attn computes them: new row at position p takes the listed blocks' rows, n = min(blocks, number of
 * blocks up to its own) of them, the last listed one up to row p % page_size. Lists are those of bd_block_select, or
 * others of that form (n blocks, the row's own last; an entry outside the row's blocks stands for the nearest one).
 * Workspace as for bd_paged_attn (bd_paged_attn_workspace). */
BD_API int32_t bd_sparse_attn(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_paged_cache* cache,
                              const bd_blocks* blocks, bd_tensor* out, bd_rowstat* lse, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BD_PAGED_H */
