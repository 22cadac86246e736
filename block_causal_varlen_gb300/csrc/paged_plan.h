// Layout of the plan blob that bd_paged_plan_build writes on the host and the
// paged-cache kernels read from device memory. All fields are int32; offsets
// count int32 words from the start of the blob.
#pragma once
#include <stdint.h>

#include "../../include/bd_paged.h"
#include "plan_layout.h"

namespace bd {

constexpr int32_t kPagedMagic = 0x50414442;  // "BDAP"
constexpr int32_t kPagedVersion = 2;
// SMs of a GB300. The persistent attention kernels' work lists are cut for one CTA
// (tiles) or two (few rows: one adds up a block while the other's loads go on) on each.
constexpr int kPagedSms = 152;
constexpr int kDecCtas = 2 * kPagedSms, kTileCtas = kPagedSms;
// A few-rows block has 8, 16, 24 (bf16, e2m1) or 32 (bf16: the others lack the registers) (new row,
// query head) pairs of one K/V head: the least that holds every sequence of the plan that goes there. e2m1
// sequences of more than 24 go in blocks of 16 (16 of 8000 rows, 20 / 32 / 48 pairs: 76 us in blocks of
// 24, 88 and 127 of 16; 32 pairs in a block of 32, whose sums spill: 127).
constexpr int dec_most_rows(int fmt) { return fmt == BD_CACHE_BF16 ? 32 : 48; }  // of a sequence that goes there
constexpr int dec_block_rows(int fmt) { return fmt == BD_CACHE_BF16 ? 32 : fmt == BD_CACHE_E2M1 ? 24 : 16; }
constexpr int dec_rows_for(int fmt, int widest) {
  const int r = (widest + 7) / 8 * 8;
  return r <= dec_block_rows(fmt) ? r : fmt == BD_CACHE_BF16 ? 32 : 16;
}
constexpr int kDecSlotRows = 32;
// Rows of the joins get a CTA each, not a warp, if a block has more parts than kWideJoin, or
// more than kWideJoinFew and every row finds a CTA at once (one sequence of 512 keys: 8.7 us by
// warps, 6.3 by CTAs).
constexpr int kWideJoin = 16, kWideJoinFew = 4, kWideCtas = 4 * kPagedSms;
constexpr int kDecUnit = 32;   // keys by which the few-rows kernel's work is cut
// Tiles (of 128 / G new rows x G heads) of one K/V head that share a key tile in the
// tile kernel, and the rows of its partial-result slots.
constexpr int tile_slots(int d) { return d == 256 ? 1 : 2; }
constexpr int tile_slot_rows(int d) { return 128 * tile_slots(d); }
// At most this many partial results of a kind: the workspace's size.
constexpr int kDecSlots = 2 * kDecCtas, kTilePartSlots = 2 * kTileCtas;

// K/V heads whose few-rows CTAs walk the same keys side by side: all of them, or the most
// that leave no more than 1 in 64 CTAs over.
constexpr int gang_of(int hkv) {
  for (int g = hkv < kDecCtas ? hkv : kDecCtas; g > 1; --g)
    if (hkv % g == 0 && kDecCtas % g * 64 <= kDecCtas) return g;
  return 1;
}

// header words (the failure status keeps the place it has in attention plans, so
// that bd_check_status reads either)
enum : int {
  PH_MAGIC = 0, PH_VERSION, PH_WORDS, PH_B, PH_H, PH_HKV, PH_D, PH_G, PH_PAGE, PH_PAGE_SHIFT, PH_NUM_PAGES,
  PH_FMT, PH_CAUSAL, PH_T, PH_KV_TOTAL, PH_WRITE_OK, PH_SCALE_BITS,
  PH_OFF_TOK,      // int32 [T]: cache row (page * page_size + row) of every new row, -1 for none
  PH_OFF_PAGES,    // int32 [npages]: the used pages of all sequences back to back
  PH_NPAGES,
  PH_OFF_PGROW,    // int32 [npages]: packed row at which the page's first row is read back
  PH_OFF_PGCNT,    // int32 [npages]: rows of the page in use
  PH_OFF_DEC,      // few-rows kernel: its pieces, CTA after CTA,
  PH_NDEC,         // their number,
  PH_NDECM,        // the joins of its split blocks,
  PH_DECM_WIDE,    // whether their rows get a CTA each (by kWideJoin, kWideJoinFew and kWideCtas),
  PH_DEC_LIVE,     // the most rows of a block in use,
  PH_DEC_ROWS,     // and the rows of a block
  PH_OFF_TILE,     // the same for the tile kernel
  PH_NTILE,
  PH_NTILEM,
  PH_OFF_POS,      // int32 [T]: position of every new row, negative for none
  PH_OFF_TOUCH,    // int32 [NTOUCH]: entries of the page list that hold new rows, every page once
  PH_NTOUCH,
  PH_BOUNDS_OK,    // whether no two sequences have new rows in a page (causal plans)
  PH_BLOCKS,       // sparse plans: blocks of a list (0: not sparse), first and recent ones
  PH_FIRST,
  PH_RECENT,
  PH_OFF_ROWPG,    // int32 [T]: word offset of the pages of every new row's sequence
  PH_SEL_CAP,      // a power of two that no new row has more blocks than
  PH_SEL_ROWS,     // rows of a group whose blocks are selected together (1: every row is one)
  PH_OFF_SELG,     // int32 [NSELG][2]: first row and number of rows of every group, none where rows are groups
  PH_NSELG,
  PH_SEL_SPLIT,    // CTAs that share out a row's scores (a cluster; 1 where rows go together)
  PH_STATUS = H_STATUS, PH_STATUS_DETAIL = H_STATUS_DETAIL, // 5 few-rows attention, 6 tile attention
  kPagedHdrWords = kHdrWords
};

// A piece: some keys of one block of rows of one (sequence, K/V head). Row r of a
// block is (new row, head of the group) number PC_ROW0 + r, new-row-major.
enum : int {
  PC_Q0 = 0,    // packed row of the sequence's first new row
  PC_QLEN, PC_KVLEN,
  PC_PAGES,     // word offset of the sequence's pages
  PC_HKV,       // K/V head
  PC_ROW0,      // first (new row, head) number of the block
  PC_NROWS,     // rows of the block that exist
  PC_K0, PC_K1, // keys [k0, k1); k0 a multiple of the kernel's unit
  PC_SLOT,      // partial-result slot, -1: the whole key range, written to the output
  PC_T0,        // PC_ROW0 / G: the block's first new row
  PC_NBLK,      // sparse plans: blocks of the sequence up to the row's own
  kPieceWords = 12
};

// Where a CTA starts reading: its pieces [p0, p1) and a copy of the first one, so that
// no lookup stands between a launch and its first loads.
enum : int { RC_P0 = 0, RC_P1, RC_RESERVED0, RC_RESERVED1, RC_PIECE, kRecordWords = RC_PIECE + kPieceWords };

// A join of the n partial results in slots slot0, slot0 + 1, ... of one block.
enum : int { MG_SLOT0 = 0, MG_N, MG_Q0, MG_HKV, MG_ROW0, MG_NROWS, MG_RESERVED0, MG_RESERVED1, kMergeWords = 8 };

static_assert(PH_SEL_SPLIT < PH_STATUS, "header words");

// Records and joins have fixed places and room for the most there can be (a join has
// two slots at least).
constexpr int kOffDecRec = kPagedHdrWords;
constexpr int kOffDecMerge = kOffDecRec + kDecCtas * kRecordWords;
constexpr int kOffTileRec = kOffDecMerge + kDecSlots / 2 * kMergeWords;
constexpr int kOffTileMerge = kOffTileRec + kTileCtas * kRecordWords;
constexpr int kOffLists = kOffTileMerge + kTilePartSlots / 2 * kMergeWords;

// Sparse plans: the most blocks of a list, and of a sequence (its scores stay in one CTA's
// shared memory).
constexpr int kMostListed = 4096, kMostBlocks = 16384;
// Groups of up to kSelRows rows of a sequence select their blocks together, where that leaves
// enough CTAs and their scores and codes take no more than kSelSmem bytes.
constexpr int kSelRows = 8, kSelCtas = 2 * kPagedSms;
constexpr int64_t kSelSmem = 48 << 10;
// Where PH_SEL_CAP is past kSelSplitCap, rows get a cluster of 2 or 4 CTAs each if every one of them has an
// SM to itself (4 sequences of 938 blocks, 8 heads: 12 us by a CTA a row and head, 8.8 by four; 16 of them by two,
// two on an SM: 12 and 14.6; 2 of them by eight, which find no room side by side: 12.3).
constexpr int kSelSplitCap = 512, kSelMostSplit = 4;
// Shared memory of the selection: codes of q (bytes of a (row, head): two lots of d, and what
// sets eight of them apart in the banks), a power of two and a place each, a score for each block and row.
constexpr int select_pitch(int d) { return 2 * d + (d == 64 ? 64 : 16); }
constexpr int64_t select_smem(int rows, int G, int d, int cap) {
  return (int64_t(rows) * G + 7) / 8 * 8 * (select_pitch(d) + 8) + int64_t(rows) * cap * 4;
}
constexpr int64_t kSelMostSmem = select_smem(1, 128, 256, kMostBlocks);
static_assert(kSelMostSmem <= 232448 - 1024, "selection over the per-CTA limit of shared memory");

// Bytes of one head's K (or V) of a cached row, and of its scales' alignment (e2m1).
constexpr int row_bytes(int fmt, int d) { return fmt == BD_CACHE_BF16 ? 2 * d : fmt == BD_CACHE_E4M3 ? d : d / 2; }
constexpr int elem_bytes(int fmt) { return fmt == BD_CACHE_BF16 ? 2 : 1; }  // of a cache's strides
constexpr int scale_align(int d) { return d == 64 ? 4 : 8; }

// Validated view of a host plan blob.
int32_t view_paged_plan(const void* plan_host, const int32_t** out);

}  // namespace bd
