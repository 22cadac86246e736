// Layout of the plan blob that bd_paged_plan_build writes on the host and the
// paged-cache kernels read from device memory. All fields are int32; offsets
// count int32 words from the start of the blob.
#pragma once
#include <stdint.h>

#include "../../include/bd_paged.h"
#include "plan_layout.h"

namespace bd {

constexpr int32_t kPagedMagic = 0x50414442;  // "BDAP"
constexpr int32_t kPagedVersion = 1;
// SMs of a GB300. The persistent attention kernels' work lists are cut for one CTA
// (tiles) or two (few rows: one adds up a block while the other's loads go on) on each.
constexpr int kPagedSms = 152;
constexpr int kDecCtas = 2 * kPagedSms, kTileCtas = kPagedSms;
// A few-rows block has 8, 16 or (bf16: e4m3 lacks the registers) 24 or 32 (new row, query head)
// pairs of one K/V head: the least that holds every sequence of the plan that goes there.
constexpr int dec_most_rows(int fmt) { return fmt == BD_CACHE_BF16 ? 32 : 48; }  // of a sequence that goes there
constexpr int dec_block_rows(int fmt) { return fmt == BD_CACHE_BF16 ? 32 : 16; }
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
  PC_RESERVED0,
  kPieceWords = 12
};

// Where a CTA starts reading: its pieces [p0, p1) and a copy of the first one, so that
// no lookup stands between a launch and its first loads.
enum : int { RC_P0 = 0, RC_P1, RC_RESERVED0, RC_RESERVED1, RC_PIECE, kRecordWords = RC_PIECE + kPieceWords };

// A join of the n partial results in slots slot0, slot0 + 1, ... of one block.
enum : int { MG_SLOT0 = 0, MG_N, MG_Q0, MG_HKV, MG_ROW0, MG_NROWS, MG_RESERVED0, MG_RESERVED1, kMergeWords = 8 };

// Records and joins have fixed places and room for the most there can be (a join has
// two slots at least).
constexpr int kOffDecRec = kPagedHdrWords;
constexpr int kOffDecMerge = kOffDecRec + kDecCtas * kRecordWords;
constexpr int kOffTileRec = kOffDecMerge + kDecSlots / 2 * kMergeWords;
constexpr int kOffTileMerge = kOffTileRec + kTileCtas * kRecordWords;
constexpr int kOffLists = kOffTileMerge + kTilePartSlots / 2 * kMergeWords;

// Validated view of a host plan blob.
int32_t view_paged_plan(const void* plan_host, const int32_t** out);

}  // namespace bd
