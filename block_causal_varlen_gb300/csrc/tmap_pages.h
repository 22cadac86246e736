// TMA descriptors of the paged-cache kernels (defined beside the others in
// host_util.cpp).
#pragma once
#include "host_util.h"

namespace bd {

// Encodes a 5-D tiled TMA map over packed bf16 rows [rows, heads, d] (t's b and c
// dimensions unused) whose box is 64 columns of box_heads heads x box_rows rows,
// 128-byte swizzle: in shared memory row-major [row][head][64].
int32_t make_tmap_group_bf16(CUtensorMap* map, const bd_tensor* t, int64_t heads, int64_t d, const char* name,
                             int box_heads, int box_rows);

// Encodes a 5-D tiled TMA map over a paged cache's K or V (esize 2: bf16, 1: bytes of codes, the
// unit of t's strides) with row_bytes bytes of a head in a row: dims (piece of `piece` = 32, 64 or
// 128 bytes of them, row of a page, piece, head, page), box = box_rows rows of one piece of one
// head, swizzled over the piece's bytes: in shared memory [row][bytes]. neighbours: what lies
// beside a box's rows is read at the same time.
int32_t make_tmap_pages(CUtensorMap* map, const bd_tensor* t, int64_t pages, int64_t heads, int64_t row_bytes, int esize,
                        const char* name, int box_rows, bool neighbours, int piece);

}  // namespace bd
