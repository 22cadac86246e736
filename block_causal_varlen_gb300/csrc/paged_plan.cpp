// Host side of the paged K/V cache: validation of a step's lengths and pages, and
// the plan blob the kernels read.
//
// The attention's work is cut on the host. A block of query rows (the (new row,
// query head) pairs of one K/V head) and its keys are an item; items are given out
// whole or cut by keys, so that every CTA gets about the same number of key units.
// Parts of cut items write partial results (running maximum, sum, unnormalised O)
// that a second kernel joins. One long sequence is thereby spread over every SM, and
// a ragged batch leaves none idle, without counters or atomics on the device.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <stdexcept>
#include <tuple>
#include <utility>
#include <vector>

#include "common.h"
#include "paged_plan.h"

namespace bd {

int32_t view_paged_plan(const void* plan_host, const int32_t** out) {
  if (!plan_host) return fail(BD_ERR_ARG, "plan_host is NULL");
  const int32_t* w = static_cast<const int32_t*>(plan_host);
  if (w[PH_MAGIC] != kPagedMagic || w[PH_VERSION] != kPagedVersion)
    return fail(BD_ERR_PLAN, "not a paged plan blob (bad magic/version)");
  const int64_t words = w[PH_WORDS];
  auto in = [&](int64_t off, int64_t n, int stride) { return off >= kOffLists && n >= 0 && off + n * stride <= words; };
  if (!in(w[PH_OFF_TOK], w[PH_T], 1) || !in(w[PH_OFF_PAGES], w[PH_NPAGES], 1) || !in(w[PH_OFF_PGROW], w[PH_NPAGES], 1) ||
      !in(w[PH_OFF_PGCNT], w[PH_NPAGES], 1) || !in(w[PH_OFF_DEC], w[PH_NDEC], kPieceWords) ||
      !in(w[PH_OFF_POS], w[PH_T], 1) || !in(w[PH_OFF_TOUCH], w[PH_NTOUCH], 1) ||
      (w[PH_BLOCKS] && (!in(w[PH_OFF_ROWPG], w[PH_T], 1) || w[PH_SEL_ROWS] < 1 || w[PH_SEL_ROWS] > kSelRows ||
                        w[PH_SEL_SPLIT] < 1 || w[PH_SEL_SPLIT] > kSelMostSplit ||
                        (w[PH_SEL_ROWS] > 1 && !in(w[PH_OFF_SELG], w[PH_NSELG], 2)))) ||
      !in(w[PH_OFF_TILE], w[PH_NTILE], kPieceWords) || w[PH_NDECM] < 0 || w[PH_NDECM] > kDecSlots / 2 ||
      w[PH_NTILEM] < 0 || w[PH_NTILEM] > kTilePartSlots / 2)
    return fail(BD_ERR_PLAN, "paged plan blob offsets are inconsistent");
  *out = w;
  return BD_OK;
}

namespace {

// seq: a sequence of the batch or, in sparse plans, a new row, which has keys of its own
struct Item {
  int32_t seq, hkv, row0, nrows, keys;
};

// What the pieces say of the sequences (or new rows) that items belong to.
struct Seqs {
  std::vector<int32_t> q0, q_len, kv_len, page_off, nblk;
};

// Some key units of an item, and the CTA that takes them.
struct Part {
  int32_t item, u0, u1, cta;
};

struct Lists {
  std::vector<int32_t> records;  // [CTAs][kRecordWords]
  std::vector<int32_t> pieces, merges;
};

int32_t units_of(const Item& it, int unit) { return int32_t((int64_t(it.keys) + unit - 1) / unit); }

// Cuts the items, in order, into n stretches of at most `t` key units, where a part
// costs its units plus `over`; false if they do not fit.
bool stretch(const std::vector<Item>& items, int unit, int over, int64_t t, int n, std::vector<Part>* parts) {
  int cta = 0;
  int64_t cap = t;
  for (size_t i = 0; i < items.size(); ++i) {
    const int32_t units = units_of(items[i], unit);
    int32_t at = 0;
    for (;;) {
      const int64_t rem = units - at;
      if (rem + over <= cap) {
        if (parts) parts->push_back({int32_t(i), at, units, cta});
        cap -= rem + over;
        break;
      }
      const int64_t part = std::min(cap - over, rem - 1);
      if (part >= 1) {
        if (parts) parts->push_back({int32_t(i), at, int32_t(at + part), cta});
        at += int32_t(part);
      } else if (cap == t) {
        return false;
      }
      if (++cta == n) return false;
      cap = t;
    }
  }
  return true;
}

// The shortest stretches that hold everything: equal work for every CTA, at most two
// parts of cut items in each.
int64_t cut_evenly(const std::vector<Item>& items, int unit, int over, int ctas, std::vector<Part>* parts) {
  int64_t total = 0;
  for (const Item& it : items) total += units_of(it, unit) + over;
  int64_t lo = std::max<int64_t>(over + 1, (total + ctas - 1) / ctas), hi = lo;
  while (!stretch(items, unit, over, hi, ctas, nullptr)) {
    lo = hi + 1;
    hi += std::max<int64_t>(1, hi / 8);
  }
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (stretch(items, unit, over, mid, ctas, nullptr)) hi = mid;
    else lo = mid + 1;
  }
  stretch(items, unit, over, hi, ctas, parts);
  return hi;
}

// Items of more than `most` units in equal parts, the longest part first to that of `num` CTAs
// with the least; returns the longest load, or -1 if the parts of cut items are more
// than there are slots.
int64_t cut_longest(const std::vector<Item>& items, int unit, int over, int64_t most, int num, std::vector<Part>* parts) {
  parts->clear();
  int64_t split = 0;
  for (size_t i = 0; i < items.size(); ++i) {
    const int64_t units = units_of(items[i], unit), n = std::max<int64_t>(1, (units + most - 1) / most);
    if (n > 1 && (split += n) > kTilePartSlots) return -1;
    for (int64_t k = 0; k < n; ++k)
      parts->push_back({int32_t(i), int32_t(units * k / n), int32_t(units * (k + 1) / n), 0});
  }
  std::stable_sort(parts->begin(), parts->end(), [](const Part& a, const Part& b) { return a.u1 - a.u0 > b.u1 - b.u0; });
  typedef std::pair<int64_t, int> Load;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> ctas;
  for (int c = 0; c < num; ++c) ctas.push({0, c});
  int64_t longest = 0;
  for (Part& p : *parts) {
    Load l = ctas.top();
    ctas.pop();
    p.cta = l.second;
    l.first += p.u1 - p.u0 + over;
    longest = std::max(longest, l.first);
    ctas.push(l);
  }
  std::stable_sort(parts->begin(), parts->end(), [](const Part& a, const Part& b) { return a.cta < b.cta; });
  return longest;
}

// Whole items, longest first, to the CTA with the least, as long as its load stays
// within `t`; the others cut to fill what is left of the CTAs. False if that does not
// hold everything (gaps of less than 4 units beyond a part's cost stay empty).
bool fill(const std::vector<Item>& items, int unit, int over, int64_t t, std::vector<Part>* parts) {
  parts->clear();
  std::vector<int32_t> order(items.size()), left;
  for (size_t i = 0; i < items.size(); ++i) order[i] = int32_t(i);
  std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) { return items[a].keys > items[b].keys; });
  typedef std::pair<int64_t, int> Load;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> ctas;
  for (int c = 0; c < kTileCtas; ++c) ctas.push({0, c});
  for (int32_t i : order) {
    Load l = ctas.top();
    const int64_t units = units_of(items[i], unit);
    if (l.first + units + over > t) {
      left.push_back(i);
      continue;
    }
    ctas.pop();
    parts->push_back({i, 0, int32_t(units), l.second});
    l.first += units + over;
    ctas.push(l);
  }
  int64_t split = 0;
  for (int32_t i : left) {
    const int64_t units = units_of(items[i], unit);
    int64_t at = 0, n = 0;
    while (at < units) {
      Load l = ctas.top();
      const int64_t part = std::min(t - l.first - over, units - at);
      if (part < std::min<int64_t>(4, units - at)) return false;
      ctas.pop();
      parts->push_back({i, int32_t(at), int32_t(at + part), l.second});
      l.first += part + over;
      ctas.push(l);
      at += part;
      ++n;
    }
    if (n > 1 && (split += n) > kTilePartSlots) return false;
  }
  std::stable_sort(parts->begin(), parts->end(), [](const Part& a, const Part& b) { return a.cta < b.cta; });
  return true;
}

// Writes the parts (in CTA order) down as pieces, records and joins.
void write_lists(const bd_paged_desc& D, const std::vector<Item>& items, const std::vector<Part>& parts, const Seqs& S,
                 int unit, int ctas, Lists* L) {
  L->records.assign(size_t(ctas) * kRecordWords, 0);
  // slots of an item's parts in key order, items in order
  std::vector<int32_t> count(items.size(), 0), slot0(items.size(), -1);
  for (const Part& p : parts) ++count[p.item];
  int32_t slots = 0;
  for (size_t i = 0; i < items.size(); ++i) {
    if (count[i] < 2) continue;
    const Item& it = items[i];
    int32_t m[kMergeWords] = {0};
    slot0[i] = m[MG_SLOT0] = slots;
    m[MG_N] = count[i]; m[MG_Q0] = S.q0[it.seq]; m[MG_HKV] = it.hkv; m[MG_ROW0] = it.row0; m[MG_NROWS] = it.nrows;
    L->merges.insert(L->merges.end(), m, m + kMergeWords);
    slots += count[i];
  }
  std::vector<std::vector<int32_t>> starts(items.size());  // first units of a cut item's parts
  for (const Part& p : parts)
    if (slot0[p.item] >= 0) starts[p.item].push_back(p.u0);
  for (auto& v : starts) std::sort(v.begin(), v.end());
  for (size_t i = 0; i < parts.size(); ++i) {
    const Part& x = parts[i];
    const Item& it = items[x.item];
    int32_t p[kPieceWords] = {0};
    p[PC_Q0] = S.q0[it.seq]; p[PC_QLEN] = S.q_len[it.seq]; p[PC_KVLEN] = S.kv_len[it.seq];
    p[PC_PAGES] = S.page_off[it.seq]; p[PC_NBLK] = S.nblk[it.seq]; p[PC_HKV] = it.hkv; p[PC_ROW0] = it.row0; p[PC_NROWS] = it.nrows;
    p[PC_K0] = x.u0 * unit;
    p[PC_K1] = int32_t(std::min<int64_t>(it.keys, int64_t(x.u1) * unit));
    p[PC_T0] = it.row0 / (D.H / D.Hkv);
    p[PC_SLOT] = -1;
    if (slot0[x.item] >= 0) {
      const auto& v = starts[x.item];
      p[PC_SLOT] = slot0[x.item] + int32_t(std::lower_bound(v.begin(), v.end(), x.u0) - v.begin());
    }
    L->pieces.insert(L->pieces.end(), p, p + kPieceWords);
    int32_t* R = &L->records[size_t(x.cta) * kRecordWords];
    if (R[RC_P1] == 0) {
      R[RC_P0] = int32_t(i);
      std::copy(p, p + kPieceWords, R + RC_PIECE);
    }
    R[RC_P1] = int32_t(i) + 1;
  }
}

// Few-rows blocks: short against their keys, cheap to join: cut evenly, unless whole blocks
// take no more than a join does longer (8 units of 32 keys, 4 at head dim 256: one sequence
// of 128 keys takes 4.4 us whole and 5.6 cut, of 256 keys 5.9 and 5.8, and a launch less on
// the host). A piece's own cost (its q, adding up the warps' results, the pipeline's start) is some
// 8 units of 32 keys (64 ragged e4m3 sequences of 32 heads: 352 us counting 6, 348 counting 8,
// 351 counting 14). One head's blocks are cut into as many stretches as there are gangs
// of CTAs, a CTA for each head: neighbouring CTAs then read neighbouring heads' parts
// of the same rows at the same time, which HBM serves faster than rows of a head on their own
// (64 ragged sequences: e4m3 rows of 8 x 128 bytes 105 -> 94 us, 8 x 256 bytes of bf16 177
// -> 172).
void dec_lists(const bd_paged_desc& D, const std::vector<Item>& items, const Seqs& S, Lists* L) {
  constexpr int kOver = 8;
  const int join = D.d == 256 ? 4 : 8;
  std::vector<Part> parts;
  if (!items.empty()) {
    const int gang = gang_of(D.Hkv);
    std::vector<Item> lead;           // the blocks of every gang's first head
    std::vector<int32_t> at, blocks;  // their places in `items`; the next head's are `blocks` on
    for (size_t i = 0; i < items.size();) {
      size_t n = 1;  // blocks of this sequence and a head
      while (i + n < items.size() && items[i + n].seq == items[i].seq && items[i + n].hkv == items[i].hkv) ++n;
      for (int32_t h = 0; h < D.Hkv; h += gang)
        for (size_t k = 0; k < n; ++k) {
          at.push_back(int32_t(i + h * n + k));
          blocks.push_back(int32_t(n));
          lead.push_back(items[at.back()]);
        }
      i += n * D.Hkv;
    }
    std::vector<Part> first, whole;
    const int64_t even = cut_evenly(lead, kDecUnit, kOver, kDecCtas / gang, &first);
    if (cut_longest(lead, kDecUnit, kOver, INT32_MAX, kDecCtas / gang, &whole) <= even + join) first.swap(whole);
    parts.reserve(first.size() * gang);
    for (size_t i = 0, j = 0; i < first.size(); i = j) {
      while (j < first.size() && first[j].cta == first[i].cta) ++j;
      for (int g = 0; g < gang; ++g)
        for (size_t k = i; k < j; ++k) {
          const Part& x = first[k];
          parts.push_back({at[x.item] + g * blocks[x.item], x.u0, x.u1, x.cta * gang + g});
        }
    }
  }
  write_lists(D, items, parts, S, kDecUnit, kDecCtas, L);
}

// Tiles: a partial result is up to 256 rows of O in fp32, written and read again, so
// blocks are cut only where that shortens the whole: the best of no cuts, equal parts
// of the longest blocks, and whole blocks with the gaps filled by parts of the others,
// by their longest load in key tiles (a piece costs kOver more, a join of n partial
// results about 3 + n / 40).
void tile_lists(const bd_paged_desc& D, const std::vector<Item>& items, const Seqs& S, Lists* L) {
  constexpr int kOver = 2;
  std::vector<Part> best, parts;
  if (!items.empty()) {
    int64_t total = 0;
    for (const Item& it : items) total += units_of(it, kTile) + kOver;
    const int64_t share = (total + kTileCtas - 1) / kTileCtas;
    int64_t least = cut_longest(items, kTile, kOver, INT32_MAX, kTileCtas, &best);
    std::vector<int32_t> count(items.size());
    auto joined = [&](const std::vector<Part>& v) {
      std::fill(count.begin(), count.end(), 0);
      for (const Part& p : v) ++count[p.item];
      int64_t n = 0;
      for (int32_t c : count) n += c > 1 ? c : 0;
      return n ? 3 + n / 40 : 0;
    };
    auto better = [&](int64_t t) {
      const int64_t cost = t + joined(parts);
      if (cost >= least) return;
      least = cost;
      best.swap(parts);
    };
    // (within 1.5% of an even share nothing is gained)
    const int64_t fine = share + share / 64;
    for (int k = 1; k <= 4 && least > fine; ++k) {
      const int64_t t = cut_longest(items, kTile, kOver, std::max<int64_t>(1, share / k), kTileCtas, &parts);
      if (t < 0) break;
      better(t);
    }
    // the least t that can be filled, between one that cannot (or an even share) and one
    // that can, to 0.5%
    int64_t lo = share, step = 1 + share / 200, hi = lo + step;
    if (least <= fine) hi = least;
    while (hi + 3 < least && !fill(items, kTile, kOver, hi, &parts)) {
      lo = hi;
      step *= 2;
      hi += step;
    }
    while (hi + 3 < least && hi - lo > 1 + share / 200) {
      const int64_t mid = (lo + hi) / 2;
      if (fill(items, kTile, kOver, mid, &parts)) hi = mid;
      else lo = mid;
    }
    if (hi + 3 < least && fill(items, kTile, kOver, hi, &parts)) better(hi);
  }
  write_lists(D, items, best, S, kTile, kTileCtas, L);
}

int32_t validate(const bd_paged_desc* D, int64_t* T, int64_t* kv, int64_t* npages) {
  if (!D) return fail(BD_ERR_ARG, "desc is NULL");
  if (D->B <= 0) return fail(BD_ERR_ARG, "B must be positive");
  if (!D->q_len || !D->kv_len || !D->page_offsets) return fail(BD_ERR_ARG, "q_len, kv_len or page_offsets is NULL");
  if (D->d != 64 && D->d != 128 && D->d != 256) return fail(BD_ERR_UNSUPPORTED, "head dim %d (64, 128, 256 supported)", D->d);
  if (D->H <= 0 || D->Hkv <= 0) return fail(BD_ERR_ARG, "H and Hkv must be positive");
  if (D->H % D->Hkv != 0 || D->H / D->Hkv > 128)
    return fail(BD_ERR_UNSUPPORTED, "H = %d must be a multiple of Hkv = %d, at most 128 times it", D->H, D->Hkv);
  if (D->page_size < 16 || D->page_size > 1024 || (D->page_size & (D->page_size - 1)))
    return fail(BD_ERR_UNSUPPORTED, "page_size %d (a power of two from 16 to 1024)", D->page_size);
  if (D->num_pages <= 0) return fail(BD_ERR_ARG, "num_pages must be positive");
  if (int64_t(D->num_pages) * D->page_size > INT32_MAX) return fail(BD_ERR_CAPACITY, "num_pages * page_size past 2^31 - 1");
  if (D->fmt != BD_CACHE_BF16 && D->fmt != BD_CACHE_E4M3 && D->fmt != BD_CACHE_E2M1) return fail(BD_ERR_ARG, "cache format %d", D->fmt);
  if (D->causal != 0 && D->causal != 1) return fail(BD_ERR_ARG, "causal must be 0 or 1");
  *T = *kv = *npages = 0;
  for (int32_t b = 0; b < D->B; ++b) {
    const int32_t q = D->q_len[b], n = D->kv_len[b];
    if (q < 0 || n < 0) return fail(BD_ERR_ARG, "sequence %d: q_len %d or kv_len %d negative", b, q, n);
    // (kernels step up to a tile past a sequence's end)
    if (n > INT32_MAX - 4096) return fail(BD_ERR_CAPACITY, "sequence %d: kv_len %d", b, n);
    const int32_t o0 = D->page_offsets[b], o1 = D->page_offsets[b + 1];
    if (o0 < 0 || o1 < o0) return fail(BD_ERR_ARG, "page_offsets decrease or are negative at sequence %d", b);
    const int64_t used = (int64_t(n) + D->page_size - 1) / D->page_size;
    if (used > int64_t(o1) - o0)
      return fail(BD_ERR_ARG, "sequence %d: %d pages listed, kv_len %d takes %lld", b, o1 - o0, n, (long long)used);
    if (used && !D->pages) return fail(BD_ERR_ARG, "pages is NULL");
    for (int64_t i = 0; i < used; ++i)
      if (D->pages[o0 + i] < 0 || D->pages[o0 + i] >= D->num_pages)
        return fail(BD_ERR_ARG, "sequence %d: page %d (entry %lld) outside [0, %d)", b, D->pages[o0 + i], (long long)i,
                    D->num_pages);
    *T += q; *kv += n; *npages += used;
  }
  // (the read back counts groups of 8 rows of pages, also of pages used in part)
  if (*npages > INT32_MAX / (D->page_size / 8)) return fail(BD_ERR_CAPACITY, "pages in use times page_size past 2^34");
  if (*T > INT32_MAX / D->H || *kv > INT32_MAX) return fail(BD_ERR_CAPACITY, "new rows times H, or cached rows, past 2^31 - 1");
  return BD_OK;
}

struct Built {
  int64_t T, kv, npages, ntouch = 0;
  std::vector<Item> dec_items, tile_items;
  Seqs S;                          // of the items
  std::vector<int32_t> page_off;   // of the sequences
  int32_t dec_rows, dec_live = 0, sel_cap = 0, sel_rows = 1, sel_split = 1;
  int64_t sel_groups = 0;
};

int32_t check_sparse(const bd_paged_desc* D, const bd_sparse_desc* X) {
  if (!X) return fail(BD_ERR_ARG, "sparse is NULL");
  if (!D) return fail(BD_ERR_ARG, "desc is NULL");
  if (X->first < 0 || X->recent < 1 || X->blocks < 1 || X->blocks > kMostListed)
    return fail(BD_ERR_ARG, "lists of %d blocks with %d first and %d recent ones (1..%d, at least 0 and 1)", X->blocks, X->first,
                X->recent, kMostListed);
  if (int64_t(X->first) + X->recent > X->blocks)
    return fail(BD_ERR_ARG, "lists of %d blocks do not hold %d first and %d recent ones", X->blocks, X->first, X->recent);
  if (D->causal != 1) return fail(BD_ERR_ARG, "rows of a plan that is not causal have no position: it cannot be sparse");
  return BD_OK;
}

// Validates a description and lists its blocks.
int32_t prepare(const bd_paged_desc* D, const bd_sparse_desc* X, Built* B) {
  int32_t st = validate(D, &B->T, &B->kv, &B->npages);
  if (st) return st;
  const int G = D->H / D->Hkv, P = D->page_size;
  std::vector<int32_t> q0(D->B);
  B->page_off.resize(D->B);
  int64_t t = 0, pg = kOffLists + B->T;
  for (int32_t b = 0; b < D->B; ++b) {
    const int32_t q = D->q_len[b], n = D->kv_len[b];
    q0[b] = int32_t(t);
    B->page_off[b] = int32_t(pg);
    t += q;
    pg += (int64_t(n) + P - 1) / P;
    if (pg > INT32_MAX) return fail(BD_ERR_CAPACITY, "plan blob past 2^31 words");
    if (D->causal && q > 0 && n > 0) B->ntouch += (n - 1) / P - std::max(0, n - q) / P + 1;
    if (X && (int64_t(n) + P - 1) / P > kMostBlocks)
      return fail(BD_ERR_UNSUPPORTED, "sequence %d: kv_len %d is more than %d blocks of %d rows", b, n, kMostBlocks, P);
  }
  // Sequences of up to 32 (bf16) or 48 (8 and 4 bits) (new row, head) pairs of a K/V head go to the
  // few-rows kernel, in blocks of one size (a tile of 32 rows in use costs what one of 128
  // does). 16 sequences of 8000 rows, bf16 d 256, 32 pairs: 220 us, as tiles 253; d 128, 48
  // pairs: 195 and 138; e4m3 d 128, 48 pairs in three blocks: 144, as tiles 167; 64 pairs of
  // 300-8000 rows: 66 and 63; e2m1, 48 pairs of 8 K/V heads: d 64 91, as tiles 136, d 128 127 and 153, d 256 276 and
  // 329 (64 of 300-8000 rows 355 and 343; of 2 heads 72 and 68, 4 of 3000 rows 15 and 22: past 32 pairs of
  // long sequences tiles gain some 5% there, and take 1.4 to 2.4 times as long for short ones). Rows with blocks of
  // their own go there one by one.
  const int most = dec_most_rows(D->fmt);
  int32_t widest = 1;
  if (X) widest = G;
  else
    for (int32_t b = 0; b < D->B; ++b)
      if (int64_t(D->q_len[b]) * G <= most) widest = std::max(widest, D->q_len[b] * G);
  B->dec_rows = dec_rows_for(D->fmt, widest);
  // every row block of a (sequence, K/V head): keys up to what its last row sees
  std::vector<Item>&dec = B->dec_items, &tile = B->tile_items;
  int64_t nitems = 0;
  for (int32_t b = 0; b < D->B; ++b)
    nitems += X ? int64_t(D->q_len[b]) * ((G + 7) / 8) * D->Hkv : (int64_t(D->q_len[b]) * G + 7) / 8 * D->Hkv;
  if (nitems > (1 << 26)) return fail(BD_ERR_CAPACITY, "plan of more than 2^26 row blocks");
  if (X) {
    Seqs& S = B->S;
    int32_t widest_row = 1;
    for (int32_t b = 0; b < D->B; ++b)
      for (int32_t i = 0; i < D->q_len[b]; ++i) {
        const int64_t pos = int64_t(D->kv_len[b]) - D->q_len[b] + i;
        const int32_t nblk = pos < 0 ? 0 : int32_t(pos / P) + 1, n = std::min(nblk, X->blocks);
        const int32_t keys = pos < 0 ? 0 : int32_t((n - 1) * P + pos % P + 1);
        const int32_t row = int32_t(S.q0.size());
        widest_row = std::max(widest_row, nblk);
        S.q0.push_back(row);
        S.q_len.push_back(1);
        S.kv_len.push_back(keys);
        S.page_off.push_back(B->page_off[b]);
        S.nblk.push_back(nblk);
        for (int32_t g = 0; g < D->Hkv; ++g)
          for (int32_t r0 = 0; r0 < G; r0 += B->dec_rows) {
            const int32_t r1 = std::min(G, r0 + B->dec_rows);
            B->dec_live = std::max(B->dec_live, r1 - r0);
            dec.push_back({row, g, r0, r1 - r0, keys});
          }
      }
    B->sel_cap = 512;
    while (B->sel_cap < widest_row) B->sel_cap *= 2;
    auto groups = [&](int rows) {
      int64_t n = 0;
      for (int32_t b = 0; b < D->B; ++b) n += (int64_t(D->q_len[b]) + rows - 1) / rows;
      return n;
    };
    B->sel_rows = kSelRows;
    while (B->sel_rows > 1 && (groups(B->sel_rows) * D->Hkv < kSelCtas || select_smem(B->sel_rows, G, D->d, B->sel_cap) > kSelSmem))
      B->sel_rows /= 2;
    B->sel_groups = groups(B->sel_rows);
    if (B->sel_rows == 1 && B->sel_cap > kSelSplitCap)
      while (B->sel_split < kSelMostSplit && 2 * B->sel_split * B->sel_groups * D->Hkv <= kPagedSms) B->sel_split *= 2;
    return BD_OK;
  }
  for (int32_t b = 0; b < D->B; ++b) {
    const int32_t q = D->q_len[b], n = D->kv_len[b], rows = q * G;
    const bool few = rows <= most;
    const int32_t step = few ? B->dec_rows : 128 / G * G * tile_slots(D->d);
    for (int32_t g = 0; g < D->Hkv; ++g)
      for (int32_t r0 = 0; r0 < rows; r0 += step) {
        const int32_t r1 = std::min(rows, r0 + step);
        const int64_t seen = D->causal ? int64_t(n) - q + (r1 - 1) / G + 1 : n;
        if (few) B->dec_live = std::max(B->dec_live, r1 - r0);
        (few ? dec : tile).push_back({b, g, r0, r1 - r0, int32_t(std::max<int64_t>(0, seen))});
      }
  }
  B->S.q0 = q0;
  B->S.q_len.assign(D->q_len, D->q_len + D->B);
  B->S.kv_len.assign(D->kv_len, D->kv_len + D->B);
  B->S.page_off = B->page_off;
  B->S.nblk.assign(D->B, 0);
  return BD_OK;
}

// The pieces are read 16 bytes at a time: each list starts on a multiple of 4 words.
int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

// Words of the header, the fixed places and the lists of rows and pages.
int64_t list_words(const Built& X, bool sparse) {
  return up4(kOffLists + (sparse ? 3 : 2) * X.T + 3 * X.npages + X.ntouch + (X.sel_rows > 1 ? 2 * X.sel_groups : 0));
}

// Words that hold the plan however its blocks are cut: a cut block's parts but one come
// out of the slots.
int64_t most_words(const Built& X, bool sparse) {
  int64_t w = list_words(X, sparse);
  if (!X.dec_items.empty()) w += (int64_t(X.dec_items.size()) + kDecSlots) * kPieceWords;
  if (!X.tile_items.empty()) w += (int64_t(X.tile_items.size()) + kTilePartSlots) * kPieceWords;
  return w;
}

}  // namespace

}  // namespace bd

using namespace bd;

// No exception leaves the library: running out of host memory is an error like others.
template <class F>
static int32_t guarded(F&& f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(BD_ERR_CAPACITY, "out of host memory");
  } catch (const std::length_error&) {
    return fail(BD_ERR_CAPACITY, "plan too large for host memory");
  }
}

static int32_t plan_bytes(const bd_paged_desc* desc, const bd_sparse_desc* sparse, size_t* bytes) {
  if (!bytes) return fail(BD_ERR_ARG, "bytes is NULL");
  Built X;
  int32_t st = prepare(desc, sparse, &X);
  if (st) return st;
  const int64_t w = most_words(X, sparse);
  if (w > INT32_MAX) return fail(BD_ERR_CAPACITY, "plan blob past 2^31 words");
  *bytes = size_t(w) * 4;
  return ok();
}

static int32_t plan_build(const bd_paged_desc* desc, const bd_sparse_desc* sparse, void* blob, size_t blob_bytes) {
  if (!blob || reinterpret_cast<uintptr_t>(blob) % 16) return fail(BD_ERR_ARG, "blob NULL or not 16-byte aligned");
  Built X;
  int32_t st = prepare(desc, sparse, &X);
  if (st) return st;
  const int64_t most = most_words(X, sparse);
  if (most > INT32_MAX) return fail(BD_ERR_CAPACITY, "plan blob past 2^31 words");
  if (blob_bytes < size_t(most) * 4)
    return fail(BD_ERR_CAPACITY, "plan blob of %zu bytes, %lld needed", blob_bytes, (long long)most * 4);
  const bd_paged_desc& D = *desc;
  Lists dec, tile;
  dec_lists(D, X.dec_items, X.S, &dec);
  tile_lists(D, X.tile_items, X.S, &tile);
  const int64_t words = list_words(X, sparse) + int64_t(dec.pieces.size()) + int64_t(tile.pieces.size());
  int32_t* w = static_cast<int32_t*>(blob);
  std::memset(w, 0, size_t(words) * 4);
  const int32_t P = D.page_size;
  w[PH_MAGIC] = kPagedMagic; w[PH_VERSION] = kPagedVersion; w[PH_WORDS] = int32_t(words);
  w[PH_B] = D.B; w[PH_H] = D.H; w[PH_HKV] = D.Hkv; w[PH_D] = D.d; w[PH_G] = D.H / D.Hkv;
  w[PH_PAGE] = P;
  while ((1 << w[PH_PAGE_SHIFT]) < P) ++w[PH_PAGE_SHIFT];
  w[PH_NUM_PAGES] = D.num_pages; w[PH_FMT] = D.fmt; w[PH_CAUSAL] = D.causal;
  w[PH_T] = int32_t(X.T); w[PH_KV_TOTAL] = int32_t(X.kv);
  const float scale = 1.0f / std::sqrt(float(D.d));
  std::memcpy(&w[PH_SCALE_BITS], &scale, 4);
  w[PH_NPAGES] = int32_t(X.npages);
  w[PH_OFF_TOK] = kOffLists;
  w[PH_OFF_PAGES] = int32_t(w[PH_OFF_TOK] + X.T);
  w[PH_OFF_PGROW] = int32_t(w[PH_OFF_PAGES] + X.npages);
  w[PH_OFF_PGCNT] = int32_t(w[PH_OFF_PGROW] + X.npages);
  w[PH_OFF_POS] = int32_t(w[PH_OFF_PGCNT] + X.npages);
  w[PH_OFF_TOUCH] = int32_t(w[PH_OFF_POS] + X.T);
  w[PH_NTOUCH] = int32_t(X.ntouch);
  if (sparse) {
    w[PH_BLOCKS] = sparse->blocks; w[PH_FIRST] = sparse->first; w[PH_RECENT] = sparse->recent;
    w[PH_OFF_ROWPG] = int32_t(w[PH_OFF_TOUCH] + X.ntouch);
    w[PH_SEL_CAP] = X.sel_cap; w[PH_SEL_ROWS] = X.sel_rows; w[PH_SEL_SPLIT] = X.sel_split;
    w[PH_OFF_SELG] = int32_t(w[PH_OFF_ROWPG] + X.T);
    w[PH_NSELG] = int32_t(X.sel_groups);
    int32_t* group = w + w[PH_OFF_SELG];
    for (int32_t b = 0, t = 0; X.sel_rows > 1 && b < D.B; t += D.q_len[b++])
      for (int32_t i = 0; i < D.q_len[b]; i += X.sel_rows) {
        *group++ = t + i;
        *group++ = std::min(X.sel_rows, D.q_len[b] - i);
      }
    std::copy(X.S.page_off.begin(), X.S.page_off.end(), w + w[PH_OFF_ROWPG]);
  }
  int64_t tok = 0, pg = 0, kv = 0, touch = 0;
  struct Entered { int32_t page, rows, entry; };
  std::vector<Entered> entered;  // pages that new rows enter, once a sequence
  struct Range { int32_t lo, hi; };
  std::vector<Range> written;  // cache rows the new rows take, one range per page touched
  for (int32_t b = 0; b < D.B; ++b) {
    const int32_t q = D.q_len[b], n = D.kv_len[b];
    const int32_t* pages = n ? D.pages + D.page_offsets[b] : nullptr;  // (pages may be NULL when nothing is cached)
    for (int32_t j = 0; j < n; j += P) {
      w[w[PH_OFF_PAGES] + pg] = pages[j / P];
      w[w[PH_OFF_PGROW] + pg] = int32_t(kv + j);
      w[w[PH_OFF_PGCNT] + pg] = std::min(P, n - j);
      if (D.causal && j + P > n - q && q > 0) {
        w[w[PH_OFF_TOUCH] + touch++] = int32_t(pg);
        entered.push_back({pages[j / P], std::min(P, n - j), int32_t(pg)});
      }
      ++pg;
    }
    for (int32_t i = 0; i < q; ++i) {
      const int64_t pos = int64_t(n) - q + i;
      const int32_t row = pos < 0 ? -1 : pages[pos / P] * P + int32_t(pos % P);
      w[w[PH_OFF_POS] + tok] = int32_t(std::max<int64_t>(pos, -1));
      w[w[PH_OFF_TOK] + tok++] = row;
      if (row < 0) continue;
      if (!written.empty() && written.back().hi == row && row % P) written.back().hi = row + 1;
      else written.push_back({row, row + 1});
    }
    kv += n;
  }
  std::sort(written.begin(), written.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  w[PH_WRITE_OK] = D.causal;
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].lo < written[i - 1].hi) w[PH_WRITE_OK] = 0;
  std::sort(entered.begin(), entered.end(), [](const Entered& a, const Entered& b) {
    return std::tie(a.page, b.rows, a.entry) < std::tie(b.page, a.rows, b.entry);
  });
  auto same = [](const Entered& a, const Entered& b) { return a.page == b.page; };
  w[PH_BOUNDS_OK] = D.causal && std::adjacent_find(entered.begin(), entered.end(), same) == entered.end();
  if (!w[PH_BOUNDS_OK]) {
    // bd_block_bounds refuses such a plan, but it may be replayed under a call captured with another:
    // each page once, with the most rows of it that are used, so that no two CTAs write the same bounds
    entered.erase(std::unique(entered.begin(), entered.end(), same), entered.end());
    w[PH_NTOUCH] = int32_t(entered.size());
    for (size_t i = 0; i < entered.size(); ++i) w[w[PH_OFF_TOUCH] + i] = entered[i].entry;
  }
  int64_t at = list_words(X, sparse);
  auto put = [&](const Lists& L, int off, int n, int nm, int rec, int mrg) {
    w[off] = int32_t(at);
    w[n] = int32_t(L.pieces.size() / kPieceWords);
    w[nm] = int32_t(L.merges.size() / kMergeWords);
    std::copy(L.records.begin(), L.records.end(), w + rec);
    std::copy(L.merges.begin(), L.merges.end(), w + mrg);
    std::copy(L.pieces.begin(), L.pieces.end(), w + at);
    at += int64_t(L.pieces.size());
  };
  w[PH_DEC_ROWS] = X.dec_rows;
  w[PH_DEC_LIVE] = X.dec_live;
  int32_t most_parts = 0;
  for (size_t i = 0; i < dec.merges.size(); i += kMergeWords) most_parts = std::max(most_parts, dec.merges[i + MG_N]);
  const int64_t joined = int64_t(dec.merges.size() / kMergeWords) * X.dec_live;
  w[PH_DECM_WIDE] = most_parts > kWideJoin || (most_parts > kWideJoinFew && joined <= kWideCtas);
  put(dec, PH_OFF_DEC, PH_NDEC, PH_NDECM, kOffDecRec, kOffDecMerge);
  put(tile, PH_OFF_TILE, PH_NTILE, PH_NTILEM, kOffTileRec, kOffTileMerge);
  return ok();
}

extern "C" int32_t bd_paged_plan_bytes(const bd_paged_desc* desc, size_t* bytes) {
  return guarded([&] { return plan_bytes(desc, nullptr, bytes); });
}

extern "C" int32_t bd_paged_plan_build(const bd_paged_desc* desc, void* blob, size_t blob_bytes) {
  return guarded([&] { return plan_build(desc, nullptr, blob, blob_bytes); });
}

extern "C" int32_t bd_sparse_plan_bytes(const bd_paged_desc* desc, const bd_sparse_desc* sparse, size_t* bytes) {
  int32_t st = check_sparse(desc, sparse);
  return st ? st : guarded([&] { return plan_bytes(desc, sparse, bytes); });
}

extern "C" int32_t bd_sparse_plan_build(const bd_paged_desc* desc, const bd_sparse_desc* sparse, void* blob, size_t blob_bytes) {
  int32_t st = check_sparse(desc, sparse);
  return st ? st : guarded([&] { return plan_build(desc, sparse, blob, blob_bytes); });
}

extern "C" int32_t bd_paged_plan_key(const void* plan_host, uint64_t* key) {
  if (!key) return fail(BD_ERR_ARG, "key is NULL");
  const int32_t* w = nullptr;
  int32_t st = view_paged_plan(plan_host, &w);
  if (st) return st;
  // what a captured launch holds of the plan (FNV-1a over the words)
  const int32_t fields[] = {w[PH_H], w[PH_HKV], w[PH_D], w[PH_PAGE], w[PH_NUM_PAGES], w[PH_FMT], w[PH_CAUSAL],
                            w[PH_WRITE_OK], w[PH_T] > 0, w[PH_NPAGES] > 0, w[PH_NDEC] > 0 ? w[PH_DEC_ROWS] : 0,
                            w[PH_NDECM] > 0 ? 1 + w[PH_DECM_WIDE] : 0, w[PH_NTILE] > 0, w[PH_NTILEM] > 0,
                            w[PH_BLOCKS], w[PH_FIRST], w[PH_RECENT], w[PH_SEL_CAP], w[PH_SEL_ROWS], w[PH_SEL_SPLIT]};
  uint64_t h = 1469598103934665603ull;
  for (int32_t f : fields)
    for (int i = 0; i < 4; ++i) h = (h ^ ((uint32_t(f) >> (8 * i)) & 255u)) * 1099511628211ull;
  *key = h;
  return ok();
}
