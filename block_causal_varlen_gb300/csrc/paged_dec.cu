// Attention of few query rows over a paged K/V cache, and the join of split key
// ranges, on sm_103a. (dec_e2m1.cu and dec_blocks.cu take the kernel and its launch from here
// for other instantiations: the units are compiled side by side.)
//
// A block of up to 32 rows (the (new row, query head) pairs of one K/V head) over
// keys [k0, k1) computes, per row, m = max_j s_j, l = sum_j 2^(s_j - m) and
// O = sum_j 2^(s_j - m) v_j with s_j = log2(e) q . k_j / sqrt(d), in one pass.
//
// What bounds it is reading K and V once (e2m1: turning them into operands): a few rows use 2 x 2 x rows x d operations
// per key and 4 d bytes, far below the tensor rate, so the products use the
// register-operand matrix instructions (m16n8k16), which want no TMEM and no 128-row
// tiles, and everything is laid out to keep HBM busy:
//   - two persistent CTAs per SM; the host cuts all keys of the batch into equal
//     stretches, one a CTA, so that no SM waits for another, and one CTA's loads go on
//     while the other adds up a block. CTAs of neighbouring heads walk the same keys;
//   - every warp runs on its own: it takes every NW-th chunk of 16 or 32 keys, loads its
//     chunks by TMA into a ring of its own (mbarriers, no CTA-wide barrier in the
//     loop) and keeps its own m, l and O in registers. The ring runs ahead over the
//     ends of blocks, so loads never stop; the warps meet only to add up a block;
//   - the products are S^T = K Q^T and O^T = V^T P^T: keys and head columns fill the 16
//     rows of the A operand, the block's rows its 8 columns, so a block of up to 8 rows
//     (a group's heads of one new row) wastes nothing, and up to 32 rows reuse K's and
//     V's fragments;
//   - e4m3 chunks go from shared memory to fp16 fragments in registers (exact). The
//     contraction order of q . k is permuted so that a lane reads 32 neighbouring
//     codes, the row order of V^T so that it reads 16 of a V row, both free of bank
//     conflicts. Exponents never touch the codes: K's is a factor of the score, V's an
//     addend of the base-2 exponent (m is then the maximum of s_j + e_j, l still the sum of
//     2^(s_j - m)). q is fp16 as well, each row scaled by a power of two to a maximum of 2^14
//     first: exact but for what is below 2^-31 of the row's largest, zero below 2^-40;
//   - e2m1 chunks likewise: a lane's codes of a key share one scale (V) or two (K), which
//     multiply the converted pairs (exact: six significant bits).
// P is rounded to the type of V's operand: bf16 for a bf16 cache (2^-8 relative at
// most, like O itself), fp16 for e4m3 and e2m1 (2^-11; its subnormals, p 2^e (e2m1: p) below
// 2^-21 of the row's largest, to 2^-32 of that), scaled by 2^7 for their sake.
//
// 64 ragged sequences of 500-16000 rows, 8 K/V heads of 128: bf16 (4 pairs a head) 164 us,
// 6.8 TB/s; e4m3 (2 pairs) 92 us, 6.1 TB/s; e2m1 (4 pairs) 73 us, 4.3 TB/s, no longer HBM's: 700
// instructions a chunk of 32 keys, 256 of them the conversions and the scales' products, one
// behind the other in 12 warps an SM, which leave the ALU (it converts at half rate) 52% and the issue
// slots 53% busy. One sequence of 4096 rows 7.5-7.8 us in a graph. (Blocks of 32 bf16 rows at d 128
// and 256 spill some 30 registers, 132 bytes, over lists of blocks 45, 180.)
//
// A row takes nothing from a key it does not see, whatever is there: V's infinities
// and NaN, which a probability of zero would turn to NaN, stay out of the products of
// chunks that some row does not see in full, and are added for the rows that do see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <cstring>
#include <type_traits>

#include "paged.h"
#include "paged_quant.cuh"
#include "ptx.cuh"

namespace bd {
using namespace dev;

namespace {

template <int D, int FMT, int NB>
struct DecCfg {
  static constexpr bool kF8 = FMT == BD_CACHE_E4M3, kF4 = FMT == BD_CACHE_E2M1;
  static constexpr bool kF16 = kF8 || kF4;                    // operands of the products are fp16
  // head dim 256: two warps share a chunk's keys, each with half of the columns. Each
  // loads its half, forms its half of the scores, and adds the other's to them (through
  // shared memory); O's columns are its own.
  static constexpr int kDim = D == 256 ? 128 : D, kSplit = D / kDim;
  static constexpr int kRowBytes = row_bytes(FMT, kDim);      // a warp's part of a key's K (or V) of one head
  static constexpr int kPieces = kRowBytes <= 128 ? 1 : kRowBytes / 128;  // 128-byte pieces of it
  static constexpr int kPieceBytes = kRowBytes / kPieces;
  // keys a warp takes at a time: 32 where that is no more than 8 KB and registers allow
  // (what a chunk costs besides its products then counts half)
  static constexpr int kChunk = kRowBytes <= 128 && NB <= 2 ? 32 : 16;
  static constexpr int kMatBytes = kChunk * kRowBytes;        // K (or V) of a chunk
  static constexpr int kStageBytes = 2 * kMatBytes;
  // (e2m1 turns codes into operands all the time: with 4, 6 and 8 warps 64 ragged sequences took 81.6, 73.0
  // and 73.5 us, one of 4096 rows 7.6, 7.8 and 8.1. More warps cost more at a block's end)
  static constexpr int kWarps = kF4 && NB == 1 ? 6 : 4, kLanes = kWarps / kSplit;  // kLanes: chunks in work at a time
  static constexpr int kThreads = 32 * kWarps;
  // a warp's share of a block is added up 8 rows x kCols columns at a time; head dim 256's
  // scores pass through the same place, two chunks in turn
  static constexpr int kCols = D == 64 ? 32 : 64, kPitch = kCols + 4, kSumFloats = 8 * kPitch;
  static constexpr int kXchg = kSplit == 2 ? kChunk / 16 * NB * 512 : 0;  // a warp's scores
  static constexpr int kSumBytes = kWarps * (kSumFloats * 4 > 2 * kXchg ? kSumFloats * 4 : 2 * kXchg);
  // ring depth: 64 KB of chunks a CTA. (Some 45 KB per SM must be in flight to cover HBM's
  // latency at its rate. More than 128 spreads the SMs' reads over too many pages of HBM:
  // with 96 KB a CTA 64 ragged bf16 sequences took 175 us, 166.5 now; 32 e4m3 heads 352
  // and 339, bf16 d 64 94 and 91.)
  static constexpr int kStages = 65536 / (kWarps * kStageBytes);
  static_assert(kStages >= 2, "a ring of two chunks at least");
  static constexpr int kOffRing = 0;
  static constexpr int kOffSum = kOffRing + kWarps * kStages * kStageBytes;
  static constexpr int kOffMl = kOffSum + kSumBytes;                   // m, l [kWarps][8 NB]
  static constexpr int kOffInv = kOffMl + kWarps * 8 * NB * 2 * 4;     // 1 / l of the block's rows
  static constexpr int kOffRow = kOffInv + 8 * NB * 4;                 // their places in O
  // e4m3: 4-byte words around K's and V's exponent bytes of a chunk's keys, and the low
  // bits of the bytes' addresses relative to k_exp and v_exp
  // (e2m1: kScale scale bytes of a warp's part of a key's K or V instead)
  static constexpr int kScale = kF8 ? 4 : kF4 ? kDim / 16 : 0;
  static constexpr int kOffExp = kOffRow + 8 * NB * 8;                 // [kWarps][kStages][2][kChunk]
  static constexpr int kOffRef = kOffExp + kWarps * kStages * 2 * kChunk * kScale;
  static constexpr int kOffBar = kOffRef + (kF8 ? kWarps * kStages * kChunk : 0);
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmem = kOffAbort + 16 + 1024;         // + alignment slack
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs do not fit an SM's shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), operands bf16 or fp16
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 codes (low, high 16 bits of x) -> two fp16 pairs
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// l times 2^x, x <= 0. An e4m3 cache's m is the maximum of s_j + e_j, l the sum of 2^(s_j - m):
// up to 2^60 for a key, which a single factor, zero below 2^-126, would lose while the
// product still counts (l is 2^-60 at least in the end). O's terms have their 2^e_j already.
__device__ __forceinline__ float weigh_l(float l, float x) {
  return l * ex2(fmaxf(x, -64.f)) * ex2(fminf(x + 64.f, 0.f));
}

// Transpose of an 8 x 8 matrix of 16-bit values: a lane's pair (row lane / 4, columns
// 2 (lane % 4)..) becomes (column lane / 4, rows 2 (lane % 4)..).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// BEHIND: launched behind the tile kernel of the same call (a parameter looked at in the kernel
// instead costs 0.1 us of the smallest calls' 3.7). BLOCKS: pieces are of single new rows, whose
// keys are those of the row's listed blocks, one after another.
template <int D, int FMT, int NB, bool BEHIND, bool BLOCKS>
__global__ void __launch_bounds__(DecCfg<D, FMT, NB>::kThreads, 2)
    bd_paged_dec_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const AttnArgs a) {
  using Cfg = DecCfg<D, FMT, NB>;
  constexpr bool F8 = Cfg::kF8, F4 = Cfg::kF4, F16 = Cfg::kF16;
  constexpr int NW = Cfg::kWarps, NST = Cfg::kStages, kChunk = Cfg::kChunk;
  constexpr int DW = Cfg::kDim, PW = Cfg::kSplit, NL = Cfg::kLanes;
  constexpr int KT = kChunk / 16;            // 16-key tiles of a chunk
  constexpr int KS = DW / 16, MT = DW / 16;  // contraction steps of q . k, 16-column tiles of O
  constexpr float kPShift = 7.f;             // fp16: P is held times 2^7
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 3, rw = lane >> 2;
  const int half = warp % PW, kl = warp / PW;  // this warp's columns, and its place among the chunks
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffAbort);
  const uint32_t ring = sbase + Cfg::kOffRing + warp * NST * Cfg::kStageBytes;
  const uint32_t bars = sbase + Cfg::kOffBar + warp * NST * 8;
  volatile uint8_t* eref = smem + Cfg::kOffRef + warp * NST * kChunk;  // low address bits of the exponents
  const uint32_t exps = sbase + Cfg::kOffExp + warp * NST * kChunk * 2 * Cfg::kScale;
  const int32_t* plan = a.plan;
  const int32_t* rec = plan + kOffDecRec + blockIdx.x * kRecordWords;
  if constexpr (BEHIND) {
    if (threadIdx.x == 0) abort_flag[1] = take_go(a.go + blockIdx.x);
    __syncthreads();
    if (!abort_flag[1]) grid_wait();
    else fence_proxy_async_all();
  } else {
    grid_wait();
  }
  const int p0 = rec[RC_P0], p1 = rec[RC_P1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join: it waits for this grid's end
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (p0 == p1) {
    if constexpr (BEHIND) grid_wait();
    return;
  }
  const int32_t* pieces = plan + plan[PH_OFF_DEC];
  auto piece = [&](int p) { return p == p0 ? rec + RC_PIECE : pieces + p * kPieceWords; };
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    // a chunk's arrivals: the copies' and every lane's exponents or scales
    for (int s = 0; s < NST; ++s) mbar_init(bars + 8 * s, F16 ? 33 : 1);
    fence_barrier_init();
  }
  __syncthreads();
  const int G = a.G, causal = a.causal, pshift = a.page_shift;

  const int brows = min(1 << pshift, kChunk);  // rows of a copy: a chunk's keys lie in one page or, of pages of 16, in two

  // ---- loads: a cursor over this warp's chunks of all pieces, NST chunks ahead of
  // the products. The next chunk's page number is fetched when the one before is
  // issued, so that issuing waits for nothing.
  int cp = p0 - 1, ck = 0, ck1 = 0, chkv = 0, cpages = 0, cpage = 0;  // cpage: of key ck + lane (mod kChunk)
  const int32_t* list = nullptr;  // BLOCKS: the row's list, its entry for the chunk after next, its blocks' number
  int entry = 0, nblk = 0;
  int ceo = 0;  // e2m1: offset of the head's scales
  auto next_chunk = [&]() {
    ck += kChunk * NL;
    bool other = false;  // another piece
    while (ck >= ck1) {
      if (++cp >= p1) return;
      const int32_t* W = piece(cp);
      ck = W[PC_K0] + kChunk * kl;
      ck1 = W[PC_K1];
      chkv = W[PC_HKV];
      cpages = W[PC_PAGES];
      if constexpr (BLOCKS) {
        list = a.blocks + W[PC_Q0] * a.b_sr + chkv * a.b_sh;
        nblk = W[PC_NBLK];
        other = true;
      }
      if constexpr (F4) ceo = chkv * int(a.e_sh) + half * Cfg::kScale;
    }
    const int k = min(ck + lane % kChunk, ck1 - 1);
    if constexpr (BLOCKS) {
      // (whatever the list holds, no block but the row's own sequence's is read)
      if (other) entry = list[k >> pshift];
      cpage = plan[cpages + min(max(entry, 0), nblk - 1)];
      entry = list[min(ck + kChunk * NL + lane % kChunk, ck1 - 1) >> pshift];
    } else {
      cpage = plan[cpages + (k >> pshift)];
    }
  };
  int is = 0;  // stage of the next chunk to come
  uint32_t issued = 0;
  auto issue = [&]() {
    const uint32_t full = bars + 8 * is;
    // row of key ck + lane (mod kChunk) in its page, past the keys' end of the last key in its own
    const int keys = ck1 - ck, row = min(ck + lane % kChunk, ck1 - 1) & ((1 << pshift) - 1);
    const bool two = kChunk == 32 && brows == 16 && keys > 16;  // copies of K and of V: one, or two
    if constexpr (F4) {
      const int64_t o = int64_t(cpage) * a.e_sp + (row * int(a.e_sr) + ceo);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (kChunk == 32 || (lane >> 4) == m)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(exps + ((is * 2 + m) * kChunk + lane % kChunk) * Cfg::kScale),
                       "l"((m ? a.v_exp : a.k_exp) + o), "n"(F4 ? Cfg::kScale : 4)
                       : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
    }
    if constexpr (F8) {
      // the 4-byte words of K's and V's exponents; a word's low address bits for later
      const int64_t o = int64_t(cpage) * a.e_sp + row * int(a.e_sr) + chkv * int(a.e_sh);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (kChunk == 32 || (lane >> 4) == m) {
          const uintptr_t at = reinterpret_cast<uintptr_t>((m ? a.v_exp : a.k_exp) + o);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(exps + ((is * 2 + m) * kChunk + lane % kChunk) * 4),
                       "l"(at & ~uintptr_t(3))
                       : "memory");
        }
      eref[is * kChunk + lane % kChunk] = uint8_t(o & 3);
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
    }
    if (lane == 0) mbar_expect_tx(full, uint32_t(2 * Cfg::kRowBytes) * uint32_t(two ? kChunk : brows));
    __syncwarp();
    if (lane == 0 || (two && lane == 16)) {  // lane 16 is at the second page's first key
      const uint32_t dst = ring + is * Cfg::kStageBytes + lane * Cfg::kPieceBytes;
#pragma unroll
      for (int c = 0; c < Cfg::kPieces; ++c) {
        tma_load_5d(dst + c * kChunk * Cfg::kPieceBytes, &tm_k, full, 0, row, half * Cfg::kPieces + c, chkv, cpage);
        tma_load_5d(dst + Cfg::kMatBytes + c * kChunk * Cfg::kPieceBytes, &tm_v, full, 0, row, half * Cfg::kPieces + c, chkv, cpage);
      }
    }
    is = is + 1 == NST ? 0 : is + 1;
    ++issued;
    next_chunk();
  };

  next_chunk();
  bool ok = true;
  for (int i = 0; i < NST && cp < p1; ++i) issue();
  __syncwarp();
  int cs = 0;  // stage and phase of the next chunk to use
  uint32_t phase = 0, cs2 = 0;

  // ---- q of a block's rows rw + 8 b as B fragments (bf16 as it is)
  uint32_t qb[KS][NB][2];
  auto load_q = [&](int q0, int hkv, int row0, int nrows) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = rw + 8 * b, n = row0 + r, t = n / G;
      const bool live = r < nrows;
      const __nv_bfloat16* qp = a.q + int64_t(q0 + t) * a.q_sr + int64_t(hkv * G + n % G) * a.q_sh + half * DW;
      if constexpr (!F16) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qb[s][b][0] = live ? *reinterpret_cast<const uint32_t*>(qp + 16 * s + 2 * j) : 0u;
          qb[s][b][1] = live ? *reinterpret_cast<const uint32_t*>(qp + 16 * s + 8 + 2 * j) : 0u;
        }
      } else {
        // lane j contracts over codes [x, x + 16) of the row, x as in the K loads below;
        // step s takes four of them
#pragma unroll
        for (int s = 0; s < KS; s += 4) {
          const int x = D == 64 ? 16 * j : 32 * j + (s >> 2) * 16;
          uint4 u = make_uint4(0, 0, 0, 0), v = u;
          if (live) {
            u = *reinterpret_cast<const uint4*>(qp + x);
            v = *reinterpret_cast<const uint4*>(qp + x + 8);
          }
          qb[s][b][0] = u.x; qb[s][b][1] = u.y; qb[s + 1][b][0] = u.z; qb[s + 1][b][1] = u.w;
          qb[s + 2][b][0] = v.x; qb[s + 2][b][1] = v.y; qb[s + 3][b][0] = v.z; qb[s + 3][b][1] = v.w;
        }
      }
    }
  };
  load_q(rec[RC_PIECE + PC_Q0], rec[RC_PIECE + PC_HKV], rec[RC_PIECE + PC_ROW0], rec[RC_PIECE + PC_NROWS]);

  for (int p = p0; p < p1; ++p) {
    const int32_t* W = piece(p);
    const int q0 = W[PC_Q0], qlen = W[PC_QLEN], kvlen = W[PC_KVLEN], hkv = W[PC_HKV], row0 = W[PC_ROW0];
    const int nrows = W[PC_NROWS], k0 = W[PC_K0], k1 = W[PC_K1], slot = W[PC_SLOT];
    // the next block's rows, for its q
    const int32_t* X = piece(min(p + 1, p1 - 1));
    const int xq0 = X[PC_Q0], xhkv = X[PC_HKV], xrow0 = X[PC_ROW0], xnrows = X[PC_NROWS];
    // ---- the rows of this lane's scores, 2 j + e + 8 b: the keys they see, their score
    // factors (fp16: log2(e) / sqrt(d) and the power of two taken out of q)
    float qs[NB][2];
    int lim[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float up_inv = 1.f;
      if constexpr (F16) {
        uint32_t mx = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          mx = __vmaxu2(mx, __vmaxu2(qb[s][b][0] & 0x7fff7fffu, qb[s][b][1] & 0x7fff7fffu));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float2 up = q_factors(mx, &up_inv);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t u = qb[s][b][h];
            qb[s][b][h] = pack_f16(bf16_lo(u) * up.x * up.y, bf16_hi(u) * up.x * up.y);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * j + e + 8 * b;
        lim[b][e] = r >= nrows ? 0 : causal ? kvlen - qlen + (row0 + r) / G + 1 : kvlen;
        qs[b][e] = a.scale_log2 * (F16 ? __shfl_sync(0xffffffffu, up_inv, 4 * (2 * j + e)) : 1.f);
      }
    }
    float m[NB][2], l[NB][2], o[MT][NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      m[b][0] = m[b][1] = -CUDART_INF_F;
      l[b][0] = l[b][1] = 0.f;
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][b][e] = 0.f;
    }
    // keys every live row sees (rows that do not exist see nothing: they need no mask)
    const int all_see = causal ? kvlen - qlen + row0 / G + 1 : kvlen;

    for (int k = k0 + kChunk * kl; k < k1; k += kChunk * NL) {
      const uint32_t st = ring + cs * Cfg::kStageBytes;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * cs, phase, abort_flag))) ok = false;
      // ---- S^T: tiles of 16 keys x 8 rows. Element (e, h) of a tile: row 2 j + e, key
      // rw + 8 h
      float s[KT][NB][4];
#pragma unroll
      for (int y = 0; y < KT; ++y)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[y][b][e] = 0.f;
      if constexpr (F4) {
        // a lane's 32 (head dim 64: 16) neighbouring codes of keys rw + 8 y, and their scales
        uint4 u[2 * KT];
        uint32_t sc[2 * KT];
#pragma unroll
        for (int y = 0; y < 2 * KT; ++y) {
          const int key = 8 * y + rw;
          const uint32_t at = exps + (cs * 2 * kChunk + key) * Cfg::kScale;
          if constexpr (D == 64) {
            const uint2 t = lds64(st + key * 32 + (((j >> 1) ^ ((key >> 2) & 1)) << 4) + (j & 1) * 8);
            u[y] = make_uint4(t.x, t.y, 0u, 0u);
            sc[y] = lds8(at + j);
          } else {
            u[y] = lds128(st + key * 64 + ((j ^ ((key >> 1) & 3)) << 4));
            sc[y] = lds16(at + 2 * j);
          }
        }
#pragma unroll
        for (int x = 0; x < KS / 2; ++x)
#pragma unroll
          for (int y = 0; y < KT; ++y) {
            auto word = [&](const uint4& v) { return x == 0 ? v.x : x == 1 ? v.y : x == 2 ? v.z : v.w; };
            uint32_t f[4], g[4];
            e2m1x8_to_f16(word(u[2 * y]), f);
            e2m1x8_to_f16(word(u[2 * y + 1]), g);
            const uint32_t fs = scale_twice(D == 64 ? sc[2 * y] : x < 2 ? sc[2 * y] & 255u : sc[2 * y] >> 8);
            const uint32_t gs = scale_twice(D == 64 ? sc[2 * y + 1] : x < 2 ? sc[2 * y + 1] & 255u : sc[2 * y + 1] >> 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f[i] = mul_f16x2(f[i], fs);
              g[i] = mul_f16x2(g[i], gs);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int b = 0; b < NB; ++b)
                mma16<true>(s[y][b], f[2 * i], g[2 * i], f[2 * i + 1], g[2 * i + 1], qb[2 * x + i][b][0], qb[2 * x + i][b][1]);
          }
      } else if constexpr (!F8) {
#pragma unroll
        for (int c = 0; c < KS; ++c)
#pragma unroll
          for (int y = 0; y < KT; ++y) {
            uint32_t x[4];
            const uint32_t ch = uint32_t(2 * c + (lane >> 4));
            ldsm4(st + (16 * y + (lane & 15)) * 128 + (ch >> 3) * (kChunk * 128) + (((ch & 7) ^ (lane & 7)) << 4), x);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16<false>(s[y][b], x[0], x[1], x[2], x[3], qb[c][b][0], qb[c][b][1]);
          }
      } else {
#pragma unroll
        for (int c = 0; c < KS / 4; ++c) {
          uint4 u[2 * KT];
#pragma unroll
          for (int y = 0; y < 2 * KT; ++y) {
            const int key = 8 * y + rw;
            if constexpr (D == 64) u[y] = lds128(st + key * 64 + ((j ^ ((key >> 1) & 3)) << 4));
            else u[y] = lds128(st + key * 128 + (((2 * j + c) ^ (key & 7)) << 4));
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < KT; ++y) {
              uint32_t f[4];
              auto word = [&](const uint4& v) { return x == 0 ? v.x : x == 1 ? v.y : x == 2 ? v.z : v.w; };
              e4m3x4_to_f16(word(u[2 * y]), f[0], f[2]);
              e4m3x4_to_f16(word(u[2 * y + 1]), f[1], f[3]);
#pragma unroll
              for (int b = 0; b < NB; ++b)
                mma16<true>(s[y][b], f[0], f[1], f[2], f[3], qb[4 * c + x][b][0], qb[4 * c + x][b][1]);
            }
        }
      }
      if constexpr (PW == 2) {
        // the halves of the scores, each times its factor, meet
        const uint32_t xb = sbase + Cfg::kOffSum + ((cs2 * NW + warp) * KT * NB * 32 + lane) * 16;
        const uint32_t xo = sbase + Cfg::kOffSum + ((cs2 * NW + (warp ^ 1)) * KT * NB * 32 + lane) * 16;
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[y][b][e] *= qs[b][e & 1];
            st_shared_v4(xb + (y * NB + b) * 512, __float_as_uint(s[y][b][0]), __float_as_uint(s[y][b][1]),
                         __float_as_uint(s[y][b][2]), __float_as_uint(s[y][b][3]));
          }
        named_bar_sync(1 + kl, 64);
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 u = lds128(xo + (y * NB + b) * 512);
            s[y][b][0] += __uint_as_float(u.x);
            s[y][b][1] += __uint_as_float(u.y);
            s[y][b][2] += __uint_as_float(u.z);
            s[y][b][3] += __uint_as_float(u.w);
          }
        cs2 ^= 1;
      }
      // what is left to multiply the scores by
      auto factor = [&](int b, int e) { return PW == 2 ? 1.f : F16 ? qs[b][e] : a.scale_log2; };
      // ---- e4m3: the scores times K's factors; ve, V's exponents of this lane's keys
      // k + 8 y + rw
      float ve[2 * KT];
      bool vnan = false;
      uint32_t vb = 0;
      if constexpr (F8) {
        uint32_t kb, low = eref[cs * kChunk + lane % kChunk];
        const uint32_t at = exps + (cs * 2 * kChunk + lane % kChunk) * 4;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(kb) : "r"(at) : "memory");
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(vb) : "r"(at + kChunk * 4) : "memory");
        kb = (kb >> (8 * ((low + uint32_t(reinterpret_cast<uintptr_t>(a.k_exp))) & 3u))) & 255u;
        vb = (vb >> (8 * ((low + uint32_t(reinterpret_cast<uintptr_t>(a.v_exp))) & 3u))) & 255u;
        vnan = __any_sync(0xffffffffu, vb == 255u);
        const float kf = exp_factor(kb), vf = vb == 255u ? 0.f : float(int(vb) - 127);
#pragma unroll
        for (int y = 0; y < 2 * KT; ++y) {
          const float f = __shfl_sync(0xffffffffu, kf, 8 * y + rw);
          ve[y] = __shfl_sync(0xffffffffu, vf, 8 * y + rw);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            s[y >> 1][b][2 * (y & 1)] *= f;
            s[y >> 1][b][2 * (y & 1) + 1] *= f;
          }
        }
      }
      if (k + kChunk > all_see) {
#pragma unroll
        for (int y = 0; y < 2 * KT; ++y)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (k + 8 * y + rw >= lim[b][e]) s[y >> 1][b][2 * (y & 1) + e] = -CUDART_INF_F;
      }
      // ---- running maximum. It moves only when it grows by more than 2^8 (exact: l and O
      // use the same one); f: how far it moves, then as a factor
      float f[NB][2];
      bool grow = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -CUDART_INF_F;
          if constexpr (F4) {  // (the factor is positive)
#pragma unroll
            for (int y = 0; y < KT; ++y) mx = max3f(mx, s[y][b][e], s[y][b][2 + e]);
            mx *= factor(b, e);
          } else {
#pragma unroll
            for (int y = 0; y < 2 * KT; ++y) {
              const float v = s[y >> 1][b][2 * (y & 1) + e];
              mx = fmaxf(mx, F8 ? fmaf(v, factor(b, e), ve[y]) : v * factor(b, e));
            }
          }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          f[b][e] = 0.f;
          if (mx > m[b][e] + 8.f) {
            f[b][e] = m[b][e] - mx;
            m[b][e] = mx;
            grow = true;
          }
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = f[b][e];
            f[b][e] = ex2(x);
            l[b][e] = F8 ? weigh_l(l[b][e], x) : l[b][e] * f[b][e];
          }
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][b][e] *= f[b][e & 1];
      }
      // ---- P^T as B operands: rows 2 j, 2 j + 1 of key rw, turned into keys 2 j, 2 j + 1 of
      // row rw
      uint32_t pb[KT][NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float me[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) me[e] = (m[b][e] == -CUDART_INF_F ? 0.f : m[b][e]) - (F4 ? kPShift : 0.f);
        if constexpr (F4) {  // l is held times 2^kPShift, too
          const float2 f2 = make_float2(factor(b, 0), factor(b, 1)), r2 = make_float2(-me[0], -me[1]);
          float2 sum = make_float2(l[b][0], l[b][1]);
#pragma unroll
          for (int y = 0; y < 2 * KT; ++y) {
            float2 v = ffma2(make_float2(s[y >> 1][b][2 * (y & 1)], s[y >> 1][b][2 * (y & 1) + 1]), f2, r2);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            sum = fadd2(sum, v);
            pb[y >> 1][b][y & 1] = transpose8(pack_f16(v.x, v.y));
          }
          l[b][0] = sum.x;
          l[b][1] = sum.y;
          continue;
        }
#pragma unroll
        for (int y = 0; y < 2 * KT; ++y) {
          const float x0 = fmaf(s[y >> 1][b][2 * (y & 1)], factor(b, 0), -me[0]);
          const float x1 = fmaf(s[y >> 1][b][2 * (y & 1) + 1], factor(b, 1), -me[1]);
          const float p0f = ex2(x0), p1f = ex2(x1);
          l[b][0] += p0f;
          l[b][1] += p1f;
          uint32_t w;
          if constexpr (F8) {
            w = pack_f16(ex2(x0 + (ve[y] + kPShift)), ex2(x1 + (ve[y] + kPShift)));
            if (vnan) {  // a V row of NaN makes P NaN for the rows that see its key
              const int key = 8 * y + rw;
              if (__shfl_sync(0xffffffffu, vb, key) == 255u)
                w |= (k + key < lim[b][0] ? 0x7e00u : 0u) | (k + key < lim[b][1] ? 0x7e000000u : 0u);
            }
          } else {
            w = pack_bf16(p0f, p1f);
          }
          pb[y >> 1][b][y & 1] = transpose8(w);
        }
      }
      // ---- O^T += V^T P^T. Keys at or past k1 may hold anything: their V become zeros. So
      // do V's infinities and NaN where some row does not see every key (e4m3: where a row
      // of V is NaN, which P says to those who see it).
      const uint32_t sv = st + Cfg::kMatBytes;
      uint32_t odd = 0;
      auto values = [&](auto cut) {
        constexpr bool TAIL = decltype(cut)::value;
        auto clean = [&](uint32_t& x) {
          const uint32_t u = __vcmpeq2(x & 0x7f807f80u, 0x7f807f80u);
          x &= ~u;
          odd |= u;
        };
#pragma unroll
        for (int y = 0; y < KT; ++y) {
          uint32_t vm[2] = {~0u, ~0u};
          if constexpr (TAIL) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int key = k + 16 * y + 8 * n + 2 * j;
              vm[n] = (key < k1 ? 0xffffu : 0u) | (key + 1 < k1 ? 0xffff0000u : 0u);
              if constexpr (F8) {
                const int at = 16 * y + 8 * n + 2 * j;
                const uint32_t e0 = __shfl_sync(0xffffffffu, vb, at), e1 = __shfl_sync(0xffffffffu, vb, at + 1);
                vm[n] &= (e0 == 255u ? 0u : 0xffffu) | (e1 == 255u ? 0u : 0xffff0000u);
              }
            }
          }
          if constexpr (F4) {
            // this lane's 16 (head dim 64: 8) neighbouring codes of keys 2 j, 2 j + 1, 8 + 2 j,
            // 9 + 2 j: codes of two keys side by side in a byte, their scales in a pair
            uint32_t x[4][2], sb[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int key = 16 * y + 8 * (z >> 1) + 2 * j + (z & 1);
              const uint32_t at = exps + ((cs * 2 + 1) * kChunk + key) * Cfg::kScale;
              if constexpr (D == 64) {
                x[z][0] = lds32(sv + key * 32 + (((rw >> 2) ^ ((key >> 2) & 1)) << 4) + (rw & 3) * 4);
                sb[z] = lds8(at + (rw >> 1));
              } else {
                const uint2 u = lds64(sv + key * 64 + (((rw >> 1) ^ ((key >> 1) & 3)) << 4) + (rw & 1) * 8);
                x[z][0] = u.x; x[z][1] = u.y;
                sb[z] = lds8(at + rw);
              }
              if constexpr (TAIL) {
                if (k + key >= k1) sb[z] = 0u;
                if (sb[z] > kMostScale) { sb[z] = 0u; odd = 1u; }
              }
            }
            const uint32_t s0 = scale_pair(sb[0] | (sb[1] << 16)), s1 = scale_pair(sb[2] | (sb[3] << 16));
#pragma unroll
            for (int w4 = 0; w4 < (D == 64 ? 1 : 2); ++w4) {
              uint32_t g[4][4];
              auto even = [](uint32_t p, uint32_t q) { return (p & 0x0f0f0f0fu) | ((q << 4) & 0xf0f0f0f0u); };
              auto odds = [](uint32_t p, uint32_t q) { return ((p >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u); };
              e2m1x8_to_f16(even(x[0][w4], x[1][w4]), g[0]);
              e2m1x8_to_f16(odds(x[0][w4], x[1][w4]), g[1]);
              e2m1x8_to_f16(even(x[2][w4], x[3][w4]), g[2]);
              e2m1x8_to_f16(odds(x[2][w4], x[3][w4]), g[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = mul_f16x2(g[0][i], s0), a1 = mul_f16x2(g[1][i], s0);
                const uint32_t a2 = mul_f16x2(g[2][i], s1), a3 = mul_f16x2(g[3][i], s1);
#pragma unroll
                for (int b = 0; b < NB; ++b) mma16<true>(o[w4 * 4 + i][b], a0, a1, a2, a3, pb[y][b][0], pb[y][b][1]);
              }
            }
          } else if constexpr (!F8) {
            const uint32_t vrow = sv + (16 * y + ((lane >> 4) & 1) * 8 + (lane & 7)) * 128;
#pragma unroll
            for (int n = 0; n < MT; ++n) {
              uint32_t x[4];
              const uint32_t ch = uint32_t(2 * n + ((lane >> 3) & 1));
              ldsm4t(vrow + (ch >> 3) * (kChunk * 128) + (((ch & 7) ^ (lane & 7)) << 4), x);
              if constexpr (TAIL) {
                x[0] &= vm[0]; x[1] &= vm[0]; x[2] &= vm[1]; x[3] &= vm[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) clean(x[i]);
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) mma16<false>(o[n][b], x[0], x[1], x[2], x[3], pb[y][b][0], pb[y][b][1]);
            }
          } else {
            // A's rows rw and rw + 8 of a tile are neighbouring columns of V: of this lane's
            // 16 (8) neighbouring codes of keys 2 j, 2 j + 1, 8 + 2 j, 9 + 2 j, paired key by key
            uint32_t x[4][4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int key = 16 * y + 8 * (z >> 1) + 2 * j + (z & 1);
              if constexpr (D == 64) {
                const uint2 u = lds64(sv + key * 64 + (((rw >> 1) ^ ((key >> 1) & 3)) << 4) + (rw & 1) * 8);
                x[z][0] = u.x; x[z][1] = u.y;
              } else {
                const uint4 u = lds128(sv + key * 128 + ((rw ^ (key & 7)) << 4));
                x[z][0] = u.x; x[z][1] = u.y; x[z][2] = u.z; x[z][3] = u.w;
              }
            }
#pragma unroll
            for (int w4 = 0; w4 < (D == 64 ? 2 : 4); ++w4)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                // bytes (k, k') of codes 0, 1 (c = 0) or 2, 3 of the word
                uint32_t g[4];
                e4m3x4_to_f16(__byte_perm(x[0][w4], x[1][w4], c ? 0x7362 : 0x5140), g[0], g[1]);
                e4m3x4_to_f16(__byte_perm(x[2][w4], x[3][w4], c ? 0x7362 : 0x5140), g[2], g[3]);
                if constexpr (TAIL) { g[0] &= vm[0]; g[1] &= vm[0]; g[2] &= vm[1]; g[3] &= vm[1]; }
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  mma16<true>(o[w4 * 2 + c][b], g[0], g[1], g[2], g[3], pb[y][b][0], pb[y][b][1]);
              }
          }
        }
      };
      if (k + kChunk > min(k1, all_see) || (F8 && vnan)) values(std::true_type());
      else values(std::false_type());
      if constexpr (F4) {
        if (__any_sync(0xffffffffu, odd != 0)) {
          for (int key = 0; key < min(kChunk, k1 - k); ++key) {  // this lane's columns are of one scale
            if (lds8(exps + ((cs * 2 + 1) * kChunk + key) * Cfg::kScale + (D == 64 ? rw >> 1 : rw)) <= kMostScale) continue;
#pragma unroll
            for (int n = 0; n < MT; ++n)
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (k + key < lim[b][e & 1]) o[n][b][e] = CUDART_NAN_F;
          }
        }
      }
      if constexpr (!F16) {
        if (__any_sync(0xffffffffu, odd != 0)) {
          for (int key = 0; key < min(kChunk, k1 - k); ++key)
#pragma unroll
            for (int n = 0; n < 2 * MT; ++n) {  // this lane's columns 8 n + rw
              uint16_t u;
              const uint32_t at = sv + key * 128 + (n >> 3) * (kChunk * 128) + (((n & 7) ^ (key & 7)) << 4) + rw * 2;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
              if ((u & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (k + key < lim[b][e]) o[n >> 1][b][2 * (n & 1) + e] += __uint_as_float(uint32_t(u) << 16);
            }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (ok && cp < p1) issue();
      __syncwarp();
      cs = cs + 1 == NST ? 0 : cs + 1;
      phase ^= cs == 0 ? 1u : 0u;
    }

    // the next block's q comes while this block's results are added up
    if (p + 1 < p1) load_q(xq0, xhkv, xrow0, xnrows);

    // ---- add the warps' results up
    float* ml = reinterpret_cast<float*>(smem + Cfg::kOffMl);  // [NW][8 NB][2]
    float* inv = reinterpret_cast<float*>(smem + Cfg::kOffInv);
    int64_t* orow = reinterpret_cast<int64_t*>(smem + Cfg::kOffRow);
    float* sum = reinterpret_cast<float*>(smem + Cfg::kOffSum);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], x);
        // NaN scores leave the maximum alone: what they gave was taken relative to 0
        if (m[b][e] == -CUDART_INF_F && l[b][e] != 0.f) m[b][e] = 0.f;
        if constexpr (F4) m[b][e] -= kPShift;  // l and O are relative to this
        if (rw == 0)
          *reinterpret_cast<float2*>(&ml[(warp * 8 * NB + 8 * b + 2 * j + e) * 2]) = make_float2(m[b][e], l[b][e]);
      }
    __syncthreads();
    float* part = slot < 0 ? nullptr : a.part + int64_t(slot) * slot_floats(kDecSlotRows, D);
    if (int(threadIdx.x) < nrows) {
      const int r = threadIdx.x, n = row0 + r, t = q0 + n / G, h = hkv * G + n % G;
      float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * 8 * NB + r) * 2]);
#pragma unroll
      for (int w = 0; w < NW; w += PW) {
        const float mw = ml[(w * 8 * NB + r) * 2];
        const float lw = ml[(w * 8 * NB + r) * 2 + 1];
        L += mw == -CUDART_INF_F ? 0.f : F8 ? weigh_l(lw, mw - M) : lw * ex2(mw - M);
      }
      inv[r] = M == -CUDART_INF_F ? 0.f : 1.f / L;
      orow[r] = int64_t(t) * a.o_sr + int64_t(h) * a.o_sh;
      if (part) {
        part[r] = M;
        part[kDecSlotRows + r] = L;
      } else if (a.lse) {
        a.lse[int64_t(h) * a.l_sh + t] = M == -CUDART_INF_F ? -CUDART_INF_F : (M + lg2(L)) * 0.69314718055994531f;
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float fac[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[(w * 8 * NB + 8 * b + 2 * j + e) * 2]);
        fac[e] = (m[b][e] == -CUDART_INF_F ? 0.f : ex2(m[b][e] - M)) * (F8 ? 0.0078125f : 1.f);  // 2^-kPShift
      }
#pragma unroll
      for (int rd = 0; rd < DW / Cfg::kCols; ++rd) {
        if (b || rd) __syncthreads();
        // fp16: a lane has columns [16 rw, 16 rw + 16) of 128 (8 of 64), half of which, W, go
        // in a round, kept together
        constexpr int NR = Cfg::kCols / 16, W = Cfg::kCols / 8;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x0 = o[rd * NR + n][b][e] * fac[e], x1 = o[rd * NR + n][b][2 + e] * fac[e];
            float* S = sum + warp * Cfg::kSumFloats + (2 * j + e) * Cfg::kPitch;
            if constexpr (F16) {
              *reinterpret_cast<float2*>(&S[W * rw + 2 * n]) = make_float2(x0, x1);
            } else {
              S[16 * n + rw] = x0;
              S[16 * n + 8 + rw] = x1;
            }
          }
        __syncthreads();
        const int rows = min(8, nrows - 8 * b);
        for (int x = threadIdx.x; x < rows * (PW * Cfg::kCols / 4); x += Cfg::kThreads) {
          const int r = x / (PW * Cfg::kCols / 4), hs = x / (Cfg::kCols / 4) % PW, c = 4 * (x % (Cfg::kCols / 4));
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < NL; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(&sum[(w * PW + hs) * Cfg::kSumFloats + r * Cfg::kPitch + c]);
            t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
          }
          const int col = hs * DW + (F16 ? (c / W) * (DW / 8) + rd * W + c % W : rd * Cfg::kCols + c);
          if (part) {
            *reinterpret_cast<float4*>(part + 2 * kDecSlotRows + (8 * b + r) * D + col) = t;
          } else {
            const float g = inv[8 * b + r];
            *reinterpret_cast<uint2*>(a.o + orow[8 * b + r] + col) = make_uint2(pack_bf16(t.x * g, t.y * g), pack_bf16(t.z * g, t.w * g));
          }
        }
      }
    }
    __syncthreads();
  }
  if constexpr (BEHIND) grid_wait();  // (who waits for this grid's end, waits for the tile kernel's)
  if (!ok) {
    // every copy issued has been waited for in turn; wait (with a limit) for those a
    // wait gave up on, then say so
    for (uint32_t s = 0; s < uint32_t(NST) && s < issued; ++s) {
      const uint32_t last = issued - 1 - ((issued - 1 - s) % NST);
      mbar_wait_drain(bars + 8 * s, (last / NST) & 1);
    }
    if (lane == 0) {
      atomicExch(const_cast<int32_t*>(plan) + PH_STATUS, DEV_TIMEOUT);
      atomicExch(const_cast<int32_t*>(plan) + PH_STATUS_DETAIL, 5);
    }
  }
}

template <int D, int FMT, int NB, bool BEHIND, bool BLOCKS>
int32_t launch_dec_tb(const int32_t* w, const bd_paged_cache* c, const AttnArgs& a, cudaStream_t s) {
  using Cfg = DecCfg<D, FMT, NB>;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(bd_paged_dec_kernel<D, FMT, NB, BEHIND, BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged few-rows)");
    if (dev < 64) done[dev].store(true, std::memory_order_release);
  }
  const int rows = w[PH_PAGE] < Cfg::kChunk ? w[PH_PAGE] : Cfg::kChunk;
  // (256-byte promotion where heads go in gangs: 64 ragged sequences of 32 e4m3 heads 370 -> 349 us)
  const bool near = gang_of(w[PH_HKV]) > 1;
  CUtensorMap mk, mv;
  int32_t st;
  if ((st = make_tmap_pages(&mk, &c->k, c->num_pages, w[PH_HKV], row_bytes(FMT, D), elem_bytes(FMT), "cache k", rows, near,
                            Cfg::kPieceBytes))) return st;
  if ((st = make_tmap_pages(&mv, &c->v, c->num_pages, w[PH_HKV], row_bytes(FMT, D), elem_bytes(FMT), "cache v", rows, near,
                            Cfg::kPieceBytes))) return st;
  const cudaError_t e = launch_kernel(bd_paged_dec_kernel<D, FMT, NB, BEHIND, BLOCKS>, kDecCtas, Cfg::kThreads, Cfg::kSmem, s, mk, mv, a);
  return e == cudaSuccess ? BD_OK : cuda_fail(e, "bd_paged_dec_kernel launch");
}

template <int D, int FMT, int NB, bool BLOCKS>
int32_t launch_dec_t(const int32_t* w, const bd_paged_cache* c, const AttnArgs& a, cudaStream_t s) {
  if constexpr (BLOCKS) return launch_dec_tb<D, FMT, NB, false, true>(w, c, a, s);
  else return a.go ? launch_dec_tb<D, FMT, NB, true, false>(w, c, a, s) : launch_dec_tb<D, FMT, NB, false, false>(w, c, a, s);
}

template <int D, int FMT, bool BLOCKS>
int32_t launch_dec_rows(const int32_t* w, const bd_paged_cache* c, const AttnArgs& a, cudaStream_t s) {
  const int rows = w[PH_DEC_ROWS];
  if (rows == 8) return launch_dec_t<D, FMT, 1, BLOCKS>(w, c, a, s);
  if (rows == 16) return launch_dec_t<D, FMT, 2, BLOCKS>(w, c, a, s);
  if constexpr (dec_block_rows(FMT) >= 24)
    if (rows == 24) return launch_dec_t<D, FMT, 3, BLOCKS>(w, c, a, s);
  if constexpr (dec_block_rows(FMT) >= 32)
    if (rows == 32) return launch_dec_t<D, FMT, 4, BLOCKS>(w, c, a, s);
  return fail(BD_ERR_PLAN, "few-rows blocks of %d rows at head dim %d", rows, D);
}

template <int FMT, bool BLOCKS>
int32_t launch_dec_fmt(const int32_t* w, const bd_paged_cache* c, const AttnArgs& a, cudaStream_t s) {
  const int d = w[PH_D];
  return d == 64    ? launch_dec_rows<64, FMT, BLOCKS>(w, c, a, s)
         : d == 128 ? launch_dec_rows<128, FMT, BLOCKS>(w, c, a, s)
                    : launch_dec_rows<256, FMT, BLOCKS>(w, c, a, s);
}

}  // namespace

}  // namespace bd

#ifndef BD_DEC_KERNEL_ONLY

namespace bd {

namespace {

template <int V>
__device__ __forceinline__ void load_cols(const float* p, float (&o)[V]) {
  if constexpr (V == 2) {
    const float2 t = __ldcg(reinterpret_cast<const float2*>(p));
    o[0] = t.x; o[1] = t.y;
  } else {
#pragma unroll
    for (int v = 0; v < V; v += 4) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(p + v));
      o[v] = t.x; o[v + 1] = t.y; o[v + 2] = t.z; o[v + 3] = t.w;
    }
  }
}

// A row's result from its total l relative to m and this lane's D / 32 columns of O.
template <int V>
__device__ __forceinline__ void store_row(const MergeArgs& a, int t, int h, int lane, float m, float l, const float (&acc)[V]) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  __nv_bfloat16* o = a.o + int64_t(t) * a.o_sr + int64_t(h) * a.o_sh + lane * V;
#pragma unroll
  for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(o + v) = pack_bf16(acc[v] * inv, acc[v + 1] * inv);
  if (lane == 0 && a.lse) a.lse[int64_t(h) * a.l_sh + t] = l == 0.f ? -CUDART_INF_F : (m + lg2(l)) * 0.69314718055994531f;
}

// One row of `cnt` slots by one warp: the maximum and the weights 2^(m_i - M), then the
// sums, whose loads do not depend on one another. P: the row's m in the first slot; l is
// ROWS floats on, O at `o` floats (this lane's columns). Slots first, first + by, ...
template <int D, int ROWS>
__device__ __forceinline__ void join_row(const float* P, int64_t o, int cnt, int first, int by, int lane, float* M, float* L,
                                         float (&acc)[D / 32]) {
  constexpr int V = D / 32;
  constexpr int64_t SL = slot_floats(ROWS, D);
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  float mx = -CUDART_INF_F, l = 0.f;
  for (int i0 = first; i0 < cnt; i0 += 32 * by) {  // 32 slots at a time, lane by lane
    const int i = i0 + lane * by, n = min(32, (cnt - i0 + by - 1) / by);
    const float mi = i < cnt ? __ldcg(P + i * SL) : -CUDART_INF_F, li = i < cnt ? __ldcg(P + i * SL + ROWS) : 0.f;
    float ov[4][V];  // the first slots' O come along with their m and l
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) load_cols(P + o + (i0 + k * by) * SL, ov[k]);
    float mn = mi;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
    mn = fmaxf(mn, mx);
    const float f = mx == -CUDART_INF_F ? 0.f : ex2(mx - mn), w = mi == -CUDART_INF_F ? -1.f : ex2(mi - mn);
    float ls = w < 0.f ? 0.f : weigh_l(li, mi - mn);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
    l = (mx == -CUDART_INF_F ? 0.f : weigh_l(l, mx - mn)) + ls;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= f;
    mx = mn;
    auto add = [&](int k, const float (&x)[V]) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += wk < 0.f ? 0.f : x[v] * wk;
    };
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) add(k, ov[k]);
#pragma unroll 4
    for (int k = 4; k < n; ++k) {
      float t[V];
      load_cols(P + o + (i0 + k * by) * SL, t);
      add(k, t);
    }
  }
  *M = mx;
  *L = l;
}

// Joins of the few-rows kernel, a warp per row. Bound by latency: the plan's entry, then the
// slots. With no shared memory and few registers, a CTA or two find room beside the
// attention's.
template <int D>
__global__ void __launch_bounds__(256) bd_paged_merge_kernel(const MergeArgs a) {
  constexpr int ROWS = kDecSlotRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  const int n = a.plan[PH_NDECM], live = a.plan[PH_DEC_LIVE];
  for (int x = blockIdx.x * 8 + warp; x < n * live; x += gridDim.x * 8) {
    const int32_t* M = a.plan + kOffDecMerge + (x / live) * kMergeWords;
    const int r = x % live, cnt = M[MG_N], slot0 = M[MG_SLOT0], nr = M[MG_ROW0] + r;
    const int t = M[MG_Q0] + nr / a.G, h = M[MG_HKV] * a.G + nr % a.G;
    if (r >= M[MG_NROWS]) continue;
    float acc[D / 32], m, l;
    join_row<D, ROWS>(a.part + int64_t(slot0) * slot_floats(ROWS, D) + r, 2 * ROWS - r + r * D + lane * (D / 32), cnt, 0, 1,
                      lane, &m, &l, acc);
    store_row(a, t, h, lane, m, l, acc);
  }
}

// The same where blocks have many slots (few long sequences, cut over every SM): a CTA
// per row, its warps every eighth slot each.
template <int D>
__global__ void __launch_bounds__(256) bd_paged_wide_merge_kernel(const MergeArgs a) {
  constexpr int V = D / 32, ROWS = kDecSlotRows;
  __shared__ float s_o[8][D];
  __shared__ float s_m[8], s_l[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_wait();
  const int n = a.plan[PH_NDECM], live = a.plan[PH_DEC_LIVE];
  for (int x = blockIdx.x; x < n * live; x += gridDim.x) {
    const int32_t* M = a.plan + kOffDecMerge + (x / live) * kMergeWords;
    const int r = x % live, cnt = M[MG_N], slot0 = M[MG_SLOT0], nr = M[MG_ROW0] + r;
    const int t = M[MG_Q0] + nr / a.G, h = M[MG_HKV] * a.G + nr % a.G;
    if (r >= M[MG_NROWS]) continue;
    float acc[V], m, l;
    join_row<D, ROWS>(a.part + int64_t(slot0) * slot_floats(ROWS, D) + r, 2 * ROWS - r + r * D + lane * V, cnt, warp, 8, lane,
                      &m, &l, acc);
#pragma unroll
    for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = acc[v];
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
    __syncthreads();
    if (warp == 0) {
      float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) mm = fmaxf(mm, s_m[w]);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (s_m[w] == -CUDART_INF_F) continue;
        const float f = ex2(s_m[w] - mm);
        ll += weigh_l(s_l[w], s_m[w] - mm);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += s_o[w][lane * V + v] * f;
      }
      store_row(a, t, h, lane, mm, ll, acc);
    }
    __syncthreads();
  }
}

// Joins of the tile kernel: a warp per row, rows of all split blocks over the grid.
template <int D>
__global__ void __launch_bounds__(256) bd_paged_tile_merge_kernel(const MergeArgs a) {
  constexpr int V = D / 32, ROWS = tile_slot_rows(D);
  grid_wait();
  const int n = a.plan[PH_NTILEM], G = a.G, per = 128 / G * G;  // rows in use of each 128 of a slot
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int x = blockIdx.x * 8 + warp; x < n * ROWS; x += gridDim.x * 8) {
    const int r = x % ROWS, br = (r >> 7) * per + (r & 127);  // row of the block
    const int32_t* M = a.plan + kOffTileMerge + (x / ROWS) * kMergeWords;
    const int cnt = M[MG_N], slot0 = M[MG_SLOT0], nr = M[MG_ROW0] + br;
    const int t = M[MG_Q0] + nr / G, h = M[MG_HKV] * G + nr % G;
    if ((r & 127) >= per || br >= M[MG_NROWS]) continue;
    float acc[V], m, l;
    join_row<D, ROWS>(a.part + int64_t(slot0) * slot_floats(ROWS, D) + r, 2 * ROWS - r + int64_t(r) * D + lane * V, cnt, 0, 1,
                      lane, &m, &l, acc);
    store_row(a, t, h, lane, m, l, acc);
  }
}

}  // namespace

int32_t launch_merge(const MergeArgs& a, int d, bool tile, bool wide, cudaStream_t s) {
  typedef void (*Kernel)(MergeArgs);
  auto pick = [d](Kernel k64, Kernel k128, Kernel k256) { return d == 64 ? k64 : d == 128 ? k128 : k256; };
  const Kernel k = tile   ? pick(bd_paged_tile_merge_kernel<64>, bd_paged_tile_merge_kernel<128>, bd_paged_tile_merge_kernel<256>)
                   : wide ? pick(bd_paged_wide_merge_kernel<64>, bd_paged_wide_merge_kernel<128>, bd_paged_wide_merge_kernel<256>)
                          : pick(bd_paged_merge_kernel<64>, bd_paged_merge_kernel<128>, bd_paged_merge_kernel<256>);
  const cudaError_t e = launch_kernel(k, tile ? kPagedSms * 8 : kWideCtas, 256, 0, s, a);
  return e == cudaSuccess ? BD_OK : cuda_fail(e, "paged join launch");
}

int32_t launch_dec(const int32_t* w, const AttnArgs& a, const bd_paged_cache* c, cudaStream_t s) {
  if (a.blocks) return launch_dec_blocks(w, a, c, s);
  return c->fmt == BD_CACHE_BF16   ? launch_dec_fmt<BD_CACHE_BF16, false>(w, c, a, s)
         : c->fmt == BD_CACHE_E4M3 ? launch_dec_fmt<BD_CACHE_E4M3, false>(w, c, a, s)
                                   : launch_dec_e2m1(w, a, c, s);
}

}  // namespace bd

using namespace bd;

// Partial results of the few-rows kernel, then of the tile kernel (at most
// kDecSlots and kTilePartSlots slots, whatever the lengths; none for a kernel that is not launched).
static size_t dec_part_bytes(const int32_t* w) {
  return w[PH_NDEC] ? size_t(kDecSlots) * slot_floats(kDecSlotRows, w[PH_D]) * 4 : 0;
}
static size_t part_bytes(const int32_t* w) {
  return dec_part_bytes(w) + (w[PH_NTILE] ? size_t(kTilePartSlots) * slot_floats(tile_slot_rows(w[PH_D]), w[PH_D]) * 4 : 0);
}
// ... and behind them the words that order the kernels.
static size_t workspace_size(const int32_t* w) {
  return part_bytes(w) + (w[PH_NDEC] && w[PH_NTILE] ? kDecCtas * sizeof(unsigned long long) : 0);
}

extern "C" int32_t bd_paged_attn_workspace(const void* plan_host, size_t* bytes) {
  if (!bytes) return fail(BD_ERR_ARG, "bytes is NULL");
  const int32_t* w = nullptr;
  int32_t st = view_paged_plan(plan_host, &w);
  if (st) return st;
  *bytes = workspace_size(w);
  return ok();
}

// bd_paged_attn, or with lists of blocks bd_sparse_attn.
static int32_t attend(bool sparse, const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_paged_cache* cache,
                      const bd_blocks* blocks, bd_tensor* out, bd_rowstat* lse, void* workspace, size_t workspace_bytes,
                      void* stream) {
  const int32_t* w = nullptr;
  int32_t st = check_paged(plan_host, plan_dev, cache, &w);
  if (st) return st;
  if (sparse != (w[PH_BLOCKS] > 0))
    return fail(BD_ERR_PLAN, sparse ? "not a sparse plan" : "a sparse plan: its rows attend over lists of blocks (bd_sparse_attn)");
  if (w[PH_T] == 0) return ok();
  if (sparse && (st = check_blocks(blocks, w))) return st;
  if ((st = check_tensor(q, "q", 2, 1, 1, w[PH_H], true))) return st;
  if ((st = check_tensor(out, "out", 2, 1, 1, w[PH_H], false))) return st;
  if (q->rows < w[PH_T] || out->rows < w[PH_T])
    return fail(BD_ERR_ARG, "q/out rows %d/%d < %d new rows of the plan", q->rows, out->rows, w[PH_T]);
  if (lse && (!lse->ptr || reinterpret_cast<uintptr_t>(lse->ptr) % 4))
    return fail(BD_ERR_ARG, "lse: NULL pointer or not 4-byte aligned");
  if (lse && w[PH_H] > 1 && lse->stride_head < w[PH_T])
    return fail(BD_ERR_ARG, "lse stride_head %lld < %d rows", (long long)lse->stride_head, w[PH_T]);
  const size_t need = workspace_size(w);
  if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256))
    return fail(BD_ERR_ARG, "workspace NULL or not 256-byte aligned");
  if (workspace_bytes < need) return fail(BD_ERR_CAPACITY, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
  AttnArgs a;
  a.plan = static_cast<const int32_t*>(plan_dev);
  a.q = static_cast<const __nv_bfloat16*>(q->ptr);
  a.q_sr = q->stride_row; a.q_sh = q->stride_head;
  a.o = static_cast<__nv_bfloat16*>(out->ptr);
  a.o_sr = out->stride_row; a.o_sh = out->stride_head;
  a.lse = lse ? lse->ptr : nullptr;
  a.l_sh = lse ? lse->stride_head : 0;
  a.part = static_cast<float*>(workspace);
  a.blocks = sparse ? blocks->ptr : nullptr;
  a.b_sr = sparse ? blocks->stride_row : 0; a.b_sh = sparse ? blocks->stride_head : 0;
  const int64_t es = elem_bytes(cache->fmt);
  a.vc = static_cast<const uint8_t*>(cache->v.ptr);
  a.v_sp = cache->v.stride_b * es; a.v_sr = cache->v.stride_row * es; a.v_sh = cache->v.stride_head * es;
  a.k_exp = cache->k_exp; a.v_exp = cache->v_exp;
  a.e_sp = cache->exp_stride_page; a.e_sr = cache->exp_stride_row; a.e_sh = cache->exp_stride_head;
  float scale;
  memcpy(&scale, &w[PH_SCALE_BITS], 4);
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.G = w[PH_G]; a.causal = w[PH_CAUSAL]; a.page_shift = w[PH_PAGE_SHIFT];
  float* const dec_part = a.part;
  float* const tile_part = a.part + dec_part_bytes(w) / 4;
  const bool dec = w[PH_NDEC] > 0, tile = w[PH_NTILE] > 0;
  a.go = dec && tile ? reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) + part_bytes(w)) : nullptr;
  // tiles first: their CTAs leave their SMs at different times, which few-rows CTAs fill
  if (tile) {
    a.part = tile_part;
    if ((st = launch_tile(w, a, q, cache, s))) return st;
  }
  if (dec) {
    a.part = dec_part;
    if ((st = launch_dec(w, a, cache, s))) return st;
  }
  MergeArgs m = {a.plan, dec_part, a.o, a.o_sr, a.o_sh, a.lse, a.l_sh, a.G};
  if (w[PH_NDECM] && (st = launch_merge(m, w[PH_D], false, w[PH_DECM_WIDE] != 0, s))) return st;
  m.part = tile_part;
  if (w[PH_NTILEM] && (st = launch_merge(m, w[PH_D], true, false, s))) return st;
  return ok();
}

extern "C" int32_t bd_paged_attn(const void* plan_host, const void* plan_dev, const bd_tensor* q,
                                 const bd_paged_cache* cache, bd_tensor* out, bd_rowstat* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return attend(false, plan_host, plan_dev, q, cache, nullptr, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int32_t bd_sparse_attn(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_paged_cache* cache,
                                  const bd_blocks* blocks, bd_tensor* out, bd_rowstat* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return attend(true, plan_host, plan_dev, q, cache, blocks, out, lse, workspace, workspace_bytes, stream);
}

#endif  // BD_DEC_KERNEL_ONLY
