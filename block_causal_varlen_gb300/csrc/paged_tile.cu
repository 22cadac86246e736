// Attention of many query rows over a paged K/V cache on sm_103a: 128-row tiles on
// the tcgen05 tensor cores.
//
// Per row i: O_i = sum_j 2^(s_ij - m_i) v_j / l_i over the keys j below the row's
// limit, s_ij = log2(e) q_i . k_j / sqrt(d), in one pass over key tiles of 128
// (bd_paged_dec_kernel gives the formulas; this kernel takes the blocks whose rows
// fill enough of a tile).
//
// A tile's 128 rows are (new row, head of the group) pairs of ONE K/V head, new-row-
// major: 128 / G new rows of all G heads. Every key tile in shared memory then serves
// 128 rows per slot however the group is shaped, and the causal edge of a tile is
// 128 / G positions wide instead of 128. Two slots (one at head dim 256, whose O
// takes half of TMEM) take neighbouring tiles and the same K/V; while one slot's
// softmax runs, the tensor core works on the other.
//
//   warp 0       TMA: Q tiles (a box of G heads x 128 / G rows), then the key tiles, one
//                box per page (32 lanes look up and issue pages at once)
//   warps 1, 2   one thread per slot issues its tcgen05 products, taking turns:
//                S = Q K^T into TMEM, O += P V with P read from TMEM
//   warp 3       bf16: clears V rows past the keys' end (a page's unused rows may hold
//                anything, and 0 x NaN is NaN), and infinities and NaN out of V rows that
//                not every row sees; those who see them get them at the block's end, read
//                from the cache (a rare and slow path)
//   warps 4-11   softmax, thread = row; they also store the results (e2m1 at head dim 256: 4-7)
//   warps 12-15  e4m3: turn raw tiles into bf16 ones. A code's bits, shifted into
//                a bf16, are its value times 2^-120; one packed multiplication by
//                2^(120 + e) gives the exact value (e: the row's exponent). e2m1 (at head
//                dim 256 warps 8-15): turn raw tiles, and Q's, into fp16 ones, where a conversion
//                and a multiplication give two exact values; Q's rows are scaled by a power of two to a maximum
//                of 2^14 first (exact but for what is below 2^-31 of the row's largest), and
//                P is fp16 as well
// Work comes from the plan: every CTA walks its own list of pieces (block, key range).
// A piece that is not its block's whole key range stores m, l and O for the join.
//
// What bounds it is the chain softmax -> P V -> next S of a slot: a tile pair takes 3250
// cycles for 2048 of products (4000 with the conversion beside it), a block some 4500
// more. 4096 rows over 16384 keys, 32 / 8 heads of 128: bf16 653 us (1473 TFLOP/s), e4m3 792, e2m1 743
// (1295), with pauses between calls; bf16 681-696 in a row, under the power cap; at d 256 bf16 1493, e4m3
// 2703, e2m1 2020. (The converting kernels spill 9 to 17 registers, 36-68 bytes, the bf16 one at d 256 two.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "paged.h"
#include "paged_quant.cuh"
#include "ptx.cuh"

namespace bd {
using namespace dev;

namespace {

template <int D, int FMT>
struct TileCfg {
  static constexpr bool kF8 = FMT == BD_CACHE_E4M3, kF4 = FMT == BD_CACHE_E2M1;
  static constexpr bool kConv = kF8 || kF4;       // tiles are converted
  static constexpr int kSlots = tile_slots(D);
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows x D bf16
  static constexpr int kStages = D == 256 ? 1 : D == 128 ? 2 : 4;
  static constexpr int kRowBytes = row_bytes(FMT, D);
  static constexpr int kPieceBytes = kRowBytes < 128 ? kRowBytes : 128;  // of a row in shared memory
  static constexpr int kRawBytes = kConv ? 128 * kRowBytes : 0;
  static constexpr int kRawStages = !kConv ? 0 : kF4 && D == 256 ? 2 : D == 256 ? 1 : D == 128 ? 2 : 4;  // K, V, K, V, ...
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kSlots * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffRaw = kOffV + kStages * kTileBytes;
  // Results leave in 128-byte pieces of rows that 8 lanes turn into stores of whole pieces:
  // in registers, or through 4 KB of shared memory per softmax warp; e4m3 has none left
  // for that and takes the slot's Q tile, which then is free only after the results are
  // out. 4096 rows over 16384 (10 ragged sequences for e4m3) in registers and through
  // shared memory: bf16 d 64 624 and 590 us, d 128 650 and 672, d 256 1856 and 1872; e4m3
  // d 128 274 and 272.
  static constexpr bool kTurnInRegs = !kF8 && D >= 128;
  static constexpr bool kStageInQ = kF8 && D >= 128;
  static constexpr int kOffStage = kOffRaw + kRawStages * kRawBytes;
  static constexpr int kOffBar = kOffStage + (kStageInQ || kTurnInRegs ? 0 : kSlots * 16384);
  static constexpr int kOffPieces = kOffBar + 512;
  static constexpr int kPre = kF4 ? 8 : 16;       // pieces kept in shared memory
  static constexpr int kOffQs = kOffPieces + kPre * kPieceWords * 4;  // e2m1: score factors of the rows of two blocks
  static constexpr int kSmem = kOffQs + (kF4 ? 2 * 128 * kSlots * 4 : 0) + 1024;  // + alignment slack
  static constexpr int kOCol = 256;               // first O column in TMEM
  // Whether P is handed to the tensor core in halves. With one slot the first half of P V
  // runs while the second half of P is made (4096 rows over 16384 at d 256: 2090 ->
  // 1890 us); with two the other slot's products fill that time, and the early half only
  // gets in their way (d 128: 668 -> 724).
  static constexpr bool kPHalves = kSlots == 1;
  static constexpr int kThreads = kConv ? 512 : 384;
  // warps from here on convert: with one slot four softmax warps more (e2m1, whose rows go in halves then)
  static constexpr int kConvWarp = kF4 && kSlots == 1 ? 8 : 12;
  static constexpr int kConvThreads = 32 * (16 - kConvWarp);
  // registers after setmaxnreg: warps 0-3, the softmax warps, the converting warps
  static constexpr int kRegsCtl = kConv ? 40 : 72, kRegsSoftmax = kConvWarp == 8 ? 240 : kConv ? 200 : 216, kRegsConv = kConvWarp == 8 ? 112 : 72;
  static constexpr int kRegsLaunch = kConv ? 128 : 168;
  static_assert(128 * kRegsCtl + 32 * (kConvWarp - 4) * kRegsSoftmax + (kConv ? kConvThreads * kRegsConv : 0) <= kRegsLaunch * kThreads,
                "register split exceeds the launch's registers");
  static_assert(kSmem <= 232448, "shared memory over the per-CTA limit");
  static_assert(kOCol + kSlots * D <= 512, "O accumulators exceed TMEM");
};

// barrier indices (8 bytes each)
enum : int {
  T_QFULL = 0, T_QEMPTY, T_KFULL = 4, T_KEMPTY = 8, T_VFULL = 12, T_VEMPTY = 16, T_RFULL = 20, T_REMPTY = 24,
  T_SFULL = 28, T_PFULL = 30, T_OFINAL = 32, T_OEMPTY = 34, T_TURN = 36, T_DRAIN = 38, T_VTAIL = 40, T_PHALF = 44,
  T_QCONV = 46, T_QSEEN = 47, T_COUNT = 48
};
constexpr int kOddMarks = 8;  // at most 4 key tiles, so 4 blocks, are under way at a time
static_assert(8 * T_COUNT + 16 + 4 * kOddMarks <= 512, "barriers, TMEM slot, abort flag and marks overflow their region");

struct Piece {
  int q0, qlen, kvlen, pages, hkv, t0, k0, k1, slot, nt, ns;
  int clear;  // keys that every row of the block sees: below this
};

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;  // subnormal operands keep their values
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four codes as two bf16 pairs times 2^-120: sign, 4 exponent and 3 mantissa bits of
// each at bits 15, 10..7 and 6..4
__device__ __forceinline__ void e4m3x4_bits(uint32_t x, uint32_t& a, uint32_t& b) {
  const uint32_t lo = (x << 4) & 0xf0f0f0f0u;
  const uint32_t hi = (x & 0x80808080u) | ((x >> 4) & 0x07070707u);
  a = __byte_perm(lo, hi, 0x5140);
  b = __byte_perm(lo, hi, 0x7362);
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}

template <int D, int FMT>
__global__ void __launch_bounds__(TileCfg<D, FMT>::kThreads, 1)
    bd_paged_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const AttnArgs a) {
  using Cfg = TileCfg<D, FMT>;
  constexpr bool F8 = Cfg::kF8, F4 = Cfg::kF4, CONV = Cfg::kConv;
  constexpr int NS = Cfg::kSlots, NST = Cfg::kStages, NR = CONV ? Cfg::kRawStages : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + Cfg::kOffQ, sK = sbase + Cfg::kOffK, sV = sbase + Cfg::kOffV, sR = sbase + Cfg::kOffRaw;
  const uint32_t bars = sbase + Cfg::kOffBar;
  auto bar = [&](int i) { return bars + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffBar + 8 * T_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::kOffBar + 8 * T_COUNT + 8);
  // of the n-th block with keys (n = 1, 2, ...): odd[(n - 1) % kOddMarks] >= n if V values
  // were taken out (or if a later block has written over the mark)
  volatile uint32_t* odd = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffBar + 8 * T_COUNT + 16);
  int32_t* pre = reinterpret_cast<int32_t*>(smem + Cfg::kOffPieces);
  // e2m1: score factors of the n-th block's rows at ((n - 1) & 1) * 128 NS. They are read before the
  // block's first P goes to the tensor core, and the block after next is not turned before that
  volatile float* qs = reinterpret_cast<volatile float*>(smem + Cfg::kOffQs);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* plan = a.plan;
  const int32_t* rec = plan + kOffTileRec + blockIdx.x * kRecordWords;
  grid_wait();
  static_assert(kDecCtas == 2 * kTileCtas, "a word for two few-rows CTAs each");
  if (a.go && threadIdx.x < 2) give_go(a.go + 2 * blockIdx.x + threadIdx.x);
  const int p0 = rec[RC_P0], p1 = rec[RC_P1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join: it waits for this grid's end
  if (p0 == p1) return;
  const int32_t* pieces = plan + plan[PH_OFF_TILE];
  const int G = a.G, causal = a.causal, pshift = a.page_shift;
  const int TPS = 128 / G;   // new rows of a slot's tile
  // the record has the first piece; a CTA with more fetches them now
  if (threadIdx.x < kPieceWords) pre[threadIdx.x] = rec[RC_PIECE + threadIdx.x];
  for (int i = kPieceWords + threadIdx.x; i < min(p1 - p0, Cfg::kPre) * kPieceWords; i += Cfg::kThreads)
    pre[i] = pieces[p0 * kPieceWords + i];

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    mbar_init(bar(T_QFULL), 1);
    if (F4) {
      mbar_init(bar(T_QCONV), Cfg::kConvThreads);
      mbar_init(bar(T_QSEEN), Cfg::kConvThreads / 32);
    }
    mbar_init(bar(T_QEMPTY), Cfg::kStageInQ ? 4 * NS : NS);  // softmax warps, or MMA threads
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar(T_KFULL + s), CONV ? Cfg::kConvThreads : 1);
      mbar_init(bar(T_KEMPTY + s), NS);
      mbar_init(bar(T_VFULL + s), CONV ? Cfg::kConvThreads : 1);
      mbar_init(bar(T_VEMPTY + s), NS);
      mbar_init(bar(T_VTAIL + s), 1);
    }
    for (int s = 0; s < NR; ++s) {
      mbar_init(bar(T_RFULL + s), 1);
      mbar_init(bar(T_REMPTY + s), Cfg::kConvThreads);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(T_SFULL + s), 1);
      mbar_init(bar(T_PFULL + s), 128);
      mbar_init(bar(T_PHALF + s), 128);
      mbar_init(bar(T_OFINAL + s), 1);
      mbar_init(bar(T_OEMPTY + s), 128);
      mbar_init(bar(T_TURN + s), 1);
      mbar_init(bar(T_DRAIN + s), 1);
    }
    for (int i = 0; i < kOddMarks; ++i) odd[i] = 0;
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto piece = [&](int p) {
    const int32_t* W = p - p0 < Cfg::kPre ? pre + (p - p0) * kPieceWords : pieces + p * kPieceWords;
    Piece P;
    P.q0 = W[PC_Q0]; P.qlen = W[PC_QLEN]; P.kvlen = W[PC_KVLEN]; P.pages = W[PC_PAGES]; P.hkv = W[PC_HKV];
    P.t0 = W[PC_T0]; P.k0 = W[PC_K0]; P.k1 = W[PC_K1]; P.slot = W[PC_SLOT];
    P.nt = (P.k1 - P.k0 + 127) >> 7;
    P.ns = NS == 2 && P.t0 + TPS < P.qlen ? 2 : 1;
    P.clear = min(P.k1, causal ? P.kvlen - P.qlen + P.t0 + 1 : P.kvlen);
    return P;
  };

  if (warp < 4) {
    regs_set<Cfg::kRegsCtl, Cfg::kRegsLaunch>();
    if (warp == 0) {
      // -------------------------------------------------------- producer (whole warp)
      const int rows = min(1 << pshift, 128);   // rows of a copy
      const int rshift = min(pshift, 7);
      constexpr int kPieceBytes = Cfg::kPieceBytes, kPieces = Cfg::kRowBytes / kPieceBytes;
      uint32_t it = 0, rit = 0, qi = 0;
      bool ok = true;
      // one matrix of the key tile at `pos`, `n` copies, into `dst`
      auto load = [&](const CUtensorMap* m, uint32_t dst, uint32_t full, int n, int pos, int page, int hkv) {
        if (lane == 0) mbar_expect_tx(full, uint32_t(n * rows * kPieceBytes * kPieces));
        __syncwarp();
        if (lane < n) {
          const int row = (pos + lane * rows) & ((1 << pshift) - 1);
#pragma unroll
          for (int c = 0; c < kPieces; ++c)
            tma_load_5d(dst + c * 128 * kPieceBytes + lane * rows * kPieceBytes, m, full, 0, row, c, hkv, page);
        }
        __syncwarp();
      };
      for (int p = p0; p < p1 && ok; ++p) {
        const Piece P = piece(p);
        if (P.nt == 0) continue;
        auto load_q = [&]() -> bool {
          if (!__all_sync(0xffffffffu, mbar_wait(bar(T_QEMPTY), (qi & 1) ^ 1, abort_flag))) return false;
          if (lane == 0) {
            mbar_expect_tx(bar(T_QFULL), uint32_t(P.ns * TPS * G * D * 2));
            for (int s = 0; s < P.ns; ++s)
              for (int c = 0; c < D / 64; ++c)
                tma_load_5d(sQ + s * Cfg::kTileBytes + c * 16384, &tm_q, bar(T_QFULL), c * 64, P.hkv * G,
                            P.q0 + P.t0 + s * TPS, 0, 0);
          }
          __syncwarp();
          ++qi;
          return true;
        };
        // this lane's page of a tile; the next tile's is fetched one tile ahead
        auto page_of = [&](int pos) { return pos + lane * rows < P.k1 && lane * rows < 128 ? plan[P.pages + ((pos + lane * rows) >> pshift)] : 0; };
        int page = page_of(P.k0);
        for (int j = 0; j < P.nt; ++j, ++it) {
          const int pos = P.k0 + 128 * j;
          const int n = (min(P.k1 - pos, 128) + rows - 1) >> rshift;
          const int next = j + 1 < P.nt ? page_of(pos + 128) : 0;
          if constexpr (!CONV) {
            const int s = it % NST;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_KEMPTY + s), ((it / NST) & 1) ^ 1, abort_flag)))) break;
            load(&tm_k, sK + s * Cfg::kTileBytes, bar(T_KFULL + s), n, pos, page, P.hkv);
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_VEMPTY + s), ((it / NST) & 1) ^ 1, abort_flag)))) break;
            // a tile with rows past the keys' end, or that some row does not see, goes by
            // way of warp 3
            load(&tm_v, sV + s * Cfg::kTileBytes, bar((pos + 128 > P.clear ? T_VTAIL : T_VFULL) + s), n, pos, page, P.hkv);
          } else {
            for (int h = 0; h < 2 && ok; ++h, ++rit) {
              const int s = rit % NR;
              if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_REMPTY + s), ((rit / NR) & 1) ^ 1, abort_flag)))) break;
              load(h ? &tm_v : &tm_k, sR + s * Cfg::kRawBytes, bar(T_RFULL + s), n, pos, page, P.hkv);
            }
            if (!ok) break;
          }
          if (j == 0 && !(ok = load_q())) break;
          page = next;
        }
      }
      if (!ok) {
        // let copies already issued land before the CTA's shared memory goes away (what
        // has landed returns at once; each wait is bounded)
        if constexpr (!CONV) {
          for (int s = 0; s < NST; ++s) {
            const uint32_t lk = it + 1;  // K may be one tile further than V
            for (uint32_t x = lk > uint32_t(NST) ? lk - NST : 0; x < lk; ++x)
              if (int(x % NST) == s) mbar_wait_drain(bar(T_KFULL + s), (x / NST) & 1);
            if (it > 0 && it > uint32_t(s)) {
              const uint32_t last = it - 1 - ((it - 1 - s) % NST);
              mbar_wait_drain(bar(T_VFULL + s), (last / NST) & 1);
            }
          }
        } else {
          for (int s = 0; s < NR; ++s)
            if (rit > uint32_t(s)) {
              const uint32_t last = rit - 1 - ((rit - 1 - s) % NR);
              mbar_wait_drain(bar(T_RFULL + s), (last / NR) & 1);
            }
        }
        if (qi > 0) mbar_wait_drain(bar(T_QFULL), (qi - 1) & 1);
      }
    } else if (warp == 1 || (warp == 2 && NS == 2)) {
      // -------------------------------------------------------- MMA issuers, one per slot
      if (lane == 0) {
        const int s = warp - 1;
        uint32_t my_turn = 0;  // groups (a product P V and the next S) this slot has passed
        auto take_turn = [&]() -> bool {
          if (NS == 1 || (s == 0 && my_turn == 0)) return true;
          const uint32_t k = s == 0 ? my_turn - 1 : my_turn;
          return mbar_wait_spin(bar(T_TURN + s), k & 1, abort_flag);
        };
        auto pass_turn = [&]() {
          if (NS == 2) mbar_arrive(bar(T_TURN + (s ^ 1)));
          ++my_turn;
        };
        constexpr uint32_t idS = F4 ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
        constexpr uint32_t idPV = F4 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
        const uint32_t d_s = tmem + s * 128, d_o = tmem + Cfg::kOCol + s * D;
        const uint32_t qa = sdesc_lo(sQ + s * Cfg::kTileBytes, 16);
        auto issue_s = [&](int st) {
          const uint32_t kb = sdesc_lo(sK + st * Cfg::kTileBytes, 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = uint32_t(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
            mma_ss_lo(d_s, qa + off, kb + off, idS, kk > 0);
          }
        };
        // V's tile is free when P V is done, not when the next S is: with one slot and one stage the next
        // tile of V waits for that (4096 rows over 16384 at d 256, bf16: 1854 -> 1493 us). Where tiles are
        // converted, V's then gets in the way of K's (e4m3 2703 -> 2840, e2m1 2020 -> 2038); with two slots
        // it only costs a commit.
        constexpr bool kEarlyV = NS == 1 && !CONV;
        constexpr int kHalf = Cfg::kPHalves ? 4 : 0;  // steps of P V that start after the first half of P
        auto issue_pv = [&](auto from, auto to, int st, bool acc) {
          const uint32_t vb = sdesc_lo(sV + st * Cfg::kTileBytes, 16384);
#pragma unroll
          for (int kk = from; kk < to; ++kk) mma_ts_lo(d_o, d_s + kk * 8, vb + uint32_t(kk * 128), idPV, (acc || kk > 0) ? 1u : 0u);
        };
        using Steps0 = std::integral_constant<int, 0>;
        using StepsH = std::integral_constant<int, kHalf>;
        using Steps8 = std::integral_constant<int, 8>;
        // this slot's part of releasing the Q tiles, after its last product S
        auto release_q = [&](bool act) {
          if (act && !Cfg::kStageInQ) tc_commit(bar(T_QEMPTY));
          if (!act) mbar_arrive_n(bar(T_QEMPTY), Cfg::kStageInQ ? 4 : 1);
        };
        // it: key tiles (stages); qi: blocks; tc, ai: this slot's tiles and blocks
        uint32_t it = 0, qi = 0, tc = 0, ai = 0;
        bool ok = true;
        for (int p = p0; p < p1 && ok; ++p) {
          const Piece P = piece(p);
          if (P.nt == 0) continue;
          const bool act = s < P.ns;
          if (!(ok = mbar_wait(bar(F4 ? T_QCONV : T_QFULL), qi & 1, abort_flag))) break;
          ++qi;
          {
            const int sk = it % NST;
            if (!(ok = mbar_wait(bar(T_KFULL + sk), (it / NST) & 1, abort_flag))) break;
            if (!(ok = take_turn())) break;
            if (act) {
              tc_fence_after();
              issue_s(sk);
              pass_turn();
              tc_commit(bar(T_SFULL + s));
              tc_commit(bar(T_KEMPTY + sk));
            } else {
              pass_turn();
              mbar_arrive(bar(T_KEMPTY + sk));
            }
            if (P.nt == 1) release_q(act);
          }
          for (int j = 1; j <= P.nt; ++j) {
            const uint32_t itp = it + j - 1, itn = it + j;
            const int svp = itp % NST, skn = itn % NST;
            if (act) {
              if (!(ok = mbar_wait_spin(bar((kHalf ? T_PHALF : T_PFULL) + s), (tc + j - 1) & 1, abort_flag))) break;
              if (j == 1 && !(ok = mbar_wait(bar(T_OEMPTY + s), (ai & 1) ^ 1, abort_flag))) break;
            }
            if (!(ok = mbar_wait(bar(T_VFULL + svp), (itp / NST) & 1, abort_flag))) break;
            if constexpr (kHalf > 0) {
              if (act) {
                tc_fence_after();
                issue_pv(Steps0{}, StepsH{}, svp, j > 1);
                if (!(ok = mbar_wait_spin(bar(T_PFULL + s), (tc + j - 1) & 1, abort_flag))) break;
              }
            }
            if (j < P.nt && !(ok = mbar_wait(bar(T_KFULL + skn), (itn / NST) & 1, abort_flag))) break;
            if (!(ok = take_turn())) break;
            if (act) {
              tc_fence_after();
              issue_pv(StepsH{}, Steps8{}, svp, j > 1);
              if (kEarlyV) tc_commit(bar(T_VEMPTY + svp));
              if (j < P.nt) issue_s(skn);
              pass_turn();
              if (!kEarlyV) tc_commit(bar(T_VEMPTY + svp));
              if (j < P.nt) {
                tc_commit(bar(T_SFULL + s));
                tc_commit(bar(T_KEMPTY + skn));
              } else {
                tc_commit(bar(T_OFINAL + s));
              }
            } else {
              pass_turn();
              mbar_arrive(bar(T_VEMPTY + svp));
              if (j < P.nt) mbar_arrive(bar(T_KEMPTY + skn));
            }
            if (j == P.nt - 1) release_q(act);
          }
          it += P.nt;
          if (act) {
            tc += P.nt;
            ++ai;
          }
        }
        if (!ok) {
          tc_commit(bar(T_DRAIN + s));
          mbar_wait_drain(bar(T_DRAIN + s), 0);
        }
      }
    } else if (warp == 3 && !CONV) {
      // -------------------------------------------------------- V rows some do not see
      // Such a tile's load completes T_VTAIL of its stage; this warp completes T_VFULL.
      uint32_t it = 0, n = 0, parity = 0;  // bit s: phase of T_VTAIL + s (a stage's next such load waits for its products)
      bool ok = true;
      for (int p = p0; p < p1 && ok; ++p) {
        const Piece P = piece(p);
        if (P.nt == 0) continue;
        ++n;
        for (int j = max(0, P.clear - P.k0) >> 7; j < P.nt; ++j) {
          const int st = (it + j) % NST, pos = P.k0 + 128 * j;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_VTAIL + st), (parity >> st) & 1, abort_flag)))) break;
          parity ^= 1u << st;
          const uint32_t v = sV + st * Cfg::kTileBytes;
          const int r0 = max(0, P.clear - pos), r1 = min(128, P.k1 - pos);
          // 16-byte pieces of rows [r0, r1), then of those past the end
          uint32_t bad = 0;
#pragma unroll 2
          for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint32_t at = v + c * 16384 + i * 16;
              const uint4 x = ld_shared_u4(at);
              // bit 15 of a half is set if its exponent is all ones
              auto ones = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
              if (((ones(x.x) | ones(x.y) | ones(x.z) | ones(x.w)) & 0x80008000u) == 0) continue;
              auto clean = [](uint32_t w) { return w & ~__vcmpeq2(w & 0x7f807f80u, 0x7f807f80u); };
              st_shared_v4(at, clean(x.x), clean(x.y), clean(x.z), clean(x.w));
              bad = 1;
            }
          for (int i = r1 * 8 + lane; i < 1024; i += 32)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) st_shared_v4(v + c * 16384 + i * 16, 0u, 0u, 0u, 0u);
          if (bad) odd[(n - 1) % kOddMarks] = n;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(T_VFULL + st));
        }
        it += P.nt;
      }
    }
  } else if (warp < Cfg::kConvWarp) {
    regs_set<Cfg::kRegsSoftmax, Cfg::kRegsLaunch>();
    // ---------------------------------------------------------- softmax
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row within the tile == TMEM lane
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + s * 128, tO = tmem + lane_base + Cfg::kOCol + s * D;
    const int tl = r / G, hg = r - tl * G;
    constexpr float kPShift = 7.f;  // e2m1: P, and with it l and O, are held times 2^this
    uint32_t tc = 0, ai = 0, n = 0;
    bool ok = s < NS;
    for (int p = p0; p < p1 && ok; ++p) {
      const Piece P = piece(p);
      n += P.nt > 0 ? 1 : 0;
      if (s >= P.ns) continue;
      const int t = P.t0 + s * TPS + tl, h = P.hkv * G + hg;
      const bool live = tl < TPS && t < P.qlen;
      const int lim = !live ? 0 : causal ? P.kvlen - P.qlen + t + 1 : P.kvlen;
      __nv_bfloat16* orow = a.o + int64_t(P.q0 + t) * a.o_sr + int64_t(h) * a.o_sh;
      float* part = P.slot < 0 ? nullptr : a.part + int64_t(P.slot) * slot_floats(tile_slot_rows(D), D);
      if (P.nt == 0) {  // rows that see nothing
        if (live) {
#pragma unroll
          for (int k = 0; k < D / 8; ++k) reinterpret_cast<uint4*>(orow)[k] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[int64_t(h) * a.l_sh + P.q0 + t] = -CUDART_INF_F;
        }
        continue;
      }
      float m_run = -CUDART_INF_F, l_run = 0.f, row_scale = 0.f;
      for (int j = 0; j < P.nt; ++j, ++tc) {
        // (warps leave together: what follows is warp-wide)
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_SFULL + s), tc & 1, abort_flag)))) break;
        tc_fence_after();
        if (F4 && j == 0) row_scale = qs[((n - 1) & 1) * 128 * NS + s * 128 + r];
        uint32_t u[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, u[q]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) reg_fence(u[q]);
        float x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e) x[q * 32 + e] = __uint_as_float(u[q][e]);
        const float scale = F4 ? row_scale : a.scale_log2;
        // the row sees the tile's columns below `see`; per group of 32 columns the warp
        // skips what no row sees and leaves alone what every row sees
        const int see = lim - (P.k0 + 128 * j);
        uint32_t gone = 0;
        if (__any_sync(0xffffffffu, see < 128)) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (__all_sync(0xffffffffu, see <= 32 * q)) {
              gone |= 1u << q;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[32 * q + e] = -CUDART_INF_F;
            } else if (!__all_sync(0xffffffffu, see >= 32 * q + 32)) {
              const int c = see - 32 * q;
              const uint32_t seen = c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1u;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[32 * q + e] = (seen & (1u << e)) ? x[32 * q + e] : -CUDART_INF_F;
            }
          }
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = -CUDART_INF_F;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!(gone & (1u << q)))
#pragma unroll
            for (int e = 32 * q; e < 32 * q + 32; e += 16)
#pragma unroll
              for (int k = 0; k < 8; ++k) m8[k] = max3f(m8[k], x[e + k], x[e + 8 + k]);
        const float mx = fmaxf(max3f(m8[0], m8[1], m8[2]), max3f(max3f(m8[3], m8[4], m8[5]), m8[6], m8[7]));
        const float m_new = fmaxf(m_run, mx * scale);
        const bool need = m_new > m_run + 8.0f;  // O is rescaled only when the maximum grows by more than 2^8
        float factor = 1.f;
        if (need) {
          factor = ex2(m_run - m_new);
          l_run *= factor;
          m_run = m_new;
        }
        if (__any_sync(0xffffffffu, need && j > 0)) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t ov[32];
            tmem_ld32(tO + q * 32, ov);
            tmem_ld_wait();
            reg_fence(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
            tmem_st32(tO + q * 32, ov);
          }
        }
        const float m_ref = (m_run == -CUDART_INF_F) ? 0.f : m_run, m_eff = F4 ? m_ref - kPShift : m_ref;
        const float2 cs = make_float2(scale, scale), cm = make_float2(-m_eff, -m_eff);
        float2 s4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[2][32];
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          float2 v = ffma2(make_float2(x[2 * e], x[2 * e + 1]), cs, cm);
          v.x = ex2(v.x);
          v.y = ex2(v.y);
          s4[e & 3] = fadd2(s4[e & 3], v);
          pk[e >> 5][e & 31] = F4 ? pack_f16(v.x, v.y) : pack_bf16(v.x, v.y);
          if (Cfg::kPHalves && e == 31) {
            tmem_st32(tS, pk[0]);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(bar(T_PHALF + s));
          }
        }
        const float2 st = fadd2(fadd2(s4[0], s4[1]), fadd2(s4[2], s4[3]));
        l_run += st.x + st.y;
        if (!Cfg::kPHalves) tmem_st32(tS, pk[0]);
        tmem_st32(tS + 32, pk[1]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(T_PFULL + s));
      }
      if (!ok) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_OFINAL + s), ai & 1, abort_flag)))) break;
      tc_fence_after();
      ++ai;
      const bool mend = odd[(n - 1) % kOddMarks] >= n;
      // V's infinities and NaN that were taken out of columns [c0, c0 + 32), for the keys
      // this row sees
      auto put_back = [&](uint32_t (&o)[32], int c0) {
        for (int key = max(P.k0, P.clear); key < min(lim, P.k1); ++key) {
          const int64_t page = plan[P.pages + (key >> pshift)], row = key & ((1 << pshift) - 1);
          if constexpr (F8) {
            if (a.v_exp[page * a.e_sp + row * a.e_sr + P.hkv * a.e_sh] == 255u)
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0x7fffffffu;
          } else if constexpr (F4) {
            const uint8_t* b = a.v_exp + page * a.e_sp + row * a.e_sr + P.hkv * a.e_sh + c0 / 16;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (b[e / 16] > kMostScale) o[e] = 0x7fffffffu;
          } else {
            const uint4* v = reinterpret_cast<const uint4*>(a.vc + page * a.v_sp + row * a.v_sr + P.hkv * a.v_sh + c0 * 2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 x = v[c];
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t b = e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16;
                if ((b & 0x7f800000u) == 0x7f800000u) o[8 * c + e] = __float_as_uint(__uint_as_float(o[8 * c + e]) + __uint_as_float(b));
              }
            }
          }
        }
      };
      // NaN scores leave the maximum alone: what they gave was taken relative to 0
      const float m_end = m_run == -CUDART_INF_F && l_run != 0.f ? 0.f : m_run, m_fin = F4 ? m_end - kPShift : m_end;
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      if (part) {
        if (live) {
          part[s * 128 + r] = m_fin;
          part[tile_slot_rows(D) + s * 128 + r] = l_run;
        }
      } else if (live && a.lse) {
        a.lse[int64_t(h) * a.l_sh + P.q0 + t] =
            l_run == 0.f ? -CUDART_INF_F : (m_fin + lg2(l_run)) * 0.69314718055994531f;
      }
      // Rows leave in 128-byte pieces (64 columns of bf16, 32 of a partial result), 8 lanes
      // storing a piece. (Rows stored by a thread each, 32 rows in every store, held the
      // load/store unit some 9000 cycles a block.)
      const int64_t off = !live ? -1 : part ? int64_t(s * 128 + r) * D * 4 : (int64_t(P.q0 + t) * a.o_sr + int64_t(h) * a.o_sh) * 2;
      uint8_t* const dst = part ? reinterpret_cast<uint8_t*>(part + 2 * tile_slot_rows(D)) : reinterpret_cast<uint8_t*>(a.o);
      auto send = [&](uint32_t (&w)[32], int byte) {  // this row's bytes [byte, byte + 128)
        if constexpr (Cfg::kTurnInRegs) {
          // 8 lanes swap 16-byte parts until each has one part of all 8 rows
#pragma unroll
          for (int b = 1; b < 8; b <<= 1) {
            const bool up = (lane & b) != 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if ((i >> 2) & b) continue;
              const uint32_t x = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + 4 * b], b);
              w[i] = up ? x : w[i];
              w[i + 4 * b] = up ? w[i + 4 * b] : x;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int64_t o = __shfl_sync(0xffffffffu, off, (lane & 24) + i);
            if (o >= 0)
              *reinterpret_cast<uint4*>(dst + o + byte + (lane & 7) * 16) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        } else {
          // part c of row x at c ^ (x & 7) of the warp's box
          const uint32_t box = (Cfg::kStageInQ ? sQ + s * Cfg::kTileBytes : sbase + Cfg::kOffStage + s * 16384) + quarter * 4096;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared_v4(box + lane * 128 + ((c ^ (lane & 7)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int x = 4 * i + (lane >> 3);
            const int64_t o = __shfl_sync(0xffffffffu, off, x);
            const uint4 v = ld_shared_u4(box + x * 128 + (((lane & 7) ^ (x & 7)) << 4));
            if (o >= 0) *reinterpret_cast<uint4*>(dst + o + byte + (lane & 7) * 16) = v;
          }
          __syncwarp();
        }
      };
      constexpr int QH = Cfg::kTurnInRegs || D == 256 ? 2 : D / 32;  // 32-column groups taken out of TMEM at a time
#pragma unroll 1
      for (int q0 = 0; q0 < D / 32; q0 += QH) {
        __syncwarp();
        uint32_t ov[QH][32];
#pragma unroll
        for (int q = 0; q < QH; ++q) tmem_ld32(tO + (q0 + q) * 32, ov[q]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < QH; ++q) reg_fence(ov[q]);
        if (q0 + QH == D / 32) {  // the next block's first product may overwrite O
          tc_fence_before();
          mbar_arrive(bar(T_OEMPTY + s));
        }
        if (mend)
#pragma unroll
          for (int q = 0; q < QH; ++q) put_back(ov[q], (q0 + q) * 32);
        __syncwarp();
        if (part) {
#pragma unroll
          for (int q = 0; q < QH; ++q) send(ov[q], (q0 + q) * 128);
        } else {
#pragma unroll
          for (int q = 0; q < QH; q += 2) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t (&x)[32] = ov[q + (e >> 4)];
              w[e] = pack_bf16(__uint_as_float(x[2 * (e & 15)]) * inv, __uint_as_float(x[2 * (e & 15) + 1]) * inv);
            }
            send(w, (q0 + q) * 64);
          }
        }
      }
      if constexpr (Cfg::kStageInQ) {
        fence_proxy_async_smem();  // the box is Q's again
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T_QEMPTY));
      }
    }
  } else {
    if constexpr (F4) {
      regs_set<Cfg::kRegsConv, Cfg::kRegsLaunch>();
      // -------------------------------------------------------- raw tiles to fp16, thread = key (or half of one)
      const int x = threadIdx.x - 32 * Cfg::kConvWarp, r = x & 127, part = x >> 7;
      constexpr int PARTS = Cfg::kConvThreads / 128;
      constexpr int RB = Cfg::kRowBytes, CH = D / 32 / PARTS;  // 16-byte pieces of a raw row in a part
      static_assert(CH <= 4, "a part's scales are eight bytes at most");
      struct Scales { uint64_t k, v; };
      uint32_t it = 0, rit = 0, n = 0;
      bool ok = true;
      // One piece (32 codes, two scales) after another, the next one's load in flight: unrolled, the loop
      // takes more registers than these warps have.
      auto convert = [&](uint32_t src, uint32_t dst, uint64_t sc) {
        auto load = [&](int ci) {
          const int c = part * CH + ci, x = RB == 32 ? c ^ ((r >> 2) & 1) : RB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
          return ld_shared_u4(src + r * RB + (x << 4));
        };
        uint4 u = load(0);
#pragma unroll(PARTS > 1 ? 4 : 2)
        for (int ci = 0; ci < CH; ++ci, sc >>= 16) {
          const int c = part * CH + ci;
          const uint4 next = load(min(ci + 1, CH - 1));
          const uint32_t f0 = scale_twice(uint32_t(sc) & 255u), f1 = scale_twice(uint32_t(sc >> 8) & 255u);
          const uint32_t d = dst + (c >> 1) * 16384 + r * 128;
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h[4];
            e2m1x8_to_f16(w[i], h);
            const uint32_t f = i < 2 ? f0 : f1;
            st_shared_v4(d + ((((c & 1) * 4 + i) ^ (r & 7)) << 4), mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f),
                         mul_f16x2(h[3], f));
          }
          u = next;
        }
        fence_proxy_async_smem();
      };
      // Q's rows of a block: bf16 to fp16, times a power of two each (its inverse goes to the
      // row's score factor). False if a wait gave up.
      auto convert_q = [&](int ns) -> bool {
        static_assert(PARTS == 1 || NS == 1, "T_QSEEN completes once a block");
        for (int s = 0; s < ns; ++s) {
          const uint32_t q = sQ + s * Cfg::kTileBytes + r * 128;
          auto at = [&](int c) { return q + (c >> 3) * 16384 + (((c & 7) ^ (r & 7)) << 4); };
          uint32_t mx = 0;
#pragma unroll 4
          for (int c = 0; c < D / 8; ++c) mx = max(mx, absmax8(ld_shared_u4(at(c))));
          float inv;
          const float2 up = q_factors(mx, &inv);
          if (part == 0) qs[((n - 1) & 1) * 128 * NS + s * 128 + r] = a.scale_log2 * inv;
          if (PARTS > 1) {  // every part has seen the whole row (a wait with a limit: the others may have given up)
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(T_QSEEN));
            if (!__all_sync(0xffffffffu, mbar_wait(bar(T_QSEEN), (n - 1) & 1, abort_flag))) return false;
          }
#pragma unroll 2
          for (int ci = 0; ci < D / 8 / PARTS; ++ci) {
            const int c = part * (D / 8 / PARTS) + ci;
            const uint4 u = ld_shared_u4(at(c));
            auto f16 = [&](uint32_t x) { return pack_f16(bf16_lo(x) * up.x * up.y, bf16_hi(x) * up.x * up.y); };
            st_shared_v4(at(c), f16(u.x), f16(u.y), f16(u.z), f16(u.w));
          }
        }
        fence_proxy_async_smem();
        return true;
      };
      auto turn_q = [&](int ns) -> bool {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(T_QFULL), (n - 1) & 1, abort_flag))) return false;
        if (!convert_q(ns)) return false;
        mbar_arrive(bar(T_QCONV));
        return true;
      };
      for (int p = p0; p < p1 && ok; ++p) {
        const Piece P = piece(p);
        // this row's scales come one tile ahead, its page number two
        auto page_of = [&](int j) {
          const int pos = P.k0 + 128 * j + r;
          return j < P.nt && pos < P.k1 ? plan[P.pages + (pos >> pshift)] : -1;
        };
        auto scales_of = [&](int j, int page) {
          Scales x = {0, 0};
          if (page < 0) return x;
          const int64_t o = int64_t(page) * a.e_sp + int64_t((P.k0 + 128 * j + r) & ((1 << pshift) - 1)) * a.e_sr + int64_t(P.hkv) * a.e_sh + part * 2 * CH;
          if constexpr (D == 64) {
            x.k = *reinterpret_cast<const uint32_t*>(a.k_exp + o);
            x.v = *reinterpret_cast<const uint32_t*>(a.v_exp + o);
          } else {
            x.k = *reinterpret_cast<const uint64_t*>(a.k_exp + o);
            x.v = *reinterpret_cast<const uint64_t*>(a.v_exp + o);
          }
          return x;
        };
        if (P.nt == 0) continue;
        ++n;
        int pg = page_of(0);
        Scales ahead = scales_of(0, pg);
        pg = page_of(1);
        for (int j = 0; j < P.nt; ++j, ++it) {
          Scales now = ahead;  // rows past the keys' end: zeros
          ahead = scales_of(j + 1, pg);
          pg = page_of(j + 2);
          const int s = it % NST;
          // V's scales of NaN stay out of the products where some row does not see the key
          if (P.k0 + 128 * j + r >= P.clear) {
            const uint32_t lo = __vcmpgtu4(uint32_t(now.v), kMostScale * 0x01010101u);
            const uint32_t hi = __vcmpgtu4(uint32_t(now.v >> 32), kMostScale * 0x01010101u);
            now.v &= ~(uint64_t(hi) << 32 | lo);
            if (lo | hi) odd[(n - 1) % kOddMarks] = n;
          }
          for (int h = 0; h < 2; ++h, ++rit) {
            // Q between its first K and V (its tile is free when the last block's products are done)
            static_assert(!Cfg::kStageInQ, "Q would be waited for before the last block's results are out");
            if (j == 0 && h == 1 && !(ok = turn_q(P.ns))) break;
            const int rs = rit % NR;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_RFULL + rs), (rit / NR) & 1, abort_flag)))) break;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar((h ? T_VEMPTY : T_KEMPTY) + s), ((it / NST) & 1) ^ 1, abort_flag)))) break;
            convert(sR + rs * Cfg::kRawBytes, (h ? sV : sK) + s * Cfg::kTileBytes, h ? now.v : now.k);
            mbar_arrive(bar(T_REMPTY + rs));
            mbar_arrive(bar((h ? T_VFULL : T_KFULL) + s));
          }
          if (!ok) break;
        }
      }
    } else if constexpr (F8) {
      regs_set<Cfg::kRegsConv, Cfg::kRegsLaunch>();
      // -------------------------------------------------------- raw tiles to bf16, thread = key
      const int r = threadIdx.x - 384;
      uint32_t it = 0, rit = 0, n = 0;
      bool ok = true;
      // codes of this thread's row (at `src`) times 2^e into the bf16 tile at `dst`;
      // SLOW: some row of the warp is to be zeros (past the keys' end, or V of NaN that not
      // every row sees), NaN, or of an exponent that takes two factors
      auto convert = [&](auto slow, uint32_t src, uint32_t dst, uint32_t byte, bool zero) {
        constexpr bool SLOW = decltype(slow)::value;
        const int e = int(byte) - 127;
        // 2^(120 + e) fits a bf16 up to e = 7; what is left of a larger one is a second factor
        const uint32_t f1 = SLOW && byte == 255u ? 0x7fc0u : uint32_t(127 + 120 + min(e, 7)) << 7;
        const uint32_t m1 = f1 | (f1 << 16), f2 = uint32_t(127 + max(e, 7) - 7) << 7, m2 = f2 | (f2 << 16);
        const uint32_t keep = zero ? 0u : ~0u;
        constexpr int PB = D == 64 ? 64 : 128;  // bytes of a raw row's piece
        auto load = [&](int c) {
          const int pc = c * 16 / PB, cc = c % (PB / 16);
          return ld_shared_u4(src + pc * 128 * PB + r * PB + (D == 64 ? ((cc ^ ((r >> 1) & 3)) << 4) : ((cc ^ (r & 7)) << 4)));
        };
        // four 16-byte loads in flight; 16 codes give two 16-byte pieces of bf16
        uint4 u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] = load(c);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 x = u[c & 3];
          if (c + 4 < D / 16) u[c & 3] = load(c + 4);
          uint32_t w[8];
          e4m3x4_bits(x.x, w[0], w[1]);
          e4m3x4_bits(x.y, w[2], w[3]);
          e4m3x4_bits(x.z, w[4], w[5]);
          e4m3x4_bits(x.w, w[6], w[7]);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = hmul2_bf16(w[i], m1);
          if constexpr (SLOW)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = (byte == 255u ? w[i] : hmul2_bf16(w[i], m2)) & keep;
          const uint32_t d = dst + (c >> 2) * 16384 + r * 128;
          const int oc = (c & 3) * 2;
          st_shared_v4(d + ((oc ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
          st_shared_v4(d + (((oc + 1) ^ (r & 7)) << 4), w[4], w[5], w[6], w[7]);
        }
        fence_proxy_async_smem();
      };
      for (int p = p0; p < p1 && ok; ++p) {
        const Piece P = piece(p);
        // this row's exponents come one tile ahead, its page number two
        auto page_of = [&](int j) {
          const int pos = P.k0 + 128 * j + r;
          return j < P.nt && pos < P.k1 ? plan[P.pages + (pos >> pshift)] : -1;
        };
        auto exps_of = [&](int j, int page) -> uint32_t {
          if (page < 0) return 127u | (127u << 8);
          const int64_t o = int64_t(page) * a.e_sp + int64_t((P.k0 + 128 * j + r) & ((1 << pshift) - 1)) * a.e_sr + int64_t(P.hkv) * a.e_sh;
          return uint32_t(a.k_exp[o]) | (uint32_t(a.v_exp[o]) << 8);
        };
        n += P.nt > 0 ? 1 : 0;
        int pg = page_of(0);
        uint32_t ex = exps_of(0, pg);
        pg = page_of(1);
        for (int j = 0; j < P.nt; ++j, ++it) {
          const uint32_t now = ex;
          ex = exps_of(j + 1, pg);
          pg = page_of(j + 2);
          const int s = it % NST;
          const bool past = P.k0 + 128 * j + r >= P.k1;
          for (int h = 0; h < 2; ++h, ++rit) {
            const int rs = rit % NR;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar(T_RFULL + rs), (rit / NR) & 1, abort_flag)))) break;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(bar((h ? T_VEMPTY : T_KEMPTY) + s), ((it / NST) & 1) ^ 1, abort_flag)))) break;
            const uint32_t src = sR + rs * Cfg::kRawBytes, dst = (h ? sV : sK) + s * Cfg::kTileBytes;
            const uint32_t byte = (now >> (8 * h)) & 255u;
            const bool out = h && byte == 255u && !past && P.k0 + 128 * j + r >= P.clear;
            if (out) odd[(n - 1) % kOddMarks] = n;
            if (__any_sync(0xffffffffu, past || byte > 127u + 7u)) convert(std::true_type(), src, dst, byte, past || out);
            else convert(std::false_type(), src, dst, byte, false);
            mbar_arrive(bar(T_REMPTY + rs));
            mbar_arrive(bar((h ? T_VFULL : T_KFULL) + s));
          }
          if (!ok) break;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) {
    atomicExch(const_cast<int32_t*>(plan) + PH_STATUS, DEV_TIMEOUT);
    atomicExch(const_cast<int32_t*>(plan) + PH_STATUS_DETAIL, 6);
  }
}

template <int D, int FMT>
int32_t launch_tile_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                      cudaStream_t s) {
  using Cfg = TileCfg<D, FMT>;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    cudaError_t e = cudaFuncSetAttribute(bd_paged_tile_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(paged tile)");
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, bd_paged_tile_kernel<D, FMT>);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(paged tile)");
    // setmaxnreg.inc waits until registers are free: never launch a split that cannot be met
    if (fa.numRegs != Cfg::kRegsLaunch)
      return fail(BD_ERR_UNSUPPORTED, "paged tile kernel built with %d registers/thread, its register split assumes %d",
                  fa.numRegs, Cfg::kRegsLaunch);
    if (dev < 64) done[dev].store(true, std::memory_order_release);
  }
  const cudaError_t e = launch_kernel(bd_paged_tile_kernel<D, FMT>, kTileCtas, Cfg::kThreads, Cfg::kSmem, s, mq, mk, mv, a);
  return e == cudaSuccess ? BD_OK : cuda_fail(e, "bd_paged_tile_kernel launch");
}

}  // namespace

int32_t launch_tile(const int32_t* w, const AttnArgs& a, const bd_tensor* q, const bd_paged_cache* c, cudaStream_t s) {
  const int d = w[PH_D], G = w[PH_G], es = elem_bytes(c->fmt), bytes = row_bytes(c->fmt, d), piece = bytes < 128 ? bytes : 128;
  const int rows = w[PH_PAGE] < 128 ? w[PH_PAGE] : 128;
  CUtensorMap mq, mk, mv;
  int32_t st;
  if ((st = make_tmap_group_bf16(&mq, q, w[PH_H], d, "q", G, 128 / G))) return st;
  if ((st = make_tmap_pages(&mk, &c->k, c->num_pages, w[PH_HKV], bytes, es, "cache k", rows, false, piece))) return st;
  if ((st = make_tmap_pages(&mv, &c->v, c->num_pages, w[PH_HKV], bytes, es, "cache v", rows, false, piece))) return st;
  if (c->fmt == BD_CACHE_BF16)
    return d == 64 ? launch_tile_t<64, BD_CACHE_BF16>(mq, mk, mv, a, s)
           : d == 128 ? launch_tile_t<128, BD_CACHE_BF16>(mq, mk, mv, a, s)
                      : launch_tile_t<256, BD_CACHE_BF16>(mq, mk, mv, a, s);
  if (c->fmt == BD_CACHE_E2M1)
    return d == 64 ? launch_tile_t<64, BD_CACHE_E2M1>(mq, mk, mv, a, s)
           : d == 128 ? launch_tile_t<128, BD_CACHE_E2M1>(mq, mk, mv, a, s)
                      : launch_tile_t<256, BD_CACHE_E2M1>(mq, mk, mv, a, s);
  return d == 64 ? launch_tile_t<64, BD_CACHE_E4M3>(mq, mk, mv, a, s)
         : d == 128 ? launch_tile_t<128, BD_CACHE_E4M3>(mq, mk, mv, a, s)
                    : launch_tile_t<256, BD_CACHE_E4M3>(mq, mk, mv, a, s);
}

}  // namespace bd
