// Bounds of the blocks of a paged K/V cache, and the blocks that each new row attends, on
// sm_103a (the attention over them is paged_dec.cu's).
//
// A block (a page of a sequence) and K/V head is described by the least and the greatest value
// of each element of its keys, as 8-bit codes lo_c, hi_c and one power of two; q by 8-bit codes and a
// power of two for each head. For any key of the block q . k <= sum_c max(q_c lo_c, q_c hi_c), up to
// the codes' rounding: that sum is the block's score. It is a whole number below 2^23, so a score is
// exact in fp32 in whatever order it is summed, and lists do not depend on the launch.
//
// bd_block_bounds_kernel: a CTA for each (block with new rows, K/V head); a stream over the
// block's keys (a decode step's 128 blocks of 64 keys 2.6 us).
//
// bd_block_select_kernel: a CTA for some new rows of a sequence and a K/V head. Scores by
// 8-bit matrix instructions (m16n8k32): 16 blocks against 8 (row, head) columns, positive q
// against hi, negative against lo; they stay in shared memory as whole numbers of the same order.
// Choice: the threshold eight bits a pass from the highest bit in which scores differ, by counts
// of the digits, then the blocks above it and the first ones equal to it, in order. Few rows have a
// CTA of 16 warps each, bound by a chain of lookups and what one SM takes in (16 rows, 8 heads: 47 blocks 6.4 us,
// 938 blocks 12), or a cluster of them where there are SMs left (1 row: 12 -> 8.6); many
// go by eight, a warp for each one's choice, which read their bounds once (600 rows, 255 blocks: 31 us). Scores as
// fp16 products, or bounds fetched a tile ahead, were no faster (13.3 and 12.3 us for the 938 blocks).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "paged.h"
#include "paged_quant.cuh"

namespace bd {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

struct BoundsArgs {
  const int32_t* plan;
  const uint8_t* k;
  int64_t k_sp, k_sr, k_sh;  // bytes
  const uint8_t* k_exp;
  int64_t e_sp, e_sr, e_sh;
  int8_t* code;
  int64_t c_sp, c_sh, c_sb;
  uint8_t* exp;
  int64_t x_sp, x_sh;
};

// The smallest e of [-50, 50] with m <= 127 * 2^e (127 = 1.984375 * 2^6), m >= 0 finite.
__device__ __forceinline__ int pow8(float m) {
  const uint32_t u = __float_as_uint(m);
  const int e = int(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return min(50, max(-50, e));
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

constexpr int kBoundThreads = 128;

template <int D, int FMT>
__global__ void __launch_bounds__(kBoundThreads) bd_block_bounds_kernel(const BoundsArgs a) {
  constexpr int LPR = D / 8, RG = kBoundThreads / LPR;  // lanes of a key, keys at a time
  __shared__ float s_lo[RG][D], s_hi[RG][D];
  __shared__ float s_max[kBoundThreads / 32];
  const int sub = threadIdx.x % LPR, rg = threadIdx.x / LPR;
  const int32_t* plan = a.plan;
  grid_wait();
  const int Hkv = plan[PH_HKV], n = plan[PH_NTOUCH];
  const int32_t *touch = plan + plan[PH_OFF_TOUCH], *pages = plan + plan[PH_OFF_PAGES], *count = plan + plan[PH_OFF_PGCNT];
  for (int64_t x = blockIdx.x; x < int64_t(n) * Hkv; x += gridDim.x) {
    const int at = touch[x / Hkv], h = int(x % Hkv), rows = count[at];
    const int64_t page = pages[at];
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { lo[i] = CUDART_INF_F; hi[i] = -CUDART_INF_F; }
    bool bad = false;
    constexpr int U = 4;  // keys in flight
    for (int r0 = rg; r0 < rows; r0 += U * RG) {
      uint4 v[U];
      uint32_t e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = min(r0 + u * RG, rows - 1);  // past the last key that one again
        const uint8_t* p = a.k + page * a.k_sp + int64_t(r) * a.k_sr + int64_t(h) * a.k_sh;
        const int64_t eo = page * a.e_sp + int64_t(r) * a.e_sr + int64_t(h) * a.e_sh;
        if constexpr (FMT == BD_CACHE_BF16) {
          v[u] = *(reinterpret_cast<const uint4*>(p) + sub);
        } else if constexpr (FMT == BD_CACHE_E4M3) {
          const uint2 c = *(reinterpret_cast<const uint2*>(p) + sub);
          v[u].x = c.x; v[u].y = c.y;
          e[u] = a.k_exp[eo];
        } else {
          v[u].x = *(reinterpret_cast<const uint32_t*>(p) + sub);
          e[u] = a.k_exp[eo + sub / 2];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (FMT == BD_CACHE_E4M3) {
          bad |= e[u] == 255u;
          const float f = exp_factor(e[u]);
          const uint2 p = dequantise4(v[u].x, f), q = dequantise4(v[u].y, f);
          v[u] = make_uint4(p.x, p.y, q.x, q.y);
        } else if constexpr (FMT == BD_CACHE_E2M1) {
          bad |= e[u] > kMostScale;
          v[u] = dequantise8_e2m1(v[u].x, e[u]);
        } else {
          bad |= absmax8(v[u]) >= 0x7f80u;
        }
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[2 * i] = fminf(lo[2 * i], bf16_lo(w[i])); hi[2 * i] = fmaxf(hi[2 * i], bf16_lo(w[i]));
          lo[2 * i + 1] = fminf(lo[2 * i + 1], bf16_hi(w[i])); hi[2 * i + 1] = fmaxf(hi[2 * i + 1], bf16_hi(w[i]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) { s_lo[rg][sub * 8 + i] = lo[i]; s_hi[rg][sub * 8 + i] = hi[i]; }
    bad = __syncthreads_or(bad);
    constexpr int C = D > kBoundThreads ? D / kBoundThreads : 1;  // columns of a thread
    float m = 0.f;
    if (threadIdx.x < D / C)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = threadIdx.x + c * kBoundThreads;
        lo[c] = CUDART_INF_F; hi[c] = -CUDART_INF_F;
#pragma unroll
        for (int g = 0; g < RG; ++g) { lo[c] = fminf(lo[c], s_lo[g][col]); hi[c] = fmaxf(hi[c], s_hi[g][col]); }
        m = fmaxf(m, fmaxf(fabsf(lo[c]), fabsf(hi[c])));
      }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
    if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBoundThreads / 32; ++w) m = fmaxf(m, s_max[w]);
    const int e = pow8(m);
    const float f = pow2f(-e);
    int8_t* out = a.code + page * a.c_sp + int64_t(h) * a.c_sh;
    if (threadIdx.x < D / C)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = threadIdx.x + c * kBoundThreads;
        // (a product below the least float is zero, its floor or ceil is not)
        const float down = fminf(floorf(lo[c] * f), lo[c] < 0.f ? -1.f : 127.f), up = fmaxf(ceilf(hi[c] * f), hi[c] > 0.f ? 1.f : -127.f);
        out[col] = bad ? int8_t(0) : int8_t(fmaxf(down, -127.f));
        out[a.c_sb + col] = bad ? int8_t(0) : int8_t(fminf(up, 127.f));
      }
    if (threadIdx.x == 0) a.exp[page * a.x_sp + int64_t(h) * a.x_sh] = bad ? uint8_t(255) : uint8_t(e + 127);
    __syncthreads();
  }
}

struct SelectArgs {
  const int32_t* plan;
  const uint8_t* q;
  int64_t q_sr, q_sh;  // bytes
  const int8_t* code;
  int64_t c_sp, c_sh, c_sb;
  const uint8_t* exp;
  int64_t x_sp, x_sh;
  int32_t* out;
  int64_t o_sr, o_sh;
  int32_t G, Hkv, blocks, first, recent, page_shift, cap, rows, split;
};

// A score as a whole number of the same order (0: below all of them), an infinity of a block with
// NaN or infinities above all of them.
__device__ __forceinline__ uint32_t order_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kOddBlock = 0xff800000u;

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The word of another CTA of the cluster that lies where p does here.
__device__ __forceinline__ uint32_t load_cluster(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The digit of a threshold from counts of 256 digits (bins past those in use are zero): the highest
// with `want` keys in it and above. A warp, 8 digits a lane. Takes the keys above off want; `exact`: the
// digit's own keys are just as many as are wanted.
__device__ __forceinline__ uint32_t find_digit(const uint32_t* hist, int lane, int* want, bool* exact) {
  const uint4 lo = reinterpret_cast<const uint4*>(hist)[2 * lane], hi = reinterpret_cast<const uint4*>(hist)[2 * lane + 1];
  const uint32_t c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += c[i];
  uint32_t above = sum;  // of this lane and those behind it
#pragma unroll
  for (int y = 1; y < 32; y <<= 1) {
    const uint32_t v = __shfl_down_sync(kFull, above, y);
    if (lane + y < 32) above += v;
  }
  above -= sum;
  const bool mine = int(above) < *want && int(above + sum) >= *want;
  uint32_t digit = 0, over = above, own = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    if (own == 0 && int(over + c[i]) >= *want) { digit = 8 * lane + i; own = c[i]; }
    if (own == 0) over += c[i];
  }
  const int from = __ffs(__ballot_sync(kFull, mine)) - 1;
  *want -= int(__shfl_sync(kFull, over, from));
  *exact = int(__shfl_sync(kFull, own, from)) == *want;
  return __shfl_sync(kFull, digit, from);
}

// SPLIT: a row's scores are shared out to the `split` CTAs of a cluster, the first of which chooses.
template <int D, int THREADS, bool SPLIT>
__global__ void __launch_bounds__(THREADS, D == 256 || SPLIT ? 1 : 1024 / THREADS) bd_block_select_kernel(const SelectArgs a) {
  constexpr int NW = THREADS / 32;
  constexpr int S = D / 32;                // contraction steps; a lane has D / 4 neighbouring codes of a block
  constexpr int QP = select_pitch(D);
  extern __shared__ uint4 sel_smem[];
  const int cols = a.rows * a.G, colt = (cols + 7) / 8;
  uint8_t* s_q = reinterpret_cast<uint8_t*>(sel_smem);          // [8 colt]: positive, then negative codes
  float2* s_col = reinterpret_cast<float2*>(s_q + colt * 8 * QP);    // [8 colt]: q's power of two, the row's keys (-1: no row)
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_col + colt * 8);   // [rows][cap]
  __shared__ uint32_t s_red[NW][2];
  __shared__ __align__(16) uint32_t s_hist[8][256];  // a row by the CTA: one for each pass, rows by warps: for each warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = lane & 3, rw = lane >> 2;
  const int32_t* plan = a.plan;
  grid_wait();
  const int groups = plan[PH_NSELG];
  const int32_t *where = plan + plan[PH_OFF_POS], *rowpg = plan + plan[PH_OFF_ROWPG], *list = plan + plan[PH_OFF_SELG];
  const uint32_t units = uint32_t(groups) * uint32_t(a.Hkv);  // (no more than new rows times heads)
  const uint32_t parts = SPLIT ? a.split : 1, part = SPLIT ? cluster_rank() : 0;
  for (uint32_t x = blockIdx.x / parts; x < units; x += gridDim.x / parts) {
    const int gi = int(x / uint32_t(a.Hkv)), g = int(x) - gi * a.Hkv;
    const int t0 = a.rows == 1 ? gi : list[2 * gi], n = a.rows == 1 ? 1 : list[2 * gi + 1];
    auto blocks_of = [&](int r) { const int pos = where[t0 + r]; return pos < 0 ? 0 : (pos >> a.page_shift) + 1; };
    auto out_of = [&](int r) { return a.out + int64_t(t0 + r) * a.o_sr + int64_t(g) * a.o_sh; };
    const int most = blocks_of(n - 1);
    if (most <= a.blocks) {  // all there are, for every row
      for (int r = 0; r < n && part == 0; ++r) {
        const int nblk = blocks_of(r);
        for (int i = tid; i < a.blocks; i += THREADS) out_of(r)[i] = i < nblk ? i : -1;
      }
      continue;
    }
    const int32_t* pages = plan + rowpg[t0];
    // the first tile's blocks are looked up while q is turned into codes
    int pg[2];
    auto look_up = [&](int tile) {
#pragma unroll
      for (int h = 0; h < 2; ++h) pg[h] = pages[min(tile * 16 + rw + 8 * h, most - 1)];
    };
    const int step = NW * int(parts), tile0 = warp + NW * int(part);
    look_up(tile0);
    // ---- q's codes: a warp for each (row, head)
    for (int c = warp; c < colt * 8; c += NW) {
      const bool there = c < n * a.G, in = lane < D / 8;
      const uint8_t* p = a.q + int64_t(t0 + c / a.G) * a.q_sr + int64_t(g * a.G + c % a.G) * a.q_sh;
      const uint4 v = in && there ? *(reinterpret_cast<const uint4*>(p) + lane) : make_uint4(0, 0, 0, 0);
      const uint32_t mx = __reduce_max_sync(kFull, absmax8(v));
      const bool bad = mx >= 0x7f80u;
      const int e = bad ? 0 : pow8(__uint_as_float(mx << 16));
      const float f = bad ? 0.f : pow2f(-e);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t up[2] = {0, 0}, down[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        const int z = bad ? 0 : int(fminf(fmaxf(rintf(y * f), -127.f), 127.f));
        up[i >> 2] |= uint32_t(max(z, 0) & 255) << (8 * (i & 3));
        down[i >> 2] |= uint32_t(min(z, 0) & 255) << (8 * (i & 3));
      }
      if (in) {
        *reinterpret_cast<uint2*>(s_q + c * QP + lane * 8) = make_uint2(up[0], up[1]);
        *reinterpret_cast<uint2*>(s_q + c * QP + D + lane * 8) = make_uint2(down[0], down[1]);
      }
      if (lane == 0) s_col[c] = make_float2(pow2f(e), __int_as_float(there ? c / a.G * a.cap : -1));
    }
    for (int r = 0; r < n; ++r)
      for (int i = tid; i < most; i += THREADS) s_key[r * a.cap + i] = 0u;
    if (a.rows == 1)
      for (int i = tid; i < 1024; i += THREADS) s_hist[0][i] = 0u;
    __syncthreads();
    // ---- scores: 16 blocks of a warp at a time against 8 (row, head) columns
    for (int tile = tile0; tile * 16 < most; tile += step) {
      uint32_t hi[2][2 * S], lo[2][2 * S], eb[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int8_t* p = a.code + int64_t(pg[h]) * a.c_sp + int64_t(g) * a.c_sh + j * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 u = *(reinterpret_cast<const uint4*>(p + a.c_sb) + i), v = *(reinterpret_cast<const uint4*>(p) + i);
          hi[h][4 * i] = u.x; hi[h][4 * i + 1] = u.y; hi[h][4 * i + 2] = u.z; hi[h][4 * i + 3] = u.w;
          lo[h][4 * i] = v.x; lo[h][4 * i + 1] = v.y; lo[h][4 * i + 2] = v.z; lo[h][4 * i + 3] = v.w;
        }
        eb[h] = a.exp[int64_t(pg[h]) * a.x_sp + int64_t(g) * a.x_sh];
      }
      if ((tile + step) * 16 < most) look_up(tile + step);
      // (memory that never was bounds may hold any byte: with q's 2^-50..2^50 and sums below 2^23 every
      // score is a finite number)
      const float ebf[2] = {pow2f(min(max(int(eb[0]) - 127, -50), 50)), pow2f(min(max(int(eb[1]) - 127, -50), 50))};
      for (int ct = 0; ct < colt; ++ct) {
        int c[4] = {0, 0, 0, 0};
        const uint8_t* q = s_q + (ct * 8 + rw) * QP + j * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 u = *(reinterpret_cast<const uint4*>(q) + i), v = *(reinterpret_cast<const uint4*>(q + D) + i);
          mma_s8(c, hi[0][4 * i], hi[1][4 * i], hi[0][4 * i + 1], hi[1][4 * i + 1], u.x, u.y);
          mma_s8(c, hi[0][4 * i + 2], hi[1][4 * i + 2], hi[0][4 * i + 3], hi[1][4 * i + 3], u.z, u.w);
          mma_s8(c, lo[0][4 * i], lo[1][4 * i], lo[0][4 * i + 1], lo[1][4 * i + 1], v.x, v.y);
          mma_s8(c, lo[0][4 * i + 2], lo[1][4 * i + 2], lo[0][4 * i + 3], lo[1][4 * i + 3], v.z, v.w);
        }
        // this lane's columns 2 j, 2 j + 1 of blocks rw, rw + 8: the largest of a row's heads
        const float4 col = *reinterpret_cast<const float4*>(s_col + ct * 8 + 2 * j);
        const int at0 = __float_as_int(col.y), at1 = __float_as_int(col.w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int b = tile * 16 + rw + 8 * h;
          if (b >= most) continue;
          const uint32_t k0 = eb[h] == 255u ? kOddBlock : order_of(float(c[2 * h]) * (col.x * ebf[h]));
          const uint32_t k1 = eb[h] == 255u ? kOddBlock : order_of(float(c[2 * h + 1]) * (col.z * ebf[h]));
          if (at0 == at1) {
            if (at0 >= 0) atomicMax(&s_key[at0 + b], max(k0, k1));
          } else {
            if (at0 >= 0) atomicMax(&s_key[at0 + b], k0);
            if (at1 >= 0) atomicMax(&s_key[at1 + b], k1);
          }
        }
      }
    }
    if constexpr (SPLIT) {
      cluster_sync();
      if (part == 0)
        for (int i = tid; i < most; i += THREADS) {
          const uint32_t from = uint32_t(i >> 4) / NW % parts;
          if (from != 0) s_key[i] = load_cluster(&s_key[i], from);
        }
      cluster_sync();  // (the others' keys are theirs again)
      if (part != 0) continue;
    } else {
      __syncthreads();
    }
    // ---- the choice, of the blocks that are not listed always: K of [first, most - recent)
    const int K = a.blocks - a.first - a.recent;
    if (a.rows == 1) {
      // one row by the whole CTA. Keys from tid * per on are this thread's.
      int32_t* out = out_of(0);
      const int per = (most + THREADS - 1) / THREADS, i0 = min(tid * per, most), i1 = min(i0 + per, most);
      const int b0 = max(i0, a.first), b1 = min(i1, most - a.recent);
      uint32_t all1 = ~0u, any1 = 0;
      for (int i = b0; i < b1; ++i) { all1 &= s_key[i]; any1 |= s_key[i]; }
      all1 = __reduce_and_sync(kFull, all1);
      any1 = __reduce_or_sync(kFull, any1);
      if (lane == 0) { s_red[warp][0] = all1; s_red[warp][1] = any1; }
      __syncthreads();
      all1 = __reduce_and_sync(kFull, lane < NW ? s_red[lane][0] : ~0u);
      any1 = __reduce_or_sync(kFull, lane < NW ? s_red[lane][1] : 0u);
      // thr: the K-th largest key, 8 bits a pass from the first that differs; or, when all keys from
      // thr on are wanted, the number before it
      const uint32_t differ = all1 ^ any1;
      int bit = differ ? 32 - __clz(differ) : 0, want = K;
      uint32_t thr = K == 0 ? ~0u : bit == 0 ? all1 : bit == 32 ? 0u : all1 & ~((1u << bit) - 1u);
      for (int pass = 0; K > 0 && bit > 0; ++pass) {
        const int lo = max(bit - 8, 0);
        const uint32_t mask = (1u << (bit - lo)) - 1u;
        for (int i = b0; i < b1; ++i) {
          const uint32_t k = s_key[i];
          if (bit == 32 || ((k ^ thr) >> bit) == 0) atomicAdd(&s_hist[pass][(k >> lo) & mask], 1u);
        }
        __syncthreads();
        bool exact;
        thr |= find_digit(s_hist[pass], lane, &want, &exact) << lo;
        bit = lo;
        if (exact && thr > 0) {
          --thr;
          break;
        }
      }
      // those above thr, and of those equal to it the first ones, in order
      uint32_t cnt = 0;  // above in the lower 16 bits, equal in the upper ones
      auto always = [&](int i) { return i < a.first || i >= most - a.recent; };
      for (int i = i0; i < i1; ++i) cnt += always(i) || s_key[i] > thr ? 1u : s_key[i] == thr ? 0x10000u : 0u;
      uint32_t sum = cnt;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const uint32_t v = __shfl_up_sync(kFull, sum, y);
        if (lane >= y) sum += v;
      }
      __syncthreads();
      if (lane == 31) s_red[warp][0] = sum;
      __syncthreads();
      const uint32_t others = lane < NW ? s_red[lane][0] : 0u;
      const uint32_t before = sum - cnt + __reduce_add_sync(kFull, lane < warp ? others : 0u);
      const int room = a.blocks - int(__reduce_add_sync(kFull, others) & 0xffffu);  // for keys equal to thr
      int above = int(before & 0xffffu), equal = int(before >> 16);
      for (int i = i0; i < i1; ++i) {
        const uint32_t k = s_key[i];
        if (always(i) || k > thr) out[above++ + min(equal, room)] = i;
        else if (k == thr) {
          if (equal < room) out[above + equal] = i;
          ++equal;
        }
      }
    } else {
      // a row by a warp; a lane has keys lane, lane + 32, ...
      for (int r = warp; r < n; r += NW) {
        int32_t* out = out_of(r);
        const uint32_t* key = s_key + r * a.cap;
        const int nblk = blocks_of(r);
        if (nblk <= a.blocks) {
          for (int i = lane; i < a.blocks; i += 32) out[i] = i < nblk ? i : -1;
          continue;
        }
        const int b0 = a.first + lane, b1 = nblk - a.recent;
        uint32_t all1 = ~0u, any1 = 0;
        for (int i = b0; i < b1; i += 32) { all1 &= key[i]; any1 |= key[i]; }
        const uint32_t differ = __reduce_and_sync(kFull, all1) ^ __reduce_or_sync(kFull, any1);
        all1 = __reduce_and_sync(kFull, all1);
        int bit = differ ? 32 - __clz(differ) : 0, want = K;
        uint32_t thr = K == 0 ? ~0u : bit == 0 ? all1 : bit == 32 ? 0u : all1 & ~((1u << bit) - 1u);
        uint32_t* hist = s_hist[warp & 7];  // (8 warps where rows are theirs)
        while (K > 0 && bit > 0) {
          const int lo = max(bit - 8, 0);
          const uint32_t mask = (1u << (bit - lo)) - 1u;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i) reinterpret_cast<uint4*>(hist)[lane + 32 * i] = make_uint4(0, 0, 0, 0);
          __syncwarp();
          for (int i = b0; i < b1; i += 32) {
            const uint32_t k = key[i];
            if (bit == 32 || ((k ^ thr) >> bit) == 0) atomicAdd(&hist[(k >> lo) & mask], 1u);
          }
          __syncwarp();
          bool exact;
          thr |= find_digit(hist, lane, &want, &exact) << lo;
          bit = lo;
          if (exact && thr > 0) {
            --thr;
            break;
          }
        }
        auto always = [&](int i) { return i < a.first || i >= b1; };
        uint32_t over = 0;
        for (int i = lane; i < nblk; i += 32) over += always(i) || key[i] > thr ? 1u : 0u;
        const int room = a.blocks - int(__reduce_add_sync(kFull, over));
        int at = 0, equal = 0;
        for (int base = 0; base < nblk; base += 32) {
          const int i = base + lane;
          const uint32_t k = i < nblk ? key[i] : 0u;
          const bool sure = i < nblk && (always(i) || k > thr), same = i < nblk && !sure && k == thr;
          const uint32_t e = __ballot_sync(kFull, same), before = (1u << lane) - 1u;
          const bool take = sure || (same && equal + __popc(e & before) < room);
          const uint32_t m = __ballot_sync(kFull, take);
          if (take) out[at + __popc(m & before)] = i;
          at += __popc(m);
          equal += __popc(e);
        }
      }
    }
    __syncthreads();
  }
}

int32_t check_bounds(const bd_bounds* b, const int32_t* w) {
  if (!b || !b->code || !b->exp) return fail(BD_ERR_ARG, "bounds: NULL, or code or exp NULL");
  if (b->num_pages != w[PH_NUM_PAGES])
    return fail(BD_ERR_PLAN, "bounds of %d pages, the plan was built for %d", b->num_pages, w[PH_NUM_PAGES]);
  const int64_t Hkv = w[PH_HKV], d = w[PH_D];
  if (reinterpret_cast<uintptr_t>(b->code) % 16 || b->stride_bound % 16 || (Hkv > 1 && b->stride_head % 16) ||
      (b->num_pages > 1 && b->stride_page % 16))
    return fail(BD_ERR_ALIGN, "bounds: code and its strides must be multiples of 16 bytes");
  if (b->stride_bound < d || (Hkv > 1 && b->stride_head < d) || (b->num_pages > 1 && b->stride_page < d) ||
      (Hkv > 1 && b->exp_stride_head <= 0) || (b->num_pages > 1 && b->exp_stride_page <= 0))
    return fail(BD_ERR_ARG, "bounds: strides must be positive, those of code at least the head dim");
  return BD_OK;
}

template <int FMT>
cudaError_t launch_bounds(int d, int grid, cudaStream_t s, const BoundsArgs& a) {
  return d == 64    ? launch_kernel(bd_block_bounds_kernel<64, FMT>, grid, kBoundThreads, 0, s, a)
         : d == 128 ? launch_kernel(bd_block_bounds_kernel<128, FMT>, grid, kBoundThreads, 0, s, a)
                    : launch_kernel(bd_block_bounds_kernel<256, FMT>, grid, kBoundThreads, 0, s, a);
}

template <int D, int THREADS, bool SPLIT>
int32_t launch_select_t(int grid, size_t smem, cudaStream_t s, const SelectArgs& a) {
  auto kernel = bd_block_select_kernel<D, THREADS, SPLIT>;
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSelMostSmem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(block select)");
    if (dev < 64) done[dev].store(true, std::memory_order_release);
  }
  cudaError_t e;
  if constexpr (SPLIT) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid * a.split);
    c.blockDim = dim3(THREADS);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    e = cudaLaunchKernelEx(&c, kernel, a);
  } else {
    e = launch_kernel(kernel, grid, THREADS, smem, s, a);
  }
  return e == cudaSuccess ? BD_OK : cuda_fail(e, "bd_block_select_kernel launch");
}

// One row by 16 warps, or by those of a few CTAs; several rows by 8.
template <int D>
int32_t launch_select(int grid, size_t smem, cudaStream_t s, const SelectArgs& a) {
  return a.rows > 1    ? launch_select_t<D, 256, false>(grid, smem, s, a)
         : a.split > 1 ? launch_select_t<D, 512, true>(grid, smem, s, a)
                       : launch_select_t<D, 512, false>(grid, smem, s, a);
}

}  // namespace

int32_t check_blocks(const bd_blocks* b, const int32_t* w) {
  if (!b || !b->ptr || reinterpret_cast<uintptr_t>(b->ptr) % 4) return fail(BD_ERR_ARG, "blocks: NULL or not 4-byte aligned");
  if (b->rows < w[PH_T]) return fail(BD_ERR_ARG, "blocks of %d rows < %d new rows of the plan", b->rows, w[PH_T]);
  if ((w[PH_T] > 1 && b->stride_row < w[PH_BLOCKS]) || (w[PH_HKV] > 1 && b->stride_head < w[PH_BLOCKS]))
    return fail(BD_ERR_ARG, "blocks: strides less than a list of %d", w[PH_BLOCKS]);
  return BD_OK;
}

}  // namespace bd

using namespace bd;

extern "C" int32_t bd_block_bounds(const void* plan_host, const void* plan_dev, const bd_paged_cache* cache,
                                   const bd_bounds* bounds, void* stream) {
  const int32_t* w = nullptr;
  int32_t st = check_paged(plan_host, plan_dev, cache, &w);
  if (st) return st;
  if (!w[PH_CAUSAL]) return fail(BD_ERR_PLAN, "new rows of a plan that is not causal have no cache positions");
  if (!w[PH_BOUNDS_OK]) return fail(BD_ERR_PLAN, "two sequences of the batch have new rows in the same page");
  if ((st = check_bounds(bounds, w))) return st;
  if (w[PH_T] == 0) return ok();
  const int64_t es = elem_bytes(cache->fmt);
  BoundsArgs a;
  a.plan = static_cast<const int32_t*>(plan_dev);
  a.k = static_cast<const uint8_t*>(cache->k.ptr);
  a.k_sp = cache->k.stride_b * es; a.k_sr = cache->k.stride_row * es; a.k_sh = cache->k.stride_head * es;
  a.k_exp = cache->k_exp;
  a.e_sp = cache->exp_stride_page; a.e_sr = cache->exp_stride_row; a.e_sh = cache->exp_stride_head;
  a.code = bounds->code;
  a.c_sp = bounds->stride_page; a.c_sh = bounds->stride_head; a.c_sb = bounds->stride_bound;
  a.exp = bounds->exp;
  a.x_sp = bounds->exp_stride_page; a.x_sh = bounds->exp_stride_head;
  // (new rows of which none has a position enter no block, but those of a plan replayed here may)
  const int64_t ctas = int64_t(w[PH_NTOUCH] > 0 ? w[PH_NTOUCH] : 1) * w[PH_HKV];
  const int grid = int(ctas < kPagedSms * 16 ? ctas : kPagedSms * 16);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->fmt == BD_CACHE_BF16   ? launch_bounds<BD_CACHE_BF16>(w[PH_D], grid, s, a)
                        : cache->fmt == BD_CACHE_E4M3 ? launch_bounds<BD_CACHE_E4M3>(w[PH_D], grid, s, a)
                                                      : launch_bounds<BD_CACHE_E2M1>(w[PH_D], grid, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "bd_block_bounds_kernel launch");
  return ok();
}

extern "C" int32_t bd_block_select(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_bounds* bounds,
                                   bd_blocks* blocks, void* stream) {
  const int32_t* w = nullptr;
  int32_t st = view_paged_plan(plan_host, &w);
  if (st) return st;
  if (!plan_dev || reinterpret_cast<uintptr_t>(plan_dev) % 16)
    return fail(BD_ERR_ARG, "plan_dev NULL or not 16-byte aligned");
  if (!w[PH_BLOCKS]) return fail(BD_ERR_PLAN, "not a sparse plan");
  if ((st = check_bounds(bounds, w))) return st;
  if (w[PH_T] == 0) return ok();
  if ((st = check_tensor(q, "q", 2, 1, 1, w[PH_H], false))) return st;
  if (q->rows < w[PH_T]) return fail(BD_ERR_ARG, "q rows %d < %d new rows of the plan", q->rows, w[PH_T]);
  if ((st = check_blocks(blocks, w))) return st;
  SelectArgs a;
  a.plan = static_cast<const int32_t*>(plan_dev);
  a.q = static_cast<const uint8_t*>(q->ptr);
  a.q_sr = q->stride_row * 2; a.q_sh = q->stride_head * 2;
  a.code = bounds->code;
  a.c_sp = bounds->stride_page; a.c_sh = bounds->stride_head; a.c_sb = bounds->stride_bound;
  a.exp = bounds->exp;
  a.x_sp = bounds->exp_stride_page; a.x_sh = bounds->exp_stride_head;
  a.out = blocks->ptr;
  a.o_sr = blocks->stride_row; a.o_sh = blocks->stride_head;
  a.G = w[PH_G]; a.Hkv = w[PH_HKV];
  a.blocks = w[PH_BLOCKS]; a.first = w[PH_FIRST]; a.recent = w[PH_RECENT];
  a.page_shift = w[PH_PAGE_SHIFT]; a.cap = w[PH_SEL_CAP]; a.rows = w[PH_SEL_ROWS]; a.split = w[PH_SEL_SPLIT];
  const int64_t ctas = int64_t(w[PH_NSELG]) * w[PH_HKV];
  const int grid = int(ctas < kPagedSms * 8 ? ctas : kPagedSms * 8);
  const size_t smem = select_smem(a.rows, a.G, w[PH_D], a.cap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = w[PH_D] == 64 ? launch_select<64>(grid, smem, s, a) : w[PH_D] == 128 ? launch_select<128>(grid, smem, s, a)
                                                                            : launch_select<256>(grid, smem, s, a);
  return st ? st : ok();
}
