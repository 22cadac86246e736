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
// block's keys.
//
// bd_block_select_kernel: a CTA for each (new row, K/V head). Scores: d / 16 lanes take a block,
// four blocks at a time, by dp4a (positive q against hi, negative against lo); they stay in shared
// memory as whole numbers of the same order. Choice: the threshold two bits a round from the highest bit
// in which scores differ, then the blocks above it and the first ones equal to it, in order.
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
        out[col] = bad ? int8_t(0) : int8_t(fminf(fmaxf(floorf(lo[c] * f), -127.f), 127.f));
        out[a.c_sb + col] = bad ? int8_t(0) : int8_t(fminf(fmaxf(ceilf(hi[c] * f), -127.f), 127.f));
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
  int32_t G, Hkv, blocks, first, recent, page_shift, cap;
};

constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32;
// shared memory: positive and negative parts of q's codes [G][2][d], their powers of two [G], keys [cap]
constexpr size_t select_smem(int G, int d, int cap) { return size_t(G) * (2 * d + 4) + size_t(cap) * 4; }

// A score as a whole number of the same order. Above all of them: an infinity of a block with NaN
// or infinities, and the blocks that are always listed.
__device__ __forceinline__ uint32_t order_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kOddBlock = 0xff800000u, kAlways = 0xffffffffu;

template <int D>
__global__ void __launch_bounds__(kSelThreads) bd_block_select_kernel(const SelectArgs a) {
  constexpr int LPB = D / 16, GPW = 32 / LPB;  // lanes of a block; blocks of a warp at a time, times U
  constexpr int U = 4;
  static_assert(LPB >= U, "four sums meet in four lanes at least");
  extern __shared__ uint4 sel_smem[];
  uint8_t* s_q = reinterpret_cast<uint8_t*>(sel_smem);
  int* s_eq = reinterpret_cast<int*>(s_q + a.G * 2 * D);
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_eq + a.G);
  __shared__ uint32_t s_red[kSelWarps][4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t* plan = a.plan;
  grid_wait();
  const int T = plan[PH_T];
  const int32_t *where = plan + plan[PH_OFF_POS], *rowpg = plan + plan[PH_OFF_ROWPG];
  for (int64_t x = blockIdx.x; x < int64_t(T) * a.Hkv; x += gridDim.x) {
    const int t = int(x / a.Hkv), g = int(x % a.Hkv);
    const int pos = where[t], nblk = pos < 0 ? 0 : (pos >> a.page_shift) + 1;
    int32_t* out = a.out + int64_t(t) * a.o_sr + int64_t(g) * a.o_sh;
    if (nblk <= a.blocks) {  // all there are
      for (int i = tid; i < a.blocks; i += kSelThreads) out[i] = i < nblk ? i : -1;
      continue;
    }
    const int32_t* pages = plan + rowpg[t];
    // ---- q's codes: a warp for each head
    for (int h = warp; h < a.G; h += kSelWarps) {
      const uint8_t* p = a.q + int64_t(t) * a.q_sr + int64_t(g * a.G + h) * a.q_sh;
      const bool in = lane < D / 8;
      const uint4 v = in ? *(reinterpret_cast<const uint4*>(p) + lane) : make_uint4(0, 0, 0, 0);
      uint32_t mx = absmax8(v);
      mx = __reduce_max_sync(kFull, mx);
      const bool bad = mx >= 0x7f80u;
      const int e = bad ? 0 : pow8(__uint_as_float(mx << 16));
      const float f = bad ? 0.f : pow2f(-e);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t up[2] = {0, 0}, down[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        const int c = bad ? 0 : int(fminf(fmaxf(rintf(y * f), -127.f), 127.f));
        up[i >> 2] |= uint32_t(max(c, 0) & 255) << (8 * (i & 3));
        down[i >> 2] |= uint32_t(min(c, 0) & 255) << (8 * (i & 3));
      }
      if (in) {
        *reinterpret_cast<uint2*>(s_q + (h * 2) * D + lane * 8) = make_uint2(up[0], up[1]);
        *reinterpret_cast<uint2*>(s_q + (h * 2 + 1) * D + lane * 8) = make_uint2(down[0], down[1]);
      }
      if (lane == 0) s_eq[h] = e;
    }
    __syncthreads();
    // ---- scores
    const int sub = lane % LPB;
    for (int b0 = (warp * GPW + lane / LPB) * U; b0 - (lane / LPB) * U < nblk; b0 += kSelWarps * GPW * U) {
      uint4 lo[U], hi[U];
      int page[U];
#pragma unroll
      for (int u = 0; u < U; ++u) page[u] = pages[min(b0 + u, nblk - 1)];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int8_t* p = a.code + int64_t(page[u]) * a.c_sp + int64_t(g) * a.c_sh + sub * 16;
        lo[u] = *reinterpret_cast<const uint4*>(p);
        hi[u] = *reinterpret_cast<const uint4*>(p + a.c_sb);
      }
      // after the sums have met a lane has block b0 + mine
      const int mine = (sub & 1) * 2 + ((sub >> 1) & 1);
      int mypage = page[0];
#pragma unroll
      for (int u = 1; u < U; ++u) mypage = mine == u ? page[u] : mypage;
      const uint32_t eb = a.exp[int64_t(mypage) * a.x_sp + int64_t(g) * a.x_sh];
      float best = -CUDART_INF_F;
      for (int h = 0; h < a.G; ++h) {
        const uint4 p = *reinterpret_cast<const uint4*>(s_q + (h * 2) * D + sub * 16);
        const uint4 m = *reinterpret_cast<const uint4*>(s_q + (h * 2 + 1) * D + sub * 16);
        int s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          int v = __dp4a(int(p.x), int(hi[u].x), 0);
          v = __dp4a(int(p.y), int(hi[u].y), v);
          v = __dp4a(int(p.z), int(hi[u].z), v);
          v = __dp4a(int(p.w), int(hi[u].w), v);
          v = __dp4a(int(m.x), int(lo[u].x), v);
          v = __dp4a(int(m.y), int(lo[u].y), v);
          v = __dp4a(int(m.z), int(lo[u].z), v);
          s[u] = __dp4a(int(m.w), int(lo[u].w), v);
        }
        // lanes of odd number go on with blocks 2 and 3, then those with bit 1 set with 1 and 3
        const int t0 = __shfl_xor_sync(kFull, sub & 1 ? s[0] : s[2], 1), t1 = __shfl_xor_sync(kFull, sub & 1 ? s[1] : s[3], 1);
        const int r0 = (sub & 1 ? s[2] : s[0]) + t0, r1 = (sub & 1 ? s[3] : s[1]) + t1;
        int v = (sub & 2 ? r1 : r0) + __shfl_xor_sync(kFull, sub & 2 ? r0 : r1, 2);
#pragma unroll
        for (int y = 4; y < LPB; y <<= 1) v += __shfl_xor_sync(kFull, v, y);
        best = fmaxf(best, float(v) * pow2f(s_eq[h] + int(eb) - 127));
      }
      const int b = b0 + mine;
      if (sub < U && b < nblk)
        s_key[b] = b < a.first || b >= nblk - a.recent ? kAlways : eb == 255u ? kOddBlock : order_of(best);
    }
    __syncthreads();
    // ---- the blocks-th largest key. Keys from tid * per on are this thread's.
    const int per = (nblk + kSelThreads - 1) / kSelThreads;
    const int i0 = min(tid * per, nblk), i1 = min(i0 + per, nblk);
    uint32_t all1 = ~0u, any1 = 0;
    for (int i = i0; i < i1; ++i) { all1 &= s_key[i]; any1 |= s_key[i]; }
    all1 = __reduce_and_sync(kFull, all1);
    any1 = __reduce_or_sync(kFull, any1);
    if (lane == 0) { s_red[warp][0] = all1; s_red[warp][1] = any1; }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) { all1 &= s_red[w][0]; any1 |= s_red[w][1]; }
    const uint32_t differ = all1 ^ any1;
    // thr: the largest number that `blocks` keys are not below, bit by bit from the first that differs
    int bit = differ ? 31 - __clz(differ) : -1;
    uint32_t thr = bit < 0 ? all1 : bit == 31 ? 0u : all1 & ~((2u << bit) - 1u);
    while (bit >= 0) {
      const int sh = max(bit - 1, 0), steps = bit > 0 ? 3 : 1;
      const uint32_t c1 = thr + (1u << sh), c2 = steps == 3 ? thr + (2u << sh) : ~0u, c3 = steps == 3 ? thr + (3u << sh) : ~0u;
      uint32_t n1 = 0, n23 = 0;  // two counts of 16 bits
      for (int i = i0; i < i1; ++i) {
        const uint32_t k = s_key[i];
        n1 += k >= c1 ? 1u : 0u;
        n23 += (k >= c2 ? 1u : 0u) + (k >= c3 ? 0x10000u : 0u);
      }
      n1 = __reduce_add_sync(kFull, n1);
      n23 = __reduce_add_sync(kFull, n23);
      __syncthreads();
      if (lane == 0) { s_red[warp][0] = n1; s_red[warp][1] = n23; }
      __syncthreads();
      n1 = n23 = 0;
#pragma unroll
      for (int w = 0; w < kSelWarps; ++w) { n1 += s_red[w][0]; n23 += s_red[w][1]; }
      const int K = a.blocks;
      if (steps == 1) thr = int(n1) >= K ? c1 : thr;
      else thr = int(n23 >> 16) >= K ? c3 : int(n23 & 0xffffu) >= K ? c2 : int(n1) >= K ? c1 : thr;
      bit -= 2;
    }
    // ---- those above thr, and of those equal to it the first ones, in order
    uint32_t cnt = 0;  // above in the lower 16 bits, equal in the upper ones
    for (int i = i0; i < i1; ++i) cnt += s_key[i] > thr ? 1u : s_key[i] == thr ? 0x10000u : 0u;
    uint32_t sum = cnt;
#pragma unroll
    for (int y = 1; y < 32; y <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, sum, y);
      if (lane >= y) sum += v;
    }
    __syncthreads();
    if (lane == 31) s_red[warp][0] = sum;
    __syncthreads();
    uint32_t before = sum - cnt, total = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      before += w < warp ? s_red[w][0] : 0u;
      total += s_red[w][0];
    }
    const int room = a.blocks - int(total & 0xffffu);  // for keys equal to thr
    int above = int(before & 0xffffu), equal = int(before >> 16);
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = s_key[i];
      if (k > thr) out[above++ + min(equal, room)] = i;
      else if (k == thr) {
        if (equal < room) out[above + equal] = i;
        ++equal;
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

template <int D>
int32_t launch_select(int grid, size_t smem, cudaStream_t s, const SelectArgs& a) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(bd_block_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int(select_smem(128, D, kMostBlocks)));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(block select)");
    if (dev < 64) done[dev].store(true, std::memory_order_release);
  }
  const cudaError_t e = launch_kernel(bd_block_select_kernel<D>, grid, kSelThreads, smem, s, a);
  return e == cudaSuccess ? BD_OK : cuda_fail(e, "bd_block_select_kernel launch");
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
  if (w[PH_NTOUCH] == 0) return ok();
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
  const int64_t ctas = int64_t(w[PH_NTOUCH]) * w[PH_HKV];
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
  a.page_shift = w[PH_PAGE_SHIFT]; a.cap = w[PH_SEL_CAP];
  const int64_t ctas = int64_t(w[PH_T]) * w[PH_HKV];
  const int grid = int(ctas < kPagedSms * 8 ? ctas : kPagedSms * 8);
  const size_t smem = select_smem(a.G, w[PH_D], a.cap);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = w[PH_D] == 64 ? launch_select<64>(grid, smem, s, a) : w[PH_D] == 128 ? launch_select<128>(grid, smem, s, a)
                                                                            : launch_select<256>(grid, smem, s, a);
  return st ? st : ok();
}
