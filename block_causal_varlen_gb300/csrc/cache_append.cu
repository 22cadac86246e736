// Appending rows to a paged K/V cache with the position rotation on the way, on sm_103a.
//
// Pair i of a head's turned elements, at position p: (x, y) -> scale (x cos a - y sin a,
// y cos a + x sin a), a = p f_i. The angle is kept as turns: the host gives f_i / 2 pi modulo 1
// in units of 2^-64 (bd_rope_phases), so p times it modulo 2^64 is the angle's fraction of a
// turn, whatever p, and its upper 32 bits lose less than 2^-32 of a turn. No table of angles is read.
//
// A group of d / 8 lanes takes some heads of a row, 8 elements a lane: cosines and sines are made
// once and used for all of them. Pairs d / 2 apart meet by a shuffle. K goes on as
// bf16 into the cache's format (paged_quant.cuh), as bd_cache_write stores it.
//
// What bounds it is HBM, or for a few rows the launch and the chain plan - rows - stores; few
// rows are cut into many groups of few heads each. 19074 rows of 32 + 8 + 8 heads of 128 into bf16 75 us (6.25
// TB/s, 92% of a copy's rate; 114 with heads of q, K and V in one group, whose places were
// looked up head by head), 30273 into e4m3 124 (5.5 TB/s), into e2m1 127 (5.1; pairs d / 2 apart
// spill three registers, 12 bytes); 8 rows 2.3 us in a graph.
#include <cuda_runtime.h>

#include <cmath>

#include "paged.h"
#include "paged_quant.cuh"

namespace bd {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFull = 0xffffffffu;

struct AppendArgs {
  const int32_t* plan;
  const uint64_t* phase;
  float scale;
  int32_t rot;                               // turned elements of a head
  int32_t H, Hkv;                            // H = 0: no q
  int32_t per;                               // heads of a group, all of q, of K or of V
  int32_t nq, nkv, chunks;                   // groups of a row: nq of q, nkv of K, nkv of V
  const uint8_t *q, *k, *v;                  // packed bf16 rows, strides in bytes
  uint8_t* qo;
  int64_t q_sr, q_sh, k_sr, k_sh, v_sr, v_sh, o_sr, o_sh;
  uint8_t *kc, *vc;                          // cache bytes
  int64_t k_cp, k_cr, k_ch, v_cp, v_cr, v_ch;
  uint8_t *k_exp, *v_exp;
  int64_t e_sp, e_sr, e_sh;
};

template <int D, int FMT, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 4) bd_cache_append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8, RPB = kThreads / LPR;
  const int sub = threadIdx.x % LPR;
  const int32_t* plan = a.plan;
  // (the phases are weights, and not written by the kernels in front of this one, but by whom is
  // not known here: everything is read behind the wait)
  grid_wait();
  const uint32_t T = uint32_t(plan[PH_T]), n = T * uint32_t(a.chunks);
  const int32_t* tok = plan + plan[PH_OFF_TOK];
  const int32_t* where = plan + plan[PH_OFF_POS];
  const int shift = plan[PH_PAGE_SHIFT];
  const int half = a.rot / 16;                    // lanes of half of the turned elements
  const bool turns = sub < 2 * half;
  const bool upper = !PAIRS && sub >= half;       // the second elements of their pairs
  const int partner = int(threadIdx.x & 31u) - sub + (!turns || PAIRS ? sub : upper ? sub - half : sub + half);
  const uint64_t* phase = a.phase + (!turns ? 0 : PAIRS ? sub * 4 : (upper ? sub - half : sub) * 8);

  // (whole warps stay together for the shuffles: groups past the last repeat the last)
  for (uint32_t g0 = blockIdx.x * uint32_t(RPB); g0 < n; g0 += gridDim.x * uint32_t(RPB)) {
    const bool there = g0 + threadIdx.x / LPR < n;
    const uint32_t g = min(g0 + threadIdx.x / LPR, n - 1), t = g / uint32_t(a.chunks);
    const int c = int(g - t * uint32_t(a.chunks));
    const bool is_q = c < a.nq, is_k = !is_q && c < a.nq + a.nkv;
    const int h0 = (is_q ? c : is_k ? c - a.nq : c - a.nq - a.nkv) * a.per, cnt = min(a.per, (is_q ? a.H : a.Hkv) - h0);
    const int32_t row = tok[t], pos = where[t];
    const int64_t pg = row >> shift, ro = row & ((1 << shift) - 1);
    const bool store = there && (is_q || row >= 0), turn = turns && (is_q || is_k) && pos >= 0;
    // where the group's heads are read and go to, and its exponents or scales
    const int64_t ss = is_q ? a.q_sh : is_k ? a.k_sh : a.v_sh, ds = is_q ? a.o_sh : is_k ? a.k_ch : a.v_ch;
    const uint8_t* src = (is_q ? a.q + int64_t(t) * a.q_sr : is_k ? a.k + int64_t(t) * a.k_sr : a.v + int64_t(t) * a.v_sr) + h0 * ss + sub * 16;
    uint8_t* dst = (is_q ? a.qo + int64_t(t) * a.o_sr
                    : is_k ? a.kc + pg * a.k_cp + ro * a.k_cr : a.vc + pg * a.v_cp + ro * a.v_cr) + h0 * ds;
    uint8_t* exps = FMT == BD_CACHE_BF16 || is_q ? nullptr : (is_k ? a.k_exp : a.v_exp) + pg * a.e_sp + ro * a.e_sr + h0 * a.e_sh;
    constexpr int U = 4;  // heads in flight
    uint4 x[U];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < U; ++u, src += ss)
        if (h + u < cnt) x[u] = __ldcs(reinterpret_cast<const uint4*>(src));
    };
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = make_uint4(0, 0, 0, 0);
    load(0);
    // cosines and sines of this lane's four words of a head (pairs: of one pair each); the sign of a word's
    // own sine goes with its element's place in the pair
    float2 cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float cc[2], sv[2];
#pragma unroll
      for (int e = 0; e < (PAIRS ? 1 : 2); ++e) {
        const uint64_t f = __ldg(phase + (PAIRS ? i : 2 * i + e));
        const int32_t part = int32_t(uint32_t((f * uint64_t(uint32_t(max(pos, 0)))) >> 32));
        sincospif(float(part) * 4.656612873077393e-10f, &sv[e], &cc[e]);  // 2^-31: half turns
        cc[e] *= a.scale;
        sv[e] *= a.scale;
      }
      cs[i] = PAIRS ? make_float2(cc[0], cc[0]) : make_float2(cc[0], cc[PAIRS ? 0 : 1]);
      sn[i] = PAIRS ? make_float2(-sv[0], sv[0])
              : upper ? make_float2(sv[0], sv[PAIRS ? 0 : 1]) : make_float2(-sv[0], -sv[PAIRS ? 0 : 1]);
    }
    for (int hb = 0; hb < a.per; hb += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (hb + u >= a.per) break;
        uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = PAIRS ? w[i] : __shfl_sync(kFull, w[i], partner);
        if (turn) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
            const float2 o = PAIRS ? make_float2(v.y, v.x) : make_float2(bf16_lo(z[i]), bf16_hi(z[i]));
            const float2 r = dev::ffma2(v, cs[i], dev::fmul2(o, sn[i]));
            w[i] = bf16_pair(r.x, r.y);
          }
        }
        const uint4 y = make_uint4(w[0], w[1], w[2], w[3]);
        const bool mine = store && hb + u < cnt;
        if constexpr (FMT == BD_CACHE_BF16) {
          if (mine) __stcs(reinterpret_cast<uint4*>(dst) + sub, y);
        } else {
          if (mine && is_q) __stcs(reinterpret_cast<uint4*>(dst) + sub, y);
          if (__any_sync(kFull, mine && !is_q)) store_quantised<LPR, FMT>(y, sub, mine && !is_q, dst, exps);
          exps += a.e_sh;
        }
        dst += ds;
      }
      if (hb + U < a.per) load(hb + U);
    }
  }
}

template <int D, int FMT>
cudaError_t launch_append(bool pairs, int grid, cudaStream_t s, const AppendArgs& a) {
  return pairs ? launch_kernel(bd_cache_append_kernel<D, FMT, true>, grid, kThreads, 0, s, a)
               : launch_kernel(bd_cache_append_kernel<D, FMT, false>, grid, kThreads, 0, s, a);
}

template <int FMT>
cudaError_t launch_append(int d, bool pairs, int grid, cudaStream_t s, const AppendArgs& a) {
  return d == 64    ? launch_append<64, FMT>(pairs, grid, s, a)
         : d == 128 ? launch_append<128, FMT>(pairs, grid, s, a)
                    : launch_append<256, FMT>(pairs, grid, s, a);
}

}  // namespace

}  // namespace bd

using namespace bd;

extern "C" int32_t bd_rope_phases(const double* inv_freq, int32_t n, uint64_t* out) {
  if (n < 0 || (n > 0 && (!inv_freq || !out))) return fail(BD_ERR_ARG, "inv_freq or out is NULL, or n negative");
  // 1 / 2 pi in two parts, off by less than 2^-109; the product and what it lost, off by less than |f| 2^-107
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double f = inv_freq[i];
    if (!std::isfinite(f)) return fail(BD_ERR_ARG, "inv_freq[%d] is not finite", i);
    const double a = f * hi, b = std::fma(f, hi, -a) + f * lo;
    // modulo 1 as 64-bit fractions, of the magnitude (1 - |x| would lose what lies below 2^-53): the
    // parts below 1 are exact, cut at 2^-64
    auto turns = [](double x) {
      const double y = std::fabs(x), u = std::ldexp(y - std::floor(y), 32), w = std::floor(u);
      const uint64_t t = (uint64_t(w) << 32) + uint64_t(std::ldexp(u - w, 32));
      return x < 0 ? 0 - t : t;
    };
    out[i] = turns(a) + turns(b);
  }
  return ok();
}

extern "C" int32_t bd_cache_append(const void* plan_host, const void* plan_dev, const bd_tensor* q, const bd_tensor* k,
                                   const bd_tensor* v, const bd_rope* rope, const bd_paged_cache* cache, bd_tensor* q_out,
                                   void* stream) {
  const int32_t* w = nullptr;
  int32_t st = check_write(plan_host, plan_dev, k, v, cache, &w);
  if (st) return st;
  if (!rope || !rope->phase || reinterpret_cast<uintptr_t>(rope->phase) % 8)
    return fail(BD_ERR_ARG, "rope: NULL, or phase NULL or not 8-byte aligned");
  if (rope->dim <= 0 || rope->dim % 16 || rope->dim > w[PH_D])
    return fail(BD_ERR_ARG, "rope of %d elements (a multiple of 16, at most the head dim %d)", rope->dim, w[PH_D]);
  if (rope->interleaved != 0 && rope->interleaved != 1) return fail(BD_ERR_ARG, "rope: interleaved must be 0 or 1");
  if (!q != !q_out) return fail(BD_ERR_ARG, "q and q_out come together");
  if (w[PH_T] == 0) return ok();
  if (q) {
    if ((st = check_tensor(q, "q", 2, 1, 1, w[PH_H], false))) return st;
    if ((st = check_tensor(q_out, "q_out", 2, 1, 1, w[PH_H], false))) return st;
    if (q->rows < w[PH_T] || q_out->rows < w[PH_T])
      return fail(BD_ERR_ARG, "q/q_out rows %d/%d < %d new rows of the plan", q->rows, q_out->rows, w[PH_T]);
  }
  AppendArgs a = {};
  a.plan = static_cast<const int32_t*>(plan_dev);
  a.phase = rope->phase;
  a.scale = rope->scale;
  a.rot = rope->dim;
  a.H = q ? w[PH_H] : 0;
  a.Hkv = w[PH_HKV];
  if (q) {
    a.q = static_cast<const uint8_t*>(q->ptr); a.qo = static_cast<uint8_t*>(q_out->ptr);
    a.q_sr = q->stride_row * 2; a.q_sh = q->stride_head * 2;
    a.o_sr = q_out->stride_row * 2; a.o_sh = q_out->stride_head * 2;
  }
  a.k = static_cast<const uint8_t*>(k->ptr); a.v = static_cast<const uint8_t*>(v->ptr);
  a.k_sr = k->stride_row * 2; a.k_sh = k->stride_head * 2; a.v_sr = v->stride_row * 2; a.v_sh = v->stride_head * 2;
  const int64_t es = elem_bytes(cache->fmt);
  a.kc = static_cast<uint8_t*>(cache->k.ptr); a.vc = static_cast<uint8_t*>(cache->v.ptr);
  a.k_cp = cache->k.stride_b * es; a.k_cr = cache->k.stride_row * es; a.k_ch = cache->k.stride_head * es;
  a.v_cp = cache->v.stride_b * es; a.v_cr = cache->v.stride_row * es; a.v_ch = cache->v.stride_head * es;
  a.k_exp = cache->k_exp; a.v_exp = cache->v_exp;
  a.e_sp = cache->exp_stride_page; a.e_sr = cache->exp_stride_row; a.e_sh = cache->exp_stride_head;
  // heads of a group: as many as leave every SM 2048 lanes, up to 16
  const int64_t lanes = int64_t(w[PH_T]) * (a.H + 2 * a.Hkv) * (w[PH_D] / 8);
  a.per = int(lanes / (int64_t(kPagedSms) * 2048));
  a.per = a.per < 1 ? 1 : a.per > 16 ? 16 : a.per;
  a.nq = (a.H + a.per - 1) / a.per;
  a.nkv = (a.Hkv + a.per - 1) / a.per;
  a.chunks = a.nq + 2 * a.nkv;
  if (int64_t(w[PH_T]) * a.chunks > INT32_MAX) return fail(BD_ERR_CAPACITY, "new rows times heads past 2^31 - 1");
  const int64_t blocks = (int64_t(w[PH_T]) * a.chunks * (w[PH_D] / 8) + kThreads - 1) / kThreads;
  const int grid = int(blocks < kPagedSms * 8 ? blocks : kPagedSms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool pairs = rope->interleaved != 0;
  const cudaError_t e = cache->fmt == BD_CACHE_BF16   ? launch_append<BD_CACHE_BF16>(w[PH_D], pairs, grid, s, a)
                        : cache->fmt == BD_CACHE_E4M3 ? launch_append<BD_CACHE_E4M3>(w[PH_D], pairs, grid, s, a)
                                                      : launch_append<BD_CACHE_E2M1>(w[PH_D], pairs, grid, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "bd_cache_append_kernel launch");
  return ok();
}
