// Writing K/V rows into a paged cache and reading sequences back out of it, on
// sm_103a.
//
// (paged_quant.cuh has the formats' arithmetic.)
//
// Both kernels are streams: what bounds them is HBM (or, for a few rows, the
// launch). A thread takes 16 bytes of bf16 (8 values) of K and of V, so a head's
// row is d / 8 neighbouring lanes and its maximum a few shuffles. 30000 rows of 8 heads of
// 128 written: bf16 37.5 us (6607 GB/s), e4m3 33.4 (5577); 49152 read back: bf16 62.1
// (6483), e4m3 53.9 (5615). e2m1, 30273 rows written 23-28 us (6900-5700 GB/s: 16 values of a scale to
// a lane, 37 with 8), 49152 read back 43.4 (5950). Walking the rows without a division each, or scaling bf16
// pairs at once, changes nothing.
#include <cuda_runtime.h>

#include "paged.h"
#include "paged_quant.cuh"

namespace bd {

namespace {

constexpr int kThreads = 256;

struct CacheArgs {
  const int32_t* plan;
  uint8_t *k, *v;                  // cache bytes
  int64_t k_sp, k_sr, k_sh, v_sp, v_sr, v_sh;  // in bytes
  uint8_t *k_exp, *v_exp;
  int64_t e_sp, e_sr, e_sh;
  uint8_t *kx, *vx;                // packed bf16 rows
  int64_t kx_sr, kx_sh, vx_sr, vx_sh;          // in bytes
};

// Values of a row that a lane takes: of an e2m1 cache the 16 that share a scale.
constexpr int write_values(int fmt) { return fmt == BD_CACHE_E2M1 ? 16 : 8; }

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) bd_cache_write_kernel(const CacheArgs a) {
  constexpr int NV = write_values(FMT) / 8, LPR = D / (8 * NV), RPB = kThreads / LPR;  // lanes of a head's row, such rows of a block
  const int32_t* plan = a.plan;
  grid_wait();
  const uint32_t Hkv = uint32_t(plan[PH_HKV]), n = uint32_t(plan[PH_T]) * Hkv;
  const int32_t* tok = plan + plan[PH_OFF_TOK];
  const int shift = plan[PH_PAGE_SHIFT];
  const uint32_t sub = threadIdx.x % LPR;
  // (the whole warp takes part in the shuffles: rows past the last repeat the last)
  for (uint32_t r0 = blockIdx.x * uint32_t(RPB); r0 < n; r0 += gridDim.x * uint32_t(RPB)) {
    const uint32_t r = min(r0 + threadIdx.x / LPR, n - 1), t = r / Hkv, h = r - t * Hkv;
    const uint4* kp = reinterpret_cast<const uint4*>(a.kx + int64_t(t) * a.kx_sr + int64_t(h) * a.kx_sh) + sub * NV;
    const uint4* vp = reinterpret_cast<const uint4*>(a.vx + int64_t(t) * a.vx_sr + int64_t(h) * a.vx_sh) + sub * NV;
    uint4 kx[NV], vx[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) { kx[i] = __ldcs(kp + i); vx[i] = __ldcs(vp + i); }
    const int32_t row = tok[t];
    const int64_t pg = row >> shift, ro = row & ((1 << shift) - 1);
    const bool store = row >= 0 && r0 + threadIdx.x / LPR < n;
    uint8_t* kd = a.k + pg * a.k_sp + ro * a.k_sr + int64_t(h) * a.k_sh;
    uint8_t* vd = a.v + pg * a.v_sp + ro * a.v_sr + int64_t(h) * a.v_sh;
    if constexpr (FMT == BD_CACHE_BF16) {
      if (store) {
        reinterpret_cast<uint4*>(kd)[sub] = kx[0];
        reinterpret_cast<uint4*>(vd)[sub] = vx[0];
      }
    } else {
      if constexpr (FMT == BD_CACHE_E4M3) {
        uint32_t kb, vb;
        const uint2 kc = quantise8<LPR>(kx[0], &kb), vc = quantise8<LPR>(vx[0], &vb);
        if (store) {
          reinterpret_cast<uint2*>(kd)[sub] = kc;
          reinterpret_cast<uint2*>(vd)[sub] = vc;
          if (sub == 0) {
            const int64_t eo = pg * a.e_sp + ro * a.e_sr + int64_t(h) * a.e_sh;
            a.k_exp[eo] = uint8_t(kb);
            a.v_exp[eo] = uint8_t(vb);
          }
        }
      } else if (store) {
        const int64_t eo = pg * a.e_sp + ro * a.e_sr + int64_t(h) * a.e_sh;
        store_group_e2m1(kx[0], kx[NV - 1], sub, kd, a.k_exp + eo);
        store_group_e2m1(vx[0], vx[NV - 1], sub, vd, a.v_exp + eo);
      }
    }
  }
}

// A block takes kReadRows rows of a page at a time, all heads.
constexpr int kReadRows = 8;

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) bd_cache_read_kernel(const CacheArgs a) {
  constexpr uint32_t LPR = D / 8;
  constexpr int U = FMT == BD_CACHE_BF16 ? 2 : 4;  // rows in flight per thread: 64 bytes of loads
  const int32_t* plan = a.plan;
  grid_wait();
  const uint32_t Hkv = uint32_t(plan[PH_HKV]);
  const int32_t* pages = plan + plan[PH_OFF_PAGES];
  const int32_t* pgrow = plan + plan[PH_OFF_PGROW];
  const int32_t* pgcnt = plan + plan[PH_OFF_PGCNT];
  const int gshift = plan[PH_PAGE_SHIFT] - 3;  // groups of kReadRows rows in a page
  static_assert(kReadRows == 8, "gshift");
  const uint32_t ngroups = uint32_t(plan[PH_NPAGES]) << gshift;
  const uint32_t sub = threadIdx.x % LPR;
  // a group's place is looked up while the group before is copied
  auto place = [&](uint32_t g, int& page, int& dst, int& rows) {
    const uint32_t e = min(g, ngroups - 1) >> gshift;
    page = pages[e];
    dst = pgrow[e];
    rows = pgcnt[e];
  };
  int page, first, count;
  if (blockIdx.x < ngroups) place(blockIdx.x, page, first, count);
  for (uint32_t g = blockIdx.x; g < ngroups; g += gridDim.x) {
    const int r0 = int(g & ((1u << gshift) - 1)) * kReadRows;
    const int rows = min(kReadRows, count - r0);
    const int64_t pg = page, dst = int64_t(first) + r0;
    place(g + gridDim.x, page, first, count);
    if (rows <= 0) continue;
    const uint32_t n = uint32_t(rows) * Hkv;
    for (uint32_t i0 = threadIdx.x / LPR; i0 < n; i0 += U * (kThreads / LPR)) {
      uint4 x[U], y[U];
      float fk[U], fv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * (kThreads / LPR), ri = i / Hkv, h = i - ri * Hkv;
        if (i >= n) continue;
        const uint8_t* ks = a.k + pg * a.k_sp + int64_t(r0 + ri) * a.k_sr + int64_t(h) * a.k_sh;
        const uint8_t* vs = a.v + pg * a.v_sp + int64_t(r0 + ri) * a.v_sr + int64_t(h) * a.v_sh;
        if constexpr (FMT == BD_CACHE_BF16) {
          x[u] = __ldcs(reinterpret_cast<const uint4*>(ks) + sub);
          y[u] = __ldcs(reinterpret_cast<const uint4*>(vs) + sub);
        } else if constexpr (FMT == BD_CACHE_E2M1) {
          x[u].x = __ldcs(reinterpret_cast<const uint32_t*>(ks) + sub);
          y[u].x = __ldcs(reinterpret_cast<const uint32_t*>(vs) + sub);
          const int64_t eo = pg * a.e_sp + int64_t(r0 + ri) * a.e_sr + int64_t(h) * a.e_sh + sub / 2;
          x[u].y = a.k_exp[eo];
          y[u].y = a.v_exp[eo];
        } else {
          const uint2 k2 = __ldcs(reinterpret_cast<const uint2*>(ks) + sub), v2 = __ldcs(reinterpret_cast<const uint2*>(vs) + sub);
          x[u].x = k2.x; x[u].y = k2.y;
          y[u].x = v2.x; y[u].y = v2.y;
          const int64_t eo = pg * a.e_sp + int64_t(r0 + ri) * a.e_sr + int64_t(h) * a.e_sh;
          fk[u] = exp_factor(a.k_exp[eo]);
          fv[u] = exp_factor(a.v_exp[eo]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t i = i0 + u * (kThreads / LPR), ri = i / Hkv, h = i - ri * Hkv;
        if (i >= n) continue;
        if constexpr (FMT == BD_CACHE_E4M3) {
          const uint2 k0 = dequantise4(x[u].x, fk[u]), k1 = dequantise4(x[u].y, fk[u]);
          const uint2 v0 = dequantise4(y[u].x, fv[u]), v1 = dequantise4(y[u].y, fv[u]);
          x[u] = make_uint4(k0.x, k0.y, k1.x, k1.y);
          y[u] = make_uint4(v0.x, v0.y, v1.x, v1.y);
        } else if constexpr (FMT == BD_CACHE_E2M1) {
          x[u] = dequantise8_e2m1(x[u].x, x[u].y);
          y[u] = dequantise8_e2m1(y[u].x, y[u].y);
        }
        __stcs(reinterpret_cast<uint4*>(a.kx + (dst + ri) * a.kx_sr + int64_t(h) * a.kx_sh) + sub, x[u]);
        __stcs(reinterpret_cast<uint4*>(a.vx + (dst + ri) * a.vx_sr + int64_t(h) * a.vx_sh) + sub, y[u]);
      }
    }
  }
}

CacheArgs cache_args(const void* plan_dev, const bd_paged_cache* c, const bd_tensor* k, const bd_tensor* v) {
  const int64_t es = elem_bytes(c->fmt);
  CacheArgs a;
  a.plan = static_cast<const int32_t*>(plan_dev);
  a.k = static_cast<uint8_t*>(c->k.ptr); a.v = static_cast<uint8_t*>(c->v.ptr);
  a.k_sp = c->k.stride_b * es; a.k_sr = c->k.stride_row * es; a.k_sh = c->k.stride_head * es;
  a.v_sp = c->v.stride_b * es; a.v_sr = c->v.stride_row * es; a.v_sh = c->v.stride_head * es;
  a.k_exp = c->k_exp; a.v_exp = c->v_exp;
  a.e_sp = c->exp_stride_page; a.e_sr = c->exp_stride_row; a.e_sh = c->exp_stride_head;
  a.kx = static_cast<uint8_t*>(k->ptr); a.vx = static_cast<uint8_t*>(v->ptr);
  a.kx_sr = k->stride_row * 2; a.kx_sh = k->stride_head * 2;
  a.vx_sr = v->stride_row * 2; a.vx_sh = v->stride_head * 2;
  return a;
}

template <int FMT>
cudaError_t launch_write(int d, int grid, cudaStream_t s, const CacheArgs& a) {
  auto kernel = d == 64 ? bd_cache_write_kernel<64, FMT> : d == 128 ? bd_cache_write_kernel<128, FMT> : bd_cache_write_kernel<256, FMT>;
  return launch_kernel(kernel, grid, kThreads, 0, s, a);
}

template <int FMT>
cudaError_t launch_read(int d, int grid, cudaStream_t s, const CacheArgs& a) {
  auto kernel = d == 64 ? bd_cache_read_kernel<64, FMT> : d == 128 ? bd_cache_read_kernel<128, FMT> : bd_cache_read_kernel<256, FMT>;
  return launch_kernel(kernel, grid, kThreads, 0, s, a);
}

}  // namespace

int32_t check_paged(const void* plan_host, const void* plan_dev, const bd_paged_cache* c, const int32_t** out) {
  const int32_t* w = nullptr;
  int32_t st = view_paged_plan(plan_host, &w);
  if (st) return st;
  if (!plan_dev || reinterpret_cast<uintptr_t>(plan_dev) % 16)
    return fail(BD_ERR_ARG, "plan_dev NULL or not 16-byte aligned");
  if (!c) return fail(BD_ERR_ARG, "cache is NULL");
  if (c->fmt != w[PH_FMT]) return fail(BD_ERR_PLAN, "cache format %d, the plan was built for %d", c->fmt, w[PH_FMT]);
  if (c->num_pages != w[PH_NUM_PAGES] || c->k.rows != w[PH_PAGE] || c->v.rows != w[PH_PAGE])
    return fail(BD_ERR_PLAN, "cache of %d pages of %d / %d rows, the plan was built for %d of %d", c->num_pages, c->k.rows,
                c->v.rows, w[PH_NUM_PAGES], w[PH_PAGE]);
  const int es = elem_bytes(c->fmt);
  if ((st = check_tensor(&c->k, "cache k", es, c->num_pages, 1, w[PH_HKV], true))) return st;
  if ((st = check_tensor(&c->v, "cache v", es, c->num_pages, 1, w[PH_HKV], true))) return st;
  if (c->fmt != BD_CACHE_BF16) {
    if (!c->k_exp || !c->v_exp) return fail(BD_ERR_ARG, "an e4m3 or e2m1 cache needs k_exp and v_exp");
    if ((c->num_pages > 1 && c->exp_stride_page <= 0) || c->exp_stride_row <= 0 ||
        (w[PH_HKV] > 1 && c->exp_stride_head <= 0))
      return fail(BD_ERR_ARG, "exponent strides must be positive");
    if (c->exp_stride_row > INT32_MAX / w[PH_PAGE] / 2 || (w[PH_HKV] > 1 && c->exp_stride_head > INT32_MAX / w[PH_HKV] / 2))
      return fail(BD_ERR_UNSUPPORTED, "exponents of a page spread over more than 2^31 bytes");
  }
  if (c->fmt == BD_CACHE_E2M1) {
    const int al = scale_align(w[PH_D]);
    const uintptr_t p = reinterpret_cast<uintptr_t>(c->k_exp) | reinterpret_cast<uintptr_t>(c->v_exp);
    if (p % al || c->exp_stride_row % al || (c->num_pages > 1 && c->exp_stride_page % al) || (w[PH_HKV] > 1 && c->exp_stride_head % al))
      return fail(BD_ERR_ALIGN, "scales: pointers and strides must be multiples of %d bytes", al);
  }
  *out = w;
  return BD_OK;
}

int32_t check_write(const void* plan_host, const void* plan_dev, const bd_tensor* k, const bd_tensor* v,
                    const bd_paged_cache* cache, const int32_t** out) {
  int32_t st = check_paged(plan_host, plan_dev, cache, out);
  if (st) return st;
  const int32_t* w = *out;
  if (!w[PH_CAUSAL]) return fail(BD_ERR_PLAN, "new rows of a plan that is not causal have no cache positions");
  if (!w[PH_WRITE_OK]) return fail(BD_ERR_PLAN, "two new rows of the batch have the same cache row");
  if (w[PH_T] == 0) return BD_OK;
  if ((st = check_tensor(k, "k", 2, 1, 1, w[PH_HKV], false))) return st;
  if ((st = check_tensor(v, "v", 2, 1, 1, w[PH_HKV], false))) return st;
  if (k->rows < w[PH_T] || v->rows < w[PH_T])
    return fail(BD_ERR_ARG, "k/v rows %d/%d < %d new rows of the plan", k->rows, v->rows, w[PH_T]);
  return BD_OK;
}

}  // namespace bd

using namespace bd;

extern "C" int32_t bd_cache_write(const void* plan_host, const void* plan_dev, const bd_tensor* k, const bd_tensor* v,
                                  const bd_paged_cache* cache, void* stream) {
  const int32_t* w = nullptr;
  int32_t st = check_write(plan_host, plan_dev, k, v, cache, &w);
  if (st) return st;
  if (w[PH_T] == 0) return ok();
  const CacheArgs a = cache_args(plan_dev, cache, k, v);
  const int64_t blocks = (int64_t(w[PH_T]) * w[PH_HKV] * (w[PH_D] / write_values(cache->fmt)) + kThreads - 1) / kThreads;
  // three rounds of 8 CTAs an SM: 30000 / 100000 e4m3 rows of 8 heads 33.4 / 93-95 us, with
  // one round 35.5 / 97-99, with two 33.4 / 97
  const int grid = int(blocks < kPagedSms * 24 ? blocks : kPagedSms * 24);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->fmt == BD_CACHE_BF16   ? launch_write<BD_CACHE_BF16>(w[PH_D], grid, s, a)
                        : cache->fmt == BD_CACHE_E4M3 ? launch_write<BD_CACHE_E4M3>(w[PH_D], grid, s, a)
                                                      : launch_write<BD_CACHE_E2M1>(w[PH_D], grid, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "bd_cache_write_kernel launch");
  return ok();
}

extern "C" int32_t bd_cache_read(const void* plan_host, const void* plan_dev, const bd_paged_cache* cache, bd_tensor* k,
                                 bd_tensor* v, void* stream) {
  const int32_t* w = nullptr;
  int32_t st = check_paged(plan_host, plan_dev, cache, &w);
  if (st) return st;
  if (w[PH_KV_TOTAL] == 0) return ok();
  if ((st = check_tensor(k, "k", 2, 1, 1, w[PH_HKV], false))) return st;
  if ((st = check_tensor(v, "v", 2, 1, 1, w[PH_HKV], false))) return st;
  if (k->rows < w[PH_KV_TOTAL] || v->rows < w[PH_KV_TOTAL])
    return fail(BD_ERR_ARG, "k/v rows %d/%d < %d cached rows of the plan", k->rows, v->rows, w[PH_KV_TOTAL]);
  const CacheArgs a = cache_args(plan_dev, cache, k, v);
  const int64_t groups = int64_t(w[PH_NPAGES]) * (w[PH_PAGE] / kReadRows);
  const int grid = int(groups < kPagedSms * 8 ? groups : kPagedSms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->fmt == BD_CACHE_BF16   ? launch_read<BD_CACHE_BF16>(w[PH_D], grid, s, a)
                        : cache->fmt == BD_CACHE_E4M3 ? launch_read<BD_CACHE_E4M3>(w[PH_D], grid, s, a)
                                                      : launch_read<BD_CACHE_E2M1>(w[PH_D], grid, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "bd_cache_read_kernel launch");
  return ok();
}
