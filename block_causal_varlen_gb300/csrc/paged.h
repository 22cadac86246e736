// Host-side helpers shared by the paged-cache entry points, and their kernels'
// common arguments.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "host_util.h"
#include "paged_plan.h"
#include "tmap_pages.h"

namespace bd {

// Every paged kernel is launched so that its grid may start while the one in front of it in
// the stream ends: it waits in grid_wait, until that grid and all in front of it have ended
// and their writes are seen, before it reads anything, the plan included (what needs no
// memory of others comes before). One sequence of 64 keys 3.9 -> 3.7 us in a graph.
template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The few-rows kernel behind the tile kernel of its call does not depend on it, only on what
// that one waited for, and runs on SMs that its CTAs have left. A grid that starts early is
// promised others' writes by a wait of its own only, so the tile kernel's CTAs hand on what
// they have waited for: each releases a word for two few-rows CTAs, which acquire it
// before their first read, or wait for the tile kernel's end if it is not there. The CTA
// that takes a word clears it; a workspace that holds anything else needs no clearing. (10
// ragged e4m3 sequences, one row to 1024: 268 us, 280 where one kernel follows the other.)
constexpr unsigned long long kGo = 0x9e1c5a37d20b64f1ull;
constexpr int kGoTries = 64;
__device__ __forceinline__ void give_go(unsigned long long* go) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(go), "l"(kGo) : "memory");
}
// By one thread of the CTA; the others follow behind a barrier of the CTA.
__device__ __forceinline__ bool take_go(unsigned long long* go) {
  unsigned long long x = 0;
  for (int i = 0; i < kGoTries && x != kGo; ++i) asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(go) : "memory");
  if (x != kGo) grid_wait();
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(go), "l"(0ull) : "memory");
  return x == kGo;
}
// Orders what was acquired before this thread's asynchronous copies (TMA) as well.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Checks both plan copies and the cache against the plan.
int32_t check_paged(const void* plan_host, const void* plan_dev, const bd_paged_cache* cache, const int32_t** w);

// Exponent byte b of an e4m3 row as a factor 2^(b - 127); byte 255 marks a row
// that held an infinity or a NaN.
__device__ __forceinline__ float exp_factor(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// Partial results: per slot m and l of its rows, then O [rows][d]. The few-rows
// kernel's slots have kDecSlotRows rows, the tile kernel's tile_slot_rows(d): 128 for each
// of its tiles of 128 / G new rows.
__host__ __device__ constexpr int64_t slot_floats(int rows, int d) { return int64_t(rows) * (d + 2); }

struct MergeArgs {
  const int32_t* plan;
  const float* part;
  __nv_bfloat16* o;
  int64_t o_sr, o_sh;
  float* lse;
  int64_t l_sh;
  int32_t G;
};

// Joins the split blocks of the few-rows (tile = false; wide: some in many parts) or the
// tile kernel.
int32_t launch_merge(const MergeArgs& a, int d, bool tile, bool wide, cudaStream_t stream);

struct AttnArgs {
  const int32_t* plan;
  const __nv_bfloat16* q;
  int64_t q_sr, q_sh;
  __nv_bfloat16* o;
  int64_t o_sr, o_sh;
  float* lse;  // NULL: not wanted
  int64_t l_sh;
  float* part;
  const uint8_t* vc;  // the cache's V, strides in bytes
  int64_t v_sp, v_sr, v_sh;
  const uint8_t *k_exp, *v_exp;
  int64_t e_sp, e_sr, e_sh;
  float scale_log2;
  int32_t G, causal, page_shift;
  unsigned long long* go;  // a word for each few-rows CTA if both kernels run, else NULL
};

int32_t launch_tile(const int32_t* w, const AttnArgs& a, const bd_tensor* q, const bd_paged_cache* cache,
                    cudaStream_t stream);
int32_t launch_dec(const int32_t* w, const AttnArgs& a, const bd_paged_cache* cache, cudaStream_t stream);

}  // namespace bd
