// Few-rows attention over a paged K/V cache of e2m1 (the kernel of paged_dec.cu).
#define BD_DEC_KERNEL_ONLY
#include "paged_dec.cu"

namespace bd {

int32_t launch_dec_e2m1(const int32_t* w, const AttnArgs& a, const bd_paged_cache* c, cudaStream_t s) {
  return launch_dec_fmt<BD_CACHE_E2M1, false>(w, c, a, s);
}

}  // namespace bd
