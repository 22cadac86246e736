// Attention of new rows over the blocks that their lists name (the kernel of paged_dec.cu).
#define BD_DEC_KERNEL_ONLY
#include "paged_dec.cu"

namespace bd {

int32_t launch_dec_blocks(const int32_t* w, const AttnArgs& a, const bd_paged_cache* c, cudaStream_t s) {
  return c->fmt == BD_CACHE_BF16   ? launch_dec_fmt<BD_CACHE_BF16, true>(w, c, a, s)
         : c->fmt == BD_CACHE_E4M3 ? launch_dec_fmt<BD_CACHE_E4M3, true>(w, c, a, s)
                                   : launch_dec_fmt<BD_CACHE_E2M1, true>(w, c, a, s);
}

}  // namespace bd
