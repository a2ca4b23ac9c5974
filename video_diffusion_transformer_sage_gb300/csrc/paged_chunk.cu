// paged_chunk.cu -- attention of many query rows per K/V head over the paged cache: the plain kernels (causal, windowed or full).
#include "paged_chunk.cuh"

namespace sage {

cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  return launch_chunk<false>(a, c, d, s);
}

}  // namespace sage
