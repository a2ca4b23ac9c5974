// paged_few.cu -- attention of few query rows per K/V head over the paged cache: the plain kernels (causal, windowed or full).
#include "paged_few.cuh"

namespace sage {

cudaError_t launch_paged_few(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  return launch_few<false>(a, c, d, s);
}

}  // namespace sage
