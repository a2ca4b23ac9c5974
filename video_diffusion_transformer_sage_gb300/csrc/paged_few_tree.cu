// paged_few_tree.cu -- attention of few query rows per K/V head over the paged cache, the new tokens a tree.
#include "paged_few.cuh"

namespace sage {

cudaError_t launch_paged_few_tree(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  return launch_few<true>(a, c, d, s);
}

}  // namespace sage
