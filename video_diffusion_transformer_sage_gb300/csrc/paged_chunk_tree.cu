// paged_chunk_tree.cu -- attention of many query rows per K/V head over the paged cache, the new tokens a tree.
#include "paged_chunk.cuh"

namespace sage {

cudaError_t launch_paged_chunk_tree(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  return launch_chunk<true>(a, c, d, s);
}

}  // namespace sage
