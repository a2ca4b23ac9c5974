// tensor_map.h -- host side: the driver's tensor-map encoder, looked up once.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

namespace sage {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// One of a cache's two page arrays as a 4-D map {head_dim, heads, slots, pages}: boxes of box_c
// channels x 1 head x box_rows slots x 1 page, 128-byte swizzled (64-byte where a box row is 64
// bytes).  Strides in bytes; that of a dimension of extent 1 is never stepped, so any valid value
// stands in for it.
inline bool make_page_map(CUtensorMap* m, const void* base, bool e4m3, int64_t d, int64_t heads, int64_t slots,
                          int64_t pages, int64_t stride_head, int64_t stride_slot, int64_t stride_page, int box_c,
                          int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int64_t row = d * (e4m3 ? 1 : 2);
  if (heads == 1) stride_head = row;
  if (slots == 1) stride_slot = row;
  if (pages == 1) stride_page = row;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(slots),
                        static_cast<cuuint64_t>(pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride_head), static_cast<cuuint64_t>(stride_slot),
                           static_cast<cuuint64_t>(stride_page)};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(box_c), 1, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const int box_bytes = box_c * (e4m3 ? 1 : 2);
  // L2 fetches no more than a head's row at a time: the next head's would come in for another CTA, another time (24
  // heads of 64 channels, single tokens: 66 us against 74 at 256 bytes for bf16, 240 against 346 for E4M3).
  const CUtensorMapL2promotion promo = row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                       : row == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                    : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sage
