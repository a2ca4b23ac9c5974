// paged_internal.h -- what the paged-cache kernels and their C entry points share.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "paged_join.h"
#include "sage_internal.h"
#include "sage_paged.h"

namespace sage {

enum PagedWhere : int32_t { kWherePage = 16, kWhereLength = 17, kWhereRopeRow = 18, kWherePagedFull = 19,
                            kWherePagedEmpty = 20, kWherePagedMma = 21 };

// The batch as the kernels take it.
struct PagedBatchDev {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  int n_seqs;
  int n_tokens;      // rows of the call's views
  int cap;           // max_pages * page_size
  int n_pages;
  int page_shift;    // log2 of page_size
};

struct PagedAppendArgs {
  PagedBatchDev b;
  const uint16_t *q, *k, *v;
  int64_t qst, qsh, kst, ksh, vst, vsh;
  int hq, hkv;
  const float *gamma_q, *gamma_k, *rope_cos, *rope_sin;
  int64_t rope_rows;
  const int32_t* positions;
  float eps;
  uint8_t *k_pages, *v_pages;
  int64_t kp, kt, kh, vp, vt, vh;   // page, slot and head strides in bytes
  const float *k_scale, *v_scale;
  uint16_t* q_out;
  int64_t ost, osh;
  int32_t* status;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, int d, bool e4m3, cudaStream_t s);

// The rows of one partial result.
constexpr int kPagedChunkRows = 256;

struct PagedAttnArgs {
  PagedBatchDev b;
  const uint16_t* q;
  int64_t qst, qsh;
  int hq, hkv;
  int causal, window;
  float scale_log2;            // sm_scale * log2 e
  const float *k_scale, *v_scale;
  uint16_t* out;
  int64_t ost, osh;
  float* lse;
  int32_t* status;
  int32_t* counters;           // [2 kPagedMaxCtas + 2], zero between calls
  float2* part_ml;             // [slots][rows]: running maximum (log2 units) and sum
  float* part_o;               // [slots][rows][D]
};

// paged_few.cu: up to 32 query rows (tokens x query heads of one K/V head) per tile.
cudaError_t launch_paged_few(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s);
// paged_chunk.cu: 256 query rows per unit.
cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s);

}  // namespace sage
