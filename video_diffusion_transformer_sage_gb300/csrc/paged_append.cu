// paged_append.cu -- new tokens into the paged K/V cache: RMSNorm and rotation of Q and K rows (the
// row arithmetic of qk_row.cuh), K and V stored to their pages as bf16 or E4M3 codes.
//
// A CTA takes rows of one token: its Q heads, then its K heads, then its V heads, D/8 lanes per
// row with 16 bytes each, so 256 threads hold 16 (D = 128) or 32 rows at a time.  The rows are
// loaded before the chain cu_q -> kv_len -> page table is walked, which hides under them.  HBM-bound
// for many tokens; for few the chain of dependent loads is the time, and the rows of a token are
// then spread over CTAs of one batch of rows each.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged_batch.cuh"
#include "qk_row.cuh"

namespace sage {
namespace {

// A plain (coherent) load: q_out may be q itself.
__device__ __forceinline__ uint4 ld_row8(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// kBatch: batches of rows a thread holds at once (kBatch 16-byte loads in flight).
template <int D, bool kE4M3, int kBatch>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAppendArgs a) {
  constexpr int VPR = D / 8, RPP = 256 / VPR;
  const int t = blockIdx.x;
  const int c8 = threadIdx.x % VPR, rin = threadIdx.x / VPR;
  const int rows = a.hq + 2 * a.hkv;
  auto load = [&](int r) -> uint4 {
    if (r < a.hq) return ld_row8(a.q + t * a.qst + r * a.qsh + c8 * 8);
    if (r < a.hq + a.hkv) return ld_row8(a.k + t * a.kst + (r - a.hq) * a.ksh + c8 * 8);
    if (r < rows) return ld_row8(a.v + t * a.vst + (r - a.hq - a.hkv) * a.vsh + c8 * 8);
    return make_uint4(0, 0, 0, 0);
  };
  const int r0 = blockIdx.y * kBatch * RPP + rin;
  uint4 x[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) x[i] = load(r0 + i * RPP);
  // The token's place, found by every warp for itself.
  const int b = find_seq(a.b, t);
  if (b < 0) return;                       // a row of no sequence: left as it is
  const int start = __ldg(a.b.cu_q + b), end = __ldg(a.b.cu_q + b + 1), len = __ldg(a.b.kv_len + b);
  (void)start;
  const int64_t pos = static_cast<int64_t>(len) - end + t;
  int64_t row = pos;
  if (a.rope_cos && a.positions) row = __ldg(a.positions + t);
  int page = -1;
  if (pos >= 0 && pos < a.b.cap) page = __ldg(a.b.table + b * a.b.table_stride + (pos >> a.b.page_shift));
  const bool row_ok = !a.rope_cos || (row >= 0 && row < a.rope_rows);
  const bool placed = page >= 0 && page < a.b.n_pages && row_ok;
  if (!placed && pos >= 0 && threadIdx.x == 0 && blockIdx.y == 0)
    record_bad_index(a.status, pos >= a.b.cap ? kWhereLength : row_ok ? kWherePage : kWhereRopeRow);
  const int64_t slot = pos & ((1 << a.b.page_shift) - 1);
  float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.rope_cos && placed) {
    cs = __ldg(reinterpret_cast<const float4*>(a.rope_cos + row * (D / 2) + c8 * 4));
    sn = __ldg(reinterpret_cast<const float4*>(a.rope_sin + row * (D / 2) + c8 * 4));
  }
  const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int r = r0 + i * RPP;
    const bool is_q = r < a.hq, is_v = r >= a.hq + a.hkv;
    float f[8];
    unpack_bf16x8(x[i], f);
    const float* gamma = is_q ? a.gamma_q : is_v ? nullptr : a.gamma_k;
    const float sumsq = row_sumsq<VPR>(f);   // a butterfly: every lane, whatever its row
    if (r >= rows) continue;
    if (gamma) {
      float g[8];
      load_gamma8(gamma, c8, g);
      const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(sumsq, 1.0f / D), a.eps)));
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(__fmul_rn(f[j], rs), g[j]);
    }
    if (a.rope_cos && !is_v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float y0 = f[2 * j], y1 = f[2 * j + 1];
        f[2 * j] = __fsub_rn(__fmul_rn(y0, cc[j]), __fmul_rn(y1, ss[j]));
        f[2 * j + 1] = __fadd_rn(__fmul_rn(y0, ss[j]), __fmul_rn(y1, cc[j]));
      }
    }
    if (is_q) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (placed)
        o = make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7]));
      *reinterpret_cast<uint4*>(a.q_out + t * a.ost + r * a.osh + c8 * 8) = o;
    } else if (placed) {
      const int h = is_v ? r - a.hq - a.hkv : r - a.hq;
      uint8_t* dst = is_v ? a.v_pages + page * a.vp + slot * a.vt + h * a.vh
                          : a.k_pages + page * a.kp + slot * a.kt + h * a.kh;
      if (kE4M3) {
        const float s = __ldg((is_v ? a.v_scale : a.k_scale) + h);
        uint16_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e4m3x2(__fdiv_rn(f[2 * j], s), __fdiv_rn(f[2 * j + 1], s));
        *reinterpret_cast<uint2*>(dst + c8 * 8) = make_uint2(pack_h2(w[0], w[1]), pack_h2(w[2], w[3]));
      } else {
        const uint4 o = is_v ? x[i]
                             : make_uint4(bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                                          bf16x2_rne(f[6], f[7]));
        *reinterpret_cast<uint4*>(dst + c8 * 16) = o;
      }
    }
  }
}

template <int D, bool kE4M3>
cudaError_t launch_t(const PagedAppendArgs& a, cudaStream_t s) {
  constexpr int RPP = 256 / (D / 8);
  const int rows = a.hq + 2 * a.hkv;
  const int batches = (rows + RPP - 1) / RPP;
  paged_append_kernel<D, kE4M3, 1><<<dim3(a.b.n_tokens, batches), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int d, bool e4m3, cudaStream_t s) {
  if (d == 128) return e4m3 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
  return e4m3 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace sage
