// paged_append.cu -- new tokens into the paged K/V cache: RMSNorm and rotation of Q and K rows (the
// row arithmetic of qk_row.cuh), K and V stored to their pages as bf16 or E4M3 codes.
//
// A warp takes up to 4 kSteps rows (8 kSteps at D = 64) of one token: its Q heads, then its K heads,
// then its V heads.  D/16 lanes hold a row, each the 8-channel groups g and g + D/16, which are the first two that the
// row's sum of squares adds: the fold over the lanes is then the same butterfly as with a lane per group,
// and the root, the division and the address of a row are paid by half as many threads.  The rows are loaded first;
// the chain cu_q -> kv_len -> page table -> rotary row hides under them.  Warps do not wait for one another.
//
// What bounds it: HBM for many tokens, each row read once and written once: 4.77 TB/s at 3024 tokens of 168 rows of
// D = 128 (54.9 us), 3.9 TB/s at 11927 tokens of 72 rows of D = 64 into E4M3 (47.6 us), where the instructions of
// the norm weigh as much as the bytes; for few tokens the chain of dependent loads.  A warp takes three steps of rows
// where the batch fills the GPU (two: 55.9 and 51.3 us, one: 64.0 and 58.0), two where three would leave
// lanes of a token's last warp idle, one where spreading the rows over more SMs shortens the chain.
#include <cuda_bf16.h>

#include <algorithm>

#include "paged_batch.cuh"
#include "qk_row.cuh"

namespace sage {
namespace {

// kCoherent: q_out may be q itself, so its rows may not come through the read-only path.
template <bool kCoherent>
__device__ __forceinline__ uint4 ld_row8(const uint16_t* p) {
  uint4 v;
  if (kCoherent)
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  else
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

template <int D, bool kE4M3, int kSteps>
__global__ void __launch_bounds__(256, kSteps == 3 ? 3 : 4) paged_append_kernel(const PagedAppendArgs a, const uint32_t segs) {
  constexpr int kLanes = D / 16, kPer = 32 / kLanes;   // lanes of a row, rows of a step
  const int lane = threadIdx.x & 31, g = lane % kLanes;
  const int rows = a.hq + 2 * a.hkv;
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(unit / segs);
  if (t >= a.b.n_tokens) return;
  const int r0 = static_cast<int>(unit - t * segs) * (kSteps * kPer) + lane / kLanes;
  uint4 x[kSteps][2];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kPer, h = r - a.hq;
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (r < a.hq) {
      const uint16_t* p = a.q + t * a.qst + r * a.qsh + g * 8;
      x[i][0] = ld_row8<true>(p);
      x[i][1] = ld_row8<true>(p + D / 2);
    } else if (r < rows) {
      const uint16_t* p = (h < a.hkv ? a.k + t * a.kst + h * a.ksh : a.v + t * a.vst + (h - a.hkv) * a.vsh) + g * 8;
      x[i][0] = ld_row8<false>(p);
      x[i][1] = ld_row8<false>(p + D / 2);
    }
  }
  const int b = find_seq(a.b, t);
  if (b < 0) return;                       // a row of no sequence: left as it is
  const int end = __ldg(a.b.cu_q + b + 1), len = __ldg(a.b.kv_len + b);
  const int64_t pos = static_cast<int64_t>(len) - end + t;
  int64_t row = pos;
  if (a.rope_cos && a.positions) row = __ldg(a.positions + t);
  int page = -1;
  if (pos >= 0 && pos < a.b.cap) page = __ldg(a.b.table + b * a.b.table_stride + (pos >> a.b.page_shift));
  const bool row_ok = !a.rope_cos || (row >= 0 && row < a.rope_rows);
  float4 cs[2], sn[2];
  cs[0] = cs[1] = sn[0] = sn[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.rope_cos && row_ok) {
    const int64_t at = row * (D / 2) + g * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      cs[k] = __ldg(reinterpret_cast<const float4*>(a.rope_cos + at + k * (D / 4)));
      sn[k] = __ldg(reinterpret_cast<const float4*>(a.rope_sin + at + k * (D / 4)));
    }
  }
  const bool placed = page >= 0 && page < a.b.n_pages && row_ok;
  if (!placed && pos >= 0 && r0 == 0)
    record_bad_index(a.status, pos >= a.b.cap ? kWhereLength : row_ok ? kWherePage : kWhereRopeRow);
  const int64_t slot = pos & ((1 << a.b.page_shift) - 1);
  uint8_t* k_at = a.k_pages + page * a.kp + slot * a.kt;
  uint8_t* v_at = a.v_pages + page * a.vp + slot * a.vt;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = r0 + i * kPer;
    const bool is_q = r < a.hq, is_v = r >= a.hq + a.hkv;
    const float* gamma = is_q ? a.gamma_q : is_v ? nullptr : a.gamma_k;
    float f[2][8];
    unpack_bf16x8(x[i][0], f[0]);
    unpack_bf16x8(x[i][1], f[1]);
    if (__any_sync(0xffffffffu, gamma != nullptr && r < rows)) {
      // sum of squares: 8 channels in order per group, groups g and g + D/16 first, then the butterfly.
      float acc[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k] = __fadd_rn(acc[k], __fmul_rn(f[k][j], f[k][j]));
      float ss = __fadd_rn(acc[0], acc[1]);
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, s));
      if (gamma) {
        const float rs = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), a.eps)));   // = fl32(1 / root)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float gm[8];
          load_gamma8(gamma, g + k * kLanes, gm);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[k][j] = __fmul_rn(__fmul_rn(f[k][j], rs), gm[j]);
        }
      }
    }
    if (r >= rows) continue;
    if (a.rope_cos && !is_v) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float cc[4] = {cs[k].x, cs[k].y, cs[k].z, cs[k].w}, sc[4] = {sn[k].x, sn[k].y, sn[k].z, sn[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y0 = f[k][2 * j], y1 = f[k][2 * j + 1];
          f[k][2 * j] = __fsub_rn(__fmul_rn(y0, cc[j]), __fmul_rn(y1, sc[j]));
          f[k][2 * j + 1] = __fadd_rn(__fmul_rn(y0, sc[j]), __fmul_rn(y1, cc[j]));
        }
      }
    }
    if (kE4M3 && !is_q) {
      if (!placed) continue;
      const int h = is_v ? r - a.hq - a.hkv : r - a.hq;
      uint8_t* dst = is_v ? v_at + h * a.vh : k_at + h * a.kh;
      const float rs = __frcp_rn(__ldg((is_v ? a.v_scale : a.k_scale) + h));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint16_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = e4m3x2(__fmul_rn(f[k][2 * j], rs), __fmul_rn(f[k][2 * j + 1], rs));
        *reinterpret_cast<uint2*>(dst + (g + k * kLanes) * 8) = make_uint2(pack_h2(w[0], w[1]), pack_h2(w[2], w[3]));
      }
      continue;
    }
    uint4 o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      o[k] = is_v ? x[i][k]
                  : make_uint4(bf16x2(f[k][0], f[k][1]), bf16x2(f[k][2], f[k][3]), bf16x2(f[k][4], f[k][5]),
                               bf16x2(f[k][6], f[k][7]));
    uint16_t* dst;
    if (is_q) {
      dst = a.q_out + t * a.ost + r * a.osh;
      if (!placed) o[0] = o[1] = make_uint4(0, 0, 0, 0);
    } else {
      if (!placed) continue;
      dst = reinterpret_cast<uint16_t*>(is_v ? v_at + (r - a.hq - a.hkv) * a.vh : k_at + (r - a.hq) * a.kh);
    }
    *reinterpret_cast<uint4*>(dst + g * 8) = o[0];
    *reinterpret_cast<uint4*>(dst + g * 8 + D / 2) = o[1];
  }
}

template <int D, bool kE4M3, int kSteps>
cudaError_t launch_steps(const PagedAppendArgs& a, cudaStream_t s) {
  constexpr int kRows = kSteps * 32 / (D / 16);
  const int64_t segs = (a.hq + 2 * a.hkv + kRows - 1) / kRows, units = segs * a.b.n_tokens;
  paged_append_kernel<D, kE4M3, kSteps><<<static_cast<unsigned>((units + 7) / 8), 256, 0, s>>>(a, static_cast<uint32_t>(segs));
  return cudaGetLastError();
}

template <int D, bool kE4M3>
cudaError_t launch_t(const PagedAppendArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  constexpr int kPer = 512 / D;                             // rows of a step
  const int64_t rows = a.hq + 2 * a.hkv;
  if (rows * a.b.n_tokens < int64_t(sms) * 24 * kPer) return launch_steps<D, kE4M3, 1>(a, s);
  const int64_t lanes2 = (rows + 2 * kPer - 1) / (2 * kPer) * 2, lanes3 = (rows + 3 * kPer - 1) / (3 * kPer) * 3;
  return lanes3 <= lanes2 + lanes2 / 8 ? launch_steps<D, kE4M3, 3>(a, s) : launch_steps<D, kE4M3, 2>(a, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int d, bool e4m3, cudaStream_t s) {
  if (d == 128) return e4m3 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
  return e4m3 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace sage
