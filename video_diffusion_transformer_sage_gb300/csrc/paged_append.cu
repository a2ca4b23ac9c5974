// paged_append.cu -- new tokens into the paged K/V cache: RMSNorm and rotation of Q and K rows (the
// row arithmetic of qk_row.cuh), K and V stored to their pages as bf16 or E4M3 codes.
//
// A warp takes up to 4 kSteps heads (8 kSteps at D = 64) of one token, all of Q, of K or of V, so what a row needs is the
// same for all its lanes.  D/16 lanes hold a row, each the 8-channel groups g and g + D/16, which are the first two that
// the row's sum of squares adds: the fold over the lanes is then the same butterfly as with a lane per group, and the
// root, the division and the address of a row are paid by half as many threads.  Products go two to an
// instruction.  The rows are loaded first; the chain cu_q -> kv_len -> page table -> rotary row hides under them.  Warps do
// not wait for one another.
//
// What bounds it: HBM for many tokens, each row read once and written once, with about as much issue time: 5.42 TB/s at
// 3024 tokens of 168 rows of D = 128 (48.2 us), 4.31 TB/s at 11927 tokens of 72 rows of D = 64 into E4M3 (43.2 us); for few
// tokens the chain of dependent loads.  A warp takes two steps of heads where the batch fills the GPU (one: 56.0 and
// 52.1 us), three where that leaves fewer lanes idle (24 heads of D = 64: 51.6 us with two), one where spreading the rows
// over more SMs shortens the chain.
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

// Segments (runs of kSteps * kPer heads, one warp each) of a token's Q, and of its K or V.
struct AppendSegs {
  uint32_t q, kv;
};

template <int D, bool kE4M3, int kSteps>
__global__ void __launch_bounds__(256, kSteps == 1 ? 5 : 4) paged_append_kernel(const PagedAppendArgs a, const AppendSegs segs) {
  constexpr int kLanes = D / 16, kPer = 32 / kLanes;   // lanes of a row, rows of a step
  const int lane = threadIdx.x & 31, g = lane % kLanes;
  // The warp's number by shuffle: token, segment and their addresses are then computed once per warp, not per lane
  // (append_frames 49.8 -> 48.2 us, append_ragged_e4m3 45.4 -> 43.2).
  const uint32_t unit = blockIdx.x * 8 + __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), per_token = segs.q + 2 * segs.kv;
  const int t = static_cast<int>(unit / per_token);
  if (t >= a.b.n_tokens) return;
  uint32_t seg = unit - t * per_token;
  const bool first = seg == 0;
  // What the warp's rows are: all Q, all K or all V.
  const bool is_q = seg < segs.q, is_v = seg >= segs.q + segs.kv;
  seg -= is_q ? 0u : is_v ? segs.q + segs.kv : segs.q;
  const int heads = is_q ? a.hq : a.hkv;
  const int64_t sh = is_q ? a.qsh : is_v ? a.vsh : a.ksh;
  const int h0 = static_cast<int>(seg) * (kSteps * kPer) + lane / kLanes;
  const uint16_t* src = (is_q ? a.q + t * a.qst : is_v ? a.v + t * a.vst : a.k + t * a.kst) + h0 * sh + g * 8;
  uint4 x[kSteps][2];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
    if (h0 + i * kPer < heads) {
      const uint16_t* p = src + i * kPer * sh;
      if (is_q) {
        x[i][0] = ld_row8<true>(p);
        x[i][1] = ld_row8<true>(p + D / 2);
      } else {
        x[i][0] = ld_row8<false>(p);
        x[i][1] = ld_row8<false>(p + D / 2);
      }
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
  const bool placed = page >= 0 && page < a.b.n_pages && row_ok;
  if (!placed && pos >= 0 && first && lane == 0)
    record_bad_index(a.status, pos >= a.b.cap ? kWhereLength : row_ok ? kWherePage : kWhereRopeRow);
  if (!placed) {
    // Nothing stored; a Q row becomes 0.
    if (is_q) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        uint16_t* dst = a.q_out + t * a.ost + (h0 + i * kPer) * a.osh + g * 8;
        if (h0 + i * kPer < heads) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + D / 2) = make_uint4(0, 0, 0, 0);
        }
      }
    }
    return;
  }
  const int64_t slot = pos & ((1 << a.b.page_shift) - 1);
  // Row h goes to dst + h * dh (bytes).
  uint8_t* dst = is_q ? reinterpret_cast<uint8_t*>(a.q_out + t * a.ost)
                 : is_v ? a.v_pages + page * a.vp + slot * a.vt : a.k_pages + page * a.kp + slot * a.kt;
  const int64_t dh = is_q ? a.osh * 2 : is_v ? a.vh : a.kh;
  dst += h0 * dh;
  if (is_v && !kE4M3) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (h0 + i * kPer < heads) {
        uint16_t* o = reinterpret_cast<uint16_t*>(dst + i * kPer * dh) + g * 8;
        *reinterpret_cast<uint4*>(o) = x[i][0];
        *reinterpret_cast<uint4*>(o + D / 2) = x[i][1];
      }
    }
    return;
  }
  const float* gamma = is_q ? a.gamma_q : is_v ? nullptr : a.gamma_k;
  const bool turn = a.rope_cos && !is_v;
  float4 cs[2], sn[2];
  cs[0] = cs[1] = sn[0] = sn[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn) {
    const int64_t at = row * (D / 2) + g * 4;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      cs[k] = __ldg(reinterpret_cast<const float4*>(a.rope_cos + at + k * (D / 4)));
      sn[k] = __ldg(reinterpret_cast<const float4*>(a.rope_sin + at + k * (D / 4)));
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    // The 16 channels as pairs (2 j, 2 j + 1): a packed multiply is two separately rounded products.  Sums stay scalar.
    uint64_t f[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w[4] = {x[i][k].x, x[i][k].y, x[i][k].z, x[i][k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) f[k][j] = f2_pack(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
    }
    if (gamma) {
      // Sum of squares: 8 channels in order per group, groups g and g + D/16 first, then the butterfly.
      float acc[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        acc[k] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          f2_unpack(f2_mul(f[k][j], f[k][j]), lo, hi);
          acc[k] = __fadd_rn(__fadd_rn(acc[k], lo), hi);
        }
      }
      float ss = __fadd_rn(acc[0], acc[1]);
#pragma unroll
      for (int s = kLanes / 2; s > 0; s >>= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, s));
      const float rs = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), a.eps)));   // = fl32(1 / root)
      const uint64_t rs2 = f2_pack(rs, rs);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float gm[8];
        load_gamma8(gamma, g + k * kLanes, gm);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[k][j] = f2_mul(f2_mul(f[k][j], rs2), f2_pack(gm[2 * j], gm[2 * j + 1]));
      }
    }
    if (turn) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float cc[4] = {cs[k].x, cs[k].y, cs[k].z, cs[k].w}, sc[4] = {sn[k].x, sn[k].y, sn[k].z, sn[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float y0c, y1c, y0s, y1s;
          f2_unpack(f2_mul(f[k][j], f2_pack(cc[j], cc[j])), y0c, y1c);
          f2_unpack(f2_mul(f[k][j], f2_pack(sc[j], sc[j])), y0s, y1s);
          f[k][j] = f2_pack(__fsub_rn(y0c, y1s), __fadd_rn(y0s, y1c));
        }
      }
    }
    if (h0 + i * kPer >= heads) continue;
    uint8_t* out = dst + i * kPer * dh;
    if (kE4M3 && !is_q) {
      const float rs = __frcp_rn(__ldg((is_v ? a.v_scale : a.k_scale) + h0 + i * kPer));
      const uint64_t rs2 = f2_pack(rs, rs);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint16_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          f2_unpack(f2_mul(f[k][j], rs2), lo, hi);
          w[j] = e4m3x2(lo, hi);
        }
        *reinterpret_cast<uint2*>(out + (g + k * kLanes) * 8) = make_uint2(pack_h2(w[0], w[1]), pack_h2(w[2], w[3]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          f2_unpack(f[k][j], lo, hi);
          w[j] = bf16x2(lo, hi);
        }
        *reinterpret_cast<uint4*>(out + (g + k * kLanes) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

template <int D, bool kE4M3, int kSteps>
cudaError_t launch_steps(const PagedAppendArgs& a, cudaStream_t s) {
  constexpr uint32_t kRows = kSteps * 512 / D;
  const AppendSegs segs{(a.hq + kRows - 1) / kRows, (a.hkv + kRows - 1) / kRows};
  const int64_t units = static_cast<int64_t>(segs.q + 2 * segs.kv) * a.b.n_tokens;
  paged_append_kernel<D, kE4M3, kSteps><<<static_cast<unsigned>((units + 7) / 8), 256, 0, s>>>(a, segs);
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
  if (rows * a.b.n_tokens < int64_t(sms) * 32 * kPer) return launch_steps<D, kE4M3, 1>(a, s);
  // The rows that the warps' runs cover, idle ones included.
  auto covered = [&](int steps) {
    const int64_t run = int64_t(steps) * kPer;
    return (a.hq + run - 1) / run * run + 2 * ((a.hkv + run - 1) / run * run);
  };
  return covered(3) < covered(2) ? launch_steps<D, kE4M3, 3>(a, s) : launch_steps<D, kE4M3, 2>(a, s);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int d, bool e4m3, cudaStream_t s) {
  if (d == 128) return e4m3 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
  return e4m3 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
}

}  // namespace sage
