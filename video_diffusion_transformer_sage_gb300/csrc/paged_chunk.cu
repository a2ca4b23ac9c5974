// paged_chunk.cu -- attention of many query rows per K/V head over the paged cache (prompts, chunks of
// a video) on the 5th-generation tensor cores.
//
// A unit is (sequence, K/V head, 256 query rows): the rows of a K/V head are the sequence's new tokens
// times the query heads that share it, so grouped heads fill the 128-row tiles and every K and V
// tile that is loaded serves all of them.  Two 128-row tiles t = 0, 1 per unit and 128-key tiles:
//   S_t = Q_t K^T    tcgen05.mma 128 x 128 x 16, fp32 in tensor memory
//   online softmax   one thread per row: fp32 maximum and sum; P_t in 16 bits over S_t's columns
//                    (its own columns at D = 64)
//   O_t += P_t V     A from tensor memory, B = V as it lies in the cache, keys by channels: the
//                    MN-major operand of the 128-byte swizzle, so V is never transposed
// as in attn_fwd.cu (Q tiles in turn, so one tile's softmax overlaps the other's MMAs).  A unit of at most 128
// rows has one Q tile; its key tiles then go to the two slots t in turn, each with a maximum, sum and O of its
// own, joined at the end: the same overlap, and half the steps.  O is rescaled only
// when a row's maximum rises by more than 2^8 (P then stays below 2^8, or 2^15 where it is lifted for fp16, inside
// both 16-bit types and fp32): the result is the same ratio, and most tiles rescale nothing.
//
// bf16 cache: bf16 operands, one TMA box per page and 64 channels, straight into the swizzled tiles.
// E4M3 cache: the codes come by TMA into a staging tile and one warpgroup widens them to fp16 (exact) in
// the swizzled tiles; Q is held as fp16 times a power of two per row and P as fp16.
//
// One CTA per SM works through the items (units, or shares of a unit's keys), drawn from a counter; the pipeline does
// not drain between them: the next unit's Q, K and V are loaded and its first S formed while O of the last one leaves.
// Against a CTA per item, whose start and end take 7.6 us of a unit: prompts_causal 371 -> 345 us, window_e4m3
// 180 -> 168, 2048 rows over 16384 bf16 keys of 16 heads 207 -> 201; a call of one short unit per SM takes 0.8 us
// more (13.2 -> 14.0).
//
// Warp roles: warp 0 (and 3) page table and TMA, warp 1 MMA issue, warp 2 draws the items and finds their
// units; warps 4-7 and 8-11 softmax and epilogue of tile 0 and 1; with E4M3 warps 12-15 widen.  Every wait is bounded.
//
// What bounds it: 4 rows keys D FLOPs at the 16-bit tensor rate (for few rows the cache's bytes), and the softmax warps,
// which take about as long: D = 64 has half the FLOPs for the same exponentials.  The key axis is split over several
// items for the units that do not fill the SMs a last time; each then leaves (maximum, sum, O) in the workspace, and paged_join_kernel adds the parts in the order of their keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "paged_batch.cuh"
#include "tensor_map.h"

namespace sage {
namespace {

constexpr int kBM = 128, kBN = 128;
constexpr uint64_t kChunkWaitNs = 2000000000ull;
constexpr int kItemWaits = 64;   // such waits for all of an item's key tiles
constexpr float kRise = 8.0f;   // log2 of how far a maximum may fall behind before O is rescaled

template <int D, bool kE4M3>
struct ChunkCfg {
  static constexpr int kThreads = kE4M3 ? 512 : 384;
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;               // 128 rows of 64 channels
  static constexpr int kQTileBytes = kBM * D * 2;
  static constexpr int kTileBytes = kBN * D * 2;              // a K or V tile in 16 bits
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;
  // K and V of a tile have barriers of their own where the ring is short (D = 128): a K stage is free again once
  // Q K^T has read it, a softmax before P V is done with V (chunk_frames 2358 -> 2236 us).  The four stages at
  // D = 64 hide the loads anyway, and there the extra waits of the issuing warp cost 3 %.
  static constexpr bool kSplitKV = D == 128;
  static constexpr int kRawTile = kBN * D;                    // a tile of codes
  static constexpr int kRawBytes = kE4M3 ? 2 * kRawTile : 0;
  // Tensor memory columns: S_t at 128 t, O_t at 256 + D t; P_t over S_t, or at 384 + 64 t (D = 64).
  static constexpr int kColO0 = 256;
  static constexpr bool kSepP = D == 64;
  static constexpr int kColP0 = kSepP ? 384 : 0, kStepP = kSepP ? 64 : 128;
  // K and V with barriers of their own, and the two staging tiles, have a loading warp each: pages of 16 tokens are 32
  // copies a tile.
  static constexpr bool kTwoLoaders = kSplitKV || kE4M3;
  // Results leave through 16 KB of shared memory per slot while the next unit's Q is loaded; with E4M3 at D = 128 there
  // is no room for both, and they leave through the slot's Q tile first.
  static constexpr bool kEarlyQ = !(kE4M3 && D == 128);
  static constexpr int kKvOff = 2 * kQTileBytes;
  static constexpr int kRawOff = kKvOff + kStages * kStageBytes;
  static constexpr int kOutOff = kRawOff + kRawBytes;
  static constexpr int kExpOff = kOutOff + (kEarlyQ ? 2 * 16384 : 0);   // biased exponent of each Q row (E4M3)
  static constexpr int kBarOff = kExpOff + (kE4M3 ? 256 : 0);
  // q_full[2], k_full[S], v_full[S], k_empty[S], v_empty[S], s_full[2], p_full[2], pv_done[2], s_free[2], o_free[2],
  // ml_full, ml_empty, mma_final, raw_full[2] (K, V), raw_empty[2], unit_full[2], unit_empty[2], draw
  static constexpr int kNumBars = 4 * kStages + 24;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + 16 + 1024;
  // Registers a thread: launched at 168 (384 threads) or 128 (512).
  static constexpr int kRegsRoles = 72, kRegsSoftmax = kE4M3 ? 184 : 216, kRegsWiden = 72;
  static_assert(128 * kRegsRoles + 256 * kRegsSoftmax + (kE4M3 ? 128 * kRegsWiden : 0) <= (kE4M3 ? 512 * 128 : 384 * 168),
                "register split exceeds launch");
  static_assert(kSmem <= 232448 - 1408, "shared memory");
};

struct ChunkParams {
  PagedAttnArgs a;
  int group;
  int box_shift;   // log2 of the slots per TMA box (a page, or 128)
  int whole;       // units below this number are one item; each of the rest is `splits` items
  int splits;
  int halve;       // units of one row tile are split half as often
  uint32_t items;
};

__device__ __forceinline__ void give_up(int32_t* status, int32_t where, volatile int* abort_flag) {
  record_timeout(status, where);
  *abort_flag = 1;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kChunkWaitNs));
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// One unit's work; the same for every thread of a CTA.
struct Unit {
  int b, h;
  int start, n_new, len;    // first row of q, new tokens, tokens in the cache
  int row0, rows;           // first row (token x group) of the unit, rows it has (at most 256)
  int t0, nt;               // its key tiles (the item's share of them); nt < 0: no more items
  int ulo, uhi;             // keys that some row sees
  int slot;                 // of its partial result; -1: the unit is one item
  // For the softmax: keys that every row of tile t sees; this CTA's key tiles, slot t's and units of one row tile so far.
  int alo[2], ahi[2];
  uint32_t ct, mine[2], ones;
};

__device__ __forceinline__ void token_keys(const PagedAttnArgs& a, int len, int n_new, int j, int& lo, int& hi) {
  const int pos = len - n_new + j;
  hi = a.causal ? max(0, pos + 1) : len;
  lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
}

// Unit number `index` of the call, found by one warp; false past the last.  Units of a sequence and head
// lie together (they share K and V in L2), the later rows (more keys when causal) first.
__device__ __forceinline__ bool find_unit(const PagedAttnArgs& a, int group, int index, Unit& u) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int b0 = 0; b0 < a.b.n_seqs; b0 += 32) {
    int blocks = 0, seq = b0 + lane;
    if (seq < a.b.n_seqs) {
      int s, e;
      seq_rows(a.b, seq, s, e);
      blocks = ((e - s) * group + 255) / 256;
    }
    if (a.b.n_seqs > 1) {
      // Among these 32, the longest sequences' units come first: the short ones fill the last wave.
      const int n = min(32, a.b.n_seqs - b0);
      const int len = lane < n ? __ldg(a.b.kv_len + seq) : INT32_MIN;
      int rank = 0, from = lane;
      for (int k = 0; k < n; ++k) {
        const int x = __shfl_sync(0xffffffffu, len, k);
        rank += x > len || (x == len && k < lane);
      }
      for (int k = 0; k < n; ++k)
        if (__shfl_sync(0xffffffffu, rank, k) == lane) from = k;
      blocks = __shfl_sync(0xffffffffu, blocks, from);
      seq = b0 + from;
    }
    int incl = blocks * a.hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, base + incl > index);
    if (past) {
      const int l = __ffs(past) - 1;
      const int nb = __shfl_sync(0xffffffffu, blocks, l);
      const int off = index - base - (__shfl_sync(0xffffffffu, incl, l) - nb * a.hkv);
      int e;
      u.b = __shfl_sync(0xffffffffu, seq, l);
      seq_rows(a.b, u.b, u.start, e);
      u.n_new = e - u.start;
      u.len = min(max(__ldg(a.b.kv_len + u.b), 0), a.b.cap);
      u.h = off / nb;
      u.row0 = (nb - 1 - off % nb) * 256;
      u.rows = min(256, u.n_new * group - u.row0);
      int unused;
      token_keys(a, u.len, u.n_new, u.row0 / group, u.ulo, unused);
      token_keys(a, u.len, u.n_new, (u.row0 + u.rows - 1) / group, unused, u.uhi);
      u.t0 = u.ulo / kBN;
      u.nt = max(1, (u.uhi + kBN - 1) / kBN - u.t0);
      return true;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// Max of 64 consecutive fp32 values (as bits): four independent chains of 3-input maxima.
__device__ __forceinline__ float max64(const uint32_t* s) {
  auto f = [s](int i) { return __uint_as_float(s[i]); };
  float a = fmax3(f(0), f(1), f(2)), b = fmax3(f(3), f(4), f(5));
  float c = fmax3(f(6), f(7), f(8)), d = fmax3(f(9), f(10), f(11));
#pragma unroll
  for (int k = 12; k < 60; k += 8) {
    a = fmax3(a, f(k), f(k + 1));
    b = fmax3(b, f(k + 2), f(k + 3));
    c = fmax3(c, f(k + 4), f(k + 5));
    d = fmax3(d, f(k + 6), f(k + 7));
  }
  a = fmax3(a, f(60), f(61));
  b = fmax3(b, f(62), f(63));
  return fmaxf(fmax3(a, b, c), d);
}

// Instruction descriptor bits: bf16 operands (fp16 is 0), B MN-major.
constexpr uint32_t kIdescBf16 = (1u << 7) | (1u << 10), kIdescBmn = 1u << 16;
// Low descriptor word of a V tile as MN-major B: rows of 64 channels (128 bytes), 8-key groups 1024 bytes
// apart (the stride offset of kSdescHi), the next 64 channels a panel further (leading offset).
__device__ __forceinline__ uint32_t vdesc_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((128u * 128u >> 4) << 16);
}

// MMA and commit on behalf of a converged warp: one thread of it, always the same, issues.  The whole warp computes the
// operands, which are the same in all lanes and known to be so (the warp's number, shared-memory base, tile counts
// come by shuffle), so they need not be moved to uniform registers for each MMA: one lane's code spent ~93 cycles on
// each, this ~35 (D = 64, 2048 rows over 16384 bf16 keys of 16 heads 168 -> 149 us; prompts_causal 345 -> 329).
__device__ __forceinline__ void warp_mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_tc_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}

template <int D, bool kE4M3>
__device__ __forceinline__ void issue_qk(uint32_t s_tmem, uint32_t ql, uint32_t kl) {
  constexpr uint32_t idesc = idesc_f32acc(kBM, kBN) | (kE4M3 ? 0u : kIdescBf16);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * ChunkCfg<D, kE4M3>::kPanelBytes + (kk & 3) * 32) >> 4;
    warp_mma_f16_ss(s_tmem, sdesc_of_lo(ql + off), sdesc_of_lo(kl + off), idesc, kk > 0 ? 1u : 0u);
  }
}
// P: 16 keys in 8 tensor-memory columns; V: 16 keys are 2048 bytes.
template <int D, bool kE4M3>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t vl, bool first) {
  constexpr uint32_t idesc = idesc_f32acc(kBM, D) | kIdescBmn | (kE4M3 ? 0u : kIdescBf16);
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk)
    warp_mma_f16_ts(o_tmem, p_tmem + kk * 8, sdesc_of_lo(vl + kk * (2048 >> 4)), idesc, (first && kk == 0) ? 0u : 1u);
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  if (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Bit k of word w: key 32 w + k of the tile lies in [lo, hi) and its box was loaded.
__device__ __forceinline__ uint32_t key_mask(int w, int lo, int hi, uint32_t bits, int box_shift) {
  const int l = max(lo - 32 * w, 0), h = min(hi - 32 * w, 32);
  if (l >= h) return 0u;
  uint32_t m = (h == 32 ? ~0u : (1u << h) - 1u) & ~((1u << l) - 1u);
  if (box_shift >= 5) {
    if (!((bits >> ((32 * w) >> box_shift)) & 1u)) m = 0u;
  } else {
    const int box = 1 << box_shift;
    for (int k = 0; k < 32; k += box)
      if (!((bits >> ((32 * w + k) >> box_shift)) & 1u)) m &= ~(((1u << box) - 1u) << k);
  }
  return m;
}

// One 128-key tile of the online softmax for the calling thread's row (= tensor-memory lane): S is read,
// masked where `masked`, its maximum taken; P = 2^(S c - m) is written in 16 bits, l the sum of the unrounded P; O is
// multiplied by 2^(m_old - m) where the maximum rose by more than kRise.  With separate P columns S is
// released as soon as it is in registers and P waits for the P.V of the tile before (pv_done).
template <int D, bool kE4M3, typename Mask>
__device__ __forceinline__ bool softmax_step(uint32_t tS, uint32_t tO, uint32_t tP, float c, bool masked, Mask&& make_mask,
                                             bool first, float& m, float& l, uint64_t* s_free, uint64_t* pv_done, int j) {
  constexpr bool kSep = ChunkCfg<D, kE4M3>::kSepP;
  uint32_t sr[128];
  SAGE_TMEM_LD32(tS + 0, (sr + 0));
  SAGE_TMEM_LD32(tS + 32, (sr + 32));
  SAGE_TMEM_LD32(tS + 64, (sr + 64));
  SAGE_TMEM_LD32(tS + 96, (sr + 96));
  tmem_wait_ld();
  if (kSep) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(s_free);
  }
  if (masked) {
    uint32_t mask[4];
    make_mask(mask);
#pragma unroll
    for (int k = 0; k < 128; ++k)
      if (!((mask[k >> 5] >> (k & 31)) & 1u)) sr[k] = 0xFF800000u;   // -infinity
  }
  constexpr float kLift = kE4M3 ? kLiftE4M3 : 0.0f;
  const float mx = fmaxf(max64(sr), max64(sr + 64)) * c, lower = mx - kLift;
  const bool up = mx > m + (kRise + kLift);   // also the first visible key: m is -infinity before it
  const float alpha = (up && !first) ? ex2_approx(m - lower) : 1.0f;
  const bool rise = up && !first;
  if (up) m = lower;
  const float base = m == -INFINITY ? 0.0f : m;   // no key so far: every P below is 0
  const uint64_t bias2 = f2_pack(-base, -base), c2 = f2_pack(c, c);
  uint64_t l2[4][2];
  uint32_t pkeep[kSep ? 64 : 1];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t pw[16];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int k = q * 32 + w * 4;
      float p[4];
      f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), c2, bias2), p[0], p[1]);
      f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[k + 2]), __uint_as_float(sr[k + 3])), c2, bias2), p[2], p[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2_approx(p[i]);
      if (w == 0) {
        l2[q][0] = f2_pack(p[0], p[1]);
        l2[q][1] = f2_pack(p[2], p[3]);
      } else {
        l2[q][0] = f2_add(l2[q][0], f2_pack(p[0], p[1]));
        l2[q][1] = f2_add(l2[q][1], f2_pack(p[2], p[3]));
      }
      pw[2 * w] = pack2<kE4M3>(p[0], p[1]);
      pw[2 * w + 1] = pack2<kE4M3>(p[2], p[3]);
    }
    if (kSep) {
#pragma unroll
      for (int i = 0; i < 16; ++i) pkeep[q * 16 + i] = pw[i];
    } else {
      SAGE_TMEM_ST16(tS + q * 16, pw);
    }
  }
  float x, y;
  f2_unpack(f2_add(f2_add(f2_add(l2[0][0], l2[0][1]), f2_add(l2[1][0], l2[1][1])),
                   f2_add(f2_add(l2[2][0], l2[2][1]), f2_add(l2[3][0], l2[3][1]))), x, y);
  l = l * alpha + (x + y);
  if (kSep) {
    if (!first) {
      if (!warp_wait(pv_done, (j - 1) & 1)) return false;
      tc_fence_after();
    }
    SAGE_TMEM_ST32(tP, pkeep);
    SAGE_TMEM_ST32(tP + 32, (pkeep + 32));
  }
  if (__any_sync(0xffffffffu, rise)) {
    const uint64_t a2 = f2_pack(alpha, alpha);
    uint32_t o[D];
#pragma unroll
    for (int i = 0; i < D; i += 32) SAGE_TMEM_LD32(tO + i, (o + i));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < D; i += 2) {
      float lo, hi;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), lo, hi);
      o[i] = __float_as_uint(lo);
      o[i + 1] = __float_as_uint(hi);
    }
#pragma unroll
    for (int i = 0; i < D; i += 32) SAGE_TMEM_ST32(tO + i, (o + i));
  }
  tmem_wait_st();
  return true;
}

// What the roles of a CTA share.
struct ChunkShared {
  Unit unit[2];                    // the items in work and next
  int skip;
  volatile int abort;
  uint32_t bits[8], raw_bits[2];   // boxes loaded: of the last key tiles, and of the staging K and V tile
  uint32_t tmem;
  float2 ml[128];                  // slot 1's maxima and sums (units of one row tile)
};

template <int T>
struct Slot {   // a row tile's number, as a constant
  static constexpr int v = T;
};

template <int D, bool kE4M3>
__global__ void __launch_bounds__(ChunkCfg<D, kE4M3>::kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ ChunkParams p) {
  using C = ChunkCfg<D, kE4M3>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ChunkShared sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::kKvOff;
  uint8_t* q_exp = smem + C::kExpOff;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* k_full = q_full + 2;
  uint64_t* v_full = k_full + S;
  uint64_t* k_empty = v_full + S;
  uint64_t* v_empty = k_empty + S;
  uint64_t* s_full = v_empty + S;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* s_free = pv_done + 2;
  uint64_t* o_free = s_free + 2;
  uint64_t* ml_full = o_free + 2;
  uint64_t* ml_empty = ml_full + 1;
  uint64_t* mma_final = ml_empty + 1;
  uint64_t* raw_full = mma_final + 1;
  uint64_t* raw_empty = raw_full + 2;
  uint64_t* unit_full = raw_empty + 2;
  uint64_t* unit_empty = unit_full + 2;
  uint64_t* draw = unit_empty + 2;
  const PagedAttnArgs& a = p.a;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    sh.skip = *reinterpret_cast<volatile int32_t*>(a.status) == kStatusTimeout;
    sh.abort = 0;
    for (int i = 0; i < 2 * S; ++i) mbar_init(k_full + i, kE4M3 ? 128 : 1);        // and v_full
    for (int i = 0; i < 2 * S; ++i) mbar_init(k_empty + i, 1);                     // and v_empty
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 128);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(pv_done + i, 1);
      mbar_init(s_free + i, 4);
      mbar_init(o_free + i, 128);
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, 128);
      mbar_init(unit_full + i, 1);
      // The loading warps, the issuing warp, the softmax and the widening warps.
      mbar_init(unit_empty + i, (C::kTwoLoaders ? 2 : 1) + 1 + 8 + (kE4M3 ? 4 : 0));
    }
    mbar_init(ml_full, 128);
    mbar_init(ml_empty, 128);
    mbar_init(mma_final, 1);
    mbar_init(draw, 1);
    fence_mbar_init();
  }
  // Warp 2 finds an item's unit and its share of the unit's key tiles (which may be empty when there are few).
  // False past the last unit, of which the number of items is an upper bound: no later item has one either.
  auto take = [&](uint32_t item, Unit& u, bool& have) {
    have = false;
    const bool split = item >= static_cast<uint32_t>(p.whole);
    const int rest = static_cast<int>(item) - p.whole;
    if (!find_unit(a, p.group, split ? p.whole + rest / p.splits : static_cast<int>(item), u)) return false;
    if (lane == 0 && __ldg(a.b.kv_len + u.b) > a.b.cap) record_bad_index(a.status, kWhereLength);
    u.slot = -1;
    if (split) {
      // A unit of one row tile takes half as long: among others it has half as many shares that are not empty.
      const int parts = p.halve && u.rows <= 128 ? (p.splits + 1) / 2 : p.splits;
      const int per = (u.nt + parts - 1) / parts, from = min(u.nt, per * (rest % p.splits));
      u.t0 += from;
      u.nt = min(per, u.nt - from);
      u.slot = rest;
    }
    if (u.nt > 0) {
      for (int t = 0; t < 2; ++t) {
        int unused;
        const int from = u.rows > 128 ? t * 128 : 0, last = min(u.rows, from + 128) - 1;
        token_keys(a, u.len, u.n_new, (u.row0 + from) / p.group, unused, u.ahi[t]);
        token_keys(a, u.len, u.n_new, (u.row0 + last) / p.group, u.alo[t], unused);
      }
      have = true;
      return true;
    }
    for (int r = lane; r < u.rows; r += 32) a.part_ml[u.slot * kPagedChunkRows + r] = make_float2(-INFINITY, 0.0f);
    return true;
  };
  Unit u{};
  bool have = false, end = false, first = true;
  // Item k for the other roles, with the CTA's counts up to it.
  auto publish = [&](int k) {
    if (end) u.nt = -1;
    if (lane == 0) {
      sh.unit[k & 1] = u;
      mbar_arrive(unit_full + (k & 1));
    }
    __syncwarp();
    u.ct += u.nt;
    u.ones += u.rows <= 128;
    for (int t = 0; t < 2; ++t) u.mine[t] += u.rows > 128 ? u.nt : (u.nt + 1 - t) / 2;
  };
  if (warp == 2) end = !take(blockIdx.x, u, have);
  __syncthreads();
  if (sh.skip) return;   // an earlier wait ran out: no work until the status has been read
  if (warp == 2 && (have || end)) publish(0);
  if (warp == 3) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem, 0);
  const int boxes = kBN >> p.box_shift;
  // A bounded wait by a whole warp; records the first timeout.  False once anything timed out.
  auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
    if (warp_wait(bar, parity)) return true;
    if (lane == 0) give_up(a.status, where, &sh.abort);
    __syncwarp();
    return false;
  };
  // Item k's entry has been copied by the whole warp and may be replaced.
  auto release_unit = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(unit_empty + (k & 1));
  };

  if (warp < 4) {
    regs_dec<C::kRegsRoles>();
    if (warp == 2) {
      // ------------------------------------------------------------ items, one ahead
      int32_t* next_item = a.counters + 2 * kPagedMaxCtas;   // and the number of CTAs that draw no more
      uint32_t item = 0;
      for (int k = have || end ? 1 : 0;;) {
        if (!first) {
          end = item >= p.items || !take(item, u, have);
          if (have || end) {
            if (k >= 2 && !wait(unit_empty + (k & 1), ((k >> 1) - 1) & 1, kWherePagedEmpty)) break;
            publish(k++);
          }
        }
        first = false;
        if (end || __any_sync(0xffffffffu, sh.abort)) break;
        // The next item is drawn when the loads of this one are about to end: late enough that a CTA with a long item
        // holds no other, early enough that finding the unit costs no time.
        if (p.items <= gridDim.x) {
          item = p.items;
          continue;
        }
        if (have) {
          bool ready = false;
          for (int n = 0; n < kItemWaits && !ready && !sh.abort; ++n) ready = warp_wait(draw, (k - 1) & 1);
          if (!ready) {
            if (lane == 0) give_up(a.status, kWherePagedEmpty, &sh.abort);
            __syncwarp();
            break;
          }
        }
        uint32_t drawn = 0;
        if (lane == 0) drawn = static_cast<uint32_t>(atomicAdd(next_item, 1));
        item = gridDim.x + __shfl_sync(0xffffffffu, drawn, 0);
      }
      // The last CTA to draw no more leaves the counters at zero for the next call.
      if (end && p.items > gridDim.x && lane == 0 && atomicAdd(next_item + 1, 1) == static_cast<int>(gridDim.x) - 1)
        next_item[0] = next_item[1] = 0;
    } else if (warp == 0 || (C::kTwoLoaders && warp == 3)) {
      // ------------------------------------------------------------ page table and TMA
      const int kv0 = warp == 0 ? 0 : 1, kv1 = C::kTwoLoaders && warp == 0 ? 1 : 2;   // K, V or both
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
      const int box = 1 << p.box_shift;
      const uint32_t box_bytes = static_cast<uint32_t>(box) * D * (kE4M3 ? 1 : 2);
      uint32_t ct = 0, issued = 0;   // tiles so far; those whose copies were issued (of K, or of this warp's)
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = wait(unit_full + (k & 1), (k >> 1) & 1, kWherePagedEmpty);
        if (!ok) break;
        const Unit& e = sh.unit[k & 1];
        const int ntiles = e.nt, h = e.h, ulo = e.ulo, uhi = e.uhi, key00 = e.t0 * kBN + (lane << p.box_shift);
        const int32_t* row = a.b.table + e.b * a.b.table_stride;
        release_unit(k);
        if (ntiles < 0) break;
        for (int j = 0; j < ntiles && ok; ++j, ++ct) {
          const int key0 = key00 + j * kBN;
          if (warp == 0 && lane == 0 && j == max(0, ntiles - 3)) mbar_arrive(draw);
          const bool need = lane < boxes && key0 < uhi && key0 + box > ulo;
          int page = -1;
          if (need) page = __ldg(row + (key0 >> a.b.page_shift));
          const bool good = need && page >= 0 && page < a.b.n_pages;
          if (need && !good) record_bad_index(a.status, kWherePage);
          const uint32_t bits = __ballot_sync(0xffffffffu, good);
          const int slot_in_page = key0 & ((1 << a.b.page_shift) - 1);
          const uint32_t s = ct % S;
          for (int kv = kv0; kv < kv1; ++kv) {
            const CUtensorMap* map = kv ? &vmap : &kmap;
            const bool own_bar = C::kSplitKV || kv == 0;   // V shares K's barriers otherwise
            uint64_t* full = kE4M3 ? raw_full + kv : (kv && own_bar ? v_full : k_full) + s;
            if (kE4M3) {
              if (ct >= 1) ok = wait(raw_empty + kv, (ct - 1) & 1, kWherePagedEmpty);
            } else if (own_bar && ct >= S) {
              ok = wait((kv || !C::kSplitKV ? v_empty : k_empty) + s, (ct / S - 1) & 1, kWherePagedEmpty);
            }
            ok = !__any_sync(0xffffffffu, !ok || sh.abort);
            if (!ok) break;
            if (lane == 0) {
              if (kE4M3) sh.raw_bits[kv] = bits;
              else if (kv == 0) sh.bits[ct % (2 * S)] = bits;
              if (kE4M3 || own_bar)
                mbar_arrive_expect_tx(full, __popc(bits) * box_bytes * (kE4M3 || C::kSplitKV ? 1u : 2u));
            }
            __syncwarp();
            if (good) {
              if (kE4M3) {
                tma_load_4d(smem_u32(smem + C::kRawOff) + kv * C::kRawTile + (lane << p.box_shift) * D, map, full, 0, h,
                            slot_in_page, page);
              } else {
                const uint32_t dst = smem_u32(sKV + s * C::kStageBytes) + kv * C::kTileBytes + (lane << p.box_shift) * 128;
#pragma unroll
                for (int pn = 0; pn < C::kPanels; ++pn)
                  tma_load_4d(dst + pn * C::kPanelBytes, map, full, pn * 64, h, slot_in_page, page);
              }
            }
            issued = ct + 1;
          }
        }
      }
      if (!ok) {
        // After a timeout: the copies issued have landed before the CTA ends.
        if (kE4M3) {
          if (issued > 0) mbar_wait(raw_full + kv0, (issued - 1) & 1, kChunkWaitNs);
        } else {
          for (uint32_t i = issued > S ? issued - S : 0; i < issued; ++i)
            mbar_wait((kv0 ? v_full : k_full) + i % S, (i / S) & 1, kChunkWaitNs);
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issue
      const uint32_t colS = tmem, colO = tmem + C::kColO0, colP = tmem + C::kColP0;
      const uint32_t s_base = __shfl_sync(0xffffffffu, smem_u32(sQ), 0);
      const uint32_t q_lo = sdesc_lo(s_base), k_lo = sdesc_lo(s_base + C::kKvOff),
                     v_lo = vdesc_lo(s_base + C::kKvOff + C::kTileBytes);
      constexpr uint32_t kQLo = C::kQTileBytes >> 4, kStageLo = C::kStageBytes >> 4;
      // The ring stage and phase of the next K tile and of the next V tile; per slot the S, P V, units and Q tiles so
      // far.
      int sk = 0, sv = 0;
      uint32_t phk = 0, phv = 0, ns[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0}, nq[2] = {0, 0};
      bool ok = true;
      auto mwait = [&](uint64_t* x, uint32_t parity) { return warp_wait(x, parity); };
      auto step_k = [&]() {
        if (C::kSplitKV) warp_tc_commit(k_empty + sk);
        if (++sk == S) {
          sk = 0;
          phk ^= 1u;
        }
      };
      auto step_v = [&]() {
        warp_tc_commit(v_empty + sv);
        if (++sv == S) {
          sv = 0;
          phv ^= 1u;
        }
      };
      auto k_ready = [&]() { return mwait(k_full + sk, phk); };
      auto v_ready = [&]() { return !C::kSplitKV || mwait(v_full + sv, phv); };
      // S of slot T from Q tile `tile` and the current K stage, once the slot's S columns are free: read, or (P in S's
      // columns) its last P V done.
      auto s_ready = [&](auto T) {
        constexpr int t = decltype(T)::v;
        return mwait((C::kSepP ? s_free : pv_done) + t, (ns[t] - 1) & 1);
      };
      auto qk = [&](auto T, int tile) {
        constexpr int t = decltype(T)::v;
        tc_fence_after();
        issue_qk<D, kE4M3>(colS + t * kBN, q_lo + tile * kQLo, k_lo + sk * kStageLo);
        warp_tc_commit(s_full + t);
        ++ns[t];
      };
      auto p_ready = [&](auto T) {
        constexpr int t = decltype(T)::v;
        return mwait(p_full + t, np[t] & 1);
      };
      auto pv = [&](auto T, bool first) {
        constexpr int t = decltype(T)::v;
        tc_fence_after();
        issue_pv<D, kE4M3>(colO + t * D, colP + t * C::kStepP, v_lo + sv * kStageLo, first);
        warp_tc_commit(pv_done + t);
        ++np[t];
      };
      // A unit's first S of a slot; its first P V waits until the last unit's O was read.
      auto begin = [&](auto T, int tile) {
        constexpr int t = decltype(T)::v;
        if (ns[t] > 0 && !s_ready(T)) return false;
        qk(T, tile);
        return true;
      };
      auto o_ready = [&](auto T) {
        constexpr int t = decltype(T)::v;
        return no[t]++ == 0 || mwait(o_free + t, (no[t] - 2) & 1);
      };
      // One key tile of a unit of one row tile, in slot T.
      auto one_tile = [&](auto T, bool first, bool more) {
        if (C::kSepP && more) {
          if (!k_ready() || !s_ready(T)) return false;
          qk(T, 0);
          step_k();
        }
        if (!p_ready(T) || !v_ready()) return false;
        pv(T, first);
        step_v();
        if (!C::kSepP && more) {
          if (!k_ready() || !s_ready(T)) return false;
          qk(T, 0);
          step_k();
        }
        return true;
      };
      const Slot<0> s0;
      const Slot<1> s1;
      for (int k = 0; ok; ++k) {
        ok = mwait(unit_full + (k & 1), (k >> 1) & 1);
        if (!ok) break;
        const int ntiles = __shfl_sync(0xffffffffu, sh.unit[k & 1].nt, 0);
        const bool one = __shfl_sync(0xffffffffu, sh.unit[k & 1].rows, 0) <= 128;
        release_unit(k);
        if (ntiles < 0) break;
        ok = k_ready() && mwait(q_full, nq[0]++ & 1) && begin(s0, 0);
        if (one) {
          if (ok) step_k();
          if (ok && ntiles > 1) {
            ok = k_ready() && begin(s1, 0);
            if (ok) step_k();
          }
          ok = ok && o_ready(s0) && (ntiles == 1 || o_ready(s1));
          for (int j = 0; j < ntiles && ok; j += 2) {
            ok = one_tile(s0, j == 0, j + 2 < ntiles);
            if (ok && j + 1 < ntiles) ok = one_tile(s1, j == 0, j + 3 < ntiles);
          }
        } else {
          ok = ok && mwait(q_full + 1, nq[1]++ & 1) && begin(s1, 1);
          if (ok) step_k();
          ok = ok && o_ready(s0) && o_ready(s1);
          for (int j = 0; j < ntiles && ok; ++j) {
            const bool more = j + 1 < ntiles;
            if (C::kSepP) {
              // S of the next tile as soon as S is read, P V once P is written.  The slots in turn: with both S issued
              // before both P V the two softmaxes ran in step and shared the exponential units (149 -> 135 us at the
              // sizes above).
              if (more) {
                ok = k_ready() && s_ready(s0);
                if (!ok) break;
                qk(s0, 0);
              }
              ok = p_ready(s0) && v_ready();
              if (!ok) break;
              pv(s0, j == 0);
              if (more) {
                ok = s_ready(s1);
                if (!ok) break;
                qk(s1, 1);
                step_k();
              }
              ok = p_ready(s1);
              if (!ok) break;
              pv(s1, j == 0);
              step_v();
            } else {
              ok = p_ready(s0) && v_ready();
              if (!ok) break;
              pv(s0, j == 0);
              if (more) {
                ok = k_ready() && s_ready(s0);
                if (!ok) break;
                qk(s0, 0);
              }
              ok = p_ready(s1);
              if (!ok) break;
              pv(s1, j == 0);
              step_v();
              if (more) {
                ok = s_ready(s1);
                if (!ok) break;
                qk(s1, 1);
                step_k();
              }
            }
          }
        }
      }
      if (!ok && lane == 0) give_up(a.status, kWherePagedMma, &sh.abort);
      __syncwarp();
      // Every MMA issued has finished before the tensor memory is freed.
      warp_tc_commit(mma_final);
      mbar_wait(mma_final, 0, kChunkWaitNs);
    }
  } else if (kE4M3 && warp >= 12) {
    // -------------------------------------------------------------- widen the codes
    regs_dec<C::kRegsWiden>();
    const int r = threadIdx.x - 384;   // the key of the tile
    const uint32_t raw = smem_u32(smem + C::kRawOff) + r * D;
    const uint32_t rsw = D == 128 ? (r & 7) : ((r >> 1) & 3);
    uint32_t ct = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = wait(unit_full + (k & 1), (k >> 1) & 1, kWherePagedEmpty);
      if (!ok) break;
      const Unit& e = sh.unit[k & 1];
      const int ntiles = e.nt, ulo = e.ulo, uhi = e.uhi, key_r = e.t0 * kBN + r;
      release_unit(k);
      if (ntiles < 0) break;
      for (int j = 0; j < ntiles && ok; ++j, ++ct) {
        const uint32_t s = ct % S;
        uint8_t* tile = sKV + s * C::kStageBytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (ct >= S && (C::kSplitKV || kv == 0))
            ok = warp_wait((kv || !C::kSplitKV ? v_empty : k_empty) + s, (ct / S - 1) & 1);
          ok = ok && warp_wait(raw_full + kv, ct & 1);
          if (!ok) give_up(a.status, kWherePagedFull, &sh.abort);
          ok = !__any_sync(0xffffffffu, !ok || sh.abort);
          if (!ok) break;
          const uint32_t bits = sh.raw_bits[kv];
          const int key = key_r + j * kBN;
          // Keys that no row sees count as zeros, whatever their slots hold.
          const bool live = ((bits >> (r >> p.box_shift)) & 1u) && key >= ulo && key < uhi;
          uint4 v[D / 16];
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(v[ch].x), "=r"(v[ch].y), "=r"(v[ch].z), "=r"(v[ch].w)
                         : "r"(raw + kv * C::kRawTile + ((ch ^ rsw) << 4)));
          mbar_arrive(raw_empty + kv);
          if (r == 0 && kv == 0) sh.bits[ct % (2 * S)] = bits;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            const uint32_t w[4] = {v[ch].x, v[ch].y, v[ch].z, v[ch].w};
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * i]) : "h"(static_cast<uint16_t>(live ? w[i] : 0u)));
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f[2 * i + 1]) : "h"(static_cast<uint16_t>(live ? w[i] >> 16 : 0u)));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int c8 = ch * 2 + i;   // 8-channel chunk of the 16-bit row
              *reinterpret_cast<uint4*>(tile + kv * C::kTileBytes + (c8 >> 3) * C::kPanelBytes + r * 128 +
                                        (((c8 & 7) ^ (r & 7)) << 4)) =
                  make_uint4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            }
          }
          fence_proxy_async_smem();
          if (C::kSplitKV || kv == 1) mbar_arrive((kv && C::kSplitKV ? v_full : k_full) + s);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax and epilogue
    regs_inc<C::kRegsSoftmax>();
    const int t = (warp - 4) >> 2, wq = warp & 3, r = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * kBN, tO = tmem + lane_base + C::kColO0 + t * D;
    const uint32_t tP = tmem + lane_base + C::kColP0 + t * C::kStepP;
    const uint32_t all_boxes = (1u << boxes) - 1u;   // at most 16
    // Slot t's Q tile of a unit, each warp its 32 rows: started here (bf16), finished and announced when the unit begins.
    auto load_q = [&](const Unit& u) {
      if (t == 1 && u.rows <= 128) return;
      // Lane i finds row i (one division), the others get it by shuffle; rows past the last are zeros.
      uint8_t* tile = sQ + t * C::kQTileBytes;
      const int my = t * 128 + wq * 32 + lane, my_row = u.row0 + my;
      const int64_t my_at = my < u.rows ? static_cast<int64_t>(u.start + my_row / p.group) * a.qst +
                                              static_cast<int64_t>(u.h * p.group + my_row % p.group) * a.qsh
                                        : -1;
      const uint16_t* q = a.q;
      if (!kE4M3) {
        // 8 lanes to a row's 128 bytes.
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = wq * 32 + i * 4 + (lane >> 3), ch = lane & 7;
          const int64_t at = __shfl_sync(0xffffffffu, my_at, i * 4 + (lane >> 3));
          const uint32_t n = at >= 0 ? 16 : 0;
          const uint16_t* src = q + (at >= 0 ? at : 0) + ch * 8;
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             smem_u32(tile + pn * C::kPanelBytes + rr * 128 + ((ch ^ (rr & 7)) << 4))),
                         "l"(src + pn * 64), "r"(n)
                         : "memory");
        }
      } else {
        // fp16 times a power of two that brings the row's largest value into [1, 2): exact but for values
        // 2^-14 below it, which keep an absolute error of 2^-25 of the row's largest.  D/8 lanes a row.
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;
#pragma unroll 4
        for (int i = 0; i < 32 / kPer; ++i) {
          const int rr = wq * 32 + i * kPer + lane / kLanes, c8 = lane % kLanes;
          const int64_t at = __shfl_sync(0xffffffffu, my_at, i * kPer + lane / kLanes);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (at >= 0) v = __ldg(reinterpret_cast<const uint4*>(q + at + c8 * 8));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float mx = 0.0f;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[x] << 16)), fabsf(__uint_as_float(w[x] & 0xFFFF0000u))));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          int e = static_cast<int>((__float_as_uint(mx) >> 23) & 255) - 127;
          e = mx == 0.0f ? 0 : min(max(e, -126), 126);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          uint32_t f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            f[x] = pack2<true>(__uint_as_float(w[x] << 16) * down, __uint_as_float(w[x] & 0xFFFF0000u) * down);
          *reinterpret_cast<uint4*>(tile + (c8 >> 3) * C::kPanelBytes + rr * 128 + (((c8 & 7) ^ (rr & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
          if (c8 == 0) q_exp[t * 128 + rr] = static_cast<uint8_t>(127 + e);
        }
      }
    };
    auto announce_q = [&](const Unit& u) {
      if (t == 1 && u.rows <= 128) return;
      if (!kE4M3) asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(q_full + t);
    };
    // One unit, of one row tile or of two.  (Runtime, not two copies: with them window_e4m3 took 195 us instead of 168,
    // a third of the stalls for instructions.)
    auto work = [&](int k) -> bool {
      const Unit& u = sh.unit[k & 1];
      const bool one = u.rows <= 128;
      bool ok = true;
      const int ntiles = u.nt, first = one ? 0 : t * 128;   // the slot's first row
      const int steps = one ? (ntiles + 1 - t) / 2 : ntiles;
      int klo, khi;   // this row's visible keys
      token_keys(a, u.len, u.n_new, (u.row0 + min(first + r, u.rows - 1)) / p.group, klo, khi);
      const int alo = u.alo[t], ahi = u.ahi[t];
      float c = a.scale_log2;
      if (kE4M3) {
        // (In a unit of one row tile slot 0's warps wrote the exponents.)
        if (one && t == 1) ok = wait(q_full, k & 1, kWherePagedFull);
        else __syncwarp();
        c *= __ldg(a.k_scale + u.h) * __uint_as_float(static_cast<uint32_t>(q_exp[first + r]) << 23);
      }
      float m = -INFINITY, l = 0.0f;
      const int key_t0 = u.t0 * kBN;
      const uint32_t ct = u.ct, mine = u.mine[t];
      for (int i = 0; i < steps && ok; ++i) {
        ok = wait(s_full + t, (mine + i) & 1, kWherePagedMma);
        if (!ok) break;
        tc_fence_after();
        const int j = one ? 2 * i + t : i, kb = key_t0 + j * kBN;
        const uint32_t bits = sh.bits[(ct + j) % (2 * S)];
        const bool masked = kb < alo || kb + kBN > ahi || bits != all_boxes;
        ok = softmax_step<D, kE4M3>(tS, tO, tP, c, masked, [&](uint32_t mask[4]) {
          if (!kE4M3) {
            // Keys that no row of the unit sees may hold anything: their V counts as 0.
            const uint32_t s = (ct + j) % S;
            const int key = kb + r;
            if (C::kSplitKV) wait(v_full + s, ((ct + j) / S) & 1, kWherePagedFull);
            if (!(((bits >> (r >> p.box_shift)) & 1u) && key >= u.ulo && key < u.uhi)) {
              uint8_t* v = sKV + s * C::kStageBytes + C::kTileBytes + r * 128;
#pragma unroll
              for (int x = 0; x < 8 * C::kPanels; ++x)
                *reinterpret_cast<uint4*>(v + (x >> 3) * C::kPanelBytes + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) mask[w] = key_mask(w, klo - kb, khi - kb, bits, p.box_shift);
          __syncwarp();
        }, i == 0, m, l, s_free + t, pv_done + t, static_cast<int>(mine) + i);
        if (!ok) {
          if (lane == 0) give_up(a.status, kWherePagedMma, &sh.abort);
          break;
        }
        tc_fence_before();
        mbar_arrive(p_full + t);
      }
      if (ok && steps > 0) ok = wait(pv_done + t, (mine + steps - 1) & 1, kWherePagedMma);
      float own = 1.0f, other = 0.0f;   // factors of slot 0's and slot 1's O (one row tile)
      if (one && ok) {
        const uint32_t ones = u.ones;
        // Slot 1's maxima and sums to slot 0's warps, which read its O themselves: the same lanes of tensor memory.
        if (t == 1) {
          if (ones > 0) ok = wait(ml_empty, (ones - 1) & 1, kWherePagedMma);
          if (ok) sh.ml[r] = make_float2(m, l);
          mbar_arrive(ml_full);
        } else {
          ok = wait(ml_full, ones & 1, kWherePagedMma) &&
               (ntiles == 1 || wait(pv_done + 1, (u.mine[1] + ntiles / 2 - 1) & 1, kWherePagedMma));
          const float2 x = sh.ml[r];
          mbar_arrive(ml_empty);
          const float mm = fmaxf(m, x.x);
          // A slot that saw no key counts nothing.
          own = m == -INFINITY ? 0.0f : ex2_approx(m - mm);
          other = x.x == -INFINITY ? 0.0f : ex2_approx(x.x - mm);
          l = l * own + x.y * other;
          m = mm;
        }
      }
      // The next unit's Q comes under this one's epilogue (every S that reads the slot's Q tile is done).
      const Unit& next = sh.unit[(k + 1) & 1];
      ok = ok && wait(unit_full + ((k + 1) & 1), ((k + 1) >> 1) & 1, kWherePagedEmpty);
      const bool has_next = ok && next.nt >= 0;
      if (C::kEarlyQ && has_next) {
        load_q(next);
        if (kE4M3 || (one && t == 1)) announce_q(next);
      }
      if (ok && (!one || t == 0)) {
        tc_fence_after();
        const int ur = first + r;
        const bool live = ur < u.rows, whole = u.slot < 0;
        const int row = u.row0 + (live ? ur : 0);
        const int tok = u.start + row / p.group, hd = u.h * p.group + row % p.group;
        const float vs = kE4M3 ? __ldg(a.v_scale + u.h) : 1.0f;
        // A row that saw no key (l = 0) becomes 0.
        const float inv = whole ? (l > 0.0f ? vs / l : l) : 1.0f;
        const float f0 = own * inv, f1 = other * inv;
        const int64_t o_at = static_cast<int64_t>(tok) * a.ost + static_cast<int64_t>(hd) * a.osh;
        float* part = whole ? nullptr : a.part_o + (static_cast<int64_t>(u.slot) * kPagedChunkRows + first + wq * 32) * D;
        const int rows_here = u.rows - first - wq * 32;   // of this warp's 32
        uint16_t* out = a.out;
        // 32 channels of the row, times the factors.
        auto channels = [&](int c0, uint32_t o[32]) {
          __syncwarp();
          SAGE_TMEM_LD32(tO + c0, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f0);
          if (one && ntiles > 1) {
            uint32_t x[32];
            SAGE_TMEM_LD32(tO + D + c0, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(fmaf(__uint_as_float(x[i]), f1, __uint_as_float(o[i])));
          }
        };
        // Rows leave 128 bytes at a time through shared memory (64 bf16 channels, or 32 of a partial result), so that a
        // warp stores whole lines; storing 16 bytes of 32 rows at a time took 2.0 us of a unit.
        uint8_t* stage = (C::kEarlyQ ? smem + C::kOutOff + t * 16384 : sQ + t * C::kQTileBytes) + wq * 4096;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += whole ? 64 : 32) {
          uint32_t o[32];
#pragma unroll 1
          for (int h2 = 0; h2 < (whole ? 2 : 1); ++h2) {
            channels(c0 + h2 * 32, o);
            if (whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  w[x] = pack2<false>(__uint_as_float(o[i * 8 + 2 * x]), __uint_as_float(o[i * 8 + 2 * x + 1]));
                const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((h2 * 4 + i) ^ (lane & 7)) << 4)) = v;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 v = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = v;
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = i * 4 + (lane >> 3), ch = lane & 7;
            const int64_t at = __shfl_sync(0xffffffffu, o_at, rr);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
            if (rr < rows_here) {
              if (whole) *reinterpret_cast<uint4*>(out + at + c0 + ch * 8) = v;
              else *reinterpret_cast<uint4*>(part + rr * D + c0 + ch * 4) = v;
            }
          }
          __syncwarp();
          if (C::kEarlyQ && !kE4M3 && c0 == 0 && has_next) announce_q(next);
        }
        tc_fence_before();
        mbar_arrive(o_free + t);
        if (one && ntiles > 1) mbar_arrive(o_free + 1);
        if (live) {
          if (!whole) a.part_ml[u.slot * kPagedChunkRows + ur] = make_float2(m, l);
          else if (a.lse) a.lse[static_cast<int64_t>(tok) * a.hq + hd] = lse_of(m, l);
        }
      }
      if (!C::kEarlyQ && has_next) {
        load_q(next);
        announce_q(next);
      }
      release_unit(k);
      return ok;
    };
    bool ok = wait(unit_full, 0, kWherePagedEmpty);
    if (ok && sh.unit[0].nt >= 0) {
      load_q(sh.unit[0]);
      announce_q(sh.unit[0]);
    }
    for (int k = 0; ok && sh.unit[k & 1].nt >= 0; ++k) ok = work(k);
    if (!kE4M3) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The parts of split units, joined in the order of their keys: a CTA takes 8 rows of a unit, 32 threads
// a row.
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ ChunkParams p) {
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  Unit u;
  if (!find_unit(a, p.group, p.whole + blockIdx.x, u)) return;
  const int ur = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (ur >= u.rows) return;
  const float2* ml = a.part_ml + static_cast<int64_t>(blockIdx.x) * p.splits * kPagedChunkRows + ur;
  constexpr int kC = D / 32;   // channels of a lane
  using Channels = std::conditional_t<D == 128, float4, float2>;
  const float* o = a.part_o + (static_cast<int64_t>(blockIdx.x) * p.splits * kPagedChunkRows + ur) * D + lane * kC;
  const int64_t o_step = static_cast<int64_t>(kPagedChunkRows) * D;
  float m = -INFINITY, l = 0.0f;
  for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, ml[s * kPagedChunkRows].x);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  float v[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) v[i] = 0.0f;
  for (int s0 = 0; s0 < p.splits; s0 += 32) {
    // Lane i has part s0 + i's factor, 0 for one that saw no key: its O counts nothing (and may not have been written).
    float f = 0.0f;
    if (s0 + lane < p.splits) {
      const float2 x = ml[(s0 + lane) * kPagedChunkRows];
      if (x.x != -INFINITY) f = ex2_approx(x.x - m);
      else if (x.y != 0.0f) f = x.y;   // scores that are no numbers: neither is the result
      l += x.y * f;
    }
    const int n = min(32, p.splits - s0);
    for (int s = 0; s < n; s += 4) {
      float part[4][kC], g[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        g[x] = __shfl_sync(0xffffffffu, f, s + x);
        Channels c{};
        if (g[x] != 0.0f) c = *reinterpret_cast<const Channels*>(o + (s0 + s + x) * o_step);
#pragma unroll
        for (int i = 0; i < kC; ++i) part[x][i] = reinterpret_cast<const float*>(&c)[i];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < kC; ++i) v[i] = fmaf(part[x][i], g[x], v[i]);
    }
  }
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  const int row = u.row0 + ur, tok = u.start + row / p.group, hd = u.h * p.group + row % p.group;
  const float inv = l > 0.0f ? (a.v_scale ? __ldg(a.v_scale + u.h) : 1.0f) / l : l;   // 0 for a row that saw no key
  uint16_t* dst = a.out + static_cast<int64_t>(tok) * a.ost + static_cast<int64_t>(hd) * a.osh + lane * kC;
#pragma unroll
  for (int i = 0; i < kC; i += 2) *reinterpret_cast<uint32_t*>(dst + i) = pack2<false>(v[i] * inv, v[i + 1] * inv);
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(tok) * a.hq + hd] = lse_of(m, l);
}

template <int D, bool kE4M3>
cudaError_t launch_t(const PagedAttnArgs& a, const sage_paged_kv& kv, cudaStream_t s) {
  using C = ChunkCfg<D, kE4M3>;
  ChunkParams p;
  p.a = a;
  if (!kE4M3) p.a.v_scale = nullptr;
  p.group = a.hq / a.hkv;
  p.box_shift = std::min(a.b.page_shift, 7);
  const int64_t e = kE4M3 ? 1 : 2;
  CUtensorMap kmap, vmap;
  const int box_c = kE4M3 ? D : 64;
  if (!make_page_map(&kmap, kv.k_pages, kE4M3, D, kv.n_heads, kv.page_size, kv.n_pages, kv.k_stride_head * e,
                     kv.k_stride_token * e, kv.k_stride_page * e, box_c, 1 << p.box_shift) ||
      !make_page_map(&vmap, kv.v_pages, kE4M3, D, kv.n_heads, kv.page_size, kv.n_pages, kv.v_stride_head * e,
                     kv.v_stride_token * e, kv.v_stride_page * e, box_c, 1 << p.box_shift))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(paged_chunk_kernel<D, kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  // Units: sum over sequences of ceil(rows / 256), at most (all rows + 255 per sequence with tokens) / 256.
  const int64_t rows = static_cast<int64_t>(a.b.n_tokens) * p.group;
  const int64_t seqs = std::min<int64_t>(a.b.n_seqs, a.b.n_tokens);
  const int64_t units = (rows + 255 * seqs) / 256 * a.hkv;
  // Whole units fill the SMs as often as they can; those left over are split along the keys into the number of
  // parts that ends them soonest.  Their number is estimated from the mean length of a sequence.  In microseconds: an
  // item's key tiles (at most the table's) at 1.45 us for two row tiles of D = 128, 0.98 of D = 64, half for one row
  // tile; 3 between items; the parts' O written and read again at 3.4 TB/s with 6 us for the join,
  // 10 behind whole units (24 x 128 rows over 3000 keys of 8 heads: 71 us unsplit, 78 in three).
  const int64_t mean = (rows + seqs - 1) / seqs, blocks = (mean + 255) / 256;
  const bool one = mean <= 128, odd = mean - (blocks - 1) * 256 <= 128;   // units of one row tile: all, or the last ones
  const int64_t likely = std::min(units, seqs * blocks * a.hkv), whole = likely / sms * sms, rest = units - whole;
  const double count = static_cast<double>(likely - whole), tile_us = 0.51 + 0.94 * D / 128;
  const int64_t tiles = std::max(1, (a.b.cap + kBN - 1) / kBN);
  const int64_t most = std::min<int64_t>({kPagedSlots / std::max<int64_t>(rest, 1), sms, std::max<int64_t>(1, tiles / 4)});
  auto last_wave = [&](int64_t k) {
    const double items = count * static_cast<double>(k) * (odd && !one ? 1.0 - 0.5 / static_cast<double>(blocks) : 1.0);
    const double item = tile_us * (one ? 0.5 : 1.0) * static_cast<double>((tiles + k - 1) / k) + 3.0;
    const double part_bytes = std::min<double>(static_cast<double>(mean), 256.0) * D * 4;
    return std::ceil(items / sms) * item + (k > 1 ? (whole > 0 ? 10.0 : 6.0) + items * part_bytes * 2 / 3.4e6 : 0.0);
  };
  int64_t splits = 1;
  for (int64_t k = 2; k <= most; ++k)
    if (last_wave(k) < last_wave(splits)) splits = k;
  p.splits = static_cast<int>(splits);
  p.halve = !one;
  p.whole = static_cast<int>(splits > 1 ? whole : units);
  p.items = static_cast<uint32_t>(p.whole + (units - p.whole) * splits);
  paged_chunk_kernel<D, kE4M3><<<std::min<uint32_t>(p.items, sms), C::kThreads, C::kSmem, s>>>(kmap, vmap, p);
  err = cudaGetLastError();
  if (err == cudaSuccess && splits > 1)
    err = launch_dependent(true, paged_join_kernel<D>, dim3(static_cast<unsigned>(rest), kPagedChunkRows / 8), dim3(256), 0,
                           s, p);
  return err;
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  if (d == 128) return c.format == 1 ? launch_t<128, true>(a, c, s) : launch_t<128, false>(a, c, s);
  return c.format == 1 ? launch_t<64, true>(a, c, s) : launch_t<64, false>(a, c, s);
}

}  // namespace sage
