// paged_few.cu -- attention of few query rows per K/V head over the paged cache (single tokens, drafted
// tokens, short chunks): the query rows of a unit are the tokens of one sequence times the query heads
// that share one K/V head, 16 or 32 rows to a tile.
//
// What bounds it: every visible K and V byte is read once from HBM, 4 rows FLOPs per 2 (4 for E4M3)
// bytes, so the cache's bandwidth; for short contexts the chain launch -> lengths -> page table ->
// page -> result.  With so few rows the warp-level MMA (m16n8k16) keeps ahead of HBM: a 32 KB stage is
// 64 MMAs per warp of a team against ~1400 cycles of one SM's share of the bandwidth, and it leaves
// the accumulators in registers, so the warps need no barrier between key tiles.
//
// The key axis.  A unit (sequence, K/V head, row tile) has nt tiles of kKeys keys; the units' tiles are dealt to one
// CTA per SM (struct Walk), so ragged batches and single long sequences load every SM alike.  A CTA walks its tiles
// through one ring of TMA stages that does not stop at unit borders.  A unit that lies in one CTA is finished
// there.  Otherwise each CTA leaves (maximum, sum, O) of its part in the workspace and takes a ticket; the last
// one joins the parts in the order of their keys, so the result does not depend on which CTA came last (paged_join.h
// has the tickets' and slots' owners).
//
// Inside a CTA: two or four loading warps (page table entries by lane, one TMA box per page) and two teams of
// four consumer warps that take the tiles in turn, a quarter of a tile's keys to each warp.  Each warp
// keeps a running maximum, sum and O of its own keys (online softmax in fp32); the eight are
// joined through shared memory at the end of a segment.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "paged_batch.cuh"
#include "tensor_map.h"

namespace sage {
namespace {

// Warps 0-3: loads (two of them may only give up their registers); warps 4-11: consumers.
// 384 threads launch with 168 registers each; 40 / 232 after the split (128 * 40 + 256 * 232 =
// 384 * 168), which holds two row tiles' accumulators.
constexpr int kFewConsumers = 256, kFewThreads = 384;
constexpr int kFewRegsProducer = 40, kFewRegsConsumer = 232;
static_assert(128 * kFewRegsProducer + 256 * kFewRegsConsumer <= kFewThreads * 168, "register split exceeds launch");
constexpr uint64_t kFewWaitNs = 2000000000ull;
constexpr float kFewRise = 8.0f;   // log2 of how far a maximum may fall behind

template <int D, bool kE4M3, int MT>
struct FewCfg {
  static constexpr int kRows = 16 * MT;
  static constexpr int kRowBytes = D * (kE4M3 ? 1 : 2);
  static constexpr int kPanels = kRowBytes > 128 ? 2 : 1;
  static constexpr int kPanelRow = kRowBytes / kPanels;       // 128, or 64 (E4M3 at D = 64)
  static constexpr int kKeys = 16384 / kRowBytes;             // keys per stage: 64, 128 or 256
  static constexpr int kPanelBytes = kKeys * kPanelRow;
  static constexpr int kStageBytes = 32768;                   // 16 KB of K, 16 KB of V
  // Even, so that a stage is always the same team's: a team that skipped every other phase of a
  // barrier could take a phase two back, of the same parity, for the one it waits for.
  static constexpr int kStages = 4;
  static_assert(kStages % 2 == 0, "a ring stage must stay with one team");
  // K and V have a loading warp each, even and odd tiles too: a tile's load is a chain of waits (~400 cycles) that one
  // warp did not repeat fast enough (one / two / four warps: decode_e4m3 69.4 / 64.0 / 61.6 us, 16 single tokens over
  // 500-4000 keys 40.6 / 34.2 / 32.4).  Rows of 64 bytes share lines between heads, which are best read in order
  // (24 heads: 191 / 179 / 205 us), and with two row tiles the arithmetic is the limit (E4M3: 71.5 / 72 / 73.5).
  static constexpr int kTurns = MT == 1 && kRowBytes >= 128 ? 2 : 1;
  static constexpr int kWarpKeys = kKeys / 4;
  static constexpr int kNT = kWarpKeys / 8;                   // 8-key score tiles per warp
  static constexpr int kOT = D / 8;                           // 8-channel O tiles
  static constexpr int kQRow = D * 2 + 16;                    // padded Q row
  static constexpr int kMergeRow = D + 8;                     // padded merge row
  static constexpr int kQOff = kStages * kStageBytes;
  static constexpr int kMergeOff = kQOff + 2 * kRows * kQRow;
  static constexpr int kMlOff = kMergeOff + 8 * 16 * kMergeRow * 4;
  static constexpr int kScaleOff = kMlOff + 2 * 8 * 16 * 4;   // 2^e of each Q row (E4M3), per buffer
  static constexpr int kBarOff = kScaleOff + 2 * kRows * 4;
  static constexpr int kNumBars = 2 * kStages + 4;
  static constexpr int kSmem = kBarOff + kNumBars * 8 + kStages * 4 + 16 + 1024;
  static_assert(kSmem <= 232448 - 512, "shared memory");
};

__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t r[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (low byte first) as fp16x2: exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// Arrives on `bar` once this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Draws a ticket with acquire and release at the GPU's scope; true for the last of n, which resets the counter.
__device__ __forceinline__ int draw_ticket(int32_t* counter, int n) {
  int before;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
  if (before != n - 1) return 0;
  *counter = 0;
  return 1;
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

struct FewParams {
  PagedAttnArgs a;
  int group;         // query heads per K/V head
  int lock;          // K/V heads that as many CTAs take side by side
  int box_shift;     // log2 of the slots per TMA box (a page, or a stage's keys where that is less)
};

// What one sequence asks for: row tiles x K/V heads units of nt key tiles each, from tile t_lo.
struct SeqWork {
  int start, rows, len;   // first row of q, rows x group, tokens in the cache
  int n_new;
  int qt, nt, t_lo;
};
template <int kRows, int kKeys>
__device__ __forceinline__ SeqWork seq_work(const FewParams& p, int b) {
  SeqWork w;
  int end;
  seq_rows(p.a.b, b, w.start, end);
  w.n_new = end - w.start;
  w.len = min(max(__ldg(p.a.b.kv_len + b), 0), p.a.b.cap);
  w.rows = w.n_new * p.group;
  w.qt = (w.rows + kRows - 1) / kRows;
  // All keys that some row sees (the per-tile masks cut the rest): a window starts at its first row's.
  const int lo = p.a.window > 0 ? max(0, w.len - w.n_new + 1 - p.a.window) : 0;
  w.t_lo = lo / kKeys;
  w.nt = max(1, (w.len + kKeys - 1) / kKeys - w.t_lo);
  return w;
}

// The visible keys [lo, hi) of token j (0-based among the sequence's new ones).
__device__ __forceinline__ void token_keys(const PagedAttnArgs& a, const SeqWork& w, int j, int& lo, int& hi) {
  const int pos = w.len - w.n_new + j;
  hi = a.causal ? max(0, pos + 1) : w.len;
  lo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
}

// A CTA's share of the units' key tiles, walked alike by every warp of it.  One of two ways:
//  - aligned: where every unit can have CTAs of its own, a unit's tiles are dealt evenly to ceil(nt / q) CTAs, with
//    the smallest q (at least 4: below that the join costs more than the tiles) that the grid allows;
//  - even: the flat list of all tiles is cut into equal runs, whatever units they cross.  It balances many units or
//    very unequal ones, at the price of two partial units per CTA.
template <int kRows, int kKeys>
struct Walk {
  SeqWork w;
  int b;
  int u;                // unit within the sequence
  int k;                // tile within the unit
  uint32_t at, end;     // even: flat tile index now, end of the CTA's share; aligned: 0, tiles of the share
  uint32_t quota;       // even: tiles per CTA; aligned: 0
  int part, parts;      // aligned: this CTA's part of its unit

  // Units and tiles per unit of sequence b; (0, 1) past the last.
  __device__ __forceinline__ void count(const FewParams& p, int b, uint32_t& units, uint32_t& nt) {
    units = 0;   // of one of the `lock` heads
    nt = 1;
    if (b < p.a.b.n_seqs) {
      const SeqWork s = seq_work<kRows, kKeys>(p, b);
      units = s.qt * (p.a.hkv / p.lock);
      nt = s.nt;
    }
  }
  // Sum of f(units, nt) over the sequences; units, nt: this lane's sequence, where there are at most 32.
  template <typename F>
  __device__ __forceinline__ uint32_t sum(const FewParams& p, uint32_t units, uint32_t nt, F f) {
    uint32_t total = 0;
    for (int b0 = 0; b0 < p.a.b.n_seqs; b0 += 32) {
      if (p.a.b.n_seqs > 32) count(p, b0 + (threadIdx.x & 31), units, nt);
      total += f(units, nt);
    }
    return __reduce_add_sync(0xffffffffu, total);
  }
  // Sets b and w to the sequence in which the running sum of f passes `target`; `before`: the sum before it.
  template <typename F>
  __device__ __forceinline__ bool locate(const FewParams& p, uint32_t target, uint32_t units, uint32_t nt, F f,
                                         uint32_t& before) {
    const int lane = threadIdx.x & 31;
    uint32_t base = 0;
    for (int b0 = 0; b0 < p.a.b.n_seqs; b0 += 32) {
      if (p.a.b.n_seqs > 32) count(p, b0 + lane, units, nt);
      const uint32_t n = f(units, nt);
      uint32_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, base + incl > target);
      if (past) {
        const int l = __ffs(past) - 1;
        b = b0 + l;
        before = base + __shfl_sync(0xffffffffu, incl - n, l);
        w = seq_work<kRows, kKeys>(p, b);
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }

  // False if the CTA has no share.
  __device__ __forceinline__ bool init(const FewParams& p) {
    const uint32_t grid = gridDim.x / p.lock, me = blockIdx.x / p.lock;
    uint32_t units, nt, before;
    count(p, threadIdx.x & 31, units, nt);
    // Tiles and units are counted in 32 bits: a batch of 2^31 tiles (each a 32 KB read) is refused.
    uint64_t mine = 0;
    for (int b0 = 0; b0 < p.a.b.n_seqs; b0 += 32) {
      uint32_t x = units, y = nt;
      if (p.a.b.n_seqs > 32) count(p, b0 + (threadIdx.x & 31), x, y);
      mine += static_cast<uint64_t>(x) * y;
    }
    if (__any_sync(0xffffffffu, mine >= (1ull << 26))) {
      uint64_t all = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      if (all >= (1ull << 31)) {
        record_bad_index(p.a.status, kWhereLength);
        return false;
      }
    }
    const uint32_t total = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(mine));
    const uint32_t even = (total + grid - 1) / grid;
    part = parts = 0;
    if (sum(p, units, nt, [](uint32_t u, uint32_t) { return u; }) <= grid) {
      // At q = the largest nt the parts are the units, which the grid holds.
      uint32_t q = max(even, 4u);
      const uint32_t most = even + 4;
      while (q <= most && sum(p, units, nt, [q](uint32_t u, uint32_t n) { return u * ((n + q - 1) / q); }) > grid) ++q;
      if (q <= most) {
        if (!locate(p, me, units, nt, [q](uint32_t u, uint32_t n) { return u * ((n + q - 1) / q); }, before)) return false;
        const int off = static_cast<int>(me - before);
        parts = static_cast<int>((w.nt + q - 1) / q);
        u = off / parts;
        part = off - u * parts;
        // parts <= 152 and nt < 2^24: the products stay below 2^32
        k = static_cast<int>(static_cast<uint32_t>(w.nt) * part / parts);
        at = 0;
        end = static_cast<uint32_t>(w.nt) * (part + 1) / parts - k;
        quota = 0;
        return true;
      }
    }
    quota = even;
    at = quota * me;
    end = min(total, at + quota);
    if (at >= end || !locate(p, at, units, nt, [](uint32_t u, uint32_t n) { return u * n; }, before)) return false;
    const uint32_t off = at - before;
    u = static_cast<int>(off / w.nt);
    k = static_cast<int>(off - u * w.nt);
    return true;
  }
  __device__ __forceinline__ int seg_tiles() const {
    return quota ? static_cast<int>(min(static_cast<uint32_t>(w.nt - k), end - at)) : static_cast<int>(end);
  }
  // The rows of CTAs that hold parts of the current unit: n of them from the first.
  __device__ __forceinline__ void unit_parts(const FewParams& p, int& first, int& n) const {
    if (quota == 0) {
      first = static_cast<int>(blockIdx.x) / p.lock - part;
      n = parts;
      return;
    }
    first = static_cast<int>((at - k) / quota);
    n = static_cast<int>((at - k + w.nt - 1) / quota) - first + 1;
  }
  // Past the segment of n tiles; afterwards valid only while at < end.
  __device__ __forceinline__ void next(const FewParams& p, int n) {
    at += n;
    k += n;
    if (at >= end || k < w.nt) return;
    k = 0;
    if (++u < w.qt * (p.a.hkv / p.lock)) return;
    u = 0;
    do {
      if (++b >= p.a.b.n_seqs) {   // the lengths changed under the call: stop
        at = end;
        return;
      }
      w = seq_work<kRows, kKeys>(p, b);
    } while (w.qt == 0);
  }
};

// A part left in the workspace, its ticket drawn: joined at the CTA's end if it was its unit's last.
struct Pending {
  int counter, count;                   // the ticket's counter and value that makes it the last
  int first, cf, parts;                 // first part of its group; the unit's first row of CTAs and its parts
  int start, rows, h, qi;
};

template <int D, bool kE4M3, int MT>
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ FewParams p) {
  using C = FewCfg<D, kE4M3, MT>;
  constexpr int R = C::kRows, KT = C::kKeys;
  extern __shared__ uint8_t smem_raw[];
  __shared__ volatile int s_abort;
  __shared__ int s_last[2], s_skip;
  __shared__ Pending s_pending[2];   // of the CTA's first and last segment
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* q_full = empty + C::kStages;
  uint64_t* q_empty = q_full + 2;
  uint32_t* page_bits = reinterpret_cast<uint32_t*>(q_empty + 2);   // per stage: the boxes loaded
  // The warp's number by shuffle, so that what follows from it is computed once per warp (decode_e4m3 71.1 -> 69.4 us);
  // two row tiles of E4M3 have no registers to spare for it (71 -> 82).
  const int tid5 = threadIdx.x >> 5, warp = MT == 1 ? __shfl_sync(0xffffffffu, tid5, 0) : tid5;
  const int lane = threadIdx.x & 31;
  const PagedAttnArgs& a = p.a;
  const int col = static_cast<int>(blockIdx.x) % p.lock;   // which of the `lock` heads side by side

  grid_dep_wait();     // launched as a dependent: nothing is read before the kernel ahead is done
  grid_dep_launch();
  if (threadIdx.x == 0) {
    s_skip = *reinterpret_cast<volatile int32_t*>(a.status) == kStatusTimeout;
    s_abort = 0;
    s_last[0] = s_last[1] = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full + s, 2);
      mbar_init(empty + s, 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full + s, 32);
      mbar_init(q_empty + s, 8);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (s_skip) return;   // an earlier wait ran out: no work until the status has been read

  auto fail = [&](int where) {
    record_timeout(a.status, where);
    s_abort = 1;
  };

  Walk<R, KT> wk;
  if (warp < 4) {
    // ------------------------------------------------------------------ loads
    regs_dec<kFewRegsProducer>();
    // Warps 0 and 1 load K and V, of the even tiles where 2 and 3 load those of the odd ones; warp 0 Q.
    if (warp >= 2 * C::kTurns || !wk.init(p)) return;
    const int kv = warp & 1, turn = warp >> 1;
    const CUtensorMap* map = kv ? &vmap : &kmap;
    tma_prefetch_desc(map);
    const int box = 1 << p.box_shift, boxes = KT >> p.box_shift;   // boxes per stage, at most 32
    const uint32_t box_bytes = static_cast<uint32_t>(box) * C::kRowBytes;
    int it = 0, issued = 0;
    bool ok = true;
    for (int seg = 0; wk.at < wk.end && ok; ++seg) {
      const int n = wk.seg_tiles();
      const int h = wk.u / wk.w.qt * p.lock + col, qi = wk.u % wk.w.qt;
      const int buf = seg & 1;
      if (warp == 0 && seg >= 2 && !mbar_wait(q_empty + buf, ((seg >> 1) - 1) & 1, kFewWaitNs)) {
        fail(kWherePagedEmpty);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok && !s_abort);
      if (!ok) break;
      if (warp == 0) {
        const uint32_t sq = smem_u32(smem + C::kQOff + buf * R * C::kQRow);
        // Lane i finds row i (one division), the others get it by shuffle; rows past the last are zeros.
        const int my = qi * R + lane;
        const int64_t my_at = lane < R && my < wk.w.rows
                                  ? static_cast<int64_t>(wk.w.start + my / p.group) * a.qst +
                                        static_cast<int64_t>(h * p.group + my % p.group) * a.qsh
                                  : -1;
        constexpr int kLanes = D / 8;   // lanes to a row
#pragma unroll
        for (int i = 0; i < R * kLanes / 32; ++i) {
          const int r = i * (32 / kLanes) + lane / kLanes, c = lane % kLanes;
          const int64_t at = __shfl_sync(0xffffffffu, my_at, r);
          cp_async16(sq + r * C::kQRow + c * 16, a.q + (at >= 0 ? at : 0) + c * 8, at >= 0);
        }
        cp_async_arrive(q_full + buf);
      }
      // The keys any row of this tile sees.
      int ulo, uhi, unused;
      token_keys(a, wk.w, (qi * R) / p.group, ulo, unused);
      token_keys(a, wk.w, (min(qi * R + R, wk.w.rows) - 1) / p.group, unused, uhi);
      if (threadIdx.x == 0 && __ldg(a.b.kv_len + wk.b) > a.b.cap) record_bad_index(a.status, kWhereLength);
      const int32_t* row = a.b.table + wk.b * a.b.table_stride;
      const int first0 = (wk.w.t_lo + wk.k) * KT + (lane << p.box_shift);
      auto needed = [&](int i) { return i < n && lane < boxes && first0 + i * KT < uhi && first0 + i * KT + box > ulo; };
      const int i0 = it % C::kTurns != turn;
      int next = needed(i0) ? __ldg(row + ((first0 + i0 * KT) >> a.b.page_shift)) : -1;
      for (int i = i0; i < n; i += C::kTurns) {
        // The next tile's table entries are on their way while this one waits for its stage.
        const int key0 = first0 + i * KT, page = next, at = it + i;
        const bool need = needed(i);
        next = needed(i + C::kTurns) ? __ldg(row + ((key0 + C::kTurns * KT) >> a.b.page_shift)) : -1;
        const bool good = need && page >= 0 && page < a.b.n_pages;
        if (need && !good) record_bad_index(a.status, kWherePage);
        const uint32_t bits = __ballot_sync(0xffffffffu, good);
        // All that can be is done before the stage is free, and the copies go ahead of the bytes announced for them (the
        // phase cannot end before this warp's arrival).
        const int s = at % C::kStages;
        const uint32_t dst = smem_u32(smem + s * C::kStageBytes) + kv * 16384 + (lane << p.box_shift) * C::kPanelRow;
        const uint32_t bytes = __popc(bits) * box_bytes;
        const int slot = key0 & ((1 << a.b.page_shift) - 1);
        const bool go = !s_abort;
        if (at >= C::kStages && !mbar_wait(empty + s, (at / C::kStages - 1) & 1, kFewWaitNs)) {
          fail(kWherePagedEmpty);
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok && go);
        if (!ok) break;
        if (good) {
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(dst + pn * C::kPanelBytes, map, full + s, pn * 64, h, slot, page);
        }
        if (lane == 0) {
          if (kv == 0) page_bits[s] = bits;
          mbar_arrive_expect_tx(full + s, bytes);
        }
        __syncwarp();
        issued = at + 1;
      }
      if (ok) it += n;
      wk.next(p, n);
    }
    if (!ok) {
      // Every copy issued has landed before the CTA ends.
      for (int j = max(0, issued - C::kStages); j < issued; ++j)
        if (j % C::kTurns == turn) mbar_wait(full + j % C::kStages, (j / C::kStages) & 1, kFewWaitNs);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // -------------------------------------------------------------------- consumers
  regs_inc<kFewRegsConsumer>();
  if (!wk.init(p)) return;
  const int g = lane >> 2, c = lane & 3;
  const int tid = threadIdx.x - 128, cw = warp - 4;   // among the consumers
  const int team = cw >> 2, kw0 = (cw & 3) * C::kWarpKeys;
  float* merge = reinterpret_cast<float*>(smem + C::kMergeOff);
  float* sm_m = reinterpret_cast<float*>(smem + C::kMlOff);   // [8][16]
  float* sm_l = sm_m + 8 * 16;
  float* q_exp = reinterpret_cast<float*>(smem + C::kScaleOff);
  // Row r of the unit (its sequence's first q row, K/V head, row tile): four channels of the output, its lse.
  auto store4 = [&](int start, int h, int qi, int r, int d, float inv, float v0, float v1, float v2, float v3) {
    const int rr = qi * R + r, tok = rr / p.group, hq = h * p.group + rr % p.group;
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(v1 * inv), "f"(v0 * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(v3 * inv), "f"(v2 * inv));
    *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(start + tok) * a.ost + static_cast<int64_t>(hq) * a.osh + d) = w;
  };
  auto store_lse = [&](int start, int h, int qi, int r, float mm, float ll) {
    const int rr = qi * R + r, tok = rr / p.group, hq = h * p.group + rr % p.group;
    a.lse[static_cast<int64_t>(start + tok) * a.hq + hq] = lse_of(mm, ll);
  };
  int it = 0;
  for (int seg = 0; wk.at < wk.end; ++seg) {
    const int n = wk.seg_tiles();
    const int h = wk.u / wk.w.qt * p.lock + col, qi = wk.u % wk.w.qt;
    const int buf = seg & 1;
    const uint32_t sq = smem_u32(smem + C::kQOff + buf * R * C::kQRow);
    if (!s_abort && !mbar_wait(q_full + buf, (seg >> 1) & 1, kFewWaitNs)) fail(kWherePagedFull);
    __syncwarp();   // after a timeout the tiles are skipped, the barriers below still met
    if (kE4M3) {
      // Q rows as fp16 times a power of two that brings the row's largest value into [1, 2): exact but
      // for values 2^-14 below it, which keep an absolute error of 2^-25 of the row's largest.
      __half* q16 = reinterpret_cast<__half*>(smem + C::kQOff + buf * R * C::kQRow);
#pragma unroll
      for (int rr = 0; rr < R / 8; ++rr) {
        const int r = cw * (R / 8) + rr;
        uint32_t* row = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(q16) + r * C::kQRow);
        uint32_t v[D / 64];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          v[i] = row[lane + 32 * i];
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(v[i] << 16)), fabsf(__uint_as_float(v[i] & 0xFFFF0000u))));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        int e = static_cast<int>((__float_as_uint(mx) >> 23) & 255) - 127;
        e = mx == 0.0f ? 0 : min(max(e, -126), 126);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const __half2 f = __floats2half2_rn(__uint_as_float(v[i] << 16) * down,
                                              __uint_as_float(v[i] & 0xFFFF0000u) * down);
          row[lane + 32 * i] = *reinterpret_cast<const uint32_t*>(&f);
        }
        if (lane == 0) q_exp[buf * R + r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
      consumer_sync();
    }
    // Per-row score factor (log2 units) and visible keys; rows past the last take the last one's.
    float sc[MT][2], m[MT][2];
    int klo[MT][2], khi[MT][2];
    const float scale = kE4M3 ? a.scale_log2 * __ldg(a.k_scale + h) : a.scale_log2;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + e * 8 + g;
        token_keys(a, wk.w, min(qi * R + r, wk.w.rows - 1) / p.group, klo[mt][e], khi[mt][e]);
        sc[mt][e] = kE4M3 ? scale * q_exp[buf * R + r] : scale;
        m[mt][e] = -INFINITY;
      }
    // Visible to all rows: [alo, ahi); to some: [ulo, uhi).
    int alo, ahi, ulo, uhi;
    token_keys(a, wk.w, qi * R / p.group, ulo, ahi);
    token_keys(a, wk.w, (min(qi * R + R, wk.w.rows) - 1) / p.group, alo, uhi);
    float o[MT][C::kOT][4], ol[MT][4];   // ol: the sums of P, every column alike
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      ol[mt][0] = ol[mt][1] = ol[mt][2] = ol[mt][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::kOT; ++i) o[mt][i][0] = o[mt][i][1] = o[mt][i][2] = o[mt][i][3] = 0.0f;
    }
    // Q fragments: in registers for one row tile, re-read from shared memory for two.
    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    auto load_q = [&](int mt, int kk, uint32_t f[4]) {
      if (!kE4M3) {
        ldsm4(f, sq + (mt * 16 + (lane & 15)) * C::kQRow + kk * 32 + (lane >> 4) * 16);
      } else {
        // Step kk takes channels 64 (kk / 4) + 16 c + 4 (kk % 4) + 0..3 of thread c, as the K codes below.
        const uint32_t off = (64 * (kk >> 2) + 16 * c + 4 * (kk & 3)) * 2;
        const uint2 x = lds64(sq + (mt * 16 + g) * C::kQRow + off), y = lds64(sq + (mt * 16 + g + 8) * C::kQRow + off);
        f[0] = x.x;
        f[1] = y.x;
        f[2] = x.y;
        f[3] = y.y;
      }
    };
    if (MT == 1)
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) load_q(0, kk, qf[kk]);

    for (int i = 0; i < n; ++i, ++it) {
      if ((it & 1) != team) continue;
      const int s = it % C::kStages;
      if (__any_sync(0xffffffffu, s_abort)) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(full + s, (it / C::kStages) & 1, kFewWaitNs))) {
        fail(kWherePagedFull);
        continue;
      }
      const uint32_t sk = smem_u32(smem + s * C::kStageBytes), sv = sk + 16384;
      const int kb = (wk.w.t_lo + wk.k + i) * KT;
      const uint32_t bits = page_bits[s];
      const bool whole = kb >= alo && kb + KT <= ahi && bits == (KT >> p.box_shift == 32 ? ~0u : (1u << (KT >> p.box_shift)) - 1u);
      // ---- scores
      float x[MT][C::kNT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int t = 0; t < C::kNT; ++t) x[mt][t][0] = x[mt][t][1] = x[mt][t][2] = x[mt][t][3] = 0.0f;
      if (!kE4M3) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t f[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (MT == 1) {
              f[0][0] = qf[kk][0]; f[0][1] = qf[kk][1]; f[0][2] = qf[kk][2]; f[0][3] = qf[kk][3];
            } else {
              load_q(mt, kk, f[mt]);
            }
          }
#pragma unroll
          for (int t2 = 0; t2 < C::kNT / 2; ++t2) {
            const int key = kw0 + t2 * 16 + (lane >> 4) * 8 + (lane & 7), ch = (kk & 3) * 2 + ((lane >> 3) & 1);
            uint32_t b[4];
            ldsm4(b, sk + (kk >> 2) * C::kPanelBytes + key * 128 + ((ch ^ (key & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<false>(x[mt][2 * t2], f[mt], b[0], b[1]);
              mma16816<false>(x[mt][2 * t2 + 1], f[mt], b[2], b[3]);
            }
          }
        }
      } else {
        // Column n of an 8-key tile is key (n >> 1) + 4 (n & 1): lanes of a quarter warp then read rows
        // whose swizzles differ in the upper chunk bit, without bank conflicts.
        const int kperm = (g >> 1) + 4 * (g & 1);
#pragma unroll
        for (int gr = 0; gr < D / 64; ++gr) {
          uint32_t f[MT][4][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              if (MT == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[0][st][e] = qf[gr * 4 + st][e];
              } else {
                load_q(mt, gr * 4 + st, f[mt][st]);
              }
            }
#pragma unroll
          for (int t = 0; t < C::kNT; ++t) {
            const int key = kw0 + t * 8 + kperm, ch = gr * 4 + c;
            const uint32_t ad = D == 128 ? sk + key * 128 + ((ch ^ (key & 7)) << 4)
                                         : sk + key * 64 + ((ch ^ ((key >> 1) & 3)) << 4);
            const uint4 v = lds128(ad);
            const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int st = 0; st < 4; ++st) {
              const uint32_t b0 = f16x2_of_e4m3(static_cast<uint16_t>(wd[st]));
              const uint32_t b1 = f16x2_of_e4m3(static_cast<uint16_t>(wd[st] >> 16));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<true>(x[mt][t], f[mt][st], b0, b1);
            }
          }
        }
      }
      // ---- online softmax, each row over its four lanes
      auto key_of = [&](int t, int j) { return kw0 + t * 8 + (kE4M3 ? c + 4 * j : 2 * c + j); };
      uint32_t seen_bits = ~0u;   // bit t * 2 + j: the key's box was loaded and some row sees it
      if (!whole) {
        seen_bits = 0;
#pragma unroll
        for (int t = 0; t < C::kNT; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int key = key_of(t, j);
            const bool in = ((bits >> (key >> p.box_shift)) & 1u) && kb + key >= ulo && kb + key < uhi;
            seen_bits |= (in ? 1u : 0u) << (t * 2 + j);
          }
      }
      // The maximum moves only when it rises by more than 2^8 (P stays below 2^8, or 2^15 where it is lifted; the ratio is
      // the same), so O is rarely rescaled.
      constexpr float kLift = kE4M3 ? kLiftE4M3 : 0.0f;
      bool rise = false;
      float al[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!whole) {
#pragma unroll
            for (int t = 0; t < C::kNT; ++t)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int key = kb + key_of(t, j);
                if (!((seen_bits >> (t * 2 + j)) & 1u) || key < klo[mt][e] || key >= khi[mt][e])
                  x[mt][t][e * 2 + j] = -INFINITY;
              }
          }
          float mx = fmaxf(x[mt][0][e * 2], x[mt][0][e * 2 + 1]);
#pragma unroll
          for (int t = 1; t < C::kNT; ++t) mx = fmax3(mx, x[mt][t][e * 2], x[mt][t][e * 2 + 1]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sc[mt][e];
          const bool up = mx > m[mt][e] + (kFewRise + kLift);   // also the first visible key
          const float lower = mx - kLift;
          al[mt][e] = up ? ex2_approx(m[mt][e] - lower) : 1.0f;
          rise |= up;
          if (up) m[mt][e] = lower;
          const float base = m[mt][e] == -INFINITY ? 0.0f : m[mt][e];   // no key so far: every p below is 0
#pragma unroll
          for (int t = 0; t < C::kNT; ++t) {
            const float p0 = ex2_approx(fmaf(x[mt][t][e * 2], sc[mt][e], -base));
            const float p1 = ex2_approx(fmaf(x[mt][t][e * 2 + 1], sc[mt][e], -base));
            uint32_t pk;   // P in the 16 bits that multiply V
            if (kE4M3)
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk) : "f"(p1), "f"(p0));
            else
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(pk) : "f"(p1), "f"(p0));
            x[mt][t][e * 2] = __uint_as_float(pk);
          }
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          ol[mt][0] *= al[mt][0];
          ol[mt][2] *= al[mt][1];
#pragma unroll
          for (int ot = 0; ot < C::kOT; ++ot) {
            o[mt][ot][0] *= al[mt][0];
            o[mt][ot][1] *= al[mt][0];
            o[mt][ot][2] *= al[mt][1];
            o[mt][ot][3] *= al[mt][1];
          }
        }
      }
      // ---- O += P V, 16 keys at a time
#pragma unroll
      for (int t2 = 0; t2 < C::kNT / 2; ++t2) {
        uint32_t pf[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          pf[mt][0] = __float_as_uint(x[mt][2 * t2][0]);
          pf[mt][1] = __float_as_uint(x[mt][2 * t2][2]);
          pf[mt][2] = __float_as_uint(x[mt][2 * t2 + 1][0]);
          pf[mt][3] = __float_as_uint(x[mt][2 * t2 + 1][2]);
        }
        // The sums: P times ones, so of the rounded P, and the weights add up to 1.
        constexpr uint32_t kOnes = kE4M3 ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mma16816<kE4M3>(ol[mt], pf[mt], kOnes, kOnes);
        // Keys that no row sees may hold anything: their V counts as 0.
        const uint32_t vis = seen_bits >> (t2 * 4);
        if (!kE4M3) {
          const uint32_t z0 = ((vis & 1u) ? 0xFFFFu : 0u) | ((vis & 2u) ? 0xFFFF0000u : 0u);
          const uint32_t z1 = ((vis & 4u) ? 0xFFFFu : 0u) | ((vis & 8u) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int d2 = 0; d2 < D / 16; ++d2) {
            const int key = kw0 + t2 * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), ch = (d2 & 3) * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4_t(b, sv + (d2 >> 2) * C::kPanelBytes + key * 128 + ((ch ^ (key & 7)) << 4));
            if (!whole) {
              b[0] &= z0;
              b[1] &= z1;
              b[2] &= z0;
              b[3] &= z1;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma16816<false>(o[mt][2 * d2], pf[mt], b[0], b[1]);
              mma16816<false>(o[mt][2 * d2 + 1], pf[mt], b[2], b[3]);
            }
          }
        } else {
          // Column n of O tile j is channel 16 u + j, u = (n >> 1) + 4 (n & 1) (D = 128), or 8 n + j.
          constexpr int kW = D / 32;   // 32-bit words of a row per lane: 4 or 2
          uint32_t wd[4][kW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = kw0 + (2 * t2 + (e >> 1)) * 8 + c + 4 * (e & 1);
            if (D == 128) {
              const int ch = (g >> 1) + 4 * (g & 1);
              const uint4 v = lds128(sv + key * 128 + ((ch ^ (key & 7)) << 4));
              wd[e][0] = v.x; wd[e][1] = v.y; wd[e][kW - 2] = v.z; wd[e][kW - 1] = v.w;
            } else {
              const uint2 v = lds64(sv + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
              wd[e][0] = v.x; wd[e][1] = v.y;
            }
            if (!whole && !((vis >> e) & 1u))
#pragma unroll
              for (int w = 0; w < kW; ++w) wd[e][w] = 0u;
          }
#pragma unroll
          for (int w = 0; w < kW; ++w) {
            const uint32_t a0 = __byte_perm(wd[0][w], wd[1][w], 0x5140), a1 = __byte_perm(wd[0][w], wd[1][w], 0x7362);
            const uint32_t b0 = __byte_perm(wd[2][w], wd[3][w], 0x5140), b1 = __byte_perm(wd[2][w], wd[3][w], 0x7362);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t sa = q < 2 ? a0 : a1, sb = q < 2 ? b0 : b1;
              const uint32_t f0 = f16x2_of_e4m3(static_cast<uint16_t>(sa >> (16 * (q & 1))));
              const uint32_t f1 = f16x2_of_e4m3(static_cast<uint16_t>(sb >> (16 * (q & 1))));
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816<true>(o[mt][w * 4 + q], pf[mt], f0, f1);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + s);
    }

    // ---- the eight warps' results joined
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty + buf);
    const bool whole_unit = wk.k == 0 && n == wk.w.nt;
    int cf = 0, parts = 1;
    if (!whole_unit) wk.unit_parts(p, cf, parts);
    const int slot = join_part_slot(blockIdx.x, 1, 0, wk.k == 0);   // row * lock + col is the CTA's number
    const int live = min(R, wk.w.rows - qi * R);        // rows of the tile that exist
    const float vs = kE4M3 ? __ldg(a.v_scale + h) : 1.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      // Each warp leaves its maxima, sums and O of 16 rows; the readers bring them to a common maximum.
      if (c == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sm_m[cw * 16 + e * 8 + g] = m[mt][e];
          sm_l[cw * 16 + e * 8 + g] = ol[mt][2 * e];
        }
      }
      float* mine = merge + cw * 16 * C::kMergeRow;
      if (!kE4M3) {
#pragma unroll
        for (int t = 0; t < C::kOT; ++t) {
          const float* v = o[mt][t];
          *reinterpret_cast<float2*>(mine + g * C::kMergeRow + t * 8 + 2 * c) = make_float2(v[0], v[1]);
          *reinterpret_cast<float2*>(mine + (g + 8) * C::kMergeRow + t * 8 + 2 * c) = make_float2(v[2], v[3]);
        }
      } else {
        // Columns 2 c and 2 c + 1 of O tile j are channels 16 c + j and kUp further: 64 (D = 128) or 8.
        constexpr int kUp = D == 128 ? 64 : 8;
        float* at = mine + g * C::kMergeRow + 16 * c;
#pragma unroll
        for (int j = 0; j < C::kOT; ++j) {
          at[j] = o[mt][j][0];
          at[kUp + j] = o[mt][j][1];
          at[8 * C::kMergeRow + j] = o[mt][j][2];
          at[8 * C::kMergeRow + kUp + j] = o[mt][j][3];
        }
      }
      consumer_sync();
      const int r16 = tid >> 4, r = mt * 16 + r16;
      if (r < live) {
        float f[8], mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) mm = fmaxf(mm, sm_m[w * 16 + r16]);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          f[w] = mm == -INFINITY ? 0.0f : ex2_approx(sm_m[w * 16 + r16] - mm);
          ll = fmaf(sm_l[w * 16 + r16], f[w], ll);
        }
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          const int d4 = half * 64 + (tid & 15) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < 8; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(merge + (w * 16 + r16) * C::kMergeRow + d4);
            v.x = fmaf(y.x, f[w], v.x);
            v.y = fmaf(y.y, f[w], v.y);
            v.z = fmaf(y.z, f[w], v.z);
            v.w = fmaf(y.w, f[w], v.w);
          }
          if (whole_unit) {
            store4(wk.w.start, h, qi, r, d4, ll > 0.0f ? vs / ll : ll, v.x, v.y, v.z, v.w);
            if (a.lse && d4 == 0) store_lse(wk.w.start, h, qi, r, mm, ll);
          } else {
            *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * R + r) * D + d4) = v;
            if (d4 == 0) a.part_ml[slot * R + r] = make_float2(mm, ll);
          }
        }
      }
      consumer_sync();
    }
    if (!whole_unit) {
      // The loop above ended with the CTA's barrier: thread 0's release covers every thread's stores.  Whether the part
      // was the last is looked at when the CTA's tiles are done, so its next unit does not wait for the ticket.
      if (tid == 0) {
        // More than 16 parts (one sequence with few K/V heads over many SMs) are joined in groups first.
        const int groups = join_groups(parts), gr = join_group_of(parts, groups, static_cast<int>(blockIdx.x) / p.lock - cf);
        const int first = join_first(parts, groups, gr);
        Pending& d = s_pending[wk.k == 0 ? 1 : 0];
        d.counter = join_counter(cf + first, p.lock, col);
        d.first = first;
        d.count = join_first(parts, groups, gr + 1) - first;
        d.cf = cf;
        d.parts = parts;
        d.start = wk.w.start;
        d.rows = wk.w.rows;
        d.h = h;
        d.qi = qi;
        s_last[wk.k == 0 ? 1 : 0] = draw_ticket(a.counters + d.counter, d.count);
      }
    }
    wk.next(p, n);
  }

  // ---- units whose last part was this CTA's: the parts joined in the order of their keys
#pragma unroll 1
  for (int d = 0; d < 2; ++d) {
    consumer_sync();
    if (!s_last[d]) continue;
    const Pending& e = s_pending[d];
    const int cf = e.cf, parts = e.parts, live = min(R, e.rows - e.qi * R);
    const float vs = kE4M3 ? __ldg(a.v_scale + e.h) : 1.0f;
    // Parts slot_of(0) .. slot_of(count - 1) into `to`, or the output where `to` is negative.
    auto join = [&](int count, auto slot_of, int to) {
      constexpr int kAhead = 4;   // parts whose loads are in flight together
      for (int i = tid; i < live * (D / 4); i += kFewConsumers) {
        const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
        float mm = -INFINITY, ll = 0.0f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int q0 = 0; q0 < count; q0 += kAhead) {
          float2 ml[kAhead];
          float4 x[kAhead];
#pragma unroll
          for (int q = 0; q < kAhead; ++q) {
            ml[q] = make_float2(-INFINITY, 0.0f);
            x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q0 + q < count) {
              const int sl = slot_of(q0 + q);
              ml[q] = __ldcg(a.part_ml + sl * R + r);
              x[q] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (static_cast<int64_t>(sl) * R + r) * D + d4));
            }
          }
#pragma unroll
          for (int q = 0; q < kAhead; ++q) {
            // No key so far: both factors are 0, and what is added is 0, or NaN where a part's scores are no numbers.
            const float mn = fmaxf(mm, ml[q].x), base = mn == -INFINITY ? 0.0f : mn;
            const float f0 = ex2_approx(mm - base), f1 = ex2_approx(ml[q].x - base);
            ll = ll * f0 + ml[q].y * f1;
            v.x = v.x * f0 + x[q].x * f1;
            v.y = v.y * f0 + x[q].y * f1;
            v.z = v.z * f0 + x[q].z * f1;
            v.w = v.w * f0 + x[q].w * f1;
            mm = mn;
          }
        }
        if (to >= 0) {
          *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(to) * R + r) * D + d4) = v;
          if (d4 == 0) a.part_ml[to * R + r] = make_float2(mm, ll);
        } else {
          store4(e.start, e.h, e.qi, r, d4, ll > 0.0f ? vs / ll : ll, v.x, v.y, v.z, v.w);
          if (a.lse && d4 == 0) store_lse(e.start, e.h, e.qi, r, mm, ll);
        }
      }
    };
    auto part_slot = [&](int q) { return join_part_slot(cf + q, p.lock, col, q == 0); };
    const int groups = join_groups(parts);
    if (groups == 1) {
      join(parts, part_slot, -1);
    } else {
      // The group's parts into a slot of the group's; then, if that was the last group, the groups.
      const int first = e.first;
      join(e.count, [&](int q) { return part_slot(first + q); }, join_group_slot(cf + first, p.lock, col));
      consumer_sync();
      if (tid == 0) s_last[d] = draw_ticket(a.counters + join_unit_counter(cf, p.lock, col), groups);
      consumer_sync();
      if (s_last[d]) join(groups, [&](int q) { return join_group_slot(cf + join_first(parts, groups, q), p.lock, col); }, -1);
    }
  }
}

template <int D, bool kE4M3, int MT>
cudaError_t launch_t(const PagedAttnArgs& a, const sage_paged_kv& kv, cudaStream_t s) {
  using C = FewCfg<D, kE4M3, MT>;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(paged_few_kernel<D, kE4M3, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (err != cudaSuccess) return err;
  const int grid = std::min(sms, kFewMaxCtas);
  FewParams p;
  p.a = a;
  p.group = a.hq / a.hkv;
  // K/V heads that CTAs take side by side, the same keys at the same time: their rows lie together in a page, and DRAM is
  // read in runs of up to 2 KB (single tokens, E4M3, 24 heads of 64 channels: 191 us against 308 with a head to a CTA's
  // turn; bf16, 8 heads of 128: 328 against 343).  At most 1 CTA in 25 may be left over.
  const int want = 2048 / C::kRowBytes;
  p.lock = 1;
  for (int g = 2; g <= a.hkv && p.lock < want; ++g)
    if (a.hkv % g == 0 && g <= grid && (grid / g) * g * 25 >= grid * 24) p.lock = g;
  p.box_shift = a.b.page_shift;
  while ((1 << p.box_shift) > C::kKeys) --p.box_shift;
  const int64_t e = kE4M3 ? 1 : 2;
  CUtensorMap kmap, vmap;
  if (!make_page_map(&kmap, kv.k_pages, kE4M3, D, kv.n_heads, kv.page_size, kv.n_pages, kv.k_stride_head * e,
                     kv.k_stride_token * e, kv.k_stride_page * e, C::kPanelRow / int(e), 1 << p.box_shift) ||
      !make_page_map(&vmap, kv.v_pages, kE4M3, D, kv.n_heads, kv.page_size, kv.n_pages, kv.v_stride_head * e,
                     kv.v_stride_token * e, kv.v_stride_page * e, C::kPanelRow / int(e), 1 << p.box_shift))
    return cudaErrorInvalidValue;
  return launch_dependent(true, paged_few_kernel<D, kE4M3, MT>, dim3(grid / p.lock * p.lock), dim3(kFewThreads), C::kSmem,
                          s, kmap, vmap, p);
}

template <int D, bool kE4M3>
cudaError_t launch_rows(const PagedAttnArgs& a, const sage_paged_kv& kv, cudaStream_t s) {
  // Two row tiles where the batch's mean rows per sequence need more than one: K and V are then read
  // once for 32 rows.
  const int64_t rows = static_cast<int64_t>(a.b.n_tokens) * (a.hq / a.hkv);
  return rows > 16 * static_cast<int64_t>(a.b.n_seqs) ? launch_t<D, kE4M3, 2>(a, kv, s) : launch_t<D, kE4M3, 1>(a, kv, s);
}

}  // namespace

cudaError_t launch_paged_few(const PagedAttnArgs& a, const sage_paged_kv& c, int d, cudaStream_t s) {
  if (d == 128) return c.format == 1 ? launch_rows<128, true>(a, c, s) : launch_rows<128, false>(a, c, s);
  return c.format == 1 ? launch_rows<64, true>(a, c, s) : launch_rows<64, false>(a, c, s);
}

}  // namespace sage
