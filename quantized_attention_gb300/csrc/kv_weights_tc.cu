// The attention weight each cached row has received (kv_weights.cu has the
// formula), for many query rows: S^T = K Q^T on the 5th-generation tensor cores.
//
// A CTA works through units of 256 keys of one (sequence, KV head), two M = 128
// tiles, against the group's query rows (query head, token) in N = 128 tiles.
// Key = TMEM lane, so a key's sum over queries is a sum along one thread's
// columns: no shuffle, no atomic, a fixed order.  Both operands are codes,
// converted once per unit (K) or tile (Q) to exact fp16; S is an exact integer.
//
//   warp 0       TMA: the units' K codes into a ring of two raw stages
//   warps 1-2    the MMAs of the two M tiles, a thread each (one thread's waits and
//                commits left the tensor pipe idle); warp 1 owns TMEM
//   warps 4-7    K codes -> fp16 A operand in TMEM (lane = key)
//   warps 8-11   Q codes -> fp16 B tiles in shared memory, their rows' factors
//   warps 12-19  p = 2^(S c - lse2) summed along the columns; one thread a key
//
// K sits in TMEM as the A operand because shared memory feeds everything else:
// per Q tile and SM the two MMAs read 64 KB of B, the producers write 32 KB and
// the column constants take 8-16 KB of broadcasts, against ~1030 cycles of
// tensor work and as many of MUFU (one ex2 a score).  Measured: ~2000 cycles a Q tile,
// the whole 8K prefill 278 us (floor 145: 49% of the measured bf16 rate); without the
// exponentials or without the MMAs it is ~250, the summing warps' chain (wait, TMEM
// loads, 290 instructions) being what is left.  With up to kQS tiles of
// queries and consecutive units of one head, the Q tiles stay where they are and
// the kernel streams K.
#include <algorithm>
#include <type_traits>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

constexpr float kLog2e = 1.44269502162933349609375f;  // fp32(log2 e)
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kUnit = 256;    // keys of a unit
constexpr int kTileQ = 128;   // query rows of a tile
constexpr int kQS = 4;        // Q stages
constexpr int kNS = 3;        // S slots (128 TMEM columns each)
static_assert(kNS == 3, "the slots' order is written out for three");
constexpr int kThreads = 640;
constexpr uint32_t kTmemS = 128;  // first column of the S slots; A sits below

template <int D>
struct Cfg {
  static constexpr int kRaw = kUnit * D;              // a unit's K codes
  static constexpr int kQTile = kTileQ * D * 2;       // D / 64 blocks of [128][128 B]
  static constexpr int kOffQ = 2 * kRaw;
  static constexpr int kOffF = kOffQ + kQS * kQTile;  // per stage: c, -lse2, last key [128] each
  static constexpr int kFac = 3 * kTileQ * 4;
  static constexpr int kOffBar = kOffF + kQS * kFac;
  static constexpr int kBytes = kOffBar + 512 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

// Item n of the S ring (slot n % kNS) is M tile n % 2 of Q tile n / 2.  The slots'
// barriers are kept per M tile: the two tiles' threads drift apart, and on a shared
// barrier a thread could look for a completion two phases away, which a parity
// cannot tell from none.  M tile m uses a slot every third item of its own.
enum {
  kRawFull = 0,   // [2] TMA bytes
  kRawEmpty = 2,  // [2] 128 producer threads
  kAFull = 4,     // [2 M tiles] 128 producer threads
  kAEmpty = 6,    // [2 M tiles] the unit's MMAs on it are done
  kQFull = 8,     // [kQS] 128 producer threads
  kQEmpty = 12,   // [kQS] the MMAs of both M tiles, and the 256 threads that read its constants
  kSFull = 16,    // [2 M tiles][kNS] an MMA's commit
  kSEmpty = 22,   // [2 M tiles][kNS] 128 threads
  kDrain = 28,    // [2] an issuing thread's MMAs are done
  kNumBars = 30
};

// What every role walks through in the same order: this CTA's units, and the
// tiles of a unit.  Fewer than 128 tokens a head: the group's rows are packed
// into tiles regardless of the head; else a tile is 128 tokens of one head
// (aligned to the scale blocks), and a causal unit starts each head at the tile
// of the first token that sees its first key.
struct Tiling {
  bool packed;
  int heads, per_head;  // heads a unit walks through, tiles of one
};
struct Tile {
  int h, c;
};

__device__ __forceinline__ int row_count(const WeightArgs& a, int b) {
  if (!a.lengths) return a.Nk;
  if (!QATTN_IN_BOUNDS(b >= 0 && b < a.B)) return 0;
  const int n = a.lengths[b];
  if (n < 0 || n > a.Nk) {
    atomicOr(a.err, kErrDomain);
    return n < 0 ? 0 : a.Nk;
  }
  return n;
}

// nbh: (batch, head) pairs of the scales
__device__ __forceinline__ float scale_of(const float* s, int gran, int bh, int nbh, int nblk, int blk) {
  if (gran == 0) return s[0];
  if (!QATTN_IN_BOUNDS(bh < nbh && (gran == 1 || (blk >= 0 && blk < nblk)))) return 0.f;
  if (gran == 1) return s[bh];
  return s[static_cast<size_t>(bh) * nblk + blk];
}

// This CTA's units.  Few tiles a unit (Q stays): equal runs of the units that the
// lengths give, one head after the other; `first` is where the run begins.
// Many: the units ordered by key block, the first blocks (the longest, when
// causal) first, dealt back and forth over the CTAs.
struct Run {
  int b, head, kb, count;  // sequence, KV head and key block of the first unit; units
};

__device__ __forceinline__ int key_blocks(int len) { return (len + kUnit - 1) / kUnit; }

// One warp: the run of CTA blockIdx.x.
__device__ __forceinline__ void find_run(const WeightArgs& a, Run* run) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  for (int b = lane; b < a.B; b += 32) total += static_cast<long long>(a.Hkv) * key_blocks(row_count(a, b));
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) total += __shfl_xor_sync(0xffffffffu, total, sh);
  const long long begin = blockIdx.x * total / gridDim.x, end = (blockIdx.x + 1) * total / gridDim.x;
  Run r{0, 0, 0, static_cast<int>(end - begin)};
  long long before = 0;
  for (int b0 = 0; b0 < a.B && r.count > 0; b0 += 32) {
    const int kb = b0 + lane < a.B ? key_blocks(row_count(a, b0 + lane)) : 0;
    const long long n = static_cast<long long>(a.Hkv) * kb;
    long long inc = n;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, sh);
      if (lane >= sh) inc += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + inc > begin);
    if (past) {
      const int w = __ffs(past) - 1;
      const int off = static_cast<int>(begin - before - __shfl_sync(0xffffffffu, inc - n, w));
      const int blocks = __shfl_sync(0xffffffffu, kb, w);
      r.b = b0 + w;
      r.head = off / blocks;
      r.kb = off % blocks;
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) *run = r;
}

struct Walk {
  int b, hkv, bkv, k0, len, pos0;
  int first;  // first tile of a head
  bool stay;  // the unit's Q tiles stay for the unit after it
  // position
  int n, count, kb, blocks;
  bool runs;
};

__device__ __forceinline__ int first_tile(const WeightArgs& a, const Tiling& til, const Walk& w, int k0) {
  const int i = a.causal ? max(0, k0 - w.pos0) : 0;
  return til.packed ? (i < a.Nq ? 0 : til.per_head) : min(i / kTileQ, til.per_head);
}

__device__ __forceinline__ void set_sequence(const WeightArgs& a, Walk& w, int b) {
  w.b = b;
  w.len = row_count(a, b);
  w.pos0 = a.pos0_len ? w.len - a.Nq : a.pos0;
  w.blocks = key_blocks(w.len);
}

__device__ __forceinline__ Walk walk_begin(const WeightArgs& a, const Run& run, bool runs) {
  Walk w;
  w.runs = runs;
  w.n = -1;
  w.count = run.count;
  w.kb = run.kb - 1;
  w.hkv = run.head;
  if (runs) set_sequence(a, w, run.b);
  return w;
}

// The next unit of this CTA; false after the last.
__device__ __forceinline__ bool walk_next(const WeightArgs& a, const Tiling& til, int most_blocks, Walk& w) {
  if (w.runs) {
    if (++w.n >= w.count) return false;
    if (++w.kb >= w.blocks) {  // the next head, the next sequence with rows
      w.kb = 0;
      if (++w.hkv == a.Hkv) {
        w.hkv = 0;
        do set_sequence(a, w, w.b + 1);
        while (w.blocks == 0);
      }
    }
    w.bkv = w.b * a.Hkv + w.hkv;
    w.k0 = w.kb * kUnit;
    w.first = first_tile(a, til, w, w.k0);
    w.stay = w.n + 1 < w.count && w.kb + 1 < w.blocks && w.first == 0 &&
             first_tile(a, til, w, w.k0 + kUnit) == 0;
    return true;
  }
  const int G = gridDim.x, c = blockIdx.x, heads = a.B * a.Hkv, units = most_blocks * heads;
  w.stay = false;
  for (;;) {
    ++w.n;
    const long long u = static_cast<long long>(w.n) * G + ((w.n & 1) ? G - 1 - c : c);
    if (w.n > units / G) return false;
    if (u >= units) continue;
    w.bkv = static_cast<int>(u % heads);
    w.k0 = static_cast<int>(u / heads) * kUnit;
    w.hkv = w.bkv % a.Hkv;
    set_sequence(a, w, w.bkv / a.Hkv);
    if (w.k0 >= w.len) continue;
    w.first = first_tile(a, til, w, w.k0);
    return true;
  }
}

__device__ __forceinline__ bool more(const Tiling& til, const Walk& w, const Tile& t) {
  return t.h < til.heads && w.first < til.per_head;
}
__device__ __forceinline__ void next(const Tiling& til, const Walk& w, Tile& t) {
  if (++t.c == til.per_head) {
    t.c = w.first;
    ++t.h;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_tc_kernel(const __grid_constant__ CUtensorMap tmK, const WeightArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Run run_s;
  pdl_trigger();
  const uint32_t raw0 = smem_u32(raw_smem);
  const uint32_t base = (raw0 + 1023u) & ~1023u;
  uint8_t* smem = raw_smem + (base - raw0);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + 8 * kNumBars + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto wait = [&](int i, uint32_t n) {  // the n-th completion (from 0) of barrier i
    return mbar_wait_fast(bar(i), n & 1, abort_flag, a.err, kErrTimeout);
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = a.G * a.Nq;
  Tiling til;
  til.packed = a.Nq < kTileQ;
  til.heads = til.packed ? 1 : a.G;
  til.per_head = ((til.packed ? R : a.Nq) + kTileQ - 1) / kTileQ;
  const int ntile = til.heads * til.per_head;
  const int most_blocks = key_blocks(a.Nk);
  const bool runs = ntile <= kQS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= kRawEmpty && i < kRawEmpty + 2) || (i >= kAFull && i < kAFull + 2) || (i >= kQFull && i < kQFull + kQS) ||
          (i >= kSEmpty && i < kSEmpty + 2 * kNS))
        n = 128;
      if (i >= kQEmpty && i < kQEmpty + kQS) n = 258;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (runs) {
    if (warp == 0) find_run(a, &run_s);
    __syncthreads();
  }
  Walk w = walk_begin(a, run_s, runs);
  auto take = [&]() { return walk_next(a, til, most_blocks, w); };

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      bool ok = true;
      uint32_t cnt = 0;
      for (; ok && take(); ++cnt) {
        const int st = cnt & 1;
        if (cnt >= 2 && !(ok = wait(kRawEmpty + st, (cnt >> 1) - 1))) break;
        (void)QATTN_IN_BOUNDS(w.k0 < a.Nk && w.bkv < a.B * a.Hkv);  // TMA coordinates
        mbar_arrive_expect_tx(bar(kRawFull + st), C::kRaw);
        for (int m = 0; m < 2; ++m)
          tma_load_3d(base + st * C::kRaw + m * (C::kRaw / 2), &tmK, bar(kRawFull + st), 0, w.k0 + 128 * m, w.bkv);
      }
      // every load this thread issued lands before the CTA may exit
      volatile int never = 0;
      for (uint32_t back = 1; back <= 2; ++back)
        if (cnt >= back)
          mbar_wait(bar(kRawFull + ((cnt - back) & 1)), ((cnt - back) >> 1) & 1, &never, a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp < 3) {
    if (lane == 0) {
      const int m = warp - 1;
      constexpr uint32_t idesc = make_idesc(128, kTileQ, 0, 0);  // F16 x F16 -> F32
      const uint64_t desc0 = smem_desc(base + C::kOffQ, 1024, kSwizzle128B);
      const uint32_t acol = tmem + m * (D / 2);
      bool ok = true, kept = false;
      uint32_t cnt = 0, qn = 0;  // units, Q tiles released
      // this tile's items are every other one of the S ring: the slot, and which of the
      // other tile's releases of it to wait for (item n - 3 is the other tile's: none
      // for the first 2 - m items).  Counted, not divided
      int slot = m, idle = 2 - m, lap = 0, third = 0;
      for (; ok && take(); ++cnt) {
        const bool stay = w.stay;
        uint32_t q = qn;
        if (!(ok = wait(kAFull + m, cnt))) break;
        for (Tile t{0, w.first}; more(til, w, t); ++q) {
          const int st = q % kQS;
          if (!kept && !(ok = wait(kQFull + st, q / kQS))) break;
          if (idle > 0) {
            --idle;
          } else {
            if (!(ok = wait(kSEmpty + kNS * (1 - m) + slot, lap))) break;
            if (++third == 3) {
              third = 0;
              ++lap;
            }
          }
          next(til, w, t);
          tc_fence_after();
          // descriptors step by constants from the stage's first one
          const uint64_t bd = desc0 + static_cast<uint32_t>(st * (C::kQTile >> 4));
          const uint32_t dcol = tmem + kTmemS + 128 * slot;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_f16_ts(dcol, acol + 8 * k, bd + ((k / 4) * (kTileQ * 128) + 32 * (k % 4)) / 16, idesc,
                       k > 0 ? 1u : 0u);
          mma_commit(bar(kSFull + kNS * m + slot));
          if (!stay) mma_commit(bar(kQEmpty + st));
          slot += slot == 0 ? 2 : -1;  // (slot + 2) % 3
        }
        if (!ok) break;
        mma_commit(bar(kAEmpty + m));
        if (!stay) qn = q;
        kept = stay;
      }
      mma_commit(bar(kDrain + m));
      volatile int never = 0;
      mbar_wait(bar(kDrain + m), 0, &never, a.err, kErrTimeout);
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------- K codes -> A in TMEM
    const int quad = warp & 3;
    bool ok = true;
    uint32_t cnt = 0;
    for (; ok && take(); ++cnt) {
      const int st = cnt & 1;
      ok = wait(kRawFull + st, cnt >> 1);
      if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {
        const int r = quad * 32 + lane;
        const uint32_t src = base + st * C::kRaw + m * (C::kRaw / 2) + r * D;
        uint32_t x[D / 64][32];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = lds128(src + 16 * (c ^ ((D == 128) ? (r & 7) : ((r >> 1) & 3))));
          uint32_t* o = &x[c / 4][8 * (c % 4)];
          codes4_to_f16x2(v.x, o[0], o[1]);
          codes4_to_f16x2(v.y, o[2], o[3]);
          codes4_to_f16x2(v.z, o[4], o[5]);
          codes4_to_f16x2(v.w, o[6], o[7]);
        }
        if (m == 1) mbar_arrive(bar(kRawEmpty + st));
        ok = cnt == 0 || wait(kAEmpty + m, cnt - 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
          tmem_st32(tmem + (static_cast<uint32_t>(quad * 32) << 16) + m * (D / 2) + 32 * e, x[e]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kAFull + m));
      }
      if (!ok) break;
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 8 && warp < 12) {
    // ---------------------------------------------------- Q codes -> B tiles
    // Thread: 16-byte chunk cc of column block cb of rows rw, rw + 128 / RS, ...;
    // eight lanes of a store (four chunks of two rows) hit eight bank groups.
    constexpr int NB = D / 64, RS = 32 / NB;  // column blocks; rows 128 threads cover at once
    constexpr int CH = kTileQ / RS;           // rows of a thread
    const int tid = threadIdx.x - 256;
    const int cc = tid & 3, rw = ((tid >> 2) & 1) | ((tid >> (3 + NB - 1)) << 1), cb = NB == 2 ? (tid >> 3) & 1 : 0;
    const int nqb = (a.Nq + 127) / 128;
    bool ok = true, kept = false;
    uint32_t qn = 0;
    while (ok && take()) {
      const bool stay = w.stay;
      uint32_t q = qn;
      if (!kept) {
        const size_t row0 = (static_cast<size_t>(w.b) * a.Hq + w.hkv * a.G) * a.Nq;
        const size_t rows_total = static_cast<size_t>(a.B) * a.Hq * a.Nq;
        uint4 v[CH];
        float s_next = 0.f, e_next = kNegInf;
        int i_next = 0;
        auto fetch = [&](const Tile& t) {
          const int r0 = t.h * a.Nq + t.c * kTileQ;
          const int n_rows = min(kTileQ, (til.packed ? R : a.Nq) - t.c * kTileQ);
          const uint4* src = reinterpret_cast<const uint4*>(a.q_codes + (row0 + r0 + rw) * D + 64 * cb + 16 * cc);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rw + RS * i < n_rows && QATTN_IN_BOUNDS(row0 + r0 + rw + RS * i < rows_total))
              v[i] = src[RS * i * (D / 16)];
          }
          s_next = 0.f;
          e_next = kNegInf;
          if (tid < n_rows && QATTN_IN_BOUNDS(row0 + r0 + tid < rows_total)) {
            const int hq = til.packed ? (r0 + tid) / a.Nq : t.h;
            i_next = r0 + tid - hq * a.Nq;
            s_next = scale_of(a.q_scales, a.q_gran, w.b * a.Hq + w.hkv * a.G + hq, a.B * a.Hq, nqb, i_next / 128);
            e_next = a.lse[row0 + r0 + tid];
          }
        };
        Tile t{0, w.first};
        if (more(til, w, t)) fetch(t);
        for (; more(til, w, t); ++q) {
          const int st = q % kQS;
          if (q >= static_cast<uint32_t>(kQS)) {
            ok = wait(kQEmpty + st, q / kQS - 1);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
          }
          const uint32_t dst = base + C::kOffQ + st * C::kQTile + cb * (kTileQ * 128) + rw * 128;
          const uint32_t c0 = ((2 * cc) ^ (rw & 7)) << 4, c1 = ((2 * cc + 1) ^ (rw & 7)) << 4;  // RS is a multiple of 8
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            uint32_t h[8];
            codes4_to_f16x2(v[i].x, h[0], h[1]);
            codes4_to_f16x2(v[i].y, h[2], h[3]);
            codes4_to_f16x2(v[i].z, h[4], h[5]);
            codes4_to_f16x2(v[i].w, h[6], h[7]);
            sts128(dst + RS * 128 * i + c0, h[0], h[1], h[2], h[3]);
            sts128(dst + RS * 128 * i + c1, h[4], h[5], h[6], h[7]);
          }
          // row tid's constants: {factor sq sm log2 e, -lse2, last visible key}; a row
          // past the end, or one that saw nothing, gives 2^-inf = 0
          float* fac = reinterpret_cast<float*>(smem + C::kOffF + st * C::kFac);
          fac[tid] = weight_factor(s_next, a.sm_scale, e_next);
          fac[128 + tid] = e_next == kNegInf ? kNegInf : -e_next * kLog2e;
          reinterpret_cast<int*>(fac)[256 + tid] = a.causal ? w.pos0 + i_next : 0x7fffffff;
          fence_proxy_async_smem();
          mbar_arrive(bar(kQFull + st));
          next(til, w, t);
          if (more(til, w, t)) fetch(t);
        }
      }
      if (!ok) break;
      if (!stay) qn = kept ? qn + ntile : q;
      kept = stay;
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 12) {
    // ---------------------------------------------------- sums along the columns
    const int m = (warp - 12) >> 2, quad = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int nkb = (a.Nk + 127) / 128;
    // one factor for a tile: its rows share a scale
    const bool one = !til.packed || a.q_gran == 0 || a.G == 1;
    bool ok = true;
    uint32_t qn = 0;
    bool ahead = false;
    float old_next = 0.f, sk_next = 1.f;
    int slot = m, lap = 0, third = 0;  // this half's items are every other one of the S ring
    while (ok && take()) {
      const bool stay = w.stay;
      const int key = w.k0 + 128 * m + quad * 32 + lane;
      const size_t o = static_cast<size_t>(w.bkv) * a.cap + key;
      const bool live = key < w.len;
      auto base_of = [&](int k) {
        if (k >= w.len || !a.base || !QATTN_IN_BOUNDS(k < a.cap)) return 0.f;
        return a.base[static_cast<size_t>(w.bkv) * a.cap + k];
      };
      auto key_scale = [&](int k0) {
        return a.k_scales ? scale_of(a.k_scales, a.k_gran, w.bkv, a.B * a.Hkv, nkb, min(k0 / 128 + m, nkb - 1)) : 1.f;
      };
      // base and scale of a unit that follows in the same head come a unit ahead: their
      // latency would stand before every unit's first column
      const float old = ahead ? old_next : base_of(key), sk = ahead ? sk_next : key_scale(w.k0);
      ahead = w.runs && w.n + 1 < w.count && w.kb + 1 < w.blocks;
      if (ahead) {
        old_next = base_of(key + kUnit);
        sk_next = key_scale(w.k0 + kUnit);
      }
      const float2 sk2 = make_float2(sk, sk);
      float total = 0.f;
      uint32_t q = qn;
      for (Tile t{0, w.first}; more(til, w, t); next(til, w, t), ++q) {
        const int st = q % kQS;
        ok = wait(kQFull + st, q / kQS) && wait(kSFull + kNS * m + slot, lap);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float* fac = reinterpret_cast<const float*>(smem + C::kOffF + st * C::kFac);
        const float* nl = fac + 128;
        const int* last = reinterpret_cast<const int*>(fac) + 256;
        // every key of this M tile visible to every row of the tile
        const bool all = !a.causal || w.k0 + 128 * m + 127 <= w.pos0 + (til.packed ? 0 : t.c * kTileQ);
        float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
        const uint32_t src = tmem + lane_base + kTmemS + 128 * slot;
        const float c0 = fac[0] * sk;
        // 32 columns; ONE: one factor for the tile, ALL: no key hidden from any row
        auto sum32 = [&](auto one_c, auto all_c, const uint32_t (&v)[32], int j) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 c01 = make_float2(c0, c0), c23 = c01;
            if constexpr (!one_c.value) {
              const float4 c4 = *reinterpret_cast<const float4*>(fac + 32 * j + e);
              c01 = fmul2(make_float2(c4.x, c4.y), sk2);
              c23 = fmul2(make_float2(c4.z, c4.w), sk2);
            }
            const float4 l4 = *reinterpret_cast<const float4*>(nl + 32 * j + e);
            float2 t0 = ffma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c01,
                              make_float2(l4.x, l4.y));
            float2 t1 = ffma2(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), c23,
                              make_float2(l4.z, l4.w));
            if constexpr (!all_c.value) {
              const int4 k4 = *reinterpret_cast<const int4*>(last + 32 * j + e);
              t0 = make_float2(key <= k4.x ? t0.x : kNegInf, key <= k4.y ? t0.y : kNegInf);
              t1 = make_float2(key <= k4.z ? t1.x : kNegInf, key <= k4.w ? t1.y : kNegInf);
            }
            s0 = fadd2(s0, make_float2(ex2_approx(t0.x), ex2_approx(t0.y)));
            s1 = fadd2(s1, make_float2(ex2_approx(t1.x), ex2_approx(t1.y)));
          }
        };
        auto tile = [&](auto one_c, auto all_c) {
          // the next 32 columns load while these compute
          uint32_t va[32], vb[32];
          tmem_ld32(src, va);
          tmem_wait_ld();
          tmem_ld32(src + 32, vb);
          sum32(one_c, all_c, va, 0);
          tmem_wait_ld();
          tmem_ld32(src + 64, va);
          sum32(one_c, all_c, vb, 1);
          tmem_wait_ld();
          tmem_ld32(src + 96, vb);
          sum32(one_c, all_c, va, 2);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(bar(kSEmpty + kNS * m + slot));
          sum32(one_c, all_c, vb, 3);
        };
        if (all) {
          if (one) tile(std::true_type{}, std::true_type{});
          else tile(std::false_type{}, std::true_type{});
        } else {  // (a tile or two of a unit)
#pragma unroll 1
          for (int j = 0; j < kTileQ / 32; ++j) {
            uint32_t v[32];
            tmem_ld32(src + 32 * j, v);
            tmem_wait_ld();
            if (j == kTileQ / 32 - 1) {
              tc_fence_before();
              mbar_arrive(bar(kSEmpty + kNS * m + slot));
            }
            sum32(std::false_type{}, std::false_type{}, v, j);
          }
        }
        slot += slot == 0 ? 2 : -1;  // (slot + 2) % 3
        if (++third == 3) {
          third = 0;
          ++lap;
        }
        total += (s0.x + s0.y) + (s1.x + s1.y);
        if (!stay) mbar_arrive(bar(kQEmpty + st));
      }
      if (!ok) break;
      if (live && QATTN_IN_BOUNDS(key < a.cap)) a.weights[o] = old + total;
      if (!stay) qn = q;
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const WeightArgs& a, cudaStream_t s) {
  constexpr int smem = Cfg<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kv_weights_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>((a.Nk + kUnit - 1) / kUnit) * a.B * a.Hkv;
  const int grid = static_cast<int>(std::min<long long>(num_sms(), units));
  return launch_pdl(kv_weights_tc_kernel<D>, dim3(grid), dim3(kThreads), smem, s, tk, a);
}

}  // namespace

unsigned int check_take_kv_weights_tc() { return check_take_local(); }

cudaError_t launch_kv_weights_tc(const CUtensorMap& tk, const WeightArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(tk, a, s) : launch_d<128>(tk, a, s);
}

}  // namespace qattn
