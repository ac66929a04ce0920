// Attention over a paged 8-bit KV cache (qattn_paged_fwd), for many query rows of a KV head
// (kPagedFewRows): on the 5th-generation tensor cores.  Mathematics as in paged_warp.cu.
//
// A CTA works on a block of 256 query rows (two tiles of 128) in steps of 128 keys:
//   warp 0       issues the MMAs (d = 64: warps 0 and 1, a tile each)
//   warp 2       walks the share: its segments go to the others through shared memory
//   warps 4-7    codes -> fp16 tiles K16, V16 [key][channel] in shared memory, straight
//                from the pages: a warp takes 32 rows of every tile (they lie in one
//                page), the next half tile's (d = 64: the next step's) loads in flight
//   warps 8-11   softmax of tile 0, warps 12-15 of tile 1: a thread a row
// Per tile and step: S = Q K16^T (both in shared memory), P = 2^(t - m) rounded to fp16
// in place of S, O += P V16 (P in TMEM, V16 as it lies: the B operand with its N index
// fastest).  TMEM: S0, S1 and O0, O1, 512 columns at d = 128, so P lies in S's columns
// and a tile's QK follows its PV; the other tile's MMAs run under a tile's softmax.  The
// issuing order PV(0, j), QK(0, j + 1), PV(1, j), QK(1, j + 1) makes one barrier do for
// "S is there", "O is done" and "P has been read".  d = 64 leaves room for a P beside S: a
// tile's next QK follows the moment S has been read.
// A block of at most 128 rows gives both tiles the same rows and every other step each
// (dual); their parts are joined from TMEM at the end.
// Codes widened once serve 256 rows: 64 KB written and 192 KB read by the MMAs a step,
// ~2050 cycles of shared memory against as many of tensor work (d = 128).
//
// What bounds it.  d = 128, 2048 tokens of 32 heads on 8 at the end of 32K rows: 758 us,
// 1.41 PFLOP/s, 73% of a bf16 matrix product's rate; ~3450 cycles a step, of which the tensor
// pipe works 62%: shared memory, which conversion and MMAs share, and a tile's softmax
// between its QK and its PV.  d = 64, four whole prompts of 1.4K to 4.1K tokens, 12 heads:
// 144 us, 460 TFLOP/s: the two softmax warps of a scheduler take ~3850 cycles a step for what
// is 1020 of exponentials, with 192 registers each too few instructions in flight (46% of the
// issue slots used); per block ~9K cycles to bring Q and to write O.  Dual: the converting
// warps, ~2000 cycles a step at d = 64 and ~3300 at d = 128; a few tokens of 8 sequences of 1K
// to 16K rows, d = 64: 44 us, 1.6 TB/s.
// The reference m is set 7 below a row's maximum and moves only when that has grown by
// another 8 (P stays at or below 2^15), so O is rarely rescaled: P keeps its eleven bits
// where P s_v is down to 2^-21 of the row's largest, and is off by at most 2^-32 of it.
#include "paged_common.cuh"

namespace qattn {
namespace {

constexpr int kStep = kPagedTcStep;
constexpr int kRows = kPagedTcRows;
static_assert(kStep == 128 && kRows == 256, "two tiles of 128 TMEM lanes, one block of keys per step");
// Four warpgroups: the issuing and the planning warp's, the converting one, softmax of
// tile 0 and of tile 1.  Registers a thread: 128 at launch, shared out.
constexpr int kThreads = 512;
constexpr int kIssueRegs = 48, kConvRegs = 80, kSoftRegs = 192;
static_assert(kIssueRegs + kConvRegs + 2 * kSoftRegs == 4 * 128, "the split takes what the launch holds");
constexpr int kHead = 7;      // of the exponentials' reference (pg_head)
constexpr float kLazy = 8.f;  // log2 growth of a row's maximum that moves its reference
static_assert(kHead + kLazy <= 15.f, "P stays inside fp16");
constexpr int kGroups = kStep / 32;       // groups of keys that lie in one page
constexpr int kWinSteps = 32 / kGroups;   // steps of a warp's window of scales

template <int D>
struct Cfg {
  static constexpr int kTile = 128 * D * 2;  // fp16 Q, K16 or V16: D / 64 blocks of [128][128 B]
  // TMEM columns of tile t: S at 128 t, P at kTmP + kTmPStep t, O at kTmO + D t.  d = 64
  // leaves room for a P of its own: the next QK then follows the moment S has been read.
  static constexpr bool kOwnP = D == 64;
  static constexpr uint32_t kTmP = kOwnP ? 256 : 0, kTmPStep = kOwnP ? 64 : 128, kTmO = kOwnP ? 384 : 256;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + 2 * kTile;
  static constexpr int kOffML = kOffV + 2 * kTile;                 // m and l of both tiles (dual)
  static constexpr int kOffBar = kOffML + 2 * 2 * 128 * 4;
  static constexpr int kOffSeg = kOffBar + 256;                    // [2] PagedSeg
  static constexpr int kBytes = kOffSeg + 2 * 64;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

enum {
  kKFull = 0,   // [2] 128 converting threads
  kKEmpty = 2,  // [2] each issuer's: the step's QK MMAs
  kVFull = 4,   // [2] 128 converting threads
  kVEmpty = 6,  // [2] each issuer's: the step's PV MMAs
  kSFull = 8,   // [2 tiles] QK (and every MMA of the tile before it) is done
  kPFull = 10,  // [2 tiles][2 halves] 128 threads: P is there, O rescaled
  kQFull = 14,  // [2 tiles] 128 threads wrote Q
  kOFull = 16,  // [2 tiles] a segment's last PV is done
  kMerge = 18,  // [2] 256 threads: m and l are there; O has been read (dual)
  kDrain = 20,  // every issuer's MMAs
  kSegFull = 21,   // [2] the planning thread
  kSegEmpty = 23,  // [2] every other thread that works: the issuers, 128 + 256
  kSFree = 25,     // [2 tiles] 128 threads have S in registers (kOwnP)
  kPvDone = 27,    // [2 tiles] a step's PV: P and O are free (kOwnP)
  kNumBars = 29
};

// f(constant 0), f(constant 1), ...
template <int V>
struct Const {
  static constexpr int value = V;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll(F f) {
  if constexpr (I < N) {
    f(Const<I>{});
    unroll<N, I + 1>(f);
  }
}

// Whether both tiles hold the block's rows and take its steps in turn.
__device__ __forceinline__ bool is_dual(const PagedArgs& a, const PagedSeg& s) {
  return s.seq.n * a.G - s.rb * kRows <= 128;
}

// 16 codes -> 16 fp16, exact.
template <bool E4M3>
__device__ __forceinline__ void widen16(const uint4& v, uint32_t (&h)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (E4M3) {
      h[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
      h[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
    } else {
      codes4_to_f16x2(w[e], h[2 * e], h[2 * e + 1]);
    }
  }
}

// 32 channels ch .. of a row, times inv, to the output.
__device__ __forceinline__ void write_out32(const PagedArgs& a, size_t row, int ch, const float (&x)[32], float inv) {
  if (!QATTN_IN_BOUNDS(row < a.rows_total && ch + 32 <= a.d)) return;
  if (a.out_bf16) {
    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.d + ch);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * k + 2 * e] * inv, x[8 * k + 2 * e + 1] * inv);
        w[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
      dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * a.d + ch);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      dst[k] = make_float4(x[4 * k] * inv, x[4 * k + 1] * inv, x[4 * k + 2] * inv, x[4 * k + 3] * inv);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const PagedArgs a) {
  using C = Cfg<D>;
  constexpr uint32_t kIssuers = C::kOwnP ? 2 : 1;  // threads that issue MMAs
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + 8 * kNumBars + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto wait = [&](int i, uint32_t n) {  // the n-th completion (from 0) of barrier i
    return mbar_wait(bar(i), n & 1, abort_flag, a.err, kErrTimeout);
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= kKFull && i < kKFull + 2) || (i >= kVFull && i < kVFull + 2) || (i >= kPFull && i < kPFull + 4) ||
          (i >= kQFull && i < kQFull + 2) || (i >= kSFree && i < kSFree + 2))
        n = 128;
      if (i >= kMerge && i < kMerge + 2) n = 256;
      if (i >= kSegEmpty && i < kSegEmpty + 2) n = kIssuers + 128 + 256;
      if ((i >= kKEmpty && i < kKEmpty + 2) || (i >= kVEmpty && i < kVEmpty + 2) || i == kDrain) n = kIssuers;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  // Segment `seg` (from 0) of this CTA's share; n() == 0: there is none.
  PagedSeg* const slots = reinterpret_cast<PagedSeg*>(smem + C::kOffSeg);
  auto fetch = [&](uint32_t seg, const PagedSeg*& sg) {
    sg = &slots[seg & 1];
    return wait(kSegFull + (seg & 1), seg >> 1);
  };

  if (warp < 4) {
    reg_dec<kIssueRegs>();
    if (warp == 2) {
      // ------------------------------------------------------------ segments
      PagedWalk walk = pg_walk<kRows, kStep>(a, blockIdx.x, gridDim.x);
      if (lane == 0) {
        pg_put_plan(a, walk);
        bool ok = true, some = true;
        for (uint32_t seg = 0; ok && some; ++seg) {
          PagedSeg sg{};
          some = pg_next<kRows, kStep>(a, walk, sg);
          if (!some) sg.s0 = sg.s1 = 0;
          if (seg >= 2 && !(ok = wait(kSegEmpty + (seg & 1), (seg >> 1) - 1))) break;
          slots[seg & 1] = sg;
          mbar_arrive(bar(kSegFull + (seg & 1)));
        }
        if (!ok) *abort_flag = 1;
      }
      __syncwarp();
    } else if ((warp == 0 || (C::kOwnP && warp == 1)) && elect_one()) {
      // ------------------------------------------------------------ MMA
      constexpr uint32_t idesc_qk = make_idesc(128, kStep, 0, 0);
      constexpr uint32_t idesc_pv = make_idesc(128, D, 0, 0) | kIdescBMnMajor;
      constexpr uint32_t high = desc_high(1024, kSwizzle128B);  // of Q, K16 and V16
      const uint32_t q0 = static_cast<uint32_t>(smem_desc(base + C::kOffQ, 1024, kSwizzle128B));
      const uint32_t k0 = static_cast<uint32_t>(smem_desc(base + C::kOffK, 1024, kSwizzle128B));
      const uint32_t v0 = static_cast<uint32_t>(smem_desc_mn(base + C::kOffV, kStep * 128, 1024));
      constexpr uint32_t tile = C::kTile >> 4;
      bool ok = true;
      uint32_t it = 0;  // steps done
      auto qk = [&](int t, uint32_t step) {
        const uint32_t qd = q0 + t * tile, kd = k0 + (step & 1) * tile, d = tmem + 128 * t;
        unroll<D / 16>([&](auto k) {
          constexpr int i = decltype(k)::value;
          mma_f16_at<((i / 4) * (128 * 128) + 32 * (i % 4)) / 16, high, idesc_qk>(d, qd, kd, i > 0 ? 1u : 0u);
        });
        mma_commit(bar(kSFull + t));
      };
      // half h (64 keys) of tile t's PV; more: O is added to
      auto pv = [&](auto h, int t, uint32_t step, uint32_t more) {
        const uint32_t vd = v0 + (step & 1) * tile;
        const uint32_t o = tmem + C::kTmO + D * t, p = tmem + C::kTmP + C::kTmPStep * t;
        unroll<4>([&](auto k) {
          constexpr int i = 4 * decltype(h)::value + decltype(k)::value;
          mma_f16_ts_at<8 * i, 128 * i, high, idesc_pv>(o, p, vd, i > 0 ? 1u : more);
        });
      };
      if constexpr (C::kOwnP) {
        // A thread for each tile: QK(j + 1) once S has been read, PV(j) once P is there.  (One
        // thread that looks round for what is ready takes ~500 cycles to see it.)
        const int t = warp;
        uint32_t ns = 0, np = 0;  // the tile's QKs and PVs
        for (uint32_t seg = 0;; ++seg) {
          const PagedSeg* sg;
          if (!(ok = fetch(seg, sg))) break;
          const int n = sg->s1 - sg->s0;
          const bool dual = is_dual(a, *sg);
          mbar_arrive(bar(kSegEmpty + (seg & 1)));
          if (n == 0) break;
          const int ahead = dual ? 2 : 1;  // to the tile's next step
          auto release = [&](int i) {      // (both tiles' MMAs, or the one tile's)
            mma_commit(bar(i));
            if (dual) mbar_arrive(bar(i));
          };
          if (!(ok = wait(kQFull + t, seg))) break;
          const int first = dual ? t : 0;
          auto next_qk = [&](int j) {
            if (j >= n) return true;
            const uint32_t step = it + j;
            if (!wait(kKFull + (step & 1), step >> 1) || (j > first && !wait(kSFree + t, ns - 1))) return false;
            tc_fence_after();
            qk(t, step);
            release(kKEmpty + (step & 1));
            ++ns;
            return true;
          };
          if (first >= n) mbar_arrive(bar(kOFull + t));  // no step for this tile
          ok = next_qk(first);
          for (int j = first; ok && j < n; j += ahead) {
            const uint32_t step = it + j;
            // (dual: two steps on, K comes after P)
            if (!dual && !(ok = next_qk(j + ahead))) break;
            if (!(ok = wait(kVFull + (step & 1), step >> 1) && wait(kPFull + 2 * t, np))) break;  // keys 0 - 63
            tc_fence_after();
            pv(Const<0>{}, t, step, j >= ahead ? 1u : 0u);
            if (!(ok = wait(kPFull + 2 * t + 1, np))) break;  // keys 64 - 127
            tc_fence_after();
            pv(Const<1>{}, t, step, 1u);
            mma_commit(bar(kPvDone + t));
            release(kVEmpty + (step & 1));
            if (j + ahead >= n) mma_commit(bar(kOFull + t));
            ++np;
            if (dual) ok = next_qk(j + ahead);
          }
          if (!ok) break;
          it += n;
        }
      } else {
        // One thread for both tiles, in turn: that keeps them half a step apart, so that one
        // tile's MMAs run under the other's softmax.  (A thread for each lets both wait and
        // then contend: 1021 us against 910 for 2048 tokens over 32K.)
        uint32_t np[2] = {0, 0};  // PVs of each tile
        for (uint32_t seg = 0;; ++seg) {
          const PagedSeg* sg;
          if (!(ok = fetch(seg, sg))) break;
          const int n = sg->s1 - sg->s0;
          const bool dual = is_dual(a, *sg);
          mbar_arrive(bar(kSegEmpty + (seg & 1)));
          if (n == 0) break;
          // the first QK of each tile
          for (int t = 0; ok && t < 2; ++t) {
            if (!(ok = wait(kQFull + t, seg))) break;
            if (dual && t >= n) {  // no step for this tile
              mbar_arrive(bar(kOFull + t));
              continue;
            }
            const uint32_t step = it + (dual ? t : 0);
            if ((dual || t == 0) && !(ok = wait(kKFull + (step & 1), step >> 1))) break;
            tc_fence_after();
            qk(t, step);
            if (dual || t == 1) mma_commit(bar(kKEmpty + (step & 1)));
          }
          const int ahead = dual ? 2 : 1;  // to a tile's next step
          for (int j = 0; ok && j < n; ++j, ++it) {
            const uint32_t st = it & 1;
            const int t0 = dual ? (j & 1) : 0, t1 = dual ? t0 + 1 : 2;
            for (int t = t0; ok && t < t1; ++t) {
              const uint32_t done = t == 0 ? np[0] : np[1];
              auto next_qk = [&] {
                if (j + ahead >= n) return true;
                const uint32_t step = it + ahead;
                if (t == t0 && !wait(kKFull + (step & 1), step >> 1)) return false;
                tc_fence_after();
                qk(t, step);
                if (t == t1 - 1) mma_commit(bar(kKEmpty + (step & 1)));
                return true;
              };
              if (t == t0 && !(ok = wait(kVFull + st, it >> 1))) break;
              if (!(ok = wait(kPFull + 2 * t, done))) break;  // keys 0 - 63
              tc_fence_after();
              pv(Const<0>{}, t, it, j >= ahead ? 1u : 0u);
              if (!(ok = wait(kPFull + 2 * t + 1, done))) break;  // keys 64 - 127
              tc_fence_after();
              pv(Const<1>{}, t, it, 1u);
              if (t == 0) ++np[0];
              else ++np[1];
              if (t == t1 - 1) mma_commit(bar(kVEmpty + st));
              if (j + ahead >= n) mma_commit(bar(kOFull + t));
              ok = next_qk();
            }
          }
          if (!ok) break;
        }
      }
      if (!ok) *abort_flag = 1;
      mma_commit(bar(kDrain));
      volatile int never = 0;
      mbar_wait(bar(kDrain), 0, &never, a.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp < 8) {
    // -------------------------------------------------------------- codes -> fp16
    reg_dec<kConvRegs>();
    // Warp w takes rows 32 w .. 32 w + 31 of every tile, K and V of a step in turn, so that
    // each waits for every stage in order.  The eight lanes of a store take four chunks of
    // rows r and r ^ 5, which differ in the swizzle's low and high bit: eight bank groups.
    constexpr int NB = D / 64;  // 64-channel blocks
    const int w = warp - 4;
    const int cc = lane & 3, u = (lane >> 3) ^ (((lane >> 2) & 1) * 5);  // chunk of a block, row of eight
    const uint32_t dst = base + (32 * w + u) * 128;
    const uint32_t c0 = ((2 * cc) ^ u) << 4, c1 = ((2 * cc + 1) ^ u) << 4;
    bool ok = true;
    uint32_t it = 0;  // steps done
    for (uint32_t seg = 0;; ++seg) {
      const PagedSeg* at_seg;
      if (!(ok = __all_sync(0xffffffffu, fetch(seg, at_seg)))) break;
      const PagedSeg sg = *at_seg;
      mbar_arrive(bar(kSegEmpty + (seg & 1)));
      const int n = sg.s1 - sg.s0, len = sg.seq.len;
      if (n == 0) break;
      // pages of this warp's rows in the next 32 steps, one a lane, and in the 32 after
      auto look_up = [&](int j0) {
        const int key = (sg.s0 + j0 + lane) * kStep + 32 * w;
        int p = -1;
        if (j0 + lane < n && key < len && QATTN_IN_BOUNDS((key >> a.page_shift) < a.max_pages && sg.b < a.B)) {
          p = a.page_table[static_cast<size_t>(sg.b) * a.max_pages + (key >> a.page_shift)];
          if (p < 0 || p >= a.n_pages) p = -1;  // (the softmax warps report it)
        }
        return p;
      };
      int cur = look_up(0), nxt = n > 32 ? look_up(32) : -1;
      // where step j's rows start in the pool (in bytes), or -1
      auto place = [&](int j) -> long long {
        if (j > 0 && j % 32 == 0) {
          cur = nxt;
          if (j + 32 < n) nxt = look_up(j + 32);
        }
        const int p = __shfl_sync(0xffffffffu, cur, j & 31);
        if (p < 0) return -1;
        const int key = (sg.s0 + j) * kStep + 32 * w;
        const long long row = ((static_cast<long long>(p) * a.Hkv + sg.hkv) << a.page_shift) +
                              (key & ((1 << a.page_shift) - 1)) + u;
        return row * D + 16 * cc;
      };
      // x: d = 128: a tile's rows in two halves of 16; d = 64: K's and V's rows
      uint4 x[2][4];
      auto load = [&](int h, const uint8_t* pages, long long at, int j) {
        const int left = len - (sg.s0 + j) * kStep - 32 * w - u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = (D == 128 ? 16 * h : 0) + 8 * (k / NB);
          x[h][k] = make_uint4(0u, 0u, 0u, 0u);
          // rows behind the sequence may hold any byte: zeros stand in
          if (at >= 0 && r < left) x[h][k] = *reinterpret_cast<const uint4*>(pages + at + r * D + 64 * (k % NB));
        }
      };
      auto convert = [&](int h, uint32_t tile) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t y[8];
          widen16<E4M3>(x[h][k], y);
          const uint32_t d = dst + tile + (k % NB) * (128 * 128) + ((D == 128 ? 16 * h : 0) + 8 * (k / NB)) * 128;
          sts128(d + c0, y[0], y[1], y[2], y[3]);
          sts128(d + c1, y[4], y[5], y[6], y[7]);
        }
      };
      long long at = place(0);
      load(0, a.k_pages, at, 0);
      load(1, D == 128 ? a.k_pages : a.v_pages, at, 0);
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t st = it & 1;
        ok = it < 2 || wait(kKEmpty + st, (it >> 1) - 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint32_t tk = C::kOffK + st * C::kTile, tv = C::kOffV + st * C::kTile;
        const bool more = j + 1 < n;
        if constexpr (D == 128) {
          convert(0, tk);
          load(0, a.v_pages, at, j);
          convert(1, tk);
          load(1, a.v_pages, at, j);
        } else {
          if (more) at = place(j + 1);
          convert(0, tk);
          if (more) load(0, a.k_pages, at, j + 1);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(kKFull + st));
        if (D == 128 && more) at = place(j + 1);
        ok = it < 2 || wait(kVEmpty + st, (it >> 1) - 1);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if constexpr (D == 128) {
          convert(0, tv);
          if (more) load(0, a.k_pages, at, j + 1);
          convert(1, tv);
          if (more) load(1, a.k_pages, at, j + 1);
        } else {
          convert(1, tv);
          if (more) load(1, a.v_pages, at, j + 1);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(kVFull + st));
      }
      if (!ok) break;
    }
    if (!ok) *abort_flag = 1;
  } else {
    // -------------------------------------------------------------- softmax
    reg_inc<kSoftRegs>();
    const int t = (warp - 8) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // TMEM lane, row of the tile
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * t, tO = tmem + lane_base + C::kTmO + D * t;
    const uint32_t tP = tmem + lane_base + C::kTmP + C::kTmPStep * t;
    float* ml = reinterpret_cast<float*>(smem + C::kOffML);  // [tile][m, l][128]
    uint32_t ns = 0, merges = 0;  // this tile's steps, dual segments
    bool ok = true;
    for (uint32_t seg = 0;; ++seg) {
      const PagedSeg* at_seg;
      if (!(ok = __all_sync(0xffffffffu, fetch(seg, at_seg)))) break;
      const int n = at_seg->s1 - at_seg->s0;
      if (n == 0) break;
      const bool dual = is_dual(a, *at_seg);
      const int s0 = at_seg->s0;
      // ---- the scales' windows, one group a lane: pages two windows ahead, scales one
      auto page_of = [&](int w) {
        const int key = s0 * kStep + 32 * (32 * w + lane);
        int p = -1;
        if (32 * w + lane < kGroups * n && key < at_seg->seq.len &&
            QATTN_IN_BOUNDS((key >> a.page_shift) < a.max_pages && at_seg->b < a.B)) {
          p = a.page_table[static_cast<size_t>(at_seg->b) * a.max_pages + (key >> a.page_shift)];
          if (p < 0 || p >= a.n_pages) {
            atomicOr(a.err, kErrDomain);
            p = -1;
          }
        }
        return p;
      };
      auto scales_of = [&](int p, float& ks, float& vs) {
        ks = vs = 0.f;
        if (p < 0) return;
        const size_t sc = static_cast<size_t>(p) * a.Hkv + at_seg->hkv;
        ks = a.k_scales[sc];
        vs = a.v_scales[sc];
      };
      int p1 = page_of(0), p2 = page_of(1);
      float ks1, vs1;
      // ---- Q's row -> fp16 in shared memory
      float rf;
      bool fin;
      int lim;
      {
        const PagedSeg sg = *at_seg;
        const int rr = sg.rb * kRows + (dual ? 0 : 128 * t) + r;
        const int tok = rr / a.G, hq = sg.hkv * a.G + rr - tok * a.G;
        const bool in = tok < sg.seq.n;
        // (a row that is none sees everything: its scores are 0, and it asks for no mask)
        lim = in ? min(pg_limit(a, sg.seq, tok), sg.seq.len) : 0x7fffffff;
        const uint16_t* src = a.q + sg.b * a.qsB + hq * a.qsH + tok * a.qsN;
        uint4 x[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          x[k] = make_uint4(0u, 0u, 0u, 0u);
          if (in && QATTN_IN_BOUNDS(sg.b < a.B && hq < a.Hq && tok < a.T)) x[k] = *reinterpret_cast<const uint4*>(src + 8 * k);
        }
        scales_of(p1, ks1, vs1);  // (behind Q's loads)
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
        }
        fin = top < 0x7f800000u;  // else the row is NaN once it sees a key
        float up, down;
        pg_row_shift(top, up, down);
        rf = __fmul_rn(__fmul_rn(a.sm_scale, kPgLog2e), down);
        const uint32_t row = base + C::kOffQ + t * C::kTile + r * 128;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(fin ? bf16_bits_to_f32(w[e] & 0xffffu) * up : 0.f,
                                                fin ? __uint_as_float(w[e] & 0xffff0000u) * up : 0.f);
            f[e] = *reinterpret_cast<const uint32_t*>(&h);
          }
          sts128(row + (k / 8) * (128 * 128) + (((k % 8) ^ (r & 7)) << 4), f[0], f[1], f[2], f[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(kQFull + t));
      float m = -kPgInf, l = 0.f;  // the row's reference and its sum
      const int first = dual ? t : 0, pace = dual ? 2 : 1;
      float c[kGroups], e[kGroups], inv[kGroups];  // the step's scales
      uint32_t rare = 0;
      // a window's scales, a lane for a group, and its groups that are out of the ordinary
      // (kept from shared memory: the MMAs' reads leave a load there waiting for ~1500 cycles)
      float wk = 0.f, we = 0.f, winv = 1.f;
      uint32_t hidden = 0, zero_v = 0, bad = 0;
      auto scales = [&](int j) {
        if (j % kWinSteps == first) {  // a new window
          const PageScale ps = pg_scale(ks1, vs1);
          wk = ps.k;
          we = ps.e;
          winv = ps.inv;
          hidden = __ballot_sync(0xffffffffu, p1 < 0);
          zero_v = __ballot_sync(0xffffffffu, ps.keep == 0u);
          bad = __ballot_sync(0xffffffffu, ps.nan);
          p1 = p2;
          scales_of(p1, ks1, vs1);
          p2 = page_of(j / kWinSteps + 2);
        }
        const int q0 = kGroups * (j % kWinSteps);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          c[g] = fmaxf(rf * __shfl_sync(0xffffffffu, wk, q0 + g), 1e-30f);
          e[g] = __shfl_sync(0xffffffffu, we, q0 + g);
          inv[g] = __shfl_sync(0xffffffffu, winv, q0 + g);
        }
        rare = ((hidden | zero_v | bad) >> q0) & ((1u << kGroups) - 1u);
      };
      if (first < n) scales(first);
      for (int j = first; j < n; j += pace, ++ns) {
        const int q0 = kGroups * (j % kWinSteps);
        const int room = lim - (s0 + j) * kStep;  // visible keys of the step
        const bool masked = __any_sync(0xffffffffu, room < kStep || rare != 0u);
        // The reference seldom moves, so the exponentials begin with the one that stands
        // while the other scores are on their way; should the maxima ask for another, S is
        // read again.  0: try; 1: settle the reference first; 2: settled.
        int mode = masked || __any_sync(0xffffffffu, m == -kPgInf) ? 1 : 0;
        ok = wait(kSFull + t, ns);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        bool pv_over = false;  // the tile's PV before this step is done (else S comes after it)
        auto pv_done = [&] {
          if (!C::kOwnP || pv_over || j == first) return true;
          pv_over = true;
          if (!__all_sync(0xffffffffu, wait(kPvDone + t, ns - 1))) return false;
          tc_fence_after();
          return true;
        };
        for (;;) {
          uint32_t v[kGroups][32];
          float mx[kGroups];
          tmem_ld32_max(tS, v[0], mx[0]);
          tmem_wait_ld();
#pragma unroll
          for (int g = 1; g < kGroups; ++g) tmem_ld32_max(tS + 32 * g, v[g], mx[g]);
          if (mode != 0) tmem_wait_ld();
          if (masked) {  // hidden keys' scores to -inf
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const uint32_t vis = pg_first_bits(((hidden >> (q0 + g)) & 1u) ? 0 : room - 32 * g);
              if (vis != 0u && ((bad >> (q0 + g)) & 1u)) fin = false;
              if (__all_sync(0xffffffffu, vis == 0xffffffffu)) continue;
              mx[g] = -kPgInf;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                if (!((vis >> k) & 1u)) v[g][k] = __float_as_uint(-kPgInf);
                mx[g] = fmaxf(mx[g], __uint_as_float(v[g][k]));
              }
            }
          }
          auto largest = [&] {
            float top = -kPgInf;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              float x = fmaf(mx[g], c[g], e[g]);
              if ((zero_v >> (q0 + g)) & 1u) x = fmaf(mx[g], c[g], kPgZeroE);
              top = fmaxf(top, x);
            }
            return top;
          };
          auto moves = [&](float top, float head) {
            return top > m + (head == 0.f ? 0.f : kHead + kLazy) || (m == -kPgInf && top > -kPgInf);
          };
          if (mode == 1) {
            const float top = largest(), head = pg_head(top, kHead);
            const bool moved = moves(top, head);
            const float mn = moved ? top - head : m;
            const float al = !moved ? 1.f : m == -kPgInf ? 0.f : ex2_approx(m - mn);
            l *= al;
            m = mn;
            if (j > first && __any_sync(0xffffffffu, moved)) {
              ok = pv_done();
              if (!ok) break;
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t x[32];
                tmem_ld32(tO + 32 * k, x);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q) x[q] = __float_as_uint(__uint_as_float(x[q]) * al);
                tmem_st32(tO + 32 * k, x);
              }
              tmem_wait_st();
              mode = 2;
              continue;  // (the scores made room for O)
            }
          }
          const float ref = m == -kPgInf ? 0.f : m;
          float add = 0.f;
          uint32_t pk[2][32];
          auto weigh = [&](int g) {
            const float off = e[g] - ref;
            const float2 c2 = make_float2(c[g], c[g]), n2 = make_float2(off, off);
            float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              float2 x0 = ffma2(make_float2(__uint_as_float(v[g][k]), __uint_as_float(v[g][k + 1])), c2, n2);
              float2 x1 = ffma2(make_float2(__uint_as_float(v[g][k + 2]), __uint_as_float(v[g][k + 3])), c2, n2);
              x0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
              x1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
              sum0 = fadd2(sum0, x0);
              sum1 = fadd2(sum1, x1);
              const __half2 h0 = __floats2half2_rn(x0.x, x0.y), h1 = __floats2half2_rn(x1.x, x1.y);
              pk[g / 2][16 * (g % 2) + k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
              pk[g / 2][16 * (g % 2) + k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
            }
            add = fmaf((sum0.x + sum0.y) + (sum1.x + sum1.y), inv[g], add);
            if ((zero_v >> (q0 + g)) & 1u) {
#pragma unroll
              for (int k = 0; k < 16; ++k) pk[g / 2][16 * (g % 2) + k] = 0u;
            }
          };
          weigh(0);
          if (mode == 0) {
            tmem_wait_ld();
            const float top = largest();
            if (__any_sync(0xffffffffu, moves(top, pg_head(top, kHead)))) {
              mode = 1;
              continue;
            }
          }
          if (C::kOwnP) {  // S may be overwritten
            tc_fence_before();
            mbar_arrive(bar(kSFree + t));
          }
          weigh(1);
          ok = pv_done();
          if (!ok) break;
          tmem_st32(tP, pk[0]);
          weigh(2);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kPFull + 2 * t));
          weigh(3);
          tmem_st32(tP + 32, pk[1]);
          l += add;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(kPFull + 2 * t + 1));
          break;
        }
        if (!ok) break;
        if (j + pace < n) scales(j + pace);
      }
      if (!ok) break;
      // ---- the segment's share
      if (!fin && m > -kPgInf) l = __uint_as_float(0x7fffffffu);  // saw a key through something not finite
      ok = __all_sync(0xffffffffu, wait(kOFull + t, seg));
      if (!ok) break;
      float fa = 1.f, fb = 0.f;  // weights of this tile's O and (dual) the other's
      if (dual) {
        ml[(2 * t) * 128 + r] = m;
        ml[(2 * t + 1) * 128 + r] = l;
        tc_fence_before();
        mbar_arrive(bar(kMerge));
        ok = wait(kMerge, merges);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const float mo = ml[(2 * (1 - t)) * 128 + r], lo = ml[(2 * (1 - t) + 1) * 128 + r];
        const float mm = fmaxf(m, mo);
        fa = m == -kPgInf ? 0.f : ex2_approx(m - mm);
        fb = mo == -kPgInf ? 0.f : ex2_approx(mo - mm);
        l = fa * l + fb * lo;
        m = mm;
      }
      tc_fence_after();
      const PagedSeg sg = *at_seg;
      mbar_arrive(bar(kSegEmpty + (seg & 1)));
      const int pr = (dual ? 0 : 128 * t) + r;  // row of the block
      const int rr = sg.rb * kRows + pr, tok = rr / a.G, hq = sg.hkv * a.G + rr - tok * a.G;
      const bool in = tok < sg.seq.n;
      const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (sg.s0 > 0 ? 0 : 1);
      const size_t row = (static_cast<size_t>(sg.b) * a.Hq + hq) * a.T + tok;
      const float rl = l == 0.f ? 0.f : 1.f / l;
      const uint32_t tOther = tmem + lane_base + C::kTmO + D * (1 - t);
#pragma unroll 1
      for (int k = dual ? t * (D / 64) : 0; k < (dual ? (t + 1) * (D / 64) : D / 32); ++k) {
        uint32_t x[32];
        float y[32];
        tmem_ld32(tO + 32 * k, x);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 32; ++q) y[q] = fa == 0.f ? 0.f : __uint_as_float(x[q]) * fa;
        if (dual) {
          tmem_ld32(tOther + 32 * k, x);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; ++q) y[q] = fb == 0.f ? y[q] : fmaf(__uint_as_float(x[q]), fb, y[q]);
        }
        if (whole) {
          if (in) write_out32(a, row, 32 * k, y, rl);
        } else if (in && QATTN_IN_BOUNDS(slot < a.slots)) {
          // chunks of four channels, each for all rows: a warp writes 512 consecutive bytes
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(a.part_o + ((slot * (D / 4) + 8 * k + q / 4) * kRows + pr) * 4) =
                make_float4(y[q], y[q + 1], y[q + 2], y[q + 3]);
        }
      }
      if (in && (!dual || t == 0)) {
        if (whole) {
          if (a.lse && QATTN_IN_BOUNDS(row < a.rows_total))
            a.lse[row] = l == 0.f ? -kPgInf : ((m + kHead) + log2f(l * (1.f / (1 << kHead)))) * kPgLn2;
        } else if (QATTN_IN_BOUNDS(slot < a.slots)) {
          a.part_m[slot * kRows + pr] = m;
          a.part_l[slot * kRows + pr] = l;
        }
      }
      tc_fence_before();  // the next segment's MMAs overwrite O
      if (dual) {
        mbar_arrive(bar(kMerge + 1));
        ok = wait(kMerge + 1, merges);  // the other tile's threads have read this one's O
        ++merges;
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The join: CTAs (c, y) work for the boundary between the shares of CTAs c and c + 1, if
// it is the first one inside a block (PagedPlan).  A lane for a row, a warp for four channels
// of it (blockIdx.y: 16 channels, then 32 rows), so that every load of a share takes 512
// consecutive bytes; four shares' loads in flight.
template <int D>
__global__ void __launch_bounds__(kPgJoinThreads) paged_join_rows_kernel(const PagedArgs a) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = 32 * (blockIdx.y / (D / 16)) + lane;
  const int c = 4 * (4 * (blockIdx.y % (D / 16)) + warp);
  pdl_wait();
  pdl_trigger();
  const PagedPlan w = pg_get_plan(a, blockIdx.x + 1);
  const int rr = w.rb * kRows + r, c0 = w.c0, c1 = w.c1;
  if (c1 < 0 || rr / a.G >= w.n) return;
  float m = -kPgInf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int cb = c0; cb <= c1; cb += U) {
    float mc[U], lc[U], mn = m;
    float4 y[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int ci = cb + i;
      const size_t slot = 2 * static_cast<size_t>(ci) + (ci == c0 ? 1 : 0);
      mc[i] = -kPgInf;
      if (ci <= c1 && QATTN_IN_BOUNDS(slot < a.slots)) {
        mc[i] = a.part_m[slot * kRows + r];
        lc[i] = a.part_l[slot * kRows + r];
        y[i] = *reinterpret_cast<const float4*>(a.part_o + ((slot * (D / 4) + c / 4) * kRows + r) * 4);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) mn = fmaxf(mn, mc[i]);
    if (mn == -kPgInf) continue;
    const float f = m == -kPgInf ? 0.f : ex2_approx(m - mn);
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (mc[i] == -kPgInf) continue;
      const float g = ex2_approx(mc[i] - mn);
      l = fmaf(g, lc[i], l);
      o.x = fmaf(g, y[i].x, o.x);
      o.y = fmaf(g, y[i].y, o.y);
      o.z = fmaf(g, y[i].z, o.z);
      o.w = fmaf(g, y[i].w, o.w);
    }
    m = mn;
  }
  pg_write_out<D, kHead>(a, w.b, w.hkv, w.n, rr, c, o, m, l);
}

template <int D, bool E4M3>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t s) {
  constexpr int smem = Cfg<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(paged_tc_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_tc_kernel<D, E4M3>, dim3(a.ctas), dim3(kThreads), smem, s, a);
  if (e != cudaSuccess || a.ctas == 1) return e;
  const int groups = (min(kRows, a.G * a.T) + 31) / 32;  // of 32 rows, in the longest block
  return launch_pdl(paged_join_rows_kernel<D>, dim3(a.ctas - 1, groups * (D / 16)), dim3(kPgJoinThreads), 0, s, a);
}

}  // namespace

unsigned int check_take_paged_tc() { return check_take_local(); }

cudaError_t launch_paged_tc(const PagedArgs& a, cudaStream_t s) {
  if (a.e4m3) return a.d == 64 ? launch_d<64, true>(a, s) : launch_d<128, true>(a, s);
  return a.d == 64 ? launch_d<64, false>(a, s) : launch_d<128, false>(a, s);
}

}  // namespace qattn
