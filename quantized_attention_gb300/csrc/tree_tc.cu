// Attention of drafted tokens over an int8 KV cache (qattn_tree_decode), for
// more than 16 query rows of a KV head: 128 rows at a time on the
// 5th-generation tensor cores.  Mathematics, work division and joining as in
// tree_warp.cu, with steps of 128 keys.
//
//   warp 0       TMA: the steps' K and V codes into a ring of raw stages
//   warp 1       TMEM and the MMAs
//   warps 4-11   softmax: two threads a row (keys 0-63 and 64-127 of a step)
//   warps 12-15  codes -> fp16 tiles K16, V16 [key][channel] in shared memory; a
//                drafted step's codes are made by these and the softmax warps first
//
// Per step: S = Q K16^T (Q as the A operand in TMEM), P = 2^(S c - m) rounded to
// fp16 into TMEM, O += P V16 (V16 as it lies: the B operand with its N index
// fastest).  Q and P in TMEM leave shared memory to the codes: 32 KB in, 32 KB
// read, 64 KB of fp16 written and 64 KB read by the MMAs a step, ~1540 cycles
// against ~1460 of the step's share of HBM and ~1030 of tensor work.  Measured: ~2250
// cycles a step: the converting warps (~1050 a tile, two a step: 180 instructions a
// thread, the proxy fence) and the softmax warps (scores 480, the halves' maxima
// exchanged 300, exponentials 810, the last PV 380, P 130, loop 140) each nearly fill
// it, and the issuing thread's K16 comes late; 26-node trees over eight caches of 5K
// to 32K rows 94 us (floor 47), 64 nodes over 32K 49 (floor 18; 33 of it the steps, 6
// up to the first scores, 5 the join and its launch).  Six or eight converting warps,
// two issuing threads, PV ahead of the next QK, setmaxnreg with more registers for the
// softmax, and softmax groups that take steps in turn (a thread a row) measured no
// faster or slower.
// The reference m is set 7 below a row's maximum and moves only when that has grown by
// another 8 (P stays at or below 2^15, inside fp16), so O is rarely rescaled: a key down
// to 2^-21 of the row's largest (14.5 nats) is off by at most 2^-11, further down by at
// most 2^-32 of the largest.
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"
#include "tree_common.cuh"

namespace qattn {
namespace {

constexpr int kStep = kTreeTcStep;
constexpr int kRows = kTreeTcRows;
static_assert(kStep == 128 && kRows == 128, "one TMEM lane per row, one block of keys per step");
constexpr int kThreads = 512;
constexpr int kRaw = 6;      // raw ring: K and V tiles of codes, one after the other
constexpr int kEncode = 384; // threads that encode a drafted step: softmax and converting warps
// Shares a head, on average, from which four warps join a row.  One against four warps,
// us: 9.5 shares (16 heads of 16K rows) 30.9 / 32.3, 19 (8 of 8K) 21.7 / 18.7, 152 (one of
// 32K) 44.1 / 22.5.
constexpr int kJoinShares = 12;
constexpr int kHead = 7;      // of the exponentials' reference (tree_head)
constexpr float kLazy = 8.f;  // log2 growth of a row's maximum that moves its reference
static_assert(kHead + kLazy <= 15.f, "P stays inside fp16");
constexpr uint32_t kTmS = 0, kTmO = 256, kTmP = 384, kTmQ = 448;  // TMEM columns

template <int D>
struct Cfg {
  static constexpr int kRawTile = kStep * D;          // K (or V) codes of a step
  static constexpr int kHalf = kStep * D * 2;         // K16 (or V16): D / 64 blocks of [128][128 B]
  static constexpr int kOff16 = kRaw * kRawTile;      // after the raw ring
  static constexpr int kOffX = kOff16 + 2 * 2 * kHalf;
  static constexpr int kOffBar = kOffX + 2 * 2 * kRows * 4;  // row maxima: [buffer][half][row]
  static constexpr int kBytes = kOffBar + 512;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
  static_assert(4 * kRows * D + 8 * kRows <= kOff16, "a CTA's O, m and l for its cluster do not fit the raw ring");
};

enum {
  kRawFull = 0,    // [kRaw] TMA bytes (a drafted step: the loader's arrival)
  kRawEmpty = 6,   // [kRaw] 128 converting threads
  kKFull = 12,     // [2] 128
  kVFull = 14,     // [2] 128
  kSFull = 16,     // [2] the step's QK MMAs: S is there, K16 is free
  kPvDone = 18,    // [2] the step's PV MMAs: O and P are free, and V16
  kQReady = 20,    // 128 threads wrote Q
  kPReady = 21,    // 256
  kXFull = 22,     // [2 buffers][4 quadrants] 64
  kDrafts = 30,    // kEncode threads wrote a drafted step's codes
  kDrain = 31,
  kNumBars = 32
};

// Place of 16-byte chunk c of row r of a CTA's O in shared memory (a thread writes a
// row: eight rows of a store hit eight bank groups).
__device__ __forceinline__ int share_chunk(int r, int c) { return c ^ (r & 7); }

template <int D, bool CL>
__global__ void __launch_bounds__(kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const TreeArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  uint8_t* smem = dyn_smem;
  const uint32_t base = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + 8 * kNumBars + 4);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto wait = [&](int i, uint32_t n) {  // the n-th completion (from 0) of barrier i
    return mbar_wait_fast(bar(i), n & 1, abort_flag, a.err, kErrTimeout);
  };
  auto raw = [&](uint32_t slot) { return base + slot * C::kRawTile; };
  auto k16 = [&](int st) { return base + C::kOff16 + st * 2 * C::kHalf; };
  auto v16 = [&](int st) { return base + C::kOff16 + st * 2 * C::kHalf + C::kHalf; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t n = 1;
      if ((i >= kRawEmpty && i < kRawEmpty + kRaw) || (i >= kKFull && i < kKFull + 2) ||
          (i >= kVFull && i < kVFull + 2) || i == kQReady)
        n = 128;
      if (i == kDrafts) n = kEncode;
      if (i == kPReady) n = 256;
      if (i >= kXFull && i < kXFull + 8) n = 64;
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
  pdl_trigger();  // after the wait: the join reads the lengths before its own
  TreeWalk walk;
  TreeSeg sg{};
  if constexpr (CL) {
    walk = tree_cluster_walk(a, kStep, sg);
  } else {
    walk = tree_walk(a, kStep);
  }
  // the next segment: of this CTA's share, or (once) its part of its own head
  auto next_segment = [&] { return CL ? tree_once(walk, sg) : tree_next(a, kStep, walk, sg); };

  // A drafted step's codes, into its raw tiles n and n + 1: the softmax warps (idle
  // until the segment's first scores) and the converting ones together, thread e of
  // kEncode.  Returns when every one has written.
  auto encode = [&](uint32_t n, int s, int e, uint32_t nd) -> bool {
    bool ok = wait(kRawFull + n % kRaw, n / kRaw) && wait(kRawFull + (n + 1) % kRaw, (n + 1) / kRaw);
    if (!__all_sync(0xffffffffu, ok)) return false;
    uint8_t* kr = smem + (n % kRaw) * C::kRawTile;
    uint8_t* vr = smem + ((n + 1) % kRaw) * C::kRawTile;
    auto at = [](uint8_t* t, int r, int c) {
      return t + r * D + 16 * (c ^ ((D == 128) ? (r & 7) : ((r >> 1) & 3)));
    };
    tree_encode_drafts<D>(a, sg.b, sg.hkv, s * kStep, kStep, e, kEncode,
                          [&](int r, int c) { return at(kr, r, c); }, [&](int r, int c) { return at(vr, r, c); });
    fence_proxy_async_smem();  // the tiles go back to the TMA engine
    mbar_arrive(bar(kDrafts));
    ok = wait(kDrafts, nd);
    return __all_sync(0xffffffffu, ok);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA
      if (a.Nk > 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
      bool ok = true;
      uint32_t n = 0;  // tiles: K and V of each step
      while (ok && next_segment()) {
        const int bkv = sg.b * a.Hkv + sg.hkv;
        for (int s = sg.s0; ok && s < sg.s1; ++s) {
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t slot = n % kRaw;
            if (n >= kRaw && !(ok = wait(kRawEmpty + slot, n / kRaw - 1))) break;
            if (s < a.drafts) {
              mbar_arrive(bar(kRawFull + slot));
            } else {
              (void)QATTN_IN_BOUNDS((s - a.drafts) * kStep < a.Nk && bkv < a.B * a.Hkv);  // TMA coordinates
              mbar_arrive_expect_tx(bar(kRawFull + slot), C::kRawTile);
              tma_load_3d(raw(slot), kv ? &tmV : &tmK, bar(kRawFull + slot), 0, (s - a.drafts) * kStep, bkv);
            }
          }
        }
      }
      // every load this thread issued lands before the CTA may exit
      volatile int never = 0;
      for (uint32_t back = 1; back <= kRaw; ++back)
        if (n >= back)
          mbar_wait(bar(kRawFull + (n - back) % kRaw), ((n - back) / kRaw) & 1, &never, a.err, kErrTimeout);
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // ------------------------------------------------------------ MMA
      constexpr uint32_t idesc_qk = make_idesc(kRows, kStep, 0, 0);
      constexpr uint32_t idesc_pv = make_idesc(kRows, D, 0, 0) | kIdescBMnMajor;
      const uint64_t kd0 = smem_desc(k16(0), 1024, kSwizzle128B);
      const uint64_t vd0 = smem_desc_mn(v16(0), kStep * 128, 1024);
      bool ok = true;
      uint32_t it = 0, seg = 0;  // steps and segments done
      auto qk = [&](uint32_t t) -> bool {
        const uint32_t st = t & 1;
        if (!wait(kKFull + st, t >> 1)) return false;
        tc_fence_after();
        const uint64_t kd = kd0 + st * (2 * C::kHalf >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ts(tmem + kTmS + 128 * st, tmem + kTmQ + 8 * k, kd + ((k / 4) * (kStep * 128) + 32 * (k % 4)) / 16,
                     idesc_qk, k > 0 ? 1u : 0u);
        mma_commit(bar(kSFull + st));
        return true;
      };
      for (; ok && next_segment(); ++seg) {
        const int n = sg.s1 - sg.s0;
        if (!(ok = wait(kQReady, seg))) break;
        if (!(ok = qk(it))) break;
        for (int j = 0; j < n; ++j, ++it) {
          if (j + 1 < n && !(ok = qk(it + 1))) break;
          const uint32_t st = it & 1;
          if (!(ok = wait(kVFull + st, it >> 1) && wait(kPReady, it))) break;
          tc_fence_after();
          const uint64_t vd = vd0 + st * (2 * C::kHalf >> 4);
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k)
            mma_f16_ts(tmem + kTmO, tmem + kTmP + 8 * k, vd + (k * 2048) / 16, idesc_pv,
                       (j > 0 || k > 0) ? 1u : 0u);
          mma_commit(bar(kPvDone + st));
        }
      }
      mma_commit(bar(kDrain));
      volatile int never = 0;
      mbar_wait(bar(kDrain), 0, &never, a.err, kErrTimeout);
      if (!ok) *abort_flag = 1;
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // -------------------------------------------------------------- softmax
    const int quad = warp & 3, hf = (warp - 4) >> 2;
    const int r = quad * 32 + lane;  // TMEM lane, row of the block
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const int R = a.G * a.T;
    float* xch = reinterpret_cast<float*>(smem + C::kOffX);
    uint32_t it = 0, nx = 0, nd = 0;
    bool ok = true;
    // this half's value to the other half's thread of the row, and back
    auto exchange = [&](float v, float& other) -> bool {
      const int b2 = nx & 1;
      xch[(b2 * 2 + hf) * kRows + r] = v;
      mbar_arrive(bar(kXFull + 4 * b2 + quad));
      const bool o = wait(kXFull + 4 * b2 + quad, nx >> 1);
      ++nx;
      if (!__all_sync(0xffffffffu, o)) return false;
      other = xch[(b2 * 2 + 1 - hf) * kRows + r];
      return true;
    };
    while (ok && next_segment()) {
      for (int s = sg.s0; ok && s < min(sg.s1, a.drafts); ++s) {
        ok = encode(2 * (it + s - sg.s0), s, threadIdx.x - 128, nd);
        ++nd;
      }
      if (!ok) break;
      const int rr = sg.rb * kRows + r;
      const bool in = rr < R;
      const int hq = in ? rr / a.T : 0, tok = in ? rr % a.T : 0;
      const size_t row = (static_cast<size_t>(sg.b) * a.Hq + sg.hkv * a.G + hq) * a.T + tok;
      if (hf == 0) {  // Q's row -> A in TMEM
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
          uint32_t x[32];
          const uint4* src = reinterpret_cast<const uint4*>(a.q_codes + row * D) + 4 * e;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (in && QATTN_IN_BOUNDS(row < a.rows_total)) v = src[c];
            codes4_to_f16x2(v.x, x[8 * c + 0], x[8 * c + 1]);
            codes4_to_f16x2(v.y, x[8 * c + 2], x[8 * c + 3]);
            codes4_to_f16x2(v.z, x[8 * c + 4], x[8 * c + 5]);
            codes4_to_f16x2(v.w, x[8 * c + 6], x[8 * c + 7]);
          }
          tmem_st32(tmem + lane_base + kTmQ + 32 * e, x);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kQReady));
      }
      bool fin = true;
      const float cf = in ? tree_factor(a, sg.b, sg.hkv * a.G + hq, fin) : 1.f;
      const int lim = tree_limit(a, sg.len, tok);
      float m = kNegInf, l = 0.f;  // the row's reference; this half's share of the sum
      for (int s = sg.s0; s < sg.s1; ++s, ++it) {
        const uint32_t st = it & 1;
        ok = wait(kSFull + st, it >> 1);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v0[32], v1[32];
        float mx0, mx1;
        const uint32_t src = tmem + lane_base + kTmS + 128 * st + 64 * hf;
        tmem_ld32_max(src, v0, mx0);
        tmem_ld32_max(src + 32, v1, mx1);
        tmem_wait_ld();
        // ---- visibility
        uint32_t w0 = 0xffffffffu, w1 = 0xffffffffu;
        if (s < a.drafts) {
          w0 = tree_draft_word(a, sg.b, tok, 4 * s + 2 * hf);
          w1 = tree_draft_word(a, sg.b, tok, 4 * s + 2 * hf + 1);
        } else {
          const int room = lim - (s - a.drafts) * kStep - 64 * hf;
          w0 = first_bits(room);
          w1 = first_bits(room - 32);
        }
        if (!__all_sync(0xffffffffu, (w0 & w1) == 0xffffffffu)) {
          mx0 = mx1 = kNegInf;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!((w0 >> k) & 1u)) v0[k] = __float_as_uint(kNegInf);
            if (!((w1 >> k) & 1u)) v1[k] = __float_as_uint(kNegInf);
            mx0 = fmaxf(mx0, __uint_as_float(v0[k]));
            mx1 = fmaxf(mx1, __uint_as_float(v1[k]));
          }
        }
        float mx = fmaxf(mx0, mx1), other;
        if (!(ok = exchange(mx, other))) break;
        mx = fmaxf(mx, other);
        // max S c = c max S (c > 0); a row that sees nothing stays at -inf
        const float top = mx * cf, head = tree_head(top, kHead);
        const float mn = top > m + (head == 0.f ? 0.f : kHead + kLazy) || m == kNegInf ? top - head : m;
        const float ref = mn == kNegInf ? 0.f : mn;
        const float2 c2 = make_float2(cf, cf), n2 = make_float2(-ref, -ref);
        float2 s0 = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
        uint32_t pk[32];
        auto half = [&](const uint32_t (&v)[32], uint32_t* out) {
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float2 t0 = ffma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, n2);
            float2 t1 = ffma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), c2, n2);
            t0 = make_float2(ex2_approx(t0.x), ex2_approx(t0.y));
            t1 = make_float2(ex2_approx(t1.x), ex2_approx(t1.y));
            s0 = fadd2(s0, t0);
            s1 = fadd2(s1, t1);
            const __half2 h0 = __floats2half2_rn(t0.x, t0.y), h1 = __floats2half2_rn(t1.x, t1.y);
            out[k / 2] = *reinterpret_cast<const uint32_t*>(&h0);
            out[k / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          }
        };
        half(v0, pk);
        half(v1, pk + 16);
        const float al = m == kNegInf ? 0.f : ex2_approx(m - ref);
        l = l * (mn == m ? 1.f : al) + ((s0.x + s0.y) + (s1.x + s1.y));
        // ---- O and P belong to the previous step's PV until it is done
        if (it > 0) {
          ok = wait(kPvDone + ((it - 1) & 1), (it - 1) >> 1);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        if (s > sg.s0 && __any_sync(0xffffffffu, mn != m)) {
          const float f = mn == m ? 1.f : al;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[16];
            const uint32_t oc = tmem + lane_base + kTmO + (D / 2) * hf + 16 * c;
            tmem_ld16(oc, x);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
            tmem_st16(oc, x);
          }
        }
        tmem_st32(tmem + lane_base + kTmP + 32 * hf, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kPReady));
        m = mn;
      }
      if (!ok) break;
      // ---- the segment's share: O from TMEM, l of both halves
      float l_other;
      if (!(ok = exchange(l, l_other))) break;
      l = tree_sum(l + l_other, fin);
      ok = wait(kPvDone + ((it - 1) & 1), (it - 1) >> 1);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (sg.s0 > 0 ? 0 : 1);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[16];
        const int ch = (D / 2) * hf + 16 * c;
        tmem_ld16(tmem + lane_base + kTmO + ch, x);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 y = make_float4(__uint_as_float(x[k]), __uint_as_float(x[k + 1]), __uint_as_float(x[k + 2]),
                                       __uint_as_float(x[k + 3]));
          if constexpr (CL) {  // the raw ring is free: every tile has been converted
            *reinterpret_cast<float4*>(smem + 4 * (r * D) + 16 * share_chunk(r, (ch + k) / 4)) = y;
          } else if (whole) {
            tree_write_out<D, kHead>(a, sg.b, sg.hkv, rr, ch + k, y, m, l);
          } else if (in && QATTN_IN_BOUNDS(slot < a.slots)) {
            // chunks of four channels, each for all rows: a warp writes 512 consecutive bytes
            *reinterpret_cast<float4*>(a.part_o + ((slot * (D / 4) + (ch + k) / 4) * kRows + r) * 4) = y;
          }
        }
      }
      if constexpr (CL) {
        if (hf == 0) {
          float* ml = reinterpret_cast<float*>(smem + 4 * kRows * D);
          ml[r] = m;
          ml[kRows + r] = l;
        }
      } else if (!whole && in && hf == 0 && QATTN_IN_BOUNDS(slot < a.slots)) {
        a.part_m[slot * kRows + r] = m;
        a.part_l[slot * kRows + r] = l;
      }
      tc_fence_before();  // the next segment's MMAs overwrite O
    }
    if (!ok) *abort_flag = 1;
  } else if (warp >= 12) {
    // -------------------------------------------------------------- codes -> fp16
    // Thread: 16-byte chunk 4 cb + cc of rows rw, rw + RS, ...  The eight lanes of an
    // access take four chunks of rows r and r ^ 5, which differ in the swizzle's
    // low and high bit: eight bank groups for the loads and for the stores.
    constexpr int NB = D / 64, RS = 32 / NB, CH = kStep / RS;
    const int tid = threadIdx.x & 127;
    const int cc = tid & 3, cb = NB == 2 ? (tid >> 3) & 1 : 0;
    const int u = tid >> (3 + NB - 1);  // row pair: 4 of an 8-row group
    const int rw = 8 * (u >> 2) + ((u & 3) ^ (((tid >> 2) & 1) * 5));
    const int chunk = 4 * cb + cc;
    const uint32_t src0 = rw * D + 16 * (chunk ^ ((D == 128) ? (rw & 7) : ((rw >> 1) & 3)));
    const uint32_t dst0 = cb * (kStep * 128) + rw * 128;
    const uint32_t c0 = ((2 * cc) ^ (rw & 7)) << 4, c1 = ((2 * cc + 1) ^ (rw & 7)) << 4;
    uint4 v[CH];  // a tile's codes: all loads before the first store
    auto load = [&](uint32_t slot) {
#pragma unroll
      for (int i = 0; i < CH; ++i) v[i] = lds128(raw(slot) + src0 + RS * D * i);
    };
    auto convert = [&](uint32_t dst) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        uint32_t h[8];
        codes4_to_f16x2(v[i].x, h[0], h[1]);
        codes4_to_f16x2(v[i].y, h[2], h[3]);
        codes4_to_f16x2(v[i].z, h[4], h[5]);
        codes4_to_f16x2(v[i].w, h[6], h[7]);
        sts128(dst + dst0 + RS * 128 * i + c0, h[0], h[1], h[2], h[3]);
        sts128(dst + dst0 + RS * 128 * i + c1, h[4], h[5], h[6], h[7]);
      }
    };
    bool ok = true;
    uint32_t it = 0, nd = 0;
    uint32_t slot = 0, lap = 0;  // the raw tile to convert next: counted, not divided
    while (ok && next_segment()) {
      bool loaded = false;  // v holds the next tile already
      for (int s = sg.s0; ok && s < sg.s1; ++s, ++it) {
        const uint32_t st = it & 1;
        if (s < a.drafts) {
          ok = encode(2 * it, s, threadIdx.x - 128, nd);
          ++nd;
          if (!ok) break;
        }
#pragma unroll 1  // (unrolled: instruction fetches, 104 us against 98 for eight 26-node trees)
        for (uint32_t kv = 0; kv < 2; ++kv) {
          if (!loaded) {
            if (!(ok = wait(kRawFull + slot, lap))) break;
            load(slot);
          }
          if (it >= 2 && !(ok = wait((kv ? kPvDone : kSFull) + st, (it >> 1) - 1))) break;
          convert(kv ? v16(st) : k16(st));
          mbar_arrive(bar(kRawEmpty + slot));
          if (++slot == kRaw) {
            slot = 0;
            ++lap;
          }
          // the next tile's loads go out ahead of the fence, if it is there
          loaded = (kv == 0 || s + 1 < sg.s1) && mbar_test(bar(kRawFull + slot), lap & 1);
          if (loaded) load(slot);
          fence_proxy_async_smem();
          mbar_arrive(bar((kv ? kVFull : kKFull) + st));
        }
      }
    }
    if (!ok) *abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (CL) {
    // ---- join the cluster: CTA `rank` writes rows rank, rank + cluster, ...  Every
    // CTA reaches both barriers, one that gave up on a wait too
    const int rank = static_cast<int>(cluster_rank());
    if (threadIdx.x == 0) tmem_slot[2] = sg.s0 < sg.s1 ? 1u : 0u;  // a part of no steps has no share
    cluster_sync();
    const uint32_t ml = base + 4 * kRows * D, flags = smem_u32(tmem_slot + 2);
    for (int idx = threadIdx.x; idx < (kRows / a.cluster) * (D / 4); idx += kThreads) {
      const int r = rank + a.cluster * (idx / (D / 4)), c = 4 * (idx % (D / 4));
      if (sg.rb * kRows + r >= a.G * a.T) continue;
      float mc[kTreeCluster], lc[kTreeCluster], mx = kNegInf, lt = 0.f;
      float4 y[kTreeCluster], x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kTreeCluster; ++q) {
        mc[q] = kNegInf;
        if (q < a.cluster && ld_cluster_u32(cluster_addr(flags, q))) {
          mc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(ml + 4 * r, q)));
          lc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(ml + 4 * (kRows + r), q)));
          y[q] = ld_cluster_f4(cluster_addr(base + 4 * (r * D) + 16 * share_chunk(r, c / 4), q));
        }
      }
#pragma unroll
      for (int q = 0; q < kTreeCluster; ++q) mx = fmaxf(mx, mc[q]);
#pragma unroll
      for (int q = 0; q < kTreeCluster; ++q) {
        if (mc[q] == kNegInf) continue;
        const float f = ex2_approx(mc[q] - mx);
        lt = fmaf(f, lc[q], lt);
        x.x = fmaf(f, y[q].x, x.x);
        x.y = fmaf(f, y[q].y, x.y);
        x.z = fmaf(f, y[q].z, x.z);
        x.w = fmaf(f, y[q].w, x.w);
      }
      tree_write_out<D, kHead>(a, sg.b, sg.hkv, sg.rb * kRows + r, c, x, mx, lt);
    }
    cluster_sync();  // no CTA leaves while another reads its share
  }
}

// The join for 128 rows a head: a lane for a row, a warp for four channels of it and
// every SW-th share (blockIdx.y: 32 rows, then 16 / SW channels), so that every load of
// a share takes 512 consecutive bytes; eight shares' loads in flight.
template <int D, int SW>
__global__ void __launch_bounds__(kTreeJoinThreads) tree_join_rows_kernel(const TreeArgs a) {
  constexpr int U = 8, W = kTreeJoinThreads / 32;
  __shared__ float part[SW > 1 ? 6 : 1][W][32];  // m, l and the channels of a warp's shares
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sw = warp % SW;
  const int r = 32 * (blockIdx.y % 4) + lane;
  const int c = 4 * ((W / SW) * (blockIdx.y / 4) + warp / SW);
  const TreeOwners own = tree_owners(a, kStep, blockIdx.x);
  const int rr = own.rb * kRows + r;
  const bool in = rr < a.G * a.T;
  pdl_wait();
  pdl_trigger();
  float m = kNegInf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto scale = [&](float f) {
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  };
  auto add = [&](float w, float lw, float4 y) {
    l = fmaf(w, lw, l);
    o.x = fmaf(w, y.x, o.x);
    o.y = fmaf(w, y.y, o.y);
    o.z = fmaf(w, y.z, o.z);
    o.w = fmaf(w, y.w, o.w);
  };
  if (own.steps > 0) {  // (else nothing is visible: no cached row and no draft)
    if (own.c0 == own.c1) return;  // written whole
    for (int cb = own.c0 + sw; cb <= own.c1; cb += SW * U) {
      float mc[U], lc[U], mn = m;
      float4 y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int ci = cb + SW * i;
        const size_t slot = 2 * static_cast<size_t>(ci) + (ci == own.c0 ? 1 : 0);
        mc[i] = kNegInf;
        if (in && ci <= own.c1 && QATTN_IN_BOUNDS(slot < a.slots)) {
          mc[i] = a.part_m[slot * kRows + r];
          lc[i] = a.part_l[slot * kRows + r];
          y[i] = *reinterpret_cast<const float4*>(a.part_o + ((slot * (D / 4) + c / 4) * kRows + r) * 4);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) mn = fmaxf(mn, mc[i]);
      if (mn == kNegInf) continue;
      scale(m == kNegInf ? 0.f : ex2_approx(m - mn));
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (mc[i] != kNegInf) add(ex2_approx(mc[i] - mn), lc[i], y[i]);
      m = mn;
    }
  }
  if constexpr (SW > 1) {
    const float mine[6] = {m, l, o.x, o.y, o.z, o.w};
#pragma unroll
    for (int k = 0; k < 6; ++k) part[k][warp][lane] = mine[k];
    __syncthreads();
    if (sw != 0) return;
    float mn = m;
#pragma unroll
    for (int i = 1; i < SW; ++i) mn = fmaxf(mn, part[0][warp + i][lane]);
    if (mn != kNegInf) {
      scale(m == kNegInf ? 0.f : ex2_approx(m - mn));
#pragma unroll
      for (int i = 1; i < SW; ++i) {
        const float mw = part[0][warp + i][lane];
        if (mw != kNegInf)
          add(ex2_approx(mw - mn), part[1][warp + i][lane],
              make_float4(part[2][warp + i][lane], part[3][warp + i][lane], part[4][warp + i][lane],
                          part[5][warp + i][lane]));
      }
      m = mn;
    }
  }
  tree_write_out<D, kHead>(a, own.b, own.hkv, rr, c, o, m, l);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = Cfg<D>::kBytes;
  cudaError_t e;
  if (a.cluster > 0) {
    e = cudaFuncSetAttribute(tree_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(tree_tc_kernel<D, true>, dim3(a.ctas), dim3(kThreads), a.cluster, smem, s, tk, tv, a);
  }
  e = cudaFuncSetAttribute(tree_tc_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_tc_kernel<D, false>, dim3(a.ctas), dim3(kThreads), smem, s, tk, tv, a);
  if (e != cudaSuccess) return e;
  const int heads = a.B * a.Hkv * a.blocks;
  if (a.ctas < kJoinShares * heads)
    return launch_pdl(tree_join_rows_kernel<D, 1>, dim3(heads, 4 * (D / 16)), dim3(kTreeJoinThreads), 0, s, a);
  return launch_pdl(tree_join_rows_kernel<D, 4>, dim3(heads, 4 * (D / 4)), dim3(kTreeJoinThreads), 0, s, a);
}

}  // namespace

unsigned int check_take_tree_tc() { return check_take_local(); }

cudaError_t launch_tree_tc(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(tk, tv, a, s) : launch_d<128>(tk, tv, a, s);
}

}  // namespace qattn
