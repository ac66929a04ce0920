// Attention of a few drafted tokens over an int8 KV cache (qattn_tree_decode),
// warp-level kernel: 16 query rows (query head of the KV group, token) at a
// time against the cached K and V codes and the drafts' own codes.
//
// Mathematics.  S = q . k of the codes, an exact integer (|S| <= 128 * 127^2 <
// 2^21); t = S c with c = fp32(fp32(sq * sm_scale) * log2 e); over the visible
// keys P = 2^(t - m) with m a running maximum, l = sum P, O = sum P v; the
// parts of a head (steps of 32 keys dealt to warps, shares of steps dealt to
// CTAs) are joined by 2^(m_part - m).  P is rounded once, to fp16, for the PV
// product; l sums the unrounded P in fp32.  m lies 15 below the running maximum, so P
// fills fp16's range: a key down to 2^-29 of the row's largest (20 nats) is off by at
// most 2^-11, an eighth of a step of the bf16 output, independently from key to key;
// further down by at most 2^-40 of the largest.
//
// What it cannot do without: the cache's bytes, 2 D per key and KV head.  The rows
// of one KV head are few, so the codes are converted in registers as they are used
// (int8 -> exact fp16, ~10 instructions per 8 codes) and multiplied by
// mma.m16n8k16: at 16 rows a 128-key tile costs ~510 tensor cycles and ~400
// issue cycles of an SM against ~1460 cycles of its share of HBM.  What bounds it:
// a warp's chain (scores, maximum, exponentials, PV) a step of 32 keys at two warps a
// scheduler.  Measured: one token over 4K rows of 8 KV heads 9.6 us (launch, first
// tiles and the cluster's join; floor 1.3), four tokens for 16 sequences of 0.2 to
// 4.5K rows 27.0 us = 2.9 TB/s (floor 11.8, 42% of DRAM's time).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"
#include "tree_common.cuh"

namespace qattn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = kTreeWarpStep;  // keys per warp step
constexpr int kHead = 15;             // of the exponentials' reference (tree_head)
// Shares a head, on average, from which four warps join a row.  One against four warps,
// us: 2.4 shares 26.7 / 27.6 (d = 128; 16 sequences of 0.2 to 4.5K rows), 4.8 shares 61.5 / 59.5
// (64 heads of 5K to 32K), 38 shares 31.3 / 22.5 (8 heads of 32K).
constexpr int kJoinShares = 4;
constexpr int kRing = 3;   // stages of a warp's ring (K and V of one step each)

template <int D>
struct WarpSmem {
  static constexpr int kTile = kStep * D;       // bytes of a step's K (or V) codes
  static constexpr int kStage = 2 * kTile;
  static constexpr int kWarp = kRing * kStage;  // one warp's ring
  static constexpr int kDraft = kWarps * kWarp;  // the drafted step's codes
  static constexpr int kBytes = kDraft + kStage + 1024;
  static_assert(kTreeRows * D * 4 <= kStage, "a CTA's O does not fit the drafted step's room");
  static_assert(kTreeRows * D * 4 <= kWarp, "a warp's O does not fit its ring");
};

// Byte offset of 16-byte chunk c of row r in a tile stored with the 128-byte
// (D = 128) or 64-byte (D = 64) swizzle.
template <int D>
__device__ __forceinline__ int swz(int r, int c) {
  return r * D + 16 * (c ^ ((D == 128) ? (r & 7) : ((r >> 1) & 3)));
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Words x, y (four channels of two keys) -> four f16x2 {x_e, y_e}, exact.
__device__ __forceinline__ void pair_f16x2(uint32_t x, uint32_t y, uint32_t (&o)[4]) {
  const uint32_t p01 = __byte_perm(x, y, 0x5140u) ^ 0x80808080u;
  const uint32_t p23 = __byte_perm(x, y, 0x7362u) ^ 0x80808080u;
  o[0] = __byte_perm(p01, 0x64646464u, 0x4140u);
  o[1] = __byte_perm(p01, 0x64646464u, 0x4342u);
  o[2] = __byte_perm(p23, 0x64646464u, 0x4140u);
  o[3] = __byte_perm(p23, 0x64646464u, 0x4342u);
#pragma unroll
  for (int e = 0; e < 4; ++e) asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(o[e]) : "r"(0x64806480u));
}

// Place of 16-byte chunk c of row r of a warp's O in shared memory.
template <int D>
__device__ __forceinline__ int join_chunk(int r, int c) {
  return c ^ (((c >> ((D == 128) ? 3 : 2)) & 3) + 4 * (r & 1));
}

// ------------------------------------------------------------------ attention
// Each CTA takes an equal share of the flattened list of steps (sequence, KV head,
// 16-row block, step): balance to one step whatever the lengths.
// Each run of steps inside one head is a segment; its steps go round the four
// warps, each with its own ring of TMA tiles and its own (m, l, O), so the main
// loop has no CTA barrier.  A head's drafted steps come first and are encoded
// by the warp that takes them while its first tiles are in flight.
template <int D, bool CL>
__global__ void __launch_bounds__(kThreads, 2)
    tree_warp_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const TreeArgs a) {
  using SM = WarpSmem<D>;
  constexpr int KS = D / 16;   // k-steps of QK^T = words of K a lane holds per key
  constexpr int NT = D / 8;    // n-tiles of PV
  constexpr int VW = NT / 4;   // V words a lane reads per key
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[kWarps][kRing];
  __shared__ float red_m[kWarps][kTreeRows], red_l[kWarps][kTreeRows];
  __shared__ float cl_m[kTreeRows], cl_l[kTreeRows];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + warp * SM::kWarp;
  if (lane == 0) {
    for (int s = 0; s < kRing; ++s) mbar_init(smem_u32(&full[warp][s]), 1);
    fence_mbar_init();
    if (warp == 0) {
      abort_flag = 0;
      if (a.Nk > 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
    }
  }
  pdl_wait();
  pdl_trigger();  // after the wait: the join reads the lengths before its own
  TreeWalk walk;
  if constexpr (!CL) walk = tree_walk(a, kStep);
  __syncthreads();  // the abort flag is set
  const int R = a.G * a.T;
  uint32_t used = 0;  // tiles this warp has taken through its ring
  uint32_t sent = 0;  // lane 0: those it has issued

  TreeSeg sg;
  if constexpr (CL) walk = tree_cluster_walk(a, kStep, sg);
  while (CL || tree_next(a, kStep, walk, sg)) {
    const int bkv = sg.b * a.Hkv + sg.hkv;
    const int nd = a.drafts;  // drafted steps of a head
    // this warp's steps: sg.s0 + warp, + kWarps, ...; the first cached one
    int first = sg.s0 + warp;
    while (first < nd && first < sg.s1) first += kWarps;
    const int ntile = first < sg.s1 ? (sg.s1 - first + kWarps - 1) / kWarps : 0;
    auto issue = [&](int i) {  // lane 0: tile i of this warp
      const uint32_t q = used + i, slot = q % kRing;
      const uint32_t bar = smem_u32(&full[warp][slot]);
      const int key = (first + i * kWarps - nd) * kStep;
      sent = q + 1;
      (void)QATTN_IN_BOUNDS(key >= 0 && key < a.Nk && bkv < a.B * a.Hkv);  // TMA coordinates
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(SM::kStage));
      tma_load_3d(smem_u32(ring + slot * SM::kStage), &tmK, bar, 0, key, bkv);
      tma_load_3d(smem_u32(ring + slot * SM::kStage + SM::kTile), &tmV, bar, 0, key, bkv);
    };
    if (lane == 0)
      for (int i = 0; i < min(kRing - 1, ntile); ++i) issue(i);
    // at most 16 drafts, one step: the CTA encodes its codes while the first tiles
    // are in flight
    const bool draft = sg.s0 < nd && sg.s0 < sg.s1;
    if (draft) {
      uint8_t* st = smem + SM::kDraft;
      tree_encode_drafts<D>(a, sg.b, sg.hkv, 0, kStep, threadIdx.x, kThreads,
                            [&](int r, int c) { return st + swz<D>(r, c); },
                            [&](int r, int c) { return st + SM::kTile + swz<D>(r, c); });
    }

    // ---- this lane's rows g and g + 8 of the block: codes, factor, key limit
    uint32_t qa[KS][4];
    float cf[2];
    bool fin[2] = {true, true};
    int lim[2];
    uint32_t tok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int rr = sg.rb * kTreeRows + g + 8 * h;
      const bool in = rr < R;
      const int hq = in ? rr / a.T : 0, i = in ? rr % a.T : 0;
      const size_t row = (static_cast<size_t>(sg.b) * a.Hq + sg.hkv * a.G + hq) * a.T + i;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q_codes) + row * D + (D / 4) * t4;
#pragma unroll
      for (int w4 = 0; w4 < KS / 4; ++w4) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (in && QATTN_IN_BOUNDS(row < a.rows_total)) x = *reinterpret_cast<const uint4*>(src + 16 * w4);
        codes4_to_f16x2(x.x, qa[4 * w4 + 0][h], qa[4 * w4 + 0][2 + h]);
        codes4_to_f16x2(x.y, qa[4 * w4 + 1][h], qa[4 * w4 + 1][2 + h]);
        codes4_to_f16x2(x.z, qa[4 * w4 + 2][h], qa[4 * w4 + 2][2 + h]);
        codes4_to_f16x2(x.w, qa[4 * w4 + 3][h], qa[4 * w4 + 3][2 + h]);
      }
      cf[h] = in ? tree_factor(a, sg.b, sg.hkv * a.G + hq, fin[h]) : 1.f;
      lim[h] = tree_limit(a, sg.len, i);
      tok[h] = i;
    }
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};

    // One step of 32 keys in stage `st`: vis[h] is the visibility word of row h
    // (bit = key of the step) when masked.
    auto step = [&](const uint8_t* st, bool masked, const uint32_t (&vis)[2]) {
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int w4 = 0; w4 < KS / 4; ++w4) {
          const uint4 kw = *reinterpret_cast<const uint4*>(st + swz<D>(8 * j + g, (KS / 4) * t4 + w4));
          const uint32_t kx[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t b0, b1;
            codes4_to_f16x2(kx[e], b0, b1);
            const uint32_t(&q)[4] = qa[4 * w4 + e];
            mma16816(s[j], q[0], q[1], q[2], q[3], b0, b1);
          }
        }
      }
      if (masked) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((vis[e >> 1] >> (8 * j + 2 * t4 + (e & 1))) & 1u)) s[j][e] = kNegInf;
      }
      // running maxima less kHead: max S c = c max S (c > 0); -inf stays -inf
      float al[2], ref[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = kNegInf;
#pragma unroll
        for (int j = 0; j < 4; ++j) x = fmax3(x, s[j][2 * h], s[j][2 * h + 1]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float top = x * cf[h];
        const float mn = fmaxf(m[h], top - tree_head(top, kHead));
        ref[h] = (mn == kNegInf) ? 0.f : mn;
        al[h] = (m[h] == kNegInf) ? 0.f : ex2_approx(m[h] - ref[h]);
        m[h] = mn;
      }
      if (!__all_sync(0xffffffffu, al[0] == 1.f && al[1] == 1.f)) {
        l[0] *= al[0];
        l[1] *= al[1];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          o[n][0] *= al[0];
          o[n][1] *= al[0];
          o[n][2] *= al[1];
          o[n][3] *= al[1];
        }
      }
      uint32_t pa[4][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pr[e] = ex2_approx(fmaf(s[j][e], cf[e >> 1], -ref[e >> 1]));
        }
        l[0] += pr[0] + pr[1];
        l[1] += pr[2] + pr[3];
        pa[j][0] = pack_half2(pr[0], pr[1]);
        pa[j][1] = pack_half2(pr[2], pr[3]);
      }
      const uint8_t* sv = st + SM::kTile;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t vw[4][VW];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = 16 * kk + 2 * t4 + (u & 1) + 8 * (u >> 1);
          const uint8_t* src = sv + swz<D>(key, (4 * VW * g) >> 4) + ((4 * VW * g) & 15);
          if constexpr (VW == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(src);
            vw[u][0] = x.x;
            vw[u][1] = x.y;
            vw[u][2] = x.z;
            vw[u][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            vw[u][0] = x.x;
            vw[u][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          uint32_t b0[4], b1[4];
          pair_f16x2(vw[0][w], vw[1][w], b0);
          pair_f16x2(vw[2][w], vw[3][w], b1);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma16816(o[4 * w + e], pa[2 * kk][0], pa[2 * kk][1], pa[2 * kk + 1][0], pa[2 * kk + 1][1],
                     b0[e], b1[e]);
        }
      }
    };

    // ---- this warp's steps, the drafted one (warp 0's first) among them
    if (draft) __syncthreads();
    const bool mine_draft = draft && warp == 0;
    for (int i = mine_draft ? -1 : 0; i < ntile; ++i) {
      const uint8_t* st = smem + SM::kDraft;
      uint32_t vis[2];
      bool masked = true;
      if (i < 0) {
        vis[0] = tree_draft_word(a, sg.b, tok[0], 0);
        vis[1] = tree_draft_word(a, sg.b, tok[1], 0);
      } else {
        if (lane == 0 && i + kRing - 1 < ntile) issue(i + kRing - 1);
        const uint32_t q = used + i, slot = q % kRing;
        const bool ok = mbar_wait(smem_u32(&full[warp][slot]), (q / kRing) & 1, &abort_flag, a.err, kErrTimeout);
        if (!__all_sync(0xffffffffu, ok)) break;
        st = ring + slot * SM::kStage;
        const int key = (first + i * kWarps - nd) * kStep;
        const int room0 = lim[0] - key, room1 = lim[1] - key;  // visible keys of the step
        masked = __any_sync(0xffffffffu, room0 < kStep || room1 < kStep);
        vis[0] = first_bits(room0);
        vis[1] = first_bits(room1);
      }
      step(st, masked, vis);
      __syncwarp();  // the stage is read
    }
    used += ntile;

    // ---- join the four warps (their rings are free)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      l[h] = tree_sum(l[h], fin[h]);
      if (t4 == 0) {
        red_m[warp][g + 8 * h] = m[h];
        red_l[warp][g + 8 * h] = l[h];
      }
    }
    __syncthreads();
    if (abort_flag) {  // a wait ran out (every thread sees it here)
      // every load this warp issued lands before the CTA may exit
      if (lane == 0)
        for (uint32_t back = 1; back <= min(sent, static_cast<uint32_t>(kRing)); ++back) {
          const uint32_t q = sent - back;
          volatile int never = 0;
          mbar_wait(smem_u32(&full[warp][q % kRing]), (q / kRing) & 1, &never, a.err, kErrTimeout);
        }
      break;
    }
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, red_m[w][g + 8 * h]);
      const float f = (m[h] == kNegInf) ? 0.f : ex2_approx(m[h] - mx);
      // n-tile n, column 2 t4 (+ 1) is channel NT * column + n; 16-byte chunks XORed
      // so that the eight lanes of a store hit eight bank groups
#pragma unroll
      for (int cl = 0; cl < 2; ++cl) {
#pragma unroll
        for (int n = 0; n < NT; n += 4) {
          const int ch = (NT * (2 * t4 + cl) + n) / 4;
          *reinterpret_cast<float4*>(mine + (g + 8 * h) * D + 4 * join_chunk<D>(g, ch)) =
              make_float4(o[n][2 * h + cl] * f, o[n + 1][2 * h + cl] * f, o[n + 2][2 * h + cl] * f,
                          o[n + 3][2 * h + cl] * f);
        }
      }
    }
    __syncthreads();
    const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (sg.s0 > 0 ? 0 : 1);
    float* share = reinterpret_cast<float*>(smem + SM::kDraft);  // CL: this CTA's O, for the cluster
    for (int idx = threadIdx.x; idx < kTreeRows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), c = 4 * (idx % (D / 4));
      float mx = kNegInf, lt = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, red_m[w][r]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = red_m[w][r];
        lt += (mw == kNegInf) ? 0.f : red_l[w][r] * ex2_approx(mw - mx);
        const float4 y =
            *reinterpret_cast<const float4*>(smem + w * SM::kWarp + 4 * (r * D + 4 * join_chunk<D>(r, c / 4)));
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if constexpr (CL) {
        *reinterpret_cast<float4*>(share + r * D + c) = x;
        if (c == 0) {
          cl_m[r] = mx;
          cl_l[r] = lt;
        }
      } else if (whole) {
        tree_write_out<D, kHead>(a, sg.b, sg.hkv, sg.rb * kTreeRows + r, c, x, mx, lt);
      } else if (QATTN_IN_BOUNDS(slot < a.slots)) {
        *reinterpret_cast<float4*>(a.part_o + (slot * kTreeRows + r) * D + c) = x;
        if (c == 0) {
          a.part_m[slot * kTreeRows + r] = mx;
          a.part_l[slot * kTreeRows + r] = lt;
        }
      }
    }
    if constexpr (CL) break;
    fence_proxy_async_smem();  // the rings go back to the TMA engine
    __syncthreads();
  }
  if constexpr (CL) {
    // ---- join the cluster: CTA `rank` writes rows rank, rank + cluster, ...  Every
    // CTA reaches both barriers, one that gave up on a wait too
    cluster_sync();
    const int rank = static_cast<int>(cluster_rank());
    for (int idx = threadIdx.x; idx < (kTreeRows / a.cluster) * (D / 4); idx += kThreads) {
      const int r = rank + a.cluster * (idx / (D / 4)), c = 4 * (idx % (D / 4));
      if (sg.rb * kTreeRows + r >= R) continue;
      float mc[kTreeCluster], lc[kTreeCluster], mx = kNegInf, lt = 0.f;
      float4 y[kTreeCluster], x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kTreeCluster; ++q) {
        mc[q] = kNegInf;
        if (q < a.cluster) {
          mc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(smem_u32(&cl_m[r]), q)));
          lc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(smem_u32(&cl_l[r]), q)));
          y[q] = ld_cluster_f4(cluster_addr(smem_u32(smem + SM::kDraft) + 4 * (r * D + c), q));
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
      tree_write_out<D, kHead>(a, sg.b, sg.hkv, sg.rb * kTreeRows + r, c, x, mx, lt);
    }
    cluster_sync();  // no CTA leaves while another reads its share
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = WarpSmem<D>::kBytes;
  cudaError_t e;
  if (a.cluster > 0) {
    e = cudaFuncSetAttribute(tree_warp_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(tree_warp_kernel<D, true>, dim3(a.ctas), dim3(kThreads), a.cluster, smem, s, tk, tv,
                              a);
  }
  e = cudaFuncSetAttribute(tree_warp_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(tree_warp_kernel<D, false>, dim3(a.ctas), dim3(kThreads), smem, s, tk, tv, a);
  if (e != cudaSuccess) return e;
  // a head in few shares: a warp for a row
  const int heads = a.B * a.Hkv * a.blocks;
  if (a.ctas < kJoinShares * heads)
    return launch_pdl(tree_join_kernel<D, kHead, kTreeRows, kStep, 1>, dim3(heads, kTreeRows / 4),
                      dim3(kTreeJoinThreads), 0, s, a);
  return launch_pdl(tree_join_kernel<D, kHead, kTreeRows, kStep, 4>, dim3(heads, kTreeRows), dim3(kTreeJoinThreads), 0,
                    s, a);
}

}  // namespace

unsigned int check_take_tree_warp() { return check_take_local(); }

cudaError_t launch_tree_warp(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                             cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(tk, tv, a, s) : launch_d<128>(tk, tv, a, s);
}

}  // namespace qattn
