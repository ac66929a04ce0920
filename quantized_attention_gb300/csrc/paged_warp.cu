// Attention over a paged 8-bit KV cache (qattn_paged_fwd), warp-level kernel: up to 16
// query rows (token, query head of the KV group) of a KV head at a time against the cached
// codes.
//
// Mathematics.  Q's rows are brought to fp16 by a power of two each (exact, see
// pg_row_shift), the codes of K and V are exact in fp16 (|int8| <= 127, e4m3 <= 448),
// so S = q . k is a sum of exact products in fp32.  With a page's scales s_k, s_v:
//   t = S c + log2 s_v,  c = row factor * s_k  (row factor: sm_scale log2 e and the
//       row's power of two)
//   P = 2^(t - m),  m a reference 15 below the running maximum of t
//   O = sum P vc,   l = sum P / s_v,   out = O / l,   lse = ln 2 (m + log2 l)
// The V scale rides in the exponent: P, rounded once to fp16 for the PV product, keeps
// its eleven bits where P s_v, the key's part in O, is down to 2^-29 of the row's
// largest, and no key costs an instruction more than with one scale for all.  l sums
// the unrounded P in fp32.  Parts of a row (steps of 64 keys dealt to warps, shares of
// steps dealt to CTAs) are joined by 2^(m_part - m).
//
// What it cannot do without: the cache's bytes, 2 D per key and KV head.  32 sequences of
// 211 to 8191 rows, 8 KV heads of 128 channels (276 MB): 52 us, 5.3 TB/s, 78% of a copy; 8 of
// 16K to 32K in e4m3 (403 MB): 71 us, 83%.  Between these and the copy lie ~5 us of start
// (lengths, page numbers, the first tiles: each waits for the one before) and join, and a
// block's start in the middle of a share.  The keys are the
// products' M: S^T = K Q^T and O^T = V^T P^T by mma.m16n8k16, so that a decode step's few
// rows (N, eight at a time) leave no product half empty, and a lane holds 2 rows' worth of
// everything; P^T turns from result to operand by movmatrix.  The codes are widened in
// registers (~5 instructions for 4), which with the products is what a step takes: ~45% each of
// the ALU and the legacy tensor pipe at the rate of HBM.  Tiles of 32 keys lie in one page
// (pages of 32, 64 or 128 rows), one TMA box each at the page's plane of the pool.  A warp
// looks up the pages and scales of its next 16 steps at once, one half step a lane, ahead
// of their use.
#include "paged_common.cuh"

namespace qattn {
namespace {

constexpr int kStep = kPagedWarpStep;
constexpr int kHead = 15;   // of the exponentials' reference (pg_head)
constexpr int kTileKeys = 32;
// Tiles of a warp's ring (K or V of half a step).  3, 4, 5, 6: 32 sequences 53.3, 53.2, 54.9,
// 56.5 us; 8 of 16K to 32K rows 71.9, 71.5, 73.3, 74.2.
constexpr int kRing = 4;
static_assert(kStep == 2 * kTileKeys, "a step is two tiles of K and two of V");

template <int D, int NB, int W>
struct WarpSmem {
  static constexpr int kTile = kTileKeys * D;
  static constexpr int kWarp = kRing * kTile;    // one warp's ring
  static constexpr int kShare = W * kWarp;       // a CTA's O
  static constexpr int kBytes = kShare + 8 * NB * D * 4 + 1024;
  static_assert(8 * NB * D * 4 <= kWarp, "a warp's O does not fit its ring");
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
// An 8 x 8 matrix of 16-bit values, two neighbours of a row a lane, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes of a word -> two f16x2, exact.
template <bool E4M3>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    lo = e4m3x2_to_f16x2(w & 0xffffu);
    hi = e4m3x2_to_f16x2(w >> 16);
  } else {
    codes4_to_f16x2(w, lo, hi);
  }
}
// Words x, y (four channels of two keys) -> four f16x2 {x_e, y_e}, exact.
template <bool E4M3>
__device__ __forceinline__ void widen_pair(uint32_t x, uint32_t y, uint32_t (&o)[4]) {
  widen4<E4M3>(__byte_perm(x, y, 0x5140u), o[0], o[1]);
  widen4<E4M3>(__byte_perm(x, y, 0x7362u), o[2], o[3]);
}

// Place of 16-byte chunk c of row r of a warp's O in shared memory: the eight lanes of a
// store hit eight bank groups.
__device__ __forceinline__ int join_chunk(int r, int c) { return c ^ ((r >> 1) & 3); }

// Pages and scales of a warp's 16 steps from `base` on, one half step a lane.
struct Window {
  int page;      // -1: no such page, its keys are hidden
  float ks, vs;
};

// ------------------------------------------------------------------ attention
// Each CTA takes an equal share of the flattened list of steps (sequence, KV head,
// row block, step), or (CL) its part of its cluster's block.  Each run of steps
// inside one block is a segment; its steps go round the W warps, each with its own
// ring of TMA tiles and its own (m, l, O), so the main loop has no CTA barrier.
// NB: eights of rows of a block.  A lane (g, t4) holds rows 2 t4 and 2 t4 + 1 of each eight
// in its results, row g of it in the products' N operands.
template <int D, bool E4M3, int NB, bool CL, int W>
__global__ void __launch_bounds__(32 * W, W == 4 ? 2 : 1)
    paged_warp_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedArgs a) {
  using SM = WarpSmem<D, NB, W>;
  constexpr int kThreads = 32 * W;
  constexpr int kRows = 8 * NB;
  constexpr int KS = D / 16;   // k-steps of K Q^T = words of K a lane holds per key
  constexpr int MT = D / 16;   // m-tiles of V^T P^T
  constexpr int VW = D / 32;   // V words a lane reads per key: channels 4 VW g ..
  extern __shared__ uint8_t raw_smem[];
  uint8_t* smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[W][kRing];
  __shared__ float red_m[W][kRows], red_l[W][kRows];
  __shared__ float cl_m[kRows], cl_l[kRows];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + warp * SM::kWarp;
  if (lane == 0) {
    for (int s = 0; s < kRing; ++s) mbar_init(smem_u32(&full[warp][s]), 1);
    fence_mbar_init();
    if (warp == 0) {
      abort_flag = 0;
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  __syncthreads();  // the abort flag is set
  pdl_wait();
  pdl_trigger();
  PagedWalk walk;
  PagedSeg sg;
  bool some = true;  // CL: the block has rows
  if constexpr (CL) some = pg_cluster_seg<kRows, kStep>(a, sg);
  else walk = pg_walk<kRows, kStep>(a, blockIdx.x, gridDim.x);
  if (!CL && threadIdx.x == kThreads - 32) pg_put_plan(a, walk);  // (the warp with the fewest steps)
  uint32_t used = 0;  // tiles this warp has taken through its ring
  uint32_t sent = 0;  // and issued

  while (CL ? some : pg_next<kRows, kStep>(a, walk, sg)) {
    const int len = sg.seq.len;
    // this warp's steps: sg.s0 + warp, + W, ...
    const int first = sg.s0 + warp;
    const int nstep = first < sg.s1 ? (sg.s1 - first + W - 1) / W : 0;
    auto key_of = [&](int i) { return (first + i * W) * kStep; };
    auto look_up = [&](int i0) {  // the window of steps i0 .. i0 + 15
      Window w{-1, 0.f, 0.f};
      const int i = i0 + (lane >> 1);
      if (i < nstep) {
        const int key = key_of(i) + kTileKeys * (lane & 1), j = key >> a.page_shift;
        if (key < len && QATTN_IN_BOUNDS(j < a.max_pages && sg.b < a.B)) {
          const int p = a.page_table[static_cast<size_t>(sg.b) * a.max_pages + j];
          if (p >= 0 && p < a.n_pages) {
            const size_t sc = static_cast<size_t>(p) * a.Hkv + sg.hkv;
            w.page = p;
            w.ks = a.k_scales[sc];
            w.vs = a.v_scales[sc];
          } else {
            atomicOr(a.err, kErrDomain);
          }
        }
      }
      return w;
    };
    // ---- row g of each eight: loads first, then the pages, then the first tiles, so that
    // one latency covers another
    uint4 xq[NB][D / 32];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int rr = sg.rb * kRows + 8 * nb + g, tok = rr / a.G;
      const int hq = sg.hkv * a.G + rr - tok * a.G;
      const uint16_t* src = a.q + sg.b * a.qsB + hq * a.qsH + tok * a.qsN + (D / 4) * t4;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        xq[nb][k] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < sg.seq.n && QATTN_IN_BOUNDS(sg.b < a.B && hq < a.Hq && tok < a.T))
          xq[nb][k] = *reinterpret_cast<const uint4*>(src + 8 * k);
      }
    }
    Window raw = look_up(0), nxt{-1, 0.f, 0.f};
    int base = 0;            // the first step of the current window,
    int pages = raw.page;    // its pages
    auto issue = [&](int n) {  // tile n: K, K, V, V of each step (the whole warp calls)
      const int i = n >> 2, o = 2 * (i - base) + (n & 1);
      const int pc = __shfl_sync(0xffffffffu, pages, o & 31), pn = __shfl_sync(0xffffffffu, nxt.page, o & 31);
      if (lane == 0) {
        const uint32_t slot = sent % kRing, bar = smem_u32(&full[warp][slot]);
        // a page that does not exist: any page of the pool stands in, its keys are hidden
        const int page = max(o < 32 ? pc : pn, 0);
        const int row = (key_of(i) + kTileKeys * (n & 1)) & ((1 << a.page_shift) - 1);
        (void)QATTN_IN_BOUNDS(page < a.n_pages && row >= 0 && row + kTileKeys <= (1 << a.page_shift));  // TMA coordinates
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(SM::kTile));
        tma_load_3d(smem_u32(ring + slot * SM::kTile), n & 2 ? &tmV : &tmK, bar, 0, row, page * a.Hkv + sg.hkv);
      }
      ++sent;
    };
    for (int n = 0; n < min(kRing, 4 * nstep); ++n) issue(n);
    if (nstep > 16) nxt = look_up(16);
    uint32_t qb[NB][KS][2];
    float rf[NB][2];   // of rows 2 t4, 2 t4 + 1: the factor,
    int lim[NB][2];    // the keys they see
    bool fin[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t w[4] = {xq[nb][k].x, xq[nb][k].y, xq[nb][k].z, xq[nb][k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool number = top < 0x7f800000u;  // else the row is NaN once it sees a key
      float up, down;
      pg_row_shift(top, up, down);
      const float f = __fmul_rn(__fmul_rn(a.sm_scale, kPgLog2e), down);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t w[4] = {xq[nb][k].x, xq[nb][k].y, xq[nb][k].z, xq[nb][k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = number ? bf16_bits_to_f32(w[e] & 0xffffu) * up : 0.f;
          const float hi = number ? __uint_as_float(w[e] & 0xffff0000u) * up : 0.f;
          qb[nb][2 * k + (e >> 1)][e & 1] = pack_half2(lo, hi);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 2 * t4 + x, rr = sg.rb * kRows + 8 * nb + r, tok = rr / a.G;
        rf[nb][x] = __shfl_sync(0xffffffffu, f, 4 * r);
        fin[nb][x] = __shfl_sync(0xffffffffu, number ? 1 : 0, 4 * r) != 0;
        // (a row that is none sees everything: its scores are 0, and it asks for no mask)
        lim[nb][x] = tok < sg.seq.n ? min(pg_limit(a, sg.seq, tok), len) : 0x7fffffff;
      }
    }
    // the current window: what its scales mean, and its halves out of the ordinary
    float wk, we, winv;
    uint32_t hidden, zero_v, bad;
    auto settle = [&](const Window& w) {
      const PageScale ps = pg_scale(w.ks, w.vs);
      pages = w.page;
      wk = ps.k;
      we = ps.e;
      winv = ps.inv;
      hidden = __ballot_sync(0xffffffffu, w.page < 0);
      zero_v = __ballot_sync(0xffffffffu, ps.keep == 0u);
      bad = __ballot_sync(0xffffffffu, ps.nan);
    };
    settle(raw);
    float o[NB][MT][4];  // channel slots g and g + 8 of m-tile p: channels 4 VW g + 2 p, + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int p = 0; p < MT; ++p) o[nb][p][0] = o[nb][p][1] = o[nb][p][2] = o[nb][p][3] = 0.f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb][0] = m[nb][1] = -kPgInf;
      l[nb][0] = l[nb][1] = 0.f;
    }

    for (int i = 0; i < nstep; ++i) {
      if (i - base == 16) {
        base = i;
        settle(nxt);
        nxt = Window{-1, 0.f, 0.f};
        if (i + 16 < nstep) nxt = look_up(i + 16);
      }
      const int q0 = 2 * (i - base), key = key_of(i);
      float ks[2], e[2], inv[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ks[x] = __shfl_sync(0xffffffffu, wk, q0 + x);
        e[x] = __shfl_sync(0xffffffffu, we, q0 + x);
        inv[x] = __shfl_sync(0xffffffffu, winv, q0 + x);
      }
      const uint32_t rare = ((hidden | zero_v | bad) >> q0) & 3u;
      int least = 0x7fffffff;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) least = min(least, min(lim[nb][0], lim[nb][1]));
      const bool masked = __any_sync(0xffffffffu, least - key < kStep || rare != 0u);
      auto tile = [&](const uint8_t*& at) {  // the next tile, once it is there
        const uint32_t slot = used % kRing;
        at = ring + slot * SM::kTile;
        const bool ok = mbar_wait(smem_u32(&full[warp][slot]), (used / kRing) & 1, &abort_flag, a.err, kErrTimeout);
        return __all_sync(0xffffffffu, ok);
      };
      auto done = [&](int n) {  // the tile has been read: its place takes the next one
        __syncwarp();
        ++used;
        if (n + kRing < 4 * nstep) issue(n + kRing);
      };
      // ---- scores: s[nb][x][j]: keys 32 x + 16 j + g (+ 8), rows 2 t4 (+ 1)
      float s[NB][2][2][4];
      bool ok = true;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* st;
        if (!(ok = tile(st))) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) s[nb][x][j][0] = s[nb][x][j][1] = s[nb][x][j][2] = s[nb][x][j][3] = 0.f;
#pragma unroll
          for (int w4 = 0; w4 < KS / 4; ++w4) {
            const uint4 u = *reinterpret_cast<const uint4*>(st + swz<D>(16 * j + g, (KS / 4) * t4 + w4));
            const uint4 v = *reinterpret_cast<const uint4*>(st + swz<D>(16 * j + g + 8, (KS / 4) * t4 + w4));
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t a0, a1, a2, a3;
              widen4<E4M3>(uw[q], a0, a2);
              widen4<E4M3>(vw[q], a1, a3);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816(s[nb][x][j], a0, a1, a2, a3, qb[nb][4 * w4 + q][0], qb[nb][4 * w4 + q][1]);
            }
          }
        }
        done(4 * i + x);
      }
      if (!ok) break;
      uint32_t pb[NB][4][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float c[2][2];  // [half][row]
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) c[x][r] = fmaxf(rf[nb][r] * ks[x], 1e-30f);
        if (masked) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int room = ((hidden >> (q0 + x)) & 1u) ? 0 : lim[nb][r] - key - kTileKeys * x;
              if (room > 0 && ((bad >> (q0 + x)) & 1u)) fin[nb][r] = false;
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  if (16 * j + g + 8 * y >= room) s[nb][x][j][2 * y + r] = -kPgInf;
            }
        }
        // ---- running maxima less kHead: max t = c max S + e (c > 0); -inf stays -inf
        float al[2], ref[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float top = -kPgInf;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float ex = ((zero_v >> (q0 + x)) & 1u) ? kPgZeroE : e[x];
            const float y = fmaxf(fmax3(s[nb][x][0][r], s[nb][x][0][2 + r], s[nb][x][1][r]), s[nb][x][1][2 + r]);
            top = fmaxf(top, fmaf(y, c[x][r], ex));
          }
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
          const float mn = fmaxf(m[nb][r], top - pg_head(top, kHead));
          ref[r] = (mn == -kPgInf) ? 0.f : mn;
          al[r] = (m[nb][r] == -kPgInf) ? 0.f : ex2_approx(m[nb][r] - ref[r]);
          m[nb][r] = mn;
        }
        if (!__all_sync(0xffffffffu, al[0] == 1.f && al[1] == 1.f)) {
          l[nb][0] *= al[0];
          l[nb][1] *= al[1];
#pragma unroll
          for (int p = 0; p < MT; ++p) {
            o[nb][p][0] *= al[0];
            o[nb][p][1] *= al[1];
            o[nb][p][2] *= al[0];
            o[nb][p][3] *= al[1];
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum[2] = {0.f, 0.f};
          const float off[2] = {e[x] - ref[0], e[x] - ref[1]};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float pr[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) pr[q] = ex2_approx(fmaf(s[nb][x][j][q], c[x][q & 1], off[q & 1]));
            sum[0] += pr[0] + pr[2];
            sum[1] += pr[1] + pr[3];
            uint32_t h0 = pack_half2(pr[0], pr[1]), h1 = pack_half2(pr[2], pr[3]);
            if ((zero_v >> (q0 + x)) & 1u) h0 = h1 = 0u;
            pb[nb][2 * x + j][0] = transpose8x8(h0);  // keys 2 t4, 2 t4 + 1 of row g
            pb[nb][2 * x + j][1] = transpose8x8(h1);  // eight further
          }
          l[nb][0] = fmaf(sum[0], inv[x], l[nb][0]);
          l[nb][1] = fmaf(sum[1], inv[x], l[nb][1]);
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* sv;
        if (!(ok = tile(sv))) break;
        // rows behind the sequence (or in no page) may hold any byte: an e4m3 NaN there must
        // not meet P = 0
        const int rows = E4M3 && masked ? (((hidden >> (q0 + x)) & 1u) ? 0 : len - key - kTileKeys * x) : kTileKeys;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int kx = 16 * j + 2 * t4 + (u & 1) + 8 * (u >> 1);
            const uint8_t* src = sv + swz<D>(kx, (4 * VW * g) >> 4) + ((4 * VW * g) & 15);
            if constexpr (VW == 4) {
              const uint4 y = *reinterpret_cast<const uint4*>(src);
              vw[u][0] = y.x;
              vw[u][1] = y.y;
              vw[u][2] = y.z;
              vw[u][3] = y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(src);
              vw[u][0] = y.x;
              vw[u][1] = y.y;
            }
            if (E4M3 && kx >= rows) {
#pragma unroll
              for (int w = 0; w < VW; ++w) vw[u][w] = 0u;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            uint32_t b0[4], b1[4];
            widen_pair<E4M3>(vw[0][w], vw[1][w], b0);
            widen_pair<E4M3>(vw[2][w], vw[3][w], b1);
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816(o[nb][2 * w + p], b0[2 * p], b0[2 * p + 1], b1[2 * p], b1[2 * p + 1], pb[nb][2 * x + j][0],
                         pb[nb][2 * x + j][1]);
          }
        }
        done(4 * i + 2 + x);
      }
      if (!ok) break;
    }

    // ---- join the warps (their rings are free)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[nb][r] += __shfl_xor_sync(0xffffffffu, l[nb][r], sh);
        // a row that saw a key through something not finite is NaN.  (Its eight lanes agree:
        // what they looked at is the same for all.)
        if (!fin[nb][r] && m[nb][r] > -kPgInf) l[nb][r] = __uint_as_float(0x7fffffffu);
        if (g == 0) {
          red_m[warp][8 * nb + 2 * t4 + r] = m[nb][r];
          red_l[warp][8 * nb + 2 * t4 + r] = l[nb][r];
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
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * nb + 2 * t4 + r;
        float mx = -kPgInf;
#pragma unroll
        for (int w = 0; w < W; ++w) mx = fmaxf(mx, red_m[w][row]);
        const float f = (m[nb][r] == -kPgInf) ? 0.f : ex2_approx(m[nb][r] - mx);
        // channels 4 VW g + 2 p, + 1 are the slots g and g + 8 of m-tile p
#pragma unroll
        for (int p = 0; p < MT; p += 2)
          *reinterpret_cast<float4*>(mine + row * D + 4 * join_chunk(row, VW * g + p / 2)) =
              make_float4(o[nb][p][r] * f, o[nb][p][2 + r] * f, o[nb][p + 1][r] * f, o[nb][p + 1][2 + r] * f);
      }
    __syncthreads();
    const bool whole = sg.s0 == 0 && sg.s1 == sg.steps;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (sg.s0 > 0 ? 0 : 1);
    float* share = reinterpret_cast<float*>(smem + SM::kShare);  // CL: this CTA's O, for the cluster
    for (int idx = threadIdx.x; idx < kRows * (D / 4); idx += kThreads) {
      const int r = idx / (D / 4), c = 4 * (idx % (D / 4));
      float mx = -kPgInf, lt = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) mx = fmaxf(mx, red_m[w][r]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float mw = red_m[w][r];
        lt += (mw == -kPgInf) ? 0.f : red_l[w][r] * ex2_approx(mw - mx);
        const float4 y =
            *reinterpret_cast<const float4*>(smem + w * SM::kWarp + 4 * (r * D + 4 * join_chunk(r, c / 4)));
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
        pg_write_out<D, kHead>(a, sg.b, sg.hkv, sg.seq.n, sg.rb * kRows + r, c, x, mx, lt);
      } else if (QATTN_IN_BOUNDS(slot < a.slots)) {
        *reinterpret_cast<float4*>(a.part_o + (slot * kRows + r) * D + c) = x;
        if (c == 0) {
          a.part_m[slot * kRows + r] = mx;
          a.part_l[slot * kRows + r] = lt;
        }
      }
    }
    if constexpr (CL) break;
    fence_proxy_async_smem();  // the rings go back to the TMA engine
    __syncthreads();
  }
  if constexpr (CL) {
    // ---- join the cluster: its CTAs take the rows' chunks in turn.  Every CTA reaches both
    // barriers, one that gave up on a wait too
    cluster_sync();
    const int rank = static_cast<int>(cluster_rank());
    for (int idx = rank * kThreads + threadIdx.x; some && idx < kRows * (D / 4); idx += a.cluster * kThreads) {
      const int r = idx / (D / 4), c = 4 * (idx % (D / 4));
      if ((sg.rb * kRows + r) / a.G >= sg.seq.n) continue;
      float mc[kPagedCluster], lc[kPagedCluster], mx = -kPgInf, lt = 0.f;
      float4 y[kPagedCluster], x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kPagedCluster; ++q) {
        mc[q] = -kPgInf;
        if (q < a.cluster) {
          mc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(smem_u32(&cl_m[r]), q)));
          lc[q] = __uint_as_float(ld_cluster_u32(cluster_addr(smem_u32(&cl_l[r]), q)));
          y[q] = ld_cluster_f4(cluster_addr(smem_u32(smem + SM::kShare) + 4 * (r * D + c), q));
        }
      }
#pragma unroll
      for (int q = 0; q < kPagedCluster; ++q) mx = fmaxf(mx, mc[q]);
#pragma unroll
      for (int q = 0; q < kPagedCluster; ++q) {
        if (mc[q] == -kPgInf) continue;
        const float f = ex2_approx(mc[q] - mx);
        lt = fmaf(f, lc[q], lt);
        x.x = fmaf(f, y[q].x, x.x);
        x.y = fmaf(f, y[q].y, x.y);
        x.z = fmaf(f, y[q].z, x.z);
        x.w = fmaf(f, y[q].w, x.w);
      }
      pg_write_out<D, kHead>(a, sg.b, sg.hkv, sg.seq.n, sg.rb * kRows + r, c, x, mx, lt);
    }
    cluster_sync();  // no CTA leaves while another reads its share
  }
}

template <int D, bool E4M3, int NB, int W>
cudaError_t launch_clusters(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t s) {
  constexpr int smem = WarpSmem<D, NB, W>::kBytes;
  const auto kernel = paged_warp_kernel<D, E4M3, NB, true, W>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return e != cudaSuccess ? e : launch_pdl_cluster(kernel, dim3(a.ctas), dim3(32 * W), a.cluster, smem, s, tk, tv, a);
}
template <int D, bool E4M3, int NB>
cudaError_t launch_nb(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t s) {
  if (a.cluster > 0)
    return a.wide ? launch_clusters<D, E4M3, NB, 8>(tk, tv, a, s) : launch_clusters<D, E4M3, NB, 4>(tk, tv, a, s);
  constexpr int W = 4, smem = WarpSmem<D, NB, W>::kBytes, kRows = 8 * NB;
  const auto kernel = paged_warp_kernel<D, E4M3, NB, false, W>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(a.ctas), dim3(32 * W), smem, s, tk, tv, a);
  if (e != cudaSuccess || a.ctas == 1) return e;
  return launch_pdl(paged_join_kernel<D, kHead, kRows>, dim3(a.ctas - 1, min(kRows, a.G * a.T)),
                    dim3(kPgJoinThreads), 0, s, a);
}
template <int D, bool E4M3>
cudaError_t launch_d(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t s) {
  return a.rows == 8 ? launch_nb<D, E4M3, 1>(tk, tv, a, s) : launch_nb<D, E4M3, 2>(tk, tv, a, s);
}

}  // namespace

unsigned int check_take_paged_warp() { return check_take_local(); }

cudaError_t launch_paged_warp(const CUtensorMap& tk, const CUtensorMap& tv, const PagedArgs& a, cudaStream_t s) {
  if (a.e4m3) return a.d == 64 ? launch_d<64, true>(tk, tv, a, s) : launch_d<128, true>(tk, tv, a, s);
  return a.d == 64 ? launch_d<64, false>(tk, tv, a, s) : launch_d<128, false>(tk, tv, a, s);
}

}  // namespace qattn
