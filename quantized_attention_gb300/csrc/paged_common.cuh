// What the kernels of qattn_paged_fwd share: the division of the work into equal
// shares, the scales of a page, the output row and the pass that joins the shares
// of a row block.
//
// Query rows of a KV head are ordered by token, then by query head of the group
// (row = token * G + head), so that a block of consecutive rows ends at a token and
// needs the cached rows up to that token's own and no further.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {

constexpr float kPgLog2e = 1.44269502162933349609375f;  // fp32(log2 e)
constexpr float kPgLn2 = 0.69314718055994531f;
constexpr float kPgInf = __builtin_huge_valf();
constexpr int kPgJoinThreads = 128;

// The low n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t pg_first_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// A sequence's rows in use and new tokens.  Values out of range are the caller's
// error: they are clamped (no access leaves the cache) and reported.
struct PagedSeq {
  int len, n;
};
__device__ __forceinline__ PagedSeq pg_seq(const PagedArgs& a, int b) {
  PagedSeq s{0, 0};
  if (!QATTN_IN_BOUNDS(b >= 0 && b < a.B)) return s;
  s.len = a.lengths[b];
  s.n = a.n_new ? a.n_new[b] : a.T;
  if (s.len < 0 || s.len > a.Nk || s.n < 0 || s.n > a.T) {
    atomicOr(a.err, kErrDomain);
    s.len = min(max(s.len, 0), a.Nk);
    s.n = min(max(s.n, 0), a.T);
  }
  return s;
}
// Row blocks of a KV head, steps of block rb (at least one: a block whose rows see
// nothing is written too), and what they count in the division of the work: a block's
// start (the last block's share written out, pipelines filled) costs as much as
// a.lead steps.
template <int ROWS>
__device__ __forceinline__ int pg_blocks(const PagedArgs& a, const PagedSeq& s) {
  return (s.n * a.G + ROWS - 1) / ROWS;
}
template <int ROWS, int STEP>
__device__ __forceinline__ int pg_steps(const PagedArgs& a, const PagedSeq& s, int rb) {
  int keys = s.len;
  if (a.causal) {
    const int last = min(s.n, ((rb + 1) * ROWS - 1) / a.G + 1);  // tokens up to the block's last
    keys = min(max(s.len - s.n + last, 0), s.len);
  }
  return max(1, (keys + STEP - 1) / STEP);
}
// Cached rows visible to token i.
__device__ __forceinline__ int pg_limit(const PagedArgs& a, const PagedSeq& s, int i) {
  return a.causal ? s.len - s.n + i + 1 : s.len;
}

// Places of one KV head of a sequence (a whole warp).
template <int ROWS, int STEP>
__device__ __forceinline__ int pg_head_places(const PagedArgs& a, const PagedSeq& s) {
  const int nb = pg_blocks<ROWS>(a, s), lane = threadIdx.x & 31;
  if (!a.causal || nb <= 1) return nb > 0 ? nb * (a.lead + pg_steps<ROWS, STEP>(a, s, nb - 1)) : 0;
  int total = 0;
  for (int k = lane; k < nb; k += 32) total += a.lead + pg_steps<ROWS, STEP>(a, s, k);
  return __reduce_add_sync(0xffffffffu, total);
}

// A CTA's share of the flattened list of places (ordered by sequence, KV head, row
// block; a block's lead, then its steps; fewer than 2^31): CTA c of G takes W / G of
// them, the first W % G CTAs one more.
struct PagedWalk {
  int p, end;        // the next place of the share in the list, its end
  int b, hkv, rb;    // where p lies
  int s0;            // place in the block less a.lead
  int steps;         // of the block
  int total;         // W
  PagedSeq seq;
};
// A run of steps of a share inside one block.
struct PagedSeg {
  int b, hkv, rb, s0, s1, steps;
  PagedSeq seq;
};

// Sequence b's places, where one number gives them (a lane for a sequence; 0 past the last).
struct PagedPlaces {
  PagedSeq seq;
  int nb, one, n;  // blocks of a KV head, steps of each, places in all
};
template <int ROWS, int STEP>
__device__ __forceinline__ PagedPlaces pg_places(const PagedArgs& a, int b) {
  PagedPlaces p{{0, 0}, 0, 0, 0};
  if (b < a.B) {
    p.seq = pg_seq(a, b);
    p.nb = pg_blocks<ROWS>(a, p.seq);
    if (p.nb > 0) p.one = pg_steps<ROWS, STEP>(a, p.seq, p.nb - 1);
    p.n = p.nb > 0 ? a.Hkv * p.nb * (a.lead + p.one) : 0;
  }
  return p;
}
// Places of all sequences (a whole warp; `first`: the first 32's, a lane each).
template <int ROWS, int STEP>
__device__ __forceinline__ int pg_totals(const PagedArgs& a, const PagedPlaces& first) {
  int total = first.n;
  const int lane = threadIdx.x & 31;
  if (a.blocks == 1 || !a.causal) {
    for (int b = 32 + lane; b < a.B; b += 32) total += pg_places<ROWS, STEP>(a, b).n;
    return __reduce_add_sync(0xffffffffu, total);
  }
  total = 0;
  for (int b = 0; b < a.B; ++b) total += a.Hkv * pg_head_places<ROWS, STEP>(a, pg_seq(a, b));
  return total;
}

// Where the share of CTA c of G begins.  Called by whole warps, each for itself.
template <int ROWS, int STEP>
__device__ __forceinline__ PagedWalk pg_walk(const PagedArgs& a, int c, int G) {
  const int lane = threadIdx.x & 31;
  PagedWalk w{};
  PagedPlaces one{{0, 0}, 0, 0, 0};
  if (a.blocks == 1 || !a.causal) one = pg_places<ROWS, STEP>(a, lane);
  const int total = pg_totals<ROWS, STEP>(a, one);
  const int q = total / G, r = total - q * G;
  w.total = total;
  w.p = c * q + min(c, r);
  w.end = w.p + q + (c < r ? 1 : 0);
  if (w.p >= w.end) return w;
  int before = 0;
  if (a.blocks == 1 || !a.causal) {
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      if (b0 > 0) one = pg_places<ROWS, STEP>(a, b0 + lane);
      int inc = one.n;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, sh);
        if (lane >= sh) inc += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + inc > w.p);
      if (past) {
        const int l = __ffs(past) - 1;
        int off = w.p - before - __shfl_sync(0xffffffffu, inc - one.n, l);
        w.b = b0 + l;
        w.seq.len = __shfl_sync(0xffffffffu, one.seq.len, l);
        w.seq.n = __shfl_sync(0xffffffffu, one.seq.n, l);
        w.steps = __shfl_sync(0xffffffffu, one.one, l);
        const int nb = __shfl_sync(0xffffffffu, one.nb, l);
        const int per = a.lead + w.steps, blk = off / per;
        w.hkv = blk / nb;
        w.rb = blk - w.hkv * nb;
        w.s0 = off - blk * per - a.lead;
        return w;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    w.end = w.p;
    return w;
  }
  for (int b = 0; b < a.B; ++b) {
    const PagedSeq s = pg_seq(a, b);
    const int per = pg_head_places<ROWS, STEP>(a, s), n = a.Hkv * per;
    if (before + n <= w.p) {
      before += n;
      continue;
    }
    int off = w.p - before;
    w.b = b;
    w.seq = s;
    w.hkv = off / per;
    off -= w.hkv * per;
    const int nb = pg_blocks<ROWS>(a, s);
    for (int k0 = 0; k0 < nb; k0 += 32) {
      const int st = k0 + lane < nb ? pg_steps<ROWS, STEP>(a, s, k0 + lane) : 0;
      const int one = k0 + lane < nb ? a.lead + st : 0;
      int inc = one;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, sh);
        if (lane >= sh) inc += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, inc > off);
      if (past) {
        const int l = __ffs(past) - 1;
        w.rb = k0 + l;
        w.steps = __shfl_sync(0xffffffffu, st, l);
        w.s0 = off - __shfl_sync(0xffffffffu, inc - one, l) - a.lead;
        return w;
      }
      off -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  w.end = w.p;
  return w;
}

// The next segment of the share; false when it is done.
template <int ROWS, int STEP>
__device__ __forceinline__ bool pg_next(const PagedArgs& a, PagedWalk& w, PagedSeg& s) {
  if (w.p >= w.end) return false;
  if (w.s0 == w.steps) {  // the next block, KV head, sequence that has blocks
    w.s0 = -a.lead;
    if (++w.rb >= pg_blocks<ROWS>(a, w.seq)) {
      w.rb = 0;
      if (++w.hkv == a.Hkv) {
        w.hkv = 0;
        do {
          w.seq = pg_seq(a, ++w.b);
        } while (pg_blocks<ROWS>(a, w.seq) == 0 && w.b < a.B);
        if (w.b >= a.B) {
          w.p = w.end;
          return false;
        }
      }
    }
    w.steps = pg_steps<ROWS, STEP>(a, w.seq, w.rb);
  }
  s.b = w.b;
  s.hkv = w.hkv;
  s.rb = w.rb;
  s.seq = w.seq;
  s.steps = w.steps;
  const int n = min(w.end - w.p, w.steps - w.s0);  // places of this block
  const int skip = w.s0 < 0 ? min(n, -w.s0) : 0;   // of them in its lead
  s.s0 = w.s0 + skip;
  s.s1 = w.s0 + n;
  w.p += n;
  w.s0 += n;
  return skip < n;  // a share that ends in a block's lead holds none of its steps
}

// The clustered form: this CTA's part of its cluster's block (possibly no step), and
// whether the block has rows at all.
template <int ROWS, int STEP>
__device__ __forceinline__ bool pg_cluster_seg(const PagedArgs& a, PagedSeg& s) {
  const int rank = static_cast<int>(cluster_rank());
  int x = blockIdx.x / a.cluster;
  s.rb = x % a.blocks;
  x /= a.blocks;
  s.hkv = x % a.Hkv;
  s.b = x / a.Hkv;
  s.seq = pg_seq(a, s.b);
  s.s0 = s.s1 = s.steps = 0;
  if (s.rb >= pg_blocks<ROWS>(a, s.seq)) return false;
  s.steps = pg_steps<ROWS, STEP>(a, s.seq, s.rb);
  const int q = s.steps / a.cluster, r = s.steps - q * a.cluster;
  s.s0 = rank * q + min(rank, r);
  s.s1 = s.s0 + q + (rank < r ? 1 : 0);
  return true;
}

// ------------------------------------------------------------------ values
// The largest power of two that brings a row of magnitude `amax` (bits; finite) below
// 2^15, so that its bf16 values are fp16 values with all their bits unless they are
// 2^29 times smaller than the largest; and its inverse.
__device__ __forceinline__ void pg_row_shift(uint32_t amax, float& up, float& down) {
  int e = 14 - (static_cast<int>(amax >> 23) - 127);
  e = min(max(e, -113), 126);
  up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// What a page's scales mean for a row: t = S c + e with c = row factor * K scale and
// e = log2(V scale), so that P = 2^(t - m) carries the V scale and l takes P / V scale.
// m may move by as much as e does, and l must outlast that in fp32: V scales lie within
// 2^-48 and 2^48 (96 powers of two, 30 left for the weights).  A smaller one counts as
// 0: the page adds 2^(t - m) to l and nothing to O.  A larger one, and scales that are
// negative or not finite, give NaN to every row that sees a key of the page.
constexpr float kPgMinV = 0x1p-48f, kPgMaxV = 0x1p48f, kPgZeroE = -48.f;
struct PageScale {
  float k;       // K scale (0 for a page that counts as NaN).  A row's factor times it is held
                 // at 1e-30 or more (2^(S c) is 1 all the same), so that a hidden key's -inf stays -inf
  float e_max;   // the exponent's part in the maximum,
  float e;       // and in the exponential
  float inv;     // 1 / V scale (1 where that counts as 0)
  uint32_t keep; // 0 where the V scale counts as 0, else all ones
  bool nan;
};
__device__ __forceinline__ PageScale pg_scale(float ks, float vs) {
  PageScale p;
  p.nan = !(ks >= 0.f && ks < kPgInf) || !(vs >= 0.f && vs <= kPgMaxV);
  const bool zero = p.nan || vs < kPgMinV;
  p.k = p.nan ? 0.f : ks;
  p.e = zero ? 0.f : log2f(vs);
  p.e_max = zero ? kPgZeroE : p.e;
  p.inv = zero ? 1.f : 1.f / vs;
  p.keep = zero ? 0u : 0xffffffffu;
  return p;
}
// The exponentials' reference lies below a row's largest t, so that P in fp16 uses the
// type's range above 1 too; from |t| = 2^20 on, where the difference would round, it is
// t itself.
__device__ __forceinline__ float pg_head(float top, float head) { return fabsf(top) < 1048576.f ? head : 0.f; }

// Four channels c.. of row rr of a block's KV head: O = x / l, 0 for a row that sees
// nothing (l = 0), NaN if l is; the row's lse with channel 0.  HEAD: see pg_head.
template <int D, int HEAD>
__device__ __forceinline__ void pg_write_out(const PagedArgs& a, int b, int hkv, int n, int rr, int c,
                                             float4 x, float m, float l) {
  const int tok = rr / a.G;
  if (tok >= n) return;
  const size_t row = (static_cast<size_t>(b) * a.Hq + hkv * a.G + rr - tok * a.G) * a.T + tok;
  if (!QATTN_IN_BOUNDS(row < a.rows_total && b < a.B && hkv < a.Hkv)) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  x.x *= inv;
  x.y *= inv;
  x.z *= inv;
  x.w *= inv;
  if (a.out_bf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * D + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * D + c) = x;
  }
  if (a.lse && c == 0)
    a.lse[row] = l == 0.f ? -kPgInf : ((m + HEAD) + log2f(l * (1.f / (1 << HEAD)))) * kPgLn2;
}

// The CTA whose share holds place x of a list of `total`.
__device__ __forceinline__ int pg_owner(int x, int total, int G) {
  const int q = total / G, r = total - q * G, big = r * (q + 1);
  return x < big ? x / (q + 1) : r + (x - big) / q;
}
// What the join has to know, left by each CTA of the attention kernel about the place
// where its share begins: the block that lies across it, if that is the block's first
// such place, and the CTAs c0 .. c1 that its steps were dealt to (else c1 = -1).  CTA c left
// its share in slot 2 c when it did not have the block's first step, else in 2 c + 1.
struct __align__(16) PagedPlan {
  int b, hkv, rb, n;  // n: the sequence's new tokens
  int c0, c1, pad0, pad1;
};
__device__ __forceinline__ void pg_put_plan(const PagedArgs& a, const PagedWalk& w) {
  const int c = blockIdx.x;
  PagedPlan p{w.b, w.hkv, w.rb, w.seq.n, 0, -1, 0, 0};
  if (w.p < w.end && w.s0 > 0 && w.s0 < w.steps) {
    p.c0 = pg_owner(w.p - w.s0, w.total, a.ctas);
    if (p.c0 == c - 1) p.c1 = pg_owner(w.p - w.s0 + w.steps - 1, w.total, a.ctas);
  }
  if (a.plan && QATTN_IN_BOUNDS(c < a.ctas)) a.plan[c] = p;
}
__device__ __forceinline__ PagedPlan pg_get_plan(const PagedArgs& a, int c) {
  PagedPlan p{0, 0, 0, 0, 0, -1, 0, 0};
  if (QATTN_IN_BOUNDS(c < a.ctas)) p = a.plan[c];
  return p;
}

// The join for few rows a block (blockIdx.x: a boundary between shares, as PagedPlan has
// it; blockIdx.y: a row): four warps for a row, which take every fourth share: the weights
// 2^(m_c - m) of 32 shares come first, one a lane, then the shares' rows in independent
// loads.  (A warp for a row: 8 sequences of 16K to 32K rows 72.8 us against 71.4.)
template <int D, int HEAD, int ROWS>
__global__ void __launch_bounds__(kPgJoinThreads) paged_join_kernel(const PagedArgs a) {
  constexpr int CPL = D / 32;  // channels per lane
  constexpr int NW = kPgJoinThreads / 32;
  __shared__ float sm[NW], sl[NW];
  __shared__ __align__(16) float so[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const PagedPlan own = pg_get_plan(a, blockIdx.x + 1);
  const int c0 = own.c0, c1 = own.c1;
  if (c1 < 0 || own.rb * ROWS + r >= own.n * a.G) return;  // (the whole CTA)
  float m = -kPgInf, l = 0.f, o[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) o[k] = 0.f;
  for (int cb = c0 + warp; cb <= c1; cb += 32 * NW) {
    const int c = cb + lane * NW;
    const size_t slot = 2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0);
    const bool mine = c <= c1 && QATTN_IN_BOUNDS(slot < a.slots);
    const float mc = mine ? a.part_m[slot * ROWS + r] : -kPgInf, lc = mine ? a.part_l[slot * ROWS + r] : 0.f;
    float mx = mc;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
    const float mn = fmaxf(m, mx);
    if (mn == -kPgInf) continue;  // (the whole warp)
    const float f = m == -kPgInf ? 0.f : ex2_approx(m - mn);
    const float w = mc == -kPgInf ? 0.f : ex2_approx(mc - mn);
    float ls = w * lc;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, sh);
    l = l * f + ls;
    m = mn;
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] *= f;
    const int cnt = min(32, (c1 - cb) / NW + 1);
#pragma unroll 8
    for (int i = 0; i < cnt; ++i) {
      const int ci = cb + i * NW;
      const size_t si = 2 * static_cast<size_t>(ci) + (ci == c0 ? 1 : 0);
      const float wi = __shfl_sync(0xffffffffu, w, i);
      if (!QATTN_IN_BOUNDS(si < a.slots)) continue;
      const float* po = a.part_o + (si * ROWS + r) * D + CPL * lane;
      if constexpr (CPL == 4) {
        const float4 y = *reinterpret_cast<const float4*>(po);
        o[0] = fmaf(wi, y.x, o[0]);
        o[1] = fmaf(wi, y.y, o[1]);
        o[2] = fmaf(wi, y.z, o[2]);
        o[3] = fmaf(wi, y.w, o[3]);
      } else {
        const float2 y = *reinterpret_cast<const float2*>(po);
        o[0] = fmaf(wi, y.x, o[0]);
        o[1] = fmaf(wi, y.y, o[1]);
      }
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < CPL; ++k) so[warp][CPL * lane + k] = o[k];
  __syncthreads();
  const int c = 4 * static_cast<int>(threadIdx.x);
  if (c < D) {
    float mx = -kPgInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[w]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = sm[w] == -kPgInf ? 0.f : ex2_approx(sm[w] - mx);
      lt = fmaf(f, sl[w], lt);
      const float4 y = *reinterpret_cast<const float4*>(&so[w][c]);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    pg_write_out<D, HEAD>(a, own.b, own.hkv, own.n, own.rb * ROWS + r, c, x, mx, lt);
  }
}

}  // namespace qattn
