// What the two kernels of qattn_tree_decode share: the division of the work
// into equal shares, the drafted tokens' codes and masks, the output row and
// the pass that joins the shares of a head.
#pragma once
#include <cuda_bf16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {

constexpr float kLog2e = 1.44269502162933349609375f;  // fp32(log2 e)
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kTreeJoinThreads = 128;

// The low n bits (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Rows in use of sequence b.  A length outside 0 .. Nk is the caller's error:
// it is clamped (no access leaves the cache) and reported by the error word.
__device__ __forceinline__ int tree_length(const TreeArgs& a, int b) {
  if (!a.lengths) return a.Nk;
  if (!QATTN_IN_BOUNDS(b >= 0 && b < a.B)) return 0;
  const int n = a.lengths[b];
  if (n < 0 || n > a.Nk) {
    atomicOr(a.err, kErrDomain);
    return n < 0 ? 0 : a.Nk;
  }
  return n;
}

// Steps of one head of a sequence: its drafted steps, then its cached ones.
__device__ __forceinline__ int tree_steps(const TreeArgs& a, int len, int step) {
  return a.drafts + (len + step - 1) / step;
}
// What they count in the division of the work: the head's start (its drafts' codes,
// the last head's share written out, pipelines filled again) costs as much as
// a.lead steps.
__device__ __forceinline__ int tree_cost(const TreeArgs& a, int steps) { return steps > 0 ? a.lead + steps : 0; }

// A CTA's share of the flattened list of W places (ordered by sequence, KV head,
// row block; a head's lead, then its steps; W < 2^31): CTA c of G takes W / G of
// them, the first W % G CTAs one more.  A segment is a run of steps of the share
// inside one head.
struct TreeWalk {
  int p, end;         // the next place of the share in the list, its end
  int b, head, s0;    // where p lies: sequence, (KV head, row block), place in the head less a.lead
  int len, steps;     // the sequence's rows in use, steps of each of its heads
};

struct TreeSeg {
  int b, hkv, rb;  // sequence, KV head, row block
  int len;         // rows in use
  int s0, s1;      // steps of the head
  int steps;       // all steps of the head
};

// Steps of all sequences, and of those before sequence b0 (a whole warp).
__device__ __forceinline__ void tree_totals(const TreeArgs& a, int step, int b0, int& total, int& before) {
  const int per = a.Hkv * a.blocks, lane = threadIdx.x & 31;
  total = before = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int n = per * tree_cost(a, tree_steps(a, tree_length(a, b), step));
    total += n;
    if (b < b0) before += n;
  }
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, sh);
    before += __shfl_xor_sync(0xffffffffu, before, sh);
  }
}

// Where this CTA's share begins.  Called by whole warps, each for itself: no CTA
// barrier, one round of loads up to 32 sequences.
__device__ __forceinline__ TreeWalk tree_walk(const TreeArgs& a, int step) {
  const int per = a.Hkv * a.blocks, lane = threadIdx.x & 31;
  TreeWalk w;
  int my_len = 0, my_n = 0, total = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int len = tree_length(a, b), n = tree_steps(a, len, step);
    if (b < 32) {
      my_len = len;
      my_n = n;
    }
    total += per * tree_cost(a, n);
  }
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) total += __shfl_xor_sync(0xffffffffu, total, sh);
  const int G = gridDim.x, c = blockIdx.x, q = total / G, r = total - q * G;
  w.p = c * q + min(c, r);
  w.end = w.p + q + (c < r ? 1 : 0);
  w.b = w.head = w.s0 = w.len = w.steps = 0;
  int before = 0;
  for (int b0 = 0; b0 < a.B && w.p < w.end; b0 += 32) {
    if (b0 > 0) {
      my_len = b0 + lane < a.B ? tree_length(a, b0 + lane) : 0;
      my_n = b0 + lane < a.B ? tree_steps(a, my_len, step) : 0;
    }
    const int n = b0 + lane < a.B ? per * tree_cost(a, my_n) : 0;
    int inc = n;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, sh);
      if (lane >= sh) inc += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + inc > w.p);
    if (past) {
      const int l = __ffs(past) - 1;
      const int off = w.p - before - __shfl_sync(0xffffffffu, inc - n, l);
      w.b = b0 + l;
      w.len = __shfl_sync(0xffffffffu, my_len, l);
      w.steps = __shfl_sync(0xffffffffu, my_n, l);
      w.head = off / (a.lead + w.steps);
      w.s0 = off - w.head * (a.lead + w.steps) - a.lead;
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return w;
}

// The next segment of the share; false when it is done.
__device__ __forceinline__ bool tree_next(const TreeArgs& a, int step, TreeWalk& w, TreeSeg& s) {
  if (w.p >= w.end) return false;
  if (w.s0 == w.steps) {  // the next head; the next sequence that has steps
    w.s0 = -a.lead;
    if (++w.head == a.Hkv * a.blocks) {
      w.head = 0;
      do {
        w.len = tree_length(a, ++w.b);
        w.steps = tree_steps(a, w.len, step);
      } while (w.steps == 0 && QATTN_IN_BOUNDS(w.b < a.B));
    }
  }
  s.b = w.b;
  s.hkv = a.blocks == 1 ? w.head : w.head / a.blocks;
  s.rb = a.blocks == 1 ? 0 : w.head - s.hkv * a.blocks;
  s.len = w.len;
  s.steps = w.steps;
  // (With s0 = max(s0, 0) and s1 = max(min(..), 0) nvcc 13.0 took a caller's
  // s0 == 0 && s1 == steps for s0 == 0.)
  const int n = min(w.end - w.p, w.steps - w.s0);     // places of this head
  const int skip = w.s0 < 0 ? min(n, -w.s0) : 0;      // of them in its lead
  s.s0 = w.s0 + skip;
  s.s1 = w.s0 + n;
  w.p += n;
  w.s0 += n;
  return skip < n;  // a share that ends in a head's lead holds none of its steps
}

// The clustered form: this CTA's part of its cluster's head (the segment; possibly
// no step: s0 == s1), and a walk that yields it once.
__device__ __forceinline__ TreeWalk tree_cluster_walk(const TreeArgs& a, int step, TreeSeg& s) {
  const int rank = static_cast<int>(cluster_rank());
  int head = blockIdx.x / a.cluster;
  s.rb = head % a.blocks;
  head /= a.blocks;
  s.hkv = head % a.Hkv;
  s.b = head / a.Hkv;
  s.len = tree_length(a, s.b);
  s.steps = tree_steps(a, s.len, step);
  const int total = tree_cost(a, s.steps);  // places: the lead, then the steps
  const int q = total / a.cluster, r = total - q * a.cluster;
  const int p = rank * q + min(rank, r) - a.lead, n = q + (rank < r ? 1 : 0);
  const int skip = p < 0 ? min(n, -p) : 0;
  s.s0 = p + skip;
  s.s1 = p + n;
  TreeWalk w{};
  w.end = n - skip;
  return w;
}
__device__ __forceinline__ bool tree_once(TreeWalk& w, const TreeSeg& s) {
  if (w.p >= w.end) return false;
  w.p = w.end;
  return s.s0 < s.s1;
}

// The CTA whose share holds place x of a list of `total`.
__device__ __forceinline__ int tree_owner(int x, int total, int G) {
  const int q = total / G, r = total - q * G, big = r * (q + 1);
  return x < big ? x / (q + 1) : r + (x - big) / q;
}
// c = fp32(fp32(sq * sm_scale) * log2 e) of a query head's tokens (T <= 128: one
// scale block).  A factor of 0 (all the head's codes 0) becomes 1e-30: 2^(S c) is
// 1 all the same for every |S| < 2^21, and a hidden key's -inf stays -inf.  So does
// one that is not finite, for the sake of the row's hidden keys; tree_sum makes up for it.
__device__ __forceinline__ float tree_factor(const TreeArgs& a, int b, int hq, bool& finite) {
  const int i = a.q_gran == 0 ? 0 : b * a.Hq + hq;
  const float sq = QATTN_IN_BOUNDS(i >= 0 && i < a.B * a.Hq) ? a.q_scales[i] : 0.f;
  const float c = __fmul_rn(__fmul_rn(sq, a.sm_scale), kLog2e);
  finite = fabsf(c) < -kNegInf;
  return c == 0.f || !finite ? 1e-30f : c;
}
// A share's sum of P: NaN if its row saw keys through a factor that is not finite (and
// with it O and lse, through every join).
__device__ __forceinline__ float tree_sum(float l, bool finite) {
  return l > 0.f && !finite ? __int_as_float(0x7fffffff) : l;
}

// The exponentials' reference lies below a row's largest t, so that P = 2^(t - m) in
// fp16 uses the type's range above 1 too: P of a key keeps its 11 bits as long as it is
// not 2^(14 + head) times smaller than the row's largest.  (P <= 2^15 with every lag of
// the reference.)  From |t| = 2^20 on, where the difference would round, it is t itself:
// there the scores are so coarse that the largest alone counts.
constexpr float kFarScore = 1048576.f;
__device__ __forceinline__ float tree_head(float top, float head) { return fabsf(top) < kFarScore ? head : 0.f; }

// Cached rows visible to token i: all of them, or (tokens already appended,
// causal) those up to its own.
__device__ __forceinline__ int tree_limit(const TreeArgs& a, int len, int i) {
  return a.cached_causal ? len - a.T + i + 1 : len;
}

// Drafts 32 s .. 32 s + 31 visible to token i of sequence b, one bit each.
__device__ __forceinline__ uint32_t tree_draft_word(const TreeArgs& a, int b, int i, int s) {
  const uint32_t real = first_bits(a.T - 32 * s);
  if (real == 0u) return 0u;  // past the mask's words
  if (!a.tree_mask) return a.draft_causal ? first_bits(i + 1 - 32 * s) & real : real;
  const int words = (a.T + 31) / 32;
  if (!QATTN_IN_BOUNDS(b < a.B && i >= 0 && i < a.T && s < words)) return 0u;
  return a.tree_mask[(static_cast<size_t>(b) * a.T + i) * words + s] & real;
}

// rint(x / s) clamped to +-127, as bytes.  The quotient by the reciprocal is off
// by at most 2 ulp (3e-5 below 128), so it rounds as the IEEE quotient does unless
// it lies next to a half: a word with one of those few, or of anything not finite,
// is divided.
__device__ __forceinline__ uint32_t code_byte(float r) {
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(r, -127.f), 127.f))) & 0xffu;
}
__device__ __forceinline__ uint32_t code_word(float4 x, float4 s, float4 inv) {
  const float4 q = make_float4(x.x * inv.x, x.y * inv.y, x.z * inv.z, x.w * inv.w);
  float4 r = make_float4(rintf(q.x), rintf(q.y), rintf(q.z), rintf(q.w));
  const bool near_half = !(fabsf(q.x - r.x) <= 0.4999f) || !(fabsf(q.y - r.y) <= 0.4999f) ||
                         !(fabsf(q.z - r.z) <= 0.4999f) || !(fabsf(q.w - r.w) <= 0.4999f);
  if (near_half)
    r = make_float4(rintf(__fdiv_rn(x.x, s.x)), rintf(__fdiv_rn(x.y, s.y)), rintf(__fdiv_rn(x.z, s.z)),
                    rintf(__fdiv_rn(x.w, s.w)));
  return code_byte(r.x) | code_byte(r.y) << 8 | code_byte(r.z) << 16 | code_byte(r.w) << 24;
}
__device__ __forceinline__ float4 bf16x4_to_f32(uint2 x) {
  return make_float4(bf16_bits_to_f32(x.x & 0xffffu), bf16_bits_to_f32(x.x >> 16), bf16_bits_to_f32(x.y & 0xffffu),
                     bf16_bits_to_f32(x.y >> 16));
}

// The codes of drafts j0 .. min(j0 + n, T) - 1 of (b, hkv), as qattn_kv_append
// would store them with the header as it stands: kc = clamp(rint((K - mu) / s_k)),
// vc = clamp(rint(V / s_v)).  The step's other rows keep what they held: any byte
// is a finite code, and no query sees them.  `nthr` threads (a multiple of 32),
// this one `tid`; k_at(r, c) and v_at(r, c) give the address of 16-byte chunk c of
// row r.
template <int D, typename FK, typename FV>
__device__ __forceinline__ void tree_encode_drafts(const TreeArgs& a, int b, int hkv, int j0, int n,
                                                   int tid, int nthr, FK k_at, FV v_at) {
  constexpr int W = D / 4;  // words of a row
  constexpr int U = 4;      // rows in flight
  const int w = tid % W;    // W <= 32 divides nthr
  if (!QATTN_IN_BOUNDS(b < a.B && hkv < a.Hkv)) return;
  const size_t ch = (static_cast<size_t>(b) * a.Hkv + hkv) * D + 4 * w;
  const float4 ks = *reinterpret_cast<const float4*>(a.k_chan_scale + ch);
  const float4 mu = *reinterpret_cast<const float4*>(a.k_mean + ch);
  const float4 vs = *reinterpret_cast<const float4*>(a.v_chan_scale + ch);
  const uint16_t* K = a.k_new + b * a.ksB + hkv * a.ksH + 4 * w;
  const uint16_t* V = a.v_new + b * a.vsB + hkv * a.vsH + 4 * w;
  const int rows = min(n, a.T - j0), dr = nthr / W;
  const float4 ki = make_float4(__frcp_rn(ks.x), __frcp_rn(ks.y), __frcp_rn(ks.z), __frcp_rn(ks.w));
  const float4 vi = make_float4(__frcp_rn(vs.x), __frcp_rn(vs.y), __frcp_rn(vs.z), __frcp_rn(vs.w));
  for (int r0 = tid / W; r0 < rows; r0 += U * dr) {
    uint2 k[U], v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int r = r0 + i * dr;
      k[i] = v[i] = make_uint2(0u, 0u);
      if (r < rows && QATTN_IN_BOUNDS(j0 + r < a.T)) {
        k[i] = *reinterpret_cast<const uint2*>(K + (j0 + r) * a.ksN);
        v[i] = *reinterpret_cast<const uint2*>(V + (j0 + r) * a.vsN);
      }
    }
    // one copy of the code for all of them: it runs once or twice, and fetching its
    // instructions would take longer than running them
#pragma unroll 1
    for (int r = r0; r < min(rows, r0 + U * dr); r += dr) {
      float4 x = bf16x4_to_f32(k[0]);
      x = make_float4(__fsub_rn(x.x, mu.x), __fsub_rn(x.y, mu.y), __fsub_rn(x.z, mu.z), __fsub_rn(x.w, mu.w));
      *reinterpret_cast<uint32_t*>(k_at(r, w >> 2) + 4 * (w & 3)) = code_word(x, ks, ki);
      *reinterpret_cast<uint32_t*>(v_at(r, w >> 2) + 4 * (w & 3)) = code_word(bf16x4_to_f32(v[0]), vs, vi);
#pragma unroll
      for (int i = 0; i + 1 < U; ++i) {
        k[i] = k[i + 1];
        v[i] = v[i + 1];
      }
    }
  }
}

// Four channels c.. of row rr (query head of the group, token) of (b, hkv):
// O = x s_v / l, 0 for a row that sees nothing (l = 0), NaN if l is; the row's lse with
// channel 0.  HEAD: how far the reference m lies below the row's largest t (both shifted
// back before the logarithm, so that a sum of about 2^HEAD costs lse no bits).
template <int D, int HEAD>
__device__ __forceinline__ void tree_write_out(const TreeArgs& a, int b, int hkv, int rr, int c,
                                               float4 x, float m, float l) {
  if (rr >= a.G * a.T) return;
  const int hq = rr / a.T, i = rr % a.T;
  const size_t row = (static_cast<size_t>(b) * a.Hq + hkv * a.G + hq) * a.T + i;
  if (!QATTN_IN_BOUNDS(row < a.rows_total && b < a.B && hkv < a.Hkv)) return;
  const float4 sv =
      *reinterpret_cast<const float4*>(a.v_chan_scale + (static_cast<size_t>(b) * a.Hkv + hkv) * D + c);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  x.x *= sv.x * inv;
  x.y *= sv.y * inv;
  x.z *= sv.z * inv;
  x.w *= sv.w * inv;
  if (a.out_bf16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * D + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * D + c) = x;
  }
  if (a.lse && c == 0)
    a.lse[row] = l == 0.f ? kNegInf : ((m + HEAD) + log2f(l * (1.f / (1 << HEAD)))) * kLn2;
}

// Joins the shares of the heads that more than one CTA worked on.  A head's steps
// are the places [x0, x0 + n) of the flattened list, so its CTAs are their owners;
// CTA c left its share in slot 2 c when it did not have the head's first step, else
// in 2 c + 1.  The attention kernel releases this grid after its own dependency wait,
// so the lengths are final and the division is known before the shares arrive.
struct TreeOwners {
  int b, hkv, rb;  // the head
  int steps, c0, c1;
};
__device__ __forceinline__ TreeOwners tree_owners(const TreeArgs& a, int step, int head) {
  TreeOwners o;
  o.rb = head % a.blocks;
  head /= a.blocks;
  o.b = head / a.Hkv;
  o.hkv = head % a.Hkv;
  int tot, x0;
  tree_totals(a, step, o.b, tot, x0);
  o.steps = tree_steps(a, tree_length(a, o.b), step);
  x0 += (o.hkv * a.blocks + o.rb) * (a.lead + o.steps) + a.lead;  // the head's first step
  o.c0 = o.steps > 0 ? tree_owner(x0, tot, a.ctas) : 0;
  o.c1 = o.steps > 0 ? tree_owner(x0 + o.steps - 1, tot, a.ctas) : 0;
  return o;
}

// The join for few rows a head: NW warps for a row (blockIdx.y: 4 / NW rows), which
// take every NW-th share: the weights 2^(m_c - m) of 32 shares come first, one a
// lane, then the shares' rows in independent loads.
template <int D, int HEAD, int ROWS, int STEP, int NW>
__global__ void __launch_bounds__(kTreeJoinThreads) tree_join_kernel(const TreeArgs a) {
  constexpr int CPL = D / 32;  // channels per lane
  constexpr int RPC = kTreeJoinThreads / 32 / NW;  // rows of a CTA
  __shared__ float sm[RPC][NW], sl[RPC][NW];
  __shared__ __align__(16) float so[RPC][NW][D];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % NW, rw = (threadIdx.x >> 5) / NW;
  const int r = blockIdx.y * RPC + rw;
  const TreeOwners own = tree_owners(a, STEP, blockIdx.x);
  const int b = own.b, hkv = own.hkv, rb = own.rb, n = own.steps, c0 = own.c0, c1 = own.c1;
  const bool in = rb * ROWS + r < a.G * a.T;
  pdl_wait();
  pdl_trigger();
  if (n == 0) {  // no cached row and no draft: nothing is visible
    if (in && warp == 0 && lane < D / 4)
      tree_write_out<D, HEAD>(a, b, hkv, rb * ROWS + r, 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f), kNegInf, 0.f);
    return;
  }
  if (c0 == c1) return;  // written whole
  float m = kNegInf, l = 0.f, o[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) o[k] = 0.f;
  for (int cb = c0 + warp; in && cb <= c1; cb += 32 * NW) {
    const int c = cb + lane * NW;
    // only the head's first CTA began before the head
    const size_t slot = 2 * static_cast<size_t>(c) + (c == c0 ? 1 : 0);
    const bool mine = c <= c1 && QATTN_IN_BOUNDS(slot < a.slots);
    const float mc = mine ? a.part_m[slot * ROWS + r] : kNegInf, lc = mine ? a.part_l[slot * ROWS + r] : 0.f;
    float mx = mc;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
    const float mn = fmaxf(m, mx);
    if (mn == kNegInf) continue;  // (the whole warp)
    const float f = m == kNegInf ? 0.f : ex2_approx(m - mn);
    const float w = mc == kNegInf ? 0.f : ex2_approx(mc - mn);
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
    sm[rw][warp] = m;
    sl[rw][warp] = l;
  }
#pragma unroll
  for (int k = 0; k < CPL; ++k) so[rw][warp][CPL * lane + k] = o[k];
  if constexpr (NW > 1) __syncthreads();
  else __syncwarp();
  const int c = 4 * (NW > 1 ? static_cast<int>(threadIdx.x) : lane);
  if (in && c < D) {
    float mx = kNegInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[rw][w]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (sm[rw][w] == kNegInf) continue;
      const float f = ex2_approx(sm[rw][w] - mx);
      lt = fmaf(f, sl[rw][w], lt);
      const float4 y = *reinterpret_cast<const float4*>(&so[rw][w][c]);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    tree_write_out<D, HEAD>(a, b, hkv, rb * ROWS + r, c, x, mx, lt);
  }
}

}  // namespace qattn
