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
  const int n = a.lengths[b];
  if (n < 0 || n > a.Nk) {
    atomicOr(a.err, kErrDomain);
    return n < 0 ? 0 : a.Nk;
  }
  return n;
}

// Steps of one head of a sequence: its drafted steps, then its cached ones.
__device__ __forceinline__ long long tree_steps(const TreeArgs& a, int len, int step) {
  return a.drafts + (len + step - 1) / step;
}

struct TreePlan {
  long long begin, end;  // this CTA's steps in the flattened list
  long long total;       // all steps
  long long seq0;        // first step of sequence seq
  int seq;               // the sequence that holds `begin`
  long long warp_sum[32];
};

struct TreeSeg {
  int b, hkv, rb;  // sequence, KV head, row block
  int len;         // rows in use
  int s0, s1;      // steps of the head
  int steps;       // all steps of the head
};

// Fills the plan (all threads of the CTA; one barrier or more, the last one
// after the plan is complete).  The flattened list is ordered by sequence, KV
// head, row block, step; CTA c of G takes [c W / G, (c + 1) W / G).
__device__ __forceinline__ void tree_plan(const TreeArgs& a, int step, TreePlan* plan) {
  const int per = a.Hkv * a.blocks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = blockDim.x >> 5;
  if (!a.lengths) {
    if (threadIdx.x == 0) {
      const long long seq = per * tree_steps(a, a.Nk, step);
      plan->total = seq * a.B;
      plan->begin = blockIdx.x * plan->total / gridDim.x;
      plan->end = (blockIdx.x + 1) * plan->total / gridDim.x;
      plan->seq = seq > 0 ? static_cast<int>(plan->begin / seq) : 0;
      plan->seq0 = plan->seq * seq;
    }
    __syncthreads();
    return;
  }
  long long sum = 0;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) sum += per * tree_steps(a, tree_length(a, b), step);
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
  if (lane == 0) plan->warp_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    long long total = lane < nw ? plan->warp_sum[lane] : 0;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) total += __shfl_xor_sync(0xffffffffu, total, sh);
    const long long begin = blockIdx.x * total / gridDim.x;
    // the sequence that holds `begin`: 32 sequences at a time
    long long base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const long long n = b0 + lane < a.B ? per * tree_steps(a, tree_length(a, b0 + lane), step) : 0;
      long long inc = n;
#pragma unroll
      for (int sh = 1; sh < 32; sh <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, sh);
        if (lane >= sh) inc += o;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, base + inc > begin);
      if (past) {
        const int w = __ffs(past) - 1;
        const long long before = __shfl_sync(0xffffffffu, inc - n, w);
        if (lane == 0) {
          plan->seq = b0 + w;
          plan->seq0 = base + before;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      plan->total = total;
      plan->begin = begin;
      plan->end = (blockIdx.x + 1) * total / gridDim.x;
    }
  }
  __syncthreads();
}

// The segment that starts at step p (plan.begin <= p < plan.end) of the
// flattened list, cut at the plan's end.  Segments are taken in order.
__device__ __forceinline__ TreeSeg tree_segment(const TreeArgs& a, TreePlan& plan, long long p, int step) {
  TreeSeg s;
  int b = plan.seq;
  long long seq0 = plan.seq0;
  const long long per = static_cast<long long>(a.Hkv) * a.blocks;
  s.len = tree_length(a, b);
  long long n = tree_steps(a, s.len, step);
  while (p >= seq0 + per * n && b + 1 < a.B) {  // sequences of no steps are passed over
    seq0 += per * n;
    s.len = tree_length(a, ++b);
    n = tree_steps(a, s.len, step);
  }
  const long long off = p - seq0, head = off / n;
  s.b = b;
  s.hkv = static_cast<int>(head / a.blocks);
  s.rb = static_cast<int>(head % a.blocks);
  s.steps = static_cast<int>(n);
  s.s0 = static_cast<int>(off - head * n);
  const long long left = plan.end - p;
  s.s1 = static_cast<int>(min(static_cast<long long>(s.s0) + left, n));
  return s;
}

// c = fp32(fp32(sq * sm_scale) * log2 e) of a query head's tokens (T <= 128: one
// scale block).  A factor of 0 (all the head's codes 0) becomes 1e-30: 2^(S c) is
// 1 all the same for every |S| < 2^21, and a hidden key's -inf stays -inf.
__device__ __forceinline__ float tree_factor(const TreeArgs& a, int b, int hq) {
  const float sq = a.q_gran == 0 ? a.q_scales[0] : a.q_scales[b * a.Hq + hq];
  const float c = __fmul_rn(__fmul_rn(sq, a.sm_scale), kLog2e);
  return c > 0.f ? c : 1e-30f;
}

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
  return a.tree_mask[(static_cast<size_t>(b) * a.T + i) * words + s] & real;
}

__device__ __forceinline__ uint32_t code_byte(float x) {
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(x), -127.f), 127.f))) & 0xffu;
}

// The codes of drafts j0 .. j0 + n - 1 (zero past T) of (b, hkv), as
// qattn_kv_append would store them with the header as it stands: kc =
// clamp(rint((K - mu) / s_k)), vc = clamp(rint(V / s_v)).  `nthr` threads (a
// multiple of 32), this one `tid`; k_at(r, c) and v_at(r, c) give the address of
// 16-byte chunk c of row r.
template <int D, typename FK, typename FV>
__device__ __forceinline__ void tree_encode_drafts(const TreeArgs& a, int b, int hkv, int j0, int n,
                                                   int tid, int nthr, FK k_at, FV v_at) {
  constexpr int W = D / 4;  // words of a row
  const int w = tid % W;    // W <= 32 divides nthr
  const size_t ch = (static_cast<size_t>(b) * a.Hkv + hkv) * D + 4 * w;
  const float4 ks = *reinterpret_cast<const float4*>(a.k_chan_scale + ch);
  const float4 mu = *reinterpret_cast<const float4*>(a.k_mean + ch);
  const float4 vs = *reinterpret_cast<const float4*>(a.v_chan_scale + ch);
  const uint16_t* K = a.k_new + b * a.ksB + hkv * a.ksH + 4 * w;
  const uint16_t* V = a.v_new + b * a.vsB + hkv * a.vsH + 4 * w;
  for (int r = tid / W; r < n; r += nthr / W) {
    uint32_t kc = 0u, vc = 0u;
    if (j0 + r < a.T) {
      const uint2 k = *reinterpret_cast<const uint2*>(K + (j0 + r) * a.ksN);
      const uint2 v = *reinterpret_cast<const uint2*>(V + (j0 + r) * a.vsN);
      kc = code_byte(__fdiv_rn(__fsub_rn(bf16_bits_to_f32(k.x & 0xffffu), mu.x), ks.x)) |
           code_byte(__fdiv_rn(__fsub_rn(bf16_bits_to_f32(k.x >> 16), mu.y), ks.y)) << 8 |
           code_byte(__fdiv_rn(__fsub_rn(bf16_bits_to_f32(k.y & 0xffffu), mu.z), ks.z)) << 16 |
           code_byte(__fdiv_rn(__fsub_rn(bf16_bits_to_f32(k.y >> 16), mu.w), ks.w)) << 24;
      vc = code_byte(__fdiv_rn(bf16_bits_to_f32(v.x & 0xffffu), vs.x)) |
           code_byte(__fdiv_rn(bf16_bits_to_f32(v.x >> 16), vs.y)) << 8 |
           code_byte(__fdiv_rn(bf16_bits_to_f32(v.y & 0xffffu), vs.z)) << 16 |
           code_byte(__fdiv_rn(bf16_bits_to_f32(v.y >> 16), vs.w)) << 24;
    }
    *reinterpret_cast<uint32_t*>(k_at(r, w >> 2) + 4 * (w & 3)) = kc;
    *reinterpret_cast<uint32_t*>(v_at(r, w >> 2) + 4 * (w & 3)) = vc;
  }
}

// Four channels c.. of row rr (query head of the group, token) of (b, hkv):
// O = x s_v / l, 0 for a row that sees nothing; the row's lse with channel 0.
template <int D>
__device__ __forceinline__ void tree_write_out(const TreeArgs& a, int b, int hkv, int rr, int c,
                                               float4 x, float m, float l) {
  if (rr >= a.G * a.T) return;
  const int hq = rr / a.T, i = rr % a.T;
  const size_t row = (static_cast<size_t>(b) * a.Hq + hkv * a.G + hq) * a.T + i;
  if (!QATTN_IN_BOUNDS(row < a.rows_total)) return;
  const float4 sv =
      *reinterpret_cast<const float4*>(a.v_chan_scale + (static_cast<size_t>(b) * a.Hkv + hkv) * D + c);
  const float inv = l > 0.f ? 1.f / l : 0.f;
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
  if (a.lse && c == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
}

// Joins the shares of the heads that more than one CTA worked on: one CTA per
// (row of the block, head and row block).  A head's steps are [x0, x1) of the
// flattened list, so its CTAs are those whose shares meet that range; CTA c left
// its share in slot 2 c when the head began before it, else in 2 c + 1.
template <int D, int ROWS, int STEP>
__global__ void __launch_bounds__(kTreeJoinThreads) tree_join_kernel(const TreeArgs a) {
  constexpr int NW = kTreeJoinThreads / 32;
  constexpr int CPL = D / 32;  // channels per lane
  __shared__ TreePlan plan;
  __shared__ float sm[NW], sl[NW];
  __shared__ __align__(16) float so[NW][D];
  const int r = blockIdx.y;
  const int rb = blockIdx.x % a.blocks, bkv = blockIdx.x / a.blocks;
  const int b = bkv / a.Hkv, hkv = bkv % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (rb * ROWS + r >= a.G * a.T) return;
  pdl_wait();
  // total steps, and the steps of the sequences before b
  const int per = a.Hkv * a.blocks;
  long long tot = 0, before = 0;
  for (int x = threadIdx.x; x < a.B; x += kTreeJoinThreads) {
    const long long n = per * tree_steps(a, tree_length(a, x), STEP);
    tot += n;
    if (x < b) before += n;
  }
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) {
    tot += __shfl_xor_sync(0xffffffffu, tot, sh);
    before += __shfl_xor_sync(0xffffffffu, before, sh);
  }
  if (lane == 0) {
    plan.warp_sum[warp] = tot;
    plan.warp_sum[NW + warp] = before;
  }
  __syncthreads();
  tot = before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    tot += plan.warp_sum[w];
    before += plan.warp_sum[NW + w];
  }
  const long long n = tree_steps(a, tree_length(a, b), STEP);
  if (n == 0) {  // no cached row and no draft: nothing is visible
    if (warp == 0 && lane < D / 4)
      tree_write_out<D>(a, b, hkv, rb * ROWS + r, 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f), kNegInf, 0.f);
    return;
  }
  const long long x0 = before + (static_cast<long long>(hkv) * a.blocks + rb) * n, x1 = x0 + n;
  const long long G = a.ctas;
  // the CTA that holds step x: the largest c with floor(c W / G) <= x
  const int c0 = static_cast<int>(((x0 + 1) * G - 1) / tot);
  const int c1 = static_cast<int>((x1 * G - 1) / tot);
  if (c0 == c1) return;  // written whole
  float m = kNegInf, l = 0.f, o[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) o[k] = 0.f;
  for (int c = c0 + warp; c <= c1; c += NW) {
    const long long start = c * tot / G;
    const size_t slot = 2 * static_cast<size_t>(c) + (x0 < start ? 0 : 1);
    if (!QATTN_IN_BOUNDS(slot < a.slots)) break;
    const float mc = a.part_m[slot * ROWS + r], lc = a.part_l[slot * ROWS + r];
    const float* po = a.part_o + (slot * ROWS + r) * D + CPL * lane;
    float oc[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) oc[k] = po[k];
    if (mc == kNegInf) continue;
    const float mn = fmaxf(m, mc);
    const float f = (m == kNegInf) ? 0.f : ex2_approx(m - mn), w = ex2_approx(mc - mn);
    l = fmaf(w, lc, l * f);
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] = fmaf(w, oc[k], o[k] * f);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < CPL; ++k) so[warp][CPL * lane + k] = o[k];
  __syncthreads();
  if (threadIdx.x < D / 4) {
    const int c = 4 * threadIdx.x;
    float mx = kNegInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm[w]);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (sm[w] == kNegInf) continue;
      const float f = ex2_approx(sm[w] - mx);
      lt = fmaf(f, sl[w], lt);
      const float4 y = *reinterpret_cast<const float4*>(&so[w][c]);
      x.x = fmaf(f, y.x, x.x);
      x.y = fmaf(f, y.y, x.y);
      x.z = fmaf(f, y.z, x.z);
      x.w = fmaf(f, y.w, x.w);
    }
    tree_write_out<D>(a, b, hkv, rb * ROWS + r, c, x, mx, lt);
  }
}

}  // namespace qattn
