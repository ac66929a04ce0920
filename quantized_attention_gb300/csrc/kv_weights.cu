// The attention weight each cached row has received (qattn_kv_weights):
//   w[b][hk][k] = base + sum over the group's query heads h and tokens i that
//   see row k of 2^(t_hik - lse_hi log2 e),  t = S c (S the exact integer
//   product of the codes).
// The sum over queries of a probability matrix that is never stored.  The
// product is taken as S^T = K Q^T, so a key's sum stays with the threads that
// hold the key and no two CTAs add to one address: the order of the additions
// is fixed.
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

constexpr float kLog2e = 1.44269502162933349609375f;  // fp32(log2 e)
constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeysPerWarp = 32;
constexpr int kKeys = kWarps * kKeysPerWarp;  // keys of a CTA
constexpr int kRows = kWeightWarpRows;        // query rows, at most (a multiple of 8)
static_assert(kRows % 8 == 0, "rows come in fragments of 8");

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

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ few queries
// One CTA per 256 keys of a (sequence, KV head) and at most kWeightWarpRows query
// rows (query head of the group, token): a decode step.  A warp holds 32 keys as
// fp16 A fragments in registers (their codes are read once, straight from global
// memory); the rows wait in shared memory as fp16 B fragments with their
// constants.  Lane (g, t) takes 16-byte chunks t and t + 4 of its keys and rows
// (four lanes read 64 consecutive bytes), so a k-step's fragment is one word of
// each.  A step over 32K rows of 8 KV heads takes 12.8 us = 2.8 TB/s (floor 5.4).
// Bound by the latency of a warp's chain (load, widen, eight dependent MMAs,
// exponentials) at 16 warps an SM.  A CTA walking over several key blocks with the
// next block's loads in flight measured no faster (17.8 against 16.1 us, both before
// the rows waited as ready fragments): fewer warps fit.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_weights_warp_kernel(const WeightArgs a) {
  constexpr int KS = D / 16;
  constexpr int NC = D / 16;  // 16-byte chunks of a row's codes, 32 bytes as fp16
  __shared__ __align__(16) uint8_t sq[kRows * NC * 32];
  __shared__ float2 rowc[kRows];  // {factor sq sm log2 e, lse log2 e}
  __shared__ int rowi[kRows];     // token of the row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  pdl_trigger();
  pdl_wait();
  const int bkv = blockIdx.y, b = bkv / a.Hkv, hkv = bkv % a.Hkv;
  const int k0 = blockIdx.x * kKeys;
  const int kw = k0 + warp * kKeysPerWarp;
  const int R = a.G * a.Nq;
  const int len = row_count(a, b);
  if (k0 >= len) return;

  // the warp's 32 keys: key 16 mt + g + 8 h, this lane's chunks
  uint4 kx[2][2][KS / 4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = kw + 16 * mt + 8 * h + g;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.k_codes) +
                           (static_cast<size_t>(bkv) * a.cap + key) * D + 16 * t4;
#pragma unroll
      for (int w4 = 0; w4 < KS / 4; ++w4) {
        kx[mt][h][w4] = make_uint4(0u, 0u, 0u, 0u);
        if (key < len && QATTN_IN_BOUNDS(key < a.cap))
          kx[mt][h][w4] = *reinterpret_cast<const uint4*>(src + 64 * w4);
      }
    }
  }
  const int nkb = (a.Nk + 127) / 128, nqb = (a.Nq + 127) / 128;
  const float sk = a.k_scales ? scale_of(a.k_scales, a.k_gran, bkv, a.B * a.Hkv, nkb, min(kw, a.Nk - 1) / 128) : 1.f;
  const int pos0 = a.pos0_len ? len - a.Nq : a.pos0;
  const size_t row0 = (static_cast<size_t>(b) * a.Hq + hkv * a.G) * a.Nq;
  const size_t rows_total = static_cast<size_t>(a.B) * a.Hq * a.Nq;
  // rows, widened once: chunk c of row r at 32 (r NC + c), its two 16-byte halves
  // exchanged in odd rows (eight lanes of a read, four chunks of two rows, hit
  // eight bank groups)
  const int rows8 = (R + 7) & ~7;
  for (int x = threadIdx.x; x < rows8 * NC; x += kThreads) {
    const int r = x / NC, c = x % NC;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < R && QATTN_IN_BOUNDS(row0 + r < rows_total))
      v = *reinterpret_cast<const uint4*>(a.q_codes + (row0 + r) * D + 16 * c);
    uint32_t h[8];
    codes4_to_f16x2(v.x, h[0], h[1]);
    codes4_to_f16x2(v.y, h[2], h[3]);
    codes4_to_f16x2(v.z, h[4], h[5]);
    codes4_to_f16x2(v.w, h[6], h[7]);
    uint8_t* dst = sq + 32 * (r * NC + c);
    *reinterpret_cast<uint4*>(dst + 16 * (r & 1)) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(dst + 16 * (1 - (r & 1))) = make_uint4(h[4], h[5], h[6], h[7]);
  }
  if (threadIdx.x < rows8) {
    const int r = threadIdx.x;
    float2 f = make_float2(0.f, -kNegInf);  // a row past the end: 2^(0 - inf) = 0
    int i = 0;
    if (r < R && QATTN_IN_BOUNDS(row0 + r < rows_total)) {
      const int hq = r / a.Nq;
      i = r - hq * a.Nq;
      const float s = scale_of(a.q_scales, a.q_gran, b * a.Hq + hkv * a.G + hq, a.B * a.Hq, nqb, i / 128);
      const float e = a.lse[row0 + r];
      // a query that saw nothing (lse = -inf) gives nothing
      f = make_float2(weight_factor(s, a.sm_scale, e), e == kNegInf ? -kNegInf : e * kLog2e);
    }
    rowc[r] = f;
    rowi[r] = i;
  }
  uint32_t ka[2][KS][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int w4 = 0; w4 < KS / 4; ++w4) {
        const uint4 x = kx[mt][h][w4];
        codes4_to_f16x2(x.x, ka[mt][4 * w4 + 0][h], ka[mt][4 * w4 + 0][2 + h]);
        codes4_to_f16x2(x.y, ka[mt][4 * w4 + 1][h], ka[mt][4 * w4 + 1][2 + h]);
        codes4_to_f16x2(x.z, ka[mt][4 * w4 + 2][h], ka[mt][4 * w4 + 2][2 + h]);
        codes4_to_f16x2(x.w, ka[mt][4 * w4 + 3][h], ka[mt][4 * w4 + 3][2 + h]);
      }
    }
  }
  float old[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // the keys' base, in flight meanwhile
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = kw + 16 * mt + 8 * h + g;
      if (a.base && t4 == 0 && key < len && QATTN_IN_BOUNDS(key < a.cap))
        old[mt][h] = a.base[static_cast<size_t>(bkv) * a.cap + key];
    }
  }
  __syncthreads();
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
  for (int r0 = 0; r0 < R; r0 += 8) {
    uint32_t qb[KS][2];  // B fragments: row r0 + g, this lane's chunks
#pragma unroll
    for (int w4 = 0; w4 < KS / 4; ++w4) {
      const uint8_t* src = sq + 32 * ((r0 + g) * NC + t4 + 4 * w4);
      const uint4 lo = *reinterpret_cast<const uint4*>(src + 16 * (g & 1));
      const uint4 hi = *reinterpret_cast<const uint4*>(src + 16 * (1 - (g & 1)));
      qb[4 * w4 + 0][0] = lo.x;
      qb[4 * w4 + 0][1] = lo.y;
      qb[4 * w4 + 1][0] = lo.z;
      qb[4 * w4 + 1][1] = lo.w;
      qb[4 * w4 + 2][0] = hi.x;
      qb[4 * w4 + 2][1] = hi.y;
      qb[4 * w4 + 3][0] = hi.z;
      qb[4 * w4 + 3][1] = hi.w;
    }
    const float2 f0 = rowc[r0 + 2 * t4], f1 = rowc[r0 + 2 * t4 + 1];
    const float c0 = f0.x * sk, c1 = f1.x * sk;
    const int lim0 = a.causal ? pos0 + rowi[r0 + 2 * t4] : 0x7fffffff;
    const int lim1 = a.causal ? pos0 + rowi[r0 + 2 * t4 + 1] : 0x7fffffff;
    float s[2][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) mma16816(s[mt], ka[mt][ks], qb[ks][0], qb[ks][1]);
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = kw + 16 * mt + 8 * h + g;
        const float p0 = ex2_approx(fmaf(s[mt][2 * h], c0, -f0.y));
        const float p1 = ex2_approx(fmaf(s[mt][2 * h + 1], c1, -f1.y));
        acc[mt][h] += (key <= lim0 ? p0 : 0.f) + (key <= lim1 ? p1 : 0.f);
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = acc[mt][h];
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      const int key = kw + 16 * mt + 8 * h + g;
      if (t4 == 0 && key < len && QATTN_IN_BOUNDS(key < a.cap))
        a.weights[static_cast<size_t>(bkv) * a.cap + key] = old[mt][h] + x;
    }
  }
}

}  // namespace

unsigned int check_take_kv_weights() { return check_take_local(); }

cudaError_t launch_kv_weights_warp(const WeightArgs& a, cudaStream_t s) {
  const dim3 grid((a.Nk + kKeys - 1) / kKeys, a.B * a.Hkv);
  return a.d == 64 ? launch_pdl(kv_weights_warp_kernel<64>, grid, dim3(kThreads), 0, s, a)
                   : launch_pdl(kv_weights_warp_kernel<128>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace qattn
