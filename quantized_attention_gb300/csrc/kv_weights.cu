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
constexpr int kRowsChunk = 64;                // query rows in shared memory at a time

__device__ __forceinline__ int row_count(const WeightArgs& a, int b) {
  if (!a.lengths) return a.Nk;
  const int n = a.lengths[b];
  if (n < 0 || n > a.Nk) {
    atomicOr(a.err, kErrDomain);
    return n < 0 ? 0 : a.Nk;
  }
  return n;
}

__device__ __forceinline__ float scale_of(const float* s, int gran, int bh, int nblk, int blk) {
  if (gran == 0) return s[0];
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
// One CTA per 256 keys of a (sequence, KV head); a warp holds 32 keys as fp16 A
// fragments in registers (their codes are read once, straight from global
// memory: 4 lanes cover a key's row) and every query row of the group passes by
// in chunks of 64 rows of codes in shared memory.  Lane (g, t) takes channels
// D/4 t .. of its keys and rows, so a k-step's fragment is one word of each.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_weights_warp_kernel(const WeightArgs a) {
  constexpr int KS = D / 16;
  __shared__ __align__(16) uint8_t sq[kRowsChunk * D];
  __shared__ float2 rowc[kRowsChunk];  // {factor sq sm log2 e, lse log2 e}
  __shared__ int rowi[kRowsChunk];     // token of the row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  pdl_trigger();
  pdl_wait();
  const int bkv = blockIdx.y, b = bkv / a.Hkv, hkv = bkv % a.Hkv;
  const int len = row_count(a, b);
  const int k0 = blockIdx.x * kKeys;
  if (k0 >= len) return;
  const int kw = k0 + warp * kKeysPerWarp;
  const int pos0 = a.pos0_len ? len - a.Nq : a.pos0;

  // the warp's 32 keys: key 16 mt + g + 8 h, words of this lane's channels
  uint32_t ka[2][KS][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = kw + 16 * mt + 8 * h + g;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.k_codes) +
                           (static_cast<size_t>(bkv) * a.cap + key) * D + (D / 4) * t4;
#pragma unroll
      for (int w4 = 0; w4 < KS / 4; ++w4) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (key < len && QATTN_IN_BOUNDS(key < a.cap)) x = *reinterpret_cast<const uint4*>(src + 16 * w4);
        codes4_to_f16x2(x.x, ka[mt][4 * w4 + 0][h], ka[mt][4 * w4 + 0][2 + h]);
        codes4_to_f16x2(x.y, ka[mt][4 * w4 + 1][h], ka[mt][4 * w4 + 1][2 + h]);
        codes4_to_f16x2(x.z, ka[mt][4 * w4 + 2][h], ka[mt][4 * w4 + 2][2 + h]);
        codes4_to_f16x2(x.w, ka[mt][4 * w4 + 3][h], ka[mt][4 * w4 + 3][2 + h]);
      }
    }
  }
  const int nkb = (a.Nk + 127) / 128, nqb = (a.Nq + 127) / 128;
  const float sk = a.k_scales ? scale_of(a.k_scales, a.k_gran, bkv, nkb, min(kw, a.Nk - 1) / 128) : 1.f;
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};

  // queries that can see any of this CTA's keys: causal, tokens >= k0 - pos0
  const int i_first = a.causal ? max(0, k0 - pos0) : 0;
  for (int hq = 0; hq < a.G; ++hq) {
    const int bh = b * a.Hq + hkv * a.G + hq;
    for (int i0 = i_first; i0 < a.Nq; i0 += kRowsChunk) {
      const int n = min(kRowsChunk, a.Nq - i0);
      __syncthreads();
      const size_t row0 = static_cast<size_t>(bh) * a.Nq + i0;
      for (int x = threadIdx.x; x < kRowsChunk * (D / 16); x += kThreads) {
        const int r = x / (D / 16), c = x % (D / 16);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < n) v = *reinterpret_cast<const uint4*>(a.q_codes + (row0 + r) * D + 16 * c);
        *reinterpret_cast<uint4*>(sq + r * D + 16 * (c ^ (r & (D / 16 - 1)))) = v;
      }
      for (int r = threadIdx.x; r < kRowsChunk; r += kThreads) {
        float2 f = make_float2(0.f, -kNegInf);  // a row past the end: 2^(0 - inf) = 0
        if (r < n) {
          const float s = scale_of(a.q_scales, a.q_gran, bh, nqb, (i0 + r) / 128);
          const float e = a.lse[row0 + r];
          // a query that saw nothing (lse = -inf) gives nothing
          f = make_float2(__fmul_rn(__fmul_rn(s, a.sm_scale), kLog2e), e == kNegInf ? -kNegInf : e * kLog2e);
        }
        rowc[r] = f;
        rowi[r] = i0 + r;
      }
      __syncthreads();
      for (int r0 = 0; r0 < n; r0 += 8) {
        // B fragments: row r0 + g, this lane's channels
        uint32_t qb[KS][2];
#pragma unroll
        for (int w4 = 0; w4 < KS / 4; ++w4) {
          const int r = r0 + g, c = (KS / 4) * t4 + w4;
          const uint4 x = *reinterpret_cast<const uint4*>(sq + r * D + 16 * (c ^ (r & (D / 16 - 1))));
          codes4_to_f16x2(x.x, qb[4 * w4 + 0][0], qb[4 * w4 + 0][1]);
          codes4_to_f16x2(x.y, qb[4 * w4 + 1][0], qb[4 * w4 + 1][1]);
          codes4_to_f16x2(x.z, qb[4 * w4 + 2][0], qb[4 * w4 + 2][1]);
          codes4_to_f16x2(x.w, qb[4 * w4 + 3][0], qb[4 * w4 + 3][1]);
        }
        const float2 f0 = rowc[r0 + 2 * t4], f1 = rowc[r0 + 2 * t4 + 1];
        const float c0 = f0.x * sk, c1 = f1.x * sk;
        const int lim0 = a.causal ? pos0 + rowi[r0 + 2 * t4] : 0x7fffffff;
        const int lim1 = a.causal ? pos0 + rowi[r0 + 2 * t4 + 1] : 0x7fffffff;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) mma16816(s, ka[mt][ks], qb[ks][0], qb[ks][1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = kw + 16 * mt + 8 * h + g;
            const float p0 = ex2_approx(fmaf(s[2 * h], c0, -f0.y));
            const float p1 = ex2_approx(fmaf(s[2 * h + 1], c1, -f1.y));
            acc[mt][h] += (key <= lim0 ? p0 : 0.f) + (key <= lim1 ? p1 : 0.f);
          }
        }
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
      if (t4 == 0 && key < len && QATTN_IN_BOUNDS(key < a.cap)) {
        const size_t o = static_cast<size_t>(bkv) * a.cap + key;
        a.weights[o] = (a.base ? a.base[o] : 0.f) + x;
      }
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
