// Rotary positions (qattn_rotate) and the tokens of a serving step entered in a
// paged 8-bit KV cache (qattn_paged_append).
//
// Mathematics.  A pair (x1, x2) of channels turns by its token's angle:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,
// every product and sum rounded to fp32 by itself, so that codes made from the
// result do not depend on how a compiler fuses them.  A page of a KV head holds
// one scale, s = amax fp32(1 / top) (top: 127 or 448); a page that holds rows already
// keeps its scale, or doubles it until the new rows fit and halves the old rows'
// codes as often: doublings keep what an old row loses below one step in all,
// however often the page's scale grows.
//
// Work item: eight channels of a row.  In the half layout those are channels
// 4 i .. 4 i + 3 and their partners rot / 2 further, else eight neighbours, so
// that an item needs four cosines and four sines either way.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

// ------------------------------------------------------------------ items
struct Item8 {
  float v[8];
};

// First channels of an item's two quads: `i` of the row's d / 8 items.
__device__ __forceinline__ void item_channels(int i, int rot, bool inter, int& c0, int& c1, bool& turned) {
  turned = 8 * i < rot;
  const bool split = turned && !inter;
  c0 = split ? 4 * i : 8 * i;
  c1 = split ? rot / 2 + 4 * i : 8 * i + 4;
}
__device__ __forceinline__ Item8 load_item(const uint16_t* row, int c0, int c1) {
  Item8 x;
  uint2 a, b;
  if (c1 == c0 + 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(row + c0);
    a = make_uint2(w.x, w.y);
    b = make_uint2(w.z, w.w);
  } else {
    a = *reinterpret_cast<const uint2*>(row + c0);
    b = *reinterpret_cast<const uint2*>(row + c1);
  }
  const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x.v[2 * k] = bf16_bits_to_f32(w[k] & 0xffffu);
    x.v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  return x;
}
__device__ __forceinline__ Item8 load_item(const float* row, int c0, int c1) {
  const float4 a = *reinterpret_cast<const float4*>(row + c0), b = *reinterpret_cast<const float4*>(row + c1);
  return Item8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store_item(uint16_t* row, int c0, int c1, const Item8& x) {
  const uint2 a = make_uint2(pack_bf16(x.v[0], x.v[1]), pack_bf16(x.v[2], x.v[3]));
  const uint2 b = make_uint2(pack_bf16(x.v[4], x.v[5]), pack_bf16(x.v[6], x.v[7]));
  if (c1 == c0 + 4) {
    *reinterpret_cast<uint4*>(row + c0) = make_uint4(a.x, a.y, b.x, b.y);
  } else {
    *reinterpret_cast<uint2*>(row + c0) = a;
    *reinterpret_cast<uint2*>(row + c1) = b;
  }
}
__device__ __forceinline__ void store_item(float* row, int c0, int c1, const Item8& x) {
  *reinterpret_cast<float4*>(row + c0) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  *reinterpret_cast<float4*>(row + c1) = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}

// Four cosines and sines of item i of a position's row of the table.
__device__ __forceinline__ void load_angles(const RopeArgs& r, int pos, int i, float4& c, float4& s) {
  const float* row = r.table + static_cast<size_t>(pos) * r.rot + 4 * i;
  c = __ldg(reinterpret_cast<const float4*>(row));
  s = __ldg(reinterpret_cast<const float4*>(row + r.rot / 2));
  if (r.inverse) s = make_float4(-s.x, -s.y, -s.z, -s.w);
}
__device__ __forceinline__ void turn(Item8& x, float4 c4, float4 s4, bool inter) {
  const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
  Item8 y;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = inter ? x.v[2 * k] : x.v[k], b = inter ? x.v[2 * k + 1] : x.v[4 + k];
    const float u = __fsub_rn(__fmul_rn(a, c[k]), __fmul_rn(b, s[k]));
    const float w = __fadd_rn(__fmul_rn(b, c[k]), __fmul_rn(a, s[k]));
    if (inter) {
      y.v[2 * k] = u;
      y.v[2 * k + 1] = w;
    } else {
      y.v[k] = u;
      y.v[4 + k] = w;
    }
  }
  x = y;
}

// ------------------------------------------------------------------ rotate
constexpr int kRotateThreads = 256;
constexpr int kRotateHeads = 8;  // heads a thread turns by the same angles

template <typename T>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateArgs a) {
  const int items = a.d / 8;
  const int i = threadIdx.x % items, per = kRotateThreads / items;
  const long long tok = static_cast<long long>(blockIdx.x) * per + threadIdx.x / items;
  const int h0 = blockIdx.y * a.heads, h1 = min(a.H, h0 + a.heads);
  pdl_trigger();
  pdl_wait();
  if (tok >= static_cast<long long>(a.B) * a.T) return;
  const int b = static_cast<int>(tok / a.T), t = static_cast<int>(tok % a.T);
  const int pos = a.positions ? a.positions[tok] : t;
  if (pos < 0 || pos >= a.rope.n) {  // outside the table: the row is left as it was
    if (i == 0 && h0 == 0) atomicOr(a.err, kErrDomain);
    return;
  }
  int c0, c1;
  bool turned;
  item_channels(i, a.rope.rot, a.rope.inter, c0, c1, turned);
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turned) load_angles(a.rope, pos, i, c, s);
  const T* X = static_cast<const T*>(a.x) + b * a.xsB + t * a.xsN;
  T* Y = static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.H * a.T + t) * a.d;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    if (!QATTN_IN_BOUNDS(b < a.B && h < a.H && c1 + 4 <= a.d)) continue;
    Item8 x = load_item(X + h * a.xsH, c0, c1);
    if (turned) turn(x, c, s, a.rope.inter);
    store_item(Y + static_cast<size_t>(h) * a.T * a.d, c0, c1, x);
  }
}

// ------------------------------------------------------------------ append
// A CTA takes one page of one sequence and some heads of one kind (K, V or Q): its
// threads hold the page's new rows in registers (NIT items each), reduce the largest
// magnitude, settle the scale and write the codes.
constexpr int kItems = 8;  // rows' items a thread holds

template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    return cvt_e4m3x2(a, b) | cvt_e4m3x2(c, d) << 16;
  } else {
    auto byte = [](float x) {
      return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(x), -127.f), 127.f))) & 0xffu;
    };
    return byte(a) | byte(b) << 8 | byte(c) << 16 | byte(d) << 24;
  }
}
// The four codes of a word, divided by a power of two (mul = 2^-k) and rounded again.
template <bool E4M3>
__device__ __forceinline__ uint32_t divide4(uint32_t w, float mul) {
  float x[4];
  if constexpr (E4M3) {
    const uint32_t lo = e4m3x2_to_f16x2(w & 0xffffu), hi = e4m3x2_to_f16x2(w >> 16);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = static_cast<float>(static_cast<int8_t>(w >> (8 * k)));
  }
  return encode4<E4M3>(__fmul_rn(x[0], mul), __fmul_rn(x[1], mul), __fmul_rn(x[2], mul), __fmul_rn(x[3], mul));
}

template <bool E4M3>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedAppendArgs a) {
  constexpr float kTop = E4M3 ? 448.f : 127.f;
  __shared__ uint32_t red[2][8];
  const int b = blockIdx.z;
  // heads of this CTA: K's groups, then V's, then Q's
  int kind = 0, grp = blockIdx.x;
  const int gkv = (a.Hkv + a.heads - 1) / a.heads;
  while (kind < 2 && grp >= gkv) {
    grp -= gkv;
    ++kind;
  }
  const int H = kind == 2 ? a.Hq : a.Hkv;
  const int h0 = grp * a.heads, h1 = min(H, h0 + a.heads);
  const int items = a.d / 8, per = blockDim.x / items;
  const int i = threadIdx.x % items, rw = threadIdx.x / items;
  pdl_trigger();
  pdl_wait();
  const int len = a.lengths[b], n = a.n_new ? a.n_new[b] : a.T;
  if (n < 0 || n > a.T || len > a.Nk || len < n) {  // the sequence is left as it is
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, kErrDomain);
    return;
  }
  const int first = len - n;  // the row of token 0
  const int j = (first >> a.page_shift) + blockIdx.y, row0 = j << a.page_shift;
  if (n == 0 || row0 >= len) return;
  const bool held = row0 < first;  // rows of the page that were there before
  int page = -1;
  if (kind < 2 && QATTN_IN_BOUNDS(j < a.max_pages)) {
    page = a.page_table[static_cast<size_t>(b) * a.max_pages + j];
    if (page < 0 || page >= a.n_pages) {  // no such page: its rows are not written
      if (threadIdx.x == 0) atomicOr(a.err, kErrDomain);
      return;
    }
  }
  const bool rotated = kind != 1 && a.rope.table != nullptr;
  int c0, c1;
  bool turned;
  item_channels(i, rotated ? a.rope.rot : 0, a.rope.inter, c0, c1, turned);
  const uint16_t* X = kind == 0 ? a.k : kind == 1 ? a.v : a.q;
  const long long sB = kind == 0 ? a.ksB : kind == 1 ? a.vsB : a.qsB;
  const long long sH = kind == 0 ? a.ksH : kind == 1 ? a.vsH : a.qsH;
  const long long sN = kind == 0 ? a.ksN : kind == 1 ? a.vsN : a.qsN;
  X += b * sB;
  uint8_t* pages = kind == 0 ? a.k_pages : a.v_pages;
  float* scales = kind == 0 ? a.k_scales : a.v_scales;
  // this thread's rows of the page: rw + per k, their tokens' positions
  auto token = [&](int k) { return row0 + rw + per * k - first; };
  auto live = [&](int k) {
    const int r = rw + per * k, t = token(k);
    return r < (1 << a.page_shift) && t >= 0 && t < n;
  };
  auto position = [&](int t) {
    return a.positions ? a.positions[static_cast<size_t>(b) * a.T + t] : first + t;
  };
  uint32_t ok = 0;  // bit k: row k is written
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (!live(k)) continue;
    if (rotated) {
      const int p = position(token(k));
      if (p < 0 || p >= a.rope.n) {  // outside the table: the token is not written
        if (i == 0) atomicOr(a.err, kErrDomain);
        continue;
      }
    }
    ok |= 1u << k;
  }
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    Item8 x[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (!((ok >> k) & 1u) || !QATTN_IN_BOUNDS(token(k) < a.T && h < H)) continue;
      x[k] = load_item(X + h * sH + token(k) * sN, c0, c1);
    }
    if (turned) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (!((ok >> k) & 1u)) continue;
        float4 c, s;
        load_angles(a.rope, position(token(k)), i, c, s);
        turn(x[k], c, s, a.rope.inter);
      }
    }
    if (kind == 2) {
#pragma unroll
      for (int k = 0; k < kItems; ++k) {
        if (!((ok >> k) & 1u)) continue;
        const size_t row = (static_cast<size_t>(b) * a.Hq + h) * a.T + token(k);
        store_item(a.q_out + row * a.d, c0, c1, x[k]);
      }
      continue;
    }
    // the largest magnitude, as bits: NaN lies above infinity, infinity above every number
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (!((ok >> k) & 1u)) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[k].v[e]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) red[h & 1][threadIdx.x >> 5] = top;
    const size_t sc = static_cast<size_t>(page) * a.Hkv + h;
    const float was = held ? scales[sc] : 0.f;
    __syncthreads();  // also: every thread has the old scale
    top = 0;
    for (unsigned w = 0; w < blockDim.x / 32; ++w) top = max(top, red[h & 1][w]);
    const float amax = __uint_as_float(top);
    // the page's scale, and the doublings of the old one
    float s;
    int up = 0;
    const bool finite = top < 0x7f800000u;
    if (!finite || !(was >= 0.f && was < __builtin_huge_valf())) {
      s = __uint_as_float(0x7fffffffu);
    } else if (was >= 0x1p-100f) {
      const float fit = __fmul_rn(was, kTop);
      if (amax > fit) {
        const uint32_t f = __float_as_uint(fit);
        up = static_cast<int>(top >> 23) - static_cast<int>(f >> 23) + ((top & 0x7fffffu) > (f & 0x7fffffu) ? 1 : 0);
      }
      s = ldexpf(was, up);
    } else {
      s = amax < 0x1p-64f ? 0.f : __fmul_rn(amax, 1.f / kTop);
      up = held && s > 0.f ? 127 : 0;  // rows held with no scale are zeros, and stay so
    }
    if (threadIdx.x == 0 && QATTN_IN_BOUNDS(page >= 0 && page < a.n_pages)) scales[sc] = s;
    uint8_t* P = pages + (sc << a.page_shift) * a.d;
    if (up > 0) {  // the rows that were there: their codes halved as often
      const float mul = up > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      const int words = (first - row0) * a.d / 16;
      for (int w = threadIdx.x; w < words; w += blockDim.x) {
        if (!QATTN_IN_BOUNDS(16 * w < (a.d << a.page_shift))) continue;
        uint4 v = *reinterpret_cast<const uint4*>(P + 16 * w);
        v = make_uint4(divide4<E4M3>(v.x, mul), divide4<E4M3>(v.y, mul), divide4<E4M3>(v.z, mul),
                       divide4<E4M3>(v.w, mul));
        *reinterpret_cast<uint4*>(P + 16 * w) = v;
      }
    }
    const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;  // (0 for NaN: codes of zero)
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      if (!((ok >> k) & 1u)) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = finite && inv > 0.f ? __fmul_rn(x[k].v[e], inv) : 0.f;
      const uint32_t lo = encode4<E4M3>(y[0], y[1], y[2], y[3]), hi = encode4<E4M3>(y[4], y[5], y[6], y[7]);
      uint8_t* row = P + (rw + per * k) * a.d;
      if (c1 == c0 + 4) {
        *reinterpret_cast<uint2*>(row + c0) = make_uint2(lo, hi);
      } else {
        *reinterpret_cast<uint32_t*>(row + c0) = lo;
        *reinterpret_cast<uint32_t*>(row + c1) = hi;
      }
    }
  }
}

}  // namespace

unsigned int check_take_paged_cache() { return check_take_local(); }

cudaError_t launch_rotate(RotateArgs a, cudaStream_t s) {
  const int per = kRotateThreads / (a.d / 8);
  const long long tokens = static_cast<long long>(a.B) * a.T;
  a.heads = kRotateHeads;
  const dim3 grid(static_cast<unsigned int>((tokens + per - 1) / per), static_cast<unsigned int>((a.H + a.heads - 1) / a.heads));
  return a.f32 ? launch_pdl(rotate_kernel<float>, grid, dim3(kRotateThreads), 0, s, a)
               : launch_pdl(rotate_kernel<uint16_t>, grid, dim3(kRotateThreads), 0, s, a);
}

cudaError_t launch_paged_append(PagedAppendArgs a, cudaStream_t s) {
  const int page = 1 << a.page_shift;
  const int threads = page * (a.d / 8) / kItems;
  // pages that a sequence's new rows touch, at most
  const int touched = (a.T + page - 2) / page + 1;
  a.heads = 1;
  const int groups = 2 * ((a.Hkv + a.heads - 1) / a.heads) + (a.q ? (a.Hq + a.heads - 1) / a.heads : 0);
  const dim3 grid(groups, touched, a.B);
  return a.e4m3 ? launch_pdl(paged_append_kernel<true>, grid, dim3(threads), 0, s, a)
                : launch_pdl(paged_append_kernel<false>, grid, dim3(threads), 0, s, a);
}

}  // namespace qattn
