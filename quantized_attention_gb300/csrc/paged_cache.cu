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
// Work item: W channels of a row (8, or 16 where the rotated and the other channels are
// multiples of it).  In the half layout those are W / 2 channels and their partners
// rot / 2 further, else W neighbours, so that an item needs W / 2 cosines and as many
// sines either way.
//
// Both are bound by memory: 3 products and sums a channel against 4 bytes moved (Q) or 3
// (K, V).  The figures below are for inputs that do not lie in L2, of 6.78 TB/s copied.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

// ------------------------------------------------------------------ items
template <int W>
struct Place {  // first channels of an item's halves
  int c0, c1;
  bool turned;
};
template <int W>
__device__ __forceinline__ Place<W> item_place(int i, int rot, bool inter) {
  Place<W> p;
  p.turned = W * i < rot;
  const bool split = p.turned && !inter;
  p.c0 = split ? (W / 2) * i : W * i;
  p.c1 = split ? rot / 2 + (W / 2) * i : W * i + W / 2;
  return p;
}
template <int W>
struct Item {
  float v[W];
};
template <int W>
struct Raw {  // an item as it lies: bf16 pairs
  uint32_t w[W / 2];
};
template <int W>
__device__ __forceinline__ Raw<W> load_raw(const uint16_t* row, const Place<W>& p) {
  Raw<W> x;
  if constexpr (W == 8) {
    const uint2 a = *reinterpret_cast<const uint2*>(row + p.c0), b = *reinterpret_cast<const uint2*>(row + p.c1);
    x.w[0] = a.x;
    x.w[1] = a.y;
    x.w[2] = b.x;
    x.w[3] = b.y;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(row + p.c0), b = *reinterpret_cast<const uint4*>(row + p.c1);
    x.w[0] = a.x;
    x.w[1] = a.y;
    x.w[2] = a.z;
    x.w[3] = a.w;
    x.w[4] = b.x;
    x.w[5] = b.y;
    x.w[6] = b.z;
    x.w[7] = b.w;
  }
  return x;
}
template <int W>
__device__ __forceinline__ Item<W> values(const Raw<W>& r) {
  Item<W> x;
#pragma unroll
  for (int k = 0; k < W / 2; ++k) {
    x.v[2 * k] = bf16_bits_to_f32(r.w[k] & 0xffffu);
    x.v[2 * k + 1] = __uint_as_float(r.w[k] & 0xffff0000u);
  }
  return x;
}
__device__ __forceinline__ Item<8> load_item(const float* row, const Place<8>& p) {
  const float4 a = *reinterpret_cast<const float4*>(row + p.c0), b = *reinterpret_cast<const float4*>(row + p.c1);
  return Item<8>{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
template <int W>
__device__ __forceinline__ Item<W> load_item(const uint16_t* row, const Place<W>& p) {
  return values<W>(load_raw<W>(row, p));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int W>
__device__ __forceinline__ void store_item(uint16_t* row, const Place<W>& p, const Item<W>& x) {
  uint32_t w[W / 2];
#pragma unroll
  for (int k = 0; k < W / 2; ++k) w[k] = pack_bf16(x.v[2 * k], x.v[2 * k + 1]);
  if constexpr (W == 8) {
    *reinterpret_cast<uint2*>(row + p.c0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(row + p.c1) = make_uint2(w[2], w[3]);
  } else {
    *reinterpret_cast<uint4*>(row + p.c0) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(row + p.c1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void store_item(float* row, const Place<8>& p, const Item<8>& x) {
  *reinterpret_cast<float4*>(row + p.c0) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
  *reinterpret_cast<float4*>(row + p.c1) = make_float4(x.v[4], x.v[5], x.v[6], x.v[7]);
}

template <int W>
struct Angles {
  float c[W / 2], s[W / 2];
};
// Cosines and sines of item i of a position's row of the table.
template <int W>
__device__ __forceinline__ Angles<W> load_angles(const RopeArgs& r, int pos, int i) {
  Angles<W> a;
  const float* row = r.table + static_cast<size_t>(pos) * r.rot + (W / 2) * i;
#pragma unroll
  for (int k = 0; k < W / 2; k += 4) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + k));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + r.rot / 2 + k));
    a.c[k] = c.x;
    a.c[k + 1] = c.y;
    a.c[k + 2] = c.z;
    a.c[k + 3] = c.w;
    a.s[k] = r.inverse ? -s.x : s.x;
    a.s[k + 1] = r.inverse ? -s.y : s.y;
    a.s[k + 2] = r.inverse ? -s.z : s.z;
    a.s[k + 3] = r.inverse ? -s.w : s.w;
  }
  return a;
}
template <int W>
__device__ __forceinline__ Item<W> turn(const Item<W>& x, const Angles<W>& a, bool inter) {
  Item<W> y;
#pragma unroll
  for (int k = 0; k < W / 2; ++k) {
    const float p = inter ? x.v[2 * k] : x.v[k], q = inter ? x.v[2 * k + 1] : x.v[W / 2 + k];
    const float u = __fsub_rn(__fmul_rn(p, a.c[k]), __fmul_rn(q, a.s[k]));
    const float w = __fadd_rn(__fmul_rn(q, a.c[k]), __fmul_rn(p, a.s[k]));
    if (inter) {
      y.v[2 * k] = u;
      y.v[2 * k + 1] = w;
    } else {
      y.v[k] = u;
      y.v[W / 2 + k] = w;
    }
  }
  return y;
}

// ------------------------------------------------------------------ rotate
constexpr int kRotateThreads = 256;

// A thread turns one item of a token in kRotateHeads heads by the same angles.  32 heads of
// 128 channels, 8192 tokens: 26 us, 5.3 TB/s, 78% of a copy; what is left is the start and
// the last, partly filled wave (16384 tokens run at 85%).  8 channels an item instead of 16:
// 32.5 us; three CTAs an SM instead of four: 30.
template <typename T, int W>
__global__ void __launch_bounds__(kRotateThreads, 4) rotate_kernel(const RotateArgs a) {
  const int items = a.d / W, per = kRotateThreads / items;
  const int i = threadIdx.x % items;
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
  const Place<W> p = item_place<W>(i, a.rope.rot, a.rope.inter);
  Angles<W> ang{};
  if (p.turned) ang = load_angles<W>(a.rope, pos, i);
  const T* X = static_cast<const T*>(a.x) + b * a.xsB + t * a.xsN;
  T* Y = static_cast<T*>(a.y) + (static_cast<size_t>(b) * a.H * a.T + t) * a.d;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    if (!QATTN_IN_BOUNDS(b < a.B && h < a.H && p.c1 + W / 2 <= a.d)) continue;
    Item<W> x = load_item(X + h * a.xsH, p);
    if (p.turned) x = turn(x, ang, a.rope.inter);
    store_item(Y + static_cast<size_t>(h) * a.T * a.d, p, x);
  }
}

// ------------------------------------------------------------------ append
template <bool E4M3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (E4M3) {
    return cvt_e4m3x2(a, b) | cvt_e4m3x2(c, d) << 16;
  } else {
    // 1.5 2^23 + x: the integer nearest to x (half to even) in the low bits.  No clamp: a scale
    // is such that |x| is 127 and a few roundings at most
    auto bits = [](float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); };
    return __byte_perm(__byte_perm(bits(a), bits(b), 0x0040u), __byte_perm(bits(c), bits(d), 0x0040u), 0x5410u);
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

// The new rows of a sequence, checked.
struct NewRows {
  int first, len, n;  // the row of token 0, rows in use, new ones (0: nothing to do)
};
__device__ __forceinline__ NewRows new_rows(const PagedAppendArgs& a, int b, bool report) {
  NewRows s{0, a.lengths[b], a.n_new ? a.n_new[b] : a.T};
  if (s.n < 0 || s.n > a.T || s.len > a.Nk || s.len < s.n) {  // the sequence is left as it is
    if (report) atomicOr(a.err, kErrDomain);
    s.n = 0;
  }
  s.first = s.len - s.n;
  return s;
}
__device__ __forceinline__ int position(const PagedAppendArgs& a, int b, int first, int t) {
  return a.positions ? a.positions[static_cast<size_t>(b) * a.T + t] : first + t;
}

// Whose threads hold a page's new rows: a warp or a CTA.
template <bool CTA>
struct Team {
  uint32_t (*red)[32];  // [2][warps] (CTA)
  __device__ __forceinline__ int size() const { return CTA ? blockDim.x : 32; }
  __device__ __forceinline__ int rank() const { return CTA ? threadIdx.x : threadIdx.x & 31; }
  // The largest x of the team.  What its threads read and wrote before lies before what they
  // do after it (the page's scale: all read it, one then writes it; a warp's reduction alone
  // does not order memory).
  __device__ __forceinline__ uint32_t largest(uint32_t x, int turn) const {
    x = __reduce_max_sync(0xffffffffu, x);
    if constexpr (!CTA) {
      __syncwarp();
    } else {
      if ((threadIdx.x & 31) == 0) red[turn & 1][threadIdx.x >> 5] = x;
      __syncthreads();
      x = 0;
      for (unsigned w = 0; w < blockDim.x / 32; ++w) x = max(x, red[turn & 1][w]);
    }
    return x;
  }
};

// One page of a sequence and heads h0 .. h1 - 1 of K or V, by a team: the new rows of a
// head (NP items a thread, rows rw + per k) are held as they came; their largest magnitude
// settles the scale; the codes follow.  K's rows are turned twice, for the maximum and for
// the codes: angles come from L1 and the registers stay few (rows held as they were turned:
// 71 us against 61 for the prompts below).  The rows are asked for before the page is known
// (66 us after it).
template <bool E4M3, int NP, bool CTA>
__device__ __forceinline__ void append_page(const PagedAppendArgs& a, const Team<CTA> team, int b, const NewRows& s,
                                            int j, bool is_v, int h0, int h1) {
  constexpr float kTop = E4M3 ? 448.f : 127.f;
  const int row0 = j << a.page_shift;
  const bool held = row0 < s.first;  // rows of the page that were there before
  if (!QATTN_IN_BOUNDS(j < a.max_pages)) return;
  const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + j];
  const int items = a.d / 8, per = team.size() / items;
  const int i = team.rank() % items, rw = team.rank() / items;
  const bool rotated = !is_v && a.rope.table != nullptr;
  const Place<8> pl = item_place<8>(i, rotated ? a.rope.rot : 0, a.rope.inter);
  const uint16_t* X = (is_v ? a.v + b * a.vsB : a.k + b * a.ksB);
  const long long sH = is_v ? a.vsH : a.ksH, sN = is_v ? a.vsN : a.ksN;
  // rows of the page in turn from the first new one: `shift` + rw + per k
  const int shift = held ? s.first - row0 : 0, t0 = row0 + shift - s.first;  // its token
  const int rows = min(min(1 << a.page_shift, s.len - row0) - shift, s.n - t0);
  uint32_t ok = 0;  // bit k: row k is written
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    if (rw + per * k >= rows) continue;
    if (rotated) {
      const int pos = position(a, b, s.first, t0 + rw + per * k);
      if (pos < 0 || pos >= a.rope.n) {  // outside the table: the token is not written
        if (i == 0) atomicOr(a.err, kErrDomain);
        continue;
      }
    }
    ok |= 1u << k;
  }
  uint8_t* const pages = is_v ? a.v_pages : a.k_pages;
  float* const scales = is_v ? a.v_scales : a.k_scales;
  Raw<8> x[NP];
  auto value = [&](int k) {
    Item<8> v = values<8>(x[k]);
    if (pl.turned) v = turn(v, load_angles<8>(a.rope, position(a, b, s.first, t0 + rw + per * k), i), a.rope.inter);
    return v;
  };
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      x[k] = Raw<8>{};
      if (((ok >> k) & 1u) && QATTN_IN_BOUNDS(t0 + rw + per * k < a.T && h < a.Hkv))
        x[k] = load_raw<8>(X + h * sH + (t0 + rw + per * k) * sN, pl);
    }
    if (page < 0 || page >= a.n_pages) {  // no such page: its rows are not written
      if (team.rank() == 0) atomicOr(a.err, kErrDomain);
      return;
    }
    const size_t sc = static_cast<size_t>(page) * a.Hkv + h;
    const float was = held ? scales[sc] : 0.f;
    // the largest magnitude, NaN if one is
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (!((ok >> k) & 1u)) continue;
      const Item<8> v = value(k);
#pragma unroll
      for (int e = 0; e < 8; e += 2) big = fmax3_abs_nan(big, v.v[e], v.v[e + 1]);
    }
    // as bits: NaN lies above infinity, infinity above every number
    const uint32_t top = team.largest(__float_as_uint(big), h);  // (every thread has the old scale)
    const float amax = __uint_as_float(top);
    // the page's scale, and the doublings of the old one
    float sc_new;
    int up = 0;
    const bool finite = top < 0x7f800000u;
    if (!finite || !(was >= 0.f && was < __builtin_huge_valf())) {
      sc_new = __uint_as_float(0x7fffffffu);
    } else if (was >= 0x1p-100f) {
      const float fit = __fmul_rn(was, kTop);
      if (amax > fit) {
        const uint32_t f = __float_as_uint(fit);
        up = static_cast<int>(top >> 23) - static_cast<int>(f >> 23) + ((top & 0x7fffffu) > (f & 0x7fffffu) ? 1 : 0);
      }
      sc_new = ldexpf(was, up);
    } else {
      sc_new = amax < 0x1p-64f ? 0.f : __fmul_rn(amax, 1.f / kTop);
      up = held && sc_new > 0.f ? 127 : 0;  // rows held with no scale are zeros, and stay so
    }
    if (team.rank() == 0 && rows > 0 && QATTN_IN_BOUNDS(page >= 0 && page < a.n_pages)) scales[sc] = sc_new;
    uint8_t* P = pages + (sc << a.page_shift) * a.d;
    if (up > 0) {  // the rows that were there: their codes halved as often
      const float mul = up > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
      const int words = shift * a.d / 16;
#pragma unroll 4
      for (int w = team.rank(); w < words; w += team.size()) {
        if (!QATTN_IN_BOUNDS(16 * w < (a.d << a.page_shift))) continue;
        uint4 v = *reinterpret_cast<const uint4*>(P + 16 * w);
        v = make_uint4(divide4<E4M3>(v.x, mul), divide4<E4M3>(v.y, mul), divide4<E4M3>(v.z, mul),
                       divide4<E4M3>(v.w, mul));
        *reinterpret_cast<uint4*>(P + 16 * w) = v;
      }
    }
    const float inv = finite && sc_new > 0.f ? __fdiv_rn(1.f, sc_new) : 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if (!((ok >> k) & 1u)) continue;
      const Item<8> v = value(k);
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = __fmul_rn(v.v[e], inv);
      uint8_t* row = P + (shift + rw + per * k) * a.d;
      const bool some = inv > 0.f;  // (else codes of zero, beside NaN too)
      *reinterpret_cast<uint32_t*>(row + pl.c0) = some ? encode4<E4M3>(q[0], q[1], q[2], q[3]) : 0u;
      *reinterpret_cast<uint32_t*>(row + pl.c1) = some ? encode4<E4M3>(q[4], q[5], q[6], q[7]) : 0u;
    }
  }
}

// Q rotated: item i of token t in heads h0 .. h1 - 1.
template <int W>
__device__ __forceinline__ void append_q(const PagedAppendArgs& a, int b, const NewRows& s, int t, int i, int h0, int h1) {
  if (t >= s.n) return;
  const bool rotated = a.rope.table != nullptr;
  const Place<W> p = item_place<W>(i, rotated ? a.rope.rot : 0, a.rope.inter);
  Angles<W> ang{};
  if (rotated) {
    const int pos = position(a, b, s.first, t);
    if (pos < 0 || pos >= a.rope.n) {
      if (i == 0) atomicOr(a.err, kErrDomain);
      return;
    }
    if (p.turned) ang = load_angles<W>(a.rope, pos, i);
  }
  const uint16_t* X = a.q + b * a.qsB + t * a.qsN;
  uint16_t* Y = a.q_out + (static_cast<size_t>(b) * a.Hq * a.T + t) * a.d;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    if (!QATTN_IN_BOUNDS(b < a.B && t < a.T && h < a.Hq)) continue;
    Item<W> x = load_item<W>(X + h * a.qsH, p);
    if (p.turned) x = turn(x, ang, a.rope.inter);
    store_item(Y + static_cast<size_t>(h) * a.T * a.d, p, x);
  }
}

// Many tokens (y: page, z: sequence): x begins with CTAs that rotate Q, a part of a page's
// tokens and a head group each, the larger pieces (last: 1 to 2% slower); then a CTA a kind and
// KV head.  Four prompts of 1.4K to 4.1K tokens, 32 + 2 x 8 heads of 128 channels, 252 MB: 59 us,
// 4.3 TB/s (63%).  Q alone would take 34 us at the rate of the rotation; K and V, 67 MB, are
// bound by latency: a CTA's way from the lengths to the rows, the maximum over the page, the
// codes, with two CTAs an SM at 64 registers, 28 bytes of them spilled (three, at 40
// registers: 74 us).
constexpr int kPageItems = 4;  // items of a page that a thread holds
template <bool E4M3, int WQ>
__global__ void __launch_bounds__(512, 2) paged_append_kernel(const PagedAppendArgs a) {
  __shared__ uint32_t red[2][32];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.z;
  const NewRows s = new_rows(a, b, threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0);
  if (s.n == 0) return;
  const int q_ctas = gridDim.x - 2 * a.kv_groups;
  int g = static_cast<int>(blockIdx.x) - q_ctas;
  if (g >= 0) {
    const bool is_v = g >= a.kv_groups;
    if (is_v) g -= a.kv_groups;
    const int j = (s.first >> a.page_shift) + blockIdx.y;
    if ((j << a.page_shift) >= s.len) return;
    append_page<E4M3, kPageItems, true>(a, Team<true>{red}, b, s, j, is_v, g * a.heads, min(a.Hkv, (g + 1) * a.heads));
    return;
  }
  // Q: a part of a page's tokens (as many as the CTA has rows of items) and a head group
  g = blockIdx.x;
  constexpr int kParts = 8 * kPageItems / WQ;
  const int items = a.d / WQ, per = blockDim.x / items;
  const int part = g % kParts;
  g /= kParts;
  const int t = (blockIdx.y << a.page_shift) + part * per + threadIdx.x / items;
  append_q<WQ>(a, b, s, t, threadIdx.x % items, g * a.q_heads, min(a.Hq, (g + 1) * a.q_heads));
}

// A few tokens: a warp a page and head of K or V; then warps that rotate Q, a token and a
// head group each.  x: units of a sequence, 8 a CTA; y: sequence.  Bound by latency: 64
// sequences' next tokens (1.5 MB) take what a launch and four dependent loads take.
constexpr int kFewWarps = 8;
template <bool E4M3, int NP>
__global__ void __launch_bounds__(32 * kFewWarps) paged_append_few_kernel(const PagedAppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  int u = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  const NewRows s = new_rows(a, b, (threadIdx.x & 31) == 0 && u == 0);
  if (s.n == 0) return;
  const int kv = 2 * a.Hkv * a.touched;
  if (u < kv) {
    const int h = u % a.Hkv;
    u /= a.Hkv;
    const int j = (s.first >> a.page_shift) + (u >> 1);
    if ((j << a.page_shift) >= s.len) return;
    append_page<E4M3, NP, false>(a, Team<false>{}, b, s, j, u & 1, h, h + 1);
    return;
  }
  u -= kv;
  const int groups = (a.Hq + a.q_heads - 1) / a.q_heads;
  const int t = u / groups, g = u % groups;
  if (a.q == nullptr || t >= a.T) return;
  // 32 lanes: items of `per` heads at once
  const int items = a.d / 8, per = 32 / items, sub = (threadIdx.x & 31) / items;
  const int h0 = g * a.q_heads, h1 = min(a.Hq, h0 + a.q_heads), each = (h1 - h0 + per - 1) / per;
  append_q<8>(a, b, s, t, (threadIdx.x & 31) % items, min(h1, h0 + sub * each), min(h1, h0 + (sub + 1) * each));
}

}  // namespace

unsigned int check_take_paged_cache() { return check_take_local(); }

cudaError_t launch_rotate(RotateArgs a, cudaStream_t s) {
  const bool wide = !a.f32 && a.rope.rot % 16 == 0 && a.d % 16 == 0;
  const int per = kRotateThreads / (a.d / (wide ? 16 : 8));
  const long long tokens = static_cast<long long>(a.B) * a.T, blocks = (tokens + per - 1) / per;
  a.heads = kRotateHeads;
  const dim3 grid(static_cast<unsigned int>(blocks), static_cast<unsigned int>((a.H + a.heads - 1) / a.heads));
  if (a.f32) return launch_pdl(rotate_kernel<float, 8>, grid, dim3(kRotateThreads), 0, s, a);
  return wide ? launch_pdl(rotate_kernel<uint16_t, 16>, grid, dim3(kRotateThreads), 0, s, a)
              : launch_pdl(rotate_kernel<uint16_t, 8>, grid, dim3(kRotateThreads), 0, s, a);
}

namespace {
template <bool E4M3>
cudaError_t launch_append(PagedAppendArgs a, cudaStream_t s) {
  const int page = 1 << a.page_shift;
  a.touched = (a.T + page - 2) / page + 1;  // pages that a sequence's new rows touch, at most
  if (a.T <= kAppendFew) {
    a.q_heads = kFewQHeads;
    const long long units = 2LL * a.Hkv * a.touched + (a.q ? static_cast<long long>(a.T) * ((a.Hq + a.q_heads - 1) / a.q_heads) : 0);
    const dim3 grid(static_cast<unsigned int>((units + kFewWarps - 1) / kFewWarps), a.B);
    constexpr int kRows = 8;  // items a lane holds: 16 rows of 128 channels, 32 of 64
    static_assert(kAppendFew <= kRows * 2, "a warp holds a page's new rows");
    return launch_pdl(paged_append_few_kernel<E4M3, kRows>, grid, dim3(32 * kFewWarps), 0, s, a);
  }
  a.heads = kAppendHeads;
  a.q_heads = kAppendQHeads;
  a.kv_groups = (a.Hkv + a.heads - 1) / a.heads;
  const bool wide = a.rope.rot % 16 == 0;
  const int parts = 8 * kPageItems / (wide ? 16 : 8);
  const dim3 grid(2 * a.kv_groups + (a.q ? parts * ((a.Hq + a.q_heads - 1) / a.q_heads) : 0), a.touched, a.B);
  const dim3 block(page * (a.d / 8) / kPageItems);
  return wide ? launch_pdl(paged_append_kernel<E4M3, 16>, grid, block, 0, s, a)
                              : launch_pdl(paged_append_kernel<E4M3, 8>, grid, block, 0, s, a);
}
}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  return a.e4m3 ? launch_append<true>(a, s) : launch_append<false>(a, s);
}

}  // namespace qattn
