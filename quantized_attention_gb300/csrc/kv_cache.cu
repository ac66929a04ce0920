// Upkeep of the int8 KV cache in a serving loop: the accepted path of a drafted
// tree appended to it (qattn_tree_commit), and its rows of most weight gathered
// into a shorter cache (qattn_kv_evict).
#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

// ------------------------------------------------------------------ commit
// One cluster per sequence, one thread per (KV head, channel): the accepted
// tokens pass in order, each quantized against the running mean of the tokens
// before it (the steps of qattn_kv_append, one IEEE operation each).  The chain
// mean -> difference -> quotient -> mean bounds it: ~60 cycles a token; the
// tokens' loads do not depend on it.  The new length is written after every CTA
// of the cluster has read the old one, so the two may be one array.
constexpr int kCommitThreads = 256;
constexpr int kCommitCluster = 8;

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitArgs a) {
  const int b = blockIdx.y;
  const int nch = a.Hkv * a.d;
  pdl_trigger();
  pdl_wait();
  const int len = a.lengths[b];
  const int seen = a.seen ? a.seen[b] : len;
  int n = a.n_accept[b];
  const int32_t* path = a.path + static_cast<size_t>(b) * a.T;
  bool bad = n < 0 || n > a.T || len < 0 || seen < 0 || seen > 0x7fffffff - max(n, 0) ||
             len + static_cast<long long>(n) > a.cap;
  if (!bad)
    for (int t = threadIdx.x; t < n; t += kCommitThreads)
      bad |= !QATTN_IN_BOUNDS(t < a.T) || path[t] < 0 || path[t] >= a.T;
  bad = __syncthreads_or(bad);
  if (bad) {  // nothing of this sequence is appended
    n = 0;
    if (threadIdx.x == 0) atomicOr(a.err, kErrDomain);
  }
  for (int x = blockIdx.x * kCommitThreads + threadIdx.x; x < nch; x += gridDim.x * kCommitThreads) {
    const int h = x / a.d, c = x % a.d;
    const size_t ch = static_cast<size_t>(b) * nch + x;
    float mu = a.k_mean[ch], am = a.v_code_amax[ch];
    const float sk = a.k_chan_scale[ch], sv = a.v_chan_scale[ch];
    const uint16_t* K = a.k_new + b * a.ksB + h * a.ksH + c;
    const uint16_t* V = a.v_new + b * a.vsB + h * a.vsH + c;
    const size_t row0 = (static_cast<size_t>(b) * a.Hkv + h) * a.cap + len;
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      if (!QATTN_IN_BOUNDS(t < a.T && path[t] >= 0 && path[t] < a.T)) continue;
      const long long j = path[t];
      const float k = bf16_bits_to_f32(K[j * a.ksN]), v = bf16_bits_to_f32(V[j * a.vsN]);
      const float diff = __fsub_rn(k, mu);
      const float qk = fminf(fmaxf(rintf(__fdiv_rn(diff, sk)), -127.f), 127.f);
      mu = __fadd_rn(mu, __fdiv_rn(diff, static_cast<float>(seen + t + 1)));
      const float qv = fminf(fmaxf(rintf(__fdiv_rn(v, sv)), -127.f), 127.f);
      am = fmaxf(am, fabsf(qv));
      if (QATTN_IN_BOUNDS(len + t < a.cap)) {
        a.k_codes[(row0 + t) * a.d + c] = static_cast<int8_t>(qk);
        a.v_codes[(row0 + t) * a.d + c] = static_cast<int8_t>(qv);
        if (a.weights && c == 0) a.weights[row0 + t] = 0.f;
      }
    }
    a.k_mean_out[ch] = mu;
    a.v_code_amax_out[ch] = am;
  }
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.lengths_out[b] = len + n;
    if (a.seen_out) a.seen_out[b] = seen + n;
  }
}

// ------------------------------------------------------------------ eviction
// One cluster per (sequence, KV head), of a size that fills the GPU.  Selection:
// each CTA holds the ordered keys of a contiguous slice of rows in shared memory
// (re-read from global memory where a slice does not fit); four rounds of 8-bit
// histograms, summed over the cluster through distributed shared memory, give the
// budget-th largest key exactly, and with it how many rows of the slices before this
// one lie above it or tie with it; the rows above it and the first of its ties are
// kept, in row order, at positions from a prefix sum.  (Three rounds of 11 bits read
// 64 KB of other CTAs' counts each: 22.9 us for 8 heads of 32K rows against 18.4.)  Then the
// cluster copies the kept rows, each CTA an equal share of the output, 16 bytes a
// thread, the V codes' channel maxima on the way.  The weights are read once, the
// kept rows read and written once; a short cache is bound by the rounds' barriers
// (~1 us each), a long one by the copy.  Measured: 128 heads of ~2K rows cut to 1999
// (d = 64) 17.7 us = 3.8 TB/s, 8 heads of 32K cut to 4K 16.2 us (64 CTAs; 17.3 with all
// weights equal); two kernels (select, gather) took 79 and 23, counting with one
// addition per distinct bin of a warp 18.5 and 17.5.
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kSelRows = 40960;  // rows of a slice kept in shared memory (160 KB)

// Order-preserving key of a weight: larger weight, larger key; NaN counts as
// -inf and -0 as 0.  Protected rows are above every weight.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -__builtin_huge_valf();
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int rows_in_use(const EvictArgs& a, int b) {
  if (!a.lengths) return a.Nk;
  const int n = a.lengths[b];
  if (n < 0 || n > a.Nk) {
    atomicOr(a.err, kErrDomain);
    return n < 0 ? 0 : a.Nk;
  }
  return n;
}

__device__ __forceinline__ uint32_t abs4_max(uint32_t m, uint32_t x) { return __vmaxu4(m, __vabs4(x)); }

template <int D>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictArgs a) {
  constexpr int LPR = D / 16;                  // threads per row of the copy
  constexpr int RPI = kEvictThreads / LPR;     // rows the CTA copies at once
  constexpr int U = 4;                         // of them in flight
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2][kBins];          // this CTA's counts of a round, alternating
  __shared__ uint32_t wsum[2][kEvictWarps];
  __shared__ uint32_t pick[2][4];              // a round's bin, the rows still wanted in it; of the
                                               // slices before: rows above the bin, rows in it
  __shared__ uint4 red[kEvictWarps][LPR];
  const int NC = a.cluster;
  const uint32_t rank = NC > 1 ? cluster_rank() : 0u;
  const int bkv = blockIdx.x / NC, b = bkv / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto sync = [&] {
    if (NC > 1) cluster_sync();
    else __syncthreads();
  };
  pdl_trigger();
  pdl_wait();
  const int len = rows_in_use(a, b);
  const int want = min(len, a.budget);
  const int slice = (len + NC - 1) / NC;
  const int r0 = min(len, static_cast<int>(rank) * slice), nr = min(len, r0 + slice) - r0;
  const float* w = a.weights + static_cast<size_t>(bkv) * a.cap;
  const bool fits = slice <= kSelRows;
  auto fresh = [&](int r) {
    if (r < a.n_sink || r >= len - a.n_recent || !QATTN_IN_BOUNDS(r < a.cap)) return 0xffffffffu;
    return weight_key(w[r]);
  };
  auto key = [&](int i) { return fits ? keys[i] : fresh(r0 + i); };
  if (fits)
    for (int i = threadIdx.x; i < nr; i += kEvictThreads) keys[i] = fresh(r0 + i);
  if (rank == 0) {  // the header's maxima start from 0; the copies raise them
    if (threadIdx.x < D) a.v_code_amax[static_cast<size_t>(bkv) * D + threadIdx.x] = 0.f;
    if (threadIdx.x == 0 && bkv % a.Hkv == 0) a.lengths_out[b] = want;
  }
  if (want == 0) return;  // the whole cluster: no row in use
  if (threadIdx.x < kBins) hist[0][threadIdx.x] = 0u;
  __syncthreads();

  uint32_t prefix = 0, left = want;  // the threshold's leading bits; rows wanted among its ties
  const bool all = want == len;      // nothing to choose: every row is above the threshold
  uint32_t gt0 = all ? r0 : 0, eq0 = 0;  // rows of the slices before above / at the threshold
#pragma unroll 1
  for (int round = 0; round < 4 && !all; ++round) {
    const int shift = 24 - 8 * round;
    const uint32_t high = round == 0 ? 0u : (0xffffffffu << (shift + 8));
    uint32_t* h = hist[round & 1];
    for (int i = threadIdx.x; i < nr; i += kEvictThreads) {
      const uint32_t k = key(i);
      if ((k & high) == prefix) atomicAdd(&h[(k >> shift) & 255u], 1u);
    }
    sync();  // the cluster's counts are in
    // thread i < 256: bin 255 - i, counted from the top: c, and p in the slices before
    uint32_t c = 0, p = 0;
    if (threadIdx.x < kBins) {
      hist[(round + 1) & 1][threadIdx.x] = 0u;  // last read a round ago, behind a barrier
      const uint32_t addr = smem_u32(&h[kBins - 1 - threadIdx.x]);
      if (NC == 1) {
        c = h[kBins - 1 - threadIdx.x];
      } else {
#pragma unroll 8
        for (uint32_t q = 0; q < static_cast<uint32_t>(NC); ++q) {
          const uint32_t x = ld_cluster_u32(cluster_addr(addr, q));
          c += x;
          p += q < rank ? x : 0u;
        }
      }
    }
    uint32_t inc = c, pinc = p;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, inc, sh), po = __shfl_up_sync(0xffffffffu, pinc, sh);
      if (lane >= sh) {
        inc += o;
        pinc += po;
      }
    }
    if (lane == 31) {
      wsum[0][warp] = inc;
      wsum[1][warp] = pinc;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      uint32_t before = inc - c, pbefore = pinc - p;
      for (int q = 0; q < warp; ++q) {
        before += wsum[0][q];
        pbefore += wsum[1][q];
      }
      if (before < left && before + c >= left) {
        pick[round & 1][0] = kBins - 1 - threadIdx.x;
        pick[round & 1][1] = left - before;
        pick[round & 1][2] = pbefore;
        pick[round & 1][3] = p;
      }
    }
    __syncthreads();
    prefix |= pick[round & 1][0] << shift;
    left = pick[round & 1][1];
    gt0 += pick[round & 1][2];
    eq0 = pick[round & 1][3];
  }
  // keep keys above the threshold, and the first `left` of its ties
  const uint32_t thr = all ? 0u : prefix;  // (no key is 0: the lowest is that of -inf)
  if (all) left = 0;  // (eq0 is 0)

  // each thread owns a run of consecutive rows (an odd length: no bank conflicts)
  const int run = ((nr + kEvictThreads - 1) / kEvictThreads) | 1;
  const int i0 = min(nr, static_cast<int>(threadIdx.x) * run), i1 = min(nr, i0 + run);
  uint32_t gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    gt += k > thr;
    eq += k == thr;
  }
  uint32_t ig = gt, ie = eq;
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const uint32_t og = __shfl_up_sync(0xffffffffu, ig, sh), oe = __shfl_up_sync(0xffffffffu, ie, sh);
    if (lane >= sh) {
      ig += og;
      ie += oe;
    }
  }
  __syncthreads();  // wsum's last readers are done
  if (lane == 31) {
    wsum[0][warp] = ig;
    wsum[1][warp] = ie;
  }
  __syncthreads();
  // the warps' sums: one a lane, exclusive prefixes by shuffles
  uint32_t vg = wsum[0][lane], ve = wsum[1][lane], sg = vg, se = ve;
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const uint32_t og = __shfl_up_sync(0xffffffffu, sg, sh), oe = __shfl_up_sync(0xffffffffu, se, sh);
    if (lane >= sh) {
      sg += og;
      se += oe;
    }
  }
  uint32_t pg = gt0 + __shfl_sync(0xffffffffu, sg - vg, warp) + ig - gt;
  uint32_t pe = eq0 + __shfl_sync(0xffffffffu, se - ve, warp) + ie - eq;
  int32_t* kept = a.kept + static_cast<size_t>(bkv) * a.budget;
  float* wo = a.weights_out + static_cast<size_t>(bkv) * a.out_cap;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > thr || (k == thr && pe < left)) {
      const uint32_t pos = pg + min(pe, left);
      if (QATTN_IN_BOUNDS(pos < static_cast<uint32_t>(want) && r0 + i < a.cap)) {
        kept[pos] = r0 + i;
        wo[pos] = w[r0 + i];
      }
    }
    pg += k > thr;
    pe += k == thr;
  }
  sync();  // the list is complete, and no CTA reads another's counts any more

  // ---- copy this CTA's share of the kept rows
  const int p0 = static_cast<int>(static_cast<long long>(want) * rank / NC);
  const int p1 = static_cast<int>(static_cast<long long>(want) * (rank + 1) / NC);
  const int c = threadIdx.x % LPR;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_codes + static_cast<size_t>(bkv) * a.cap * D) + c;
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_codes + static_cast<size_t>(bkv) * a.cap * D) + c;
  uint4* ko = reinterpret_cast<uint4*>(a.k_out + static_cast<size_t>(bkv) * a.out_cap * D) + c;
  uint4* vo = reinterpret_cast<uint4*>(a.v_out + static_cast<size_t>(bkv) * a.out_cap * D) + c;
  uint4 m = make_uint4(0u, 0u, 0u, 0u);
  for (int p = p0 + threadIdx.x / LPR; p < p1; p += U * RPI) {
    int row[U];
    uint4 kx[U], vx[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      row[i] = p + i * RPI < p1 && QATTN_IN_BOUNDS(p + i * RPI < a.budget) ? kept[p + i * RPI] : -1;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row[i] >= 0 && QATTN_IN_BOUNDS(row[i] < a.cap)) {
        kx[i] = ks[static_cast<size_t>(row[i]) * LPR];
        vx[i] = vs[static_cast<size_t>(row[i]) * LPR];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (row[i] >= 0 && QATTN_IN_BOUNDS(p + i * RPI < a.out_cap)) {
        ko[static_cast<size_t>(p + i * RPI) * LPR] = kx[i];
        vo[static_cast<size_t>(p + i * RPI) * LPR] = vx[i];
      }
      m.x = abs4_max(m.x, vx[i].x);
      m.y = abs4_max(m.y, vx[i].y);
      m.z = abs4_max(m.z, vx[i].z);
      m.w = abs4_max(m.w, vx[i].w);
    }
  }
  // ---- the channel maxima: lanes of a column, warps, then the cluster's CTAs
#pragma unroll
  for (int sh = LPR; sh < 32; sh <<= 1) {
    m.x = __vmaxu4(m.x, __shfl_xor_sync(0xffffffffu, m.x, sh));
    m.y = __vmaxu4(m.y, __shfl_xor_sync(0xffffffffu, m.y, sh));
    m.z = __vmaxu4(m.z, __shfl_xor_sync(0xffffffffu, m.z, sh));
    m.w = __vmaxu4(m.w, __shfl_xor_sync(0xffffffffu, m.w, sh));
  }
  if (lane < LPR) red[warp][lane] = m;
  __syncthreads();
  if (threadIdx.x < D) {
    const int col = threadIdx.x / 16, word = (threadIdx.x / 4) % 4, byte = threadIdx.x % 4;
    uint32_t x = 0;
#pragma unroll
    for (int q = 0; q < kEvictWarps; ++q)
      x = max(x, (reinterpret_cast<const uint32_t*>(&red[q][col])[word] >> (8 * byte)) & 0xffu);
    // non-negative floats order like their bits
    atomicMax(reinterpret_cast<int*>(a.v_code_amax + static_cast<size_t>(bkv) * D + threadIdx.x),
              __float_as_int(static_cast<float>(x)));
  }
}

template <int D>
cudaError_t launch_evict_d(EvictArgs a, cudaStream_t s) {
  // CTAs per head: as many as fill the SMs, and enough that a slice fits.  (Clusters
  // of 16 took 36.6 us where 8 take 18.4, 8 heads of 32K rows: the chip places fewer
  // than eight of them at once.)
  const long long heads = static_cast<long long>(a.B) * a.Hkv;
  const int sms = num_sms();
  a.cluster = 1;
  while (a.cluster < kMaxCluster && (2 * a.cluster * heads <= sms || a.Nk > static_cast<long long>(a.cluster) * kSelRows))
    a.cluster *= 2;
  const int slice = (a.Nk + a.cluster - 1) / a.cluster;
  const int smem = 4 * min(slice, kSelRows);
  cudaError_t e = cudaFuncSetAttribute(evict_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kSelRows);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned int>(heads * a.cluster));
  if (a.cluster == 1) return launch_pdl(evict_kernel<D>, grid, dim3(kEvictThreads), smem, s, a);
  return launch_pdl_cluster(evict_kernel<D>, grid, dim3(kEvictThreads), a.cluster, smem, s, a);
}

}  // namespace

unsigned int check_take_kv_cache() { return check_take_local(); }

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t s) {
  const int nch = a.Hkv * a.d;
  const int ctas = min(kCommitCluster, (nch + kCommitThreads - 1) / kCommitThreads);
  return launch_pdl_cluster(tree_commit_kernel, dim3(ctas, a.B), dim3(kCommitThreads), ctas, 0, s, a);
}

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s) {
  return a.d == 32 ? launch_evict_d<32>(a, s) : a.d == 64 ? launch_evict_d<64>(a, s) : launch_evict_d<128>(a, s);
}

}  // namespace qattn
