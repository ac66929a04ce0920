// Upkeep of the int8 KV cache in a serving loop: the accepted path of a drafted
// tree appended to it (qattn_tree_commit), and its rows of most weight gathered
// into a shorter cache (qattn_kv_evict).
#include "qattn_check.cuh"
#include "qattn_internal.h"
#include "sm103_ptx.cuh"

namespace qattn {
namespace {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A 32-bit word of another CTA's shared memory (the same offset as `p` here).
__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t addr, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

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
  bool bad = n < 0 || n > a.T || len < 0 || seen < 0 || len + static_cast<long long>(n) > a.cap;
  if (!bad)
    for (int t = threadIdx.x; t < n; t += kCommitThreads) bad |= path[t] < 0 || path[t] >= a.T;
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
// Selection: one cluster of 8 CTAs per (sequence, KV head); each holds the
// ordered keys of a contiguous slice of rows in shared memory (re-read from
// global memory where a slice does not fit).  Three histogram rounds (11, 11
// and 10 bits, the cluster's counts summed through distributed shared memory)
// give the budget-th largest key exactly; the rows above it and the first of
// its ties are kept, in row order, at positions from a prefix sum over the
// slices.  One read of the weights; bound by the rounds' barriers.
constexpr int kSelThreads = 512;
constexpr int kSelCluster = 8;
constexpr int kBins = 2048;
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

__global__ void __cluster_dims__(kSelCluster, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins];      // this CTA's counts of a round
  __shared__ uint32_t total[kBins];     // the cluster's
  __shared__ uint32_t wsum[2][kSelThreads / 32];
  __shared__ uint32_t pick[2];          // the round's bin, rows still wanted in it
  __shared__ uint32_t mine[2];          // this slice's rows above / at the threshold
  const int bkv = blockIdx.y, b = bkv / a.Hkv;
  const uint32_t rank = cluster_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int len = rows_in_use(a, b);
  const int want = min(len, a.budget);
  const int slice = (len + kSelCluster - 1) / kSelCluster;
  const int r0 = min(len, static_cast<int>(rank) * slice), r1 = min(len, r0 + slice);
  const int nr = r1 - r0;
  const float* w = a.weights + static_cast<size_t>(bkv) * a.cap;
  const bool fits = slice <= kSelRows;
  auto fresh = [&](int r) {
    return (r < a.n_sink || r >= len - a.n_recent) ? 0xffffffffu : weight_key(w[r]);
  };
  auto key = [&](int i) { return fits ? keys[i] : fresh(r0 + i); };
  if (fits)
    for (int i = threadIdx.x; i < nr; i += kSelThreads) keys[i] = fresh(r0 + i);
  if (rank == 0) {  // the header's maxima start from 0; the gather raises them
    for (int c = threadIdx.x; c < a.d; c += kSelThreads)
      a.v_code_amax[static_cast<size_t>(bkv) * a.d + c] = 0.f;
    if (threadIdx.x == 0 && bkv % a.Hkv == 0) a.lengths_out[b] = want;
  }
  if (want == 0) return;  // the whole cluster: no row in use

  uint32_t prefix = 0, left = want;  // the threshold's leading bits; rows wanted among its ties
  int shift = 32;
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int bits = round == 2 ? 10 : 11;
    const uint32_t high = shift == 32 ? 0u : (0xffffffffu << shift);
    shift -= bits;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < nr; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & high) == prefix) {
        const uint32_t bin = (k >> shift) & ((1u << bits) - 1u);
        // one addition for the lanes that agree with the first one (runs of
        // equal weights would otherwise queue up on one bin)
        const uint32_t act = __activemask();
        const uint32_t same = __ballot_sync(act, bin == __shfl_sync(act, bin, __ffs(act) - 1));
        if ((same >> lane) & 1u) {
          if (lane == __ffs(same) - 1) atomicAdd(&hist[bin], __popc(same));
        } else {
          atomicAdd(&hist[bin], 1u);
        }
      }
    }
    cluster_sync();
    for (int i = threadIdx.x; i < (1 << bits); i += kSelThreads) {
      uint32_t c = 0;
#pragma unroll
      for (int q = 0; q < kSelCluster; ++q) c += ld_cluster(&hist[i], q);
      total[i] = c;
    }
    __syncthreads();
    // the bin that holds the left-th largest: thread i owns bins from the top
    const int per = (1 << bits) / kSelThreads;
    uint32_t sum = 0;
    for (int e = 0; e < per; ++e) sum += total[(1 << bits) - 1 - (threadIdx.x * per + e)];
    uint32_t inc = sum;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, inc, sh);
      if (lane >= sh) inc += o;
    }
    if (lane == 31) wsum[0][warp] = inc;
    __syncthreads();
    uint32_t before = inc - sum;
    for (int q = 0; q < warp; ++q) before += wsum[0][q];
    if (before < left && before + sum >= left) {
      for (int e = 0; e < per; ++e) {
        const int bin = (1 << bits) - 1 - (threadIdx.x * per + e);
        if (before + total[bin] >= left) {
          pick[0] = bin;
          pick[1] = left - before;
          break;
        }
        before += total[bin];
      }
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    left = pick[1];
    cluster_sync();  // every CTA has read this round's counts
  }
  const uint32_t thr = prefix;  // keep keys above it, and the first `left` ties

  // each thread owns a run of consecutive rows (an odd length: no bank conflicts)
  const int run = ((nr + kSelThreads - 1) / kSelThreads) | 1;
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
  if (lane == 31) {
    wsum[0][warp] = ig;
    wsum[1][warp] = ie;
  }
  __syncthreads();
  uint32_t pg = ig - gt, pe = ie - eq, tg = 0, te = 0;
  for (int q = 0; q < kSelThreads / 32; ++q) {
    if (q < warp) {
      pg += wsum[0][q];
      pe += wsum[1][q];
    }
    tg += wsum[0][q];
    te += wsum[1][q];
  }
  if (threadIdx.x == 0) {
    mine[0] = tg;
    mine[1] = te;
  }
  cluster_sync();
  for (uint32_t q = 0; q < rank; ++q) {
    pg += ld_cluster(&mine[0], q);
    pe += ld_cluster(&mine[1], q);
  }
  int32_t* kept = a.kept + static_cast<size_t>(bkv) * a.budget;
  float* wo = a.weights_out + static_cast<size_t>(bkv) * a.out_cap;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > thr || (k == thr && pe < left)) {
      const uint32_t pos = pg + min(pe, left);
      if (QATTN_IN_BOUNDS(pos < static_cast<uint32_t>(want))) {
        kept[pos] = r0 + i;
        wo[pos] = w[r0 + i];
      }
    }
    pg += k > thr;
    pe += k == thr;
  }
  cluster_sync();  // no CTA leaves while another reads its counts
}

// Gather: a warp takes kRowsPerWarp kept rows, 16 bytes a lane, all loads of a
// batch before its stores; the V codes' channel maxima stay in registers and
// meet in one integer maximum per channel and CTA.
constexpr int kGatherWarps = 8;
constexpr int kRowsPerWarp = 16;

__device__ __forceinline__ uint32_t abs4_max(uint32_t m, uint32_t x) { return __vmaxu4(m, __vabs4(x)); }

template <int D>
__global__ void __launch_bounds__(32 * kGatherWarps) evict_gather_kernel(const EvictArgs a) {
  constexpr int LPR = D / 16;        // lanes per row
  constexpr int RPI = 32 / LPR;      // rows per warp load
  constexpr int NI = kRowsPerWarp / RPI;
  __shared__ uint4 red[kGatherWarps][32];
  const int bkv = blockIdx.y, b = bkv / a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, c = lane % LPR;
  pdl_trigger();
  pdl_wait();
  const int n = a.lengths_out[b];
  const int p0 = (blockIdx.x * kGatherWarps + warp) * kRowsPerWarp;
  if (blockIdx.x * kGatherWarps * kRowsPerWarp >= n) return;
  const int32_t* kept = a.kept + static_cast<size_t>(bkv) * a.budget;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_codes + static_cast<size_t>(bkv) * a.cap * D);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_codes + static_cast<size_t>(bkv) * a.cap * D);
  uint4* ko = reinterpret_cast<uint4*>(a.k_out + static_cast<size_t>(bkv) * a.out_cap * D);
  uint4* vo = reinterpret_cast<uint4*>(a.v_out + static_cast<size_t>(bkv) * a.out_cap * D);
  uint4 kx[NI], vx[NI];
  int row[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = p0 + RPI * i + sub;
    row[i] = p < n ? kept[p] : -1;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row[i] >= 0 && QATTN_IN_BOUNDS(row[i] < a.cap)) {
      kx[i] = ks[static_cast<size_t>(row[i]) * LPR + c];
      vx[i] = vs[static_cast<size_t>(row[i]) * LPR + c];
    }
  }
  uint4 m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = p0 + RPI * i + sub;
    if (p < n && QATTN_IN_BOUNDS(p < a.out_cap)) {
      ko[static_cast<size_t>(p) * LPR + c] = kx[i];
      vo[static_cast<size_t>(p) * LPR + c] = vx[i];
    }
    m.x = abs4_max(m.x, vx[i].x);
    m.y = abs4_max(m.y, vx[i].y);
    m.z = abs4_max(m.z, vx[i].z);
    m.w = abs4_max(m.w, vx[i].w);
  }
  red[warp][lane] = m;
  __syncthreads();
  // thread c < D: channel c's byte over the warps and row lanes
  if (threadIdx.x < D) {
    const int l0 = threadIdx.x / 16, word = (threadIdx.x / 4) % 4, byte = threadIdx.x % 4;
    uint32_t x = 0;
#pragma unroll
    for (int w = 0; w < kGatherWarps; ++w) {
#pragma unroll
      for (int q = 0; q < RPI; ++q) {
        const uint32_t v = reinterpret_cast<const uint32_t*>(&red[w][q * LPR + l0])[word];
        x = max(x, (v >> (8 * byte)) & 0xffu);
      }
    }
    // non-negative floats order like their bits
    atomicMax(reinterpret_cast<int*>(a.v_code_amax + static_cast<size_t>(bkv) * D + threadIdx.x),
              __float_as_int(static_cast<float>(x)));
  }
}

template <int D>
cudaError_t launch_gather(const EvictArgs& a, cudaStream_t s) {
  const int per = kGatherWarps * kRowsPerWarp;
  const int most = min(a.budget, a.Nk);
  if (most == 0) return cudaSuccess;
  return launch_pdl(evict_gather_kernel<D>, dim3((most + per - 1) / per, a.B * a.Hkv),
                    dim3(32 * kGatherWarps), 0, s, a);
}

}  // namespace

unsigned int check_take_kv_cache() { return check_take_local(); }

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t s) {
  const int nch = a.Hkv * a.d;
  const int ctas = min(kCommitCluster, (nch + kCommitThreads - 1) / kCommitThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, a.B);
  cfg.blockDim = dim3(kCommitThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_commit_kernel, a);
}

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s) {
  const int slice = (a.Nk + kSelCluster - 1) / kSelCluster;
  const int smem = 4 * min(slice, kSelRows);
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       4 * kSelRows);
  if (e != cudaSuccess) return e;
  e = launch_pdl(evict_select_kernel, dim3(kSelCluster, a.B * a.Hkv), dim3(kSelThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  return a.d == 32 ? launch_gather<32>(a, s) : a.d == 64 ? launch_gather<64>(a, s) : launch_gather<128>(a, s);
}

}  // namespace qattn
