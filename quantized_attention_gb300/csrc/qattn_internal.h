// Internal launch interface between the C ABI (qattn_api.cu) and the
// kernels (quant_kernels.cu, attn_fwd.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace qattn {

// Launches `kernel` on stream s with programmatic stream serialization, so it
// may start while the previous kernel of the stream finishes (the kernels call
// pdl_wait before touching their inputs).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// The same with clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, int cluster,
                                      size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned int>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Streaming multiprocessors of the current device (1 if the query fails).
inline int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  return n;
}

// Unique id (cuCtxGetId) of the CUDA context current on the calling thread;
// false when no context is current or the driver cannot say.  The library
// caches device addresses of its own __device__ symbols per device and per
// context, so that a context destroyed by cudaDeviceReset (and replaced by a
// new one) never leaves a stale address behind.
bool current_context_id(unsigned long long* id);

// Bits of the device error word.
constexpr unsigned int kErrTimeout = 1u;
constexpr unsigned int kErrDomain = 2u;  // device-held scales outside a kernel's domain

// The checked build's bounds-check words, one per kernel translation unit
// (qattn_check.cuh): each call reads and clears its unit's word (always 0 in
// the normal build).
unsigned int check_take_attn_fwd();
unsigned int check_take_quant();
unsigned int check_take_decode();
unsigned int check_take_short();
unsigned int check_take_exact24();
unsigned int check_take_intsm();
unsigned int check_take_tree_warp();
unsigned int check_take_tree_tc();
unsigned int check_take_kv_weights();
unsigned int check_take_kv_weights_tc();
unsigned int check_take_kv_cache();
// One guard that fails for 16 of 32 threads, touching no memory (quant_kernels.cu).
cudaError_t launch_bounds_probe(cudaStream_t s);

struct AttnArgs {
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;
  int pos0;  // key position of query row 0 (causal only)
  float sm_scale;
  int q_gran, k_gran;
  const float* q_scales;
  const float* k_scales;
  const float* v_scales;
  const float* bias;
  long long bias_head_stride;
  int pv_int8;  // P quantized as int8 rint(127 P) (ablation) instead of e4m3(448 P)
  void* out;
  int out_bf16;
  float* lse;
  unsigned int* err;
};

// ---- attn_short.cu: the recipe on the warp-level tensor cores for short
// non-causal key sequences (d in {32, 64}, Nk <= kShortMaxNk)
constexpr int kShortMaxNk = 256;
constexpr int kWindowMax = 64;  // Nq, Nk of the window kernel
bool attn_short_eligible(const AttnArgs& a);
cudaError_t launch_attn_short(const AttnArgs& a, const int8_t* q_codes, const int8_t* k_codes,
                              const uint8_t* v8t, long long ldv, cudaStream_t s);

// ---- quant_kernels.cu
// An input tensor [B][H][N][d] (bf16 or int8) at any strides, in elements: row
// t of (batch, head) bh = b H + h starts at p + b sB + h sH + t sN and its d
// elements are contiguous.  Dense: sB = H N d, sH = N d, sN = d.
struct Src {
  const void* p;
  long long sB, sH, sN;
  int H;
};
inline Src dense_src(const void* p, int H, long long N, int d) {
  return Src{p, static_cast<long long>(H) * N * d, N * d, static_cast<long long>(d), H};
}

cudaError_t launch_smooth_k(const Src& K, int BH, int Nk, int d, long long* ws, float* mu,
                            cudaStream_t s);
size_t smooth_k_ws_bytes(long long BH, long long Nk, long long d);

// One tensor to quantize per 128-token block rows (a2): X [B*H][N][d] bf16.
//   mode 0: x = X;  1: x = X - chan[b][h][:] (Hchan = H);
//   2: x = X * chan[b][h / group][:] (chan has Hchan heads, group = H / Hchan)
struct RowsJob {
  const uint16_t* X;
  long long sB, sH, sN;  // X's strides in elements (see Src)
  int H, N;
  const float* chan;
  int Hchan, group, gran;
  int8_t* codes;
  float* scales;
  float* ws_amax;  // B*H*nblk block maxima (tensor / head granules only)
  uint16_t* carrier;  // nullable: the codes again as exact fp16, same layout
  int nblk, BH;    // 128-token blocks per head; B*H (0: no job)
  float* ones;     // nullable (job 0 only): n_ones floats set to 1 by the
  long long n_ones;  // launch (the K scales of an int8 cache)
};
// Quantizes j0 (mode m0) and j1 (mode m1) in the same launches.  Supported:
// (m0, m1) = (0, 0), (0, 1), or (2, -) with j1.BH = 0.
cudaError_t launch_quantize_rows(const RowsJob& j0, int m0, const RowsJob& j1, int m1, int d,
                                 cudaStream_t s);
size_t quantize_rows_ws_bytes(long long B, long long H, long long N, int gran);
// The pre-pass for bf16 Q, K, V with block granules: jq (Q, mode 0), jk (K
// minus jk.chan = the mean it writes, mode 1), V's e4m3 transpose.  One launch
// for heads of at most 128 tokens and d <= 64, else two (ws zeroed here).
// ws: prepare_ws_bytes().
cudaError_t launch_prepare(const RowsJob& jq, const RowsJob& jk, const Src& V, int d,
                           uint8_t* v8t, long long ldv, float* v_scales, void* ws, cudaStream_t s);
size_t prepare_ws_bytes(long long BH, long long d);
int prepare_launch_count(int d, int Nq, int Nk);  // 1 for short heads, else 2
// The same pre-pass with tensor granules (jq.gran = jk.gran = 0): two launches,
// one warp per head, for d in {32, 64} and 1 <= Nk <= 256.  ws: 8 bytes (the
// two maxima, zeroed here).
bool prepare_tensor_eligible(int d, int Nq, int Nk);
cudaError_t launch_prepare_tensor(const RowsJob& jq, const RowsJob& jk, const Src& V, int d,
                                  uint8_t* v8t, long long ldv, float* v_scales, void* ws,
                                  cudaStream_t s);

cudaError_t launch_quantize_v(const Src& V, int is_i8, const float* chan, int BH, int Nk, int d,
                              uint8_t* v8t, long long ldv, float* v_scales, unsigned int* ws_amax,
                              cudaStream_t s);

cudaError_t launch_codes_to_f16(const int8_t* src, uint16_t* dst, size_t n, cudaStream_t s);

// max |code| per channel of int8 V codes [BH][rows][d], rows 0 .. Nk-1
// (out: [BH][d] fp32, zeroed first)
cudaError_t launch_v_code_amax(const int8_t* v_codes, int BH, int Nk, long long rows, int d,
                               float* out, cudaStream_t s);

// Rows that see no key (Nk = 0): out = 0 (out_bytes of it), lse = -inf for
// `rows` rows when lse is not null.
cudaError_t launch_no_key_rows(void* out, size_t out_bytes, float* lse, size_t rows, cudaStream_t s);

// ---- decode.cu
constexpr int kMaxDecodeRows = 16;  // (Hq / Hkv) * Nq rows per KV head

struct DecodeArgs {
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;
  int pos0;
  float sm_scale;
  int q_gran, k_gran;
  const int8_t* q_codes;
  const float* q_scales;
  const int8_t* k_codes;
  const float* k_scales;
  const int8_t* v_codes;       // [B*Hkv][Nk][d], row-major as cached
  const float* v_chan_scale;   // [B*Hkv][d]
  const float* v_code_amax;    // [B*Hkv][d]: max |code| per channel
  void* out;
  int out_bf16;
  float* lse;
  // set by launch_decode: the split and the workspace regions
  int bpc;                        // key blocks per chunk
  int nch;                        // chunks per (batch, KV head)
  unsigned long long epoch;       // this call's tag (low 32 bits), unique per call
  unsigned long long* ctr;        // unit counter: (tag << 32) | units taken
  float* part_o;                  // [B*Hkv][nch][R][d]  chunk shares of O
  float* part_l;                  // [B*Hkv][nch][R]     their l
  float* part_m;                  // [B*Hkv][nch][R]     their running max
  unsigned long long* rec;        // [B*Hkv][nch][R]     chunk maxima: (tag << 32) | bits
  unsigned int* err;  // device error word (a bounded wait that ran out)
};
size_t decode_ws_bytes(long long B, long long Hq, long long Hkv, long long Nq, long long Nk,
                       long long d);
// tk, tv: maps over the int8 K and V codes [B*Hkv][Nk][d], box d x 128 x 1,
// 128-byte swizzle for d = 128, 64-byte for d = 64.
cudaError_t launch_decode(const CUtensorMap& tk, const CUtensorMap& tv, DecodeArgs a, void* ws,
                          cudaStream_t s);
cudaError_t launch_kv_append(const uint16_t* K_new, const uint16_t* V_new, int BH, int d, int T,
                             int pos, long long cap, const float* k_chan_scale,
                             const float* v_chan_scale, float* k_mean, float* v_code_amax,
                             int8_t* k_codes, int8_t* v_codes, cudaStream_t s);

// ---- tree_warp.cu, tree_tc.cu (tree_common.cuh): qattn_tree_decode
constexpr int kTreeMaxTokens = 128;  // drafted tokens of a sequence
// Query rows of the warp-level kernel's block, and the most of a KV head that it takes:
// beyond them the tensor-core kernel runs, which reads the cache once for up to 128.
// Measured, warp-level against tensor cores, us (d = 128, four query heads a KV head; 8
// heads of 4K, 8 of 32K, 128 of 0.1 to 4K, 64 of 5K to 32K rows): 16 rows 10.0 / 13.4,
// 23.0 / 27.4, 27.9 / 43.7, 61 / 90; 20 rows 11.6 / 13.5, 30.1 / 27.8, 36.2 / 44.0, 110 /
// 90; 32 rows 11.8 / 13.6, 30.7 / 27.8, 38.3 / 44.3, 108 / 90; 64 rows 12.5 / 14.7, 47.8 /
// 28.7, 63.6 / 46.4, 195 / 92.
constexpr int kTreeRows = 16;
constexpr int kTreeWarpCtas = 304;   // its CTAs, at most (152 SMs, two each; the workspace's size
                                     // is asked for without a device, so not num_sms())
constexpr int kTreeTcRows = 128;     // query rows of the tensor-core kernel's block
constexpr int kTreeTcCtas = 152;     // its CTAs, at most
constexpr int kTreeWarpStep = 32, kTreeTcStep = 128;  // keys of a step
// Steps that a head's start counts for in equal shares (the last head's share joined
// and written, the drafts' codes, the pipeline filled again) and, its drafts alone, in
// a cluster.  Shares without and with it: 39.4 and 27.8 us (16 sequences of 0.2 to
// 4.5K rows, four drafts), 114 and 104 (eight of 5K to 32K, 26).
constexpr int kTreeWarpLead = 18, kTreeTcLead = 6;
constexpr int kTreeWarpDraftLead = 5, kTreeTcDraftLead = 3;
constexpr int kTreeCluster = 8;      // most CTAs of a head's own cluster
// CTAs of the cluster a head gets to itself in the warp-level kernel: as many (a
// power of two) as are placed at once, two CTAs an SM (38 clusters of 8 are not: 25
// us against 18 in shares).  0 -- equal shares of all heads' steps, joined by a
// second kernel, 2.5 us more of host time -- once the busiest CTA would take 10 steps
// more than its share (the few-head cases that this would take at 4K gain nothing).
// Measured, clusters against shares, us (d = 128): 8 heads of 2K / 8K / 32K rows 8.0 /
// 15.2 / 36.4 against 10.1 / 14.1 / 22.7; 16 of 4K / 8K / 16K 12.8 / 18.0 / 28.2 against
// 14.0 / 18.0 / 22.3; 32 of 8K / 16K 20.9 / 30.9 against 21.9 / 31.7; 64 of 4K 20.8 / 22.3,
// of 5K to 32K 71.7 / 59.4; 128 of 2K 21.2 / 26.1, of 100 to 4K 27.9 / 25.7, to 8K 47.5 /
// 36.5; 256 of 300 / 2K 15.1 / 32.9 against 21.5 / 39.6.  The same rule serves d = 64: 8 of
// 2K / 8K / 32K 6.6 / 10.9 / 27.9 against 8.7 / 11.2 / 17.5; 32 of 4K / 16K 11.4 / 24.9
// against 13.0 / 21.9; 64 of 5K to 32K 63.5 / 40.0; 128 of 2K 16.8 / 17.4, of 100 to 4K 21.9 /
// 18.1 (taken as clusters); 256 of 300 / 2K 10.1 / 26.3 against 12.2 / 25.2.
inline int tree_cluster(long long heads, long long steps) {
  const int c = heads <= 32 ? kTreeCluster : heads <= kTreeWarpCtas / 4 ? 4 : heads <= kTreeWarpCtas / 2 ? 2 : 1;
  const long long waves = (heads * c + kTreeWarpCtas - 1) / kTreeWarpCtas;
  const long long extra = steps * (waves * kTreeWarpCtas - heads * c) / (c * kTreeWarpCtas);
  return extra <= 10 + (heads < 8 ? 10 : 80 / heads) ? c : 0;
}
// The same for the tensor-core kernel (heads: KV heads x row blocks; one CTA an SM).
// The chip places 32 clusters of 4 at once and 8 of 8, not as many as its SMs would
// hold (38 in fours: 44 us against 29 in shares).  Equal shares cost a plan, a join
// and kTreeTcLead steps (of 1.2 us) a head: they pay once the busiest CTA of a
// cluster would take so many steps more than its share (few for up to 12 heads, whose
// rows four warps join).  Measured, clusters against shares, us (d = 128): one head of
// 2K / 8K / 32K rows 14.7 / 19.3 / 44.9 against 11.3 / 12.6 / 22.5; 4 of 8K 19.8 / 17.1; 8
// of 2K / 8K / 32K 15.5 / 20.9 / 46.5 against 14.6 / 18.7 / 29.9; 16 of 4K / 8K / 16K 19.3 /
// 27.9 / 45.0 against 20.3 / 24.0 / 30.9; 32 of 4K / 8K / 16K 20.3 / 28.8 / 46.9 against
// 24.1 / 31.0 / 44.6; 64 of 4K 30.5 / 35.6, of 5K to 32K 119 / 89; 128 of 2K 33.8 / 44.7, of
// 100 to 4K 48.6 / 51.5, to 8K 81.8 / 68.0; 256 of 2K 66.0 / 74.3.  At d = 64: 8 of 2K / 8K /
// 32K 12.1 / 16.4 / 39.6 against 11.8 / 14.3 / 24.5; 32 of 4K / 16K 16.5 / 39.1 against 20.1 /
// 38.3; 64 of 4K 25.1 / 27.3, of 5K to 32K 129 / 78; 128 of 2K 27.5 / 31.7, of 100 to 4K
// 41.7 / 33.9 (taken as clusters); 256 of 300 / 2K 29.7 / 53.8 against 31.7 / 54.1.
inline int tree_tc_cluster(long long heads, long long steps) {
  const int c = heads <= 8 ? kTreeCluster : heads <= 32 ? 4 : heads <= kTreeTcCtas / 2 ? 2 : 1;
  const long long waves = (heads * c + kTreeTcCtas - 1) / kTreeTcCtas;
  const long long extra = steps * (waves * kTreeTcCtas - heads * c) / (c * kTreeTcCtas);
  const long long most = heads <= 12 ? 1 : heads < 25 ? 4 : 3 + heads / 25;
  return extra <= most ? c : 0;
}
struct TreeArgs {
  int B, Hq, Hkv, G, T, Nk, d;   // G = Hq / Hkv; Nk: most rows in use
  int blocks;                    // row blocks of a head
  int drafts;                    // drafted steps of a head (0: no drafts)
  int draft_causal;              // no mask given: draft j visible to token i iff j <= i (else all)
  int cached_causal;             // no drafts: cached row k visible to token i iff k <= len - T + i
  int q_gran;                    // GRAN_TENSOR, else one scale per (sequence, query head)
  float sm_scale;
  const int8_t* q_codes;         // [B][Hq][T][d]
  const float* q_scales;
  const float* k_chan_scale;     // [B][Hkv][d]
  const float* v_chan_scale;     // [B][Hkv][d]
  const float* k_mean;           // [B][Hkv][d]
  const int32_t* lengths;        // [B] or null (all Nk)
  const uint16_t* k_new;         // bf16 drafts, element strides
  const uint16_t* v_new;
  long long ksB, ksH, ksN, vsB, vsH, vsN;
  const uint32_t* tree_mask;     // [B][T][ceil(T/32)] or null
  void* out;                     // [B][Hq][T][d]
  int out_bf16;
  float* lse;                    // [B][Hq][T] or null
  unsigned int* err;
  // the split and its workspace
  int cluster;                   // CTAs of the cluster that has a head to itself: no join, no
                                 // workspace (0: shares of all heads' steps, then the join)
  int ctas;
  int lead;                      // steps that a head's start counts for in the division
  size_t slots, rows_total;      // 2 ctas; B Hq T
  float* part_o;                 // [slots][block rows][d]
  float* part_m;                 // [slots][block rows]
  float* part_l;
};
// tk, tv: maps over the int8 K and V codes, box d x (keys of a step) x 1
// (128-byte swizzle for d = 128, 64-byte for d = 64).
cudaError_t launch_tree_warp(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                             cudaStream_t s);
cudaError_t launch_tree_tc(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a,
                           cudaStream_t s);

// ---- kv_weights.cu
struct WeightArgs {
  int B, Hq, Hkv, G, Nq, Nk, d;
  long long cap;             // cache rows per (sequence, KV head)
  int causal;
  int pos0_len;              // 1: query row 0 sits on row length - Nq; 0: on pos0
  int pos0;
  float sm_scale;
  int q_gran, k_gran;
  const int8_t* q_codes;     // [B][Hq][Nq][d]
  const float* q_scales;
  const int8_t* k_codes;     // [B][Hkv][cap][d]
  const float* k_scales;     // null: 1
  const float* lse;          // [B][Hq][Nq]
  const int32_t* lengths;    // [B] or null
  const float* base;         // [B][Hkv][cap] or null
  float* weights;            // [B][Hkv][cap]
  unsigned int* err;
};
// A query row's factor sq sm log2 e; 0 for a query that gives nothing (lse = -inf) if
// its scale is not finite: 0 S - inf is -inf, where NaN would hide every other query.
__device__ __forceinline__ float weight_factor(float sq, float sm_scale, float lse) {
  const float c = __fmul_rn(__fmul_rn(sq, sm_scale), 1.44269502162933349609375f);  // fp32(log2 e)
  return fabsf(c) < __builtin_huge_valf() || lse != -__builtin_huge_valf() ? c : 0.f;
}
// Query rows (query heads of the group x tokens) up to which the warp-level kernel
// runs; above, the tensor-core one, which works in tiles of 128.  Measured on 8
// heads of 32K rows, warp-level against tensor cores, us: 16 rows 13.8 / 22.8, 32
// rows 16.3 / 22.9, 64 rows 21.8 / 22.9, and the latter still 23 at 128.
constexpr int kWeightWarpRows = 64;
cudaError_t launch_kv_weights_warp(const WeightArgs& a, cudaStream_t s);
// ---- kv_weights_tc.cu.  tk: map over the K codes, box d x 128 x 1.
cudaError_t launch_kv_weights_tc(const CUtensorMap& tk, const WeightArgs& a, cudaStream_t s);

// ---- kv_cache.cu
struct CommitArgs {
  int B, Hkv, T, d;
  long long cap;
  const uint16_t *k_new, *v_new;
  long long ksB, ksH, ksN, vsB, vsH, vsN;
  const int32_t *path, *n_accept;      // [B][T], [B]
  const float *k_chan_scale, *v_chan_scale;
  const int32_t *lengths, *seen;       // seen null: lengths
  const float *k_mean, *v_code_amax;
  int32_t *lengths_out, *seen_out;
  float *k_mean_out, *v_code_amax_out;
  float* weights;                      // null, or [B][Hkv][cap]: new rows zeroed
  int8_t *k_codes, *v_codes;
  unsigned int* err;
};
cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t s);

struct EvictArgs {
  int B, Hkv, Nk, d;
  long long cap, out_cap;
  int budget, n_sink, n_recent;
  const int8_t *k_codes, *v_codes;
  const float* weights;
  const int32_t* lengths;
  int8_t *k_out, *v_out;
  float* weights_out;
  int32_t* kept;        // [B][Hkv][budget]
  int32_t* lengths_out;
  float* v_code_amax;
  unsigned int* err;
  int cluster;          // CTAs per (sequence, KV head); set by launch_kv_evict
};
cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t s);

// ---- exact24.cu
struct Exact24Args {
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;
  int pos0;
  float sm_scale;
  long long cap;                // cache rows per (batch, KV head)
  const void* Q;                // bf16 [B][Hq][Nq][d]
  const float* k_chan_scale;    // [B][Hkv][d]
  const int8_t* k_codes;        // [B][Hkv][cap][d]
  const int8_t* v_codes;
  const float* v_chan_scale;
  void* out;
  int out_bf16;
  float* lse;
  void* ws;                     // exact24_ws_bytes
  unsigned int* err;            // device error word (a bounded wait that ran out)
};
size_t exact24_ws_bytes(long long B, long long Hq, long long Hkv, long long Nq, long long Nk,
                        long long d);
cudaError_t launch_exact24(const Exact24Args& x, cudaStream_t s);

// ---- intsm.cu
cudaError_t launch_intsoftmax(int B, int Hq, int Hkv, int Nq, int Nk, int d, float sm_scale,
                              const int8_t* q_codes, const float* q_scale, const int8_t* k_codes,
                              const float* k_scale, const int8_t* v_codes, int8_t* out,
                              unsigned int* err, cudaStream_t s);

// 3-D tiled TMA map over a dense [planes][rows][inner] tensor (qattn_api.cu):
// row_stride_bytes between rows, plane_rows rows between planes (0 = rows);
// false if the driver entry point is missing or rejects the map.
bool encode_tiled_3d(CUtensorMap* map, CUtensorMapDataType dt, const void* ptr, uint64_t inner,
                     uint64_t rows, uint64_t planes, uint64_t row_stride_bytes, uint32_t box_inner,
                     uint32_t box_rows, CUtensorMapSwizzle swz, uint64_t plane_rows = 0);

// ---- attn_fwd.cu
// tq: int8 Q codes; tk: fp16 K carriers; tv: e4m3 V^T; to: the output
// [B*Hq][Nq][d] (bf16 or fp32) in boxes of 128-byte rows x 32 rows, 128B
// swizzle (unused, and may be left zero, for bf16 with d = 32).
cudaError_t launch_attn_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                            const CUtensorMap& to, const AttnArgs& a, cudaStream_t s);
cudaError_t launch_qk_debug(const CUtensorMap& tq, const CUtensorMap& tk, int B, int Hq, int Hkv,
                            int Nq, int Nk, int d, int32_t* S, unsigned int* err,
                            cudaStream_t s);

}  // namespace qattn
