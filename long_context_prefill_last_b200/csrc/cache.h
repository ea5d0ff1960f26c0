// Internal declarations of the cache operators: attention over a key/value
// cache (window, scored, shared prefix) and eviction (not part of the ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "crisp.h"
#include "internal.h"

namespace crisp {

constexpr int kMaxBatch = 1024;          // sequences of one call
constexpr int kMaxCacheLen = 1 << 24;    // key slots per sequence
constexpr int kMaxDraft = 16;            // query tokens of a scored or shared-prefix call, and of the bf16 decode kernel
constexpr int kNoWindow = 1 << 30;       // window = 0: every earlier key
constexpr int kStatusLen = 4;            // status slot: a sequence length outside [0, n_k] (it was clamped)

struct Strides {   // elements; d is contiguous
  int64_t seq, head, token;
};

// A validated cache configuration.
struct CacheShape {
  int batch, n_q, n_k, h_q, h_kv, group;
  int window;              // kNoWindow when unlimited
  int sinks;
  int n_prefix, budget, recent, n_new;
  bool fp32;
  float scale_log2;
  Strides q, k, v, out, k_prefix, v_prefix, k_new, v_new;
};

// The keys that the queries of one unit read, as one list: the first `se`
// keys, then keys lo, lo + 1, ... Entry u is key u for u < se, else
// lo + (u - se).
struct KeyList {
  int se, lo, total;
#ifdef __CUDACC__
  __host__ __device__ int key(int u) const { return u < se ? u : lo + (u - se); }
#endif
};

// Union of the keys that query tokens i0..i1 of a sequence of len keys see.
// Token i is at position len - n_q + i and sees key j when 0 <= j <= position
// and (j < sinks or j > position - window).
#ifdef __CUDACC__
__host__ __device__
#endif
inline KeyList key_list(int len, int n_q, int i0, int i1, int window, int sinks) {
  KeyList r;
  const int first = len - n_q + i0;
  const int hi = len - n_q + i1 + 1;           // one past the last position (<= len)
  if (hi <= 0) {
    r.se = r.lo = r.total = 0;
    return r;
  }
  r.se = sinks < hi ? sinks : hi;
  const int low = first - window + 1;
  r.lo = low > r.se ? low : r.se;
  r.total = r.se + (hi - r.lo);
  return r;
}

// Units and rows of an attention launch: a unit is one key/value head of one
// sequence; its rows are its (token, head of the group) pairs, token-major. For
// the shared prefix a unit is one key/value head and its rows are those of
// every sequence, one after another.

// Where an attention launch leaves a row's partial results: runs of
// consecutive slots of `block` rows each. kSplits: slot = job * splits + s.
// kStair: the launch's key tiles are dealt to `ctas` CTAs as equal runs of one
// flat list; slot = (CTA + job) * splits + s (unique: CTA and job only grow
// along the list), with `splits` results per CTA and job.
// kBoxes: the tcgen05 kernel's row tiles, two per job; slot = job * splits + s.
enum PartMode : int { kPartNone = 0, kSplits = 1, kStair = 2, kBoxes = 3 };
struct PartSrc {
  int mode;
  const float* o;       // [slot][block][128], not normalised
  const float2* ml;     // [slot][block]: maximum (log2 domain), sum
  int block;            // rows per slot
  int blocks;           // row blocks per unit
  int splits;
  const int2* table;    // kStair: [job] first and last CTA
  int tok_box, seq_box; // kBoxes
};

// x / d as (x * div_magic(d)) >> 36, exact while x * d < 2^36 (rows < 2^28, d <= 256).
inline uint64_t div_magic(int d) { return (((uint64_t)1 << 36) + d - 1) / d; }

// Arguments shared by the attention kernels.
struct CacheArgs {
  const void *q, *k, *v;
  void* out;
  const int32_t* kv_len;   // NULL: n_keys for every sequence
  int32_t* status;
  int batch;               // sequences (1 unit group for the prefix)
  int n_keys;              // key slots per sequence, or the prefix length
  int h_kv, group, n_q, window, sinks;
  int rows, per_seq;       // rows per unit; rows per sequence within it
  int sets_status;         // the call's only kernel that reports: it sets the status words instead of a memset
  int cluster;             // bf16 decode kernel: CTAs of a cluster that has a job to itself (0: runs of the flat list)
  int chained;             // launched beside the kernel before it: it ends after that one has
  int prefix;              // rows run over every sequence, every key is seen
  int tok_box, seq_box;    // tcgen05 kernel: tokens and sequences of a row tile
  int row_tiles;           // per unit
  int n_seqs;              // sequences of q
  uint64_t group_mul, seq_mul;   // div_magic(group), div_magic(per_seq)
  float scale_log2;
  Strides sq, sk, sv, so;
  // partial results (NULL: write the output rows)
  float* part_o;
  float2* part_ml;
  int block, blocks, splits, ctas;   // block: rows of a partial slot
  int2* table;             // decode kernel: [job] first and last CTA that had a tile of it
  // scored: scaled logits [unit][row][pitch] by list index
  float* logits;
  int64_t pitch;
  float* score;            // [batch][h_kv][n_keys]
};

#ifdef __CUDACC__
namespace dev {

__device__ __forceinline__ int cache_len(const CacheArgs& a, int b) {
  if (a.kv_len == nullptr) return a.n_keys;
  int n = a.kv_len[b];
  if (n < 0 || n > a.n_keys) {
    a.status[kStatusLen] = CRISP_ERR_INVALID_ARG;   // every writer writes the same value
    n = n < 0 ? 0 : a.n_keys;
  }
  return n;
}

// Key list of query tokens i0..i1 of sequence b (every key for the prefix).
__device__ __forceinline__ KeyList unit_keys(const CacheArgs& a, int len, int i0, int i1) {
  if (a.prefix) {
    KeyList r;
    r.se = 0;
    r.lo = 0;
    r.total = len;
    return r;
  }
  return key_list(len, a.n_q, i0, i1, a.window, a.sinks);
}

// Row r of unit (b, g): sequence, token and query head.
struct Row {
  int b, i, h;
};
__device__ __forceinline__ Row unit_row(const CacheArgs& a, int b, int g, int r) {
  Row x;
  x.b = b;
  if (a.prefix) {
    x.b = (int)(((uint64_t)r * a.seq_mul) >> 36);
    r -= x.b * a.per_seq;
  }
  x.i = (int)(((uint64_t)r * a.group_mul) >> 36);
  x.h = g * a.group + (r - x.i * a.group);
  return x;
}

// Position of query token i: keys past it are not seen. Prefix rows see every key.
__device__ __forceinline__ int row_pos(const CacheArgs& a, int len, int i) {
  return a.prefix ? (1 << 29) : len - a.n_q + i;
}

__device__ __forceinline__ int clamp_len(const int32_t* kv_len, int b, int n_keys, bool* bad = nullptr) {
  if (kv_len == nullptr) return n_keys;
  const int n = kv_len[b];
  if (n >= 0 && n <= n_keys) return n;
  if (bad != nullptr) *bad = true;
  return n < 0 ? 0 : n_keys;
}
__device__ __forceinline__ int clamped_len(const CacheArgs& a, int b) { return clamp_len(a.kv_len, b, a.n_keys); }

// Key tiles of every sequence, summed: cum[b] = tiles of the sequences before
// b, cum[batch] = all. Called by a whole CTA; ends with a barrier. tmp: int[32].
// Returns whether some length was outside [0, n_keys].
__device__ __forceinline__ bool stair_scan(const int32_t* kv_len, int batch, int n_keys, int n_q, int window, int sinks,
                                           bool prefix, int tile, int* cum, int* tmp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (batch + blockDim.x - 1) / blockDim.x;
  bool bad = false;
  auto tiles_of = [&](int b) {
    const int n = clamp_len(kv_len, b, n_keys, &bad);
    return ((prefix ? n : key_list(n, n_q, 0, n_q - 1, window, sinks).total) + tile - 1) / tile;
  };
  if (batch == 1) {
    if (tid == 0) {
      cum[0] = 0;
      cum[1] = tiles_of(0);
    }
    return __syncthreads_or(bad) != 0;
  }
  int mine = 0;
  if (per == 1) {
    mine = tid < batch ? tiles_of(tid) : 0;
  } else {
    for (int i = 0; i < per; ++i)
      if (tid * per + i < batch) mine += tiles_of(tid * per + i);
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (batch <= 32) {   // one warp's work
    if (warp == 0) {
      if (lane < batch) cum[lane] = inc - mine;
      if (lane == 31) cum[batch] = inc;
    }
    return __syncthreads_or(bad) != 0;
  }
  if (lane == 31) tmp[warp] = inc;
  __syncthreads();
  int at = inc - mine;
  for (int w = 0; w < warp; ++w) at += tmp[w];
  if (per == 1) {
    if (tid < batch) cum[tid] = at;
    if (tid == batch - 1) cum[batch] = at + mine;
  } else {
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b < batch) {
        cum[b] = at;
        at += tiles_of(b);
        if (b == batch - 1) cum[batch] = at;
      }
    }
  }
  return __syncthreads_or(bad) != 0;
}

// A place in the flat list of key tiles that the decode kernels deal to their
// CTAs: sequence after sequence, in each its jobs (key/value head, row block)
// and in each job its key tiles.
struct Place {
  int b, jj, t;      // sequence, job within it, next key tile of the job
  int T, len;        // key tiles of the sequence's jobs, tokens
  KeyList list;
  __device__ void enter(const CacheArgs& a, const int* cum) {   // after b, jj, t are set
    T = cum[b + 1] - cum[b];
    len = clamped_len(a, b);
    list = unit_keys(a, len, 0, a.n_q - 1);
  }
  __device__ void next_job(const CacheArgs& a, const int* cum, int per_seq) {
    t = 0;
    if (++jj == per_seq) {
      jj = 0;
      do ++b; while (cum[b + 1] == cum[b]);
      enter(a, cum);
    }
  }
};

// L2 policy for data that is read once.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t evict_normal() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// 16-byte asynchronous copy; bytes = 0 fills with zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::128B [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(bytes), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Programmatic launch: let the next kernel of the stream start its set-up
// early / wait until the kernels before have finished and their writes show.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launches() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The sequence that holds tile x of the summed list (sequences without tiles are passed over).
__device__ __forceinline__ int stair_find(const int* cum, int batch, int x) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The start of the CTA's run of tiles, and its length (0: none): runs differ
// by one tile at most.
template <typename U>
__device__ __forceinline__ int stair_run(const CacheArgs& a, const int* cum, Place& p) {
  const U per_seq = a.h_kv * a.blocks, all = (U)cum[a.batch] * per_seq;
  const U ctas = all < (U)a.ctas ? all : (U)a.ctas, c = blockIdx.x;   // every one of them has a tile
  if (c >= ctas) return 0;
  const U base = all / ctas, extra = all - base * ctas;
  const U x0 = c * base + (c < extra ? c : extra);
  p.b = stair_find(cum, a.batch, (int)(x0 / per_seq));
  const U rem = x0 - (U)cum[p.b] * per_seq;
  const U T = cum[p.b + 1] - cum[p.b];
  p.jj = (int)(rem / T);
  p.t = (int)(rem - (U)p.jj * T);
  p.enter(a, cum);
  return (int)(base + (c < extra ? 1 : 0));
}
__device__ __forceinline__ int stair_start(const CacheArgs& a, const int* cum, Place& p) {
  // 64-bit divisions cost a few hundred cycles each
  const int64_t all = (int64_t)cum[a.batch] * a.h_kv * a.blocks;
  return all < ((int64_t)1 << 32) ? stair_run<uint32_t>(a, cum, p) : stair_run<uint64_t>(a, cum, p);
}

}  // namespace dev
#endif

// ---- plans: grid shapes and workspace pieces of one call, fixed by the shape ----
struct AttnPlan {
  int kernel;        // AttnKernel
  int block, blocks, splits, ctas, tile;
  int slot_rows;     // rows of a partial slot: the block's, or the unit's where it has only one block
  int tok_box, seq_box, row_tiles;   // kTileTc
  int run;           // kTileSimt: key tiles of a CTA, at most
  int units;
  int cluster;       // kDecodeMma: CTAs per job that join their results themselves (0: see kStair)
  size_t slots;      // partial slots (0: the kernel writes the output itself)
};
enum AttnKernel : int { kTileSimt = 0, kDecodeMma = 1, kTileTc = 2, kDecodeSimt = 3 };

struct CachePlan {
  AttnPlan main, pre;       // the sequences' own keys; the shared prefix
  bool has_pre;
  int64_t pitch;            // scored: logits per row
  int warps_per_row;        // of the finishing kernel
  size_t off_ml, off_o, off_table, off_pre_ml, off_pre_o, off_pre_table, off_logits;
  size_t total;
};

CachePlan plan_cache(const CacheShape& s, int op);

// ---- launchers (each enqueues on `st`; return cudaGetLastError()) ----
cudaError_t launch_cache_tc(const CacheArgs& a, const AttnPlan& p, cudaStream_t st);
cudaError_t launch_cache_decode(const CacheArgs& a, const AttnPlan& p, cudaStream_t st);
cudaError_t launch_cache_decode_fp32(const CacheArgs& a, const AttnPlan& p, cudaStream_t st);
cudaError_t launch_cache_tile(const CacheArgs& a, const AttnPlan& p, cudaStream_t st);   // fp32

// Launches a kernel in clusters of `cluster` CTAs; with `beside` it may start
// before the one before it in the stream has finished.
template <typename... P, typename... A>
inline cudaError_t launch_clusters(void (*kernel)(P...), unsigned grid, unsigned cluster, int threads, size_t smem,
                                   cudaStream_t st, bool beside, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {};
  unsigned n = 0;
  if (beside) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
inline cudaError_t launch_kernel(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, bool beside,
                                 const A&... args) {
  return launch_clusters(kernel, grid, 1, threads, smem, st, beside, args...);
}

struct FinishArgs {
  PartSrc main, pre;
  const int32_t* kv_len;
  int batch, n_q, n_k, h_kv, group, window, sinks;
  void* out;
  Strides so;
  bool fp32;
  int warps_per_row;       // 1, 2, 4 or 8
  // scored
  const float* logits;     // [unit][row][pitch], by list index; NULL: no scores
  int64_t pitch;
  float* score;            // [batch][h_kv][n_k]
  int out_ctas, score_ctas;   // set by the launcher; score CTAs per unit
};
cudaError_t launch_cache_finish(const FinishArgs& a, cudaStream_t st);

struct EvictArgs {
  const void *k, *v;
  const float* score;
  const int32_t* kv_len;
  void *k_new, *v_new;
  float* score_new;
  int32_t *kept, *new_len, *status;
  Strides sk, sv, skn, svn;
  int batch, h_kv, n_k, sinks, recent, budget, n_new;
  int row_bytes;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace crisp
