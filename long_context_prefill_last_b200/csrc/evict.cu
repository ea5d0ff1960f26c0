// Eviction from a key/value cache by accumulated attention weight. Per
// sequence and key/value head, of len keys: all are kept when len <= budget;
// else the first `sinks`, the last `recent`, and of those between them the
// budget - sinks - recent with the largest score (equal scores: the lower
// index first; NaN below every number). The kept keys, values and scores move
// to the new cache in their old order.
//
// Selection: the cut is found by a radix select on order-preserving 32-bit
// keys (11 + 11 + 10 bits, counts in shared memory); the counts also say how
// many survivors each CTA has, and so where its first one goes. One cluster of
// 1 to 8 CTAs per head shares the counts through distributed shared memory; a
// head is a few hundred KB of scores, read once and kept in shared memory, so
// this is bound by the latency of its few barriers. The move is bound by memory:
// 8 heads of 131072 keys cut to 16384 take 27 us for the selection and 20 us
// for the move of 134 MB, of which HBM has read 72 MB and written 12 MB by its
// end (half of its rate; the other writes are still in L2).
#include <cooperative_groups.h>
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace crisp {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCachedKeys = 40960;   // keys of a CTA's stretch held in shared memory (160 KB)
constexpr int kMoveKeys = 8;         // keys per warp of the move

// Order-preserving 32-bit key of a score: -0 counts as +0, NaN as the lowest.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of one value per thread over the CTA.
__device__ __forceinline__ int cta_scan(int x, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int w = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp == 0 ? 0 : before) + inc - x;
}

// One cluster per (sequence, key/value head): the indices that stay, ascending.
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(EvictArgs a, int cs) {
  extern __shared__ uint32_t cached[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ int warp_sums[32];
  __shared__ uint32_t found_bin;
  __shared__ int found_above;
  __shared__ int warp_above[kSelWarps];
  __shared__ __align__(8) int cta_counts[2];   // above the cut, equal to it
  const cg::cluster_group cluster = cg::this_cluster();
  const int unit = blockIdx.x / cs, rank = blockIdx.x - unit * cs, b = unit / a.h_kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int everyone = cs * kSelThreads, me = rank * kSelThreads + tid;
  dev::launch_dependents();

  if (blockIdx.x == 0) {   // the call's status: a length outside [0, n_k]?
    bool bad = false;
    for (int i = tid; i < a.batch; i += kSelThreads) dev::clamp_len(a.kv_len, i, a.n_k, &bad);
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      a.status[kStatusCode] = 0;
      a.status[kStatusLen] = bad ? CRISP_ERR_INVALID_ARG : 0;
    }
  }
  const int len = dev::clamp_len(a.kv_len, b, a.n_k);
  int32_t* kept = a.kept + (int64_t)unit * a.budget;
  const int keep = min(len, a.budget);
  if (me == 0 && unit == b * a.h_kv) a.new_len[b] = keep;
  for (int i = keep + me; i < a.budget; i += everyone) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = me; i < len; i += everyone) kept[i] = i;
    return;
  }
  const float* score = a.score + (int64_t)unit * a.n_k;
  const int m0 = a.sinks, m1 = len - a.recent;      // the keys between compete
  for (int i = me; i < m0; i += everyone) kept[i] = i;
  for (int i = me; i < a.recent; i += everyone) kept[a.budget - a.recent + i] = m1 + i;
  int want = a.budget - a.sinks - a.recent;         // < m1 - m0
  if (want == 0) return;

  // this CTA's stretch
  const int seg = ((m1 - m0 + cs - 1) / cs + 31) & ~31;
  const int s0 = min(m1, m0 + rank * seg), n = min(m1, s0 + seg) - s0;
  const bool hold = seg <= kCachedKeys;
  for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[i / kBins][i % kBins] = 0;
  __syncthreads();
  const float* mine = score + s0;
  auto key_at = [&](int i) { return hold ? cached[i] : score_key(mine[i]); };

  uint32_t prefix = 0, mask = 0;
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
  for (int lev = 0; lev < 3; ++lev) {
    const uint32_t bm = (1u << bits[lev]) - 1u;
    if (lev == 0) {
      int i = tid;
      for (; i + 7 * kSelThreads < n; i += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = mine[i + q * kSelThreads];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t key = score_key(x[q]);
          if (hold) cached[i + q * kSelThreads] = key;
          atomicAdd(&hist[0][key >> shift[0]], 1);
        }
      }
      for (; i < n; i += kSelThreads) {
        const uint32_t key = score_key(mine[i]);
        if (hold) cached[i] = key;
        atomicAdd(&hist[0][key >> shift[0]], 1);
      }
    } else {
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t key = key_at(i);
        if ((key & mask) == prefix) atomicAdd(&hist[lev][(key >> shift[lev]) & bm], 1);
      }
    }
    if (cs > 1) cluster.sync(); else __syncthreads();
    // bins from the top: thread t owns bins top = last - 2t and top - 1, summed over the cluster
    const int top = kBins - 1 - 2 * tid;
    int c0 = 0, c1 = 0;
    if (cs > 1) {
      int2 c[8];   // the cluster's counts, all loads in flight at once
#pragma unroll
      for (int r = 0; r < 8; ++r)
        c[r] = r < cs ? *reinterpret_cast<const int2*>(cluster.map_shared_rank(hist[lev], r) + top - 1) : make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        c0 += c[r].y;
        c1 += c[r].x;
      }
    } else {
      const int2 c = *reinterpret_cast<const int2*>(hist[lev] + top - 1);
      c0 = c.y;
      c1 = c.x;
    }
    const int above = cta_scan(c0 + c1, warp_sums);
    if (above < want && above + c0 >= want) {
      found_bin = (uint32_t)top;
      found_above = above;
    } else if (above + c0 < want && above + c0 + c1 >= want) {
      found_bin = (uint32_t)(top - 1);
      found_above = above + c0;
    }
    __syncthreads();
    prefix |= found_bin << shift[lev];
    mask |= bm << shift[lev];
    want -= found_above;
    __syncthreads();
  }
  // Keys above the cut stay, and the first `want` equal to it. How many of
  // either this CTA has, for those that come after it, follows from its own counts.
  const uint32_t cut = prefix;
  if (cs > 1) {
    int up = 0;
#pragma unroll
    for (int lev = 0; lev < 3; ++lev) {
      const int bin = (int)((cut >> shift[lev]) & ((1u << bits[lev]) - 1u));
      for (int i = tid; i < kBins; i += kSelThreads) up += i > bin ? hist[lev][i] : 0;
    }
    int total = up;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) warp_above[warp] = total;
    __syncthreads();
    if (warp == 0) {
      total = warp_above[lane];
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
      if (lane == 0) {
        cta_counts[0] = total;
        cta_counts[1] = hist[2][cut & ((1u << bits[2]) - 1u)];
      }
    }
  }
  int before_above = 0, before_ties = 0;
  if (cs > 1) {
    cluster.sync();
    int2 c[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      c[r] = r < rank ? *reinterpret_cast<const int2*>(cluster.map_shared_rank(cta_counts, r)) : make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      before_above += c[r].x;
      before_ties += c[r].y;
    }
    cluster.sync();   // nobody reads the counts, or this CTA's totals, any more
  }
  // 32 keys a word, 1024 words a round: warps set the words' bits (the counts'
  // memory serves again), a scan gives each word its place, warps write the survivors
  uint32_t* ups = reinterpret_cast<uint32_t*>(hist[0]);
  uint32_t* tie = reinterpret_cast<uint32_t*>(hist[1]);
  int2* first = reinterpret_cast<int2*>(hist[2]);   // survivors before a word: above the cut, equal to it
  for (int base = 0; base < n; base += 32 * kSelThreads) {
    const int words = min(kSelThreads, (n - base + 31) / 32);
#pragma unroll 4
    for (int w = warp; w < words; w += kSelWarps) {
      const int i = base + w * 32 + lane;
      const uint32_t key = i < n ? key_at(i) : 0u;
      const uint32_t x = __ballot_sync(0xffffffffu, i < n && key > cut);
      const uint32_t y = __ballot_sync(0xffffffffu, i < n && key == cut);
      if (lane == 0) {
        ups[w] = x;
        tie[w] = y;
      }
    }
    __syncthreads();
    const uint32_t x = tid < words ? ups[tid] : 0u, y = tid < words ? tie[tid] : 0u;
    // both prefix sums at once: a round has at most 32768 of either
    const int both = cta_scan(__popc(x) | (__popc(y) << 16), warp_sums);
    const int at = before_above + (both & 0xffff), t = before_ties + (int)((uint32_t)both >> 16);
    first[tid] = make_int2(at, t);
    __syncthreads();
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll 4
    for (int w = warp; w < words; w += kSelWarps) {
      const uint32_t xs = ups[w], ys = tie[w];
      const int2 f = first[w];
      const int up = f.x + __popc(xs & lower), ti = f.y + __popc(ys & lower);
      if (((xs >> lane) & 1u) || (((ys >> lane) & 1u) && ti < want)) kept[m0 + up + min(ti, want)] = s0 + base + w * 32 + lane;
    }
    __syncthreads();   // the words have been read
    if (base + 32 * kSelThreads < n) {
      if (tid == kSelThreads - 1) {
        cta_counts[0] = at + __popc(x);
        cta_counts[1] = t + __popc(y);
      }
      __syncthreads();
      before_above = cta_counts[0];
      before_ties = cta_counts[1];
      __syncthreads();
    }
  }
}

// Eight kept keys per warp: their key rows, value rows and scores; the scores
// behind the last kept key become 0. All loads of a warp are in flight at
// once. VEC: 16-byte pieces of a key's K and V rows per lane (1 bf16, 2 fp32).
template <int VEC>
__global__ void __launch_bounds__(256) evict_move_kernel(EvictArgs a) {
  const int unit = blockIdx.y, b = unit / a.h_kv, g = unit - b * a.h_kv;
  const int lane = threadIdx.x & 31;
  const int i0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kMoveKeys;
  if (i0 >= a.n_new) return;
  constexpr int es = VEC * 2;   // element size
  constexpr int row16 = VEC * 16;   // 16-byte pieces per row
  dev::wait_for_launches();
  int j = -1;
  float sc = 0.f;
  if (lane < kMoveKeys && i0 + lane < a.budget) {
    j = a.kept[(int64_t)unit * a.budget + i0 + lane];
    if (j >= 0) sc = a.score[(int64_t)unit * a.n_k + j];
  }
  const char* k0 = static_cast<const char*>(a.k) + (b * a.sk.seq + g * a.sk.head) * es;
  const char* v0 = static_cast<const char*>(a.v) + (b * a.sv.seq + g * a.sv.head) * es;
  char* kn = static_cast<char*>(a.k_new) + (b * a.skn.seq + g * a.skn.head) * es;
  char* vn = static_cast<char*>(a.v_new) + (b * a.svn.seq + g * a.svn.head) * es;
  uint4 x[kMoveKeys][VEC];
  int from[kMoveKeys];
#pragma unroll
  for (int q = 0; q < kMoveKeys; ++q) {
    from[q] = __shfl_sync(0xffffffffu, j, q);
    if (from[q] >= 0) {
#pragma unroll
      for (int p = 0; p < VEC; ++p) {
        const int c = p * 32 + lane;
        const char* src = c < row16 ? k0 + (int64_t)from[q] * a.sk.token * es + c * 16
                                    : v0 + (int64_t)from[q] * a.sv.token * es + (c - row16) * 16;
        x[q][p] = __ldcs(reinterpret_cast<const uint4*>(src));
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kMoveKeys; ++q) {
    if (from[q] >= 0) {
#pragma unroll
      for (int p = 0; p < VEC; ++p) {
        const int c = p * 32 + lane;
        char* dst = c < row16 ? kn + (int64_t)(i0 + q) * a.skn.token * es + c * 16
                              : vn + (int64_t)(i0 + q) * a.svn.token * es + (c - row16) * 16;
        *reinterpret_cast<uint4*>(dst) = x[q][p];
      }
    }
  }
  if (lane < kMoveKeys && i0 + lane < a.n_new) a.score_new[(int64_t)unit * a.n_new + i0 + lane] = sc;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int units = a.batch * a.h_kv;
  // a cluster per head: about 8192 keys per CTA, while that does not ask for more than two CTAs per SM
  int cs = 1;
  while (cs < 8 && (int64_t)cs * 8192 < a.n_k && 2 * cs * units <= 296) cs *= 2;
  while (cs < 8 && (int64_t)cs * kCachedKeys < a.n_k) cs *= 2;   // or the keys would be read from memory four times
  const int64_t stretch = ((a.n_k + cs - 1) / cs + 31) / 32 * 32;
  const size_t smem = 4 * (size_t)(stretch < kCachedKeys ? stretch : kCachedKeys);
  cudaError_t e =
      cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kCachedKeys);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cs)) != cudaSuccess) return e;
  cfg.gridDim = dim3((a.n_new + 8 * kMoveKeys - 1) / (8 * kMoveKeys), units);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return a.row_bytes == 2 * kHeadDim ? cudaLaunchKernelEx(&cfg, evict_move_kernel<1>, a)
                                     : cudaLaunchKernelEx(&cfg, evict_move_kernel<2>, a);
}

}  // namespace crisp
