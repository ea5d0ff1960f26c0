// Eviction from a key/value cache by accumulated attention weight. Per
// sequence and key/value head, of len keys: all are kept when len <= budget;
// else the first `sinks`, the last `recent`, and of those between them the
// budget - sinks - recent with the largest score (equal scores: the lower
// index first; NaN below every number). The kept keys, values and scores move
// to the new cache in their old order.
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace crisp {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;   // 11 bits a level: 32 bits in three levels (11, 11, 10)

// Order-preserving 32-bit key of a score: -0 counts as +0, NaN as the lowest.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of one value per thread over the CTA; *total gets the sum.
__device__ __forceinline__ int cta_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int before = warp == 0 ? 0 : warp_sums[warp - 1];
  *total = warp_sums[31];
  __syncthreads();
  return before + inc - x;
}

// One CTA per (sequence, key/value head): the indices that stay, ascending.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ uint32_t found_bin;
  __shared__ int found_above;
  const int unit = blockIdx.x, b = unit / a.h_kv, tid = threadIdx.x;
  int len = a.kv_len != nullptr ? a.kv_len[b] : a.n_k;
  if (len < 0 || len > a.n_k) {
    if (tid == 0) a.status[kStatusLen] = CRISP_ERR_INVALID_ARG;
    len = len < 0 ? 0 : a.n_k;
  }
  int32_t* kept = a.kept + (int64_t)unit * a.budget;
  const int keep = min(len, a.budget);
  if (tid == 0 && unit % a.h_kv == 0) a.new_len[b] = keep;
  for (int i = keep + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  if (len <= a.budget) {
    for (int i = tid; i < len; i += kSelThreads) kept[i] = i;
    return;
  }
  const float* score = a.score + (int64_t)unit * a.n_k;
  const int m0 = a.sinks, m1 = len - a.recent;      // the keys that compete
  int want = a.budget - a.sinks - a.recent;         // < m1 - m0
  // radix select: the want-th largest key, level by level
  uint32_t prefix = 0, mask = 0;
  const int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
  if (want > 0) {
    for (int lev = 0; lev < 3; ++lev) {
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t bm = (1u << bits[lev]) - 1u;
      for (int j = m0 + tid; j < m1; j += kSelThreads) {
        const uint32_t key = score_key(score[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift[lev]) & bm], 1);
      }
      __syncthreads();
      // bins from the top: thread t owns bins top - 2t and top - 2t - 1
      const int top = kBins - 1 - 2 * tid;
      const int c0 = hist[top], c1 = hist[top - 1];
      int total;
      const int above = cta_scan(c0 + c1, warp_sums, &total);
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
  }
  // keys above the cut stay, and the first `want` equal to it
  const uint32_t cut = prefix;
  const bool any = a.budget > a.sinks + a.recent;
  int done = 0, ties = 0;
  for (int j0 = 0; j0 < len; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool stay = false, tie = false;
    if (j < len) {
      if (j < m0 || j >= m1) {
        stay = true;
      } else if (any) {
        const uint32_t key = score_key(score[j]);
        stay = key > cut;
        tie = key == cut;
      }
    }
    int n_tie, n_stay;
    const int t = ties + cta_scan(tie ? 1 : 0, warp_sums, &n_tie);
    if (tie && t < want) stay = true;
    const int at = done + cta_scan(stay ? 1 : 0, warp_sums, &n_stay);
    if (stay) kept[at] = j;
    ties += n_tie;
    done += n_stay;
  }
}

// One warp per kept key: its key row, value row and score; the scores behind
// the last kept key become 0.
__global__ void __launch_bounds__(256) evict_gather_kernel(EvictArgs a) {
  const int unit = blockIdx.y, b = unit / a.h_kv, g = unit - b * a.h_kv;
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= a.n_new) return;
  const int j = i < a.budget ? a.kept[(int64_t)unit * a.budget + i] : -1;
  float* sn = a.score_new + (int64_t)unit * a.n_new + i;
  if (j < 0) {
    if (lane == 0) *sn = 0.f;
    return;
  }
  const int es = a.row_bytes / kHeadDim;   // element size
  auto row = [&](const void* p, const Strides& s, int64_t t) {
    return static_cast<const char*>(p) + (b * s.seq + g * s.head + t * s.token) * es;
  };
  const char* ks = row(a.k, a.sk, j);
  const char* vs = row(a.v, a.sv, j);
  char* kd = const_cast<char*>(row(a.k_new, a.skn, i));
  char* vd = const_cast<char*>(row(a.v_new, a.svn, i));
  for (int o = lane * 16; o < 2 * a.row_bytes; o += 512) {
    if (o < a.row_bytes)
      *reinterpret_cast<uint4*>(kd + o) = *reinterpret_cast<const uint4*>(ks + o);
    else
      *reinterpret_cast<uint4*>(vd + o - a.row_bytes) = *reinterpret_cast<const uint4*>(vs + o - a.row_bytes);
  }
  if (lane == 0) *sn = a.score[(int64_t)unit * a.n_k + j];
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  const int units = a.batch * a.h_kv;
  evict_select_kernel<<<units, kSelThreads, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_gather_kernel<<<dim3((a.n_new + 7) / 8, units), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace crisp
