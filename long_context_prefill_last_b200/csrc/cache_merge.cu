// Joins the partial results of split key lists, and adds softmax weights to
// the keys' accumulated scores.
//   M = max_i m_i, L = sum_i 2^(m_i - M) l_i, o = sum_i 2^(m_i - M) O_i / L
// The pieces of a row are joined in slot order, so the result does not depend
// on the order in which CTAs ran.
#include <cuda_bf16.h>
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace crisp {
namespace {

__device__ __forceinline__ int merge_len(const int32_t* kv_len, int b, int n) {
  if (kv_len == nullptr) return n;
  const int x = kv_len[b];
  return x < 0 ? 0 : (x > n ? n : x);
}

// One CTA per output row (sequence, query head, token); thread = column.
template <typename T>
__global__ void __launch_bounds__(128) cache_merge_kernel(MergeArgs a) {
  const int row = blockIdx.x, c = threadIdx.x;
  const int i = row % a.n_q, bh = row / a.n_q;
  const int h_q = a.h_kv * a.group;
  const int b = bh / h_q, h = bh - b * h_q;
  const int g = h / a.group, j = h - g * a.group;
  float M = -INFINITY, L = 0.f, o = 0.f;
  for (int src = 0; src < 2; ++src) {
    const PartSrc& p = src == 0 ? a.main : a.pre;
    if (p.mode == kPartNone) continue;
    const int unit = src == 0 ? b * a.h_kv + g : g;
    const int r = src == 0 ? i * a.group + j : (b * a.n_q + i) * a.group + j;
    const int blk = r / p.block, in = r - blk * p.block;
    const int64_t first = ((int64_t)unit * p.blocks + blk) * p.splits;
    const int count = p.splits;
    for (int s = 0; s < count; ++s) {
      const int64_t at = (first + s) * p.block + in;
      const float2 ml = p.ml[at];
      if (ml.y == 0.f) continue;   // the piece holds no key that this row sees
      const float x = p.o[at * kHeadDim + c];
      const float mn = fmaxf(M, ml.x);
      const float f0 = exp2f(M - mn), f1 = exp2f(ml.x - mn);
      L = L * f0 + ml.y * f1;
      o = o * f0 + x * f1;
      M = mn;
    }
  }
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);   // no key: 0; NaN stays NaN
  T* dst = static_cast<T*>(a.out) + b * a.so.seq + h * a.so.head + i * a.so.token;
  dst[c] = dev::from_f32<T>(o * inv);
  if (a.final_ml != nullptr && c == 0)
    a.final_ml[(int64_t)(b * a.h_kv + g) * a.n_q * a.group + i * a.group + j] = make_float2(M == -INFINITY ? 0.f : M, inv);
}

// score[key] += sum over the unit's rows of 2^(x - M) / L, a thread per key
// and the rows in order: no atomics, the sum's order is fixed.
__global__ void __launch_bounds__(256) cache_score_kernel(ScoreArgs a) {
  extern __shared__ float2 fin[];
  const int unit = blockIdx.y, b = unit / a.h_kv;
  const int rows = a.n_q * a.group;
  for (int r = threadIdx.x; r < rows; r += blockDim.x) fin[r] = a.final_ml[(int64_t)unit * rows + r];
  __syncthreads();
  const KeyList list = key_list(merge_len(a.kv_len, b, a.n_k), a.n_q, 0, a.n_q - 1, a.window, a.sinks);
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= list.total) return;
  const float* x = a.logits + (int64_t)unit * rows * a.pitch + u;
  float sum = 0.f;
  for (int r = 0; r < rows; ++r) {
    const float y = x[r * a.pitch];
    if (y != -INFINITY) sum += exp2f(y - fin[r].x) * fin[r].y;   // -inf: the row does not see the key
  }
  float* dst = a.score + (int64_t)unit * a.n_k + list.key(u);
  *dst += sum;
}

}  // namespace

cudaError_t launch_cache_merge(const MergeArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.batch * a.h_kv * a.group * a.n_q;
  if (rows > INT32_MAX) return cudaErrorInvalidValue;
  if (a.fp32)
    cache_merge_kernel<float><<<(unsigned)rows, kHeadDim, 0, st>>>(a);
  else
    cache_merge_kernel<__nv_bfloat16><<<(unsigned)rows, kHeadDim, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_score(const ScoreArgs& a, cudaStream_t st) {
  const int64_t most = (int64_t)a.sinks + a.window + a.n_q - 1;
  const int keys = most < a.n_k ? (int)most : a.n_k;
  const dim3 grid((keys + 255) / 256, a.batch * a.h_kv);
  cache_score_kernel<<<grid, 256, a.n_q * a.group * sizeof(float2), st>>>(a);
  return cudaGetLastError();
}

}  // namespace crisp
