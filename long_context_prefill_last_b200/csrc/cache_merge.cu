// Joins the partial results of split key lists, and adds softmax weights to
// the keys' accumulated scores.
//   M = max_i m_i, L = sum_i 2^(m_i - M) l_i, o = sum_i 2^(m_i - M) O_i / L
//   score_j += sum over the rows of 2^(x_rj - M_r) / L_r
// The pieces of a row are joined in a fixed order and a thread adds up a key's
// rows in order, so results do not depend on the order in which CTAs ran.
// Bound by latency (a few KB per row), so both happen in one launch: the first
// CTAs take output rows, the others keys, each of them computing the (M, L)
// that it needs from the pieces' own. Measured: 4 to 8 us for outputs; about
// 23 us with 67 MB of logits and 34 MB of scores (one token on 524288 tokens).
#include <cuda_bf16.h>
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace crisp {
namespace {

constexpr int kThreads = 256;
constexpr int kScoreKeys = 4;   // keys per thread, a CTA's width apart
constexpr int kScoreRows = 4;   // rows per step

struct Pieces {
  int64_t at[2];   // first piece's row, in rows of the source
  int count[2];
};

// The pieces of row r of unit (b, g) in both sources.
__device__ __forceinline__ Pieces find_pieces(const FinishArgs& a, int b, int g, int i, int j) {
  Pieces p;
#pragma unroll
  for (int src = 0; src < 2; ++src) {
    const PartSrc& s = src == 0 ? a.main : a.pre;
    p.count[src] = 0;
    p.at[src] = 0;
    if (s.mode == kPartNone) continue;
    const int unit = src == 0 ? b * a.h_kv + g : g;
    const int r = src == 0 ? i * a.group + j : (b * a.n_q + i) * a.group + j;
    int blk, in;
    if (s.mode == kBoxes) {
      const int it = i / s.tok_box;
      int ti = it, row = (i - it * s.tok_box) * a.group + j;
      if (src == 1) {
        const int bt = b / s.seq_box;
        ti += bt * ((a.n_q + s.tok_box - 1) / s.tok_box);
        row += (b - bt * s.seq_box) * s.tok_box * a.group;
      }
      blk = s.block == 256 ? ti >> 1 : ti;
      in = s.block == 256 ? (ti & 1) * 128 + row : row;
    } else {
      blk = r / s.block;
      in = r - blk * s.block;
    }
    const int job = unit * s.blocks + blk;
    int64_t first = (int64_t)job * s.splits;
    int count = s.splits;
    if (s.mode == kStair) {
      // a job without key tiles has no entry of its own
      const bool any = src == 1 || dev::clamp_len(a.kv_len, b, a.n_k) > 0;
      const int2 ctas = any ? s.table[job] : make_int2(0, -1);
      first = ((int64_t)ctas.x + job) * s.splits;
      count = (ctas.y - ctas.x + 1) * s.splits;
    }
    p.at[src] = first * s.block + in;
    p.count[src] = count;
  }
  return p;
}

__device__ __forceinline__ float2 piece_ml(const FinishArgs& a, const Pieces& p, int i) {
  const bool own = i < p.count[0];
  const PartSrc& s = own ? a.main : a.pre;
  return s.ml[p.at[own ? 0 : 1] + (int64_t)(own ? i : i - p.count[0]) * s.block];
}

// Row statistics by `lanes` neighbouring lanes (a power of two): the base that
// exponents subtract (0 when the row sees no key) and the sum.
__device__ __forceinline__ float2 row_stats(const FinishArgs& a, const Pieces& p, int lane, int lanes) {
  const int n = p.count[0] + p.count[1], l0 = lane & (lanes - 1);
  float M = -INFINITY, L = 0.f;
  for (int i0 = l0; i0 < n; i0 += 4 * lanes) {
    float2 ml[4];   // four loads in flight
#pragma unroll
    for (int e = 0; e < 4; ++e)
      ml[e] = i0 + e * lanes < n ? piece_ml(a, p, i0 + e * lanes) : make_float2(-INFINITY, 0.f);
    const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
    const float base = mn == -INFINITY ? 0.f : mn;
    L *= exp2f(M - base);
    M = mn;
#pragma unroll
    for (int e = 0; e < 4; ++e) L += exp2f(ml[e].x - base) * ml[e].y;
  }
  float top = M;
  for (int d = lanes >> 1; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -INFINITY ? 0.f : top;
  L *= exp2f(M - base);
  for (int d = lanes >> 1; d >= 1; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  return make_float2(base, L);
}

// 1 / L; 0 for a row that sees no key; NaN stays NaN.
__device__ __forceinline__ float inverse(float L) { return L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L); }

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(dev::pack_bf16x2(v.x, v.y), dev::pack_bf16x2(v.z, v.w));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_finish_kernel(FinishArgs a) {
  __shared__ float4 join[8][32];
  __shared__ float2 fin[kMaxDraft * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dev::wait_for_launches();

  if ((int)blockIdx.x < a.out_ctas) {
    // ------------------------------------------------ output rows, warps_per_row warps each
    const int W = a.warps_per_row, part = warp % W;
    const int64_t row = (int64_t)blockIdx.x * (8 / W) + warp / W;
    const int h_q = a.h_kv * a.group;
    const bool in = row < (int64_t)a.batch * h_q * a.n_q;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    int i = 0, b = 0, h = 0;
    if (in) {
      i = (int)(row % a.n_q);
      const int bh = (int)(row / a.n_q);
      b = bh / h_q;
      h = bh - b * h_q;
      const int g = h / a.group, j = h - g * a.group;
      const Pieces p = find_pieces(a, b, g, i, j);
      const float2 st = row_stats(a, p, lane, 32);
      L = st.y;
      const int n = p.count[0] + p.count[1];
      for (int i0 = 0; i0 < n; i0 += 32) {
        float w = 0.f;
        if (i0 + lane < n) w = exp2f(piece_ml(a, p, i0 + lane).x - st.x);
        const int m = n - i0 < 32 ? n - i0 : 32;
        for (int c0 = part; c0 < m; c0 += 4 * W) {
          float4 x[4];
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = c0 + e * W, q = i0 + c;
            f[e] = __shfl_sync(0xffffffffu, w, c & 31);
            x[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c >= m) f[e] = 0.f;
            if (f[e] != 0.f) {   // else nothing of the piece counts (it may not even be written)
              const bool own = q < p.count[0];
              const PartSrc& s = own ? a.main : a.pre;
              const int64_t at = p.at[own ? 0 : 1] + (int64_t)(own ? q : q - p.count[0]) * s.block;
              x[e] = *reinterpret_cast<const float4*>(s.o + at * kHeadDim + lane * 4);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o.x += f[e] * x[e].x, o.y += f[e] * x[e].y, o.z += f[e] * x[e].z, o.w += f[e] * x[e].w;
        }
      }
    }
    if (W > 1) {
      join[warp][lane] = o;
      __syncthreads();
      if (part == 0)
        for (int c = 1; c < W; ++c) {
          const float4 x = join[warp + c][lane];
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
    }
    if (in && part == 0) {
      const float inv = inverse(L);
      T* dst = static_cast<T*>(a.out) + b * a.so.seq + h * a.so.head + i * a.so.token;
      store4(dst + lane * 4, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
    return;
  }
  // ------------------------------------------------ scores: one thread per key, the rows in order
  const int id = blockIdx.x - a.out_ctas;
  const int unit = id / a.score_ctas, b = unit / a.h_kv, g = unit - b * a.h_kv;
  const KeyList list = key_list(dev::clamp_len(a.kv_len, b, a.n_k), a.n_q, 0, a.n_q - 1, a.window, a.sinks);
  const int stride = a.score_ctas * kThreads * kScoreKeys;
  int u = (id - unit * a.score_ctas) * kThreads * kScoreKeys;
  if (u >= list.total) return;
  const int rows = a.n_q * a.group;
  // as many rows at once as their pieces allow: each costs a chain of loads
  const int lanes = a.warps_per_row >= 4 ? 32 : a.warps_per_row * 4;
  for (int r0 = 0; r0 < rows; r0 += kThreads / lanes) {   // same trips for every lane
    const int r = r0 + (int)threadIdx.x / lanes;
    Pieces p{{0, 0}, {0, 0}};
    if (r < rows) p = find_pieces(a, b, g, r / a.group, r % a.group);
    const float2 st = row_stats(a, p, lane, lanes);
    if (r < rows && (lane & (lanes - 1)) == 0) fin[r] = make_float2(st.x, inverse(st.y));
  }
  __syncthreads();
  // Steps of kScoreRows rows x kScoreKeys keys per thread; a step's loads are
  // issued before the arithmetic of the one before.
  const int steps = (rows + kScoreRows - 1) / kScoreRows;
  const float* x0 = a.logits + (int64_t)unit * rows * a.pitch + threadIdx.x;
  float* dst = a.score + (int64_t)unit * a.n_k;
  float y[kScoreRows][kScoreKeys], next[kScoreRows][kScoreKeys], old[kScoreKeys], sum[kScoreKeys];
  auto fetch = [&](float (&v)[kScoreRows][kScoreKeys], int base, int r0) {
#pragma unroll
    for (int q = 0; q < kScoreRows; ++q)
#pragma unroll
      for (int c = 0; c < kScoreKeys; ++c)
        v[q][c] = base + (int)threadIdx.x + c * kThreads < list.total && r0 + q < rows
                      ? __ldcs(x0 + (r0 + q) * a.pitch + base + c * kThreads)
                      : -INFINITY;
  };
  fetch(y, u, 0);
  while (u < list.total) {
#pragma unroll
    for (int c = 0; c < kScoreKeys; ++c) {
      const int at = u + (int)threadIdx.x + c * kThreads;
      old[c] = at < list.total ? dst[list.key(at)] : 0.f;
      sum[c] = 0.f;
    }
    for (int n = 0; n < steps; ++n) {
      if (n + 1 < steps)
        fetch(next, u, (n + 1) * kScoreRows);
      else
        fetch(next, u + stride, 0);
#pragma unroll
      for (int q = 0; q < kScoreRows; ++q) {
        const float2 f = fin[n * kScoreRows + q < rows ? n * kScoreRows + q : 0];
#pragma unroll
        for (int c = 0; c < kScoreKeys; ++c) {
          const float w = dev::ex2(y[q][c] - f.x) * f.y;
          sum[c] += y[q][c] == -INFINITY ? 0.f : w;   // -inf: the row does not see the key
        }
      }
#pragma unroll
      for (int q = 0; q < kScoreRows; ++q)
#pragma unroll
        for (int c = 0; c < kScoreKeys; ++c) y[q][c] = next[q][c];
    }
#pragma unroll
    for (int c = 0; c < kScoreKeys; ++c) {
      const int at = u + (int)threadIdx.x + c * kThreads;
      if (at < list.total) dst[list.key(at)] = old[c] + sum[c];
    }
    u += stride;
  }
}

}  // namespace

cudaError_t launch_cache_finish(const FinishArgs& args, cudaStream_t st) {
  FinishArgs a = args;
  const int64_t rows = (int64_t)a.batch * a.h_kv * a.group * a.n_q;
  const int64_t per_cta = 8 / a.warps_per_row;
  const int64_t out_ctas = (rows + per_cta - 1) / per_cta;
  int64_t score_ctas = 0;
  if (a.logits != nullptr) {
    const int64_t most = (int64_t)a.sinks + a.window + a.n_q - 1;
    const int64_t keys = most < a.n_k ? most : a.n_k;
    score_ctas = (keys + kThreads * kScoreKeys - 1) / (kThreads * kScoreKeys);
    // about four CTAs per SM, each going through its share of a unit's keys:
    // the row statistics that every CTA computes are a few us
    const int64_t most_ctas = 592 / ((int64_t)a.batch * a.h_kv);
    score_ctas = score_ctas < most_ctas ? score_ctas : (most_ctas > 1 ? most_ctas : 1);
  }
  const int64_t grid = out_ctas + score_ctas * a.batch * a.h_kv;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  a.out_ctas = (int)out_ctas;
  a.score_ctas = (int)score_ctas;
  return launch_kernel(a.fp32 ? cache_finish_kernel<float> : cache_finish_kernel<__nv_bfloat16>, (unsigned)grid, kThreads, 0,
                       st, true, a);
}

}  // namespace crisp
