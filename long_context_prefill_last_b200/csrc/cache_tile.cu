// Attention over a key/value cache on CUDA cores (FFMA, fp32 accumulation):
// the fp32 path of the window, scored and shared-prefix operators. For query
// row r at position p and the keys j it sees (0 <= j <= p, and j < sinks or
// j > p - window):
//     o_r = sum_j 2^(x_rj - m_r) v_j / l_r,   x_rj = scale * log2(e) * q_r . k_j
// with the running maximum m and sum l carried over key tiles in one pass.
//
// One CTA per (unit, 64-row block, split of the key list), 256 threads as
// 16 x 16: thread (ty, tx) holds logits of rows 4 ty .. 4 ty + 3 against keys
// tx + 16 j, and output columns 4 tx .. 4 tx + 3 and 64 + 4 tx .. of the same
// rows. A row of a unit is a (token, head of the group) pair, so a key tile is
// read once for all query heads that share it.
//
// Bound: FMA and shared memory (12 wavefronts of loads per 32 packed FMA in the
// logits, 20 per 32 in the output). Measured: 4096 tokens of one head through a
// 512-key window in 50 us, 62% of the FMA pipe on SMs that hold two CTAs.
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace crisp {
namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kPitch = kHeadDim + 4;      // floats per staged Q or K row: 16 rows x 16 bytes fall in 2 wavefronts
constexpr int kPPitch = kRows + 4;        // floats per key of the staged probabilities
constexpr int kHold = 64;                 // tiles whose sums the registers hold, before they go to what is held
constexpr int kSmem = (2 * kRows * kPitch + kKeys * kHeadDim) * 4;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// HOLD: a CTA may take more than kHold key tiles. Without, the code that this
// needs is left out (4096 tokens through a 512-key window: 60 us, 61.4 with).
template <bool HOLD>
__global__ void __launch_bounds__(256, 2) cache_tile_kernel(CacheArgs a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ float2 held[kRows];   // maximum and sum of a row's held results
  float* qs = sm;
  float* ks = qs + kRows * kPitch;
  float* vs = ks + kKeys * kPitch;
  float* ps = ks;   // the probabilities take the K tile's place once the logits are done
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ty = tid >> 4, tx = tid & 15;
  const int split = blockIdx.x % a.splits;
  const int job = blockIdx.x / a.splits;
  const int rb = job % a.blocks, unit = job / a.blocks;
  const int b = unit / a.h_kv, g = unit - b * a.h_kv;
  const int r0 = rb * kRows;
  const int len = dev::cache_len(a, b);
  const int last = min(r0 + kRows, a.rows) - 1;
  // with logits kept, list indices have to be those of the whole unit
  const KeyList list = a.prefix || a.logits != nullptr ? dev::unit_keys(a, len, 0, a.n_q - 1)
                                                       : dev::unit_keys(a, len, r0 / a.group, last / a.group);
  const int tiles = (list.total + kKeys - 1) / kKeys;
  const int t0 = (int)((int64_t)tiles * split / a.splits), t1 = (int)((int64_t)tiles * (split + 1) / a.splits);

  // queries, scaled; rows past the unit's end are zero
  for (int r = warp; r < kRows; r += 8) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < a.rows) {
      const dev::Row w = dev::unit_row(a, b, g, r0 + r);
      x = load4(static_cast<const float*>(a.q) + w.b * a.sq.seq + w.h * a.sq.head + w.i * a.sq.token + lane * 4);
    }
    *reinterpret_cast<float4*>(qs + r * kPitch + lane * 4) = x;
  }
  int pos[4];
  float m[4], l[4];
  float4 o[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    pos[i] = r < a.rows ? dev::row_pos(a, len, dev::unit_row(a, b, g, r).i) : -1;
    m[i] = -INFINITY;
    l[i] = 0.f;
    o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float* kp = static_cast<const float*>(a.k) + b * a.sk.seq + g * a.sk.head + lane * 4;
  const float* vp = static_cast<const float*>(a.v) + b * a.sv.seq + g * a.sv.head + lane * 4;

  const uint32_t ks_at = dev::smem_u32(ks) + lane * 16, vs_at = dev::smem_u32(vs) + lane * 16;
  const uint64_t policy = dev::evict_normal();   // row blocks share the keys through L2
  // Long key lists: sums of up to kHold tiles are collected in registers and then
  // added to those held in the destination row (one long running sum's roundings
  // fall to one side where tiles are alike: 2048 tiles, 2e-5).
  auto dest = [&](int i) -> float* {
    const int r = r0 + ty * 4 + i;
    if (a.part_o != nullptr) return a.part_o + (((int64_t)job * a.splits + split) * kRows + ty * 4 + i) * kHeadDim;
    const dev::Row w = dev::unit_row(a, b, g, r);
    return static_cast<float*>(a.out) + w.b * a.so.seq + w.h * a.so.head + w.i * a.so.token;
  };
  auto add_held = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (r0 + ty * 4 + i >= a.rows) continue;
      const float2 h = held[ty * 4 + i];
      const float f = exp2f(h.x - (m[i] == -INFINITY ? 0.f : m[i]));
      const float* src = dest(i);
      l[i] = fmaf(h.y, f, l[i]);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float4 x = load4(src + n * 64 + tx * 4);
        o[i][n].x = fmaf(x.x, f, o[i][n].x), o[i][n].y = fmaf(x.y, f, o[i][n].y);
        o[i][n].z = fmaf(x.z, f, o[i][n].z), o[i][n].w = fmaf(x.w, f, o[i][n].w);
      }
    }
    __syncwarp();   // a row's 16 threads have read its statistics
  };
  for (int t = t0; t < t1; ++t) {
    if (HOLD && t > t0 && (t - t0) % kHold == 0) {
      if (t - t0 > kHold) add_held();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r0 + ty * 4 + i < a.rows) {
          store4(dest(i) + tx * 4, o[i][0]);
          store4(dest(i) + 64 + tx * 4, o[i][1]);
          held[ty * 4 + i] = make_float2(m[i], l[i]);   // the same from all 16 threads
        }
        l[i] = 0.f;
        o[i][0] = o[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      __syncwarp();
    }
    __syncthreads();
    // keys first; the values land while the logits are computed
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int c = i * 8 + warp, u = t * kKeys + c;
        const bool in = u < list.total;
        const int64_t j = in ? list.key(u) : 0;
        if (which == 0)
          dev::cp16(ks_at + c * kPitch * 4, kp + j * a.sk.token, in ? 16u : 0u, policy);
        else
          dev::cp16(vs_at + c * kHeadDim * 4, vp + j * a.sv.token, in ? 16u : 0u, policy);
      }
      dev::cp_commit();
    }
    dev::cp_wait<1>();
    __syncthreads();
    // logits: two partial sums (even and odd pairs of dims) per entry
    uint64_t acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll 4
    for (int d = 0; d < kHeadDim; d += 4) {
      ulonglong2 qv[4], kv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const ulonglong2*>(qs + (ty * 4 + i) * kPitch + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * j) * kPitch + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = dev::f2_fma(qv[i].x, kv[j].x, acc[i][j]);
          acc[i][j] = dev::f2_fma(qv[i].y, kv[j].y, acc[i][j]);
        }
    }
    float x[4][4], tmax[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tmax[i] = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float s0, s1;
        dev::f2_unpack(acc[i][j], s0, s1);
        const int u = t * kKeys + tx + 16 * j, key = list.key(u);
        const bool seen = u < list.total && key <= pos[i] && (key < a.sinks || key > pos[i] - a.window);
        x[i][j] = seen ? (s0 + s1) * a.scale_log2 : -INFINITY;
        tmax[i] = fmaxf(tmax[i], x[i][j]);
      }
    }
    if (a.logits != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty * 4 + i;
        if (r < a.rows) {
          float* dst = a.logits + ((int64_t)unit * a.rows + r) * a.pitch + t * kKeys;
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[tx + 16 * j] = x[i][j];
        }
      }
    }
    dev::cp_wait<0>();
    __syncthreads();   // the K tile has been read by everyone; the values are there
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) tmax[i] = fmaxf(tmax[i], __shfl_xor_sync(0xffffffffu, tmax[i], w));
      const float mn = fmaxf(m[i], tmax[i]);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = exp2f(x[i][j] - base);
        sum += x[i][j];
      }
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * f + sum;
      o[i][0].x *= f, o[i][0].y *= f, o[i][0].z *= f, o[i][0].w *= f;
      o[i][1].x *= f, o[i][1].y *= f, o[i][1].z *= f, o[i][1].w *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(ps + (tx + 16 * j) * kPPitch + ty * 4) =
          make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
    __syncthreads();
    // the tile's own sum first, then added to the running one: the rounding
    // error of a long sum grows with the number of tiles, not of keys
    uint64_t s2[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = 0ull;
#pragma unroll 4
    for (int c = 0; c < kKeys; ++c) {
      const float4 p = *reinterpret_cast<const float4*>(ps + c * kPPitch + ty * 4);
      const ulonglong2 v0 = *reinterpret_cast<const ulonglong2*>(vs + c * kHeadDim + tx * 4);
      const ulonglong2 v1 = *reinterpret_cast<const ulonglong2*>(vs + c * kHeadDim + 64 + tx * 4);
      const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t pp = dev::f2_pack(pr[i], pr[i]);
        s2[i][0] = dev::f2_fma(pp, v0.x, s2[i][0]);
        s2[i][1] = dev::f2_fma(pp, v0.y, s2[i][1]);
        s2[i][2] = dev::f2_fma(pp, v1.x, s2[i][2]);
        s2[i][3] = dev::f2_fma(pp, v1.y, s2[i][3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float e0, e1, e2, e3;
        dev::f2_unpack(s2[i][2 * h], e0, e1);
        dev::f2_unpack(s2[i][2 * h + 1], e2, e3);
        o[i][h].x += e0, o[i][h].y += e1, o[i][h].z += e2, o[i][h].w += e3;
      }
  }
  if (HOLD && t1 - t0 > kHold) add_held();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= a.rows) continue;
    if (a.part_o != nullptr) {
      const int64_t at = ((int64_t)job * a.splits + split) * kRows + ty * 4 + i;
      store4(a.part_o + at * kHeadDim + tx * 4, o[i][0]);
      store4(a.part_o + at * kHeadDim + 64 + tx * 4, o[i][1]);
      if (tx == 0) a.part_ml[at] = make_float2(m[i], l[i]);
    } else {
      const dev::Row w = dev::unit_row(a, b, g, r);
      const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);   // no key: 0; NaN stays NaN
      float* dst = static_cast<float*>(a.out) + w.b * a.so.seq + w.h * a.so.head + w.i * a.so.token;
      store4(dst + tx * 4, make_float4(o[i][0].x * inv, o[i][0].y * inv, o[i][0].z * inv, o[i][0].w * inv));
      store4(dst + 64 + tx * 4, make_float4(o[i][1].x * inv, o[i][1].y * inv, o[i][1].z * inv, o[i][1].w * inv));
    }
  }
}

}  // namespace

cudaError_t launch_cache_tile(const CacheArgs& a, const AttnPlan& p, cudaStream_t st) {
  const int64_t grid = (int64_t)p.units * p.blocks * p.splits;
  if (grid <= 0 || grid > INT32_MAX) return cudaErrorInvalidValue;
  const auto kernel = p.run > kHold ? cache_tile_kernel<true> : cache_tile_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)grid, 256, kSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace crisp
