// Decode attention over a key/value cache, fp32 (FFMA): up to 16 query rows
// per job (tokens of a draft x query heads of the group) against a long key
// list, in one pass with running softmax statistics.
//
// Bound: HBM. A key costs 1024 bytes per key/value head, 42 cycles of an SM's
// share of the bandwidth; R rows cost 2 R cycles of FMA and about 2 (R + 4) of
// shared memory, so up to 16 rows stay below that. The job list, the ring that
// runs on across jobs and the partial results are those of cache_decode.cu.
//
// Per tile of 32 keys, 128 threads: four lanes take a key's logits, a quarter
// of the dims each, for all rows (their 16-byte steps are rotated against one
// another so that the quarters fall in different banks); a warp takes a row's
// softmax, a lane per key; then a thread takes an output column for all rows.
//
// Measured: 2 sequences of 4096 and 8191 tokens, 8 heads of their own keys: 101
// MB in 27 us (3.7 TB/s; 20 tiles per CTA).
// The compensation of the running sums costs 0.5 us of a call's 32.5.
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace crisp {
namespace {

using dev::cp16;
using dev::cp_commit;
using dev::cp_wait;

constexpr int kKeys = 32;
constexpr int kStages = 3;
constexpr int kThreads = 128;
constexpr uint32_t kKPitch = kHeadDim * 4 + 16;   // bytes: eight keys' 16-byte pieces fall in different banks
constexpr uint32_t kVPitch = kHeadDim * 4;
constexpr uint32_t OFF_V = kKeys * kKPitch;
constexpr uint32_t kStageBytes = kKeys * (kKPitch + kVPitch);
constexpr uint32_t OFF_Q = kStages * kStageBytes;

template <int R>
struct Layout {
  static constexpr uint32_t x = OFF_Q + R * kHeadDim * 4;        // float[R][kKeys + 1] logits
  static constexpr uint32_t p = (x + R * (kKeys + 1) * 4 + 15) / 16 * 16;   // float[kKeys][R] weights
  static constexpr uint32_t f = p + kKeys * R * 4;               // float[R] factors of the running sums
  static constexpr uint32_t cum = f + R * 4;                     // int[batch + 1]
};

template <int R>
__global__ void __launch_bounds__(kThreads, 2) cache_decode_fp32_kernel(CacheArgs a) {
  using L = Layout<R>;
  constexpr int RW = R / 4;   // rows of a warp's softmax
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan_tmp[32];
  float* qs = reinterpret_cast<float*>(smem + OFF_Q);
  float* xs = reinterpret_cast<float*>(smem + L::x);
  float* ps = reinterpret_cast<float*>(smem + L::p);
  float* fs = reinterpret_cast<float*>(smem + L::f);
  int* cum = reinterpret_cast<int*>(smem + L::cum);
  const uint32_t sbase = dev::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  dev::launch_dependents();
  const bool bad = dev::stair_scan(a.kv_len, a.batch, a.n_keys, a.n_q, a.window, a.sinks, a.prefix != 0, kKeys, cum,
                                   scan_tmp);
  if (blockIdx.x == 0 && tid == 0) {
    if (a.sets_status) a.status[kStatusCode] = 0;
    if (a.sets_status || bad) a.status[kStatusLen] = bad ? CRISP_ERR_INVALID_ARG : 0;
  }
  const int per_seq = a.h_kv * a.blocks;
  dev::Place ld;
  const int n_all = dev::stair_start(a, cum, ld);
  if (n_all == 0) return;
  dev::Place cp = ld;

  // loads, kStages - 1 tiles ahead, across jobs: a warp copies a key row per step
  const float *kp, *vp;
  auto bind = [&]() {
    const int g = ld.jj / a.blocks;
    kp = static_cast<const float*>(a.k) + ld.b * a.sk.seq + g * a.sk.head + lane * 4;
    vp = static_cast<const float*>(a.v) + ld.b * a.sv.seq + g * a.sv.head + lane * 4;
  };
  bind();
  const uint64_t policy = dev::evict_first();
  int loaded = 0;
  auto load = [&]() {
    if (loaded < n_all) {
      if (ld.t == ld.T) {
        ld.next_job(a, cum, per_seq);
        bind();
      }
      const uint32_t dst = sbase + (loaded % kStages) * kStageBytes + lane * 16;
#pragma unroll
      for (int i = 0; i < kKeys / 4; ++i) {
        const int c = i * 4 + warp, u = ld.t * kKeys + c;
        const bool in = u < ld.list.total;
        const int64_t j = in ? ld.list.key(u) : 0;
        cp16(dst + c * kKPitch, kp + j * a.sk.token, in ? 16u : 0u, policy);
        cp16(dst + OFF_V + c * kVPitch, vp + j * a.sv.token, in ? 16u : 0u, policy);
      }
      ++ld.t;
      ++loaded;
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load();

  int done = 0;
  while (done < n_all) {
    const int run = n_all - done < cp.T - cp.t ? n_all - done : cp.T - cp.t;   // tiles of this job here
    const int g = cp.jj / a.blocks, rb = cp.jj - g * a.blocks;
    const int unit = cp.b * a.h_kv + g;
    const KeyList list = cp.list;
    // queries (rows past the unit's end are zero); the last readers of the
    // previous job's passed the barrier after its last logits
    for (int r = warp; r < R; r += 4) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (rb * R + r < a.rows) {
        const dev::Row w = dev::unit_row(a, cp.b, g, rb * R + r);
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + w.b * a.sq.seq + w.h * a.sq.head +
                                             w.i * a.sq.token + lane * 4);
      }
      *reinterpret_cast<float4*>(qs + r * kHeadDim + lane * 4) = x;
    }
    int pos[RW];
    float m[RW], l[RW], lc[RW], o[R], oc[R];   // lc, oc: what the roundings of l and o have added too much
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = rb * R + i * 4 + warp;
      pos[i] = r < a.rows ? dev::row_pos(a, cp.len, dev::unit_row(a, cp.b, g, r).i) : -1;
      m[i] = -INFINITY;
      l[i] = lc[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) o[r] = oc[r] = 0.f;

    for (int it = 0; it < run; ++it) {
      cp_wait<kStages - 2>();
      __syncthreads();
      load();
      const int t = cp.t + it;
      const uint8_t* stage = smem + ((done + it) % kStages) * kStageBytes;
      {   // logits
        const int key = warp * 8 + (lane >> 2), part = lane & 3;
        const float* kr = reinterpret_cast<const float*>(stage + key * kKPitch) + part * 32;
        const float* qr = qs + part * 32;
        uint64_t acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = 0ull;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int d = ((s + 2 * part) & 7) * 4;
          const ulonglong2 kv = *reinterpret_cast<const ulonglong2*>(kr + d);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qr + r * kHeadDim + d);
            acc[r] = dev::f2_fma(qv.x, kv.x, acc[r]);
            acc[r] = dev::f2_fma(qv.y, kv.y, acc[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float s0, s1;
          dev::f2_unpack(acc[r], s0, s1);
          float x = s0 + s1;
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          x += __shfl_xor_sync(0xffffffffu, x, 2);
          if (part == (r & 3)) xs[r * (kKeys + 1) + key] = x;
        }
      }
      __syncthreads();
      // softmax: lane = key
      const int u = t * kKeys + lane, key = list.key(u);
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r = i * 4 + warp;
        const bool seen = u < list.total && key <= pos[i] && (key < a.sinks || key > pos[i] - a.window);
        const float x = seen ? xs[r * (kKeys + 1) + lane] * a.scale_log2 : -INFINITY;
        if (a.logits != nullptr && rb * R + r < a.rows)
          a.logits[((int64_t)unit * a.rows + rb * R + r) * a.pitch + u] = x;
        float mx = x;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[i] - base), p = exp2f(x - base);
        m[i] = mn;
        float sum = p;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        // the running sums are compensated (Kahan): where tiles are alike a plain
        // sum's roundings fall to one side (4096 tiles: 4e-5), in scores as in outputs
        const float y = fmaf(-lc[i], f, sum), z = fmaf(l[i], f, y);
        lc[i] = fmaf(-l[i], f, z) - y;
        l[i] = z;
        ps[lane * R + r] = p;
        if (lane == 0) fs[r] = f;
      }
      __syncthreads();
      // output: the tile's own sum first, then added to the running one
      const float* vc = reinterpret_cast<const float*>(stage + OFF_V) + tid;
      float s2[R];
#pragma unroll
      for (int r = 0; r < R; ++r) s2[r] = 0.f;
#pragma unroll 8
      for (int c = 0; c < kKeys; ++c) {
        const float v = vc[c * kHeadDim];
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 p = *reinterpret_cast<const float4*>(ps + c * R + r);
          s2[r] = fmaf(p.x, v, s2[r]);
          s2[r + 1] = fmaf(p.y, v, s2[r + 1]);
          s2[r + 2] = fmaf(p.z, v, s2[r + 2]);
          s2[r + 3] = fmaf(p.w, v, s2[r + 3]);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = fs[r], y = fmaf(-oc[r], f, s2[r]), z = fmaf(o[r], f, y);
        const float e = fmaf(-o[r], f, z) - y;
        oc[r] = e == e ? e : 0.f;   // an infinite sum stays one
        o[r] = z;
      }
    }
    const int64_t slot = (int64_t)blockIdx.x + (int64_t)cp.b * per_seq + cp.jj;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (rb * R + r < a.rows) a.part_o[(slot * a.block + r) * kHeadDim + tid] = o[r];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = i * 4 + warp;
      if (lane == 0 && rb * R + r < a.rows) a.part_ml[slot * a.block + r] = make_float2(m[i], l[i]);
    }
    if (tid == 0) {
      int* entry = reinterpret_cast<int*>(a.table + cp.b * per_seq + cp.jj);
      if (cp.t == 0) entry[0] = blockIdx.x;
      if (cp.t + run == cp.T) entry[1] = blockIdx.x;
    }
    done += run;
    cp.t += run;
    if (cp.t == cp.T && done < n_all) cp.next_job(a, cum, per_seq);
  }
  if (a.chained) dev::wait_for_launches();
}

template <int R>
cudaError_t launch(const CacheArgs& a, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache_decode_fp32_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Layout<R>::cum + 4 * (kMaxBatch + 1));
  if (e != cudaSuccess) return e;
  return launch_kernel(cache_decode_fp32_kernel<R>, a.ctas, kThreads, Layout<R>::cum + 4 * (a.batch + 1), st,
                       a.chained != 0, a);
}

}  // namespace

cudaError_t launch_cache_decode_fp32(const CacheArgs& a, const AttnPlan& p, cudaStream_t st) {
  if (p.block == 4) return launch<4>(a, st);
  if (p.block == 8) return launch<8>(a, st);
  return launch<16>(a, st);
}

}  // namespace crisp
