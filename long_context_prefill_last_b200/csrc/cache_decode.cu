// Decode attention over a key/value cache, bf16: a few query rows per
// key/value head (tokens of a draft x query heads of the group, up to 64)
// against a long key list, in one pass with running softmax statistics.
//
// Bound: HBM. A key costs 512 bytes per key/value head and 4 * 128 FLOP per
// row, so at 64 rows the legacy tensor instruction (m16n8k16, operands in
// registers) still keeps up with memory, and with 4 .. 28 rows a tcgen05 tile
// of 128 rows would compute mostly padding. Keys and values come through a
// three-stage cp.async ring (64 keys x 512 bytes a stage, two CTAs per SM);
// per-row copies let the key list jump from the first keys to the window
// without a hole, and zero-fill past its end.
//
// The key tiles of all jobs (sequence, key/value head, row block) form one
// list that is dealt to the CTAs in equal runs, so a ragged batch keeps every
// SM busy however its lengths lie; the lengths are read on the device, and the
// ring runs on across jobs. Each (CTA, job) pair leaves one partial result,
// joined by cache_merge.cu.
//
// 4 warps: RT = 1, 2 or 4 of them along the rows (16 each), KW = 4 / RT along
// the keys of a tile, each with its own statistics and output: a run leaves KW
// partial results per job, without a barrier between the warps at its end.
// Keys and values, each read once, are copied with the evict-first policy,
// which leaves the L2 cache to the logits that a scored call writes here and
// reads in its second launch.
//
// Small calls (CL): a cluster of 1 to 8 CTAs has a job to itself, each CTA a
// part of its key tiles (at most 20, so that one long sequence among short
// ones, which the flat list would deal to every SM, costs little); they join
// their results through distributed shared memory, write the output rows and
// add the scores of their own keys, in one launch (about 3 us on the GPU and 2
// on the host less than two).
//
// Measured: one token of 32 query and 8 key/value heads on 524288 tokens, 2.15
// GB of keys and values and 67 MB of logits in 326 us (6.8 TB/s); 125 MB of
// windows of 32 sequences in 27 us a call (4.7 TB/s: 3 us until the first
// copies are under way, 17 tiles per CTA).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>

#include "cache.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace crisp {
namespace {

constexpr int kKeys = 64;
constexpr int kStages = 3;
constexpr int kThreads = 128;
constexpr uint32_t kTileBytes = kKeys * kHeadDim * 2;   // K or V of one stage
constexpr uint32_t kStageBytes = 2 * kTileBytes;
constexpr uint32_t OFF_CUM = kStages * kStageBytes;      // int[batch + 1]
constexpr uint32_t smem_bytes(int batch) { return OFF_CUM + 4 * (batch + 1); }
static_assert(2 * (smem_bytes(kMaxBatch) + 1024 + 128) <= 228 * 1024, "two CTAs per SM");
// what a cluster's join keeps, over the ring: the warps' rows and statistics,
// the CTA's (read by the others), the job's final statistics
constexpr int kOPitch = kHeadDim + 4;
constexpr uint32_t OFF_WO = 0;                                   // float[4][16][kOPitch]
constexpr uint32_t OFF_WML = OFF_WO + 4 * 16 * kOPitch * 4;      // float2[4][16]
constexpr int kClusterRows = 32;                                 // rows of a cluster's job
constexpr uint32_t OFF_CO = OFF_WML + 4 * 16 * 8;                // float[kClusterRows][128]
constexpr uint32_t OFF_CML = OFF_CO + kClusterRows * kHeadDim * 4;   // float2[kClusterRows]
constexpr uint32_t OFF_FIN = OFF_CML + kClusterRows * 8;         // float2[kClusterRows]
static_assert(OFF_FIN + kClusterRows * 8 <= OFF_CUM, "the join aliases the ring");

using dev::cp16;
using dev::cp_commit;
using dev::cp_wait;
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int RT, bool CL>
__global__ void __launch_bounds__(kThreads, 2) cache_decode_kernel(CacheArgs a) {
  constexpr int KW = 4 / RT;            // warps along the keys
  constexpr int NK = kKeys / KW;        // keys of a tile per warp
  constexpr int NT = NK / 8;            // 8-key accumulator tiles per warp
  constexpr int BLOCK = 16 * RT;        // rows per job
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scan_tmp[32];
  int* cum = reinterpret_cast<int*>(smem + OFF_CUM);
  const uint32_t sbase = dev::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = warp % RT, kw = warp / RT;
  const int gq = lane >> 2, tq = lane & 3;

  dev::launch_dependents();
  const int per_seq = a.h_kv * a.blocks;                       // jobs per sequence
  dev::Place ld;
  int n_all;                                                   // tiles of this CTA
  const int rank = CL ? blockIdx.x % a.cluster : 0;
  if constexpr (CL) {
    const int job = blockIdx.x / a.cluster;
    ld.b = job / per_seq;
    ld.jj = job - ld.b * per_seq;
    ld.len = dev::clamped_len(a, ld.b);
    ld.list = dev::unit_keys(a, ld.len, 0, a.n_q - 1);
    ld.T = (ld.list.total + kKeys - 1) / kKeys;
    ld.t = ld.T * rank / a.cluster;
    n_all = ld.T * (rank + 1) / a.cluster - ld.t;
    if (blockIdx.x == 0) {
      bool bad = false;
      for (int i = tid; i < a.batch; i += kThreads) dev::clamp_len(a.kv_len, i, a.n_keys, &bad);
      bad = __syncthreads_or(bad);
      if (tid == 0) {
        a.status[kStatusCode] = 0;
        a.status[kStatusLen] = bad ? CRISP_ERR_INVALID_ARG : 0;
      }
    }
  } else {
    const bool bad = dev::stair_scan(a.kv_len, a.batch, a.n_keys, a.n_q, a.window, a.sinks, a.prefix != 0, kKeys, cum,
                                     scan_tmp);
    if (blockIdx.x == 0 && tid == 0) {
      if (a.sets_status) a.status[kStatusCode] = 0;
      if (a.sets_status || bad) a.status[kStatusLen] = bad ? CRISP_ERR_INVALID_ARG : 0;
    }
    n_all = dev::stair_start(a, cum, ld);
    if (n_all == 0) return;
  }
  dev::Place cp = ld;

  // The loads run kStages - 1 tiles ahead of the arithmetic, across jobs.
  const int lrow = tid >> 4, lchunk = tid & 15;
  const uint64_t policy = dev::evict_first();
  const char *kp, *vp;
  auto bind = [&]() {
    const int g = ld.jj / a.blocks;
    kp = static_cast<const char*>(a.k) + (ld.b * a.sk.seq + g * a.sk.head) * 2 + lchunk * 16;
    vp = static_cast<const char*>(a.v) + (ld.b * a.sv.seq + g * a.sv.head) * 2 + lchunk * 16;
  };
  // the next job's queries towards the L2 cache, two tiles before they are needed
  auto fetch_q = [&]() {
    const int g = ld.jj / a.blocks, r = (ld.jj - g * a.blocks) * BLOCK + (tid >> 1);
    if ((tid >> 1) < BLOCK && r < a.rows) {
      const dev::Row w = dev::unit_row(a, ld.b, g, r);
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const __nv_bfloat16*>(a.q) + w.b * a.sq.seq +
                                                     w.h * a.sq.head + w.i * a.sq.token + (tid & 1) * 64));
    }
  };
  bind();
  int loaded = 0;
  auto load = [&]() {
    if (loaded < n_all) {
      if (ld.t == ld.T) {
        ld.next_job(a, cum, per_seq);
        bind();
        fetch_q();
      }
      const uint32_t dst = sbase + (loaded % kStages) * kStageBytes + lrow * 256 + ((lchunk ^ lrow) << 4);
#pragma unroll
      for (int i = 0; i < kKeys / 8; ++i) {
        const int u = ld.t * kKeys + i * 8 + lrow;
        const bool in = u < ld.list.total;
        const int64_t j = in ? ld.list.key(u) : 0;
        cp16(dst + i * 8 * 256, kp + j * a.sk.token * 2, in ? 16u : 0u, policy);
        cp16(dst + kTileBytes + i * 8 * 256, vp + j * a.sv.token * 2, in ? 16u : 0u, policy);
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
    const int r0 = rb * BLOCK + rt * 16;                        // this warp's first row
    const KeyList list = cp.list;

    // Q fragments (rows past the unit's end are zero) and the rows' positions
    uint32_t qf[8][4];
    int pos[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = r0 + half * 8 + gq;
      const bool in = r < a.rows;
      const dev::Row w = dev::unit_row(a, cp.b, g, in ? r : 0);
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + w.b * a.sq.seq +
                                                             w.h * a.sq.head + w.i * a.sq.token) + tq;
      pos[half] = in ? dev::row_pos(a, cp.len, w.i) : -1;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qf[ks][half] = in ? qp[ks * 8] : 0u;
        qf[ks][2 + half] = in ? qp[ks * 8 + 4] : 0u;
      }
    }
    float o[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lc[2] = {0.f, 0.f};
    const int first_pos = a.prefix ? (1 << 29) : cp.len - a.n_q, last_pos = a.prefix ? 0 : cp.len - 1;

    for (int it = 0; it < run; ++it) {
      cp_wait<kStages - 2>();
      __syncthreads();   // everyone's copies have landed, and the stage that is filled next has been read
      load();
      const int t = cp.t + it;
      const uint32_t ks_base = sbase + ((done + it) % kStages) * kStageBytes, vs_base = ks_base + kTileBytes;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
#pragma unroll
        for (int n2 = 0; n2 < NT / 2; ++n2) {
          const int key = kw * NK + n2 * 16 + ((lane >> 4) << 3) + (lane & 7);
          const int chunk = ks * 2 + ((lane >> 3) & 1);
          uint32_t f[4];
          ldsm4(ks_base + key * 256 + ((chunk ^ (key & 7)) << 4), f);
          mma16816(s[2 * n2], qf[ks], f[0], f[1]);
          mma16816(s[2 * n2 + 1], qf[ks], f[2], f[3]);
        }
      // scaled logits; unseen keys get -inf. Tiles whose every key every row sees skip the tests.
      const int u_last = t * kKeys + kKeys - 1;
      const int wu = t * kKeys > list.se ? t * kKeys : list.se;    // first entry of the window's part
      const bool whole = u_last < list.total && list.key(u_last) <= first_pos &&
                         (u_last < list.se || list.key(wu) > last_pos - a.window);
      float tmax[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = s[n][e] * a.scale_log2;
          if (!whole) {
            const int u = t * kKeys + kw * NK + n * 8 + tq * 2 + (e & 1), key = list.key(u), p = pos[e >> 1];
            const bool seen = u < list.total && key <= p && (key < a.sinks || key > p - a.window);
            y = seen ? y : -INFINITY;
          }
          s[n][e] = y;
          tmax[e >> 1] = fmaxf(tmax[e >> 1], y);
        }
      if (a.logits != nullptr) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = r0 + half * 8 + gq;
          if (r < a.rows) {
            float* dst = a.logits + ((int64_t)unit * a.rows + r) * a.pitch + t * kKeys + kw * NK + tq * 2;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              *reinterpret_cast<float2*>(dst + n * 8) = make_float2(s[n][2 * half], s[n][2 * half + 1]);
          }
        }
      }
      float base[2], f[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        tmax[half] = fmaxf(tmax[half], __shfl_xor_sync(0xffffffffu, tmax[half], 1));
        tmax[half] = fmaxf(tmax[half], __shfl_xor_sync(0xffffffffu, tmax[half], 2));
        const float mn = fmaxf(m[half], tmax[half]);
        base[half] = mn == -INFINITY ? 0.f : mn;
        f[half] = dev::ex2(m[half] - base[half]);
        m[half] = mn;
      }
      if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
        l[0] *= f[0], lc[0] *= f[0];
        l[1] *= f[1], lc[1] *= f[1];
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= f[0];
          o[n][1] *= f[0];
          o[n][2] *= f[1];
          o[n][3] *= f[1];
        }
      }
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = dev::ex2(s[n][e] - base[e >> 1]);
          part[e >> 1] += s[n][e];
        }
      // the running sum is compensated (Kahan): scores need it to a few 2^-24
      // after thousands of tiles
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float y = part[half] - lc[half], z = l[half] + y;
        lc[half] = (z - l[half]) - y;
        l[half] = z;
      }
      // weights rounded to bf16 for the product with V (fp32 accumulation), as the
      // tensor instruction takes them: a second product with their remainders would
      // double the work for 0.4e-3 of the error; l keeps them in fp32
#pragma unroll
      for (int k16 = 0; k16 < NT / 2; ++k16) {
        const uint32_t pf[4] = {dev::pack_bf16x2(s[2 * k16][0], s[2 * k16][1]),
                                dev::pack_bf16x2(s[2 * k16][2], s[2 * k16][3]),
                                dev::pack_bf16x2(s[2 * k16 + 1][0], s[2 * k16 + 1][1]),
                                dev::pack_bf16x2(s[2 * k16 + 1][2], s[2 * k16 + 1][3])};
        const int key = kw * NK + k16 * 16 + (lane & 15);
#pragma unroll
        for (int d2 = 0; d2 < 8; ++d2) {
          const int chunk = d2 * 2 + (lane >> 4);
          uint32_t vf[4];
          ldsm4_t(vs_base + key * 256 + ((chunk ^ (key & 7)) << 4), vf);
          mma16816(o[2 * d2], pf, vf[0], vf[1]);
          mma16816(o[2 * d2 + 1], pf, vf[2], vf[3]);
        }
      }
    }

#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    }
    if constexpr (CL) {   // the job's only run here
      __syncthreads();    // the ring has been read
      float* wo = reinterpret_cast<float*>(smem + OFF_WO) + (warp * 16 + gq) * kOPitch + tq * 2;
      float2* wml = reinterpret_cast<float2*>(smem + OFF_WML) + warp * 16 + gq;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int n = 0; n < 16; ++n)
          *reinterpret_cast<float2*>(wo + half * 8 * kOPitch + n * 8) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
        if (tq == 0) wml[half * 8] = make_float2(m[half], l[half]);
      }
      break;
    }
    const int64_t slot = ((int64_t)blockIdx.x + (int64_t)cp.b * per_seq + cp.jj) * KW + kw;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (r0 + half * 8 + gq >= a.rows) continue;
      const int64_t at = slot * a.block + rt * 16 + half * 8 + gq;
      float* dst = a.part_o + at * kHeadDim + tq * 2;
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * half], o[n][2 * half + 1]);
      if (tq == 0) a.part_ml[at] = make_float2(m[half], l[half]);
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
  if constexpr (CL) {
    const cg::cluster_group cluster = cg::this_cluster();
    const float* wo = reinterpret_cast<const float*>(smem + OFF_WO);
    const float2* wml = reinterpret_cast<const float2*>(smem + OFF_WML);
    float* co = reinterpret_cast<float*>(smem + OFF_CO);
    float2* cml = reinterpret_cast<float2*>(smem + OFF_CML);
    float2* fin = reinterpret_cast<float2*>(smem + OFF_FIN);
    __syncthreads();
    const int g = ld.jj;
    auto put = [&](int r, float o) {
      const dev::Row w = dev::unit_row(a, cp.b, g, r);
      static_cast<__nv_bfloat16*>(a.out)[w.b * a.so.seq + w.h * a.so.head + w.i * a.so.token + tid] = __float2bfloat16_rn(o);
    };
    // 1 / L; 0 for a row that sees no key; NaN stays NaN
    auto inverse = [](float L) { return L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L); };
    // the CTA's result: its warps joined, a thread per column
#pragma unroll 4
    for (int r = 0; r < a.rows; ++r) {
      float M = -INFINITY, L = 0.f, O = 0.f;
      if (n_all > 0) {
        const int w0 = (r >> 4) * 16 + (r & 15);
#pragma unroll
        for (int c = 0; c < KW; ++c) M = fmaxf(M, wml[w0 + RT * c * 16].x);
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int c = 0; c < KW; ++c) {
          const float2 ml = wml[w0 + RT * c * 16];
          const float f = dev::ex2(ml.x - base);
          L += f * ml.y;
          O += f * wo[(w0 + RT * c * 16) * kOPitch + tid];
        }
      }
      if (a.cluster == 1) {
        put(r, O * inverse(L));
        if (tid == 0) fin[r] = make_float2(M == -INFINITY ? 0.f : M, inverse(L));
      } else {
        co[r * kHeadDim + tid] = O;
        if (tid == 0) cml[r] = make_float2(M, L);
      }
    }
    if (a.cluster > 1) {
      cluster.sync();
      // the job's: every CTA needs every row's statistics, and writes its share of the rows
      for (int r = tid; r < a.rows; r += kThreads) {
        float2 ml[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          ml[k] = k < a.cluster ? *cluster.map_shared_rank(cml + r, k) : make_float2(-INFINITY, 0.f);
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) M = fmaxf(M, ml[k].x);
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < 8; ++k) L += dev::ex2(ml[k].x - base) * ml[k].y;
        fin[r] = make_float2(base, inverse(L));
      }
      __syncthreads();
#pragma unroll 2
      for (int r = rank; r < a.rows; r += a.cluster) {
        float x[8], f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = k < a.cluster ? *cluster.map_shared_rank(co + r * kHeadDim + tid, k) : 0.f;
          f[k] = k < a.cluster ? dev::ex2(cluster.map_shared_rank(cml + r, k)->x - fin[r].x) : 0.f;
        }
        float O = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) O += f[k] * x[k];
        put(r, O * fin[r].y);
      }
    } else {
      __syncthreads();   // fin
    }
    if (a.logits != nullptr) {
      // scores of this CTA's keys, whose logits it wrote itself
      const int unit = cp.b * a.h_kv + g;
      const int t0 = cp.T * rank / a.cluster, end = min((t0 + n_all) * kKeys, cp.list.total);
      float* score = a.score + (int64_t)unit * a.n_keys;
      for (int u = t0 * kKeys + tid; u < end; u += kThreads) {
        const float* x = a.logits + (int64_t)unit * a.rows * a.pitch + u;
        float* dst = score + cp.list.key(u);
        const float old = *dst;
        float sum = 0.f;
#pragma unroll 4
        for (int r = 0; r < a.rows; ++r) {
          const float y = x[r * a.pitch];
          const float p = dev::ex2(y - fin[r].x) * fin[r].y;
          sum += y == -INFINITY ? 0.f : p;   // -inf: the row does not see the key
        }
        *dst = old + sum;
      }
    }
    if (a.cluster > 1) cluster.sync();   // nobody leaves while its results may be read
  }
}

template <int RT>
cudaError_t launch(const CacheArgs& a, const AttnPlan& p, cudaStream_t st) {
  if constexpr (16 * RT <= kClusterRows) {
    if (p.cluster > 0) {
      const auto kernel = cache_decode_kernel<RT, true>;
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(1));
      if (e != cudaSuccess) return e;
      return launch_clusters(kernel, (unsigned)(p.units * p.cluster), p.cluster, kThreads, smem_bytes(1), st, false, a);
    }
  }
  if (p.cluster > 0) return cudaErrorInvalidValue;
  const auto kernel = cache_decode_kernel<RT, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kMaxBatch));
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, a.ctas, kThreads, smem_bytes(a.batch), st, a.chained != 0, a);
}

}  // namespace

cudaError_t launch_cache_decode(const CacheArgs& a, const AttnPlan& p, cudaStream_t st) {
  if (p.block == 16) return launch<1>(a, p, st);
  if (p.block == 32) return launch<2>(a, p, st);
  return launch<4>(a, p, st);
}

}  // namespace crisp
