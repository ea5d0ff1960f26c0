// Attention over a key/value cache on the 5th-generation tensor cores
// (tcgen05.mma, accumulators in TMEM, keys and values staged by TMA), bf16:
// prompts and appended chunks through a window, and a prefix shared by many
// rows. For query row r at position p and the keys j it sees (0 <= j <= p,
// and j < sinks or j > p - window), in one pass over the keys:
//     o_r = sum_j 2^(x_rj - m_r) v_j / l_r,   x_rj = scale * log2(e) * q_r . k_j
//
// Bound: the tensor pipe (4 * 128 FLOP per row and key) beside the softmax's
// issue slots. One CTA takes one or two row tiles of a unit (A and B, up to 128
// rows each) and a range of its key tiles. A row tile is a TMA box of the query
// tensor: the group's heads x a run of tokens (x sequences, for the prefix),
// so the query heads that share a key/value head read its tiles once, and the
// keys that a CTA's rows span beyond the window are few (64 tokens at 4 heads
// a group). The same box of the output tensor takes the result. Key tiles
// start at the first key that the CTA's rows see, wherever that is: TMA boxes
// need no alignment along the tokens.
//
// A tile of at most 32 keys (a few first keys, a window's last ones) is
// narrow: 32 columns of S, two K = 16 steps of P V, and a softmax over 32
// columns.
//
// Warps, TMEM columns, register split and MMA order follow attn_tc.cu:
//   warp 0       TMA producer: Q_A, Q_B, then K (3-stage ring) and V (2-stage
//                ring; a CTA of one row tile has one stage of each); clears the
//                V rows behind the last key of a list segment, whose weights
//                are zero but whose content may be anything
//   warp 1       TMEM allocation; one elected lane issues every tcgen05.mma
//   warps 4..7   softmax of tile A, warps 8..11 of tile B (row = TMEM lane)
// TMEM: S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512) (one row tile:
// S_A [0,128), O_A [128,256)); P (bf16) over the first 64 columns of S. Issue order per key tile u:
//     S_B(u) = Q_B K_u^T,  O_A += P_A(u) V_u,  S_A(u+1) = Q_A K_{u+1}^T,  O_B += P_B(u) V_u
// S_X(u) landing means O_X already holds P_X(u-1) V, so a softmax warp may
// rescale O_X then; it does when a row's maximum grew by more than 2^8.
//
// Measured: 32768 tokens of 32 heads through a 4096-key window in 2.18 ms, 970
// TFLOP/s of seen pairs. A key tile takes a row-tile pair 3530 cycles, 2048 of
// them tensor work: a tile's softmax (1800: 1024 of MUFU, then the loads, the
// maximum and the stores) and its two products follow one another. The start
// and end of a job (set-up, first loads, the drained output) come on top: over
// a launch of 8192 tokens the tensor pipe is busy 52% of the SMs' active
// cycles, and the SMs are active 90% of the time. Starting the exponentials
// before the tile's maximum is known was slower (2.49 ms: the registers spill).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "cache.h"
#include "ptx.cuh"
#include "tmap.h"

namespace crisp {
namespace {

constexpr uint32_t kTileBytes = 128 * 128 * 2;   // a bf16 128x128 tile: two 64-column halves
constexpr uint32_t kHalfBytes = 128 * 128;       // 128 rows x 128 bytes

// What a CTA of NX row tiles (1 or 2) has.
template <int NX>
struct Cta {
  static constexpr int threads = 128 + 128 * NX;
  static constexpr int per_sm = NX == 2 ? 1 : 2;
  static constexpr int regs_launch = NX == 2 ? 168 : 128;
  static constexpr int regs_control = NX == 2 ? 64 : 40;
  static constexpr int regs_softmax = 216;
  static_assert(128 * regs_control + 128 * NX * regs_softmax <= threads * regs_launch, "register split exceeds the launch");
  static constexpr int k_stages = NX == 2 ? 3 : 1;
  static constexpr int v_stages = NX == 2 ? 2 : 1;
  static constexpr uint32_t off_q = 0;                    // A, then B
  static constexpr uint32_t off_k = NX * kTileBytes;
  static constexpr uint32_t off_v = off_k + k_stages * kTileBytes;
  static constexpr uint32_t off_bar = off_v + v_stages * kTileBytes;
  enum {
    b_kfull = 0,
    b_kempty = b_kfull + k_stages,
    b_vfull = b_kempty + k_stages,
    b_vempty = b_vfull + v_stages,
    b_vclear = b_vempty + v_stages,  // the rows behind a segment's end are zero (one arrival per tile)
    b_sfull = b_vclear + v_stages,   // [2]: S_X landed
    b_pfull = b_sfull + 2,           // [2]: P_X written (128 arrivals)
    b_done = b_pfull + 2,            // [2]: last P_X V landed
    b_q = b_done + 2,                // [2]: Q_X landed
    b_drain = b_q + 2,
    b_count = b_drain + 1
  };
  static constexpr uint32_t off_tmemptr = off_bar + 8 * b_count;
  static constexpr uint32_t off_abort = off_tmemptr + 4;
  static constexpr uint32_t smem = off_abort + 4 + 1024;   // + slack to align the base to 1024
  static_assert(per_sm * (smem + 1024) <= 228 * 1024, "shared memory budget");
  static constexpr uint32_t tmem_cols = 256 * NX;          // S_X, then O_X
  static __device__ __forceinline__ uint32_t bar(uint32_t base, int i) { return base + off_bar + 8u * i; }
};
constexpr float kRescaleLog2 = 8.f;
constexpr int kNarrow = 32;

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status,
                                          int where) {
  const bool ok = dev::mbar_wait(bar, parity, abort_flag, status, where);
  return __all_sync(0xffffffffu, ok);
}

// 4-D tiled load; x is a multiple of 64 elements.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(dst), "l"(tmap), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// 4-D tiled store; x is a multiple of 64 elements, no coordinate is negative.
__device__ __forceinline__ void tma_store_4d(uint32_t src, const void* tmap, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(tmap), "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Two K = 16 steps of D (+)= A * B, A in tensor memory (8 columns a step), B
// MN-major, 128-byte swizzled in shared memory (128 in the start-address field a step).
__device__ __forceinline__ void umma_ts2_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 r, t;\n\t.reg .b64 b;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 p0, %4, 0;\n\t"
      "setp.eq.b32 pt, %4, %4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
      "add.u32 t, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %3, pt;\n\t"
      "}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Bits lo .. hi - 1 of a 32-bit word (bounds may lie outside it).
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t skip = lo >= 32 ? 0xffffffffu : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below & ~skip;
}

// Per-row softmax state of a warp's 32 rows (one per lane).
struct SoftRow {
  float m_ref, l;
};

// One key tile of NC columns: logits from TMEM, unseen ones masked, running
// statistics, weights back to TMEM as bf16. Column c is key k0 + c: seen for
// low < c <= high or c < front, c <= high, when `part`.
template <int NC>
__device__ __forceinline__ void soft_tile(SoftRow& st, uint32_t s_col, uint32_t o_col, bool first, bool part, int low,
                                          int high, int front, float sl2, uint32_t p_bar) {
  float s[NC];
#pragma unroll
  for (int c0 = 0; c0 < NC; c0 += 32) dev::tmem_ld32(s_col + c0, reinterpret_cast<uint32_t(&)[32]>(s[c0]));
  dev::tmem_wait_ld();
  if (part) {
#pragma unroll
    for (int c0 = 0; c0 < NC; c0 += 32) {
      const uint32_t seen = (bit_range(low + 1 - c0, 32) | bit_range(0, front - c0)) & bit_range(0, high + 1 - c0);
#pragma unroll
      for (int c = 0; c < 32; ++c) s[c0 + c] = (seen & (1u << c)) != 0u ? s[c0 + c] : -INFINITY;
    }
  }
  float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int c = 4; c < NC - 4; c += 8) {
    mx[0] = dev::max3(mx[0], s[c], s[c + 1]);
    mx[1] = dev::max3(mx[1], s[c + 2], s[c + 3]);
    mx[2] = dev::max3(mx[2], s[c + 4], s[c + 5]);
    mx[3] = dev::max3(mx[3], s[c + 6], s[c + 7]);
  }
  mx[0] = dev::max3(mx[0], s[NC - 4], s[NC - 3]);
  mx[1] = dev::max3(mx[1], s[NC - 2], s[NC - 1]);
  const float tmax = fmaxf(dev::max3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
  const bool need = tmax > st.m_ref + kRescaleLog2 || (st.m_ref == -INFINITY && tmax > -INFINITY);
  const float factor = need ? dev::ex2(st.m_ref - tmax) : 1.f;   // 0 when m_ref = -inf
  if (!first && __any_sync(0xffffffffu, need)) {
    // O holds P V of every earlier tile (it completed before S landed)
#pragma unroll 1
    for (int c0 = 0; c0 < 128; c0 += 32) {
      uint32_t v[32];
      dev::tmem_ld32(o_col + c0, v);
      dev::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * factor);
      dev::tmem_st32(o_col + c0, v);
    }
  }
  if (need) {
    st.l *= factor;
    st.m_ref = tmax;
  }
  const float neg_m = st.m_ref == -INFINITY ? 0.f : -st.m_ref;
  // P = 2^(x - m), rounded to bf16, the type of V, for their product (a second
  // one with the remainders would cost half as much again; l keeps fp32); chunk c0 goes to S columns [c0/2, c0/2 + 16), already consumed
  const uint64_t scale2 = dev::f2_pack(sl2, sl2), negm2 = dev::f2_pack(neg_m, neg_m);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int c0 = 0; c0 < NC; c0 += 32) {
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int c = c0 + 2 * j;
      const uint64_t x2 = dev::f2_fma(dev::f2_pack(s[c], s[c + 1]), scale2, negm2);
      float x0, x1;
      dev::f2_unpack(x2, x0, x1);
      const float p0 = dev::ex2(x0), p1 = dev::ex2(x1);
      acc[j & 3] = dev::f2_add(acc[j & 3], dev::f2_pack(p0, p1));
      pk[j] = dev::pack_bf16x2(p0, p1);
    }
    dev::tmem_st16(s_col + (c0 >> 1), pk);
  }
  float sum[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) dev::f2_unpack(acc[j], sum[2 * j], sum[2 * j + 1]);
  dev::tmem_wait_st();
  dev::tc_fence_before();
  dev::mbar_arrive(p_bar);
  st.l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
}

enum Kind : int { kNone = 0, kWhole = 1, kPart = 2 };

// The CTA's key tiles: those of the first keys [0, se), then those of [lo, hi).
struct Sched {
  int se, lo, hi, sink_tiles, t0, t1;
  int window, sinks;
  int first[2], last[2];   // positions of the first and last row of A and B (B absent: last < 0)
  __device__ int key0(int t) const { return t < sink_tiles ? t * 128 : lo + (t - sink_tiles) * 128; }
  __device__ int end(int t) const {   // one past the tile's last key
    const int k = key0(t) + 128, e = t < sink_tiles ? se : hi;
    return k < e ? k : e;
  }
  __device__ bool narrow(int t) const { return end(t) - key0(t) <= kNarrow; }
  __device__ int kind(int x, int t) const {
    const int k0 = key0(t), k1 = end(t);
    if (k0 > last[x] || (k0 >= sinks && k1 - 1 <= first[x] - window)) return kNone;
    if (k1 - k0 == 128 && k1 - 1 <= first[x] && (k0 > last[x] - window || k1 <= sinks)) return kWhole;
    return kPart;
  }
  // next tile >= t that A or B needs; false at the end
  __device__ bool next(int& t, int& ka, int& kb) const {
    for (; t < t1; ++t) {
      ka = kind(0, t);
      kb = kind(1, t);
      if (ka != kNone || kb != kNone) return true;
    }
    return false;
  }
};

template <int NX>
__global__ void __launch_bounds__(Cta<NX>::threads, Cta<NX>::per_sm)
cache_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, CacheArgs a) {
  using C = Cta<NX>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = dev::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + C::off_abort);
  uint32_t* tmem_ptr_smem = reinterpret_cast<uint32_t*>(sgen + C::off_tmemptr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int split = blockIdx.x % a.splits;
  const int job = blockIdx.x / a.splits;
  const int pair = job % a.blocks, unit = job / a.blocks;
  const int b = unit / a.h_kv, g = unit - b * a.h_kv;
  const int len = dev::cache_len(a, b);   // in flight over the set-up

  if (threadIdx.x == 0) {
    *abort_flag = dev::load_volatile(a.status) != 0 ? 1 : 0;   // an earlier failure: do nothing
    for (int s = 0; s < C::k_stages; ++s) {
      dev::mbar_init(C::bar(sbase, C::b_kfull + s), 1);
      dev::mbar_init(C::bar(sbase, C::b_kempty + s), 1);
    }
    for (int s = 0; s < C::v_stages; ++s) {
      dev::mbar_init(C::bar(sbase, C::b_vfull + s), 1);
      dev::mbar_init(C::bar(sbase, C::b_vempty + s), 1);
      dev::mbar_init(C::bar(sbase, C::b_vclear + s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      dev::mbar_init(C::bar(sbase, C::b_sfull + x), 1);
      dev::mbar_init(C::bar(sbase, C::b_pfull + x), 128);
      dev::mbar_init(C::bar(sbase, C::b_done + x), 1);
      dev::mbar_init(C::bar(sbase, C::b_q + x), 1);
    }
    dev::mbar_init(C::bar(sbase, C::b_drain), 1);
    dev::fence_mbar_init();
  }
  if (warp == 1) {
    dev::tmem_alloc(dev::smem_u32(tmem_ptr_smem), C::tmem_cols);
    dev::tmem_relinquish();
  }
  dev::tc_fence_before();
  __syncthreads();
  dev::tc_fence_after();
  const uint32_t tmem = *tmem_ptr_smem;
  if (*abort_flag) {   // uniform: written before the barrier; later failures are met in the waits
    if (warp == 1) dev::tmem_dealloc(tmem, C::tmem_cols);
    return;
  }

  // the row tiles: tokens [tok0, tok0 + tok_box) of sequences [seq0, seq0 + seq_box)
  const bool hasB = NX == 2 && 2 * pair + 1 < a.row_tiles;
  const int seq_tiles = (a.n_q + a.tok_box - 1) / a.tok_box;   // row tiles along a sequence's tokens
  int tok0[2], seq0[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int ti = NX * pair + x, s = a.prefix ? ti / seq_tiles : 0;
    seq0[x] = a.prefix ? s * a.seq_box : b;
    tok0[x] = (ti - s * seq_tiles) * a.tok_box;
  }
  if (threadIdx.x == 0) {
    const int y = g * a.group;
    const uint32_t half = (uint32_t)(a.group * a.tok_box * a.seq_box) * 128u;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x == 1 && !hasB) break;
      const uint32_t dst = sbase + C::off_q + x * kTileBytes, bq = C::bar(sbase, C::b_q + x);
      dev::mbar_arrive_expect_tx(bq, 2 * half);
      tma_load_4d(dst, &tm_q, bq, 0, y, tok0[x], seq0[x]);
      tma_load_4d(dst + kHalfBytes, &tm_q, bq, 64, y, tok0[x], seq0[x]);
    }
  }

  Sched sc;
  {
    const int end = tok0[hasB ? 1 : 0] + a.tok_box;
    const int i_last = (end < a.n_q ? end : a.n_q) - 1;
    const KeyList list = dev::unit_keys(a, len, tok0[0], i_last);
    sc.se = list.se;
    sc.lo = list.lo;
    sc.hi = list.lo + (list.total - list.se);
    if (sc.lo <= sc.se) {   // the window begins at the end of the first keys: one segment
      sc.se = 0;
      sc.lo = 0;
    }
    sc.sink_tiles = (sc.se + 127) / 128;
    const int tiles = sc.sink_tiles + (sc.hi - sc.lo + 127) / 128;   // <= 2^17 + 1; splits <= 296
    sc.t0 = a.splits == 1 ? 0 : tiles * split / a.splits;
    sc.t1 = a.splits == 1 ? tiles : tiles * (split + 1) / a.splits;
    sc.window = a.window;
    sc.sinks = a.sinks;
    const int a_end = tok0[0] + a.tok_box;
    sc.first[0] = dev::row_pos(a, len, tok0[0]);
    sc.last[0] = dev::row_pos(a, len, (a_end < a.n_q ? a_end : a.n_q) - 1);
    sc.first[1] = hasB ? dev::row_pos(a, len, tok0[1]) : -1;
    sc.last[1] = hasB ? dev::row_pos(a, len, i_last) : -1;
  }

  if (warp < 4) dev::regs_release<C::regs_control>();
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    if (lane == 0) {
      dev::prefetch_tmap(&tm_k);
      dev::prefetch_tmap(&tm_v);
    }
    int u = 0, t = sc.t0, ka = 0, kb = 0, prev_t = -1;
    int issued_k = 0, issued_v = 0;
    bool ok = true, more = true;
    while (ok && (more || prev_t >= 0)) {
      more = more && sc.next(t, ka, kb);
      if (more) {   // K of tile u
        const int s = u % C::k_stages;
        if (!warp_wait(C::bar(sbase, C::b_kempty + s), ((u / C::k_stages) & 1) ^ 1, abort_flag, a.status, 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t bk = C::bar(sbase, C::b_kfull + s);
          dev::mbar_arrive_expect_tx(bk, kTileBytes);
          tma_load_4d(sbase + C::off_k + s * kTileBytes, &tm_k, bk, 0, sc.key0(t), g, b);
          tma_load_4d(sbase + C::off_k + s * kTileBytes + kHalfBytes, &tm_k, bk, 64, sc.key0(t), g, b);
        }
        ++issued_k;
      }
      // V of the tile before, whose weights are still being computed; with one
      // stage of each, of this tile: it waits for the product before it alone
      const int tv = NX == 1 ? (more ? t : -1) : prev_t;
      if (tv >= 0) {
        const int uv = NX == 1 ? u : u - 1, s = uv % C::v_stages;
        const uint32_t vbase = C::off_v + s * kTileBytes, bv = C::bar(sbase, C::b_vfull + s);
        if (!warp_wait(C::bar(sbase, C::b_vempty + s), ((uv / C::v_stages) & 1) ^ 1, abort_flag, a.status, 2)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          dev::mbar_arrive_expect_tx(bv, kTileBytes);
          tma_load_4d(sbase + vbase, &tm_v, bv, 0, sc.key0(tv), g, b);
          tma_load_4d(sbase + vbase + kHalfBytes, &tm_v, bv, 64, sc.key0(tv), g, b);
        }
        ++issued_v;
        const int valid = sc.end(tv) - sc.key0(tv);
        const int used = valid <= kNarrow ? kNarrow : 128;   // rows that the product reads
        if (valid < used) {   // rows behind the segment's end: whatever the cache holds there, 0 * x has to be 0
          if (!warp_wait(bv, (uv / C::v_stages) & 1, abort_flag, a.status, 9)) {
            ok = false;
            break;
          }
          for (int e = lane; e < (used - valid) * 16; e += 32) {
            const int row = valid + (e >> 4), c = e & 15;
            *reinterpret_cast<uint4*>(sgen + vbase + (c >> 3) * kHalfBytes + row * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          dev::fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) dev::mbar_arrive(C::bar(sbase, C::b_vclear + s));
      }
      prev_t = NX == 2 && more ? t : -1;
      if (more) {
        ++t;
        ++u;
      }
    }
    // Every copy lands before the CTA exits: after an error (here or, reported
    // through the status word, in another CTA) the others may not have waited for it
    dev::mbar_drain(C::bar(sbase, C::b_q), 0);
    if (hasB) dev::mbar_drain(C::bar(sbase, C::b_q + 1), 0);
    for (int s = 0; s < C::k_stages && s < issued_k; ++s) {
      const int last = issued_k - 1 - ((issued_k - 1 - s) % C::k_stages);
      dev::mbar_drain(C::bar(sbase, C::b_kfull + s), (last / C::k_stages) & 1);
    }
    for (int s = 0; s < C::v_stages && s < issued_v; ++s) {
      const int last = issued_v - 1 - ((issued_v - 1 - s) % C::v_stages);
      dev::mbar_drain(C::bar(sbase, C::b_vfull + s), (last / C::v_stages) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t idesc_qk = dev::umma_idesc_bf16(128, 128, false);
    const uint32_t idesc_narrow = dev::umma_idesc_bf16(128, kNarrow, false);
    const uint32_t idesc_pv = dev::umma_idesc_bf16(128, 128, true);
    const uint64_t QD0 = dev::smem_desc_sw128(sbase + C::off_q, 16, 1024);
    const uint64_t KD0 = dev::smem_desc_sw128(sbase + C::off_k, 16, 1024);
    const uint64_t VD0 = dev::smem_desc_sw128(sbase + C::off_v, kHalfBytes, 1024);
    int kx0 = 0, kx1 = 0;   // P.V issued per row tile
    auto qk = [&](int x, int u, bool narrow) {
      dev::umma_ss8_w(tmem + (uint32_t)x * 128u, QD0 + (uint64_t)(x * (kTileBytes >> 4)),
                      KD0 + (uint64_t)((u % C::k_stages) * (kTileBytes >> 4)), narrow ? idesc_narrow : idesc_qk, 0u);
      dev::umma_commit_w(C::bar(sbase, C::b_sfull + x));
    };
    auto pv = [&](int x, int u, bool narrow) -> bool {
      const int kx = x == 0 ? kx0 : kx1;
      if (!warp_wait(C::bar(sbase, C::b_pfull + x), kx & 1, abort_flag, a.status, 4 + x)) return false;
      dev::tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(NX + x) * 128u, p = tmem + (uint32_t)x * 128u;
      const uint64_t vd = VD0 + (uint64_t)((u % C::v_stages) * (kTileBytes >> 4));
      if (narrow)
        umma_ts2_w(d, p, vd, idesc_pv, kx > 0 ? 1u : 0u);
      else
        dev::umma_ts8_w(d, p, vd, idesc_pv, kx > 0 ? 1u : 0u);
      if (x == 0) ++kx0; else ++kx1;
      return true;
    };
    int t = sc.t0, ka = 0, kb = 0;
    bool ok = warp_wait(C::bar(sbase, C::b_q), 0, abort_flag, a.status, 14) &&
              (!hasB || warp_wait(C::bar(sbase, C::b_q + 1), 0, abort_flag, a.status, 15));
    bool have = ok && sc.next(t, ka, kb);
    if (have) {
      ok = warp_wait(C::bar(sbase, C::b_kfull + 0), 0, abort_flag, a.status, 6);
      dev::tc_fence_after();
      if (ok && ka != kNone) qk(0, 0, sc.narrow(t));
    }
    int u = 0;
    while (ok && have) {
      if (kb != kNone) qk(1, u, sc.narrow(t));
      dev::umma_commit_w(C::bar(sbase, C::b_kempty + u % C::k_stages));
      int t2 = t + 1, ka2 = 0, kb2 = 0;
      const bool have2 = sc.next(t2, ka2, kb2);
      if (!warp_wait(C::bar(sbase, C::b_vfull + u % C::v_stages), (u / C::v_stages) & 1, abort_flag, a.status, 7) ||
          !warp_wait(C::bar(sbase, C::b_vclear + u % C::v_stages), (u / C::v_stages) & 1, abort_flag, a.status, 3)) {
        ok = false;
        break;
      }
      dev::tc_fence_after();
      if (ka != kNone && !pv(0, u, sc.narrow(t))) {
        ok = false;
        break;
      }
      if (have2) {
        if (!warp_wait(C::bar(sbase, C::b_kfull + (u + 1) % C::k_stages), ((u + 1) / C::k_stages) & 1, abort_flag, a.status,
                       8)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        if (ka2 != kNone) qk(0, u + 1, sc.narrow(t2));
      }
      if (kb != kNone && !pv(1, u, sc.narrow(t))) {
        ok = false;
        break;
      }
      dev::umma_commit_w(C::bar(sbase, C::b_vempty + u % C::v_stages));
      t = t2;
      ka = ka2;
      kb = kb2;
      have = have2;
      ++u;
    }
    if (ok) {
      dev::umma_commit_w(C::bar(sbase, C::b_done + 0));
      dev::umma_commit_w(C::bar(sbase, C::b_done + 1));
    }
    // every MMA issued must complete before TMEM is released
    dev::umma_commit_w(C::bar(sbase, C::b_drain));
    dev::mbar_drain(C::bar(sbase, C::b_drain), 0);
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax warps
    dev::regs_acquire<C::regs_softmax>();
    const int x = (warp - 4) >> 2;                // 0: tile A, 1: tile B
    const int quarter = warp & 3;                 // TMEM lane quarter of this warp
    const int r = quarter * 32 + lane;            // row inside the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = tmem + lane_base + (uint32_t)x * 128;
    const uint32_t o_col = tmem + lane_base + (uint32_t)(NX + x) * 128;
    if (x == 0 || hasB) {
      // the lane's row: a (sequence, token, head of the group) of the tile's box
      const int rest = (int)(((uint64_t)r * a.group_mul) >> 36);
      const int ds = a.seq_box == 1 ? 0 : rest / a.tok_box;
      const int tok = tok0[x] + rest - ds * a.tok_box;
      const bool in = r < a.group * a.tok_box * a.seq_box && tok < a.n_q && seq0[x] + ds < a.n_seqs;
      const int pos = in ? dev::row_pos(a, len, tok) : -1;
      const float sl2 = a.scale_log2;
      SoftRow st{-INFINITY, 0.f};
      int k = 0;
      bool ok = true;
      for (int t = sc.t0; t < sc.t1; ++t) {
        const int kind = sc.kind(x, t);
        if (kind == kNone) continue;
        if (!warp_wait(C::bar(sbase, C::b_sfull + x), k & 1, abort_flag, a.status, 10 + x)) {
          ok = false;
          break;
        }
        dev::tc_fence_after();
        const int k0 = sc.key0(t), e = sc.end(t) - 1;
        const int high = (pos < e ? pos : e) - k0, low = pos - a.window - k0, front = a.sinks - k0;
        if (sc.narrow(t))
          soft_tile<kNarrow>(st, s_col, o_col, k == 0, kind == kPart, low, high, front, sl2, C::bar(sbase, C::b_pfull + x));
        else
          soft_tile<128>(st, s_col, o_col, k == 0, kind == kPart, low, high, front, sl2, C::bar(sbase, C::b_pfull + x));
        ++k;
      }
      if (ok && k > 0) {
        ok = warp_wait(C::bar(sbase, C::b_done + x), 0, abort_flag, a.status, 12 + x);
        dev::tc_fence_after();
      }
      // Results leave through the tile's Q, which no MMA reads any more (a
      // tile without keys has read nothing, but its load has to have landed)
      ok = ok && warp_wait(C::bar(sbase, C::b_q + x), 0, abort_flag, a.status, 16 + x);
      uint8_t* stage = sgen + C::off_q + x * kTileBytes;
      if (ok && a.part_o != nullptr) {
        // float rows, half the columns at a time through the warp's 8 KB, so
        // that half a warp writes 256 bytes of a row
        uint8_t* own = stage + quarter * 8192;
        const int piece = lane & 15;
        const int64_t at0 = ((int64_t)job * a.splits + split) * (128 * NX) + x * 128 + quarter * 32;
        if (in) a.part_ml[at0 + lane] = make_float2(st.m_ref, st.l);
        const uint32_t rows_in = __ballot_sync(0xffffffffu, in);
        if (k > 0) {   // without a key tile the piece has weight 0 and is not read
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              uint32_t v[32];
              dev::tmem_ld32(o_col + half * 64 + c0, v);
              dev::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(own + lane * 256 + (((c0 >> 2) + j) ^ (lane & 7)) * 16) =
                    make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
            __syncwarp();
#pragma unroll 4
            for (int e = 0; e < 16; ++e) {
              const int q = e * 2 + (lane >> 4);
              const uint4 y = *reinterpret_cast<const uint4*>(own + q * 256 + (piece ^ (q & 7)) * 16);
              if ((rows_in >> q) & 1u)
                *reinterpret_cast<uint4*>(a.part_o + (at0 + q) * kHeadDim + half * 64 + piece * 4) = y;
            }
            __syncwarp();
          }
        }
      } else if (ok) {
        // bf16 rows in the box's swizzled layout, then one TMA store per half
        const float inv = st.l > 0.f ? 1.f / st.l : (st.l == 0.f ? 0.f : st.l);   // no key: 0; NaN stays NaN
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 32) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
          if (k > 0) {
            dev::tmem_ld32(o_col + c0, v);
            dev::tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[e] = dev::pack_bf16x2(__uint_as_float(v[8 * j + 2 * e]) * inv, __uint_as_float(v[8 * j + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + (c0 >> 6) * kHalfBytes + r * 128 + ((((c0 >> 3) + j) & 7) ^ (r & 7)) * 16) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      if (a.part_o == nullptr) {
        dev::fence_proxy_async_smem();
        asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");   // the tile's four warps
        if (ok && quarter == 0 && lane == 0) {
          const uint32_t src = sbase + C::off_q + x * kTileBytes;
          tma_store_4d(src, &tm_o, 0, g * a.group, tok0[x], seq0[x]);
          tma_store_4d(src + kHalfBytes, &tm_o, 64, g * a.group, tok0[x], seq0[x]);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // before the CTA's memory goes
        }
      }
    }
    dev::tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    dev::tc_fence_after();
    dev::tmem_dealloc(tmem, C::tmem_cols);
  }
  if (a.chained) dev::wait_for_launches();
}

// A 4-D map with boxes of 64 columns (128 bytes), 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* ptr, const int (&ext)[3], const int64_t (&stride)[3], const int (&rows)[3]) {
  auto fn = tmap_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)ext[0], (cuuint64_t)ext[1], (cuuint64_t)ext[2]};
  cuuint64_t strides[3] = {(cuuint64_t)stride[0] * 2, (cuuint64_t)stride[1] * 2, (cuuint64_t)stride[2] * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)rows[0], (cuuint32_t)rows[1], (cuuint32_t)rows[2]};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_cache_tc(const CacheArgs& a, const AttnPlan& p, cudaStream_t st) {
  CUtensorMap mq, mo, mk, mv;
  const int kv[3] = {a.n_keys, a.h_kv, a.batch}, kv_box[3] = {128, 1, 1};
  const int qo[3] = {a.h_kv * a.group, a.n_q, a.n_seqs}, qo_box[3] = {a.group, a.tok_box, a.seq_box};
  if (!make_map(&mk, a.k, kv, {a.sk.token, a.sk.head, a.sk.seq}, kv_box) ||
      !make_map(&mv, a.v, kv, {a.sv.token, a.sv.head, a.sv.seq}, kv_box) ||
      !make_map(&mq, a.q, qo, {a.sq.head, a.sq.token, a.sq.seq}, qo_box) ||
      !make_map(&mo, a.out, qo, {a.so.head, a.so.token, a.so.seq}, qo_box))
    return cudaErrorInvalidValue;
  const int64_t grid = (int64_t)p.units * p.blocks * p.splits;
  if (grid <= 0 || grid > INT32_MAX) return cudaErrorInvalidValue;
  const auto kernel = p.block == 256 ? cache_tc_kernel<2> : cache_tc_kernel<1>;
  const int smem = p.block == 256 ? Cta<2>::smem : Cta<1>::smem;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, (unsigned)grid, p.block == 256 ? Cta<2>::threads : Cta<1>::threads, smem, st,
                       a.chained != 0, mq, mo, mk, mv, a);
}

}  // namespace crisp
