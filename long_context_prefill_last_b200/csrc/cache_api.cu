// C ABI of the cache operators: argument checks, plans (grid shapes and
// workspace pieces) and the order of launches. Nothing here synchronises
// except crisp_cache_device_status.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "cache.h"
#include "crisp.h"

namespace crisp {
namespace {

constexpr int kSms = 148;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// One tensor's strides: zeros mean contiguous, axes of length 1 get a harmless stride.
crisp_status make_strides(const crisp_strides& in, int64_t seqs, int64_t heads, int64_t tokens, int elem, Strides* out) {
  if (in.seq == 0 && in.head == 0 && in.token == 0) {
    out->token = kHeadDim;
    out->head = tokens * kHeadDim;
    out->seq = heads * out->head;
    return CRISP_OK;
  }
  const int64_t ext[3] = {seqs, heads, tokens}, st[3] = {in.seq, in.head, in.token};
  int64_t got[3];
  for (int i = 0; i < 3; ++i) {
    if (ext[i] <= 1) {
      got[i] = kHeadDim;
      continue;
    }
    if (st[i] < kHeadDim || st[i] > ((int64_t)1 << 36)) return CRISP_ERR_SHAPE;
    if (st[i] * elem % 16 != 0) return CRISP_ERR_ALIGN;
    got[i] = st[i];
  }
  *out = Strides{got[0], got[1], got[2]};
  return CRISP_OK;
}

crisp_status make_cache_shape(const crisp_cache_cfg* c, int op, CacheShape* s) {
  if (c == nullptr || c->reserved != 0) return CRISP_ERR_INVALID_ARG;
  if (op < CRISP_CACHE_WINDOW || op > CRISP_CACHE_EVICT) return CRISP_ERR_INVALID_ARG;
  if (c->dtype != CRISP_BF16 && c->dtype != CRISP_FP32) return CRISP_ERR_DTYPE;
  if (c->d != kHeadDim) return CRISP_ERR_SHAPE;
  if (c->batch < 1 || c->batch > kMaxBatch || c->n_k < 1 || c->n_k > kMaxCacheLen) return CRISP_ERR_SHAPE;
  if (c->h_q <= 0 || c->h_kv <= 0 || c->h_q % c->h_kv != 0 || c->h_q / c->h_kv > 16 || c->h_q > kMaxHeads ||
      (int64_t)c->batch * c->h_q > 65535)
    return CRISP_ERR_SHAPE;
  if (!isfinite(c->sm_scale) || c->window < 0 || c->sinks < 0) return CRISP_ERR_INVALID_ARG;
  const bool attends = op != CRISP_CACHE_EVICT;
  if (attends && (c->n_q < 1 || c->n_q > c->n_k)) return CRISP_ERR_SHAPE;
  if ((op == CRISP_CACHE_SCORED || op == CRISP_CACHE_PREFIX) && c->n_q > kMaxDraft) return CRISP_ERR_SHAPE;
  if (op == CRISP_CACHE_PREFIX) {
    if (c->n_prefix < 1 || c->n_prefix > kMaxCacheLen) return CRISP_ERR_SHAPE;
    if (c->window != 0 || c->sinks != 0) return CRISP_ERR_UNSUPPORTED;
  }
  if (op == CRISP_CACHE_EVICT) {
    if (c->budget < 1 || c->recent < 0 || (int64_t)c->sinks + c->recent > c->budget) return CRISP_ERR_INVALID_ARG;
    if (c->n_new < c->budget || c->n_new > kMaxCacheLen) return CRISP_ERR_SHAPE;
  }
  memset(s, 0, sizeof(*s));
  s->batch = c->batch;
  s->n_q = attends ? c->n_q : 1;
  s->n_k = c->n_k;
  s->h_q = c->h_q;
  s->h_kv = c->h_kv;
  s->group = c->h_q / c->h_kv;
  s->window = c->window == 0 || c->window > kNoWindow ? kNoWindow : c->window;
  s->sinks = std::min(c->sinks, op == CRISP_CACHE_EVICT ? INT32_MAX : c->n_k);
  s->n_prefix = c->n_prefix;
  s->budget = c->budget;
  s->recent = c->recent;
  s->n_new = c->n_new;
  s->fp32 = c->dtype == CRISP_FP32;
  const float scale = c->sm_scale > 0.f ? c->sm_scale : 1.f / sqrtf((float)c->d);
  s->scale_log2 = scale * 1.4426950408889634f;
  return CRISP_OK;
}

crisp_status cache_strides(const crisp_cache_cfg* c, int op, CacheShape* s) {
  const int e = s->fp32 ? 4 : 2;
  crisp_status r;
  if ((r = make_strides(c->k, s->batch, s->h_kv, s->n_k, e, &s->k)) != CRISP_OK) return r;
  if ((r = make_strides(c->v, s->batch, s->h_kv, s->n_k, e, &s->v)) != CRISP_OK) return r;
  if (op == CRISP_CACHE_EVICT) {
    if ((r = make_strides(c->k_new, s->batch, s->h_kv, s->n_new, e, &s->k_new)) != CRISP_OK) return r;
    return make_strides(c->v_new, s->batch, s->h_kv, s->n_new, e, &s->v_new);
  }
  if ((r = make_strides(c->q, s->batch, s->h_q, s->n_q, e, &s->q)) != CRISP_OK) return r;
  if ((r = make_strides(c->out, s->batch, s->h_q, s->n_q, e, &s->out)) != CRISP_OK) return r;
  if (op == CRISP_CACHE_PREFIX) {
    if ((r = make_strides(c->k_prefix, 1, s->h_kv, s->n_prefix, e, &s->k_prefix)) != CRISP_OK) return r;
    return make_strides(c->v_prefix, 1, s->h_kv, s->n_prefix, e, &s->v_prefix);
  }
  return CRISP_OK;
}

crisp_status check_tensor(const void* p) {
  if (p == nullptr) return CRISP_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % 16 != 0 ? CRISP_ERR_ALIGN : CRISP_OK;
}
crisp_status check_words(const void* p, bool optional) {
  if (p == nullptr) return optional ? CRISP_OK : CRISP_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % 4 != 0 ? CRISP_ERR_ALIGN : CRISP_OK;
}
crisp_status check_workspace(const crisp_cache_cfg* c, size_t need) {
  if (c->workspace == nullptr) return CRISP_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(c->workspace) % 256 != 0) return CRISP_ERR_ALIGN;
  return c->workspace_bytes < need ? CRISP_ERR_WORKSPACE : CRISP_OK;
}

// The bytes from a tensor's first to its last element.
struct Range {
  const char *from, *to;
  bool meets(const Range& o) const { return from < o.to && o.from < to; }
};
Range cache_range(const void* p, const Strides& t, int tokens, const CacheShape& s) {
  const int64_t elems = (s.batch - 1) * t.seq + (s.h_kv - 1) * t.head + (int64_t)(tokens - 1) * t.token + kHeadDim;
  return Range{static_cast<const char*>(p), static_cast<const char*>(p) + elems * (s.fp32 ? 4 : 2)};
}
Range word_range(const void* p, int64_t n) {   // NULL: empty
  return Range{static_cast<const char*>(p), static_cast<const char*>(p) + (p == nullptr ? 0 : n * 4)};
}

// How many CTAs share a job's key tiles. Splitting shortens the longest CTA but
// leaves partial results to join: measured, about 5 us for the second launch
// and 0.2 ns per row and split. `cost` is a key tile's time in us; the splits
// fill at most `room` CTAs. (512 tokens of 32 heads through a 128-key window:
// 12 us in one piece, 29 us in two; a chunk of 32 tokens on 4096 keys: 63 us
// in one, 19 us in sixteen.)
int plan_splits(int64_t jobs, int tiles, int64_t rows, int room, double cost) {
  int best = 1;
  double best_us = tiles * cost;
  const int64_t most = std::min<int64_t>(room / jobs, tiles / 2);
  for (int s = 2; s <= most; ++s) {
    const double us = (tiles + s - 1) / s * cost + 5.0 + 2e-4 * (double)rows * s;
    if (us < best_us) {
      best = s;
      best_us = us;
    }
  }
  return best;
}

// Grid of the CUDA-core tile kernel, two CTAs per SM: a 64-key tile takes 4.5 us
// on an SM of its own, and key lists are not split beyond that use.
AttnPlan plan_tile(int units, int rows, int keys) {
  AttnPlan p{};
  p.kernel = kTileSimt;
  p.units = units;
  p.tile = 64;
  p.block = p.slot_rows = 64;
  p.blocks = (rows + 63) / 64;
  const int64_t jobs = (int64_t)units * p.blocks;
  p.splits = plan_splits(jobs, (keys + 63) / 64, (int64_t)units * rows, 2 * kSms, 4.5);
  p.run = ((keys + 63) / 64 + p.splits - 1) / p.splits;
  p.slots = (size_t)jobs * p.splits;
  return p;
}

// Grid of the tcgen05 kernel. A row tile holds up to 128 rows: the group's
// heads of as many tokens as fit (of as many sequences as fit, for the
// prefix). CTAs of two row tiles read the keys once for both and run one per
// SM; CTAs of one run two per SM and hide each other's start and end, which
// counts while there are few key tiles. Measured on 16384 tokens of 32 heads
// (one / two row tiles): 64 keys 127 / 148 us, 512 keys 233 / 261, 1536 keys
// 445 / 462, 2048 keys 573 / 558, 4096 keys of 32768 tokens 2.23 / 2.15 ms.
AttnPlan plan_tc(int units, int group, int n_q, int seqs, bool prefix, int keys) {
  AttnPlan p{};
  p.kernel = kTileTc;
  p.units = units;
  p.tile = 128;
  p.block = p.slot_rows = keys <= 1792 ? 128 : 256;
  p.tok_box = std::min(n_q, 128 / group);
  p.seq_box = prefix && p.tok_box == n_q ? std::min(seqs, 128 / (group * n_q)) : 1;
  p.row_tiles = (n_q + p.tok_box - 1) / p.tok_box * (prefix ? (seqs + p.seq_box - 1) / p.seq_box : 1);
  p.blocks = p.block == 256 ? (p.row_tiles + 1) / 2 : p.row_tiles;
  const int64_t jobs = (int64_t)units * p.blocks;
  p.splits = plan_splits(jobs, (keys + 127) / 128, (int64_t)units * group * n_q * (prefix ? seqs : 1),
                         p.block == 256 ? kSms : 2 * kSms, 2.0);
  p.slots = (size_t)jobs * p.splits;
  return p;
}

// Grid of the decode kernels: two CTAs per SM, or one per key tile when there
// are fewer.
AttnPlan plan_decode(int units, int rows, int keys, bool fp32) {
  AttnPlan p{};
  p.kernel = fp32 ? kDecodeSimt : kDecodeMma;
  p.units = units;
  p.tile = fp32 ? 32 : 64;
  p.block = fp32 ? (rows <= 4 ? 4 : rows <= 8 ? 8 : 16) : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  p.blocks = (rows + p.block - 1) / p.block;
  p.slot_rows = std::min(p.block, rows);
  const int64_t jobs = (int64_t)units * p.blocks;
  p.ctas = (int)std::min<int64_t>(2 * kSms, jobs * ((keys + p.tile - 1) / p.tile));
  p.splits = fp32 ? 1 : 64 / p.block;   // results per CTA and job
  p.slots = (size_t)(jobs + p.ctas) * p.splits;
  return p;
}

// A cluster per job instead of runs of the flat list and a second launch, for up
// to 32 rows, whose join is short. The lengths are not known here, so two
// things bound a CTA's share of a full cache: it stays within kClusterMore tiles
// of the flat list's, for sequences of like lengths, and within kClusterTiles
// tiles of 16 rows, for a long one among short ones, where the flat list deals
// its tiles to every SM and a cluster walks them alone. Measured in us (cluster /
// flat list; 32 query and 8 key/value heads, one token, 64-key tiles of a CTA in
// brackets), every sequence full, lengths even from 1 up, and one full sequence
// among others of 64 tokens:
//   37 x  512 keys [8]    22 / 29     18 / 29     16 / 20
//   32 x 1024 keys [16]   31 / 37     27 / 33     22 / 22
//   32 x 2048 keys [32]   51 / 59     41 / 45     37 / 31
//   37 x 8192 keys [128] 199 / 205   139 / 117   117 / 49
// 74 sequences, 4 key/value heads, 21 rows (32 computed):
//   74 x  512 keys [8]    29 / 33     27 / 35     22 / 22
//   74 x 1024 keys [16]   41 / 47     37 / 47     33 / 25
// and with scores, where a CTA also goes through its keys' logits on its own
// (all full, one full):
//   16 x 1536 keys [12]   33 / 33     25 / 27
//   32 x 1024 keys [16]   37 / 39     29 / 22
// So a skewed batch loses a few us at most. The host saves another 2 us.
constexpr int kClusterMore = 4;
constexpr int kClusterTiles = 20, kClusterTilesScored = 12;
void plan_cluster(AttnPlan* p, int keys, bool scored) {
  if (p->blocks != 1 || p->block > 32 || p->units > 2 * kSms) return;
  const int tiles = (keys + 63) / 64;
  int cs = 1;
  while (cs < 8 && 2 * cs * p->units <= 2 * kSms && 2 * cs <= tiles) cs *= 2;
  const int mine = (tiles + cs - 1) / cs, flat = (int)(((int64_t)p->units * tiles + 2 * kSms - 1) / (2 * kSms));
  if (mine > flat + kClusterMore || mine * (p->block / 16) > (scored ? kClusterTilesScored : kClusterTiles)) return;
  p->cluster = cs;
  p->slots = 0;
}

bool decodes(const AttnPlan& p) { return p.kernel == kDecodeMma || p.kernel == kDecodeSimt; }

}  // namespace

CachePlan plan_cache(const CacheShape& s, int op) {
  CachePlan p{};
  size_t off = 256;   // status
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  auto parts = [&](AttnPlan& a, size_t* ml, size_t* o, size_t* table) {
    *table = take(decodes(a) ? (size_t)a.units * a.blocks * 8 : 0);
    *ml = take(a.slots * a.slot_rows * 8);
    *o = take(a.slots * a.slot_rows * kHeadDim * 4);
  };
  if (op != CRISP_CACHE_EVICT) {
    const int units = s.batch * s.h_kv, rows = s.n_q * s.group;
    // keys that one CTA's rows can span: tokens in its rows, the window and the first keys
    const int tokens = std::min(s.n_q, s.fp32 ? 64 : 256);
    const int64_t seen = (int64_t)s.window + s.sinks + tokens - 1;
    const int keys = (int)std::min<int64_t>(s.n_k, seen);
    p.has_pre = op == CRISP_CACHE_PREFIX;
    // Few rows (a draft's, or those of all sequences for the prefix) take a
    // decode kernel, more a tile kernel. In bf16 up to 64 rows (of 16 tokens),
    // where the legacy tensor instruction still keeps up with memory and one job
    // holds them all (a second row block would read every key again); in fp32 up
    // to 32, where two passes of 16 rows over the keys (80 cycles a key) beat the
    // 64-row tile (128). Scores in bf16 need the decode kernel's logits.
    // Measured on bf16 drafts (decode kernel / tcgen05 kernel, us): 70 rows of 7
    // heads a group, 1 x 4096 keys 22 / 18, 1 x 65536 86 / 45, 8 x 8192 86 / 45, 64
    // x 600 76 / 29; 256 rows of 16 heads, 1 x 65536 57 / 31, 64 x 600 51 / 20. A
    // window of 512 keys of one sequence is the other way round, 14 / 18.
    auto plan = [&](int n_units, int n_rows, int n_keys, bool few, bool prefix) {
      return few      ? plan_decode(n_units, n_rows, n_keys, s.fp32)
             : s.fp32 ? plan_tile(n_units, n_rows, n_keys)
                      : plan_tc(n_units, s.group, s.n_q, s.batch, prefix, n_keys);
    };
    const int most_rows = s.fp32 ? 32 : 64;
    const bool few = rows <= most_rows && (s.fp32 || s.n_q <= kMaxDraft);
    p.main = plan(units, rows, keys, few || (!s.fp32 && op == CRISP_CACHE_SCORED), false);
    if (p.main.kernel == kDecodeMma && !p.has_pre) plan_cluster(&p.main, keys, op == CRISP_CACHE_SCORED);
    if (p.has_pre) p.pre = plan(s.h_kv, s.batch * rows, s.n_prefix, s.batch * rows <= most_rows, true);
    // output rows straight away when no row's keys are split
    if (op == CRISP_CACHE_WINDOW && !decodes(p.main) && p.main.splits == 1) p.main.slots = 0;
    // a row's pieces are read by one warp while there are few, by up to eight when there are many
    auto pieces = [](const AttnPlan& a) {
      return a.slots == 0 ? 0 : decodes(a) ? (a.ctas / (a.units * a.blocks) + 1) * a.splits : a.splits;
    };
    const int most = pieces(p.main) + pieces(p.pre);
    p.warps_per_row = most > 32 ? 8 : most > 16 ? 4 : most > 8 ? 2 : 1;
    parts(p.main, &p.off_ml, &p.off_o, &p.off_table);
    if (p.has_pre) parts(p.pre, &p.off_pre_ml, &p.off_pre_o, &p.off_pre_table);
    if (op == CRISP_CACHE_SCORED) {
      p.pitch = (keys + 63) / 64 * 64;
      p.off_logits = take((size_t)units * rows * p.pitch * 4);
    }
  }
  p.total = off;
  return p;
}

namespace {

#define CACHE_TRY(expr)                         \
  do {                                          \
    if ((expr) != cudaSuccess) {                \
      (void)cudaGetLastError();                 \
      return CRISP_ERR_CUDA;                    \
    }                                           \
  } while (0)

crisp_status run_attention(const void* q, const void* kp, const void* vp, const void* k, const void* v, void* out,
                           float* score, const int32_t* kv_len, const CacheShape& s, const CachePlan& p, char* ws,
                           cudaStream_t st) {
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  // a decode kernel on its own sets the status words; otherwise they are cleared first and kernels only report
  const bool clear = !decodes(p.main) || (p.has_pre && !decodes(p.pre));
  if (clear) CACHE_TRY(cudaMemsetAsync(status, 0, 32, st));
  auto launch = [&](const AttnPlan& pl, const CacheArgs& a) {
    return pl.kernel == kDecodeMma ? launch_cache_decode(a, pl, st)
           : pl.kernel == kDecodeSimt ? launch_cache_decode_fp32(a, pl, st)
           : pl.kernel == kTileTc ? launch_cache_tc(a, pl, st)
                                  : launch_cache_tile(a, pl, st);
  };
  CacheArgs a{};
  a.q = q;
  a.out = out;
  a.status = status;
  a.h_kv = s.h_kv;
  a.group = s.group;
  a.n_q = s.n_q;
  a.per_seq = s.n_q * s.group;
  a.n_seqs = s.batch;
  a.group_mul = div_magic(a.group);
  a.seq_mul = div_magic(a.per_seq);
  a.scale_log2 = s.scale_log2;
  a.sq = s.q;
  a.so = s.out;
  const CacheArgs base = a;   // what the prefix's launch shares with the sequences' own
  FinishArgs m{};
  auto source = [&](const AttnPlan& pl, size_t off_ml, size_t off_o, size_t off_table, CacheArgs* x) {
    PartSrc src{};
    x->block = pl.slot_rows;
    x->blocks = pl.blocks;
    x->splits = pl.splits;
    x->ctas = pl.ctas;
    x->tok_box = pl.tok_box;
    x->seq_box = pl.seq_box;
    x->row_tiles = pl.row_tiles;
    x->cluster = pl.cluster;
    if (pl.slots == 0) return src;
    x->part_ml = reinterpret_cast<float2*>(ws + off_ml);
    x->part_o = reinterpret_cast<float*>(ws + off_o);
    src.mode = decodes(pl) ? kStair : pl.kernel == kTileTc ? kBoxes : kSplits;
    src.tok_box = pl.tok_box;
    src.seq_box = pl.seq_box;
    src.o = x->part_o;
    src.ml = x->part_ml;
    src.block = pl.slot_rows;
    src.blocks = pl.blocks;
    src.splits = pl.splits;
    src.table = x->table = reinterpret_cast<int2*>(ws + off_table);
    return src;
  };
  a.k = k;
  a.v = v;
  a.sk = s.k;
  a.sv = s.v;
  a.kv_len = kv_len;
  a.batch = s.batch;
  a.n_keys = s.n_k;
  a.rows = a.per_seq;
  a.window = s.window;
  a.sinks = s.sinks;
  a.sets_status = clear ? 0 : 1;
  m.main = source(p.main, p.off_ml, p.off_o, p.off_table, &a);
  if (score != nullptr) {
    a.logits = reinterpret_cast<float*>(ws + p.off_logits);
    a.pitch = p.pitch;
    a.score = score;
    m.logits = a.logits;
    m.pitch = p.pitch;
    m.score = score;
  }
  CACHE_TRY(launch(p.main, a));
  if (p.has_pre) {
    CacheArgs x = base;
    x.k = kp;
    x.v = vp;
    x.sk = s.k_prefix;
    x.sv = s.v_prefix;
    x.batch = 1;
    x.n_keys = s.n_prefix;
    x.rows = s.batch * a.per_seq;
    x.prefix = 1;
    x.window = kNoWindow;
    m.pre = source(p.pre, p.off_pre_ml, p.off_pre_o, p.off_pre_table, &x);
    // the two read nothing of each other: the prefix may start while a decode
    // kernel on the sequences' own keys still runs (it lets it), and ends after it
    x.chained = decodes(p.main) && p.pre.kernel != kTileSimt ? 1 : 0;
    CACHE_TRY(launch(p.pre, x));
  }
  if (p.main.slots == 0) return CRISP_OK;
  m.kv_len = kv_len;
  m.batch = s.batch;
  m.n_q = s.n_q;
  m.n_k = s.n_k;
  m.h_kv = s.h_kv;
  m.group = s.group;
  m.window = s.window;
  m.sinks = s.sinks;
  m.out = out;
  m.so = s.out;
  m.fp32 = s.fp32;
  m.warps_per_row = p.warps_per_row;
  CACHE_TRY(launch_cache_finish(m, st));
  return CRISP_OK;
}

// The checks that every operator makes, in the order of the prefill entry points.
crisp_status prepare_cache(const crisp_cache_cfg* cfg, int op, const void* const* tensors, int n_tensors, CacheShape* s,
                           CachePlan* p) {
  crisp_status r = make_cache_shape(cfg, op, s);
  if (r != CRISP_OK) return r;
  if ((r = cache_strides(cfg, op, s)) != CRISP_OK) return r;
  for (int i = 0; i < n_tensors; ++i)
    if ((r = check_tensor(tensors[i])) != CRISP_OK) return r;
  *p = plan_cache(*s, op);
  return check_workspace(cfg, p->total);
}

}  // namespace
}  // namespace crisp

using namespace crisp;

extern "C" {

crisp_status crisp_cache_cfg_init(crisp_cache_cfg* cfg, int32_t batch, int32_t n_q, int32_t n_k, int32_t h_q,
                                  int32_t h_kv, int32_t d, int32_t dtype) {
  if (cfg == nullptr) return CRISP_ERR_INVALID_ARG;
  memset(cfg, 0, sizeof(*cfg));
  cfg->batch = batch;
  cfg->n_q = n_q;
  cfg->n_k = n_k;
  cfg->h_q = h_q;
  cfg->h_kv = h_kv;
  cfg->d = d;
  cfg->dtype = dtype;
  return CRISP_OK;
}

crisp_status crisp_cache_workspace_size(const crisp_cache_cfg* cfg, int32_t op, size_t* bytes) {
  CacheShape s;
  crisp_status r = make_cache_shape(cfg, op, &s);
  if (r != CRISP_OK) return r;
  if (bytes == nullptr) return CRISP_ERR_INVALID_ARG;
  *bytes = plan_cache(s, op).total;
  return CRISP_OK;
}

crisp_status crisp_window_attention(const void* q, const void* k, const void* v, void* out, const int32_t* kv_len,
                                    const crisp_cache_cfg* cfg, void* stream) {
  CacheShape s;
  CachePlan p;
  const void* t[] = {q, k, v, out};
  crisp_status r = prepare_cache(cfg, CRISP_CACHE_WINDOW, t, 4, &s, &p);
  if (r != CRISP_OK) return r;
  if ((r = check_words(kv_len, true)) != CRISP_OK) return r;
  return run_attention(q, nullptr, nullptr, k, v, out, nullptr, kv_len, s, p, static_cast<char*>(cfg->workspace),
                       static_cast<cudaStream_t>(stream));
}

crisp_status crisp_scored_attention(const void* q, const void* k, const void* v, void* out, float* score,
                                    const int32_t* kv_len, const crisp_cache_cfg* cfg, void* stream) {
  CacheShape s;
  CachePlan p;
  const void* t[] = {q, k, v, out};
  crisp_status r = prepare_cache(cfg, CRISP_CACHE_SCORED, t, 4, &s, &p);
  if (r != CRISP_OK) return r;
  if ((r = check_words(score, false)) != CRISP_OK) return r;
  if ((r = check_words(kv_len, true)) != CRISP_OK) return r;
  return run_attention(q, nullptr, nullptr, k, v, out, score, kv_len, s, p, static_cast<char*>(cfg->workspace),
                       static_cast<cudaStream_t>(stream));
}

crisp_status crisp_shared_prefix_attention(const void* q, const void* k_prefix, const void* v_prefix, const void* k,
                                           const void* v, void* out, const int32_t* kv_len,
                                           const crisp_cache_cfg* cfg, void* stream) {
  CacheShape s;
  CachePlan p;
  const void* t[] = {q, k_prefix, v_prefix, k, v, out};
  crisp_status r = prepare_cache(cfg, CRISP_CACHE_PREFIX, t, 6, &s, &p);
  if (r != CRISP_OK) return r;
  if ((r = check_words(kv_len, true)) != CRISP_OK) return r;
  return run_attention(q, k_prefix, v_prefix, k, v, out, nullptr, kv_len, s, p, static_cast<char*>(cfg->workspace),
                       static_cast<cudaStream_t>(stream));
}

crisp_status crisp_evict(const void* k, const void* v, const float* score, const int32_t* kv_len, void* k_new,
                         void* v_new, float* score_new, int32_t* kept, int32_t* new_len,
                         const crisp_cache_cfg* cfg, void* stream) {
  CacheShape s;
  CachePlan p;
  const void* t[] = {k, v, k_new, v_new};
  crisp_status r = prepare_cache(cfg, CRISP_CACHE_EVICT, t, 4, &s, &p);
  if (r != CRISP_OK) return r;
  const void* words[] = {score, score_new, kept, new_len};
  for (const void* w : words)
    if ((r = check_words(w, false)) != CRISP_OK) return r;
  if ((r = check_words(kv_len, true)) != CRISP_OK) return r;
  // nothing that is written may be an input, or another output; k_new and v_new may lie interleaved
  const int64_t units = (int64_t)s.batch * s.h_kv;
  const Range in[] = {cache_range(k, s.k, s.n_k, s), cache_range(v, s.v, s.n_k, s), word_range(score, units * s.n_k),
                      word_range(kv_len, s.batch)};
  const Range out[] = {cache_range(k_new, s.k_new, s.n_new, s), cache_range(v_new, s.v_new, s.n_new, s),
                       word_range(score_new, units * s.n_new), word_range(kept, units * s.budget),
                       word_range(new_len, s.batch)};
  if (k_new == v_new) return CRISP_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i) {
    for (const Range& x : in)
      if (out[i].meets(x)) return CRISP_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (i > 1 && out[i].meets(out[j])) return CRISP_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(cfg->workspace);
  EvictArgs a{};
  a.k = k;
  a.v = v;
  a.score = score;
  a.kv_len = kv_len;
  a.k_new = k_new;
  a.v_new = v_new;
  a.score_new = score_new;
  a.kept = kept;
  a.new_len = new_len;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.sk = s.k;
  a.sv = s.v;
  a.skn = s.k_new;
  a.svn = s.v_new;
  a.batch = s.batch;
  a.h_kv = s.h_kv;
  a.n_k = s.n_k;
  a.sinks = s.sinks;
  a.recent = s.recent;
  a.budget = s.budget;
  a.n_new = s.n_new;
  a.row_bytes = kHeadDim * (s.fp32 ? 4 : 2);
  CACHE_TRY(launch_evict(a, st));
  return CRISP_OK;
}

crisp_status crisp_cache_device_status(const crisp_cache_cfg* cfg, void* stream, int32_t* device_status) {
  if (cfg == nullptr || device_status == nullptr) return CRISP_ERR_INVALID_ARG;
  const crisp_status r = check_workspace(cfg, 256);
  if (r != CRISP_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t word[8] = {0};
  // all on `st`: the default stream would wait for other streams' work, and what
  // follows on `st` would not wait for its clearing
  CACHE_TRY(cudaMemcpyAsync(word, cfg->workspace, sizeof(word), cudaMemcpyDeviceToHost, st));
  CACHE_TRY(cudaMemsetAsync(cfg->workspace, 0, sizeof(word), st));
  CACHE_TRY(cudaStreamSynchronize(st));
  *device_status = word[kStatusCode] != 0 ? word[kStatusCode] : word[kStatusLen];
  return CRISP_OK;
}

}  // extern "C"
