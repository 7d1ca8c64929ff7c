// C-ABI layer of the attention calls: argument validation, how key ranges are
// split over the SMs, workspace layout, launches.  No device memory is
// allocated and no exception leaves an entry point: plans live on the stack.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "attn_internal.h"
#include "dosa_device.cuh"

namespace dosa {

int attn_sm_count() {
  static std::atomic<int> known[64];       // per device
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 148;          // without a device only sizes are asked for
  }
  if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms <= 0) {
    cudaGetLastError();
    return 148;
  }
  if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace dosa

using namespace dosa;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;   // rows and keys are 32-bit indices in the kernels

const AttnHandle* handle(dosa_attn_t h) { return reinterpret_cast<const AttnHandle*>(h); }

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A view of n rows of `heads` 128-element vectors (no rows: any address).
bool rows_ok(const dosa_rows* r, int heads, int64_t n) {
  return r && (r->ptr || n == 0) && aligned(r->ptr, 16) && r->row_stride % 8 == 0 && r->head_stride % 8 == 0 &&
         r->row_stride >= (n > 1 ? 8 : 0) && r->head_stride >= (heads > 1 ? 8 : 0) &&
         r->row_stride < ((int64_t)1 << 38) && r->head_stride < ((int64_t)1 << 38);
}
// The same for results: no two vectors overlap.
bool out_rows_ok(const dosa_rows* r, int heads, int64_t n) {
  if (!rows_ok(r, heads, n)) return false;
  if (heads > 1 && r->head_stride < kHeadDim) return false;
  if (n > 1 && r->row_stride < kHeadDim) return false;
  if (heads <= 1 || n <= 1) return true;
  // one stride spans all vectors of the other
  return r->row_stride >= (heads - 1) * r->head_stride + kHeadDim ||
         r->head_stride >= (n - 1) * r->row_stride + kHeadDim;
}

Rows16 rows16(const dosa_rows* r) {
  Rows16 o;
  o.ptr = static_cast<uint16_t*>(r->ptr);
  o.rs = r->row_stride;
  o.hs = r->head_stride;
  return o;
}

bool cache_ok(const dosa_cache4* c) {
  return c && c->k_codes && c->k_params && c->v_codes && c->v_params && c->capacity >= 0 &&
         c->capacity <= kMaxRows && aligned(c->k_codes, 16) && aligned(c->k_params, 16) &&
         aligned(c->v_codes, 16) && aligned(c->v_params, 16) && aligned(c->weight, 4);
}

Cache4View cache_view(const dosa_cache4* c) {
  Cache4View v;
  v.kc = static_cast<uint8_t*>(c->k_codes);
  v.kp = static_cast<uint8_t*>(c->k_params);
  v.vc = static_cast<uint8_t*>(c->v_codes);
  v.vp = static_cast<uint8_t*>(c->v_params);
  v.weight = c->weight;
  v.cap = c->capacity;
  return v;
}

dosa_status check_batch(const int64_t* so, int B) {
  if (!so || B < 1) return DOSA_ERR_INVALID_ARG;
  if (so[0] != 0 || so[1] != 0) return DOSA_ERR_INVALID_ARG;
  for (int b = 0; b < B; ++b) {
    const int64_t *r = so + 3 * b, *n = r + 3;
    const int64_t nq = n[0] - r[0], nk = n[1] - r[1];
    if (n[0] < r[0] || n[1] < r[1] || r[2] < 0) return DOSA_ERR_INVALID_ARG;
    if (n[0] > kMaxRows || n[1] > kMaxRows || r[2] > kMaxRows) return DOSA_ERR_UNSUPPORTED;
    if (nq > 0 && r[2] + nq > nk) return DOSA_ERR_INVALID_ARG;
  }
  return DOSA_OK;
}

// ---- plans -------------------------------------------------------------------

// How a call cuts its work.  Computed from the batch alone, so the workspace
// query and the call agree.
struct Plan {
  int chunk;            // keys per part (attend) or key tiles per part (prompt)
  int64_t vectors;      // partial vectors of split sequences
};

constexpr int kPromptTile = 128;     // keys per tile, packed query rows per MMA tile

int prompt_tokens(const AttnHandle* h) { return 2 * (kPromptTile / h->G); }   // rows per unit

// Key tiles a sequence's longest unit walks, and its units without splitting.
void prompt_shape(const AttnHandle* h, const int64_t* r, int64_t* tiles, int64_t* units) {
  const int64_t rows = r[3] - r[0];
  *tiles = rows > 0 ? (r[2] + rows + kPromptTile - 1) / kPromptTile : 0;
  *units = (rows + prompt_tokens(h) - 1) / prompt_tokens(h) * h->cfg.Hkv;
}

// Parts of a sequence's key axis for parts of at most `chunk` tiles, and the even
// share of each.
int64_t prompt_parts(int64_t tiles, int64_t chunk) { return tiles > 0 ? (tiles + chunk - 1) / chunk : 1; }

// Batches of few rows: every unit of a sequence is alike, and the time is that of
// parts handed out longest first to the SMs.  items: (tiles, how many), at most
// kEvenSeqs kinds.  SMs of equal load are one group, kept in ascending order.
constexpr int kEvenSeqs = 64, kEvenSms = 256;
struct PartKind {
  int tiles;
  int64_t count;
};
int64_t longest_first_time(PartKind* items, int n, int sms) {
  std::sort(items, items + n, [](const PartKind& a, const PartKind& b) { return a.tiles > b.tiles; });
  struct {
    int64_t load;
    int count;
  } g[kEvenSms + 1];
  int groups = 1;
  g[0] = {0, sms};
  for (int i = 0; i < n; ++i)
    for (int64_t left = items[i].count; left > 0;) {
      const int take = (int)std::min<int64_t>(left, g[0].count);
      const int64_t load = g[0].load + items[i].tiles;
      left -= take;
      g[0].count -= take;
      int to = 1;                                  // first group that is not below `load`
      while (to < groups && g[to].load < load) ++to;
      if (to < groups && g[to].load == load) {
        g[to].count += take;
      } else {
        for (int j = groups; j > to; --j) g[j] = g[j - 1];
        g[to] = {load, take};
        ++groups;
      }
      if (g[0].count == 0) {
        --groups;
        for (int j = 0; j < groups; ++j) g[j] = g[j + 1];
      }
    }
  return g[groups - 1].load;
}

// The chunk: the time of a chunk is estimated in tiles as the work per SM (a
// unit costs 3 tiles beyond its own, 5 when it is a part whose result has to be
// joined) and a quarter of the longest unit for the uneven end, or the longest
// unit if that is more.  Where the batch has few rows, the chunks that come
// within an eighth of the best are compared by handing their parts out (16 rows
// over 5K to 16K keys, 64 heads over 8: 159 -> 146 us).
Plan prompt_plan(const AttnHandle* h, const int64_t* so, int B) {
  const int64_t sms = attn_sm_count();
  int64_t longest = 0;
  for (int b = 0; b < B; ++b) {
    int64_t t, u;
    prompt_shape(h, so + 3 * b, &t, &u);
    if (t > longest) longest = t;
  }
  auto estimate = [&](int64_t chunk) {
    double work = 0, unit = 0;
    int64_t parts = 0;
    for (int b = 0; b < B; ++b) {
      int64_t t, u;
      prompt_shape(h, so + 3 * b, &t, &u);
      if (t == 0) continue;
      // causal units of one sequence walk from the first row's tiles to the last's
      const int64_t t0 = (so[3 * b + 2] + kPromptTile) / kPromptTile;
      const int64_t ns = prompt_parts(t, chunk);
      const double extra = ns > 1 ? 5.0 : 3.0;
      work += (double)u * (0.5 * (t + t0) + extra * ns);
      parts += u * ns;
      const double len = (double)((t + ns - 1) / ns) + extra;
      if (len > unit) unit = len;
    }
    const double even = work / sms + (parts > sms ? 0.25 * unit : 0.0);
    return even > unit ? even : unit;
  };
  Plan p;
  int64_t best = longest > 0 ? longest : 1;
  double best_t = estimate(best), t_of[65];
  int last = 1;
  t_of[1] = best_t;
  for (int n = 2; n <= 64 && longest / n >= 3; ++n) {
    const int64_t chunk = (longest + n - 1) / n;
    const double t = t_of[last = n] = estimate(chunk);
    if (t < best_t) {
      best_t = t;
      best = chunk;
    }
  }
  bool alike = B <= kEvenSeqs && sms <= kEvenSms;
  for (int b = 0; b < B && alike; ++b) alike = so[3 * b + 3] - so[3 * b] <= prompt_tokens(h);
  if (alike && last > 1) {
    int64_t even_t = INT64_MAX;
    for (int n = 1; n <= last; ++n) {
      if (t_of[n] > 1.125 * best_t) continue;
      const int64_t chunk = (longest + n - 1) / n;
      PartKind items[kEvenSeqs];
      int kinds = 0;
      int64_t parts = 0, most = 1;
      for (int b = 0; b < B; ++b) {
        int64_t t, u;
        prompt_shape(h, so + 3 * b, &t, &u);
        if (t == 0) continue;
        const int64_t ns = prompt_parts(t, chunk);
        items[kinds++] = {(int)((t + ns - 1) / ns) + 3, u * ns};
        parts += u * ns;
        most = std::max(most, ns);
      }
      if (parts > 8 * sms) continue;               // their end is even enough
      // the join reads every part: a tile's time per 8 of them
      const int64_t t = 8 * longest_first_time(items, kinds, (int)sms) + most;
      if (t < even_t) {
        even_t = t;
        best = chunk;
      }
    }
  }
  p.chunk = (int)best;
  p.vectors = 0;
  for (int b = 0; b < B; ++b) {
    int64_t t, u;
    prompt_shape(h, so + 3 * b, &t, &u);
    const int64_t ns = prompt_parts(t, best);
    if (ns > 1) p.vectors += ns * (so[3 * b + 3] - so[3 * b]) * h->cfg.Hq;
  }
  return p;
}

// Units of an attend sequence per part.
int64_t attend_groups(const AttnHandle* h, int64_t rows, bool selected) {
  const int nc = attend_columns(*h, (int)rows, selected);
  const int64_t cols = selected ? h->G : rows * h->G;
  return (cols + nc - 1) / nc * h->cfg.Hkv * (selected ? rows : 1);
}

// One wave: the shortest chunk of keys (a multiple of 128: one 16-token slice
// per warp) for which all parts of all units are resident at once, two CTAs
// per SM, one where a unit has more than 8 columns (registers).  Sequences of each
// column width have launches of their own, one after another, and so a plan.
Plan attend_plan(const AttnHandle* h, const int64_t* so, int B, int K, int width) {
  const bool selected = K > 0;
  auto rows_of = [&](int b) {                      // 0: nothing to do, or another width
    const int64_t rows = so[3 * b + 3] - so[3 * b];
    return rows > 0 && attend_columns(*h, (int)rows, selected) == width ? rows : 0;
  };
  int64_t longest = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t rows = rows_of(b);
    const int64_t len = rows > 0 ? (selected ? K : so[3 * b + 2] + rows) : 0;
    if (len > longest) longest = len;
  }
  const int64_t slots = (width > 8 ? 1 : 2) * (int64_t)attn_sm_count();
  auto parts = [&](int64_t blocks) {
    int64_t n = 0;
    for (int b = 0; b < B; ++b) {
      const int64_t rows = rows_of(b);
      if (rows == 0) continue;
      const int64_t len = selected ? K : so[3 * b + 2] + rows;
      n += (len + 128 * blocks - 1) / (128 * blocks) * attend_groups(h, rows, selected);
    }
    return n;
  };
  int64_t lo = 1, hi = (longest + 127) / 128;
  if (hi < 1) hi = 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (parts(mid) <= slots) hi = mid;
    else lo = mid + 1;
  }
  Plan p;
  p.chunk = (int)(lo * 128);
  p.vectors = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t rows = rows_of(b);
    if (rows == 0) continue;
    const int64_t len = selected ? K : so[3 * b + 2] + rows;
    const int64_t ns = (len + p.chunk - 1) / p.chunk;
    if (ns > 1) p.vectors += ns * rows * h->cfg.Hq;
  }
  return p;
}

// The widths' plans; returns their partial vectors.
constexpr int kWidths = 3;                         // 8, 16, 32 columns
int64_t attend_plans(const AttnHandle* h, const int64_t* so, int B, int K, Plan (&p)[kWidths]) {
  int64_t vectors = 0;
  for (int i = 0; i < kWidths; ++i) {
    p[i] = attend_plan(h, so, B, K, 8 << i);
    vectors += p[i].vectors;
  }
  return vectors;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of a selection with weights that one launch takes: their scores (4 bytes
// per list entry and head) are kept for the weights, in at most 64 MB (a row's,
// if that is more), which is half of L2.
constexpr int64_t kScoreBytes = (int64_t)64 << 20;
int64_t score_rows(const AttnHandle* h, int64_t Tq, int K) {
  const int64_t n = kScoreBytes / ((int64_t)K * h->cfg.Hq * 4);
  return std::min(Tq, std::max<int64_t>(n, 1));
}

struct Layout {
  size_t part_o, part_lse, lse2, row_weight, scores, total;
};
Layout layout(const AttnHandle* h, int64_t vectors, int64_t Tq, int K, bool weights) {
  Layout L;
  size_t at = kWsHeaderBytes;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += round256(n);
    return o;
  };
  L.part_o = take((size_t)vectors * kHeadDim * 4);
  L.part_lse = take((size_t)vectors * 4);
  L.lse2 = take(weights ? (size_t)Tq * h->cfg.Hq * 4 : 0);
  const size_t entries = weights && K ? (size_t)score_rows(h, Tq, K) * K : 0;
  L.row_weight = take(entries * 4);
  L.scores = take(entries * h->cfg.Hq * 4);
  L.total = at;
  return L;
}

AttnSeq seq_of(const int64_t* so, int b) {
  AttnSeq s;
  s.k0 = so[3 * b + 1];
  s.q0 = (int)so[3 * b];
  s.rows = (int)(so[3 * b + 3] - so[3 * b]);
  s.pos0 = (int)so[3 * b + 2];
  s.part0 = -1;
  s.unit0 = 0;
  s.nsplit = 1;
  s.chunk = 0;
  return s;
}

// The table of a launch's split sequences for the joining kernel: units are
// their (row, head) vectors.
AttnTable join_table(const AttnTable& t, int Hq) {
  AttnTable j;
  j.n = 0;
  j.units = 0;
  for (int i = 0; i < t.n; ++i) {
    if (t.s[i].nsplit <= 1) continue;
    j.s[j.n] = t.s[i];
    j.s[j.n].unit0 = j.units;
    j.units += t.s[i].rows * Hq;
    ++j.n;
  }
  return j;
}

// Reorder the table's sequences by the key tiles of their longest unit, longest
// first, and renumber their units.
void longest_first(AttnTable* t, int Hkv, int tokens) {
  for (int i = 1; i < t->n; ++i) {
    const AttnSeq s = t->s[i];
    int k = i;
    for (; k > 0 && t->s[k - 1].chunk < s.chunk; --k) t->s[k] = t->s[k - 1];
    t->s[k] = s;
  }
  int units = 0;
  for (int i = 0; i < t->n; ++i) {
    t->s[i].unit0 = units;
    units += (t->s[i].rows + tokens - 1) / tokens * Hkv * t->s[i].nsplit;
  }
}

dosa_status check_cache_call(const AttnHandle* h, const dosa_cache4* cache,
                             const int64_t* seq_offsets, int B) {
  if (!h || !cache_ok(cache)) return DOSA_ERR_INVALID_ARG;
  const dosa_status st = check_batch(seq_offsets, B);
  if (st != DOSA_OK) return st;
  // every sequence's slots lie in the cache
  if (seq_offsets[3 * B + 1] > cache->capacity) return DOSA_ERR_INVALID_ARG;
  return DOSA_OK;
}

// Append and read: tables whose units are the rows of the batch.
template <class F>
dosa_status for_row_tables(const int64_t* so, int B, F launch) {
  AttnTable t;
  for (int b = 0; b < B;) {
    t.n = 0;
    t.units = 0;
    for (; b < B && t.n < kSeqsPerLaunch; ++b) {
      AttnSeq s = seq_of(so, b);
      if (s.rows == 0) continue;
      s.unit0 = t.units;
      t.units += s.rows;
      t.s[t.n++] = s;
    }
    if (t.units > 0 && launch(t) != cudaSuccess) return DOSA_ERR_CUDA;
  }
  return DOSA_OK;
}

// Spans out of order are compared pairwise.
constexpr int kUnorderedSpans = 4096;

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

}  // namespace

extern "C" {

void dosa_attn_config_default(dosa_attn_config* cfg) {
  if (!cfg) return;
  cfg->Hq = 64;
  cfg->Hkv = 8;
  cfg->d = kHeadDim;
  cfg->dtype = DOSA_BF16;
  cfg->scale = 0.f;
}

dosa_status dosa_attn_create(const dosa_attn_config* cfg, dosa_attn_t* out) {
  if (!cfg || !out) return DOSA_ERR_INVALID_ARG;
  *out = nullptr;
  if (cfg->Hq < 1 || cfg->Hkv < 1 || cfg->Hq > 4096 || cfg->Hq % cfg->Hkv != 0 ||
      !std::isfinite(cfg->scale) || cfg->scale < 0.f)
    return DOSA_ERR_INVALID_ARG;
  if (cfg->d != kHeadDim || cfg->Hq / cfg->Hkv > 128 ||
      (cfg->dtype != DOSA_BF16 && cfg->dtype != DOSA_FP16))
    return DOSA_ERR_UNSUPPORTED;
  AttnHandle* h = new (std::nothrow) AttnHandle;
  if (!h) return DOSA_ERR_INVALID_ARG;
  h->cfg = *cfg;
  h->G = cfg->Hq / cfg->Hkv;
  const double scale = cfg->scale != 0.f ? (double)cfg->scale : 1.0 / std::sqrt((double)kHeadDim);
  h->scale_log2 = (float)(scale * 1.4426950408889634);
  h->fp16 = cfg->dtype == DOSA_FP16;
  *out = reinterpret_cast<dosa_attn_t>(h);
  return DOSA_OK;
}

void dosa_attn_destroy(dosa_attn_t h) { delete reinterpret_cast<AttnHandle*>(h); }

dosa_status dosa_attn_prompt_workspace_size(dosa_attn_t hh, const int64_t* seq_offsets, int B,
                                            size_t* bytes) {
  const AttnHandle* h = handle(hh);
  if (!h || !bytes) return DOSA_ERR_INVALID_ARG;
  const dosa_status st = check_batch(seq_offsets, B);
  if (st != DOSA_OK) return st;
  *bytes = layout(h, prompt_plan(h, seq_offsets, B).vectors, 0, 0, false).total;
  return DOSA_OK;
}

dosa_status dosa_attn_prompt(dosa_attn_t hh, const dosa_rows* q, const dosa_rows* k,
                             const dosa_rows* v, const int64_t* seq_offsets, int B,
                             const dosa_rows* out, float* lse, void* workspace, size_t ws_bytes,
                             void* stream_) {
  const AttnHandle* h = handle(hh);
  if (!h) return DOSA_ERR_INVALID_ARG;
  const dosa_status st = check_batch(seq_offsets, B);
  if (st != DOSA_OK) return st;
  const int64_t Tq = seq_offsets[3 * B], S = seq_offsets[3 * B + 1];
  if (!rows_ok(q, h->cfg.Hq, Tq) || !rows_ok(k, h->cfg.Hkv, S) || !rows_ok(v, h->cfg.Hkv, S) ||
      !out_rows_ok(out, h->cfg.Hq, Tq) ||
      !aligned(lse, 4))
    return DOSA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return DOSA_ERR_INVALID_ARG;
  const Plan plan = prompt_plan(h, seq_offsets, B);
  const Layout L = layout(h, plan.vectors, 0, 0, false);
  if (ws_bytes < L.total) return DOSA_ERR_WORKSPACE;
  if (Tq == 0) return DOSA_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part_o = reinterpret_cast<float*>(ws + L.part_o);
  float* part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  int64_t part0 = 0;
  AttnTable t;
  for (int b = 0; b < B;) {
    t.n = 0;
    t.units = 0;
    for (; b < B && t.n < kSeqsPerLaunch; ++b) {
      AttnSeq s = seq_of(seq_offsets, b);
      if (s.rows == 0) continue;
      int64_t tiles, units;
      prompt_shape(h, seq_offsets + 3 * b, &tiles, &units);
      s.nsplit = (int)prompt_parts(tiles, plan.chunk);
      s.chunk = (int)((tiles + s.nsplit - 1) / s.nsplit);
      units *= s.nsplit;
      if (units > kMaxRows || (t.n > 0 && t.units + units > kMaxRows)) {
        if (t.n == 0) return DOSA_ERR_UNSUPPORTED;
        break;
      }
      if (s.nsplit > 1) {
        s.part0 = part0;
        part0 += (int64_t)s.nsplit * s.rows * h->cfg.Hq;
      }
      s.unit0 = t.units;
      t.units += (int)units;
      t.s[t.n++] = s;
    }
    if (t.n == 0) continue;
    // units of a sequence run longest first; so do the sequences
    longest_first(&t, h->cfg.Hkv, prompt_tokens(h));
    if (launch_prompt(*h, rows16(q), rows16(k), rows16(v), Tq, S, t, rows16(out), lse, part_o,
                      part_lse, static_cast<int*>(workspace), stream) != cudaSuccess)
      return DOSA_ERR_CUDA;
    if (launch_join(*h, DOSA_KERNEL_PROMPT, join_table(t, h->cfg.Hq), rows16(out), lse, nullptr,
                    part_o, part_lse, stream) != cudaSuccess)
      return DOSA_ERR_CUDA;
  }
  return DOSA_OK;
}

dosa_status dosa_cache4_append(dosa_attn_t hh, const dosa_cache4* cache, const dosa_rows* k,
                               const dosa_rows* v, const int64_t* seq_offsets, int B,
                               void* stream) {
  const AttnHandle* h = handle(hh);
  const dosa_status st = check_cache_call(h, cache, seq_offsets, B);
  if (st != DOSA_OK) return st;
  const int64_t Tq = seq_offsets[3 * B];
  if (!rows_ok(k, h->cfg.Hkv, Tq) || !rows_ok(v, h->cfg.Hkv, Tq)) return DOSA_ERR_INVALID_ARG;
  return for_row_tables(seq_offsets, B, [&](const AttnTable& t) {
    return launch_cache_append(*h, cache_view(cache), rows16(k), rows16(v), t,
                               static_cast<cudaStream_t>(stream));
  });
}

dosa_status dosa_cache4_read(dosa_attn_t hh, const dosa_cache4* cache, const int64_t* seq_offsets,
                             int B, const dosa_rows* k, const dosa_rows* v, void* stream) {
  const AttnHandle* h = handle(hh);
  const dosa_status st = check_cache_call(h, cache, seq_offsets, B);
  if (st != DOSA_OK) return st;
  const int64_t Tq = seq_offsets[3 * B];
  if (!out_rows_ok(k, h->cfg.Hkv, Tq) || !out_rows_ok(v, h->cfg.Hkv, Tq))
    return DOSA_ERR_INVALID_ARG;
  return for_row_tables(seq_offsets, B, [&](const AttnTable& t) {
    return launch_cache_read(*h, cache_view(cache), rows16(k), rows16(v), t,
                             static_cast<cudaStream_t>(stream));
  });
}

dosa_status dosa_cache4_attend_workspace_size(dosa_attn_t hh, const int64_t* seq_offsets, int B,
                                              int K, int add_weights, size_t* bytes) {
  const AttnHandle* h = handle(hh);
  if (!h || !bytes || K < 0 || K > kMaxRows) return DOSA_ERR_INVALID_ARG;
  const dosa_status st = check_batch(seq_offsets, B);
  if (st != DOSA_OK) return st;
  Plan plans[kWidths];
  *bytes = layout(h, attend_plans(h, seq_offsets, B, K, plans), seq_offsets[3 * B], K,
                  add_weights != 0)
               .total;
  return DOSA_OK;
}

dosa_status dosa_cache4_attend(dosa_attn_t hh, const dosa_cache4* cache, const dosa_rows* q,
                               const int64_t* seq_offsets, int B, const int32_t* sel_idx, int K,
                               int add_weights, const dosa_rows* out, float* lse,
                               void* workspace, size_t ws_bytes, void* stream_) {
  const AttnHandle* h = handle(hh);
  dosa_status st = check_cache_call(h, cache, seq_offsets, B);
  if (st != DOSA_OK) return st;
  const int64_t Tq = seq_offsets[3 * B];
  if (!rows_ok(q, h->cfg.Hq, Tq) || !out_rows_ok(out, h->cfg.Hq, Tq) || !aligned(lse, 4) || !aligned(sel_idx, 4))
    return DOSA_ERR_INVALID_ARG;
  if (sel_idx ? (K < 1 || K > kMaxRows) : K != 0) return DOSA_ERR_INVALID_ARG;
  if (add_weights && !cache->weight) return DOSA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return DOSA_ERR_INVALID_ARG;
  Plan plans[kWidths];
  const Layout L = layout(h, attend_plans(h, seq_offsets, B, K, plans), Tq, K, add_weights != 0);
  if (ws_bytes < L.total) return DOSA_ERR_WORKSPACE;
  // the weights over every key read q again when out has been written
  if (add_weights && !sel_idx && Tq > 0 && out->ptr == q->ptr) return DOSA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* part_o = reinterpret_cast<float*>(ws + L.part_o);
  float* part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  float* lse2 = add_weights ? reinterpret_cast<float*>(ws + L.lse2) : nullptr;
  const bool list_weights = add_weights && K;
  float* row_weight = list_weights ? reinterpret_cast<float*>(ws + L.row_weight) : nullptr;
  float* scores = list_weights ? reinterpret_cast<float*>(ws + L.scores) : nullptr;
  const int64_t row_limit = list_weights ? score_rows(h, Tq, K) : Tq;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const Cache4View c = cache_view(cache);
  const bool selected = sel_idx != nullptr;
  int64_t part0 = 0;
  // launches take sequences of one column width each; narrow ones first
  AttnTable t;
  for (int i = 0; i < kWidths; ++i) {
    const int width = 8 << i;
    const Plan& plan = plans[i];
    int r0 = 0;                                    // rows of sequence b already launched
    for (int b = 0; b < B;) {
      t.n = 0;
      t.units = 0;
      int64_t rows = 0;
      while (b < B && t.n < kSeqsPerLaunch && (rows < row_limit || t.n == 0)) {
        AttnSeq s = seq_of(seq_offsets, b);
        const int all = s.rows;
        if (all == 0 || attend_columns(*h, all, selected) != width) {
          ++b;
          continue;
        }
        if (list_weights) {
          s.q0 += r0;
          s.pos0 += r0;
          s.rows -= r0;
          if (s.rows > row_limit - rows) s.rows = (int)(row_limit - rows);
        }
        const int64_t len = selected ? K : (int64_t)s.pos0 + s.rows;
        s.chunk = plan.chunk;
        s.nsplit = (int)((len + plan.chunk - 1) / plan.chunk);
        const int64_t units = attend_groups(h, s.rows, selected) * s.nsplit;
        if (units > kMaxRows || (t.n > 0 && t.units + units > kMaxRows)) {
          if (t.n == 0) return DOSA_ERR_UNSUPPORTED;
          break;
        }
        if (s.nsplit > 1) {
          s.part0 = part0;
          part0 += (int64_t)s.nsplit * s.rows * h->cfg.Hq;
        }
        s.unit0 = t.units;
        t.units += (int)units;
        rows += s.rows;
        t.s[t.n++] = s;
        r0 += s.rows;
        if (r0 == all) {
          r0 = 0;
          ++b;
        }
      }
      if (t.n == 0) continue;
      if (launch_attend(*h, c, rows16(q), t, sel_idx, K, rows16(out), lse, lse2, part_o, part_lse,
                        scores, stream) != cudaSuccess)
        return DOSA_ERR_CUDA;
      const AttnTable j = join_table(t, h->cfg.Hq);
      if (launch_join(*h, DOSA_KERNEL_ATTEND, j, rows16(out), lse, lse2, part_o, part_lse, stream) !=
          cudaSuccess)
        return DOSA_ERR_CUDA;
      const cudaError_t we =
          !add_weights ? cudaSuccess
          : selected   ? launch_list_weights(*h, t, sel_idx, K, scores, lse2, row_weight, c.weight,
                                             stream)
                       : launch_attend_weights(*h, c, rows16(q), t, lse2, stream);
      if (we != cudaSuccess)
        return DOSA_ERR_CUDA;
    }
  }
  return DOSA_OK;
}

dosa_status dosa_cache4_evict(dosa_attn_t hh, const dosa_cache4* src, const dosa_cache4* dst,
                              const int64_t* spans, int B, int64_t first, int64_t last,
                              int32_t* kept_idx, int64_t kept_ld, void* stream) {
  const AttnHandle* h = handle(hh);
  if (!h || !cache_ok(src) || !cache_ok(dst) || !src->weight || !spans || B < 1 ||
      (!kept_idx && kept_ld != 0) || !aligned(kept_idx, 4) || first < 0 || last < 0 || first > kMaxRows || last > kMaxRows ||
      kept_ld < 0)
    return DOSA_ERR_INVALID_ARG;
  const size_t Hkv = (size_t)h->cfg.Hkv;
  const size_t sc = Hkv * src->capacity, dc = Hkv * dst->capacity;
  const struct { const void* p; size_t n; } from[5] = {
      {src->k_codes, sc * kVecCodes}, {src->k_params, sc * kVecParams},
      {src->v_codes, sc * kVecCodes}, {src->v_params, sc * kVecParams},
      {src->weight, (size_t)src->capacity * 4}};
  const struct { const void* p; size_t n; } to[5] = {
      {dst->k_codes, dc * kVecCodes}, {dst->k_params, dc * kVecParams},
      {dst->v_codes, dc * kVecCodes}, {dst->v_params, dc * kVecParams},
      {dst->weight, (size_t)dst->capacity * 4}};
  for (const auto& a : from)
    for (const auto& b : to)
      if (overlaps(a.p, a.n, b.p, b.n)) return DOSA_ERR_INVALID_ARG;
  int64_t end = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t *s = spans + 4 * b, n = s[1], keep = s[3];
    if (s[0] < 0 || n < 0 || s[2] < 0 || keep < 0 || n > kMaxRows) return DOSA_ERR_INVALID_ARG;
    const int64_t kept = n < keep ? n : keep;
    if (n > keep && first + last > keep) return DOSA_ERR_INVALID_ARG;
    if (kept > kept_ld) return DOSA_ERR_INVALID_ARG;
    if (s[0] > src->capacity - n || s[2] > dst->capacity - kept) return DOSA_ERR_INVALID_ARG;
    // destination spans must be disjoint
    if (kept == 0) continue;
    if (s[2] >= end) {                             // behind all before it
      end = s[2] + kept;
      continue;
    }
    if (B > kUnorderedSpans) return DOSA_ERR_UNSUPPORTED;
    for (int e = 0; e < b; ++e) {
      const int64_t* o = spans + 4 * e;
      const int64_t ok = o[1] < o[3] ? o[1] : o[3];
      if (s[2] < o[2] + ok && o[2] < s[2] + kept) return DOSA_ERR_INVALID_ARG;
    }
  }
  if (kept_ld == 0) return DOSA_OK;                // nothing is kept or listed
  EvictTable t;
  for (int b = 0; b < B;) {
    t.n = 0;
    int64_t total = 0;
    int max_n = 0;
    for (; b < B && t.n < kSeqsPerLaunch; ++b) {
      const int64_t* s = spans + 4 * b;
      EvictSeq& e = t.s[t.n];
      e.src0 = s[0];
      e.dst0 = s[2];
      e.n = (int)s[1];
      e.keep = (int)(s[1] < s[3] ? s[1] : s[3]);
      if (t.n > 0 && total + e.keep > kMaxRows / 2) break;
      e.j0 = (int)total;
      e.out = b;
      total += e.keep;
      if (e.n > max_n) max_n = e.n;
      ++t.n;
    }
    // the move indexes 4 chunks per token with 32 bits
    if (total > kMaxRows / 2) return DOSA_ERR_UNSUPPORTED;
    t.total = (int)total;
    if (launch_evict(*h, cache_view(src), cache_view(dst), t, (int)first, (int)last, max_n,
                     kept_idx, kept_ld, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return DOSA_ERR_CUDA;
  }
  return DOSA_OK;
}

}  // extern "C"
