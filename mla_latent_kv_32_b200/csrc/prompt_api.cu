// Entry points of the prompt-side operators: argument checks, the scaled RoPE
// table, the planner of the expanded attention.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <queue>
#include <vector>

#include "internal.h"

namespace mla {
namespace {

mla_status_t check_layout(int layout) {
  MLA_CHECK_ARG(layout == MLA_ROPE_INTERLEAVED || layout == MLA_ROPE_HALF,
                "layout %d is neither MLA_ROPE_INTERLEAVED nor MLA_ROPE_HALF", layout);
  return MLA_OK;
}

// Whether rows (stride ld) of n_h heads (stride hs) of `width` elements are
// apart from one another, token-major or head-major: for outputs.
bool apart(long long T, long long ld, long long n_h, long long hs, long long width) {
  const bool by_token = hs >= width && (T == 1 || ld >= (n_h - 1) * hs + width);
  const bool by_head = ld >= width && (n_h == 1 || hs >= (T - 1) * ld + width);
  return by_token || by_head;
}

mla_status_t norm_append_entry(NormAppendArgs &a, int layout, mla_stream_t stream) {
  clear_error();
  MLA_CHECK_ARG(a.n_tokens >= 0, "n_tokens < 0");
  mla_status_t st = check_layout(layout);
  if (st != MLA_OK) return st;
  a.half = layout == MLA_ROPE_HALF;
  if (a.n_tokens == 0) return MLA_OK;
  MLA_CHECK_ARG(a.block_table && a.seq_idx && a.pos && a.c_kv && a.k_pe && a.rope_table,
                "NULL device pointer");
  MLA_CHECK_ARG(a.num_pages > 0 && a.batch > 0 && a.max_pages > 0 && a.max_pos > 0,
                "sizes must be positive");
  MLA_CHECK_ARG(aligned16(a.c_kv) && aligned16(a.k_pe) && aligned16(a.rope_table) &&
                    (a.w_kv == nullptr || aligned16(a.w_kv)),
                "c_kv, w_kv, k_pe and rope_table must be 16-byte aligned");
  MLA_CHECK_ARG(a.ld_c >= MLA_D_C && a.ld_c % 8 == 0, "ld_c must be >= 512 and a multiple of 8");
  MLA_CHECK_ARG(a.ld_k >= MLA_D_R && a.ld_k % 8 == 0, "ld_k must be >= 64 and a multiple of 8");
  MLA_CHECK_ARG(isfinite(a.eps) && a.eps >= 0.f, "eps must be finite and not negative");
  MLA_CHECK_ARG(a.q_dim >= 0 && a.q_dim % 8 == 0, "q_dim must be 0 or a multiple of 8");
  if (a.q_dim > 0) {
    MLA_CHECK_ARG(a.c_q && a.q_out, "NULL query latent");
    MLA_CHECK_ARG(aligned16(a.c_q) && aligned16(a.q_out) && (a.w_q == nullptr || aligned16(a.w_q)),
                  "c_q, w_q and q_out must be 16-byte aligned");
    MLA_CHECK_ARG(a.ld_q >= a.q_dim && a.ld_q % 8 == 0 && a.ld_qo >= a.q_dim && a.ld_qo % 8 == 0,
                  "ld_q and ld_qo must be >= q_dim and multiples of 8");
    MLA_CHECK_ARG(a.c_q != a.q_out || a.ld_q == a.ld_qo,
                  "q_out may be c_q itself only with the same leading dimension");
  }
  st = require_sm100();
  if (st != MLA_OK) return st;
  return launch_norm_append(a, (cudaStream_t)stream);
}

mla_status_t gather_entry(GatherArgs &a, bool fp8, mla_stream_t stream) {
  clear_error();
  MLA_CHECK_ARG(a.n_rows >= 0 && a.batch >= 0, "negative size");
  if (a.n_rows == 0 || a.batch == 0) return MLA_OK;
  MLA_CHECK_ARG(a.cache && a.block_table && a.cu_rows && a.rows, "NULL device pointer");
  MLA_CHECK_ARG(!fp8 || a.scales8 != nullptr, "the FP8 cache needs its scales");
  MLA_CHECK_ARG(a.num_pages > 0 && a.max_pages > 0, "num_pages and max_pages must be positive");
  MLA_CHECK_ARG(aligned16(a.cache) && aligned16(a.rows) && (!fp8 || aligned16(a.scales8)),
                "cache, scales and rows must be 16-byte aligned");
  MLA_CHECK_ARG(a.ld_rows >= MLA_ROW && a.ld_rows % 8 == 0,
                "ld_rows must be >= 576 and a multiple of 8");
  mla_status_t st = require_sm100();
  if (st != MLA_OK) return st;
  return launch_cache_gather(a, (cudaStream_t)stream);
}

// -------------------------------------------------- planner of the prompt ---

size_t align16(size_t x) { return (x + 15) & ~(size_t)15; }

// (query tile, head) units of a batch; -1 when a length is negative
long long prefill_units(const int32_t *q_lens, int batch, int n_h) {
  long long tiles = 0;
  for (int b = 0; b < batch; ++b) {
    if (q_lens[b] < 0) return -1;
    tiles += ((long long)q_lens[b] + kPrefillRows - 1) / kPrefillRows;
  }
  return tiles * n_h;
}

// Units cut into parts of at least total / (kMaxCuts * num_ctas) tiles make at
// most this many items.
constexpr int kMaxCuts = 4;

size_t prefill_bytes(long long units, int num_ctas) {
  return sizeof(PrefillHeader) + align16(sizeof(int32_t) * ((size_t)num_ctas + 1)) +
         ((size_t)units + (size_t)kMaxCuts * num_ctas) * sizeof(PrefillItem) +
         (size_t)units * sizeof(PrefillCombine);
}

mla_status_t prefill_ctas(int *num_ctas) {
  if (*num_ctas > 0) return MLA_OK;
  return device_info(num_ctas, nullptr, nullptr);   // one CTA per SM
}

// Costs in eighths of a full item's key tile (about 1.8 us); a tile that the
// streams take in turn costs about 1.45. An item: query load, first scores, last
// output, epilogue. A merge pass: its launch, and the partial rows written and
// read, 1 KB each, by all SMs together.
constexpr int kTileCost = 8, kTurnCost = 6, kItemCost = 12, kMergeCost = 20;
constexpr int kPartialRowsPerCost = 1300;

struct Unit {
  int q_row, q_rows, h, k_row, k_len, lim0, tiles;
};
struct Piece {
  int unit, begin, end, tile_cost;
};

long long piece_cost(const Piece &p) {
  return (long long)(p.end - p.begin) * p.tile_cost + kItemCost;
}

// No dealing ends before this.
long long cost_bound(const std::vector<Piece> &pieces, int lists) {
  long long sum = 0, longest = 0;
  for (const Piece &p : pieces) {
    sum += piece_cost(p);
    longest = std::max(longest, piece_cost(p));
  }
  return std::max(longest, (sum + lists - 1) / lists);
}

// Deals the pieces to the lists, each to the list with the least work so far:
// longest first, or in their own order. list_of[i]: piece i's list. Returns the
// busiest list's cost.
long long deal_in(const std::vector<Piece> &pieces, int lists, bool longest_first,
                  std::vector<int> &order, std::vector<int> &list_of) {
  order.resize(pieces.size());
  list_of.resize(pieces.size());
  for (size_t i = 0; i < order.size(); ++i) order[i] = (int)i;
  if (longest_first)
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) {
      return piece_cost(pieces[x]) > piece_cost(pieces[y]);
    });
  typedef std::pair<long long, int> Load;
  std::vector<Load> store;
  store.reserve(lists);
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> heap(std::greater<Load>(),
                                                                        std::move(store));
  for (int c = 0; c < lists; ++c) heap.push({0, c});
  long long worst = 0;
  for (int i : order) {
    Load l = heap.top();
    heap.pop();
    list_of[i] = l.second;
    l.first += piece_cost(pieces[i]);
    worst = std::max(worst, l.first);
    heap.push(l);
  }
  return worst;
}

// In their own order the query tiles of a head run side by side and share its
// keys and values in L2; longest first balances better when lengths differ.
// The first is taken while it ends at most 1/32 later. (`order`: the pieces in
// the order they were dealt.)
long long deal(const std::vector<Piece> &pieces, int lists, std::vector<int> &order,
               std::vector<int> &list_of) {
  const long long own = deal_in(pieces, lists, false, order, list_of);
  const long long bound = cost_bound(pieces, lists);
  if (own <= bound + bound / 32) return own;
  const long long sorted = deal_in(pieces, lists, true, order, list_of);
  if (own > sorted + sorted / 32) return sorted;
  return deal_in(pieces, lists, false, order, list_of);
}

// The units in parts of at most `most` tiles; units of more than `rows` query
// rows stay whole. *partials: the rows of partial results that this takes.
std::vector<Piece> cut(const std::vector<Unit> &units, int most, int rows, long long *partials) {
  std::vector<Piece> pieces;
  pieces.reserve(units.size());
  *partials = 0;
  for (size_t u = 0; u < units.size(); ++u) {
    const int n = units[u].tiles;
    const int parts = units[u].q_rows > rows
                          ? 1
                          : (int)std::max(1ll, ((long long)n + most - 1) / most);
    for (int p = 0; p < parts; ++p)
      pieces.push_back({(int)u, (int)((long long)n * p / parts),
                        (int)((long long)n * (p + 1) / parts),
                        units[u].q_rows <= kTurnRows ? kTurnCost : kTileCost});
    if (parts > 1) *partials += (long long)parts * units[u].q_rows;
  }
  return pieces;
}

mla_status_t build_prefill_plan(const int32_t *q_lens, const int32_t *kv_lens, int batch, int n_h,
                                int causal, int num_ctas, int max_split, unsigned char *base,
                                size_t need, mla_plan_info_t *info) {
  std::vector<Unit> units;
  long long q0 = 0, k0 = 0, total = 0;
  int longest = 0;
  size_t small_units = 0;
  for (int b = 0; b < batch; ++b) {
    const int lq = q_lens[b], lk = kv_lens[b];
    for (int h = 0; h < n_h; ++h)
      for (int r = (lq - 1) / kPrefillRows * kPrefillRows; r >= 0 && lq > 0; r -= kPrefillRows) {
        const int rows = std::min(kPrefillRows, lq - r);
        const long long lim0 = causal ? (long long)lk - lq + r + 1 : lk;
        const long long seen = std::min<long long>(lk, causal ? lim0 + rows - 1 : lk);
        const int tiles = seen <= 0 ? 0 : (int)((seen + kPrefillKeys - 1) / kPrefillKeys);
        units.push_back({(int)q0 + r, rows, h, (int)k0, lk, (int)lim0, tiles});
        total += tiles;
        longest = std::max(longest, tiles);
        small_units += rows <= kPrefillRows / 2;
      }
    q0 += lq;
    k0 += lk;
  }
  // Whole units, or units cut into parts of at most a 2 / (k num_ctas) share of
  // all tiles (all units, or only those of up to 128 rows, whose partial
  // results are small), whichever ends first by the estimate.
  long long partials = 0;
  std::vector<Piece> best = cut(units, INT_MAX, kPrefillRows, &partials);
  std::vector<int> order, list_of;
  if (max_split != 1 && longest > 0) {
    long long cost = max_split < 0 ? deal(best, num_ctas, order, list_of) : LLONG_MAX;
    for (int k = 2; k <= 2 * kMaxCuts; ++k) {
      const int most = (int)std::max<long long>(
          2, (2 * total + (long long)k * num_ctas - 1) / ((long long)k * num_ctas));
      if (most >= longest) continue;
      for (int c = 0; c < (k == 2 ? 8 : 2); ++c) {
        if ((c & 1) && small_units * (units.size() - small_units) == 0) continue;
        // (a little more than the share, so that the parts of a few long units
        // can come out one a list)
        std::vector<Piece> pieces = cut(units, most + most * (c >> 1) / 16,
                                        c & 1 ? kPrefillRows / 2 : kPrefillRows, &partials);
        const long long merge = kMergeCost + partials / kPartialRowsPerCost;
        if (cost_bound(pieces, num_ctas) + merge >= cost) continue;
        const long long est = deal(pieces, num_ctas, order, list_of) + merge;
        if (est < cost) {
          cost = est;
          best.swap(pieces);
        }
      }
    }
  }
  const int lists = units.empty() ? 0 : (int)std::min<long long>(num_ctas, best.size());
  if (lists > 0) deal(best, lists, order, list_of);

  // partial-result rows and merges of the units that were cut (their pieces
  // follow one another)
  std::vector<int> slot(best.size(), -1);
  std::vector<PrefillCombine> comb;
  long long rows = 0;
  int merge_rows = 0;
  for (size_t i = 0; i < best.size();) {
    size_t j = i;
    while (j < best.size() && best[j].unit == best[i].unit) ++j;
    if (j - i > 1) {
      const Unit &u = units[best[i].unit];
      comb.push_back({u.q_row, u.q_rows, u.h, (int)rows, (int)(j - i), {0, 0, 0}});
      merge_rows = std::max(merge_rows, u.q_rows);
      for (size_t k = i; k < j; ++k) {
        slot[k] = (int)rows;
        rows += u.q_rows;
        if (rows > INT_MAX) return fail(MLA_ERR_UNSUPPORTED, "too many partial results");
      }
    }
    i = j;
  }
  PrefillHeader h = {};
  h.magic = kPrefillMagic;
  h.version = kPrefillVersion;
  h.q_total = (int)q0;
  h.k_total = (int)k0;
  h.n_h = n_h;
  h.causal = causal ? 1 : 0;
  h.num_items = lists > 0 ? (int)best.size() : 0;
  h.num_ctas = lists;
  h.num_partials = (int)rows;
  h.num_combine = (int)comb.size();
  h.max_merge_rows = merge_rows;
  h.cta_off = (int)sizeof(PrefillHeader);
  h.items_off = h.cta_off + (int)align16(sizeof(int32_t) * ((size_t)num_ctas + 1));
  const size_t comb_off = (size_t)h.items_off + (size_t)h.num_items * sizeof(PrefillItem);
  const size_t used = comb_off + comb.size() * sizeof(PrefillCombine);
  if (used > need)
    return fail(MLA_ERR_INVALID_ARGUMENT, "planner produced %zu bytes (bound %zu)", used, need);
  h.combine_off = (int)comb_off;
  memset(base, 0, used);
  memcpy(base, &h, sizeof(h));
  int32_t *cta_begin = reinterpret_cast<int32_t *>(base + h.cta_off);
  PrefillItem *items = reinterpret_cast<PrefillItem *>(base + h.items_off);
  for (int l : list_of) ++cta_begin[l + 1];
  for (int c = 0; c < lists; ++c) cta_begin[c + 1] += cta_begin[c];
  std::vector<int> at(cta_begin, cta_begin + lists);
  // full items first: the kernel lays its shared memory out for one kind, then for
  // the other
  int turns = 0;
  for (int small = 0; small < 2; ++small)
    for (int i : order) {
      const Unit &u = units[best[i].unit];
      const bool in_turn = u.q_rows <= kTurnRows && best[i].end - best[i].begin >= kTurnTiles;
      if (in_turn != (small != 0)) continue;
      items[at[list_of[i]]++] = PrefillItem{u.q_row, u.q_rows, u.h, u.k_row, u.k_len, u.lim0,
                                            best[i].begin, best[i].end, slot[i], {0, 0, 0}};
      turns |= in_turn;
    }
  reinterpret_cast<PrefillHeader *>(base)->turns = turns;
  if (!comb.empty()) memcpy(base + comb_off, comb.data(), comb.size() * sizeof(PrefillCombine));
  if (info) {
    info->num_items = h.num_items;
    info->num_ctas = lists;
    info->num_partials = (int)rows;
    info->num_combine = h.num_combine;
    info->plan_bytes = used;
    info->workspace_bytes = prefill_ws_bytes((int)rows);
  }
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" {

mla_status_t mla_rope_table_scaled(float *table, int max_pos, int dim, double base, int method,
                                   double factor, int original_max_pos, double beta_fast,
                                   double beta_slow, double attn_factor) {
  clear_error();
  MLA_CHECK_ARG(table != nullptr, "rope table pointer is NULL");
  MLA_CHECK_ARG(max_pos > 0, "max_pos must be positive (got %d)", max_pos);
  MLA_CHECK_ARG(dim >= 2 && dim % 2 == 0 && dim <= MLA_ROPE_MAX_DIM,
                "dim must be even and in [2, %d] (got %d)", MLA_ROPE_MAX_DIM, dim);
  MLA_CHECK_ARG(isfinite(base) && base > 1.0, "RoPE base must exceed 1 (got %g)", base);
  MLA_CHECK_ARG(method >= MLA_ROPE_SCALE_NONE && method <= MLA_ROPE_SCALE_YARN,
                "unknown scaling method %d", method);
  MLA_CHECK_ARG(method == MLA_ROPE_SCALE_NONE || (isfinite(factor) && factor >= 1.0),
                "factor must be at least 1 (got %g)", factor);
  MLA_CHECK_ARG(isfinite(attn_factor) && attn_factor > 0.0, "attn_factor must be positive");
  MLA_CHECK_ARG(method != MLA_ROPE_SCALE_NTK || dim > 2, "NTK scaling needs dim > 2");
  double theta[MLA_ROPE_MAX_DIM / 2];
  const double b = method == MLA_ROPE_SCALE_NTK ? base * pow(factor, dim / (dim - 2.0)) : base;
  for (int j = 0; j < dim / 2; ++j) theta[j] = 1.0 / pow(b, 2.0 * j / dim);
  if (method == MLA_ROPE_SCALE_LINEAR)
    for (int j = 0; j < dim / 2; ++j) theta[j] /= factor;
  if (method == MLA_ROPE_SCALE_YARN) {
    MLA_CHECK_ARG(original_max_pos > 0, "original_max_pos must be positive");
    MLA_CHECK_ARG(isfinite(beta_fast) && beta_fast > beta_slow && beta_slow > 0.0,
                  "beta_fast must exceed beta_slow, and both be positive");
    // the pair that makes n turns over the original context
    const double two_pi = 6.283185307179586476925286766559;
    auto pair_of = [&](double n) {
      return dim * log(original_max_pos / (n * two_pi)) / (2.0 * log(base));
    };
    const double low = std::max(0.0, floor(pair_of(beta_fast)));
    double high = std::min(dim - 1.0, ceil(pair_of(beta_slow)));
    if (high <= low) high = low + 0.001;
    for (int j = 0; j < dim / 2; ++j) {
      const double ramp = std::min(1.0, std::max(0.0, (j - low) / (high - low)));
      theta[j] = theta[j] * (1.0 - ramp) + theta[j] / factor * ramp;
    }
  }
  for (int p = 0; p < max_pos; ++p)
    for (int j = 0; j < dim / 2; ++j) {
      const double th = p * theta[j];
      table[(size_t)p * dim + 2 * j] = (float)(attn_factor * cos(th));
      table[(size_t)p * dim + 2 * j + 1] = (float)(attn_factor * sin(th));
    }
  return MLA_OK;
}

mla_status_t mla_rope_heads(const mla_bf16_t *x, int ld_x, int hs_x, const int32_t *pos,
                            const float *rope_table, int max_pos, int T, int n_h, int dim,
                            int layout, mla_bf16_t *out, int ld_o, int hs_o, uint32_t *status,
                            mla_stream_t stream) {
  clear_error();
  MLA_CHECK_ARG(T >= 0 && n_h >= 0, "negative size");
  mla_status_t st = check_layout(layout);
  if (st != MLA_OK) return st;
  if (T == 0 || n_h == 0) return MLA_OK;
  if (dim < 16 || dim > MLA_ROPE_MAX_DIM || dim % 16 != 0)
    return fail(MLA_ERR_UNSUPPORTED, "dim = %d (supported: multiples of 16 up to %d)", dim,
                MLA_ROPE_MAX_DIM);
  MLA_CHECK_ARG(x && pos && rope_table && out, "NULL device pointer");
  MLA_CHECK_ARG(max_pos > 0, "max_pos must be positive");
  MLA_CHECK_ARG(aligned16(x) && aligned16(out) && aligned16(rope_table),
                "x, out and rope_table must be 16-byte aligned");
  MLA_CHECK_ARG(ld_x > 0 && hs_x >= dim && ld_x % 8 == 0 && hs_x % 8 == 0 && ld_o > 0 &&
                    hs_o >= dim && ld_o % 8 == 0 && hs_o % 8 == 0,
                "strides must be positive multiples of 8, head strides at least dim");
  MLA_CHECK_ARG(x != out || (ld_x == ld_o && hs_x == hs_o),
                "out may be x itself only with the same strides");
  MLA_CHECK_ARG(apart(T, ld_o, n_h, hs_o, dim), "rows of out overlap");
  st = require_sm100();
  if (st != MLA_OK) return st;
  RopeHeadsArgs a;
  a.x = x;
  a.ld_x = ld_x;
  a.hs_x = hs_x;
  a.pos = pos;
  a.rope_table = rope_table;
  a.max_pos = max_pos;
  a.T = T;
  a.n_h = n_h;
  a.dim = dim;
  a.half = layout == MLA_ROPE_HALF;
  a.out = out;
  a.ld_o = ld_o;
  a.hs_o = hs_o;
  a.status = status;
  return launch_rope_heads(a, (cudaStream_t)stream);
}

mla_status_t mla_norm_append(mla_bf16_t *cache, int num_pages, const int32_t *block_table,
                             int batch, int max_pages, const int32_t *seq_idx, const int32_t *pos,
                             const mla_bf16_t *c_kv, int ld_c, const mla_bf16_t *w_kv,
                             const mla_bf16_t *k_pe, int ld_k, const float *rope_table,
                             int max_pos, int layout, float eps, int n_tokens,
                             const mla_bf16_t *c_q, int ld_q, const mla_bf16_t *w_q, int q_dim,
                             mla_bf16_t *q_out, int ld_qo, uint32_t *status, mla_stream_t stream) {
  NormAppendArgs a = {cache, nullptr, nullptr, num_pages, block_table, batch, max_pages, seq_idx,
                      pos, c_kv, ld_c, w_kv, k_pe, ld_k, rope_table, max_pos, 0, eps, n_tokens,
                      c_q, ld_q, w_q, q_dim, q_out, ld_qo, status};
  if (n_tokens > 0) {
    clear_error();
    MLA_CHECK_ARG(cache != nullptr && aligned16(cache), "cache must be a 16-byte aligned pointer");
  }
  return norm_append_entry(a, layout, stream);
}

mla_status_t mla_norm_append_fp8(uint8_t *cache, float *scales, int num_pages,
                                 const int32_t *block_table, int batch, int max_pages,
                                 const int32_t *seq_idx, const int32_t *pos,
                                 const mla_bf16_t *c_kv, int ld_c, const mla_bf16_t *w_kv,
                                 const mla_bf16_t *k_pe, int ld_k, const float *rope_table,
                                 int max_pos, int layout, float eps, int n_tokens,
                                 const mla_bf16_t *c_q, int ld_q, const mla_bf16_t *w_q, int q_dim,
                                 mla_bf16_t *q_out, int ld_qo, uint32_t *status,
                                 mla_stream_t stream) {
  NormAppendArgs a = {nullptr, cache, scales, num_pages, block_table, batch, max_pages, seq_idx,
                      pos, c_kv, ld_c, w_kv, k_pe, ld_k, rope_table, max_pos, 0, eps, n_tokens,
                      c_q, ld_q, w_q, q_dim, q_out, ld_qo, status};
  if (n_tokens > 0) {
    clear_error();
    MLA_CHECK_ARG(cache != nullptr && aligned16(cache), "cache must be a 16-byte aligned pointer");
    MLA_CHECK_ARG(scales != nullptr && aligned16(scales),
                  "scales must be a 16-byte aligned pointer");
  }
  return norm_append_entry(a, layout, stream);
}

mla_status_t mla_cache_gather(const mla_bf16_t *cache, int num_pages, const int32_t *block_table,
                              int batch, int max_pages, const int32_t *start,
                              const int32_t *cu_rows, int n_rows, mla_bf16_t *rows, int ld_rows,
                              uint32_t *status, mla_stream_t stream) {
  GatherArgs a = {cache, nullptr, num_pages, block_table, batch, max_pages, start, cu_rows, n_rows,
                  rows, ld_rows, status};
  return gather_entry(a, false, stream);
}

mla_status_t mla_cache_gather_fp8(const uint8_t *cache, const float *scales, int num_pages,
                                  const int32_t *block_table, int batch, int max_pages,
                                  const int32_t *start, const int32_t *cu_rows, int n_rows,
                                  mla_bf16_t *rows, int ld_rows, uint32_t *status,
                                  mla_stream_t stream) {
  GatherArgs a = {cache, scales, num_pages, block_table, batch, max_pages, start, cu_rows, n_rows,
                  rows, ld_rows, status};
  return gather_entry(a, true, stream);
}

size_t mla_prefill_plan_bytes(const int32_t *q_lens, int batch, int n_h, int num_ctas) {
  if (batch < 0 || n_h < 1 || (batch > 0 && q_lens == nullptr)) return 0;
  if (prefill_ctas(&num_ctas) != MLA_OK) return 0;
  const long long units = prefill_units(q_lens, batch, n_h);
  const size_t need = units < 0 ? 0 : prefill_bytes(units, num_ctas);
  return need > INT_MAX ? 0 : need;
}

mla_status_t mla_prefill_plan(const int32_t *q_lens, const int32_t *kv_lens, int batch, int n_h,
                              int causal, int num_ctas, int max_split, void *plan,
                              size_t plan_bytes, mla_plan_info_t *info) {
  clear_error();
  MLA_CHECK_ARG(batch >= 0, "batch < 0");
  if (n_h < 1 || n_h > 128) return fail(MLA_ERR_UNSUPPORTED, "n_h = %d (supported: 1..128)", n_h);
  MLA_CHECK_ARG(batch == 0 || (q_lens != nullptr && kv_lens != nullptr), "lengths are NULL");
  MLA_CHECK_ARG(plan != nullptr, "plan is NULL");
  long long tq = 0, tk = 0;
  for (int b = 0; b < batch; ++b) {
    MLA_CHECK_ARG(q_lens[b] >= 0 && kv_lens[b] >= 0, "sequence %d has a negative length", b);
    tq += q_lens[b];
    tk += kv_lens[b];
  }
  if (tq > INT_MAX || tk > INT_MAX) return fail(MLA_ERR_UNSUPPORTED, "over 2^31 - 1 rows");
  mla_status_t st = prefill_ctas(&num_ctas);
  if (st != MLA_OK) return st;
  const size_t need = prefill_bytes(prefill_units(q_lens, batch, n_h), num_ctas);
  if (need > INT_MAX) return fail(MLA_ERR_UNSUPPORTED, "the plan would take %zu bytes", need);
  if (plan_bytes < need)
    return fail(MLA_ERR_WORKSPACE_TOO_SMALL, "plan buffer %zu B < %zu B", plan_bytes, need);
  try {
    return build_prefill_plan(q_lens, kv_lens, batch, n_h, causal, num_ctas, max_split,
                              static_cast<unsigned char *>(plan), need, info);
  } catch (const std::bad_alloc &) {
    return fail(MLA_ERR_INVALID_ARGUMENT, "out of host memory while planning");
  }
}

mla_status_t mla_prefill_attention(const mla_bf16_t *q_nope, int ld_qn, int hs_qn,
                                   const mla_bf16_t *q_pe, int ld_qp, int hs_qp,
                                   const mla_bf16_t *k_nope, int ld_kn, int hs_kn,
                                   const mla_bf16_t *v, int ld_v, int hs_v, const mla_bf16_t *k_pe,
                                   int ld_kp, int T_q, int T_k, int n_h, float scale,
                                   const void *plan_host, const void *plan_dev, void *workspace,
                                   size_t workspace_bytes, mla_bf16_t *o, int ld_o, int hs_o,
                                   float *lse, uint32_t *status, mla_stream_t stream) {
  clear_error();
  MLA_CHECK_ARG(plan_host != nullptr && plan_dev != nullptr, "plan pointers are NULL");
  const PrefillHeader *ph = static_cast<const PrefillHeader *>(plan_host);
  MLA_CHECK_ARG(ph->magic == kPrefillMagic && ph->version == kPrefillVersion, "not a prefill plan");
  MLA_CHECK_ARG(ph->n_h == n_h, "plan was built for n_h %d", ph->n_h);
  MLA_CHECK_ARG(T_q >= ph->q_total && T_k >= ph->k_total,
                "the plan covers %d query rows and %d keys, the buffers hold %d and %d",
                ph->q_total, ph->k_total, T_q, T_k);
  if (ph->num_items == 0) return MLA_OK;
  MLA_CHECK_ARG(q_nope && q_pe && o, "NULL device pointer");
  MLA_CHECK_ARG(ph->k_total == 0 || (k_nope && v && k_pe), "NULL keys or values");
  MLA_CHECK_ARG(aligned16(q_nope) && aligned16(q_pe) && aligned16(o) && aligned16(plan_dev) &&
                    (workspace == nullptr || aligned16(workspace)) &&
                    (ph->k_total == 0 || (aligned16(k_nope) && aligned16(v) && aligned16(k_pe))),
                "pointers must be 16-byte aligned");
  const bool keys = ph->k_total > 0;
  // without keys their strides are not read
  const int wide[] = {ld_qn, hs_qn, ld_o, hs_o, ld_kn, hs_kn, ld_v, hs_v};
  const int narrow[] = {ld_qp, hs_qp, ld_kp};
  for (int i = 0; i < (keys ? 8 : 4); ++i)
    MLA_CHECK_ARG(wide[i] >= 128 && wide[i] % 8 == 0,
                  "strides of q_nope, k_nope, v and o must be multiples of 8 and at least 128");
  for (int i = 0; i < (keys ? 3 : 2); ++i)
    MLA_CHECK_ARG(narrow[i] >= 64 && narrow[i] % 8 == 0,
                  "strides of q_pe and k_pe must be multiples of 8 and at least 64");
  MLA_CHECK_ARG(apart(T_q, ld_o, n_h, hs_o, MLA_D_V), "rows of o overlap");
  MLA_CHECK_ARG(isfinite(scale) && scale > 0.f, "scale must be finite and positive");
  const size_t need = prefill_ws_bytes(ph->num_partials);
  if (ph->num_partials > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(MLA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu B < %zu B", workspace_bytes, need);
  mla_status_t st = require_sm100();
  if (st != MLA_OK) return st;
  PrefillArgs a;
  a.q_nope = q_nope;
  a.q_pe = q_pe;
  a.k_nope = k_nope;
  a.v = v;
  a.k_pe = k_pe;
  a.ld_qn = ld_qn;
  a.hs_qn = hs_qn;
  a.ld_qp = ld_qp;
  a.hs_qp = hs_qp;
  // without keys their strides only have to be valid for a map that is not read
  a.ld_kn = keys ? ld_kn : 128;
  a.hs_kn = keys ? hs_kn : 128;
  a.ld_v = keys ? ld_v : 128;
  a.hs_v = keys ? hs_v : 128;
  a.ld_kp = keys ? ld_kp : 64;
  a.T_q = T_q;
  a.T_k = keys ? T_k : 0;
  a.n_h = n_h;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.plan_host = ph;
  a.plan_dev = static_cast<const unsigned char *>(plan_dev);
  a.ws_o = static_cast<float *>(workspace);
  a.ws_lse = workspace ? reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) +
                                                   prefill_ws_o_bytes(ph->num_partials))
                       : nullptr;
  a.o = o;
  a.ld_o = ld_o;
  a.hs_o = hs_o;
  a.lse = lse;
  a.status = status;
  return launch_prefill(a, (cudaStream_t)stream);
}

}  // extern "C"
