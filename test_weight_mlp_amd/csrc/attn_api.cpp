// C ABI of the attention half: argument validation, the plan (built on the
// host), workspace layout and the launches.  Nothing is launched and nothing is
// written unless every argument checks out; nothing here allocates or throws.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/ipttt.h"
#include "attn.h"

using ipttt::attn::JoinItem;
using ipttt::attn::KeyItem;
using ipttt::attn::kBwdKeys;
using ipttt::attn::kBwdRows;
using ipttt::attn::KeyJoin;
using ipttt::attn::kFewRows;
using ipttt::attn::kKeys;
using ipttt::attn::kPartRows;
using ipttt::attn::kMagic;
using ipttt::attn::kRows;
using ipttt::attn::kShortKeys;
using ipttt::attn::PlanHeader;
using ipttt::attn::RowItem;
using ipttt::attn::View;

namespace {

constexpr int64_t kMaxInt = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;  // workgroups of 256 threads in a grid's x dimension
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxRowStride = int64_t(1) << 22;
constexpr int64_t kMaxHeadStride = int64_t(1) << 40;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
ipttt_status hip_status(hipError_t e) { return e == hipSuccess ? IPTTT_OK : IPTTT_ERR_HIP; }

ipttt_status check_dims(int64_t heads, int64_t kv_heads, int64_t head_dim, int32_t dtype) {
  if (dtype != IPTTT_F32 && dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (heads < 1 || heads > kMaxHeads || kv_heads < 1 || kv_heads > kMaxHeads) return IPTTT_ERR_SHAPE;
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0) return IPTTT_ERR_SHAPE;
  return IPTTT_OK;
}

// One [rows, heads, D] tensor.  A tile's rows are addressed with 32-bit byte
// offsets from the tile's first row: tile_rows rows of tile_heads heads have to
// fit.  The stride of a dimension of one element is not looked at.
ipttt_status check_heads(const ipttt_heads* t, int64_t rows, int64_t heads, int64_t D, int32_t dtype,
                         int64_t tile_rows, int64_t tile_heads, View* v) {
  if (t == nullptr || t->data == nullptr) return IPTTT_ERR_NULL;
  if (!aligned(t->data, 16)) return IPTTT_ERR_ALIGN;
  const int64_t row = rows == 1 ? D : t->row_stride, head = heads == 1 ? D : t->head_stride;
  if (row < D || head < D || row % 8 != 0 || head % 8 != 0) return IPTTT_ERR_SHAPE;
  if (row > kMaxRowStride || head > kMaxHeadStride) return IPTTT_ERR_SHAPE;
  const int64_t es = dtype == IPTTT_BF16 ? 2 : 4;
  if ((tile_rows * row + (tile_heads - 1) * head + D) * es > kMaxInt - 15) return IPTTT_ERR_SHAPE;
  *v = View{t->data, row, head};
  return IPTTT_OK;
}

// ------------------------------------------------------------------- plan

ipttt_status check_attn(const ipttt_attn_problem* p) {
  if (p == nullptr) return IPTTT_ERR_NULL;
  const ipttt_status s = check_dims(p->heads, p->kv_heads, p->head_dim, p->dtype);
  if (s != IPTTT_OK) return s;
  if (p->heads % p->kv_heads != 0) return IPTTT_ERR_SHAPE;
  if (p->n_seqs < 1 || p->n_seqs > kMaxInt || p->q_rows < 0 || p->k_rows < 0) return IPTTT_ERR_SHAPE;
  const int64_t G = p->heads / p->kv_heads;
  // flat rows, and the rows and keys of a tile past them, fit 31 bits
  if (p->q_rows > (kMaxInt >> 1) / G - 512 || p->k_rows > (kMaxInt >> 1) / G - 512) return IPTTT_ERR_SHAPE;
  if (p->q_start == nullptr || p->q_len == nullptr || p->k_start == nullptr || p->k_len == nullptr)
    return IPTTT_ERR_NULL;
  int64_t end = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i) {
    if (p->q_len[i] < 0 || p->k_len[i] < 0 || p->q_start[i] < end || p->k_start[i] < 0) return IPTTT_ERR_SEGMENTS;
    if (p->q_len[i] > p->q_rows || p->q_start[i] > p->q_rows - p->q_len[i]) return IPTTT_ERR_SEGMENTS;
    if (p->k_len[i] > p->k_rows || p->k_start[i] > p->k_rows - p->k_len[i]) return IPTTT_ERR_SEGMENTS;
    end = p->q_start[i] + p->q_len[i];
  }
  return IPTTT_OK;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Keys that some row of the tile [r0, r0 + n) of sequence i sees.
int64_t tile_keys(const ipttt_attn_problem* p, int64_t i, int64_t r0, int64_t n) {
  const int64_t G = p->heads / p->kv_heads, last = std::min(r0 + n, p->q_len[i] * G) - 1;
  return std::max<int64_t>(0, p->k_len[i] - p->q_len[i] + last / G + 1);
}

// The first flat row that sees key k0 of sequence i, and the steps from it on.
int64_t key_rows(const ipttt_attn_problem* p, int64_t i, int64_t k0) {
  const int64_t t = std::max<int64_t>(0, k0 - (p->k_len[i] - p->q_len[i]));
  return std::min(p->q_len[i], t) * (p->heads / p->kv_heads);
}
int64_t key_steps(const ipttt_attn_problem* p, int64_t i, int64_t k0) {
  return div_up(p->q_len[i] * (p->heads / p->kv_heads) - key_rows(p, i, k0), kBwdRows);
}

constexpr int64_t kCus = 256;
// Workgroups that run at once: two a CU (one, of fp32 tiles wider than 64).
constexpr int64_t kGroups = 2 * kCus;

// How far the tiles are cut into parts.
struct Cut {
  bool rows;      // whether there are tiles of many rows
  int64_t keys;   // most keys of a forward part
  int64_t few;    // most keys of a part of few rows
  int64_t dq;     // most keys of a dQ part
  int64_t steps;  // most steps of a dK, dV part
};

// A sequence of few rows: the kernel for them reads the keys with every wave.
// Over few keys it is worth no launch of its own beside the tiles of many rows.
// One without queries (a pool's idle slot) has no rows and no part in the forward.
bool fits_few(const ipttt_attn_problem* p, int64_t i) { return p->q_len[i] * (p->heads / p->kv_heads) <= kFewRows; }
bool few_rows(const ipttt_attn_problem* p, const Cut& cut, int64_t i) {
  return p->q_len[i] > 0 && fits_few(p, i) && !(cut.rows && p->k_len[i] <= 4 * kKeys);
}

// Whether the workgroups of a forward call are alone on their CUs.
bool alone(const ipttt_attn_problem* p) { return p->dtype == IPTTT_F32 && p->head_dim > 64; }
// Whether a call's workgroups all start at once, two on some CUs.  The second then
// comes to a CU in the order of the first, so the shortest should meet the longest.
bool folded(const ipttt_attn_problem* p, int64_t groups) { return !alone(p) && kCus < groups && groups <= kGroups; }

// The most steps (of kKeys keys) of a part of a forward tile of many rows; kMaxInt
// leaves every tile whole.  Two workgroups on a CU take about as long as one of both
// lengths, so a call takes as long as the CU with the most steps, the longest
// parts handed out first; a lone bf16 workgroup a tenth longer.  Of n-ths of the
// longest tile and even shares of all work, the part is the one for which that ends
// first, with some steps' time for each part's start and for a join, if any: 4 and
// 12, fp32 (whose steps take longer) 1/2 and 3/2.  Calls of two tiles a CU and more
// (fp32: four) stay whole.  Over 62 shapes of 32 to 900 tiles that is some 2 % above
// the best part of a sweep; cutting wherever a workgroup had less than an even share
// of 512: 10 % (bf16) and 6 % (fp32).  Heads 32 over 8 of width 128, 1000 tokens: whole
// 22 us, cut in shares 31; 100 tokens over 16000: whole 240, cut 46.
int64_t forward_part(const ipttt_attn_problem* p, const Cut& cut) {
  const bool f32 = p->dtype == IPTTT_F32;
  constexpr int64_t kMost = 4 * kCus;
  const int64_t G = p->heads / p->kv_heads, copies = p->kv_heads;
  const int64_t start = f32 ? 1 : 8, join = f32 ? 3 : 24, least = f32 ? 2 : 4;  // start and join in half steps
  const int64_t whole = f32 ? kMost : kGroups, limit = f32 ? kMost : 3 * kCus;
  const auto tiles = [&](auto&& f) {
    for (int64_t i = 0; i < p->n_seqs; ++i) {
      if (few_rows(p, cut, i)) continue;
      for (int64_t r0 = 0; r0 < p->q_len[i] * G; r0 += kRows)
        if (!f(div_up(tile_keys(p, i, r0, kRows), kKeys))) return;
    }
  };
  int64_t longest = 0, work = 0, n = 0;
  tiles([&](int64_t steps) {
    longest = std::max(longest, steps);
    work += steps * copies;
    return (n += copies) < whole;
  });
  if (n >= whole) return kMaxInt;
  int64_t best = INT64_MAX, part = kMaxInt;
  for (int64_t nth : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256, -1, -2}) {
    const int64_t most = nth > 0 ? std::max<int64_t>(1, div_up(longest, nth)) : div_up(work, -nth * kCus);
    if (nth != 1 && (most < least || most >= longest)) continue;
    int64_t size[kMost], load[kCus] = {}, sum = 0;
    bool fits = true;
    n = 0;  // parts of one key head
    tiles([&](int64_t steps) {
      for (; fits; steps -= most) {
        fits = (n + 1) * copies <= limit;
        if (fits) sum += size[n++] = start + 2 * std::min(steps, most);
        if (steps <= most) break;
      }
      return fits;
    });
    if (!fits) continue;
    std::sort(size, size + n, [](int64_t x, int64_t y) { return x > y; });
    const int64_t total = n * copies, more = nth == 1 ? 0 : join;
    if (n == 0 || std::max(sum * copies / kCus, size[0]) + more >= best) continue;  // it cannot be the one
    for (int64_t i = 0; i < total;) {
      std::sort(load, load + kCus);
      for (int64_t j = 0; j < kCus && i < total; ++j, ++i) load[j] += size[i / copies];
    }
    int64_t time = *std::max_element(load, load + kCus);
    // beyond two a CU the second comes to a CU in the order of the first
    if (!alone(p) && total > kGroups) time = std::max(time, size[0] + size[kCus / copies]);
    if (!f32 && total <= kCus) time += time / 10;
    if (time + more >= best) continue;
    best = time + more;
    part = nth == 1 ? kMaxInt : most;
  }
  return part;
}

// The most keys of a part of few rows: a multiple of 64, a block of 32 for each of a
// workgroup's two waves.  Only reading matters, and a second workgroup on a CU reads
// no sooner than the first: the shortest parts that are no more than the CUs (one
// token over 16000 keys, 8 key heads of width 128: 21.2 us in parts of 512, 32.8 of
// 128).  A long sequence's are at least 128, as a join is longer for each (4000 keys
// of one head: 10.8 us, 13.0 of 64).  Where that takes parts of more than 1024,
// shares of 2048 workgroups, whose ends even out, but at least 512 keys (16 tokens
// over 3000, 8 key heads of width 64: 26.3 us, 29.2 of 1024, 28.2 of 192).
int64_t few_part(const ipttt_attn_problem* p, const Cut& cut) {
  int64_t keys = 0, longest = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i) {
    if (!few_rows(p, cut, i)) continue;
    keys += p->k_len[i];
    longest = std::max(longest, p->k_len[i]);
  }
  int64_t most = longest > 2048 ? 128 : 64;
  const auto fits = [&] {
    int64_t n = 0;
    for (int64_t i = 0; i < p->n_seqs; ++i)
      if (few_rows(p, cut, i)) n += div_up(p->k_len[i], most);
    return n * p->kv_heads <= kCus;
  };
  while (most <= 1024 && !fits()) most += 64;
  if (most > 1024) most = std::max<int64_t>(512, div_up(div_up(keys * p->kv_heads, 4 * kGroups), 64) * 64);
  return most;
}

// Backward: the first keys of a causal sequence meet all its rows and the last
// almost none, and a call's last workgroup ends it, so no tile of keys is longer
// than what a workgroup gets on average (32 heads over 8 of width 128, forward and
// backward: 2500 tokens 415 us uncut, 268 cut and joined; 4000: 740 and 564; 8192 and
// more: equal); where workgroups would stay idle, tiles of rows are cut alike, and
// those of keys in parts of 1.5 shares, which leaves fewer (bf16, 1000 tokens: 88 us,
// 95 in even shares; 4000 tokens, whose tiles fill the CUs: 600 and 563; fp32: even
// shares everywhere).  A step of rows is 128 x 64 x 3 products, one of keys
// 32 x 128 x 4: three to two.
Cut cut_of(const ipttt_attn_problem* p) {
  const bool f32 = p->dtype == IPTTT_F32;
  const int64_t least = (f32 ? 2 : 4) * kKeys, least_steps = f32 ? 4 : 8;
  const int64_t G = p->heads / p->kv_heads;
  Cut c = {};
  for (int64_t i = 0; i < p->n_seqs; ++i) c.rows = c.rows || !fits_few(p, i);
  int64_t bwd_tiles = 0, work = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i) {
    if (p->q_len[i] == 0) continue;  // its keys' tiles only write zeros
    for (int64_t r0 = 0; r0 < p->q_len[i] * G; r0 += kRows) {
      const int64_t n = tile_keys(p, i, r0, kRows);
      ++bwd_tiles;
      work += 3 * div_up(n, kKeys);
    }
    for (int64_t k0 = 0; k0 < p->k_len[i]; k0 += kBwdKeys) {
      ++bwd_tiles;
      work += 2 * key_steps(p, i, k0);
    }
  }
  const int64_t part = forward_part(p, c);
  c.keys = part == kMaxInt ? kMaxInt : part * kKeys;
  c.few = few_part(p, c);
  const int64_t each = div_up(work * p->kv_heads, kGroups);
  const bool some = bwd_tiles * p->kv_heads < kGroups;
  c.steps = std::max(least_steps, div_up(some && !f32 ? 3 * each : 2 * each, 4));
  c.dq = !some ? kMaxInt : std::max(least, div_up(each, 3) * kKeys);
  return c;
}

// Walks every item of the plan in sequence order.
template <class Rows, class FewRows, class Join, class Tiles, class Dq, class DqJoin, class Key, class KJoin>
void walk(const ipttt_attn_problem* p, const Cut& cut, Rows&& rows, FewRows&& few, Join&& join, Tiles&& tiles, Dq&& dq,
          DqJoin&& dq_join, Key&& key, KJoin&& kjoin) {
  const int64_t G = p->heads / p->kv_heads;
  int64_t slots = 0, dq_slots = 0, key_slots = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i) {
    const int32_t off = (int32_t)(p->k_len[i] - p->q_len[i]);
    const int32_t qs = (int32_t)p->q_start[i], ql = (int32_t)p->q_len[i], ks = (int32_t)p->k_start[i];
    // one tile over its keys, in parts of `most` (the last may be shorter), each
    // of `step` slots
    const auto tile = [&](int64_t r0, int64_t n, int64_t most, int64_t step, int64_t& slot, auto& emit, auto& joined) {
      const int64_t parts = std::max<int64_t>(1, div_up(n, most));
      if (parts == 1) {
        emit(RowItem{qs, ql, (int32_t)r0, ks, off, 0, (int32_t)n, -1});
        return;
      }
      joined(JoinItem{qs, ql, (int32_t)r0, (int32_t)slot, (int32_t)parts, (int32_t)step});
      for (int64_t j = 0; j < parts; ++j, slot += step)
        emit(RowItem{qs, ql, (int32_t)r0, ks, off, (int32_t)(j * most), (int32_t)std::min(n, (j + 1) * most),
                     (int32_t)slot});
    };
    const bool is_few = few_rows(p, cut, i);
    if (is_few) tile(0, tile_keys(p, i, 0, kFewRows), cut.few, 1, slots, few, join);
    for (int64_t r0 = 0; r0 < p->q_len[i] * G; r0 += kRows) {
      const int64_t n = tile_keys(p, i, r0, kRows);
      tiles(RowItem{qs, ql, (int32_t)r0, ks, off, 0, (int32_t)n, -1});
      tile(r0, n, cut.dq, kRows / kPartRows, dq_slots, dq, dq_join);
      if (!is_few) tile(r0, n, cut.keys, kRows / kPartRows, slots, rows, join);
    }
    for (int64_t k0 = 0; k0 < p->k_len[i]; k0 += kBwdKeys) {
      const int64_t r0 = key_rows(p, i, k0), end = p->q_len[i] * G;
      const int64_t parts = std::max<int64_t>(1, div_up(key_steps(p, i, k0), cut.steps));
      if (parts == 1) {
        key(KeyItem{qs, ql, (int32_t)r0, (int32_t)end, ks, off, (int32_t)k0, -1});
        continue;
      }
      const int64_t rows_each = div_up(key_steps(p, i, k0), parts) * kBwdRows;
      int64_t n = 0;
      for (int64_t r = r0; r < end; r += rows_each, ++n)
        key(KeyItem{qs, ql, (int32_t)r, (int32_t)std::min(end, r + rows_each), ks, off, (int32_t)k0,
                    (int32_t)(key_slots + n)});
      kjoin(KeyJoin{(int32_t)(p->k_start[i] + k0), (int32_t)std::min<int64_t>(kBwdKeys, p->k_len[i] - k0),
                    (int32_t)key_slots, (int32_t)n});
      key_slots += n;
    }
  }
}

struct Range {
  int64_t start, len;
};

struct Sizes {
  int64_t rows = 0, few = 0, join = 0, tiles = 0, dq = 0, dq_join = 0, key = 0, kjoin = 0;
  int64_t parts = 0, dq_parts = 0, key_parts = 0, join_rows = 0;
  bool rows_cut = false;
  int64_t o_rows, o_few, o_join, o_tiles, o_dq_join, o_dq, o_key, o_kjoin, o_ranges, bytes;
};

// Counts and offsets; false if the plan would not fit its own 31-bit fields.
bool sizes_of(const ipttt_attn_problem* p, const Cut& cut, Sizes* s) {
  const int64_t G = p->heads / p->kv_heads;
  walk(
      p, cut,
      [&](const RowItem& x) {
        ++s->rows;
        s->rows_cut = s->rows_cut || x.part >= 0;
      },
      [&](const RowItem&) { ++s->few; },
      [&](const JoinItem& x) {
        ++s->join;
        s->parts += (int64_t)x.n * x.step;
        s->join_rows = std::max(s->join_rows, std::min<int64_t>(x.step * kPartRows, x.q_len * G - x.r0));
      },
      [&](const RowItem&) { ++s->tiles; }, [&](const RowItem&) { ++s->dq; },
      [&](const JoinItem& x) {
        ++s->dq_join;
        s->dq_parts += (int64_t)x.n * x.step;
      },
      [&](const KeyItem& x) {
        ++s->key;
        s->key_parts += x.part >= 0;
      },
      [&](const KeyJoin&) { ++s->kjoin; });
  s->o_rows = sizeof(PlanHeader);
  s->o_few = s->o_rows + s->rows * (int64_t)sizeof(RowItem);
  s->o_tiles = s->o_few + s->few * (int64_t)sizeof(RowItem);
  s->o_dq = s->o_tiles + s->tiles * (int64_t)sizeof(RowItem);
  s->o_key = s->o_dq + s->dq * (int64_t)sizeof(RowItem);
  s->o_join = s->o_key + s->key * (int64_t)sizeof(KeyItem);
  s->o_dq_join = s->o_join + s->join * (int64_t)sizeof(JoinItem);
  s->o_kjoin = (s->o_dq_join + s->dq_join * (int64_t)sizeof(JoinItem) + 15) / 16 * 16;
  s->o_ranges = s->o_kjoin + s->kjoin * (int64_t)sizeof(KeyJoin);
  s->bytes = s->o_ranges + p->n_seqs * (int64_t)sizeof(Range);
  const int64_t most = std::max(std::max(s->rows, s->few), std::max(s->tiles, s->dq + s->key));
  return s->bytes <= kMaxInt && most <= kMaxGroups / p->kv_heads;
}

const PlanHeader* header(const void* plan) {
  if (plan == nullptr || !aligned(plan, 8)) return nullptr;
  const PlanHeader* h = static_cast<const PlanHeader*>(plan);
  return h->magic == kMagic ? h : nullptr;
}

struct FwdLayout {
  size_t o, lse, total;
};
FwdLayout fwd_layout(const PlanHeader* h) {
  FwdLayout l;
  const size_t rows = (size_t)h->parts * h->kv_heads * kPartRows;
  l.o = 0;
  l.lse = align256(rows * h->head_dim * sizeof(float));
  l.total = l.lse + align256(rows * sizeof(float));
  return l;
}

// -lse / scale of every row | -delta of every row | partial dK, dV | partial dQ
struct BwdLayout {
  size_t nlse, ndelta, keys, dq, total;
};
BwdLayout bwd_layout(const PlanHeader* h) {
  BwdLayout l;
  const size_t stat = align256((size_t)h->q_rows * h->heads * sizeof(float));
  const size_t row = (size_t)h->kv_heads * h->head_dim * sizeof(float);
  l.nlse = 0;
  l.ndelta = stat;
  l.keys = 2 * stat;
  l.dq = l.keys + align256((size_t)h->key_parts * 2 * kBwdKeys * row);
  l.total = l.dq + align256((size_t)h->dq_parts * kPartRows * row);
  return l;
}

ipttt_status check_call(const void* plan, const void* plan_dev, float scale, void* ws, size_t ws_bytes, size_t need) {
  if (plan == nullptr || plan_dev == nullptr) return IPTTT_ERR_NULL;
  if (!aligned(plan, 8) || !aligned(plan_dev, 16)) return IPTTT_ERR_ALIGN;
  if (header(plan) == nullptr || !std::isfinite(scale) || scale <= 0.0f) return IPTTT_ERR_ARG;
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return IPTTT_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 256)) return IPTTT_ERR_ALIGN;
  return IPTTT_OK;
}

// q and o by tiles of rows (of every head of a group), k and v by tiles of keys.
// A tensor of no rows may be NULL: no tile reads or writes it.
ipttt_status q_view(const PlanHeader* h, const ipttt_heads* t, View* v) {
  if (h->q_rows == 0) return IPTTT_OK;
  return check_heads(t, h->q_rows, h->heads, h->head_dim, h->dtype, kRows + 1, h->heads / h->kv_heads, v);
}
ipttt_status k_view(const PlanHeader* h, const ipttt_heads* t, View* v) {
  if (h->k_rows == 0) return IPTTT_OK;
  return check_heads(t, h->k_rows, h->kv_heads, h->head_dim, h->dtype, kBwdKeys, 1, v);
}

ipttt::attn::Args base_args(const PlanHeader* h, float scale) {
  ipttt::attn::Args a = {};
  a.dtype = h->dtype;
  a.heads = h->heads;
  a.kv_heads = h->kv_heads;
  a.G = h->heads / h->kv_heads;
  a.D = h->head_dim;
  a.scale = scale;
  return a;
}

// ------------------------------------------------------- norm and rotation

ipttt_status check_qk(const ipttt_qk_problem* p) {
  if (p == nullptr) return IPTTT_ERR_NULL;
  const ipttt_status s = check_dims(p->heads, p->kv_heads, p->head_dim, p->dtype);
  if (s != IPTTT_OK) return s;
  if (p->tokens < 1 || p->tokens > 4 * kMaxGroups || p->table_rows < 1 || p->table_rows > kMaxInt) return IPTTT_ERR_SHAPE;
  if (p->out_rows < 0 || p->out_rows > kMaxInt) return IPTTT_ERR_SHAPE;
  if (!std::isfinite(p->eps) || p->eps < 0.0f) return IPTTT_ERR_ARG;
  return IPTTT_OK;
}

// Every address is 64-bit here: only the strides' own rules apply.  A tensor of no
// rows may be NULL.
ipttt_status qk_view(const ipttt_qk_problem* p, const ipttt_heads* t, int64_t rows, int64_t heads, View* v) {
  if (rows == 0) return IPTTT_OK;
  return check_heads(t, rows, heads, p->head_dim, p->dtype, 1, 1, v);
}

bool same(const View& a, const View& b) { return a.p == b.p && a.row == b.row && a.head == b.head; }

size_t qk_part_bytes(const ipttt_qk_problem* p) {
  return align256((size_t)ipttt::kQkParts * 2 * (size_t)p->head_dim * sizeof(float));
}

ipttt::QkArgs qk_args(const ipttt_qk_problem* p, const void* w_q, const void* w_k, const int32_t* positions,
                      const float* table) {
  ipttt::QkArgs a = {};
  a.dtype = p->dtype;
  a.heads = (int)p->heads;
  a.kv_heads = (int)p->kv_heads;
  a.D = (int)p->head_dim;
  a.tokens = p->tokens;
  a.table_rows = p->table_rows;
  a.out_rows = p->out_rows;
  a.eps = p->eps;
  a.w_q = w_q;
  a.w_k = w_k;
  a.pos = positions;
  a.table = table;
  return a;
}

ipttt_status check_qk_inputs(const void* w_q, const void* w_k, const int32_t* positions, const float* table) {
  if (w_q == nullptr || w_k == nullptr || positions == nullptr || table == nullptr) return IPTTT_ERR_NULL;
  if (!aligned(w_q, 16) || !aligned(w_k, 16) || !aligned(table, 16) || !aligned(positions, 4)) return IPTTT_ERR_ALIGN;
  return IPTTT_OK;
}

}  // namespace

#define IPTTT_TRY(expr)                       \
  do {                                        \
    const ipttt_status status_ = (expr);      \
    if (status_ != IPTTT_OK) return status_;  \
  } while (0)

extern "C" {

ipttt_status ipttt_qk_norm_rope(const ipttt_qk_problem* p, const ipttt_heads* q, const ipttt_heads* k, const void* w_q,
                                const void* w_k, const int32_t* positions, const float* table,
                                const ipttt_heads* q_out, const ipttt_heads* k_out, const ipttt_heads* v,
                                const ipttt_heads* v_out, const int32_t* rows, void* stream) {
  IPTTT_TRY(check_qk(p));
  IPTTT_TRY(check_qk_inputs(w_q, w_k, positions, table));
  ipttt::QkArgs a = qk_args(p, w_q, w_k, positions, table);
  IPTTT_TRY(qk_view(p, q, p->tokens, p->heads, &a.q));
  IPTTT_TRY(qk_view(p, k, p->tokens, p->kv_heads, &a.k));
  IPTTT_TRY(qk_view(p, q_out, p->tokens, p->heads, &a.q_out));
  IPTTT_TRY(qk_view(p, k_out, p->out_rows, p->kv_heads, &a.k_out));
  if ((v == nullptr) != (v_out == nullptr)) return IPTTT_ERR_NULL;
  if (v != nullptr) {
    IPTTT_TRY(qk_view(p, v, p->tokens, p->kv_heads, &a.v));
    IPTTT_TRY(qk_view(p, v_out, p->out_rows, p->kv_heads, &a.v_out));
  }
  if (!aligned(rows, 4)) return IPTTT_ERR_ALIGN;
  if (rows == nullptr && p->out_rows < p->tokens) return IPTTT_ERR_SHAPE;
  // an output over its input has to be that input, row for row
  if (a.q_out.p == a.q.p && !same(a.q_out, a.q)) return IPTTT_ERR_ARG;
  if (a.k_out.p == a.k.p && (rows != nullptr || !same(a.k_out, a.k))) return IPTTT_ERR_ARG;
  if (v != nullptr && a.v_out.p == a.v.p && (rows != nullptr || !same(a.v_out, a.v))) return IPTTT_ERR_ARG;
  a.rows = rows;
  return hip_status(ipttt::launch_qk(a, static_cast<hipStream_t>(stream)));
}

size_t ipttt_qk_backward_workspace_bytes(const ipttt_qk_problem* p) {
  return check_qk(p) == IPTTT_OK ? qk_part_bytes(p) : 0;
}

ipttt_status ipttt_qk_norm_rope_backward(const ipttt_qk_problem* p, const ipttt_heads* q, const ipttt_heads* k,
                                         const void* w_q, const void* w_k, const int32_t* positions,
                                         const float* table, const ipttt_heads* dq_out, const ipttt_heads* dk_out,
                                         const ipttt_heads* dq, const ipttt_heads* dk, float* dw_q, float* dw_k,
                                         void* ws, size_t ws_bytes, void* stream) {
  IPTTT_TRY(check_qk(p));
  IPTTT_TRY(check_qk_inputs(w_q, w_k, positions, table));
  ipttt::QkArgs a = qk_args(p, w_q, w_k, positions, table);
  IPTTT_TRY(qk_view(p, q, p->tokens, p->heads, &a.q));
  IPTTT_TRY(qk_view(p, k, p->tokens, p->kv_heads, &a.k));
  IPTTT_TRY(qk_view(p, dq_out, p->tokens, p->heads, &a.q_out));
  IPTTT_TRY(qk_view(p, dk_out, p->tokens, p->kv_heads, &a.k_out));
  IPTTT_TRY(qk_view(p, dq, p->tokens, p->heads, &a.dq));
  IPTTT_TRY(qk_view(p, dk, p->tokens, p->kv_heads, &a.dk));
  if (dw_q == nullptr || dw_k == nullptr) return IPTTT_ERR_NULL;
  if (!aligned(dw_q, 16) || !aligned(dw_k, 16)) return IPTTT_ERR_ALIGN;
  if (a.dq.p == a.q_out.p && !same(a.dq, a.q_out)) return IPTTT_ERR_ARG;
  if (a.dk.p == a.k_out.p && !same(a.dk, a.k_out)) return IPTTT_ERR_ARG;
  if (ws == nullptr || ws_bytes < qk_part_bytes(p)) return IPTTT_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return IPTTT_ERR_ALIGN;
  a.dw_q = dw_q;
  a.dw_k = dw_k;
  a.part = static_cast<float*>(ws);
  return hip_status(ipttt::launch_qk_backward(a, static_cast<hipStream_t>(stream)));
}

ipttt_status ipttt_attn_validate(const ipttt_attn_problem* p) {
  IPTTT_TRY(check_attn(p));
  Sizes s;
  return sizes_of(p, cut_of(p), &s) ? IPTTT_OK : IPTTT_ERR_SHAPE;
}

size_t ipttt_attn_plan_bytes(const ipttt_attn_problem* p) {
  Sizes s;
  return check_attn(p) == IPTTT_OK && sizes_of(p, cut_of(p), &s) ? (size_t)s.bytes : 0;
}

ipttt_status ipttt_attn_plan(const ipttt_attn_problem* p, void* plan, size_t plan_bytes) {
  IPTTT_TRY(check_attn(p));
  const Cut cut = cut_of(p);
  Sizes s;
  if (!sizes_of(p, cut, &s)) return IPTTT_ERR_SHAPE;
  if (plan == nullptr || plan_bytes < (size_t)s.bytes) return IPTTT_ERR_WORKSPACE;
  if (!aligned(plan, 8)) return IPTTT_ERR_ALIGN;
  std::memset(plan, 0, (size_t)s.bytes);
  char* base = static_cast<char*>(plan);
  RowItem* rows = reinterpret_cast<RowItem*>(base + s.o_rows);
  RowItem* dq = reinterpret_cast<RowItem*>(base + s.o_dq);
  KeyItem* key = reinterpret_cast<KeyItem*>(base + s.o_key);
  JoinItem* join = reinterpret_cast<JoinItem*>(base + s.o_join);
  RowItem* tiles = reinterpret_cast<RowItem*>(base + s.o_tiles);
  JoinItem* dq_join = reinterpret_cast<JoinItem*>(base + s.o_dq_join);
  KeyJoin* kjoin = reinterpret_cast<KeyJoin*>(base + s.o_kjoin);
  RowItem* few = reinterpret_cast<RowItem*>(base + s.o_few);
  walk(p, cut, [&](const RowItem& x) { *rows++ = x; }, [&](const RowItem& x) { *few++ = x; },
       [&](const JoinItem& x) { *join++ = x; }, [&](const RowItem& x) { *tiles++ = x; },
       [&](const RowItem& x) { *dq++ = x; }, [&](const JoinItem& x) { *dq_join++ = x; },
       [&](const KeyItem& x) { *key++ = x; },
       [&](const KeyJoin& x) { *kjoin++ = x; });
  // the longest first, so that the last workgroups to start are short ones
  const auto longer = [](const RowItem& x, const RowItem& y) {
    const int32_t a = x.k_end - x.k_begin, b = y.k_end - y.k_begin;
    if (a != b) return a > b;
    return x.q_start != y.q_start ? x.q_start < y.q_start : x.r0 != y.r0 ? x.r0 < y.r0 : x.k_begin < y.k_begin;
  };
  std::sort(rows - s.rows, rows, longer);
  // (3900 tokens, 16 heads over 8 of width 64: 49.4 us without, 47.4; fp32 351 and 258)
  if (folded(p, s.rows * p->kv_heads)) std::reverse(rows - s.rows + kCus / p->kv_heads, rows);
  std::sort(few - s.few, few, longer);
  std::sort(dq - s.dq, dq, longer);
  std::sort(key - s.key, key, [](const KeyItem& x, const KeyItem& y) {
    const int32_t a = x.r_end - x.r_begin, b = y.r_end - y.r_begin;
    if (a != b) return a > b;
    return x.k_start != y.k_start ? x.k_start < y.k_start : x.key0 != y.key0 ? x.key0 < y.key0 : x.r_begin < y.r_begin;
  });
  // whether two sequences share keys
  Range* r = reinterpret_cast<Range*>(base + s.o_ranges);
  int64_t n = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i)
    if (p->k_len[i] > 0) r[n++] = Range{p->k_start[i], p->k_len[i]};
  std::sort(r, r + n, [](const Range& x, const Range& y) { return x.start < y.start; });
  bool overlap = false;
  for (int64_t i = 1; i < n; ++i) overlap = overlap || r[i].start < r[i - 1].start + r[i - 1].len;

  PlanHeader* h = static_cast<PlanHeader*>(plan);
  h->magic = kMagic;
  h->dtype = p->dtype;
  h->heads = (int32_t)p->heads;
  h->kv_heads = (int32_t)p->kv_heads;
  h->head_dim = (int32_t)p->head_dim;
  h->n_seqs = (int32_t)p->n_seqs;
  h->q_rows = (int32_t)p->q_rows;
  h->k_rows = (int32_t)p->k_rows;
  h->n_rows = (int32_t)s.rows;
  h->n_tiles = (int32_t)s.tiles;
  h->o_tiles = (int32_t)s.o_tiles;
  h->n_dq_join = (int32_t)s.dq_join;
  h->o_dq_join = (int32_t)s.o_dq_join;
  h->dq_parts = (int32_t)s.dq_parts;
  h->n_few = (int32_t)s.few;
  h->o_few = (int32_t)s.o_few;
  h->join_rows = (int32_t)s.join_rows;
  h->rows_cut = s.rows_cut;
  h->shorts = 0;
  for (int64_t i = 0; i < p->n_seqs; ++i) h->shorts |= p->q_len[i] > 0 && p->k_len[i] <= kShortKeys;
  h->n_join = (int32_t)s.join;
  h->n_dq = (int32_t)s.dq;
  h->n_key = (int32_t)s.key;
  h->o_rows = (int32_t)s.o_rows;
  h->o_join = (int32_t)s.o_join;
  h->o_dq = (int32_t)s.o_dq;
  h->o_key = (int32_t)s.o_key;
  h->n_key_join = (int32_t)s.kjoin;
  h->o_key_join = (int32_t)s.o_kjoin;
  h->key_parts = (int32_t)s.key_parts;
  h->parts = (int32_t)s.parts;
  h->overlap = overlap;
  h->bytes = (int32_t)s.bytes;
  return IPTTT_OK;
}

size_t ipttt_attn_workspace_bytes(const void* plan) {
  const PlanHeader* h = header(plan);
  return h == nullptr ? 0 : fwd_layout(h).total;
}

size_t ipttt_attn_backward_workspace_bytes(const void* plan) {
  const PlanHeader* h = header(plan);
  return h == nullptr ? 0 : bwd_layout(h).total;
}

ipttt_status ipttt_attention(const void* plan, const void* plan_dev, float scale, const ipttt_heads* q,
                             const ipttt_heads* k, const ipttt_heads* v, const ipttt_heads* o, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  IPTTT_TRY(check_call(plan, plan_dev, scale, ws, ws_bytes, ipttt_attn_workspace_bytes(plan)));
  const PlanHeader* h = header(plan);
  ipttt::attn::Args a = base_args(h, scale);
  IPTTT_TRY(q_view(h, q, &a.q));
  IPTTT_TRY(k_view(h, k, &a.k));
  IPTTT_TRY(k_view(h, v, &a.v));
  IPTTT_TRY(q_view(h, o, &a.o));
  if (lse == nullptr && h->q_rows > 0) return IPTTT_ERR_NULL;
  if (!aligned(lse, 16)) return IPTTT_ERR_ALIGN;
  const FwdLayout l = fwd_layout(h);
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + l.o);
  a.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + l.lse);
  const char* dev = static_cast<const char*>(plan_dev);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (h->n_rows > 0) {
    a.items = dev + h->o_rows;
    a.n_items = h->n_rows;
    a.cut = h->rows_cut != 0;
    IPTTT_TRY(hip_status(ipttt::attn::launch_forward(a, st)));
  }
  if (h->n_few > 0) {
    a.items = dev + h->o_few;
    a.n_items = h->n_few;
    IPTTT_TRY(hip_status(ipttt::attn::launch_few(a, st)));
  }
  if (h->n_join == 0) return IPTTT_OK;
  return hip_status(ipttt::attn::launch_join(a, dev + h->o_join, h->n_join, h->join_rows, st));
}

ipttt_status ipttt_attention_backward(const void* plan, const void* plan_dev, float scale, const ipttt_heads* q,
                                      const ipttt_heads* k, const ipttt_heads* v, const ipttt_heads* o,
                                      const float* lse, const ipttt_heads* dO, const ipttt_heads* dq,
                                      const ipttt_heads* dk, const ipttt_heads* dv, void* ws, size_t ws_bytes,
                                      void* stream) {
  IPTTT_TRY(check_call(plan, plan_dev, scale, ws, ws_bytes, ipttt_attn_backward_workspace_bytes(plan)));
  const PlanHeader* h = header(plan);
  if (h->overlap) return IPTTT_ERR_SEGMENTS;
  ipttt::attn::Args a = base_args(h, scale);
  IPTTT_TRY(q_view(h, q, &a.q));
  IPTTT_TRY(k_view(h, k, &a.k));
  IPTTT_TRY(k_view(h, v, &a.v));
  IPTTT_TRY(q_view(h, o, &a.o));
  IPTTT_TRY(q_view(h, dO, &a.dO));
  IPTTT_TRY(q_view(h, dq, &a.dq));
  IPTTT_TRY(k_view(h, dk, &a.dk));
  IPTTT_TRY(k_view(h, dv, &a.dv));
  if (lse == nullptr && h->q_rows > 0) return IPTTT_ERR_NULL;
  if (!aligned(lse, 16)) return IPTTT_ERR_ALIGN;
  a.lse = const_cast<float*>(lse);
  const BwdLayout l = bwd_layout(h);
  const auto region = [ws](size_t at) { return reinterpret_cast<float*>(static_cast<char*>(ws) + at); };
  a.nlse = region(l.nlse);
  a.ndelta = region(l.ndelta);
  a.part_o = region(l.keys);
  a.part_dq = region(l.dq);
  const char* dev = static_cast<const char*>(plan_dev);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (h->n_tiles > 0) {
    a.items = dev + h->o_tiles;
    a.n_items = h->n_tiles;
    IPTTT_TRY(hip_status(ipttt::attn::launch_delta(a, st)));
  }
  if (h->n_key + h->n_dq > 0) {
    a.items = dev + h->o_key;
    a.n_items = h->n_key;
    a.dq_items = dev + h->o_dq;
    a.n_dq = h->n_dq;
    a.shorts = h->shorts != 0;
    IPTTT_TRY(hip_status(ipttt::attn::launch_backward(a, st)));
  }
  if (h->n_dq_join + h->n_key_join == 0) return IPTTT_OK;
  return hip_status(ipttt::attn::launch_join_backward(a, dev + h->o_dq_join, h->n_dq_join, dev + h->o_key_join,
                                                      h->n_key_join, st));
}

}  // extern "C"
