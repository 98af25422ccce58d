// Host side of the attention: the plan (documents cut into work for the kernels), buffer sizes and the checks of
// arguments that both directions share.
#include <math.h>

#include <algorithm>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "attention.cuh"

namespace dit6 {
namespace attn {

constexpr int SMS = 152;  // a plan is made on the host, for this chip

struct Costed {
  Item item;
  double cost;
};

// The end of the last of `pieces` on `places` processors that take them in order.
static double makespan(std::vector<double> pieces, int heads, int places) {
  std::sort(pieces.begin(), pieces.end(), std::greater<double>());
  std::priority_queue<double, std::vector<double>, std::greater<double>> ends;
  double last = 0.0;
  for (double c : pieces)
    for (int h = 0; h < heads; ++h) {
      double begin = 0.0;
      if ((int)ends.size() == places) {
        begin = ends.top();
        ends.pop();
      }
      ends.push(begin + c);
      last = std::max(last, begin + c);
    }
  return last;
}

// Forward times in tiles of two blocks of rows (0.8 us with up to 64 dimensions, 1.8 with up to 128): a CTA's start and end; what a piece of
// a split item adds, which writes a partial result; the joining kernel whatever it joins; and for each partial row of it.
// A tile of one block of rows takes as long as one of two, a chain of waits (LONE); where it is cut into pieces anyway, the
// CTA's halves take its tiles in turn (TURNS).
struct Times {
  double start, split_end, join, join_row;
};
constexpr Times TIMES[2] = {{5.0, 2.0, 5.0, 1.5e-4}, {3.0, 1.2, 3.0, 0.7e-4}};
constexpr double LONE = 0.95, TURNS = 0.5;
// Short items: with one block of rows to a CTA and two CTAs to an SM the start and end of one hide behind the other's tiles, but each block
// streams its own keys, and the ring holds two tiles instead of six.  With 64 dimensions (heads in brackets), two blocks and
// one: 32 documents of 77 tokens (30) 30.9 and 18.1 us, 32 of 156 42.6 and 38.4, 16 of 300 45.5 and 33.8, 9 of 1000 92.5 and
// 86.9, 5 of 2000, 16 tiles, 153.9 and 153.1; one of 4096 (9) 33.0 and 36.1, of 17,776 (30) 1788 and 1850.
constexpr int64_t SHORT_TILES = 16;
constexpr double BACK_START = 5.0;  // of a backward CTA, in tiles

static dit_status make_plan(const int64_t* queries, const int64_t* keys, const int64_t* begins, const int64_t* prefix,
                            int64_t documents, int64_t frame, int heads, int kv_heads, int dim, int training,
                            dit_attention_plan_t* plan, int32_t* table, int64_t table_ints) {
  if (!plan || documents < 0 || (documents > 0 && (!queries || !keys)) || frame < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads || dim < 1)
    return DIT_ERR_INVALID_ARG;
  const int group = heads / kv_heads;
  if (documents > MAX_DOCUMENTS || heads > MAX_HEADS || group > MAX_GROUP || dim % 8 || dim > MAX_DIM || frame > MAX_ROWS) return DIT_ERR_UNSUPPORTED;
  *plan = dit_attention_plan_t{};
  plan->documents = (int32_t)documents;
  plan->heads = heads;
  plan->kv_heads = kv_heads;
  plan->dim = dim;
  plan->frame = (int32_t)frame;
  plan->training = training ? 1 : 0;
  std::vector<Doc> docs((size_t)documents);
  int64_t q_rows = 0, k_next = 0, tiles = 0;
  for (int64_t i = 0; i < documents; ++i) {
    const int64_t begin = begins ? begins[i] : k_next, pre = prefix ? prefix[i] : 0;
    if (queries[i] < 0 || keys[i] < 0 || begin < 0 || pre < 0 || queries[i] > MAX_ROWS || keys[i] > MAX_ROWS || begin > MAX_ROWS ||
        pre > MAX_ROWS || q_rows + queries[i] > MAX_ROWS || begin + keys[i] > MAX_ROWS)
      return DIT_ERR_INVALID_ARG;
    if (frame == 0 && pre > 0) return DIT_ERR_INVALID_ARG;
    docs[(size_t)i] = Doc{(int32_t)q_rows, (int32_t)queries[i], keys[i] ? (int32_t)begin : 0, (int32_t)keys[i], (int32_t)pre, (int32_t)tiles};
    q_rows += queries[i];
    k_next = begin + keys[i];
    if (keys[i] && k_next > plan->k_rows) plan->k_rows = k_next;
    tiles += (queries[i] + TILE - 1) / TILE;
  }
  if (tiles > MAX_ROWS) return DIT_ERR_UNSUPPORTED;
  plan->q_rows = q_rows;
  plan->padded_rows = tiles * TILE;
  if (training) {
    std::vector<std::pair<int64_t, int64_t>> spans;
    for (const Doc& d : docs)
      if (d.keys) spans.push_back({d.k0, (int64_t)d.k0 + d.keys});
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
      if (spans[i].first < spans[i - 1].second) return DIT_ERR_INVALID_ARG;
  }

  const int cols = BACK_COLS, rt = rows_per_tile(group), pd = padded_dim(dim);
  const Times& time = TIMES[pd > 64];
  std::vector<Costed> lists[DIT_ATTENTION_LISTS];
  // forward: `blocks` row blocks to an item, an item to a head of keys
  std::vector<Costed>& items = lists[FORWARD];
  auto list_items = [&](int blocks) {
    items.clear();
    for (const Doc& d : docs)
      for (int64_t r = 0; r < d.queries; r += blocks * rt) {
        const int64_t last = std::min<int64_t>(d.queries, r + blocks * rt) - 1;
        const int64_t n = (seen_end(d, frame, last) + FORWARD_COLS - 1) / FORWARD_COLS;
        const double each = blocks == 1 || last - r >= rt ? 1.0 : LONE;
        items.push_back({Item{d, (int32_t)r, 0, (int32_t)n, -1, 0, {}}, time.start + each * (double)n});
      }
  };
  auto ends = [&](int places) {
    std::vector<double> all;
    for (const Costed& c : items) all.push_back(c.cost);
    return makespan(all, kv_heads, places);
  };
  bool brief = pd == 64;
  for (const Doc& d : docs) brief = brief && (d.queries == 0 || seen_end(d, frame, d.queries - 1) <= SHORT_TILES * FORWARD_COLS);
  double apart = HUGE_VAL;  // the end with one block to an item, where there may be either
  if (brief) {
    list_items(1);
    if ((int64_t)items.size() * kv_heads < 8 * SMS) apart = ends(2 * SMS);
  }
  plan->row_blocks = pd == 64 ? 2 : 1;
  list_items(plan->row_blocks);
  const int wide = plan->row_blocks * rt, places = plan->row_blocks == 2 ? SMS : 2 * SMS;  // queries of an item, CTAs at a time
  // Few items: the keys of some are cut into pieces of up to `len` tiles, of one size (even) or all but the last of `len`, whichever
  // brings the end of the last CTA forward most.  Which items: those that are left when zero to three rounds of the SMs have whole ones,
  // since what is cut has to be joined.  Lone blocks of rows first, whose halves work at a piece together, then the longest.  With
  // all items cut alike 1350 queries over 8326 keys took 105 us (30 heads of 64), with five of six whole 86.
  auto cut = [](int64_t n, int64_t len, bool even, int64_t k) {  // where piece k begins
    const int64_t pieces = (n + len - 1) / len;
    return even ? n * k / pieces : std::min(n, k * len);
  };
  auto lone = [&](const Item& it) { return wide > rt && it.row0 + rt >= it.doc.queries; };
  const int64_t ctas = (int64_t)items.size() * kv_heads;
  if (ctas && ctas < 4 * places) {
    std::stable_sort(items.begin(), items.end(), [&](const Costed& a, const Costed& b) {
      return lone(a.item) != lone(b.item) ? lone(a.item) : a.item.end > b.item.end;
    });
    std::vector<double> now;
    int64_t most = 0;
    for (const Costed& c : items) most = std::max<int64_t>(most, c.item.end);
    double best = std::min(apart, ends(places));
    int64_t longest = 0, cuts = 0;  // tiles of a piece, 0: items stay whole; the items that may be cut
    bool evenly = true;
    for (int rounds = 0; rounds < 4; ++rounds) {
      const int64_t may = (int64_t)items.size() - rounds * places / kv_heads;
      if (may <= 0) break;
      for (int64_t len = most; len >= 2; len = len > 24 ? len * 15 / 16 : len - 1) {
        int64_t total = 0;
        for (int64_t i = 0; i < may; ++i) total += std::max<int64_t>((items[(size_t)i].item.end + len - 1) / len, 1);
        if (total * kv_heads > 6 * places) break;
        for (int even = 0; even < 2; ++even) {
          now.clear();
          int64_t joined = 0;
          for (int64_t i = 0; i < (int64_t)items.size(); ++i) {
            const Costed& c = items[(size_t)i];
            const int64_t n = c.item.end, pieces = i < may ? (n + len - 1) / len : 1;
            const double each = lone(c.item) ? TURNS : 1.0;
            if (pieces <= 1) {
              now.push_back(c.cost);
              continue;
            }
            joined += std::min<int64_t>(wide, c.item.doc.queries - c.item.row0) * pieces * (lone(c.item) ? 2 : 1);
            for (int64_t k = 0; k < pieces; ++k) now.push_back(time.start + time.split_end + each * (double)(cut(n, len, even, k + 1) - cut(n, len, even, k)));
          }
          const double join = time.join + time.join_row * (double)joined * heads;
          // no order ends before the work shared evenly, nor before the longest piece
          double sum = 0.0, top = 0.0;
          for (double c : now) sum += c, top = std::max(top, c);
          if (std::max(sum * kv_heads / places, top) + join >= best) continue;
          const double t = makespan(now, kv_heads, places) + join;
          if (t < best) {
            best = t;
            longest = len;
            cuts = may;
            evenly = even;
          }
        }
      }
    }
    if (longest) {
      std::vector<Costed> whole;
      whole.swap(items);
      for (int64_t i = 0; i < (int64_t)whole.size(); ++i) {
        const Costed& c = whole[(size_t)i];
        const int64_t n = c.item.end, pieces = i < cuts ? (n + longest - 1) / longest : 1;
        if (pieces <= 1) {
          items.push_back(c);
          continue;
        }
        const Doc& d = c.item.doc;
        const int32_t rows = (int32_t)std::min<int64_t>(wide, d.queries - c.item.row0);
        const bool turns = lone(c.item);
        const double each = turns ? TURNS : 1.0;
        lists[JOIN].push_back({Item{d, c.item.row0, plan->slots, (int32_t)(turns ? 2 * pieces : pieces), rows, 0, {}}, 1.0});
        for (int64_t k = 0; k < pieces; ++k) {
          Item it = c.item;
          it.begin = (int32_t)cut(n, longest, evenly, k);
          it.end = (int32_t)cut(n, longest, evenly, k + 1);
          it.slot = plan->slots;
          it.turns = turns;
          plan->slots += turns ? 2 * rows : rows;
          items.push_back({it, time.start + time.split_end + each * (double)(it.end - it.begin)});
        }
      }
    }
  }
  if (brief && lists[JOIN].empty()) {
    plan->row_blocks = 1;
    list_items(1);
  }
  if (training)
    for (size_t i = 0; i < docs.size(); ++i) {
      const Doc& d = docs[i];
      for (int64_t r = 0; r < d.queries; r += TILE) {
        const int64_t n = (seen_end(d, frame, std::min<int64_t>(d.queries, r + TILE) - 1) + cols - 1) / cols;
        lists[GRAD_Q].push_back({Item{d, (int32_t)r, 0, (int32_t)n, -1, 0, {}}, BACK_START + (double)n});
      }
      const int64_t end = ((int64_t)d.queries + cols - 1) / cols;
      for (int64_t k = 0; k < d.keys; k += TILE) {
        const int64_t begin = std::min(end, seen_from(d, frame, k) / cols);
        lists[GRAD_KV].push_back({Item{d, (int32_t)k, (int32_t)begin, (int32_t)end, -1, 0, {}}, BACK_START + (double)(end - begin)});
      }
    }
  std::vector<std::pair<int32_t, int32_t>> buckets[DIT_ATTENTION_LISTS];
  for (int l = 0; l < DIT_ATTENTION_LISTS; ++l) {
    auto& list = lists[l];
    if ((int64_t)list.size() * heads > MAX_ROWS) return DIT_ERR_UNSUPPORTED;
    std::stable_sort(list.begin(), list.end(), [](const Costed& a, const Costed& b) { return a.cost > b.cost; });
    double top = 0.0;
    for (size_t i = 0; i < list.size(); ++i) {
      if (i == 0 || (list[i].cost < 0.7 * top && buckets[l].size() < DIT_ATTENTION_BUCKETS)) {
        buckets[l].push_back({(int32_t)i, 0});
        top = list[i].cost;
      }
      ++buckets[l].back().second;
    }
    plan->items[l] = (int32_t)list.size();
    plan->buckets[l] = (int32_t)buckets[l].size();
    for (size_t b = 0; b < buckets[l].size(); ++b) {
      plan->bucket[l][2 * b] = buckets[l][b].first;
      plan->bucket[l][2 * b + 1] = buckets[l][b].second;
    }
  }
  plan->table_ints = first_item(*plan, DIT_ATTENTION_LISTS);
  plan->saved_bytes = training ? (int64_t)heads * plan->padded_rows * 4 : 0;
  const int64_t joins = (int64_t)heads * plan->slots * partial_floats(pd) * 4, deltas = plan->saved_bytes;
  plan->scratch_bytes = std::max(joins, deltas);
  if (!table) return DIT_OK;
  if (table_ints < plan->table_ints) return DIT_ERR_INVALID_ARG;
  std::fill(table, table + plan->table_ints, 0);
  for (int l = 0; l < DIT_ATTENTION_LISTS; ++l) {
    int32_t* o = table + first_item(*plan, l);
    for (const Costed& c : lists[l]) {
      std::copy_n(reinterpret_cast<const int32_t*>(&c.item), ITEM_INTS, o);
      o += ITEM_INTS;
    }
  }
  return DIT_OK;
}

bool plan_ok(const dit_attention_plan_t* p) {
  if (!p || p->documents < 0 || p->heads < 1 || p->heads > MAX_HEADS || p->kv_heads < 1 || p->heads % p->kv_heads || p->heads / p->kv_heads > MAX_GROUP ||
      p->dim < 8 || p->dim > MAX_DIM || p->dim % 8 || p->frame < 0 || p->q_rows < 0 || p->q_rows > MAX_ROWS || p->k_rows < 0 || p->k_rows > MAX_ROWS ||
      p->padded_rows < p->q_rows || p->padded_rows % TILE || p->slots < 0 ||
      (p->dim > 64 ? p->row_blocks != 1 : p->row_blocks != 2 && (p->row_blocks != 1 || p->items[JOIN])))
    return false;
  for (int l = 0; l < DIT_ATTENTION_LISTS; ++l)
    if (p->items[l] < 0 || (int64_t)p->items[l] * p->heads > MAX_ROWS || p->buckets[l] < 0 || p->buckets[l] > DIT_ATTENTION_BUCKETS || (p->items[l] && !p->buckets[l])) return false;
  const int64_t saved = p->training ? (int64_t)p->heads * p->padded_rows * 4 : 0;
  return p->table_ints == first_item(*p, DIT_ATTENTION_LISTS) && p->saved_bytes == saved &&
         p->scratch_bytes == std::max(saved, (int64_t)p->heads * p->slots * partial_floats(padded_dim(p->dim)) * 4);
}

// A view's checks; strides that no access uses are replaced by ones that a tensor map takes.
dit_status check_view(const dit_heads_t* v, int heads, int64_t rows, int dim, Heads* o) {
  if (!v || v->heads != heads || (!v->ptr && rows > 0)) return DIT_ERR_INVALID_ARG;
  *o = Heads{reinterpret_cast<__nv_bfloat16*>(const_cast<void*>(v->ptr)), rows > 1 ? v->token_stride : dim, heads > 1 ? v->head_stride : dim};
  if (o->row <= 0 || o->head <= 0) return DIT_ERR_INVALID_ARG;
  if (o->row > 0x7fffffff || o->head > 0x7fffffff) return DIT_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(o->ptr) & 15) || o->row % 8 || o->head % 8) return DIT_ERR_ALIGNMENT;
  return DIT_OK;
}

dit_status check_output(const dit_heads_t* v, int heads, int64_t rows, int dim, Heads* o) {
  const dit_status e = check_view(v, heads, rows, dim, o);
  return e == DIT_OK && !heads_apart(rows, heads, dim, o->row, o->head) ? DIT_ERR_INVALID_ARG : e;
}

bool buffers_apart(const dit_attention_plan_t& p, const void* saved, const void* scratch, const void* ws) {
  const size_t kept = (size_t)p.saved_bytes, free = (size_t)p.scratch_bytes;
  return bytes_apart(saved, kept, scratch, free) && bytes_apart(saved, kept, ws, WS_BYTES) && bytes_apart(scratch, free, ws, WS_BYTES);
}

bool map_heads(CUtensorMap* map, const Heads& t, int dim, int heads, int64_t rows, int box_heads, int box_rows) {
  return encode_tmap_heads(map, t.ptr, (uint64_t)dim, (uint64_t)heads, (uint64_t)rows, (uint64_t)t.head * 2, (uint64_t)t.row * 2,
                           (uint32_t)box_heads, (uint32_t)box_rows);
}

}  // namespace attn
}  // namespace dit6

extern "C" dit_status dit_attention_plan(const int64_t* queries, const int64_t* keys, const int64_t* begins, const int64_t* prefix,
                                         int64_t documents, int64_t frame, int heads, int kv_heads, int dim, int training,
                                         dit_attention_plan_t* plan, int32_t* table, int64_t table_ints) {
  try {
    return dit6::attn::make_plan(queries, keys, begins, prefix, documents, frame, heads, kv_heads, dim, training, plan, table, table_ints);
  } catch (...) {  // out of host memory
    return DIT_ERR_UNSUPPORTED;
  }
}
