// How the attention kernels over a paged cache divide their work.
//
// The new tokens of a sequence and the query heads that share a K/V head form
// the rows of one matrix product against that head's keys: row r is token
// r / group, query head r % group of the group. An item is one K/V head of one
// sequence with one tile of kRows rows; its work is counted in units of kKeys
// keys, over the keys that at least one of its rows can see: a prefix (the sink
// tokens) and a run that ends at its last token.
//
// All units of all items stand in one line (sequence, K/V head, row tile, key
// tile), each as long as it costs, and CTA c takes the c-th equal share of it. So a
// batch of unlike lengths, one long sequence and many short ones all load the GPU
// evenly, and the lengths are read where they are, on the device. An item that a boundary
// cuts is finished from partial results: each CTA writes its output (normalised,
// f32) and log-sum-exp to the workspace, and the CTA that arrives last joins
// them, always in the order of the keys, so results do not depend on timing.
#pragma once

#include "attention_internal.h"
#include "kaio_device.cuh"

namespace kaio {

// What the scores and masks are: kPlain has no prefixes and documents, the others do. Each
// is a kernel of its own: the chunks' loop over a row's scores leaves no register to spare, and
// code that is passed over is fetched all the same (one token over 1037 keys with slopes: 13.3 us
// with the cap's code in the kernel, 13.2 without).
enum class Form : int { kPlain, kMasks, kCapped, kDistance, kCappedDistance };
__host__ __device__ constexpr bool is_capped(Form f) { return f == Form::kCapped || f == Form::kCappedDistance; }
__host__ __device__ constexpr bool has_distance(Form f) { return f == Form::kDistance || f == Form::kCappedDistance; }

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMaxFloat = 3.4028234663852886e38f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

// kScored in what follows: with prefixes and documents (of the scored kernels; the others
// have no code for them).
struct PagedSeq {
  int q0, n, kv;     // first token, new tokens, positions in the cache
  int prefix;        // leading positions that all its tokens see
};

template <bool kScored>
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  if (p.q_starts) {
    s.q0 = min(max(p.q_starts[b], 0), p.tokens);
    s.n = min(max(p.q_starts[b + 1], s.q0), p.tokens) - s.q0;
  } else {
    s.q0 = b;
    s.n = 1;
  }
  const long long room = static_cast<long long>(p.max_pages) << p.page_shift;
  s.kv = static_cast<int>(min(static_cast<long long>(max(p.kv_lens[b], 0)),
                              min(room, static_cast<long long>(kPagedMaxLen))));
  s.prefix = kScored && p.prefix_lens ? min(max(p.prefix_lens[b], 0), s.kv) : 0;
  return s;
}

// Where the document of a sequence's row r begins.
template <bool kScored>
__device__ __forceinline__ int paged_doc(const PagedParams& p, const PagedSeq& s, int r) {
  return kScored && p.doc_starts ? min(max(p.doc_starts[s.q0 + p.group_div.div(r)], 0), kPagedMaxLen) : 0;
}

// Keys that the rows [r0, r1) of a sequence see: [from, first) and [lo, hi), and
// the key tiles that hold them. `from` is the document's begin of the first row: they do
// not decrease, so no row sees anything before it. A prefix that passes the causal end is
// that end, and otherwise as good as sink tokens. The units go through the run's tiles, the one at
// the window's edge last (its keys are hidden from some rows, and a poor maximum to
// begin with would have to be renewed), and then through those of the prefix.
template <int kKeys, bool kScored>
struct PagedSpan {
  int from, first, lo, hi;   // (an empty [from, first) is [0, 0))
  int lo_tile, run;    // the run's first tile, and its tiles
  int units;           // at least 1, so that every item is visited
  bool nearest_first;  // (scored) scores lose with distance: the run's tiles in reverse, or every tile would raise the maximum
  __device__ __forceinline__ bool back() const { return kScored && nearest_first; }
  __device__ __forceinline__ PagedSpan(const PagedParams& p, const PagedSeq& s, int r0, int r1, int doc) {
    const int t0 = p.group_div.div(r0), t1 = p.group_div.div(r1 - 1);
    hi = p.causal ? min(max(s.kv - s.n + t1 + 1, 0), s.kv) : s.kv;
    if (kScored) hi = max(hi, s.prefix);
    lo = p.window > 0 ? min(max(s.kv - s.n + t0 - p.window + 1, 0), hi) : 0;
    if (kScored) lo = min(max(lo, doc), hi);
    first = min(kScored ? max(p.sinks, s.prefix) : p.sinks, lo);
    from = 0;
    if (kScored) {
      if (first > doc) from = doc;
      else first = 0;
      if (lo == hi && first == 0) lo = hi = 0;
    }
    nearest_first = kScored && p.slopes != nullptr;
    lo_tile = lo / kKeys;
    run = (hi + kKeys - 1) / kKeys - lo_tile;
    units = max(1, run + max(min((first + kKeys - 1) / kKeys, lo_tile) - from / kKeys, 0));
  }
  __device__ __forceinline__ int key0(int unit) const {
    int tile = unit + lo_tile;
    if (back()) {
      tile = unit < run ? lo_tile + run - 1 - unit : unit - run + from / kKeys;
    } else if (lo > 0) {
      if (unit >= run) tile = unit - run + (kScored ? from / kKeys : 0);
      else tile = unit + 1 < run ? tile + 1 : lo_tile;
    }
    return tile * kKeys;
  }
};

// Keys that one row sees: from <= j < hi and (j >= lo or j < first); pos is its own place.
template <bool kScored>
struct PagedRow {
  int pos, from, first, lo, hi;
  __device__ __forceinline__ PagedRow(const PagedParams& p, const PagedSeq& s, int r, int doc) {
    pos = s.kv - s.n + p.group_div.div(r);
    hi = p.causal ? min(max(pos + 1, 0), s.kv) : s.kv;
    if (kScored) hi = max(hi, s.prefix);
    lo = p.window > 0 ? min(max(pos - p.window + 1, 0), hi) : 0;
    first = kScored ? max(p.sinks, s.prefix) : p.sinks;
    from = kScored ? doc : 0;
  }
  __device__ __forceinline__ bool sees(int j) const {
    return j < hi && (j >= lo || j < first) && (!kScored || j >= from);
  }
};

// a / b for 0 <= a < 2^53, 0 < b < 2^31, by a rounded estimate and its correction
// (the compiler's 64-bit division is some hundred instructions, and code is fetched
// slowly at a kernel's start).
__device__ __forceinline__ long long paged_div(long long a, int b) {
  const float inv = 1.0f / static_cast<float>(b);
  long long q = static_cast<long long>(static_cast<float>(a) * inv);
  long long r = a - q * b;
#pragma unroll 1
  while (r < 0 || r >= b) {
    long long step = static_cast<long long>(static_cast<float>(r) * inv);
    if (step == 0) step = r < 0 ? -1 : 1;
    q += step;
    r -= step * b;
  }
  return q;
}

// One CTA's share [begin, end) of a line of `total` cost among `ctas` CTAs: the
// first total % ctas shares have one more than the others.
struct PagedShare {
  long long begin, end, each;    // each = total / ctas
  int ctas, more;                // more = total % ctas
  int snap;                      // a boundary this near to an item's moves there
  int whole;                     // items of so many units are not cut at all
  __device__ __forceinline__ int owner(long long at) const {
    const long long first = (each + 1) * more;
    if (at < first) return static_cast<int>(paged_div(at, static_cast<int>(each + 1)));
    return more + static_cast<int>(paged_div(at - first, static_cast<int>(each)));
  }
};

// A place in the line of work: an item, and a unit in it. The constants of `Work`:
//   kScored               with prefixes and documents
//   kRows, kKeys          rows of a tile, keys of a unit
//   kCost, kSmallCost     length of a unit in the line; the second for items of at most
//                         kSmallRows rows
//   kItemCost             what an item costs besides its units
//   kPartWorth            what joining a part costs, in units, in the size of shares
//   kWhole, kJoin         An item that is not split waits for one CTA, a split one for its
//                         parts to be written and joined. With at most as many items as
//                         CTAs, none longer than kWhole units or than a share and kJoin,
//                         all stay whole and belong to the share that holds their
//                         beginning. (By their ends, the last tile of a causal head, its
//                         longest, would share a CTA with the first ones of the next.)
//                         Otherwise those of kWholeOfMany units do.
//   kSnap                 A boundary inside another item moves to its begin or end if that
//                         is nearer than half a share and than kSnap: a CTA with parts of
//                         two items does all that precedes and follows their units twice.
//                         (One token over 1037 keys of 32 heads, 9 shares to an item: 15.5
//                         us with boundaries where they fall, 11.6 us so; 100 tokens over
//                         9000, 32/8 heads: 73 and 59.)
//   kFewRows              Where no item is split and there are at most half as many as
//                         CTAs, the rows of a tile instead (three chunks of 77 tokens over
//                         613 keys, 15/3 heads: 15.5 us in 18 tiles, 13.1 us in 36; four
//                         of 60 over 1000, 16/4 heads: 19.9 and 15.0).
template <typename Work>
struct PagedWalk : Work {
  static constexpr bool kScored = Work::kScored;
  using Span = PagedSpan<Work::kKeys, kScored>;
  using Work::kRows, Work::kFewRows, Work::kKeys, Work::kCost, Work::kSmallCost, Work::kSmallRows, Work::kItemCost;
  static_assert(kSmallCost <= kCost && kCost < 8);
  int tile_rows;              // kRows or kFewRows
  int b, h, tile, tiles;      // item: sequence, K/V head, row tile of `tiles`
  int unit, units, cost;      // unit within the item; cost of one
  long long at;               // where in the line the item begins
  PagedSeq s;

  __device__ __forceinline__ int row_tiles(const PagedParams& p, const PagedSeq& s) const {
    return (s.n * p.group + step() - 1) / step();
  }
  __device__ __forceinline__ int step() const { return kFewRows < kRows ? tile_rows : kRows; }
  __device__ __forceinline__ int row0() const { return tile * step(); }
  __device__ __forceinline__ int row1(const PagedParams& p) const { return min(tile * step() + step(), s.n * p.group); }
  __device__ __forceinline__ int item_units(const PagedParams& p, const PagedSeq& s, int tile) const {
    return item_units(p, s, tile, paged_doc<kScored>(p, s, tile * step()));
  }
  __device__ __forceinline__ int item_units(const PagedParams& p, const PagedSeq& s, int tile, int doc) const {
    return Span(p, s, tile * step(), min(tile * step() + step(), s.n * p.group), doc).units;
  }
  __device__ __forceinline__ int item_cost(const PagedParams& p, const PagedSeq& s, int tile) const {
    return s.n * p.group - tile * step() <= kSmallRows || (kFewRows <= kSmallRows && step() == kFewRows) ? kSmallCost : kCost;
  }
  __device__ __forceinline__ int length() const { return kItemCost + units * cost; }
  // (divisions by constants)
  __device__ __forceinline__ int whole_units(int length) const {
    return kSmallCost != kCost && cost == kSmallCost ? length / kSmallCost : length / kCost;
  }
  __device__ __forceinline__ long long head_length(const PagedParams& p, const PagedSeq& s, int* longest) const {   // (8 units + cost)
    long long u = 0;
    const int tiles = row_tiles(p, s);
    auto add = [&](int i, int doc) {
      const int units = item_units(p, s, i, doc), cost = item_cost(p, s, i);
      u += kItemCost + units * cost;
      *longest = max(*longest, 8 * units + cost);
    };
    if (kScored && p.doc_starts) {
      // (eight documents' begins at a time: one after another they take a round trip each)
#pragma unroll 1
      for (int i = 0; i < tiles; i += 8) {
        int doc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) doc[k] = paged_doc<kScored>(p, s, min(i + k, tiles - 1) * step());
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < tiles) add(i + k, doc[k]);
      }
      return u;
    }
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) add(i, 0);
    return u;
  }
  // The unit at which a boundary of shares cuts this item: 0 and `units` for those before and past it.
  __device__ __forceinline__ int cut(long long boundary, const PagedShare& share) const {
    const long long to = boundary - at;
    if (to <= 0 || to >= length()) return to <= 0 ? 0 : units;
    if (units <= share.whole) return units;
    const int into = static_cast<int>(to);
    return into <= share.snap ? 0 : length() - into <= share.snap ? units : whole_units(max(into - kItemCost, 0));
  }
  // The CTAs that hold its first and its last unit.
  __device__ __forceinline__ int first_owner(const PagedShare& share) const {
    return share.owner(at + max(kItemCost + cost - 1, share.snap));
  }
  __device__ __forceinline__ int last_owner(const PagedShare& share) const {
    return share.owner(at + max(length() - share.snap - 1, share.snap));
  }
  // To the first unit of the next item (past the line's end: b == batch).
  __device__ __forceinline__ void next_item(const PagedParams& p) {
    at += length();
    unit = 0;
    if (++tile == tiles) {
      tile = 0;
      if (++h == p.kv_heads) {
        h = 0;
        do {
          if (++b >= p.batch) return;
          s = paged_seq<kScored>(p, b);
          tiles = row_tiles(p, s);
        } while (tiles == 0);
      }
    }
    units = item_units(p, s, tile);
    cost = item_cost(p, s, tile);
  }
};

// Found by all threads of the CTA together: the share of CTA `cta`, and the place of
// its first unit. Every thread sums a run of sequences; a scan gives the total and
// the run in which the share begins. `sums` holds a value for each warp in shared memory.
// Returns false if the share is empty.
template <int kThreads, typename Walk>
__device__ bool paged_share(const PagedParams& p, int cta, int grid, long long* sums, Walk* place,
                            PagedShare* share) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  constexpr int kWarps = kThreads / 32;
  // Few sequences with documents: a warp takes each, its lanes the row tiles (three prompts of 2500
  // tokens, a thread each: the first tile is found after 21000-28000 cycles, so after half of it; prompts of 1000 tokens
  // in documents take 127 us for 12 sequences, by warps, 141 for 13, by threads, where 10.6 a sequence would give 138).
  const bool by_warps = Walk::kScored && Walk::kRows > 32 && p.batch <= kWarps;
  constexpr bool kTwoSizes = Walk::kFewRows < Walk::kRows;
  Walk w;
  long long mine, upto, total, head = 0;
  int longest, items;
#pragma unroll 1
  for (w.tile_rows = Walk::kRows;; w.tile_rows = Walk::kFewRows) {
    mine = 0, total = 0, longest = 0, items = 0;
    if (by_warps && (tid >> 5) < p.batch) {
      w.s = paged_seq<Walk::kScored>(p, tid >> 5);
      w.tiles = w.row_tiles(p, w.s);
#pragma unroll 1
      for (int i = lane; i < w.tiles; i += 32) {
        const int units = w.item_units(p, w.s, i), cost = w.item_cost(p, w.s, i);
        mine += Walk::kItemCost + units * cost;
        longest = max(longest, 8 * units + cost);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
      head = mine;
      mine = lane == 0 ? mine * p.kv_heads : 0;
      if (kTwoSizes) items = lane == 0 ? min(p.kv_heads * w.tiles, 1 << 20) : 0;
    }
#pragma unroll 1
    for (int b = by_warps ? b1 : b0; b < b1; ++b) {
      const PagedSeq s = paged_seq<Walk::kScored>(p, b);
      mine += p.kv_heads * w.head_length(p, s, &longest);
      if (kTwoSizes) items = min(items + p.kv_heads * w.row_tiles(p, s), 1 << 20);
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long add = __shfl_up_sync(0xFFFFFFFFu, upto, d);
      if ((tid & 31) >= d) upto += add;
    }
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    if (kTwoSizes) items = __reduce_add_sync(0xFFFFFFFFu, items);
    if ((tid & 31) == 31) {
      sums[tid >> 5] = upto;
      sums[kWarps + (tid >> 5)] = longest | static_cast<long long>(items) << 32;
    }
    __syncthreads();
    items = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == (tid >> 5)) upto += total;
      total += sums[i];
      longest = max(longest, static_cast<int>(sums[kWarps + i]));
      if (kTwoSizes) items += static_cast<int>(sums[kWarps + i] >> 32);
    }
    if (!kTwoSizes || w.tile_rows == Walk::kFewRows || (longest >> 3) > Walk::kWhole || 2 * items > grid) break;
    __syncthreads();                                       // sums have been read
  }
  if (total == 0) return false;
  // The share has to be worth its CTA: one unit where no item is split. An item of U units
  // in shares of u takes about u units' time, and then U / u parts to join one after another;
  // with a part at kPartWorth units the sum is least for u = sqrt(kPartWorth U).
  const int units = longest >> 3, cost = longest & 7;
  const int least = units <= Walk::kWhole ? 1 : max(1, static_cast<int>(sqrtf(Walk::kPartWorth * static_cast<float>(units))));
  // (tiles of one size take a sequence's few rows: one item for each K/V head, not counted)
  const bool few = kTwoSizes ? items <= grid : static_cast<long long>(p.batch) * p.kv_heads <= grid;
  // (A share that cuts an item holds a unit at least. Where nothing is cut: enough shares that no item meets another, and no more, since idle
  // CTAs slow the others' start: 10 sequences of 4 keys, 4 K/V heads: 6.4 us on 120, 6.2 on 40.)
  const bool uncut = units <= (few ? Walk::kWhole : Walk::kWholeOfMany);
  const long long length = uncut && kTwoSizes ? total - items * Walk::kItemCost : total;
  const int worth = !uncut ? max(least * cost, Walk::kCost) : kTwoSizes ? cost : Walk::kItemCost + cost;
  share->ctas = static_cast<int>(min(static_cast<long long>(grid), max(1ll, paged_div(length, worth))));
  if (cta >= share->ctas) return false;
  share->each = paged_div(total, share->ctas);
  share->more = static_cast<int>(total - share->each * share->ctas);
  const int each = static_cast<int>(min(share->each, 1ll << 30));
  const int limit = max(Walk::kWhole, Walk::kJoin + each / Walk::kCost);
  share->whole = few && units <= limit ? limit : Walk::kWholeOfMany;
  share->snap = min(Walk::kSnap, (each + 1) / 2);
  share->begin = cta * share->each + min(cta, share->more);
  share->end = share->begin + share->each + (cta < share->more ? 1 : 0);
  if (by_warps) {
    const long long from = upto - head * p.kv_heads;
    if ((tid >> 5) < p.batch && share->begin >= from && share->begin < upto) {
      long long left = share->begin - from;
      w.b = tid >> 5;
#pragma unroll 1
      for (w.h = 0; left >= head; ++w.h) left -= head;
#pragma unroll 1
      for (int t0 = 0;; t0 += 32) {
        const int t = min(t0 + lane, w.tiles - 1);
        w.units = w.item_units(p, w.s, t);
        w.cost = w.item_cost(p, w.s, t);
        long long end = t0 + lane < w.tiles ? w.length() : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long add = __shfl_up_sync(0xFFFFFFFFu, end, d);
          if (lane >= d) end += add;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, end > left);
        if (past != 0) {
          if (lane == __ffs(past) - 1) {
            w.tile = t;
            w.at = share->begin - (left - (end - w.length()));
            w.unit = w.cut(share->begin, *share);
            if (w.unit == w.units) w.next_item(p);
            *place = w;
          }
          break;
        }
        left -= __shfl_sync(0xFFFFFFFFu, end, 31);
      }
    }
    __syncthreads();
    return true;
  }
  const long long from = upto - mine;
  if (share->begin >= from && share->begin < upto) {
    long long left = share->begin - from;
#pragma unroll 1
    for (w.b = b0;; ++w.b) {
      w.s = paged_seq<Walk::kScored>(p, w.b);
      const long long head = w.head_length(p, w.s, &longest);
      if (left < head * p.kv_heads) {
        w.tiles = w.row_tiles(p, w.s);
#pragma unroll 1
        for (w.h = 0; left >= head; ++w.h) left -= head;
        break;
      }
      left -= head * p.kv_heads;
    }
#pragma unroll 1
    for (w.tile = 0;; ++w.tile) {
      w.units = w.item_units(p, w.s, w.tile);
      w.cost = w.item_cost(p, w.s, w.tile);
      if (left < w.length()) break;
      left -= w.length();
    }
    w.at = share->begin - left;
    w.unit = w.cut(share->begin, *share);
    if (w.unit == w.units) w.next_item(p);
    *place = w;
  }
  __syncthreads();
  return true;
}

// A slope times log2(e). Where that passes f32's range it is the largest number: the token's own key, at a
// distance of zero, then keeps a bias of zero.
__device__ __forceinline__ float slope_log2(float slope) {
  const float s = slope * kLog2e;
  return fabsf(s) <= kMaxFloat ? s : copysignf(kMaxFloat, s) + 0.f * slope;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace kaio
