// How the prompt attention shares its work among the CTAs: plain integer
// arithmetic on the sequences' lengths, the same in every CTA (and replayed on
// the CPU by tests/prompt_split_check.cpp).
//
// An item is a tile of `unit` (128 or 256) queries of a sequence for one of its
// `hp` heads (or pairs of heads).  Items lie end to end, ordered by sequence,
// head, tile (the tiles of a head read the same keys: side by side, they find
// them in L2); one takes as many units as the 128-key blocks its last query
// sees, and kPromptItem for what an item costs besides.  CTA c gets the units
// from bound c to bound c + 1, `chunk` apart, so that all CTAs get the same
// amount whatever the lengths.  A bound inside an item splits its blocks, unless
// fewer than kPromptEdge blocks would be left on one side; where no item is long
// enough for that to pay, bounds move to the nearer end of the item, or, with no
// more items than CTAs, every item is one unit.
#pragma once

#ifdef __CUDACC__
#define DS_HD __host__ __device__ __forceinline__
#else
#define DS_HD inline
#endif

namespace ds {

constexpr int kPromptEdge = 4;  // least blocks of a part
constexpr int kPromptItem = 2;  // units of an item besides its blocks
constexpr int kPromptParts = 8; // about as many parts as an item may be cut into
constexpr int kPromptLanes = 32; // most lanes (a thread of a warp each)
constexpr int kPromptJoin = 8;  // what a cut costs a CTA, in units: storing its parts, joining one

struct PromptSeq {
  int q0 = 0, lq = 0, k0 = 0, lk = 0;  // first packed rows, and lengths
};
struct PromptBound {
  int b = 0, t = 0, h = 0, j = 0;  // item (sequence, tile, head) and block; j = its blocks: behind the item
  long long u0 = 0;                // the item's first unit
};

DS_HD int prompt_tiles(const PromptSeq& s, int unit) { return (s.lq + unit - 1) / unit; }
// 128-key blocks that the last query of tile t sees.
DS_HD int prompt_blocks(const PromptSeq& s, int unit, int t) {
  const long long end = (long long)(t + 1) * unit;
  const long long seen = (long long)s.lk - s.lq + (end < s.lq ? end : s.lq);
  return seen > 0 ? (int)((seen + 127) >> 7) : 0;
}
// Units of one head of tiles 0 .. t-1, in closed form: all tiles but the last
// see a + k (unit / 128) blocks, k = 1, 2, ..., where that is positive.
DS_HD long long prompt_units(const PromptSeq& s, int unit, int t) {
  const int T = prompt_tiles(s, unit);
  const long long a = ((long long)s.lk - s.lq + 127) >> 7, d = unit >> 7;  // (>> rounds down: a ceiling)
  const long long k = t < T ? t : (T > 0 ? T - 1 : 0);                      // tiles of the series
  long long m = 0;                                                           // of them, those that see nothing
  if (a < 0) m = (-a) / d < k ? (-a) / d : k;
  long long u = kPromptItem * k + (k - m) * a + d * (k * (k + 1) - m * (m + 1)) / 2;
  if (t >= T && T > 0) u += prompt_blocks(s, unit, T - 1) + kPromptItem;
  return u;
}
struct PromptPlan {
  long long chunk = 1;  // units from one bound to the next
  int cut = 0;          // whether bounds may cut items
  int flat = 0;         // every item is one unit
  int lanes = 0;        // shares lie in lanes: units are counted from the lane's start,
  int base = 0;         // its first CTA
};
// An even share of `total` units.  Whole items make some CTA late by what the
// longest is over that, or by half of it; they are cut where that costs more
// than the cuts, into parts that are worth one and not too many to join.
DS_HD PromptPlan prompt_plan(long long total, long long items, int grid, int longest) {
  PromptPlan p;
  const long long even = (total + grid - 1) / grid;
  const long long late = even > longest ? longest / 2 : longest + kPromptItem - even;
  p.cut = late > kPromptJoin;
  long long least = 1 + kPromptItem;
  if (p.cut) {
    least = (longest + kPromptParts - 1) / kPromptParts;
    if (least < 2 * kPromptEdge) least = 2 * kPromptEdge;
  }
  p.chunk = even > least ? even : least;
  if (!p.cut && items <= grid) {
    p.flat = 1;
    p.chunk = 1;
  }
  return p;
}
// Lanes: the least share for which they fit into `grid` CTAs, 0 where that is more
// than a sixteenth above the even share or parts would be too short.  ctas(c) is
// the number of CTAs that all lanes take at c units each.
template <class F>
DS_HD int prompt_lane_share(long long total, long long lanes, int grid, const PromptPlan& p, const F& ctas) {
  if (!p.cut || lanes > kPromptLanes || lanes * 8 > grid || total >= (1LL << 30)) return 0;
  int lo = (int)((total + grid - 1) / grid), hi = lo + lo / 16;
  if (p.chunk > lo || ctas(hi) > grid) return 0;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ctas(mid) <= grid) hi = mid;
    else lo = mid + 1;
  }
  return hi;
}
// CTAs of a lane whose sequence's last tile sees `top` blocks, at c units each.
DS_HD int prompt_lane_ctas(int hp, int top, int c) { return (hp * (top + kPromptItem) + c - 1) / c; }

// Units of each of a lane's k shares; lanes are not taken where that is below
// 2 kPromptEdge for one of them.
DS_HD int prompt_lane_chunk(int hp, int n, int k) { return (hp * (n + kPromptItem) + k - 1) / k; }

// Block j of an item of n as a bound.
DS_HD int prompt_edge(const PromptPlan& p, int j, int n) {
  return !p.cut || j < kPromptEdge || n - j < kPromptEdge ? (2 * j < n || j < 1 ? 0 : n) : j;
}
// The bound at unit v of tile t's lane of sequence b.
DS_HD PromptBound prompt_lane_locate(const PromptPlan& p, int b, int t, int n, long long v) {
  PromptBound r;
  r.b = b;
  r.t = t;
  r.h = (int)(v / (n + kPromptItem));
  r.u0 = (long long)r.h * (n + kPromptItem);
  r.j = prompt_edge(p, (int)(v - r.u0) - kPromptItem, n);
  return r;
}
// The bound at unit v (0 <= v < the units of all heads) of sequence b, whose
// first unit is `before`.
DS_HD PromptBound prompt_locate(const PromptSeq& s, int unit, const PromptPlan& p, int b, long long before, long long v) {
  const int T = prompt_tiles(s, unit);
  const long long per_head = p.flat ? T : prompt_units(s, unit, T);
  PromptBound r;
  r.b = b;
  r.h = (int)(v / per_head);
  v -= r.h * per_head;
  if (p.flat) {
    r.t = (int)v;
    r.u0 = before + r.h * per_head + v;
    return r;
  }
  int lo = 0, hi = T - 1;  // the last tile that starts at or before v
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (prompt_units(s, unit, mid) <= v) lo = mid;
    else hi = mid - 1;
  }
  r.t = lo;
  const int n = prompt_blocks(s, unit, lo);
  const long long first = prompt_units(s, unit, lo);
  r.u0 = before + r.h * per_head + first;
  r.j = prompt_edge(p, (int)(v - first) - kPromptItem, n);
  return r;
}
// The CTAs that hold parts of the item of n blocks at unit u0: *first and the
// ones after it, their number returned (1: the item is whole).
DS_HD int prompt_parts(long long u0, int n, const PromptPlan& p, int* first) {
  const long long chunk = p.chunk;
  const long long c_lo = (u0 + kPromptItem + kPromptEdge + chunk - 1) / chunk;
  const long long c_hi = (u0 + kPromptItem + n - kPromptEdge) / chunk;
  *first = p.base + (int)(c_lo - 1);
  return p.cut && n >= 2 * kPromptEdge && c_hi >= c_lo ? (int)(c_hi - c_lo) + 2 : 1;
}

// The items of a share, one after the other.  seq_of(b) gives sequence b.
struct PromptItem {
  int b = 0, t = 0, h = 0, n = 0;  // n: its blocks
  long long u0 = 0;
  PromptSeq s;
};
template <class F>
DS_HD PromptItem prompt_after(PromptItem x, const PromptPlan& p, int batch, int unit, int hp, const F& seq_of) {
  x.u0 += p.flat ? 1 : x.n + kPromptItem;
  if (p.lanes) {
    if (++x.h >= hp) x.b = batch;
    return x;
  }
  ++x.t;
  while (x.t >= prompt_tiles(x.s, unit)) {
    x.t = 0;
    if (prompt_tiles(x.s, unit) > 0 && ++x.h < hp) break;
    x.h = 0;
    if (++x.b >= batch) return x;  // behind the last item
    x.s = seq_of(x.b);
  }
  x.n = prompt_blocks(x.s, unit, x.t);
  return x;
}
// The first item of the share between two bounds and its first block; b =
// batch where the share is empty.
template <class F>
DS_HD PromptItem prompt_first(const PromptBound& from, const PromptBound& till, const PromptPlan& p, int batch, int unit, int hp,
                              const F& seq_of, int* j0) {
  PromptItem x;
  *j0 = 0;
  x.b = batch;
  if (from.b >= batch || (from.b == till.b && from.u0 == till.u0 && from.j == till.j)) return x;
  x.b = from.b;
  x.t = from.t;
  x.h = from.h;
  x.u0 = from.u0;
  x.s = seq_of(x.b);
  x.n = prompt_blocks(x.s, unit, x.t);
  if (from.j > 0 && from.j == x.n) return prompt_after(x, p, batch, unit, hp, seq_of);
  *j0 = from.j;
  return x;
}
// Whether item x is the one in which bound `till` lies.
DS_HD bool prompt_last(const PromptItem& x, const PromptBound& till) { return x.b == till.b && x.u0 == till.u0; }

}  // namespace ds
