// Replays the lanes of the prompt attention's work split (csrc/prompt_split.h)
// on the CPU over random batches, as prompt_split_check.cpp does for items laid
// end to end: each block of each item in exactly one CTA, in order within its
// lane; the CTAs of a split item as prompt_parts gives them; at most one part
// that continues an item and one that is continued per CTA; no part under
// kPromptEdge blocks; no share more than a sixteenth above the even one (and what
// a bound moves); all lanes of a sequence over as many CTAs.
// Prints "ok <batches with lanes>" or the first violation.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "prompt_split.h"

using namespace ds;

#define REQUIRE(x)                                                              \
  do {                                                                          \
    if (!(x)) {                                                                 \
      printf("violated: %s (case %d)\n", #x, g_case);                           \
      exit(1);                                                                  \
    }                                                                           \
  } while (0)
static int g_case = 0;

struct Lane {
  int b, t, n, top;
};

static bool check(const std::vector<PromptSeq>& seqs, int unit, int hp, int grid) {
  const int B = (int)seqs.size();
  auto seq_of = [&](int b) { return seqs[b]; };
  long long total = 0, items = 0;
  int longest = 0;
  std::vector<Lane> lanes;
  for (int b = 0; b < B; ++b) {
    const int T = prompt_tiles(seqs[b], unit);
    total += hp * prompt_units(seqs[b], unit, T);
    items += (long long)hp * T;
    if (seqs[b].lq > 0) longest = std::max(longest, (seqs[b].lk + 127) / 128);
    for (int t = 0; t < T; ++t)
      lanes.push_back({b, t, prompt_blocks(seqs[b], unit, t), prompt_blocks(seqs[b], unit, T - 1)});
  }
  PromptPlan plan = prompt_plan(total, items, grid, longest);
  auto ctas = [&](int c) {
    int k = 0;
    for (const auto& l : lanes) k += prompt_lane_ctas(hp, l.top, c);
    return k;
  };
  const int share = prompt_lane_share(total, (long long)lanes.size(), grid, plan, ctas);
  if (share == 0) return false;
  REQUIRE(plan.cut && ctas(share) <= grid);
  for (const auto& l : lanes)
    if (prompt_lane_chunk(hp, l.n, prompt_lane_ctas(hp, l.top, share)) < 2 * kPromptEdge) return false;
  const long long even = (total + grid - 1) / grid;
  REQUIRE(share <= even + even / 16);
  plan.lanes = 1;
  int base = 0;
  for (const auto& l : lanes) {
    const int k = prompt_lane_ctas(hp, l.top, share), chunk = prompt_lane_chunk(hp, l.n, k);
    const long long units = (long long)hp * (l.n + kPromptItem);
    plan.base = base;
    plan.chunk = chunk;
    int h = 0, at = 0;  // what comes next: item and block
    for (int c = 0; c < k; ++c) {
      PromptBound bound[2];
      for (int i = 0; i < 2; ++i) {
        bound[i].b = B;
        if ((long long)(c + i) * chunk < units) bound[i] = prompt_lane_locate(plan, l.b, l.t, l.n, (long long)(c + i) * chunk);
      }
      int j0, continues = 0, continued = 0;
      long long work = 0;
      PromptItem x = prompt_first(bound[0], bound[1], plan, B, unit, hp, seq_of, &j0);
      while (x.b < B) {
        const bool last = prompt_last(x, bound[1]);
        if (last && bound[1].j <= j0) break;
        const int j1 = last ? bound[1].j : x.n;
        REQUIRE(x.b == l.b && x.t == l.t && x.h == h && x.n == l.n && j0 == at && (j1 > j0 || x.n == 0));
        REQUIRE(x.u0 == (long long)h * (l.n + kPromptItem));
        work += j1 - j0 + (j0 == 0 ? kPromptItem : 0);
        int first = -1;
        const int parts = prompt_parts(x.u0, x.n, plan, &first), mine = base + c;
        const bool whole = j0 == 0 && j1 >= x.n;
        REQUIRE(whole == (parts == 1));
        if (!whole) {
          REQUIRE(first >= base && mine >= first && mine < first + parts && first + parts <= base + k);
          REQUIRE((mine == first) == (j0 == 0) && (mine == first + parts - 1) == (j1 == x.n));
          REQUIRE(j1 - j0 >= kPromptEdge);
          if (j0 > 0) ++continues;
          else ++continued;
        }
        at = j1 >= x.n ? 0 : j1;
        if (j1 >= x.n) ++h;
        if (last) break;
        x = prompt_after(x, plan, B, unit, hp, seq_of);
        j0 = 0;
      }
      REQUIRE(continues <= 1 && continued <= 1);
      REQUIRE(work <= chunk + 2 * kPromptEdge + kPromptItem);
    }
    REQUIRE(h == hp && at == 0);
    base += k;
  }
  REQUIRE(base <= grid);
  return true;
}

int main(int argc, char** argv) {
  const int cases = argc > 1 ? atoi(argv[1]) : 20000;
  std::mt19937 rng(54321);
  auto uni = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int with = 0;
  for (g_case = 0; g_case < cases; ++g_case) {
    const int B = uni(1, 6), most_q = g_case % 3 == 0 ? 300 : (g_case % 3 == 1 ? 1000 : 5000);
    std::vector<PromptSeq> seqs(B);
    for (auto& s : seqs) {
      s.lq = uni(0, 4) == 0 ? 0 : uni(0, most_q);
      const int kind = uni(0, 5);
      s.lk = kind == 0 ? s.lq : (kind == 1 ? uni(0, s.lq) : (kind == 2 ? 0 : s.lq + uni(0, 100000)));
    }
    with += check(seqs, uni(0, 1) ? 128 : 256, uni(1, 80), uni(0, 3) ? 152 : uni(1, 200));
  }
  REQUIRE(with > cases / 20);
  printf("ok %d\n", with);
  return 0;
}
