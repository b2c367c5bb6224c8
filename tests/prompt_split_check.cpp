// Replays the prompt attention's work split (csrc/prompt_split.h) on the CPU
// over random batches: the closed form of the units against a sum, and the
// walk of every CTA against what the kernel relies on -- each block of each
// item in exactly one CTA, in order; the parts of a split item numbered from
// prompt_parts' first CTA without gaps; at most one part that continues an
// item and one that is continued per CTA; no part under kPromptEdge blocks.
// Prints "ok <batches>" or the first violation.
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

static void check(const std::vector<PromptSeq>& seqs, int unit, int hp, int grid) {
  const int B = (int)seqs.size();
  auto seq_of = [&](int b) { return seqs[b]; };
  std::vector<long long> before(B + 1, 0);
  long long items = 0;
  for (int b = 0; b < B; ++b) {
    const int T = prompt_tiles(seqs[b], unit);
    long long u = 0;
    for (int t = 0; t < T; ++t) {
      REQUIRE(prompt_units(seqs[b], unit, t) == u);
      const long long last_q = std::min((long long)(t + 1) * unit, (long long)seqs[b].lq) - 1;
      const long long sees = seqs[b].lk - seqs[b].lq + last_q + 1;  // keys 0 .. of the tile's last query
      REQUIRE(prompt_blocks(seqs[b], unit, t) == (sees > 0 ? (sees + 127) / 128 : 0));
      u += prompt_blocks(seqs[b], unit, t) + kPromptItem;
    }
    REQUIRE(prompt_units(seqs[b], unit, T) == u);
    before[b + 1] = before[b] + hp * u;
    items += (long long)hp * T;
  }
  const long long total = before[B];
  int longest = 0;
  for (const auto& s : seqs) longest = std::max(longest, s.lq > 0 ? (s.lk + 127) / 128 : 0);
  const PromptPlan plan = prompt_plan(total, items, grid, longest);
  if (plan.flat)
    for (int b = 0; b < B; ++b) before[b + 1] = before[b] + (long long)hp * prompt_tiles(seqs[b], unit);
  const long long chunk = plan.chunk;
  REQUIRE(chunk * grid >= before[B]);
  auto bound = [&](long long u) {
    PromptBound r;
    r.b = B;
    for (int b = 0; b < B; ++b)
      if (u >= before[b] && u < before[b + 1]) return prompt_locate(seqs[b], unit, plan, b, before[b], u - before[b]);
    return r;
  };
  // what comes next: item (b, t, h) and block
  long long seen_items = 0;
  PromptItem want;
  int want_j = 0;
  bool any = false;
  want.b = 0;
  for (want.b = 0; want.b < B && prompt_tiles(seqs[want.b], unit) == 0;) ++want.b;
  if (want.b < B) {
    want.s = seqs[want.b];
    want.n = prompt_blocks(want.s, unit, 0);
    want.u0 = before[want.b];
  }
  for (int c = 0; c < grid; ++c) {
    const PromptBound from = bound((long long)c * chunk), till = bound(((long long)c + 1) * chunk);
    int j0, continues = 0, continued = 0;
    long long share = 0;
    PromptItem x = prompt_first(from, till, plan, B, unit, hp, seq_of, &j0);
    while (x.b < B) {
      const bool last = prompt_last(x, till);
      if (last && till.j <= j0) break;
      const int j1 = last ? till.j : x.n;
      REQUIRE(x.b == want.b && x.t == want.t && x.h == want.h && x.u0 == want.u0 && x.n == want.n && j0 == want_j);
      REQUIRE(j1 > j0 || x.n == 0);
      share += j1 - j0 + (j0 == 0 ? kPromptItem : 0);
      const bool whole = j0 == 0 && j1 >= x.n;
      int first = -1;
      const int parts = prompt_parts(x.u0, x.n, plan, &first);
      REQUIRE(whole == (parts == 1));
      REQUIRE(parts <= kPromptParts + 2);
      if (!whole) {
        REQUIRE(c >= first && c < first + parts && first >= 0);
        REQUIRE((c == first) == (j0 == 0) && (c == first + parts - 1) == (j1 == x.n));
        REQUIRE(j1 - j0 >= kPromptEdge);
        if (j0 > 0) ++continues;
        else ++continued;
      }
      any = true;
      if (j1 >= x.n) {
        ++seen_items;
        want = prompt_after(want, plan, B, unit, hp, seq_of);
        want_j = 0;
      } else {
        want_j = j1;
      }
      if (last) break;
      x = prompt_after(x, plan, B, unit, hp, seq_of);
      j0 = 0;
    }
    REQUIRE(continues <= 1 && continued <= 1);
    REQUIRE(share <= (plan.flat ? longest : chunk + (plan.cut ? 2 * kPromptEdge : longest)) + kPromptItem);
  }
  REQUIRE(seen_items == items);
  REQUIRE(!any == (items == 0));
}

int main(int argc, char** argv) {
  const int cases = argc > 1 ? atoi(argv[1]) : 4000;
  std::mt19937 rng(12345);
  auto uni = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (g_case = 0; g_case < cases; ++g_case) {
    const int B = uni(1, g_case % 7 == 0 ? 60 : 6);
    const int most_q = g_case % 3 == 0 ? 300 : (g_case % 3 == 1 ? 3000 : 20000);
    std::vector<PromptSeq> seqs(B);
    for (auto& s : seqs) {
      s.lq = uni(0, 4) == 0 ? 0 : uni(0, most_q);
      const int kind = uni(0, 4);
      s.lk = kind == 0 ? s.lq : (kind == 1 ? uni(0, s.lq) : (kind == 2 ? s.lq + uni(0, 40000) : (kind == 3 ? 0 : s.lq + uni(0, 200))));
    }
    check(seqs, uni(0, 1) ? 128 : 256, uni(1, 40), uni(0, 3) ? 152 : uni(1, 200));
  }
  printf("ok %d\n", cases);
  return 0;
}
