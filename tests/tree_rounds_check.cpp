// Checks how csrc/chunk_plan.h shares trees out in rounds of whole row tiles: the
// kernel's own functions, put together as its plan does, cover every (row tile, key
// tile) exactly once, evenly, with at most two cut row tiles a pair. Compiled by the
// host compiler with traps on undefined arithmetic; prints "ok".
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <random>
#include <vector>

#include "chunk_plan.h"

using namespace dsakv;
using std::vector;

#define CHECK(x)                                                            \
  do {                                                                      \
    if (!(x)) {                                                             \
      printf("line %d: %s\n", __LINE__, #x);                                \
      exit(1);                                                              \
    }                                                                       \
  } while (0)

struct Args {
  const Request* r;
  int B, H;
  bool causal;
};
static Request request(const Args& a, int b) { return a.r[b]; }

// Returns the rounds that the plan takes (0: stretches alone).
static int check(const vector<Request>& rs, int H, int pairs) {
  const Args a{rs.data(), int(rs.size()), H, false};
  int64_t total = 0;
  vector<int> first(1, 0), units;
  for (const Request& r : rs) {
    const int t = row_tiles(H, r);
    first.push_back(first.back() + t);
    units.push_back(key_tiles(r.ctx));
    total += int64_t(t) * units.back();
  }
  int rounds = first.back() / pairs - 1;
  vector<int> load(pairs, 0);
  int64_t within = 0;
  for (int p = 0; rounds > 0 && p < pairs; ++p) {
    for (int b = 0; b < a.B; ++b) {
      const int mine = round_tiles(pairs, rounds, p, first[b], first[b + 1]);
      int counted = 0;  // one by one
      for (int i = first[b]; i < first[b + 1]; ++i) counted += i % pairs == p && i / pairs < rounds;
      CHECK(mine == counted);
      load[p] += mine * units[b];
    }
    within += load[p];
  }
  bool fits = rounds > 0;
  for (int p = 0; p < pairs; ++p) fits = fits && load[p] < stretch_of(total, pairs, p).count;
  if (!fits) return 0;

  std::map<std::pair<int, int>, vector<char>> seen;  // (request, row tile): its key tiles
  for (int p = 0; p < pairs; ++p) {
    const Stretch rest = stretch_behind(total, pairs, p, load.data());
    CHECK(rest.count >= 1 && rest.count + load[p] == stretch_of(total, pairs, p).count);
    if (p == 0) CHECK(rest.from == within);
    // where the stretch begins, as the kernel's threads find it
    Walk w{0, 0, 0, rest.count};
    int64_t before = 0;
    for (int b = 0; b < a.B; ++b) {
      const int t = row_tiles(H, rs[b]);
      const int64_t u = t ? units_before(H, false, rs[b], t, t) : 0;
      if (u && rest.from >= before && rest.from < before + u) {
        const Place at = place_of(H, false, rs[b], rest.from - before);
        w.b = b, w.j = at.j, w.u = at.u;
      }
      before += u;
    }
    Walker<true> walk{w, rounds, pairs, 0, p};
    Segment s;
    int heads = 0, tails = 0, whole = 0;
    while (walk.next(a, s)) {
      CHECK(s.rows > 0 && s.rows <= kRows && s.row0 % kRows == 0 && s.t0 < s.t1);
      vector<char>& keys = seen[{s.b, s.row0 / kRows}];
      keys.resize(units[s.b], 0);
      CHECK(s.t1 <= units[s.b] && s.starts == (s.t0 == 0) && s.ends == (s.t1 == units[s.b]));
      for (int t = s.t0; t < s.t1; ++t) CHECK(!keys[t]++);
      if (!(s.starts && s.ends)) ++(s.starts ? heads : tails);
      else ++whole;
    }
    CHECK(heads <= 1 && tails <= 1 && whole >= rounds);
  }
  int64_t covered = 0;
  for (const auto& k : seen)
    for (char c : k.second) covered += c;
  CHECK(covered == total);
  return rounds;
}

int main() {
  std::mt19937 g(1);
  auto pick = [&](int lo, int hi) { return int(lo + g() % uint32_t(hi - lo + 1)); };
  long long taken = 0, cases = 0;
  CHECK(check(vector<Request>(16, Request{0, 64, 8192}), 128, 76) == 12);
  for (int i = 0; i < 4000; ++i) {
    vector<Request> rs(pick(1, 64));
    const int H = pick(1, 200), pairs = pick(1, 80), longest = pick(1, 6000);
    for (Request& r : rs) {
      r.q0 = 0;
      r.n = pick(0, 90);
      r.ctx = pick(0, longest);
    }
    taken += check(rs, H, pairs) > 0;
    ++cases;
  }
  CHECK(taken > 500);
  printf("ok %lld of %lld\n", taken, cases);
  return 0;
}
