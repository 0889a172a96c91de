// Checks csrc/chunk_plan.h, the kernel's own functions, against counts made one
// by one in 64 bits. Compiled by the host compiler with traps on undefined
// arithmetic (signed overflow among them); prints "ok" and the cases' number.
#include <stdio.h>
#include <stdlib.h>

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

static long long cases = 0;

// The definitions, in 64 bits.
static int64_t tiles_of(int H, const Request& r) { return (int64_t(r.n) * H + 127) / 128; }
static int64_t end_of(int H, bool causal, const Request& r, int64_t j) {
  if (!causal) return r.ctx;
  int64_t last = j * 128 + 127;                    // the tile's last row
  if (last > int64_t(r.n) * H - 1) last = int64_t(r.n) * H - 1;
  const int64_t end = int64_t(r.ctx) - r.n + last / H + 1;
  return end < 0 ? 0 : end;
}
static int64_t units_of(int64_t end) { return end <= 256 ? 1 : (end + 255) / 256; }

// Every row tile's first unit, and where units at a tile's ends belong.
static void closed_form(int H, bool causal, Request r) {
  const int tiles = row_tiles(H, r);
  CHECK(tiles == tiles_of(H, r));
  int64_t s = 0;
  for (int j = 0; j < tiles; ++j) {
    const int64_t end = end_of(H, causal, r, j), units = units_of(end);
    CHECK(key_end(H, causal, r, j) == end);
    CHECK(key_tiles(static_cast<int>(end)) == units);
    CHECK(units_before(H, causal, r, tiles, j) == s);
    if (j < 300 || j % 4099 == 0 || j + 300 > tiles) {
      const Place first = place_of(H, causal, r, s), last = place_of(H, causal, r, s + units - 1);
      CHECK(first.j == j && first.u == 0);
      CHECK(last.j == j && last.u == units - 1);
    }
    s += units;
  }
  CHECK(units_before(H, causal, r, tiles, tiles) == s);
  ++cases;
}

struct Line {
  vector<Request> r;
  int B, H;
  bool causal;
};
static Request request(const Line& a, int b) { return a.r[b]; }

// All pairs' stretches: every unit of the line once and in order, a pair's cut
// row tiles at most one that it begins and one that it does not, each cut tile
// begun by one pair and ended by a later one.
static void stretches(const Line& a, int max_pairs) {
  vector<int64_t> before(1, 0);
  for (const Request& r : a.r) {
    const int t = row_tiles(a.H, r);
    before.push_back(before.back() + (r.n ? units_before(a.H, a.causal, r, t, t) : 0));
  }
  const int64_t total = before.back();
  int64_t at = 0;                                   // next unit of the line
  int b = 0, j = 0;
  int64_t u = 0;                                    // and where it lies
  auto skip = [&] {
    while (b < a.B && j >= tiles_of(a.H, a.r[b])) ++b, j = 0;
  };
  skip();
  for (int pair = 0; pair < max_pairs; ++pair) {
    const Stretch st = stretch_of(total, max_pairs, pair);
    CHECK(st.count >= 0 && (st.count == 0 || st.from == at));
    if (!st.count) continue;
    int rb = 0;
    while (st.from >= before[rb + 1]) ++rb;
    const Place p = place_of(a.H, a.causal, a.r[rb], st.from - before[rb]);
    Walk walk{rb, p.j, p.u, st.count};
    Segment s;
    int begun = 0, taken_over = 0;
    while (walk.next(a, s)) {
      CHECK(s.b == b && s.row0 == j * 128 && s.t0 == u);
      const int64_t end = end_of(a.H, a.causal, a.r[b], j), units = units_of(end);
      CHECK(s.end == end && s.t1 > s.t0 && s.t1 <= units);
      const int64_t rows = int64_t(a.r[b].n) * a.H - s.row0;
      CHECK(s.rows == (rows < 128 ? rows : 128) && s.rows > 0);
      CHECK(s.starts == (u == 0) && s.ends == (s.t1 == units));
      for (int t = s.t0; t < s.t1 && t < s.t0 + 3; ++t) {
        const int64_t keys = end - int64_t(t) * 256;
        CHECK(groups(s.end, t) == (keys <= 0 ? 0 : keys >= 256 ? 4 : (keys + 63) / 64));
      }
      if (!(s.starts && s.ends)) ++(s.starts ? begun : taken_over);
      at += s.t1 - s.t0;
      u = s.t1;
      if (s.ends) u = 0, ++j, skip();
    }
    CHECK(at == st.from + st.count);
    CHECK(begun <= 1 && taken_over <= 1);
  }
  CHECK(at == total && b == a.B);
  ++cases;
}

int main() {
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
  const int heads[] = {1, 5, 16, 20, 64, 127, 128, 130, 1000, 1024};
  for (int H : heads)
    for (int i = 0; i < 200; ++i) {
      const int n = i % 5 == 0 ? pick(1, 4) : pick(1, 900);
      const int ctx = i % 4 == 0 ? pick(0, n) : i % 4 == 1 ? n : pick(0, 60000);
      closed_form(H, i % 3 != 0, {0, n, ctx});
    }
  // the largest: contexts of 2^27 (a pair of positions below and at it), 1024
  // heads, T H just below 2^31 - 128
  for (bool causal : {true, false}) {
    for (int ctx : {kMaxCtx, kMaxCtx - 1, 1 << 21, 0})
      for (int n : {1, 3, 2097151}) closed_form(1024, causal, {0, n, ctx});
    closed_form(1, causal, {0, 2147483647 - 128, kMaxCtx});
    closed_form(1000, causal, {0, 2147483, 2147483});
  }
  for (int pairs : {1, 2, 7, 76})
    for (int i = 0; i < 150; ++i) {
      Line a;
      a.H = heads[pick(0, 9)];
      a.causal = i % 3 != 0;
      a.B = pick(1, 12);
      for (int b = 0; b < a.B; ++b) {
        const int n = pick(0, 3) ? pick(0, 5) : pick(0, 300);
        a.r.push_back({0, n, pick(0, 4) ? pick(0, 9000) : pick(0, n)});
      }
      stretches(a, pairs);
    }
  stretches({{{0, 2000, kMaxCtx}, {0, 0, 5}, {0, 90000, kMaxCtx - 3}, {0, 7, 0}}, 4, 1024, true}, 76);
  stretches({{{0, 2097151, kMaxCtx}}, 1, 1024, true}, 76);
  stretches({{{0, 0, 5}, {0, 0, 0}}, 2, 16, true}, 76);
  printf("ok %lld\n", cases);
}
