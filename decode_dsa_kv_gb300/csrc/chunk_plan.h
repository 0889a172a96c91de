// How sfa_mla_chunk splits its work: the arithmetic of its row tiles, key tiles
// and stretches. Plain functions, shared by the kernel and (compiled by the host
// compiler alone) its tests.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PLAN_INLINE __host__ __device__ __forceinline__
#define PLAN_CALL static __host__ __device__ __noinline__
#else
#define PLAN_INLINE inline
#define PLAN_CALL inline
#endif

namespace dsakv {

constexpr int kRows = 128;         // query rows of a pair's tile
constexpr int kKeys = 256;         // keys of a tile
constexpr int kMaxCtx = 1 << 27;   // with H <= 1024, every count of the plan fits 32 bits

template <class T>
PLAN_INLINE T least(T a, T b) {
  return a < b ? a : b;
}
template <class T>
PLAN_INLINE T most(T a, T b) {
  return a > b ? a : b;
}

// One request, its values brought into range: first token, tokens, positions.
struct Request {
  int q0, n, ctx;
};

PLAN_INLINE int row_tiles(int H, const Request& r) {
  return (r.n * H + kRows - 1) / kRows;  // (T H < 2^31 - 128)
}
// Keys that the last row of row tile j attends to.
PLAN_INLINE int key_end(int H, bool causal, const Request& r, int j) {
  if (!causal) return r.ctx;
  // (T H < 2^31)
  const int last = least(r.n * H - 1, j * kRows + kRows - 1);
  return most(0, r.ctx - r.n + last / H + 1);
}
PLAN_INLINE int key_tiles(int end) { return most(1, (end + kKeys - 1) / kKeys); }
// x / y of whole numbers >= 0, in 32 bits where they fit (64-bit division is
// some 100 clocks of serial code).
PLAN_CALL int64_t divide(int64_t x, int y) {
  return (x >> 32) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}
// Sum of floor(i / G) over 0 <= i < N.
PLAN_INLINE int64_t quotients_below(int N, uint32_t G) {
  const uint32_t x = most(N, 0), k = x / G;
  return int64_t(G) * (int64_t(k) * (int64_t(k) - 1) / 2) + int64_t(k) * (x - k * G);
}
// Units (key tiles) of a request's first j row tiles, in closed form: row tile
// i before the last ends with token (128 i + 127) / H, so it has
//   1 + max(0, floor((ctx - n + (128 i + 127) / H) / 256))
//     = 1 + max(0, floor((i + c) / 2H)),  c = floor(((ctx - n) H + 127) / 128)
// key tiles (nested floors of quotients fold into one).
PLAN_CALL int64_t units_before(int H, bool causal, const Request r, int tiles, int j) {
  if (!causal) return int64_t(j) * key_tiles(r.ctx);
  int64_t s = 0;
  const int m = least(j, tiles - 1);
  if (m > 0) {
    const uint32_t G = 2 * H;
    const int c = static_cast<int>((int64_t(r.ctx - r.n) * H + kRows - 1) >> 7);
    s = m + quotients_below(m + c, G) - quotients_below(c, G);
  }
  if (j == tiles) s += key_tiles(key_end(H, causal, r, tiles - 1));
  return s;
}

// The units `from` .. `from + count` of the line of all units that a pair takes.
struct Stretch {
  int64_t from, count;
};
PLAN_INLINE Stretch stretch_of(int64_t total, int max_pairs, int pair) {
  const int pairs = static_cast<int>(least(int64_t(max_pairs), total));
  const int64_t share = pairs ? divide(total, pairs) : 0;
  const int more = static_cast<int>(total - share * pairs);  // pairs with one unit more
  return {share * pair + least(pair, more), pair < pairs ? share + (pair < more ? 1 : 0) : 0};
}

// Row tiles first .. last - 1 of the line of all row tiles that pair p takes when
// `pairs` pairs take them in turn, `rounds` each.
PLAN_INLINE int round_tiles(int pairs, int rounds, int p, int first, int last) {
  auto below = [&](int x) {  // those numbers i < x with i % pairs = p
    return least(rounds, (x - p + pairs - 1) / pairs);
  };
  return below(last) - below(first);
}

// The row tile and key tile of a request that its unit `at` is: the last row
// tile that begins at or before it.
struct Place {
  int j, u;
};
PLAN_INLINE Place place_of(int H, bool causal, const Request& r, int64_t at) {
  const int tiles = row_tiles(H, r);
  int lo = 0, hi = tiles - 1;
#ifdef __CUDACC__
#pragma unroll 1
#endif
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (units_before(H, causal, r, tiles, mid) <= at) lo = mid;
    else hi = mid - 1;
  }
  return {lo, static_cast<int>(at - units_before(H, causal, r, tiles, lo))};
}

// A row tile over a range of its key tiles.
struct Segment {
  int b, row0;     // request; first row of the tile within the request's n x H
  Request r;
  int rows;        // rows of the tile
  int t0, t1;      // key tiles
  int end;         // keys the tile's last row attends to
  bool starts, ends;
};
// Walks the segments of a stretch of `left` units that begins at key tile u of
// row tile j of request b; every role of both CTAs walks alike. `request(a, b)`
// gives a request of the arguments a.
struct Walk {
  int b, j, u;
  int64_t left;
  template <class Args>
  PLAN_INLINE bool next(const Args& a, Segment& s) {
    if (left <= 0) return false;
    int tiles;
    for (;; ++b, j = 0) {
      if (b >= a.B) return false;
      s.r = request(a, b);
      tiles = row_tiles(a.H, s.r);
      if (j < tiles) break;
    }
    s.b = b;
    s.row0 = j * kRows;
    s.rows = static_cast<int>(least(int64_t(kRows), int64_t(s.r.n) * a.H - s.row0));
    s.end = key_end(a.H, a.causal, s.r, j);
    const int units = key_tiles(s.end);
    s.t0 = u;
    s.t1 = static_cast<int>(least(int64_t(units), u + left));
    s.starts = u == 0;
    s.ends = s.t1 == units;
    left -= s.t1 - s.t0;
    if (s.ends) u = 0, ++j;
    else u = s.t1;
    return true;
  }
};

// What a pair takes behind rounds of whole row tiles, of which pair p has load[p]
// units: an equal share of everything less its load (which has to be below it).
PLAN_INLINE Stretch stretch_behind(int64_t total, int pairs, int pair, const int* load) {
  const Stretch st = stretch_of(total, pairs, pair);
  int64_t all = 0, before = 0;
#ifdef __CUDACC__
#pragma unroll 1
#endif
  for (int p = 0; p < pairs; ++p) {
    if (p < pair) before += load[p];
    all += load[p];
  }
  return {all + st.from - before, st.count - load[pair]};
}

// A pair's segments: of a tree, first `rounds` whole row tiles, every pairs-th
// from row tile j of request b on (not causal: all of a request's row tiles have
// all of its keys), then its stretch.
template <bool kTree>
struct Walker {
  Walk walk;
  int rounds, pairs, b, j;
  template <class Args>
  PLAN_INLINE bool next(const Args& a, Segment& s) {
    if (!kTree || rounds == 0) return walk.next(a, s);
    --rounds;
    for (;; ++b) {  // (there are that many row tiles)
      s.r = request(a, b);
      const int tiles = row_tiles(a.H, s.r);
      if (j < tiles) break;
      j -= tiles;
    }
    s.b = b;
    s.row0 = j * kRows;
    s.rows = static_cast<int>(least(int64_t(kRows), int64_t(s.r.n) * a.H - s.row0));
    s.end = s.r.ctx;
    s.t0 = 0;
    s.t1 = key_tiles(s.end);
    s.starts = s.ends = true;
    j += pairs;
    return true;
  }
};

// 64-key groups of key tile t that hold keys below `end`.
PLAN_INLINE int groups(int end, int t) {
  return least(4, most(0, (end - t * kKeys + 63) >> 6));
}

}  // namespace dsakv
