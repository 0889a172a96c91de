// ts_beam_select: the n best of a request's K x V continuations, and
// dsa_cache_fork: the sequences' block tables and last pages in their new order.
//
// Two kernels. beam_rows_kernel reads the logits, once: a CTA takes a piece of
// one beam's row into registers and leaves the piece's n best and its sum of
// exponentials. beam_merge_kernel, a CTA a request, joins the sums and takes
// the n best of the pieces' best. What bounds them is the one read of the
// logits and, with 16-bit ones, the instructions for each value.
//
// The n best of many values without sorting them: cut the values into groups,
// at least n of them; the n-th largest of the groups' maxima is a bound that at
// least n values reach and, unless the large values sit in few groups, not many
// more. Those few are listed in shared memory, and a value's place is the number
// of larger ones. Where more reach the bound than the list holds (rows of equal
// values, or sorted ones), the bound is raised by bisection until they fit.
//
// A sum of exponentials is s e^m. For a piece m is E log 2 with E whole, and
// exp(x - m) is taken as 2^(x log2(e) - E) with log2(e) in two floats: pieces then
// join exactly, by powers of two, and no rounding of a maximum, which the whole
// row would share, enters the result. (Where a piece's largest value is past
// 2^20 in size, rows of a type's lowest value, m is that value itself.)
#include <algorithm>
#include <climits>

#include "cache.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxN = 128;
constexpr int kList = 512;
constexpr float kLog2eHi = 1.44269502162933349609f, kLog2eLo = 1.92596299112661746887e-8f;

// A float's bits in the values' order; -0 is 0.
__device__ __forceinline__ uint32_t in_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_order(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
// The same of a double.
__device__ __forceinline__ uint64_t in_order64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ double from_order64(uint64_t k) {
  return __longlong_as_double(
      static_cast<long long>(k >> 63 ? k & ~(uint64_t(1) << 63) : ~k));
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A value of a row and its place: larger values first, then lower places. The
// place is kept inverted, so that keys compare as whole numbers; 0: nothing.
__device__ __forceinline__ uint64_t key_of(float x, int t) {
  return uint64_t(in_order(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(t));
}
constexpr uint32_t kNoValue = 0x007fffffu;  // in_order(-infinity): never a candidate

struct Piece {
  float s;    // sum of exp(x - m)
  int e;      // m = e log 2, or
  float top;  // (where e is kWide) this
  __device__ __forceinline__ double m() const;
};
constexpr int kWide = INT_MAX;
constexpr double kLn2 = 0.693147180559945309417;
__device__ __forceinline__ double Piece::m() const { return e == kWide ? double(top) : e * kLn2; }

template <class T>
struct Quad;  // 16 bytes of a row
template <>
struct Quad<float> {
  static constexpr int kValues = 4;
  static __device__ __forceinline__ void widen(const uint4& q, float* x) {
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
};
template <>
struct Quad<__nv_bfloat16> {
  static constexpr int kValues = 8;
  static __device__ __forceinline__ void widen(const uint4& q, float* x) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
};

// Threads whose maximum is a group's: as many groups as a power of two from 4 n
// on, if there are threads for it.
__host__ __device__ inline int group_threads(int n) {
  return n <= 8 ? 8 : n <= 16 ? 4 : n <= 32 ? 2 : 1;
}

// The n-th largest of the first `groups` words of `of` (all different, or equal
// ones in the order of their places), found by thread i < groups for word i.
__device__ __forceinline__ bool is_nth(const uint32_t* of, int groups, int i, int n) {
  const uint32_t v = of[i];
  int above = 0;
  for (int j = 0; j < groups; ++j) above += of[j] > v || (of[j] == v && j < i);
  return above == n - 1;
}

// kQuads 16-byte loads a thread.
template <class T, int kQuads>
__global__ void __launch_bounds__(kThreads)
    beam_rows_kernel(const T* __restrict__ logits, int64_t row_stride, int V, int n, int pieces,
                     uint64_t* __restrict__ best, Piece* __restrict__ sums, int32_t* err) {
  constexpr int kValues = Quad<T>::kValues, kEach = kQuads * kValues;
  __shared__ uint32_t maxima[kThreads];
  __shared__ uint64_t list[kList];
  __shared__ uint64_t bound;
  __shared__ int listed;
  __shared__ uint32_t warp_top[kWarps];
  __shared__ float warp_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces;
  const T* p = logits + row * row_stride;
  // the row from the 16-byte boundary at or below its first value on
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int t0 = (piece * kThreads * kQuads + tid) * kValues - shift;  // of this thread's first load
  constexpr int kStep = kThreads * kValues;                            // tokens between its loads
  float x[kEach];
  uint4 raw[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int t = t0 + i * kStep;
    if (t >= 0 && t + kValues <= V) raw[i] = __ldcs(reinterpret_cast<const uint4*>(p + t));
  }
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int t = t0 + i * kStep;
    if (t >= 0 && t + kValues <= V) {
      Quad<T>::widen(raw[i], x + i * kValues);
    } else {
#pragma unroll
      for (int c = 0; c < kValues; ++c)
        x[i * kValues + c] = t + c >= 0 && t + c < V ? Quad<T>::one(p + t + c) : -INFINITY;
    }
  }
  if (tid == 0) listed = 0;
  // NaN and +infinity count as -infinity. (A maximum passes NaNs over; they show
  // in the sum.)
  float mx = -INFINITY;
  auto take_out = [&]() {
    report(err, TS_DEVERR_NAN);
    mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (!(x[j] < INFINITY)) x[j] = -INFINITY;
      mx = fmaxf(mx, x[j]);
    }
  };
#pragma unroll
  for (int j = 0; j < kEach; ++j) mx = fmaxf(mx, x[j]);
  if (mx == INFINITY) take_out();
  // the groups' maxima
  const int per = group_threads(n), groups = kThreads / per;
  {
    uint32_t m = in_order(mx);
    for (int d = 1; d < per; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (tid % per == 0) maxima[tid / per] = m;
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) warp_top[warp] = m;
  }
  __syncthreads();
  if (tid < groups && is_nth(maxima, groups, tid, n)) bound = uint64_t(maxima[tid]) << 32;
  uint32_t most = warp_top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) most = max(most, warp_top[w]);
  const float top = from_order(most);
  const bool wide = fabsf(top) > 0x1p20f && top > -INFINITY;
  const float e = wide || top == -INFINITY ? 0.f : ceilf(top * kLog2eHi);
  auto sum = [&]() -> float {
    float s[4] = {};
    if (!wide) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        s[j & 3] += fast_exp2(fmaf(x[j], kLog2eLo, fmaf(x[j], kLog2eHi, -e)));
    } else {
      for (int j = 0; j < kEach; ++j) s[j & 3] += fast_exp2((x[j] - top) * kLog2eHi);
    }
    float all = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xffffffffu, all, d);
    return all;
  };
  float all = sum();
  if (!(all < INFINITY)) {  // (the whole warp)
    take_out();
    all = sum();
  }
  if (lane == 0) warp_sum[warp] = all;
  __syncthreads();
  launch_dependents();
  if (tid == 0) {
    float s = warp_sum[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += warp_sum[w];
    sums[blockIdx.x] = {top == -INFINITY ? 0.f : s, wide ? kWide : static_cast<int>(e), top};
  }
  auto add_above = [&](uint64_t least) {
    if (uint64_t(in_order(mx)) << 32 < (least & ~0xffffffffull)) return;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint64_t k = key_of(x[j], t0 + (j / kValues) * kStep + j % kValues);
      if (k >= least && (k >> 32) > kNoValue) {
        const int at = atomicAdd(&listed, 1);
        if (at < kList) list[at] = k;
      }
    }
  };
  uint64_t least = bound;
  add_above(least);
  __syncthreads();
  if (listed > kList) {
    // raised until at least n and at most kList keys (all different) reach it
    uint64_t lo = least, hi = ~0ull;  // n or more reach lo, none hi
    for (;;) {
      const uint64_t mid = lo + (hi - lo) / 2;
      int mine = 0;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const uint64_t k = key_of(x[j], t0 + (j / kValues) * kStep + j % kValues);
        mine += k >= mid && (k >> 32) > kNoValue;
      }
      __syncthreads();
      if (tid == 0) listed = 0;
      __syncthreads();
      mine = __reduce_add_sync(0xffffffffu, mine);
      if (lane == 0) atomicAdd(&listed, mine);
      __syncthreads();
      const int all = listed;
      if (all >= n) lo = mid;
      else hi = mid;
      if ((all >= n && all <= kList) || hi - lo <= 1) break;
    }
    __syncthreads();
    if (tid == 0) listed = 0;
    __syncthreads();
    add_above(lo);
    __syncthreads();
  }
  const int count = min(listed, kList);
  uint64_t* out = best + int64_t(blockIdx.x) * n;
  for (int i = tid; i < count; i += kThreads) {
    const uint64_t k = list[i];
    int above = 0;
    for (int j = 0; j < count; ++j) above += list[j] > k;
    if (above < n) out[above] = k;
  }
  for (int i = count + tid; i < n; i += kThreads) out[i] = 0;
}

// A candidate: its score, then its place (beam, token), lower first.
struct Candidate {
  uint64_t score;  // in_order64
  uint32_t place;  // inverted
  __device__ __forceinline__ bool above(const Candidate& o) const {
    return score > o.score || (score == o.score && place > o.place);
  }
};

// A beam: a continuation's score is (x - m) + rest.
struct Beam {
  double m, rest;
};

__global__ void __launch_bounds__(kThreads)
    beam_merge_kernel(const uint64_t* best, const Piece* sums, const float* cum, int K, int V,
                      int n, int pieces, Beam* beams, int32_t* tokens, int32_t* parents,
                      float* scores, int32_t* err) {
  __shared__ uint64_t score[kList];
  __shared__ uint32_t place[kList];
  __shared__ float maxima[kThreads];
  __shared__ float bound;
  __shared__ int listed;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  wait_previous_kernel();
  if (tid == 0) {
    listed = 0;
    bound = -INFINITY;
  }
  // every beam's sum of exponentials; a warp a beam
  beams += int64_t(b) * K;
  for (int k = warp; k < K; k += kWarps) {
    const Piece* of = sums + (int64_t(b) * K + k) * pieces;
    double m = -INFINITY;
    int e = INT_MIN;  // of the pieces that are not wide
    for (int i = lane; i < pieces; i += 32) {
      const Piece p = of[i];
      if (p.s > 0.f) m = fmax(m, p.m());
      if (p.s > 0.f && p.e != kWide) e = max(e, p.e);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, d));
    e = __reduce_max_sync(0xffffffffu, e);
    const bool whole = e != INT_MIN && m == e * kLn2;  // m is a power of two's
    double s = 0;
    for (int i = lane; i < pieces; i += 32) {
      const Piece p = of[i];
      if (!(p.s > 0.f)) continue;
      if (whole && p.e != kWide) s += double(ldexpf(p.s, max(p.e - e, -200)));
      else s += p.s * exp(p.m() - m);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) {
      float c = cum[int64_t(b) * K + k];
      if (!(c < INFINITY)) {
        report(err, TS_DEVERR_NAN);
        c = -INFINITY;
      }
      beams[k] = {m, s > 0 && c > -INFINITY ? double(c) - log(s) : -INFINITY};
    }
  }
  __syncthreads();
  // Warps take beams, or (few beams) equal slices of them; candidates lie in
  // order of (beam, piece, place there).
  const int slices = K < kWarps ? kWarps / K : 1;
  const int each = pieces * n, slice = (each + slices - 1) / slices;
  best += int64_t(b) * K * each;
  auto walk = [&](auto&& f) {
    for (int u = warp; u < K * slices; u += kWarps) {
      const int k = u / slices, from = (u - k * slices) * slice, to = min(each, from + slice);
      const Beam beam = beams[k];
      if (beam.rest == -INFINITY) continue;
      for (int i = from + lane; i < to; i += 32) {
        const uint64_t key = best[int64_t(k) * each + i];
        if (key) f(k, beam, key);
      }
    }
  };
  auto candidate = [&](int k, const Beam& beam, uint64_t key) -> Candidate {
    const double x = from_order(static_cast<uint32_t>(key >> 32));
    const uint32_t t = 0xffffffffu - static_cast<uint32_t>(key);
    return {in_order64((x - beam.m) + beam.rest),
            0xffffffffu - (static_cast<uint32_t>(k) * V + t)};
  };
  // In fp32 first (fp64 takes 16 clocks an instruction): a score lies within
  // `off` of y, so n scores reach the n-th largest of the groups' maxima of y -
  // off, and those n best of all are among the ones whose y + off does.
  auto about = [](const Beam& beam, uint64_t key, float* off) -> float {
    const float x = from_order(static_cast<uint32_t>(key >> 32)), m = static_cast<float>(beam.m),
                rest = static_cast<float>(beam.rest);
    // (five roundings, each of a sum of some of these or of one of them)
    *off = 0x1p-21f * (fabsf(x) + fabsf(m) + fabsf(rest));
    return (x - m) + rest;
  };
  float mine = -INFINITY;
  walk([&](int, const Beam& beam, uint64_t key) {
    float off;
    const float y = about(beam, key, &off);
    mine = fmaxf(mine, y - off);
  });
  const int per = group_threads(n), groups = kThreads / per;
  for (int d = 1; d < per; d <<= 1)
    mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, d));
  if (tid % per == 0) maxima[tid / per] = mine;
  __syncthreads();
  if (tid < groups) {
    const float v = maxima[tid];
    int above = 0;
    for (int j = 0; j < groups; ++j) above += maxima[j] > v || (maxima[j] == v && j < tid);
    if (above == n - 1) bound = v;
  }
  __syncthreads();
  const float least_about = bound;
  auto put = [&](const Candidate& c) {
    const int at = atomicAdd(&listed, 1);
    if (at < kList) {
      score[at] = c.score;
      place[at] = c.place;
    }
  };
  walk([&](int k, const Beam& beam, uint64_t key) {
    float off;
    const float y = about(beam, key, &off);
    if (!(y + off < least_about)) put(candidate(k, beam, key));
  });
  __syncthreads();
  if (listed > kList) {
    // the list's bound raised by bisection, first the score, then the place
    auto reach = [&](const Candidate& l) -> int {
      int m = 0;
      walk([&](int k, const Beam& beam, uint64_t key) { m += !l.above(candidate(k, beam, key)); });
      __syncthreads();
      if (tid == 0) listed = 0;
      __syncthreads();
      m = __reduce_add_sync(0xffffffffu, m);
      if (lane == 0) atomicAdd(&listed, m);
      __syncthreads();
      return listed;
    };
    // n or more reach (lo, from), fewer than n (hi, 0) or (lo, to)
    uint64_t lo = 0, hi = ~0ull;
    int got = kList + 1;
    while (got > kList && hi - lo > 1) {
      const uint64_t mid = lo + (hi - lo) / 2;
      const int r = reach({mid, 0});
      if (r >= n) lo = mid, got = r;
      else hi = mid;
    }
    uint32_t from = 0, to = 0xffffffffu;
    while (got > kList && to - from > 1) {
      const uint32_t mid = from + (to - from) / 2;
      const int r = reach({lo, mid});
      if (r >= n) from = mid, got = r;
      else to = mid;
    }
    __syncthreads();
    if (tid == 0) listed = 0;
    __syncthreads();
    const Candidate least = {lo, from};
    walk([&](int k, const Beam& beam, uint64_t key) {
      const Candidate c = candidate(k, beam, key);
      if (!least.above(c)) put(c);
    });
    __syncthreads();
  }
  const int count = min(listed, kList);
  const int64_t out = int64_t(b) * n;
  for (int i = tid; i < count; i += kThreads) {
    const Candidate c = {score[i], place[i]};
    int above = 0;
    for (int j = 0; j < count; ++j) above += Candidate{score[j], place[j]}.above(c);
    if (above >= n) continue;
    const uint32_t at = 0xffffffffu - c.place;
    tokens[out + above] = static_cast<int>(at % V);
    parents[out + above] = static_cast<int>(at / V);
    scores[out + above] = static_cast<float>(from_order64(c.score));
  }
  for (int i = count + tid; i < n; i += kThreads) {
    tokens[out + i] = parents[out + i] = -1;
    scores[out + i] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// A page's rows lie side by side, so a partial last page is one copy of whole
// 16-byte pieces. A CTA takes 16 KB of a sequence's; the first writes its table
// row too.
constexpr int kCopyPieces = 4;  // 16 bytes each, a thread's
constexpr int kCopyBytes = kThreads * kCopyPieces * 16;

struct Fork {
  uint8_t* cache;
  int64_t pages;
  int row_bytes, shift, max_ctx, parts;
  const int32_t* table;
  int64_t stride;
  const int32_t *ctx_len, *parents, *spare;
  int K, n;
  int32_t *new_table, *new_len, *err;
};

__global__ void __launch_bounds__(kThreads) cache_fork_kernel(const __grid_constant__ Fork a) {
  wait_previous_kernel();
  const int64_t i = blockIdx.x / a.parts;  // the new sequence
  const int part = blockIdx.x % a.parts, tid = threadIdx.x;
  const bool reports = part == 0 && tid == 0;
  int p = a.parents[i];
  if (p < -1 || p >= a.K) {
    if (reports) report(a.err, TS_DEVERR_PARENT);
    p = -1;
  }
  int ctx = 0;
  const int32_t* old = nullptr;
  if (p >= 0) {
    const int64_t from = i / a.n * a.K + p;
    old = a.table + from * a.stride;
    ctx = a.ctx_len[from];
    if (ctx < 0 || ctx > a.max_ctx) {
      if (reports) report(a.err, TS_DEVERR_CTX);
      ctx = min(max(ctx, 0), a.max_ctx);
    }
  }
  const int last = ctx >> a.shift, rows = ctx & ((1 << a.shift) - 1);
  if (part == 0 && a.new_table) {
    int32_t* row = a.new_table + i * a.stride;
    for (int64_t j = tid; j < a.stride; j += kThreads)
      row[j] = j < last ? old[j] : j == last && p >= 0 ? a.spare[i] : -1;
    if (tid == 0) a.new_len[i] = ctx;
  }
  if (rows == 0) return;  // (and a sequence that is none)
  const int64_t src = old[last], dst = a.spare[i];
  if (src < 0 || src >= a.pages || dst < 0 || dst >= a.pages) {
    if (reports) report(a.err, TS_DEVERR_SLOT_RANGE);
    return;
  }
  if (src == dst) return;
  const int64_t page_bytes = int64_t(a.row_bytes) << a.shift;
  const int whole = rows * a.row_bytes / 16, first = part * kThreads * kCopyPieces + tid;
  const uint4* s = reinterpret_cast<const uint4*>(a.cache + src * page_bytes);
  uint4* d = reinterpret_cast<uint4*>(a.cache + dst * page_bytes);
  uint4 v[kCopyPieces];
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k)
    if (first + k * kThreads < whole) v[k] = s[first + k * kThreads];
#pragma unroll
  for (int k = 0; k < kCopyPieces; ++k)
    if (first + k * kThreads < whole) d[first + k * kThreads] = v[k];
}

__host__ inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// How a row is cut: pieces of kThreads x quads x 16 bytes.
struct Cut {
  int quads, pieces;
};
Cut cut_of(int64_t rows, int V, int size) {
  const int values = 16 / size;
  auto pieces = [&](int quads) -> int {
    const int64_t each = int64_t(kThreads) * quads * values;
    return static_cast<int>((V + values - 1 + each - 1) / each);
  };
  // 128 bytes a thread, or 64 of 16-bit values (32 values either way); where
  // that leaves SMs without a piece, a quarter
  const int most = size == 4 ? 8 : 4;
  const int quads = rows * pieces(most) < sm_count() ? most / 4 : most;
  return {quads, pieces(quads)};
}

bool beam_sizes_ok(int B, int K, int V, int n) {
  return n <= kMaxN && int64_t(K) * V < INT_MAX && int64_t(B) * K < (1 << 24);
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" size_t ts_beam_workspace_size(int B, int K, int V, int n) {
  if (B <= 0 || K <= 0 || V <= 0 || n <= 0 || !beam_sizes_ok(B, K, V, n)) return 0;
  const int64_t rows = int64_t(B) * K;
  // (either type's)
  size_t pieces = std::max(cut_of(rows, V, 4).pieces, cut_of(rows, V, 2).pieces);
  return align256(rows * sizeof(Beam)) + align256(rows * pieces * sizeof(Piece)) +
         rows * pieces * n * sizeof(uint64_t);
}

extern "C" ts_status ts_beam_select(const void* logits, int dtype, int64_t row_stride,
                                    const float* cum, int B, int K, int V, int n, int32_t* tokens,
                                    int32_t* parents, float* scores, void* ws, size_t ws_bytes,
                                    int32_t* err, cudaStream_t stream) {
  if (B < 0 || K <= 0 || V <= 0 || n <= 0 || (dtype != TS_FP32 && dtype != TS_BF16))
    return TS_ERR_INVALID_ARG;
  if (B == 0) return TS_OK;
  const int size = dtype == TS_FP32 ? 4 : 2;
  if (!logits || !cum || !tokens || !parents || !scores || !ws || row_stride < V ||
      reinterpret_cast<uintptr_t>(logits) % size != 0)
    return TS_ERR_INVALID_ARG;
  if (!beam_sizes_ok(B, K, V, n)) return TS_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
      ws_bytes < ts_beam_workspace_size(B, K, V, n))
    return TS_ERR_WORKSPACE;
  const int64_t rows = int64_t(B) * K;
  const Cut cut = cut_of(rows, V, size);
  if (rows * cut.pieces > INT_MAX || int64_t(K) * cut.pieces * n > INT_MAX)
    return TS_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  Beam* beams = reinterpret_cast<Beam*>(w);
  w += align256(rows * sizeof(Beam));
  Piece* sums = reinterpret_cast<Piece*>(w);
  w += align256(rows * cut.pieces * sizeof(Piece));
  uint64_t* best = reinterpret_cast<uint64_t*>(w);
  auto launch = [&](auto kernel, auto* x) {
    kernel<<<static_cast<unsigned>(rows * cut.pieces), kThreads, 0, stream>>>(
        x, row_stride, V, n, cut.pieces, best, sums, err);
  };
  if (dtype == TS_FP32) {
    const auto* x = static_cast<const float*>(logits);
    if (cut.quads == 8) launch(beam_rows_kernel<float, 8>, x);
    else launch(beam_rows_kernel<float, 2>, x);
  } else {
    const auto* x = static_cast<const __nv_bfloat16*>(logits);
    if (cut.quads == 4) launch(beam_rows_kernel<__nv_bfloat16, 4>, x);
    else launch(beam_rows_kernel<__nv_bfloat16, 1>, x);
  }
  const ts_status st = launch_status();
  if (st != TS_OK) return st;
  return launch_after(beam_merge_kernel, unsigned(B), kThreads, stream, best, sums, cum, K, V, n,
                      cut.pieces, beams, tokens, parents, scores, err);
}

extern "C" ts_status dsa_cache_fork(void* cache, int64_t num_slots, int fmt,
                                    const int32_t* block_table, int64_t table_stride,
                                    int page_size, const int32_t* ctx_len, const int32_t* parents,
                                    const int32_t* spare, int B, int K, int n, int32_t* new_table,
                                    int32_t* new_len, int32_t* err, cudaStream_t stream) {
  ts_status st = cache_check(cache, num_slots, fmt);
  if (st == TS_OK) st = paging_check(block_table, table_stride, page_size, num_slots);
  if (st != TS_OK) return st;
  if (B < 0 || K <= 0 || n <= 0 || (new_table == nullptr) != (new_len == nullptr))
    return TS_ERR_INVALID_ARG;
  if (B == 0) return TS_OK;
  if (!ctx_len || !parents || !spare) return TS_ERR_INVALID_ARG;
  Fork a = {};
  a.cache = static_cast<uint8_t*>(cache);
  a.pages = num_slots / page_size;
  a.row_bytes = cache_row_bytes(fmt);
  a.shift = __builtin_ctz(page_size);
  a.max_ctx = static_cast<int>(std::min(table_stride, int64_t(INT_MAX) / page_size) * page_size);
  a.parts = ((page_size - 1) * a.row_bytes + kCopyBytes - 1) / kCopyBytes;
  a.table = block_table;
  a.stride = table_stride;
  a.ctx_len = ctx_len;
  a.parents = parents;
  a.spare = spare;
  a.K = K;
  a.n = n;
  a.new_table = new_table;
  a.new_len = new_len;
  a.err = err;
  if (int64_t(B) * n * a.parts > INT_MAX || int64_t(B) * K > INT_MAX) return TS_ERR_UNSUPPORTED;
  return launch_after(cache_fork_kernel, static_cast<unsigned>(int64_t(B) * n * a.parts), kThreads,
                      stream, a);
}
