// ts_beam_select: the n best of a request's K x V continuations, and
// dsa_cache_fork: the sequences' block tables and last pages in their new order.
//
// Two kernels. beam_rows_kernel reads the logits: a CTA streams a piece of one
// beam's row and leaves the piece's n best and its sums of exponentials.
// beam_merge_kernel, a CTA a request, joins the sums and takes the n best of the
// pieces' best.
//
// The n best of many values without sorting them: cut the values into groups,
// at least n of them; the n-th largest of the groups' maxima is a bound that at
// least n values reach and, unless the large values sit in few groups, not many
// more. While a row streams by, a thread keeps only the maximum of each 64 bytes
// it reads; with the bound it reads again the few that reach it. The values
// above the bound are listed in shared memory, and a value's place is the number
// of larger ones. Where more reach the bound than the list holds (rows of equal
// values, or sorted ones), the bound is raised by bisection until they fit, at a
// second reading of the piece a step: 64 x 8 beams over 131,072 bf16 logits of one
// value 2.8 ms, of a type's lowest value but for five 6.2 ms, rising by 1e-3 1.4 ms,
// where normal ones, a mask of the lowest value in nine of ten places or of
// -infinity, and logits in whole quarters all take 37 us.
//
// A sum of exponentials is s e^m. For a warp m is E log 2 with E whole, and
// exp(x - m) is taken as 2^(x log2(e) - E) with log2(e) in two floats: sums then
// join exactly, by powers of two, and no rounding of a maximum, which the whole
// row would share, enters the result. (Where a warp's largest value is past 2^20
// in size, rows of a type's lowest value, m is that value itself.)
//
// What a log-sum may be off by: the exponential's 2^-22; its argument's two roundings,
// below 2^-19.5 for a value within 32 powers of two of the reference (smaller ones add
// up to less than V 2^-32); 64 additions of a thread's and 7 of the threads', 2^-24
// each: below 2^-17 in all, and 2^-20 where one token has nearly everything. The
// roundings go both ways: 5e-8 root mean square over rows of normal logits.
//
// Measured: 64 x 8 beams over 131,072 bf16 logits (134 MB) 35 us, 0.57 of the
// measured copy rate: the stream alone is 25, a piece's end (reductions, bound,
// the hits' second reading, places) some 3 us of which other pieces hide a part,
// the merge 4 behind it. 16 x 10 over 50,257 fp32 (32 MB) 16.1 us; 1 x 4 over
// 32,000 8 us, its two launches and their chains.
#include <algorithm>
#include <climits>

#include "cache.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxN = 64;
constexpr int kMaxRounds = 8;
constexpr int kStages = 3;  // rounds of a piece on their way or in use
constexpr int kList = 512;
// Powers of two that a value may lie above its warp's reference (beyond, it becomes
// the reference): the argument of its exponential is then off by 2^-21 of a power.
// With 64 a row's one large token left its log off by up to 2e-6, with 8 by 6e-7, at
// equal times (a row's values seldom pass the first round's largest by 5.5).
constexpr float kLag = 8.f;
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

struct Piece {
  float s;    // sum of exp(x - m), in [1, 2) unless m is a value (or s is 0)
  int e;      // m = e log 2, or
  float top;  // (where e is kWide) this
  __device__ __forceinline__ double m() const;
};
constexpr int kWide = INT_MAX;
constexpr double kLn2 = 0.693147180559945309417;
__device__ __forceinline__ double Piece::m() const { return e == kWide ? double(top) : e * kLn2; }

// Packed pairs of fp32 values.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
  return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}

// Word i of four that hold 16 bytes of a row.
__device__ __forceinline__ uint32_t& word(uint4& q, int i) {
  return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
}
__device__ __forceinline__ uint32_t word(const uint4& q, int i) {
  return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
}

// 16 bytes of a row, kept as they came; a round of them.
constexpr int kQuads = 4;
template <class T>
struct Quad;
template <>
struct Quad<float> {
  static constexpr int kValues = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // a word of -infinity
  static __device__ __forceinline__ float value(const uint4& q, int c) {
    return __uint_as_float(word(q, c));
  }
  static __device__ __forceinline__ void set(uint4& q, int c, float x) {
    word(q, c) = __float_as_uint(x);
  }
  static __device__ __forceinline__ float load(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ float top(const uint4 (&x)[kQuads]) {
    float m[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
      m[i] = fmaxf(fmaxf(value(x[i], 0), value(x[i], 1)), fmaxf(value(x[i], 2), value(x[i], 3)));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  }
};
template <>
struct Quad<__nv_bfloat16> {
  static constexpr int kValues = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ float value(const uint4& q, int c) {
    const uint32_t w = word(q, c >> 1);
    return __uint_as_float(c & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ void set(uint4& q, int c, float x) {
    uint32_t& w = word(q, c >> 1);
    const uint32_t b = __float_as_uint(x);
    w = c & 1 ? (w & 0xffffu) | (b & 0xffff0000u) : (w & 0xffff0000u) | b >> 16;
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) {
    return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
  static __device__ __forceinline__ float top(const uint4 (&x)[kQuads]) {
    auto as2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
      m[i] = __hmax2(__hmax2(as2(x[i].x), as2(x[i].y)), __hmax2(as2(x[i].z), as2(x[i].w)));
    const __nv_bfloat162 all = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(__low2float(all), __high2float(all));
  }
};

// Threads of a CTA's whose maximum is a group's: as many groups as a power of two
// from 4 n on, or as there are threads (n above 32: from 2 n on).
__device__ __forceinline__ int group_threads(int threads, int n) {
  return max(1, threads / (n <= 8 ? 32 : n <= 16 ? 64 : n <= 32 ? 128 : 256));
}

// The n-th largest of the first `groups` words of `of` (all different, or equal
// ones in the order of their places), found by thread i < groups for word i.
// (a power of two from 32 on; 16-byte aligned)
__device__ __forceinline__ bool is_nth(const uint32_t* of, int groups, int i, int n) {
  const uint32_t v = of[i];
  int above = 0;
#pragma unroll 2
  for (int j = 0; j < groups; j += 4) {
    const uint4 o = *reinterpret_cast<const uint4*>(of + j);
    above += (o.x > v || (o.x == v && j < i)) + (o.y > v || (o.y == v && j + 1 < i)) +
             (o.z > v || (o.z == v && j + 2 < i)) + (o.w > v || (o.w == v && j + 3 < i));
  }
  return above == n - 1;
}

// A piece is `rounds` rounds of kQuads 16-byte loads a thread. They go through
// shared memory, each thread's through places of its own, so that the next two
// rounds are on their way without a register (in registers, one round ahead, the
// compiler spilled: 64 x 8 over 131,072 took 64 us where this took 50). 8 rounds at
// most: 30.9 us for the kernel, 34.7 with 4 and 35.2 with 16.
template <class T>
__global__ void __launch_bounds__(kThreads, 7)
    beam_rows_kernel(const T* __restrict__ logits, int64_t row_stride, int V, int n, int pieces,
                     int rounds, uint64_t* __restrict__ best, Piece* __restrict__ sums,
                     int32_t* err) {
  using Q = Quad<T>;
  constexpr int kValues = Q::kValues;
  constexpr int kStep = kThreads * kValues;   // tokens between a thread's loads
  constexpr int kRound = kStep * kQuads;      // tokens of a round
  __shared__ __align__(16) uint32_t maxima[kThreads];
  __shared__ uint32_t bound, most;
  __shared__ int listed, hit;
  extern __shared__ __align__(16) uint4 ring[];  // [kStages][kQuads][kThreads]
  float* round_top = reinterpret_cast<float*>(ring + kStages * kQuads * kThreads);  // [rounds][kThreads]
  // once the rounds are through: the values above the bound, and where they are
  uint64_t* list = reinterpret_cast<uint64_t*>(ring);
  uint32_t* hits = reinterpret_cast<uint32_t*>(list + kList);
  static_assert(kList * 8 + kMaxRounds * kThreads * 4 <= kStages * kQuads * kThreads * 16, "lists");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / pieces;
  const int piece = blockIdx.x - static_cast<int>(row) * pieces;
  const T* p = logits + row * row_stride;
  // the row from the 16-byte boundary at or below its first value on
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
  const int from = piece * rounds * kRound - shift;  // the piece's first token
  const int t0 = from + tid * kValues;               // of this thread's first load
  // the row's ends: whole loads where they lie inside, else value by value
  auto load_end = [&](uint4& x, int t) {
    x = make_uint4(Q::kNone, Q::kNone, Q::kNone, Q::kNone);
    if (t >= 0 && t + kValues <= V) {
      x = __ldcs(reinterpret_cast<const uint4*>(p + t));
    } else if (t < V && t + kValues > 0) {
#pragma unroll
      for (int c = 0; c < kValues; ++c)
        if (t + c >= 0 && t + c < V) Q::set(x, c, Q::load(p + t + c));
    }
  };
  auto send = [&](int r) {
    if (r < rounds) {
      uint4* to = ring + (r % kStages) * (kQuads * kThreads) + tid;
      const int at = from + r * kRound, t = t0 + r * kRound;
      if (at >= 0 && at + kRound <= V) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           smem_addr(to + i * kThreads)),
                       "l"(p + (t + i * kStep))
                       : "memory");
      } else {
#pragma unroll 1
        for (int i = 0; i < kQuads; ++i) load_end(to[i * kThreads], t + i * kStep);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (tid == 0) {
    listed = hit = 0;
    most = 0;
  }

  // ---- the stream ----
  float mine = -INFINITY;  // this thread's maximum
  // the warp's reference: E, or (wide) its maximum, or nothing yet; a value past
  // `limit` needs another one
  float e = 0.f, ref = -INFINITY, limit = -INFINITY;
  bool wide = false;
  uint64_t sum[2] = {};
  auto add = [&](const uint4 (&x)[kQuads]) {
    if (wide) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
#pragma unroll
        for (int c = 0; c < kValues; ++c) s += fast_exp2((Q::value(x[i], c) - ref) * kLog2eHi);
      sum[0] = add2(sum[0], pair(s, 0.f));
      return;
    }
    const uint64_t hi = pair(kLog2eHi, kLog2eHi), lo = pair(kLog2eLo, kLog2eLo),
                   minus_e = pair(-e, -e);
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
#pragma unroll
      for (int c = 0; c < kValues; c += 2) {
        const uint64_t v = pair(Q::value(x[i], c), Q::value(x[i], c + 1));
        const float2 y = unpair(fma2(v, lo, fma2(v, hi, minus_e)));
        sum[c >> 1 & 1] = add2(sum[c >> 1 & 1], pair(fast_exp2(y.x), fast_exp2(y.y)));
      }
  };
  // NaN and +infinity count as -infinity. (A maximum passes NaNs over; they show
  // in the sums.)
  auto take_out = [&](uint4 (&x)[kQuads]) {
    report(err, TS_DEVERR_NAN);
#pragma unroll
    for (int i = 0; i < kQuads; ++i)
#pragma unroll
      for (int c = 0; c < kValues; ++c)
        if (!(Q::value(x[i], c) < INFINITY)) Q::set(x[i], c, -INFINITY);
  };
  auto round = [&](uint4 (&x)[kQuads], int r) {
    float top = Q::top(x);
    if (__any_sync(0xffffffffu, !(top <= limit))) {
      // (the first round, a much larger value, NaNs alone or an infinity)
      if (!(top < INFINITY)) {
        take_out(x);
        top = Q::top(x);
      }
      const float all = from_order(__reduce_max_sync(0xffffffffu, in_order(fmaxf(top, mine))));
      if (!(all <= limit)) {
        const bool was_wide = wide, none = limit == -INFINITY;
        const float was_e = e, was_ref = ref;
        wide = fabsf(all) > 0x1p20f;
        ref = all;
        e = wide ? 0.f : ceilf(all * kLog2eHi);
        limit = wide ? all : (e + kLag) * static_cast<float>(kLn2);
        float f = 0.f;
        if (!none && !was_wide && !wide) f = ldexpf(1.f, max(static_cast<int>(was_e - e), -200));
        else if (!none)
          f = static_cast<float>(exp((was_wide ? double(was_ref) : was_e * kLn2) -
                                     (wide ? double(ref) : e * kLn2)));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 y = unpair(sum[k]);
          sum[k] = pair(y.x * f, y.y * f);
        }
      }
    }
    const uint64_t before[2] = {sum[0], sum[1]};
    add(x);
    {
      const float2 y = unpair(add2(sum[0], sum[1]));
      if (__any_sync(0xffffffffu, !(y.x + y.y < INFINITY))) {
        take_out(x);
        sum[0] = before[0];
        sum[1] = before[1];
        add(x);
      }
    }
    round_top[r * kThreads + tid] = top;
    mine = fmaxf(mine, top);
  };
  {
#pragma unroll
    for (int r = 0; r < kStages - 1; ++r) send(r);
#pragma unroll 1
    for (int r = 0; r < rounds; ++r) {
      send(r + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      uint4 x[kQuads];
      const uint4* at = ring + (r % kStages) * (kQuads * kThreads) + tid;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) x[i] = at[i * kThreads];
      round(x, r);
    }
  }
  launch_dependents();
  {
    const float2 y = unpair(add2(sum[0], sum[1]));
    float s = y.x + y.y;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    // s is brought to [1, 2), its exponent goes to E (exact): E is that of the first
    // rounds' values, s up to 2^(kLag + 13)
    int whole = static_cast<int>(e);
    if (!wide && s >= 0x1p-126f) {
      const uint32_t bits = __float_as_uint(s);
      whole += static_cast<int>(bits >> 23) - 127;
      s = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    }
    if (lane == 0) sums[int64_t(blockIdx.x) * kWarps + warp] = {s, wide ? kWide : whole, ref};
  }

  // ---- the n best ----
  const int per = group_threads(kThreads, n), groups = kThreads / per;
  {
    uint32_t m = in_order(mine);
    for (int d = 1; d < per; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (tid % per == 0) maxima[tid / per] = m;
  }
  __syncthreads();
  if (tid < groups) {
    if (is_nth(maxima, groups, tid, n)) bound = maxima[tid];
    atomicMax(&most, maxima[tid]);
  }
  __syncthreads();
  auto put = [&](uint64_t k) {
    const int at = atomicAdd(&listed, 1);
    if (at < kList) list[at] = k;
  };
  const float least = from_order(bound);
  // the threads' rounds that reach it, then all of their loads at once
  if (mine >= least)
#pragma unroll 4
    for (int r = 0; r < rounds; ++r)
      if (round_top[r * kThreads + tid] >= least) hits[atomicAdd(&hit, 1)] = r * kThreads + tid;
  __syncthreads();
#pragma unroll 1
  for (int j = tid; j < hit * kQuads; j += kThreads) {
    const int at = hits[j / kQuads], r = at / kThreads, i = j % kQuads;
    const int t = from + r * kRound + i * kStep + (at % kThreads) * kValues;
    uint4 x;
    load_end(x, t);
#pragma unroll
    for (int c = 0; c < kValues; ++c) {
      const float v = Q::value(x, c);
      if (v >= least && v > -INFINITY && v < INFINITY) put(key_of(v, t + c));
    }
  }
  __syncthreads();
  if (listed > kList) {
    // raised until at least n and at most kList keys (all different) reach it
    auto keys = [&](auto&& f) {
#pragma unroll 1
      for (int t = max(from, 0) + tid; t < min(from + rounds * kRound, V); t += kThreads) {
        const float v = Q::load(p + t);
        if (v > -INFINITY && v < INFINITY) f(key_of(v, t));
      }
    };
    // n or more reach lo, none hi
    uint64_t lo = uint64_t(bound) << 32, hi = (uint64_t(most) << 32) + (uint64_t(1) << 32);
    for (;;) {
      const uint64_t mid = lo + (hi - lo) / 2;
      int reach = 0;
      keys([&](uint64_t k) { reach += k >= mid; });
      __syncthreads();
      if (tid == 0) listed = 0;
      __syncthreads();
      reach = __reduce_add_sync(0xffffffffu, reach);
      if (lane == 0) atomicAdd(&listed, reach);
      __syncthreads();
      reach = listed;
      if (reach >= n) lo = mid;
      else hi = mid;
      if ((reach >= n && reach <= kList) || hi - lo <= 1) break;
    }
    __syncthreads();
    if (tid == 0) listed = 0;
    __syncthreads();
    keys([&](uint64_t k) {
      if (k >= lo) put(k);
    });
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

// log s of s >= 2^-44, within 2^-29 (2^25 values tried): s = 2^k c (1 + r) with c a float of
// [1/sqrt 2, sqrt 2] and |r| below 2^-24, log c = 2 artanh(q), q = (c - 1) / (c +
// 1), of which only q itself needs two floats. (CUDA's own of a double takes 1.2
// us here, where fp64 is slow: a third of the kernel.)
__device__ __forceinline__ double log_of(double s) {
  int k = static_cast<int>(static_cast<uint64_t>(__double_as_longlong(s)) >> 52) - 1023;
  double f = __longlong_as_double((__double_as_longlong(s) & 0xfffffffffffffll) |
                                  0x3ff0000000000000ll);  // in [1, 2)
  if (f > 1.41421356) {
    f *= 0.5;
    ++k;
  }
  const float c = static_cast<float>(f), r = static_cast<float>(f - double(c)) / c;
  const float above = c - 1.f, below = c + 1.f;  // (the first is exact)
  const float low = c < 1.f ? c - (below - 1.f) : 1.f - (below - c);  // what the second lost
  const float q = above / below;
  const float rest = fmaf(-q, low, fmaf(-q, below, above)) / below;
  const float q2 = q * q;
  // 1/3 + q2 / 5 + .. (q2 < 0.0295: the next term is below 2^-37 of q)
  const float series =
      fmaf(q2, fmaf(q2, fmaf(q2, fmaf(q2, fmaf(q2, 1.f / 13, 1.f / 11), 1.f / 9), 1.f / 7), 0.2f),
           1.f / 3);
  const float small = fmaf(2.f, fmaf(q * q2, series, rest), r);
  return k * kLn2 + (2.0 * q + small);
}

// A beam: a continuation's score is (x - m) + rest.
struct Beam {
  double m, rest;
};

// One CTA a request. Its time is its chain: the pieces' sums and best, which are
// all on their way from the start, a logarithm for each beam, and the barriers
// between those, the bound, the list and the places.
constexpr int kMergeThreads = 256;
constexpr int kAhead = 4;  // candidates a thread holds in registers
// A row has at most 2^18 parts below 2 (2^30 values in pieces of 2^14, four warps a
// piece): their sum stays below 2^64, and what each loses adds up to less than 2^-26.
constexpr int kShift = 44;
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const uint64_t* best, const Piece* sums, const float* cum, int K, int V,
                      int n, int pieces, Beam* beams, int32_t* tokens, int32_t* parents,
                      float* scores, int32_t* err) {
  __shared__ uint64_t score[kList];
  __shared__ uint32_t place[kList];
  __shared__ __align__(16) uint32_t maxima[kMergeThreads];
  __shared__ uint32_t bound;
  __shared__ int listed;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  wait_previous_kernel();
  // candidates lie in the order of (beam, piece, place there)
  const uint32_t each = pieces * n, all = K * each;
  best += int64_t(b) * all;
  uint64_t ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const uint32_t i = tid + j * kMergeThreads;
    ahead[j] = i < all ? best[i] : 0;
  }
  if (tid == 0) listed = 0;
  // every beam's sum of exponentials, in whole multiples of 2^-kShift of 2^e, e the
  // largest of its parts' (each below 2): a warp a beam
  beams += int64_t(b) * K;
  for (int k = warp; k < K; k += kMergeThreads / 32) {
    const int parts = pieces * kWarps;
    const Piece* of = sums + (int64_t(b) * K + k) * parts;
    Piece first = {0.f, 0, 0.f};
    if (lane < parts) first = of[lane];
    const float c = cum[int64_t(b) * K + k];
    auto piece = [&](int i) { return i == lane ? first : of[i]; };
    int e = INT_MIN;  // of the pieces that are not wide
    uint32_t top = 0; // of those that are
    for (int i = lane; i < parts; i += 32) {
      const Piece p = piece(i);
      if (p.s > 0.f && p.e != kWide) e = max(e, p.e);
      if (p.s > 0.f && p.e == kWide) top = max(top, in_order(p.top));
    }
    e = __reduce_max_sync(0xffffffffu, e);
    top = __reduce_max_sync(0xffffffffu, top);
    const double whole_m = e != INT_MIN ? e * kLn2 : -INFINITY;
    const double wide_m = top ? double(from_order(top)) : -INFINITY;
    Beam beam = {fmax(whole_m, wide_m), 0};
    double s = 0;
    if (!(wide_m > whole_m - 200)) {  // (a wide part that far below adds nothing)
      uint64_t whole = 0;
      for (int i = lane; i < parts; i += 32) {
        const Piece p = piece(i);
        if (p.s > 0.f && p.e != kWide)
          whole += __float2ull_rn(ldexpf(p.s, max(p.e - e, -100) + kShift));
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, d);
      s = static_cast<double>(whole) * (1.0 / (uint64_t(1) << kShift));
    } else {
      for (int i = lane; i < parts; i += 32) {
        const Piece p = piece(i);
        if (p.s > 0.f) s += p.s * exp(p.m() - beam.m);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    if (lane == 0) {
      if (!(c < INFINITY)) report(err, TS_DEVERR_NAN);
      beam.rest = c < INFINITY && c > -INFINITY ? s : 0;
      beams[k] = beam;
    }
  }
  __syncthreads();
  for (int k = tid; k < K; k += kMergeThreads) {
    const double s = beams[k].rest;
    beams[k].rest = s > 0 ? double(cum[int64_t(b) * K + k]) - log_of(s) : -INFINITY;
  }
  __syncthreads();
  auto walk = [&](auto&& f) {
    auto one = [&](uint32_t i, uint64_t key) {
      const int k = i / each;
      const Beam beam = beams[k];
      if (key && beam.rest > -INFINITY) f(k, beam, key);
    };
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (ahead[j]) one(tid + j * kMergeThreads, ahead[j]);
    for (uint32_t i = tid + kAhead * kMergeThreads; i < all; i += kMergeThreads) one(i, best[i]);
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
  const int per = group_threads(kMergeThreads, n), groups = kMergeThreads / per;
  for (int d = 1; d < per; d <<= 1)
    mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, d));
  if (tid % per == 0) maxima[tid / per] = in_order(mine);
  __syncthreads();
  if (tid < groups && is_nth(maxima, groups, tid, n)) bound = maxima[tid];
  __syncthreads();
  const float least_about = from_order(bound);
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
  for (int i = tid; i < count; i += kMergeThreads) {
    const Candidate c = {score[i], place[i]};
    int above = 0;
    for (int j = 0; j < count; ++j) above += Candidate{score[j], place[j]}.above(c);
    if (above >= n) continue;
    const uint32_t at = 0xffffffffu - c.place;
    tokens[out + above] = static_cast<int>(at % V);
    parents[out + above] = static_cast<int>(at / V);
    scores[out + above] = static_cast<float>(from_order64(c.score));
  }
  for (int i = count + tid; i < n; i += kMergeThreads) {
    tokens[out + i] = parents[out + i] = -1;
    scores[out + i] = -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// A page's rows lie side by side, so a partial last page is one copy of whole
// 16-byte pieces. A CTA takes 8 KB of a sequence's; the first writes its table
// row too. Bound by its chain (parent, its length and page, rows) and its launch:
// 512 sequences with 44 rows of 656 bytes (30 MB moved) 8 us, 0.55 of the measured
// copy rate.
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
  if (rows == 0) {  // (and a sequence that is none)
    if (reports && p >= 0 && last < a.stride && (a.spare[i] < 0 || a.spare[i] >= a.pages))
      report(a.err, TS_DEVERR_SLOT_RANGE);
    return;
  }
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

// How a row is cut: as many pieces as fill the SMs' 7 CTAs once, of whole rounds
// and at most kMaxRounds of them.
struct Cut {
  int rounds, pieces;
};
Cut cut_of(int64_t rows, int V, int size, bool even) {
  const int values = 16 / size, each = kThreads * kQuads * values;
  const int units = (V + (even ? 0 : values - 1) + each - 1) / each;  // (odd: a row's shift)
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(units, sm_count() * 7 / rows));
  const int rounds = std::min<int>(kMaxRounds, (units + want - 1) / want);
  return {rounds, (units + rounds - 1) / rounds};
}

bool beam_sizes_ok(int B, int K, int V, int n) {
  return n <= kMaxN && V <= (1 << 30) && int64_t(K) * V < INT_MAX && int64_t(B) * K < (1 << 24);
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" size_t ts_beam_workspace_size(int B, int K, int V, int n) {
  if (B <= 0 || K <= 0 || V <= 0 || n <= 0 || !beam_sizes_ok(B, K, V, n)) return 0;
  const int64_t rows = int64_t(B) * K;
  // (either type's and alignment's)
  const size_t pieces = std::max(std::max(cut_of(rows, V, 4, false).pieces, cut_of(rows, V, 4, true).pieces),
                                 std::max(cut_of(rows, V, 2, false).pieces, cut_of(rows, V, 2, true).pieces));
  return align256(rows * sizeof(Beam)) + align256(rows * pieces * kWarps * sizeof(Piece)) +
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
  const bool even = aligned16(logits) && row_stride * size % 16 == 0;
  const Cut cut = cut_of(rows, V, size, even);
  if (rows * cut.pieces > INT_MAX || int64_t(K) * cut.pieces * std::max(n, kWarps) > INT_MAX)
    return TS_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  Beam* beams = reinterpret_cast<Beam*>(w);
  w += align256(rows * sizeof(Beam));
  Piece* sums = reinterpret_cast<Piece*>(w);
  w += align256(rows * cut.pieces * kWarps * sizeof(Piece));
  uint64_t* best = reinterpret_cast<uint64_t*>(w);
  const unsigned grid = static_cast<unsigned>(rows * cut.pieces);
  const int smem = kThreads * (kStages * kQuads * 16 + cut.rounds * 4);
  if (dtype == TS_FP32)
    beam_rows_kernel<<<grid, kThreads, smem, stream>>>(static_cast<const float*>(logits), row_stride,
                                                       V, n, cut.pieces, cut.rounds, best, sums, err);
  else
    beam_rows_kernel<<<grid, kThreads, smem, stream>>>(static_cast<const __nv_bfloat16*>(logits),
                                                       row_stride, V, n, cut.pieces, cut.rounds,
                                                       best, sums, err);
  const ts_status st = launch_status();
  if (st != TS_OK) return st;
  return launch_after(beam_merge_kernel, unsigned(B), kMergeThreads, stream, best, sums, cum, K, V, n,
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
