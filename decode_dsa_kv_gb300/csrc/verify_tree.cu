// ts_verify_tree: a drafted tree against the target's probabilities, by a walk
// from the root: draw a token from the node's row, go on to the child that has
// it.
//
// One cluster of up to 8 CTAs a request. A step reads one row of V
// probabilities; steps depend on one another, so what bounds the walk is a
// step's chain: the row's loads, all on their way at once and kept in registers
// (a warp takes up to 2048 tokens side by side), the warps' sums, sent to every
// CTA, a cluster barrier, the drawn token, found by the warp that holds it in
// what it already has, its child, sent to every CTA, a cluster barrier. Weights
// are whole multiples of 2^-60 (verify.cuh): the drawn token does not depend on
// the split.
//
// Measured: 32 trees over 131,072 tokens, at most 4 drafts accepted, 22 us from L2,
// some 4.3 a step, of which (clocks of a step with every request on its way) the
// loads take 2000 to 3000, the sums 2000, waiting for the slowest CTA 1300, the sums'
// scan 1200, the draw 1800, the child 400 and the second barrier 550. Two CTAs an
// SM of 256 threads, eight a request: as requests end, the others' rows are spread
// over more SMs (four of 512 threads: 34 us; 16 of 128: 24.5 where this took 26.8,
// but clusters above 8 are not portable). One greedy tree over 32,000: 6.2 us.
#include <algorithm>

#include "verify.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSub = 4;                 // quads (4 tokens) a lane has of a piece
constexpr int kPiece = 32 * 4 * kSub;   // 512 tokens
constexpr int kMaxHeld = 4;             // pieces of a warp at once
constexpr int kMaxCluster = 8;
constexpr int kMaxV = 1 << 20;

struct Args {
  const int32_t *tokens, *parent, *cu_q;
  int T;
  const float* target;
  int64_t stride;
  const float* u;
  int V, depth, cluster, rounds;  // rounds of cluster * kWarps * held pieces
  int parts, kept;                // places in shared memory for sums and for nodes
  int32_t *path, *next, *accepted, *err;
};

// One row of probabilities, seen from the 16-byte boundary at or below its
// first: quad g holds tokens 4 g - shift .. 4 g - shift + 3, whole quads are
// one load and nothing outside the row is read.
struct Row {
  const float* p;
  int shift, V;
  __device__ __forceinline__ float4 quad(int g, float none) const {
    const int t = 4 * g - shift;
    if (t >= 0 && t + 3 < V) return __ldg(reinterpret_cast<const float4*>(p + t));
    float4 v;
    v.x = t >= 0 && t < V ? __ldg(p + t) : none;
    v.y = t + 1 >= 0 && t + 1 < V ? __ldg(p + t + 1) : none;
    v.z = t + 2 >= 0 && t + 2 < V ? __ldg(p + t + 2) : none;
    v.w = t + 3 >= 0 && t + 3 < V ? __ldg(p + t + 3) : none;
    return v;
  }
  // kHeld pieces from `piece` on.
  template <int kHeld>
  __device__ __forceinline__ void load(float4 (&v)[kHeld][kSub], int piece, float none) const {
    const int lane = threadIdx.x & 31, t0 = piece * kPiece - shift;
    if (t0 >= 0 && t0 + kHeld * kPiece <= V) {  // (the whole warp)
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
#pragma unroll
        for (int i = 0; i < kSub; ++i)
          v[j][i] = __ldg(reinterpret_cast<const float4*>(p + t0) + (kSub * j + i) * 32 + lane);
      return;
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
#pragma unroll
      for (int i = 0; i < kSub; ++i)
        v[j][i] = quad((piece + j) * (kPiece / 4) + 32 * i + lane, none);
  }
};

// A lane's sums of the parts of up to 16 values (verify.cuh: below 2^22 each) and
// the largest bits among the values.
struct Lane {
  uint32_t h, l, m, top;
  __device__ __forceinline__ void add(float x, float y) {
    const Split s = split(pack2(x, y));
    constexpr uint32_t four = 0x40800000u;
    h += static_cast<uint32_t>(s.h) + static_cast<uint32_t>(s.h >> 32) - 2 * four;
    l += static_cast<uint32_t>(s.l) + static_cast<uint32_t>(s.l >> 32) - 2 * four;
    m += static_cast<uint32_t>(s.m) + static_cast<uint32_t>(s.m >> 32) - 2 * four;
    top = max(top, max(__float_as_uint(x), __float_as_uint(y)));
  }
  __device__ __forceinline__ void add(const float4& v) {
    add(v.x, v.y);
    add(v.z, v.w);
  }
  // The warp's sum, in every lane, unless a value is bad (2 or more, NaN or
  // negative) or the sum may be 16 (2^64) or more. (None of the three can pass 32
  // bits.)
  __device__ __forceinline__ bool warp(uint64_t* sum) const {
    const uint32_t H = __reduce_add_sync(0xffffffffu, h);
    *sum = (uint64_t(H) << 39) + (uint64_t(__reduce_add_sync(0xffffffffu, l)) << 17) +
           __reduce_add_sync(0xffffffffu, m);
    return H < (1u << 25) - (1u << 10) && !__any_sync(0xffffffffu, top >= 0x40000000u);
  }
};
// The sum of a warp's values; where need be value by value, bad ones left out.
template <int kQuads>
__device__ __forceinline__ uint64_t sum_of(const float4 (&v)[kQuads], int* bad) {
  Lane a = {};
#pragma unroll
  for (int i = 0; i < kQuads; ++i) a.add(v[i]);
  uint64_t s;
  if (a.warp(&s)) return s;
  s = 0;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    s = add_full(s, fixed(v[i].x, bad) + fixed(v[i].y, bad));
    s = add_full(s, fixed(v[i].z, bad) + fixed(v[i].w, bad));
  }
  return warp_sum(s);
}
// The sums of a warp's first pieces, together with those before them.
template <int kHeld>
__device__ __forceinline__ void sums_of(const float4 (&v)[kHeld][kSub], uint64_t (&upto)[kHeld],
                                        int* bad) {
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const uint64_t s = sum_of(v[j], bad);
    upto[j] = j ? add_full(upto[j - 1], s) : s;
  }
}

// Inclusive sums over the lanes, which stop at 2^64 - 1.
__device__ __forceinline__ uint64_t inclusive(uint64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = add_full(v, o);
  }
  return v;
}

// The token, counted from the warp's first, that `rest` falls on: the piece, its
// row of 128 tokens, then the lane, then its token.
template <int kHeld>
__device__ __forceinline__ int draw(const float4 (&v)[kHeld][kSub], const uint64_t (&upto)[kHeld],
                                    uint64_t rest) {
  const int lane = threadIdx.x & 31;
  int ignored = 0, j = 0, row = 0;
  float4 piece[kSub], x = {};
  uint64_t before = 0;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const bool is = k == 0 || rest >= upto[k - 1];  // (ascending: the last one that is)
    if (is && k) j = k, before = upto[k - 1];
#pragma unroll
    for (int i = 0; i < kSub; ++i)
      piece[i] = make_float4(is ? v[k][i].x : piece[i].x, is ? v[k][i].y : piece[i].y,
                             is ? v[k][i].z : piece[i].z, is ? v[k][i].w : piece[i].w);
  }
  rest -= before;
  before = 0;
  uint64_t all = 0;
#pragma unroll
  for (int i = 0; i < kSub; ++i) {
    const bool is = i == 0 || rest >= all;
    if (is) row = i, before = all;
    x = make_float4(is ? piece[i].x : x.x, is ? piece[i].y : x.y, is ? piece[i].z : x.z,
                    is ? piece[i].w : x.w);
    if (i < kSub - 1) {
      const float4 one[1] = {piece[i]};
      all += sum_of(one, &ignored);
    }
  }
  rest -= before;
  const uint64_t w[4] = {fixed(x.x, &ignored), fixed(x.y, &ignored), fixed(x.z, &ignored),
                         fixed(x.w, &ignored)};
  const uint64_t own = (w[0] + w[1]) + (w[2] + w[3]), inc = inclusive(own);
  uint64_t left = rest - (inc - own);
  int c = 0;
  if (left >= w[0]) {
    left -= w[0], c = 1;
    if (left >= w[1]) {
      left -= w[1], c = 2;
      if (left >= w[2]) c = 3;
    }
  }
  const int who = __ffs(__ballot_sync(0xffffffffu, rest < inc)) - 1;
  return __shfl_sync(0xffffffffu, j * kPiece + 128 * row + 4 * lane + c, who);
}

// A float's bits in the values' order (-0 is 0).
__device__ __forceinline__ uint32_t in_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
// Two warps' sums.
struct __align__(16) uint2x64 {
  uint64_t x, y;
};
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u;
  return uint64_t(hi) << 32 | __reduce_max_sync(0xffffffffu, lo);
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// kHeld pieces a warp and round, in registers.
template <int kHeld>
__global__ void __launch_bounds__(kThreads, 2) verify_tree_kernel(const __grid_constant__ Args a) {
  // all CTAs' warps' sums, round by round; greedy: their best
  extern __shared__ __align__(16) uint64_t parts[];
  // the first nodes' parents and tokens
  int2* const nodes = reinterpret_cast<int2*>(parts + a.parts);
  __shared__ uint32_t drawn, chosen;
  const int b = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warps = a.cluster * kWarps, me = rank * kWarps + warp;
  launch_dependents();
  // Another CTA's shared memory may be written only once that CTA has started: every
  // CTA arrives here, and waits for the others behind the first row's loads.
  cluster_arrive_relaxed();
  bool started = false;
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1);
  const int q0 = min(max(c0, 0), a.T), n = max(min(c1, a.T) - q0, 0);
  int32_t* path = a.path + int64_t(b) * (a.depth + 1);
  int32_t* next = a.next + int64_t(b) * (a.depth + 1);
  if (rank == 0 && tid == 0 && (c0 < 0 || c1 < c0 || c1 > a.T)) report(a.err, TS_DEVERR_ORDER);
  int bad = 0, nan = 0, node = 0, step = n ? 0 : -1;
  auto node_at = [&](int i) -> int2 {
    return make_int2(a.parent ? __ldg(a.parent + q0 + i) : i - 1, __ldg(a.tokens + q0 + i));
  };
  for (int i = tid; i < min(n, a.kept); i += kThreads) nodes[i] = node_at(i);
  // (read behind the first step's barrier)
  // the lowest child of x with token t, or -1: 32 nodes at a time
  auto child_of = [&](int x, int t) -> int {
    if (t < 0 || step >= a.depth) return -1;
#pragma unroll 1
    for (int i0 = x + 1; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      int2 is = make_int2(-1, -1);
      if (i < a.kept) is = nodes[min(i, n - 1)];
      else if (i < n) is = node_at(i);
      const uint32_t who = __ballot_sync(0xffffffffu, i < n && is.x == x && is.y == t);
      if (who) return i0 + __ffs(who) - 1;
    }
    return -1;
  };
  while (step >= 0) {  // (every branch on the walk's state is the same in all of the cluster)
    Row row;
    row.p = a.target + (int64_t(q0) + node) * a.stride;
    row.shift = (reinterpret_cast<uintptr_t>(row.p) & 15u) >> 2;
    row.V = a.V;
    float4 v[kHeld][kSub];
    // (greedy: two sets of parts, of even and odd steps; one barrier a step)
    uint64_t* part = parts + (a.u ? 0 : (step & 1) * warps);
    const float point = a.u ? __ldg(a.u + int64_t(b) * (a.depth + 1) + step) : 0.f;
    uint64_t best = 0, upto[kHeld];
#pragma unroll 1
    for (int r = 0; r < a.rounds; ++r) {
      const int first = (r * warps + me) * kHeld;
      row.load(v, first, a.u ? 0.f : -INFINITY);
      if (!started) {
        __syncwarp();
        cluster_wait();
        started = true;
      }
      if (a.u) {
        sums_of(v, upto, &bad);
        if (lane < a.cluster)
          st_dsmem_u64(dsmem_addr(parts + r * warps + me, lane), upto[kHeld - 1]);
      } else {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            const float4 x = v[j][i];
            nan |= (x.x != x.x) | (x.y != x.y) | (x.z != x.z) | (x.w != x.w);
            top = fmaxf(fmaxf(top, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
          }
        const uint32_t most = __reduce_max_sync(0xffffffffu, in_order(top));
        uint32_t at = 0;  // the lowest token of it, inverted
        if (in_order(top) == most) {
#pragma unroll
          for (int j = kHeld - 1; j >= 0; --j)
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
              const float x[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
              const int t = (first + j) * kPiece + 128 * i + 4 * lane - row.shift;
#pragma unroll
              for (int c = 3; c >= 0; --c)
                if (x[c] == top && t + c >= 0 && t + c < a.V) at = ~static_cast<uint32_t>(t + c);
            }
        }
        const uint64_t key = uint64_t(most) << 32 | __reduce_max_sync(0xffffffffu, at);
        // (a warp of NaNs, or past the row's end, has no token)
        if (static_cast<uint32_t>(key) && key > best) best = key;
      }
    }
    int found = -1, child = -1;
    if (!a.u) {
      if (lane < a.cluster) st_dsmem_u64(dsmem_addr(part + me, lane), best);
      __syncwarp();
      cluster_sync_all();
      best = 0;
      for (int i = lane; i < warps; i += 32) best = max(best, part[i]);
      best = warp_max(best);
      if (best) found = static_cast<int>(~static_cast<uint32_t>(best));
      child = child_of(node, found);
    } else {
      __syncwarp();
      cluster_sync_all();
      // (a round has 64 warps at most: two a lane)
      auto both = [&](int r) -> uint2x64 {
        if (2 * lane >= warps) return {0, 0};
        return *reinterpret_cast<const uint2x64*>(parts + r * warps + 2 * lane);
      };
      uint64_t own = 0;
      for (int r = 0; r < a.rounds; ++r) {
        const uint2x64 e = both(r);
        own = add_full(own, add_full(e.x, e.y));
      }
      uint64_t inc = inclusive(own);
      const uint64_t total = __shfl_sync(0xffffffffu, inc, 31);
      bool mine = false;
      if (total == 0 || total == kFull) {
        bad |= rank == 0 && tid == 0;
        mine = me == 0;
      } else {
        uint64_t rest = __umul64hi(fixed_u(point), total);
        for (int r = 0; r < a.rounds; ++r) {
          const uint2x64 e = both(r);
          if (a.rounds > 1) inc = inclusive(e.x + e.y);
          const uint32_t past = __ballot_sync(0xffffffffu, rest < inc);
          if (!past) {
            rest -= __shfl_sync(0xffffffffu, inc, 31);
            continue;
          }
          const int who = __ffs(past) - 1;
          rest -= __shfl_sync(0xffffffffu, inc - (e.x + e.y), who);
          const uint64_t x = __shfl_sync(0xffffffffu, e.x, who);
          const bool second = rest >= x;
          if (second) rest -= x;
          mine = 2 * who + second == me;
          if (mine) {
            const int first = (r * warps + me) * kHeld;
            if (r != a.rounds - 1) {
              int again;
              row.load(v, first, 0.f);
              sums_of(v, upto, &again);
            }
            found = first * kPiece + draw(v, upto, rest) - row.shift;
          }
          break;
        }
      }
      if (mine) {
        child = child_of(node, found);
        if (lane < a.cluster) {
          st_dsmem_u32(dsmem_addr(&drawn, lane), static_cast<uint32_t>(found));
          st_dsmem_u32(dsmem_addr(&chosen, lane), static_cast<uint32_t>(child));
        }
      }
      __syncwarp();
      cluster_sync_all();
      found = static_cast<int>(drawn);
      child = static_cast<int>(chosen);
    }
    if (rank == 0 && tid == 0) {
      path[step] = node;
      next[step] = found;
    }
    if (child < 0) break;
    node = child;
    ++step;
  }
  if (bad) report(a.err, TS_DEVERR_PROB);
  if (nan) report(a.err, TS_DEVERR_NAN);
  if (rank == 0) {
    if (tid == 0) a.accepted[b] = step;
    for (int i = step + 1 + tid; i <= a.depth; i += kThreads) path[i] = next[i] = -1;
  }
  // (greedy: the last step's parts may still be on their way to a CTA)
  __syncwarp();
  if (!started) cluster_wait();  // (a request without a node)
  cluster_sync_all();
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" ts_status ts_verify_tree(const int32_t* tokens, const int32_t* parent,
                                    const int32_t* cu_q, int T, int B, const float* target,
                                    int64_t target_stride, const float* u, int V, int depth,
                                    int32_t* path, int32_t* next, int32_t* accepted, int32_t* err,
                                    cudaStream_t stream) {
  if (B < 0 || T < 0 || V <= 0 || depth < 0) return TS_ERR_INVALID_ARG;
  if (B == 0) return TS_OK;
  if (!cu_q || !path || !next || !accepted || (T > 0 && (!tokens || !target)))
    return TS_ERR_INVALID_ARG;
  if (target_stride < V || (reinterpret_cast<uintptr_t>(target) & 3u) != 0)
    return TS_ERR_INVALID_ARG;
  if (V > kMaxV || depth > TS_MAX_TREE || int64_t(B) * kMaxCluster > 2147483647)
    return TS_ERR_UNSUPPORTED;
  const bool even = aligned16(target) && target_stride % 4 == 0;  // (else a row's shift)
  const int pieces = (V + (even ? 0 : 3) + kPiece - 1) / kPiece;
  // As many CTAs a request as the GPU holds at once for all of them, two an SM
  // (a second wave would wait for the first's whole walk), and no more than
  // have pieces; then as few pieces a warp as make one round of it.
  int cluster = 1, held = 1;
  while (cluster < kMaxCluster && cluster * kWarps < pieces &&
         int64_t(B) * cluster <= sm_count())
    cluster *= 2;
  while (held < kMaxHeld && cluster * kWarps * held < pieces) held *= 2;
  Args a = {};
  a.tokens = tokens;
  a.parent = parent;
  a.cu_q = cu_q;
  a.T = T;
  a.target = target;
  a.stride = target_stride;
  a.u = u;
  a.V = V;
  a.depth = depth;
  a.cluster = cluster;
  const int round_pieces = cluster * kWarps * held;
  a.rounds = (pieces + round_pieces - 1) / round_pieces;
  a.parts = cluster * kWarps * std::max(a.rounds, 2);  // (greedy: two sets)
  a.kept = std::min(T, TS_MAX_TREE);
  a.path = path;
  a.next = next;
  a.accepted = accepted;
  a.err = err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 8 * (a.parts + a.kept);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = held == 1   ? verify_tree_kernel<1>
                : held == 2 ? verify_tree_kernel<2>
                            : verify_tree_kernel<4>;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return TS_ERR_CUDA;
  }
  return launch_status();
}
