// ts_verify_tree: a drafted tree against the target's probabilities, by a walk
// from the root: draw a token from the node's row, go on to the child that has
// it.
//
// One cluster of up to 8 CTAs a request. A step reads one row of V
// probabilities; steps depend on one another, so what bounds the walk is a
// step's chain: loads, sums, cluster barrier, the drawn token found, cluster
// barrier. To keep it short a warp takes 1024 tokens side by side, in registers,
// so the warp that holds the drawn point finds the token in what it already has
// (where a CTA has one such round; else it reads those 4 KB again), looks for
// the child itself and sends both to every CTA. Weights are whole multiples of
// 2^-60 (verify.cuh): the drawn token does not depend on the split.
#include "verify.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kQuads = 8;                  // of 4 tokens, a lane's of a piece
constexpr int kPiece = 32 * 4 * kQuads;    // 1024 tokens, a warp's
constexpr int kMaxCluster = 8;
constexpr int kMaxPieces = 1040;           // of a CTA: 8 KB of sums
constexpr int kMaxV = 1 << 23;
static_assert(int64_t(kMaxPieces) * kMaxCluster * kPiece >= kMaxV + 3 &&
                  kMaxPieces % kWarps == 0, "pieces");

struct Args {
  const int32_t *tokens, *parent, *cu_q;
  int T;
  const float* target;
  int64_t stride;
  const float* u;
  int V, depth, cluster, rounds;  // a CTA's rounds of kWarps pieces
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
  __device__ __forceinline__ void load(float4 (&v)[kQuads], int piece, float none) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) v[i] = quad(piece * (kPiece / 4) + 32 * i + lane, none);
  }
};

// The sum of a warp's piece, in every lane; *top gathers the largest bits, and
// the sum is exact as long as they stay below those of 2.
__device__ __forceinline__ uint64_t piece_sum(const float4 (&v)[kQuads], uint32_t* top) {
  uint32_t h = 0, l = 0, m = 0;  // l, m: 32 values below 2^22
  uint32_t most = 0;
  auto add = [&](float x, float y) {
    const Split s = split(pack2(x, y));
    constexpr uint32_t four = 0x40800000u;
    h += static_cast<uint32_t>(s.h) + static_cast<uint32_t>(s.h >> 32) - 2 * four;
    l += static_cast<uint32_t>(s.l) + static_cast<uint32_t>(s.l >> 32) - 2 * four;
    m += static_cast<uint32_t>(s.m) + static_cast<uint32_t>(s.m >> 32) - 2 * four;
    most = max(most, max(__float_as_uint(x), __float_as_uint(y)));
  };
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    add(v[i].x, v[i].y);
    add(v[i].z, v[i].w);
  }
  // (a lane that adds up to 16 or more: the warp's h could pass 32 bits; l and m,
  // 1024 values below 2^22 each, cannot)
  if (h >= 1u << 25) most = ~0u;
  *top = max(*top, most);
  h = __reduce_add_sync(0xffffffffu, h);
  l = __reduce_add_sync(0xffffffffu, l);
  m = __reduce_add_sync(0xffffffffu, m);
  return (uint64_t(h) << 39) + (uint64_t(l) << 17) + m;
}
// The same value by value, the bad ones left out.
__device__ __forceinline__ uint64_t careful_sum(const float4 (&v)[kQuads], int* bad) {
  uint64_t s = 0;
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    s = add_full(s, fixed(v[i].x, bad) + fixed(v[i].y, bad));
    s = add_full(s, fixed(v[i].z, bad) + fixed(v[i].w, bad));
  }
  return warp_sum(s);
}

// A float's bits in the values' order (-0 is 0); NaN below all others.
__device__ __forceinline__ uint32_t in_order(float x, int* nan) {
  if (x != x) {
    *nan = 1;
    return 0;
  }
  const uint32_t b = __float_as_uint(x + 0.f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u;
  return uint64_t(hi) << 32 | __reduce_max_sync(0xffffffffu, lo);
}

__global__ void __launch_bounds__(kThreads, 1) verify_tree_kernel(const __grid_constant__ Args a) {
  __shared__ uint64_t part[kMaxPieces];
  __shared__ uint64_t cta_sum;
  __shared__ uint32_t drawn, chosen;
  const int b = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pieces = a.rounds * kWarps;
  launch_dependents();
  const int q0 = min(max(__ldg(a.cu_q + b), 0), a.T);
  const int n = max(min(__ldg(a.cu_q + b + 1), a.T) - q0, 0);
  int32_t* path = a.path + int64_t(b) * (a.depth + 1);
  int32_t* next = a.next + int64_t(b) * (a.depth + 1);
  if (rank == 0 && tid == 0 && (__ldg(a.cu_q + b) < 0 || __ldg(a.cu_q + b + 1) < __ldg(a.cu_q + b) ||
                                __ldg(a.cu_q + b + 1) > a.T))
    report(a.err, TS_DEVERR_ORDER);
  int bad = 0, nan = 0, node = 0, step = 0;
  if (n == 0) step = -1;  // (the same in every CTA of the cluster)
  for (; step >= 0;) {
    Row row;
    row.p = a.target + (int64_t(q0) + node) * a.stride;
    row.shift = (reinterpret_cast<uintptr_t>(row.p) & 15u) >> 2;
    row.V = a.V;
    const int piece0 = rank * pieces;
    float4 v[kQuads];
    uint32_t top = 0;
    uint64_t best = 0;
    for (int i = 0; i < a.rounds; ++i) {
      row.load(v, piece0 + i * kWarps + warp, a.u ? 0.f : -INFINITY);
      if (a.u) {
        const uint64_t s = piece_sum(v, &top);
        if (lane == 0) part[i * kWarps + warp] = s;
      } else {
        const int t0 = (piece0 + i * kWarps + warp) * kPiece + 4 * lane - row.shift;
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
          const float x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int t = t0 + 128 * k + c;
            if (t >= 0 && t < a.V) {
              const uint64_t key = uint64_t(in_order(x[c], &nan)) << 32 | (0xffffffffu - t);
              if (key > best) best = key;
            }
          }
        }
      }
    }
    int found = -1;  // the token, where this warp has it
    bool mine = false;
    if (a.u) {
      if (__syncthreads_or(top >= 0x40000000u)) {
        for (int i = 0; i < a.rounds; ++i) {
          row.load(v, piece0 + i * kWarps + warp, 0.f);
          const uint64_t s = careful_sum(v, &bad);
          if (lane == 0) part[i * kWarps + warp] = s;
        }
        __syncthreads();
      }
      if (warp == 0) {
        uint64_t s = 0;
        for (int i = lane; i < pieces; i += 32) s = add_full(s, part[i]);
        s = warp_sum(s);
        if (lane == 0) cta_sum = s;
      }
      __syncwarp();
      cluster_sync_all();
      uint64_t sum = lane < a.cluster ? ld_dsmem_u64(dsmem_addr(&cta_sum, lane)) : 0;
      const uint64_t total = warp_sum(sum);
      uint64_t before = 0;  // (used only where the total fits)
      for (int r = 0; r < rank; ++r) before += __shfl_sync(0xffffffffu, sum, r);
      sum = __shfl_sync(0xffffffffu, sum, rank);
      if (total == 0 || total == kFull) {
        bad |= rank == 0 && tid == 0;
        mine = rank == 0 && warp == 0;
      } else {
        const uint64_t r =
            __umul64hi(fixed_u(__ldg(a.u + int64_t(b) * (a.depth + 1) + step)), total);
        if (r >= before && r - before < sum) {
          uint64_t rest = r - before;
          // the piece: 32 at a time, every warp alike
          int piece = 0;
          for (int i0 = 0; i0 < pieces; i0 += 32) {
            uint64_t inc = i0 + lane < pieces ? part[i0 + lane] : 0;
            const uint64_t own = inc;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const uint64_t o = __shfl_up_sync(0xffffffffu, inc, d);
              if (lane >= d) inc += o;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, rest < inc);
            if (past) {
              const int i = __ffs(past) - 1;
              piece = i0 + i;
              rest -= __shfl_sync(0xffffffffu, inc - own, i);
              break;
            }
            rest -= __shfl_sync(0xffffffffu, inc, 31);
          }
          mine = piece % kWarps == warp;
          if (mine) {
            if (piece / kWarps != a.rounds - 1) row.load(v, piece0 + piece, 0.f);
            // the row of 128 tokens, then the lane, then its token
            uint64_t s[kQuads];
            int quad = -1;
            int ignored = 0;
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
              s[k] = fixed(v[k].x, &ignored) + fixed(v[k].y, &ignored) + fixed(v[k].z, &ignored) +
                     fixed(v[k].w, &ignored);
              const uint64_t all = warp_sum(s[k]);
              if (quad < 0) {
                if (rest < all) quad = k;
                else rest -= all;
              }
            }
            float4 x = v[0];
            uint64_t inc = s[0];
#pragma unroll
            for (int k = 1; k < kQuads; ++k)
              if (quad == k) x = v[k], inc = s[k];
            const uint64_t own = inc;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const uint64_t o = __shfl_up_sync(0xffffffffu, inc, d);
              if (lane >= d) inc += o;
            }
            const int who = __ffs(__ballot_sync(0xffffffffu, rest < inc)) - 1;
            uint64_t left = rest - (inc - own);
            const uint64_t w[3] = {fixed(x.x, &ignored), fixed(x.y, &ignored),
                                   fixed(x.z, &ignored)};
            int c = 0;
            if (left >= w[0]) {
              left -= w[0], c = 1;
              if (left >= w[1]) {
                left -= w[1], c = 2;
                if (left >= w[2]) c = 3;
              }
            }
            found = (piece0 + piece) * kPiece + 128 * quad + 4 * lane + c - row.shift;
            found = __shfl_sync(0xffffffffu, found, who);
          }
        }
      }
    } else {
      best = warp_max(best);
      if (lane == 0) part[warp] = best;
      __syncthreads();
      if (warp == 0) {
        best = warp_max(lane < kWarps ? part[lane] : 0);
        if (lane == 0) cta_sum = best;
      }
      __syncwarp();
      cluster_sync_all();
      best = warp_max(lane < a.cluster ? ld_dsmem_u64(dsmem_addr(&cta_sum, lane)) : 0);
      mine = rank == 0 && warp == 0;
      if (best >> 32) found = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
    }
    if (mine) {
      // the child: 32 nodes at a time
      int child = -1;
      const bool on = found >= 0 && step < a.depth;
      for (int i0 = node + 1; on && child < 0 && i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const bool is = i < n && (a.parent ? __ldg(a.parent + q0 + i) : i - 1) == node &&
                        __ldg(a.tokens + q0 + i) == found;
        const uint32_t who = __ballot_sync(0xffffffffu, is);
        if (who) child = i0 + __ffs(who) - 1;
      }
      if (lane < a.cluster) {
        st_dsmem_u32(dsmem_addr(&drawn, lane), static_cast<uint32_t>(found));
        st_dsmem_u32(dsmem_addr(&chosen, lane), static_cast<uint32_t>(child));
      }
    }
    __syncwarp();
    cluster_sync_all();
    const int child = static_cast<int>(chosen);
    if (rank == 0 && tid == 0) {
      path[step] = node;
      next[step] = static_cast<int>(drawn);
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
  if (V >= kMaxV || depth > TS_MAX_TREE || int64_t(B) * kMaxCluster > 2147483647)
    return TS_ERR_UNSUPPORTED;
  const bool even = aligned16(target) && target_stride % 4 == 0;  // (else a row's shift)
  const int pieces = (V + (even ? 0 : 3) + kPiece - 1) / kPiece;
  // As many CTAs a request as the GPU holds at once for all of them, one an SM
  // (a second wave would wait for the first's whole walk), and no more than
  // have pieces; but no CTA has more pieces than its shared memory has sums for.
  int cluster = 1;
  while (cluster < kMaxCluster && cluster * kWarps < pieces &&
         (int64_t(B) * cluster * 2 <= sm_count() || pieces > kMaxPieces * cluster))
    cluster *= 2;
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
  a.rounds = (pieces + cluster * kWarps - 1) / (cluster * kWarps);
  a.path = path;
  a.next = next;
  a.accepted = accepted;
  a.err = err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, verify_tree_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return TS_ERR_CUDA;
  }
  return launch_status();
}
