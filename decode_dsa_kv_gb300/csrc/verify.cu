// ts_verify_drafts: acceptance of drafted tokens (speculative sampling) and
// the draw of the token after them.
//
// One cluster of up to 8 CTAs per request. The acceptance of a request's n
// drafts reads 2 n probabilities; what costs is the one pass over the row
// (two rows after a refusal) that the next token is drawn from: 4 or 8 bytes
// a token of the vocabulary, bound by memory. Each CTA sums its slice of the
// vocabulary by tiles of kTile tokens, the slices' sums meet through
// distributed shared memory, and the CTA that holds the drawn point finds its
// tile in its tile sums and re-reads only that tile.
//
// The weights are whole multiples of 2^-60 in 64 bits: sums are exact, so the
// drawn token depends neither on the split nor on the order, and an integer
// add costs a fraction of an FP64 one here. (An fp32 running sum over 10^5
// tokens would move the borders between tokens by about 1e-6.) A probability
// is cut into three whole numbers by additions rounded towards zero, on the
// full-rate fp32 pipe: shifting its mantissa into 64 bits takes some 12
// half-rate integer instructions a value instead, and was what bounded the
// pass (128 requests x 131,072 tokens, 118 MB: 86 us; so 35 us, 0.51 of the
// measured copy rate: the rest is each cluster's chain of sums, cluster barrier
// and second look at one tile, and the pass's own instructions, 0.60 of the issue
// slots over the launch).
#include "common.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 512;
constexpr int kPer = 8;                 // tokens of a tile per thread
constexpr int kTile = kThreads * kPer;  // 4096
constexpr int kMaxCluster = 8;
constexpr int kMaxTiles = 256;  // of a CTA: 34 KB of sums
constexpr int kMaxV = kMaxTiles * kMaxCluster * kTile;
constexpr int kFrac = 60;

// p in [0, 2) as a multiple of 2^-60 (what lies below is cut off: nothing of a
// p of 2^-37 or more, whose last bit is at least 2^-60, and less than 2^-60 of a
// smaller one, all of it below 2^-60); anything else is 0 and sets *bad.
__device__ __forceinline__ uint64_t fixed(float p, int* bad) {
  const uint32_t b = __float_as_uint(p);
  if (b >= 0x40000000u) {  // 2 and more, NaN, or a sign
    if (b != 0x80000000u) *bad = 1;
    return 0;
  }
  const int sh = static_cast<int>(b >> 23) - (150 - kFrac);
  const uint64_t m = (b >> 23) ? ((b & 0x7fffffu) | 0x800000u) : 0u;  // subnormals: below 2^-126
  return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0);
}

// floor(p 2^60) = H 2^39 + L 2^17 + M of p in [0, 2), each as the bits of a
// float 4 + x: 4 + p rounded down is 4 + H 2^-21; what that leaves, times 2^22,
// gives L in the same way, and its rest, times 2^17, M. For two values at
// once (packed fp32), of which the numbers' differences come back: the 4's
// bits cancel.
struct Parts {
  int32_t h, l, m;
};
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ int32_t bits_apart(uint64_t v) {
  return static_cast<int32_t>(static_cast<uint32_t>(v) - static_cast<uint32_t>(v >> 32));
}
__device__ __forceinline__ Parts parts_apart(float p, float q) {
  const uint64_t x = pack2(p, q), four = pack2(4.f, 4.f), minus4 = pack2(-4.f, -4.f),
                 one = pack2(-1.f, -1.f), up22 = pack2(0x1p22f, 0x1p22f),
                 up17 = pack2(0x1p17f, 0x1p17f);
  uint64_t a, b, c, t, r, s;
  asm("add.rz.f32x2 %0, %1, %2;" : "=l"(a) : "l"(x), "l"(four));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(a), "l"(minus4));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(t), "l"(one), "l"(x));  // exact: < 2^-21
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(b) : "l"(r), "l"(up22), "l"(four));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(b), "l"(one), "l"(four));  // 4 - b, exact
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(s) : "l"(r), "l"(up22), "l"(t));    // exact: < 2^-21
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(c) : "l"(s), "l"(up17), "l"(four));
  return {bits_apart(a), bits_apart(b), bits_apart(c)};
}

// u in [0, 1) as a multiple of 2^-64; outside it the nearest end.
__device__ __forceinline__ uint64_t fixed_u(float u) {
  if (!(u > 0.f)) return 0;
  if (u >= 1.f) return ~0ull;
  const uint32_t b = __float_as_uint(u);
  const int sh = static_cast<int>(b >> 23) - (150 - 64);
  const uint64_t m = (b >> 23) ? ((b & 0x7fffffu) | 0x800000u) : 0u;
  return sh >= 0 ? m << sh : (sh > -24 ? m >> -sh : 0);
}

// Sums of weights stop at 2^64 - 1: a row that adds up to 16 or more is told by
// its total, whatever the order of summation.
constexpr uint64_t kFull = ~0ull;
__device__ __forceinline__ uint64_t add_full(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  return s < a ? kFull : s;
}

struct Weights {
  const float* p;
  const float* q;  // NULL: none, or one-hot at `hot`
  int hot;         // -1: none
  bool plain;      // the fallback: p itself
  __device__ __forceinline__ uint64_t at(int t, int V, int* bad) const {
    if (t >= V) return 0;
    const uint64_t a = fixed(__ldg(p + t), bad);
    if (plain) return a;
    if (q) {
      const uint64_t c = fixed(__ldg(q + t), bad);
      return a > c ? a - c : 0;
    }
    return t == hot ? 0 : a;
  }
  // This thread's tokens of a tile: t, t + kThreads, ..
  struct Tile {
    float a[kPer], b[kPer];
  };
  __device__ __forceinline__ void load(Tile& x, int64_t t, int V) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t k = t + j * kThreads;
      x.a[j] = k < V ? __ldg(p + k) : 0.f;
      x.b[j] = q && !plain && k < V ? __ldg(q + k) : 0.f;
    }
  }
  // The warp's share of the tile's sum, in every lane; exact as long as *top
  // (the largest bits) stays below those of 2.
  static constexpr int32_t kLargeH = (1 << 25) - (1 << 9);
  __device__ __forceinline__ uint64_t warp_tile_sum(const Tile& x, int64_t t, uint32_t* top) const {
    int32_t h = 0, l = 0, m = 0;  // |each| below kPer 2^22, the warp's below 2^30
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      *top = max(*top, max(__float_as_uint(x.a[j]), __float_as_uint(x.b[j])));
      const Parts u = parts_apart(x.a[j], x.b[j]);
      if (x.a[j] > x.b[j] && (plain || t + j * kThreads != hot)) {
        h += u.h;
        l += u.l;
        m += u.m;
      }
    }
    h = __reduce_add_sync(0xffffffffu, h);
    l = __reduce_add_sync(0xffffffffu, l);
    m = __reduce_add_sync(0xffffffffu, m);
    // below 2^64 as long as H 2^39 is below it by more than |L| 2^17 + |M| < 2^48:
    // else (a tile's share of some 16) value by value
    if (h >= kLargeH) *top = ~0u;
    return (int64_t(h) << 39) + (int64_t(l) << 17) + m;
  }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = add_full(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

__device__ __forceinline__ uint64_t ld_dsmem_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads, 2)
    verify_kernel(const int32_t* __restrict__ drafts, const int32_t* __restrict__ n_draft,
                  const float* __restrict__ target, int64_t target_stride,
                  const float* __restrict__ draft, int64_t draft_stride,
                  const float* __restrict__ u, int n, int V, int cluster, int tiles_per_cta,
                  int32_t* __restrict__ tokens, int32_t* __restrict__ accepted, int32_t* err) {
  extern __shared__ uint64_t tile_sum[];  // this CTA's tiles, then their warps' parts
  uint64_t* part = tile_sum + tiles_per_cta;
  __shared__ uint64_t cta_sum;
  __shared__ uint64_t warp_part[kThreads / 32];
  __shared__ int first_refused;
  const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0, bad_id = 0;

  // ---- acceptance ----
  const int nd = n_draft ? min(max(__ldg(n_draft + b), 0), n) : n;
  if (tid == 0) first_refused = nd;
  __syncthreads();
  for (int i = tid; i < nd; i += kThreads) {
    const int x = __ldg(drafts + int64_t(b) * n + i);
    bool take = false;
    if (x >= 0 && x < V) {
      const float p = __ldg(target + (int64_t(b) * (n + 1) + i) * target_stride + x);
      const float q = draft ? __ldg(draft + (int64_t(b) * n + i) * draft_stride + x) : 1.f;
      // u q and p in double: the product of two floats is exact there
      take = double(__ldg(u + int64_t(b) * (n + 1) + i)) * double(q) < double(p);
      if (!(p >= 0.f && p < 2.f && q >= 0.f && q < 2.f)) {
        bad = 1;
        take = false;
      }
    } else {
      bad_id = 1;
    }
    if (!take) atomicMin(&first_refused, i);
  }
  __syncthreads();
  const int a = first_refused;
  Weights w;
  w.p = target + (int64_t(b) * (n + 1) + a) * target_stride;
  w.q = draft && a < nd ? draft + (int64_t(b) * n + a) * draft_stride : nullptr;
  w.hot = !draft && a < nd ? __ldg(drafts + int64_t(b) * n + a) : -1;
  w.plain = false;

  // ---- the next token ----
  const int tile0 = rank * tiles_per_cta;
  int next = -1;
  for (int pass = 0; pass < 2; ++pass) {
    // every warp's part of every tile's sum; the tiles' sums follow
    uint32_t top = 0;  // the largest bits seen: 2 and more, NaN or a sign (or a sum too large)
    Weights::Tile ahead;
    w.load(ahead, int64_t(tile0) * kTile + tid, V);
    for (int i = 0; i < tiles_per_cta; ++i) {
      const int64_t t = int64_t(tile0 + i) * kTile + tid;
      const Weights::Tile x = ahead;
      if (i + 1 < tiles_per_cta) w.load(ahead, t + kTile, V);
      const uint64_t v = w.warp_tile_sum(x, t, &top);
      if (lane == 0) part[i * (kThreads / 32) + warp] = v;
    }
    if (__syncthreads_or(top >= 0x40000000u)) {  // value by value, the bad ones left out
      for (int i = 0; i < tiles_per_cta; ++i) {
        const int64_t t0 = int64_t(tile0 + i) * kTile;
        uint64_t v = 0;  // (kPer values below 2: below 2^64)
        for (int j = 0; j < kPer && t0 < V; ++j)
          v += w.at(static_cast<int>(t0) + j * kThreads + tid, V, &bad);
        v = warp_sum(v);
        if (lane == 0) part[i * (kThreads / 32) + warp] = v;
      }
      __syncthreads();
    }
    for (int i = tid; i < tiles_per_cta; i += kThreads) {
      uint64_t v = 0;
      for (int k = 0; k < kThreads / 32; ++k) v = add_full(v, part[i * (kThreads / 32) + k]);
      tile_sum[i] = v;
    }
    __syncthreads();
    if (warp == 0) {
      uint64_t v = 0;
      for (int i = lane; i < tiles_per_cta; i += 32) v = add_full(v, tile_sum[i]);
      v = warp_sum(v);
      if (lane == 0) cta_sum = v;
    }
    cluster_sync_all();
    uint64_t before = 0, total = 0;
    for (int r = 0; r < cluster; ++r) {
      const uint64_t v = ld_dsmem_u64(dsmem_addr(&cta_sum, r));
      if (r < rank) before += v;  // (used only where the total fits)
      total = add_full(total, v);
    }
    const uint64_t mine = cta_sum;
    cluster_sync_all();  // every CTA has read the sums: they may change, or the CTA leave
    if (total == kFull) break;  // (this and the next: the same in every CTA of the cluster)
    if (total == 0) {
      if (w.plain || (!w.q && w.hot < 0)) break;
      w.plain = true;
      continue;
    }
    const uint64_t r = __umul64hi(fixed_u(__ldg(u + int64_t(b) * (n + 1) + n)), total);
    if (r < before || r - before >= mine) {
      next = -2;  // another CTA's
      break;
    }
    uint64_t rest = r - before;
    int i = 0;
    while (rest >= tile_sum[i]) rest -= tile_sum[i++];  // ends: the CTA's sum is above rest
    // within the tile, in token order: thread t holds tokens t * kPer ..
    const int t0 = (tile0 + i) * kTile + tid * kPer;
    uint64_t v[kPer], s = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += v[j] = w.at(t0 + j, V, &bad);
    uint64_t inc = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) warp_part[warp] = inc;
    __syncthreads();
    uint64_t ex = inc - s;
    for (int k = 0; k < warp; ++k) ex += warp_part[k];
    if (rest >= ex && rest - ex < s) {
      uint64_t left = rest - ex;
      int j = 0;
#pragma unroll
      for (int k = 0; k < kPer - 1; ++k)
        if (j == k && left >= v[k]) left -= v[k], j = k + 1;
      next = t0 + j;
    }
    if (next < 0) next = -2;
    break;
  }

  // ---- results: the thread that holds the token, or (a row without weight, or
  // with too much) the first CTA's first thread ----
  if (bad) report(err, TS_DEVERR_PROB);
  if (bad_id && rank == 0) report(err, TS_DEVERR_ID_RANGE);
  if (next == -1 && (rank != 0 || tid != 0)) next = -2;
  if (next != -2) {
    if (next < 0) report(err, TS_DEVERR_PROB);
    tokens[int64_t(b) * (n + 1) + a] = next;
    accepted[b] = a;
  }
  if (rank == 0)
    for (int i = tid; i <= n; i += kThreads)
      if (i != a)
        tokens[int64_t(b) * (n + 1) + i] = i < a ? __ldg(drafts + int64_t(b) * n + i) : -1;
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" ts_status ts_verify_drafts(const int32_t* drafts, const int32_t* n_draft,
                                      const float* target, int64_t target_stride,
                                      const float* draft, int64_t draft_stride, const float* u,
                                      int B, int n, int V, int32_t* tokens, int32_t* accepted,
                                      int32_t* err, cudaStream_t stream) {
  if (B < 0 || n < 0 || V <= 0) return TS_ERR_INVALID_ARG;
  if (B == 0) return TS_OK;
  if (!target || !u || !tokens || !accepted || (n > 0 && !drafts)) return TS_ERR_INVALID_ARG;
  if (target_stride < V || (draft && draft_stride < V)) return TS_ERR_INVALID_ARG;
  if (V >= kMaxV || n > 65535 || int64_t(B) * kMaxCluster > 2147483647) return TS_ERR_UNSUPPORTED;
  const int tiles = (V + kTile - 1) / kTile;
  // As many CTAs a request as the GPU holds at once for all of them (two an
  // SM): a second wave would wait for the first's whole chain of loads. But no
  // CTA has more tiles than its shared memory has sums for.
  int cluster = 1;
  while (cluster < kMaxCluster && cluster < tiles &&
         (int64_t(B) * cluster <= sm_count() || tiles > kMaxTiles * cluster))
    cluster *= 2;
  const int per = (tiles + cluster - 1) / cluster;
  const int smem = per * 8 * (1 + kThreads / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, verify_kernel, drafts, n_draft, target, target_stride, draft,
                         draft_stride, u, n, V, cluster, per, tokens, accepted, err) !=
      cudaSuccess) {
    cudaGetLastError();
    return TS_ERR_CUDA;
  }
  return launch_status();
}
