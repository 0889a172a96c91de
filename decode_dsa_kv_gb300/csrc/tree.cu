// dsa_tree_plan: what a drafted tree's parents mean for the other calls, and
// dsa_cache_keep: the rows of its accepted path moved together.
#include <algorithm>
#include <climits>

#include "cache.cuh"
#include "chunk_plan.h"

namespace dsakv {
namespace {

constexpr int kPlanThreads = 256;

struct Table {
  const int32_t* entries;  // [B][stride], or NULL
  int64_t stride;
  int shift;       // log2 of the page size
  int64_t pages;   // of the cache
  int max_ctx;     // positions that a row has room for, at most kMaxCtx
  // The slot of request b's position t, or -1.
  __device__ __forceinline__ int slot(int b, int t) const {
    if (t < 0 || t >= max_ctx) return -1;
    const int64_t page = entries[b * stride + (t >> shift)];
    if (page < 0 || page >= pages) return -1;
    return static_cast<int>((page << shift) + (t & ((1 << shift) - 1)));
  }
};

// One request, its values brought into range and reported where they were not.
__device__ __forceinline__ Request tree_of(const int32_t* cu_q, int T, const int32_t* ctx_len,
                                           int max_ctx, int b, bool reports, int32_t* err) {
  const int c0 = cu_q[b], c1 = cu_q[b + 1], ctx = ctx_len[b];
  Request r;
  r.q0 = min(max(c0, 0), T);
  r.n = max(min(c1, T) - r.q0, 0);
  r.ctx = min(max(ctx, 0), max_ctx);
  if (reports) {
    if (c0 < 0 || c1 < c0 || c1 > T) report(err, TS_DEVERR_ORDER);
    if (ctx < 0 || ctx > max_ctx || r.n > r.ctx) report(err, TS_DEVERR_CTX);
  }
  return r;
}

// A CTA a request, a thread a node, which walks up its parents in shared
// memory; they descend, so the mask is written word by word on the way. Bound
// by its launch and two dependent loads (lengths, parents); a walk's step is
// one shared load: 32 trees of up to 61 nodes 2 us. The last CTA clears the tokens that no request has.
__global__ void __launch_bounds__(kPlanThreads)
    tree_plan_kernel(const int32_t* parent, const int32_t* cu_q, int T,
                     int B, const int32_t* ctx_len, const Table table,
                     int32_t* pos, int32_t* slots,
                     uint32_t* mask, int words, int32_t* err) {
  __shared__ int32_t up[TS_MAX_TREE];
  launch_dependents();
  wait_previous_kernel();
  const int b = blockIdx.x, tid = threadIdx.x;
  auto none = [&](int t) {
    if (pos) pos[t] = 0;
    if (slots) slots[t] = -1;
    if (mask)
      for (int k = 0; k < words; ++k) mask[int64_t(t) * words + k] = 0;
  };
  if (b == B) {
    const int c0 = cu_q[0], c1 = cu_q[B];
    int falls = c0 < 0 | c1 > T;
    for (int i = tid; i < B; i += kPlanThreads) falls |= cu_q[i] > cu_q[i + 1];  // (all at once)
    const int first = min(max(c0, 0), T), last = min(max(c1, 0), T);
    if (!__syncthreads_or(falls)) {
      for (int t = tid; t < first; t += kPlanThreads) none(t);
      for (int64_t t = int64_t(last) + tid; t < T; t += kPlanThreads) none(static_cast<int>(t));
      return;
    }
    // (reported; requests may then lie anywhere among the tokens: one by one)
    for (int64_t t = tid; t < T; t += kPlanThreads) {
      bool has = false;
      for (int i = 0; i < B && !has; ++i) {
        const int q0 = min(max(cu_q[i], 0), T);
        has = t >= q0 && t < min(cu_q[i + 1], T);
      }
      if (!has) none(static_cast<int>(t));
    }
    return;
  }
  const Request r = tree_of(cu_q, T, ctx_len, table.max_ctx, b, tid == 0, err);
  const int planned = parent ? min(r.n, TS_MAX_TREE) : r.n;
  if (tid == 0 && (planned < r.n || (mask && r.n > 32 * words))) report(err, TS_DEVERR_COUNT);
  if (parent) {
    for (int i = tid; i < planned; i += kPlanThreads) {
      int p = parent[r.q0 + i];
      if (p < -1 || p >= i) {
        report(err, TS_DEVERR_PARENT);
        p = -1;
      }
      up[i] = p;
    }
    __syncthreads();
  }
  for (int i = tid; i < r.n; i += kPlanThreads) {
    const int t = r.q0 + i;
    if (i >= planned) {
      none(t);
      continue;
    }
    uint32_t* row = mask + int64_t(t) * words;
    // words `from` and below, down to `to` and above it
    auto put = [&](int from, int to, uint32_t v) {
      if (mask)
        for (int k = min(from, words - 1); k > to; --k) row[k] = v;
    };
    int w = i >> 5, depth = i;
    put(words - 1, w, 0u);
    if (parent) {
      uint32_t bits = 0;
      depth = -1;
      for (int x = i; x >= 0; x = up[x], ++depth) {
        if ((x >> 5) != w) {
          put(w, w - 1, bits);
          put(w - 1, x >> 5, 0u);
          w = x >> 5;
          bits = 0;
        }
        bits |= 1u << (x & 31);
      }
      put(w, w - 1, bits);
      put(w - 1, -1, 0u);
    } else {
      put(w, w - 1, 0xffffffffu >> (31 - (i & 31)));
      put(w - 1, -1, 0xffffffffu);
    }
    const int at = r.ctx - r.n + i;
    if (pos) pos[t] = r.ctx - r.n + depth;
    if (slots) {
      const int s = table.slot(b, at);
      if (s < 0 && at >= 0) report(err, TS_DEVERR_SLOT_RANGE);
      slots[t] = s;
    }
  }
}

// A CTA a request, a warp a row. Row path[i] goes to place i <= path[i], and a
// path ascends, so rows read together are read before any of them is written,
// and later ones lie past every place written so far (path[j] >= j). Bound by
// its launch and the chain of path, block table, row: 2.5 us.
constexpr int kKeepWarps = 8;
template <int kFmt>
__global__ void __launch_bounds__(32 * kKeepWarps)
    cache_keep_kernel(uint8_t* cache, const Table table, const int32_t* cu_q, int T,
                      const int32_t* ctx_len, const int32_t* path, int depth,
                      const int32_t* accepted, int32_t* new_len, int32_t* err) {
  constexpr int kPieces = cache_row_bytes(kFmt) / 16, kEach = (kPieces + 31) / 32;
  wait_previous_kernel();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Request r = tree_of(cu_q, T, ctx_len, table.max_ctx, b, tid == 0, err);
  const int a = accepted[b], base = r.ctx - r.n;
  const int32_t* x = path + int64_t(b) * (depth + 1);
  bool ascends = a >= -1 && a <= depth, paged = true;
  for (int i = tid; ascends && i <= a; i += 32 * kKeepWarps) {
    const int node = x[i];
    ascends = node < r.n && (i == 0 ? node == 0 : node > x[i - 1]);
    // (the last row's place is looked up even where it stays)
    if (ascends) paged = paged && table.slot(b, base + node) >= 0 && table.slot(b, base + i) >= 0;
  }
  ascends = __syncthreads_and(ascends);
  paged = __syncthreads_and(paged);
  if (tid == 0) {
    if (!ascends) report(err, TS_DEVERR_PARENT);
    else if (!paged) report(err, TS_DEVERR_SLOT_RANGE);
    if (new_len) new_len[b] = max(0, base) + (ascends ? a + 1 : 0);
  }
  if (!ascends || !paged) return;
  for (int i0 = 1; i0 <= a; i0 += kKeepWarps) {
    const int i = i0 + warp, node = i <= a ? x[i] : i;
    uint4 v[kEach];
    if (node != i) {
      const uint4* src = reinterpret_cast<const uint4*>(
          cache + int64_t(table.slot(b, base + node)) * cache_row_bytes(kFmt));
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (lane + 32 * k < kPieces) v[k] = src[lane + 32 * k];
    }
    __syncthreads();
    if (node != i) {
      uint4* dst = reinterpret_cast<uint4*>(
          cache + int64_t(table.slot(b, base + i)) * cache_row_bytes(kFmt));
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (lane + 32 * k < kPieces) dst[lane + 32 * k] = v[k];
    }
    __syncthreads();
  }
}

Table make_table(const int32_t* block_table, int64_t table_stride, int page_size,
                 int64_t num_slots) {
  Table t = {};
  t.entries = block_table;
  t.stride = table_stride;
  t.max_ctx = kMaxCtx;
  if (!block_table) return t;
  t.shift = __builtin_ctz(page_size);
  t.pages = num_slots / page_size;
  t.max_ctx = static_cast<int>(
      std::min(std::min(table_stride, int64_t(kMaxCtx)) * page_size, int64_t(kMaxCtx)));
  return t;
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" ts_status dsa_tree_plan(const int32_t* parent, const int32_t* cu_q, int T, int B,
                                   const int32_t* ctx_len, const int32_t* block_table,
                                   int64_t table_stride, int page_size, int64_t num_slots,
                                   int32_t* pos, int32_t* slots, uint32_t* mask, int words,
                                   int32_t* err, cudaStream_t stream) {
  if (T < 0 || B <= 0 || (mask && words <= 0) || (slots && !block_table))
    return TS_ERR_INVALID_ARG;
  if (block_table) {
    const ts_status st = paging_check(block_table, table_stride, page_size, num_slots);
    if (st != TS_OK) return st;
    if (num_slots > INT_MAX) return TS_ERR_UNSUPPORTED;
  }
  if (T == 0) return TS_OK;
  if (!cu_q || !ctx_len) return TS_ERR_INVALID_ARG;
  if (B == INT_MAX || (mask && words > TS_MAX_TREE / 32)) return TS_ERR_UNSUPPORTED;
  return launch_after(tree_plan_kernel, unsigned(B) + 1, kPlanThreads, stream, parent, cu_q, T, B,
                      ctx_len, make_table(block_table, table_stride, page_size, num_slots), pos,
                      slots, mask, words, err);
}

extern "C" ts_status dsa_cache_keep(void* cache, int64_t num_slots, int fmt,
                                    const int32_t* block_table, int64_t table_stride,
                                    int page_size, const int32_t* cu_q, int T,
                                    const int32_t* ctx_len, int B, const int32_t* path, int depth,
                                    const int32_t* accepted, int32_t* new_len, int32_t* err,
                                    cudaStream_t stream) {
  ts_status st = cache_check(cache, num_slots, fmt);
  if (st == TS_OK) st = paging_check(block_table, table_stride, page_size, num_slots);
  if (st != TS_OK) return st;
  if (B < 0 || T < 0 || depth < 0) return TS_ERR_INVALID_ARG;
  if (num_slots > INT_MAX || depth > TS_MAX_TREE) return TS_ERR_UNSUPPORTED;
  if (B == 0) return TS_OK;
  if (!cu_q || !ctx_len || !path || !accepted) return TS_ERR_INVALID_ARG;
  auto kernel = fmt == DSA_CACHE_BF16 ? cache_keep_kernel<DSA_CACHE_BF16>
                                      : cache_keep_kernel<DSA_CACHE_E4M3>;
  return launch_after(kernel, unsigned(B), 32 * kKeepWarps, stream, static_cast<uint8_t*>(cache),
                      make_table(block_table, table_stride, page_size, num_slots), cu_q, T,
                      ctx_len, path, depth, accepted, new_len, err);
}
