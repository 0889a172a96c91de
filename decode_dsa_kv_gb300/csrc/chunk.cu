// sfa_mla_chunk: absorbed-MLA attention of each request's newest tokens over
// its paged latent cache. One CTA per (token, 8 heads), a warp a head: 32 keys
// at a time go to shared memory as bf16, lane j takes key j's score, and every
// lane then adds the weighted rows into its 16 of the 512 output dims.
#include <climits>
#include <cmath>

#include "cache.cuh"

namespace dsakv {
namespace {

constexpr int kKeys = 32;
constexpr int kHeadsCta = 8;
constexpr int kThreads = kHeadsCta * 32;
constexpr int kPitch = DSA_D + 8;  // bf16 values of a key's row in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    chunk_kernel(const __nv_bfloat16* __restrict__ q, int64_t q_stride,
                 const int32_t* __restrict__ cu_q, int T, int B, int H,
                 const uint8_t* __restrict__ cache, int64_t num_slots,
                 const int32_t* __restrict__ block_table, int64_t table_stride, int page_shift,
                 const int32_t* __restrict__ ctx_len, int causal, float scale_log2,
                 __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int32_t* err) {
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16* ks = reinterpret_cast<__nv_bfloat16*>(smem);
  float* qs = reinterpret_cast<float*>(smem + kKeys * kPitch * 2);
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kHeadsCta + warp;
  if (t == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i <= B; i += kThreads)
      if (__ldg(cu_q + i) > T || __ldg(cu_q + i) < (i ? __ldg(cu_q + i - 1) : 0))
        report(err, TS_DEVERR_ORDER);
  // the request of token t: the last with a start at or before t
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu_q + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  if (lo == B || t < __ldg(cu_q)) return;
  const int b = lo, first = __ldg(cu_q + b), n = min(__ldg(cu_q + b + 1), T) - first;
  int ctx = __ldg(ctx_len + b);
  const int64_t most = min(table_stride << page_shift, int64_t(INT_MAX));
  if (ctx < 0 || ctx > most) {
    if (threadIdx.x == 0) report(err, TS_DEVERR_CTX);
    ctx = ctx < 0 ? 0 : static_cast<int>(most);
  }
  const int limit = causal ? max(0, ctx - n + (t - first) + 1) : ctx;
  if (h < H)
    for (int d = lane; d < DSA_D; d += 32)
      qs[warp * DSA_D + d] = __bfloat162float(q[int64_t(t) * q_stride + int64_t(h) * DSA_D + d]);
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int k0 = 0; k0 < limit; k0 += kKeys) {
    __syncthreads();
    for (int j = warp; j < kKeys; j += kHeadsCta) {
      const int key = min(k0 + j, limit - 1);
      const int64_t page = __ldg(block_table + b * table_stride + (key >> page_shift));
      int64_t slot = (page << page_shift) + (key & ((1 << page_shift) - 1));
      if (slot < 0 || slot >= num_slots) {
        if (lane == 0) report(err, TS_DEVERR_SLOT_RANGE);
        slot = 0;
      }
      const uint8_t* src = cache + slot * cache_row_bytes(kFmt);
      uint4* dst = reinterpret_cast<uint4*>(ks + j * kPitch);
      if (kFmt == DSA_CACHE_BF16) {
        for (int c = lane; c < DSA_ROW_CHUNKS; c += 32)
          dst[c] = __ldg(reinterpret_cast<const uint4*>(src) + c);
      } else {
        uint4 o[2];
        e4m3x16_to_bf16(__ldg(reinterpret_cast<const uint4*>(src) + lane),
                        __ldg(reinterpret_cast<const float*>(src + TS_D_LATENT) + (lane >> 3)), o);
        dst[2 * lane] = o[0];
        dst[2 * lane + 1] = o[1];
        if (lane < 8) dst[64 + lane] = __ldg(reinterpret_cast<const uint4*>(src + kE4m3Rope) + lane);
      }
    }
    __syncthreads();
    if (h >= H) continue;
    float s = 0.f;
    const uint4* kr = reinterpret_cast<const uint4*>(ks + lane * kPitch);
    for (int c = 0; c < DSA_ROW_CHUNKS; ++c) {
      const uint4 v = kr[c];
      const float* qq = qs + warp * DSA_D + c * 8;
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s += qq[2 * i] * __uint_as_float(w[i] << 16);
        s += qq[2 * i + 1] * __uint_as_float(w[i] & 0xffff0000u);
      }
    }
    s = k0 + lane < limit ? s * scale_log2 : -INFINITY;
    float mx = s;
#pragma unroll
    for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float mn = fmaxf(m, mx), f = exp2f(m - mn), p = exp2f(s - mn);
    float ps = p;
#pragma unroll
    for (int d = 16; d; d >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, d);
    m = mn;
    l = l * f + ps;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= f;
    for (int j = 0; j < kKeys; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      const uint4* vr = reinterpret_cast<const uint4*>(ks + j * kPitch) + 2 * lane;
      const uint4 v0 = vr[0], v1 = vr[1];
      const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[2 * i] += pj * __uint_as_float(w[i] << 16);
        acc[2 * i + 1] += pj * __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  if (h >= H) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* dst = reinterpret_cast<uint4*>(out + (int64_t(t) * H + h) * DSA_DV) + 2 * lane;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  if (lse && lane == 0) lse[int64_t(t) * H + h] = l > 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" size_t sfa_chunk_workspace_size(int T, int B, int H) {
  if (T <= 0 || B <= 0 || H <= 0) return 0;
  return 256;
}

extern "C" ts_status sfa_mla_chunk(const void* q, int64_t q_stride, const int32_t* cu_q, int T,
                                   int B, int H, const void* cache, int64_t num_slots, int fmt,
                                   const int32_t* block_table, int64_t table_stride,
                                   int page_size, const int32_t* ctx_len, int causal, float scale,
                                   void* out, float* lse, void* ws, size_t ws_bytes, int32_t* err,
                                   cudaStream_t stream) {
  ts_status st = cache_check(cache, num_slots, fmt);
  if (st == TS_OK) st = paging_check(block_table, table_stride, page_size, num_slots);
  if (st != TS_OK) return st;
  if (T < 0 || B <= 0 || H <= 0 || !std::isfinite(scale)) return TS_ERR_INVALID_ARG;
  if (T == 0) return TS_OK;
  if (!q || !cu_q || !ctx_len || !out || !ws || !aligned16(q) || !aligned16(out))
    return TS_ERR_INVALID_ARG;
  if (q_stride < int64_t(H) * DSA_D || q_stride % 8 != 0) return TS_ERR_INVALID_ARG;
  if (H > 1024 || int64_t(T) * H >= INT_MAX - 127) return TS_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
      ws_bytes < sfa_chunk_workspace_size(T, B, H))
    return TS_ERR_WORKSPACE;
  const int smem = kKeys * kPitch * 2 + kHeadsCta * DSA_D * 4;
  const dim3 grid(T, (H + kHeadsCta - 1) / kHeadsCta);
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* c = static_cast<const uint8_t*>(cache);
  auto* o = static_cast<__nv_bfloat16*>(out);
  const int shift = __builtin_ctz(page_size);
  static std::atomic<uint64_t> set[2];
  const void* fn = fmt == DSA_CACHE_BF16
                       ? reinterpret_cast<const void*>(chunk_kernel<DSA_CACHE_BF16>)
                       : reinterpret_cast<const void*>(chunk_kernel<DSA_CACHE_E4M3>);
  if (!raise_smem_limit(fn, smem, set[fmt])) return TS_ERR_CUDA;
  if (fmt == DSA_CACHE_BF16)
    chunk_kernel<DSA_CACHE_BF16><<<grid, kThreads, smem, stream>>>(
        qb, q_stride, cu_q, T, B, H, c, num_slots, block_table, table_stride, shift, ctx_len,
        causal, scale * kLog2e, o, lse, err);
  else
    chunk_kernel<DSA_CACHE_E4M3><<<grid, kThreads, smem, stream>>>(
        qb, q_stride, cu_q, T, B, H, c, num_slots, block_table, table_stride, shift, ctx_len,
        causal, scale * kLog2e, o, lse, err);
  return launch_status();
}
