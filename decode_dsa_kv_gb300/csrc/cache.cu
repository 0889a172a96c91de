// The paged latent cache's rows: written (bf16, or quantised to e4m3 with a
// power-of-two scale for each 128 latent values) and read back as bf16.
#include <cuda_fp8.h>

#include <climits>

#include "cache.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The exponent e of a group's scale 2^e: the smallest e >= -120 with
// amax <= 448 * 2^e = 1.75 * 2^(8 + e). With amax = f * 2^a, 1 <= f < 2, that
// is a - 8 for f <= 1.75 and a - 7 above; read off the float's bits (zero and
// subnormals end up at the lower limit, infinity, a = 128 and f = 1, at 120).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int a = static_cast<int>(b >> 23) - 127;
  return max(a - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), -120);
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// One warp a row; lane i holds the latent values 16 i .. 16 i + 15, so a group
// of 128 is eight lanes. One pass: a row is read once, its maxima are found in
// the lanes that hold it, and it is written once. Bound by memory: 32,768 rows
// quantised (59 MB) in 8.5 us with them in L2, 17.5 us (0.51 of the measured
// copy rate) from HBM; up to a few hundred rows by its launch, 4.3 us.
template <int kFmt>
__global__ void __launch_bounds__(kThreads)
    cache_write_kernel(const __nv_bfloat16* __restrict__ latent, int64_t latent_stride,
                       const __nv_bfloat16* __restrict__ rope, int64_t rope_stride,
                       const int32_t* __restrict__ slots, int n, uint8_t* __restrict__ cache,
                       int64_t num_slots, int32_t* err) {
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= n) return;
  const int32_t slot = __ldg(slots + row);
  if (slot < 0) return;
  if (slot >= num_slots) {
    if (lane == 0) report(err, TS_DEVERR_SLOT_RANGE);
    return;
  }
  uint8_t* dst = cache + int64_t(slot) * cache_row_bytes(kFmt);
  const uint4* src = reinterpret_cast<const uint4*>(latent + int64_t(row) * latent_stride);
  const uint4* rsrc = reinterpret_cast<const uint4*>(rope + int64_t(row) * rope_stride);
  if (kFmt == DSA_CACHE_BF16) {
    uint4* d = reinterpret_cast<uint4*>(dst);
    d[lane] = __ldg(src + lane);
    d[lane + 32] = __ldg(src + lane + 32);
    if (lane < 8) d[64 + lane] = __ldg(rsrc + lane);
    return;
  }
  const uint4 x[2] = {__ldg(src + 2 * lane), __ldg(src + 2 * lane + 1)};
  uint4 r = {};
  if (lane < 8) r = __ldg(rsrc + lane);
  float v[16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(x)[i];
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));  // a NaN drops out
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  const int e = scale_exponent(amax);
  const float inv = exp2i(-e);  // exact; so is every product below
  uint32_t codes[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    codes[i] = lo | (hi << 16);
  }
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
  if ((lane & 7) == 0) reinterpret_cast<float*>(dst + TS_D_LATENT)[lane >> 3] = exp2i(e);
  if (lane < 8) reinterpret_cast<uint4*>(dst + kE4m3Rope)[lane] = r;
}

// kReadRows rows a warp: their positions and pages are looked up by as many
// lanes at once, and every row's pieces are on their way before the first is
// stored. Four rows a warp where there are rows for every SM, else one
// (measured, 8-bit rows: 65,536 rows 30.9 us with one and 25.1 with four, 256
// rows 4.3 and 6.2). Bound by the latency of its loads: those 65,536 rows are 119
// MB, 0.71 of the measured copy rate; as bf16 rows 151 MB in 27.0 us, 0.84.
template <int kFmt, int kReadRows>
__global__ void __launch_bounds__(kThreads)
    cache_read_kernel(const uint8_t* __restrict__ cache, int64_t num_slots,
                      const int32_t* __restrict__ block_table, int64_t table_stride,
                      int page_shift, const int32_t* __restrict__ pos,
                      const int32_t* __restrict__ ctx_len, int64_t rows, int k,
                      uint8_t* __restrict__ sel, int32_t* err) {
  const int64_t row0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kReadRows;
  const int lane = threadIdx.x & 31;
  int32_t slot = -1;
  if (lane < kReadRows && row0 + lane < rows) {
    const int b = static_cast<int>((row0 + lane) / k);
    const int32_t t = __ldg(pos + row0 + lane);
    if (t < 0 || t >= __ldg(ctx_len + b)) {
      report(err, TS_DEVERR_ID_RANGE);
    } else {
      const int page_i = t >> page_shift;
      int64_t at = -1;
      if (page_i < table_stride)
        at = (int64_t(__ldg(block_table + b * table_stride + page_i)) << page_shift) +
             (t & ((1 << page_shift) - 1));
      if (at < 0 || at >= num_slots) report(err, TS_DEVERR_SLOT_RANGE);
      else slot = static_cast<int32_t>(at);
    }
  }
  uint4 x[kReadRows][kFmt == DSA_CACHE_BF16 ? 3 : 2];
  float scale[kReadRows];
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    const int32_t at = __shfl_sync(0xffffffffu, slot, i);
    if (at < 0) continue;
    const uint8_t* src = cache + int64_t(at) * cache_row_bytes(kFmt);
    const uint4* s = reinterpret_cast<const uint4*>(src);
    x[i][0] = __ldg(s + lane);
    if (kFmt == DSA_CACHE_BF16) {
      x[i][1] = __ldg(s + lane + 32);
      if (lane < 8) x[i][2] = __ldg(s + 64 + lane);
    } else {
      scale[i] = __ldg(reinterpret_cast<const float*>(src + TS_D_LATENT) + (lane >> 3));
      if (lane < 8) x[i][1] = __ldg(reinterpret_cast<const uint4*>(src + kE4m3Rope) + lane);
    }
  }
#pragma unroll
  for (int i = 0; i < kReadRows; ++i) {
    if (__shfl_sync(0xffffffffu, slot, i) < 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(sel + (row0 + i) * DSA_ROW_BYTES);
    if (kFmt == DSA_CACHE_BF16) {
      dst[lane] = x[i][0];
      dst[lane + 32] = x[i][1];
      if (lane < 8) dst[64 + lane] = x[i][2];
    } else {
      uint4 o[2];
      e4m3x16_to_bf16(x[i][0], scale[i], o);
      dst[2 * lane] = o[0];
      dst[2 * lane + 1] = o[1];
      if (lane < 8) dst[64 + lane] = x[i][1];
    }
  }
}

}  // namespace

ts_status cache_check(const void* cache, int64_t num_slots, int fmt) {
  if (!cache || !aligned16(cache) || num_slots <= 0) return TS_ERR_INVALID_ARG;
  if (fmt != DSA_CACHE_BF16 && fmt != DSA_CACHE_E4M3) return TS_ERR_INVALID_ARG;
  return TS_OK;
}

ts_status paging_check(const int32_t* block_table, int64_t table_stride, int page_size,
                       int64_t num_slots) {
  if (!block_table || table_stride <= 0 || page_size <= 0) return TS_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return TS_ERR_UNSUPPORTED;
  return num_slots < page_size ? TS_ERR_INVALID_ARG : TS_OK;
}

}  // namespace dsakv

using namespace dsakv;

extern "C" size_t dsa_cache_row_bytes(int fmt) {
  return fmt == DSA_CACHE_BF16 || fmt == DSA_CACHE_E4M3 ? cache_row_bytes(fmt) : 0;
}

extern "C" ts_status dsa_cache_write(const void* latent, int64_t latent_stride, const void* rope,
                                     int64_t rope_stride, const int32_t* slots, int n,
                                     void* cache, int64_t num_slots, int fmt, int32_t* err,
                                     cudaStream_t stream) {
  const ts_status st = cache_check(cache, num_slots, fmt);
  if (st != TS_OK) return st;
  if (n < 0) return TS_ERR_INVALID_ARG;
  if (n == 0) return TS_OK;
  if (!latent || !rope || !slots || !aligned16(latent) || !aligned16(rope))
    return TS_ERR_INVALID_ARG;
  if (latent_stride < TS_D_LATENT || latent_stride % 8 != 0 || rope_stride < TS_D - TS_D_LATENT ||
      rope_stride % 8 != 0)
    return TS_ERR_INVALID_ARG;
  const auto* l = static_cast<const __nv_bfloat16*>(latent);
  const auto* r = static_cast<const __nv_bfloat16*>(rope);
  auto* c = static_cast<uint8_t*>(cache);
  const unsigned grid = static_cast<unsigned>((int64_t(n) + kWarps - 1) / kWarps);
  if (fmt == DSA_CACHE_BF16)
    cache_write_kernel<DSA_CACHE_BF16><<<grid, kThreads, 0, stream>>>(
        l, latent_stride, r, rope_stride, slots, n, c, num_slots, err);
  else
    cache_write_kernel<DSA_CACHE_E4M3><<<grid, kThreads, 0, stream>>>(
        l, latent_stride, r, rope_stride, slots, n, c, num_slots, err);
  return launch_status();
}

extern "C" ts_status dsa_cache_read(const void* cache, int64_t num_slots, int fmt,
                                    const int32_t* block_table, int64_t table_stride,
                                    int page_size, const int32_t* pos, const int32_t* ctx_len,
                                    int B, int k, void* sel, int32_t* err, cudaStream_t stream) {
  ts_status st = cache_check(cache, num_slots, fmt);
  if (st == TS_OK) st = paging_check(block_table, table_stride, page_size, num_slots);
  if (st != TS_OK) return st;
  if (!pos || !ctx_len || !sel || !aligned16(sel) || B <= 0 || k <= 0) return TS_ERR_INVALID_ARG;
  const int64_t rows = int64_t(B) * k;
  if (rows > INT_MAX || num_slots > INT_MAX) return TS_ERR_UNSUPPORTED;
  const auto* c = static_cast<const uint8_t*>(cache);
  auto* o = static_cast<uint8_t*>(sel);
  const int shift = __builtin_ctz(page_size);
  auto launch = [&](auto kernel, int rows_warp) {
    const unsigned grid = static_cast<unsigned>((rows + kWarps * rows_warp - 1) / (kWarps * rows_warp));
    kernel<<<grid, kThreads, 0, stream>>>(c, num_slots, block_table, table_stride, shift, pos,
                                          ctx_len, rows, k, o, err);
  };
  const bool many = rows >= int64_t(sm_count()) * kWarps * 8;  // a full SM's warps
  if (fmt == DSA_CACHE_BF16) {
    if (many) launch(cache_read_kernel<DSA_CACHE_BF16, 4>, 4);
    else launch(cache_read_kernel<DSA_CACHE_BF16, 1>, 1);
  } else {
    if (many) launch(cache_read_kernel<DSA_CACHE_E4M3, 4>, 4);
    else launch(cache_read_kernel<DSA_CACHE_E4M3, 1>, 1);
  }
  return launch_status();
}
