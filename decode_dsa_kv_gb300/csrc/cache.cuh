// Row formats of the paged latent cache, shared by its kernels.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dsakv {

constexpr int kE4m3RowBytes = 656;  // 512 codes, 4 float scales, 64 bf16 rope values
constexpr int kE4m3Rope = 528;      // byte offset of the rope values

__host__ __device__ constexpr int cache_row_bytes(int fmt) {
  return fmt == DSA_CACHE_BF16 ? DSA_ROW_BYTES : kE4m3RowBytes;
}

// Argument checks that the calls on a cache share.
ts_status cache_check(const void* cache, int64_t num_slots, int fmt);
ts_status paging_check(const int32_t* block_table, int64_t table_stride, int page_size,
                       int64_t num_slots);

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

// A row's latent part as codes: lane i of a warp holds the values 16 i .. 16 i +
// 15 (x) and stores their codes, so a group of 128 is eight lanes, and the
// first of them stores its scale.
__device__ __forceinline__ void store_codes(uint8_t* dst, const uint4 (&x)[2], int lane) {
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
}

// 16 e4m3 codes times a power-of-two scale as 16 bf16 values (exact: e4m3 has
// 4 significant bits and bf16 8; a scale of at least 2^-120 keeps the
// smallest product, 2^-9 of it, a multiple of bf16's subnormal step).
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4& c, float scale, uint4 (&o)[2]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto code = static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
    const __half2 h(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3));
    const float2 f = __half22float2(h);
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  o[0] = make_uint4(r[0], r[1], r[2], r[3]);
  o[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

}  // namespace dsakv
