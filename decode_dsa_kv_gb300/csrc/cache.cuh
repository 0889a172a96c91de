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
