// dsa_cache_append: new tokens' rows into their slots and their queries made
// ready, the rope parts of both turned by their positions on the way.
#include "cache.cuh"

namespace dsakv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 16;  // of a warp's share of a token's queries

struct Turns {
  float cos[8], sin[8];
};

// The angles of this lane's 8 rope values: lane c of every eight holds the
// values 8 c .. 8 c + 7 of a rope part. pos * freq / 2 pi modulo one turn, in
// whole 2^-64 turns: freq / 2 pi is rounded once (2^-56 of a turn for a freq of
// at most 1), the product with pos is exact, so an angle is off by pos times
// that, and no range reduction of a large angle is needed (a double angle of
// position 10^6 is off by 2^-34, and its fp64 arithmetic takes 16 clocks an
// instruction here). A freq that is infinite or no number gives no number. Lane i
// computes pair i, the lanes that hold its values fetch it.
template <bool kPairs>
__device__ __forceinline__ Turns turns_of(const double* freq, int pos, int lane) {
  const double f = freq[lane], turn = f * 0.15915494309189533577;  // 1 / 2 pi
  const uint64_t step = static_cast<uint64_t>(__double2ull_rz((turn - floor(turn)) * 0x1p64));
  const int64_t at = static_cast<int64_t>(step * static_cast<uint64_t>(int64_t(pos)));
  // to fp32 from both halves, the lower one signed (one instruction for 64 bits takes
  // longer; a half turn's sign may change: the same angle)
  const int lo = static_cast<int>(at), hi = static_cast<int>((at + 0x80000000ll) >> 32);
  const float unit = (__double2hiint(f) & 0x7ff00000) == 0x7ff00000 ? NAN : 0x1p-31f;
  float s, c;
  sincospif(fmaf(static_cast<float>(lo), 0x1p-32f, static_cast<float>(hi)) * unit, &s, &c);
  Turns t;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int pair = kPairs ? (lane & 7) * 4 + (j >> 1) : (lane & 3) * 8 + j;
    t.cos[j] = __shfl_sync(0xffffffffu, c, pair);
    t.sin[j] = __shfl_sync(0xffffffffu, s, pair);
  }
  return t;
}

// Lane c's 8 values of a rope part, turned; fp32, rounded once.
template <bool kPairs>
__device__ __forceinline__ uint4 turned(const uint4& x, const Turns& t, int lane) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float v[8], y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  if (kPairs) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      y[j] = v[j] * t.cos[j] - v[j + 1] * t.sin[j];
      y[j + 1] = v[j] * t.sin[j] + v[j + 1] * t.cos[j];
    }
  } else {
    // the other half's value of each pair is four lanes on
    const float sign = (lane & 4) ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], 4);
      y[2 * i] = v[2 * i] * t.cos[2 * i] + sign * (__uint_as_float(o << 16) * t.sin[2 * i]);
      y[2 * i + 1] = v[2 * i + 1] * t.cos[2 * i + 1] +
                     sign * (__uint_as_float(o & 0xffff0000u) * t.sin[2 * i + 1]);
    }
  }
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

struct Args {
  const __nv_bfloat16 *latent, *rope;
  int64_t latent_stride, rope_stride;
  const int32_t *pos, *slots;
  int n;
  const double* freq;
  uint8_t* cache;
  int64_t num_slots;
  const __nv_bfloat16* q_rope;
  int64_t q_rope_stride, q_rope_head;
  int H, shares;  // a token's warps: its row, and 16 heads each
  __nv_bfloat16* q;
  int64_t q_stride;
  int32_t* err;
};

// A warp takes a token's row, or 16 heads of its queries: four heads an
// instruction, all sixteen on their way before the angles are computed. Bound by
// memory: 4095 tokens of 128 heads (144 MB, the queries' parts 128 bytes of every
// 384 read and of every 1152 written) in 25.7 us, 0.83 of the measured copy rate;
// with 8 heads a warp 27.9, with 32 27.1, in blocks of 256 threads 27.1. 991 nodes of
// 32 trees, 8-bit rows, behind their plan: 8.0 us; one token of 16 heads 1.6.
template <int kFmt, bool kPairs>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);  // (below 2^32)
  const uint32_t number = item / uint32_t(a.shares);
  const int share = static_cast<int>(item - number * a.shares);
  wait_previous_kernel();
  if (number >= uint32_t(a.n)) return;
  const int row = static_cast<int>(number);
  const int pos = a.pos[row];
  if (share > 0) {
    const int head0 = (share - 1) * kHeads + (lane >> 3), c = lane & 7;
    const __nv_bfloat16* src = a.q_rope + row * a.q_rope_stride + c * 8;
    uint4 x[kHeads / 4] = {};
#pragma unroll
    for (int i = 0; i < kHeads / 4; ++i)
      if (head0 + 4 * i < a.H)
        x[i] = *reinterpret_cast<const uint4*>(src + (head0 + 4 * i) * a.q_rope_head);
    const Turns t = turns_of<kPairs>(a.freq, pos, lane);
    __nv_bfloat16* dst = a.q + row * a.q_stride + DSA_DV + c * 8;
#pragma unroll
    for (int i = 0; i < kHeads / 4; ++i) {
      const uint4 y = turned<kPairs>(x[i], t, lane);
      if (head0 + 4 * i < a.H)
        *reinterpret_cast<uint4*>(dst + int64_t(head0 + 4 * i) * DSA_D) = y;
    }
    return;
  }
  const int32_t slot = a.slots[row];
  const uint4* src = reinterpret_cast<const uint4*>(a.latent + row * a.latent_stride);
  // (codes: a lane's 16 values side by side)
  const uint4 x[2] = {src[kFmt == DSA_CACHE_BF16 ? lane : 2 * lane],
                      src[kFmt == DSA_CACHE_BF16 ? lane + 32 : 2 * lane + 1]};
  const uint4 r =
      reinterpret_cast<const uint4*>(a.rope + row * a.rope_stride)[lane & 7];
  const uint4 y = turned<kPairs>(r, turns_of<kPairs>(a.freq, pos, lane), lane);
  if (slot < 0) return;
  if (slot >= a.num_slots) {
    if (lane == 0) report(a.err, TS_DEVERR_SLOT_RANGE);
    return;
  }
  uint8_t* dst = a.cache + int64_t(slot) * cache_row_bytes(kFmt);
  if (kFmt == DSA_CACHE_BF16) {
    reinterpret_cast<uint4*>(dst)[lane] = x[0];
    reinterpret_cast<uint4*>(dst)[lane + 32] = x[1];
    if (lane < 8) reinterpret_cast<uint4*>(dst)[64 + lane] = y;
  } else {
    store_codes(dst, x, lane);
    if (lane < 8) reinterpret_cast<uint4*>(dst + kE4m3Rope)[lane] = y;
  }
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" ts_status dsa_cache_append(const void* latent, int64_t latent_stride, const void* rope,
                                      int64_t rope_stride, const int32_t* pos,
                                      const int32_t* slots, int n, const double* freq, int pairs,
                                      void* cache, int64_t num_slots, int fmt, const void* q_rope,
                                      int64_t q_rope_stride, int64_t q_rope_head, int H, void* q,
                                      int64_t q_stride, int32_t* err, cudaStream_t stream) {
  const ts_status st = cache_check(cache, num_slots, fmt);
  if (st != TS_OK) return st;
  if (n < 0) return TS_ERR_INVALID_ARG;
  if (n == 0) return TS_OK;
  if (!latent || !rope || !pos || !slots || !freq || !aligned16(latent) || !aligned16(rope) ||
      (reinterpret_cast<uintptr_t>(freq) & 7u) != 0)
    return TS_ERR_INVALID_ARG;
  constexpr int kRope = TS_D - TS_D_LATENT;
  if (latent_stride < TS_D_LATENT || latent_stride % 8 != 0 || rope_stride < kRope ||
      rope_stride % 8 != 0)
    return TS_ERR_INVALID_ARG;
  if (q_rope) {
    if (!q || !aligned16(q) || !aligned16(q_rope) || H <= 0 || q_rope_head < kRope ||
        q_rope_head % 8 != 0 || q_rope_stride < kRope || q_rope_stride % 8 != 0 ||
        q_stride < int64_t(H) * TS_D || q_stride % 8 != 0)
      return TS_ERR_INVALID_ARG;
    if (H > 1024) return TS_ERR_UNSUPPORTED;
  }
  Args a = {};
  a.latent = static_cast<const __nv_bfloat16*>(latent);
  a.rope = static_cast<const __nv_bfloat16*>(rope);
  a.latent_stride = latent_stride;
  a.rope_stride = rope_stride;
  a.pos = pos;
  a.slots = slots;
  a.n = n;
  a.freq = freq;
  a.cache = static_cast<uint8_t*>(cache);
  a.num_slots = num_slots;
  a.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  a.q_rope_stride = q_rope_stride;
  a.q_rope_head = q_rope_head;
  a.H = H;
  a.shares = 1 + (q_rope ? (H + kHeads - 1) / kHeads : 0);
  a.q = static_cast<__nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.err = err;
  const int64_t blocks = (int64_t(n) * a.shares + kWarps - 1) / kWarps;
  if (blocks * kWarps > 0xffffffffll) return TS_ERR_UNSUPPORTED;
  auto kernel = fmt == DSA_CACHE_BF16 ? (pairs ? cache_append_kernel<DSA_CACHE_BF16, true>
                                               : cache_append_kernel<DSA_CACHE_BF16, false>)
                                      : (pairs ? cache_append_kernel<DSA_CACHE_E4M3, true>
                                               : cache_append_kernel<DSA_CACHE_E4M3, false>);
  return launch_after(kernel, static_cast<unsigned>(blocks), kThreads, stream, a);
}
