// sfa_mla_chunk: absorbed-MLA attention of each request's newest tokens over
// its paged latent cache.
//
// A request's n x H query rows (token-major: one latent row is every head's
// key and value, so heads and tokens fold into one long row axis) are cut into
// tiles of 128 rows, the cached positions into tiles of 256 keys. A pair of
// CTAs (cta_group::2) takes a row tile over a range of key tiles:
//   S[128 x 256] = Q[128 x 576] K[256 x 576]^T    36 products of K = 16
//   O[128 x 512] += P[128 x 256] V[256 x 512]     32 products, N = 256 each
// Why a pair: O for 128 rows in fp32 is all of one SM's tensor memory (512
// columns) and leaves none for S. With M = 128 over two CTAs each holds 64
// rows, its O in 256 columns (lanes 0-63 dims 0-255, lanes 64-127 dims
// 256-511 of the same rows) and two S buffers in the other 256, so the scores
// of the next tile are computed while the softmax of this one runs. N = 256 is
// what the pair needs for its full rate (a product of M = 128 takes 64 clocks
// at N = 128 and at N = 256, measured).
//
// Work is split evenly whatever the lengths: the units (row tile, key tile) of
// all requests form one line, and each of the SMs' pairs takes an equal
// stretch of it. A row tile cut by a stretch's end leaves partial sums in the
// workspace, which chunk_merge_kernel joins in order (no atomics: results do
// not depend on timing).
//
// Measured on GB300: 2048 tokens x 128 heads over 8192 bf16 positions 2.5 to
// 2.6 ms back to back, 0.82 to 0.86 of the measured bf16 burst rate, and 2.43 ms,
// 0.88, as one launch behind an L2 flush, which lets the power recover (bound by
// the products and their issue); 32 single tokens x 128 heads over 32,768
// positions each 280 us, 4.3 TB/s (only the K stages come from HBM, and the ring
// does not reach over the V stages between them); one token x 16 heads over 4096
// positions 19 us (latency: plan, first loads, softmax, epilogue, merge). A row
// tile of one key tile more costs a pair 6 us, a key tile more in the row tile it
// has 2 to 4: a row tile is drained before the next one's scores begin.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "cache.cuh"
#include "chunk_plan.h"

namespace dsakv {
namespace {

constexpr int kRowsCta = 64;   // the rows of a tile that each CTA of the pair holds
constexpr int kBlocks = 9;     // 64-wide blocks of the 576 dims
constexpr uint32_t kQBlock = kRowsCta * 128;     // 64 rows x 64 dims
constexpr uint32_t kQBytes = kBlocks * kQBlock;  // 72 KB, resident for a row tile
constexpr uint32_t kPBlock = kRowsCta * 128;     // 64 rows x 64 keys
constexpr uint32_t kPBytes = 4 * kPBlock;        // 64 rows x 256 keys
constexpr uint32_t kStageBytes = 16384;  // K: 128 keys x 64 dims; V: 64 keys x 2 x 64 dims
constexpr uint32_t kVBox = 64 * 128;     // V: 64 keys x 64 dims
constexpr uint32_t kBarBytes = 2944;
// Warp roles. bf16 rows: warps 0..7 softmax, 8..10 load by TMA (every third
// stage each), 11 issues the products. 8-bit rows: warps 0..3 softmax, 4..11
// convert (every eighth half of a stage each), 12 walks the work for them and
// loads Q, 15 issues the products; 13 and 14 fill the warpgroup.
constexpr int kTmaWarps = 3, kConvertWarps = 8;
constexpr int kPhases = 3;  // 8-bit rows: phase records on their way to the converting warps
constexpr uint32_t kRawUnit = 4096;  // 64 keys x 64 codes
template <int kFmt>
struct Layout {
  static constexpr bool k8 = kFmt == DSA_CACHE_E4M3;
  static constexpr int kSoftmaxWarps = k8 ? 4 : 8;
  static constexpr int kParts = kSoftmaxWarps / 4;  // threads of a TMEM lane
  static constexpr int kLoaders = k8 ? kConvertWarps + 3 : kTmaWarps;
  static constexpr int kMmaWarp = kSoftmaxWarps + kLoaders;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kStages = k8 ? 4 : 7;
  static constexpr uint32_t kRawBytes = k8 ? kConvertWarps * kRawUnit : 0;
  static constexpr uint32_t kSmem =
      kQBytes + kPBytes + kStages * kStageBytes + kRawBytes + kBarBytes;
  static_assert(kSmem <= 227 * 1024, "dynamic shared memory of one CTA");
  // Registers a thread after the split, of 384 x 168, or 512 x 128, at launch:
  // such that little spills, because nearly all of the L1 is shared memory and
  // what is spilled comes back at L2's distance (bf16 rows, 88 bytes spilled by
  // the loaders at 104 registers: 2680 against 2540 us at 2048 x 128 over 8192).
  // The kernel of bf16 rows spills nothing. That of 8-bit rows stores 120 bytes
  // and loads 220, none of them in the converting warps (without these the count
  // stays as it is, without the softmax's code it is zero).
  static constexpr int kSoftmaxRegs = k8 ? 200 : 176, kConvertRegs = 104, kLastRegs = k8 ? 104 : 152;
  static constexpr int kConvertThreads = kThreads - 32 * kSoftmaxWarps - 128;
  static_assert(32 * kSoftmaxWarps * kSoftmaxRegs + kConvertThreads * kConvertRegs +
                        128 * kLastRegs <= kThreads * (k8 ? 128 : 168), "register split");
};
constexpr int kMaxStages = 7;
constexpr int kMaxPairs = 80;
constexpr uint32_t kOCol = 256;  // TMEM columns: S buffers 0..127 and 128..255, O 256..511
constexpr uint64_t kWaitLimit = 2000000000ull;  // 2 s of global timer per wait
constexpr uint64_t kDrainNs = 2000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The running maximum follows only when a tile's exceeds it by this much (in
// powers of two): weights then stay below 2^8, which costs bf16 and the fp32
// sums no precision, and O is seldom rescaled.
constexpr float kSlack = 8.f;

// 8-bit rows: what the converting warps need to know of a phase (a key tile's
// K units and the V units of the tile before it).
struct Phase {
  int slot[16];  // of the tile's 16-key steps
  int units;     // of the phase; -1: no more
  int k_units;   // the first of them
  int rest;      // keys of the context from the tile on
};

struct Bars {
  uint64_t full[kMaxStages];   // even CTA: a stage's parts in both CTAs have landed
  // both: the products reading the stage are done; a place's uses alternate
  // between two barriers
  uint64_t empty[2][kMaxStages];
  uint64_t q_full;          // even CTA: Q of the row tile in both CTAs
  uint64_t q_empty;         // both: the row tile's last score product is done
  uint64_t s_full[2];       // both: a tile's scores are complete
  uint64_t p_full;          // even CTA: P written and S read in both CTAs
  uint64_t pv_done;         // both: a tile's value products are complete
  uint64_t phase_full[kPhases], phase_empty[kPhases];
  Phase phase[kPhases];
  uint64_t raw[kConvertWarps];  // a converting warp's unit of codes
  uint64_t drain;
  uint64_t sum[16];
  uint32_t tmem_slot;
  int abort;
  int start_b, start_j, start_u;  // where the pair's stretch of work begins
  int64_t count;                  // and its length in units
  float red[2][2][kRows];         // exchange between a row's threads
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

struct Args {
  const uint8_t* q;
  int64_t q_stride;  // bytes between tokens
  bool q_dense;      // the tokens lie side by side: Q by TMA
  const int32_t* cu_q;
  int T, B, H;
  const uint8_t* cache;
  int64_t pages;
  const int32_t* block_table;
  int64_t table_stride;
  int page_shift;
  int max_ctx;  // positions that the table has room for, at most kMaxCtx
  const int32_t* ctx_len;
  bool causal;
  float scale_log2;  // |scale| log2(e)
  bool negate;       // scale < 0
  __nv_bfloat16* out;
  float* lse;
  int4* meta;    // [pairs][2]: {first output row, rows, flags, 0} of a pair's partial row tiles
  float2* ml;    // [pairs][2][part_rows]: running maximum (log2) and sum
  float* opart;  // [pairs][2][part_rows][512]
  int part_rows;
  int pairs;
  uint64_t wait_ns;
  int32_t* err;
};
constexpr uint32_t kIdescNegateA = 1u << 13;
constexpr int kStarts = 1, kEnds = 2;  // meta flags: holds the row tile's first / last keys

// One request of the arguments, its values brought into range.
__device__ __forceinline__ Request request(const Args& a, int b) {
  Request r;
  r.q0 = min(max(__ldg(a.cu_q + b), 0), a.T);
  r.n = max(min(__ldg(a.cu_q + b + 1), a.T) - r.q0, 0);
  r.ctx = min(max(__ldg(a.ctx_len + b), 0), a.max_ctx);
  return r;
}

// The pair's stretch of the line of all units: thread-per-request sums, then
// the request, row tile and key tile that the stretch begins in.
__device__ __forceinline__ void plan(const Args& a, Bars* bars, int pair) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  auto units_of = [&](int b) -> int64_t {
    if (b >= a.B) return 0;
    const Request r = request(a, b);
    return r.n ? units_before(a.H, a.causal, r, row_tiles(a.H, r), row_tiles(a.H, r)) : 0;
  };
  // inclusive scan over the block; *all gets the sum
  auto scan = [&](int64_t v, int64_t* all) -> int64_t {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += o;
    }
    if (lane == 31) bars->sum[warp] = v;
    __syncthreads();
    *all = 0;
#pragma unroll 1
    for (int w = 0; w < threads >> 5; ++w) {
      if (w < warp) v += bars->sum[w];
      *all += bars->sum[w];
    }
    __syncthreads();
    return v;
  };
  // (one request a thread: its sum and its place in the scan are the same)
  const bool small = a.B <= threads;
  int64_t mine = 0, total;
#pragma unroll 1
  for (int b = tid; b < a.B; b += threads) mine += units_of(b);
  int64_t inc = scan(mine, &total);
  const Stretch st = stretch_of(total, a.pairs, pair);
  const int64_t from = st.from, count = st.count;
  if (tid == 0) bars->count = count;
  int64_t base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B && base <= from && count; b0 += threads) {
    const int b = b0 + tid;
    int64_t u = mine, all = total;
    if (!small) {
      u = units_of(b);
      inc = scan(u, &all);
    }
    const int64_t before = base + inc - u;
    if (u && from >= before && from < before + u) {
      const Place at = place_of(a.H, a.causal, request(a, b), from - before);
      bars->start_b = b;
      bars->start_j = at.j;
      bars->start_u = at.u;
    }
    base += all;
  }
  __syncthreads();
}

// Reports lengths out of range (once per launch).
__device__ __forceinline__ void check_lengths(const Args& a) {
#pragma unroll 1
  for (int b = threadIdx.x; b < a.B; b += int(blockDim.x)) {
    const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), ctx = __ldg(a.ctx_len + b);
    if (c0 < 0 || c1 < c0 || c1 > a.T) report(a.err, TS_DEVERR_ORDER);
    if (ctx < 0 || ctx > a.max_ctx) report(a.err, TS_DEVERR_CTX);
  }
}

// 2^x on the special-function unit (relative error far below the bf16
// rounding the weights then get).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16_zfill(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// Barrier of the softmax warps (named barrier 1).
template <int kThreads>
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}
// The same, and whether `ok` holds in every thread of them.
template <int kThreads>
__device__ __forceinline__ bool softmax_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, r;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred r, 1, %2, p;\n selp.u32 %0, 1, 0, r;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "n"(kThreads)
      : "memory");
  return all != 0;
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 8 bf16 values times a power of two.
__device__ __forceinline__ uint4 scaled(const uint4& x, float f) {
  const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
  auto mul = [&](uint32_t v) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), f2);
    return *reinterpret_cast<const uint32_t*>(&y);
  };
  return make_uint4(mul(x.x), mul(x.y), mul(x.z), mul(x.w));
}

// 16 e4m3 codes times 2^-120 f as bf16 values (f is 2^120 times the codes'
// scale). Two codes are spread over a word's halves, each below copies of its
// sign; shifted by 4 and masked, sign, exponent and mantissa bits lie in a
// bf16's places. A subnormal code becomes a bf16 subnormal of the same value,
// so no code is special but NaN (which the cache may not hold below ctx_len).
// 8 instructions for four codes; through the conversions to half and float it
// is 12.
__device__ __forceinline__ void widen_codes(const uint4& c, float f, uint4 (&o)[2]) {
  // (bit 3 of a byte's selector takes its sign in all eight bits)
  auto spread = [](uint32_t w, uint32_t bytes) {
    uint32_t x;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(x) : "r"(w), "r"(bytes));
    return (x << 4) & 0x87f087f0u;
  };
  auto low = [&](uint32_t w) { return spread(w, 0x9180); };
  auto high = [&](uint32_t w) { return spread(w, 0xb3a2); };
  o[0] = scaled(make_uint4(low(c.x), high(c.x), low(c.y), high(c.y)), f);
  o[1] = scaled(make_uint4(low(c.z), high(c.z), low(c.w), high(c.w)), f);
}

struct Maps {
  CUtensorMap q;     // [T H rows][9 blocks of 64], box 64 rows x 9 blocks
  CUtensorMap k;     // cache rows, box min(page, 128) rows x 1 block; 8-bit rows: their rope
                     // part, box min(page, 64) rows
  CUtensorMap v;     // cache rows, box min(page, 64) rows x 2 blocks (1 below 64)
  CUtensorMap code;  // 8-bit rows: the codes, box min(page, 64) rows x 64
};

// What the loading warps share.
struct Loader {
  const Args& a;
  const Maps& maps;
  Bars* bars;
  uint8_t *q_tile, *ring, *raw;
  uint32_t rank, q_full, full;  // cluster addresses of the even CTA's barriers
  int lane;
  bool el;  // this lane issues
  volatile int* abort;
  // 16-key steps that one TMA box of a K stage and of 64 keys covers
  int k_step, v_step;

  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return mbar_warp_wait<false>(bar, parity, abort, a.wait_ns);
  }
  // The place of a stage's use number `wrap` is free once the use before is
  // consumed. Uses alternate between two barriers, so a warp that has not
  // looked at this place for two uses is still told apart (a barrier's parity
  // tells two phases): its stages may be up to 2 * kStages apart.
  __device__ __forceinline__ bool wait_free(uint32_t s, uint32_t wrap) {
    return wrap == 0 || wait(&bars->empty[(wrap - 1) & 1][s], ((wrap - 1) >> 1) & 1);
  }
  // The slot of every 16-key step of a segment's key tile t: lanes 0..15 (-1:
  // no such page; keys past the context need none). In two halves: the loaders
  // of bf16 rows read the table's entries a tile before they use them.
  __device__ __forceinline__ bool needs(const Segment& g, int t) {
    return lane < 16 && t < g.t1 && t * kKeys + lane * 16 < g.r.ctx;
  }
  __device__ __forceinline__ int pages_of(const Segment& g, int t) {
    if (!needs(g, t)) return -1;
    return __ldg(a.block_table + g.b * a.table_stride + ((t * kKeys + lane * 16) >> a.page_shift));
  }
  __device__ __forceinline__ int slots_of(const Segment& g, int t, int64_t page) {
    if (!needs(g, t)) return -1;
    if (page < 0 || page >= a.pages) {
      report(a.err, TS_DEVERR_SLOT_RANGE);
      return -1;
    }
    const int key = t * kKeys + lane * 16;
    return static_cast<int>((page << a.page_shift) + (key & ((1 << a.page_shift) - 1)));
  }
  // Q of a row tile that starts at output row `row0`: by TMA (rows past the
  // tile's are other rows' values, or zeros past the last; their scores are
  // never used) ...
  __device__ __forceinline__ void q_by_tma(int row0, int rows, uint32_t bar) {
    const bool any = int(rank) * kRowsCta < rows;
    if (!el) return;
    if (any) {
      mbar_expect_tx_cluster(bar, kQBytes);
      tma_load_3d_pair(q_tile, &maps.q, bar, 0, row0 + rank * kRowsCta, 0);
    } else {
      mbar_arrive_cluster(bar);
    }
  }
  // ... or, tokens further apart, row by row by `warps` warps.
  __device__ __forceinline__ void q_by_copy(int row0, int rows, int w, int warps) {
#pragma unroll 1
    for (int i = w; i < kRowsCta; i += warps) {
      const int rr = rank * kRowsCta + i;
      const bool valid = rr < rows;
      const int row = row0 + (valid ? rr : 0);
      const uint8_t* src =
          a.q + int64_t(row / a.H) * a.q_stride + int64_t(row % a.H) * DSA_ROW_BYTES;
#pragma unroll 1
      for (int c = lane; c < DSA_ROW_CHUNKS; c += 32)
        cp_async16_zfill(q_tile + (c >> 3) * kQBlock + i * 128 + (((c & 7) ^ (i & 7)) << 4),
                         src + c * 16, valid);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  // K stage: this CTA's 128 keys of a tile, 64 dims of block kb; box i of the
  // tile starts at slot[i]. (Unrolled: a TMA costs its warp 50 clocks so, and
  // 97 in a loop that shuffles its slot first.)
  struct KBoxes {
    int slot[8];
    uint32_t bytes;
  };
  __device__ __forceinline__ KBoxes k_boxes(int slots) {
    KBoxes k;
    uint32_t boxes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      k.slot[i] = __shfl_sync(0xffffffffu, slots, rank * 8 + i);
      if (i & (k_step - 1)) k.slot[i] = -1;
      boxes += k.slot[i] >= 0;
    }
    k.bytes = boxes * k_step * 2048;
    return k;
  }
  __device__ __forceinline__ void k_by_tma(const KBoxes& k, int kb, uint8_t* dst, uint32_t bar) {
    if (!el) return;
    mbar_expect_tx_cluster(bar, k.bytes);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k.slot[i] >= 0) tma_load_3d_pair(dst + i * 2048, &maps.k, bar, 0, k.slot[i], kb);
  }
  // V stage: 64 keys from key0 on (group g of the tile), dims of blocks kb, kb + 1.
  __device__ __forceinline__ void v_by_tma(int slots, int key0, int ctx, int g, int kb,
                                           uint8_t* dst, uint32_t bar) {
    const bool gaps = __any_sync(0xffffffffu, lane >> 2 == g && slots < 0);
    if (key0 + 64 > ctx || gaps) {
      // V rows that are not the request's must be zeros: their weights are,
      // but the rows may hold anything, and 0 times NaN is NaN
#pragma unroll 4
      for (int i = 0; i < 32; ++i) {
        const int row = i * 2 + (lane >> 4), c = lane & 15;  // a row's 16 pieces
        int slot = __shfl_sync(0xffffffffu, slots, g * 4 + (row >> 4));
        const bool valid = key0 + row < ctx && slot >= 0;
        slot = max(slot, 0) + (valid ? row & 15 : 0);
        cp_async16_zfill(dst + (c >> 3) * kVBox + row * 128 + (((c & 7) ^ (row & 7)) << 4),
                         a.cache + int64_t(slot) * DSA_ROW_BYTES + kb * 128 + c * 16, valid);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (el) mbar_arrive_cluster(bar);
      return;
    }
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = __shfl_sync(0xffffffffu, slots, g * 4 + i);
    if (!el) return;
    mbar_expect_tx_cluster(bar, kStageBytes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & (v_step - 1)) continue;
      tma_load_3d_pair(dst + i * 2048, &maps.v, bar, 0, slot[i], kb);
      if (v_step < 4) tma_load_3d_pair(dst + kVBox + i * 2048, &maps.v, bar, 0, slot[i], kb + 1);
    }
  }
};

// The stages of a segment in the order the products take them: for each tile
// t its nine K stages, then the V stages of tile t - 1 (64-key group v / 2,
// dims half v % 2). Stages of phase t of a segment:
__device__ __forceinline__ int stages_of(const Segment& g, int t) {
  return (t < g.t1 ? kBlocks : 0) + (t > g.t0 ? 2 * groups(g.end, t - 1) : 0);
}

// bf16 rows: warp w of kTmaWarps. (Whole pages sent to L2 two tiles ahead, so
// that a row's nine pieces come from there, made every case slower: the long
// prefetches hold the TMA unit up. 32 x 32,768 positions, one token: 402 us
// with them, 269 without.)
__device__ __forceinline__ void load_bf16(Loader& ld, Walk walk, int w) {
  constexpr int kStages = Layout<DSA_CACHE_BF16>::kStages;
  const Args& a = ld.a;
  Segment sg;
  static_assert(kTmaWarps <= 2 * kStages, "wait_free");
  uint32_t s = 0, wrap = 0, qn = 0;
  int turn = 0;  // whose stage is next
  bool ok = true;
  while (ok && walk.next(a, sg)) {
    int here = -1, now_page = ld.pages_of(sg, sg.t0), next_page = ld.pages_of(sg, sg.t0 + 1);
    if (w == 0 || !a.q_dense) {
      if (qn > 0) ok = ld.wait(&ld.bars->q_empty, (qn - 1) & 1);
      if (!ok) break;
      const int row0 = sg.r.q0 * a.H + sg.row0;
      if (a.q_dense) {
        ld.q_by_tma(row0, sg.rows, ld.q_full);
      } else {
        ld.q_by_copy(row0, sg.rows, w, kTmaWarps);
        fence_proxy_async_smem();
        __syncwarp();
        if (ld.el) mbar_arrive_cluster(ld.q_full);
      }
    }
    ++qn;
    for (int t = sg.t0; t <= sg.t1 && ok; ++t) {
      const bool scores = t < sg.t1;
      const int now = ld.slots_of(sg, t, now_page);
      now_page = next_page;
      next_page = ld.pages_of(sg, t + 2);
      const int n = stages_of(sg, t);
      const Loader::KBoxes k = ld.k_boxes(now);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        if (turn == w) {
          ok = ld.wait_free(s, wrap);
          if (ok) {
            uint8_t* dst = ld.ring + s * kStageBytes;
            const uint32_t bar = ld.full + s * 8;
            if (scores && i < kBlocks) {
              ld.k_by_tma(k, i, dst, bar);
            } else {
              const int v = scores ? i - kBlocks : i;
              ld.v_by_tma(here, (t - 1) * kKeys + (v >> 1) * 64, sg.r.ctx, v >> 1,
                          ld.rank * 4 + (v & 1) * 2, dst, bar);
            }
          }
        }
        if (++turn == kTmaWarps) turn = 0;
        if (++s == kStages) s = 0, ++wrap;
      }
      here = now;
    }
  }
}

// 8-bit rows: walks the pair's work for the converting warps, which have too
// few registers for it (what they spill comes back at L2's distance: nearly all
// of the L1 is shared memory here), and loads Q.
__device__ __forceinline__ void load_q_8bit(Loader& ld, Walk walk) {
  const Args& a = ld.a;
  Bars* bars = ld.bars;
  Segment sg;
  uint32_t qn = 0, at = 0, wrap = 0;
  bool ok = true;
  auto publish = [&](int slots, int units, int k_units, int rest) {
    if (wrap > 0) ok = ld.wait(&bars->phase_empty[at], (wrap - 1) & 1);
    if (!ok) return;
    Phase& p = bars->phase[at];
    if (ld.lane < 16) p.slot[ld.lane] = slots;
    if (ld.lane == 16) p.units = units;
    if (ld.lane == 17) p.k_units = k_units;
    if (ld.lane == 18) p.rest = rest;
    __syncwarp();
    if (ld.el) mbar_arrive(&bars->phase_full[at]);
    if (++at == kPhases) at = 0, ++wrap;
  };
  while (ok && walk.next(a, sg)) {
    int page = ld.pages_of(sg, sg.t0);
#pragma unroll 1
    for (int t = sg.t0; t <= sg.t1 && ok; ++t) {
      const int slots = ld.slots_of(sg, t, page);
      page = ld.pages_of(sg, t + 1);
      publish(slots, 2 * stages_of(sg, t), t < sg.t1 ? 2 * kBlocks : 0, sg.r.ctx - t * kKeys);
      if (t > sg.t0 || !ok) continue;
      // Q, behind the first phase: a converting warp asks for its next unit's
      // phase before it places a unit of the row tile before, and that tile's
      // last score products wait for those
      if (qn > 0) ok = ld.wait(&bars->q_empty, (qn - 1) & 1);
      if (!ok) break;
      ++qn;
      const int row0 = sg.r.q0 * a.H + sg.row0;
      if (a.q_dense) {
        ld.q_by_tma(row0, sg.rows, ld.q_full);
      } else {
        ld.q_by_copy(row0, sg.rows, 0, 1);
        fence_proxy_async_smem();
        __syncwarp();
        if (ld.el) mbar_arrive_cluster(ld.q_full);
      }
    }
  }
  if (ok) publish(-1, -1, 0, 0);
}

// 8-bit rows: warp w of kConvertWarps. A stage is two units, its halves of 64
// keys x 64 dims, dealt to the warps in turn; lane i takes the keys i and
// i + 32. A unit's codes come by TMA (64-byte swizzle: the lanes' reads of one
// piece of every row meet no bank twice) into the warp's raw space; once they
// are in registers the next unit's are sent for, and land while this one is
// converted. What bounds this kernel is the shared memory's bandwidth: of some
// 9500 clocks a tile, 5400 are wavefronts of its loads and stores (counted),
// and the products' operands and the codes' arrival add about 4200; the
// products by themselves take 4556. (Ten converting warps, or a ring of five
// stages, take the same time as eight and four. Codes loaded straight into
// registers, or widened before the wait for their place, took 1.2 to 1.5 times
// as long: the warps then spilled.)
__device__ __forceinline__ void load_codes(Loader& ld, int w) {
  constexpr int kStages = Layout<DSA_CACHE_E4M3>::kStages;
  static_assert(kConvertWarps <= 2 * kBlocks, "every warp has a unit of a row tile's first phase");
  static_assert(kConvertWarps == 2 * kStages, "a warp's units all go to one place");
  const Args& a = ld.a;
  Bars* bars = ld.bars;
  const int lane = ld.lane;
  uint8_t* raw = ld.raw + w * kRawUnit;
  uint64_t* raw_bar = &bars->raw[w];
  const uint32_t at = w >> 1, half = w & 1, bar = ld.full + at * 8;
  uint8_t* dst = ld.ring + at * kStageBytes + half * kVBox;
  const uint32_t read = lane * 64, read_x = (lane >> 1 & 3) << 4;
  const uint32_t write = lane * 128, write_x = (lane & 7) << 4;
  // the unit in flight: whether it is rope, its valid 16-key steps, its keys of
  // the context, its slots and scales
  bool have = false, rope = false;
  uint32_t wrap = 0, valid = 0;
  int count = 0, unit_slots = -1;
  float scale0 = 0.f, scale1 = 0.f;
  uint32_t landed = 0;
  // this warp's next unit is number i of the phase's n, of which the first
  // k_units are K's; the slots and keys of the phase's tile and the one before
  bool over = false;
  int i = w, n = 0, k_units = 0, here = -1, now = -1, rest_here = 0, rest = 0;
  uint32_t ph = 0, ph_parity = 0;
  for (;;) {
    bool ok = true;
    while (ok && !over && i >= n) {  // on to the phase that holds the next unit
      i -= n;
      here = now;
      rest_here = rest;
      ok = ld.wait(&bars->phase_full[ph], ph_parity);
      const Phase& p = bars->phase[ph];
      n = p.units;
      k_units = p.k_units;
      rest = p.rest;
      now = lane < 16 ? p.slot[lane] : -1;
      over = n < 0;
      __syncwarp();
      if (ld.el) mbar_arrive(&bars->phase_empty[ph]);
      if (++ph == kPhases) ph = 0, ph_parity ^= 1;
    }
    if (!ok) break;
    if (over && !have) break;

    // the unit in flight: its codes into registers
    uint4 code[8];
    float f0 = scale0, f1 = scale1;
    if (have && !rope) {
      if (!ld.wait(raw_bar, landed & 1)) break;
      ++landed;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        code[k] = *reinterpret_cast<const uint4*>(raw + read + (k >> 2) * 2048 +
                                                  (((k & 3) << 4) ^ read_x));
      if (count < 64 || valid != 15) {
        // keys that are not the request's: codes of 0 and a scale that is no NaN
        const bool in0 = lane < count && (valid >> (lane >> 4) & 1);
        const bool in1 = lane + 32 < count && (valid >> (2 + (lane >> 4)) & 1);
        f0 = in0 ? f0 : 0.f;
        f1 = in1 ? f1 : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (!(k < 4 ? in0 : in1)) code[k] = make_uint4(0, 0, 0, 0);
      }
    }
    __syncwarp();

    // the next one's sent for
    bool next_rope = false;
    uint32_t next_valid = 0;
    int next_count = 0, slots = -1;
    if (!over) {
      int v = i >> 1, step, kb;
      if (i < k_units) {
        slots = now;
        step = ld.rank * 8 + half * 4;
        next_count = rest - int(ld.rank) * 128 - int(half) * 64;
        kb = v;
        next_rope = v == kBlocks - 1;
      } else {
        v -= k_units >> 1;  // 64-key group v / 2, dims half v % 2
        slots = here;
        step = (v >> 1) * 4;
        next_count = rest_here - (v >> 1) * 64;
        kb = ld.rank * 4 + (v & 1) * 2 + half;
      }
      next_count = min(max(next_count, 0), 64);
      next_valid = __ballot_sync(0xffffffffu, slots >= 0) >> step & 15;
      // (from here on lanes 0..3 hold the unit's slots)
      slots = __shfl_sync(0xffffffffu, slots, (step + lane) & 31);
      if (!next_rope) {
        const uint32_t boxes = next_valid & (ld.v_step == 4 ? 1u : ld.v_step == 2 ? 5u : 15u);
        if (ld.el) {
          if (boxes) mbar_expect_tx(raw_bar, __popc(boxes) * ld.v_step * 1024);
          else mbar_arrive(raw_bar);
        }
#pragma unroll 1
        for (int k = 0; k < 4; k += ld.v_step) {
          const int at = __shfl_sync(0xffffffffu, slots, k);
          if (ld.el && at >= 0) tma_load_3d(raw + k * 1024, &ld.maps.code, raw_bar, kb * 64, at, 0);
        }
        // (without a condition, which would wait for the values here)
        const int slot0 = max(__shfl_sync(0xffffffffu, slots, lane >> 4), 0) + (lane & 15);
        const int slot1 = max(__shfl_sync(0xffffffffu, slots, 2 + (lane >> 4)), 0) + (lane & 15);
        const uint8_t* scales = a.cache + TS_D_LATENT + (kb >> 1) * 4;
        scale0 = __ldg(reinterpret_cast<const float*>(scales + int64_t(slot0) * kE4m3RowBytes));
        scale1 = __ldg(reinterpret_cast<const float*>(scales + int64_t(slot1) * kE4m3RowBytes));
      }
    }

    // the unit in flight: into its place
    if (have) {
      if (!ld.wait_free(at, wrap++)) break;
      if (rope) {  // bf16 as it is, by TMA
        const uint32_t boxes = valid & (ld.v_step == 4 ? 1u : ld.v_step == 2 ? 5u : 15u);
        if (ld.el) mbar_expect_tx_cluster(bar, __popc(boxes) * ld.v_step * 2048);
#pragma unroll 1
        for (int k = 0; k < 4; k += ld.v_step) {
          const int slot = __shfl_sync(0xffffffffu, unit_slots, k);
          if (slot >= 0 && ld.el) tma_load_3d_pair(dst + k * 2048, &ld.maps.k, bar, 0, slot, 0);
        }
      } else {
        // (2^120 scale is past bf16's range for a scale above 2^7: those codes
        // get their scale in a second product)
        const bool big = __any_sync(0xffffffffu, fmaxf(f0, f1) > 128.f);
        const float g0 = big ? 0x1p120f : f0 * 0x1p120f, g1 = big ? 0x1p120f : f1 * 0x1p120f;
        auto place = [&](int k) -> uint4* {
          return reinterpret_cast<uint4*>(dst + write + (k >> 3) * 4096 +
                                          (((k & 7) << 4) ^ write_x));
        };
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint4 o[2];
          widen_codes(code[k], k < 4 ? g0 : g1, o);
          *place(2 * k) = o[0];
          *place(2 * k + 1) = o[1];
        }
        if (big) {
#pragma unroll 1
          for (int k = 0; k < 16; ++k) *place(k) = scaled(*place(k), k < 8 ? f0 : f1);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (ld.el) mbar_arrive_cluster(bar);
      }
    }
    have = !over;
    rope = next_rope;
    valid = next_valid;
    count = next_count;
    unit_slots = slots;
    i += kConvertWarps;
  }
}

template <int kFmt>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Layout<kFmt>::kThreads, 1)
    chunk_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
  using Lay = Layout<kFmt>;
  constexpr int kStages = Lay::kStages, kMmaWarp = Lay::kMmaWarp;
  constexpr int kSoftmaxWarps = Lay::kSoftmaxWarps, kParts = Lay::kParts;
  constexpr int kCols = 128 / kParts;  // score columns of a softmax thread
  extern __shared__ __align__(1024) uint8_t q_tile[];  // (swizzled tiles: 1024-byte aligned)
  uint8_t* p_tile = q_tile + kQBytes;
  uint8_t* ring = p_tile + kPBytes;
  uint8_t* raw = ring + kStages * kStageBytes;
  Bars* bars = reinterpret_cast<Bars*>(raw + Lay::kRawBytes);
  volatile int* abort = &bars->abort;
  const int pair = blockIdx.x >> 1;
  const uint32_t rank = cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wait_ns = a.wait_ns;

  launch_dependents();
  if (threadIdx.x == 32) {
    if (a.q_dense) tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(Lay::k8 ? &maps.code : &maps.v);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], Lay::k8 ? 4 : 2);
      mbar_init(&bars->empty[0][s], 1);
      mbar_init(&bars->empty[1][s], 1);
    }
    mbar_init(&bars->q_full, Lay::k8 || a.q_dense ? 2 : 2 * kTmaWarps);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->s_full[0], 1);
    mbar_init(&bars->s_full[1], 1);
    mbar_init(&bars->p_full, 2 * Lay::kSoftmaxWarps);
    mbar_init(&bars->pv_done, 1);
    for (int i = 0; i < kConvertWarps; ++i) mbar_init(&bars->raw[i], 1);
    for (int i = 0; i < kPhases; ++i) {
      mbar_init(&bars->phase_full[i], 1);
      mbar_init(&bars->phase_empty[i], kConvertWarps);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&bars->tmem_slot, 512);
    tmem_relinquish_pair();
  }
  // (the cluster meets over the plan: the barriers are there, and the tensor
  // memory's address is read behind the plan's own barriers)
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  if (blockIdx.x == 0) check_lengths(a);
  plan(a, bars, pair);
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;

  auto make_loader = [&]() -> Loader {
    const int k_step = min(8, (1 << a.page_shift) >> 4);
    return Loader{a, maps, bars, q_tile, ring, raw, rank, dsmem_addr(&bars->q_full, 0),
                  dsmem_addr(&bars->full[0], 0), lane, elect_one(), abort, k_step, min(4, k_step)};
  };
  Walk walk{bars->start_b, bars->start_j, bars->start_u, bars->count};
  Segment sg;
  if (warp < kSoftmaxWarps) {
    // ---------------- softmax and epilogue: kParts threads per TMEM lane ----------------
    // Lanes r and r + 64 hold row r: of S keys 0..127 and 128..255, of O dims
    // 0..255 and 256..511; of either, a lane's threads take equal parts of the
    // columns.
    regs_inc<Lay::kSoftmaxRegs>();
    const int L = (warp & 3) * 32 + lane, r = L & 63, half = L >> 6, part = warp >> 2;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t p_full = dsmem_addr(&bars->p_full, 0);
    if (rank == 0 && threadIdx.x == 0)
      a.meta[pair * 2] = a.meta[pair * 2 + 1] = make_int4(-1, 0, 0, 0);
    uint32_t tg = 0;  // tiles so far
    bool ok = true;
    while (ok && walk.next(a, sg)) {
      const int rr = rank * kRowsCta + r;  // row within the tile
      int limit = 0;
      if (rr < sg.rows)
        limit = a.causal ? max(0, sg.r.ctx - sg.r.n + (sg.row0 + rr) / a.H + 1) : sg.r.ctx;
      // (the sum in parts of 64 columns, whatever the threads: both formats then
      // add in one order, and equal rows give equal results)
      float m = -INFINITY, l64[kCols / 64] = {};
      for (int t = sg.t0; t < sg.t1; ++t, ++tg) {
        const uint32_t ts = trow + (tg & 1) * 128 + part * kCols;
        const int nv = min(max(limit - t * kKeys - half * 128 - part * kCols, 0), kCols);
        const bool whole = __all_sync(0xffffffffu, nv == kCols);
        if (ok) ok = mbar_warp_wait<false>(&bars->s_full[tg & 1], (tg >> 1) & 1, abort, wait_ns);
        // the thread's scores, once, into registers
        uint32_t x[kCols / 32][32];
        float mx = -INFINITY;
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) tmem_ld32(ts + 32 * c, x[c]);
          tmem_wait_ld();
          if (!whole) {
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (i >= nv) x[i >> 5][i & 31] = __float_as_uint(-INFINITY);
          }
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < kCols; i += 2)
            m4[(i >> 1) & 3] =
                fmaxf(fmaxf(m4[(i >> 1) & 3], __uint_as_float(x[i >> 5][i & 31])),
                      __uint_as_float(x[i >> 5][(i & 31) + 1]));
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          mx *= a.scale_log2;
        }
        bars->red[tg & 1][part][L] = mx;
        softmax_sync<32 * Lay::kSoftmaxWarps>();
        {
          const auto& e = bars->red[tg & 1];
#pragma unroll
          for (int k = 0; k < kParts; ++k) mx = fmaxf(mx, fmaxf(e[k][r], e[k][r + 64]));
        }
        // the tile before this one is in O, and its P read. (Only now the weights:
        // they go to P as they come, and the products are busy with the next
        // tile's scores meanwhile. Held in registers over this wait they made the
        // threads spill, and what is spilled comes back at L2's distance.)
        if (ok && tg > 0) ok = mbar_warp_wait<false>(&bars->pv_done, (tg - 1) & 1, abort, wait_ns);
        if (!ok) continue;  // the barrier above stays matched in every warp
        const bool moves = mx > m + kSlack;
        const float f = moves ? fast_exp2(m - mx) : 1.f;
        if (moves) m = mx;
        if (t > sg.t0 && __any_sync(0xffffffffu, moves)) {
          tc_fence_after();
          uint32_t v[32];
#pragma unroll 1
          for (int c = part * (256 / kParts); c < (part + 1) * (256 / kParts); c += 32) {
            tmem_ld32(trow + kOCol + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st32(trow + kOCol + c, v);
          }
          tmem_wait_st();
        }
        // The weights are rounded to bf16 for the value products, half a step of
        // 2^-8 each, which is what the tensor cores' bf16 rate takes (as in the
        // sparse decode): 2048 x 128 over 8192, the outputs' error against 64 bits
        // goes from 0.0016 of their size, the rounding of the outputs themselves,
        // to 0.0018. Their sum adds them unrounded, in fp32.
        const float mu = m == -INFINITY ? 0.f : m;
        uint8_t* prow = p_tile + (half * 2 + part * (kCols / 64)) * kPBlock + r * 128;
#pragma unroll
        for (int k = 0; k < kCols / 64; ++k) {
          float l4[4] = {};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t packed[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const int c = k * 64 + j * 8 + i;
              const float p0 = fast_exp2(fmaf(__uint_as_float(x[c >> 5][c & 31]), a.scale_log2, -mu));
              const float p1 =
                  fast_exp2(fmaf(__uint_as_float(x[c >> 5][(c & 31) + 1]), a.scale_log2, -mu));
              l4[i & 3] += p0;
              l4[(i & 3) + 1] += p1;
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
              packed[i / 2] = *reinterpret_cast<const uint32_t*>(&h2);
            }
            *reinterpret_cast<uint4*>(prow + k * kPBlock + ((j ^ (r & 7)) << 4)) =
                make_uint4(packed[0], packed[1], packed[2], packed[3]);
          }
          l64[k] = l64[k] * f + ((l4[0] + l4[1]) + (l4[2] + l4[3]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full);
      }
      // the row tile's sums: O from TMEM, normalised into the output or raw
      // into the workspace
#pragma unroll
      for (int k = 0; k < kCols / 64; ++k) bars->red[tg & 1][part + k][L] = l64[k];
      softmax_sync<32 * Lay::kSoftmaxWarps>();
      float l;
      {
        const auto& e = bars->red[tg & 1];
        l = (e[0][r] + e[0][r + 64]) + (e[1][r] + e[1][r + 64]);
      }
      if (ok) ok = mbar_warp_wait<false>(&bars->pv_done, (tg - 1) & 1, abort, wait_ns);
      ok = softmax_all<32 * Lay::kSoftmaxWarps>(ok);  // the same in every warp: all go on, or none
      if (!ok) break;
      tc_fence_after();
      const int64_t grow = int64_t(sg.r.q0) * a.H + sg.row0 + rr;  // output row
      const bool valid = rr < sg.rows;
      // Through shared memory (P's, which is free now), 512 bytes of every row
      // a pass, so that the stores are whole lines: a thread holds one row's
      // columns, and stores of 16 bytes at 32 rows each took 5 us a row tile.
      // Of a row's four segments of 128 dims a thread has one (or, one thread
      // a lane, two).
      const bool direct = sg.starts && sg.ends;
      const int slot = pair * 2 + (sg.starts ? 1 : 0);
      const int seg_bytes = direct ? 256 : 512;
      uint8_t* dst = direct ? reinterpret_cast<uint8_t*>(a.out) + (grow - r) * (DSA_DV * 2)
                            : reinterpret_cast<uint8_t*>(a.opart) +
                                  (int64_t(slot) * a.part_rows + rr - r) * (DSA_DV * 4);
      const bool empty = l == 0.f;  // no key (a NaN is kept)
      const float inv = empty ? 0.f : 1.f / l;
      const int mine = min(kRowsCta, sg.rows - int(rank) * kRowsCta);  // rows to store
#pragma unroll 1
      for (int pass = 0; pass < (direct ? 2 : 4); ++pass) {
#pragma unroll
        for (int k = 0; k < 2 / kParts; ++k) {
          const int seg = half * 2 + part + k;
          const uint32_t col = trow + kOCol + (part + k) * 128;
          uint8_t* stage = p_tile + r * 512 + seg * 128;
          auto put = [&](int piece, const uint4& x) {
            *reinterpret_cast<uint4*>(stage + ((piece ^ (r & 7)) << 4)) = x;
          };
          uint32_t v[32];
          if (direct) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tmem_ld32(col + pass * 64 + h * 32, v);
              tmem_wait_ld();
              uint32_t o[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                // (a row without a key has no O: zeros, whatever lies there)
                const float x0 = empty ? 0.f : __uint_as_float(v[2 * i]) * inv;
                const float x1 = empty ? 0.f : __uint_as_float(v[2 * i + 1]) * inv;
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(x0, x1);
                o[i] = *reinterpret_cast<const uint32_t*>(&h2);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                put(h * 4 + j, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
            }
          } else {
            tmem_ld32(col + pass * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              put(j, make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
          }
        }
        softmax_sync<32 * Lay::kSoftmaxWarps>();
#pragma unroll 2
        for (int i = warp; i < mine; i += kSoftmaxWarps)
          *reinterpret_cast<uint4*>(dst + int64_t(i) * seg_bytes * 4 + (lane >> 3) * seg_bytes +
                                    pass * 128 + (lane & 7) * 16) =
              *reinterpret_cast<const uint4*>(p_tile + i * 512 + (lane >> 3) * 128 +
                                              (((lane & 7) ^ (i & 7)) << 4));
        softmax_sync<32 * Lay::kSoftmaxWarps>();
      }
      if (valid && half == 0 && part == 0) {
        if (!direct) a.ml[int64_t(slot) * a.part_rows + rr] = make_float2(m, l);
        else if (a.lse) a.lse[grow] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      if (!direct && rank == 0 && threadIdx.x == 0)
        a.meta[slot] = make_int4(static_cast<int>(int64_t(sg.r.q0) * a.H + sg.row0), sg.rows,
                                 (sg.starts ? kStarts : 0) | (sg.ends ? kEnds : 0), 0);
      tc_fence_before();
    }
  } else if (Lay::k8 && warp < kSoftmaxWarps + kConvertWarps) {
    // ---------------- 8-bit rows: the K and V stages ----------------
    regs_dec<Lay::kConvertRegs>();
    const int w = warp - kSoftmaxWarps;
    Loader ld = make_loader();
    load_codes(ld, w);
  } else {
    // (one instruction for all of a warpgroup's warps)
    regs_dec<Lay::kLastRegs>();
    if (warp < kMmaWarp) {
      // ---------------- Q; bf16 rows: the K and V stages ----------------
      Loader ld = make_loader();
      if (!Lay::k8) load_bf16(ld, walk, warp - kSoftmaxWarps);
      else if (warp == kSoftmaxWarps + kConvertWarps) load_q_8bit(ld, walk);
    } else if (rank == 0) {
      // ---------------- MMA issuer (the even CTA's, for both) ----------------
      // a negative scale negates Q (its bit of the instruction descriptor)
      const uint32_t id_s =
          idesc_bf16_f32(kRows, kKeys, false, false) | (a.negate ? kIdescNegateA : 0u);
      const uint32_t id_pv = idesc_bf16_f32(kRows, 256, false, true);
      // descriptors of the first 16-wide step; later ones differ in the start
      // address (16-byte units, no carry out of its field)
      const uint64_t q_desc = smem_desc_sw128(smem_addr(q_tile), 16, 1024);
      const uint64_t p_desc = smem_desc_sw128(smem_addr(p_tile), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_addr(ring), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_addr(ring), kVBox, 1024);
      const bool el = elect_one();
      uint32_t s = 0, phase = 0, tg = 0, qn = 0;
      bool ok = true;
      // the next stage, in both CTAs
      auto landed = [&]() -> bool {
        if (!__all_sync(0xffffffffu, mbar_try_wait(&bars->full[s], phase)))
          ok = mbar_warp_wait<false>(&bars->full[s], phase, abort, wait_ns);
        tc_fence_after();
        return ok;
      };
      auto advance = [&]() {
        if (++s == kStages) s = 0, phase ^= 1;
      };
      while (ok && walk.next(a, sg)) {
        ok = mbar_warp_wait<true>(&bars->q_full, qn & 1, abort, wait_ns);
        ++qn;
        for (int t = sg.t0; t <= sg.t1 && ok; ++t) {
          if (t < sg.t1) {
            const uint32_t d = tmem + (tg & 1) * 128;
            // (unrolled: the issue of a stage's products has to stay below their own
            // 257 clocks; 2048 x 128 over 8192: 2565 -> 2490 us)
#pragma unroll 3
            for (int kb = 0; kb < kBlocks && landed(); ++kb) {
              const uint64_t qd = q_desc + kb * (kQBlock >> 4);
              const uint64_t kd = k_desc + s * (kStageBytes >> 4);
              if (el) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_bf16_pair(d, qd + kk * 2, kd + kk * 2, id_s, (kb | kk) != 0);
                tc_commit_pair(&bars->empty[phase][s]);
              }
              advance();
            }
            if (!ok) break;
            if (el) {
              tc_commit_pair(&bars->s_full[tg & 1]);
              if (t == sg.t1 - 1) tc_commit_pair(&bars->q_empty);
            }
            ++tg;
          }
          if (t > sg.t0) {
            // the tile before: tg counts one more when this one's scores were issued
            const uint32_t tp = t < sg.t1 ? tg - 2 : tg - 1;
            ok = mbar_warp_wait<true>(&bars->p_full, tp & 1, abort, wait_ns);
            if (!ok) break;
            tc_fence_after();
            const int g1 = groups(sg.end, t - 1);
            const bool first = t - 1 == sg.t0;
#pragma unroll 2
            for (int v = 0; v < 2 * g1 && landed(); ++v) {  // group v / 2, dims half v % 2
              const uint64_t pd = p_desc + (v >> 1) * (kPBlock >> 4);
              const uint64_t vd = v_desc + s * (kStageBytes >> 4);
              const uint32_t d = tmem + kOCol + (v & 1) * 128;
              if (el) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_bf16_pair(d, pd + kk * 2, vd + kk * (2048 >> 4), id_pv,
                                   !first || (v >> 1 | kk) != 0);
                tc_commit_pair(&bars->empty[phase][s]);
              }
              advance();
            }
            if (ok && el) tc_commit_pair(&bars->pv_done);
          }
        }
      }
    }
  }

  // ---------------- teardown ----------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  const bool aborted = bars->abort != 0;
  if (aborted) {
    if (threadIdx.x == 0) report(a.err, TS_DEVERR_TIMEOUT);
    // copies in flight land, and every tcgen05 operation issued completes,
    // before the CTA may leave
    if (threadIdx.x == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
    if (warp == kMmaWarp && rank == 0 && elect_one()) {
      tc_commit_pair(&bars->drain);
      mbar_wait_timed(&bars->drain, 0, kWaitLimit);
    }
    __syncthreads();
  }
  // (relaxed: nobody here reads the sums on their way, and every arrival sent to
  // the other CTA has been waited for, unless a wait gave up)
  if (aborted) cluster_arrive();
  else cluster_arrive_relaxed();
  cluster_wait();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Joins the partial sums of the row tiles that stretches of work have cut: the
// head (a pair's segment that holds a row tile's first keys) and the pairs
// after it up to the segment that holds its last,
//   out = sum_i w_i O_i / sum_i w_i l_i,  w_i = 2^(m_i - max m).
// A warp a row; pairs without a head leave at once.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) chunk_merge_kernel(const Args a) {
  wait_previous_kernel();
  const int pair = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 head = a.meta[pair * 2 + 1];
  const int r = blockIdx.y * kMergeWarps + warp;
  if (head.x < 0 || r >= head.y) return;
  // the segments: slot 1 of this pair, slot 0 of the next ones
  int parts = 0;
  for (int p0 = pair + 1; p0 < a.pairs && !parts; p0 += 32) {
    const int p = p0 + lane;
    const bool last = p < a.pairs && a.meta[p * 2].x >= 0 && (a.meta[p * 2].z & kEnds);
    const uint32_t who = __ballot_sync(0xffffffffu, last);
    if (who) parts = p0 + __ffs(who) - pair;
  }
  auto row_of = [&](int i) -> int64_t {
    return int64_t(i == 0 ? pair * 2 + 1 : (pair + i) * 2) * a.part_rows + r;
  };
  float mx = -INFINITY;
#pragma unroll 1
  for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, a.ml[row_of(i)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  const float base = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, acc[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) acc[c] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float2 e = i0 + lane < parts ? a.ml[row_of(i0 + lane)] : make_float2(-INFINITY, 0.f);
    const float w = exp2f(e.x - base);
    sum += w * e.y;
    const int n = min(parts - i0, 32);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float4* src = reinterpret_cast<const float4*>(a.opart + row_of(i0 + i) * DSA_DV) + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 x = __ldcs(src + 32 * c);
        acc[4 * c] += wi * x.x;
        acc[4 * c + 1] += wi * x.y;
        acc[4 * c + 2] += wi * x.z;
        acc[4 * c + 3] += wi * x.w;
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t row = int64_t(head.x) + r;
  uint2* dst = reinterpret_cast<uint2*>(a.out + row * DSA_DV) + lane;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[4 * c] * inv, acc[4 * c + 1] * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[4 * c + 2] * inv, acc[4 * c + 3] * inv);
    dst[32 * c] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                             *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// 3-D map over rows of `blocks` blocks of `inner` values: dims {inner, rows,
// blocks}; box {64, box_rows, box_blocks}. bf16 values swizzled by 128 bytes, or
// (codes) bytes swizzled by 64.
bool make_map(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t row_bytes,
              uint64_t inner, uint64_t blocks, uint32_t box_rows, uint32_t box_blocks,
              bool codes = false) {
  EncodeTiled enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {inner, rows, blocks};
  const cuuint64_t strides[2] = {row_bytes, 128};
  const cuuint32_t box[3] = {64, box_rows, box_blocks};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int part_rows(int T, int H) { return static_cast<int>(std::min(int64_t(T) * H, int64_t(kRows))); }

// The attention's launch; the maps and the merge are the caller's.
template <int kFmt>
ts_status launch_chunk(const Maps& maps, const Args& a, cudaStream_t stream) {
  using Lay = Layout<kFmt>;
  static std::atomic<uint64_t> smem_set{0};
  if (!raise_smem_limit(reinterpret_cast<const void*>(chunk_kernel<kFmt>), Lay::kSmem, smem_set))
    return TS_ERR_CUDA;
  chunk_kernel<kFmt><<<2 * a.pairs, Lay::kThreads, Lay::kSmem, stream>>>(maps, a);
  return launch_status();
}

}  // namespace
}  // namespace dsakv

using namespace dsakv;

extern "C" size_t sfa_chunk_workspace_size(int T, int B, int H) {
  if (T <= 0 || B <= 0 || H <= 0) return 0;
  const size_t slots = 2 * kMaxPairs, rows = slots * part_rows(T, H);
  return align256(slots * sizeof(int4)) + align256(rows * sizeof(float2)) + rows * DSA_DV * 4;
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
  if (H > 1024 || int64_t(T) * H >= INT_MAX - 127 || num_slots > INT_MAX)
    return TS_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
      ws_bytes < sfa_chunk_workspace_size(T, B, H))
    return TS_ERR_WORKSPACE;
  Args a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride * 2;
  a.q_dense = q_stride == int64_t(H) * DSA_D || T == 1;
  a.cu_q = cu_q;
  a.T = T;
  a.B = B;
  a.H = H;
  a.cache = static_cast<const uint8_t*>(cache);
  a.pages = num_slots / page_size;
  a.block_table = block_table;
  a.table_stride = table_stride;
  a.page_shift = __builtin_ctz(page_size);
  a.max_ctx = static_cast<int>(
      std::min(std::min(table_stride, int64_t(kMaxCtx)) * page_size, int64_t(kMaxCtx)));
  a.ctx_len = ctx_len;
  a.causal = causal != 0;
  // (above 0: a masked score, minus infinity, times 0 would be no number)
  a.scale_log2 = std::max(std::fabs(scale) * kLog2e, FLT_MIN);
  a.negate = scale < 0.f;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.part_rows = part_rows(T, H);
  a.pairs = std::max(1, std::min(kMaxPairs, sm_count() / 2));
  const size_t slots = 2 * kMaxPairs, rows = slots * a.part_rows;
  char* w = static_cast<char*>(ws);
  a.meta = reinterpret_cast<int4*>(w);
  w += align256(slots * sizeof(int4));
  a.ml = reinterpret_cast<float2*>(w);
  w += align256(rows * sizeof(float2));
  a.opart = reinterpret_cast<float*>(w);
  a.wait_ns = wait_limit_ns(kWaitLimit);
  a.err = err;
  Maps maps = {};
  bool made = !a.q_dense || make_map(&maps.q, q, int64_t(T) * H, DSA_ROW_BYTES, 64, kBlocks,
                                     kRowsCta, kBlocks);
  if (fmt == DSA_CACHE_BF16) {
    made = made &&
           make_map(&maps.k, cache, num_slots, DSA_ROW_BYTES, 64, kBlocks, std::min(page_size, 128),
                    1) &&
           make_map(&maps.v, cache, num_slots, DSA_ROW_BYTES, 64, kBlocks, std::min(page_size, 64),
                    page_size >= 64 ? 2 : 1);
    st = made ? launch_chunk<DSA_CACHE_BF16>(maps, a, stream) : TS_ERR_CUDA;
  } else {
    made = made &&
           make_map(&maps.k, a.cache + kE4m3Rope, num_slots, kE4m3RowBytes, 64, 1,
                    std::min(page_size, 64), 1) &&
           make_map(&maps.code, cache, num_slots, kE4m3RowBytes, TS_D_LATENT, 1,
                    std::min(page_size, 64), 1, true);
    st = made ? launch_chunk<DSA_CACHE_E4M3>(maps, a, stream) : TS_ERR_CUDA;
  }
  if (st != TS_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.pairs, (a.part_rows + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, chunk_merge_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return TS_ERR_CUDA;
  }
  return TS_OK;
}
