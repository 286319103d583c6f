// dsa_paged.cu - dense attention over the paged latent cache, one new token per request, and the
// attention weight each cached position receives (dsa_paged_attn, dsa_paged_attn_mass).
//
// For token t of request r, head h and position j of the token's range [a, b):
//   u_hj = sm_scale q_h . k_j, capped by cap * tanh(u / cap), minus slope_h |qpos - kpos_j|
//   out_h = sum_j softmax_j(u_h) k_j,  lse_h = log sum_j exp(u_hj)
//   mass_out[r, j] = mass[r, j] + sum_h exp(u_hj - lse_h)
// The latent row k_j is key and value of every head: a position costs 264 (FP8) or 512 (bf16) bytes
// and 4 * 256 operations per head, so with 64 heads a bf16 cache is bound by HBM and an FP8 one by
// HBM and the tensor core about equally. What a tile takes is set by its chains of hand-offs: 128 tokens x
// 32768 FP8 positions take 444 us (2.5 TB/s; 167 at HBM's rate), some 4100 cycles a tile. With parts of
// the work left out, when the whole took 453: 372 (no softmax arithmetic), 390 (next to no products), 343 (no
// copies and no widening), 271 (none of the three: the hand-offs between the warps alone). No unit is full,
// shared memory is the busiest: a product step of N = 64 reads 6 KB, all that its 48 cycles can carry, and
// with copies, widening and weights a tile moves some 2800 cycles' worth. 64 ragged bf16 requests, 144 MB of
// rows, take 50 us (2.9 TB/s; 21 at HBM's rate).
//
// Shape of the computation
//  * Transposed products: S^T[key, head] = K Q^T with M = 128 keys, N = 64 heads, then
//    O^T[column, head] += V^T P^T in two M = 128 halves of the 256 columns, V^T read MN-major from
//    the same K tile (tcgen05 kind::f16, bf16 operands, fp32 accumulators in tensor memory). A
//    token has at most 64 heads per pass: heads as M would leave half of the tensor core idle.
//  * FP8 rows: scores run on the e4m3 codes as they are (kind::f8f6f4), the bf16 query split into two
//    e4m3 terms per head, scaled by a power of two: hi + lo is the bf16 component for every component
//    within 2^9 of the head's largest, and off by at most 2^-17 of the largest otherwise. S keeps one
//    accumulator per scale tile and the fp32 scales multiply there. The value product takes the codes
//    widened to f16, which is exact and one conversion per two codes (to bf16 it is four instructions), and
//    one f16 weight matrix per scale tile: p * scale relative to a reference, the head's largest p * scale so far, 2^22 of normal range
//    below it. (The largest scale would not do: a row of large scale that a head ignores would take the
//    range from those it reads.) The first tile's reference is taken off the scores with the running
//    maximum, and the second's differs from it by about the same factor in all heads of a group, so a
//    weight is one product, p times a factor of the key. Where the heads differ by more, theirs come in
//    between the two tiles (128 x 32768 positions when it was tried: 430 us; 530 with a factor per head for
//    every weight). The references cost a row's first tile up to 2 us: 8 x 2112 positions take 27.8 us from
//    a graph, 25.7 with the largest scale as the reference. e4m3 weights (as two terms) would need no widening but lose what
//    many far positions add up to beside one strong one. So the keys are the exact products code * scale.
//  * Softmax with one thread per key and 16 heads: four groups of four warps, a warp per lane quarter of
//    tensor memory in each. The warps of a group share running maxima and synchronise among themselves. The
//    running maximum of a head is raised, and O and the sums rescaled, only when some score exceeds it by
//    2^20 (FP8: when some weight may leave the range of f16): p and its sums are floating point, so a stale
//    maximum costs no precision, and the exact path runs for a segment's first tile and almost never again.
//  * Persistent CTAs, one per SM. Each computes the same split from the lengths (they live on the
//    device): rows (token, group of 64 heads) cost their 128-position tiles plus a constant, and
//    CTA c takes the c-th of G equal parts of the total. A row cut by a border leaves unnormalised
//    parts in the workspace, which a second, dependent launch joins in the order of the parts.
//  * Warp roles: 0-15 softmax, 16 scheduler (walks the CTA's rows and finds the slots of each tile's
//    positions, up to eight tiles ahead), 17 score products, 18 value products, 19 query loads, 20-23
//    row loads, 24-27 FP8: query split and widening. Every wait is bounded. Every job has warps of its
//    own with no polling between jobs, and the arithmetic is on pairs. The registers are split anew after
//    the start (a spill in the loop would leave the L1 that the tiles leave over: a tile took 9500 cycles
//    with spills).
//  * bf16 tiles without a masked position come by TMA, in boxes of as many rows as a page and a tile
//    share; other bf16 tiles and FP8 rows (264 bytes: no tensor map takes that pitch) by cp.async
//    straight to their swizzled place. Either way every free stage of the ring holds loads in flight
//    and no register does. FP8: other warps widen the rows into a second ring while the softmax
//    of their tile runs.
//  * The mass kernel is the same without the value product: with the lse given, each key's thread
//    adds the weights of all 64 heads; four groups of four warps take tiles in turn.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "dsa_host.h"
#include "dsa_paged_split.h"
#include "dsa_paged_wait.cuh"
#include "dsa_ptx.cuh"

namespace dsa {
namespace paged {

constexpr int kD = 256;
constexpr int kMaxHeads = 128;
constexpr int kHG = 64;    // heads per row (MMA N)
constexpr int kBN = 128;   // positions per tile (MMA M)
constexpr int kSoftmaxWarps = 16;
constexpr int kWarpSched = 16, kWarpScore = 17, kWarpValue = 18, kWarpQuery = 19, kWarpLoad0 = 20, kWarpWiden0 = 24;
constexpr int kGroups = kSoftmaxWarps / 4;   // head groups
constexpr int kHW = kHG / kGroups;           // heads per group
constexpr int kLoadWarps = 4, kWidenWarps = 4;
constexpr int kLoadRows = kBN / kLoadWarps;
constexpr int kWarps = kWarpWiden0 + kWidenWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpRows = 256;     // rows whose costs one warp sums up, eight per lane
constexpr int kSegs = 8;           // segment ring depth
constexpr int kMaps = 8;           // tiles whose slots are known ahead
// Smallest page whose rows the scheduler prefetches into L2 (an eighth of a tile per request), FP8
// only. It shortens the start of short shares: 8 heads with a distance bias 45 us with it and 48 without
// when it was tried; 128 x 32768 positions took the same (488 and 487). bf16 tiles come by TMA in any
// case, and 64 ragged requests took 72 us with it, 66 without.
constexpr int kPrefetchPage = 16;
constexpr int kRowOverhead = 1;    // a row's start and end, in tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.402823466e38f;  // maximum of no score: below every finite one
// bf16: a score may exceed the running maximum by 2^20. FP8: by what the sums hold (2^55 and 2^64 of kOwn
// are finite together), and a weight p * scale the head's reference by what f16 holds, kMostWeight =
// 2^kWeightShift * 2^6 or so.
constexpr float kStale = 20.0f, kStaleF8 = 55.0f, kMostWeight = 65000.0f;
constexpr int kWeightShift = 10;
// FP8: the heads of a group share the second tile's factor while theirs lie within 2^kSpread of one another:
// the smallest of them leaves 2^(14 + kWeightShift - kSpread) = 2^22 of normal range below each reference.
// Else a head's own is at most 2^kOwn of the smallest.
constexpr int kSpread = 2, kOwn = 64;
// References are powers of two between these. What of the first tile's is taken off the scores goes kFoldLow
// down from the group's largest, and no factor falls below 2^-126.
constexpr int kRefLow = -80, kRefHigh = 127, kFoldLow = -40;
__device__ __forceinline__ float fold_of(float ref0, float ref1, float base) {
  return fmaxf(ref0 - base, fmaxf((float)kFoldLow, ref1 - (float)(126 + kWeightShift)));
}

struct Params {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int64_t T;
  int H, HG;  // heads, groups of 64 heads
  const uint8_t* cache;
  int64_t num_slots;
  const int32_t* bt;
  int64_t bt_stride;
  int page_size;
  uint32_t pg_mul;  // x / page_size == (x * pg_mul) >> pg_shift for 0 <= x < 2^31
  int pg_shift;
  int64_t pos_limit;  // addressable positions of a request
  int box_rows;       // bf16: rows of a TMA box (0: none, a page and a tile share fewer than eight)
  int64_t num_requests;
  const int32_t* req;
  const int32_t* starts;
  const int32_t* lengths;
  const int32_t* qpos;
  const int32_t* kpos;
  int64_t kp_stride;
  float sm_scale, cap;
  const float* slopes;
  uint16_t* out;
  int64_t out_st, out_sh;
  float* lse;
  int64_t lse_st;
  const float* mass;
  int64_t mass_st;
  float* mass_out;
  int64_t mass_out_st;
  int32_t* err;
  int G;            // CTAs
  float* ws_o;      // [2 G][64 heads][256] unnormalised partial outputs: slot 2c the row CTA c
                    // continues, 2c + 1 the row it starts and does not finish
  float* ws_ml;     // [2 G][2][64] their maxima (exp2 domain) and sums
  int4* ws_split;   // [G] split rows, entry r for row r when there are at most G rows, else entry c for the
                    // row that CTA c starts: the row (-1: not split, none), the CTAs that start and
                    // finish it, and the split's total cost
};

struct Seg {
  int type;  // 0: done, 1: a row's tiles
  int t, hg, req;
  int a, b;           // range of positions, clipped
  int tile0, ntiles;  // tiles of 128 positions from a rounded down to a multiple of 128
  int kind;           // 0: whole row, 1: its start, 2: a later part
  int pad[7];
};
static_assert(sizeof(Seg) == 64, "segment ring entry");

template <int KIND, bool MASS>
struct Cfg {
  static constexpr bool F8 = KIND == DSA_CACHE_FP8_SCALED;
  static constexpr int RB = F8 ? 264 : 512;
  static constexpr int NSB = MASS ? 4 : 2;            // score buffers (3: 128 x 32768 FP8 454 us for 458, but
                                                      // one token over 131071 positions 44 for 42)
  static constexpr int S_COLS = F8 ? 128 : 64;        // columns of one (FP8: one 64 per scale tile)
  static constexpr int O_COL = NSB * S_COLS;          // O^T halves at O_COL and O_COL + 64
  static constexpr int TMEM_USED = O_COL + (MASS ? 0 : 128);
  static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
  // FP8: ring of tile scales; a load warp may run this far ahead of the tile's reader
  static constexpr int NV = MASS ? 8 : 4;
  static constexpr bool WIDEN = F8 && !MASS;
  // K ring: halves of a tile (128 keys x 128 columns), as stored; FP8 values: a ring of widened halves
  static constexpr int HALF_BYTES = kBN * (F8 ? 128 : 256);
  static constexpr int NST = F8 ? (MASS ? 8 : 5) : 4;
  static constexpr int NW = 2;
  static constexpr int WIDE_BYTES = WIDEN ? kBN * 256 : 0;
  static constexpr int PBUF = F8 ? 1 : 2;
  static constexpr int PN = F8 ? 2 : 1;               // weight matrices per tile
  static constexpr int P_BYTES = MASS ? 0 : PN * kBN * 128;
  static constexpr int Q_OFF = 0, Q_BYTES = kHG * kD * 2;  // FP8: hi terms of both tiles, then lo
  static constexpr int K_OFF = Q_OFF + Q_BYTES;
  static constexpr int W_OFF = K_OFF + NST * HALF_BYTES;
  static constexpr int P_OFF = W_OFF + NW * WIDE_BYTES;
  static constexpr int SEG_OFF = P_OFF + PBUF * P_BYTES;
  static constexpr int MAP_OFF = SEG_OFF + kSegs * 64;        // [kMaps][128] slots, -1: masked
  static constexpr int FULL_OFF = MAP_OFF + kMaps * 512;      // [kMaps] no position of the tile is masked
  static constexpr int SC_OFF = FULL_OFF + kMaps * 4;        // FP8: [NV][128][2] tile scales
  static constexpr int SQ_OFF = SC_OFF + (F8 ? NV * 1024 : 0); // FP8: [kSegs][64] query scales
  static constexpr int NL_OFF = SQ_OFF + (F8 ? kSegs * 256 : 0);  // mass: [kSegs][64] -lse, exp2 domain
  static constexpr int SL_OFF = NL_OFF + (MASS ? kSegs * 256 : 0);  // slopes [128]
  // -m [2][64], alpha [64], part [4][64], inverse sums [64], raise of m [64]; FP8: largest weights of the
  // tile [4][2][64], then the accumulators' factors [2][64]; the weights' factors [2][64]; references
  // [2][64], log2; the heads' own factors [64]; per group both tiles' factors [2], the largest first
  // reference, and the second tile's largest factor
  static constexpr int RED_OFF = SL_OFF + 512;
  static constexpr int PLAN_OFF = RED_OFF + 9 * 256 + (WIDEN ? 13 * 256 + 64 : 0);  // block scans: 2 x kWarps int64; start row, its cost
  static constexpr int BAR_OFF = PLAN_OFF + 2 * 8 * kWarps + 64;
  static constexpr int NBARS = 2 + 2 * NST + 3 * kSegs + 2 * kMaps + 2 * NSB + 2 * 2 + 2 + 2 * NW;
  static constexpr int MISC_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(TMEM_USED <= 512, "TMEM budget");
};

// Instruction descriptor, kind::f16 with f16 A/B and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn_major, int b_mn_major) {
  return (1u << 4) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Warp-wide maximum (NaN ignored).
__device__ __forceinline__ float redux_max_f32(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// 2-D tiled tensor load (coordinates innermost first).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void set_err(int32_t* err, int bits) {
  if (err) atomicOr(err, bits);
}
__device__ __forceinline__ float u2f(uint32_t u) { return __uint_as_float(u); }
__device__ __forceinline__ uint32_t f2u(float f) { return __float_as_uint(f); }

struct Row {
  int req, a, b, n;  // range, tiles
  bool bad;          // something of it is not addressable
};
// Range of row `row` clipped to the addressable positions, and its tiles (0: nothing to read).
__device__ __forceinline__ Row row_of(const Params& p, int row) {
  const int t = p.HG == 1 ? row : row >> 1;
  const int req = p.req ? p.req[t] : t;
  const int s = p.starts ? p.starts[t] : 0;
  Row r;
  r.req = req;
  r.a = s < 0 ? 0 : s;
  r.b = p.lengths[t];
  r.n = 0;
  r.bad = false;
  if (r.a >= r.b) return r;
  if (req < 0 || req >= p.num_requests) {
    r.bad = true;
    return r;
  }
  if (r.b > p.pos_limit) {
    r.b = (int)p.pos_limit;
    r.bad = true;
  }
  if (r.a < r.b) r.n = ((r.b - 1) >> 7) - (r.a >> 7) + 1;
  return r;
}

// 2 log2(e) / cap: the cap's exponential is exp2(-|u| times this). Held finite (a cap below 2^-127 gives
// infinity, and a score of 0 would turn NaN).
__device__ __forceinline__ float cap_factor(float cap) { return cap > 0.0f ? fminf(2.0f * kLog2e / cap, 3.402823466e38f) : 0.0f; }

// One score in natural units -> exp2 domain, with cap and distance bias.
__device__ __forceinline__ float modify(float u, float cap, float inv_cap2, float bias) {
  if (cap > 0.0f) {
    // cap * tanh(z), z = u / cap. From |z| = 1/4 on cap * (1 - e) / (1 + e), e = exp(-2 |z|), with u's sign:
    // e's relative error (2^-22, and |z| 2^-22 of its argument) comes to 2.4 * 2^-22 of the result there
    // and falls from there on. Below, 1 - e would cancel (an error of cap * 2^-24, whatever u is), and
    // tanh's Taylor series as u * (1 - z^2 / 3 + 2 z^4 / 15 - 17 z^6 / 315 + 62 z^8 / 2835) is off by the next
    // term at most, 1382 / 155925 z^10 < 2^-26.
    const float w = fabsf(u) * inv_cap2;  // 2 log2(e) |z|
    constexpr float kZ = 0.5f * kLn2;     // z = kZ w
    constexpr float c1 = -kZ * kZ / 3.0f, c2 = kZ * kZ * kZ * kZ * (2.0f / 15.0f),
                    c3 = -kZ * kZ * kZ * kZ * kZ * kZ * (17.0f / 315.0f),
                    c4 = kZ * kZ * kZ * kZ * kZ * kZ * kZ * kZ * (62.0f / 2835.0f);
    const float w2 = w * w;
    const float series = fmaf(u, w2 * fmaf(w2, fmaf(w2, fmaf(w2, c4, c3), c2), c1), u);
    const float e = ex2_approx(-w);
    const float far = copysignf(__fdividef(cap * (1.0f - e), 1.0f + e), u);
    u = w < 0.25f / kZ ? series : far;
  }
  return (u - bias) * kLog2e;
}

// Exclusive sum over the block, and its total; `buf` holds kWarps values.
__device__ __forceinline__ int block_sum(int v, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int w = lane < kWarps ? buf[lane] : 0;  // every warp sums up the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + x - v;
}
// Exclusive running maximum over the block.
__device__ __forceinline__ int block_max(int v, int* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, y);
  }
  if (lane == 31) buf[warp] = x;
  int ex = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) ex = INT32_MIN;
  __syncthreads();
  int w = lane < warp ? buf[lane] : INT32_MIN;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
  return max(ex, w);
}
static_assert(kWarps <= 32, "one lane per warp in the block scans");

// Barrier of the four softmax warps of a head group, which returns the OR of `v`. They take the same
// path through the tiles: a warp whose wait runs out goes on with what it has, waiting no more, and
// the four leave together between two segments, so none is left behind at a barrier.
__device__ __forceinline__ bool group_any(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\nbarrier.cta.red.or.pred q, %1, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(1 + group), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// Splits query rows h0 .. h0 + HEADS - 1 of a row (zero past `heads`) into e4m3 hi and lo terms, lane
// l columns 8 l .. 8 l + 7, per head scaled by 2^-e so that the largest component lies in
// [128, 256); sq[h] = f * 2^e. One head per round of a short loop, the next one on its way meanwhile
// (the first call meets a cold instruction cache, and an unrolled body cost it 4 us).
template <int HEADS>
__device__ __forceinline__ void split_query(const uint16_t* q, int64_t q_sh, int h0, int heads, float f, uint8_t* qbuf,
                                            float* sq) {
  const int lane = threadIdx.x & 31;
  const int gl = lane & 15, tile = lane >> 4;
  auto load = [&](int h) {
    return h < heads ? *reinterpret_cast<const uint4*>(q + h * q_sh + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
  };
  // two lanes and two 128-byte lines each per head
  if (HEADS > 1 && lane < 2 * HEADS && h0 + (lane >> 1) < heads) {
    const uint16_t* a = q + (h0 + (lane >> 1)) * q_sh + 128 * (lane & 1);
    asm volatile("prefetch.global.L2 [%0];\nprefetch.global.L2 [%1];" ::"l"(a), "l"(a + 64));
  }
  uint4 next = load(h0);
#pragma unroll 1
  for (int h = h0; h < h0 + HEADS; ++h) {
    const uint32_t w[4] = {next.x, next.y, next.z, next.w};
    if (h + 1 < h0 + HEADS) next = load(h + 1);
    uint32_t a = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
    a = __reduce_max_sync(0xffffffffu, a);
    int e = (int)(a >> 23) - 127 - 7;
    e = a == 0u ? 0 : (e < -126 ? -126 : e);
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float x[4], r[4];
      x[0] = __uint_as_float(w[2 * j] << 16) * inv;
      x[1] = __uint_as_float(w[2 * j] & 0xFFFF0000u) * inv;
      x[2] = __uint_as_float(w[2 * j + 1] << 16) * inv;
      x[3] = __uint_as_float(w[2 * j + 1] & 0xFFFF0000u) * inv;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // four significant bits; none below e4m3's normal range (2^-6), where hi would round as well as lo
        const uint32_t bits = __float_as_uint(x[c]);
        r[c] = __uint_as_float(bits & ((bits & 0x7F800000u) < 0x3C800000u ? 0u : 0xFFF00000u));
      }
      hi[j] = (uint32_t)f32x2_to_e4m3x2(r[0], r[1]) | ((uint32_t)f32x2_to_e4m3x2(r[2], r[3]) << 16);
      lo[j] = (uint32_t)f32x2_to_e4m3x2(x[0] - r[0], x[1] - r[1]) |
              ((uint32_t)f32x2_to_e4m3x2(x[2] - r[2], x[3] - r[3]) << 16);
    }
    uint8_t* d = qbuf + tile * (kHG * 128) + h * 128 + (((gl >> 1) ^ (h & 7)) << 4) + 8 * (gl & 1);
    *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(d + 2 * kHG * 128) = make_uint2(lo[0], lo[1]);
    // an infinite or NaN component makes the head's scores NaN
    if (lane == 0)
      sq[h] = a >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : f * __uint_as_float((uint32_t)(127 + e) << 23);
  }
}

template <int KIND, bool MASS, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tmap) {
  using C = Cfg<KIND, MASS>;
  constexpr bool F8 = C::F8;
  extern __shared__ uint8_t smem_raw[];
  // an offset, not a rounded address: the compiler keeps knowing that this is shared memory (8 heads with
  // a distance bias 39 us; 46 with the rounded address, whose accesses are generic)
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  const uint32_t bar0 = sbase + C::BAR_OFF;
  const uint32_t q_full = bar0, q_empty = bar0 + 8;
  auto k_full = [&](uint32_t s) { return bar0 + 16 + 8 * s; };
  auto k_empty = [&](uint32_t s) { return bar0 + 16 + 8 * (C::NST + s); };
  const uint32_t b1 = bar0 + 16 + 16 * C::NST;
  auto g_full = [&](uint32_t s) { return b1 + 8 * s; };                 // segment ring
  auto g_empty = [&](uint32_t s) { return b1 + 8 * (kSegs + s); };
  auto aux_full = [&](uint32_t s) { return b1 + 8 * (2 * kSegs + s); };  // the segment's -lse, query scales
  const uint32_t b2 = b1 + 24 * kSegs;
  auto map_full = [&](uint32_t s) { return b2 + 8 * s; };               // slots of a tile
  auto map_empty = [&](uint32_t s) { return b2 + 8 * (kMaps + s); };
  const uint32_t b2s = b2 + 16 * kMaps;
  auto s_full = [&](uint32_t s) { return b2s + 8 * s; };
  auto s_empty = [&](uint32_t s) { return b2s + 8 * (C::NSB + s); };
  const uint32_t b3 = b2s + 16 * C::NSB;
  auto p_full = [&](uint32_t s) { return b3 + 8 * s; };
  auto pv_done = [&](uint32_t s) { return b3 + 16 + 8 * s; };
  auto drain = [&](uint32_t s) { return b3 + 32 + 8 * s; };
  auto w_full = [&](uint32_t s) { return b3 + 48 + 8 * s; };  // widened halves
  auto w_empty = [&](uint32_t s) { return b3 + 48 + 8 * (C::NW + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  volatile int* progress = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);  // tiles mapped
  Seg* segs = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  float* s_slopes = reinterpret_cast<float*>(smem + C::SL_OFF);

  asm volatile("griddepcontrol.launch_dependents;");
  // a barrier per thread, in the order of their addresses
  if (threadIdx.x < C::NBARS) {
    constexpr int B0 = 2, B1 = B0 + C::NST, B2 = B1 + C::NST, B3 = B2 + kSegs, B4 = B3 + kSegs, B5 = B4 + kSegs,
                  B6 = B5 + kMaps, B7 = B6 + kMaps, B8 = B7 + C::NSB, B9 = B8 + C::NSB, B10 = B9 + 2, B11 = B10 + 4,
                  B12 = B11 + C::NW;
    const int i = threadIdx.x;
    int n = 1;                                                 // pv_done, drain, w_empty, q_empty, g_full, map_full
    if (i == 0) n = F8 ? kSoftmaxWarps : 32;                   // q_full (bf16: an asynchronous arrival per thread)
    else if (i >= B0 && i < B1) n = 32 * kLoadWarps;           // k_full: an asynchronous arrival per thread
    else if (i >= B1 && i < B2) n = 1 + (C::WIDEN ? kWidenWarps : 0);  // k_empty: the last product, the widening
    else if (i >= B3 && i < B4)                                // g_empty: softmax, issuers, query warp, widening
      n = kSoftmaxWarps + 1 + (MASS ? 0 : 1) + (C::WIDEN ? 0 : 1) + (F8 ? kWidenWarps : 0);
    else if (i >= B4 && i < B5) n = (MASS ? 1 : 0) + (F8 ? kSoftmaxWarps : 0) + (!MASS && !F8 ? 1 : 0);  // aux_full
    else if (i >= B6 && i < B7) n = MASS ? 4 : kSoftmaxWarps;  // map_empty
    else if (i >= B7 && i < B8) n = 2;                         // s_full: the product, and its issuer
    else if (i >= B8 && i < B9) n = MASS ? 4 : kSoftmaxWarps;  // s_empty
    else if (i >= B9 && i < B10) n = kSoftmaxWarps;            // p_full
    else if (i >= B11 && i < B12) n = kWidenWarps;             // w_full
    mbar_init(bar0 + 8 * i, n);
    if (i == 0) *abort_flag = *progress = 0;
    fence_mbar_init();
  }
  if (MODS && threadIdx.x < kMaxHeads)
    s_slopes[threadIdx.x] = p.slopes && threadIdx.x < p.H ? p.slopes[threadIdx.x] : 0.0f;
  if (warp == kWarpScore) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }

  // ---- the split: the total cost of the rows, and the row in which this CTA's share begins. Up to
  // kWarpRows rows the scheduler alone finds them (no block barrier waits for the lengths), else all.
  int* plan = reinterpret_cast<int*>(smem + C::PLAN_OFF);
  int* plan_start = plan + 2 * kWarps;  // row, its cost offset, running maximum of the requests
  const int nrows = (int)(p.T * p.HG);
  int total = 0, row = 0, cost = 0;  // the scheduler's: where its walk begins
  int run = INT32_MIN;
  auto cost_of = [&](const Row& r, int& run) -> int {
    bool ok = true;
    if (MASS && p.req) {
      ok = r.req > run;
      run = max(run, r.req);
    }
    return (ok ? r.n : 0) + kRowOverhead;
  };
  if (nrows > kWarpRows) {
    const int per = (nrows + kThreads - 1) / kThreads;
    const int i0 = min((int)threadIdx.x * per, nrows), i1 = min(i0 + per, nrows);
    int mx = INT32_MIN;
    if (MASS && p.req) {
      int m = INT32_MIN;
      for (int i = i0; i < i1; ++i) m = max(m, p.req[i]);
      mx = block_max(m, plan);
    }
    int sum = 0;
    run = mx;
    for (int i = i0; i < i1; ++i) sum += cost_of(row_of(p, i), run);
    const int pre = block_sum(sum, plan + kWarps, &total);
    const int c0 = share(cta, total, p.G);
    if (pre <= c0 && c0 < pre + sum) {
      int at = pre, i = i0;
      run = mx;
      for (;; ++i) {
        int next = run;
        const int c = cost_of(row_of(p, i), next);
        if (c0 < at + c) break;
        at += c;
        run = next;
      }
      plan_start[0] = i;
      plan_start[1] = at;
      plan_start[2] = run;
    }
  } else if (warp == kWarpSched) {
    constexpr int PER = kWarpRows / 32;
    const int per = (nrows + 31) / 32, i0 = lane * per;
    Row r[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (k < per && i0 + k < nrows) r[k] = row_of(p, i0 + k);
    int mx = INT32_MIN;
    if (MASS && p.req) {
      int m = INT32_MIN;
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (k < per && i0 + k < nrows) m = max(m, r[k].req);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) m = max(m, y);
      }
      mx = __shfl_up_sync(0xffffffffu, m, 1);
      if (lane == 0) mx = INT32_MIN;
    }
    int mine = 0;
    int rn = mx;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (k < per && i0 + k < nrows) mine += cost_of(r[k], rn);
    int cum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, cum, o);
      if (lane >= o) cum += y;
    }
    total = __shfl_sync(0xffffffffu, cum, 31);
    // the last 32 rows at most are walked from the lane whose rows hold the start
    const int c0 = share(cta, total, p.G), pre = cum - mine;
    const uint32_t in = __ballot_sync(0xffffffffu, pre <= c0 && c0 < cum);
    const int src = __ffs(in) - 1;  // some lane: c0 < total
    row = src * per;
    cost = __shfl_sync(0xffffffffu, pre, src);
    run = __shfl_sync(0xffffffffu, mx, src);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&]() {
    set_err(p.err, DSA_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  auto wait = [&](uint32_t bar, uint32_t par) -> bool {
    if (bar_wait(bar, par, abort_flag)) return true;
    fail();
    return false;
  };
  // FP8: the first segment's query, by the softmax warps
  auto split_first = [&](const Seg& s, uint32_t slot) {
    constexpr int HEADS = kHG / kSoftmaxWarps;
    split_query<HEADS>(p.q + (int64_t)s.t * p.q_st + (int64_t)s.hg * kHG * p.q_sh, p.q_sh, HEADS * warp,
                       min(kHG, p.H - s.hg * kHG), MODS ? p.sm_scale : p.sm_scale * kLog2e, smem + C::Q_OFF,
                       reinterpret_cast<float*>(smem + C::SQ_OFF) + kHG * slot);
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(q_full);
      mbar_arrive(aux_full(slot));
    }
  };
  // the whole warp waits, and agrees on the outcome
  auto wait_warp = [&](uint32_t bar, uint32_t par) -> bool {
    if (__all_sync(0xffffffffu, bar_wait(bar, par, abort_flag))) return true;
    fail();
    return false;
  };

  // for warps that have nothing to do between two rows' starts
  auto wait_row = [&](uint32_t bar, uint32_t par) -> bool {
    if (__all_sync(0xffffffffu, bar_wait_row(bar, par, abort_flag, progress))) return true;
    fail();
    return false;
  };

  // 896 threads x 72 registers at launch; 512 x 80 + 384 x 56 is within that total. (No function is
  // called from here on: ptxas allocates past the launch's 72 only without calls.)
  static_assert(32 * kWarps == 896 && 32 * kWarps * 72 >= 512 * 80 + 384 * 56, "register split");
  if (warp >= kSoftmaxWarps) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == kWarpSched) {
    // ================================================================== scheduler ====
    uint32_t sc = 0;
    uint32_t g = 0;  // tiles mapped
    int split_row = -1, split_last = 0;  // the row this CTA starts and does not finish
    bool ok = true;
    auto map_slot = [&](bool& good) -> int4* {
      const uint32_t m = g % kMaps;
      good = g < kMaps || wait_warp(map_empty(m), ((g / kMaps) & 1) ^ 1);
      return reinterpret_cast<int4*>(smem + C::MAP_OFF + m * 512) + lane;
    };
    auto map_done = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(map_full(g % kMaps));
      ++g;
      if (lane == 0) *progress = (int)g;
    };
    // the slots of `n` tiles from position `base` of the range [a, b): lane l rows 4 l .. 4 l + 3
    auto map_tiles = [&](int req, uint32_t a, uint32_t b, uint32_t base, int n) -> bool {
      const int32_t* bt = p.bt ? p.bt + req * p.bt_stride : nullptr;
      for (int k = 0; k < n; ++k, base += kBN) {
        bool good;
        int4* dst = map_slot(good);
        if (!good) return false;
        int sl[4];
        bool bad = false;
        const uint32_t pos0 = base + 4 * lane;
        uint32_t pg = 0, off = pos0;
        if (bt) {
          pg = (uint32_t)(((uint64_t)pos0 * p.pg_mul) >> p.pg_shift);
          off = pos0 - pg * (uint32_t)p.page_size;
        }
        if (pos0 >= a && pos0 + 4 <= b && (!bt || off + 4 <= (uint32_t)p.page_size)) {
          // four rows of one page
          int64_t s0 = off;
          if (bt) {
            const int64_t page = bt[pg];
            s0 = page < 0 ? p.num_slots : page * p.page_size + off;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sl[i] = s0 + i < p.num_slots ? (int)s0 + i : -1;
          bad = sl[3] < 0;
        } else {
#pragma unroll 1
          for (int i = 3; i >= 0; --i) {
            const uint32_t pos = pos0 + i;
            int v = -1;
            if (pos >= a && pos < b) {
              int64_t slot = pos;
              if (bt) {
                pg = (uint32_t)(((uint64_t)pos * p.pg_mul) >> p.pg_shift);
                const int64_t page = bt[pg];
                slot = page < 0 ? p.num_slots : page * p.page_size + (pos - pg * (uint32_t)p.page_size);
              }
              if (slot < p.num_slots) v = (int)slot;
              else bad = true;
            }
            sl[3] = sl[2];
            sl[2] = sl[1];
            sl[1] = sl[0];
            sl[0] = v;
          }
        }
        if (bad) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        *dst = make_int4(sl[0], sl[1], sl[2], sl[3]);
        const bool full = __all_sync(0xffffffffu, sl[0] >= 0 && sl[1] >= 0 && sl[2] >= 0 && sl[3] >= 0);
        if (lane == 0) reinterpret_cast<int*>(smem + C::FULL_OFF)[g % kMaps] = full;
        // the tile's rows into L2, one request per page
        if (F8 && bt && p.page_size >= kPrefetchPage) {
          const uint32_t lo = max(base, a), hi = min(base + (uint32_t)kBN, b);
          const uint32_t pg = (uint32_t)(((uint64_t)lo * p.pg_mul) >> p.pg_shift) + lane;
          const uint64_t first = (uint64_t)pg * (uint32_t)p.page_size;
          if (first < hi) {
            const uint64_t from = first > lo ? first : lo;
            const uint64_t to = first + p.page_size < hi ? first + p.page_size : hi;
            const int64_t s0 = (int64_t)bt[pg] * p.page_size + (int64_t)(from - first);
            if (s0 >= 0 && s0 + (int64_t)(to - from) <= p.num_slots) {
              const uint64_t b0 = (uint64_t)(s0 * C::RB) & ~15ull;
              const uint32_t bytes = (uint32_t)((uint64_t)((s0 + (int64_t)(to - from)) * C::RB) - b0) & ~15u;
              if (bytes)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.cache + b0), "r"(bytes) : "memory");
            }
          }
        }
        map_done();
      }
      return true;
    };
    if (nrows > kWarpRows) {
      row = plan_start[0];
      cost = plan_start[1];
      run = plan_start[2];
    }
    const int c0 = share(cta, total, p.G), c1 = share(cta + 1, total, p.G);
    if (c0 < c1) {
      while (ok && cost < c1 && row < nrows) {
        const int i = row + lane;
        Row r{};
        int c = 0;
        bool order = true;
        if (i < nrows) {
          r = row_of(p, i);
          c = 1;
        }
        if (MASS && p.req) {
          int x = i < nrows ? r.req : INT32_MIN;
          int before = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x = max(x, y);
          }
          before = __shfl_up_sync(0xffffffffu, x, 1);
          before = lane == 0 ? run : max(before, run);
          run = max(run, __shfl_sync(0xffffffffu, x, 31));
          order = r.req > before;
        }
        const int n = order ? r.n : 0;
        int cum = c ? n + kRowOverhead : 0;
        const int mine = cum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, cum, o);
          if (lane >= o) cum += y;
        }
        const int at = cost + cum - mine;  // this row's cost offset
        int lo = c0 - at - kRowOverhead, hi = c1 - at - kRowOverhead;
        lo = lo < 0 ? 0 : lo;
        hi = hi > n ? n : hi;
        const bool owner = c && at >= c0 && at < c1;
        if (owner && r.bad && order) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        if (owner && !order && r.a < r.b) set_err(p.err, DSA_DEVERR_REQUEST_ORDER);
        const bool has = c && (n > 0 ? lo < hi : owner && !MASS);
        const int kind = lo > 0 ? 2 : (hi < n ? 1 : 0);
        // the CTA of a split row's last tile: the largest whose share starts at or before it
        int last = 0;
        if (kind == 1) {
          // from the quotient's estimate: shares are total / G long, give or take one
          last = min(p.G - 1, (int)((float)(at + kRowOverhead + n) * ((float)p.G / (float)total)));
          while (last > 0 && share(last, total, p.G) >= at + kRowOverhead + n) --last;
          while (last + 1 < p.G && share(last + 1, total, p.G) < at + kRowOverhead + n) ++last;
        }
        if (!MASS && nrows <= p.G && has && kind != 2) {
          p.ws_split[i] = make_int4(kind == 1 ? i : -1, cta, last, total);
        }
        uint32_t todo = __ballot_sync(0xffffffffu, has);
        if (!MASS) {
          const uint32_t st = __ballot_sync(0xffffffffu, has && kind == 1);
          if (st) {  // at most one, the CTA's last
            split_row = row + (31 - __clz(st));
            split_last = __shfl_sync(0xffffffffu, last, 31 - __clz(st));
          }
        }
        while (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          const uint32_t slot = sc % kSegs;
          if (sc >= kSegs && !wait_warp(g_empty(slot), ((sc / kSegs) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == src) {
            Seg* s = segs + slot;
            s->type = 1;
            s->t = p.HG == 1 ? i : i >> 1;
            s->hg = p.HG == 1 ? 0 : i & 1;
            s->req = r.req;
            s->a = r.a;
            s->b = r.b;
            s->tile0 = lo;
            s->ntiles = n > 0 ? hi - lo : 0;
            s->kind = kind;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(g_full(slot));
          ++sc;
          const int a = __shfl_sync(0xffffffffu, r.a, src), b = __shfl_sync(0xffffffffu, r.b, src);
          const int t0 = __shfl_sync(0xffffffffu, lo, src);
          const int nt = __shfl_sync(0xffffffffu, n > 0 ? hi - lo : 0, src);
          const int req = __shfl_sync(0xffffffffu, r.req, src);
          if (!map_tiles(req, (uint32_t)a, (uint32_t)b, (uint32_t)(a & ~127) + 128u * (uint32_t)t0, nt)) {
            ok = false;
            break;
          }
        }
        row += 32;
        cost += __shfl_sync(0xffffffffu, cum, 31);
      }
    }
    if (!MASS && nrows > p.G && lane == 0) p.ws_split[cta] = make_int4(split_row, cta, split_last, total);
    if (ok) {
      bool good;
      int4* dst = map_slot(good);
      if (good) {  // no more tiles
        *dst = make_int4(-2, -2, -2, -2);
        map_done();
      }
      const uint32_t slot = sc % kSegs;
      if (sc < kSegs || wait_warp(g_empty(slot), ((sc / kSegs) & 1) ^ 1)) {
        if (lane == 0) {
          segs[slot].type = 0;
          mbar_arrive(g_full(slot));
        }
      }
    }
  } else if (warp == kWarpScore) {
    // ============================================================= score products ====
    if (lane == 0) {
      constexpr uint32_t idS = F8 ? idesc_e4m3(kBN, kHG, 0, 0) : idesc_bf16(kBN, kHG, 0, 0);
      const uint64_t dq = sw128_desc(sbase + C::Q_OFF, 16, 1024);
      const uint32_t q_lo = (uint32_t)dq, q_hi = (uint32_t)(dq >> 32);
      const uint32_t k_hi = (uint32_t)(sw128_desc(0, 16, 1024) >> 32);
      uint32_t g = 0, qc = 0;
      bool ok = true;
      for (uint32_t sc = 0; ok; ++sc) {
        const uint32_t slot = sc % kSegs;
        if (!wait(g_full(slot), (sc / kSegs) & 1)) break;
        const int type = segs[slot].type, ntiles = segs[slot].ntiles;
        mbar_arrive(g_empty(slot));
        if (type == 0) break;
        if (ntiles == 0) continue;
        if (!wait(q_full, qc & 1)) break;
        ++qc;
        for (int k = 0; k < ntiles && ok; ++k, ++g) {
          const uint32_t sb = g % C::NSB;
          if (g >= C::NSB && !wait(s_empty(sb), ((g / C::NSB) & 1) ^ 1)) {
            ok = false;
            break;
          }
          // the slots' and (with k_full) the scales' writes are this thread's to pass on with s_full
          if (!wait(map_full(g % kMaps), (g / kMaps) & 1)) {
            ok = false;
            break;
          }
          const uint32_t d0 = tmem + sb * C::S_COLS;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t hs = 2 * g + h, st = hs % C::NST;
            if (!wait(k_full(st), (hs / C::NST) & 1)) {
              ok = false;
              break;
            }
            // the operands were written through the generic proxy
            fence_proxy_async_smem();
            tc_fence_after();
            const uint32_t k_lo = (uint32_t)sw128_desc(sbase + C::K_OFF + st * C::HALF_BYTES, 16, 1024);
            const uint32_t d = F8 ? d0 + 64 * h : d0;
            if constexpr (F8) {
              // 32 columns per step, hi term then lo term (two chunks further)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t qa = q_lo + (uint32_t)((h * (kHG * 128) + 32 * kk) >> 4);
                if (kk == 0) mma_f8_lohi<0>(d, k_lo, k_hi, qa, q_hi, idS);
                else mma_f8_lohi<1>(d, k_lo + 2 * kk, k_hi, qa, q_hi, idS);
                mma_f8_lohi<1>(d, k_lo + 2 * kk, k_hi, qa + ((2 * kHG * 128) >> 4), q_hi, idS);
              }
            } else {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t ka = (uint32_t)((kk >> 2) * ((kBN * 128) >> 4) + (kk & 3) * 2);
                const uint32_t qa = (uint32_t)((2 * h + (kk >> 2)) * ((kHG * 128) >> 4) + (kk & 3) * 2);
                if (kk == 0 && h == 0) mma_bf16_lohi<0>(d, k_lo + ka, k_hi, q_lo + qa, q_hi, idS);
                else mma_bf16_lohi<1>(d, k_lo + ka, k_hi, q_lo + qa, q_hi, idS);
              }
            }
            if (MASS || F8) mma_commit(k_empty(st));
          }
          if (ok) {
            mma_commit(s_full(sb));
            mbar_arrive(s_full(sb));
          }
        }
        if (ok) mma_commit(q_empty);
      }
      mma_commit(drain(0));
      bar_wait(drain(0), 0, nullptr);  // (products in flight end before the block does)
    }
    __syncwarp();
  } else if (warp == kWarpValue) {
    // ============================================================= value products ====
    if (!MASS && lane == 0) {
      constexpr uint32_t idPV = F8 ? idesc_f16(kBN, kHG, 1, 1) : idesc_bf16(kBN, kHG, 1, 1);
      const uint32_t mn_hi = (uint32_t)(sw128_desc(0, kBN * 128, 1024) >> 32);
      uint32_t g = 0;
      bool ok = true;
      for (uint32_t sc = 0; ok; ++sc) {
        const uint32_t slot = sc % kSegs;
        if (!wait(g_full(slot), (sc / kSegs) & 1)) break;
        const int type = segs[slot].type, ntiles = segs[slot].ntiles;
        mbar_arrive(g_empty(slot));
        if (type == 0) break;
        for (int k = 0; k < ntiles; ++k, ++g) {
          const uint32_t pb = g % C::PBUF;
          if (!wait(p_full(pb), (g / C::PBUF) & 1)) {
            ok = false;
            break;
          }
          // weights and rows were written through the generic proxy: ordered here, by the thread that
          // has waited for them (a writer's fence would also wait for its copies in flight)
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t hs = 2 * g + h, st = hs % (C::WIDEN ? C::NW : C::NST);
            if (C::WIDEN) {
              if (!wait(w_full(st), (hs / C::NW) & 1)) {
                ok = false;
                break;
              }
              fence_proxy_async_smem();
              tc_fence_after();
            }
            const uint32_t v_lo = (uint32_t)sw128_desc(
                sbase + (C::WIDEN ? C::W_OFF + st * C::WIDE_BYTES : C::K_OFF + st * C::HALF_BYTES), kBN * 128, 1024);
            const uint32_t p_lo = (uint32_t)sw128_desc(
                sbase + C::P_OFF + pb * C::P_BYTES + (F8 ? h * kBN * 128 : 0), kBN * 128, 1024);
            const uint32_t d = tmem + C::O_COL + 64 * h;
            // the first step of a segment overwrites the accumulator
            mma_bf16(d, ((uint64_t)mn_hi << 32) | v_lo, ((uint64_t)mn_hi << 32) | p_lo, idPV, k == 0 ? 0u : 1u);
#pragma unroll
            for (int j = 1; j < kBN / 16; ++j)
              mma_bf16_lohi<1>(d, v_lo + 128 * j, mn_hi, p_lo + 128 * j, mn_hi, idPV);
            mma_commit(C::WIDEN ? w_empty(st) : k_empty(st));
          }
          if (!ok) break;
          mma_commit(pv_done(g & 1));
        }
      }
      mma_commit(drain(1));
      bar_wait(drain(1), 0, nullptr);
    }
    __syncwarp();
  } else if (warp == kWarpQuery) {
    // ================================================================ query loads ====
    // 64 heads x 256 columns in four 128-byte-swizzled chunks; heads past the row's are zero.
    // FP8: the softmax and the widening warps split the query, and for the attention nothing is left to do here.
    uint32_t qc = 0;
    for (uint32_t sc = 0; !C::WIDEN; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!wait_row(g_full(slot), (sc / kSegs) & 1)) break;
      const Seg s = segs[slot];
      if (s.type == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(g_empty(slot));
        break;
      }
      const int heads = min(kHG, p.H - s.hg * kHG);
      if (s.ntiles > 0) {
        if (MASS) {
          float* nl = reinterpret_cast<float*>(smem + C::NL_OFF) + slot * kHG;
          for (int h = lane; h < kHG; h += 32)
            nl[h] = h < heads ? -p.lse[s.t * p.lse_st + s.hg * kHG + h] * kLog2e : -INFINITY;
          __syncwarp();
          if (lane == 0) mbar_arrive(aux_full(slot));
        }
      }
      if (!F8 && s.ntiles > 0) {
        if (qc > 0 && !wait_warp(q_empty, (qc - 1) & 1)) break;
        ++qc;
        const uint16_t* q = p.q + (int64_t)s.t * p.q_st + (int64_t)s.hg * kHG * p.q_sh;
#pragma unroll 8
        for (int h = 0; h < kHG; ++h) {
          // lane = 16-byte granule of the head's row
          const uint32_t dst = sbase + C::Q_OFF + (lane >> 3) * (kHG * 128) + h * 128 + (((lane & 7) ^ (h & 7)) << 4);
          const uint16_t* src = h < heads ? q + h * p.q_sh + 8 * lane : p.q;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(h < heads ? 16 : 0)
                       : "memory");
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(q_full) : "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(g_empty(slot));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kWarpWiden0) {
    // ================================================================== row loads ====
    // Warp w takes rows 32 w .. 32 w + 31 of every tile, in two column halves; by cp.async the 16 lanes of
    // a half warp share a row.
    const int lw = warp - kWarpLoad0;
    const int gl = lane & 15, hi16 = lane >> 4;
    const int r0 = kLoadRows * lw + hi16;
    // byte offset of the lane's piece (16 bytes; FP8: 8) of row r0 + 2 i in a half as stored: rows of
    // 128 bytes, 16-byte granules swizzled by the row, which repeats every four i
    uint32_t piece[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 2 * i;
      piece[i] = F8 ? (uint32_t)(r * 128 + (((gl >> 1) ^ (r & 7)) << 4) + 8 * (gl & 1))
                    : (uint32_t)((gl >> 3) * (kBN * 128) + r * 128 + (((gl & 7) ^ (r & 7)) << 4));
    }
    constexpr int PIECE = F8 ? 8 : 16, HALF_ROW = F8 ? 128 : 256;
    // FP8 rows that follow one another from an even slot (a slot is 264 bytes, the base is 16-byte aligned):
    // even rows start on 16 bytes and go in 16-byte pieces, four rows per instruction, odd ones in 8-byte
    // pieces, two rows per instruction (128 tokens x 32768 keys when it was tried: 489 us; 549 with 8-byte
    // pieces alone)
    const int er = 2 * (lane >> 3);  // even row 8 i + er, granule lane % 8
    const uint32_t even = (uint32_t)((kLoadRows * lw + er) * 128 + (((lane & 7) ^ er) << 4));
    uint32_t odd[2];                 // odd row 4 i + 2 hi16 + 1, which is 4 (i % 2) + 2 hi16 + 1 of eight
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 4 * i + 2 * hi16 + 1;
      odd[i] = (uint32_t)((kLoadRows * lw + r) * 128 + (((gl >> 1) ^ r) << 4) + 8 * (gl & 1));
    }
    uint32_t issued = 0;  // halves
    for (uint32_t g = 0;; ++g) {
      if (!wait_warp(map_full(g % kMaps), (g / kMaps) & 1)) break;
      const int own = reinterpret_cast<const int*>(smem + C::MAP_OFF + (g % kMaps) * 512)[kLoadRows * lw + lane];
      if (__any_sync(0xffffffffu, own == -2)) break;
      const int first = __shfl_sync(0xffffffffu, own, 0);
      const bool run = __all_sync(0xffffffffu, first >= 0 && own == first + lane);  // rows that follow one another
      const bool boxes = !F8 && p.box_rows > 0 && reinterpret_cast<const int*>(smem + C::FULL_OFF)[g % kMaps];
      bool stop = false;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t hs = 2 * g + h, st = hs % C::NST;
        if (hs >= C::NST && !wait_warp(k_empty(st), ((hs / C::NST) & 1) ^ 1)) {
          stop = true;
          break;
        }
        if (F8 && h == 0) {
          // the two scales of the lane's row
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(sbase + C::SC_OFF + 1024 * (g % C::NV) +
                                                                            8 * (kLoadRows * lw + lane)),
                       "l"(p.cache + (own >= 0 ? (int64_t)own * C::RB + 256 : 0)), "r"(own >= 0 ? 8 : 0)
                       : "memory");
        }
        issued = hs + 1;
        const uint32_t dst = sbase + C::K_OFF + st * C::HALF_BYTES;
        if (boxes) {
          // boxes of 64 columns x box_rows rows, a box by the warp its first row belongs to
          const int per = p.box_rows < kLoadRows ? kLoadRows / p.box_rows : 1;
          const bool mine = p.box_rows < kLoadRows || (kLoadRows * lw) % p.box_rows == 0;
          if (mine && lane == 0) mbar_arrive_expect_tx(k_full(st), 2 * per * p.box_rows * 128);
          else mbar_arrive(k_full(st));
          __syncwarp();
          const int c = lane & 1, r = (lane >> 1) * p.box_rows;
          const int y = __shfl_sync(0xffffffffu, own, r & 31);
          if (mine && lane < 2 * per)
            tma_load_2d(dst + c * (kBN * 128) + (kLoadRows * lw + r) * 128, &tmap, 128 * h + 64 * c, y, k_full(st));
          continue;
        }
        if (F8 && run && (first & 1) == 0) {
          const uint8_t* src = p.cache + (int64_t)first * C::RB + HALF_ROW * h;
          const uint8_t* se = src + er * C::RB + 16 * (lane & 7);
          const uint8_t* so = src + (2 * hi16 + 1) * C::RB + 8 * gl;
#pragma unroll
          for (int i = 0; i < kLoadRows / 8; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + even + 1024 * i), "l"(se + 8 * C::RB * i)
                         : "memory");
#pragma unroll
          for (int i = 0; i < kLoadRows / 4; ++i)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + odd[i & 1] + 1024 * (i >> 1)),
                         "l"(so + 4 * C::RB * i)
                         : "memory");
        } else if (run) {
          const uint8_t* src = p.cache + (int64_t)(first + hi16) * C::RB + HALF_ROW * h + PIECE * gl;
#pragma unroll
          for (int i = 0; i < kLoadRows / 2; ++i) {
            if constexpr (F8)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + piece[i & 3] + 1024 * (i >> 2)),
                           "l"(src + 2 * C::RB * i)
                           : "memory");
            else
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + piece[i & 3] + 1024 * (i >> 2)),
                           "l"(src + 2 * C::RB * i)
                           : "memory");
          }
        } else {
#pragma unroll 4
          for (int i = 0; i < kLoadRows / 2; ++i) {
            const int sl = __shfl_sync(0xffffffffu, own, 2 * i + hi16);
            const uint8_t* src = p.cache + (sl >= 0 ? (int64_t)sl * C::RB + HALF_ROW * h + PIECE * gl : 0);
            if constexpr (F8)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + piece[i & 3] + 1024 * (i >> 2)),
                           "l"(src), "r"(sl >= 0 ? 8 : 0)
                           : "memory");
            else
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + piece[i & 3] + 1024 * (i >> 2)),
                           "l"(src), "r"(sl >= 0 ? 16 : 0)
                           : "memory");
          }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(k_full(st)) : "memory");
      }
      if (stop) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (!F8) {
      // boxes in flight land before the block ends (after a wait that ran out a load warp may lack another's
      // arrivals: the first wait then takes its whole limit, which is the time they had)
      for (uint32_t hs = issued; hs > 0 && issued - hs < (uint32_t)C::NST; --hs)
        if (!bar_wait(k_full((hs - 1) % C::NST), ((hs - 1) / C::NST) & 1, nullptr)) break;
    }
  } else if constexpr (F8) {
    // ================================================= FP8: query split and widening ====
    // Warp w splits heads 16 w .. of a segment's query (the CTA's first is split by the softmax warps,
    // which have nothing else to do yet), then widens rows 32 w .. 32 w + 31 of its tiles.
    const int ww = warp - kWarpWiden0;
    // In round t a lane takes a 16-byte granule (4 t + lane % 4) of a row and writes two. Eight lanes
    // that access memory together take rows k and k ^ 5 of a group of eight, whose swizzles keep the
    // four granules read, and the four written, of one row off the other's banks.
    const int g4 = lane & 3, r7 = (lane >> 3) ^ (lane & 4 ? 5 : 0);
    const uint32_t row = (uint32_t)(32 * ww + r7) * 128;
    const uint32_t from[2] = {row + ((g4 ^ r7) << 4), row + (((4 + g4) ^ r7) << 4)};
    const uint32_t to[2] = {row + (((2 * g4) ^ r7) << 4), row + (((2 * g4 + 1) ^ r7) << 4)};
    uint32_t hs = 0, qn = 0;  // halves widened, queries split
    bool ok = true;
    for (uint32_t sc = 0; ok; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!(C::WIDEN ? wait_warp(g_full(slot), (sc / kSegs) & 1) : wait_row(g_full(slot), (sc / kSegs) & 1))) break;
      const Seg s = segs[slot];
      if (s.type == 0) break;
      const bool split = s.ntiles > 0 && qn > 0;
      if (split) {
        if (!wait_warp(q_empty, (qn - 1) & 1)) break;
        split_query<kHG / kWidenWarps>(p.q + (int64_t)s.t * p.q_st + (int64_t)s.hg * kHG * p.q_sh, p.q_sh,
                                       kHG / kWidenWarps * ww, min(kHG, p.H - s.hg * kHG),
                                       MODS ? p.sm_scale : p.sm_scale * kLog2e, smem + C::Q_OFF,
                                       reinterpret_cast<float*>(smem + C::SQ_OFF) + kHG * slot);
      }
      __syncwarp();
      // (an arrival for each of the softmax warps, who arrive at the first segment's)
      if (lane < kSoftmaxWarps / kWidenWarps) {
        if (split) mbar_arrive(q_full);
        if (split || s.ntiles == 0) mbar_arrive(aux_full(slot));
      }
      if (lane == 0) mbar_arrive(g_empty(slot));
      qn += s.ntiles > 0;
      if constexpr (C::WIDEN) {
        const uint32_t end = hs + 2 * (uint32_t)s.ntiles;
        for (; hs < end; ++hs) {
          const uint32_t st = hs % C::NST, sw = hs % C::NW;
          if (!wait_warp(k_full(st), (hs / C::NST) & 1) ||
              (hs >= C::NW && !wait_warp(w_empty(sw), ((hs / C::NW) & 1) ^ 1))) {
            ok = false;
            break;
          }
          const uint8_t* raw = smem + C::K_OFF + st * C::HALF_BYTES;
          uint8_t* wide = smem + C::W_OFF + sw * C::WIDE_BYTES;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint4 v[4];  // row groups 2 part, 2 part + 1, both rounds
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4*>(raw + from[i & 1] + 1024 * (2 * part + (i >> 1)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t c[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint4*>(wide + to[j] + (i & 1) * (kBN * 128) + 1024 * (2 * part + (i >> 1))) = make_uint4(
                    e4m3x2_to_f16x2((uint16_t)c[2 * j]), e4m3x2_to_f16x2((uint16_t)(c[2 * j] >> 16)),
                    e4m3x2_to_f16x2((uint16_t)c[2 * j + 1]), e4m3x2_to_f16x2((uint16_t)(c[2 * j + 1] >> 16)));
            }
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(w_full(sw));
            mbar_arrive(k_empty(st));
          }
        }
      }
    }
  }
  } else {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
  if constexpr (MASS) {
    // ================================================== weights of a key, 16 warps ===
    const int qd = warp & 3, gi = warp >> 2;
    const int tr = 32 * qd + lane;
    const float inv_cap2 = MODS ? cap_factor(p.cap) : 0.0f;
    const float c_log2 = p.sm_scale * kLog2e;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t sc = 0; ok; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!wait_warp(g_full(slot), (sc / kSegs) & 1)) break;
      const Seg s = segs[slot];
      if (s.type == 0) break;
      if (F8 && sc == 0) split_first(s, slot);  // (a mass segment has tiles)
      if (!wait_warp(aux_full(slot), (sc / kSegs) & 1)) break;
      const float* sq = reinterpret_cast<const float*>(smem + C::SQ_OFF) + kHG * slot;
      const int heads = min(kHG, p.H - s.hg * kHG);
      const float* nl = reinterpret_cast<const float*>(smem + C::NL_OFF) + slot * kHG;
      const float* slopes = s_slopes + s.hg * kHG;
      const int64_t qp = MODS && p.qpos ? p.qpos[s.t] : (int64_t)p.lengths[s.t] - 1;
      for (int k = 0; k < s.ntiles; ++k, ++g) {
        if (g % kGroups != (uint32_t)gi) continue;
        const uint32_t sb = g % C::NSB;
        const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16) + sb * C::S_COLS;
        const uint32_t pos = (uint32_t)(s.a & ~127) + 128u * (uint32_t)(s.tile0 + k) + tr;
        const bool in = pos >= (uint32_t)s.a && pos < (uint32_t)s.b;
        float old = 0.0f, dist = 0.0f;
        if (in) {
          old = p.mass[s.req * p.mass_st + pos];
          if (MODS && p.slopes) {
            const int64_t kp = p.kpos ? p.kpos[s.req * p.kp_stride + pos] : (int64_t)pos;
            dist = fabsf((float)(qp - kp));
          }
        }
        if (!wait_warp(s_full(sb), (g / C::NSB) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool valid = reinterpret_cast<const int*>(smem + C::MAP_OFF + (g % kMaps) * 512)[tr] >= 0;
        float2 scl = make_float2(1.0f, 1.0f);
        if (F8) scl = reinterpret_cast<const float2*>(smem + C::SC_OFF + 1024 * (g % C::NV))[tr];
        const float f = MODS ? p.sm_scale : c_log2;
        const float2 s0 = make_float2(scl.x, scl.x), s1 = make_float2(scl.y, scl.y), f2 = make_float2(f, f);
        float2 w2 = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int ch = 0; ch < (heads + 15) >> 4; ++ch) {
          uint32_t x0[16], x1[16];
          tmem_ld32_x16(tl + 16 * ch, x0);
          if (F8) tmem_ld32_x16(tl + 64 + 16 * ch, x1);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 n = *reinterpret_cast<const float2*>(nl + 16 * ch + i);
            float2 x = make_float2(u2f(x0[i]), u2f(x0[i + 1]));
            float2 q = f2;
            if (F8) {
              x = __ffma2_rn(make_float2(u2f(x1[i]), u2f(x1[i + 1])), s1, __fmul2_rn(x, s0));
              q = *reinterpret_cast<const float2*>(sq + 16 * ch + i);
            }
            if (MODS) {
              x = __fmul2_rn(x, q);
              x.x = modify(x.x, p.cap, inv_cap2, slopes[16 * ch + i] * dist) + n.x;
              x.y = modify(x.y, p.cap, inv_cap2, slopes[16 * ch + i + 1] * dist) + n.y;
            } else {
              x = __ffma2_rn(x, q, n);
            }
            w2 = __fadd2_rn(w2, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
          }
        }
        const float w = w2.x + w2.y;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s_empty(sb));
          mbar_arrive(map_empty(g % kMaps));
        }
        if (in) p.mass_out[s.req * p.mass_out_st + pos] = valid ? old + w : old;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(g_empty(slot));
    }
  } else {
    // ===================================================== softmax and outputs, 16 warps ===
    // Warp = lane quarter qd (keys 32 qd ..; output columns 32 qd .. of both halves), head group hq: the
    // heads from kHW hq on
    const int qd = warp & 3, hq = warp >> 2;
    constexpr int CH = kHW / 16, NP = kHW / 2;  // chunks of 16 heads, pairs
    const int hb = kHW * hq;
    const int tr = 32 * qd + lane;
    const int gid = threadIdx.x & 127;  // thread of the head group
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    float* red = reinterpret_cast<float*>(smem + C::RED_OFF);  // -m [2 buffers][64]
    float* red_alpha = red + 128;
    float* red_part = red + 192;  // [4 quarters][64 heads]
    float* red_inv = red + 448;
    float* red_raise = red + 512;
    float* red_top = red + 576;    // FP8: log2 of the tile's largest p * |scale|, [4 quarters][2 tiles][64], then
                                   // [2][64] what the accumulators take when m and the factors change
    float* red_wf = red + 1088;    // FP8: [2][64] weight = p * scale * this, a power of two
    float* red_ref = red + 1216;   // FP8: [2][64] log2 of the reference, relative to m
    float* red_own = red + 1344;   // FP8: [64] red_wf of the second tile over the group's factor
    float* red_grp = red + 1408 + 4 * hq;  // FP8: the group's factors of both tiles [2], its largest reference
                                           // of the first tile, its largest red_wf of the second
    const float inv_cap2 = MODS ? cap_factor(p.cap) : 0.0f;
    const float f = MODS ? p.sm_scale : p.sm_scale * kLog2e;
    uint32_t g = 0, mb = 0;
    bool first_query = true;
    bool failed = false;  // a wait ran out: go on without waiting, and leave with the group
    auto await = [&](uint32_t bar, uint32_t par) {
      if (failed || __all_sync(0xffffffffu, bar_wait(bar, par, abort_flag))) return;
      fail();
      failed = true;
    };
    auto pv_wait = [&](uint32_t last) { await(pv_done(last & 1), (last >> 1) & 1); };
    const uint32_t o_addr = tl + C::O_COL + hb;  // O^T half 0 (half 1 64 columns on), the group's heads
    // -m of a segment without a valid key so far is 0
    if (gid < kHW) red[hb + gid] = 0.0f;
    for (uint32_t sc = 0;; ++sc) {
      const uint32_t slot = sc % kSegs;
      await(g_full(slot), (sc / kSegs) & 1);
      if (F8 && !failed && segs[slot].type != 0) {
        if (first_query && segs[slot].ntiles > 0) {
          split_first(segs[slot], slot);
          first_query = false;
        }
        await(aux_full(slot), (sc / kSegs) & 1);
      }
      if (group_any(hq, failed)) break;
      const Seg& s = segs[slot];  // read where it is needed: registers are short in the loop over the tiles
      if (s.type == 0) break;
      const int heads = min(kHG, p.H - s.hg * kHG);
      // chunks of 16 heads in use: the weights of the others meet only unused columns of O^T
      const int nch = max(0, min(CH, (heads - hb + 15) >> 4));
      const float* slopes = s_slopes + s.hg * kHG + hb;
      const float* sq = reinterpret_cast<const float*>(smem + C::SQ_OFF) + kHG * slot + hb;
      int qp = 0;
      if (MODS) qp = p.qpos ? p.qpos[s.t] : (int)((uint32_t)p.lengths[s.t] - 1u);  // (used where there are tiles: a length above 0)
      float2 lsum[NP];  // heads 2 i, 2 i + 1 of the group
#pragma unroll
      for (int i = 0; i < NP; ++i) lsum[i] = make_float2(0.0f, 0.0f);
      bool fresh = true;  // no valid key so far: m counts as 0, no reference scale
      const int ntiles = s.ntiles;
      for (int k = 0; k < ntiles; ++k, ++g) {
        const uint32_t sb = g % C::NSB;
        float dist = 0.0f;
        if (MODS && p.slopes) {
          const uint32_t pos = (uint32_t)(s.a & ~127) + 128u * (uint32_t)(s.tile0 + k) + tr;
          int kp = (int)pos;
          if (p.kpos && pos >= (uint32_t)s.a && pos < (uint32_t)s.b) kp = p.kpos[s.req * p.kp_stride + pos];
          dist = fabsf((float)((int64_t)qp - kp));
        }
        await(s_full(sb), (g / C::NSB) & 1);
        tc_fence_after();
        const bool valid = reinterpret_cast<const int*>(smem + C::MAP_OFF + (g % kMaps) * 512)[tr] >= 0;
        float2 scl = make_float2(0.0f, 0.0f);
        if (F8) scl = reinterpret_cast<const float2*>(smem + C::SC_OFF + 1024 * (g % C::NV))[tr];
        // y = score - m, exp2 domain
        float2 y[NP];
        float top = -INFINITY;
        const float2 s0 = make_float2(scl.x, scl.x), s1 = make_float2(scl.y, scl.y), f2 = make_float2(f, f);
        const float* m = red + 64 * mb + hb;
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          if (ch < nch) {
            uint32_t x0[16], x1[16];
            tmem_ld32_x16(tl + sb * C::S_COLS + hb + 16 * ch, x0);
            if (F8) tmem_ld32_x16(tl + sb * C::S_COLS + 64 + hb + 16 * ch, x1);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 n = *reinterpret_cast<const float4*>(m + 16 * ch + i);
              float2 xa = make_float2(u2f(x0[i]), u2f(x0[i + 1])), xb = make_float2(u2f(x0[i + 2]), u2f(x0[i + 3]));
              float2 qa = f2, qb = f2;
              if (F8) {
                xa = __ffma2_rn(make_float2(u2f(x1[i]), u2f(x1[i + 1])), s1, __fmul2_rn(xa, s0));
                xb = __ffma2_rn(make_float2(u2f(x1[i + 2]), u2f(x1[i + 3])), s1, __fmul2_rn(xb, s0));
                const float4 q = *reinterpret_cast<const float4*>(sq + 16 * ch + i);
                qa = make_float2(q.x, q.y);
                qb = make_float2(q.z, q.w);
              }
              if (MODS) {
                const float* sl = slopes + 16 * ch + i;
                xa = __fmul2_rn(xa, qa);
                xb = __fmul2_rn(xb, qb);
                xa.x = modify(xa.x, p.cap, inv_cap2, sl[0] * dist) + n.x;
                xa.y = modify(xa.y, p.cap, inv_cap2, sl[1] * dist) + n.y;
                xb.x = modify(xb.x, p.cap, inv_cap2, sl[2] * dist) + n.z;
                xb.y = modify(xb.y, p.cap, inv_cap2, sl[3] * dist) + n.w;
              } else {
                xa = __ffma2_rn(xa, qa, make_float2(n.x, n.y));
                xb = __ffma2_rn(xb, qb, make_float2(n.z, n.w));
              }
              y[8 * ch + i / 2] = xa;
              y[8 * ch + i / 2 + 1] = xb;
              top = fmaxf(fmaxf(fmaxf(top, xa.x), fmaxf(xa.y, xb.x)), xb.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[8 * ch + i] = make_float2(-INFINITY, -INFINITY);
          }
        }
        if (__any_sync(0xffffffffu, !valid)) {
          if (!valid) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NP; ++i) y[i] = make_float2(-INFINITY, -INFINITY);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s_empty(sb));
          mbar_arrive(map_empty(g % kMaps));
        }
        bool exact = fresh;
        if (!exact) {
          bool stale = top > (F8 ? kStaleF8 : kStale);
          // (the most that any of the group's heads can make of this key: one that none of them reads passes,
          // whatever its scales; heads with factors far apart may take the exact path more often than they must)
          if (F8) stale = stale || ex2_approx(top) * fmaxf(fabsf(scl.x) * red_grp[0], fabsf(scl.y) * red_grp[3]) > kMostWeight;
          exact = group_any(hq, stale);
        }
        if (exact) {
          // exact maximum of the tile per head; the running maxima are raised to it. FP8: the largest weights
          // as well (unrolled: in a loop over the three the compiler spills, 488 us for 430 at 128 x 32768)
          float mine = -INFINITY;  // lane i ends with head i's
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float m0 = redux_max_f32(y[i].x), m1 = redux_max_f32(y[i].y);
            mine = lane == 2 * i ? m0 : (lane == 2 * i + 1 ? m1 : mine);
          }
          if (lane < kHW) red_part[64 * qd + hb + lane] = mine;
          if (F8) {
#pragma unroll 2
            for (int t = 0; t < 2; ++t) {
              const float ls = __log2f(fabsf(t == 0 ? scl.x : scl.y));
#pragma unroll
              for (int i = 0; i < NP; ++i) {
                const float m0 = redux_max_f32(y[i].x + ls), m1 = redux_max_f32(y[i].y + ls);
                mine = lane == 2 * i ? m0 : (lane == 2 * i + 1 ? m1 : mine);
              }
              if (lane < kHW) red_top[64 * (2 * qd + t) + hb + lane] = mine;
            }
          }
          const bool some = group_any(hq, valid);
          static_assert(2 * kHW == 32, "a lane of one warp per tile and head");
          if (gid < (F8 ? 2 * kHW : kHW)) {
            const int h = hb + (gid & (kHW - 1)), t = gid / kHW;
            // relative to what y was taken from; a first maximum may be below it. FP8: that is m plus the fold,
            // what of the first tile's reference is taken off as well
            const float* pt = red_part + h;
            const float up = fmaxf(fmaxf(pt[0], pt[64]), fmaxf(pt[128], pt[192]));
            const float mo = fresh ? 0.0f : -red[64 * mb + h];
            float fold = F8 && !fresh ? fold_of(red_ref[h], red_ref[64 + h], red_grp[2]) : 0.0f;
            float raise = fresh ? (up > kNoMax ? up : 0.0f) : fmaxf(up, -fold);
            if (F8) {
              // the power of two at or above the largest p * |scale| so far, p relative to the new m
              const int at = 64 * t + h;
              const float* tt = red_top + at;
              const float old = fresh ? -INFINITY : red_ref[at] - fold;
              const float seen = fmaxf(fmaxf(fmaxf(tt[0], tt[128]), fmaxf(tt[256], tt[384])), old) - raise;
              const float ref = fminf(fmaxf(ceilf(seen), (float)kRefLow), (float)kRefHigh);
              const float other = __shfl_xor_sync(0xffffffffu, ref, kHW);
              const float ref0 = t == 0 ? ref : other, ref1 = t == 0 ? other : ref;
              const int base = __reduce_max_sync(0xffffffffu, (int)ref0);
              fold = fold_of(ref0, ref1, (float)base);
              raise += fold;
              // the factors' exponents, biased; the first tile's are one another's but for folds at their limit
              const int w1 = 127 + kWeightShift - (int)ref1 + (int)fold;
              const int lo = __reduce_min_sync(0xffffffffu, w1), spread = __reduce_max_sync(0xffffffffu, w1) - lo;
              const int own = spread > kSpread ? min(w1 - lo, kOwn) : 0;
              const int e = t == 0 ? 127 + kWeightShift - base : lo + own;
              red_top[at] = ex2_approx((float)(e - (int)(f2u(red_wf[at]) >> 23)) - raise);
              red_wf[at] = u2f((uint32_t)e << 23);
              red_ref[at] = ref;
              if (t == 0) red_own[h] = u2f((uint32_t)(127 + own) << 23);
              if (gid == 0) {
                red_grp[0] = u2f((uint32_t)e << 23);
                red_grp[1] = u2f((uint32_t)lo << 23);
                red_grp[2] = (float)base;
                red_grp[3] = u2f((uint32_t)(lo + (spread > kSpread ? min(spread, kOwn) : 0)) << 23);
              }
            }
            if (t == 0) {
              red[64 * (mb ^ 1) + h] = -(mo + raise);
              red_raise[h] = raise;
              red_alpha[h] = ex2_approx(-raise);
            }
          }
          group_sync(hq);
          mb ^= 1;
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float2 up = *reinterpret_cast<const float2*>(red_raise + hb + 2 * i);
            y[i] = make_float2(y[i].x - up.x, y[i].y - up.y);
          }
          if (!fresh) {
#pragma unroll
            for (int i = 0; i < NP; ++i) lsum[i] = __fmul2_rn(lsum[i], *reinterpret_cast<const float2*>(red_alpha + hb + 2 * i));
            pv_wait(g - 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2 * CH; ++c) {  // half c / CH, 16 heads
              const int half = c / CH, h16 = 16 * (c % CH);
              const uint32_t addr = o_addr + 64 * half + h16;
              const float* al = (F8 ? red_top + 64 * half : red_alpha) + hb + h16;
              uint32_t o[16];
              tmem_ld32_x16(addr, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = f2u(u2f(o[i]) * al[i]);
              tmem_st32_x16(addr, o);
            }
            tc_wait_st();
          }
          fresh = fresh && !some;
        }
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          if (ch < nch) {
#pragma unroll
            for (int i = 8 * ch; i < 8 * ch + 8; ++i) {
              y[i] = make_float2(ex2_approx(y[i].x), ex2_approx(y[i].y));
              lsum[i] = __fadd2_rn(lsum[i], y[i]);
            }
          }
        }
        // the weights' buffer is free once the value product that read it is complete
        if (g >= C::PBUF) pv_wait(g - C::PBUF);
        uint8_t* prow = smem + C::P_OFF + (g % C::PBUF) * C::P_BYTES + tr * 128;
        const int sw = tr & 7;
#pragma unroll
        for (int h = 0; h < C::PN; ++h) {
          float wf = 1.0f;
          if (F8) {
            // the key's factor, held finite (a weight of 0 stays 0)
            wf = fminf(fmaxf((h == 0 ? scl.x : scl.y) * red_grp[h], -3.402823466e38f), 3.402823466e38f);
            if (h == 1 && red_grp[1] != red_grp[3]) {  // the heads' own factors
#pragma unroll
              for (int i = 0; i < NP; ++i) y[i] = __fmul2_rn(y[i], *reinterpret_cast<const float2*>(red_own + hb + 2 * i));
            }
          }
#pragma unroll
          for (int ch = 0; ch < CH; ++ch) {
            if (ch < nch) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (F8) {
                  const float2 v = __fmul2_rn(y[8 * ch + i], make_float2(wf, wf));
                  w[i] = f32x2_to_f16x2(v.x, v.y);
                } else {
                  w[i] = f32x2_to_bf16x2(y[8 * ch + i].x, y[8 * ch + i].y);
                }
              }
              uint8_t* d = prow + h * (kBN * 128);
              const int gr = (hb >> 3) + 2 * ch;
              *reinterpret_cast<uint4*>(d + ((gr ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(d + (((gr + 1) ^ sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(g % C::PBUF));
      }
      // ---- the segment's end: sums over the keys, then the group's columns of O^T
      {
        // reduce-scatter over the lanes: head i of the group ends in lanes i * 32 / kHW ..
        float v[kHW];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          v[2 * i] = lsum[i].x;
          v[2 * i + 1] = lsum[i].y;
        }
        constexpr int R = 32 / kHW;  // lanes per head
#pragma unroll
        for (int w = kHW / 2; w > 0; w >>= 1) {
          const bool upper = lane & (w * R);
#pragma unroll
          for (int i = 0; i < w; ++i)
            v[i] = (upper ? v[i + w] : v[i]) + __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + w], w * R);
        }
#pragma unroll
        for (int o = R / 2; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        if (lane % R == 0) red_part[64 * qd + hb + lane / R] = v[0];
      }
      group_sync(hq);
      const int part = 2 * cta + (s.kind == 1 ? 1 : 0);
      if (gid < kHW) {
        const int h = hb + gid;
        const float L = (red_part[h] + red_part[64 + h]) + (red_part[128 + h] + red_part[192 + h]);
        const float m = -red[64 * mb + h];
        red[64 * mb + h] = 0.0f;  // for the next segment
        red_inv[h] = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
        if (s.kind != 0) {
          p.ws_ml[(int64_t)part * 2 * kHG + h] = L == 0.0f ? kNoMax : m;
          p.ws_ml[(int64_t)part * 2 * kHG + kHG + h] = L;
        } else if (p.lse && h < heads) {
          p.lse[s.t * p.lse_st + s.hg * kHG + h] = L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
        }
      }
      group_sync(hq);
      if (s.ntiles > 0) pv_wait(g - 1);
      tc_fence_after();
      uint16_t* orow = p.out + (int64_t)s.t * p.out_st + (int64_t)s.hg * kHG * p.out_sh;
#pragma unroll 1
      for (int c = 0; c < 2 * CH; ++c) {  // half c / CH, 16 heads
        const int half = c / CH, h16 = 16 * (c % CH), h0 = hb + h16;
        if (h0 >= heads) continue;
        uint32_t o[16];
        if (s.ntiles > 0) {
          tmem_ld32_x16(o_addr + 64 * half + h16, o);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0u;
        }
        // FP8: the inverse of the weights' factor, a power of two, by its bits
        auto back = [&](int h) -> float { return F8 && !fresh ? u2f(0x7F000000u - f2u(red_wf[64 * half + h])) : 1.0f; };
        const int dv = 128 * half + tr;
        if (s.kind != 0) {
          float* prt = p.ws_o + ((int64_t)part * kHG + h0) * kD + dv;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (h0 + i < heads) prt[i * kD] = u2f(o[i]) * back(h0 + i);
        } else {
          // lanes 2i and 2i + 1 hold neighbouring columns: they swap heads, so that each writes
          // two columns of one head
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float e = u2f(o[2 * i]) * back(h0 + 2 * i) * red_inv[h0 + 2 * i];
            const float d = u2f(o[2 * i + 1]) * back(h0 + 2 * i + 1) * red_inv[h0 + 2 * i + 1];
            const bool odd = lane & 1;
            const float other = __shfl_xor_sync(0xffffffffu, odd ? e : d, 1);
            const uint32_t w = odd ? f32x2_to_bf16x2(other, d) : f32x2_to_bf16x2(e, other);
            const int h = h0 + 2 * i + (odd ? 1 : 0);
            if (h < heads) *reinterpret_cast<uint32_t*>(orow + h * p.out_sh + (dv & ~1)) = w;
          }
        }
      }
      // (the barrier at the next segment's start keeps it from rewriting sums still being read)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(g_empty(slot));
    }
  }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpScore) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Joins the parts of each split row in the order of the parts. Block (x, y) takes row x (when there
// are at most G rows; else the row that CTA x starts) and 64 / gridDim.y of its heads: 4 at once when
// there are at most kFewParts parts, else one after the other with 4 parts at a time, 64 threads for
// the 256 columns of each.
constexpr int kJoinThreads = 256;
constexpr int kFewParts = 8;
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Params p) {
  __shared__ int s_part[kMaxCtas + 1];
  __shared__ float s_w[kMaxCtas + 1];
  __shared__ int s_cnt[8];
  __shared__ float s_red[2][8];
  __shared__ float4 s_acc[kJoinThreads / 64][64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = p.ws_split[blockIdx.x];
  const int row = rec.x, c = rec.y, last = rec.z, total = rec.w;
  if (!record_valid(row, c, last, total, p.T * p.HG, p.G, (int)blockIdx.x)) return;  // (-1: a row that is not split)
  // the parts: of the CTA that starts the row, and of those after it to the one that finishes it whose
  // share is not empty (there are more CTAs than tiles then)
  const int k = c + 1 + tid;  // G is below the block's threads
  const uint32_t mem = __ballot_sync(0xffffffffu, k <= last && share(k, total, p.G) < share(k + 1, total, p.G));
  if (lane == 0) s_cnt[warp] = __popc(mem);
  __syncthreads();
  int at = 1, n = 1;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) at += s_cnt[w];
    n += s_cnt[w];
  }
  if ((mem >> lane) & 1) s_part[at + __popc(mem & ((1u << lane) - 1u))] = 2 * k;
  if (tid == 0) s_part[0] = 2 * c + 1;
  __syncthreads();
  const int64_t t = p.HG == 1 ? row : row >> 1;
  const int hg = p.HG == 1 ? 0 : row & 1;
  const int heads = min(kHG, p.H - hg * kHG);
  const int per = kHG / gridDim.y;
  const int col = tid & 63, pg = tid >> 6;
  if (n <= kFewParts) {
    // few parts: 4 heads at a time, 64 threads each, which read the parts' maxima and sums themselves
    for (int h = blockIdx.y * per + pg; h < (int)(blockIdx.y + 1) * per && h < heads; h += kJoinThreads / 64) {
      float m[kFewParts], l[kFewParts];
      float4 v[kFewParts];
      float M = kNoMax;
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        m[i] = kNoMax;
        l[i] = 0.0f;
        if (i < n) {
          const int64_t part = s_part[i];
          m[i] = p.ws_ml[part * 2 * kHG + h];
          l[i] = p.ws_ml[part * 2 * kHG + kHG + h];
          v[i] = *reinterpret_cast<const float4*>(p.ws_o + (part * kHG + h) * kD + 4 * col);
        }
      }
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) M = fmaxf(M, m[i]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float L = 0.0f;
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        if (i < n) {
          const float w = ex2_approx(m[i] - M);
          L = fmaf(w, l[i], L);
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
      }
      const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
      *reinterpret_cast<uint2*>(p.out + t * p.out_st + (int64_t)(hg * kHG + h) * p.out_sh + 4 * col) =
          make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
      if (col == 0 && p.lse) p.lse[t * p.lse_st + hg * kHG + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    return;
  }
  const int my_part = tid < n ? s_part[tid] : -1;  // n <= kMaxCtas + 1 < 256
  for (int h = blockIdx.y * per; h < (int)(blockIdx.y + 1) * per && h < heads; ++h) {
    // the parts' weights 2^(m - M), M their largest maximum, and the sum of the weighted sums
    float m = kNoMax, l = 0.0f;
    if (my_part >= 0) {
      m = p.ws_ml[(int64_t)my_part * 2 * kHG + h];
      l = p.ws_ml[(int64_t)my_part * 2 * kHG + kHG + h];
    }
    // the first loads of the sum do not wait for the weights
    constexpr int kGroups = kJoinThreads / 64, kAhead = 8;
    float4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int q = pg + kGroups * i;
      if (q < n) v[i] = *reinterpret_cast<const float4*>(p.ws_o + ((int64_t)s_part[q] * kHG + h) * kD + 4 * col);
    }
    if (warp < 8) {
      float x = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      if (lane == 0) s_red[0][warp] = x;
    }
    __syncthreads();
    float M = s_red[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) M = fmaxf(M, s_red[0][w]);
    if (warp < 8) {
      const float w = ex2_approx(m - M);
      if (my_part >= 0) s_w[tid] = w;
      float x = w * l;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) s_red[1][warp] = x;
    }
    __syncthreads();
    float L = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) L += s_red[1][w];
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int q0 = pg; q0 < n; q0 += kGroups * kAhead) {
      if (q0 != pg) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int q = q0 + kGroups * i;
          if (q < n) v[i] = *reinterpret_cast<const float4*>(p.ws_o + ((int64_t)s_part[q] * kHG + h) * kD + 4 * col);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int q = q0 + kGroups * i;
        if (q < n) {
          const float w = s_w[q];
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
      }
    }
    s_acc[pg][col] = acc;
    __syncthreads();
    if (pg == 0) {
      const float inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
      for (int i = 1; i < kGroups; ++i) {
        const float4 x = s_acc[i][col];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      *reinterpret_cast<uint2*>(p.out + t * p.out_st + (int64_t)(hg * kHG + h) * p.out_sh + 4 * col) =
          make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
      if (tid == 0 && p.lse) p.lse[t * p.lse_st + hg * kHG + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    __syncthreads();
  }
}

// Host checks shared by the entry points.
dsa_status_t check(const dsa_paged_args_t* a, bool mass) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->kind != DSA_CACHE_BF16 && a->kind != DSA_CACHE_FP8_SCALED) return DSA_ERR_INVALID_ARGUMENT;
  if (a->T < 0 || a->H < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (a->H > kMaxHeads || a->T > (1 << 24) || a->d_nope != kD || a->d_rope != 0 || a->d_v != kD)
    return DSA_ERR_UNSUPPORTED;
  if (a->T == 0) return DSA_OK;
  // more rows than any device holds: slots fit 31 bits
  if (a->num_slots > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
  if (!a->q || !a->cache || !a->lengths || a->num_slots < 0 || a->num_requests < 1) return DSA_ERR_INVALID_ARGUMENT;
  if (!a->req_of_token && a->T > a->num_requests) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(a->q, 16) || a->q_stride_t % 8 || a->q_stride_h % 8 || a->q_stride_t < 0 || a->q_stride_h < 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(a->cache, 16) || !aligned(a->lengths, 4)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->block_table && (a->page_size < 1 || a->max_pages < 0 || a->bt_stride < a->max_pages))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->key_positions && (a->kp_width < 0 || a->kp_stride < a->kp_width)) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(a->sm_scale) || !std::isfinite(a->logit_cap) || a->logit_cap < 0.0f)
    return DSA_ERR_INVALID_ARGUMENT;
  if (mass) return a->lse ? DSA_OK : DSA_ERR_INVALID_ARGUMENT;
  if (!a->out || !aligned(a->out, 16) || a->out_stride_t % 8 || a->out_stride_h % 8 || a->out_stride_h < kD ||
      a->out_stride_t < 0 || (a->T > 1 && a->out_stride_t < kD))
    return DSA_ERR_INVALID_ARGUMENT;
  return DSA_OK;
}

Params make_params(const dsa_paged_args_t* a) {
  Params p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_st = a->q_stride_t;
  p.q_sh = a->q_stride_h;
  p.T = a->T;
  p.H = a->H;
  p.HG = (a->H + kHG - 1) / kHG;
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.num_slots = a->num_slots;
  p.bt = a->block_table;
  p.bt_stride = a->bt_stride;
  p.page_size = a->block_table ? a->page_size : 1;
  {
    // round-up reciprocal: with l = ceil(log2 d) and m = ceil(2^(31+l) / d) < 2^32,
    // floor(x * m / 2^(31+l)) == floor(x / d) for every 0 <= x < 2^31
    const uint64_t d = (uint64_t)p.page_size;
    int l = 0;
    while ((1ull << l) < d) ++l;
    p.pg_mul = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
    p.pg_shift = 31 + l;
  }
  p.pos_limit = a->block_table ? (int64_t)a->max_pages * a->page_size : a->num_slots;
  if (a->key_positions && a->kp_width < p.pos_limit) p.pos_limit = a->kp_width;
  p.num_requests = a->num_requests;
  p.req = a->req_of_token;
  p.starts = a->starts;
  p.lengths = a->lengths;
  p.qpos = a->q_positions;
  p.kpos = a->key_positions;
  p.kp_stride = a->kp_stride;
  p.sm_scale = a->sm_scale;
  p.cap = a->logit_cap;
  p.slopes = a->slopes;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_st = a->out_stride_t;
  p.out_sh = a->out_stride_h;
  p.lse = a->lse;
  p.lse_st = a->H;
  p.err = a->error_word;
  return p;
}

// Workspace: partial outputs, their maxima and sums, then the split's records.
struct Ws {
  size_t o, ml, split, bytes;
};
Ws ws_layout(int G) {
  Ws w;
  w.o = 0;
  w.ml = w.o + (size_t)2 * G * kHG * kD * 4;
  w.split = w.ml + (size_t)2 * G * 2 * kHG * 4;
  w.bytes = w.split + (size_t)G * sizeof(int4);
  return w;
}

int64_t most_tiles(const Params& p) { return (p.pos_limit < 0x7FFFFFFF ? p.pos_limit : 0x7FFFFFFF) / kBN + 1; }
// The rows' costs must add up within 31 bits.
bool splittable(const Params& p) { return p.T * p.HG * (most_tiles(p) + kRowOverhead) <= 0x7FFFFFFF; }

// One CTA per SM, and no more than there can be tiles.
int grid_of(const Params& p, const DeviceInfo& dev) {
  const int sms = dev.sm_count < kMaxCtas ? dev.sm_count : kMaxCtas;
  const int64_t most = p.T * p.HG * most_tiles(p);
  return (int)(most < sms ? most : sms);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// 2-D map over the bf16 rows, box 64 columns x p->box_rows rows, 128-byte swizzle: the K-major layout
// the products read. box_rows is what a page and a tile share, a power of two; the swizzle repeats
// every eight rows, so smaller shares go without a map.
dsa_status_t encode_rows(Params* p, CUtensorMap* map) {
  int box = kBN;
  if (p->bt)
    while (p->page_size % box) box >>= 1;
  p->box_rows = 0;
  if (box < 8 || p->num_slots < box) return DSA_OK;
  static std::mutex mu;
  static EncodeFn fn = nullptr;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!fn) {
      void* f = nullptr;
      cudaDriverEntryPointQueryResult qres;
      const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qres);
      if (e != cudaSuccess) return cuda_fail(e);
      if (!f || qres != cudaDriverEntryPointSuccess) return cuda_fail(cudaErrorSymbolNotFound);
      fn = reinterpret_cast<EncodeFn>(f);
    }
  }
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)p->num_slots};
  const cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
  const cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  const cuuint32_t es[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint8_t*>(p->cache), dims, strides, boxes, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return cuda_fail(cudaErrorInvalidValue);
  p->box_rows = box;
  return DSA_OK;
}

template <int KIND, bool MASS, bool MODS>
cudaError_t launch_one(const Params& p, const CUtensorMap& map, cudaStream_t s) {
  paged_kernel<KIND, MASS, MODS><<<(unsigned)p.G, kThreads, Cfg<KIND, MASS>::SMEM_BYTES, s>>>(p, map);
  return cudaGetLastError();
}

template <bool MASS>
dsa_status_t launch(Params p, int kind, cudaStream_t s) {
  const bool mods = p.cap > 0.0f || p.slopes;
  CUtensorMap map{};
  cudaError_t e;
  if (kind == DSA_CACHE_BF16) {
    const dsa_status_t st = encode_rows(&p, &map);
    if (st != DSA_OK) return st;
    e = mods ? launch_one<DSA_CACHE_BF16, MASS, true>(p, map, s) : launch_one<DSA_CACHE_BF16, MASS, false>(p, map, s);
  } else {
    e = mods ? launch_one<DSA_CACHE_FP8_SCALED, MASS, true>(p, map, s)
             : launch_one<DSA_CACHE_FP8_SCALED, MASS, false>(p, map, s);
  }
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

template <int KIND, bool MASS, bool MODS>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(paged_kernel<KIND, MASS, MODS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<KIND, MASS>::SMEM_BYTES);
}

// The kernels' shared-memory limits, once per device.
dsa_status_t prepare_kernels(int device) {
  static std::mutex mu;
  static bool done[64];
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return DSA_OK;
  cudaError_t e = cudaSuccess;
  if ((e = allow_smem<DSA_CACHE_BF16, false, false>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_BF16, false, true>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_BF16, true, false>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_BF16, true, true>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_FP8_SCALED, false, false>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_FP8_SCALED, false, true>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_FP8_SCALED, true, false>()) != cudaSuccess ||
      (e = allow_smem<DSA_CACHE_FP8_SCALED, true, true>()) != cudaSuccess)
    return cuda_fail(e);
  done[device] = true;
  return DSA_OK;
}

}  // namespace paged
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_paged_attn_workspace_size(const dsa_paged_args_t* a, size_t* bytes) {
  if (!a || !bytes || a->T < 0 || a->H < 1) return DSA_ERR_INVALID_ARGUMENT;
  DeviceInfo dev;
  const dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  *bytes = paged::ws_layout(dev.sm_count < paged::kMaxCtas ? dev.sm_count : paged::kMaxCtas).bytes;
  return DSA_OK;
}

extern "C" dsa_status_t dsa_paged_attn(const dsa_paged_args_t* a, void* stream) {
  dsa_status_t st = paged::check(a, false);
  if (st != DSA_OK || a->T == 0) return st;
  paged::Params p = paged::make_params(a);
  if (!paged::splittable(p)) return DSA_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  p.G = paged::grid_of(p, dev);
  const paged::Ws w = paged::ws_layout(p.G);
  if (!a->workspace || !aligned(a->workspace, 256)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->workspace_bytes < w.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p.ws_o = reinterpret_cast<float*>(ws + w.o);
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
  p.ws_split = reinterpret_cast<int4*>(ws + w.split);
  if ((st = paged::prepare_kernels(dev.device)) != DSA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = paged::launch<false>(p, a->kind, s)) != DSA_OK) return st;
  if (p.G == 1) return DSA_OK;  // no border, nothing to join
  // the join's blocks: a row (or CTA) each, times a head each where few rows can have many parts, four
  // heads (one pass over few parts) where there are more rows
  const int64_t nrows = p.T * p.HG;
  const int x = (int)(nrows <= p.G ? nrows : p.G);
  const int y = x <= 16 ? 64 : 16;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)x, (unsigned)y);
  cfg.blockDim = dim3(paged::kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged::join_kernel, p);
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

extern "C" dsa_status_t dsa_paged_attn_mass(const dsa_paged_args_t* a, const float* mass, int64_t mass_stride,
                                            float* mass_out, int64_t mass_out_stride, int64_t mass_width,
                                            void* stream) {
  dsa_status_t st = paged::check(a, true);
  if (st != DSA_OK || a->T == 0) return st;
  if (!mass || !mass_out || mass_width < 0 || mass_stride < mass_width || mass_out_stride < mass_width)
    return DSA_ERR_INVALID_ARGUMENT;
  if (mass_out == mass && mass_out_stride != mass_stride) return DSA_ERR_INVALID_ARGUMENT;  // in place: the same rows
  paged::Params p = paged::make_params(a);
  if (mass_width < p.pos_limit) p.pos_limit = mass_width;
  if (!paged::splittable(p)) return DSA_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  p.mass = mass;
  p.mass_st = mass_stride;
  p.mass_out = mass_out;
  p.mass_out_st = mass_out_stride;
  p.HG = 1;
  p.G = paged::grid_of(p, dev);
  if ((st = paged::prepare_kernels(dev.device)) != DSA_OK) return st;
  // 64 heads per launch: a second one adds the others' weights to the first's result
  for (int h = 0; h < a->H; h += paged::kHG) {
    p.q = static_cast<const uint16_t*>(a->q) + h * a->q_stride_h;
    p.lse = a->lse + h;
    p.slopes = a->slopes ? a->slopes + h : nullptr;
    p.H = a->H - h < paged::kHG ? a->H - h : paged::kHG;
    if ((st = paged::launch<true>(p, a->kind, static_cast<cudaStream_t>(stream))) != DSA_OK) return st;
    p.mass = mass_out;
    p.mass_st = mass_out_stride;
  }
  return DSA_OK;
}
