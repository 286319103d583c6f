// dsa_block_scores.cu - a cheap score of each block (page) for each token:
//   scores[t, b] = sum_h w[t,h] * max(0, sm_scale * q[t,h] . summary[page of b]).
//
// Transposed products: S^T[block, head] = P Q^T with M = 128 blocks and, as N, the heads of up to
// 256 / H neighbouring tokens (tcgen05 kind::f16, fp32 accumulators in tensor memory). A block is then a
// lane of tensor memory, so the sum over heads stays within a thread: no shuffle, and what a block's row
// holds (NaN, infinities, nothing) reaches its own scores only. Tokens of one request share the tile of
// summaries; where a group of tokens has several requests, each run of equal ones is a product of its
// own over its part of the query rows.
//
// One CTA per SM walks units (group of tokens, part of its block tiles). Warps 0-15 sum up and store, 16-19 load
// summaries (cp.async, row by row: pages are scattered), a column quarter each, through a ring of three halves of a
// tile, 20 issues the products, 21-22 load queries, up to four groups ahead where they are small, 23 loads weights.
// Two accumulators let the products of a tile run while the one before it is summed up. Every wait is bounded.
//
// 4096 tokens of 64 heads, half of them over 2016 to 2048 blocks and half over 909 to 941, 198 GFLOP, take 144
// us in a graph of calls (1.37 PFLOP/s). At the measured matrix rate, 1929.7 TFLOP/s, it would be 103, 107 with the tiles'
// empty rows, and 116 for the 88 tiles of the busiest SM (the mean is 81); by the tensor pipe's own cycles at the 1.92 GHz
// seen here, 92 for those 88. With parts of the work left out, the whole being 146 as the replay of one call: 121
// without queries and sums (what is above the products is waits and commits between them), 129 without queries, 139
// without sums. A group's queries fill the room that there is for them, so the next ones come in between two
// groups. The warp that issues keeps all its state uniform and elects
// a thread: with a fixed thread the operands went through registers first, 168 us for 152.
// 256 requests of up to 512 blocks, 47 MB, take 18.5 us, 11.6 where they lie in L2 (HBM: 7): 128 units of two tokens,
// so 24 SMs have none and the busiest has 7 tiles of a mean of 4.6; and chains of loads (lengths, pages, rows) at
// the start of each, and of hand-offs per tile.
//
// Two issuing warps taking tiles in turn ran the products faster (111 without queries and sums) and the whole slower
// (166 with a token between them, 183 to 210 without: tiles that run at the same time end at the same time, and their
// sums then have nothing to run beside).
// Queries by TMA: 142 to 144 for 146, for a tensor map that each call has to encode (1 us of a small call's 10).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "dsa_host.h"
#include "dsa_paged_wait.cuh"
#include "dsa_ptx.cuh"

namespace dsa {
namespace scores {

using paged::bar_wait;
using paged::bar_wait_row;

constexpr int kD = 256;
constexpr int kMaxHeads = 128;
constexpr int kBM = 128;     // blocks per tile (MMA M)
constexpr int kMaxN = 256;   // query rows per group (MMA N)
constexpr int kChunks = kD / 64;
constexpr int N = 16;        // heads summed up per step
constexpr int kStages = 3;   // halves of a tile's columns
constexpr int kTurns = 2;    // warps per accumulator and lane quarter: they take its tokens in turn
constexpr int kSumWarps = 8 * kTurns;
constexpr int kWarpLoad0 = kSumWarps, kLoadWarps = 4, kWarpMma = kWarpLoad0 + kLoadWarps, kWarpQuery = kWarpMma + 1,
              kQueryWarps = 2, kWarpWeights = kWarpQuery + kQueryWarps;
constexpr int kWarps = kWarpWeights + 1;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSlots = 4;  // query groups in shared memory, where they are small
constexpr uint32_t kChunkBytes = kBM * 128;
constexpr uint32_t kQueryBytes = kMaxN * kD * 2;
constexpr uint32_t kRingOff = kQueryBytes;
constexpr uint32_t kWeightOff = kRingOff + kStages * 2 * kChunkBytes;
constexpr uint32_t kMiscOff = kWeightOff + kMaxN * 4;
constexpr uint32_t kSmemBytes = kMiscOff + 512 + 1024;  // and room to align

struct Params {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int64_t T;
  int H, HP;  // heads, rounded up to a multiple of 16
  int G;      // tokens per group
  int slots;  // groups of query rows that fit
  int parts;  // units per group
  int units;
  const uint16_t* summary;
  int64_t num_pages;
  const int32_t* bt;
  int64_t bt_st;
  int page;
  int most;   // blocks that the table and the scores hold
  int64_t num_requests;
  const int32_t *req, *lengths;
  float scale;
  const float* w;
  float* out;
  int64_t out_st;
  int32_t* err;
};

// max(x, 0) that passes NaN on
__device__ __forceinline__ float relu(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Waits for tensor-memory loads; the registers pass through, so that no use of them moves before it.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One thread of the warp, chosen by the hardware: the same one every time (a commit covers its own thread's products).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void set_err(int32_t* err, int bit) {
  if (err) atomicOr(err, bit);
}

// The tiles of this CTA's units in order; every warp walks them for itself. Lane i holds token i of the
// unit's group; the requests and lengths of the next two units are on their way meanwhile (units may be
// one tile long, shorter than a load).
struct Walk {
  int u;                 // unit
  int t0, part;          // first token of its group, its part of the tiles
  int step_t, step_part; // from one unit of this CTA to the next, before the carry
  int req, nb;           // lane: request, blocks
  int count;             // tokens of the group
  int a, b;              // the run: tokens a .. b - 1 share a request
  int blocks;            // most blocks of a token of the run
  int m, m_end;          // tile, end of the run's tiles in this part
  int ahead_t, ahead_part;
  int req1, len1, req2, len2;

  __device__ __forceinline__ void advance(const Params& p, int& t, int& part_) const {
    t += step_t;
    part_ += step_part;
    if (part_ >= p.parts) {
      part_ -= p.parts;
      t += p.G;
    }
  }
  __device__ __forceinline__ void fetch(const Params& p, int unit, int first, int& r, int& len) const {
    const int lane = threadIdx.x & 31;
    r = len = 0;
    if (unit < p.units && lane < p.G && first + lane < p.T) {
      r = p.req ? p.req[first + lane] : first + lane;
      len = p.lengths[first + lane];
    }
  }
  __device__ __forceinline__ void start(const Params& p) {
    const int grid = (int)gridDim.x;
    step_t = grid / p.parts * p.G;
    step_part = grid % p.parts;
    u = (int)blockIdx.x - grid;
    ahead_t = (int)blockIdx.x / p.parts * p.G;
    ahead_part = (int)blockIdx.x % p.parts;
    a = b = count = m = m_end = t0 = part = 0;
    fetch(p, u + grid, ahead_t, req1, len1);
    int t = ahead_t, q = ahead_part;
    advance(p, t, q);
    fetch(p, u + 2 * grid, t, req2, len2);
  }
  // The next tile; false at the end. `report`: whether this warp tells of tokens that cannot be scored.
  __device__ __forceinline__ bool next(const Params& p, bool report = false) {
    if (++m < m_end) return true;
    const int lane = threadIdx.x & 31, grid = (int)gridDim.x;
    for (;;) {
      if (b >= count) {  // the next unit
        u += grid;
        if (u >= p.units) return false;
        t0 = ahead_t;
        part = ahead_part;
        advance(p, ahead_t, ahead_part);
        count = p.T - t0 < p.G ? (int)(p.T - t0) : p.G;
        req = req1;
        const int n = len1 > 0 ? (int)((uint32_t)(len1 - 1) / (uint32_t)p.page) + 1 : 0;
        req1 = req2;
        len1 = len2;
        nb = n < p.most ? n : p.most;
        bool bad = n > p.most;
        if (req < 0 || req >= p.num_requests) {
          bad = true;
          nb = 0;
        }
        if (lane >= count) nb = 0;
        if (report && bad && lane < count && part == 0) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        b = 0;
        int t = ahead_t, q = ahead_part;
        advance(p, t, q);
        fetch(p, u + 2 * grid, t, req2, len2);
      }
      a = b;
      const int r = __shfl_sync(0xffffffffu, req, a);
      const uint32_t other = __ballot_sync(0xffffffffu, lane > a && (lane >= count || req != r));
      b = other ? __ffs(other) - 1 : 32;
      blocks = __reduce_max_sync(0xffffffffu, lane >= a && lane < b ? nb : 0);
      const int tiles = (blocks + kBM - 1) / kBM;
      m = 0;
      m_end = tiles;
      if (p.parts > 1) {
        m = tiles * part / p.parts;
        m_end = tiles * (part + 1) / p.parts;
      }
      if (m < m_end) return true;
    }
  }
  __device__ __forceinline__ int64_t run_req() const { return __shfl_sync(0xffffffffu, req, a); }
};

// WHOLE: the heads fill steps of N.
template <bool WEIGHTS, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 1) scores_kernel(const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t bars = base + kMiscOff;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  constexpr int kQBar = 2 * kStages, kAccBar = kQBar + 2 * kMaxSlots, kWBar = kAccBar + 4;
  auto q_full = [&](int s) { return bars + 8 * (kQBar + s); };
  auto q_empty = [&](int s) { return bars + 8 * (kQBar + kMaxSlots + s); };
  auto acc_full = [&](int s) { return bars + 8 * (kAccBar + s); };
  auto acc_empty = [&](int s) { return bars + 8 * (kAccBar + 2 + s); };
  const uint32_t w_full = bars + 8 * kWBar, w_empty = w_full + 8;
  constexpr int kBars = kWBar + 3;
  static_assert(8 * kBars + 12 <= 512, "barriers");
  const uint32_t drained = bars + 8 * (kBars - 1);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + kMiscOff + 8 * kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff + 8 * kBars + 4);
  volatile int* progress = reinterpret_cast<volatile int*>(smem + kMiscOff + 8 * kBars + 8);  // tiles issued
  float* weights = reinterpret_cast<float*>(smem + kWeightOff);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), kLoadWarps / 2);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(q_full(s), kQueryWarps);
      mbar_init(q_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full(s), 1);
      mbar_init(acc_empty(s), kSumWarps / 2);
    }
    mbar_init(w_full, 1);
    mbar_init(w_empty, kSumWarps);
    mbar_init(drained, 1);
    *abort = *progress = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&]() {
    *abort = 1;
    if (lane == 0) set_err(p.err, DSA_DEVERR_TIMEOUT);
  };
  // one answer for the warp, also where the limit runs out between two lanes' attempts
  auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity, abort)) != 0; };
  // for all tiles of a unit, however many: the limit starts anew with every tile
  auto wait_unit = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, bar_wait_row(bar, parity, abort, progress)) != 0;
  };
  const uint32_t row_bytes_q = (uint32_t)(p.G * p.HP) * 128;  // one column quarter of a group's rows
  Walk k;
  k.start(p);

  if (warp >= kWarpLoad0 && warp < kWarpLoad0 + kLoadWarps) {
    // ---- summaries: warp w brings column quarter w of every tile, four rows per instruction. (All four on each
    // quarter, 32 rows each, took a hand-over per warp and quarter: 512 cycles, a quarter's products, did not do.)
    const int w = warp - kWarpLoad0;
    const uint32_t sub = lane >> 3, piece = lane & 7;
    uint32_t dst[2];  // rows 4 i + sub alternate between two places in the swizzle
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) dst[i] = (4 * i + sub) * 128 + ((piece ^ (4 * i + sub)) << 4);
    // the next tile's pages (rows 32 i + lane) are loaded ahead, and looked at when its turn has come
    int page[4], blocks = 0;
    bool more;
    auto load_pages = [&]() {
      more = k.next(p, w == 0);
      if (!more) return;
      const int32_t* from = p.bt + k.run_req() * p.bt_st + k.m * kBM + lane;
      blocks = k.blocks - k.m * kBM;
#pragma unroll
      for (int i = 0; i < 4; ++i) page[i] = 32 * i + lane < blocks ? from[32 * i] : -1;
    };
    int stage = w >> 1;
    uint32_t phase = 0;
    load_pages();
    while (more) {
      int now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        now[i] = page[i];
        if (now[i] >= p.num_pages) now[i] = -1;
        if (w == 0 && now[i] < 0 && 32 * i + lane < blocks) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
      }
      load_pages();
      // (one issuing warp reads the halves in order: so the phase two rounds before, of the same parity, is past)
      if (!wait(empty(stage), phase ^ 1)) {
        give_up();
        break;
      }
      // rows without a summary keep what the stage holds: their lanes are not read
      const uint32_t to = base + kRingOff + (2 * stage + (w & 1)) * kChunkBytes;
      const uint16_t* from = p.summary + 64 * w + 8 * piece;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int pg = __shfl_sync(0xffffffffu, now[i >> 3], 4 * (i & 7) + sub);
        if (pg >= 0) cp16(to + dst[i & 1] + 1024 * (i >> 1), from + (int64_t)pg * kD);
      }
      // the writer's fence makes the copies visible to the tensor core: one at the reader would hold up the products
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(stage));
      stage += 2;
      if (stage >= kStages) {
        stage -= kStages;
        phase ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kWarpQuery && warp < kWarpQuery + kQueryWarps) {
    // ---- queries: a group's rows once per unit
    const int w = warp - kWarpQuery;
    int slot = 0;
    uint32_t phase = 0;
    int last = -1;
    while (k.next(p)) {
      if (k.u == last) continue;
      last = k.u;
      if (!wait_unit(q_empty(slot), phase ^ 1)) {
        give_up();
        break;
      }
      const uint32_t c = lane >> 3, piece = lane & 7;
      const uint32_t to = base + (uint32_t)slot * kChunks * row_bytes_q + c * row_bytes_q;
      for (int i = 0; i < k.count; ++i) {
        const uint16_t* src = p.q + (int64_t)(k.t0 + i) * p.q_st + 8 * lane;
        const int n0 = i * p.HP;
#pragma unroll 8
        for (int h = w; h < p.H; h += kQueryWarps)
          cp16(to + (n0 + h) * 128 + ((piece ^ (h & 7)) << 4), src + h * p.q_sh);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(slot));
      if (p.slots == 1 && k.u + (int)gridDim.x < p.units) {
        const int n = (int)(p.T - k.ahead_t < p.G ? p.T - k.ahead_t : p.G) * p.H;
        for (int i = w * 32 + lane; i < n; i += 32 * kQueryWarps)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                           p.q + (int64_t)(k.ahead_t + i / p.H) * p.q_st + (int64_t)(i % p.H) * p.q_sh),
                       "r"(2 * kD)
                       : "memory");
        __syncwarp();
      }
      if (++slot == p.slots) {
        slot = 0;
        phase ^= 1;
      }
    }
  } else if (warp == kWarpWeights) {
    // ---- weights: w * sm_scale, a group's once per unit, the next one's in registers by the time their place is free
    uint32_t phase = 0;
    int last = -1;
    while (WEIGHTS && k.next(p)) {
      if (k.u == last) continue;
      last = k.u;
      float v[kMaxN / 32];
      const float* from = p.w + (int64_t)k.t0 * p.H;
#pragma unroll
      for (int z = 0; z < kMaxN / 32; ++z) {
        const int n = 32 * z + lane, i = n / p.HP, h = n - i * p.HP;
        v[z] = i < k.count && h < p.H ? from[i * p.H + h] : 0.0f;
      }
      if (!wait_unit(w_empty, phase ^ 1)) {
        give_up();
        break;
      }
#pragma unroll
      for (int z = 0; z < kMaxN / 32; ++z) weights[32 * z + lane] = v[z] * p.scale;
      __syncwarp();
      if (lane == 0) mbar_arrive(w_full);
      phase ^= 1;
    }
  } else if (warp == kWarpMma) {
    // ---- products
    const uint64_t d0 = sw128_desc(0, 16, 1024);
    const uint32_t d_hi = (uint32_t)(d0 >> 32), d_lo = (uint32_t)d0;
    int stage = 0, slot = -1, buf = 0;
    uint32_t phase = 0, q_phase = 0, acc_phase = 0;
    int last = -1, tiles = 0;
    bool ok = true, released = true;
    bool more = k.next(p);
    while (more) {
      const bool fresh = k.u != last;
      if (fresh) {
        if (!released && elect_one()) mma_commit(q_empty(slot));
        __syncwarp();
        if (++slot == p.slots) {
          slot = 0;
          q_phase ^= 1;
        }
        last = k.u;
        released = false;
      }
      // after a unit's last tile its query rows may go; else the next unit finds out
      const bool ends = k.m + 1 >= k.m_end && !__any_sync(0xffffffffu, lane >= k.b && k.nb > 0);
      released |= ends;
      const uint32_t idesc = idesc_bf16(kBM, (k.b - k.a) * p.HP, 0, 0);
      const uint32_t acc = tmem + buf * kMaxN;
      const uint32_t q_lo = d_lo | ((base + (uint32_t)slot * kChunks * row_bytes_q + (uint32_t)(k.a * p.HP) * 128) >> 4);
      if (!wait(acc_empty(buf), acc_phase ^ 1) || (fresh && !wait(q_full(slot), q_phase))) {
        give_up();
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {  // a half: one wait and one commit for eight products
        if (!wait(full(stage), phase)) {
          give_up();
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t a_lo = d_lo | ((base + kRingOff + 2 * stage * kChunkBytes) >> 4);
          const uint32_t b_lo = q_lo + c * (row_bytes_q >> 4);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t da = (s >> 2) * (kChunkBytes >> 4) + 2 * (s & 3), db = (s >> 2) * (row_bytes_q >> 4) + 2 * (s & 3);
            if (c == 0 && s == 0)
              mma_bf16_lohi<0>(acc, a_lo, d_hi, b_lo, d_hi, idesc);
            else
              mma_bf16_lohi<1>(acc, a_lo + da, d_hi, b_lo + db, d_hi, idesc);
          }
          mma_commit(empty(stage));
          if (c + 2 == kChunks) {
            mma_commit(acc_full(buf));
            if (ends) mma_commit(q_empty(slot));
          }
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
        if (c == 0) more = k.next(p);  // while the products of the first half run
      }
      if (!ok) break;
      if (lane == 0) *progress = ++tiles;
      buf ^= 1;
      acc_phase ^= buf == 0;
    }
    // every product ends before tensor memory is given back
    if (elect_one()) mma_commit(drained);
    __syncwarp();
    bar_wait(drained, 0, nullptr);
  } else {
    // ---- sums over heads: a block per lane, tiles in turn between the warps of either accumulator
    const int buf = warp / (4 * kTurns), first = (warp >> 2) % kTurns, quarter = warp & 3;
    uint32_t phase = 0, w_phase = 0;
    int last = -1;
    bool mine = buf != 0;
    const uint64_t scale2 = pack2(p.scale, p.scale);
    const uint32_t acc0 = tmem + buf * kMaxN + ((uint32_t)(32 * quarter) << 16);
    while (k.next(p)) {
      mine = !mine;
      if (WEIGHTS && k.u != last) {
        if (last >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(w_empty);
        }
        last = k.u;
        if (!wait(w_full, w_phase)) {
          give_up();
          break;
        }
        w_phase ^= 1;
      }
      if (!mine) continue;
      const int row = k.m * kBM + 32 * quarter + lane;  // the thread's block
      const int64_t r = k.run_req();
      int page = -1;
      if (row < k.blocks) page = p.bt[r * p.bt_st + row];
      if (!wait(acc_full(buf), phase)) {
        give_up();
        break;
      }
      phase ^= 1;
      tc_fence_after();
      // while one warp waits for its products, the others of its scheduler sum up theirs
      for (int i = k.a + first; i < k.b; i += kTurns) {
        const uint32_t col = acc0 + (i - k.a) * p.HP;
        const float4* w = reinterpret_cast<const float4*>(weights + i * p.HP);
        uint64_t sum[4] = {0, 0, 0, 0};  // chains of pairs of heads
        for (int h0 = 0; h0 < p.HP; h0 += N) {
          uint32_t x[N];
          tmem_ld32_x16(col + h0, x);
          wait_ld(x);
#pragma unroll
          for (int j = 0; j < N / 4; ++j) {
            float u[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              u[z] = relu(__uint_as_float(x[4 * j + z]));
              if (!WHOLE && h0 + 4 * j + z >= p.H) u[z] = 0.0f;  // heads that are not there
            }
            if (WEIGHTS) {
              const float4 f = w[h0 / 4 + j];
              sum[2 * (j & 1)] = fma2(pack2(u[0], u[1]), pack2(f.x, f.y), sum[2 * (j & 1)]);
              sum[2 * (j & 1) + 1] = fma2(pack2(u[2], u[3]), pack2(f.z, f.w), sum[2 * (j & 1) + 1]);
            } else {
              sum[2 * (j & 1)] = fma2(pack2(u[0], u[1]), scale2, sum[2 * (j & 1)]);
              sum[2 * (j & 1) + 1] = fma2(pack2(u[2], u[3]), scale2, sum[2 * (j & 1) + 1]);
            }
          }
        }
        const float2 s0 = unpack2(sum[0]), s1 = unpack2(sum[1]), s2 = unpack2(sum[2]), s3 = unpack2(sum[3]);
        const float total = ((s0.x + s0.y) + (s1.x + s1.y)) + ((s2.x + s2.y) + (s3.x + s3.y));
        const int nb = __shfl_sync(0xffffffffu, k.nb, i);
        if (row < nb)
          p.out[(int64_t)(k.t0 + i) * p.out_st + row] = page < 0 || page >= p.num_pages ? -INFINITY : total;
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty(buf));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The kernels' shared-memory limits, once per device.
dsa_status_t prepare(int device) {
  static std::mutex mu;
  static bool done[64];
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return DSA_OK;
  cudaError_t e = cudaSuccess;
  for (const void* f : {(const void*)scores_kernel<false, false>, (const void*)scores_kernel<true, false>,
                        (const void*)scores_kernel<false, true>, (const void*)scores_kernel<true, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return cuda_fail(e);
  done[device] = true;
  return DSA_OK;
}

}  // namespace scores
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_block_scores(const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t T, int H,
                                         const void* summary, int64_t num_pages, const int32_t* block_table,
                                         int64_t bt_stride, int page_size, int max_pages, int64_t num_requests,
                                         const int32_t* req_of_token, const int32_t* lengths, float sm_scale,
                                         const float* weights, float* scores_out, int64_t score_stride, int64_t width,
                                         int32_t* error_word, void* stream) {
  if (T < 0 || H < 1 || page_size < 1 || max_pages < 0 || bt_stride < max_pages || num_pages < 0 || width < 1 ||
      score_stride < width || !std::isfinite(sm_scale) || !(sm_scale > 0.0f))
    return DSA_ERR_INVALID_ARGUMENT;
  if (H > scores::kMaxHeads || T > (1 << 24) || width > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!q || !summary || !block_table || !lengths || !scores_out || num_requests < 1 || (!req_of_token && T > num_requests))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(q, 16) || q_stride_t < 0 || q_stride_h < 0 || q_stride_t % 8 || q_stride_h % 8 || !aligned(summary, 16))
    return DSA_ERR_INVALID_ARGUMENT;
  for (const void* x : {(const void*)block_table, (const void*)req_of_token, (const void*)lengths, (const void*)weights,
                        (const void*)scores_out, (const void*)error_word})
    if (!aligned(x, 4)) return DSA_ERR_INVALID_ARGUMENT;
  DeviceInfo dev;
  dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  scores::Params p{};
  p.q = static_cast<const uint16_t*>(q);
  p.q_st = q_stride_t;
  p.q_sh = q_stride_h;
  p.T = T;
  p.H = H;
  p.summary = static_cast<const uint16_t*>(summary);
  p.num_pages = num_pages;
  p.bt = block_table;
  p.bt_st = bt_stride;
  p.page = page_size;
  p.num_requests = num_requests;
  p.req = req_of_token;
  p.lengths = lengths;
  p.scale = sm_scale;
  p.w = weights;
  p.out = scores_out;
  p.out_st = score_stride;
  p.err = error_word;
  p.most = (int)(width < max_pages ? width : max_pages);
  const int64_t tiles = p.most > 0 ? (p.most + scores::kBM - 1) / scores::kBM : 1;
  const int sms = dev.sm_count;
  // As many tokens in a group as an MMA takes, while their tiles are three times the SMs: neighbours of one
  // request share its summaries (1024 tokens of 4 requests x 1024 blocks, 32 heads: 27 us with 8 in a group, 67
  // with 1), but a unit is as long as all its tokens' tiles (8 requests x 2048 blocks: 10.5 us with 1 and 14.4
  // with 4). Tokens that do not name their requests have one each. These rules, and those below, go by the table's width,
  // since the lengths are on the device: rows much shorter than it get fewer, longer units than they would bear (32
  // requests of up to 512 blocks: 5.8 us in a table of 513 columns, 10.0 in 8208; 64: 6.6 and 9.9; 256: 11.6 and 12.9).
  p.HP = (H + 15) / 16 * 16;
  p.G = req_of_token ? scores::kMaxN / p.HP : 1;
  while (p.G > 1 && (T + p.G - 1) / p.G * tiles < 3 * sms) p.G >>= 1;
  // Few tiles do not cover the time that the next group's queries take: two groups must fit then (1495 tokens x 128
  // heads x 19 blocks: 31 us for 37; 4096 x 64 x 256: 45 for 53; x 1024: 96 for 80. Their floors are 15 and 21 us: the
  // queries are waited for all the same).
  while (p.G > 1 && tiles <= 4 && p.G * p.HP > scores::kMaxN / 2) p.G >>= 1;
  const int64_t groups = (T + p.G - 1) / p.G;
  // As many parts of a group's tiles as end first, a unit's start (lengths, pages, queries) being worth a tile (256
  // requests of up to 512 blocks: 18.7 us in one part, 21.5 in two; 64 such requests: 12.3 in one, 10.2 in two).
  int64_t parts = 1;
  double best = 0.0;
  for (int64_t n = 1; n <= tiles && (n - 1) * groups <= 2 * sms; ++n) {
    const double cost = (double)((groups * n + sms - 1) / sms) * ((double)tiles / n + 1.0);
    if (n > 1 && cost >= best) continue;
    best = cost;
    parts = n;
  }
  p.parts = (int)parts;
  p.units = (int)(groups * p.parts);
  p.slots = (int)(scores::kQueryBytes / ((uint32_t)(p.G * p.HP) * scores::kD * 2));
  if (p.slots > scores::kMaxSlots) p.slots = scores::kMaxSlots;
  if ((st = scores::prepare(dev.device)) != DSA_OK) return st;
  const unsigned grid = (unsigned)(p.units < sms ? p.units : sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool whole = H % scores::N == 0;
  auto kernel = weights ? (whole ? scores::scores_kernel<true, true> : scores::scores_kernel<true, false>)
                        : (whole ? scores::scores_kernel<false, true> : scores::scores_kernel<false, false>);
  kernel<<<grid, scores::kThreads, scores::kSmemBytes, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
