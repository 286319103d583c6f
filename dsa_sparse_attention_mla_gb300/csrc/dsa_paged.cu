// dsa_paged.cu - dense attention over the paged latent cache, one new token per request, and the
// attention weight each cached position receives (dsa_paged_attn, dsa_paged_attn_mass).
//
// For token t of request r, head h and position j of the token's range [a, b):
//   u_hj = sm_scale q_h . k_j, capped by cap * tanh(u / cap), minus slope_h |qpos - kpos_j|
//   out_h = sum_j softmax_j(u_h) k_j,  lse_h = log sum_j exp(u_hj)
//   mass_out[r, j] = mass[r, j] + sum_h exp(u_hj - lse_h)
// The latent row k_j is key and value of every head: a position costs 264 (FP8) or 512 (bf16) bytes
// and 4 * 256 operations per head, so with 64 heads a bf16 cache is bound by HBM and an FP8 one
// about equally by HBM and the tensor core.
//
// Shape of the computation
//  * Transposed products: S^T[key, head] = K Q^T with M = 128 keys, N = 64 heads, then
//    O^T[column, head] += V^T P^T in two M = 128 halves of the 256 columns, V^T read MN-major from
//    the same K tile (tcgen05 kind::f16, bf16 operands, fp32 accumulators in tensor memory). A
//    token has at most 64 heads per pass: heads as M would leave half of the tensor core idle.
//  * FP8 rows: the e4m3 codes are widened to bf16 exactly on their way into shared memory. The two
//    tile scales of a row never touch them: S keeps one accumulator per scale tile and they are
//    multiplied there in fp32, and the value product takes one weight matrix per scale tile,
//    p * scale, so the keys are the exact products code * scale.
//  * Softmax with one thread per key and 16 heads (four warps per lane quarter). The running maximum
//    of a head is raised, and O and the sums rescaled, only when some score exceeds it by 2^20: p
//    and its sums are floating point, so a stale maximum costs no precision, and the exact path runs
//    for a segment's first tile and almost never again.
//  * Persistent CTAs, one per SM. Each computes the same split from the lengths (they live on the
//    device): rows (token, group of 64 heads) cost their 128-position tiles plus a constant, and
//    CTA c takes the c-th of G equal parts of the total. A row cut by a border leaves unnormalised
//    parts in the workspace, which a second, dependent launch joins in the order of the parts.
//  * Warp roles: 0-15 softmax, 16 scheduler (walks the CTA's rows), 17 score products, 18 value
//    products, 19 query loads, 20-27 row loads. Every wait is bounded.
//  * The mass kernel is the same without the value product: with the lse given, each key's thread
//    adds the weights of all 64 heads; four warp groups take tiles in turn, with an accumulator
//    buffer each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>

#include "dsa_host.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace paged {

constexpr int kD = 256;
constexpr int kMaxHeads = 128;
constexpr int kHG = 64;    // heads per row (MMA N)
constexpr int kBN = 128;   // positions per tile (MMA M)
constexpr int kSoftmaxWarps = 16;
constexpr int kWarpSched = 16, kWarpScore = 17, kWarpValue = 18, kWarpQuery = 19, kWarpLoad0 = 20;
constexpr int kLoadWarps = 8;
constexpr int kWarps = kWarpLoad0 + kLoadWarps;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 192;      // the join's lists
constexpr int kSegs = 8;           // segment ring depth
constexpr int kRowOverhead = 1;    // a row's start and end, in tiles
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -1e30f;   // running maximum before the first valid score
constexpr float kStale = 20.0f;    // a score may exceed the running maximum by 2^20

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
  int64_t* ws_tail; // [G] the row CTA c starts and does not finish, or -1
  int* ws_head;     // [G] 0: continues no row, 1: continues one to its border, 2: finishes one
  int* ws_first;    // [T * HG], when that is at most G: the CTA that starts a split row, or -1
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
  static constexpr int NSB = MASS ? 4 : 2;            // score buffers
  static constexpr int S_COLS = F8 ? 128 : 64;        // columns of one (FP8: one 64 per scale tile)
  static constexpr int O_COL = NSB * S_COLS;          // O^T halves at O_COL and O_COL + 64
  static constexpr int TMEM_USED = O_COL + (MASS ? 0 : 128);
  static constexpr int TMEM_COLS = TMEM_USED <= 256 ? 256 : 512;
  // rings of a tile's valid mask and scales: a load warp may run this far ahead of the tile's reader
  static constexpr int NV = MASS ? 8 : 4;
  static constexpr int NST = 4;                       // K ring: halves of a tile (128 keys x 128 columns)
  static constexpr int HALF_BYTES = kBN * 256;
  static constexpr int PBUF = F8 ? 1 : 2;
  static constexpr int PN = F8 ? 2 : 1;               // weight matrices per tile
  static constexpr int P_BYTES = MASS ? 0 : PN * kBN * 128;
  static constexpr int Q_OFF = 0, Q_BYTES = kHG * kD * 2;
  static constexpr int K_OFF = Q_OFF + Q_BYTES;
  static constexpr int P_OFF = K_OFF + NST * HALF_BYTES;
  static constexpr int SEG_OFF = P_OFF + PBUF * P_BYTES;
  static constexpr int VM_OFF = SEG_OFF + kSegs * 64;         // [NV] valid masks of a tile, 128 bits
  static constexpr int SC_OFF = VM_OFF + 16 * NV;             // FP8: [NV][128][2] tile scales
  static constexpr int NL_OFF = SC_OFF + (F8 ? NV * 1024 : 0); // mass: [kSegs][64] -lse, exp2 domain
  static constexpr int SL_OFF = NL_OFF + (MASS ? kSegs * 256 : 0);  // slopes [128]
  static constexpr int RED_OFF = SL_OFF + 512;  // m [2][64], alpha [64], part [4][64], inverse sums [64]
  static constexpr int VOTE_OFF = RED_OFF + 8 * 256;
  static constexpr int PLAN_OFF = VOTE_OFF + 128;  // block scans: 2 x kWarps int64; start row, its cost
  static constexpr int BAR_OFF = PLAN_OFF + 2 * 8 * kWarps + 64;
  static constexpr int NBARS = 2 + 2 * NST + 3 * kSegs + NV + 2 * NSB + 2 * 2 + 1 + 2;
  static constexpr int MISC_OFF = BAR_OFF + 8 * NBARS;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(TMEM_USED <= 512, "TMEM budget");
};

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
__device__ __forceinline__ Row row_of(const Params& p, int64_t row) {
  const int64_t t = p.HG == 1 ? row : row >> 1;
  const int req = p.req ? p.req[t] : (int)t;
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

// One score in natural units -> exp2 domain, with cap and distance bias.
__device__ __forceinline__ float modify(float u, float cap, float inv_cap2, float bias) {
  if (cap > 0.0f) {
    // cap * tanh(u / cap) = cap * (1 - e) / (1 + e), e = exp(-2 |u| / cap), with u's sign
    const float e = ex2_approx(-fabsf(u) * inv_cap2);
    u = copysignf(__fdividef(cap * (1.0f - e), 1.0f + e), u);
  }
  return (u - bias) * kLog2e;
}

// Sums over the block, exclusive per thread (v), and in total; `buf` holds kWarps values.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* buf, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int64_t base = 0, sum = 0;
  for (int w = 0; w < kWarps; ++w) {
    const int64_t s = buf[w];
    if (w < warp) base += s;
    sum += s;
  }
  *total = sum;
  return base + x - v;
}
// Exclusive running maximum over the block.
__device__ __forceinline__ int block_max(int v, int64_t* buf) {
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
  for (int w = 0; w < warp; ++w) ex = max(ex, (int)buf[w]);
  return ex;
}

// Exchange among the softmax warps (one arrival each on `xbar`, phase `n` of it): returns the OR
// of `v` over the warps, with every warp's earlier shared-memory writes visible, or -1 when a warp
// did not arrive within the time limit.
static __device__ __forceinline__ int exchange(uint32_t xbar, int* votes, uint32_t n, bool v) {
  const int lane = threadIdx.x & 31;
  const int slot = n & 1;
  const bool any = __any_sync(0xffffffffu, v);
  __syncwarp();
  if (lane == 0) {
    votes[slot * kSoftmaxWarps + (threadIdx.x >> 5)] = any ? 1 : 0;
    mbar_arrive(xbar);
  }
  const bool ok = mbar_wait(xbar, n & 1, kWaitNs);
  if (!__all_sync(0xffffffffu, ok)) return -1;
  const int mine = votes[slot * kSoftmaxWarps + (lane & (kSoftmaxWarps - 1))];
  return __any_sync(0xffffffffu, mine != 0) ? 1 : 0;
}

template <int KIND, bool MASS, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(const __grid_constant__ Params p) {
  using C = Cfg<KIND, MASS>;
  constexpr bool F8 = C::F8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
  auto nl_full = [&](uint32_t s) { return b1 + 8 * (2 * kSegs + s); };  // mass: the segment's -lse
  const uint32_t b2 = b1 + 24 * kSegs;
  auto v_full = [&](uint32_t s) { return b2 + 8 * s; };                 // valid mask and scales of a tile
  auto s_full = [&](uint32_t s) { return b2 + 8 * (C::NV + s); };
  auto s_empty = [&](uint32_t s) { return b2 + 8 * (C::NV + C::NSB + s); };
  const uint32_t b3 = b2 + 8 * C::NV + 16 * C::NSB;
  auto p_full = [&](uint32_t s) { return b3 + 8 * s; };
  auto pv_done = [&](uint32_t s) { return b3 + 16 + 8 * s; };
  const uint32_t xbar = b3 + 32;
  auto drain = [&](uint32_t s) { return b3 + 40 + 8 * s; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  Seg* segs = reinterpret_cast<Seg*>(smem + C::SEG_OFF);
  float* s_slopes = reinterpret_cast<float*>(smem + C::SL_OFF);

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    mbar_init(q_full, 32);
    mbar_init(q_empty, 1);
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(k_full(s), F8 ? kLoadWarps : 32 * kLoadWarps);  // bf16: one asynchronous arrival per thread
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(g_full(s), 1);
      // softmax warps, load warps, query warp, score issuer, value issuer
      mbar_init(g_empty(s), kSoftmaxWarps + kLoadWarps + 2 + (MASS ? 0 : 1));
      mbar_init(nl_full(s), 1);
    }
    for (int s = 0; s < C::NV; ++s) mbar_init(v_full(s), kLoadWarps);
    for (int s = 0; s < C::NSB; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_empty(s), MASS ? 4 : kSoftmaxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(p_full(s), kSoftmaxWarps);
      mbar_init(pv_done(s), 1);
      mbar_init(drain(s), 1);
    }
    mbar_init(xbar, kSoftmaxWarps);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (MODS && threadIdx.x < kMaxHeads)
    s_slopes[threadIdx.x] = p.slopes && threadIdx.x < p.H ? p.slopes[threadIdx.x] : 0.0f;
  if (warp == kWarpScore) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }

  // ---- the split: total cost of the rows, and the row in which this CTA's share begins
  int64_t* plan = reinterpret_cast<int64_t*>(smem + C::PLAN_OFF);
  int64_t* plan_start = plan + 2 * kWarps;  // row, its cost offset, running maximum of the requests
  const int64_t nrows = p.T * p.HG;
  int64_t c0, c1;
  {
    const int64_t per = (nrows + kThreads - 1) / kThreads;
    const int64_t i0 = threadIdx.x * per, i1 = i0 + per < nrows ? i0 + per : nrows;
    int mx = INT32_MIN;
    if (MASS && p.req) {
      int m = INT32_MIN;
      for (int64_t i = i0; i < i1; ++i) m = max(m, p.req[i]);
      mx = block_max(m, plan);
    }
    auto cost_of = [&](int64_t i, int& run) -> int64_t {
      const Row r = row_of(p, i);
      bool ok = true;
      if (MASS && p.req) {
        ok = r.req > run;
        run = max(run, r.req);
      }
      return (ok ? r.n : 0) + kRowOverhead;
    };
    int64_t sum = 0;
    int run = mx;
    for (int64_t i = i0; i < i1; ++i) sum += cost_of(i, run);
    int64_t total;
    const int64_t pre = block_sum(sum, plan + kWarps, &total);
    c0 = cta * total / p.G;
    c1 = (cta + 1) * total / p.G;
    if (c0 < c1 && pre <= c0 && c0 < pre + sum) {
      int64_t at = pre, i = i0;
      run = mx;
      for (;; ++i) {
        int next = run;
        const int64_t c = cost_of(i, next);
        if (c0 < at + c) break;
        at += c;
        run = next;
      }
      plan_start[0] = i;
      plan_start[1] = at;
      plan_start[2] = run;
    }
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
    if (mbar_wait(bar, par, kWaitNs)) return true;
    fail();
    return false;
  };
  // the whole warp waits, and agrees on the outcome
  auto wait_warp = [&](uint32_t bar, uint32_t par) -> bool {
    if (__all_sync(0xffffffffu, mbar_wait(bar, par, kWaitNs))) return true;
    fail();
    return false;
  };

  if (warp == kWarpSched) {
    // ================================================================== scheduler ====
    uint32_t sc = 0;
    int64_t tail = -1;
    int head = 0;
    bool ok = true;
    if (c0 < c1) {
      int64_t row = plan_start[0], cost = plan_start[1];
      int run = (int)plan_start[2];
      while (ok && cost < c1 && row < nrows) {
        const int64_t i = row + lane;
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
        int64_t cum = c ? (int64_t)n + kRowOverhead : 0;
        const int64_t mine = cum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, cum, o);
          if (lane >= o) cum += y;
        }
        const int64_t at = cost + cum - mine;  // this row's cost offset
        int64_t lo = c0 - at - kRowOverhead, hi = c1 - at - kRowOverhead;
        lo = lo < 0 ? 0 : lo;
        hi = hi > n ? n : hi;
        const bool owner = c && at >= c0 && at < c1;
        if (owner && r.bad && order) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        if (owner && !order && r.a < r.b) set_err(p.err, DSA_DEVERR_REQUEST_ORDER);
        const bool has = c && (n > 0 ? lo < hi : owner && !MASS);
        const int kind = lo > 0 ? 2 : (hi < n ? 1 : 0);
        if (!MASS && nrows <= p.G && has && kind != 2) p.ws_first[i] = kind == 1 ? cta : -1;
        uint32_t todo = __ballot_sync(0xffffffffu, has);
        if (!MASS) {
          const uint32_t st = __ballot_sync(0xffffffffu, has && kind == 1);
          if (st) tail = row + (31 - __clz(st));
          const uint32_t co = __ballot_sync(0xffffffffu, has && kind == 2 && n > 0);
          if (co) head = __shfl_sync(0xffffffffu, hi < n ? 1 : 2, 31 - __clz(co));
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
            s->t = (int)(p.HG == 1 ? i : i >> 1);
            s->hg = p.HG == 1 ? 0 : (int)(i & 1);
            s->req = r.req;
            s->a = r.a;
            s->b = r.b;
            s->tile0 = (int)lo;
            s->ntiles = n > 0 ? (int)(hi - lo) : 0;
            s->kind = kind;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(g_full(slot));
          ++sc;
        }
        row += 32;
        cost += __shfl_sync(0xffffffffu, cum, 31);
      }
    }
    if (!MASS && lane == 0) {
      p.ws_tail[cta] = tail;
      p.ws_head[cta] = head;
    }
    if (ok) {
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
      constexpr uint32_t idS = idesc_bf16(kBN, kHG, 0, 0);
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
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t ka = (uint32_t)((kk >> 2) * ((kBN * 128) >> 4) + (kk & 3) * 2);
              const uint32_t qa = (uint32_t)((2 * h + (kk >> 2)) * ((kHG * 128) >> 4) + (kk & 3) * 2);
              if (kk == 0 && (F8 || h == 0)) mma_bf16_lohi<0>(d, k_lo + ka, k_hi, q_lo + qa, q_hi, idS);
              else mma_bf16_lohi<1>(d, k_lo + ka, k_hi, q_lo + qa, q_hi, idS);
            }
            if (MASS) mma_commit(k_empty(st));
          }
          if (ok) mma_commit(s_full(sb));
        }
        if (ok) mma_commit(q_empty);
      }
      mma_commit(drain(0));
      mbar_wait(drain(0), 0, kWaitNs);
    }
    __syncwarp();
  } else if (warp == kWarpValue) {
    // ============================================================= value products ====
    if (!MASS && lane == 0) {
      constexpr uint32_t idPV = idesc_bf16(kBN, kHG, 1, 1);
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
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t st = (2 * g + h) % C::NST;
            const uint32_t v_lo = (uint32_t)sw128_desc(sbase + C::K_OFF + st * C::HALF_BYTES, kBN * 128, 1024);
            const uint32_t p_lo = (uint32_t)sw128_desc(
                sbase + C::P_OFF + pb * C::P_BYTES + (F8 ? h * kBN * 128 : 0), kBN * 128, 1024);
            const uint32_t d = tmem + C::O_COL + 64 * h;
            // the first step of a segment overwrites the accumulator
            mma_bf16(d, ((uint64_t)mn_hi << 32) | v_lo, ((uint64_t)mn_hi << 32) | p_lo, idPV, k == 0 ? 0u : 1u);
#pragma unroll
            for (int j = 1; j < kBN / 16; ++j)
              mma_bf16_lohi<1>(d, v_lo + 128 * j, mn_hi, p_lo + 128 * j, mn_hi, idPV);
            mma_commit(k_empty(st));
          }
          mma_commit(pv_done(g & 1));
        }
      }
      mma_commit(drain(1));
      mbar_wait(drain(1), 0, kWaitNs);
    }
    __syncwarp();
  } else if (warp == kWarpQuery) {
    // ================================================================ query loads ====
    // 64 heads x 256 columns in four 128-byte-swizzled chunks; heads past the row's are zero.
    uint32_t qc = 0;
    for (uint32_t sc = 0;; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!wait_warp(g_full(slot), (sc / kSegs) & 1)) break;
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
          if (lane == 0) mbar_arrive(nl_full(slot));
        }
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
  } else if (warp >= kWarpLoad0) {
    // ================================================================== row loads ====
    // Warp w takes rows 16 w .. 16 w + 15 of every tile, in two column halves. Lane l < 16 finds
    // row l's slot, one tile ahead of the copies.
    const int lw = warp - kWarpLoad0;
    uint32_t g = 0;  // tiles so far, and the segment being read
    uint32_t sc = 0;
    int k = 0;
    Seg s{};
    s.ntiles = 0;
    bool ok = true, more = true;
    int64_t slot_n = -1;      // slot of this lane's row in the next tile
    float2 scale_n = make_float2(0.0f, 0.0f);
    // finds the next tile's slots; false when there is none
    auto advance = [&]() -> bool {
      while (k >= s.ntiles) {
        const uint32_t ring = sc % kSegs;
        if (!wait_warp(g_full(ring), (sc / kSegs) & 1)) {
          ok = false;
          return false;
        }
        s = segs[ring];
        __syncwarp();
        if (lane == 0) mbar_arrive(g_empty(ring));
        ++sc;
        k = 0;
        if (s.type == 0) return false;
      }
      const uint32_t pos = (uint32_t)(s.a & ~127) + 128u * (uint32_t)(s.tile0 + k) + 16 * lw + (lane & 15);
      int64_t slot = -1;
      if (pos >= (uint32_t)s.a && pos < (uint32_t)s.b) {
        if (p.bt) {
          const uint32_t pg = (uint32_t)(((uint64_t)pos * p.pg_mul) >> p.pg_shift);
          const int64_t page = p.bt[s.req * p.bt_stride + pg];
          slot = page * p.page_size + (pos - pg * (uint32_t)p.page_size);
          if (page < 0 || slot >= p.num_slots) slot = -2;
        } else {
          slot = pos;
        }
      }
      if (slot == -2) {
        if (lane < 16) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        slot = -1;
      }
      slot_n = slot;
      if (F8) {
        scale_n = make_float2(0.0f, 0.0f);
        if (slot >= 0 && lane < 16) scale_n = *reinterpret_cast<const float2*>(p.cache + slot * C::RB + 256);
      }
      ++k;
      return true;
    };
    const int gl = lane & 15, hi16 = lane >> 4;
    // FP8: the 16 lanes of a half warp read one row's 128 codes of a half
    auto load_half = [&](uint2 (&v)[8], int64_t slot, int h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t sl = __shfl_sync(0xffffffffu, slot, 2 * i + hi16);
        v[i] = make_uint2(0u, 0u);
        if (sl >= 0) v[i] = __ldcs(reinterpret_cast<const uint2*>(p.cache + sl * C::RB + 128 * h + 8 * gl));
      }
    };
    auto store_half = [&](const uint2 (&v)[8], uint32_t st) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 16 * lw + 2 * i + hi16;
        const uint32_t c[2] = {v[i].x, v[i].y};
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(c[j] & 0xFFFFu)));
          const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(c[j] >> 16)));
          w[2 * j] = f32x2_to_bf16x2(a.x, a.y);
          w[2 * j + 1] = f32x2_to_bf16x2(b.x, b.y);
        }
        uint8_t* d = smem + C::K_OFF + st * C::HALF_BYTES + (gl >> 3) * (kBN * 128) + r * 128 + (((gl & 7) ^ (r & 7)) << 4);
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    // the tile's valid rows and scales, for the softmax warps
    auto publish = [&](int64_t slot, float2 scale) {
      const uint32_t m = __ballot_sync(0xffffffffu, slot >= 0) & 0xFFFFu;
      if (lane == 0) reinterpret_cast<uint16_t*>(smem + C::VM_OFF + 16 * (g % C::NV))[lw] = (uint16_t)m;
      if (F8 && lane < 16)
        reinterpret_cast<float2*>(smem + C::SC_OFF + 1024 * (g % C::NV))[16 * lw + lane] = scale;
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(g % C::NV));
    };
    more = advance();
    if constexpr (F8) {
      uint2 va[8], vb[8];
      int64_t slot = slot_n;
      float2 scale = scale_n;
      if (more) load_half(va, slot, 0);
      while (more) {
        load_half(vb, slot, 1);
        const int64_t cur = slot;
        const float2 cur_scale = scale;
        more = advance();
        slot = slot_n;
        scale = scale_n;
        {
          const uint32_t hs = 2 * g, st = hs % C::NST;
          if (hs >= C::NST && !wait_warp(k_empty(st), ((hs / C::NST) & 1) ^ 1)) break;
          publish(cur, cur_scale);
          store_half(va, st);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full(st));
        }
        if (more) load_half(va, slot, 0);
        {
          const uint32_t hs = 2 * g + 1, st = hs % C::NST;
          if (hs >= C::NST && !wait_warp(k_empty(st), ((hs / C::NST) & 1) ^ 1)) break;
          store_half(vb, st);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(k_full(st));
        }
        ++g;
      }
    } else {
      while (more) {
        const int64_t slot = slot_n;
        bool stop = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hs = 2 * g + h, st = hs % C::NST;
          if (hs >= C::NST && !wait_warp(k_empty(st), ((hs / C::NST) & 1) ^ 1)) {
            stop = true;
            break;
          }
          if (h == 0) publish(slot, scale_n);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int64_t sl = __shfl_sync(0xffffffffu, slot, 2 * i + hi16);
            const int r = 16 * lw + 2 * i + hi16;
            const uint32_t dst = sbase + C::K_OFF + st * C::HALF_BYTES + (gl >> 3) * (kBN * 128) + r * 128 +
                                 (((gl & 7) ^ (r & 7)) << 4);
            const uint8_t* src = p.cache + (sl >= 0 ? sl * C::RB + 256 * h + 16 * gl : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(sl >= 0 ? 16 : 0)
                         : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(k_full(st)) : "memory");
          if (h == 0) more = advance();
        }
        if (stop) break;
        ++g;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
    (void)ok;
  } else if constexpr (MASS) {
    // ================================================= weights of a key, 16 warps ====
    const int qd = warp & 3, gi = warp >> 2;
    const int tr = 32 * qd + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16) + gi * C::S_COLS;
    const float inv_cap2 = MODS && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
    const float c_log2 = p.sm_scale * kLog2e;
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t sc = 0; ok; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!wait_warp(g_full(slot), (sc / kSegs) & 1)) break;
      const Seg s = segs[slot];
      if (s.type == 0) break;
      if (s.ntiles > 0 && !wait_warp(nl_full(slot), (sc / kSegs) & 1)) break;
      const float* nl = reinterpret_cast<const float*>(smem + C::NL_OFF) + slot * kHG;
      const float* slopes = s_slopes + s.hg * kHG;
      const int64_t qp = MODS && p.qpos ? p.qpos[s.t] : (int64_t)p.lengths[s.t] - 1;
      for (int k = 0; k < s.ntiles; ++k, ++g) {
        if ((g & 3) != (uint32_t)gi) continue;
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
        if (!wait_warp(v_full(g % C::NV), (g / C::NV) & 1) || !wait_warp(s_full(gi), (g >> 2) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool valid = (reinterpret_cast<const uint32_t*>(smem + C::VM_OFF + 16 * (g % C::NV))[qd] >> lane) & 1;
        float2 scl = make_float2(1.0f, 1.0f);
        if (F8) scl = reinterpret_cast<const float2*>(smem + C::SC_OFF + 1024 * (g % C::NV))[tr];
        const float f = MODS ? p.sm_scale : c_log2;
        const float f0 = F8 ? scl.x * f : f, f1 = scl.y * f;
        float w = 0.0f;
#pragma unroll
        for (int ch = 0; ch < kHG / 16; ++ch) {
          uint32_t x0[16], x1[16];
          tmem_ld32_x16(tl + 16 * ch, x0);
          if (F8) tmem_ld32_x16(tl + 64 + 16 * ch, x1);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x = u2f(x0[i]) * f0;
            if (F8) x = fmaf(u2f(x1[i]), f1, x);
            if (MODS) x = modify(x, p.cap, inv_cap2, slopes[16 * ch + i] * dist);
            w += ex2_approx(x + nl[16 * ch + i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty(gi));
        if (in) p.mass_out[s.req * p.mass_out_st + pos] = valid ? old + w : old;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(g_empty(slot));
    }
  } else {
    // ==================================================== softmax and outputs, 16 warps ====
    // Warp = lane quarter qd (keys 32 qd ..; output columns 32 qd .. of both halves), heads 16 hq ..
    const int qd = warp & 3, hq = warp >> 2;
    const int tr = 32 * qd + lane;
    const int sid = threadIdx.x;  // 0 .. 511
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    float* red = reinterpret_cast<float*>(smem + C::RED_OFF);
    float* red_alpha = red + 128;
    float* red_part = red + 192;  // [4 quarters][64 heads]
    float* red_inv = red + 448;
    int* votes = reinterpret_cast<int*>(smem + C::VOTE_OFF);
    const float inv_cap2 = MODS && p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
    const float c_log2 = p.sm_scale * kLog2e;
    uint32_t g = 0, xc = 0, mb = 0;
    auto xsync = [&](bool v) -> int {
      const int r = exchange(xbar, votes, xc++, v);
      if (r < 0) fail();
      return r;
    };
    auto pv_wait = [&](uint32_t last) -> bool { return wait_warp(pv_done(last & 1), (last >> 1) & 1); };
    // O^T columns this warp handles: half oh, heads 32 * (hq & 1) ..
    const int oh = hq >> 1, ob = 32 * (hq & 1);
    const uint32_t o_addr = tl + C::O_COL + 64 * oh + ob;
    bool ok = true;
    for (uint32_t sc = 0; ok; ++sc) {
      const uint32_t slot = sc % kSegs;
      if (!wait_warp(g_full(slot), (sc / kSegs) & 1)) break;
      const Seg s = segs[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(g_empty(slot));
      if (s.type == 0) break;
      const int heads = min(kHG, p.H - s.hg * kHG);
      const float* slopes = s_slopes + s.hg * kHG + 16 * hq;
      int64_t qp = 0;
      if (MODS) qp = p.qpos ? p.qpos[s.t] : (int64_t)p.lengths[s.t] - 1;
      float lsum[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) lsum[i] = 0.0f;
      for (int k = 0; k < s.ntiles; ++k, ++g) {
        const uint32_t sb = g % C::NSB;
        float dist = 0.0f;
        if (MODS && p.slopes) {
          const uint32_t pos = (uint32_t)(s.a & ~127) + 128u * (uint32_t)(s.tile0 + k) + tr;
          int64_t kp = pos;
          if (p.kpos && pos >= (uint32_t)s.a && pos < (uint32_t)s.b) kp = p.kpos[s.req * p.kp_stride + pos];
          dist = fabsf((float)(qp - kp));
        }
        if (!wait_warp(v_full(g % C::NV), (g / C::NV) & 1) || !wait_warp(s_full(sb), (g / C::NSB) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool valid = (reinterpret_cast<const uint32_t*>(smem + C::VM_OFF + 16 * (g % C::NV))[qd] >> lane) & 1;
        float2 scl = make_float2(1.0f, 1.0f);
        if (F8) scl = reinterpret_cast<const float2*>(smem + C::SC_OFF + 1024 * (g % C::NV))[tr];
        float x[16];
        {
          uint32_t x0[16], x1[16];
          tmem_ld32_x16(tl + sb * C::S_COLS + 16 * hq, x0);
          if (F8) tmem_ld32_x16(tl + sb * C::S_COLS + 64 + 16 * hq, x1);
          tc_wait_ld();
          const float f = MODS ? p.sm_scale : c_log2;
          const float f0 = F8 ? scl.x * f : f, f1 = scl.y * f;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = u2f(x0[i]) * f0;
            if (F8) x[i] = fmaf(u2f(x1[i]), f1, x[i]);
            if (MODS) x[i] = modify(x[i], p.cap, inv_cap2, slopes[i] * dist);
            if (!valid) x[i] = -INFINITY;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty(sb));
        bool exact = k == 0;
        if (!exact) {
          float top = -INFINITY;
          const float* m = red + 64 * mb + 16 * hq;
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, x[i] - m[i]);
          const int r = xsync(top > kStale);
          if (r < 0) {
            ok = false;
            break;
          }
          exact = r != 0;
        }
        if (exact) {
          // exact maximum of the tile per head; the running maxima are raised to it
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int mx = redux_max_s32(f2ord(x[i]));
            if (lane == i) red_part[64 * qd + 16 * hq + i] = ord2f(mx);
          }
          if (xsync(false) < 0) {
            ok = false;
            break;
          }
          if (sid < kHG) {
            const float mo = k == 0 ? kNoMax : red[64 * mb + sid];
            const float mt = fmaxf(fmaxf(red_part[sid], red_part[64 + sid]), fmaxf(red_part[128 + sid], red_part[192 + sid]));
            const float mn = fmaxf(mo, mt);
            red[64 * (mb ^ 1) + sid] = mn;
            red_alpha[sid] = ex2_approx(mo - mn);
          }
          if (xsync(false) < 0) {
            ok = false;
            break;
          }
          mb ^= 1;
          if (k > 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) lsum[i] *= red_alpha[16 * hq + i];
            if (!pv_wait(g - 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int ch = 0; ch < 2; ++ch) {
              uint32_t o[16];
              tmem_ld32_x16(o_addr + 16 * ch, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = f2u(u2f(o[i]) * red_alpha[ob + 16 * ch + i]);
              tmem_st32_x16(o_addr + 16 * ch, o);
            }
            tc_wait_st();
          }
        }
        {
          const float* m = red + 64 * mb + 16 * hq;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = ex2_approx(x[i] - m[i]);
            lsum[i] += x[i];
          }
        }
        // the weights' buffer is free once the value product that read it is complete
        if (g >= C::PBUF && !pv_wait(g - C::PBUF)) {
          ok = false;
          break;
        }
        uint8_t* prow = smem + C::P_OFF + (g % C::PBUF) * C::P_BYTES + tr * 128;
        const int sw = tr & 7;
#pragma unroll
        for (int h = 0; h < C::PN; ++h) {
          const float f = F8 ? (h == 0 ? scl.x : scl.y) : 1.0f;
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = F8 ? f32x2_to_bf16x2(x[2 * i] * f, x[2 * i + 1] * f) : f32x2_to_bf16x2(x[2 * i], x[2 * i + 1]);
          *reinterpret_cast<uint4*>(prow + h * (kBN * 128) + (((2 * hq) ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(prow + h * (kBN * 128) + (((2 * hq + 1) ^ sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(g % C::PBUF));
      }
      if (!ok) break;
      // ---- the segment's end: sums over the keys, then this warp's columns of O^T
      {
        // reduce-scatter over the lanes: lanes 2i and 2i + 1 end with the warp's sum of head i
        float v8[8], v4[4], v2[2];
        const bool b4 = lane & 16, b3_ = lane & 8, b2_ = lane & 4, b1_ = lane & 2;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v8[i] = (b4 ? lsum[i + 8] : lsum[i]) + __shfl_xor_sync(0xffffffffu, b4 ? lsum[i] : lsum[i + 8], 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) v4[i] = (b3_ ? v8[i + 4] : v8[i]) + __shfl_xor_sync(0xffffffffu, b3_ ? v8[i] : v8[i + 4], 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) v2[i] = (b2_ ? v4[i + 2] : v4[i]) + __shfl_xor_sync(0xffffffffu, b2_ ? v4[i] : v4[i + 2], 4);
        float v1 = (b1_ ? v2[1] : v2[0]) + __shfl_xor_sync(0xffffffffu, b1_ ? v2[0] : v2[1], 2);
        v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
        if ((lane & 1) == 0) red_part[64 * qd + 16 * hq + (lane >> 1)] = v1;
      }
      if (xsync(false) < 0) break;
      const int part = 2 * cta + (s.kind == 1 ? 1 : 0);
      if (sid < kHG) {
        const float L = (red_part[sid] + red_part[64 + sid]) + (red_part[128 + sid] + red_part[192 + sid]);
        const float m = red[64 * mb + sid];
        red_inv[sid] = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
        if (s.kind != 0) {
          p.ws_ml[(int64_t)part * 2 * kHG + sid] = s.ntiles > 0 ? m : kNoMax;
          p.ws_ml[(int64_t)part * 2 * kHG + kHG + sid] = L;
        } else if (p.lse && sid < heads) {
          p.lse[s.t * p.lse_st + s.hg * kHG + sid] = L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
        }
      }
      if (xsync(false) < 0) break;
      if (s.ntiles > 0 && !pv_wait(g - 1)) break;
      tc_fence_after();
      const int dv = 128 * oh + tr;
      uint16_t* orow = p.out + (int64_t)s.t * p.out_st + (int64_t)s.hg * kHG * p.out_sh;
      float* prt = p.ws_o + (int64_t)part * kHG * kD + dv;
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        const int h0 = ob + 16 * ch;
        if (h0 >= heads) break;
        uint32_t o[16];
        if (s.ntiles > 0) {
          tmem_ld32_x16(o_addr + 16 * ch, o);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0u;
        }
        if (s.kind != 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (h0 + i < heads) prt[(h0 + i) * kD] = u2f(o[i]);
        } else {
          // lanes 2i and 2i + 1 hold neighbouring columns: they swap heads, so that each writes
          // two columns of one head
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float e = u2f(o[2 * i]) * red_inv[h0 + 2 * i], f = u2f(o[2 * i + 1]) * red_inv[h0 + 2 * i + 1];
            const bool odd = lane & 1;
            const float other = __shfl_xor_sync(0xffffffffu, odd ? e : f, 1);
            const uint32_t w = odd ? f32x2_to_bf16x2(other, f) : f32x2_to_bf16x2(e, other);
            const int h = h0 + 2 * i + (odd ? 1 : 0);
            if (h < heads) *reinterpret_cast<uint32_t*>(orow + h * p.out_sh + (dv & ~1)) = w;
          }
        }
      }
      tc_fence_before();
      // the sums and weights of this segment are read before the next one rewrites them
      if (xsync(false) < 0) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpScore) tmem_dealloc(tmem, C::TMEM_COLS);
}

// Joins the parts of each split row in the order of the parts. Block (x, y) takes row x (when there
// are at most G rows; else the row that CTA x starts) and heads y * 64 / gridDim.y ..
// 256 threads: 64 columns of four times 4 parts at a time, heads one after the other.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params p) {
  __shared__ int s_part[kMaxCtas + 1];
  __shared__ float s_w[kMaxCtas + 1];
  __shared__ int s_fin[8], s_cnt[8], s_n;
  __shared__ float4 s_acc[4][64];
  __shared__ float s_L;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int64_t nrows = p.T * p.HG;
  int64_t row;
  int c;
  if (nrows <= p.G) {
    row = blockIdx.x;
    c = p.ws_first[row];
    if (c < 0) return;
  } else {
    c = blockIdx.x;
    row = p.ws_tail[c];
    if (row < 0) return;
  }
  // parts in order: the start, then every CTA that continues the row, to the one that finishes it
  {
    const int lane = tid & 31, warp = tid >> 5;
    const int k = c + 1 + tid;
    const int h = k < p.G ? p.ws_head[k] : 0;
    const uint32_t fin = __ballot_sync(0xffffffffu, h == 2);
    if (lane == 0) s_fin[warp] = fin ? 32 * warp + __ffs(fin) - 1 : 1 << 20;
    __syncthreads();
    int last = s_fin[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) last = min(last, s_fin[w]);
    const uint32_t mem = __ballot_sync(0xffffffffu, h != 0 && tid <= last);
    if (lane == 0) s_cnt[warp] = __popc(mem);
    __syncthreads();
    int at = 1, total = 1;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += s_cnt[w];
      total += s_cnt[w];
    }
    if ((mem >> lane) & 1) s_part[at + __popc(mem & ((1u << lane) - 1u))] = 2 * k;
    if (tid == 0) {
      s_part[0] = 2 * c + 1;
      s_n = total;
    }
  }
  __syncthreads();
  const int n = s_n;
  const int64_t t = p.HG == 1 ? row : row >> 1;
  const int hg = p.HG == 1 ? 0 : (int)(row & 1);
  const int heads = min(kHG, p.H - hg * kHG);
  const int per = kHG / gridDim.y;
  for (int h = blockIdx.y * per; h < (int)(blockIdx.y + 1) * per && h < heads; ++h) {
    if (tid < 32) {
      float M = kNoMax, L = 0.0f;
      for (int i = tid; i < n; i += 32) M = fmaxf(M, p.ws_ml[(int64_t)s_part[i] * 2 * kHG + h]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      for (int i = tid; i < n; i += 32) {
        const float w = ex2_approx(p.ws_ml[(int64_t)s_part[i] * 2 * kHG + h] - M);
        s_w[i] = w;
        L += w * p.ws_ml[(int64_t)s_part[i] * 2 * kHG + kHG + h];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (tid == 0) {
        s_L = L;
        if (p.lse) p.lse[t * p.lse_st + hg * kHG + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
      }
    }
    __syncthreads();
    const int col = tid & 63, pg = tid >> 6;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = pg; i < n; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p.ws_o + ((int64_t)s_part[i] * kHG + h) * kD + 4 * col);
      const float w = s_w[i];
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
    s_acc[pg][col] = acc;
    __syncthreads();
    if (pg == 0) {
      const float L = s_L, inv = L > 0.0f ? 1.0f / L : (L == 0.0f ? 0.0f : L);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const float4 v = s_acc[i][col];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      *reinterpret_cast<uint2*>(p.out + t * p.out_st + (int64_t)(hg * kHG + h) * p.out_sh + 4 * col) =
          make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
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
  size_t o, ml, tail, head, first, bytes;
};
Ws ws_layout(int G) {
  Ws w;
  w.o = 0;
  w.ml = w.o + (size_t)2 * G * kHG * kD * 4;
  w.tail = w.ml + (size_t)2 * G * 2 * kHG * 4;
  w.head = w.tail + (size_t)G * 8;
  w.first = w.head + (size_t)G * 4;
  w.bytes = w.first + (size_t)G * 4;
  return w;
}

// One CTA per SM, and no more than there can be tiles.
int grid_of(const Params& p, const DeviceInfo& dev) {
  const int64_t tiles = (p.pos_limit < 0x7FFFFFFF ? p.pos_limit : 0x7FFFFFFF) / kBN + 1;
  const int sms = dev.sm_count < kMaxCtas ? dev.sm_count : kMaxCtas;
  const int64_t most = p.T * p.HG * tiles;
  return (int)(most < sms ? most : sms);
}

template <int KIND, bool MASS, bool MODS>
cudaError_t launch_one(const Params& p, cudaStream_t s) {
  paged_kernel<KIND, MASS, MODS><<<(unsigned)p.G, kThreads, Cfg<KIND, MASS>::SMEM_BYTES, s>>>(p);
  return cudaGetLastError();
}

template <bool MASS>
cudaError_t launch(const Params& p, int kind, cudaStream_t s) {
  const bool mods = p.cap > 0.0f || p.slopes;
  if (kind == DSA_CACHE_BF16)
    return mods ? launch_one<DSA_CACHE_BF16, MASS, true>(p, s) : launch_one<DSA_CACHE_BF16, MASS, false>(p, s);
  return mods ? launch_one<DSA_CACHE_FP8_SCALED, MASS, true>(p, s) : launch_one<DSA_CACHE_FP8_SCALED, MASS, false>(p, s);
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
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  paged::Params p = paged::make_params(a);
  p.G = paged::grid_of(p, dev);
  const paged::Ws w = paged::ws_layout(p.G);
  if (!a->workspace || !aligned(a->workspace, 256)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->workspace_bytes < w.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p.ws_o = reinterpret_cast<float*>(ws + w.o);
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml);
  p.ws_tail = reinterpret_cast<int64_t*>(ws + w.tail);
  p.ws_head = reinterpret_cast<int*>(ws + w.head);
  p.ws_first = reinterpret_cast<int*>(ws + w.first);
  if ((st = paged::prepare_kernels(dev.device)) != DSA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = paged::launch<false>(p, a->kind, s);
  if (e != cudaSuccess) return cuda_fail(e);
  if (p.G == 1) return DSA_OK;  // no border, nothing to join
  // the join's blocks: a row (or CTA) each, its heads over as many blocks as fill the device
  const int64_t nrows = p.T * p.HG;
  const int x = (int)(nrows <= p.G ? nrows : p.G);
  int y = 64;
  while (y > 8 && x * y > 16 * dev.sm_count) y >>= 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)x, (unsigned)y);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged::join_kernel, p);
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
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  paged::Params p = paged::make_params(a);
  if (mass_width < p.pos_limit) p.pos_limit = mass_width;
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
    const cudaError_t e = paged::launch<true>(p, a->kind, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    p.mass = mass_out;
    p.mass_st = mass_out_stride;
  }
  return DSA_OK;
}
