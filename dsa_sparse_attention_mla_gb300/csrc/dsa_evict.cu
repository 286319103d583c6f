// dsa_evict.cu - eviction from the paged latent cache by accumulated attention weight
// (dsa_cache_evict).
//
// Request r holds n positions with a mass each and may keep b < n. Kept are the b largest masses
// (protected positions rank as +inf, ties to the lower position): with order-preserving integer
// keys, the positions whose key exceeds the b-th largest key u*, and the first ones at u*. The
// kept positions at or past b move into the evicted positions below b, in order: as many of one
// as of the other, and sources and destinations are disjoint, so rows move in place and at once
// and no more than the evicted number of them.
//
// Two launches.
//  * select: one CTA per request. The keys are made once and kept in shared memory (rows past
//    kKeys positions are made anew in every pass). u* by a radix selection of 11, 11 and 10 bits on
//    an integer histogram in shared memory: a log-normal mass fills few of 256 leading bytes, and the
//    atomics on them collide, but some fifty of 2048 leading elevens. Then each warp takes a
//    contiguous share of the positions, and ballots and a scan over the warps number the ties at u*,
//    the holes below b and the movers past it in position order (no atomic decides an order); the
//    lists go to the workspace, and masses and positions follow them.
//  * move: the rows, over the whole device, four rows in flight per warp.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "dsa_host.h"

namespace dsa {
namespace evict {

constexpr int kBins = 2048;
constexpr int kKeys = 49152;      // keys that shared memory holds (192 KB)
// Threads of a select CTA, by the rows' width: passes over few positions are bound by what every
// thread does beside them (scans, barriers). Both launches from a captured graph behind an L2 flush, of
// which an empty replay takes 7 us: 256 requests of 1088 positions 24 us with 512, 32 with 1024; 48 of
// 8192 46 and 42 when it was tried (40 now). Calls from the host, one after another: 26 - 32 us for the
// former with either (the host's own time), 36.9 for the latter.
constexpr int kFew = 512, kMany = 1024;
constexpr int kFewWidth = 4096;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;      // rows in flight per warp

struct Params {
  uint8_t* cache;
  int64_t num_slots;
  const int32_t* bt;
  int64_t bt_stride;
  int page_size;
  int64_t pos_limit;
  const int32_t* lengths;
  const int32_t* budgets;
  int budget, sink, recent;
  int64_t width;
  int keys;  // keys in shared memory
  const float* mass;
  int64_t mass_st;
  const int32_t* pos;
  int64_t pos_st;
  float* mass_out;
  int64_t mass_out_st;
  int32_t* pos_out;
  int64_t pos_out_st;
  int32_t* len_out;
  int32_t* moves;   // [R] rows to move
  int32_t* lists;   // [R][2][list_st]: sources, destinations
  int64_t list_st;
  int32_t* err;
};

// larger mass <=> larger key; -0 as +0
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t b = __float_as_uint(m == 0.0f ? 0.0f : m);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ int64_t slot_of(const Params& p, int64_t r, int j) {
  if (!p.bt) return j;
  const uint32_t pg = (uint32_t)j / (uint32_t)p.page_size;
  return (int64_t)p.bt[r * p.bt_stride + pg] * p.page_size + ((uint32_t)j - pg * (uint32_t)p.page_size);
}

// Exclusive sum over the NW warps of one count per warp (lane 0's `v` counts), and the total.
template <int NW>
__device__ __forceinline__ int warp_scan(int v, int* buf, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();  // earlier readers of buf are done
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  const int x = lane < NW ? buf[lane] : 0;
  int s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  return __shfl_sync(0xffffffffu, s - x, warp);
}
template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ Params p) {
  constexpr int kWarps = kThreads / 32, kPer = kBins / kThreads;  // bins per thread
  static_assert(kWarps <= 32 && kPer * kThreads == kBins, "one lane per warp in the scans");
  extern __shared__ uint32_t s_keys[];
  __shared__ int hist[kBins];
  __shared__ int wbuf[kWarps];
  __shared__ int s_newest, s_digit, s_need;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x;
  const float* mass = p.mass + r * p.mass_st;
  const int32_t* pos = p.pos ? p.pos + r * p.pos_st : nullptr;
  float* mass_out = p.mass_out + r * p.mass_out_st;
  int32_t* pos_out = p.pos_out ? p.pos_out + r * p.pos_out_st : nullptr;
  const int64_t len = p.lengths[r];
  const int n = (int)(len < 0 ? 0 : (len < p.width ? len : p.width));
  const int bq = p.budgets ? p.budgets[r] : p.budget;
  const int b = bq < 0 ? 0 : bq;

  // the request's pages, and its newest token position
  int bad = len > p.width || len > p.pos_limit;
  if (tid == 0) s_newest = INT32_MIN;
  __syncthreads();
  if (!bad && n > b) {
    if (p.bt) {
      const int pages = (n - 1) / p.page_size + 1;
      for (int i = tid; i < pages; i += kThreads) {
        const int64_t pg = p.bt[r * p.bt_stride + i];
        const int64_t last = i + 1 < pages ? p.page_size - 1 : (n - 1) % p.page_size;
        bad |= pg < 0 || pg * p.page_size + last >= p.num_slots;
      }
    }
    if (pos && p.recent > 0) {
      int nw = INT32_MIN;
      for (int j = tid; j < n; j += kThreads) nw = max(nw, pos[j]);
      nw = __reduce_max_sync(0xffffffffu, nw);
      if (lane == 0) atomicMax(&s_newest, nw);
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
  if (bad || n <= b) {
    if (mass_out != mass)
      for (int j = tid; j < n; j += kThreads) mass_out[j] = mass[j];
    if (pos_out && pos_out != pos)
      for (int j = tid; j < n; j += kThreads) pos_out[j] = pos ? pos[j] : j;
    if (tid == 0) {
      p.len_out[r] = (int32_t)len;
      p.moves[r] = 0;
    }
    return;
  }
  const int64_t newest = pos ? s_newest : n - 1;
  auto make_key = [&](int j) -> uint32_t {
    const int64_t k = pos ? pos[j] : j;
    if (k < p.sink || (p.recent > 0 && k > newest - p.recent)) return 0xFF800000u;  // the key of +inf
    return mass_key(mass[j]);
  };
  const bool cached = n <= p.keys;
  auto key_of = [&](int j) -> uint32_t { return cached ? s_keys[j] : make_key(j); };

  // the b-th largest key u*; `need` of the keys equal to it are kept
  uint32_t prefix = 0;
  int need = b;
  if (b > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      if (pass == 0) {
        for (int j = tid; j < n; j += kThreads) {
          const uint32_t k = make_key(j);
          if (cached) s_keys[j] = k;
          atomicAdd(&hist[k >> 21], 1);
        }
      } else {
        for (int j = tid; j < n; j += kThreads) {
          const uint32_t k = key_of(j);
          if (((k ^ prefix) >> (shift + bits)) == 0) atomicAdd(&hist[(k >> shift) & ((1 << bits) - 1)], 1);
        }
      }
      __syncthreads();
      // the digit at which the counts from the top reach `need`: thread t takes the kPer bins that end
      // at 2047 - kPer t, and sums run downwards
      int c[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        c[i] = hist[kBins - 1 - kPer * tid - i];
        mine += c[i];
      }
      int s = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      int total;
      const int in_warp = __shfl_sync(0xffffffffu, s, 31);
      int above = warp_scan<kWarps>(in_warp, wbuf, &total) + s - mine;  // keys with a digit above this thread's
      if (above < need && above + mine >= need) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (above < need && above + c[i] >= need) {
            s_digit = kBins - 1 - kPer * tid - i;
            s_need = need - above;
          }
          above += c[i];
        }
      }
      __syncthreads();
      prefix |= (uint32_t)s_digit << shift;
      need = s_need;
    }
  }
  if (b == 0) __syncthreads();

  // a contiguous share of whole strips of 32 positions per warp
  const int strips = (n + 31) / 32, per = (strips + kWarps - 1) / kWarps;
  const int j0 = warp * per * 32, j1 = min(n, j0 + per * 32);
  int ties = 0;
  if (b > 0)
    for (int j = j0 + lane; j - lane < j1; j += 32)
      ties += __popc(__ballot_sync(0xffffffffu, j < j1 && key_of(j) == prefix));
  int total;
  const int tie0 = warp_scan<kWarps>(ties, wbuf, &total);
  // whether position j is kept (all lanes of a strip at once); t counts the ties before the strip
  auto kept = [&](int j, int& t) -> bool {
    if (b == 0) return false;
    const uint32_t k = j < j1 ? key_of(j) : 0u;
    const bool tie = j < j1 && k == prefix;
    const uint32_t m = __ballot_sync(0xffffffffu, tie);
    const int rank = t + __popc(m & ((1u << lane) - 1u));
    t += __popc(m);
    return j < j1 && (k > prefix || (tie && rank < need));
  };
  int holes = 0, movers = 0;
  {
    int t = tie0;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      const bool keep = kept(j, t);
      holes += __popc(__ballot_sync(0xffffffffu, j < j1 && j < b && !keep));
      movers += __popc(__ballot_sync(0xffffffffu, j >= b && keep));
    }
  }
  int count;
  int hole0 = warp_scan<kWarps>(holes, wbuf, &total), mover0 = warp_scan<kWarps>(movers, wbuf, &count);
  int32_t* src = p.lists + r * 2 * p.list_st;
  int32_t* dst = src + p.list_st;
  {
    int t = tie0;
    const uint32_t below = (1u << lane) - 1u;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      const bool keep = kept(j, t);
      const bool hole = j < j1 && j < b && !keep, mover = j >= b && keep;
      const uint32_t hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
      if (hole) dst[hole0 + __popc(hm & below)] = j;
      if (mover) src[mover0 + __popc(mm & below)] = j;
      hole0 += __popc(hm);
      mover0 += __popc(mm);
      if (keep && j < b) {
        if (mass_out != mass) mass_out[j] = mass[j];
        if (pos_out && pos_out != pos) pos_out[j] = pos ? pos[j] : j;
      }
    }
  }
  if (tid == 0) {
    p.moves[r] = count;
    p.len_out[r] = b;
  }
  __syncthreads();  // the lists are complete
  for (int i = tid; i < count; i += kThreads) {
    const int s = src[i], d = dst[i];
    mass_out[d] = mass[s];
    if (pos_out) pos_out[d] = pos ? pos[s] : s;
  }
  __syncthreads();  // in place: the movers' masses are read before they are cleared
  for (int j = b + tid; j < n; j += kThreads) mass_out[j] = 0.0f;
}

// Rows of 8 * WORDS bytes. Block (x, y) moves rows of request y: four per warp at a time, all read
// before the first is written (sources and destinations are disjoint anyhow).
template <int WORDS>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ Params p) {
  constexpr int PER = (WORDS + 31) / 32;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t r = blockIdx.y;
  const int n = p.moves[r];
  const int32_t* list = p.lists + r * 2 * p.list_st;
  const int warps = gridDim.x * (kMoveThreads / 32);
  for (int i0 = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kMoveRows; i0 < n; i0 += warps * kMoveRows) {
    // lanes 0 - 3: source slots, 4 - 7: destinations
    int64_t slot = -1;
    const int i = i0 + (lane & 3);
    if (lane < 8 && i < n) slot = slot_of(p, r, list[(lane >> 2) * p.list_st + i]);
    uint2 v[kMoveRows][PER];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int64_t s = __shfl_sync(0xffffffffu, slot, k);
#pragma unroll
      for (int w = 0; w < PER; ++w)
        if (s >= 0 && 32 * w + lane < WORDS)
          v[k][w] = reinterpret_cast<const uint2*>(p.cache + s * (8 * WORDS))[32 * w + lane];
    }
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int64_t d = __shfl_sync(0xffffffffu, slot, 4 + k);
#pragma unroll
      for (int w = 0; w < PER; ++w)
        if (d >= 0 && 32 * w + lane < WORDS) reinterpret_cast<uint2*>(p.cache + d * (8 * WORDS))[32 * w + lane] = v[k][w];
    }
  }
}

struct Ws {
  size_t moves, lists, bytes;
  int64_t list_st;
};
// At most half of a request's positions move: a source and a destination each.
Ws ws_layout(int64_t requests, int64_t width) {
  Ws w;
  w.list_st = (width + 1) / 2;
  w.lists = 0;
  w.moves = (size_t)requests * (size_t)w.list_st * 8;
  w.bytes = w.moves + (size_t)requests * 4;
  return w;
}

dsa_status_t prepare(int device) {
  static std::mutex mu;
  static bool done[64];
  std::lock_guard<std::mutex> lock(mu);
  if (done[device]) return DSA_OK;
  cudaError_t e = cudaFuncSetAttribute(select_kernel<kFew>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeys * 4);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(select_kernel<kMany>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeys * 4);
  if (e != cudaSuccess) return cuda_fail(e);
  done[device] = true;
  return DSA_OK;
}

template <int WORDS>
cudaError_t launch_move(const Params& p, dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, move_kernel<WORDS>, p);
}

}  // namespace evict
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_cache_evict_workspace_size(int64_t num_requests, int64_t width, size_t* bytes) {
  if (!bytes || num_requests < 0 || width < 1 || width > (1 << 30)) return DSA_ERR_INVALID_ARGUMENT;
  *bytes = evict::ws_layout(num_requests, width).bytes;
  return DSA_OK;
}

extern "C" dsa_status_t dsa_cache_evict(const dsa_evict_args_t* a, void* stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->kind != DSA_CACHE_BF16 && a->kind != DSA_CACHE_FP8_SCALED) return DSA_ERR_INVALID_ARGUMENT;
  if (!((a->d_nope == 256 && a->d_rope == 0) || (a->d_nope == 512 && a->d_rope == 64))) return DSA_ERR_UNSUPPORTED;
  if (a->num_requests < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (a->num_requests == 0) return DSA_OK;
  if (a->num_requests > 65535) return DSA_ERR_UNSUPPORTED;
  if (!a->cache || !aligned(a->cache, 8) || a->num_slots < 0 || !a->lengths || !a->mass || !a->mass_out ||
      !a->lengths_out)
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->block_table) {
    if (a->page_size < 1 || a->max_pages < 0 || a->bt_stride < a->max_pages) return DSA_ERR_INVALID_ARGUMENT;
  } else if (a->num_requests != 1) {
    return DSA_ERR_INVALID_ARGUMENT;
  }
  if (a->sink < 0 || a->recent < 0 || (!a->budgets && a->budget < 0)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->width < 1 || a->width > (1 << 30)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->mass_stride < a->width || a->mass_out_stride < a->width) return DSA_ERR_INVALID_ARGUMENT;
  if (a->positions && (a->positions_stride < a->width || !a->positions_out)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->positions_out && a->positions_out_stride < a->width) return DSA_ERR_INVALID_ARGUMENT;
  // in place means the same rows
  if (a->mass_out == a->mass && a->mass_out_stride != a->mass_stride) return DSA_ERR_INVALID_ARGUMENT;
  if (a->positions && a->positions_out == a->positions && a->positions_out_stride != a->positions_stride)
    return DSA_ERR_INVALID_ARGUMENT;
  const evict::Ws w = evict::ws_layout(a->num_requests, a->width);
  if (!a->workspace || !aligned(a->workspace, 8)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->workspace_bytes < w.bytes) return DSA_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  dsa_status_t st = current_device(&dev);
  if (st != DSA_OK || (st = evict::prepare(dev.device)) != DSA_OK) return st;
  evict::Params p{};
  p.cache = static_cast<uint8_t*>(a->cache);
  p.num_slots = a->num_slots;
  p.bt = a->block_table;
  p.bt_stride = a->bt_stride;
  p.page_size = a->block_table ? a->page_size : 1;
  p.pos_limit = a->block_table ? (int64_t)a->max_pages * a->page_size : a->num_slots;
  p.lengths = a->lengths;
  p.budgets = a->budgets;
  p.budget = a->budget;
  p.sink = a->sink;
  p.recent = a->recent;
  p.width = a->width;
  p.keys = (int)(a->width < evict::kKeys ? a->width : evict::kKeys);
  p.mass = a->mass;
  p.mass_st = a->mass_stride;
  p.pos = a->positions;
  p.pos_st = a->positions_stride;
  p.mass_out = a->mass_out;
  p.mass_out_st = a->mass_out_stride;
  p.pos_out = a->positions_out;
  p.pos_out_st = a->positions_out_stride;
  p.len_out = a->lengths_out;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  p.lists = reinterpret_cast<int32_t*>(ws + w.lists);
  p.moves = reinterpret_cast<int32_t*>(ws + w.moves);
  p.list_st = w.list_st;
  p.err = a->error_word;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->width <= evict::kFewWidth)
    evict::select_kernel<evict::kFew><<<(unsigned)a->num_requests, evict::kFew, (size_t)p.keys * 4, s>>>(p);
  else
    evict::select_kernel<evict::kMany><<<(unsigned)a->num_requests, evict::kMany, (size_t)p.keys * 4, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e);
  // blocks per request: the device eight blocks deep, and no more than the most moves can use
  const int64_t rows_per_block = evict::kMoveRows * (evict::kMoveThreads / 32);
  const int64_t most = (w.list_st + rows_per_block - 1) / rows_per_block;
  int64_t x = (8 * (int64_t)dev.sm_count + a->num_requests - 1) / a->num_requests;
  if (x > most) x = most;
  const dim3 grid((unsigned)x, (unsigned)a->num_requests);
  switch (dsa_cache_row_bytes(a->kind, a->d_nope, a->d_rope)) {
    case 264: e = evict::launch_move<33>(p, grid, s); break;
    case 512: e = evict::launch_move<64>(p, grid, s); break;
    case 656: e = evict::launch_move<82>(p, grid, s); break;
    default: e = evict::launch_move<144>(p, grid, s); break;
  }
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
