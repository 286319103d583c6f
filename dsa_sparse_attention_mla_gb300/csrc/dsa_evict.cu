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
// One CTA per request. The b-th largest key is found by a radix selection, eight bits per pass
// over the masses, on an integer histogram in shared memory; holes and movers are numbered by
// block scans in position order (no atomics decide an order); the holes go into the workspace, and
// warps then copy row by row.
#include <cuda_runtime.h>

#include <cstdint>

#include "dsa_host.h"

namespace dsa {
namespace evict {

constexpr int kThreads = 512;

struct Params {
  uint8_t* cache;
  int64_t num_slots;
  int row_words;  // cache row in 8-byte words
  const int32_t* bt;
  int64_t bt_stride;
  int page_size;
  int64_t pos_limit;
  const int32_t* lengths;
  const int32_t* budgets;
  int budget, sink, recent;
  int64_t width;
  const float* mass;
  int64_t mass_st;
  const int32_t* pos;
  int64_t pos_st;
  float* mass_out;
  int64_t mass_out_st;
  int32_t* pos_out;
  int64_t pos_out_st;
  int32_t* len_out;
  int32_t* ws;
  int64_t ws_st;  // workspace entries per request
  int32_t* err;
};

// larger mass <=> larger key; -0 as +0
__device__ __forceinline__ uint32_t mass_key(float m) {
  const uint32_t b = __float_as_uint(m == 0.0f ? 0.0f : m);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ int64_t slot_of(const Params& p, int64_t r, int64_t j) {
  if (!p.bt) return j;
  return (int64_t)p.bt[r * p.bt_stride + j / p.page_size] * p.page_size + j % p.page_size;
}

// exclusive sum over the block of v (a count per thread); *total gets the block's sum
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int s = warp_sums[w];
    if (w < warp) base += s;
    sum += s;
  }
  __syncthreads();
  *total = sum;
  return base + x - v;
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ Params p) {
  __shared__ int hist[256];
  __shared__ int wsum[kThreads / 32];
  __shared__ int s_newest;
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const float* mass = p.mass + r * p.mass_st;
  const int32_t* pos = p.pos ? p.pos + r * p.pos_st : nullptr;
  float* mass_out = p.mass_out + r * p.mass_out_st;
  int32_t* pos_out = p.pos_out ? p.pos_out + r * p.pos_out_st : nullptr;
  int32_t* holes = p.ws + r * p.ws_st;
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
    if (pos) {
      int nw = INT32_MIN;
      for (int j = tid; j < n; j += kThreads) nw = max(nw, pos[j]);
      atomicMax(&s_newest, nw);
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
  if (bad || n <= b) {
    if (mass_out != mass)
      for (int j = tid; j < n; j += kThreads) mass_out[j] = mass[j];
    if (pos_out && pos_out != pos)
      for (int j = tid; j < n; j += kThreads) pos_out[j] = pos ? pos[j] : j;
    if (tid == 0) p.len_out[r] = (int32_t)len;
    return;
  }
  const int64_t newest = pos ? s_newest : n - 1;
  auto key_of = [&](int j) -> uint32_t {
    const int64_t k = pos ? pos[j] : j;
    if (k < p.sink || k > newest - p.recent) return 0xFF800000u;  // the key of +inf
    return mass_key(mass[j]);
  };

  // the b-th largest key
  uint32_t prefix = 0;
  int need = b;  // of the keys that share the prefix, how many are kept
  for (int shift = 24; shift >= 0 && b > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int j = tid; j < n; j += kThreads) {
      const uint32_t k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, d = 255;
      for (; d > 0 && hist[d] < left; --d) left -= hist[d];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }

  // one pass in position order: number the ties at u*, the holes below b and the movers past it
  int ties = 0, nholes = 0, nmove = 0;
  for (int j0 = 0; j0 < n; j0 += kThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < n && b > 0 ? key_of(j) : 0u;
    const bool tie = j < n && b > 0 && k == prefix;
    int total;
    const int tr = ties + block_scan(tie ? 1 : 0, wsum, &total);
    ties += total;
    const bool keep = j < n && b > 0 && (k > prefix || (tie && tr < need));
    const bool hole = j < b && !keep, mover = j >= b && keep;
    const int packed = block_scan((hole ? 1 : 0) | (mover ? 1 << 16 : 0), wsum, &total);
    if (hole) holes[nholes + (packed & 0xFFFF)] = j;
    nholes += total & 0xFFFF;
    // every hole is below every mover, but a chunk may hold both: its holes are written first
    __syncthreads();
    if (j < b && keep) {
      if (mass_out != mass) mass_out[j] = mass[j];
      if (pos_out && pos_out != pos) pos_out[j] = pos ? pos[j] : j;
    }
    if (mover) {
      const int i = nmove + (packed >> 16);
      const int dst = holes[i];
      mass_out[dst] = mass[j];
      if (pos_out) pos_out[dst] = pos ? pos[j] : j;
      holes[i] = j;
      // the destination's place is known by rank again when the rows move
      p.ws[r * p.ws_st + p.ws_st / 2 + i] = dst;
    }
    nmove += total >> 16;
  }
  __syncthreads();
  for (int j = b + tid; j < n; j += kThreads) mass_out[j] = 0.0f;
  if (tid == 0) p.len_out[r] = b;

  const int lane = tid & 31;
  for (int i = tid >> 5; i < nmove; i += kThreads / 32) {
    const int64_t src = slot_of(p, r, holes[i]), dst = slot_of(p, r, holes[p.ws_st / 2 + i]);
    const uint2* s = reinterpret_cast<const uint2*>(p.cache + src * 8 * p.row_words);
    uint2* d = reinterpret_cast<uint2*>(p.cache + dst * 8 * p.row_words);
    for (int w = lane; w < p.row_words; w += 32) d[w] = s[w];
  }
}

}  // namespace evict
}  // namespace dsa

using namespace dsa;

// At most half of a request's positions move: a source and a destination each.
extern "C" dsa_status_t dsa_cache_evict_workspace_size(int64_t num_requests, int64_t width, size_t* bytes) {
  if (!bytes || num_requests < 0 || width < 1 || width > (1 << 30)) return DSA_ERR_INVALID_ARGUMENT;
  *bytes = (size_t)num_requests * (size_t)((width + 1) / 2) * 8;
  return DSA_OK;
}

extern "C" dsa_status_t dsa_cache_evict(const dsa_evict_args_t* a, void* stream) {
  if (!a) return DSA_ERR_INVALID_ARGUMENT;
  if (a->kind != DSA_CACHE_BF16 && a->kind != DSA_CACHE_FP8_SCALED) return DSA_ERR_INVALID_ARGUMENT;
  if (!((a->d_nope == 256 && a->d_rope == 0) || (a->d_nope == 512 && a->d_rope == 64))) return DSA_ERR_UNSUPPORTED;
  if (a->num_requests < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (a->num_requests == 0) return DSA_OK;
  if (a->num_requests > 0x7FFFFFFF) return DSA_ERR_UNSUPPORTED;
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
  size_t need = 0;
  dsa_status_t st = dsa_cache_evict_workspace_size(a->num_requests, a->width, &need);
  if (st != DSA_OK) return st;
  if (!a->workspace || !aligned(a->workspace, 8)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->workspace_bytes < need) return DSA_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  evict::Params p{};
  p.cache = static_cast<uint8_t*>(a->cache);
  p.num_slots = a->num_slots;
  p.row_words = (int)(dsa_cache_row_bytes(a->kind, a->d_nope, a->d_rope) / 8);
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
  p.mass = a->mass;
  p.mass_st = a->mass_stride;
  p.pos = a->positions;
  p.pos_st = a->positions_stride;
  p.mass_out = a->mass_out;
  p.mass_out_st = a->mass_out_stride;
  p.pos_out = a->positions_out;
  p.pos_out_st = a->positions_out_stride;
  p.len_out = a->lengths_out;
  p.ws = static_cast<int32_t*>(a->workspace);
  p.ws_st = (a->width + 1) / 2 * 2;
  p.err = a->error_word;
  evict::evict_kernel<<<(unsigned)a->num_requests, evict::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
