// dsa_plan.cu - the batch plan of a serving step: block tables brought to the requests' lengths
// through a stack of free pages, and the slot maps of the tokens that the step adds.
//
// Three prefix sums over the requests carry it: pages given back, then pages wanted and tokens
// wanted (whose inclusive sums decide what is refused), then both again over what is granted. Every
// page moved finds its request by a binary search in the sums of its chunk of requests, so a step
// with one long prompt and one with many short ones cost the same per page.
//
// The sums need every request, and a decode step has a few hundred: a cluster of blocks does the step,
// each block all the sums (for itself, so that no value has to be passed on) and its share of the pages
// and tokens. Between the parts lies a barrier of the cluster. What bounds it is the chain of dependent
// loads (state, table, stack, table again), not bytes: 256 requests that add a token each, 16 of which end
// and give back their pages, take 9.0 us in a graph of twenty calls, 48 prompts of 201038 tokens with 12564 pages 11.0.
// (As the replay of a single call, two to three us more: 10.3, 18.5 with one block; 14.4, 26.6 with one block and no
// overlap of the tokens' launch.) More than 1024 requests have one block: 4096 take 61 us where they move 25420
// pages and add 3840 tokens, 147 where they move 104622 and add 65255.
#include <cuda_runtime.h>

#include <climits>

#include "dsa_host.h"

namespace dsa {
namespace plan {

constexpr int kThreads = 1024;     // requests of a chunk, one per thread
constexpr int kCluster = 8;
constexpr int kAhead = 4;          // pages a thread moves at a time, their loads in flight together
constexpr int kFillThreads = 256;
constexpr int64_t kMaxFill = 16384;  // tokens that the plan's own blocks write

struct Params {
  int64_t R;
  const int32_t *lengths, *add, *held;
  int32_t* bt;
  int64_t bt_st;
  int page, max_pages;
  int32_t* stack;
  int64_t cap;
  const int32_t* num_free;
  int32_t *len_out, *held_out, *num_free_out;
  int64_t T;
  int32_t *cu, *req, *pos, *tlen;
  int64_t* loc;
  int32_t* err;
  const int32_t* seen;
  int32_t *seen_out, *tok, *kpos;
  int64_t kp_st;
  int kp_width;  // INT_MAX without kpos
};

// Inclusive sums over the block of two values per thread; *total receives the sums over all threads.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2 (&s_warp)[32], longlong2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  longlong2 w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  total->x = __shfl_sync(0xffffffffu, w.x, 31);
  total->y = __shfl_sync(0xffffffffu, w.y, 31);
  if (warp > 0) {
    v.x += __shfl_sync(0xffffffffu, w.x, warp - 1);
    v.y += __shfl_sync(0xffffffffu, w.y, warp - 1);
  }
  return v;
}

// The first of n ascending entries that exceeds i.
template <class V>
__device__ __forceinline__ int64_t first_above(const V* a, int64_t n, int64_t i) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (a[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// The entries of token slot i of request r, whose new length is `len`, which has been given `seen` tokens by now and
// whose tokens end before slot `next`. The table's entries may have been written by another block of the cluster: past L1.
__device__ __forceinline__ void fill(const Params& p, int64_t i, int64_t r, int next, int len, int seen) {
  const int pos = len - next + (int)i, tok = seen - next + (int)i;
  const int page = __ldcg(p.bt + r * p.bt_st + pos / p.page);
  p.req[i] = (int)r;
  p.pos[i] = pos;
  p.tlen[i] = pos + 1;
  p.loc[i] = page < 0 ? -1 : (int64_t)page * p.page + pos % p.page;
  if (p.tok) p.tok[i] = tok;
  if (p.kpos) p.kpos[r * p.kp_st + pos] = tok;
}
__device__ __forceinline__ void fill_padding(const Params& p, int64_t i) {
  p.req[i] = 0;
  p.pos[i] = -1;
  p.tlen[i] = 0;
  p.loc[i] = -1;
  if (p.tok) p.tok[i] = -1;
}

// All blocks of the cluster: what each wrote before is seen by the others after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Want {
  uint32_t after, need;  // the request's length and pages if it is granted (below 2^32 both)
  uint32_t seen_after;   // and the tokens it has been given
  int l, h, seen;
  bool fits;
  long long back, take, tokens;
};

__device__ __forceinline__ Want want_of(const Params& p, int64_t r) {
  Want w;
  w.l = max(p.lengths[r], 0);
  w.h = min(max(p.held[r], 0), p.max_pages);
  const int n = p.add[r];
  w.after = n < 0 ? 0 : (uint32_t)w.l + (uint32_t)n;
  w.need = w.after ? (w.after - 1) / (uint32_t)p.page + 1 : 0;
  w.seen = p.seen ? max(p.seen[r], 0) : w.l;
  w.seen_after = n < 0 ? 0 : (uint32_t)w.seen + (uint32_t)n;
  w.fits = w.need <= (uint32_t)p.max_pages && max(w.after, w.seen_after) <= (uint32_t)INT_MAX &&
           (n <= 0 || w.after <= (uint32_t)p.kp_width);
  w.back = w.need < (uint32_t)w.h ? w.h - (int)w.need : 0;
  w.take = w.fits && w.need > (uint32_t)w.h ? (int)w.need - w.h : 0;
  w.tokens = w.fits && n > 0 ? n : 0;
  return w;
}

// Moves the pages of a chunk that are this block's share: page i is the j-th of request k of the chunk
// (`sums`: its inclusive sums), load(k, j, i) gives it and store(k, j, i, page) takes it.
template <class Load, class Store>
__device__ __forceinline__ void each_page(const long long* sums, int64_t total, int rank, int blocks, Load load, Store store) {
  const int64_t step = (int64_t)blocks * kThreads;
  for (int64_t i0 = (int64_t)rank * kThreads + threadIdx.x; i0 < total; i0 += kAhead * step) {
    int k[kAhead], v[kAhead];
    int64_t j[kAhead];
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int64_t i = i0 + z * step;
      if (i >= total) break;
      k[z] = (int)first_above(sums, kThreads, i);
      j[z] = i - (k[z] ? sums[k[z] - 1] : 0);
      v[z] = load(k[z], j[z], i);
    }
#pragma unroll
    for (int z = 0; z < kAhead; ++z) {
      const int64_t i = i0 + z * step;
      if (i >= total) break;
      store(k[z], j[z], i, v[z]);
    }
  }
}

// `blocks` of the cluster (1: no cluster). More than one only where one chunk holds all requests: then no
// block reads the requests' state after the first barrier, and it may change in place.
__global__ void __launch_bounds__(kThreads) plan_kernel(const Params p, const int blocks, const int fill_here) {
  __shared__ longlong2 s_warp[32];
  __shared__ long long s_sum[kThreads];  // inclusive page sums of the chunk
  __shared__ int s_first[kThreads];      // first table entry that a request gives back or takes
  __shared__ int s_cu[kThreads + 1], s_len[kThreads], s_seen[kThreads];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, rank = blocks > 1 ? (int)blockIdx.x : 0;
  const int64_t nf = min((int64_t)max(*p.num_free, 0), p.cap);
  const bool one = p.R <= kThreads;
  auto sync = [&]() {
    if (blocks > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  int bad = 0;
  longlong2 total;
  Want w{};
  // pages given back go onto the stack
  int64_t have = nf;
  for (int64_t r0 = 0; r0 < p.R; r0 += kThreads) {
    const int64_t r = r0 + tid;
    w = Want{};
    if (r < p.R) w = want_of(p, r);
    const longlong2 sum = block_scan(make_longlong2(w.back, 0), s_warp, &total);
    s_sum[tid] = sum.x;
    s_first[tid] = (int)w.need;
    __syncthreads();
    each_page(
        s_sum, total.x, rank, blocks,
        [&](int k, int64_t j, int64_t) { return __ldcg(p.bt + (r0 + k) * p.bt_st + s_first[k] + j); },
        [&](int, int64_t, int64_t i, int page) {
          if (have + i < p.cap)
            p.stack[have + i] = page;
          else
            bad = DSA_DEVERR_SLOT_OUT_OF_RANGE;
        });
    have += total.x;
    __syncthreads();
  }
  if (have > p.cap) have = p.cap;
  sync();
  // what is wanted, what of it is granted, and the pages taken from the top
  longlong2 wanted = make_longlong2(0, 0), granted = make_longlong2(0, 0);
  for (int64_t r0 = 0; r0 < p.R; r0 += kThreads) {
    const int64_t r = r0 + tid;
    if (!one) {
      w = Want{};
      if (r < p.R) w = want_of(p, r);
    }
    longlong2 sum = block_scan(make_longlong2(w.take, w.tokens), s_warp, &total);
    const bool no_page = w.take > 0 && wanted.x + sum.x > have;
    const bool no_room = w.tokens > 0 && wanted.y + sum.y > p.T;
    wanted.x += total.x;
    wanted.y += total.y;
    const bool ok = w.fits && !no_page && !no_room;
    // (a chunk that is granted whole has its sums already)
    const bool whole = __syncthreads_and(r >= p.R || ok || (w.take == 0 && w.tokens == 0));
    if (r < p.R && rank == 0) {
      if (!w.fits) bad |= DSA_DEVERR_INDEX_OUT_OF_RANGE;
      if (no_page) bad |= DSA_DEVERR_OUT_OF_PAGES;
      if (no_room) bad |= DSA_DEVERR_TOKEN_CAPACITY;
    }
    if (!ok) w.take = w.tokens = 0;
    if (!whole) sum = block_scan(make_longlong2(w.take, w.tokens), s_warp, &total);
    s_sum[tid] = sum.x;
    s_first[tid] = w.h;
    if (r < p.R) {
      const int len = ok ? (int)w.after : w.l, cu = (int)(granted.y + sum.y), seen = ok ? (int)w.seen_after : w.seen;
      s_cu[tid + 1] = cu;
      s_len[tid] = len;
      s_seen[tid] = seen;
      if (rank == 0) {
        p.len_out[r] = len;
        if (p.seen) p.seen_out[r] = seen;
        p.held_out[r] = w.take > 0 || w.need < (uint32_t)w.h ? (int)w.need : w.h;
        p.cu[r + 1] = cu;
      }
    }
    __syncthreads();
    each_page(
        s_sum, total.x, rank, blocks,
        [&](int, int64_t, int64_t i) { return __ldcg(p.stack + have - 1 - granted.x - i); },
        [&](int k, int64_t j, int64_t, int page) { p.bt[(r0 + k) * p.bt_st + s_first[k] + j] = page; });
    granted.x += total.x;
    granted.y += total.y;
    __syncthreads();
  }
  if (tid == 0 && rank == 0) {
    p.cu[0] = 0;
    *p.num_free_out = (int)(have - granted.x);
  }
  if (bad && p.err) atomicOr(p.err, bad);
  if (!fill_here) return;
  sync();
  const int64_t step = (int64_t)blocks * kThreads;
  for (int64_t i = (int64_t)rank * kThreads + tid; i < p.T; i += step) {
    if (i >= granted.y) {
      fill_padding(p, i);
    } else if (one) {
      const int r = (int)first_above(s_cu + 1, p.R, i);
      fill(p, i, r, s_cu[r + 1], s_len[r], s_seen[r]);
    } else {
      const int64_t r = first_above(p.cu + 1, p.R, i);
      const int len = p.len_out[r];
      fill(p, i, r, p.cu[r + 1], len, p.seen ? p.seen_out[r] : len);
    }
  }
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(const Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * kFillThreads + threadIdx.x;
  if (i >= p.T) return;
  if (i >= p.cu[p.R]) {
    fill_padding(p, i);
    return;
  }
  const int64_t r = first_above(p.cu + 1, p.R, i);
  const int len = p.len_out[r];
  fill(p, i, r, p.cu[r + 1], len, p.seen ? p.seen_out[r] : len);
}

}  // namespace plan
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_batch_plan(const dsa_plan_args_t* a, void* stream) {
  if (!a || a->num_requests < 0 || a->T < 0 || a->free_capacity < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (a->num_requests > (1 << 20) || a->T > (1 << 30) || a->free_capacity > INT_MAX) return DSA_ERR_UNSUPPORTED;
  if (a->page_size < 1 || a->max_pages < 0 || a->bt_stride < a->max_pages) return DSA_ERR_INVALID_ARGUMENT;
  if (!a->num_free || !a->num_free_out || !a->cu_tokens || (a->free_capacity > 0 && !a->free_pages))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->num_requests > 0 && (!a->lengths || !a->new_tokens || !a->held || !a->lengths_out || !a->held_out ||
                              (a->max_pages > 0 && !a->block_table)))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->T > 0 && (!a->req_of_token || !a->positions || !a->token_lengths || !a->out_loc)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->num_requests > 0 && a->seen && !a->seen_out) return DSA_ERR_INVALID_ARGUMENT;
  if (a->key_positions && (a->kp_width < 0 || a->kp_stride < a->kp_width)) return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(a->out_loc, 8)) return DSA_ERR_INVALID_ARGUMENT;
  for (const void* q : {(const void*)a->lengths, (const void*)a->new_tokens, (const void*)a->held, (const void*)a->block_table,
                        (const void*)a->free_pages, (const void*)a->num_free, (const void*)a->lengths_out,
                        (const void*)a->held_out, (const void*)a->num_free_out, (const void*)a->cu_tokens,
                        (const void*)a->req_of_token, (const void*)a->positions, (const void*)a->token_lengths,
                        (const void*)a->error_word, (const void*)a->seen, (const void*)a->seen_out,
                        (const void*)a->token_positions, (const void*)a->key_positions})
    if (!aligned(q, 4)) return DSA_ERR_INVALID_ARGUMENT;
  DeviceInfo dev;
  const dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  plan::Params p{};
  p.R = a->num_requests;
  p.lengths = a->lengths;
  p.add = a->new_tokens;
  p.held = a->held;
  p.bt = a->block_table;
  p.bt_st = a->bt_stride;
  p.page = a->page_size;
  p.max_pages = a->max_pages;
  p.stack = a->free_pages;
  p.cap = a->free_capacity;
  p.num_free = a->num_free;
  p.len_out = a->lengths_out;
  p.held_out = a->held_out;
  p.num_free_out = a->num_free_out;
  p.T = a->T;
  p.cu = a->cu_tokens;
  p.req = a->req_of_token;
  p.pos = a->positions;
  p.tlen = a->token_lengths;
  p.loc = a->out_loc;
  p.err = a->error_word;
  p.seen = a->seen;
  p.seen_out = a->seen_out;
  p.tok = a->token_positions;
  p.kpos = a->key_positions;
  p.kp_st = a->kp_stride;
  p.kp_width = a->key_positions && a->kp_width < INT_MAX ? (int)a->kp_width : INT_MAX;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool here = p.T <= plan::kMaxFill;
  // One block where it can have little to move, and where the requests take several chunks (see the kernel).
  const bool little = p.T <= plan::kThreads && (double)p.R * p.max_pages <= plan::kAhead * plan::kThreads;
  const int blocks = p.R <= plan::kThreads && !little ? plan::kCluster : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(plan::kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, plan::plan_kernel, (const plan::Params)p, blocks, (int)here);
  if (e != cudaSuccess) return cuda_fail(e);
  if (!here) {
    cfg.gridDim = dim3((unsigned)((p.T + plan::kFillThreads - 1) / plan::kFillThreads));
    cfg.blockDim = dim3(plan::kFillThreads);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    e = cudaLaunchKernelEx(&cfg, plan::fill_kernel, (const plan::Params)p);
  }
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
