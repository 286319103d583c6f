// dsa_block.cu - blocks (pages) of the latent cache: the mean row of each block that a step's tokens
// lie in, and the choice of the blocks that each token attends to.
//
// Pool: summary[page] = mean of the block's rows. The tokens of a step name the blocks: a token leads
// its block when the token before it lies in another one, so no list of blocks has to be made first.
// The leader's block of threads reads the rows, one row per warp at a time, and the warps' fp32 sums
// are joined in a fixed order. 101739 bf16 rows in blocks of 64 (54 MB) take 8.1 us in a graph of calls on one
// state, whose rows lie in L2, and 15.1 after a write that takes them out of it: 3.6 TB/s, where the copy would take 8.0.
// A leader's loads form a chain (positions, then table and lengths, then rows) with nothing of the next leader on its way.
//
// Select: the m-th largest key of a row decides, found bit by bit: scores map to unsigned keys of the
// same order, blocks that are always chosen to the largest one, and up to 32 counts of the keys at or
// above a trial value build it from the top bit down. The keys stay in registers; ballots and their
// prefix sums put the chosen blocks in ascending order. 8192 rows of up to 512 blocks take 19.1 us in a graph of
// calls on one state, some 7 of it the search's chain of counts, the rest not taken apart (2048 blocks of threads in 1.7
// waves); 256 rows of up to 2048 take 8.0. With the inputs out of L2: 24.5 and 11.1. Rows of more than 8704 blocks read
// their keys anew for every count: 64 of up to 16384 take 49 us.
#include <cuda_runtime.h>

#include <climits>

#include "dsa_host.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace block {

// -------------------------------------------------------------------------------------- pool --
constexpr int kD = 256;
constexpr int kPoolThreads = 128;
constexpr int kPoolWarps = kPoolThreads / 32;
constexpr int kAhead = 8;  // rows a warp has in flight

struct PoolParams {
  const uint8_t* cache;
  int64_t num_slots;
  const int32_t* bt;
  int64_t bt_st;
  int page, max_pages;
  int64_t num_requests;
  const int32_t *pos, *req;
  int64_t T;
  const int32_t* lengths;
  uint16_t* summary;
  int64_t num_pages;
  int32_t* err;
  int per_block;  // tokens per block of threads
};

template <int KIND>
struct Piece;  // a lane's eight columns of a row
template <>
struct Piece<DSA_CACHE_BF16> {
  static constexpr int64_t RB = 2 * kD;
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) { v = *reinterpret_cast<const uint4*>(row + 16 * lane); }
  __device__ __forceinline__ void add(float (&s)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] += __uint_as_float(w[i] << 16);
      s[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Piece<DSA_CACHE_FP8_SCALED> {
  static constexpr int64_t RB = kD + 8;
  uint2 v;
  float scale;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    v = *reinterpret_cast<const uint2*>(row + 8 * lane);
    scale = *reinterpret_cast<const float*>(row + kD + 4 * (lane >> 4));
  }
  __device__ __forceinline__ void add(float (&s)[8]) const {
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
      s[2 * i] = fmaf(c.x, scale, s[2 * i]);
      s[2 * i + 1] = fmaf(c.y, scale, s[2 * i + 1]);
    }
  }
};

// Token t's (request, block); block -1 for padding.
__device__ __forceinline__ int2 block_of(const PoolParams& p, int64_t t) {
  const int pos = p.pos[t];
  return make_int2(p.req ? p.req[t] : (int)t, pos < 0 ? -1 : pos / p.page);
}

template <int KIND>
__global__ void __launch_bounds__(kPoolThreads) pool_kernel(const PoolParams p) {
  __shared__ float s_sum[kPoolWarps][kD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * p.per_block;
  // per_block <= 32: every warp finds the leaders for itself
  bool leads = false;
  int2 mine = make_int2(0, -1);
  if (lane < p.per_block && t0 + lane < p.T) {
    mine = block_of(p, t0 + lane);
    leads = mine.y >= 0;
    if (leads && t0 + lane > 0) {
      const int2 before = block_of(p, t0 + lane - 1);
      leads = before.x != mine.x || before.y != mine.y;
    }
  }
  for (uint32_t todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const int r = __shfl_sync(0xffffffffu, mine.x, src), b = __shfl_sync(0xffffffffu, mine.y, src);
    int64_t page = -1;
    int count = 0;
    if (r >= 0 && r < p.num_requests && b < p.max_pages) {
      const int64_t left = (int64_t)p.lengths[r] - (int64_t)b * p.page;
      count = (int)(left < p.page ? left : p.page);
      page = p.bt[r * p.bt_st + b];
    }
    if (page < 0 || page >= p.num_pages || count <= 0 || page * p.page + count > p.num_slots) {
      if (threadIdx.x == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
      continue;  // the same for every thread
    }
    const uint8_t* rows = p.cache + page * p.page * Piece<KIND>::RB;
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = warp; j < count; j += kAhead * kPoolWarps) {
      Piece<KIND> x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (j + i * kPoolWarps < count) x[i].load(rows + (int64_t)(j + i * kPoolWarps) * Piece<KIND>::RB, lane);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (j + i * kPoolWarps < count) x[i].add(s);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4*>(&s_sum[warp][8 * lane + 4 * i]) = make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
    __syncthreads();
    float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kPoolWarps; ++w) {
      const float2 u = *reinterpret_cast<const float2*>(&s_sum[w][2 * threadIdx.x]);
      v.x += u.x;
      v.y += u.y;
    }
    reinterpret_cast<uint32_t*>(p.summary + page * kD)[threadIdx.x] =
        f32x2_to_bf16x2(__fdiv_rn(v.x, (float)count), __fdiv_rn(v.y, (float)count));
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------ select --
struct SelectParams {
  const float* scores;
  int64_t score_st;
  int64_t width;
  int64_t T;
  const int32_t* bt;
  int64_t bt_st;
  int page, max_pages;
  int64_t num_requests;
  const int32_t *req, *lengths;
  int K, sink, recent;
  int32_t* blocks;
  int64_t blocks_st;
  int32_t* table;
  int64_t table_st;
  int32_t* len_out;
  int32_t* err;
};

// An unsigned key of the score's order, -0.0 as +0.0, below the one of the blocks always chosen.
__device__ __forceinline__ uint32_t key_of(float x) {
  uint32_t u = __float_as_uint(x);
  if (u == 0x80000000u) u = 0;
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return u == 0xFFFFFFFFu ? 0xFFFFFFFEu : u;
}

// Sum over the group of W warps that share a row (a whole block, or one warp).
template <int W>
__device__ __forceinline__ int group_sum(int v, int (&s)[2][32], int& turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  if (W == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) s[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < W ? s[turn][lane] : 0;
  turn ^= 1;  // the next sum writes elsewhere: one barrier per sum
  return __reduce_add_sync(0xffffffffu, v);
}

// W warps per row, N keys per thread and chunk of 32 W N blocks, thread g of the group holding blocks g, g + 32 W,
// ...: loads are whole lines, and a ballot is 32 neighbouring blocks. A row of one chunk (ONE) keeps its keys in
// registers and lists the chosen blocks in shared memory; a longer one reads them anew for every count.
template <int W, int N, bool ONE>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W, W == 1 ? 8 : 1) select_kernel(const SelectParams p) {
  constexpr int GT = 32 * W, CHUNK = GT * N, ROWS = W == 1 ? 4 : 1;
  __shared__ int s[2][32];
  __shared__ int s_last;
  __shared__ int s_list[ONE ? ROWS : 1][ONE ? CHUNK : 1];
  __shared__ uint32_t s_above[W == 1 ? 1 : N * W], s_equal[W == 1 ? 1 : N * W];    // bits of 32 blocks each
  __shared__ int s_above0[W == 1 ? 1 : N * W], s_equal0[W == 1 ? 1 : N * W];       // and how many before them
  int turn = 0;
  const int lane = threadIdx.x & 31, warp = W == 1 ? 0 : threadIdx.x >> 5;
  const int g = W == 1 ? lane : (int)threadIdx.x;  // thread of the group
  const int64_t t = W == 1 ? (int64_t)blockIdx.x * ROWS + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  if (t >= p.T) return;  // whole warps (W == 1), or nobody
  int* list = s_list[ONE && W == 1 ? threadIdx.x >> 5 : 0];
  const int len = max(p.lengths[t], 0);
  const int64_t r = p.req ? p.req[t] : t;
  int nb = len > 0 ? (len - 1) / p.page + 1 : 0;
  const int most = (int)(p.width < p.max_pages ? p.width : p.max_pages);
  bool bad = nb > most;
  const bool cut = bad;
  if (bad) nb = most;
  if (r < 0 || r >= p.num_requests) {
    bad = true;
    nb = 0;
  }
  if (bad && g == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
  const int n = nb;
  const int m = n < p.K ? n : p.K;
  const float* row = p.scores + t * p.score_st;
  const int32_t* pages = p.bt + (n ? r * p.bt_st : 0);
  const int end_sink = p.sink, from_recent = n - p.recent;
  uint32_t key[N];
  auto load = [&](int c0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int b = c0 + i * GT + g;
      key[i] = 0;  // below every score
      if (ONE && i * GT >= n) continue;
      if (b < n) key[i] = b < end_sink || b >= from_recent ? 0xFFFFFFFFu : key_of(row[b]);
    }
  };
  auto count = [&](uint32_t at_least) {
    int c = 0;
    for (int c0 = 0; c0 < n; c0 += CHUNK) {
      if (!ONE) load(c0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (ONE && i % 4 == 0 && i * GT >= n) break;  // (short rows: 8192 causal ones 18.9 us for 21.8 with these)
        c += key[i] >= at_least;
      }
      if (ONE) break;
    }
    return group_sum<W>(c, s, turn);
  };
  if (ONE) load(0);
  // The largest value that at least m keys reach is the m-th largest key, found from the top bit down; a value
  // that exactly m keys reach ends the search. Chosen: the keys above `u`, and the first `ties` of those equal.
  uint32_t u = 0;
  int ties = 0;
  if (m < n) {
    int c = 0;
    for (int bit = 31; bit >= 0 && c != m; --bit) {
      const uint32_t trial = u | (1u << bit);
      const int reach = count(trial);
      if (reach >= m) {
        u = trial;
        c = reach;
      }
    }
    if (c == m)
      --u;  // all that reach it
    else
      ties = m - (u == 0xFFFFFFFFu ? 0 : count(u + 1));
  }
  const bool all = m == n;
  if (W > 1) {
    if (threadIdx.x == 0) s_last = 0;
    __syncthreads();
  }
  bool last = false;
  auto choose = [&](int b, int at) {
    if (ONE) {
      list[at] = b;
    } else {
      if (p.blocks) p.blocks[t * p.blocks_st + at] = b;
      p.table[t * p.table_st + at] = pages[b];
    }
    last |= b == n - 1;
  };
  const uint32_t lower = (1u << lane) - 1;
  int above0 = 0, equal0 = 0;  // before this chunk (W == 1: before these 32)
  for (int c0 = 0; c0 < n; c0 += CHUNK) {
    if (!ONE) load(c0);
    uint32_t above[N], equal[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      above[i] = equal[i] = 0;
      if (ONE && i * GT >= n) continue;
      const bool in = c0 + i * GT + g < n;
      above[i] = __ballot_sync(0xffffffffu, in && (all || key[i] > u));
      equal[i] = __ballot_sync(0xffffffffu, in && !all && key[i] == u);
    }
    if (W > 1) {
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          s_above[i * W + warp] = above[i];
          s_equal[i * W + warp] = equal[i];
        }
      }
      __syncthreads();
      if (warp == 0) {  // the words in order, neighbouring ones in one lane
        constexpr int PER = (N * W + 31) / 32;
        int a = 0, e = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int word = lane * PER + k;
          if (word < N * W) {
            a += __popc(s_above[word]);
            e += __popc(s_equal[word]);
          }
        }
        int as = a, es = e;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, as, o), y = __shfl_up_sync(0xffffffffu, es, o);
          if (lane >= o) {
            as += x;
            es += y;
          }
        }
        as -= a;
        es -= e;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          const int word = lane * PER + k;
          if (word < N * W) {
            s_above0[word] = above0 + as;
            s_equal0[word] = equal0 + es;
            as += __popc(s_above[word]);
            es += __popc(s_equal[word]);
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (ONE && i * GT >= n) break;
      const int b = c0 + i * GT + g;
      int a, e;
      if (W == 1) {
        a = above0;
        e = equal0;
        above0 += __popc(above[i]);
        equal0 += __popc(equal[i]);
      } else {
        a = s_above0[i * W + warp];
        e = s_equal0[i * W + warp];
      }
      a += __popc(above[i] & lower);
      e += __popc(equal[i] & lower);
      const bool up = (above[i] >> lane) & 1, tie = (equal[i] >> lane) & 1;
      if (up || (tie && e < ties)) choose(b, a + (e < ties ? e : ties));
    }
    if (W > 1 && !ONE) {
      above0 = s_above0[N * W - 1] + __popc(s_above[N * W - 1]);
      equal0 = s_equal0[N * W - 1] + __popc(s_equal[N * W - 1]);
      __syncthreads();
    }
    if (ONE) break;
  }
  if (W == 1) {
    last = __any_sync(0xffffffffu, last);
    __syncwarp();
  } else {
    if (last) s_last = 1;
    __syncthreads();
    last = s_last != 0;
  }
  for (int i = (ONE ? 0 : m) + g; i < p.K; i += GT) {
    const int b = ONE && i < m ? list[i] : -1;
    if (p.blocks) p.blocks[t * p.blocks_st + i] = b;
    p.table[t * p.table_st + i] = b < 0 ? -1 : pages[b];
  }
  if (g == 0) {
    int64_t out = (int64_t)m * p.page;
    if (last && !cut) out -= (int64_t)nb * p.page - len;
    p.len_out[t] = (int)(out < INT_MAX ? out : INT_MAX);
  }
}

template <int W, int N, bool ONE>
cudaError_t launch_select(const SelectParams& p, cudaStream_t s) {
  const int threads = W == 1 ? 128 : 32 * W, rows = W == 1 ? 4 : 1;
  select_kernel<W, N, ONE><<<(unsigned)((p.T + rows - 1) / rows), threads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace block
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_block_pool(const void* cache, dsa_cache_kind_t kind, int64_t num_slots,
                                       const int32_t* block_table, int64_t bt_stride, int page_size, int max_pages,
                                       int64_t num_requests, const int32_t* positions, const int32_t* req_of_token,
                                       int64_t T, const int32_t* lengths, void* summary, int64_t num_pages,
                                       int32_t* error_word, void* stream) {
  if (kind != DSA_CACHE_BF16 && kind != DSA_CACHE_FP8_SCALED) return DSA_ERR_INVALID_ARGUMENT;
  if (T < 0 || page_size < 1 || max_pages < 0 || bt_stride < max_pages || num_slots < 0 || num_pages < 0)
    return DSA_ERR_INVALID_ARGUMENT;
  if (T > (1 << 24) || num_slots > INT_MAX) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!cache || !block_table || !positions || !lengths || !summary || num_requests < 1 || (!req_of_token && T > num_requests))
    return DSA_ERR_INVALID_ARGUMENT;
  if (!aligned(cache, 16) || !aligned(summary, 16) || !aligned(block_table, 4) || !aligned(positions, 4) ||
      !aligned(req_of_token, 4) || !aligned(lengths, 4) || !aligned(error_word, 4))
    return DSA_ERR_INVALID_ARGUMENT;
  DeviceInfo dev;
  const dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  block::PoolParams p{};
  p.cache = static_cast<const uint8_t*>(cache);
  p.num_slots = num_slots;
  p.bt = block_table;
  p.bt_st = bt_stride;
  p.page = page_size;
  p.max_pages = max_pages;
  p.num_requests = num_requests;
  p.pos = positions;
  p.req = req_of_token;
  p.T = T;
  p.lengths = lengths;
  p.summary = static_cast<uint16_t*>(summary);
  p.num_pages = num_pages;
  p.err = error_word;
  // A decode step's tokens all lead a block: one each, spread over the device. Of a prefill's one in page_size
  // does, and blocks of threads that find none cost their start: eight per SM, of up to 32 tokens. (101739 tokens in
  // pages of 64: 13.1 us, 19.2 with 8 tokens each; 8192 that all lead: 20.4, 61 with 32 each; replays of one call,
  // rows in L2.)
  const int64_t share = T / (8 * dev.sm_count);
  p.per_block = (int)(share < 1 ? 1 : share > 32 ? 32 : share);
  const unsigned grid = (unsigned)((T + p.per_block - 1) / p.per_block);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (kind == DSA_CACHE_BF16)
    block::pool_kernel<DSA_CACHE_BF16><<<grid, block::kPoolThreads, 0, s>>>(p);
  else
    block::pool_kernel<DSA_CACHE_FP8_SCALED><<<grid, block::kPoolThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}

extern "C" dsa_status_t dsa_block_select(const float* scores, int64_t score_stride, int64_t width, int64_t T,
                                         const int32_t* block_table, int64_t bt_stride, int page_size, int max_pages,
                                         int64_t num_requests, const int32_t* req_of_token, const int32_t* lengths, int K,
                                         int sink, int recent, int32_t* blocks, int64_t blocks_stride, int32_t* table,
                                         int64_t table_stride, int32_t* lengths_out, int32_t* error_word, void* stream) {
  if (T < 0 || page_size < 1 || max_pages < 0 || bt_stride < max_pages || width < 1 || score_stride < width)
    return DSA_ERR_INVALID_ARGUMENT;
  if (K < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > K) return DSA_ERR_INVALID_ARGUMENT;
  if (T > (1 << 24) || width > (1 << 24) || K > 16384) return DSA_ERR_UNSUPPORTED;
  if ((blocks && blocks_stride < K) || table_stride < K) return DSA_ERR_INVALID_ARGUMENT;
  if (T == 0) return DSA_OK;
  if (!scores || !block_table || !lengths || !table || !lengths_out || num_requests < 1 || (!req_of_token && T > num_requests))
    return DSA_ERR_INVALID_ARGUMENT;
  for (const void* q : {(const void*)scores, (const void*)block_table, (const void*)req_of_token, (const void*)lengths,
                        (const void*)blocks, (const void*)table, (const void*)lengths_out, (const void*)error_word})
    if (!aligned(q, 4)) return DSA_ERR_INVALID_ARGUMENT;
  DeviceInfo dev;
  const dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  block::SelectParams p{};
  p.scores = scores;
  p.score_st = score_stride;
  p.width = width;
  p.T = T;
  p.bt = block_table;
  p.bt_st = bt_stride;
  p.page = page_size;
  p.max_pages = max_pages;
  p.num_requests = num_requests;
  p.req = req_of_token;
  p.lengths = lengths;
  p.K = K;
  p.sink = sink;
  p.recent = recent;
  p.blocks = blocks;
  p.blocks_st = blocks_stride;
  p.table = table;
  p.table_st = table_stride;
  p.len_out = lengths_out;
  p.err = error_word;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t most = width < max_pages ? width : max_pages;
  cudaError_t e;
  // a warp per row up to 544 blocks, then as few warps as hold the keys (tables are a little wider than a
  // round number of blocks as a rule). The table's width decides, since the lengths are on the device: rows much shorter
  // than it pay for it (8192 rows of up to 512 blocks: 21 us in a table of 513 columns, 71 in 2052, 288 in 8208, 641 in
  // 16416). A table sliced to the longest request's pages avoids that.
  if (most <= 160)
    e = block::launch_select<1, 5, true>(p, s);
  else if (most <= 288)
    e = block::launch_select<1, 9, true>(p, s);
  else if (most <= 544)
    e = block::launch_select<1, 17, true>(p, s);
  else if (most <= 1152)
    e = block::launch_select<4, 9, true>(p, s);
  else if (most <= 2304)
    e = block::launch_select<8, 9, true>(p, s);
  else if (most <= 4608)
    e = block::launch_select<16, 9, true>(p, s);
  else if (most <= 8704)
    e = block::launch_select<16, 17, true>(p, s);
  else
    e = block::launch_select<32, 8, false>(p, s);
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
