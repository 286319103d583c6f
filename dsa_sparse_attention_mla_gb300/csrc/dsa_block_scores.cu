// dsa_block_scores.cu - a cheap score of each block (page) for each token:
//   scores[t, b] = sum_h w[t,h] * max(0, sm_scale * q[t,h] . summary[page of b]).
//
// A warp per block of a token: its lanes hold the summary row, eight columns each, and go through the
// heads.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "dsa_host.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace scores {

constexpr int kD = 256;
constexpr int kMaxHeads = 128;
constexpr int kThreads = 256;

struct Params {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int64_t T;
  int H;
  const uint16_t* summary;
  int64_t num_pages;
  const int32_t* bt;
  int64_t bt_st;
  int page, max_pages;
  int64_t num_requests;
  const int32_t *req, *lengths;
  float scale;
  const float* w;
  float* out;
  int64_t out_st, width;
  int32_t* err;
};

__device__ __forceinline__ void widen(const uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// max(x, 0) that passes NaN on
__device__ __forceinline__ float relu(float x) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
  return r;
}

__global__ void __launch_bounds__(kThreads) scores_kernel(const Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int64_t r = p.req ? p.req[t] : t;
  const int64_t most = p.width < p.max_pages ? p.width : p.max_pages;
  int64_t n = ((int64_t)max(p.lengths[t], 0) + p.page - 1) / p.page;
  bool bad = n > most;
  if (bad) n = most;
  if (r < 0 || r >= p.num_requests) {
    bad = true;
    n = 0;
  }
  if (bad && threadIdx.x == 0 && blockIdx.y == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
  for (int64_t b = (int64_t)blockIdx.y * (kThreads / 32) + warp; b < n; b += (int64_t)gridDim.y * (kThreads / 32)) {
    const int64_t page = p.bt[r * p.bt_st + b];
    float total = -INFINITY;
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
    } else {
      float k[8];
      widen(*reinterpret_cast<const uint4*>(p.summary + page * kD + 8 * lane), k);
      total = 0.0f;
      for (int h = 0; h < p.H; ++h) {
        float x[8], dot = 0.0f;
        widen(*reinterpret_cast<const uint4*>(p.q + t * p.q_st + h * p.q_sh + 8 * lane), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(x[i], k[i], dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        total = fmaf(p.w ? p.w[t * p.H + h] : 1.0f, relu(dot * p.scale), total);
      }
    }
    if (lane == 0) p.out[t * p.out_st + b] = total;
  }
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
  const dsa_status_t st = current_device(&dev);
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
  p.max_pages = max_pages;
  p.num_requests = num_requests;
  p.req = req_of_token;
  p.lengths = lengths;
  p.scale = sm_scale;
  p.w = weights;
  p.out = scores_out;
  p.out_st = score_stride;
  p.width = width;
  p.err = error_word;
  const int64_t most = width < max_pages ? width : max_pages;
  const int64_t y = (most + 31) / 32;
  scores::scores_kernel<<<dim3((unsigned)T, (unsigned)(y < 1 ? 1 : y > 1024 ? 1024 : y)), scores::kThreads, 0,
                          static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
