// dsa_paged.cu - dense attention over the paged latent cache, one new token per request, and the
// attention weight each cached position receives (dsa_paged_attn, dsa_paged_attn_mass).
//
// For token t of request r, head h and position j of the token's range [start, end):
//   u_hj = sm_scale q_h . k_j, capped by cap * tanh(u / cap), minus slope_h |qpos - kpos_j|
//   out_h = sum_j softmax_j(u_h) k_j,  lse_h = log sum_j exp(u_hj)
//   mass_out[r, j] = mass[r, j] + sum_h exp(u_hj - lse_h)
// The latent row k_j is key and value of every head, so a position costs 264 (FP8) or 512 (bf16)
// bytes and 4 * 256 * H operations.
//
// One warp takes one position at a time, lane l columns 8l .. 8l + 7; eight warps of a CTA share a
// token and head (attention, online softmax per warp, joined at the end) or a token (mass).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "dsa_host.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace paged {

constexpr int kD = 256;
constexpr int kMaxHeads = 128;

struct Params {
  const uint16_t* q;
  int64_t q_st, q_sh;
  int64_t T;
  int H;
  const uint8_t* cache;
  int64_t num_slots;
  const int32_t* bt;
  int64_t bt_stride;
  int page_size;
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
  const float* mass;
  int64_t mass_stride;
  float* mass_out;
  int64_t mass_out_stride;
  int32_t* err;
};

__device__ __forceinline__ void set_err(int32_t* err, int bits) {
  if (err) atomicOr(err, bits);
}

// The range of token t, clipped to the addressable positions; false when there is nothing to read.
__device__ __forceinline__ bool token_range(const Params& p, int64_t t, int64_t* req, int64_t* a, int64_t* b) {
  *req = p.req ? p.req[t] : t;
  const int64_t s = p.starts ? p.starts[t] : 0, e = p.lengths[t];
  *a = s < 0 ? 0 : s;
  *b = e;
  if (*a >= *b) return false;
  if (*req < 0 || *req >= p.num_requests) {
    set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
    return false;
  }
  if (*b > p.pos_limit) {
    set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
    *b = p.pos_limit;
  }
  return *a < *b;
}

__device__ __forceinline__ int64_t slot_of(const Params& p, int64_t req, int64_t j) {
  if (!p.bt) return j;
  const int64_t page = p.bt[req * p.bt_stride + j / p.page_size];
  if (page < 0) return -1;
  const int64_t s = page * p.page_size + j % p.page_size;
  return s < p.num_slots ? s : -1;
}

template <int KIND>
__device__ __forceinline__ void load_row(const Params& p, int64_t slot, int lane, float (&k)[8]) {
  if constexpr (KIND == DSA_CACHE_BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p.cache + slot * 512 + 16 * lane);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[2 * i] = __uint_as_float(w[i] << 16);
      k[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint8_t* r = p.cache + slot * 264;
    const uint2 c = *reinterpret_cast<const uint2*>(r + 8 * lane);
    const float sc = *reinterpret_cast<const float*>(r + 256 + 4 * (lane >> 4));
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] & 0xFFFFu)));
      const float2 b = f16x2_to_f32x2(e4m3x2_to_f16x2((uint16_t)(w[i] >> 16)));
      k[4 * i] = a.x * sc;
      k[4 * i + 1] = a.y * sc;
      k[4 * i + 2] = b.x * sc;
      k[4 * i + 3] = b.y * sc;
    }
  }
}

__device__ __forceinline__ void load_q(const Params& p, int64_t t, int h, int lane, float (&q)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p.q + t * p.q_st + h * p.q_sh + 8 * lane);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[2 * i] = __uint_as_float(w[i] << 16);
    q[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// score in natural units from the dot product
__device__ __forceinline__ float modify(const Params& p, float dot, int h, float dist) {
  float u = dot * p.sm_scale;
  if (p.cap > 0.0f) u = p.cap * tanhf(u / p.cap);
  if (p.slopes) u -= p.slopes[h] * dist;
  return u;
}

__device__ __forceinline__ float warp_dot(const float (&a)[8], const float (&b)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ float distance(const Params& p, int64_t t, int64_t req, int64_t j) {
  if (!p.slopes) return 0.0f;
  const int64_t qp = p.qpos ? p.qpos[t] : (int64_t)p.lengths[t] - 1;
  const int64_t kp = p.kpos ? p.kpos[req * p.kp_stride + j] : j;
  return fabsf((float)(qp - kp));
}

template <int KIND>
__global__ void __launch_bounds__(256) attn_kernel(const __grid_constant__ Params p) {
  __shared__ float sm_m[8], sm_l[8], sm_o[8][kD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y;
  int64_t req, a, b;
  const bool any = token_range(p, t, &req, &a, &b);
  float q[8], o[8], m = -INFINITY, l = 0.0f;
  load_q(p, t, h, lane, q);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.0f;
  if (any) {
    for (int64_t j = a + warp; j < b; j += 8) {
      const int64_t slot = slot_of(p, req, j);
      if (slot < 0) {
        if (lane == 0) set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
        continue;
      }
      float k[8];
      load_row<KIND>(p, slot, lane, k);
      const float u = modify(p, warp_dot(q, k), h, distance(p, t, req, j));
      const float mn = fmaxf(m, u);
      const float f = m == mn ? 1.0f : __expf(m - mn), e = __expf(u - mn);
      l = l * f + e;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * f + e * k[i];
      m = mn;
    }
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sm_o[warp][8 * lane + i] = o[i];
  __syncthreads();
  float M = -INFINITY, L = 0.0f, acc = 0.0f;
  for (int w = 0; w < 8; ++w) M = fmaxf(M, sm_m[w]);
  for (int w = 0; w < 8; ++w) {
    if (sm_l[w] == 0.0f) continue;  // a warp that read nothing
    const float f = __expf(sm_m[w] - M);
    L += f * sm_l[w];
    acc += f * sm_o[w][threadIdx.x];
  }
  const float r = L == 0.0f ? 0.0f : acc / L;
  __nv_bfloat16 bo = __float2bfloat16_rn(r);
  p.out[t * p.out_st + h * p.out_sh + threadIdx.x] = *reinterpret_cast<uint16_t*>(&bo);
  if (p.lse && threadIdx.x == 0) p.lse[t * p.H + h] = L == 0.0f ? -INFINITY : M + logf(L);
}

template <int KIND>
__global__ void __launch_bounds__(256) mass_kernel(const __grid_constant__ Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  int64_t req, a, b;
  if (!token_range(p, t, &req, &a, &b)) return;
  if (p.req) {
    bool bad = false;
    for (int64_t i = threadIdx.x; i < t; i += 256) bad |= p.req[i] >= req;
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) set_err(p.err, DSA_DEVERR_REQUEST_ORDER);
      return;
    }
  }
  for (int64_t j = a + warp + 8 * blockIdx.y; j < b; j += 8 * gridDim.y) {
    const int64_t slot = slot_of(p, req, j);
    float w = 0.0f;
    if (slot >= 0) {
      float k[8], q[8];
      load_row<KIND>(p, slot, lane, k);
      const float d = distance(p, t, req, j);
      for (int h = 0; h < p.H; ++h) {
        load_q(p, t, h, lane, q);
        w += __expf(modify(p, warp_dot(q, k), h, d) - p.lse[t * p.H + h]);
      }
    } else if (lane == 0) {
      set_err(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
    }
    if (lane == 0) p.mass_out[req * p.mass_out_stride + j] = p.mass[req * p.mass_stride + j] + w;
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
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.num_slots = a->num_slots;
  p.bt = a->block_table;
  p.bt_stride = a->bt_stride;
  p.page_size = a->block_table ? a->page_size : 1;
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
  p.err = a->error_word;
  return p;
}

}  // namespace paged
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_paged_attn_workspace_size(const dsa_paged_args_t* a, size_t* bytes) {
  if (!a || !bytes || a->T < 0 || a->H < 1) return DSA_ERR_INVALID_ARGUMENT;
  *bytes = 0;
  return DSA_OK;
}

extern "C" dsa_status_t dsa_paged_attn(const dsa_paged_args_t* a, void* stream) {
  dsa_status_t st = paged::check(a, false);
  if (st != DSA_OK || a->T == 0) return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != DSA_OK) return st;
  const paged::Params p = paged::make_params(a);
  const dim3 grid((unsigned)a->T, (unsigned)a->H);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->kind == DSA_CACHE_BF16) paged::attn_kernel<DSA_CACHE_BF16><<<grid, 256, 0, s>>>(p);
  else paged::attn_kernel<DSA_CACHE_FP8_SCALED><<<grid, 256, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
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
  p.mass_stride = mass_stride;
  p.mass_out = mass_out;
  p.mass_out_stride = mass_out_stride;
  const dim3 grid((unsigned)a->T, 64);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->kind == DSA_CACHE_BF16) paged::mass_kernel<DSA_CACHE_BF16><<<grid, 256, 0, s>>>(p);
  else paged::mass_kernel<DSA_CACHE_FP8_SCALED><<<grid, 256, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
