// dsa_qk.cu - the norm of every query head and of the latent key, the rotation of their RoPE columns
// and the key's cache row, in one pass.
//
// y_d = x_d * rsqrt(mean x^2 + eps) * w_d over the first n columns, then the last d_rope turn by the
// token's angles. One warp per row holds it in registers: lane l the columns 8 l .. 8 l + 7 of each 256
// of the NoPE part and the pair 2 l, 2 l + 1 of the RoPE part, whose partner columns come from the lane
// itself (interleaved) or from lane l ^ 16 (halves). A row is thus read and written once; bytes bound
// it at large sizes, the launch at small ones.
//
// Everything is in fp32 until the one rounding at the end. The packed row takes the unrounded fp32
// values: a bf16 row in between would round twice.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>

#include "dsa_host.h"
#include "dsa_ptx.cuh"

namespace dsa {
namespace qk {

constexpr int kThreads = 128;
// Per SM: every row in flight counts (8192 x 64 rows of 1152 bytes: 200 us with 16 and 215 with 12 when it was chosen; now
// 187 in a graph, 6.6 TB/s)
constexpr int kBlocks = 16;
constexpr int kWarps = kThreads / 32;

struct Params {
  int64_t T;
  uint32_t rows;  // T * H query rows, then T key rows
  uint32_t q_rows;
  uint32_t H;
  const uint16_t* q;
  int64_t q_st, q_sh;
  uint16_t* qo;
  int64_t qo_st, qo_sh;
  int q_norm;
  const uint16_t* q_w;
  const uint16_t* k;
  int64_t k_st;
  int k_norm;
  const uint16_t* k_w;
  uint8_t* cache;
  int64_t num_slots;
  const int64_t* loc;
  float eps;
  const int32_t* pos;
  const float* cs;
  int64_t cs_st, num_pos;
  int inter;
  int32_t* err;
};

__device__ __forceinline__ float lo_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ void widen(const uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo_bf16(w[i]);
    x[2 * i + 1] = hi_bf16(w[i]);
  }
}
__device__ __forceinline__ uint4 narrow(const float* x) {
  return make_uint4(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(x[4], x[5]),
                    f32x2_to_bf16x2(x[6], x[7]));
}

template <int KIND, int D_NOPE, int D_ROPE>
__global__ void __launch_bounds__(kThreads, kBlocks) qk_kernel(const Params p) {
  constexpr int NV = D_NOPE / 256;  // 16-byte pieces per lane
  constexpr int D = D_NOPE + D_ROPE;
  constexpr int TILES = D_NOPE / 128;
  constexpr int64_t RB = KIND == DSA_CACHE_BF16 ? 2 * D : D_NOPE + 4 * TILES + 2 * D_ROPE;
  const int lane = threadIdx.x & 31;
  const uint32_t row = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  const bool is_q = row < p.q_rows;
  const uint32_t t = is_q ? row / p.H : row - p.q_rows;
  const uint32_t h = is_q ? row - t * p.H : 0;
  int64_t at = 0;
  if (p.pos) {
    at = p.pos[t];
    if (at < 0) return;
    if (p.cs && at >= p.num_pos) {
      if (lane == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INDEX_OUT_OF_RANGE);
      return;
    }
  }
  int64_t slot = 0;
  if (!is_q) {
    slot = p.loc ? p.loc[t] : t;
    if (slot < 0) return;
    if (slot >= p.num_slots) {
      if (lane == 0 && p.err) atomicOr(p.err, DSA_DEVERR_SLOT_OUT_OF_RANGE);
      return;
    }
  }
  const uint16_t* src = is_q ? p.q + t * p.q_st + h * p.q_sh : p.k + t * p.k_st;
  // every load of the row at once; it stays in bf16 until its pieces are worked on, one after another
  uint4 raw[NV];
  uint32_t raw_tail = 0;
  float2 cos = make_float2(1.0f, 1.0f), sin = make_float2(0.0f, 0.0f);  // of the lane's two RoPE columns
#pragma unroll
  for (int v = 0; v < NV; ++v) raw[v] = *reinterpret_cast<const uint4*>(src + 256 * v + 8 * lane);
  if (D_ROPE > 0) {
    raw_tail = *reinterpret_cast<const uint32_t*>(src + D_NOPE + 2 * lane);
    if (p.cs) {
      const float* cs = p.cs + at * p.cs_st;
      if (p.inter) {
        cos.x = cs[lane];
        sin.x = cs[D_ROPE / 2 + lane];
      } else {
        const int i = 2 * (lane & 15);
        cos = make_float2(cs[i], cs[i + 1]);
        sin = make_float2(cs[D_ROPE / 2 + i], cs[D_ROPE / 2 + i + 1]);
      }
    }
  }
  float a = lo_bf16(raw_tail), b = hi_bf16(raw_tail);
  const int n = is_q ? p.q_norm : p.k_norm;
  const uint16_t* wt = nullptr;
  float r = 1.0f;
  if (n > 0) {
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[8];
      widen(raw[v], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    }
    if (D_ROPE > 0 && n == D) ss = fmaf(a, a, fmaf(b, b, ss));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    r = rsqrtf(ss / (float)n + p.eps);
    wt = is_q ? p.q_w : p.k_w;
    if (D_ROPE > 0 && n == D) {
      a *= r;
      b *= r;
      if (wt) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(wt + D_NOPE + 2 * lane);
        a *= lo_bf16(w);
        b *= hi_bf16(w);
      }
    }
  }
  if (D_ROPE > 0 && p.cs) {
    if (p.inter) {
      const float u = a * cos.x - b * sin.x;
      b = b * cos.x + a * sin.x;
      a = u;
    } else {
      // lanes 0-15 hold the first halves of the pairs, lanes 16-31 the second ones
      const float pa = __shfl_xor_sync(0xffffffffu, a, 16), pb = __shfl_xor_sync(0xffffffffu, b, 16);
      const float sign = lane < 16 ? -1.0f : 1.0f;
      a = a * cos.x + sign * (pa * sin.x);
      b = b * cos.y + sign * (pb * sin.y);
    }
  }
  const bool packed = !is_q && KIND == DSA_CACHE_FP8_SCALED;
  uint16_t* dst = is_q ? p.qo + t * p.qo_st + h * p.qo_sh : reinterpret_cast<uint16_t*>(p.cache + slot * RB);
  uint8_t* row_out = p.cache + slot * RB;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float x[8];
    widen(raw[v], x);
    if (wt) {
      float w[8];
      widen(*reinterpret_cast<const uint4*>(wt + 256 * v + 8 * lane), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= r;
    }
    if (!packed) {
      *reinterpret_cast<uint4*>(dst + 256 * v + 8 * lane) = narrow(x);
      continue;
    }
    // a 128-column tile is half a warp's 8-column pieces
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float scale = __fdiv_rn(amax, 448.0f);
    uint32_t code[2] = {0, 0};
    if (scale > 0.0f) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        code[i] = (uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)) |
                  ((uint32_t)f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)) << 16);
    } else {
      // values below 448 * 2^-150, which count as zeros (the unrounded row can hold them), or NaN, which the maximum
      // passes over: a norm makes a whole row of it, and zeros would hide that
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x[i] != x[i]) code[i >> 2] |= 0x7Fu << (8 * (i & 3));
    }
    *reinterpret_cast<uint2*>(row_out + 256 * v + 8 * lane) = make_uint2(code[0], code[1]);
    if ((lane & 15) == 0) *reinterpret_cast<float*>(row_out + D_NOPE + 4 * (2 * v + (lane >> 4))) = scale;
  }
  if (D_ROPE > 0) {
    const uint32_t tail = f32x2_to_bf16x2(a, b);
    if (packed)
      *reinterpret_cast<uint32_t*>(row_out + D_NOPE + 4 * TILES + 4 * lane) = tail;
    else
      *reinterpret_cast<uint32_t*>(dst + D_NOPE + 2 * lane) = tail;
  }
}

template <int KIND, int D_NOPE, int D_ROPE>
cudaError_t launch(const Params& p, cudaStream_t s) {
  qk_kernel<KIND, D_NOPE, D_ROPE><<<(p.rows + kWarps - 1) / kWarps, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace qk
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status_t dsa_qk_norm_rope(const dsa_qk_args_t* a, void* stream) {
  if (!a || a->T < 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!((a->d_nope == 256 && a->d_rope == 0) || (a->d_nope == 512 && a->d_rope == 64)) || a->T > (1 << 24))
    return DSA_ERR_UNSUPPORTED;
  const int D = a->d_nope + a->d_rope;
  if (!a->q && !a->k && a->T > 0) return DSA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(a->eps) || !(a->eps > 0.0f)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->q) {
    if (a->H < 1) return DSA_ERR_INVALID_ARGUMENT;
    if (a->H > 128) return DSA_ERR_UNSUPPORTED;
    if (!a->q_out || !aligned(a->q, 16) || !aligned(a->q_out, 16) || !aligned(a->q_weight, 16) || a->q_stride_t < 0 ||
        a->q_stride_h < 0 || a->q_stride_t % 8 || a->q_stride_h % 8 || a->q_out_stride_t % 8 || a->q_out_stride_h % 8)
      return DSA_ERR_INVALID_ARGUMENT;
    // rows of the result that overlap would be written twice
    if ((a->H > 1 && a->q_out_stride_h < D) || (a->T > 1 && a->q_out_stride_t < D) ||
        (a->H > 1 && a->T > 1 && a->q_out_stride_t < (a->H - 1) * a->q_out_stride_h + D &&
         a->q_out_stride_h < (a->T - 1) * a->q_out_stride_t + D))
      return DSA_ERR_INVALID_ARGUMENT;
    if (a->q_out == a->q && ((a->T > 1 && a->q_out_stride_t != a->q_stride_t) || (a->H > 1 && a->q_out_stride_h != a->q_stride_h)))
      return DSA_ERR_INVALID_ARGUMENT;
    if (a->q_norm != 0 && a->q_norm != a->d_nope && a->q_norm != D) return DSA_ERR_INVALID_ARGUMENT;
  }
  if (a->k) {
    if (a->kind != DSA_CACHE_BF16 && a->kind != DSA_CACHE_FP8_SCALED) return DSA_ERR_INVALID_ARGUMENT;
    if (!a->cache || a->num_slots < 0 || !aligned(a->k, 16) || !aligned(a->cache, 16) || !aligned(a->k_weight, 16) ||
        !aligned(a->out_loc, 8) || a->k_stride_t < 0 || a->k_stride_t % 8)
      return DSA_ERR_INVALID_ARGUMENT;
    if (a->k_norm != 0 && a->k_norm != a->d_nope && a->k_norm != D) return DSA_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(a->positions, 4) || !aligned(a->error_word, 4)) return DSA_ERR_INVALID_ARGUMENT;
  if (a->cos_sin && (a->d_rope == 0 || (!a->positions && a->T > 0) || !aligned(a->cos_sin, 4) || a->cs_stride < a->d_rope || a->num_positions < 0))
    return DSA_ERR_INVALID_ARGUMENT;
  if (a->T == 0) return DSA_OK;
  DeviceInfo dev;
  const dsa_status_t st = current_device(&dev);
  if (st != DSA_OK) return st;
  qk::Params p{};
  p.T = a->T;
  p.H = a->q ? a->H : 1;
  p.q_rows = a->q ? (uint32_t)(a->T * a->H) : 0;
  p.rows = p.q_rows + (a->k ? (uint32_t)a->T : 0);
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_st = a->q_stride_t;
  p.q_sh = a->q_stride_h;
  p.qo = static_cast<uint16_t*>(a->q_out);
  p.qo_st = a->q_out_stride_t;
  p.qo_sh = a->q_out_stride_h;
  p.q_norm = a->q_norm;
  p.q_w = static_cast<const uint16_t*>(a->q_weight);
  p.k = static_cast<const uint16_t*>(a->k);
  p.k_st = a->k_stride_t;
  p.k_norm = a->k_norm;
  p.k_w = static_cast<const uint16_t*>(a->k_weight);
  p.cache = static_cast<uint8_t*>(a->cache);
  p.num_slots = a->num_slots;
  p.loc = a->out_loc;
  p.eps = a->eps;
  p.pos = a->positions;
  p.cs = a->cos_sin;
  p.cs_st = a->cs_stride;
  p.num_pos = a->num_positions;
  p.inter = a->interleaved;
  p.err = a->error_word;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool packed = a->k && a->kind == DSA_CACHE_FP8_SCALED;
  cudaError_t e;
  if (a->d_nope == 256)
    e = packed ? qk::launch<DSA_CACHE_FP8_SCALED, 256, 0>(p, s) : qk::launch<DSA_CACHE_BF16, 256, 0>(p, s);
  else
    e = packed ? qk::launch<DSA_CACHE_FP8_SCALED, 512, 64>(p, s) : qk::launch<DSA_CACHE_BF16, 512, 64>(p, s);
  return e == cudaSuccess ? DSA_OK : cuda_fail(e);
}
