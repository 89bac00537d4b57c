// Queries and keys before attention, for sm_103a: the RMS norm of each head and the
// rotation by position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;   (a, b) -> (a cos - b sin, b cos + a sin)
//
// for the pairs (a, b) of a head's first R values, pair i by the angle
// position * f_i on the position axis the pair belongs to (one axis for text;
// time, height and width for images and video).
//
// HBM-bound: each value is read once and written once, 8 flops between, so the
// kernel is 16-byte loads, a reduction over the lanes that hold a head, and
// 16-byte stores.
//  * One CTA takes one token (or a part of its heads, where there are few tokens):
//    the R/2 sines and cosines are computed once in shared memory and used by all
//    of its heads.
//  * The angle is computed in whole numbers: f is given in units of 2^-64 turns, so
//    position * f wraps modulo one turn by itself, exactly, however far the
//    position; its top 32 bits then go to sincospif.  A product in fp32 would be off
//    by whole radians at position 10^6 and beyond.
//  * D/8 lanes hold a row, 8 values each, so a pair's two halves (R/2 apart) are in
//    two lanes: one shuffle exchanges them.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_rope = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_rope, 0, code); }

constexpr int kThreads = 256;
constexpr int kMaxAxes = 8;

struct RopeParams {
  const __half* q;
  const __half* k;
  const __half* q_weight;
  const __half* k_weight;
  const int32_t* positions;
  const int64_t* frequencies;
  const int32_t* pair_axis;
  __half* q_out;
  __half* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  int num_axes, rotary_dim, num_tokens, num_heads, num_kv_heads;
  int rows_per_cta;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& raw, float (&x)[8]) {
  const __half2* h2 = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(h2[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}

// grid (tokens, parts of a token's query and key heads)
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 8;                        // lanes per row
  constexpr int RPP = kThreads / LPR;               // rows per pass
  constexpr int U = 3;                              // passes whose loads are in flight together
  __shared__ float2 turn[D / 2];                    // (cos, sin) of each pair
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int t = blockIdx.x;
  const int tid = threadIdx.x, c = tid % LPR;
  const int total = p.num_heads + p.num_kv_heads;
  const int begin = blockIdx.y * p.rows_per_cta, end = min(total, begin + p.rows_per_cta);
  auto load = [&](int row) {
    return row >= end ? make_uint4(0, 0, 0, 0)
           : row < p.num_heads
               ? *reinterpret_cast<const uint4*>(p.q + t * p.q_stride + row * D + c * 8)
               : *reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (row - p.num_heads) * D + c * 8);
  };
  const int first = begin + tid / LPR;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load(first + u * RPP);
  if (tid < p.rotary_dim / 2) {
    const int axis = p.pair_axis == nullptr ? 0 : p.pair_axis[tid];
    float cs = 1.f, sn = 0.f;
    if (axis >= 0 && axis < p.num_axes) {
      const int64_t pos = p.positions[static_cast<int64_t>(axis) * p.num_tokens + t];
      // turns modulo one in [-1/2, 1/2), as a signed 64-bit fraction; its top 32 bits are 2^-32 turns
      const uint64_t turns = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.frequencies[tid]);
      const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
      sincospif(half_turns, &sn, &cs);
    } else if (blockIdx.y == 0) {
      record_error(PKV_DEV_BAD_AXIS);
    }
    turn[tid] = make_float2(cs, sn);
  }
  float wq[8], wk[8];
  const bool norm_q = p.q_weight != nullptr, norm_k = p.k_weight != nullptr;
  unpack8(norm_q ? *reinterpret_cast<const uint4*>(p.q_weight + c * 8) : make_uint4(0, 0, 0, 0), wq);
  unpack8(norm_k ? *reinterpret_cast<const uint4*>(p.k_weight + c * 8) : make_uint4(0, 0, 0, 0), wk);
  __syncthreads();
  // this lane's turns: of its 8 values' pairs (half layout), or of its 4 pairs (interleaved)
  constexpr int NT = INTERLEAVED ? 4 : 8;
  const int lanes = p.rotary_dim / 8;               // lanes that hold turned values
  const bool turned = c < lanes;
  const bool upper = c >= lanes / 2;                // half layout: this lane holds the pairs' second values
  float2 cs[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int pair = INTERLEAVED ? c * 4 + i : (upper ? c - lanes / 2 : c) * 8 + i;
    cs[i] = turned ? turn[pair] : make_float2(1.f, 0.f);
  }
  // half layout: the lane that holds the other values of this lane's pairs
  const int lane = tid & 31;
  const int other = !turned ? lane : upper ? lane - lanes / 2 : lane + lanes / 2;

  // whole passes, so that every lane of a warp takes part in the shuffles
  for (int row = first; row - tid / LPR < end; row += U * RPP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      const bool is_q = r < p.num_heads;
      float x[8];
      unpack8(raw[u], x);
      raw[u] = load(r + U * RPP);
      if (is_q ? norm_q : norm_k) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        const unsigned row_lanes = (LPR == 16 ? 0xffffu : 0xffu) << (lane & ~(LPR - 1));
#pragma unroll
        for (int o = LPR / 2; o > 0; o /= 2) ss += __shfl_xor_sync(row_lanes, ss, o);
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv * (is_q ? wq[i] : wk[i]);
      }
      float y[8];
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[2 * i] = turned ? x[2 * i] * cs[i].x - x[2 * i + 1] * cs[i].y : x[2 * i];
          y[2 * i + 1] = turned ? x[2 * i + 1] * cs[i].x + x[2 * i] * cs[i].y : x[2 * i + 1];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xffffffffu, x[i], other);
          const float turned_x = upper ? x[i] * cs[i].x + o * cs[i].y : x[i] * cs[i].x - o * cs[i].y;
          y[i] = turned ? turned_x : x[i];
        }
      }
      if (r < end) {
        uint4 w;
        __half2* h2 = reinterpret_cast<__half2*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) h2[e] = __floats2half2_rn(y[2 * e], y[2 * e + 1]);
        __half* dst = is_q ? p.q_out + t * p.q_out_stride + r * D
                           : p.k_out + t * p.k_out_stride + (r - p.num_heads) * D;
        *reinterpret_cast<uint4*>(dst + c * 8) = w;
      }
    }
  }
}

template <int D>
cudaError_t launch_rope(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t st) {
  return interleaved ? pkv::launch_pdl(qk_norm_rope_kernel<D, true>, grid, dim3(kThreads), 0, st, p)
                     : pkv::launch_pdl(qk_norm_rope_kernel<D, false>, grid, dim3(kThreads), 0, st, p);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int read_device_error_rope(int reset, int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_dev_error_rope, sizeof(int));
  if (e == cudaSuccess && reset && v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_dev_error_rope, &zero, sizeof(int));
  }
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, "reading the rotation check word: %s", cudaGetErrorString(e));
  *code = v;
  return PKV_OK;
}
}  // namespace pkv

extern "C" {

int pkv_qk_norm_rope(const uint16_t* q, const uint16_t* key, const uint16_t* q_weight, const uint16_t* k_weight,
                     float eps, const int32_t* positions, int num_axes, const int64_t* frequencies,
                     const int32_t* pair_axis, int rotary_dim, int interleaved, int num_tokens, int num_heads,
                     int num_kv_heads, int head_dim, int64_t q_stride, int64_t k_stride, uint16_t* q_out,
                     uint16_t* k_out, int64_t q_out_stride, int64_t k_out_stride, void* stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_axes <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_qk_norm_rope: num_tokens=%d num_heads=%d num_kv_heads=%d num_axes=%d",
                     num_tokens, num_heads, num_kv_heads, num_axes);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "pkv_qk_norm_rope: head_dim %d not in {64, 128}", head_dim);
  if (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "pkv_qk_norm_rope: rotary_dim %d not a multiple of 16 in [16, %d]", rotary_dim,
                     head_dim);
  if (num_axes > kMaxAxes || num_heads > 65535 || num_kv_heads > 65535)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "pkv_qk_norm_rope: more than %d axes or 65535 heads", kMaxAxes);
  if (!std::isfinite(eps) || eps < 0.f)
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_qk_norm_rope: eps must be finite and not negative");
  if (num_tokens == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (!q || !key || !positions || !frequencies || !q_out || !k_out)
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_qk_norm_rope: null pointer");
  if (!aligned16(q) || !aligned16(key) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
      !aligned16(k_weight))
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_qk_norm_rope: q, key, weights and outputs must be 16-byte aligned");
  const int64_t q_row = static_cast<int64_t>(num_heads) * head_dim, k_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < q_row || q_out_stride < q_row || k_stride < k_row || k_out_stride < k_row || q_stride % 8 ||
      q_out_stride % 8 || k_stride % 8 || k_out_stride % 8)
    return pkv::fail(PKV_ERR_INVALID_ARG,
                     "pkv_qk_norm_rope: strides must be multiples of 8 and at least a token's length");
  if ((q_out == q && q_out_stride != q_stride) || (k_out == key && k_out_stride != k_stride))
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_qk_norm_rope: in place needs equal strides");
  RopeParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k = reinterpret_cast<const __half*>(key);
  p.q_weight = reinterpret_cast<const __half*>(q_weight);
  p.k_weight = reinterpret_cast<const __half*>(k_weight);
  p.positions = positions;
  p.frequencies = frequencies;
  p.pair_axis = pair_axis;
  p.q_out = reinterpret_cast<__half*>(q_out);
  p.k_out = reinterpret_cast<__half*>(k_out);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_out_stride = q_out_stride;
  p.k_out_stride = k_out_stride;
  p.num_axes = num_axes;
  p.rotary_dim = rotary_dim;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.eps = eps;
  // one CTA per token; with too few tokens to give every SM a few CTAs, a token's heads are split
  const int rpp = kThreads / (head_dim / 8), rows = num_heads + num_kv_heads;
  const int passes = (rows + rpp - 1) / rpp;
  int splits = num_tokens >= 1024 ? 1 : (1024 + num_tokens - 1) / num_tokens;
  if (splits > passes) splits = passes;
  const int per = (passes + splits - 1) / splits;
  p.rows_per_cta = per * rpp;
  const dim3 grid(num_tokens, (passes + per - 1) / per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = head_dim == 128 ? launch_rope<128>(p, interleaved != 0, grid, st)
                                  : launch_rope<64>(p, interleaved != 0, grid, st);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "pkv_qk_norm_rope launch: %s", cudaGetErrorString(e));
  pkv::clear_error();
  return PKV_OK;
}

int pkv_rope_frequencies(const double* inv_freq, int n, int64_t* frequencies_out) {
  if (n < 0 || (n > 0 && (!inv_freq || !frequencies_out)))
    return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_rope_frequencies: n=%d or a null pointer", n);
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i]))
      return pkv::fail(PKV_ERR_INVALID_ARG, "pkv_rope_frequencies: frequency %d is not finite", i);
  }
  for (int i = 0; i < n; ++i) {
    // turns per position in [-1/2, 1/2]; 2^64 times it is exact in fp64's exponent range
    const double turns = inv_freq[i] / (2.0 * 3.14159265358979323846);
    const double part = turns - std::nearbyint(turns);
    // |part| <= 1/2: half a turn forward and half a turn back are the same
    frequencies_out[i] = part >= 0.5 ? INT64_MIN : static_cast<int64_t>(std::nearbyint(part * 0x1p64));
  }
  pkv::clear_error();
  return PKV_OK;
}

}  // extern "C"
