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
//  * One warp takes one token (or a part of its heads, where there are few tokens, or two
//    tokens of few heads): it computes the token's R/2 sines and cosines once and uses them
//    for all of its heads.  No CTA barrier: warps run free of one another.
//  * The angle is computed in whole numbers: f is given in units of 2^-64 turns, so
//    position * f wraps modulo one turn by itself, exactly, however far the
//    position; its top 32 bits then go to sincospif.  A product in fp32 would be off
//    by whole radians at position 10^6 and beyond.
//  * D/16 lanes hold a row, each eight pairs: eight first values and their eight second
//    values, R/2 further on (or interleaved with them).  No shuffle is needed to turn
//    them, and weights times sines are formed once per token, so a pair takes four fused
//    operations (two to an instruction) and the product with the norm.
// Measured: 32768 tokens of 40 + 8 heads of 128 with norms and three axes, 122 us, 98 % of the
// copy rate, and with interleaved pairs 139 us, 85 % (122 registers against 80, four CTAs to an SM against
// six); 64 tokens of 40 + 40 heads 4.6 us in a row of such calls, a launch and two round trips.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_rope = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_rope, 0, code); }

constexpr int kWarps = 4;            // per CTA
constexpr int kMaxAxes = 8;
// From kPairTokens tokens of at most kPairPasses warps' worth of rows each, half a warp takes a token: there a
// warp's time is its chain of loads, angles and stores, and two chains share it (32768 tokens, 8 + 1 heads of
// 64, 37 -> 24 us, of 128, 43 -> 34).  8192 tokens of 32 + 8 heads of 128 would go from 33 to 40 us.
constexpr int kPairTokens = 2 * pkv::kFullWarps, kPairPasses = 4;

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
  int rows_per_warp;
  float eps;
};

// two fp32 products, sums or fused products in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// grid (tokens / (kWarps TPW), parts of a token's query and key heads); TPW tokens to a warp
template <int D, bool INTERLEAVED, int TPW>
__global__ void __launch_bounds__(kWarps * 32, INTERLEAVED ? 4 : 6) qk_norm_rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 16;                       // lanes per row
  constexpr int LANES = 32 / TPW;                   // lanes per token
  constexpr int RPP = LANES / LPR;                  // rows they take at a time
  constexpr int PF = 2;                             // of which so many are in flight
  __shared__ __align__(16) float cos_tab[kWarps * TPW][D / 2], sin_tab[kWarps * TPW][D / 2];
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int lane = threadIdx.x & (LANES - 1), c = lane % LPR, slot = threadIdx.x / LANES;
  const int wanted = blockIdx.x * kWarps * TPW + slot;
  if (wanted - slot % TPW >= p.num_tokens) return;  // a whole warp
  const bool live = TPW == 1 || wanted < p.num_tokens;
  const int t = TPW == 1 ? wanted : min(wanted, p.num_tokens - 1);
  const int total = p.num_heads + p.num_kv_heads;
  const int begin = blockIdx.y * p.rows_per_warp, end = min(total, begin + p.rows_per_warp);
  // this lane's values of a row: eight from first_off and eight from second_off.  The lanes past the
  // turned ones hold 16 values in a row as they are.
  const int turned_lanes = p.rotary_dim / 16;
  const bool turned = c < turned_lanes;
  const int first_off = INTERLEAVED || !turned ? c * 16 : c * 8;
  const int second_off = INTERLEAVED || !turned ? c * 16 + 8 : c * 8 + p.rotary_dim / 2;
  const __half* q = p.q + t * p.q_stride;
  const __half* k = p.k + t * p.k_stride - static_cast<int64_t>(p.num_heads) * D;
  __half* q_out = p.q_out + t * p.q_out_stride;
  __half* k_out = p.k_out + t * p.k_out_stride - static_cast<int64_t>(p.num_heads) * D;
  uint4 raw[PF][2];
  auto load = [&](int r, uint4 (&x)[2]) {
    if (r < end) {
      const __half* src = (r < p.num_heads ? q : k) + r * D;
      x[0] = *reinterpret_cast<const uint4*>(src + first_off);
      x[1] = *reinterpret_cast<const uint4*>(src + second_off);
    } else {
      x[0] = x[1] = make_uint4(0, 0, 0, 0);
    }
  };
  const int sub = lane / LPR;
#pragma unroll
  for (int u = 0; u < PF; ++u) load(begin + u * RPP + sub, raw[u]);

  for (int pair = lane; pair < p.rotary_dim / 2; pair += LANES) {
    const int axis = p.pair_axis == nullptr ? 0 : p.pair_axis[pair];
    float cs = 1.f, sn = 0.f;
    if (axis >= 0 && axis < p.num_axes) {
      const int64_t pos = p.positions[static_cast<int64_t>(axis) * p.num_tokens + t];
      // turns modulo one as a signed 64-bit fraction: the top 32 bits are 2^-32 turns in [-1/2, 1/2)
      const uint64_t turns = static_cast<uint64_t>(pos) * static_cast<uint64_t>(p.frequencies[pair]);
      sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &sn, &cs);
    } else if (blockIdx.y == 0) {
      record_error(PKV_DEV_BAD_AXIS);
    }
    cos_tab[slot][pair] = cs;
    sin_tab[slot][pair] = sn;
  }
  __syncwarp();

  // the query rows, then the key rows: each with its weight folded into the turn
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int r1 = part == 0 ? min(end, p.num_heads) : end;
    const int r0 = part == 0 ? begin : max(begin, p.num_heads);
    if (r0 >= r1) continue;
    const __half* weight = part == 0 ? p.q_weight : p.k_weight;
    // first  <- first * fc - second * fs,   second <- second * sc + first * ss   (two pairs a register pair)
    float2 fc[4], fs[4], sc[4], ss[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w1[2] = {1.f, 1.f}, w2[2] = {1.f, 1.f};
      if (weight != nullptr) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = 2 * i + j;
          w1[j] = __half2float(weight[INTERLEAVED && turned ? c * 16 + 2 * e : first_off + e]);
          w2[j] = __half2float(weight[INTERLEAVED && turned ? c * 16 + 2 * e + 1 : second_off + e]);
        }
      }
      float2 cs = make_float2(1.f, 1.f), sn = make_float2(0.f, 0.f);
      if (turned) {
        cs = *reinterpret_cast<const float2*>(&cos_tab[slot][c * 8 + 2 * i]);
        sn = *reinterpret_cast<const float2*>(&sin_tab[slot][c * 8 + 2 * i]);
      }
      fc[i] = make_float2(w1[0] * cs.x, w1[1] * cs.y);
      fs[i] = make_float2(-w2[0] * sn.x, -w2[1] * sn.y);
      sc[i] = make_float2(w2[0] * cs.x, w2[1] * cs.y);
      ss[i] = make_float2(w1[0] * sn.x, w1[1] * sn.y);
    }
    __half* dst_base = part == 0 ? q_out : k_out;
    // the prefetched rows run on from the query rows into the key rows only where a pass ends there:
    // otherwise the key rows start anew
    if (part == 1 && begin < p.num_heads) {
#pragma unroll
      for (int u = 0; u < PF; ++u) load(r0 + u * RPP + sub, raw[u]);
    }
    for (int row = r0; row < r1; row += PF * RPP) {
#pragma unroll
      for (int u = 0; u < PF; ++u) {
        const int r = row + u * RPP + sub;
        float2 a[4], b[4];
        {
          const __half2* h0 = reinterpret_cast<const __half2*>(&raw[u][0]);
          const __half2* h1 = reinterpret_cast<const __half2*>(&raw[u][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (INTERLEAVED && turned) {
              // pairs lie side by side: (a0 b0 a1 b1 ..)
              const __half2* h = i < 2 ? h0 : h1;
              const float2 x = __half22float2(h[2 * (i & 1)]), y = __half22float2(h[2 * (i & 1) + 1]);
              a[i] = make_float2(x.x, y.x);
              b[i] = make_float2(x.y, y.y);
            } else {
              a[i] = __half22float2(h0[i]);
              b[i] = __half22float2(h1[i]);
            }
          }
        }
        load(r + PF * RPP, raw[u]);
        float inv = 1.f;
        if (weight != nullptr) {
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) s2 = fma2(b[i], b[i], fma2(a[i], a[i], s2));
          float s = s2.x + s2.y;
#pragma unroll
          for (int o = LPR / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
          inv = rsqrtf(s * (1.f / D) + p.eps);
        }
        const float2 inv2 = make_float2(inv, inv);
        uint4 w[2];
        __half2* o0 = reinterpret_cast<__half2*>(&w[0]);
        __half2* o1 = reinterpret_cast<__half2*>(&w[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 x = mul2(a[i], fc[i]), y = mul2(b[i], sc[i]);
          if (turned) {
            x = fma2(b[i], fs[i], x);
            y = fma2(a[i], ss[i], y);
          }
          x = mul2(x, inv2);
          y = mul2(y, inv2);
          if (INTERLEAVED && turned) {
            __half2* o = i < 2 ? o0 : o1;
            o[2 * (i & 1)] = __floats2half2_rn(x.x, y.x);
            o[2 * (i & 1) + 1] = __floats2half2_rn(x.y, y.y);
          } else {
            o0[i] = __floats2half2_rn(x.x, x.y);
            o1[i] = __floats2half2_rn(y.x, y.y);
          }
        }
        if (r < r1 && live) {
          __half* dst = dst_base + r * D;
          *reinterpret_cast<uint4*>(dst + first_off) = w[0];
          *reinterpret_cast<uint4*>(dst + second_off) = w[1];
        }
      }
    }
  }
}

template <int D, int TPW>
cudaError_t launch_rope(const RopeParams& p, bool interleaved, dim3 grid, cudaStream_t st) {
  return interleaved ? pkv::launch_pdl(qk_norm_rope_kernel<D, true, TPW>, grid, dim3(kWarps * 32), 0, st, p)
                     : pkv::launch_pdl(qk_norm_rope_kernel<D, false, TPW>, grid, dim3(kWarps * 32), 0, st, p);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int device_error_word_rope(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_rope));
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
  // a warp per token, or half a one; where that leaves SMs short of warps, a token's heads are split
  const int rpp = 512 / head_dim, rows = num_heads + num_kv_heads, passes = (rows + rpp - 1) / rpp;
  int splits = num_tokens >= pkv::kFullWarps ? 1 : (pkv::kFullWarps + num_tokens - 1) / num_tokens;
  if (splits > passes) splits = passes;
  const int per = (passes + splits - 1) / splits;
  p.rows_per_warp = per * rpp;
  const int tpw = passes <= kPairPasses && num_tokens >= kPairTokens ? 2 : 1;
  const dim3 grid((num_tokens - 1) / (kWarps * tpw) + 1, (passes + per - 1) / per);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = interleaved != 0;
  cudaError_t e = head_dim == 128 ? (tpw == 2 ? launch_rope<128, 2>(p, inter, grid, st) : launch_rope<128, 1>(p, inter, grid, st))
                                  : (tpw == 2 ? launch_rope<64, 2>(p, inter, grid, st) : launch_rope<64, 1>(p, inter, grid, st));
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
