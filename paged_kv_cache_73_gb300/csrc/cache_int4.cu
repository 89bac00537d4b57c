// Rows into and out of the four-bit K/V cache, for sm_103a.
//
// A row x of D values is held as n = round((x - lo) / s) in 0..15 with lo = min x and
// s = (max x - lo) / 15: half a byte a value and four bytes a row (s and lo in fp16),
// 68 bytes for D = 128 where fp16 takes 256.  It stands for lo + s * n.
//
// Both kernels are HBM-bound: 16 bytes of fp16 against 4 bytes of packed values per
// lane, D/8 lanes a row, one CTA a token.  A row's minimum and maximum are taken on
// packed fp16 pairs and reduced over its lanes by shuffles.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_cache_int4 = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_cache_int4, 0, code); }

constexpr int kThreads = 256;

struct Int4RowParams {
  const __half* key;
  const __half* value;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  __half* key_out;
  __half* value_out;
  int64_t key_stride, value_stride;
  int64_t num_slots;
  int num_heads;
  int log2_block;
  int tile_bytes;
  int rows_per_cta;
};

// n of one value by the definition, from the estimate n0 (off by at most one): n s against d = x - lo,
// halves to even.  n s is exact in fp32 (4 + 11 bits), and so is 2 (d - n s) next to a border.
__device__ __forceinline__ unsigned nearest_exact(float d, float s, float n0) {
  float n = fminf(fmaxf(n0, 0.f), 15.f);
  const float r2 = 2.f * fmaf(-n, s, d);
  const bool odd = (static_cast<int>(n) & 1) != 0;
  if (r2 > s || (r2 == s && odd)) n += 1.f;
  if (r2 < -s || (r2 == -s && odd)) n -= 1.f;
  return static_cast<unsigned>(fminf(fmaxf(n, 0.f), 15.f));
}

// grid (tokens, parts of a token's K and V rows)
template <int D>
__global__ void __launch_bounds__(kThreads) reshape_and_cache_int4_kernel(const Int4RowParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPP = kThreads / LPR;
  constexpr int U = 3;                              // passes whose loads are in flight together
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int t = blockIdx.x;
  const int tid = threadIdx.x, c = tid % LPR;
  const int H = p.num_heads;
  const int begin = blockIdx.y * p.rows_per_cta, end = min(2 * H, begin + p.rows_per_cta);
  const int first = begin + tid / LPR;
  auto load = [&](int r) {
    return r >= end ? make_uint4(0, 0, 0, 0)
           : r < H  ? *reinterpret_cast<const uint4*>(p.key + t * p.key_stride + r * D + c * 8)
                    : *reinterpret_cast<const uint4*>(p.value + t * p.value_stride + (r - H) * D + c * 8);
  };
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) raw[u] = load(first + u * RPP);
  const int64_t slot = p.slots[t];
  if (slot < 0) return;                             // padding token
  if (slot >= p.num_slots) {
    if (tid == 0 && blockIdx.y == 0) record_error(PKV_DEV_BAD_SLOT);
    return;
  }
  const int64_t blk = slot >> p.log2_block;
  const int in_block = static_cast<int>(slot & ((1 << p.log2_block) - 1));
  const int64_t block_base = blk * H * p.tile_bytes;
  const int data_off = in_block * (D / 2) + c * 4;
  const int meta_off = ((D / 2) << p.log2_block) + in_block * 4;
  for (int row = first; row - tid / LPR < end; row += U * RPP) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      const uint4 x4 = raw[u];
      raw[u] = load(r + U * RPP);
      const __half2* h2 = reinterpret_cast<const __half2*>(&x4);
      // NaN-keeping minimum and maximum: a row that holds a NaN gets a NaN scale
      __half2 lo2 = __hmin2_nan(__hmin2_nan(h2[0], h2[1]), __hmin2_nan(h2[2], h2[3]));
      __half2 hi2 = __hmax2_nan(__hmax2_nan(h2[0], h2[1]), __hmax2_nan(h2[2], h2[3]));
      // lowest and (negated) highest side by side: one shuffle a step
      __half2 both = __halves2half2(__hmin_nan(__low2half(lo2), __high2half(lo2)),
                                    __hneg(__hmax_nan(__low2half(hi2), __high2half(hi2))));
#pragma unroll
      for (int o = LPR / 2; o > 0; o /= 2) both = __hmin2_nan(both, __shfl_xor_sync(0xffffffffu, both, o));
      const __half lo_h = __low2half(both);
      const float lo = __half2float(lo_h), hi = -__half2float(__high2half(both));
      __half s_h = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
      const float s = __half2float(s_h);
      if (!(s <= 65504.f)) s_h = __ushort_as_half(0x7fff);   // a row that is not finite stands for NaNs
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
      // d / s to the nearest whole number: adding 1.5 * 2^23 rounds u = d * inv there.  u is within
      // 2^-18 of the quotient, so only a fraction that close to one half (or a quotient past 15,
      // where a scale below 2^-14 was rounded) needs the exact rule.
      constexpr float kMagic = 12582912.f;
      float d[8];
      unsigned word = 0;
      float far = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(h2[e]);
        d[2 * e] = f.x - lo;
        d[2 * e + 1] = f.y - lo;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = d[i] * inv;
        const float m = v + kMagic;
        far = fmaxf(far, fabsf(v - (m - kMagic)));
        word += __float_as_uint(m) << (4 * i);
      }
      // the whole numbers sit in the low bits of 0x4B400000 + n: take the constants' sum off
      constexpr unsigned kOnes = 0x11111111u;
      word -= 0x4B400000u * kOnes;
      if (far >= 0.5f - 0x1p-18f || (hi - lo) * inv > 15.25f) {
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= s > 0.f ? nearest_exact(d[i], s, rintf(d[i] * inv)) << (4 * i) : 0u;
      }
      if (r < end) {
        uint8_t* tile = (r < H ? p.k_cache : p.v_cache) + block_base + static_cast<int64_t>(r < H ? r : r - H) * p.tile_bytes;
        *reinterpret_cast<unsigned*>(tile + data_off) = word;
        if (c == 0) *reinterpret_cast<__half2*>(tile + meta_off) = __halves2half2(s_h, lo_h);
      }
    }
  }
}

// grid (tokens, parts of a token's K and V rows)
template <int D>
__global__ void __launch_bounds__(kThreads) gather_cache_int4_kernel(const Int4RowParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPP = kThreads / LPR;
  constexpr int U = 5;                              // rows a lane has in flight together
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int t = blockIdx.x;
  const int tid = threadIdx.x, c = tid % LPR;
  const int H = p.num_heads;
  const int begin = blockIdx.y * p.rows_per_cta, end = min(2 * H, begin + p.rows_per_cta);
  const int64_t slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (tid == 0 && blockIdx.y == 0) record_error(PKV_DEV_BAD_SLOT);
    return;
  }
  const int64_t blk = slot >> p.log2_block;
  const int in_block = static_cast<int>(slot & ((1 << p.log2_block) - 1));
  const int64_t block_base = blk * H * p.tile_bytes;
  const int data_off = in_block * (D / 2) + c * 4;
  const int meta_off = ((D / 2) << p.log2_block) + in_block * 4;
  for (int row = begin + tid / LPR; row < end; row += U * RPP) {
    unsigned word[U];
    __half2 meta[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      if (r < end) {
        const uint8_t* tile = (r < H ? p.k_cache : p.v_cache) + block_base + static_cast<int64_t>(r < H ? r : r - H) * p.tile_bytes;
        word[u] = *reinterpret_cast<const unsigned*>(tile + data_off);
        meta[u] = *reinterpret_cast<const __half2*>(tile + meta_off);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      if (r < end) {
        const __half2 s2 = __low2half2(meta[u]), z2 = __high2half2(meta[u]);
        uint4 out;
        unsigned* o = reinterpret_cast<unsigned*>(&out);
        unsigned pair[4];
        // 1024 + n has n in its low bits in fp16; the fused product rounds zero + scale * n once
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned bits = ((word[u] >> (4 * i)) & 0x000f000fu) | 0x64006400u;      // values i and i + 4
          const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&bits), __float2half2_rn(1024.f));
          const __half2 y = __hfma2(n, s2, z2);
          pair[i] = *reinterpret_cast<const unsigned*>(&y);
        }
        o[0] = __byte_perm(pair[0], pair[1], 0x5410);
        o[1] = __byte_perm(pair[2], pair[3], 0x5410);
        o[2] = __byte_perm(pair[0], pair[1], 0x7632);
        o[3] = __byte_perm(pair[2], pair[3], 0x7632);
        __half* dst = (r < H ? p.key_out : p.value_out) + (static_cast<int64_t>(t) * H + (r < H ? r : r - H)) * D + c * 8;
        *reinterpret_cast<uint4*>(dst) = out;
      }
    }
  }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

int check_shape(const char* fn, int num_tokens, int num_heads, int head_dim, int block_size, int num_blocks) {
  if (num_tokens < 0 || num_heads <= 0 || num_blocks <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_tokens=%d num_kv_heads=%d num_blocks=%d", fn, num_tokens, num_heads,
                     num_blocks);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: block_size %d not in {4, 8, 16, 32}", fn, block_size);
  if (num_heads > 65535) return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: num_kv_heads above 65535", fn);
  return PKV_OK;
}

// One CTA per token; with few tokens a token's 2 H rows are split over CTAs.
template <typename Kernel>
int launch_rows(const char* fn, Kernel k64, Kernel k128, Int4RowParams p, int num_tokens, int head_dim, int block_size,
                int num_blocks, void* stream) {
  int lb = 0;
  while ((1 << lb) < block_size) ++lb;
  p.log2_block = lb;
  p.tile_bytes = block_size * (head_dim / 2 + 4);
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  const int rpp = kThreads / (head_dim / 8), passes = (2 * p.num_heads + rpp - 1) / rpp;
  int splits = num_tokens >= 1024 ? 1 : (1024 + num_tokens - 1) / num_tokens;
  if (splits > passes) splits = passes;
  const int per = (passes + splits - 1) / splits;
  p.rows_per_cta = per * rpp;
  const dim3 grid(num_tokens, (passes + per - 1) / per);
  cudaError_t e = pkv::launch_pdl(head_dim == 128 ? k128 : k64, grid, dim3(kThreads), 0,
                                  static_cast<cudaStream_t>(stream), p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  pkv::clear_error();
  return PKV_OK;
}

}  // namespace

namespace pkv {
int read_device_error_cache_int4(int reset, int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_dev_error_cache_int4, sizeof(int));
  if (e == cudaSuccess && reset && v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_dev_error_cache_int4, &zero, sizeof(int));
  }
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, "reading the four-bit cache's check word: %s", cudaGetErrorString(e));
  *code = v;
  return PKV_OK;
}
}  // namespace pkv

extern "C" {

int pkv_reshape_and_cache_int4(const uint16_t* key, const uint16_t* value, uint8_t* k_cache, uint8_t* v_cache,
                               const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
                               int block_size, int num_blocks, int64_t key_stride, int64_t value_stride,
                               void* stream) {
  const char* fn = "pkv_reshape_and_cache_int4";
  int rc = check_shape(fn, num_tokens, num_kv_heads, head_dim, block_size, num_blocks);
  if (rc != PKV_OK) return rc;
  if (num_tokens == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (!key || !value || !k_cache || !v_cache || !slot_mapping)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: key, value and caches must be 16-byte aligned", fn);
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (key_stride < row || value_stride < row || key_stride % 8 || value_stride % 8)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: strides must be multiples of 8 and at least a token's length", fn);
  Int4RowParams p{};
  p.key = reinterpret_cast<const __half*>(key);
  p.value = reinterpret_cast<const __half*>(value);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slots = slot_mapping;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.num_heads = num_kv_heads;
  return launch_rows(fn, reshape_and_cache_int4_kernel<64>, reshape_and_cache_int4_kernel<128>, p, num_tokens, head_dim,
                     block_size, num_blocks, stream);
}

int pkv_gather_cache_int4(const uint8_t* k_cache, const uint8_t* v_cache, const int64_t* slot_mapping,
                          uint16_t* key, uint16_t* value, int num_tokens, int num_kv_heads, int head_dim,
                          int block_size, int num_blocks, void* stream) {
  const char* fn = "pkv_gather_cache_int4";
  int rc = check_shape(fn, num_tokens, num_kv_heads, head_dim, block_size, num_blocks);
  if (rc != PKV_OK) return rc;
  if (num_tokens == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (!key || !value || !k_cache || !v_cache || !slot_mapping)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: key, value and caches must be 16-byte aligned", fn);
  Int4RowParams p{};
  p.k_cache = const_cast<uint8_t*>(k_cache);
  p.v_cache = const_cast<uint8_t*>(v_cache);
  p.slots = slot_mapping;
  p.key_out = reinterpret_cast<__half*>(key);
  p.value_out = reinterpret_cast<__half*>(value);
  p.num_heads = num_kv_heads;
  return launch_rows(fn, gather_cache_int4_kernel<64>, gather_cache_int4_kernel<128>, p, num_tokens, head_dim, block_size,
                     num_blocks, stream);
}

}  // extern "C"
