// Rows into and out of the four-bit K/V cache, for sm_103a.
//
// A row x of D values is held as n = round((x - lo) / s) in 0..15 with lo = min x and
// s = (max x - lo) / 15: half a byte a value and four bytes a row (s and lo in fp16),
// 68 bytes for D = 128 where fp16 takes 256.  It stands for lo + s * n.
//
// Both kernels are HBM-bound.  A warp takes a token's rows (or a part of them, where there
// are few tokens), so that every access of a row is contiguous over its lanes in whole
// sectors.  The read-back has 16 values to a lane in two 16-byte chunks half a row apart, and
// runs at 98 % of the copy rate (160k tokens of 8 + 8 rows of 128: 124 us).
//
// The write has about 9 values to handle per clock and SM at HBM rate, so it counts
// instructions: 32 values to a lane, which halves what a row costs beside its values (7 us of the
// 139 that write and read-back of 16 411 tokens of 2 x 40 rows of 128 take); minimum and
// maximum on packed fp16 pairs; the quotients two to an instruction.  u = x / s - lo / s is
// rounded by adding and taking off 1.5 * 2^23, whose low bytes are then gathered; only where
// u comes nearer to a half than its error bound (some 2^-16 of all values) is n decided by
// the exact remainder.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_cache_int4 = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_cache_int4, 0, code); }

constexpr int kWarps = 4;            // per CTA

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
  int num_tokens;
  int rows_per_warp;
};

// n of one value by the definition: n s against x - lo, halves to even.  n s is exact in fp32 (4 + 11 bits).  x - lo
// can take 40 bits: d is its rounding to fp32 and rest, by a two-sum, exactly what that left.  The estimate
// d inv is 2^-17 off at most, so a little less than it rounds to n or, at and just past a half, to n - 1: only
// whether 2 (x - lo - n s) reaches s is left to see.  There r = d - n s is exact too, and d is below 16 s (below 22 s
// where s is below the normals, and exact there), so its last place is 2^-19 of s's leading bit at most:
// 2 r and s are multiples of twice d's last place, 2 rest is at most one, and decides where 2 r meets s.
__device__ __forceinline__ unsigned nearest_exact(float x, float lo, float s, float inv) {
  const float d = x - lo, back = d - x, rest = (x - (d - back)) - (lo + back);
  const float n = fminf(fmaxf(rintf(fmaf(d, inv, -0x1p-10f)), 0.f), 15.f);
  const float over = fmaf(2.f, rest, 2.f * fmaf(-n, s, d) - s);
  const unsigned whole = static_cast<unsigned>(n);
  return min(whole + (over > 0.f || (over == 0.f && (whole & 1u)) ? 1u : 0u), 15u);
}

// two fp32 sums or fused products in one instruction
__device__ __forceinline__ float2 add2(float2 a, float b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %6};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight values' n, four bits each.  d / s = u + e with u = x inv + b, b = -lo inv: inv is off by 2^-23
// relative and the sum by 2^-24 of it, so e is below 2^-18 + 2^-23 |b|; `sure` is one half less more
// than that.
__device__ __forceinline__ unsigned pack8(const uint4& raw, float inv, float b, float lo, float s, float sure) {
  constexpr float kMagic = 12582912.f;              // 1.5 * 2^23: the sum's low byte is the whole number
  const __half2* h2 = reinterpret_cast<const __half2*>(&raw);
  unsigned m[8];
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 u = fma2(__half22float2(h2[e]), inv, make_float2(b, b));
    const float2 n = add2(u, kMagic);
    const float2 r = fma2(add2(n, -kMagic), -1.f, u);
    far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
    m[2 * e] = __float_as_uint(n.x);
    m[2 * e + 1] = __float_as_uint(n.y);
  }
  const unsigned even = __byte_perm(__byte_perm(m[0], m[2], 0x0040), __byte_perm(m[4], m[6], 0x0040), 0x5410);
  const unsigned odd = __byte_perm(__byte_perm(m[1], m[3], 0x0040), __byte_perm(m[5], m[7], 0x0040), 0x5410);
  unsigned word = even + (odd << 4);
  if (!(far < sure)) {
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? __high2float(h2[i / 2]) : __low2float(h2[i / 2]);
      word |= s > 0.f ? nearest_exact(x, lo, s, inv) << (4 * i) : 0u;
    }
  }
  return word;
}

// grid (tokens / (kWarps TPW), parts of a token's K and V rows); TPW tokens to a warp
template <int D, int TPW>
__global__ void __launch_bounds__(kWarps * 32, 7) reshape_and_cache_int4_kernel(const Int4RowParams p) {
  constexpr int LPR = D / 32;                       // lanes per row: 16 values of each half of it to a lane
  constexpr int LANES = 32 / TPW;                   // lanes per token
  constexpr int RPP = LANES / LPR;                  // rows they take at a time
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int lane = threadIdx.x & (LANES - 1), c = lane % LPR, place = threadIdx.x / LANES;
  const int wanted = blockIdx.x * kWarps * TPW + place;
  if (wanted - place % TPW >= p.num_tokens) return;  // a whole warp
  bool live = TPW == 1 || wanted < p.num_tokens;
  const int t = TPW == 1 ? wanted : min(wanted, p.num_tokens - 1);
  const int H = p.num_heads;
  const int begin = blockIdx.y * p.rows_per_warp, end = min(2 * H, begin + p.rows_per_warp);
  const __half* key = p.key + t * p.key_stride + c * 16;
  const __half* value = p.value + t * p.value_stride + c * 16 - static_cast<int64_t>(H) * D;
  uint4 raw[4];
  auto load = [&](int r, uint4 (&x)[4]) {
    if (r < end) {
      const __half* src = (r < H ? key : value) + r * D;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const uint4*>(src + (k >> 1) * (D / 2) + (k & 1) * 8);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = make_uint4(0, 0, 0, 0);
    }
  };
  const int first = begin + lane / LPR;
  load(first, raw);
  int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.num_slots) {
    if (slot >= 0 && live && lane == 0 && blockIdx.y == 0) record_error(PKV_DEV_BAD_SLOT);
    if (TPW == 1) return;
    live = false;                                   // padding token or bad slot, beside others in its warp
    slot = 0;
  }
  const int in_block = static_cast<int>(slot & ((1 << p.log2_block) - 1));
  const int64_t block_base = (slot >> p.log2_block) * H * p.tile_bytes;
  uint8_t* k_block = p.k_cache + block_base;
  uint8_t* v_block = p.v_cache + block_base - static_cast<int64_t>(H) * p.tile_bytes;
  const int data_off = in_block * (D / 2) + c * 8;
  const int meta_off = ((D / 2) << p.log2_block) + in_block * 4;
  for (int r = first; r - lane / LPR < end; r += RPP) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = raw[k];
    load(r + RPP, raw);
    // NaN-keeping minimum and maximum: a row that holds a NaN gets a NaN scale
    __half2 lo2 = *reinterpret_cast<const __half2*>(&x[0]), hi2 = lo2;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2* h2 = reinterpret_cast<const __half2*>(&x[k]);
#pragma unroll
      for (int e = k == 0 ? 1 : 0; e < 4; ++e) {
        lo2 = __hmin2_nan(lo2, h2[e]);
        hi2 = __hmax2_nan(hi2, h2[e]);
      }
    }
    // lowest and negated highest side by side: one shuffle a step
    __half2 both = __hmin2_nan(__lows2half2(lo2, __hneg2(hi2)), __highs2half2(lo2, __hneg2(hi2)));
#pragma unroll
    for (int o = LPR / 2; o > 0; o /= 2) both = __hmin2_nan(both, __shfl_xor_sync(0xffffffffu, both, o));
    const float lo = __low2float(both), span = -__high2float(both) - lo;
    // span / 15 correctly rounded: one step of Markstein's division by a constant
    constexpr float kFifteenth = 1.f / 15.f;
    const float s0 = span * kFifteenth;
    __half s_h = __float2half_rn(fmaf(fmaf(-s0, 15.f, span), kFifteenth, s0));
    const float s = __half2float(s_h);
    if (!(s <= 65504.f)) s_h = __ushort_as_half(0x7fff);   // a row that is not finite stands for NaNs
    const float inv = s > 0.f ? rcp_approx(s) : 0.f;
    const float b = -lo * inv;
    // past: only where a scale below 2^-14 was rounded down
    const float sure = span * inv > 15.25f ? -1.f : 0.5f - 0x1p-17f - fabsf(b) * 0x1p-22f;
    unsigned w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack8(x[k], inv, b, lo, s, sure);
    if (r < end && live) {
      uint8_t* tile = (r < H ? k_block : v_block) + static_cast<int64_t>(r) * p.tile_bytes;
      *reinterpret_cast<uint2*>(tile + data_off) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(tile + data_off + D / 4) = make_uint2(w[2], w[3]);
      if (c == 0) *reinterpret_cast<__half2*>(tile + meta_off) = __halves2half2(s_h, __low2half(both));
    }
  }
}

// Eight values of a row: 1024 + n has n in its low bits in fp16, and the fused product rounds
// zero + scale * n once.
__device__ __forceinline__ uint4 unpack8(unsigned word, __half2 s2, __half2 z2) {
  unsigned pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned bits = ((word >> (4 * i)) & 0x000f000fu) | 0x64006400u;      // values i and i + 4
    const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&bits), __float2half2_rn(1024.f));
    const __half2 y = __hfma2(n, s2, z2);
    pair[i] = *reinterpret_cast<const unsigned*>(&y);
  }
  return make_uint4(__byte_perm(pair[0], pair[1], 0x5410), __byte_perm(pair[2], pair[3], 0x5410),
                    __byte_perm(pair[0], pair[1], 0x7632), __byte_perm(pair[2], pair[3], 0x7632));
}

// grid (tokens / (kWarps TPW), parts of a token's K and V rows)
template <int D, int TPW>
__global__ void __launch_bounds__(kWarps * 32) gather_cache_int4_kernel(const Int4RowParams p) {
  constexpr int LPR = D / 16;
  constexpr int LANES = 32 / TPW;
  constexpr int RPP = LANES / LPR;
  constexpr int U = 5;                              // rows a lane has in flight together
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int lane = threadIdx.x & (LANES - 1), c = lane % LPR;
  const int t = blockIdx.x * kWarps * TPW + threadIdx.x / LANES;
  if (t >= p.num_tokens) return;
  const int H = p.num_heads;
  const int begin = blockIdx.y * p.rows_per_warp, end = min(2 * H, begin + p.rows_per_warp);
  const int64_t slot = p.slots[t];
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (lane == 0 && blockIdx.y == 0) record_error(PKV_DEV_BAD_SLOT);
    return;
  }
  const int in_block = static_cast<int>(slot & ((1 << p.log2_block) - 1));
  const int64_t block_base = (slot >> p.log2_block) * H * p.tile_bytes;
  const uint8_t* k_block = p.k_cache + block_base;
  const uint8_t* v_block = p.v_cache + block_base - static_cast<int64_t>(H) * p.tile_bytes;
  const int data_off = in_block * (D / 2) + c * 4;
  const int meta_off = ((D / 2) << p.log2_block) + in_block * 4;
  __half* key = p.key_out + static_cast<int64_t>(t) * H * D + c * 8;
  __half* value = p.value_out + static_cast<int64_t>(t) * H * D + c * 8 - static_cast<int64_t>(H) * D;
  for (int row = begin + lane / LPR; row < end; row += U * RPP) {
    unsigned word[U][2];
    __half2 meta[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      if (r < end) {
        const uint8_t* tile = (r < H ? k_block : v_block) + static_cast<int64_t>(r) * p.tile_bytes;
        word[u][0] = *reinterpret_cast<const unsigned*>(tile + data_off);
        word[u][1] = *reinterpret_cast<const unsigned*>(tile + data_off + D / 4);
        meta[u] = *reinterpret_cast<const __half2*>(tile + meta_off);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row + u * RPP;
      if (r < end) {
        const __half2 s2 = __low2half2(meta[u]), z2 = __high2half2(meta[u]);
        __half* dst = (r < H ? key : value) + r * D;
        *reinterpret_cast<uint4*>(dst) = unpack8(word[u][0], s2, z2);
        *reinterpret_cast<uint4*>(dst + D / 2) = unpack8(word[u][1], s2, z2);
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

// A warp per token; where that leaves SMs short of warps, a token's 2 H rows are split.  Many tokens of so few
// rows that a quarter of a warp has them in two passes go four to a warp: a warp's time is its chain of
// loads and stores there (16384 tokens of one head of 128: write 12.4 -> 8.3 us, read-back 8.3 -> 6.2).  Kernels:
// for D = 64 and 128, one and four tokens to a warp.
template <typename Kernel>
int launch_rows(const char* fn, const Kernel (&kernels)[2][2], int values_per_lane, Int4RowParams p, int num_tokens,
                int head_dim, int block_size, int num_blocks, void* stream) {
  int lb = 0;
  while ((1 << lb) < block_size) ++lb;
  p.log2_block = lb;
  p.tile_bytes = block_size * (head_dim / 2 + 4);
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.num_tokens = num_tokens;
  const int rpp = 32 * values_per_lane / head_dim, passes = (2 * p.num_heads + rpp - 1) / rpp;
  int splits = num_tokens >= pkv::kFullWarps ? 1 : (pkv::kFullWarps + num_tokens - 1) / num_tokens;
  if (splits > passes) splits = passes;
  const int per = (passes + splits - 1) / splits;
  p.rows_per_warp = per * rpp;
  const bool four = 4 * p.num_heads <= rpp && num_tokens >= 4 * pkv::kFullWarps;
  const dim3 grid((num_tokens - 1) / (kWarps * (four ? 4 : 1)) + 1, (passes + per - 1) / per);
  cudaError_t e = pkv::launch_pdl(kernels[head_dim == 128][four], grid, dim3(kWarps * 32), 0,
                                  static_cast<cudaStream_t>(stream), p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  pkv::clear_error();
  return PKV_OK;
}

}  // namespace

namespace pkv {
int device_error_word_cache_int4(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_cache_int4));
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
  using Kernel = void (*)(Int4RowParams);
  static constexpr Kernel kernels[2][2] = {{reshape_and_cache_int4_kernel<64, 1>, reshape_and_cache_int4_kernel<64, 4>},
                                           {reshape_and_cache_int4_kernel<128, 1>, reshape_and_cache_int4_kernel<128, 4>}};
  return launch_rows(fn, kernels, 32, p, num_tokens, head_dim, block_size, num_blocks, stream);
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
  using Kernel = void (*)(Int4RowParams);
  static constexpr Kernel kernels[2][2] = {{gather_cache_int4_kernel<64, 1>, gather_cache_int4_kernel<64, 4>},
                                           {gather_cache_int4_kernel<128, 1>, gather_cache_int4_kernel<128, 4>}};
  return launch_rows(fn, kernels, 16, p, num_tokens, head_dim, block_size, num_blocks, stream);
}

}  // extern "C"
