// Paged decode attention over a K/V cache held in four bits, for sm_103a: one query
// per (sequence, head), groups of query heads sharing a cached head.
//
// A cached row stands for z + s n (n whole numbers 0..15, s and z fp16 per row), so
//   q . k_t = s_t (q . n_t) + z_t sum(q),      o = sum_t p_t (s_t n_t + z_t) / sum_t p_t,
// and only whole numbers meet the tensor cores: the rows' scales and zero points are
// applied once per (token, head), in fp32, not once per value.
//
// What bounds it: 68 bytes a row (D = 128) where fp16 takes 256, so at HBM rate an SM
// has 3.8 times as many values to handle per clock as with fp16 rows: 24 bytes a clock
// are 45 values, times 2 flops, times the group's heads.  Two choices make that fit.
//  * Values are never converted.  A half byte n under mask 0x000f is the fp16 number
//    n 2^-24 (subnormal), under mask 0x00f0 it is 16 n 2^-24: one AND gives two fp16
//    operands, exactly.  The tensor cores take subnormals at full rate, the 2^24 goes
//    into the final fp32 factor, and the 16 into q (exactly) or the output.
//  * The products run on mma.sync with the cached rows as the 16-row operand and eight
//    query heads as the 8-column one: S^T = K q^T and O^T = V^T P^T.  A lone head wastes
//    seven columns, but the products are then still a small part of the issue slots;
//    tcgen05 would want its operands in shared memory as fp16, which is the conversion
//    that this layout saves.
//
// Layout within a warp (lane = 4 g + t): for S^T, lane (g, t) holds D/4 values of token
// rows g and g + 8; which of the row's values a lane takes is free as long as q is laid
// out the same, so a lane reads D/8 contiguous bytes.  For O^T, it holds two pairs of
// tokens (2t, 2t + 1 and those + 8) and D/8 values g D/8 .., of each; a byte permute
// joins a byte of two tokens' words into two fp16 pairs.  P^T comes from S^T's
// accumulator by an 8x8 transpose in registers (movmatrix).
//
// Softmax in base 2 with a running maximum that moves only when a chunk raises it by
// more than 2^8.  The weight that multiplies V's whole numbers is u_t = p_t s_t, rounded
// to fp16; the maximum is kept over x_t + log2 of s_t's exponent, so that u is at most
// 2^9 and its greatest is a normal number whatever the rows' scales.  With u' = fp16(u),
//   sum p (s n + z) = sum u' (n - 8) + sum p (z + 8 s) + (rounding of u) (n - 8):
// the second sum is fp32, and sum u' comes from one more product, with ones, so that a
// weight's rounding meets n - 8 and not n.
//
// Each warp streams its own tokens, 32 at a time, through a ring in shared memory by
// 16-byte cp.async: rows of any block size land in the same place, and V's rows XOR-ed so
// that four tokens' words are read without bank conflicts.  The context is split over CTAs
// and over a CTA's warps, joined by the log-sum-exp identity (second kernel for the CTAs'
// parts).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_attention_int4 = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_attention_int4, 0, code); }

#ifndef V_MINB
#define V_MINB 3
#endif
constexpr unsigned FULL = 0xffffffffu;
constexpr int NW = 4;                 // warps per CTA
constexpr int CHUNK = 32;             // tokens a warp handles at a time
constexpr int kMinPartTokens = 128;   // one chunk per warp
constexpr int kMaxPartTokens = 1024;
constexpr float kRescale = 8.f;       // the running maximum moves when a chunk passes it by this much

struct Int4Params {
  const __half* q;
  const uint8_t* k;
  const uint8_t* v;
  const int32_t* tables;
  const int32_t* lens;
  __half* out;
  float* ws_ml;  // [S, H, max_parts, 2] (m, l), base-2 log domain
  float* ws_o;   // [S, H, max_parts, D] unnormalised partial outputs
  int num_heads, num_kv_heads, group, head_tiles;
  int num_blocks, max_blocks, log2_block;
  int part_tokens, max_parts;
  float scale_log2;
};

__device__ __forceinline__ void mma16816(float (&c)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                         unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned transpose8x8(unsigned x) {
  unsigned y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&h);
}
// log2 of a scale (a non-negative fp16 number), that of the smallest fp16 for zero; it only places
// the running maximum
__device__ __forceinline__ float log2_of(float s) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return fmaxf(y, -24.f);
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int W>
__device__ __forceinline__ void load_words(unsigned (&w)[W], const uint8_t* src) {
  if constexpr (W == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (W == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const unsigned*>(src);
  }
}

#ifndef V_NST
#define V_NST 4
#endif
// A ring stage: 32 tokens' K rows, V rows (XOR-ed), K and V (scale, zero) pairs.
template <int D>
struct Ring {
  static constexpr int ROW = D / 2;                 // bytes of a row's values
  static constexpr int V_OFF = CHUNK * ROW;
  static constexpr int META_OFF = 2 * CHUNK * ROW;
  static constexpr int STAGE = META_OFF + 2 * CHUNK * 4;
  static constexpr int NST = V_NST;
  static constexpr int WARP = NST * STAGE;          // a warp's ring
};
// Byte offset of 16-byte chunk c of V row r within a stage's V rows: in each 128-byte line (2 or 4
// rows) the chunk's place is XOR-ed with twice the line's number mod 4, so the eight lanes that read
// rows 2t or 2t + 1 of one chunk pair, t = 0..3, reach different banks.
template <int D>
__device__ __forceinline__ int v_place(int r, int c) {
  const int lin = r * (D / 32) + c, line = lin >> 3;
  return line * 128 + (((lin & 7) ^ ((line & 3) << 1)) << 4);
}

// A warp's running softmax over its tokens for 8 NT heads; lane (g, t) holds heads 8 n + 2t,
// 8 n + 2t + 1.
template <int D, int NT>
struct WarpState {
  float m[NT][2], l[NT][2], c[NT][2];   // l and c: this lane's tokens only, until the end
  float acc[NT][D / 16][4];             // sum u' n: {even value, heads 2t, 2t + 1; odd value x 16, the same}
  float ones[NT][4];                    // sum u'
};

// One chunk of `valid` tokens (all 32 unless MASKED) staged at `stage`.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void chunk_update(const unsigned char* stage, int valid, const unsigned (&qf)[NT][D / 16][2],
                                             const float (&ca)[NT][2], const float (&cb)[NT][2], WarpState<D, NT>& st,
                                             int g, int t, const int (&v_off)[4]) {
  using R = Ring<D>;
  constexpr int WK = D / 32;            // words of a K row per lane
  constexpr int WV = D / 64;            // words of a V row per lane
  float x[NT][2][4];                    // tile i, {token g: heads 2t, 2t + 1; token g + 8: the same}
  float2 vm[2][2];                      // V's scale and zero + 8 scale of those tokens
  float top[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    unsigned ka[WK], kb[WK];
    load_words<WK>(ka, stage + (16 * i + g) * R::ROW + t * (D / 8));
    load_words<WK>(kb, stage + (16 * i + g + 8) * R::ROW + t * (D / 8));
    float dot[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) dot[n][0] = dot[n][1] = dot[n][2] = dot[n][3] = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const unsigned a = ka[w] >> (8 * half), b = kb[w] >> (8 * half);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma16816(dot[n], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u, qf[n][2 * w + half][0],
                   qf[n][2 * w + half][1]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 16 * i + g + 8 * r;
      const bool live = !MASKED || row < valid;
      const float2 km = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + row * 4));
      vm[i][r] = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + CHUNK * 4 + row * 4));
      if (!live) vm[i][r] = make_float2(0.f, 0.f);
      const float e = log2_of(vm[i][r].x);
      vm[i][r].y = fmaf(8.f, vm[i][r].x, vm[i][r].y);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float y = fmaf(km.x, ca[n][j] * dot[n][2 * r + j], km.y * cb[n][j]);
          x[n][i][2 * r + j] = live ? y : -INFINITY;
          top[n][j] = fmaxf(top[n][j], x[n][i][2 * r + j] + e);
        }
    }
  }
  bool moves = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) top[n][j] = fmaxf(top[n][j], __shfl_xor_sync(FULL, top[n][j], o));
      moves |= top[n][j] > st.m[n][j] + kRescale;
    }
  if (__any_sync(FULL, moves)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float m = fmaxf(st.m[n][j], top[n][j]);
        const float f = m == -INFINITY ? 1.f : exp2f(st.m[n][j] - m);
        st.m[n][j] = m;
        st.l[n][j] *= f;
        st.c[n][j] *= f;
        st.ones[n][j] *= f;
        st.ones[n][2 + j] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.acc[n][i][j] *= f;
          st.acc[n][i][2 + j] *= f;
        }
      }
  }
  unsigned pb[NT][2][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float u[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // the chunk has a valid token, so the maximum is not -inf (a NaN logit makes NaNs)
          const float w = fast_exp2(x[n][i][2 * r + j] - st.m[n][j]);
          st.l[n][j] += w;
          u[j] = w * vm[i][r].x;
          st.c[n][j] = fmaf(w, vm[i][r].y, st.c[n][j]);
        }
        pb[n][i][r] = transpose8x8(pack2(u[0], u[1]));
      }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    unsigned va[4][WV];                 // tokens 2t, 2t + 1, 2t + 8, 2t + 9 of the tile
#pragma unroll
    for (int r = 0; r < 4; ++r) load_words<WV>(va[r], stage + R::V_OFF + v_off[r] + i * 16 * R::ROW);
#pragma unroll
    for (int w = 0; w < WV; ++w)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const unsigned sel = 0x4400u + 0x1111u * b;          // byte b of the first token, byte b of the second
        const unsigned e = __byte_perm(va[0][w], va[1][w], sel), f = __byte_perm(va[2][w], va[3][w], sel);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma16816(st.acc[n][4 * w + b], e & 0x000f000fu, e & 0x00f000f0u, f & 0x000f000fu, f & 0x00f000f0u, pb[n][i][0],
                   pb[n][i][1]);
      }
    constexpr unsigned kOne2 = 0x3c003c00u;
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16816(st.ones[n], kOne2, kOne2, kOne2, kOne2, pb[n][i][0], pb[n][i][1]);
  }
}

// grid (parts, K/V heads x tiles of 8 NT heads of a group, sequences)
template <int D, int NT>
__global__ void __launch_bounds__(NW * 32, V_MINB) paged_attention_int4_kernel(const Int4Params p) {
  using R = Ring<D>;
  constexpr int HT = 8 * NT;
  constexpr int WK = D / 32;            // words of a K row per lane
  constexpr int ROW = R::ROW;
  __shared__ int64_t tile_off[kMaxPartTokens / 4];
  extern __shared__ __align__(128) unsigned char smem[];     // the warps' rings
  static_assert(HT * (D + 2) * 4 <= R::WARP, "a warp's result takes its ring's place");

  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int part = blockIdx.x, s = blockIdx.z;
  const int kvh = blockIdx.y / p.head_tiles, h_in_group = (blockIdx.y % p.head_tiles) * HT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int lb = p.log2_block, B = 1 << lb;
  const int H = p.num_heads;
  const int h0 = kvh * p.group + h_in_group;                 // first query head of this CTA
  const int nh = min(HT, p.group - h_in_group);              // heads that exist
  const int ctx = p.lens[s];
  const bool bad_len = ctx < 0 || ctx > (p.max_blocks << lb);
  const int nparts = ctx <= 0 || bad_len ? 1 : (ctx + p.part_tokens - 1) / p.part_tokens;
  if (part >= nparts) return;
  auto empty_result = [&]() {
    for (int i = tid; i < nh * D; i += NW * 32) {
      const size_t row = static_cast<size_t>(s) * H + h0 + i / D;
      if (nparts == 1) p.out[row * D + i % D] = __float2half_rn(0.f);
      else p.ws_o[(row * p.max_parts + part) * D + i % D] = 0.f;
    }
    if (nparts > 1 && tid < nh) {
      const size_t w = (static_cast<size_t>(s) * H + h0 + tid) * p.max_parts + part;
      p.ws_ml[2 * w] = -INFINITY;
      p.ws_ml[2 * w + 1] = 0.f;
    }
  };
  if (ctx <= 0 || bad_len) {
    if (bad_len && tid == 0) record_error(PKV_DEV_BAD_CONTEXT_LEN);
    empty_result();
    return;
  }
  const int begin = part * p.part_tokens, n_tok = min(p.part_tokens, ctx - begin);
  const int64_t tile_bytes = static_cast<int64_t>(ROW + 4) << lb;
  int bad = 0;
  for (int i = tid; i < (n_tok + B - 1) >> lb; i += NW * 32) {
    const int phys = p.tables[static_cast<size_t>(s) * p.max_blocks + (begin >> lb) + i];
    const bool ok = phys >= 0 && phys < p.num_blocks;
    bad |= !ok;
    tile_off[i] = ok ? (static_cast<int64_t>(phys) * p.num_kv_heads + kvh) * tile_bytes : 0;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) record_error(PKV_DEV_BAD_BLOCK_ID);
    empty_result();
    return;
  }

  // The warp takes chunks warp, warp + NW, ...; a lane copies the same pieces of every chunk: 16-byte
  // pieces of K and V rows, and of four rows' (scale, zero) pairs.  Rows past the partition's tokens
  // are not read.
  unsigned char* ring = smem + warp * R::WARP;
  constexpr int PIECES = CHUNK * ROW / 16 / 32;              // of K, and of V, per lane
  int piece_blk[PIECES], piece_off[PIECES], v_dst[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = i * 32 + lane, row = at / (ROW / 16), c = at % (ROW / 16);
    piece_blk[i] = row >> lb;
    piece_off[i] = (row & (B - 1)) * ROW + c * 16;
    v_dst[i] = R::V_OFF + v_place<D>(row, c);
  }
  const int meta_row = 4 * (lane & 7);
  const uint8_t* meta_src = (lane & 8 ? p.v : p.k) + (ROW << lb) + (meta_row & (B - 1)) * 4;
  const int n_chunks = (n_tok + CHUNK - 1) / CHUNK;
  const int my_n = n_chunks > warp ? (n_chunks - warp + NW - 1) / NW : 0;
  auto fill = [&](int k) {
    if (k < my_n) {
      const int c0 = (warp + k * NW) * CHUNK, blk0 = c0 >> lb;
      const uint32_t dst = smem_u32(ring + (k % R::NST) * R::STAGE);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (c0 + (i * 32 + lane) / (ROW / 16) < n_tok) {
          const int64_t off = tile_off[blk0 + piece_blk[i]] + piece_off[i];
          cp_async16(dst + (i * 32 + lane) * 16, p.k + off);
          cp_async16(dst + v_dst[i], p.v + off);
        }
      }
      if (lane < 16 && c0 + meta_row < n_tok)
        cp_async16(dst + R::META_OFF + lane * 16, meta_src + tile_off[blk0 + (meta_row >> lb)]);
    }
    cp_async_commit();                                       // one group a chunk, empty ones too
  };
#pragma unroll
  for (int k = 0; k < R::NST - 1; ++k) fill(k);

  // q as the 8-column operand, laid out like a K row's half bytes: word w of a lane holds values
  // 8 w .. 8 w + 7 of its D/4; AND 0x000f000f takes values (0, 4) of it, AND 0x00f000f0 16 x (1, 5),
  // and 8 bits further (2, 6) and 16 x (3, 7).  q is scaled by a power of two per head so that its
  // greatest value is near 2^9: q / 16 then loses nothing that matters.
  unsigned qf[NT][D / 16][2];
  float ca[NT][2], cb[NT][2];           // x = s (ca dot) + z cb, heads 2t, 2t + 1 of each tile
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float qv[WK][8];
    float amax = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (n * 8 + g < nh)
        raw = *reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(s) * H + h0 + n * 8 + g) * D + t * (D / 4) + w * 8);
      const __half2* h2 = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(h2[e]);
        qv[w][2 * e] = f.x;
        qv[w][2 * e + 1] = f.y;
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        sum += f.x + f.y;
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
      amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, o));
      sum += __shfl_xor_sync(FULL, sum, o);
    }
    const int e = amax > 0.f ? static_cast<int>(__float_as_uint(amax) >> 23) - 127 : 9;
    const float up = __uint_as_float(static_cast<unsigned>(9 - e + 127) << 23);
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float d = up * 0.0625f;
      qf[n][2 * w][0] = pack2(qv[w][0] * up, qv[w][4] * up);
      qf[n][2 * w][1] = pack2(qv[w][1] * d, qv[w][5] * d);
      qf[n][2 * w + 1][0] = pack2(qv[w][2] * up, qv[w][6] * up);
      qf[n][2 * w + 1][1] = pack2(qv[w][3] * d, qv[w][7] * d);
    }
    const float a = p.scale_log2 * 16777216.f * __uint_as_float(static_cast<unsigned>(e - 9 + 127) << 23);
    const float b = p.scale_log2 * sum;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      ca[n][j] = __shfl_sync(FULL, a, (2 * t + j) * 4);
      cb[n][j] = __shfl_sync(FULL, b, (2 * t + j) * 4);
    }
  }

  WarpState<D, NT> st;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      st.m[n][j] = -INFINITY;
      st.l[n][j] = st.c[n][j] = 0.f;
      st.ones[n][j] = st.ones[n][2 + j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.acc[n][i][j] = 0.f;
  }

  int v_off[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    // lane g's D/16 bytes of V rows 2t, 2t + 1, 2t + 8, 2t + 9
    const int at = g * (D / 16);
    v_off[r] = v_place<D>(2 * t + (r & 1) + 8 * (r >> 1), at / 16) + at % 16;
  }
  for (int k = 0; k < my_n; ++k) {
    cp_async_wait<R::NST - 2>();
    __syncwarp();                                            // every lane's copies; and stage k - 1 is read
    fill(k + R::NST - 1);
    const unsigned char* stage = ring + (k % R::NST) * R::STAGE;
    const int valid = n_tok - (warp + k * NW) * CHUNK;
    if (valid >= CHUNK)
      chunk_update<D, NT, false>(stage, CHUNK, qf, ca, cb, st, g, t, v_off);
    else
      chunk_update<D, NT, true>(stage, valid, qf, ca, cb, st, g, t, v_off);
  }
  cp_async_wait<0>();
  __syncwarp();                                              // the ring is free

  // the warps' results side by side: o in values, (m, l)
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) {
        st.l[n][j] += __shfl_xor_sync(FULL, st.l[n][j], o);
        st.c[n][j] += __shfl_xor_sync(FULL, st.c[n][j], o);
      }
      float* dst = reinterpret_cast<float*>(ring) + (n * 8 + 2 * t + j) * (D + 2);
      const float mid = fmaf(-8.f, st.ones[n][j], st.c[n][j]);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int d = g * (D / 8) + 2 * i;                 // word i / 4, byte i % 4: values 2 i and 2 i + 1
        dst[d] = fmaf(st.acc[n][i][j], 16777216.f, mid);
        dst[d + 1] = fmaf(st.acc[n][i][2 + j], 1048576.f, mid);
      }
      if (g == 0) {
        dst[D] = st.m[n][j];
        dst[D + 1] = st.l[n][j];
      }
    }
  __syncthreads();
  for (int i = tid; i < nh * D; i += NW * 32) {
    const int h = i / D, d = i % D;
    auto comb = [&](int w) { return reinterpret_cast<const float*>(smem + w * R::WARP) + h * (D + 2); };
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, comb(w)[D]);
    float L = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float mw = comb(w)[D];
      const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
      L = fmaf(comb(w)[D + 1], f, L);
      o = fmaf(comb(w)[d], f, o);
    }
    const size_t row = static_cast<size_t>(s) * H + h0 + h;
    if (nparts == 1) {
      p.out[row * D + d] = __float2half_rn(o / L);
    } else {
      const size_t w0 = row * p.max_parts + part;
      p.ws_o[w0 * D + d] = o;
      if (d == 0) {
        p.ws_ml[2 * w0] = M;
        p.ws_ml[2 * w0 + 1] = L;
      }
    }
  }
}

// Joins the parts of every (sequence, head) with more than one: a warp each, a lane D/32 values.
template <int D>
__global__ void __launch_bounds__(128) paged_attention_int4_merge_kernel(const Int4Params p) {
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x * 4 + warp, s = blockIdx.y;
  if (h >= p.num_heads) return;
  const int ctx = p.lens[s];
  if (ctx <= p.part_tokens || ctx > (p.max_blocks << p.log2_block)) return;   // one part (or none): written already
  const int nparts = (ctx + p.part_tokens - 1) / p.part_tokens;
  const size_t w0 = (static_cast<size_t>(s) * p.num_heads + h) * p.max_parts;
  constexpr int V = D / 32;
  float acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
  float M = -INFINITY, L = 0.f;
  for (int i = 0; i < nparts; ++i) M = fmaxf(M, p.ws_ml[2 * (w0 + i)]);
  for (int i = 0; i < nparts; ++i) {
    const float m = p.ws_ml[2 * (w0 + i)];
    const float f = m == -INFINITY ? 0.f : exp2f(m - M);
    L = fmaf(p.ws_ml[2 * (w0 + i) + 1], f, L);
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = fmaf(p.ws_o[(w0 + i) * D + lane * V + c], f, acc[c]);
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int c = 0; c < V; ++c)
    p.out[(static_cast<size_t>(s) * p.num_heads + h) * D + lane * V + c] = __float2half_rn(acc[c] * inv);
}

__host__ __device__ constexpr size_t ws_ml_floats(size_t pairs) { return (pairs * 2 + 3) / 4 * 4; }

int device_sms() {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  std::lock_guard<std::mutex> g(mu);
  if (!cache[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 152;
    cache[dev] = n;
  }
  return cache[dev];
}

// Head tiles of 8 columns, or of 16 where a group has more than 8 heads (the rows are then unpacked
// once for both).
struct Plan {
  int nt, head_tiles, part_tokens, max_parts;
};
Plan plan_for(int num_seqs, int num_heads, int num_kv_heads, int max_ctx) {
  Plan pl{};
  const int group = num_heads / num_kv_heads;
  pl.nt = group > 8 ? 2 : 1;
  pl.head_tiles = (group + 8 * pl.nt - 1) / (8 * pl.nt);
  // the longest part that still gives every SM a CTA
  const long long streams = static_cast<long long>(num_seqs) * num_kv_heads * pl.head_tiles;
  pl.part_tokens = kMinPartTokens;
  for (int pt : {1024, 512, 256}) {
    if (streams * ((max_ctx + pt - 1) / pt) >= device_sms()) {
      pl.part_tokens = pt;
      break;
    }
  }
  pl.max_parts = (max_ctx + pl.part_tokens - 1) / pl.part_tokens;
  return pl;
}

template <int D>
cudaError_t prepare_kernels() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(mu);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  constexpr int smem = NW * Ring<D>::WARP;
  e = cudaFuncSetAttribute(paged_attention_int4_kernel<D, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_attention_int4_kernel<D, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <int D>
int launch(Int4Params p, const Plan& pl, int num_seqs, void* ws, size_t ws_bytes, cudaStream_t st) {
  p.head_tiles = pl.head_tiles;
  p.part_tokens = pl.part_tokens;
  p.max_parts = pl.max_parts;
  if (p.max_parts > 1) {
    const size_t pairs = static_cast<size_t>(num_seqs) * p.num_heads * p.max_parts;
    const size_t need = (ws_ml_floats(pairs) + pairs * D) * sizeof(float);
    if (ws == nullptr || ws_bytes < need)
      return pkv::fail(PKV_ERR_WORKSPACE, "pkv_paged_attention_decode_int4: workspace of %zu bytes needed, %zu given",
                       need, ws == nullptr ? static_cast<size_t>(0) : ws_bytes);
    p.ws_ml = static_cast<float*>(ws);
    p.ws_o = p.ws_ml + ws_ml_floats(pairs);
  }
  const dim3 grid(p.max_parts, p.num_kv_heads * p.head_tiles, num_seqs);
  constexpr size_t smem = NW * Ring<D>::WARP;
  cudaError_t e = prepare_kernels<D>();
  if (e == cudaSuccess)
    e = pl.nt == 1 ? pkv::launch_pdl(paged_attention_int4_kernel<D, 1>, grid, dim3(NW * 32), smem, st, p)
                   : pkv::launch_pdl(paged_attention_int4_kernel<D, 2>, grid, dim3(NW * 32), smem, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess && p.max_parts > 1) {
    e = pkv::launch_pdl(paged_attention_int4_merge_kernel<D>, dim3((p.num_heads + 3) / 4, num_seqs), dim3(128), 0, st, p);
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  if (e != cudaSuccess)
    return pkv::fail(PKV_ERR_CUDA, "pkv_paged_attention_decode_int4 launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int read_device_error_attention_int4(int reset, int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_dev_error_attention_int4, sizeof(int));
  if (e == cudaSuccess && reset && v) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_dev_error_attention_int4, &zero, sizeof(int));
  }
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, "reading the four-bit attention's check word: %s", cudaGetErrorString(e));
  *code = v;
  return PKV_OK;
}
}  // namespace pkv

extern "C" {

size_t pkv_paged_attention_int4_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                               int max_blocks_per_seq, int block_size) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
      max_blocks_per_seq <= 0 || block_size <= 0 || static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return 0;
  const Plan pl = plan_for(num_seqs, num_heads, num_kv_heads, max_blocks_per_seq * block_size);
  if (pl.max_parts <= 1) return 0;
  const size_t pairs = static_cast<size_t>(num_seqs) * num_heads * pl.max_parts;
  return (ws_ml_floats(pairs) + pairs * head_dim) * sizeof(float);
}

int pkv_paged_attention_decode_int4(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                    int num_heads, int num_kv_heads, int head_dim, int num_blocks,
                                    int max_blocks_per_seq, float scale, int block_size, uint16_t* out,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "pkv_paged_attention_decode_int4";
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG,
                     "%s: num_seqs=%d num_heads=%d num_kv_heads=%d num_blocks=%d max_blocks_per_seq=%d", fn, num_seqs,
                     num_heads, num_kv_heads, num_blocks, max_blocks_per_seq);
  if (num_heads % num_kv_heads)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_heads=%d is not a multiple of num_kv_heads=%d", fn, num_heads,
                     num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: block_size %d not in {4, 8, 16, 32}", fn, block_size);
  if (num_seqs == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (num_seqs > 65535 || num_heads > 65535)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: num_seqs/num_heads above 65535", fn);
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: context capacity above 2^30 tokens", fn);
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q, caches, out, workspace must be 16-byte aligned", fn);
  if (!std::isfinite(scale)) return pkv::fail(PKV_ERR_INVALID_ARG, "%s: scale not finite", fn);
  Int4Params p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k = k_cache;
  p.v = v_cache;
  p.tables = block_tables;
  p.lens = context_lens;
  p.out = reinterpret_cast<__half*>(out);
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks_per_seq;
  while ((1 << p.log2_block) < block_size) ++p.log2_block;
  p.scale_log2 = scale * 1.4426950408889634f;
  const Plan pl = plan_for(num_seqs, num_heads, num_kv_heads, max_blocks_per_seq * block_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rc = head_dim == 128 ? launch<128>(p, pl, num_seqs, workspace, workspace_bytes, st)
                                 : launch<64>(p, pl, num_seqs, workspace, workspace_bytes, st);
  if (rc == PKV_OK) pkv::clear_error();
  return rc;
}

}  // extern "C"
