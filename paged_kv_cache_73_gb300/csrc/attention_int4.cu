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
// out the same, so a lane reads D/8 contiguous bytes.  For O^T a transposing matrix load takes
// V's rows as 16-bit elements: a lane gets tokens 2t, 2t + 1 of one element, that is of four
// values, in the two halves of a register.  Of the low bytes both half bytes are masked out; of the
// high bytes the low half is, and the whole byte enters as n + 16 n', whose n comes off in the
// end (byte permutes of row words and four masks took long grouped contexts 7 us more).
// P^T comes from S^T's accumulator by an 8x8 transpose in registers (movmatrix).
//
// Where each cached head has one query head, the products' other seven columns are idle, and
// so would be most of the softmax: a warp then deals the 32 logits of its one column out,
// one to a lane, and brings the weights back by one transpose and three shuffles (a fifth of
// the chunk's instructions saved).  Its second column takes what the weights' rounding to fp16
// left, which costs nothing there.
//
// Softmax in base 2 with a running maximum that moves only when a chunk raises it by
// more than 2^8.  The weight that multiplies V's whole numbers is u_t = p_t s_t, rounded
// to fp16; the maximum is kept over x_t + log2 of s_t's exponent, so that u is at most
// 2^9 and its greatest is a normal number whatever the rows' scales.  With u' = fp16(u),
//   sum p (s n + z) = sum u' (n - 8) + sum p (z + 8 s) + (rounding of u) (n - 8):
// the second sum is fp32, and sum u' comes from one more product, with ones, so that a
// weight's rounding meets n - 8 and not n.  Chunk by chunk 8 sum u' is taken off the running
// sum u' n, which so stays as small as the result.
//
// Every warp of a resident grid is a worker of its own.  The work is one line of chunks of
// 32 tokens, sequence after sequence and in each cached head after cached head, cut into
// equal pieces; a worker walks its piece through a ring in shared memory that 16-byte
// cp.async fill some chunks ahead, across the ends of streams.  (One CTA per part of a
// stream, with 1024 tokens each, lost a quarter of its time to starts: length, table and
// first rows are three round trips, with three CTAs to an SM to hide them.)  Where a
// stream is cut, its workers leave partial results that a second kernel joins by the
// log-sum-exp identity.
//
// Measured (D = 128): 64 sequences of 128 to 2048 tokens, 40 heads, 71 us = 5.3 TB/s of cached
// rows; 32 sequences of 8192 to 32768, 64 heads on 8, 118 us = 6.2 TB/s.  Copies alone take 94 and
// 96 % of that; one sequence of 2048 tokens, 40 heads, 10.8 us in a row of such calls, of which 7
// are there at 128 tokens too.  Small blocks cost: 64 sequences of 1088 tokens take 65 us with
// blocks of 32 tokens, 69 with 16 and 78 with 8 (tiles of 2176, 1088 and 544 bytes).
// Groups of 9 to 16 are held by the chain of a chunk, not by the copies: it takes 1.8 times as long as with
// 8 heads (twice the columns, and 108 to 132 bytes of spills at 168 registers) and twelve warps fill half of
// the issue slots; 32 sequences as above with 64 heads on 4 take 105 us of 54 for their bytes.  Above 16
// every 16 heads walk the rows again: 32 heads on one 62 us, 48 on one 84, of 13.5.
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

constexpr unsigned FULL = 0xffffffffu;
constexpr int NW = 12;                // warps on an SM, in one CTA; a small grid has CTAs of four
constexpr int CHUNK = 32;             // tokens a worker handles at a time
constexpr int kMinChunks = 4;         // chunks a worker takes at least
// Sixteen warps join a head's parts where there are at most kFewHeads heads in all and equal streams would be
// cut into more than kManyParts: one sequence of 131072 tokens, 8 heads on 1, 87 -> 21 us, 32 on 8, 55 -> 32;
// elsewhere one warp does: 8 sequences of 512 tokens, 40 heads, 16.5 us against 22.6, one of 128 9.4 against 10.5.
constexpr int kFewHeads = 256, kManyParts = 32;
constexpr float kRescale = 8.f;       // the running maximum moves when a chunk passes it by this much
constexpr float kLowest = -3.4028235e38f;  // its start: finite, so that a chunk without a live row gives weights of 0

struct Int4Params {
  const __half* q;
  const uint8_t* k;
  const uint8_t* v;
  const int32_t* tables;
  const int32_t* lens;
  __half* out;
  float* ws_ml;  // [slots, rows per tile, 2] (m, l), base-2 log domain
  float* ws_o;   // [slots, rows per tile, D] unnormalised partial outputs
  int num_seqs, num_heads, num_kv_heads, group, head_tiles;
  int num_blocks, max_blocks, log2_block;
  int workers;
  float scale_log2;
};

// How the line of chunks is laid out and cut, from the lengths: both kernels derive it alike.  A
// stream is one sequence's cached head (and tile of its query heads); worker w takes chunks
// [w per, (w + 1) per) of the line.  Slot w + stream is unique to that pair: along the line one of the
// two grows at every cut.
// AHEAD: read before the caller's wait for the kernels before it, and so from L2, where those that are done
// have left them.
template <bool AHEAD>
__device__ __forceinline__ int chunks_of(const Int4Params& p, int s) {
  const int len = s >= p.num_seqs ? 0 : AHEAD ? __ldcg(p.lens + s) : p.lens[s];
  return len <= 0 || len > (p.max_blocks << p.log2_block) ? 0 : (len + CHUNK - 1) / CHUNK;
}
__device__ __forceinline__ long long per_worker(long long total, int workers) {
  const long long per = (total + workers - 1) / workers;
  return per > kMinChunks ? per : kMinChunks;
}

__device__ __forceinline__ void mma16816(float (&c)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                         unsigned b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two fp32 sums in one instruction
__device__ __forceinline__ void add2(float& a, float& b, float2 x) {
  asm("{\n\t.reg .b64 ra, rx;\n\tmov.b64 ra, {%0, %1};\n\tmov.b64 rx, {%2, %3};\n\t"
      "add.rn.f32x2 ra, ra, rx;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x.x), "f"(x.y));
}
__device__ __forceinline__ unsigned transpose8x8(unsigned x) {
  unsigned y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// four 8x8 matrices of 16-bit elements, transposed: lane (g, t) gets rows 2t, 2t + 1 of column g of each
__device__ __forceinline__ void load_transposed(unsigned (&w)[4], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(row)
               : "memory");
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
// bytes = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// A ring stage: 32 tokens' K rows, V rows (XOR-ed), K and V (scale, zero) pairs.
template <int D>
struct Ring {
  static constexpr int ROW = D / 2;                 // bytes of a row's values
  static constexpr int V_OFF = CHUNK * ROW;
  static constexpr int META_OFF = 2 * CHUNK * ROW;
  static constexpr int STAGE = META_OFF + 2 * CHUNK * 4;
  static constexpr int NST = 3;
  static constexpr int WARP = NST * STAGE;          // a warp's ring
};
// Byte offset of 16-byte chunk c of V row r within a stage's V rows: in each 128-byte line (2 or 4
// rows) the chunk's place is XOR-ed with the line's number mod 4, so one chunk of eight rows lies in
// different banks.
template <int D>
__device__ __forceinline__ int v_place(int r, int c) {
  const int lin = r * (D / 32) + c, line = lin >> 3;
  return line * 128 + (((lin & 7) ^ (line & 3)) << 4);
}

// A worker's running softmax over one stream's tokens for 8 NT heads; lane (g, t) holds heads 8 n + 2t,
// 8 n + 2t + 1.  With a lone head (SOLO) m, l and c use [0][0]: m by all lanes alike, l and c for the one token
// of each chunk that a lane takes; acc and ones in lanes with t = 0 (columns 0 and 1: the weights
// and what their rounding left).
template <int D, int NT>
struct WarpState {
  float m[NT][2], l[NT][2], c[NT][2];   // l and c: this lane's tokens only, until the end
  // Value pair i: {even value, heads 2t, 2t + 1; 16 times the odd value, the same, plus the even one where i is
  // odd}, as sum u' (n - 8) over the chunks before the last and sum u' n over that.
  float acc[NT][D / 16][4];
  float ones[NT][4];                    // sum u' over the last chunk
};

// One chunk staged at `stage`.  live: the rows that count; the others (past the context, or of a block outside the
// pool) get no weight, whatever is there.
template <int D, int NT, bool SOLO>
__device__ __forceinline__ void chunk_update(const unsigned char* stage, unsigned live, const unsigned (&qf)[NT][D / 16][2],
                                             const float (&ca)[NT][2], const float (&cb)[NT][2], WarpState<D, NT>& st,
                                             int g, int t, uint32_t v_row) {
  using R = Ring<D>;
  constexpr int WK = D / 32;            // words of a K row per lane
  // the two tiles' products side by side: each is a chain of dependent accumulations
  unsigned kw[2][2][WK];
  float dot[2][NT][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    load_words<WK>(kw[i][0], stage + (16 * i + g) * R::ROW + t * (D / 8));
    load_words<WK>(kw[i][1], stage + (16 * i + g + 8) * R::ROW + t * (D / 8));
#pragma unroll
    for (int n = 0; n < NT; ++n) dot[i][n][0] = dot[i][n][1] = dot[i][n][2] = dot[i][n][3] = 0.f;
  }
#pragma unroll
  for (int w = 0; w < WK; ++w) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const unsigned a = kw[i][0][w] >> (8 * half), b = kw[i][1][w] >> (8 * half);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mma16816(dot[i][n], a & 0x000f000fu, b & 0x000f000fu, a & 0x00f000f0u, b & 0x00f000f0u,
                   qf[n][2 * w + half][0], qf[n][2 * w + half][1]);
      }
    }
  }
  unsigned pb[NT][2][2];                // P^T: tile i, rows 2t, 2t + 1 and those + 8
  if constexpr (SOLO) {
    // lane (g, t) takes the token of tile t / 2, row g + 8 (t % 2), whose dot lane (g, 0) holds
    const int from = 4 * g, row = 16 * (t >> 1) + g + 8 * (t & 1);
    const float d00 = __shfl_sync(FULL, dot[0][0][0], from), d01 = __shfl_sync(FULL, dot[0][0][2], from);
    const float d10 = __shfl_sync(FULL, dot[1][0][0], from), d11 = __shfl_sync(FULL, dot[1][0][2], from);
    const float d = t < 2 ? (t == 0 ? d00 : d01) : (t == 2 ? d10 : d11);
    const float2 km = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + row * 4));
    float2 vm = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + CHUNK * 4 + row * 4));
    float x = fmaf(km.x, ca[0][0] * d, km.y * cb[0][0]);
    if (!(live >> row & 1)) {
      vm = make_float2(0.f, 0.f);
      x = -INFINITY;
    }
    float top = x + log2_of(vm.x);
    if (__any_sync(FULL, top > st.m[0][0] + kRescale)) {
#pragma unroll
      for (int o = 1; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
      const float m = fmaxf(st.m[0][0], top), f = exp2f(st.m[0][0] - m);
      st.m[0][0] = m;
      st.l[0][0] *= f;
      st.c[0][0] *= f;
      st.ones[0][0] *= f;
      st.ones[0][1] *= f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.acc[0][i][j] *= f;
    }
    const float w = fast_exp2(x - st.m[0][0]);
    st.l[0][0] += w;
    st.c[0][0] = fmaf(w, fmaf(8.f, vm.x, vm.y), st.c[0][0]);
    // The weight in two halves, u' and what its rounding left: columns 0 and 1.  Transposed, lane (2k, t)
    // holds u' of rows 2t, 2t + 1 of the k-th eight tokens and lane (2k + 1, t) the rest; the products want
    // the four in lanes (0, t) and (1, t), and what other columns hold does not matter.
    const float u = w * vm.x;
    const __half hi = __float2half_rn(u), rest = __float2half_rn(u - __half2float(hi));
    const unsigned both = transpose8x8(static_cast<unsigned>(__half_as_ushort(hi)) | static_cast<unsigned>(__half_as_ushort(rest)) << 16);
    const int column = (4 * g + t) & 7;
    pb[0][0][0] = both;
    pb[0][0][1] = __shfl_sync(FULL, both, 8 + column);
    pb[0][1][0] = __shfl_sync(FULL, both, 16 + column);
    pb[0][1][1] = __shfl_sync(FULL, both, 24 + column);
  } else {
    float x[NT][2][4];                    // tile i, {token g: heads 2t, 2t + 1; token g + 8: the same}
    float2 vm[2][2];                      // V's scale and zero + 8 scale of those tokens
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * i + g + 8 * r;
        const float2 km = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + row * 4));
        vm[i][r] = __half22float2(*reinterpret_cast<const __half2*>(stage + R::META_OFF + CHUNK * 4 + row * 4));
        vm[i][r].y = fmaf(8.f, vm[i][r].x, vm[i][r].y);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            x[n][i][2 * r + j] = fmaf(km.x, ca[n][j] * dot[i][n][2 * r + j], km.y * cb[n][j]);
      }
    }
    if (const unsigned mine = live >> g; live != FULL) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (!(mine >> (16 * i + 8 * r) & 1)) {
            vm[i][r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n][i][2 * r] = x[n][i][2 * r + 1] = -INFINITY;
          }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float e = log2_of(vm[i][r].x);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) top[n][j] = fmaxf(top[n][j], x[n][i][2 * r + j] + e);
      }
    bool moves = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) moves |= top[n][j] > st.m[n][j] + kRescale;
    if (__any_sync(FULL, moves)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o *= 2) top[n][j] = fmaxf(top[n][j], __shfl_xor_sync(FULL, top[n][j], o));
          const float m = fmaxf(st.m[n][j], top[n][j]);
          const float f = exp2f(st.m[n][j] - m);
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
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float u[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float w = fast_exp2(x[n][i][2 * r + j] - st.m[n][j]);    // a NaN logit makes NaNs
            st.l[n][j] += w;
            u[j] = w * vm[i][r].x;
            st.c[n][j] = fmaf(w, vm[i][r].y, st.c[n][j]);
          }
          pb[n][i][r] = transpose8x8(pack2(u[0], u[1]));
        }
  }
  // The last chunk's sum u' n becomes sum u' (n - 8), late, when its products have long arrived.  Left in, the
  // 8 sum u' grew with the context while the result shrinks, and the tensor cores' sums, cut off at the
  // accumulator's last bit, cost 5.8e-4 of the result at 20 000 tokens where now 3.0e-4 are lost at any
  // length (2.1e-4 by the output's own rounding), for 3 us of long grouped contexts' 118.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 even = make_float2(st.ones[n][0] * -0x1p-21f, st.ones[n][1] * -0x1p-21f);
    const float2 odd = make_float2(st.ones[n][0] * -0x1p-17f, st.ones[n][1] * -0x1p-17f);
    const float2 both = make_float2(even.x + odd.x, even.y + odd.y);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      add2(st.acc[n][i][0], st.acc[n][i][1], even);
      add2(st.acc[n][i][2], st.acc[n][i][3], i & 1 ? both : odd);
    }
    st.ones[n][0] = st.ones[n][1] = st.ones[n][2] = st.ones[n][3] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int pair = 0; pair < D / 64; ++pair) {              // 16-byte chunks 2 pair, 2 pair + 1 of the rows
      unsigned v[4];                                         // of each: tokens 2t, 2t + 1, then those + 8
      load_transposed(v, v_row + i * 16 * R::ROW ^ pair * 32);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // the low bytes' halves apart; of the high bytes the low half and the whole (which holds 17 n at most)
          const unsigned e = h ? __byte_perm(v[2 * c], 0, 0x4341) : v[2 * c];
          const unsigned f = h ? __byte_perm(v[2 * c + 1], 0, 0x4341) : v[2 * c + 1];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma16816(st.acc[n][4 * pair + 2 * c + h], e & 0x000f000fu, h ? e : e & 0x00f000f0u, f & 0x000f000fu,
                     h ? f : f & 0x00f000f0u, pb[n][i][0], pb[n][i][1]);
        }
    }
    constexpr unsigned kOne2 = 0x3c003c00u;
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16816(st.ones[n], kOne2, kOne2, kOne2, kOne2, pb[n][i][0], pb[n][i][1]);
  }
}

// A place on the line of chunks: chunk c of the `chunks` of stream (s, y).
struct Place {
  int s, y, c, chunks, len;
};

template <int D, int NT, bool SOLO, int LB>
__global__ void __launch_bounds__(NW * 32, 1) paged_attention_int4_kernel(const Int4Params p) {
  using R = Ring<D>;
  constexpr int HT = 8 * NT, WK = D / 32, ROW = R::ROW, B = 1 << LB;
  constexpr int PIECES = CHUNK * ROW / 16 / 32;              // 16-byte pieces of K, and of V, per lane and chunk
  constexpr int RPP = 512 / ROW;                             // rows that one piece of every lane covers
  constexpr int BPC = CHUNK / B;                             // blocks per chunk
  extern __shared__ __align__(128) unsigned char smem[];     // the workers' rings

  // Every thread waits before it triggers, unlike in the other kernels: the joining kernel, launched next, may
  // start once all of this grid has triggered, and reads the lengths before it waits for this grid.  The
  // kernels before this one are done by then, so the lengths are there.
  pkv::pdl_wait();
  pkv::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int worker = warp * gridDim.x + blockIdx.x;
  const int S = p.num_seqs, H = p.num_heads, Y = p.num_kv_heads * p.head_tiles;

  // this worker's piece of the line
  Place at;
  int left;
  {
    long long total = 0;
    bool bad = false;
    for (int s = lane; s < S; s += 32) {
      total += chunks_of<false>(p, s);
      bad |= p.lens[s] < 0 || p.lens[s] > (p.max_blocks << LB);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) total += __shfl_xor_sync(FULL, total, o);
    if (bad && worker == 0) record_error(PKV_DEV_BAD_CONTEXT_LEN);
    const long long n = total * Y, per = per_worker(n, p.workers), x = worker * per;
    if (x >= n) return;
    left = static_cast<int>(min(per, n - x));
    // the sequence: the first whose chunks, all heads together, reach past x
    long long before = 0;
    int s = S, mine = 0;
    for (int base = 0; base < S; base += 32) {
      mine = chunks_of<false>(p, base + lane);
      long long upto = mine;                                 // inclusive prefix sum over the lanes
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(FULL, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned past = __ballot_sync(FULL, (before + upto) * Y > x);
      if (past) {
        const int hit = __ffs(past) - 1;
        s = base + hit;
        before += __shfl_sync(FULL, upto - mine, hit);
        mine = __shfl_sync(FULL, mine, hit);
        break;
      }
      before += __shfl_sync(FULL, upto, 31);
    }
    if (s >= S) return;                                      // the lengths changed meanwhile
    const long long rest = x - before * Y;
    at.s = s;
    at.y = static_cast<int>(rest / mine);
    at.c = static_cast<int>(rest - static_cast<long long>(at.y) * mine);
    at.chunks = mine;
    at.len = p.lens[s];
  }
  auto advance = [&](Place& x) {                             // true if the stream changed
    if (++x.c < x.chunks) return false;
    x.c = 0;
    if (++x.y == Y) {
      x.y = 0;
      do ++x.s, x.chunks = chunks_of<false>(p, x.s);
      while (x.chunks == 0 && x.s < S);
      x.len = x.s < S ? p.lens[x.s] : 0;
    }
    return true;
  };

  // ---- the ring: a lane copies the same pieces of every chunk
  unsigned char* ring = smem + warp * R::WARP;
  const uint32_t ring_u32 = smem_u32(ring);
  const int tile_bytes = (ROW + 4) * B, block_bytes = p.num_kv_heads * tile_bytes;
  const int piece_row = lane / (ROW / 16);                   // piece i: row RPP i + piece_row
  const int piece_col = lane % (ROW / 16) * 16;
  const int v_lane = R::V_OFF + v_place<D>(piece_row, lane % (ROW / 16));
  const int meta_row = 4 * (lane & 7);
  Place ahead = at;
  int to_fill = left;
  // table entries of 32 blocks around `ahead`, one a lane, and of the next 32; -1 past the context, -2 bad
  int entry = -1, entry_next = -1;
  auto read_entry = [&](int first) {
    const int j = first + lane;
    if (j * static_cast<long long>(B) >= ahead.len) return -1;
    const int phys = p.tables[static_cast<size_t>(ahead.s) * p.max_blocks + j];
    if (phys >= 0 && phys < p.num_blocks) return phys;
    record_error(PKV_DEV_BAD_BLOCK_ID);
    return -2;
  };
  unsigned gone = 0;                                         // per stage eight bits: its chunk's bad blocks
  bool fresh = true;                                         // `ahead` is at a stream's first chunk here
  int head_off = 0;                                          // of `ahead`'s cached head in a block
  const uint8_t* meta_src = (lane & 8 ? p.v : p.k) + ROW * B + (meta_row % B) * 4;
  auto fill = [&](int stage) {
    if (to_fill > 0) {
      const int blk = ahead.c * BPC, first = blk & ~31;
      if (fresh) {
        entry = read_entry(first);
        entry_next = read_entry(first + 32);
        head_off = ahead.y / p.head_tiles * tile_bytes;
        // its queries, for when the products come to it
        const int in_group = ahead.y % p.head_tiles * HT, h0 = ahead.y / p.head_tiles * p.group + in_group;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n * 8 + g < min(HT, p.group - in_group))
            asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + (static_cast<size_t>(ahead.s) * H + h0 + n * 8 + g) * D + t * (D / 4)));
        fresh = false;
      } else if (blk == first) {
        entry = entry_next;
        entry_next = read_entry(first + 32);
      }
      gone = (gone & ~(0xffu << 8 * stage)) | (__ballot_sync(FULL, entry == -2) >> (blk & 31) & ((1u << BPC) - 1)) << 8 * stage;
      const int valid = ahead.len - ahead.c * CHUNK;
      const uint32_t dst = ring_u32 + stage * R::STAGE;
      // pieces of one block (or of one pair of blocks, a half of the lanes each) share an address
      constexpr int PPB = B * ROW / 512 > 0 ? B * ROW / 512 : 1;
#pragma unroll
      for (int i0 = 0; i0 < PIECES; i0 += PPB) {
        const int row0 = RPP * i0 + piece_row;
        const int phys = __shfl_sync(FULL, entry, (blk & 31) + row0 / B);
        const int bytes = phys >= 0 ? 16 : 0;                // nothing of a bad block is read
        const int64_t off = static_cast<int64_t>(max(phys, 0)) * block_bytes + (head_off + (row0 % B) * ROW + piece_col);
        const uint8_t* ks = p.k + off;
        const uint8_t* vs = p.v + off;
#pragma unroll
        for (int i = i0; i < i0 + PPB; ++i) {
          if (RPP * i + piece_row < valid) {
            cp_async16(dst + lane * 16 + i * 512, ks + (i - i0) * 512, bytes);
            cp_async16(dst + v_lane + i * 512, vs + (i - i0) * 512, bytes);
          }
        }
      }
      {
        const int phys = __shfl_sync(FULL, entry, (blk & 31) + meta_row / B);
        if (lane < 16 && meta_row < valid)
          cp_async16(dst + R::META_OFF + lane * 16,
                     meta_src + (static_cast<int64_t>(max(phys, 0)) * block_bytes + head_off), phys >= 0 ? 16 : 0);
      }
      --to_fill;
      fresh = advance(ahead);
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
  WarpState<D, NT> st;
  auto begin_stream = [&]() {
    const int in_group = at.y % p.head_tiles * HT, h0 = at.y / p.head_tiles * p.group + in_group;
    const int nh = min(HT, p.group - in_group);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float qv[WK][8];
      float amax = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (n * 8 + g < nh)
          raw = *reinterpret_cast<const uint4*>(p.q + (static_cast<size_t>(at.s) * H + h0 + n * 8 + g) * D + t * (D / 4) + w * 8);
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
        ca[n][j] = __shfl_sync(FULL, a, SOLO ? 0 : (2 * t + j) * 4);
        cb[n][j] = __shfl_sync(FULL, b, SOLO ? 0 : (2 * t + j) * 4);
        st.m[n][j] = kLowest;
        st.l[n][j] = st.c[n][j] = 0.f;
        st.ones[n][j] = st.ones[n][2 + j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) st.acc[n][i][j] = 0.f;
    }
  };
  // the stream's result, or this worker's part of it: lane (g, t) holds values 32 k + 4 g .. of heads 2t, 2t + 1
  auto end_stream = [&](bool whole) {
    const int in_group = at.y % p.head_tiles * HT, h0 = at.y / p.head_tiles * p.group + in_group;
    const int nh = min(HT, p.group - in_group), rows = min(HT, p.group);
    const size_t slot = static_cast<size_t>(worker) + static_cast<size_t>(at.s) * Y + at.y;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < (SOLO ? 1 : 2); ++j) {
#pragma unroll
        for (int o = SOLO ? 1 : 4; o < 32; o *= 2) {
          st.l[n][j] += __shfl_xor_sync(FULL, st.l[n][j], o);
          st.c[n][j] += __shfl_xor_sync(FULL, st.c[n][j], o);
        }
        const int h = n * 8 + 2 * t + j;
        if (h >= nh) continue;
        if constexpr (SOLO) {                                // the weights' two halves
          st.ones[0][0] += st.ones[0][1];
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            st.acc[0][i][0] += st.acc[0][i][1];
            st.acc[0][i][2] += st.acc[0][i][3];
          }
        }
        const float mid = fmaf(-8.f, st.ones[n][j], st.c[n][j]);
        float o[D / 8];                                      // o[4 k ..]: values 32 k + 4 g ..
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[2 * i] = fmaf(st.acc[n][i][j], 16777216.f, mid);
          o[2 * i + 1] = fmaf(st.acc[n][i][2 + j] - (i & 1 ? st.acc[n][i][j] : 0.f), 1048576.f, mid);
        }
        if (whole) {
          const float inv = st.l[n][j] == 0.f ? 0.f : 1.f / st.l[n][j];   // 0: every block is bad
          __half* dst = p.out + (static_cast<size_t>(at.s) * H + h0 + h) * D + g * 4;
#pragma unroll
          for (int i = 0; i < D / 8; i += 4)
            *reinterpret_cast<uint2*>(dst + 8 * i) = make_uint2(pack2(o[i] * inv, o[i + 1] * inv), pack2(o[i + 2] * inv, o[i + 3] * inv));
        } else {
          const size_t w = slot * rows + h;
          float* dst = p.ws_o + w * D + g * 4;
#pragma unroll
          for (int i = 0; i < D / 8; i += 4)
            *reinterpret_cast<float4*>(dst + 8 * i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          if (g == 0) *reinterpret_cast<float2*>(p.ws_ml + 2 * w) = make_float2(st.m[n][j], st.l[n][j]);
        }
      }
  };

  // the V row and chunk whose address this lane gives: matrices are (first, second eight tokens) of a chunk,
  // then of the next
  const uint32_t v_row = ring_u32 + R::V_OFF + v_place<D>((lane & 8) + (lane & 7), lane >> 4);
  bool from_start = at.c == 0;
  begin_stream();
  int stage = 0;
  for (; left > 0; --left) {
    cp_async_wait<R::NST - 2>();
    __syncwarp();                                            // every lane's copies; and the last stage is read
    fill(stage == 0 ? R::NST - 1 : stage - 1);
    const unsigned char* src = ring + stage * R::STAGE;
    const int valid = at.len - at.c * CHUNK;
    // the rows before the context's end, of blocks that are in the pool
    unsigned live = valid < CHUNK ? (1u << valid) - 1 : FULL;
    for (unsigned bad = gone >> 8 * stage & 0xffu; bad; bad &= bad - 1) live &= ~((FULL >> (32 - B)) << (__ffs(bad) - 1) * B);
    chunk_update<D, NT, SOLO>(src, live, qf, ca, cb, st, g, t, v_row + stage * R::STAGE);
    if (++stage == R::NST) stage = 0;
    const bool to_end = at.c + 1 == at.chunks;
    if (to_end || left == 1) {
      end_stream(from_start && to_end);
      from_start = true;
      if (left > 1) {
        advance(at);
        begin_stream();
      }
    } else {
      ++at.c;
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of every cut stream, and writes the zeros of empty contexts: WPH warps per (sequence,
// head), a lane D/32 values.  Where there are few heads in all, each may have been cut into a thousand
// parts, and sixteen warps share them.  The lengths are read before the wait: this kernel's launch has to
// follow that of paged_attention_int4_kernel, whose every thread waits for the kernels before it and then
// triggers; no other kernel may come between the two.
template <int D, int WPH>
__global__ void __launch_bounds__(WPH == 1 ? 128 : WPH * 32) paged_attention_int4_merge_kernel(const Int4Params p, int head_rows) {
  constexpr int WARPS = WPH == 1 ? 4 : WPH, FLY = 8;         // warps of a CTA; parts in flight to a warp
  pkv::pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = WPH == 1 ? blockIdx.x * 4 + warp : blockIdx.x, s = blockIdx.y;
  // chunks of the sequences before s, and of all
  long long mine[2] = {0, 0};
  for (int i = threadIdx.x; i < p.num_seqs; i += WARPS * 32) {
    const int c = chunks_of<true>(p, i);
    mine[1] += c;
    if (i < s) mine[0] += c;
  }
  __shared__ long long sums[WARPS][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mine[k] += __shfl_xor_sync(FULL, mine[k], o);
    if (lane == 0) sums[warp][k] = mine[k];
  }
  __syncthreads();
  if (h >= p.num_heads) {
    pkv::pdl_wait();
    return;
  }
  long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    before += sums[i][0];
    total += sums[i][1];
  }
  constexpr int V = D / 32;
  __half* dst = p.out + (static_cast<size_t>(s) * p.num_heads + h) * D + lane * V;
  const int chunks = chunks_of<true>(p, s);
  const int Y = p.num_kv_heads * p.head_tiles, tile = h % p.group / head_rows;
  const int y = h / p.group * p.head_tiles + tile, row = h % p.group - tile * head_rows;
  const long long first = before * Y + static_cast<long long>(y) * chunks;
  const long long per = per_worker(total * Y, p.workers), w_first = first / per, w_last = (first + chunks - 1) / per;
  pkv::pdl_wait();                                           // the parts
  if (chunks == 0) {
    if (WPH == 1 || warp == 0) {
#pragma unroll
      for (int c = 0; c < V; c += 2) *reinterpret_cast<__half2*>(dst + c) = __floats2half2_rn(0.f, 0.f);
    }
    return;
  }
  if (w_first == w_last) return;                             // one worker wrote it
  const int all = static_cast<int>(w_last - w_first) + 1, rows = min(head_rows, p.group);
  // this warp's parts
  const int share = (all + WPH - 1) / WPH, part0 = WPH == 1 ? 0 : warp * share, nparts = min(share, all - part0);
  const size_t slot0 = static_cast<size_t>(w_first) + part0 + static_cast<size_t>(s) * Y + y;
  auto at = [&](int i) { return (slot0 + i) * rows + row; };  // part i's row of the workspace
  // (m, l) of 32 slots at a time, one a lane; then some slots' outputs in flight at a time
  float acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
  float M = -INFINITY, L = 0.f;
  for (int base = 0; base < nparts; base += 32) {
    const int i = base + lane;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (i < nparts) ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * at(i));
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    m = fmaxf(M, m);
    const float carry = M == -INFINITY ? 0.f : exp2f(M - m);
    M = m;
    L *= carry;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= carry;
    const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
    L = fmaf(ml.y, f, L);
    const int n = min(32, nparts - base);
    for (int j0 = 0; j0 < n; j0 += FLY) {
      float x[FLY][V];
#pragma unroll
      for (int u = 0; u < FLY; ++u) {
#pragma unroll
        for (int c = 0; c < V; ++c) x[u][c] = 0.f;
        if (j0 + u < n) {
          const float* src = p.ws_o + at(base + j0 + u) * D + lane * V;
          if constexpr (V == 4) {
            const float4 z = *reinterpret_cast<const float4*>(src);
            x[u][0] = z.x; x[u][1] = z.y; x[u][2] = z.z; x[u][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(src);
            x[u][0] = z.x; x[u][1] = z.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < FLY; ++u) {
        const float fu = __shfl_sync(FULL, f, (j0 + u) & 31);
        if (j0 + u < n) {
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(x[u][c], fu, acc[c]);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) L += __shfl_xor_sync(FULL, L, o);
  if constexpr (WPH > 1) {
    __shared__ float warp_m[WPH], warp_l[WPH];
    __shared__ __align__(16) float warp_o[WPH][D];
    if (lane == 0) {
      warp_m[warp] = M;
      warp_l[warp] = L;
    }
#pragma unroll
    for (int c = 0; c < V; ++c) warp_o[warp][lane * V + c] = acc[c];
    __syncthreads();
    if (warp != 0) return;
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < WPH; ++i) M = fmaxf(M, warp_m[i]);
    L = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll
    for (int i = 0; i < WPH; ++i) {
      const float f = warp_m[i] == -INFINITY ? 0.f : exp2f(warp_m[i] - M);
      L = fmaf(warp_l[i], f, L);
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(warp_o[i][lane * V + c], f, acc[c]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int c = 0; c < V; c += 2) *reinterpret_cast<__half2*>(dst + c) = __floats2half2_rn(acc[c] * inv, acc[c + 1] * inv);
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
// once for both).  One CTA of twelve warps to an SM, or, where even the longest contexts would not give
// each of those kMinChunks chunks, as many CTAs of four warps as that takes (smaller CTAs start sooner:
// 1.9 us less for one sequence of 2048 tokens and 40 heads).
struct Plan {
  int nt, head_tiles, head_rows, ctas, warps;
  long long slots, most_chunks;
};
Plan plan_for(int num_seqs, int num_heads, int num_kv_heads, int max_ctx) {
  Plan pl{};
  const int group = num_heads / num_kv_heads;
  pl.nt = group > 8 ? 2 : 1;
  pl.head_tiles = (group + 8 * pl.nt - 1) / (8 * pl.nt);
  pl.head_rows = group < 8 * pl.nt ? group : 8 * pl.nt;
  const long long streams = static_cast<long long>(num_seqs) * num_kv_heads * pl.head_tiles;
  pl.most_chunks = streams * ((max_ctx + CHUNK - 1) / CHUNK);
  const long long workers = (pl.most_chunks + kMinChunks - 1) / kMinChunks, sms = device_sms();
  const bool full = workers >= sms * NW;
  pl.warps = full ? NW : 4;
  pl.ctas = static_cast<int>(full ? sms : (workers + 3) / 4);
  pl.slots = streams + static_cast<long long>(pl.ctas) * pl.warps;
  return pl;
}
size_t workspace_bytes_for(const Plan& pl, int head_dim) {
  const size_t rows = static_cast<size_t>(pl.slots) * pl.head_rows;
  return (ws_ml_floats(rows) + rows * head_dim) * sizeof(float);
}

template <int D, int NT, bool SOLO, int LB>
cudaError_t launch_kernel(const Int4Params& p, const Plan& pl, cudaStream_t st) {
  constexpr int smem = NW * Ring<D>::WARP;
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> g(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(paged_attention_int4_kernel<D, NT, SOLO, LB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  e = pkv::launch_pdl(paged_attention_int4_kernel<D, NT, SOLO, LB>, dim3(pl.ctas), dim3(pl.warps * 32),
                      static_cast<size_t>(pl.warps) * Ring<D>::WARP, st, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <int D, int NT, bool SOLO>
cudaError_t launch_block_size(const Int4Params& p, const Plan& pl, cudaStream_t st) {
  switch (p.log2_block) {
    case 2: return launch_kernel<D, NT, SOLO, 2>(p, pl, st);
    case 3: return launch_kernel<D, NT, SOLO, 3>(p, pl, st);
    case 4: return launch_kernel<D, NT, SOLO, 4>(p, pl, st);
    default: return launch_kernel<D, NT, SOLO, 5>(p, pl, st);
  }
}

template <int D>
int launch(Int4Params p, const Plan& pl, void* ws, size_t ws_bytes, cudaStream_t st) {
  p.head_tiles = pl.head_tiles;
  p.workers = pl.ctas * pl.warps;
  const size_t need = workspace_bytes_for(pl, D);
  if (ws == nullptr || ws_bytes < need)
    return pkv::fail(PKV_ERR_WORKSPACE, "pkv_paged_attention_decode_int4: workspace of %zu bytes needed, %zu given", need,
                     ws == nullptr ? static_cast<size_t>(0) : ws_bytes);
  p.ws_ml = static_cast<float*>(ws);
  p.ws_o = p.ws_ml + ws_ml_floats(static_cast<size_t>(pl.slots) * pl.head_rows);
  cudaError_t e = p.group == 1 ? launch_block_size<D, 1, true>(p, pl, st)
                  : pl.nt == 1 ? launch_block_size<D, 1, false>(p, pl, st) : launch_block_size<D, 2, false>(p, pl, st);
  if (e == cudaSuccess) {
    const long long streams = static_cast<long long>(p.num_seqs) * p.num_kv_heads * p.head_tiles;
    if (static_cast<long long>(p.num_heads) * p.num_seqs <= kFewHeads && p.workers > kManyParts * streams)
      e = pkv::launch_pdl(paged_attention_int4_merge_kernel<D, 16>, dim3(p.num_heads, p.num_seqs), dim3(512), 0, st, p,
                          pl.head_rows);
    else
      e = pkv::launch_pdl(paged_attention_int4_merge_kernel<D, 1>, dim3((p.num_heads + 3) / 4, p.num_seqs), dim3(128), 0,
                          st, p, pl.head_rows);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess)
    return pkv::fail(PKV_ERR_CUDA, "pkv_paged_attention_decode_int4 launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int device_error_word_attention_int4(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_attention_int4));
}
}  // namespace pkv

extern "C" {

size_t pkv_paged_attention_int4_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                               int max_blocks_per_seq, int block_size) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
      max_blocks_per_seq <= 0 || block_size <= 0 || static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return 0;
  return workspace_bytes_for(plan_for(num_seqs, num_heads, num_kv_heads, max_blocks_per_seq * block_size), head_dim);
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
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks_per_seq;
  while ((1 << p.log2_block) < block_size) ++p.log2_block;
  p.scale_log2 = scale * 1.4426950408889634f;
  const Plan pl = plan_for(num_seqs, num_heads, num_kv_heads, max_blocks_per_seq * block_size);
  if (pl.most_chunks / (pl.ctas * pl.warps) >= (1LL << 30))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^30 chunks of %d tokens per warp", fn, CHUNK);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rc = head_dim == 128 ? launch<128>(p, pl, workspace, workspace_bytes, st)
                                 : launch<64>(p, pl, workspace, workspace_bytes, st);
  if (rc == PKV_OK) pkv::clear_error();
  return rc;
}

}  // extern "C"
