// Attention of drafted tokens over a paged fp16 cache, for sm_103a: each sequence's new tokens, a
// chain or a tree, see its context and those of each other that their mask rows name; groups of
// query heads share a cached head.
//
//   o_i = sum_t softmax_t(scale q_i . k_t) v_t   over t < ctx - n and t = ctx - n + j, bit j of row i set
//
// The n new tokens' G query heads of one cached head are the rows of one product: n G rows over
// the same keys, each cached row read once for all of them.  So it is bound by the cache's
// bytes up to about 256 rows (4 D flops a row and key against 4 D bytes a key), and
// the products run on the tensor cores from one row on: a tile of 128 rows costs 1024 clocks per 128 keys of
// D = 128 however few are real, while their 64 KB take an SM 2800 at the copy rate.
//
//  * A stream is one sequence's cached head and tile of 128 rows.  All streams' key tiles (64 positions)
//    lie on one line, cut evenly over the resident CTAs, two to an SM, each with half of the tensor memory: ragged
//    contexts and few sequences fill the GPU alike.  A CTA walks its piece through a ring of K and V tiles
//    that runs on over the ends of streams.
//  * Where a sequence has more than 128 rows, two CTAs walk two row tiles over the same keys at the same time, so
//    that the second reads from L2 what the first brought there; one after the other they read 2 x from memory (32
//    sequences of 20480 tokens, 64 heads on 8, 32 drafts: 791 us against 580).  Every row tile walks all of its
//    sequence's key tiles, without a mask too: 4096 new tokens over none compute twice what they need.
//  * A stream that is cut leaves partial results (row maximum, sum, output) that a second kernel joins by the
//    log-sum-exp identity; the first CTA of such a stream notes where they lie.  A CTA has at most
//    two such parts, the first and the last of its piece.
//  * K and V blocks come by TMA (one box per block and 64 columns) into the 128-byte swizzle.  V tiles
//    that some row does not see whole (drafts, the context's end) are looked over in shared memory before their
//    product: a masked weight of 0 times a value that is not finite would be a NaN, so such values of
//    drafts become zeros, are noted, and put back in the end for the rows that see them.
//  * Softmax as in prompt attention: a thread owns a row (a lane of tensor memory); the maximum, and with
//    it O, moves only when a tile passes it by 2^8; weights are 2^(7 + S - m) as fp16, so that those
//    lost below fp16's smallest are 2^-32 of the largest; sums are fp32 over the rounded weights.  The
//    result is off by 2.9e-4 in the 2-norm so, 2.1e-4 from the output's own rounding alone.  Weights in two fp16 halves
//    would not, but times an infinite value of V the halves give a NaN, and long contexts take 230 -> 234 us, wide trees of
//    D = 64 42 -> 49, 256 short sequences of one token 69 -> 87 or more, 256 rows 580 -> 779.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "launch.cuh"
#include "pkv_internal.h"
#include "tcgen05.cuh"

namespace {

__device__ int g_dev_error_tree_attention = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_tree_attention, 0, code); }

using namespace pkv::tc;

constexpr int BM = 128;            // rows of a product (MMA M)
constexpr int BN = 64;             // key positions per tile
// Key tiles a CTA takes at least: one sequence of 128 tokens and 40 heads takes 8.5 us with two, 9.9 with one (a
// second CTA to start for each), 11.2 with three.
constexpr int kMinTiles = 2;
// What a stream costs besides its key tiles, in key tiles: 16 wide trees over 276 to 4608 tokens (D = 64) take 49.5 us
// with 2, 45.0 with 4 and with 6; one sequence of 2048 tokens 16.1, 16.6 and 17.4.
constexpr int kStart = 4;
// Where streams are cut into more parts than this (by the longest contexts), a CTA joins four columns of one, with groups of
// threads to share the parts: one sequence of 16384 tokens, 32 heads on 8 (38 parts) 20.6 -> 17.8 us, of 131072 on one
// head (304) 66 -> 27; one of 2048 with 40 heads (8 parts) would go from 16.7 to 36.5, for so many CTAs are launched.
constexpr int kManyParts = 16;
constexpr float kRescale = 8.f;    // the running maximum moves when a tile passes it by this much
constexpr float kLift = 7.f;       // weights are kept as 2^(kLift + S - m)

// A cut stream, as its first CTA notes it for the joining kernel (parts 0: none).
struct Cut {
  int parts, slot;                 // parts lie in slots slot, then 2 (w + 1), 2 (w + 2), .. of the CTAs that follow
  int next;                        // the second part's slot
  int rows, first_row, q0, kv_head, pad;
};

struct TreeParams {
  CUtensorMap tmap_k, tmap_v;      // pools as (D, Hk B, num_blocks), boxes of 64 x B x 1, 128-byte swizzle
  const __half* q;
  const __half* k;
  const __half* v;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* qstart;
  const uint32_t* mask;
  __half* out;
  float2* ws_ml;                   // [2 workers][BM] (m, l), base-2 log domain
  float* ws_o;                     // [2 workers][D][BM] unnormalised outputs
  Cut* cuts;                       // [workers]
  int64_t q_stride;
  int mask_words, num_seqs, total_q, max_query_len;
  int num_heads, num_kv_heads, group, num_blocks, max_blocks, log2_block;
  int use_tma, out_sectors, workers;
  float scale_log2;
};

// One sequence's share of the line: kStart places that hold no work and `tiles` key tiles for each of its
// num_kv_heads * row_tiles streams.
struct Seq {
  int ctx, n, q0, tiles, row_tiles;
};
__device__ __forceinline__ Seq make_seq(const TreeParams& p, int ctx, int q0, int q1, int* code) {
  Seq x{ctx, q1 - q0, q0, 0, 0};
  if (x.n == 0) return x;
  if (x.ctx < 0 || x.ctx > (p.max_blocks << p.log2_block)) {
    *code = PKV_DEV_BAD_CONTEXT_LEN;
    return x;
  }
  if (x.n < 0 || x.n > x.ctx || x.n > p.max_query_len || x.q0 < 0 || x.q0 > p.total_q - x.n) {
    *code = PKV_DEV_BAD_QUERY_RANGE;
    return x;
  }
  x.tiles = (x.ctx + BN - 1) / BN;
  x.row_tiles = (x.n * p.group + BM - 1) / BM;
  return x;
}
__device__ __forceinline__ Seq seq_of(const TreeParams& p, int s, int* code) {
  return s < p.num_seqs ? make_seq(p, p.lens[s], p.qstart[s], p.qstart[s + 1], code) : Seq{0, 0, 0, 0, 0};
}
// Streams of a kind to a cached head: pairs of row tiles, row tiles left alone by those, or (kind ALL) every row tile.
enum Kind { ALL, PAIRS, ALONE };
__device__ __forceinline__ int streams_of(const Seq& x, Kind kind) {
  return kind == ALL ? x.row_tiles : kind == PAIRS ? x.row_tiles / 2 : x.row_tiles % 2;
}
__device__ __forceinline__ long long places_of(const Seq& x, int kv_heads, Kind kind) {
  return static_cast<long long>(x.tiles + kStart) * streams_of(x, kind) * kv_heads;
}

// QR: rows of Q that are held (a multiple of 32, the most that an item has); the product's other rows read what
// lies behind them, and depend on nothing else.
template <int D, int QR>
struct Cfg {
  static constexpr int Q_BYTES = QR * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  // ring slots for K and V: as many as two CTAs' shared memory holds
  static constexpr int NK = D == 64 ? 5 : QR == 32 ? 3 : 2;
  static constexpr int NV = D == 64 ? 6 : QR == 128 ? 2 : 3;
  // S buffers: with three S(j + 1) need not wait for PV(j - 1) (16 wide trees of D = 64, 45.0 -> 44.0 us)
  static constexpr int NB = D == 64 ? 3 : 2;
  static constexpr int BARS = 1024;
  static constexpr int BYTES = 1024 + Q_BYTES + (NK + NV) * KV_BYTES + BARS;
  // so much that no third CTA, which would wait for tensor memory, fits an SM
  static constexpr int SMEM = BYTES > 80 * 1024 ? BYTES : 80 * 1024;
  static_assert(SMEM <= 113 * 1024 && BM * D * 2 <= Q_BYTES + (NK + NV) * KV_BYTES, "two to an SM; a product's rows lie inside");
};
// Tensor memory: the O accumulator (D columns) and as many S buffers of 64 columns as a half of the SM's 512
// columns has room for.
constexpr uint32_t TMEM_COLS = 256;
constexpr int W_K = 4, W_V = 5, W_S = 6, W_PV = 7;            // warps 0 to 3: softmax
constexpr int THREADS = 256;
constexpr int NI = 2;                                         // items that may be on their way (four or eight change nothing)

// What a CTA does at a time: key tiles [tile0, tile0 + n_tiles) of one stream; n_tiles 0 ends the loop.
struct Item {
  int s, kv_head, first_row, rows, tile0, n_tiles, ctx, n, q0, slot;  // slot -1: the whole stream, to out
};

// 4-byte async copy global -> shared
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Divisions on the line: 64-bit ones take some 500 clocks, and few lines are that long.
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

__device__ __forceinline__ bool finite16(unsigned h) { return (h & 0x7c00u) != 0x7c00u; }

// Sixteen fp16 values to out: one 32-byte store where out's rows are whole sectors, else two of 16.
__device__ __forceinline__ void store16(__half* dst, const uint32_t (&w)[8], bool sectors) {
  if (sectors) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A wait for the phase of `parity`, false once another role has raised the abort flag or after 2^19
// tries (2 s: a failed try takes 3.9 us).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait_parity(bar, parity); ++i)
    if ((i & 1023u) == 0 && (*abort_flag != 0 || i >= (1u << 19))) return false;
  return true;
}

// Which of the positions key0 .. key0 + 63 node i sees, those before the drafts (at first_new and on) all.
__device__ __forceinline__ uint64_t seen_from(const TreeParams& p, int q_row, int i, int key0, int first_new) {
  const int j0 = key0 - first_new;
  if (j0 <= -BN) return ~0ull;
  if (p.mask == nullptr) {
    const int count = i + 1 - j0;
    return count <= 0 ? 0 : count >= 64 ? ~0ull : (1ull << count) - 1;
  }
  const uint32_t* row = p.mask + static_cast<int64_t>(q_row) * p.mask_words;
  auto word = [&](int w) { return w < p.mask_words ? row[w] : 0u; };
  if (j0 < 0) return ((static_cast<uint64_t>(word(1)) << 32 | word(0)) << -j0) | ((1ull << -j0) - 1);
  const int w = j0 >> 5, sh = j0 & 31;
  const uint32_t x0 = word(w), x1 = word(w + 1), x2 = word(w + 2);
  return static_cast<uint64_t>(__funnelshift_r(x1, x2, sh)) << 32 | __funnelshift_r(x0, x1, sh);
}

// Warp roles:
//   0-3   softmax: waits S(j), masks, takes the row maximum (moving the running one, and
//         O, only past 2^8), writes P over the scores and arrives on p_full; after an item's last tile its
//         output or partial result.  A warp without rows only keeps step.
//   W_K   finds the items and loads their K tiles
//   W_V   loads the V tiles
//   W_S   gathers an item's Q; one lane issues S(j) = Q K(j)^T once K(j) landed and PV(j - NB), the last
//         reader of its buffer, is done, and then releases K
//   W_PV  looks over the V tiles that some row does not see whole; one lane issues O += P(j) V(j) once
//         V(j) and P(j) are there, then releases V
// Key tiles are numbered through all of a CTA's items (j above), items too; every hand-off is an
// mbarrier, and no waiter is more than one phase behind the barrier it waits on.  Every wait is
// bounded; a role that gives up records PKV_DEV_WAIT_TIMEOUT and leaves its loop, the others give up
// in turn, and the CTA still reaches its final barrier.
template <int D, int QR>
__global__ void __launch_bounds__(THREADS, 2) tree_attention_kernel(const __grid_constant__ TreeParams p) {
  using C = Cfg<D, QR>;
  constexpr int NK = C::NK, NV = C::NV, NB = C::NB, CPR = D / 8;   // CPR: 16-byte chunks per row
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  const uint32_t sq = base, sk = sq + C::Q_BYTES, sv = sk + NK * C::KV_BYTES, bars = sv + NV * C::KV_BYTES;
  // per S buffer u (key tile j uses j % NB), per ring slot b, per item slot i (item number % NI)
  auto s_full = [&](int u) { return bars + 8u * u; };
  auto p_full = [&](int u) { return bars + 24u + 8u * u; };
  auto pv_done = [&](int u) { return bars + 48u + 8u * u; };
  auto item_full = [&](int i) { return bars + 72u + 8u * i; };
  auto item_free = [&](int i) { return bars + 72u + 8u * (NI + i); };
  constexpr uint32_t RINGS = 72 + 16 * NI + 16;
  const uint32_t q_free = bars + RINGS - 16, o_free = bars + RINGS - 8;
  auto k_full = [&](int b) { return bars + RINGS + 8u * b; };
  auto k_free = [&](int b) { return bars + RINGS + 8u * (NK + b); };
  auto v_full = [&](int b) { return bars + RINGS + 8u * (2 * NK + b); };
  auto v_free = [&](int b) { return bars + RINGS + 8u * (2 * NK + NV + b); };
  constexpr uint32_t AT = RINGS + 16 * (NK + NV);
  // Which of a tile's positions are in the context and in a block of the pool, for key tile j in place j % 8: K(j) is
  // loaded once S(j - NK) is done, and so PV(j - NK - NB) and what the softmax read for that tile.
  static_assert(NK + NB <= 8 && NB <= 3, "a tile's word is read before it is written anew");
  volatile uint2* live = reinterpret_cast<volatile uint2*>(smem + (bars + AT - base));               // [8]
  constexpr uint32_t ITEMS = AT + 64, LAST = ITEMS + NI * sizeof(Item);
  volatile Item* items = reinterpret_cast<volatile Item*>(smem + (bars + ITEMS - base));             // [NI]
  volatile int* not_finite = reinterpret_cast<volatile int*>(smem + (bars + LAST - base));           // [NI]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + (bars + LAST + 4 * NI - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bars + LAST + 4 * NI + 4 - base));
  static_assert(AT % 8 == 0 && LAST + 4 * NI + 8 <= C::BARS, "barrier area");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pkv::pdl_trigger();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  if (tid == 32) {
    for (int u = 0; u < NB; ++u) {
      mbar_init_count(s_full(u), 1);
      mbar_init_count(p_full(u), 4);
      mbar_init_count(pv_done(u), 1);
    }
    for (int u = 0; u < NI; ++u) {
      mbar_init_count(item_full(u), 1);
      mbar_init_count(item_free(u), 7);                       // 4 softmax warps, both issuers, the V loader
    }
    mbar_init_count(q_free, 1);
    mbar_init_count(o_free, 4);
    for (int b = 0; b < NK; ++b) {
      mbar_init_count(k_full(b), 1);
      mbar_init_count(k_free(b), 1);
    }
    for (int b = 0; b < NV; ++b) {
      mbar_init_count(v_full(b), 1);
      mbar_init_count(v_free(b), 1);
    }
    *abort_flag = 0;
  }
  if (tid == 64 && p.use_tma) {
    prefetch_tensormap(&p.tmap_k);
    prefetch_tensormap(&p.tmap_v);
  }
  pkv::pdl_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto t_s = [&](int u) { return tmem + D + 64u * u; };
  const uint32_t t_o = tmem;
  static_assert(D + 64 * NB <= TMEM_COLS, "tensor memory");
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag); };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  auto give_up = [&]() {
    if (!*abort_flag) record_error(PKV_DEV_WAIT_TIMEOUT);
    *abort_flag = 1;
  };
  auto take_item = [&](int it, Item& item) {
    if (!wait(item_full(it % NI), (it / NI) & 1)) return false;
    const volatile Item& x = items[it % NI];
    item.s = x.s;
    item.kv_head = x.kv_head;
    item.first_row = x.first_row;
    item.rows = x.rows;
    item.tile0 = x.tile0;
    item.n_tiles = x.n_tiles;
    item.ctx = x.ctx;
    item.n = x.n;
    item.q0 = x.q0;
    item.slot = x.slot;
    return true;
  };
  const int lb = p.log2_block, B = 1 << lb;
  bool failed = false;

  if (warp == W_K || warp == W_V) {
    // ---------------- loads ----------------
    const bool is_k = warp == W_K;
    const __half* pool = is_k ? p.k : p.v;
    const CUtensorMap* map = is_k ? &p.tmap_k : &p.tmap_v;
    const uint32_t ring = is_k ? sk : sv;
    const int slots = is_k ? NK : NV;
    int b = 0, round = 0;                                     // tile j goes to slot b = j % slots, round = j / slots
    constexpr int ROWS = 32 / CPR;                            // rows per warp-wide copy
    const int c = lane % CPR, rsub = lane / CPR;              // this lane's chunk and row offset
    const int nb = BN >> lb;                                  // blocks per tile
    // the K loader's place on the line: sequence, stream of it, place in that, and what is left of the piece
    Seq seq{};
    int s = 0, stream = 0, place = 0;
    long long left = 0;
    bool notes = false;                                       // this CTA's Cut is written
    // The CTA's kind of streams, its number among the CTAs that share them out, their count, which row tile of a
    // pair it takes, and its number in the workspace, where a kind's CTAs lie side by side.
    Kind kind = ALL;
    int number = blockIdx.x, count = gridDim.x, half = 0, worker = blockIdx.x;
    long long per = 0;
    if (is_k) {
      const int H = p.num_kv_heads;
      long long pairs = 0, alone = 0;
      int code = 0;
      // lengths and starts by way of the K ring, where nothing has landed yet: all on their way at once, and read twice
      // (waiting for each 32 sequences' loads, 4000 sequences of 60 tokens took 179 us for 111)
      constexpr int CHUNK = 4064;
      static_assert((2 * CHUNK + 1) * 4 <= NK * C::KV_BYTES && CHUNK % 32 == 0, "fits");
      const int* lens = reinterpret_cast<const int*>(smem + (sk - base));
      auto fetch = [&](int first) {
        const int n = min(CHUNK, p.num_seqs - first);
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
          cp_async4(sk + 4 * i, p.lens + first + i);
          cp_async4(sk + 4 * (CHUNK + i), p.qstart + first + i);
        }
        if (lane == 0) cp_async4(sk + 4 * (CHUNK + n), p.qstart + first + n);
        cp_async_wait_all();
        __syncwarp();
      };
      // sequence first + i, of those that are there
      auto seq_at = [&](int first, int i) {
        return first + i < p.num_seqs ? make_seq(p, lens[i], lens[CHUNK + i], lens[CHUNK + i + 1], &code) : Seq{0, 0, 0, 0, 0};
      };
#pragma unroll 1
      for (int first = 0; first < p.num_seqs; first += CHUNK) {
        __syncwarp();
        fetch(first);
#pragma unroll 1
        for (int i = lane; i < min(CHUNK, p.num_seqs - first); i += 32) {
          const Seq y = seq_at(first, i);
          pairs += places_of(y, H, PAIRS);
          alone += places_of(y, H, ALONE);
        }
      }
      if (code && blockIdx.x == 0) record_error(code);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
        alone += __shfl_xor_sync(0xffffffffu, alone, o);
      }
      const int teams = gridDim.x / 2;
      long long total = 2 * pairs + alone;
      if (pairs > 0 && teams >= 2) {
        // CTA w and CTA w + teams, which mostly share an SM, take a pair together; the others single row tiles
        const int team = blockIdx.x % teams;
        half = blockIdx.x / teams;
        int mine = static_cast<int>(divide(2 * pairs * teams + total / 2, total));
        if (alone > 0) mine = max(1, min(teams - 1, mine));
        kind = team < mine ? PAIRS : ALONE;
        count = kind == PAIRS ? mine : 2 * (teams - mine);
        number = kind == PAIRS ? team : half * (teams - mine) + team - mine;
        worker = kind == PAIRS ? half * mine + team : 2 * mine + number;
        total = kind == PAIRS ? pairs : alone;
      }
      per = divide(total + count - 1, count);
      if (per < kMinTiles + kStart) per = kMinTiles + kStart;
      const long long x = number * per;
      left = min(per, total - x);
      if (left > 0) {
        // the sequence: the first whose tiles, all streams together, reach past x
        long long before = 0;
        s = p.num_seqs;
#pragma unroll 1
        for (int at = 0; at < p.num_seqs; at += 32) {
          const int first = at / CHUNK * CHUNK;
          if (p.num_seqs > CHUNK && at == first) {
            __syncwarp();
            fetch(first);
          }
          const Seq y = seq_at(first, at - first + lane);
          const long long mine = places_of(y, H, kind);
          long long upto = mine;
#pragma unroll
          for (int o = 1; o < 32; o *= 2) {
            const long long z = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += z;
          }
          const unsigned past = __ballot_sync(0xffffffffu, before + upto > x);
          if (past) {
            const int hit = __ffs(past) - 1;
            s = at + hit;
            before += __shfl_sync(0xffffffffu, upto - mine, hit);
            seq.ctx = __shfl_sync(0xffffffffu, y.ctx, hit);
            seq.n = __shfl_sync(0xffffffffu, y.n, hit);
            seq.q0 = __shfl_sync(0xffffffffu, y.q0, hit);
            seq.tiles = __shfl_sync(0xffffffffu, y.tiles, hit);
            seq.row_tiles = __shfl_sync(0xffffffffu, y.row_tiles, hit);
            break;
          }
          before += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (streams_of(seq, kind) == 0) {
          left = 0;                                           // the lengths changed meanwhile
        } else {
          stream = static_cast<int>(divide(x - before, seq.tiles + kStart));
          place = static_cast<int>(x - before - static_cast<long long>(stream) * (seq.tiles + kStart));
        }
      }
      __syncwarp();
      fence_proxy_async_smem();                               // these reads -> the ring's copies
    }
    int j = 0;
    for (int it = 0;; ++it) {
      Item item;
      if (is_k) {
        // the next item, for all roles
        item.n_tiles = 0;
        int tile = 0;
        if (left > 0) {
          tile = max(0, place - kStart);
          const int to = static_cast<int>(min(static_cast<long long>(seq.tiles + kStart), place + left));
          left -= to - place;
          item.n_tiles = max(0, to - kStart) - tile;          // 0 where the piece ends before the stream's first
        }
        if (item.n_tiles > 0) {
          item.s = s;
          const int streams = streams_of(seq, kind), tile_no = stream % streams;
          item.kv_head = stream / streams;
          item.first_row = (kind == ALL ? tile_no : kind == PAIRS ? 2 * tile_no + half : seq.row_tiles - 1) * BM;
          item.rows = min(BM, seq.n * p.group - item.first_row);
          item.tile0 = tile;
          item.ctx = seq.ctx;
          item.n = seq.n;
          item.q0 = seq.q0;
          item.slot = item.n_tiles == seq.tiles ? -1 : 2 * worker + (it > 0);
        }
        if (it >= NI && !warp_wait(item_free(it % NI), (it / NI - 1) & 1)) {
          failed = true;
          break;
        }
        if (lane == 0) {
          volatile Item& out = items[it % NI];
          out.n_tiles = item.n_tiles;
          if (item.n_tiles > 0) {
            out.s = item.s;
            out.kv_head = item.kv_head;
            out.first_row = item.first_row;
            out.rows = item.rows;
            out.tile0 = item.tile0;
            out.ctx = item.ctx;
            out.n = item.n;
            out.q0 = item.q0;
            out.slot = item.slot;
          }
          mbar_arrive(item_full(it % NI));
        }
        __syncwarp();
      } else {
        if (!__all_sync(0xffffffffu, take_item(it, item))) {
          failed = true;
          break;
        }
      }
      if (item.n_tiles == 0) break;
      const int32_t* table = p.tables + static_cast<size_t>(item.s) * p.max_blocks;
      // the table entries of 32 of the item's blocks, one a lane, and of the next 32
      auto entries = [&](int block) {
        const int t0 = item.tile0 * BN + ((block + lane) << lb);
        return t0 < item.ctx ? __ldg(table + (t0 >> lb)) : -1;
      };
      int entry = entries(0), next_entries = entries(32);
      for (int i = 0; i < item.n_tiles; ++i, ++j) {
        const int key0 = (item.tile0 + i) * BN, t0 = key0 + (lane << lb);
        const bool in_ctx = lane < nb && t0 < item.ctx;
        const int at_block = i * nb & 31;
        if (at_block == 0 && i > 0) {
          entry = next_entries;
          next_entries = entries(i * nb + 32);
        }
        int phys = __shfl_sync(0xffffffffu, entry, at_block + lane);
        const bool good = in_ctx && phys >= 0 && phys < p.num_blocks;
        if (is_k && in_ctx && !good) record_error(PKV_DEV_BAD_BLOCK_ID);
        if (!good) phys = -1;
        const uint32_t good_mask = __ballot_sync(0xffffffffu, good);
        if (round > 0 && !warp_wait(is_k ? k_free(b) : v_free(b), (round - 1) & 1)) {
          failed = true;
          break;
        }
        const uint32_t full = is_k ? k_full(b) : v_full(b), dst = ring + b * C::KV_BYTES;
        if (++b == slots) {
          b = 0;
          ++round;
        }
        if (is_k) {
          // K rows past the context or of bad blocks may hold anything: their scores are masked
          const int valid = good ? min(B, item.ctx - t0) : 0, at = lane << lb & 31;
          const uint32_t bits = (valid >= 32 ? 0xffffffffu : (1u << valid) - 1u) << at;
          const uint32_t lo = __reduce_or_sync(0xffffffffu, lane << lb < 32 ? bits : 0u);
          const uint32_t hi = __reduce_or_sync(0xffffffffu, lane << lb < 32 ? 0u : bits);
          if (lane == 0) {
            live[j & 7].x = lo;
            live[j & 7].y = hi;
          }
        }
        // V tiles with a block outside the pool, and small blocks, come in 16-byte copies, with zeros in its place
        if (p.use_tma && (is_k || !__any_sync(0xffffffffu, in_ctx && !good))) {
          if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(good_mask)) * B * D * 2);
          __syncwarp();
          if (good) {
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_3d(dst + half * (BN * 128) + lane * B * 128, map, half * 64, item.kv_head * B, phys, full);
          }
          continue;
        }
#pragma unroll 4
        for (int r0 = 0; r0 < BN; r0 += ROWS) {
          const int pb = __shfl_sync(0xffffffffu, phys, r0 >> lb), r = r0 + rsub;   // ROWS <= 4 <= B: one block
          const __half* src = pool + (((static_cast<size_t>(max(pb, 0)) * p.num_kv_heads + item.kv_head) << lb) + (r & (B - 1))) * D + c * 8;
          cp_async16(dst + sw128(r, c, BN), src, pb >= 0 ? 16 : 0);
        }
        cp_async_wait_all();
        fence_proxy_async_smem();                             // these writes -> tensor-core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      if (failed) break;
      if (is_k) {
        if (item.tile0 == 0 && item.n_tiles < seq.tiles) {
          // a cut stream's first part: the others are the first items of the CTAs that follow
          notes = true;
          if (lane == 0) {
            Cut cut{};
            cut.parts = 1 + static_cast<int>(divide(seq.tiles - item.n_tiles + per - 1, per));
            cut.parts = min(cut.parts, count - number);
            cut.slot = item.slot;
            cut.next = 2 * (worker + 1);
            cut.rows = item.rows;
            cut.first_row = item.first_row;
            cut.q0 = item.q0;
            cut.kv_head = item.kv_head;
            p.cuts[worker] = cut;
          }
        }
        if (left > 0) {                                       // on to the next stream
          place = 0;
          if (++stream == p.num_kv_heads * streams_of(seq, kind)) {
            stream = 0;
            int code = 0;
            do seq = seq_of(p, ++s, &code);
            while (streams_of(seq, kind) == 0 && s < p.num_seqs);
            if (streams_of(seq, kind) == 0) left = 0;         // the lengths changed meanwhile
          }
        }
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(item_free(it % NI));
      }
    }
    if (is_k && !notes && lane == 0) p.cuts[worker].parts = 0;
    if (failed) give_up();
    if (*abort_flag) {
      // let the copies this warp issued land (bounded) before the CTA's shared memory is released
      for (int t = max(0, j - slots); t < j; ++t) mbar_wait(is_k ? k_full(t % NK) : v_full(t % NV), (t / slots) & 1);
    }
  } else if (warp == W_S) {
    // ---------------- Q, and S = Q K^T issue (one lane) ----------------
    constexpr uint32_t IDESC_QK = umma_idesc_f16(BM, BN, false);
    const uint64_t a0 = umma_smem_desc(sq, 16, 1024);
    int j = 0, u = 0, phase = 0;                              // tile j: S buffer u = j % NB, phase = j / NB
    for (int it = 0;; ++it) {
      Item item;
      if (!__all_sync(0xffffffffu, take_item(it, item) && (it == 0 || wait(q_free, (it - 1) & 1)))) {
        failed = true;
        break;
      }
      if (item.n_tiles == 0) break;
      // Rows past the item's hold what was there: a row of the product depends on its own alone.
      {
        constexpr int ROWS = 32 / CPR;                        // rows per warp-wide copy
        const int c = lane % CPR;
        int r = lane / CPR, i = (item.first_row + r) / p.group, g = item.first_row + r - i * p.group;
        const __half* src = p.q + (item.q0 + i) * p.q_stride + (item.kv_head * p.group + g) * D + c * 8;
#pragma unroll 1
        for (; r < item.rows; r += ROWS) {
          cp_async16(sq + sw128(r, c, QR), src, 16);
          // ROWS rows on: so many heads further, or in a later node
          g += ROWS;
          src += ROWS * D;
          while (g >= p.group) {
            g -= p.group;
            src += p.q_stride - p.group * D;
          }
        }
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(item_free(it % NI));
        for (int i = 0; i < item.n_tiles; ++i, ++j) {
          if (!wait(k_full(j % NK), (j / NK) & 1) || (phase > 0 && !wait(pv_done(u), (phase - 1) & 1))) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint64_t b0 = umma_smem_desc(sk + (j % NK) * C::KV_BYTES, 16, 1024);
          const uint32_t d = t_s(u);
          umma_ss(d, a0, b0, IDESC_QK, 0u);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk)
            umma_ss(d, a0 + (((kk >> 2) * (QR * 128) + (kk & 3) * 32) >> 4),
                    b0 + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), IDESC_QK, 1u);
          umma_commit(s_full(u));
          umma_commit(k_free(j % NK));
          if (++u == NB) {
            u = 0;
            ++phase;
          }
        }
        if (!failed) umma_commit(q_free);
      }
      j = __shfl_sync(0xffffffffu, j, 0);
      failed = __shfl_sync(0xffffffffu, failed, 0);
      if (failed) break;
    }
    if (failed) {
      give_up();
      if (j > 0) mbar_wait(s_full((j - 1) % NB), ((j - 1) / NB) & 1);
    }
  } else if (warp == W_PV) {
    // ---------------- O += P V issue (one lane); V tiles that some row does not see whole ----------------
    constexpr uint32_t IDESC_PV = umma_idesc_f16(BM, D, true);
    int j = 0, u = 0, phase = 0;
    for (int it = 0;; ++it) {
      Item item;
      if (!__all_sync(0xffffffffu, take_item(it, item))) {
        failed = true;
        break;
      }
      if (item.n_tiles == 0) break;
      if (lane == 0) not_finite[it % NI] = 0;
      __syncwarp();
      const int first_new = item.ctx - item.n;
      for (int i = 0; i < item.n_tiles; ++i, ++j) {
        const int b = j % NV, key0 = (item.tile0 + i) * BN;
        if (!warp_wait(v_full(b), (j / NV) & 1)) {
          failed = true;
          break;
        }
        if (key0 + BN > first_new) {
          // Zeros past the context's end, and for drafts' values that are not finite; four chunks in flight to a
          // lane (one after the other they took 6500 clocks of a short stream's 15000).
          unsigned char* v = smem + (sv + b * C::KV_BYTES - base);
          const int end = min(BN, item.ctx - key0) * CPR;
          const __half2 zero = __float2half2_rn(0.f);
#pragma unroll 1
          for (int k0 = max(0, first_new - key0) * CPR + lane; k0 < end; k0 += 4 * 32) {
            uint4 w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int k = k0 + h * 32;
              w[h] = make_uint4(0, 0, 0, 0);
              if (k < end) w[h] = *reinterpret_cast<const uint4*>(v + sw128(k / CPR, k % CPR, BN));
            }
            // 0 times a value is a NaN if the value is not finite; sums of those are NaN
            __half2 acc = zero;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              acc = __hfma2(*reinterpret_cast<const __half2*>(&w[h].x), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __half2*>(&w[h].y), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __half2*>(&w[h].z), zero, acc);
              acc = __hfma2(*reinterpret_cast<const __half2*>(&w[h].w), zero, acc);
            }
            if (__hisnan(__low2half(acc)) || __hisnan(__high2half(acc))) {
              not_finite[it % NI] = 1;
#pragma unroll 1
              for (int k = k0; k < min(end, k0 + 4 * 32); k += 32) {
                uint32_t* e = reinterpret_cast<uint32_t*>(v + sw128(k / CPR, k % CPR, BN));
#pragma unroll 1
                for (int h = 0; h < 4; ++h)
                  e[h] = (finite16(e[h]) ? e[h] & 0xffffu : 0u) | (finite16(e[h] >> 16) ? e[h] & 0xffff0000u : 0u);
              }
            }
          }
          // a lane's rows ROWS apart: the same chunk of each
          constexpr int ROWS = 32 / CPR;
#pragma unroll 2
          for (int r = end / CPR + lane / CPR; r < BN; r += ROWS)
            *reinterpret_cast<uint4*>(v + sw128(r, lane % CPR, BN)) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();                           // these writes -> tensor-core reads
          __syncwarp();
        }
        if (lane == 0) {
          // the first product overwrites the accumulator: the last item's output has been read
          if ((i == 0 && it > 0 && !wait(o_free, (it - 1) & 1)) || !wait(p_full(u), phase & 1)) {
            failed = true;
          } else {
            tc_fence_after();
            const uint64_t v0 = umma_smem_desc(sv + b * C::KV_BYTES, BN * 128, 1024);
            const uint32_t pa = t_s(u);
            umma_ts(t_o, pa, v0, IDESC_PV, i > 0 ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < BN / 16; ++kk) umma_ts(t_o, pa + kk * 8, v0 + ((kk * 16 * 128) >> 4), IDESC_PV, 1u);
            umma_commit(pv_done(u));
            umma_commit(v_free(b));
          }
        }
        failed = __shfl_sync(0xffffffffu, failed, 0);
        if (failed) break;
        if (++u == NB) {
          u = 0;
          ++phase;
        }
      }
      if (failed) break;
      if (lane == 0) mbar_arrive(item_free(it % NI));
    }
    if (failed) {
      give_up();
      if (j > 0) mbar_wait(pv_done((j - 1) % NB), ((j - 1) / NB) & 1);
    }
  } else {
    // ---------------- softmax and output ----------------
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    int j = 0, u = 0, phase = 0;
    uint32_t last = 0, last_phase = 0;                        // of the tile before: its pv_done barrier and phase
    for (int it = 0; !failed; ++it) {
      Item item;
      // decisions stay warp-uniform: the tcgen05.ld/st below are warp-collective
      if (!__all_sync(0xffffffffu, take_item(it, item))) failed = true;
      if (failed || item.n_tiles == 0) break;
      const bool works = warp * 32 < item.rows;
      const int row = item.first_row + min(tid, item.rows - 1), node = row / p.group, first_new = item.ctx - item.n;
      float l = 0.f, m_ref = -INFINITY;
      for (int i = 0; i < item.n_tiles; ++i, ++j) {
        const int key0 = (item.tile0 + i) * BN;
        const uint32_t ts = t_s(u), before = last, before_phase = last_phase, here = p_full(u);
        if (!warp_wait(s_full(u), phase & 1)) {
          failed = true;
          break;
        }
        last = pv_done(u);
        last_phase = phase & 1;
        if (++u == NB) {
          u = 0;
          ++phase;
        }
        if (!works) {
          if (lane == 0) mbar_arrive(here);
          continue;
        }
        tc_fence_after();
        const uint32_t live_lo = live[j & 7].x, live_hi = live[j & 7].y;
        float sv_[BN];
        tmem_ld32_nowait(ts + lane_off, *reinterpret_cast<float(*)[32]>(sv_));
        tmem_ld32_nowait(ts + lane_off + 32, *reinterpret_cast<float(*)[32]>(sv_ + 32));
        tmem_ld_wait();
        if (key0 + BN > first_new || (live_lo & live_hi) != 0xffffffffu) {
          const uint64_t seen = seen_from(p, item.q0 + node, node, key0, first_new);
          const uint32_t lo = static_cast<uint32_t>(seen) & live_lo, hi = static_cast<uint32_t>(seen >> 32) & live_hi;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (!(lo >> c & 1)) sv_[c] = -INFINITY;
            if (!(hi >> c & 1)) sv_[32 + c] = -INFINITY;
          }
        }
        float m8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) m8[e] = fmaxf(sv_[e], sv_[8 + e]);
#pragma unroll
        for (int c = 16; c < BN; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = max3(m8[e], sv_[c + e], sv_[c + 8 + e]);
        float mx = max3(max3(m8[0], m8[1], m8[2]), max3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        mx *= p.scale_log2;
        const bool rescale = mx > m_ref + kRescale;           // also the first finite maximum
        float alpha = 1.f;
        if (rescale) {
          alpha = exp2f(m_ref - mx);
          m_ref = mx;
        }
        const float nref = m_ref == -INFINITY ? 0.f : kLift - m_ref;
        if (__any_sync(0xffffffffu, rescale && i > 0)) {
          if (!warp_wait(before, before_phase)) {
            failed = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(t_o + lane_off + c * 32, o);
            uint32_t ob[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) ob[e] = __float_as_uint(o[e] * alpha);
            tmem_st32(t_o + lane_off + c * 32, ob);
          }
        }
        // P as fp16; the row sum adds the rounded weights, the ones that multiply V
        float sum8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t pk[BN / 2];
#pragma unroll
        for (int e = 0; e < BN / 2; ++e) {
          float x0, x1;
          fma2(x0, x1, sv_[2 * e], sv_[2 * e + 1], p.scale_log2, nref);
          pk[e] = pack_half2(fast_exp2(x0), fast_exp2(x1));
          add_half2(sum8[2 * (e & 3)], sum8[2 * (e & 3) + 1], pk[e]);
        }
        float sum4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum4[e] = sum8[2 * e] + sum8[2 * e + 1];
        tmem_st32(ts + lane_off, pk);
        l = l * alpha + ((sum4[0] + sum4[1]) + (sum4[2] + sum4[3]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(here);
      }
      if (!failed) failed = !warp_wait(last, last_phase);
      if (failed) break;
      tc_fence_after();
      if (works) {
        // 32 columns at a time: the row to out, whole 32-byte sectors at once, or to the workspace, where
        // a column's rows lie side by side
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a row that sees nothing is zeros
        const bool fix = not_finite[it % NI] != 0, real = tid < item.rows;
        const int head = item.kv_head * p.group + (row - node * p.group);
        __half* dst = p.out + (static_cast<size_t>(item.q0 + node) * p.num_heads + head) * D;
        float* part = p.ws_o + static_cast<size_t>(max(item.slot, 0)) * D * BM + tid;
        if (item.slot >= 0 && real) p.ws_ml[static_cast<size_t>(item.slot) * BM + tid] = make_float2(m_ref, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float x[32];
          tmem_ld32(t_o + lane_off + c * 32, x);
          if (item.slot >= 0) {
            if (real) {
#pragma unroll
              for (int e = 0; e < 32; ++e) part[(c * 32 + e) * BM] = x[e];
            }
          } else if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 16) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = pack_half2(x[e + 2 * k] * inv, x[e + 2 * k + 1] * inv);
              store16(dst + c * 32 + e, w, p.out_sectors);
            }
          }
          __syncwarp();
        }
        if (fix && real) {
          // values of drafts that are not finite were left out: added to what is stored, where the row sees them
          // (rare, so its code is small rather than fast)
          const int from = max(first_new, item.tile0 * BN), to = min(item.ctx, (item.tile0 + item.n_tiles) * BN);
#pragma unroll 1
          for (int t = from; t < to; ++t) {
            const int phys = p.tables[static_cast<size_t>(item.s) * p.max_blocks + (t >> lb)];
            if (!(seen_from(p, item.q0 + node, node, t, first_new) & 1) || phys < 0 || phys >= p.num_blocks) continue;
            const __half* v = p.v + (((static_cast<size_t>(phys) * p.num_kv_heads + item.kv_head) << lb) + (t & (B - 1))) * D;
#pragma unroll 1
            for (int e = 0; e < D; ++e) {
              if (finite16(__half_as_ushort(v[e]))) continue;
              if (item.slot >= 0) part[e * BM] += __half2float(v[e]);
              else dst[e] = __float2half_rn(__half2float(dst[e]) + __half2float(v[e]));
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free);
        mbar_arrive(item_free(it % NI));
      }
    }
    if (failed) give_up();
  }

  // every tensor-memory access is done (tcgen05.ld and .st wait inline, the products are committed)
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// ---- joining the parts of cut streams, by the log-sum-exp identity ---------------------------------
// A row's running result over parts, of which one that saw nothing (m -inf, l 0) is left out; one with a NaN is not.
struct Joined {
  float M, L, acc[4];
  __device__ __forceinline__ void add(const float2 (&ml)[4], const float (&x)[4][4]) {
    float m = M;
#pragma unroll
    for (int u = 0; u < 4; ++u) m = fmaxf(m, ml[u].x);
    const float base = m == -INFINITY ? 0.f : m, carry = exp2f(M - base);   // nothing seen so far: 0
    L *= carry;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= carry;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (ml[u].x == -INFINITY && ml[u].y == 0.f) continue;
      const float f = exp2f(ml[u].x - base);
      L = fmaf(ml[u].y, f, L);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[u][e], f, acc[e]);
    }
    M = m;
  }
  __device__ __forceinline__ void store(__half* dst) const {
    const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_half2(acc[0] * inv, acc[1] * inv), pack_half2(acc[2] * inv, acc[3] * inv));
  }
};
// Row r's (m, l) and four columns' values in parts k, k + step, ..: all of them on their way at once.
template <int D>
__device__ __forceinline__ void load_parts(const TreeParams& p, const Cut& cut, int k, int step, int r, int col,
                                           float2 (&ml)[4], float (&x)[4][4]) {
#pragma unroll
  for (int u = 0; u < 4; ++u, k += step) {
    ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[u][e] = 0.f;
    if (k < cut.parts) {
      const size_t slot = k == 0 ? cut.slot : cut.next + 2 * (k - 1);
      ml[u] = p.ws_ml[slot * BM + r];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][e] = p.ws_o[(slot * D + col + e) * BM + r];
    }
  }
}
__device__ __forceinline__ __half* row_of(const TreeParams& p, const Cut& cut, int r, int D) {
  const int row = cut.first_row + r, node = row / p.group, head = cut.kv_head * p.group + row - node * p.group;
  return p.out + (static_cast<size_t>(cut.q0 + node) * p.num_heads + head) * D;
}

// CTA (w, y): the y-th share of the columns of the stream that CTA w of the grid before noted; a thread has a row
// and four columns at a time.
constexpr int JOIN_THREADS = 256;
// One sequence of 2048 tokens and 40 heads takes 16.7 us with one share of the columns, 15.2 with four, 16.1 with eight;
// 8 of 4096 with 64 rows 44.9, 37.1 and 36.2.
constexpr int kJoinShares = 4;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) tree_attention_join_kernel(const __grid_constant__ TreeParams p) {
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts <= 1) return;
  int log2_rows = 3;                                          // the rows, to a power of two
  while ((1 << log2_rows) < cut.rows) ++log2_rows;
  const int r = threadIdx.x & ((1 << log2_rows) - 1), share = D / gridDim.y;
  if (r >= cut.rows) return;
  __half* dst = row_of(p, cut, r, D);
  for (int c = (threadIdx.x >> log2_rows) * 4; c < share; c += JOIN_THREADS >> log2_rows << 2) {
    const int col = blockIdx.y * share + c;
    Joined all{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
    for (int k = 0; k < cut.parts; k += 4) {
      float2 ml[4];
      float x[4][4];
      load_parts<D>(p, cut, k, 1, r, col, ml, x);
      all.add(ml, x);
    }
    all.store(dst + col);
  }
}

// The same where there are few streams, and so many parts: CTA (k, y) columns 4 y .. of the k-th stream that was
// noted; groups of threads share its parts.
constexpr int MANY_THREADS = 512;
template <int D>
__global__ void __launch_bounds__(MANY_THREADS) tree_attention_join_many_kernel(const __grid_constant__ TreeParams p) {
  __shared__ Joined groups[MANY_THREADS];
  __shared__ int before[MANY_THREADS / 32], found;
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) found = -1;
  int seen = 0;
  for (int w0 = 0; w0 < p.workers; w0 += MANY_THREADS) {
    const int w = w0 + tid;
    const bool is_cut = w < p.workers && p.cuts[w].parts > 1;
    const unsigned mine = __ballot_sync(0xffffffffu, is_cut);
    __syncthreads();
    before[warp] = __popc(mine);
    __syncthreads();
    int rank = seen + __popc(mine & ((1u << lane) - 1));
    for (int i = 0; i < MANY_THREADS / 32; ++i) {
      if (i < warp) rank += before[i];
      seen += before[i];
    }
    if (is_cut && rank == static_cast<int>(blockIdx.x)) found = w;
  }
  __syncthreads();
  if (found < 0) return;
  const Cut cut = p.cuts[found];
  int log2_rows = 3;
  while ((1 << log2_rows) < cut.rows) ++log2_rows;
  const int r = tid & ((1 << log2_rows) - 1), count = MANY_THREADS >> log2_rows, col = blockIdx.y * 4;
  Joined all{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  if (r < cut.rows) {
    for (int k = tid >> log2_rows; k < cut.parts; k += 4 * count) {
      float2 ml[4];
      float x[4][4];
      load_parts<D>(p, cut, k, count, r, col, ml, x);
      all.add(ml, x);
    }
  }
  groups[tid] = all;
  __syncthreads();
  if (tid >= cut.rows) return;
  all = Joined{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
  for (int g = 0; g < count; g += 4) {                        // count is at least 4
    float2 ml[4];
    float x[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const Joined& other = groups[((g + u) << log2_rows) + r];
      ml[u] = make_float2(other.M, other.L);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][e] = other.acc[e];
    }
    all.add(ml, x);
  }
  all.store(row_of(p, cut, r, D) + col);
}

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

// Two CTAs to an SM, or as many as the longest contexts would give kMinTiles key tiles each.
struct Plan {
  int workers;
  long long streams;               // at most
  long long most_tiles;
};
Plan plan_for(int num_seqs, int total_q, int max_query_len, int num_heads, int num_kv_heads, long long max_ctx) {
  Plan pl{};
  const int group = num_heads / num_kv_heads;
  // streams: a sequence has one row tile at least, and all of them no more than their rows fill
  const long long rows = static_cast<long long>(max_query_len) * group, per_seq = (rows + BM - 1) / BM;
  const long long by_rows = num_seqs + static_cast<long long>(total_q) * group / BM;
  const long long row_tiles = per_seq * num_seqs < by_rows ? per_seq * num_seqs : by_rows;
  pl.streams = row_tiles * num_kv_heads;
  pl.most_tiles = pl.streams * ((max_ctx + BN - 1) / BN);
  const long long want = (pl.most_tiles + kMinTiles - 1) / kMinTiles, most = 2 * device_sms();
  pl.workers = static_cast<int>(want < most ? want : most);
  if (rows > BM) pl.workers += pl.workers & 1;                // pairs of row tiles want pairs of CTAs
  return pl;
}
size_t ml_bytes(int workers) { return static_cast<size_t>(workers) * 2 * BM * sizeof(float2); }
size_t cut_bytes(int workers) { return static_cast<size_t>(workers) * sizeof(Cut); }
size_t workspace_bytes_for(const Plan& pl, int head_dim) {
  return ml_bytes(pl.workers) + cut_bytes(pl.workers) + static_cast<size_t>(pl.workers) * 2 * BM * head_dim * sizeof(float);
}

// A pool [num_blocks][H][B][D] fp16 as the 3-D tensor (D, H B, num_blocks); a box is one head's B rows of one
// 64-element half of the head dimension, written with the 128-byte swizzle.
int encode_pool_map(const char* fn, CUtensorMap* map, const void* pool, int D, int H, int B, int num_blocks) {
  const EncodeTiledFn encode = tensor_map_encoder();
  if (!encode) return pkv::fail(PKV_ERR_CUDA, "%s: cuTensorMapEncodeTiled is not available", fn);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H) * B, static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * B * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(B), 1};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(pool), dims, strides, box, elem,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return pkv::fail(PKV_ERR_CUDA, "%s: tensor map encoding failed (%d)", fn, static_cast<int>(r));
  return PKV_OK;
}

template <int D, int QR>
int launch(const char* fn, const TreeParams& p, int workers, int few_streams, cudaStream_t st) {
  using C = Cfg<D, QR>;
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> g(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(tree_attention_kernel<D, QR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s setup: %s", fn, cudaGetErrorString(e));
  e = pkv::launch_pdl(tree_attention_kernel<D, QR>, dim3(workers), dim3(THREADS), C::SMEM, st, p);
  if (e == cudaSuccess && workers > 1)
    e = few_streams ? pkv::launch_pdl(tree_attention_join_many_kernel<D>, dim3(few_streams, D / 4), dim3(MANY_THREADS), 0, st, p)
                    : pkv::launch_pdl(tree_attention_join_kernel<D>, dim3(workers, kJoinShares), dim3(JOIN_THREADS), 0, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  return PKV_OK;
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int device_error_word_tree_attention(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_tree_attention));
}
}  // namespace pkv

extern "C" {

size_t pkv_paged_attention_tree_workspace_size(int num_seqs, int total_q, int max_query_len, int num_heads,
                                               int num_kv_heads, int head_dim, int max_blocks_per_seq,
                                               int block_size) {
  if (num_seqs <= 0 || total_q <= 0 || max_query_len <= 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads || head_dim <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return 0;
  return workspace_bytes_for(plan_for(num_seqs, total_q, max_query_len, num_heads, num_kv_heads,
                                      static_cast<long long>(max_blocks_per_seq) * block_size),
                             head_dim);
}

int pkv_paged_attention_tree(const uint16_t* q, int64_t q_stride, const uint16_t* k_cache, const uint16_t* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                             const int32_t* tree_mask, int mask_words, int num_seqs, int total_q, int max_query_len,
                             int num_heads, int num_kv_heads, int head_dim, int num_blocks, int max_blocks_per_seq,
                             float scale, int block_size, uint16_t* out, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* fn = "pkv_paged_attention_tree";
  if (num_seqs < 0 || total_q < 0 || max_query_len < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG,
                     "%s: num_seqs=%d total_q=%d max_query_len=%d num_heads=%d num_kv_heads=%d num_blocks=%d "
                     "max_blocks_per_seq=%d",
                     fn, num_seqs, total_q, max_query_len, num_heads, num_kv_heads, num_blocks, max_blocks_per_seq);
  if (num_heads % num_kv_heads)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_heads=%d is not a multiple of num_kv_heads=%d", fn, num_heads,
                     num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: block_size %d not in {4, 8, 16, 32}", fn, block_size);
  if (tree_mask && (mask_words <= 0 || static_cast<long long>(mask_words) * 32 < max_query_len))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: %d mask words a row for max_query_len=%d", fn, mask_words, max_query_len);
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (num_seqs > 65535 || num_heads > 65535)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: num_seqs/num_heads above 65535", fn);
  if (static_cast<long long>(max_query_len) * (num_heads / num_kv_heads) > (1LL << 26))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^26 rows to a cached head", fn);
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: context capacity above 2^30 tokens", fn);
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !out)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q, caches, out, workspace must be 16-byte aligned", fn);
  if (q_stride < static_cast<int64_t>(num_heads) * head_dim || q_stride % 8)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 8 and at least a token's length", fn);
  if (!std::isfinite(scale) || !(scale > 0.f))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: scale must be finite and positive", fn);
  const Plan pl = plan_for(num_seqs, total_q, max_query_len, num_heads, num_kv_heads,
                           static_cast<long long>(max_blocks_per_seq) * block_size);
  const size_t need = workspace_bytes_for(pl, head_dim);
  if (!workspace || workspace_bytes < need)
    return pkv::fail(PKV_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                     workspace ? workspace_bytes : static_cast<size_t>(0));
  if (pl.most_tiles / pl.workers >= (1LL << 30))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^30 key tiles to a CTA", fn);
  TreeParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k = reinterpret_cast<const __half*>(k_cache);
  p.v = reinterpret_cast<const __half*>(v_cache);
  p.tables = block_tables;
  p.lens = context_lens;
  p.qstart = query_start;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.out = reinterpret_cast<__half*>(out);
  p.q_stride = q_stride;
  p.mask_words = mask_words;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_query_len = max_query_len;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks_per_seq;
  while ((1 << p.log2_block) < block_size) ++p.log2_block;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out_sectors = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.ws_ml = static_cast<float2*>(workspace);
  p.cuts = reinterpret_cast<Cut*>(static_cast<char*>(workspace) + ml_bytes(pl.workers));
  p.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml_bytes(pl.workers) + cut_bytes(pl.workers));
  // whole blocks of 8 or more rows are fetched by TMA; smaller blocks by 16-byte copies
  p.use_tma = block_size >= 8 ? 1 : 0;
  if (p.use_tma) {
    int rc = encode_pool_map(fn, &p.tmap_k, k_cache, head_dim, num_kv_heads, block_size, num_blocks);
    if (rc == PKV_OK) rc = encode_pool_map(fn, &p.tmap_v, v_cache, head_dim, num_kv_heads, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // few rows leave shared memory for more key tiles in flight
  const int rows = max_query_len * p.group;
  const int few = pl.workers > kManyParts * pl.streams ? static_cast<int>(pl.streams) : 0;
  p.workers = pl.workers;
  const int rc = head_dim == 64 ? launch<64, 128>(fn, p, pl.workers, few, st)
                 : rows <= 32   ? launch<128, 32>(fn, p, pl.workers, few, st)
                 : rows <= 64   ? launch<128, 64>(fn, p, pl.workers, few, st)
                                : launch<128, 128>(fn, p, pl.workers, few, st);
  if (rc == PKV_OK) pkv::clear_error();
  return rc;
}

}  // extern "C"
