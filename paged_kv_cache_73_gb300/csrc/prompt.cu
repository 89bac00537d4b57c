// Prompt attention for sm_103a: packed sequences of queries over contiguous keys and
// values, causal, groups of query heads sharing a key head.
//
//   o_i = sum_{t <= p} softmax_t(scale q_i . k_t) v_t,   p = m - n + i
//
// for query i of a sequence with n queries and m >= n keys ([note] "vLLM /
// PagedAttention -- 把 LLM 服务的瓶颈从显存碎片里救出来", 关键设计 1, first equation).  It serves
// requests whose K/V go to a four-bit cache: the prompt attends over its own fp16 rows
// (and over gathered rows of its cached context) before or while they are quantised.
//
// 4 D flops per (query, key) pair that the mask leaves, against two rows read per
// 128-query tile: bound by the tensor cores.  Scores and outputs live in tensor memory
// (tcgen05.mma, fp16 in, fp32 accumulation); a softmax thread owns a query row, which is
// a tensor-memory lane.
//  * One CTA takes 128 queries of one head, with a half of the tensor memory and of the
//    shared memory, so two run on an SM: each hides the other's start, end and hand-offs.
//    One CTA with two query tiles that share every K/V tile took 1242 us against 1122 for
//    eight 4096-token prompts (40 heads on 8), and 126 against 98 for ragged short ones,
//    where starts and ends are most of the time.
//  * Key tiles of 64 positions come by TMA through a ring.  Where some row of the CTA does
//    not see a tile whole (the diagonal, and the tile that holds the sequence's end), a
//    warp first looks V's tile over: a masked weight of 0 times a value that is not finite
//    would be a NaN, so such values become zeros, and are put back in the end for the rows
//    that see them.
//  * The grid is a flat list of query tiles (a tile's sequence is found by a prefix sum over
//    query_start), so a batch of ragged prompts launches few CTAs that have nothing to do.
//    Head after head, so that a head's K/V stay in L2; only the last heads' tiles go from long
//    to short, so that the CTAs end together.
//  * A CTA that runs takes over tiles of CTAs not launched yet (clusterlaunchcontrol), and its
//    roles pass from one tile to the next on their own: the next tile's K and V are loaded
//    and its first scores computed while the softmax warps write the last tile's output.
//    One launch per tile spent 4.3 us of 7.7 on starts and ends where prompts are short.
//  * Few queries over many keys (a chunk of one long request) would leave most SMs idle: there the CTAs
//    of a cluster share a query tile's keys, and each then joins a slice of the columns from all
//    parts by the log-sum-exp identity, read through distributed shared memory: no workspace and no
//    second kernel.
//  * Five kinds of warps run different code at once and share the instruction cache, so code
//    is kept small where it is not hot: waits in one loop instead of two took ragged short
//    prompts from 94 us to 74, an unrolled staging of the output had them at 107.
//
// Per 128 x 64 tile (D = 128) the products take 384 + 256 clocks: S is bound by shared memory
// (an SS product of 128 x 64 x 16 reads 6 KB), PV by math; both with the loads come to about 750
// clocks of shared-memory traffic as counted, and 685 a tile are measured on long prompts.  Two S
// buffers keep S(j + 1) running under the softmax of tile j (about 1000 clocks).
// Measured: eight 4096-token prompts, 40 heads on 8, 1100 us (1.25 PFLOP/s); 32 prompts of 1 to 512
// tokens, 40 heads, 71 us (4.7 TB/s of q, K, V and out); 16 chunks of 32 to 512 tokens over 1024
// cached ones, 32 heads on 8, D = 64, 63 us.
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "launch.cuh"
#include "pkv_internal.h"
#include "prompt_items.cuh"
#include "tcgen05.cuh"

namespace {

using namespace pkv::tc;
using namespace pkv::prompt;

__device__ int g_dev_error_prompt = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_prompt, 0, code); }

// Where the query tiles of all heads fill at most half of the resident CTAs and a query sees kSplitTiles key
// tiles or more on average, clusters of two to eight CTAs take an item each and share its key tiles (at least
// two to a CTA, and none shared below half of kSplitTiles): 128 queries over 131072 keys, 32 heads on 8, 1400
// -> 256 us; 64 over 8192, 96 -> 29; 128 over 1128, 8 heads, 18.5 -> 12.7.  Below, the clusters' start and the
// joining cost more than they save: 1024 tokens over themselves, 8 heads, 17.2 -> 18.7 us.
constexpr int kResident = 304, kSplitTiles = 12, kMostParts = 8;
constexpr float kRescale = 8.f;    // the running maximum moves when a tile passes it by this much
// Weights are kept as 2^(kLift + S - m): the largest in fp16's upper half, at most 2^15, so that those that
// fall below its smallest number are 2^-32 of the largest, not 2^-25.
constexpr float kLift = 7.f;

struct PromptParams {
  CUtensorMap tmap_q, tmap_k, tmap_v;   // (D, heads, tokens), boxes of 64 x 1 x 128 (q) or 64, 128-byte swizzle
  const __half* v;
  __half* out;
  int64_t v_stride;
  Layout layout;
  int group;
  int out_sectors;                      // out is 32-byte aligned
  float scale_log2;
};

template <int D>
struct Cfg {
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int NS = D == 64 ? 4 : 2;                  // ring slots each for K and for V
  static constexpr int BYTES = 1024 + Q_BYTES + 2 * NS * KV_BYTES + 512 + 8 * BM;
  // so much that no third CTA, which would wait for tensor memory, fits an SM
  static constexpr int SMEM = BYTES > 80 * 1024 ? BYTES : 80 * 1024;
};
// Tensor memory: the O accumulator and two S buffers of 64 columns, a half of the SM's 512 columns.
constexpr uint32_t TMEM_COLS = 256, O_COL = 0, S_COL = 128;
constexpr int W_S = 4, W_LOAD = 5, W_CHECK = 6, W_PV = 7;     // warps 0 to 3: softmax
constexpr int THREADS = 256;

__device__ __forceinline__ bool finite16(unsigned h) { return (h & 0x7c00u) != 0x7c00u; }

// Sixteen fp16 values to out: one 32-byte store where out's rows are whole sectors, else two of 16.
__device__ __forceinline__ void store16(__half* dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h, bool sectors) {
  if (sectors) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e),
                 "r"(f), "r"(g), "r"(h)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(a, b, c, d);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(e, f, g, h);
  }
}

// ---- a cluster's CTAs ----------------------------------------------------------------------------
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, int rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(rank));
  return out;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t addr, float a) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(a) : "memory");
}
__device__ __forceinline__ void st_shared(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// ---- taking over a CTA that was not launched yet -------------------------------------------------
// The answer, 16 bytes at `answer`, arrives as a transaction on `bar`.
__device__ __forceinline__ void try_cancel(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   answer),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool cancelled(uint32_t answer, int& x, int& y) {
  uint32_t ok, cx, cy;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, r;\n\t}"
      : "=r"(ok), "=r"(cx), "=r"(cy)
      : "r"(answer)
      : "memory");
  x = static_cast<int>(cx);
  y = static_cast<int>(cy);
  return ok != 0;
}

// A wait for the phase of `parity`, false once another role has raised the abort flag or after 2^19
// tries (2 s: a failed try takes 3.9 us).  Some role may wait for the whole of another's item, which
// 2^26 keys, the most that a call takes, keep under 0.8 s.  Small, because it is in a dozen places of
// roles that share the instruction cache; the flag is looked at only now and then, for a shared-memory
// read in a thread that issues products stalls it until they are done.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait_parity(bar, parity); ++i)
    if ((i & 1023u) == 0 && (*abort_flag != 0 || i >= (1u << 19))) return false;
  return true;
}

// Warp roles:
//   0-3      softmax: waits S(j), releases K slot, masks, takes the row maximum (moving the running
//            one, and O, only past 2^8), writes P = 2^(7 + S - m) as fp16 over the scores and arrives on
//            p_full; after an item's last tile, its output (with SPLIT the part of it for the cluster)
//   W_S      one lane issues S(j) = Q K(j)^T once K(j) landed and PV(j - 2), the last reader of its
//            buffer, is done
//   W_PV     one lane issues O += P(j) V(j) once V(j) and P(j) are there, then releases V
//   W_LOAD   finds the next item and one lane loads its Q and its K and V tiles into the ring
//   W_CHECK  looks the edge tiles' V over and passes them on to the PV issuer
// Key tiles are numbered through all of a CTA's items (j above), items too; every hand-off is an
// mbarrier, and no waiter is more than one phase behind the barrier it waits on.  Every wait is
// bounded; a role that gives up records PKV_DEV_WAIT_TIMEOUT and leaves its loop, the others give up
// in turn, and the CTA still reaches its final barrier.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 2) prompt_attention_kernel(const __grid_constant__ PromptParams p) {
  using C = Cfg<D>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  const uint32_t sq = base, sk = sq + C::Q_BYTES, sv = sk + NS * C::KV_BYTES, bars = sv + NS * C::KV_BYTES;
  // per S buffer u (key tile j uses j % 2), per ring slot b, per item slot i (item number % 2)
  auto s_full = [&](int u) { return bars + 8u * u; };
  auto p_full = [&](int u) { return bars + 16u + 8u * u; };
  auto pv_done = [&](int u) { return bars + 32u + 8u * u; };
  auto item_full = [&](int i) { return bars + 48u + 8u * i; };
  auto item_free = [&](int i) { return bars + 64u + 8u * i; };
  const uint32_t q_full = bars + 80, q_free = bars + 88, o_free = bars + 96, answered = bars + 104;
  auto k_full = [&](int b) { return bars + 112u + 8u * b; };
  auto v_full = [&](int b) { return bars + 112u + 8u * (NS + b); };
  auto k_free = [&](int b) { return bars + 112u + 8u * (2 * NS + b); };
  auto v_free = [&](int b) { return bars + 112u + 8u * (3 * NS + b); };
  auto v_ok = [&](int b) { return bars + 112u + 8u * (4 * NS + b); };     // edge tiles: looked over
  auto v_issued = [&](int b) { return bars + 112u + 8u * (5 * NS + b); };  // edge tiles: their load is on its way
  constexpr uint32_t AT = 112 + 48 * NS;                      // 16-byte aligned
  const uint32_t answer = bars + AT;
  volatile Item* items = reinterpret_cast<volatile Item*>(smem + (bars + AT + 16 - base));            // [2]
  volatile int* not_finite = reinterpret_cast<volatile int*>(smem + (bars + AT + 80 - base));         // [2]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + (bars + AT + 88 - base));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (bars + AT + 92 - base));
  static_assert(sizeof(Item) == 32 && AT % 16 == 0 && AT + 96 <= 512, "barrier area");
  // SPLIT: this CTA's place in its cluster, and its part of the item for the others to read: each row's
  // maximum and sum, and O as [D][BM] floats where the K and V rings were
  const int rank = SPLIT ? cluster_rank() : 0, parts = SPLIT ? cluster_size() : 1;
  const uint32_t part_ml = bars + 512, part_o = sk;
  static_assert(D * BM * 4 <= 2 * NS * C::KV_BYTES, "O fits in the rings");

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
    for (int u = 0; u < 2; ++u) {
      mbar_init_count(s_full(u), 1);
      mbar_init_count(p_full(u), 4);
      mbar_init_count(pv_done(u), 1);
      mbar_init_count(item_full(u), 1);
      mbar_init_count(item_free(u), 7);                       // 4 softmax warps, both issuers, the checker
    }
    mbar_init_count(q_full, 1);
    mbar_init_count(q_free, 1);
    mbar_init_count(o_free, 4);
    mbar_init_count(answered, 1);
    for (int b = 0; b < NS; ++b) {
      mbar_init_count(k_full(b), 1);
      mbar_init_count(v_full(b), 1);
      mbar_init_count(k_free(b), 4);
      mbar_init_count(v_free(b), 1);
      mbar_init_count(v_ok(b), 1);
      mbar_init_count(v_issued(b), 1);
    }
    *abort_flag = 0;
    if (SPLIT) items[0].rows = 0;
  }
  if (SPLIT && tid < BM) st_shared(part_ml + tid * 8, -INFINITY, 0.f);
  if (tid == 64) {
    prefetch_tensormap(&p.tmap_q);
    prefetch_tensormap(&p.tmap_k);
    prefetch_tensormap(&p.tmap_v);
  }
  pkv::pdl_wait();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto t_s = [&](int u) { return tmem + S_COL + 64u * u; };
  const uint32_t t_o = tmem + O_COL;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_phase(bar, parity, abort_flag); };
  auto give_up = [&]() {
    if (!*abort_flag) record_error(PKV_DEV_WAIT_TIMEOUT);
    *abort_flag = 1;
  };
  // The same for a softmax warp: its lanes leave the loop together (with one arrival a warp on p_full, 66.9 ->
  // 65.8 us for chunks at D = 64; one lane that waits for the others took 72, and in the loader's and the
  // checker's waits the larger code costs more than it saves).
  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
#pragma unroll 1
    for (uint32_t i = 1; !__all_sync(0xffffffffu, mbar_try_wait_parity(bar, parity)); ++i)
      if ((i & 1023u) == 0 && (__any_sync(0xffffffffu, *abort_flag != 0) || i >= (1u << 19))) return false;
    return true;
  };
  // the next item, once it is there; n_tiles 0 ends the loop
  auto take_item = [&](int it, Item& item) {
    if (!wait(item_full(it & 1), (it >> 1) & 1)) return false;
    const volatile Item& x = items[it & 1];
    item.q_row = x.q_row;
    item.rows = x.rows;
    item.first_pos = x.first_pos;
    item.k_row = x.k_row;
    item.keys = x.keys;
    item.n_tiles = x.n_tiles;
    item.edge = x.edge;
    item.head = x.head;
    return true;
  };
  bool failed = false;

  if (warp == W_LOAD) {
    // ---------------- items and loads ----------------
    ItemFinder finder;
    auto ask = [&]() {
      mbar_arrive_expect_tx(answered, 16);
      try_cancel(answer, answered);
    };
    int x = blockIdx.x / parts, y = blockIdx.y, j = 0, it = 0, asked = 0;
    int k_issued = 0, v_issued_n = 0, q_issued = 0;
    while (true) {
      Item item;
      const bool real = finder.find(p.layout, y * (static_cast<int>(gridDim.x) / parts) + x, lane, item,
                                    [](int code) { record_error(code); });
      if (SPLIT && real) {
        // this CTA's key tiles
        const int use = item.n_tiles < kSplitTiles / 2 ? 1 : min(parts, item.n_tiles / 2);
        const int t0 = item.n_tiles * min(rank, use) / use;
        item.n_tiles = item.n_tiles * min(rank + 1, use) / use - t0;
        item.first_pos -= t0 * BN;
        item.k_row += t0 * BN;
        item.keys -= t0 * BN;
        item.edge = max(0, item.edge - t0);
      }
      if (lane == 0) {
        if (real) {
          const int slot = it & 1;
          if (it >= 2 && !wait(item_free(slot), ((it >> 1) - 1) & 1)) failed = true;
          if (!failed) {
            volatile Item& out = items[slot];
            out.q_row = item.q_row;
            out.rows = item.rows;
            out.first_pos = item.first_pos;
            out.k_row = item.k_row;
            out.keys = item.keys;
            out.n_tiles = item.n_tiles;
            out.edge = item.edge;
            out.head = item.head;
            not_finite[slot] = 0;
            mbar_arrive(item_full(slot));
          }
          const int kvh = item.head / p.group;
          for (int i = 0; i < item.n_tiles && !failed; ++i, ++j) {
            const int b = j % NS;
            // Rows past the sequence's end are its neighbour's (or zeros past the tensor): K's scores are
            // masked, V's rows are looked over.
            if (j >= NS && !wait(k_free(b), (j / NS - 1) & 1)) {
              failed = true;
              break;
            }
            mbar_arrive_expect_tx(k_full(b), C::KV_BYTES);
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_3d(sk + b * C::KV_BYTES + half * (BN * 128), &p.tmap_k, half * 64, kvh, item.k_row + i * BN, k_full(b));
            ++k_issued;
            if (i == 0) {
              // Q, once the last item's scores are computed.  Rows past the sequence's queries read the
              // next one's (or zeros past the tensor): never stored.
              if (it >= 1 && !wait(q_free, (it - 1) & 1)) {
                failed = true;
                break;
              }
              mbar_arrive_expect_tx(q_full, C::Q_BYTES);
#pragma unroll
              for (int half = 0; half < D / 64; ++half)
                tma_load_3d(sq + half * (BM * 128), &p.tmap_q, half * 64, item.head, item.q_row, q_full);
              ++q_issued;
            }
            // the next item is asked for as late as its answer still comes in time (0.4 us): one taken
            // early is not there for a CTA that runs dry
            if (!SPLIT && i == item.n_tiles - 1) {
              ask();
              ++asked;
            }
            if (j >= NS && !wait(v_free(b), (j / NS - 1) & 1)) {
              failed = true;
              break;
            }
            mbar_arrive_expect_tx(v_full(b), C::KV_BYTES);
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_3d(sv + b * C::KV_BYTES + half * (BN * 128), &p.tmap_v, half * 64, kvh, item.k_row + i * BN, v_full(b));
            if (i >= item.edge) mbar_arrive(v_issued(b));
            ++v_issued_n;
          }
        } else if (!SPLIT) {
          ask();
          ++asked;
        }
      }
      it += real;
      j = __shfl_sync(0xffffffffu, j, 0);
      asked = __shfl_sync(0xffffffffu, asked, 0);
      failed = __shfl_sync(0xffffffffu, failed, 0);
      if (failed || SPLIT) break;
      // the answer: another CTA's place, or none left (after which none may be asked for)
      if (!__all_sync(0xffffffffu, wait(answered, (asked - 1) & 1))) {
        failed = true;
        break;
      }
      const bool more = cancelled(answer, x, y);
      fence_proxy_async_smem();                               // the answer is read before the next one is written
      __syncwarp();
      if (!more) break;
    }
    // (a role gave up) an answer on its way lands before the CTA's shared memory is released: bounded
    if (failed && asked > 0) mbar_wait(answered, (asked - 1) & 1);
    if (lane == 0) {
      if (!failed) {
        const int slot = it & 1;
        if (it >= 2 && !wait(item_free(slot), ((it >> 1) - 1) & 1)) {
          failed = true;
        } else {
          items[slot].n_tiles = 0;
          mbar_arrive(item_full(slot));
        }
      }
      if (failed) give_up();
      if (*abort_flag) {
        // let the copies this lane issued land (bounded) before the CTA's shared memory is released
        for (int t = max(0, k_issued - NS); t < k_issued; ++t) mbar_wait(k_full(t % NS), (t / NS) & 1);
        for (int t = max(0, v_issued_n - NS); t < v_issued_n; ++t) mbar_wait(v_full(t % NS), (t / NS) & 1);
        if (q_issued > 0) mbar_wait(q_full, (q_issued - 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == W_CHECK) {
    // ---------------- the edge tiles' V: values that are not finite, and what is past the end ----------------
    uint32_t edge_phase = 0;                                  // bit b: parity of slot b's next edge tile
    int j0 = 0;
    for (int it = 0;; ++it) {
      Item item;
      if (!__all_sync(0xffffffffu, take_item(it, item))) {
        failed = true;
        break;
      }
      if (item.n_tiles == 0) break;
      for (int i = item.edge; i < item.n_tiles; ++i) {
        const int j = j0 + i, b = j % NS;
        // v_full's phase is this tile's only once its load is issued (tile j - NS has landed by then): a
        // wait for it before that could be for an earlier tile of the same parity
        if (!__all_sync(0xffffffffu, wait(v_issued(b), (edge_phase >> b) & 1) && wait(v_full(b), (j / NS) & 1))) {
          failed = true;
          break;
        }
        edge_phase ^= 1u << b;
        unsigned char* tile = smem + (sv + b * C::KV_BYTES - base);
        // 0 times a value is a NaN if the value is not finite; sums of those are NaN
        const __half2 zero = __float2half2_rn(0.f);
        __half2 acc[4] = {zero, zero, zero, zero};
#pragma unroll 8
        for (int c = lane; c < C::KV_BYTES / 16; c += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + c * 16);
          acc[0] = __hfma2(*reinterpret_cast<const __half2*>(&x.x), zero, acc[0]);
          acc[1] = __hfma2(*reinterpret_cast<const __half2*>(&x.y), zero, acc[1]);
          acc[2] = __hfma2(*reinterpret_cast<const __half2*>(&x.z), zero, acc[2]);
          acc[3] = __hfma2(*reinterpret_cast<const __half2*>(&x.w), zero, acc[3]);
        }
        const __half2 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
        if (__any_sync(0xffffffffu, __hisnan(__low2half(sum)) || __hisnan(__high2half(sum)))) {
          for (int c = lane; c < C::KV_BYTES / 16; c += 32) {
            const int key = i * BN + (c / 8) % BN;            // 128-byte rows, a half of the head dimension each
            unsigned* w = reinterpret_cast<unsigned*>(tile + c * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const unsigned x = w[e];
              if (!finite16(x) || !finite16(x >> 16)) {
                if (key < item.keys) not_finite[it & 1] = 1;
                w[e] = (finite16(x) ? x & 0xffffu : 0u) | (finite16(x >> 16) ? x & 0xffff0000u : 0u);
              }
            }
          }
          __threadfence_block();
          fence_proxy_async_smem();                           // these stores -> tensor-core reads
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(v_ok(b));
      }
      if (failed) break;
      j0 += item.n_tiles;
      if (lane == 0) mbar_arrive(item_free(it & 1));
    }
    if (failed) give_up();
  } else if (warp == W_S) {
    // ---------------- S = Q K^T issue (one lane) ----------------
    if (lane == 0) {
      constexpr uint32_t IDESC_QK = umma_idesc_f16(BM, BN, false);
      const uint64_t a0 = umma_smem_desc(sq, 16, 1024);
      int j = 0;
      for (int it = 0; !failed; ++it) {
        Item item;
        if (!take_item(it, item) || (item.n_tiles > 0 && !wait(q_full, it & 1))) failed = true;
        if (failed || item.n_tiles == 0) break;
        mbar_arrive(item_free(it & 1));
        for (int i = 0; i < item.n_tiles; ++i, ++j) {
          const int u = j & 1;
          if (!wait(k_full(j % NS), (j / NS) & 1) || (j >= 2 && !wait(pv_done(u), ((j - 2) >> 1) & 1))) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint64_t b0 = umma_smem_desc(sk + (j % NS) * C::KV_BYTES, 16, 1024);
          const uint32_t d = t_s(u);
          umma_ss(d, a0, b0, IDESC_QK, 0u);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk)
            umma_ss(d, a0 + (((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4),
                    b0 + (((kk >> 2) * (BN * 128) + (kk & 3) * 32) >> 4), IDESC_QK, 1u);
          umma_commit(s_full(u));
        }
        if (!failed) umma_commit(q_free);
      }
      if (failed) {
        give_up();
        if (j > 0) mbar_wait(s_full((j - 1) & 1), ((j - 1) >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == W_PV) {
    // ---------------- O += P V issue (one lane) ----------------
    if (lane == 0) {
      constexpr uint32_t IDESC_PV = umma_idesc_f16(BM, D, true);
      uint32_t edge_phase = 0;
      int j = 0;
      for (int it = 0; !failed; ++it) {
        Item item;
        if (!take_item(it, item)) failed = true;
        if (failed || item.n_tiles == 0) break;
        mbar_arrive(item_free(it & 1));
        for (int i = 0; i < item.n_tiles; ++i, ++j) {
          const int u = j & 1, b = j % NS;
          bool ok = wait(v_full(b), (j / NS) & 1);
          if (ok && i >= item.edge) {
            ok = wait(v_ok(b), (edge_phase >> b) & 1);
            edge_phase ^= 1u << b;
          }
          // the first product overwrites the accumulator: the last item's output has been read
          if (ok && i == 0 && it > 0) ok = wait(o_free, (it - 1) & 1);
          if (!ok || !wait(p_full(u), (j >> 1) & 1)) {
            failed = true;
            break;
          }
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
      if (failed) {
        give_up();
        if (j > 0) mbar_wait(pv_done((j - 1) & 1), ((j - 1) >> 1) & 1);
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax and output ----------------
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    int j = 0;
    for (int it = 0; !failed; ++it) {
      Item item;
      // decisions stay warp-uniform: the tcgen05.ld/st below are warp-collective
      if (!__all_sync(0xffffffffu, take_item(it, item))) failed = true;
      if (failed || item.n_tiles == 0) break;
      const int pos = item.first_pos + tid;
      float l = 0.f, m_ref = -INFINITY;
      for (int i = 0; i < item.n_tiles; ++i, ++j) {
        const int u = j & 1;
        const uint32_t ts = t_s(u);
        if (!warp_wait(s_full(u), (j >> 1) & 1)) {
          failed = true;
          break;
        }
        tc_fence_after();
        if (lane == 0) mbar_arrive(k_free(j % NS));
        float sv_[BN];
        tmem_ld32_nowait(ts + lane_off, *reinterpret_cast<float(*)[32]>(sv_));
        tmem_ld32_nowait(ts + lane_off + 32, *reinterpret_cast<float(*)[32]>(sv_ + 32));
        tmem_ld_wait();
        const int key0 = i * BN;
        if (__any_sync(0xffffffffu, key0 + BN - 1 > pos)) {                 // keys after the query (and past the end)
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (key0 + c > pos) sv_[c] = -INFINITY;
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
          if (!warp_wait(pv_done((j - 1) & 1), ((j - 1) >> 1) & 1)) {
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
        if (lane == 0) mbar_arrive(p_full(u));
      }
      if (!failed) failed = !warp_wait(pv_done((j - 1) & 1), ((j - 1) >> 1) & 1);
      if (failed) break;
      tc_fence_after();
      // the output, 32 columns at a time: each thread normalises and stores its own row, whole 32-byte
      // sectors at once; the next columns are read meanwhile
      const float inv = 1.f / l;                              // a query sees its own key at least
      const bool fix = not_finite[it & 1] != 0;
      __half* dst = p.out + (static_cast<size_t>(item.q_row + tid) * p.layout.num_heads + item.head) * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        float x[32];
        tmem_ld32(t_o + lane_off + c * 32, x);
        if (c == D / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(o_free);
            mbar_arrive(item_free(it & 1));
          }
        }
        if constexpr (SPLIT) {
          if (fix) {                                          // of this part's tiles only: the others' have their own factor
            const int last = tid < item.rows ? min(pos, min(item.keys, item.n_tiles * BN) - 1) : -1;
            const __half* v = p.v + (item.k_row + static_cast<int64_t>(item.edge) * BN) * p.v_stride +
                              static_cast<int64_t>(item.head / p.group) * D + c * 32;
#pragma unroll 1
            for (int t = item.edge * BN; t <= last; ++t, v += p.v_stride)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!finite16(__half_as_ushort(v[e]))) x[e] += __half2float(v[e]);
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) st_shared(part_o + ((c * 32 + e) * BM + tid) * 4, x[e]);
          continue;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) fma2(x[e], x[e + 1], x[e], x[e + 1], inv, 0.f);
        if (tid < item.rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 16)
            store16(dst + c * 32 + e, pack_half2(x[e], x[e + 1]), pack_half2(x[e + 2], x[e + 3]), pack_half2(x[e + 4], x[e + 5]),
                    pack_half2(x[e + 6], x[e + 7]), pack_half2(x[e + 8], x[e + 9]), pack_half2(x[e + 10], x[e + 11]),
                    pack_half2(x[e + 12], x[e + 13]), pack_half2(x[e + 14], x[e + 15]), p.out_sectors);
        }
        __syncwarp();
      }
      if constexpr (SPLIT) {
        st_shared(part_ml + tid * 8, m_ref, l);
      } else if (fix) {
        // values that are not finite in the edge tiles were left out: added to the stored row where the
        // query sees them (rare, so its code is small rather than fast)
        const int last = tid < item.rows ? min(pos, item.keys - 1) : -1;
        const __half* v = p.v + (item.k_row + static_cast<int64_t>(item.edge) * BN) * p.v_stride + static_cast<int64_t>(item.head / p.group) * D;
#pragma unroll 1
        for (int t = item.edge * BN; t <= last; ++t, v += p.v_stride)
#pragma unroll 1
          for (int e = 0; e < D; ++e)
            if (!finite16(__half_as_ushort(v[e]))) dst[e] = __float2half_rn(__half2float(dst[e]) + __half2float(v[e]));
        __syncwarp();
      }
    }
    if (failed) give_up();
  }

  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();                                           // every CTA's part is there
    const int rows = items[0].rows;
    if (tid < rows) {
      // a row to a thread, this CTA's D / parts columns of it, by the log-sum-exp identity
      const int columns = D / parts;
      float f[kMostParts];                                    // the parts' factors
      uint32_t o_of[kMostParts];
      bool has[kMostParts];                                   // not where a part saw no key, or had none
      float M = -INFINITY, L = 0.f;
      float2 ml[kMostParts];
#pragma unroll
      for (int r = 0; r < kMostParts; ++r)
        ml[r] = r < parts ? ld_cluster2(map_to_rank(part_ml + tid * 8, r)) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int r = 0; r < kMostParts; ++r) M = fmaxf(M, ml[r].x);
#pragma unroll
      for (int r = 0; r < kMostParts; ++r) {
        has[r] = ml[r].x != -INFINITY || ml[r].y != 0.f;
        f[r] = exp2f(ml[r].x - M);
        if (has[r]) L = fmaf(ml[r].y, f[r], L);
        o_of[r] = map_to_rank(part_o + (rank * columns * BM + tid) * 4, r < parts ? r : 0);
      }
      const float inv = 1.f / L;
      __half* dst = p.out + (static_cast<size_t>(items[0].q_row + tid) * p.layout.num_heads + items[0].head) * D + rank * columns;
#pragma unroll 1
      for (int c = 0; c < columns; c += 8) {
        float v[kMostParts][8], o[8];
#pragma unroll
        for (int r = 0; r < kMostParts; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[r][e] = has[r] ? ld_cluster(o_of[r] + (c + e) * BM * 4) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[e] = 0.f;
#pragma unroll
          for (int r = 0; r < kMostParts; ++r) o[e] = has[r] ? fmaf(v[r][e], f[r], o[e]) : o[e];
        }
        *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack_half2(o[0] * inv, o[1] * inv), pack_half2(o[2] * inv, o[3] * inv),
                                                        pack_half2(o[4] * inv, o[5] * inv), pack_half2(o[6] * inv, o[7] * inv));
      }
    }
    __syncwarp();
    cluster_sync();                                           // nobody reads this CTA's part any more
  }
  // every tensor-memory access is done (tcgen05.ld and .st wait inline, the products are committed)
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// x [T][H][D] fp16, tokens `stride` elements apart, as the 3-D tensor (D, H, T); a box is `box_tokens`
// tokens of one head and one 64-element half of the head dimension, written with the 128-byte swizzle.
int encode_rows_map(CUtensorMap* map, const void* x, int D, int H, int T, int64_t stride, int box_tokens) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return pkv::fail(PKV_ERR_CUDA, "pkv_prompt_attention: cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t elem[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(x), dims, strides, box, elem,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return pkv::fail(PKV_ERR_CUDA, "pkv_prompt_attention: tensor map encoding failed (%d)", static_cast<int>(r));
  return PKV_OK;
}

template <int D, bool SPLIT>
int launch(const PromptParams& p, long long tiles, int parts, cudaStream_t st) {
  using C = Cfg<D>;
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) {
    std::lock_guard<std::mutex> g(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(prompt_attention_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "pkv_prompt_attention setup: %s", cudaGetErrorString(e));
  const dim3 grid(static_cast<unsigned>(tiles * parts), p.layout.num_heads);
  e = SPLIT ? pkv::launch_pdl_cluster(prompt_attention_kernel<D, SPLIT>, grid, dim3(THREADS), C::SMEM, st, parts, p)
            : pkv::launch_pdl(prompt_attention_kernel<D, SPLIT>, grid, dim3(THREADS), C::SMEM, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "pkv_prompt_attention launch: %s", cudaGetErrorString(e));
  return PKV_OK;
}

}  // namespace

namespace pkv {
int device_error_word_prompt(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_prompt));
}
}  // namespace pkv

extern "C" {

int pkv_prompt_attention(const uint16_t* q, const uint16_t* key, const uint16_t* value, const int32_t* query_start,
                         const int32_t* key_start, int num_seqs, int total_q, int total_k, int max_query_len,
                         int num_heads, int num_kv_heads, int head_dim, int64_t q_stride, int64_t key_stride,
                         int64_t value_stride, float scale, uint16_t* out, void* stream) {
  const char* fn = "pkv_prompt_attention";
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_query_len < 0 || num_heads <= 0 || num_kv_heads <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG,
                     "%s: num_seqs=%d total_q=%d total_k=%d max_query_len=%d num_heads=%d num_kv_heads=%d", fn, num_seqs,
                     total_q, total_k, max_query_len, num_heads, num_kv_heads);
  if (num_heads % num_kv_heads)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_heads=%d is not a multiple of num_kv_heads=%d", fn, num_heads,
                     num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (num_seqs > 65535 || num_heads > 65535)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: num_seqs/num_heads above 65535", fn);
  if (total_q > (1 << 26) || total_k > (1 << 26))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^26 tokens", fn);
  if (total_k == 0) return pkv::fail(PKV_ERR_INVALID_ARG, "%s: queries but no keys", fn);
  if (!q || !key || !value || !query_start || !out) return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(key) || !aligned16(value) || !aligned16(out))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q, key, value and out must be 16-byte aligned", fn);
  const int64_t q_row = static_cast<int64_t>(num_heads) * head_dim, k_row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (q_stride < q_row || key_stride < k_row || value_stride < k_row || q_stride % 8 || key_stride % 8 || value_stride % 8)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: strides must be multiples of 8 and at least a token's length", fn);
  if (!std::isfinite(scale) || !(scale > 0.f))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: scale must be finite and positive", fn);
  PromptParams p{};
  p.layout.qstart = query_start;
  p.layout.kstart = key_start ? key_start : query_start;
  p.layout.num_seqs = num_seqs;
  p.layout.num_heads = num_heads;
  p.layout.total_q = total_q;
  p.layout.total_k = total_k;
  const long long tiles = lay_out(p.layout, max_query_len);
  if (tiles * num_heads > INT_MAX)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 query tiles over all heads", fn);
  int rc = encode_rows_map(&p.tmap_q, q, head_dim, num_heads, total_q, q_stride, BM);
  if (rc == PKV_OK) rc = encode_rows_map(&p.tmap_k, key, head_dim, num_kv_heads, total_k, key_stride, BN);
  if (rc == PKV_OK) rc = encode_rows_map(&p.tmap_v, value, head_dim, num_kv_heads, total_k, value_stride, BN);
  if (rc != PKV_OK) return rc;
  p.v = reinterpret_cast<const __half*>(value);
  p.out = reinterpret_cast<__half*>(out);
  p.v_stride = value_stride;
  p.group = num_heads / num_kv_heads;
  p.out_sectors = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int parts = 1;
  while (parts < kMostParts && tiles * num_heads * parts * 2 <= kResident && (total_k - total_q / 2) / num_seqs >= kSplitTiles * BN)
    parts *= 2;
  if (parts > 1) rc = head_dim == 128 ? launch<128, true>(p, tiles, parts, st) : launch<64, true>(p, tiles, parts, st);
  else rc = head_dim == 128 ? launch<128, false>(p, tiles, 1, st) : launch<64, false>(p, tiles, 1, st);
  if (rc == PKV_OK) pkv::clear_error();
  return rc;
}

}  // extern "C"
