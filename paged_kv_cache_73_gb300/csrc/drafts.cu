// Around the attention over drafted tokens, for sm_103a: which drafts the target model's
// distributions let stay, and the kept ones' rows on their way to the places behind the context.
//
// Verification.  Node 0 of a sequence's drafts is its last certain token; p_c is the target's
// distribution behind node c, q_c the one that the drafts behind c were drawn from.  The children of
// the current node c are tried in ascending order, with R = p_c and M = sum R = 1 at first:
//   child j with token x stays if u_j M q_c(x) < R(x)   (q = 1 where the drafts have no distribution);
//   if not, R <- max(R - M q_c, 0), M <- sum R          (without one: M <- M - R(x), R(x) <- 0).
// Where none stays the next token is drawn from R: the least index whose running sum passes u_0 sum R.
// So each kept and drawn token is distributed as the target alone would draw it.
//
// After k refusals at a node R = max(p - C q, 0) with C = 1 + M_1 + .. + M_(k-1), the product rounded down: a pass over
// a row costs one product a value however often something was refused there.  (One product for each refusal,
// rounded by itself, differs by a unit now and then, and with 30 refusals at a node 16 sequences of 131072 tokens
// take 2302 us for 428.)
//
// R and M are whole numbers in units of 2^-60 (fp32 values up to 1 lose only what is below 2^-60):
// sums of whole numbers do not depend on their order, and the drawn token is the same however a row is
// cut up.  In fp32 a running sum over 131072 values is off by more than most of its steps.
//
// What it has to read: a few values a node, and of the vocabulary only the rows of nodes where a
// draft was refused, or where the path ends.  Those are read once per refusal, by the CTAs of a cluster (a
// row's later passes come from L2), each warp a piece of its own; the last pass's piece sums
// find the piece that holds the drawn token, and the warps of its CTA read that piece again.  The cluster's
// first CTA decides and tells the others, so that all of them come to the same barriers.  It writes into their
// shared memory, so the first barrier, which tells that they run, is arrived at ahead of all else and waited for
// behind the loads of the nodes.
//
// The move.  A path's nodes go up with their place, path[i] >= i, so a thread that takes its 16 bytes of every
// kept row in the path's order reads each row before it overwrites it: no staging, no barrier.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <functional>
#include <new>
#include <type_traits>
#include <vector>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_drafts = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_drafts, 0, code); }

typedef unsigned long long u64;

constexpr unsigned FULL = 0xffffffffu;
constexpr int kMaxNodes = 1024;      // of a sequence
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMostCtas = 8;         // of a cluster
constexpr int kResident = 4;         // CTAs to an SM: three leave 64 chains over 50257 tokens at 20 us for 16
// A cluster has eight CTAs, less where all of them would be more than kEnough: 256 chains over 32000 tokens take 42 us
// with eight each, 31 with four; 128 trees over 131072, where refusals follow one another, 77 with eight, 94 with four.
constexpr int kEnough = 1024;
constexpr u64 kOne = 1ull << 60, kMost = 1ull << 61;

// floor(p 2^60) of p in [0, 1]; what is no probability (a NaN, negative, above 1 by more than 2^-10, as rounded
// softmaxes are not) sets `bad`, and counts as 0 or 1
__device__ __forceinline__ u64 whole(float p, bool& bad) {
  bad |= !(p >= 0.f && p <= 1.0009765625f);
  const unsigned b = p >= 0.f ? __float_as_uint(fminf(p, 1.f)) & 0x7fffffffu : 0u;
  const int e = static_cast<int>(b >> 23) - 90;
  const u64 m = (b & 0x7fffffu) | 0x800000u;
  return e >= 0 ? m << e : e > -24 ? m >> -e : 0;
}
// The same of values that are all in [0, 1] (largest: the bits of the largest met, so that the
// others, whose bits are above those of 1, are noticed): a shift of the 24-bit mantissa from the top.
constexpr unsigned kOneBits = 0x3f800000u;
__device__ __forceinline__ u64 whole_fast(float p, unsigned& largest) {
  const unsigned b = __float_as_uint(p);
  largest = max(largest, b);
  return (static_cast<u64>((b << 5) & 0x0fffffe0u | 0x10000000u) << 32) >> min(127u - (b >> 23), 63u);
}
// floor(a b / 2^60), a and b up to 2^61
__device__ __forceinline__ u64 part_of(u64 a, u64 b) { return __umul64hi(a << 2, b << 2); }
// What refusals take from a value: C q with C = whole + part / 2^60; off - p is what counts, so no more than 2.
struct Taken {
  unsigned whole;
  u64 part;
};
__device__ __forceinline__ u64 less(u64 p, u64 q, const Taken& c) {
  const u64 high = static_cast<u64>(static_cast<unsigned>(q >> 32)) * c.whole;
  const u64 off = high >> 29 ? kMost : q * c.whole + part_of(c.part, q);
  return p > off ? p - off : 0;
}
// sums that stay below 2^62 whatever the rows hold
__device__ __forceinline__ u64 add_most(u64 a, u64 b) {
  const u64 c = a + b;
  return c < kMost ? c : kMost;
}

struct VerifyParams {
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* query_start;
  const float* uniforms;
  int32_t* path;
  int32_t* path_len;
  int32_t* next_token;
  int64_t target_stride, draft_stride;
  int num_seqs, total_q, vocab, max_path;
};

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
// The two halves of a barrier that only tells that every CTA of the cluster runs: shared memory of one that does
// not yet may not be written to.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t map_to_rank(const void* p, int rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(out)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return out;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A sequence's nodes, as the first CTA keeps them.
struct Nodes {
  int parent[kMaxNodes];
  int token[kMaxNodes];
  u64 has[kMaxNodes];     // p and q of the node's token behind its parent, and the node's own u
  u64 drawn[kMaxNodes];
  u64 u[kMaxNodes];
  unsigned char stays[kMaxNodes];  // where no sibling before it was refused
};

// What the first CTA tells the others: a pass over row `row` with the first `refused` of its refusals, and
// whether the next token is drawn from what it leaves.
struct Order {
  int row, refused, last;
  unsigned taken_whole;
  u64 taken_part, u0;
};

__global__ void __launch_bounds__(kThreads, kResident) verify_draft_kernel(const VerifyParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  int* refused_x = reinterpret_cast<int*>(smem);                      // without draft distributions: the refused tokens
  Nodes& nodes = *reinterpret_cast<Nodes*>(smem + kMaxNodes * 4);     // the first CTA's only
  __shared__ Order order;
  __shared__ u64 cta_sum[2][kMostCtas];
  __shared__ u64 warp_sum[kWarps], part_sum[kWarps];
  __shared__ int cta_bad[2][kMostCtas];

  cluster_arrive_relaxed();
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int rank = cluster_rank(), ctas = cluster_size(), s = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q0 = p.query_start[s], n = p.query_start[s + 1] - q0;
  // the same in every CTA of the cluster, unless the caller changes it meanwhile: the first CTA's view counts
  int ok = n > 0 && n <= kMaxNodes && q0 >= 0 && q0 <= p.total_q - n;
  if (rank == 0) {
    if (tid == 0 && n != 0 && !ok) record_error(PKV_DEV_BAD_QUERY_RANGE);
    if (ok) {
      for (int j = tid; j < n; j += kThreads) {
        const int parent = j == 0 ? -1 : p.parents[q0 + j], x = p.tokens[q0 + j];
        bool bad = false;
        const u64 u = min(whole(p.uniforms[q0 + j], bad), kOne - 1);   // 1 would pass over every token
        u64 has = 0, drawn = kOne;
        int from = parent;
        if (parent >= j) {
          record_error(PKV_DEV_BAD_TREE);
          from = -1;
        } else if (parent >= 0) {
          if (x < 0 || x >= p.vocab) {
            record_error(PKV_DEV_BAD_TOKEN);
            from = -1;
          } else {
            has = whole(p.target[static_cast<int64_t>(q0 + parent) * p.target_stride + x], bad);
            if (p.draft != nullptr) drawn = whole(p.draft[static_cast<int64_t>(q0 + parent) * p.draft_stride + x], bad);
          }
        }
        if (bad) record_error(PKV_DEV_BAD_PROBABILITY);
        nodes.parent[j] = from;
        nodes.token[j] = x;
        nodes.has[j] = has;
        nodes.drawn[j] = drawn;
        nodes.u[j] = u;
        nodes.stays[j] = part_of(drawn, u) < has;
      }
    }
    __syncthreads();
  }

  // the walk's state, in the first CTA's first warp
  int at = 0, size = 1, next = 1, k = 0;
  u64 share = kOne;
  Taken taken{0, 0};
  bool ended = false;                                         // the row's sum is all that is left to find
  const int most = p.max_path;
  if (rank == 0 && tid < p.max_path) p.path[static_cast<int64_t>(s) * most + tid] = tid == 0 && ok ? 0 : -1;
  if (rank == 0)
    for (int i = tid + kThreads; i < most; i += kThreads) p.path[static_cast<int64_t>(s) * most + i] = -1;
  __syncthreads();
  cluster_wait();                                             // from here on the first CTA writes to the others

  for (int pass = 0;; ++pass) {
    if (rank == 0 && warp == 0) {
      // on from the node where the last refusal left it, to the next refusal that needs its row's sum
      bool wants = false;
      while (ok && !ended && !wants) {
        // the next child of `at` from `next` on
        int j = n;
        if (size < most) {
          for (int base = next & ~31; base < n; base += 32) {
            const int c = base + lane;
            const unsigned hit = __ballot_sync(FULL, c >= next && c < n && nodes.parent[c] == at);
            if (hit) {
              j = base + __ffs(hit) - 1;
              break;
            }
          }
        }
        if (j >= n) {
          ended = true;
          break;
        }
        next = j + 1;
        bool stays = nodes.stays[j] != 0;
        u64 has = nodes.has[j];
        if (k > 0) {
          const u64 drawn = nodes.drawn[j];
          if (p.draft != nullptr) {
            has = less(has, drawn, taken);
          } else {
            for (int i = 0; i < k; ++i)
              if (refused_x[i] == nodes.token[j]) has = 0;
          }
          stays = part_of(part_of(share, drawn), nodes.u[j]) < has;
        }
        if (stays) {
          if (lane == 0) p.path[static_cast<int64_t>(s) * most + size] = j;
          ++size;
          at = j;
          share = kOne;
          k = 0;
          taken = Taken{0, 0};
        } else if (p.draft != nullptr) {
          const u64 c = taken.part + share;
          taken.whole += static_cast<unsigned>(c >> 60);
          taken.part = c & (kOne - 1);
          ++k;
          wants = true;                                       // M is the sum of what is left
        } else if (has > 0) {                                 // a token that is left nothing is noted already, or was 0
          __syncwarp();
          if (lane < ctas) st_cluster(map_to_rank(refused_x + k, lane), nodes.token[j]);
          ++k;
          share -= min(share, has);
        }
        __syncwarp();
      }
      // a refusal after which no sibling is left ends the path as well
      if (ok && wants) {
        int more = 0;
        for (int base = next & ~31; base < n && !more; base += 32) {
          const int c = base + lane;
          more = __any_sync(FULL, c >= next && c < n && nodes.parent[c] == at);
        }
        if (!more) ended = true;
      }
      if (lane < ctas) {
        const uint32_t to = map_to_rank(&order, lane);
        st_cluster(to, ok ? q0 + at : -1);
        st_cluster(to + 4, k);
        st_cluster(to + 8, static_cast<int>(ended));
        st_cluster(to + 12, static_cast<int>(taken.whole));
        st_cluster(to + 16, taken.part);
        st_cluster(to + 24, ok ? nodes.u[0] : 0ull);
      }
    }
    cluster_sync();
    const Order o = order;
    if (o.row < 0) break;                                     // no nodes
    const float* prow = p.target + static_cast<int64_t>(o.row) * p.target_stride;
    const float* qrow = p.draft == nullptr ? nullptr : p.draft + static_cast<int64_t>(o.row) * p.draft_stride;
    // This warp's piece of the row, in lines of 128 values that start at multiples of 16 bytes: value i of the row is
    // value i + shift of the lines.  Where the two rows lie differently, or the strides are odd, a value at a time.
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(prow) >> 2 & 3);
    const bool wide = qrow == nullptr || static_cast<int>(reinterpret_cast<uintptr_t>(qrow) >> 2 & 3) == shift;
    const int lines = (p.vocab + shift + 127) / 128, pieces = ctas * kWarps, mine = rank * kWarps + warp;
    auto first_line = [&](int piece) { return static_cast<int>(static_cast<int64_t>(lines) * piece / pieces); };
    const int first = first_line(mine), end = first_line(mine + 1);
    int refused = o.refused;
    const Taken all_taken{o.taken_whole, o.taken_part};
    bool bad = false, slow = false;
    auto left = [&](int i) {                                  // R(i) after the refusals
      u64 r = whole(prow[i], bad);
      if (qrow != nullptr) {
        if (refused > 0) r = less(r, whole(qrow[i], bad), all_taken);
      } else {
        for (int j = 0; j < refused; ++j)
          if (refused_x[j] == i) r = 0;
      }
      return r;
    };
    // the sum over lines [from, to) of this lane's values, one by one
    auto slow_sum = [&](int from, int to) {
      u64 sum = 0;
#pragma unroll 1
      for (int k = from * 128 + lane; k < to * 128; k += 32)
        if (k >= shift && k - shift < p.vocab) sum = add_most(sum, left(k - shift));
      return sum;
    };
    // the same of whole lines, 16 bytes at a time; STEPS: refusals (2: two or more)
    auto fast_sum = [&](auto steps, int from, int to) {
      constexpr int STEPS = decltype(steps)::value, FLY = STEPS == 0 ? 4 : 2;
      u64 sum = 0;
      unsigned largest = 0;
      const float4* pv = reinterpret_cast<const float4*>(prow - shift) + lane;
      const float4* qv = STEPS == 0 ? nullptr : reinterpret_cast<const float4*>(qrow - shift) + lane;
#pragma unroll 1
      for (int line = from; line < to; line += FLY) {
        float4 x[FLY], y[FLY];
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
          x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (line + u < to) {
            x[u] = pv[(line + u) * 32];
            if (STEPS > 0) y[u] = qv[(line + u) * 32];
          }
        }
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
          const float4 a = x[u], c = y[u];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float xe = e == 0 ? a.x : e == 1 ? a.y : e == 2 ? a.z : a.w;
            u64 r = whole_fast(xe, largest);
            if (STEPS > 0) {
              const float ye = e == 0 ? c.x : e == 1 ? c.y : e == 2 ? c.z : c.w;
              const u64 q = whole_fast(ye, largest);
              if (STEPS > 1) r = less(r, q, all_taken);
              else r = r > q ? r - q : 0;                     // the first refusal takes q
            }
            sum += r;                                         // eight at most before they are held down
          }
          if (u & 1) sum = add_most(sum, 0);
        }
      }
      if (__any_sync(FULL, largest > kOneBits)) {             // something is no probability
        sum = slow_sum(from, to);
        slow = true;
      }
      return sum;
    };
    u64 total = 0;
    int parity = pass & 1;
    for (int attempt = 0; attempt < 2; ++attempt) {
      u64 sum = 0;
      int fast_from = 0, fast_to = 0;
      if (wide) {
        // the lines that hold something else than the row's values apart
        const int from = first + (first == 0 && shift > 0 && end > 0), to = end - (end == lines && (p.vocab + shift) % 128 != 0 && end > from);
        if (first < from) sum = slow_sum(first, from);
        if (to < end) sum = add_most(sum, slow_sum(to, end));
        const u64 inner = qrow == nullptr || refused == 0 ? fast_sum(std::integral_constant<int, 0>(), from, to)
                          : refused == 1                  ? fast_sum(std::integral_constant<int, 1>(), from, to)
                                                          : fast_sum(std::integral_constant<int, 2>(), from, to);
        sum = add_most(sum, inner);
        fast_from = from;
        fast_to = to;
      } else {
        sum = slow_sum(first, end);
      }
#pragma unroll
      for (int d = 16; d > 0; d /= 2) sum = add_most(sum, __shfl_xor_sync(FULL, sum, d));
      if (qrow == nullptr && refused > 0 && !slow && sum >= kMost) {
        // held down before the refused tokens are taken off: no distribution, but what is left of it may be one
        sum = slow_sum(first, end);
        slow = true;
        for (int d = 16; d > 0; d /= 2) sum = add_most(sum, __shfl_xor_sync(FULL, sum, d));
      }
      if (qrow == nullptr) {
        // refused tokens have nothing left (slow_sum counts that)
        for (int j = 0; j < refused; ++j) {
          const int line = (refused_x[j] + shift) / 128;
          if (!slow && line >= fast_from && line < fast_to) sum -= min(sum, whole(prow[refused_x[j]], bad));
        }
      }
      if (lane == 0) warp_sum[warp] = sum;
      const int any_bad = __syncthreads_or(bad);
      if (tid == 0) {
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) all = add_most(all, warp_sum[w]);
        for (int c = 0; c < ctas; ++c) {
          st_cluster(map_to_rank(&cta_sum[parity][rank], c), all);
          st_cluster(map_to_rank(&cta_bad[parity][rank], c), any_bad);
        }
      }
      cluster_sync();
      total = 0;
      bad = false;
      for (int c = 0; c < ctas; ++c) {
        total = add_most(total, cta_sum[parity][c]);
        bad |= cta_bad[parity][c] != 0;
      }
      // The target gives nothing that the draft does not (a refusal only rounding allows): the node's own
      // distribution.  All CTAs see the same sums.
      if (!o.last || total != 0 || refused == 0) break;
      refused = 0;
      parity ^= 1;
    }
    if (!o.last) {
      share = total;
      if (bad && rank == 0 && tid == 0) record_error(PKV_DEV_BAD_PROBABILITY);
      continue;
    }
    // the drawn token
    const bool unusable = bad || total == 0 || total > kOne + kOne / 2;
    if (unusable) {
      if (rank == 0 && tid == 0) {
        record_error(PKV_DEV_BAD_PROBABILITY);
        p.next_token[s] = -1;
      }
    } else {
      u64 aim = part_of(total, o.u0);
      bool here = true;
      for (int c = 0; c < rank; ++c) {
        here &= aim >= cta_sum[parity][c];
        aim -= cta_sum[parity][c];
      }
      if (here && aim < cta_sum[parity][rank]) {
        // in this CTA: its warps share the piece that holds the token, and the one whose lines do goes through
        // them again, four values to a lane
        int piece = 0;
        while (piece < kWarps - 1 && aim >= warp_sum[piece]) aim -= warp_sum[piece++];
        const int from = first_line(rank * kWarps + piece), count = first_line(rank * kWarps + piece + 1) - from;
        const int l0 = from + count * warp / kWarps, l1 = from + count * (warp + 1) / kWarps;
        auto four = [&](int line, u64 (&r)[4]) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = line * 128 + lane * 4 + e - shift;
            r[e] = i >= 0 && i < p.vocab ? left(i) : 0;
          }
          return r[0] + r[1] + r[2] + r[3];
        };
        u64 r[4], sum = 0;
#pragma unroll 2
        for (int line = l0; line < l1; ++line) sum += four(line, r);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(FULL, sum, d);
        if (lane == 0) part_sum[warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) {
          here &= aim >= part_sum[w];
          aim -= part_sum[w];
        }
        if (here && aim < part_sum[warp]) {
#pragma unroll 1
          for (int line = l0; line < l1; ++line) {
            const u64 mine = four(line, r);
            u64 upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
              const u64 y = __shfl_up_sync(FULL, upto, d);
              if (lane >= d) upto += y;
            }
            const unsigned past = __ballot_sync(FULL, upto > aim);
            if (past) {
              if (lane == __ffs(past) - 1) {
                u64 rest = aim - (upto - mine);
                int e = 0;
                while (e < 3 && rest >= r[e]) rest -= r[e++];
                p.next_token[s] = line * 128 + lane * 4 + e - shift;
              }
              break;
            }
            aim -= __shfl_sync(FULL, upto, 31);
          }
        }
      }
    }
    break;
  }
  if (rank == 0 && tid == 0) {
    p.path_len[s] = ok ? size : 0;
    if (!ok) p.next_token[s] = -1;
  }
}

// ---- the move ------------------------------------------------------------------------------------

constexpr int kMaxLayersPerLaunch = 64;
constexpr int kFly = 8;              // rows in flight to a thread
constexpr int kStep = 64;            // of the path's places, whose slots a CTA looks up at a time

struct MoveParams {
  uint4* k[kMaxLayersPerLaunch];
  uint4* v[kMaxLayersPerLaunch];
  const int64_t* slots;
  const int32_t* query_start;
  const int32_t* path;
  const int32_t* path_len;
  int64_t num_slots;
  int total_q, max_path, num_kv_heads, log2_vec, log2_block;
};

// grid (sequences, layers, 2 x parts of a row's columns): K in the first half of z, V in the second
__global__ void __launch_bounds__(256) move_accepted_kernel(const __grid_constant__ MoveParams p) {
  __shared__ int64_t from[kStep], to[kStep];                  // a row's offset in its pool, head 0; from -1: no move
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int s = blockIdx.x, parts = gridDim.z / 2;
  const int q0 = p.query_start[s], n = p.query_start[s + 1] - q0, kept = p.path_len[s];
  const bool first = blockIdx.y == 0 && blockIdx.z == 0;
  if (kept <= 1) return;                                      // the root is where it belongs
  if (kept > p.max_path || q0 < 0 || n < 0 || q0 > p.total_q - n) {
    if (first && threadIdx.x == 0) record_error(PKV_DEV_BAD_QUERY_RANGE);
    return;
  }
  uint4* pool = static_cast<int>(blockIdx.z) < parts ? p.k[blockIdx.y] : p.v[blockIdx.y];
  const int columns = p.num_kv_heads << p.log2_vec, step = blockDim.x * parts;
  for (int i0 = 1; i0 < kept; i0 += kStep) {
    const int m = min(kStep, kept - i0);
    __syncthreads();
    for (int i = threadIdx.x; i < kStep; i += blockDim.x) {
      int64_t a = -1, b = -1;
      if (i < m) {
        const int at = i0 + i, node = p.path[static_cast<int64_t>(s) * p.max_path + at];
        if (node < at || node >= n) {
          if (first) record_error(PKV_DEV_BAD_TREE);
        } else if (node > at) {
          a = p.slots[q0 + node];
          b = p.slots[q0 + at];
          if (a >= p.num_slots || b >= p.num_slots) {
            if (first) record_error(PKV_DEV_BAD_SLOT);
            a = -1;
          }
          if (b < 0) a = -1;
        }
      }
      const int64_t row_mask = (1 << p.log2_block) - 1;
      auto offset = [&](int64_t slot) {
        return (((slot >> p.log2_block) * p.num_kv_heads << p.log2_block) + (slot & row_mask)) << p.log2_vec;
      };
      from[i] = a < 0 ? -1 : offset(a);
      to[i] = a < 0 ? 0 : offset(b);
    }
    __syncthreads();
    for (int e = (static_cast<int>(blockIdx.z) % parts) * blockDim.x + threadIdx.x; e < columns; e += step) {
      // column c of head h
      uint4* col = pool + ((static_cast<int64_t>(e >> p.log2_vec) << (p.log2_block + p.log2_vec)) + (e & ((1 << p.log2_vec) - 1)));
      for (int j0 = 0; j0 < m; j0 += kFly) {
        uint4 x[kFly];
#pragma unroll
        for (int u = 0; u < kFly; ++u)
          if (j0 + u < kStep && from[j0 + u] >= 0) x[u] = col[from[j0 + u]];
#pragma unroll
        for (int u = 0; u < kFly; ++u)
          if (j0 + u < kStep && from[j0 + u] >= 0) col[to[j0 + u]] = x[u];
      }
    }
  }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int device_error_word_drafts(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_drafts));
}
}  // namespace pkv

extern "C" {

int pkv_verify_draft(const float* target_probs, const float* draft_probs, const int32_t* tokens,
                     const int32_t* parents, const int32_t* query_start, const float* uniforms, int num_seqs,
                     int total_q, int vocab_size, int64_t target_stride, int64_t draft_stride, int max_path,
                     int32_t* path, int32_t* path_len, int32_t* next_token, void* stream) {
  const char* fn = "pkv_verify_draft";
  if (num_seqs < 0 || total_q < 0 || vocab_size <= 0 || max_path <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_seqs=%d total_q=%d vocab_size=%d max_path=%d", fn, num_seqs, total_q,
                     vocab_size, max_path);
  if (num_seqs > 1 << 20 || max_path > kMaxNodes || vocab_size > 1 << 24)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 2^20 sequences, %d nodes on a path or 2^24 tokens", fn, kMaxNodes);
  if (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: rows must be at least vocab_size apart", fn);
  if (num_seqs == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  // without nodes their arrays may be NULL
  if ((total_q > 0 && (!target_probs || !tokens || !parents || !uniforms)) || !query_start || !path || !path_len || !next_token)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  VerifyParams p{};
  p.target = target_probs;
  p.draft = draft_probs;
  p.tokens = tokens;
  p.parents = parents;
  p.query_start = query_start;
  p.uniforms = uniforms;
  p.path = path;
  p.path_len = path_len;
  p.next_token = next_token;
  p.target_stride = target_stride;
  p.draft_stride = draft_stride;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.vocab = vocab_size;
  p.max_path = max_path;
  constexpr int smem = kMaxNodes * 4 + static_cast<int>(sizeof(Nodes));
  static_assert(smem <= 47 * 1024, "fits without asking for more");
  int ctas = kMostCtas;
  while (ctas > 1 && num_seqs * ctas > kEnough) ctas /= 2;
  cudaError_t e = pkv::launch_pdl_cluster(verify_draft_kernel, dim3(num_seqs * ctas), dim3(kThreads), smem,
                                          static_cast<cudaStream_t>(stream), ctas, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  pkv::clear_error();
  return PKV_OK;
}

int pkv_move_accepted(uint16_t* const* k_caches, uint16_t* const* v_caches, int num_layers, const int64_t* slot_mapping,
                      const int32_t* query_start, const int32_t* path, const int32_t* path_len, int num_seqs,
                      int total_q, int max_path, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                      void* stream) {
  const char* fn = "pkv_move_accepted";
  if (num_layers <= 0 || num_seqs < 0 || total_q < 0 || max_path <= 0 || num_kv_heads <= 0 || num_blocks <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_layers=%d num_seqs=%d total_q=%d max_path=%d num_kv_heads=%d num_blocks=%d",
                     fn, num_layers, num_seqs, total_q, max_path, num_kv_heads, num_blocks);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: block_size %d not in {4, 8, 16, 32}", fn, block_size);
  if (num_kv_heads > 65535) return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: more than 65535 heads", fn);
  if (!k_caches || !v_caches) return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  for (int l = 0; l < num_layers; ++l)
    if (!k_caches[l] || !v_caches[l] || !aligned16(k_caches[l]) || !aligned16(v_caches[l]))
      return pkv::fail(PKV_ERR_INVALID_ARG, "%s: layer %d: a pool is null or not 16-byte aligned", fn, l);
  // a pool that is there twice would have its rows moved by two CTAs, each over what the other may have moved already
  try {
    std::vector<const void*> pools(k_caches, k_caches + num_layers);
    pools.insert(pools.end(), v_caches, v_caches + num_layers);
    std::sort(pools.begin(), pools.end(), std::less<const void*>());
    if (std::adjacent_find(pools.begin(), pools.end()) != pools.end())
      return pkv::fail(PKV_ERR_INVALID_ARG, "%s: a pool is given twice", fn);
  } catch (const std::bad_alloc&) {
    return pkv::fail(PKV_ERR_OOM, "%s: out of host memory", fn);
  }
  if (num_seqs == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if ((total_q > 0 && !slot_mapping) || !query_start || !path || !path_len)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  MoveParams p{};
  p.slots = slot_mapping;
  p.query_start = query_start;
  p.path = path;
  p.path_len = path_len;
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.total_q = total_q;
  p.max_path = max_path;
  p.num_kv_heads = num_kv_heads;
  p.log2_vec = head_dim == 128 ? 4 : 3;
  while ((1 << p.log2_block) < block_size) ++p.log2_block;
  const int columns = num_kv_heads << p.log2_vec, parts = columns > 256 * 64 ? 64 : (columns + 255) / 256;
  for (int l0 = 0; l0 < num_layers; l0 += kMaxLayersPerLaunch) {
    const int layers = num_layers - l0 < kMaxLayersPerLaunch ? num_layers - l0 : kMaxLayersPerLaunch;
    for (int l = 0; l < layers; ++l) {
      p.k[l] = reinterpret_cast<uint4*>(k_caches[l0 + l]);
      p.v[l] = reinterpret_cast<uint4*>(v_caches[l0 + l]);
    }
    cudaError_t e = pkv::launch_pdl(move_accepted_kernel, dim3(num_seqs, layers, 2 * parts), dim3(256), 0,
                                    static_cast<cudaStream_t>(stream), p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  }
  pkv::clear_error();
  return PKV_OK;
}

int pkv_tree_masks(const int32_t* parents, const int32_t* query_start, int num_seqs, int mask_words,
                   int32_t* masks_out, int32_t* depths_out) {
  const char* fn = "pkv_tree_masks";
  if (num_seqs < 0 || mask_words <= 0 || (num_seqs > 0 && (!parents || !query_start || !masks_out)))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_seqs=%d mask_words=%d or a null pointer", fn, num_seqs, mask_words);
  for (int s = 0; s < num_seqs; ++s) {
    const int64_t q0 = query_start[s], n = query_start[s + 1] - q0;
    if (q0 < 0 || n < 0 || n > static_cast<int64_t>(mask_words) * 32)
      return pkv::fail(PKV_ERR_INVALID_ARG, "%s: sequence %d has %lld nodes from %lld on, %d words a row", fn, s,
                       static_cast<long long>(n), static_cast<long long>(q0), mask_words);
  }
  // the starts go up, so no parent behind the last of them is read
  for (int s = 0; s < num_seqs; ++s) {
    const int64_t q0 = query_start[s], n = query_start[s + 1] - q0;
    for (int64_t j = 0; j < n; ++j)
      if (parents[q0 + j] >= j)
        return pkv::fail(PKV_ERR_INVALID_ARG, "%s: node %lld of sequence %d comes before its parent %d", fn,
                         static_cast<long long>(j), s, parents[q0 + j]);
  }
  for (int s = 0; s < num_seqs; ++s) {
    const int64_t q0 = query_start[s], n = query_start[s + 1] - q0;
    for (int64_t j = 0; j < n; ++j) {
      const int parent = parents[q0 + j];
      uint32_t* row = reinterpret_cast<uint32_t*>(masks_out) + (q0 + j) * mask_words;
      const uint32_t* up = reinterpret_cast<const uint32_t*>(masks_out) + (q0 + parent) * mask_words;
      for (int w = 0; w < mask_words; ++w) row[w] = parent >= 0 ? up[w] : 0;
      row[j / 32] |= 1u << (j % 32);
      if (depths_out) depths_out[q0 + j] = parent >= 0 ? depths_out[q0 + parent] + 1 : 0;
    }
  }
  pkv::clear_error();
  return PKV_OK;
}

}  // extern "C"
