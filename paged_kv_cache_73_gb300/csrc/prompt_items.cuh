// How prompt attention's grid is laid out: a flat list of items, each a tile of 128 queries of one head
// and one sequence, found from query_start and key_start by a warp.  Apart from the kernel so that
// tests run it on the host.
#pragma once

#include <cstdint>

#include "pkv.h"

namespace pkv {
namespace prompt {

constexpr int BM = 128;            // queries per query tile (MMA M)
constexpr int BN = 64;             // keys per tile (S MMA N, PV MMA K)
// The last kLate items (as many as CTAs run at once) come by length, in kParts steps from long to short: 69.5
// -> 67 us for chunks over cached contexts (17 to 24 key tiles an item), 1072 -> 1062 for long prompts; 912 and
// 1824 items, or 4 steps, do no better.
constexpr int kLate = 304, kParts = 8;

// A query tile: its first row of q and out, the rows that are its sequence's, the first one's position
// among the keys; the sequence's first key and their number; key tiles to visit, the first edge tile.
struct Item {
  int q_row, rows, first_pos, k_row, keys, n_tiles, edge, head;
};

// What lays the items out; both starts are device arrays of num_seqs + 1.
struct Layout {
  const int32_t* qstart;
  const int32_t* kstart;
  int num_seqs, num_heads;
  int max_query_len;
  int max_tiles;                        // query tiles per sequence that max_query_len covers
  int late;                             // heads whose query tiles come last and by length
  int total_q, total_k;
};

// Sets what follows from max_query_len; returns the places per head that the grid needs: the query tiles of num_seqs
// sequences that have total_q queries together and max_query_len at most each.
inline long long lay_out(Layout& p, int max_query_len) {
  p.max_query_len = max_query_len;
  p.max_tiles = (max_query_len - 1) / BM + 1;
  const long long by_total = p.total_q / BM + p.num_seqs, by_longest = static_cast<long long>(p.max_tiles) * p.num_seqs;
  const long long tiles = by_total < by_longest ? by_total : by_longest, late = kLate / tiles + 1;
  p.late = static_cast<int>(late < p.num_heads ? late : p.num_heads);
  return tiles;
}

// A warp's search.  32 sequences at a time, one a lane: where they start, their lengths, their query tiles
// and the key tiles that the last of those visits.  A sequence with a bad range has none; some CTA gets to
// each batch and reports it.
// A batch's items come in parts: part 0 has all query tiles of the first heads; each further part those
// of the last p.late heads that visit more than `few` key tiles and are in no part before.
struct ItemFinder {
  int q0 = 0, n = 0, k0 = 0, m = 0, tiles = 0, own = 0;
  int batch = 0, part = -1, most = 0;                         // most: the largest `own`
  int upto = 0, per_head = 0, end = 0, begin = 0;             // a head's items up to the lane's, all; the lane's tiles
  int64_t part_base = 0;                                      // the part's first item

  // Item x, false past the last one.  Batch and part are kept: a CTA's items mostly rise.
  template <typename Report>
  __device__ __forceinline__ bool find(const Layout& p, int x, int lane, Item& item, Report report) {
    if (x < part_base) {
      batch = part_base = 0;
      part = -1;
    }
    while (true) {
      const int heads = part <= 0 ? p.num_heads - p.late : p.late;
      if (part >= 0) {
        const int64_t size = static_cast<int64_t>(per_head) * heads;
        if (x - part_base < size) break;
        part_base += size;
        if (part == kParts) {
          batch += 32;
          if (batch >= p.num_seqs) {
            per_head = 0;                                     // part_base is the end: what is asked for past it is not there
            return false;
          }
          part = -1;
        }
      }
      if (++part == 0) {
        const int i = batch + lane;
        tiles = own = 0;
        if (i < p.num_seqs) {
          q0 = p.qstart[i];
          n = p.qstart[i + 1] - q0;
          k0 = p.kstart[i];
          m = p.kstart[i + 1] - k0;
          const bool ok = n >= 0 && n <= m && q0 >= 0 && q0 <= p.total_q - n && k0 >= 0 && k0 <= p.total_k - m;
          if (!ok || n > p.max_query_len) report(PKV_DEV_BAD_QUERY_RANGE);
          tiles = ok ? min((n + BM - 1) / BM, p.max_tiles) : 0;
          if (tiles > 0) own = (m - n + min(n, tiles * BM) - 1) / BN + 1;
        }
        most = __reduce_max_sync(0xffffffffu, own);
        begin = 0;
        end = tiles;
      } else {
        // begin: the lane's first query tile that visits more than `few` key tiles
        const int few = most - part * ((most + kParts - 1) / kParts);
        const int rows = few * BN + 1 - (m - n);              // so many queries of the sequence see at most that
        end = part == 1 ? tiles : begin;
        begin = part == kParts || rows <= 0 ? 0 : few >= own ? tiles : min(tiles, (rows - 1) / BM);
      }
      upto = end - begin;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      per_head = __shfl_sync(0xffffffffu, upto, 31);
    }
    const unsigned in_part = static_cast<unsigned>(x - part_base), h = in_part / static_cast<unsigned>(per_head);
    const int w = static_cast<int>(in_part - h * per_head);
    const int hit = __ffs(__ballot_sync(0xffffffffu, upto > w)) - 1;
    // a sequence's tiles from the last, which visits the most key tiles
    const int qt = __shfl_sync(0xffffffffu, begin + upto, hit) - 1 - w;
    const int s_n = __shfl_sync(0xffffffffu, n, hit), s_m = __shfl_sync(0xffffffffu, m, hit);
    const int s_q0 = __shfl_sync(0xffffffffu, q0, hit), s_k0 = __shfl_sync(0xffffffffu, k0, hit);
    const int i0 = qt * BM;
    item.q_row = s_q0 + i0;
    item.rows = min(s_n - i0, BM);
    item.first_pos = s_m - s_n + i0;
    item.k_row = s_k0;
    item.keys = s_m;
    item.n_tiles = (item.first_pos + item.rows - 1) / BN + 1;
    // tiles from here on hold keys that some row does not see, or the sequence's end
    item.edge = min((item.first_pos + 1) / BN, s_m / BN);
    item.head = static_cast<int>(h) + (part == 0 ? 0 : p.num_heads - p.late);
    return true;
  }
};

}  // namespace prompt
}  // namespace pkv
