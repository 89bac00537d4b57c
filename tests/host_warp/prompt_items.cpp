// Runs csrc/prompt_items.cuh on the host: 32 fibers stand for a warp's lanes, in turn, and a warp
// collective is the point where each hands over to the next.
//
// Reads from stdin: num_heads max_query_len total_q total_k num_seqs, query_start, key_start, then
// the number of CTAs and for each the number of places it takes and those places in order.  Prints
// "grid <places per head> <late>", per place that held an item "<place> <head> <q_row> <rows>
// <first_pos> <k_row> <keys> <n_tiles> <edge>", and "codes <n>": lanes that reported a bad range.
#include <ucontext.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#define __device__
#define __forceinline__ inline
using std::max;
using std::min;

namespace {
constexpr int LANES = 32;
ucontext_t lanes[LANES], home;
char stacks[LANES][64 * 1024];
int current;
long collectives[LANES];
int slots[2][LANES];

// Hands over to the next lane; comes back when every other lane has reached the same collective.
void next_lane() {
  const int from = current;
  current = (current + 1) % LANES;
  swapcontext(&lanes[from], &lanes[current]);
}
// Every lane's value of this collective.
const int* exchange(int value) {
  int* now = slots[collectives[current]++ & 1];
  now[current] = value;
  next_lane();
  return now;
}
}  // namespace

int __shfl_sync(unsigned, int value, int from) { return exchange(value)[from & 31]; }
int __shfl_up_sync(unsigned, int value, int by) {
  const int me = current;
  const int* all = exchange(value);
  return me >= by ? all[me - by] : value;
}
int __reduce_max_sync(unsigned, int value) {
  const int* all = exchange(value);
  return *std::max_element(all, all + LANES);
}
unsigned __ballot_sync(unsigned, bool value) {
  const int* all = exchange(value);
  unsigned mask = 0;
  for (int i = 0; i < LANES; ++i) mask |= static_cast<unsigned>(all[i] != 0) << i;
  return mask;
}
int __ffs(unsigned x) { return __builtin_ffs(static_cast<int>(x)); }

#include "prompt_items.cuh"

namespace {
pkv::prompt::Layout layout;
std::vector<std::vector<int>> ctas;
long codes;

void lane_main() {
  const int lane = current;
  for (const auto& places : ctas) {
    pkv::prompt::ItemFinder finder;
    for (const int x : places) {
      pkv::prompt::Item it;
      const bool real = finder.find(layout, x, lane, it, [](int) { ++codes; });
      if (real && lane == 0)
        std::printf("%d %d %d %d %d %d %d %d %d\n", x, it.head, it.q_row, it.rows, it.first_pos, it.k_row, it.keys,
                    it.n_tiles, it.edge);
    }
  }
  // the lanes end one after another
  if (lane == LANES - 1) swapcontext(&lanes[lane], &home);
  next_lane();
}

int number() {
  int x;
  if (std::scanf("%d", &x) != 1) std::exit(2);
  return x;
}
}  // namespace

int main() {
  layout.num_heads = number();
  const int max_query_len = number();
  layout.total_q = number();
  layout.total_k = number();
  layout.num_seqs = number();
  std::vector<int32_t> starts[2];
  for (auto& v : starts)
    for (int i = 0; i <= layout.num_seqs; ++i) v.push_back(number());
  layout.qstart = starts[0].data();
  layout.kstart = starts[1].data();
  const long long tiles = pkv::prompt::lay_out(layout, max_query_len);
  std::printf("grid %lld %d\n", tiles, layout.late);
  ctas.resize(number());
  for (auto& places : ctas) {
    places.resize(number());
    for (int& x : places) x = number();
  }
  for (int i = 0; i < LANES; ++i) {
    getcontext(&lanes[i]);
    lanes[i].uc_stack.ss_sp = stacks[i];
    lanes[i].uc_stack.ss_size = sizeof stacks[i];
    makecontext(&lanes[i], lane_main, 0);
  }
  current = 0;
  swapcontext(&home, &lanes[0]);
  std::printf("codes %ld\n", codes);
  return 0;
}
