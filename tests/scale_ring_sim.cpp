// Simulation of the attention's buffers of scales where a tile has one panel (tests/test_scale_ring.py): one warp fills them in order, the
// scores' thread and the softmax wait for every tile's, two sets of warps only for every second one. Every wait is by the parity of a phase, as
// an mbarrier's; a wait that passes before its phase is over is counted.
#include <cstdio>
#include <random>
#include <vector>

#include "mxq_rings.h"

namespace {

struct Barrier {
  int count, pending, phases = 0;
  explicit Barrier(int n) : count(n), pending(n) {}
  void arrive() {
    if (--pending == 0) pending = count, ++phases;
  }
  bool passes(int phase) const { return (phases & 1) != (phase & 1); }
  bool over(int phase) const { return phases > phase; }
};

// 1 where a wait passed too early (the run ends with it).
int simulate(int bufs, std::mt19937& rng) {
  const int tiles = 200;
  std::vector<Barrier> full, empty;
  for (int i = 0; i < bufs; ++i) full.emplace_back(1), empty.emplace_back(3);  // the scores, the softmax, the tile's set
  int filled = 0, at[4] = {0, 0, 0, 1};                                        // the scores, the softmax, the sets
  const int step[4] = {1, 1, 2, 2};
  int weight[5];  // how fast each of them is
  for (int& w : weight) w = 1 + static_cast<int>(rng() % 12);
  while (at[0] < tiles || at[1] < tiles || at[2] < tiles || at[3] < tiles) {
    int who = 0, draw = static_cast<int>(rng() % static_cast<unsigned>(weight[0] + weight[1] + weight[2] + weight[3] + weight[4]));
    while (draw >= weight[who]) draw -= weight[who++];
    if (who == 4) {
      if (filled >= tiles || !empty[filled % bufs].passes(filled / bufs - 1)) continue;
      if (filled >= bufs && !empty[filled % bufs].over(filled / bufs - 1)) return 1;
      full[filled % bufs].arrive();
      ++filled;
      continue;
    }
    const int n = at[who];
    if (n >= tiles || !full[n % bufs].passes(n / bufs)) continue;
    if (!full[n % bufs].over(n / bufs)) return 1;
    empty[n % bufs].arrive();
    at[who] += step[who];
  }
  return 0;
}

int count(int bufs, int runs) {
  std::mt19937 rng(static_cast<unsigned>(bufs));
  int early = 0;
  for (int i = 0; i < runs; ++i) early += simulate(bufs, rng);
  return early;
}

}  // namespace

int main() {
  for (int bufs = 1; bufs <= 9; ++bufs)
    if (mxq::scale_ring_ok(bufs) && count(bufs, 2000) != 0) return std::printf("%d buffers\n", bufs), 1;
  std::printf("%d\n", count(1, 2000));  // what the rule keeps out
  return 0;
}
