// Simulation of the attention's rings of panels (tests/test_rings.py): a loader fills slots in order, loads land in any order, two sets
// of warps take panels by turns, convert each into one or two chunks, and a thread uses the chunks up in order.
// Every wait is by the parity of a phase, as an mbarrier's; a wait that passes before its phase is over is counted.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "mxq_rings.h"

namespace {

struct Barrier {
  int phases = 0;  // those over
  bool passes(int phase) const { return (phases & 1) != (phase & 1); }
  bool over(int phase) const { return phases > phase; }
};

// The number of waits that passed too early (0 or 1: the run ends with the first).
int simulate(int slots, int chunks, bool shared, int short_of_ten, std::mt19937& rng) {
  const int panels = 160;
  auto chance = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); };
  std::vector<int> size(panels), first(panels + 1, 0), state(panels, 0);  // chunks of a panel; 0 not asked for, 1 in flight, 2 landed
  const int np = 1 + chance(4);
  for (int q = 0; q < panels; q += np) {
    const int n = chance(10) < short_of_ten ? 1 : 2;
    for (int p = q; p < q + np && p < panels; ++p) size[p] = n;
  }
  for (int q = 0; q < panels; ++q) first[q + 1] = first[q] + size[q];
  std::vector<Barrier> full(slots), v_full(chunks), v_empty(chunks);
  std::vector<int> converted(panels, 0), scored(panels, 0);
  int loaded = 0, score = 0, used = 0, panel[2] = {0, 1}, done[2] = {0, 0};
  bool inside[2] = {false, false};
  const int fast = 1 + chance(30);  // how seldom a load lands
  while (used < first[panels]) {
    const int who = chance(6 + fast);
    if (who == 0) {  // the loader (it waits for every use of a slot itself: its parity is right)
      if (loaded < panels && (loaded < slots || (converted[loaded - slots] && (!shared || scored[loaded - slots])))) state[loaded++] = 1;
    } else if (who == 1) {  // a load lands
      std::vector<int> flight;
      for (int q = loaded > slots ? loaded - slots : 0; q < loaded; ++q)
        if (state[q] == 1) flight.push_back(q);
      if (!flight.empty()) {
        const int q = flight[static_cast<size_t>(chance(static_cast<int>(flight.size())))];
        state[q] = 2;
        ++full[q % slots].phases;
      }
    } else if (who == 2) {  // the scores, in order
      if (score < panels && state[score] == 2) scored[score++] = 1;
    } else if (who == 3) {  // a chunk is used up
      if (v_full[used % chunks].over(used / chunks)) ++v_empty[used % chunks].phases, ++used;
    } else {  // a set of warps
      const int s = who & 1, q = panel[s];
      if (q >= panels) continue;
      if (!inside[s]) {
        if (!full[q % slots].passes(q / slots)) continue;
        if (!full[q % slots].over(q / slots)) return 1;
        inside[s] = true;
      }
      const int c = first[q] + done[s];
      if (!v_empty[c % chunks].passes(c / chunks - 1)) continue;
      if (c >= chunks && !v_empty[c % chunks].over(c / chunks - 1)) return 1;
      ++v_full[c % chunks].phases;
      if (++done[s] == size[q]) converted[q] = 1, panel[s] += 2, done[s] = 0, inside[s] = false;
    }
  }
  return 0;
}

int count(int slots, int chunks, bool shared, int runs) {
  std::mt19937 rng(static_cast<unsigned>(slots * 100 + chunks));
  int early = 0;
  for (int i = 0; i < runs; ++i) early += simulate(slots, chunks, shared, i % 11, rng);
  return early;
}

}  // namespace

int main() {
  for (int chunks = 3; chunks <= 8; ++chunks) {
    for (int slots = 6; slots <= 16; ++slots) {
      if (mxq::ring_ok(slots, chunks) && count(slots, chunks, true, 150) != 0) return std::printf("shared %d %d\n", slots, chunks), 1;
      const int v = mxq::value_ring(slots);
      if (!mxq::ring_ok(v, chunks) || v < 4 || slots - v < 2) return std::printf("value ring of %d\n", slots), 1;
      if (count(v, chunks, false, 150) != 0) return std::printf("values %d %d\n", v, chunks), 1;
    }
  }
  // what the rule keeps out: five slots and eight chunks; and two chunks, whose own waits pass too early
  std::printf("%d %d %d\n", count(5, 8, false, 2000), count(7, 8, true, 2000), count(6, 2, false, 2000));
  return 0;
}
