// Simulation of the experts' load pipeline giving up at arbitrary points (tests/test_moe_settle.py): every
// loader issues its stages in order, at most STAGES ahead of the MMA thread, and stops somewhere; some copies
// have landed, some have not. After settling by csrc/mxq_settle.h a stage's barrier must complete its phase
// exactly with the last of its copies in flight.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "mxq_settle.h"

namespace {

struct Barrier {  // one phase of an mbarrier
  int pending, tx = 0;
  bool complete() const { return pending == 0 && tx == 0; }
};

template <int PARTS>
int simulate(std::mt19937& rng, long& unsettled) {
  auto upto = [&](int n) { return static_cast<int>(rng() % static_cast<unsigned>(n + 1)); };
  const int stages = 6, weight = 16384;
  const int consumed = upto(20);
  int count[2][PARTS];
  for (auto& c : count)
    for (int& n : c) n = consumed + upto(stages);
  const int staged = consumed + upto(stages);
  int hi = 0;
  for (auto& c : count)
    for (int n : c) hi = n > hi ? n : hi;
  for (int i = consumed; i < hi; ++i) {
    const int half = 8 * (1 + upto(12));  // 8 .. 104
    const int rows = PARTS == 1 ? 32 * ((half + 23) / 32) + 8 : half;
    Barrier bar{2};
    std::vector<int> copies;
    if (i < count[0][0]) {  // the announcement
      --bar.pending;
      bar.tx += 2 * (weight + rows * 128);
    }
    for (int r = 0; r < 2; ++r)
      for (int l = 0; l < PARTS; ++l) {
        if (i >= count[r][l]) continue;
        if (l == 0) copies.push_back(weight);
        if (PARTS == 1)
          copies.push_back(rows * 128);
        else
          for (int quad = l; 4 * quad < half; quad += PARTS) copies.push_back(512);  // four rows of 128 bytes
      }
    if (i < staged) --bar.pending;
    std::shuffle(copies.begin(), copies.end(), rng);
    size_t landed = static_cast<size_t>(upto(static_cast<int>(copies.size())));
    for (size_t c = 0; c < landed; ++c) bar.tx -= copies[c];
    Barrier before = bar;
    const mxq::Owed o = mxq::owed_operands<PARTS>(i, count, staged, weight, rows * 128);
    bar.tx += o.bytes;
    bar.pending -= o.arrivals;
    for (; landed < copies.size(); ++landed) {
      if (bar.complete()) return std::printf("stage %d complete with copies in flight\n", i), 1;
      bar.tx -= copies[landed];
      before.tx -= copies[landed];
    }
    if (!bar.complete()) return std::printf("stage %d never completes\n", i), 1;
    if (bar.pending != 0) return std::printf("stage %d: arrivals\n", i), 1;
    unsettled += before.complete() ? 0 : 1;
  }
  return 0;
}

int simulate_scales(std::mt19937& rng) {
  const int bytes = 6144;
  for (int i = 0; i < 4; ++i) {
    const int c0 = static_cast<int>(rng() % 5), c1 = static_cast<int>(rng() % 5);
    Barrier bar{1};
    std::vector<int> copies;
    if (i < c0) {
      --bar.pending;
      bar.tx += 2 * bytes;
      copies.insert(copies.end(), {2048, 4096});
    }
    if (i < c1) copies.insert(copies.end(), {2048, 4096});
    std::shuffle(copies.begin(), copies.end(), rng);
    const mxq::Owed o = mxq::owed_scales(i, c0, c1, bytes);
    bar.tx += o.bytes;
    bar.pending -= o.arrivals;
    for (int c : copies) {
      if (bar.complete()) return std::printf("chunk %d complete with copies in flight\n", i), 1;
      bar.tx -= c;
    }
    if (!bar.complete()) return std::printf("chunk %d never completes\n", i), 1;
  }
  return 0;
}

}  // namespace

int main() {
  std::mt19937 rng(1);
  long unsettled = 0;
  for (int n = 0; n < 20000; ++n)
    if (simulate<4>(rng, unsettled) != 0 || simulate<1>(rng, unsettled) != 0 || simulate_scales(rng) != 0) return 1;
  std::printf("%ld\n", unsettled);
  return 0;
}
