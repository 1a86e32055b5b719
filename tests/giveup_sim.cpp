// Simulation of the attention's roles after a wait has given up (tests/test_giveup.py): the loads of panels and queries, the scale
// warp, the scores' and the outputs' threads, the four softmax warps of a half of the heads, and the two sets of warps that convert values. A
// wait passes by the parity of its phase; one of them, at a random point, gives up and sets `dead`, after which every wait that does not pass
// at once fails, and its role goes on as if it had passed, or leaves. Counted: runs in which a role waits for ever at the softmax's named barrier, or meets it in
// a barrier of another kind; and announcements of loads on a barrier whose loads before are still in flight.
#include <coroutine>
#include <cstdio>
#include <exception>
#include <random>
#include <vector>

#include "mxq_rings.h"

namespace {

struct Role {
  struct promise_type {
    Role get_return_object() { return {std::coroutine_handle<promise_type>::from_promise(*this)}; }
    std::suspend_always initial_suspend() noexcept { return {}; }
    std::suspend_always final_suspend() noexcept { return {}; }
    void return_void() {}
    void unhandled_exception() { std::terminate(); }
  };
  std::coroutine_handle<promise_type> h;
};
using Step = std::suspend_always;

struct Barrier {  // an mbarrier without bytes
  int count, pending, phases = 0;
  explicit Barrier(int n) : count(n), pending(n) {}
  void arrive() {
    if (--pending == 0) pending = count, ++phases;
  }
  bool passes(int phase) const { return (phases & 1) != (phase & 1); }
};

// count: the softmax's warps count their tiles from the lengths; else they go by marks in the buffers of scales, which the scale warp
// overwrites without a limit once waits fail. leave: a role that has not waited for panels, chunks or queries leaves, instead of handing on and
// releasing them all the same.
struct Rules {
  bool count, leave;
};

constexpr int kSf = 3;

struct Panels {  // a ring of panels and what is in flight to it
  int slots;
  std::vector<Barrier> full, empty;
  std::vector<char> flying;
  Panels(int n, int releases) : slots(n), flying(static_cast<size_t>(n), 0) {
    for (int i = 0; i < n; ++i) full.emplace_back(1), empty.emplace_back(releases);
  }
};

struct Cta {
  Rules rules;
  std::mt19937 rng;
  std::vector<int> tiles;               // of each segment
  std::vector<std::vector<int>> size;   // chunks of a panel, by segment and tile
  int np, gives_up;                     // panels of a tile; the failing try that gives up
  bool shared, dead = false;
  long early = 0, mixed = 0;
  // barriers
  std::vector<Barrier> sf_full, sf_empty;
  Barrier s_full{1}, s_empty{4}, fin_full{4}, fin_empty{1}, q_full{1}, q_empty{1}, o_full{1}, o_empty{2};
  std::vector<Barrier> p_full, p_empty, v_full, v_empty;
  Panels keys, rows;                    // rows: the values' panels, where they are not the keys
  int flags[kSf] = {0, 0, 0};           // 1: the segment's last tile, 2: the CTA's
  bool q_flying = false;
  struct Load {
    Panels* ring;                       // null: the queries
    int slot;
  };
  std::vector<Load> in_flight;
  // the named barrier
  int there = 0, round = 0, kind = -1;
  bool said = false, answer = false;

  Cta(Rules r, unsigned seed, int chunks, int slots, bool shared_kv)
      : rules(r), rng(seed), shared(shared_kv), keys(shared_kv ? slots : 4, shared_kv ? 2 : 1), rows(slots, 1) {
    np = 1 + chance(4);
    for (int i = 0; i < kSf; ++i) sf_full.emplace_back(1), sf_empty.emplace_back(7);
    for (int i = 0; i < 2; ++i) p_full.emplace_back(4), p_empty.emplace_back(1);
    for (int i = 0; i < chunks; ++i) v_full.emplace_back(1), v_empty.emplace_back(1);
    const int n = 1 + chance(5);
    for (int i = 0; i < n; ++i) {
      tiles.push_back(1 + chance(6));
      size.emplace_back(static_cast<size_t>(tiles.back()), 2);
      if (chance(2) == 0) size.back().back() = 1;
    }
    gives_up = chance(4) == 0 ? chance(4000) : chance(400);
  }
  Panels& values() { return shared ? keys : rows; }
  int chance(int n) { return static_cast<int>(rng() % static_cast<unsigned>(n)); }
  // A try of a wait: 1 passed, -1 given up, 0 again.
  int tried(const Barrier& b, int phase) {
    if (b.passes(phase)) return 1;
    if (dead || gives_up-- == 0) return dead = true, -1;
    return 0;
  }
  void announce(Panels& r, int slot) {
    early += r.flying[static_cast<size_t>(slot)];
    r.flying[static_cast<size_t>(slot)] = 1;
    in_flight.push_back({&r, slot});
  }
  void land(size_t at) {
    const Load l = in_flight[at];
    in_flight.erase(in_flight.begin() + static_cast<long>(at));
    if (l.ring == nullptr) return q_flying = false, q_full.arrive();
    l.ring->flying[static_cast<size_t>(l.slot)] = 0;
    l.ring->full[static_cast<size_t>(l.slot)].arrive();
  }
  void meet(int what, bool say) {
    if (there == 0) kind = what, said = false;
    mixed += kind != what;
    said = said || say;
    if (++there == 4) there = 0, ++round, answer = said;
  }
};

// Waits; `got`: whether it passed.
#define WAIT(got, bar, phase)                                   \
  {                                                             \
    int tried;                                                  \
    while ((tried = c.tried((bar), (phase))) == 0) co_await Step {}; \
    (got) = tried > 0;                                          \
    co_await Step {};                                           \
  }
// ... and leaves the role where that is the rule and it did not.
#define WAIT_OR_LEAVE(bar, phase)      \
  {                                    \
    bool got_;                         \
    WAIT(got_, bar, phase);            \
    if (!got_ && c.rules.leave) co_return; \
  }
#define MEET(what, say)                                     \
  {                                                         \
    const int now = c.round;                                \
    c.meet((what), (say));                                  \
    while (c.round == now) co_await Step {};                \
  }                                                         \
  co_await Step {}

Role loads(Cta& c, Panels& r) {
  int slot = 0, use = 0;
  for (size_t s = 0; s < c.tiles.size() && !c.dead; ++s)
    for (int i = 0; i < c.tiles[s]; ++i)
      for (int p = 0; p < c.np; ++p) {
        bool got;
        WAIT(got, r.empty[static_cast<size_t>(slot)], use - 1);
        if (!got) break;
        c.announce(r, slot);
        if (++slot == r.slots) slot = 0, ++use;
      }
}

Role scales(Cta& c) {
  int n = 0;
  for (size_t s = 0; s < c.tiles.size(); ++s)
    for (int i = 0; i < c.tiles[s]; ++i, ++n) {
      [[maybe_unused]] bool got;
      WAIT(got, c.sf_empty[n % kSf], n / kSf - 1);
      const bool last = i + 1 == c.tiles[s];
      c.flags[n % kSf] = (last ? 1 : 0) | (last && s + 1 == c.tiles.size() ? 2 : 0);
      co_await Step{};
      c.sf_full[n % kSf].arrive();
    }
}

Role scores(Cta& c) {
  int n = 0, panel = 0;
  [[maybe_unused]] bool got;
  for (size_t s = 0; s < c.tiles.size(); ++s) {
    WAIT_OR_LEAVE(c.q_empty, static_cast<int>(s) - 1);
    c.early += c.q_flying;
    c.q_flying = true;
    c.in_flight.push_back({nullptr, 0});
    WAIT_OR_LEAVE(c.q_full, static_cast<int>(s));
    for (int i = 0; i < c.tiles[s]; ++i, ++n) {
      WAIT(got, c.sf_full[n % kSf], n / kSf);
      WAIT(got, c.s_empty, n - 1);
      for (int p = 0; p < c.np; ++p, ++panel) {
        const int slot = panel % c.keys.slots;
        WAIT_OR_LEAVE(c.keys.full[slot], panel / c.keys.slots);
        c.keys.empty[slot].arrive();
      }
      c.s_full.arrive();
      c.sf_empty[n % kSf].arrive();
      if (i + 1 == c.tiles[s]) c.q_empty.arrive();
      co_await Step{};
    }
  }
}

Role outputs(Cta& c) {
  int n = 0, chunk = 0;
  [[maybe_unused]] bool got;
  const int chunks = static_cast<int>(c.v_full.size());
  for (size_t s = 0; s < c.tiles.size(); ++s) {
    WAIT(got, c.o_empty, static_cast<int>(s) - 1);
    for (int i = 0; i < c.tiles[s]; ++i, ++n) {
      WAIT(got, c.p_full[n % 2], n / 2);
      for (int k = 0; k < c.np * c.size[s][i]; ++k, ++chunk) {
        WAIT_OR_LEAVE(c.v_full[chunk % chunks], chunk / chunks);
        c.v_empty[chunk % chunks].arrive();
      }
      c.p_empty[n % 2].arrive();
    }
    c.o_full.arrive();
  }
}

// One of two sets of warps that take panels by turns.
Role values(Cta& c, int set) {
  int n = 0, panel = 0, chunk = 0;
  const int chunks = static_cast<int>(c.v_full.size());
  Panels& r = c.values();
  [[maybe_unused]] bool got;
  for (size_t s = 0; s < c.tiles.size(); ++s) {
    for (int i = 0; i < c.tiles[s]; ++i, ++n) {
      WAIT(got, c.sf_full[n % kSf], n / kSf);
      for (int p = 0; p < c.np; ++p, ++panel) {
        const int first = chunk;
        chunk += c.size[s][i];
        if (panel % 2 != set) continue;
        WAIT_OR_LEAVE(r.full[panel % r.slots], panel / r.slots);
        for (int k = first; k < chunk; ++k) {
          WAIT_OR_LEAVE(c.v_empty[k % chunks], k / chunks - 1);
          c.v_full[k % chunks].arrive();
        }
        r.empty[panel % r.slots].arrive();
      }
      c.sf_empty[n % kSf].arrive();
    }
    if (set == 0) {
      WAIT(got, c.fin_full, static_cast<int>(s));
      c.fin_empty.arrive();
    }
    WAIT(got, c.o_full, static_cast<int>(s));
    c.o_empty.arrive();
  }
}

enum { kPlain, kOr };

Role softmax(Cta& c) {
  int n = 0, segment = 0;
  const int segments = static_cast<int>(c.tiles.size());
  bool more = true;
  [[maybe_unused]] bool got;
  while (true) {
    MEET(kPlain, false);
    MEET(kPlain, false);
    if (!more) break;
    bool last, started = false;
    int left = segment < segments ? c.tiles[static_cast<size_t>(segment)] : 0;
    do {
      WAIT(got, c.s_full, n);
      WAIT(got, c.sf_full[n % kSf], n / kSf);
      if (c.rules.count) {
        last = --left == 0;
        more = !(last && segment + 1 == segments);
      } else {
        last = (c.flags[n % kSf] & 1) != 0;
        more = (c.flags[n % kSf] & 2) == 0;
      }
      c.sf_empty[n % kSf].arrive();
      co_await Step{};
      bool move = !started;
      while (true) {
        if (move) {
          MEET(kPlain, false);
          MEET(kPlain, false);
          if (started) WAIT(got, c.p_empty[(n + 1) % 2], (n - 1) / 2);
          break;
        }
        MEET(kOr, c.chance(6) == 0);
        move = c.answer;
        if (!move) break;
      }
      c.s_empty.arrive();
      WAIT(got, c.p_empty[n % 2], n / 2 - 1);
      c.p_full[n % 2].arrive();
      started = true;
      ++n;
      co_await Step{};
    } while (!last);
    WAIT(got, c.fin_empty, segment - 1);
    c.fin_full.arrive();
    ++segment;
  }
}

struct Counts {
  long stuck = 0, mixed = 0, early = 0, whole = 0;
};

void simulate(Rules rules, unsigned seed, bool gives_up, Counts& out) {
  std::mt19937 shape(seed);
  const int chunks = 3 + static_cast<int>(shape() % 6);
  const bool shared = shape() % 2 == 0;
  int slots = 4 + static_cast<int>(shape() % 13);
  while (!mxq::ring_ok(slots, chunks) || (shared && slots < 6)) ++slots;
  Cta c(rules, static_cast<unsigned>(shape()), chunks, slots, shared);
  if (!gives_up) c.gives_up = 1 << 30;
  std::vector<Role> roles{loads(c, c.keys), scales(c), scores(c), outputs(c), values(c, 0), values(c, 1)};
  if (!shared) roles.push_back(loads(c, c.rows));
  for (int i = 0; i < 4; ++i) roles.push_back(softmax(c));
  const int slow = 1 + c.chance(60);  // how seldom a load lands
  int idle = 0;
  while (idle < 40000) {  // (a run has some thousand steps)
    bool live = false;
    for (Role& r : roles) live = live || !r.h.done();
    if (!live) break;
    const int who = c.chance(static_cast<int>(roles.size()) + 2);
    if (who < static_cast<int>(roles.size())) {
      Role& r = roles[static_cast<size_t>(who)];
      if (!r.h.done()) r.h.resume();
    } else if (!c.in_flight.empty() && c.chance(slow) == 0) {
      c.land(static_cast<size_t>(c.chance(static_cast<int>(c.in_flight.size()))));
    }
    idle = c.dead ? idle + 1 : 0;
  }
  bool stuck = false;
  for (Role& r : roles) stuck = stuck || !r.h.done();
  out.stuck += stuck;
  out.mixed += c.mixed != 0;
  out.early += c.early != 0;
  out.whole += !c.dead;
  for (Role& r : roles) r.h.destroy();
}

Counts count(Rules rules, bool gives_up, int runs) {
  Counts n;
  for (int i = 0; i < runs; ++i) simulate(rules, static_cast<unsigned>(i), gives_up, n);
  return n;
}

}  // namespace

int main() {
  const Counts sound = count({true, true}, false, 300);
  if (sound.stuck + sound.mixed + sound.early != 0 || sound.whole != 300) return std::printf("without a wait that gives up\n"), 1;
  const Counts now = count({true, true}, true, 3000);
  if (now.stuck + now.mixed + now.early != 0)
    return std::printf("stuck %ld, mixed %ld, early %ld\n", now.stuck, now.mixed, now.early), 1;
  if (now.whole > 1500) return std::printf("too few that give up: %ld\n", 3000 - now.whole), 1;
  // what the two rules keep out
  const Counts apart = count({false, true}, true, 3000), on = count({true, false}, true, 3000);
  std::printf("%ld %ld\n", apart.stuck + apart.mixed, on.early);
  return 0;
}
