// csrc/mxq_per_device.h with a stand-in for the call that it guards (tests/test_per_device.py).
#include <cstdio>

#include "mxq_per_device.h"

#define CHECK(c) \
  if (!(c)) return std::printf("line %d: %s\n", __LINE__, #c), 1

enum Error { kOk = 0, kBad = 7 };

int main() {
  mxq::PerDevice set, other;
  int calls = 0;
  auto ok = [&] { ++calls; return kOk; };
  auto bad = [&] { ++calls; return kBad; };
  CHECK(set.once(0, ok) == kOk && calls == 1);
  CHECK(set.once(0, ok) == kOk && calls == 1);   // once
  CHECK(set.once(0, bad) == kOk && calls == 1);  // not run again
  CHECK(set.once(1, ok) == kOk && calls == 2);   // another device needs it too
  CHECK(set.once(63, ok) == kOk && set.once(63, ok) == kOk && calls == 3);
  CHECK(other.once(0, ok) == kOk && calls == 4);  // another kernel's
  CHECK(set.once(2, bad) == kBad && set.once(2, bad) == kBad && calls == 6);  // a failure is not kept
  CHECK(set.once(2, ok) == kOk && set.once(2, bad) == kOk && calls == 7);
  CHECK(set.once(64, ok) == kOk && set.once(64, ok) == kOk && calls == 9);
  CHECK(set.once(-1, ok) == kOk && set.once(0, bad) == kOk && calls == 10);
  return 0;
}
