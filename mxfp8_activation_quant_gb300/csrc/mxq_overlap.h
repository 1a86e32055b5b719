// Whether two strided matrices share a byte. Host only.
#pragma once

#include <cstdint>

namespace mxq {

// `rows` rows of width_a bytes, stride_a bytes apart, from a (stride_a >= width_a); b likewise. Exact where the
// strides are equal (two column ranges of one buffer do not overlap); otherwise by the whole spans.
inline bool rows_overlap(const void* a, int64_t stride_a, int64_t width_a, const void* b, int64_t stride_b, int64_t width_b,
                         int64_t rows) {
  const int64_t a0 = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a)), b0 = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b));
  if (a0 + (rows - 1) * stride_a + width_a <= b0 || b0 + (rows - 1) * stride_b + width_b <= a0) return false;
  if (stride_a != stride_b) return true;
  // b0 = a0 + q stride + d: b's row j begins d bytes into a's row j + q and may reach into row j + q + 1
  int64_t q = (b0 - a0) / stride_a, d = (b0 - a0) % stride_a;
  if (d < 0) {
    d += stride_a;
    --q;
  }
  return (d < width_a && q > -rows && q < rows) || (d + width_b > stride_a && q + 1 > -rows && q + 1 < rows);
}

}  // namespace mxq
