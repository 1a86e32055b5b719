// csrc/mxq_overlap.h against marking every byte (tests/test_overlap.py).
#include <cstdio>
#include <vector>

#include "mxq_overlap.h"

int main() {
  long apart = 0, n = 0;
  std::vector<char> mark(512);
  char* base = reinterpret_cast<char*>(1 << 20);  // (addresses only)
  for (int rows = 1; rows <= 4; ++rows)
    for (int stride = 1; stride <= 9; ++stride)
      for (int wa = 1; wa <= stride; ++wa)
        for (int wb = 1; wb <= stride; ++wb)
          for (int off = -60; off <= 60; ++off) {
            for (char& m : mark) m = 0;
            for (int i = 0; i < rows; ++i)
              for (int c = 0; c < wa; ++c) mark[200 + i * stride + c] = 1;
            bool want = false;
            for (int j = 0; j < rows; ++j)
              for (int c = 0; c < wb; ++c) want |= mark[200 + off + j * stride + c] != 0;
            if (mxq::rows_overlap(base, stride, wa, base + off, stride, wb, rows) != want)
              return std::printf("rows %d stride %d widths %d %d offset %d\n", rows, stride, wa, wb, off), 1;
            // other strides: never less than what is shared
            for (int sb = wb; sb <= 9; ++sb) {
              bool share = false;
              for (int j = 0; j < rows; ++j)
                for (int c = 0; c < wb; ++c) share |= mark[200 + off + j * sb + c] != 0;
              if (share && !mxq::rows_overlap(base, stride, wa, base + off, sb, wb, rows))
                return std::printf("rows %d strides %d %d offset %d\n", rows, stride, sb, off), 1;
            }
            const bool spans = off < (rows - 1) * stride + wa && -off < (rows - 1) * stride + wb;
            apart += spans && !want;
            ++n;
          }
  std::printf("%ld %ld\n", apart, n);
  return 0;
}
