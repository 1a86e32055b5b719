// What a stage's barrier still lacks when a pipeline of loads has given up: the arithmetic, for host and
// device.
//
// A loader fills stages 0, 1, 2, ... in order and counts them, so loader l of CTA r has issued its part of
// stage i exactly if i < count[r][l]. One of them, loader 0 of CTA 0, announces the bytes of all of them on
// the stage's barrier before its own part. When all have stopped, at whatever stages, the barrier is
// brought to wait for the bytes that were issued and for nothing else: then its phase completes when
// the last copy in flight has landed, and a CTA may leave shared memory.
#pragma once

#ifdef __CUDACC__
#define MXQ_HD __host__ __device__ __forceinline__
#else
#define MXQ_HD inline
#endif

namespace mxq {

// bytes: to be added to those the barrier waits for (negative: to be counted as landed). arrivals: to be
// made in the place of threads that will not come.
struct Owed {
  int bytes, arrivals;
};

// A tile's `half` token rows of 128 bytes (a multiple of 4), in quads of rows that `parts` loaders take in
// turn: the bytes of loader `part`.
MXQ_HD int quad_bytes(int half, int part, int parts) {
  const int quads = half / 4;
  return quads > part ? (quads - part + parts - 1) / parts * 512 : 0;
}

// Operand stage i: loader 0 of each CTA brings `weight_bytes` and its part of the `token_bytes`, the others
// only their parts (parts == 1: loader 0 all of them). The barrier counts the announcement and the scale
// copies, which have been made for the first `staged` stages.
template <int PARTS>
MXQ_HD Owed owed_operands(int i, const int (&count)[2][PARTS], int staged, int weight_bytes, int token_bytes) {
  int issued = 0;
  for (int r = 0; r < 2; ++r)
    for (int l = 0; l < PARTS; ++l)
      if (i < count[r][l])
        issued += (l == 0 ? weight_bytes : 0) + (PARTS == 1 ? token_bytes : quad_bytes(token_bytes / 128, l, PARTS));
  const bool announced = i < count[0][0];
  return {issued - (announced ? 2 * (weight_bytes + token_bytes) : 0), (announced ? 0 : 1) + (i < staged ? 0 : 1)};
}

// Scale chunk i, of `bytes` from each CTA's loader; the barrier counts the announcement alone.
MXQ_HD Owed owed_scales(int i, int count0, int count1, int bytes) {
  const bool announced = i < count0;
  return {(announced ? bytes : 0) + (i < count1 ? bytes : 0) - (announced ? 2 * bytes : 0), announced ? 0 : 1};
}

}  // namespace mxq
