// Scale stores shared by the streaming kernels (quantizer, RMSNorm producers): one warp holds 256
// consecutive columns of a row, 8 per lane, and a 32-element group is 4 lanes.
#pragma once

#include <cstdint>

#include "mxq_device.cuh"

namespace mxq {
namespace {

struct QuantArgs {
  const uint16_t* x;
  int64_t M, K, ldx;
  uint8_t* q;
  int64_t ldq;
  uint8_t* sf_rm;   // [M, Kg]
  uint32_t* sf_pk;  // [Kw, Mp4]
  uint8_t* sf_tl;   // F8_128x4
  int64_t Kg, Kw, Mp4, Mp128;
  int64_t rows_total;  // rows covered (padding rows write zero scale words only)
  int32_t chunks;      // warp segments per row
};

// Scales of one 256-column unit: row-major bytes, packed word, tiled word.
__device__ __forceinline__ void store_unit_scales(const QuantArgs& a, int64_t row, int64_t c, uint32_t code,
                                                  int lane) {
  if (a.sf_rm != nullptr && row < a.M && (lane & 3) == 0 && c < a.K) a.sf_rm[row * a.Kg + (c >> 5)] = code;
  uint32_t w = code;
  w |= __shfl_down_sync(0xffffffffu, code, 4) << 8;
  w |= __shfl_down_sync(0xffffffffu, code, 8) << 16;
  w |= __shfl_down_sync(0xffffffffu, code, 12) << 24;
  if ((lane & 15) == 0 && c < a.K) {
    const int64_t wi = c >> 7;
    if (a.sf_pk != nullptr && row < a.Mp4) a.sf_pk[wi * a.Mp4 + row] = w;
    if (a.sf_tl != nullptr && row < a.Mp128)
      *reinterpret_cast<uint32_t*>(a.sf_tl + tiled128x4_word_offset(row, wi, a.Kw)) = w;
  }
}

}  // namespace
}  // namespace mxq
