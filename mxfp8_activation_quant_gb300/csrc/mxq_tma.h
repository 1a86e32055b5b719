// Host side of the TMA operand maps shared by the GEMM kernels (tma_maps.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>

namespace mxq {

// cuTensorMapEncodeTiled of the loaded driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
// 2-D E4M3 tensor [rows, cols], row stride ld bytes; box = 128 bytes x box_rows, 128B swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
// Scale atoms of an F8_128x4 array as a 2-D tensor [atoms, 128 x u32]: box_atoms 512-byte atoms per box.
bool make_sf_map(CUtensorMap* m, const void* base, int64_t atoms, int box_atoms = 1);
// bf16 or fp32 [rows, cols] (row stride ld elements) in boxes of 128 elements x box_rows, unswizzled.
bool make_bf16_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
bool make_f32_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
// SMs of the current device.
int num_sms();

}  // namespace mxq
