// Quantizing keys and values as they are written into a paged cache, and reading them back
// (HBM-streaming kernels).
//
// Mapping: as the standalone quantizer's: 8 elements per lane, 4 lanes per 32-element group (amax with two
// xor-shuffles), 16 lanes per 128-element scale word, and a warp owns a segment of kUnits x 256 columns
// of a token's heads * dim row. A write moves 2 + 33/32 bytes an element, a read the same the other way: a read of a batch's
// prefixes is bound by HBM (40960 rows of 8 x 128, keys and values, 41.9 us: 0.90 of a copy's rate), a write of 8192 tokens by its
// instructions (11.0 us, 0.68 of the copy's rate; issue slots 75 % busy, DRAM 30 %, since its stores stay in L2). Keys and
// values go in one launch (grid.y), since a decode step's few tokens take less than a launch does.
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_kv_internal.h"

namespace mxq {
namespace {

constexpr int kWarps = 4;
constexpr int kUnits = 2;
// From here a warp reads four rows (one row, four, us: 2048 rows of 512 2.9, 3.3; 4096 3.5, 3.6; 8192 4.8, 4.0; 2048 of 8 x 128, keys and values
// 4.4, 4.7; 4096 6.6, 5.6; 2048 of 128 3.0, 3.2; 4096 4.2, 3.7).
constexpr int64_t kManyRows = 4096;

// Division by a number known on the host: x / d = x * (floor(2^64 / d) + 1) >> 64 for x < 2^64 / d, since the product is off by
// less than x / 2^64 < 1 / d. (d = 1: mul = 0.)
struct Divisor {
  uint64_t mul;
};
Divisor divisor(uint64_t d) { return {d == 1 ? 0 : ~uint64_t(0) / d + 1}; }
__device__ __forceinline__ uint64_t operator/(uint64_t x, Divisor d) { return d.mul == 0 ? x : __umul64hi(x, d.mul); }

struct Tensor {
  const uint16_t* rows;
  int64_t ld, ldh;
  uint8_t* data;
  uint8_t* sf;
  int64_t page, token, head, sf_page, sf_token, sf_head;
  uint32_t dim, width;  // width = heads * dim
  uint32_t chunks;      // warp segments per row
  Divisor by_dim, by_chunks;
};

struct WriteArgs {
  Tensor t[2];
  const int32_t* slots;
  int64_t T;
  uint32_t page_size, slots_end;
  Divisor by_page;
};

struct ReadArgs {
  Tensor t[2];
  const int32_t* table;
  int64_t ld_table, B, rows;
  const int32_t* cu;
  const int32_t* starts;
  uint32_t page_size, pages, table_width;
};

Tensor tensor(const KvTensor& k) {
  const mxq_kv_cache& c = k.c;
  Tensor t;
  t.rows = static_cast<const uint16_t*>(k.rows);
  t.ld = k.ld;
  t.ldh = k.ldh;
  t.data = static_cast<uint8_t*>(c.data);
  t.sf = static_cast<uint8_t*>(c.sf);
  t.page = c.page_stride;
  t.token = c.token_stride;
  t.head = c.head_stride;
  t.sf_page = c.sf_page_stride;
  t.sf_token = c.sf_token_stride;
  t.sf_head = c.sf_head_stride;
  t.dim = static_cast<uint32_t>(c.dim);
  t.width = static_cast<uint32_t>(c.heads) * t.dim;
  t.chunks = (t.width + 256 * kUnits - 1) / (256 * kUnits);
  t.by_dim = divisor(t.dim);
  t.by_chunks = divisor(t.chunks);
  return t;
}

// A write's instructions count as much as its bytes: with the compiler's divisions (the 64-bit one by a row's warps above all) 8192
// tokens of 8 x 128, keys and values, took 12.0 us, now 11.0 (4600 GB/s); 65536 tokens 84.4 and 79.2 (5140 GB/s).
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const __grid_constant__ WriteArgs a) {
  const Tensor& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t row = static_cast<uint64_t>(wid) / t.by_chunks;
  if (row >= a.T) return;
  const uint32_t slot = static_cast<uint32_t>(a.slots[row]);
  const uint32_t col0 = static_cast<uint32_t>(wid - row * t.chunks) * (256 * kUnits) + 8 * lane;

  uint4 v[kUnits];  // (asked for before the slot is looked at)
  uint32_t h[kUnits], d[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const uint32_t c = col0 + 256 * u;
    h[u] = static_cast<uint32_t>(c / t.by_dim);
    d[u] = c - h[u] * t.dim;
    v[u] = c < t.width ? ld_stream_u4(t.rows + row * t.ld + h[u] * t.ldh + d[u]) : make_uint4(0, 0, 0, 0);
  }
  if (slot >= a.slots_end) return;  // (negative ones too)
  const uint32_t page = static_cast<uint32_t>(slot / a.by_page), place = slot - page * a.page_size;
  uint8_t* const data = t.data + page * t.page + place * t.token;
  uint8_t* const sf = t.sf + page * t.sf_page + place * t.sf_token;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const bool in = col0 + 256 * u < t.width;
    uint32_t amax = absmax8(v[u]);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = ue8m0_from_bf16_amax(amax);
    if (in) *reinterpret_cast<uint2*>(data + h[u] * t.head + d[u]) = quant8(v[u], ue8m0_inverse(code));
    uint8_t* const s = sf + h[u] * t.sf_head + (d[u] >> 5);
    if (t.dim % 128 == 0) {  // 16 lanes lie in one head: whole words
      uint32_t w = code;
      w |= __shfl_down_sync(0xffffffffu, code, 4) << 8;
      w |= __shfl_down_sync(0xffffffffu, code, 8) << 16;
      w |= __shfl_down_sync(0xffffffffu, code, 12) << 24;
      if (in && (lane & 15) == 0) *reinterpret_cast<uint32_t*>(s) = w;
    } else if (in && (lane & 3) == 0) {
      *s = static_cast<uint8_t>(code);
    }
  }
}

// 2^(b - 127) as fp32; byte 255 is NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}

// Four E4M3 bytes times s, as four bf16.
__device__ __forceinline__ uint2 dequant4(uint32_t w, float s) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
  float f[4];
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[0]), "=f"(f[1]) : "r"(lo));
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f[2]), "=f"(f[3]) : "r"(hi));
  return make_uint2(bf16x2_rn(f[0] * s, f[1] * s), bf16x2_rn(f[2] * s, f[3] * s));
}

// A warp reads R consecutive rows; 32 / R lanes look up a row each, then all lanes take the rows' columns, 8 a lane.
// Three loads depend on one another before a row's first byte (its sequence, its page, itself), so many rows want a
// warp with four in flight: 40960 rows of 8 x 128, keys and values, 62.6 -> 42.2 us.
template <int R>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kLanes = 32 / R;
  const Tensor& t = a.t[blockIdx.y];
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const uint32_t group = (kLanes == 32 ? 0xffffffffu : (1u << kLanes) - 1) << (lane - sub);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * R;
  if (row0 >= a.rows) return;
  const int64_t row = row0 + lane / kLanes;
  // the last b with cu[b] <= row, kLanes candidates a step
  int64_t b = -1, n = a.B + 1;
  while (true) {
    const int64_t step = (n + kLanes - 1) / kLanes, i = sub * step, at = b < 0 ? i : b + i;
    const uint32_t le = __ballot_sync(0xffffffffu, i < n && a.cu[at] <= row) & group;
    const int64_t k = (__popc(le) - 1) * step;  // (below zero: in front of the first row)
    if (le != 0) {
      b = (b < 0 ? 0 : b) + k;
      n = min(step, n - k);
    } else {
      n = 1;
    }
    if (__all_sync(0xffffffffu, n <= 1)) break;
  }
  // 0: not to be written, 1: zeros, 2: there
  int state = row < a.rows && b >= 0 && b < a.B ? 1 : 0;
  int64_t data_at = 0, sf_at = 0;
  if (state != 0) {
    const int64_t pos = row - a.cu[b] + (a.starts != nullptr ? a.starts[b] : 0);
    if (pos >= 0 && pos < static_cast<int64_t>(a.table_width) * a.page_size) {
      const uint32_t p = static_cast<uint32_t>(pos / a.page_size), place = static_cast<uint32_t>(pos - static_cast<int64_t>(p) * a.page_size);
      const uint32_t page = static_cast<uint32_t>(a.table[b * a.ld_table + p]);
      if (page < a.pages) {
        state = 2;
        data_at = page * t.page + place * t.token;
        sf_at = page * t.sf_page + place * t.sf_token;
      }
    }
  }
  int st[R];
  const uint8_t *data[R], *sf[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    st[r] = __shfl_sync(0xffffffffu, state, r * kLanes);
    data[r] = t.data + __shfl_sync(0xffffffffu, data_at, r * kLanes);
    sf[r] = t.sf + __shfl_sync(0xffffffffu, sf_at, r * kLanes);
  }
  for (uint32_t col0 = 8 * lane; col0 < (t.width + 255u & ~255u); col0 += 256 * kUnits) {
    uint2 v[kUnits][R];
    uint32_t s[kUnits][R];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t c = col0 + 256 * u, h = c / t.dim, d = c - h * t.dim;
      const int64_t da = h * t.head + d, sa = h * t.sf_head + (d >> 5);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = st[r] == 2 && c < t.width;
        v[u][r] = in ? *reinterpret_cast<const uint2*>(data[r] + da) : make_uint2(0, 0);
        s[u][r] = in ? sf[r][sa] : 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t c = col0 + 256 * u;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (c >= t.width || st[r] == 0) continue;
        const float f = ue8m0_value(s[u][r]);
        const uint2 x = dequant4(v[u][r].x, f), y = dequant4(v[u][r].y, f);
        *reinterpret_cast<uint4*>(const_cast<uint16_t*>(t.rows) + (row0 + r) * t.ld + c) = make_uint4(x.x, x.y, y.x, y.y);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteLaunch& l, cudaStream_t stream) {
  WriteArgs a{};
  int64_t chunks = 0;
  for (int i = 0; i < l.tensors; ++i) {
    a.t[i] = tensor(l.t[i]);
    chunks = chunks > a.t[i].chunks ? chunks : a.t[i].chunks;
  }
  const int64_t warps = l.T * chunks;
  a.slots = l.slots;
  a.T = l.T;
  a.page_size = static_cast<uint32_t>(l.t[0].c.page_size);
  a.by_page = divisor(a.page_size);
  a.slots_end = static_cast<uint32_t>(l.t[0].c.pages * l.t[0].c.page_size);
  const int64_t blocks = (warps + kWarps - 1) / kWarps;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  kv_write_kernel<<<dim3(static_cast<unsigned>(blocks), l.tensors), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvReadLaunch& l, cudaStream_t stream) {
  ReadArgs a{};
  for (int i = 0; i < l.tensors; ++i) a.t[i] = tensor(l.t[i]);
  a.table = l.table;
  a.ld_table = l.ld_table;
  a.table_width = static_cast<uint32_t>(l.table_width);
  a.B = l.B;
  a.rows = l.rows;
  a.cu = l.cu;
  a.starts = l.starts;
  a.page_size = static_cast<uint32_t>(l.t[0].c.page_size);
  a.pages = static_cast<uint32_t>(l.t[0].c.pages);
  const bool many = l.rows >= kManyRows;
  const int64_t per = kWarps * (many ? 4 : 1), blocks = (l.rows + per - 1) / per;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks), l.tensors);
  if (many) kv_read_kernel<4><<<grid, kWarps * 32, 0, stream>>>(a);
  else kv_read_kernel<1><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxq
