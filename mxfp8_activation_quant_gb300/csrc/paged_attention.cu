// Attention of one new token per sequence over a paged MXFP8 cache, split over the cache's length and
// joined.
#include <cuda_runtime.h>

#include <algorithm>

#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_kv_internal.h"
#include "mxq_tma.h"

namespace mxq {
namespace {

constexpr int kTile = 32;   // tokens per step
constexpr int kHeads = 8;   // query heads per block
constexpr int kThreads = 256;

struct Cache {
  const uint8_t* data;
  const uint8_t* sf;
  int64_t page, token, head, sf_page, sf_token, sf_head;
};
struct Args {
  const uint16_t* q;
  int64_t ldq, ldqh;
  Cache k, v;
  bool shared;
  const int32_t* table;
  int64_t ld_table;
  uint32_t table_width, page_size, pages;
  const int32_t* lens;
  int32_t B, H, kv, G, D, splits, blocks;
  float scale;
  float* part;   // [B * H * splits][D + 2]
  uint16_t* o;
  uint8_t* oq;
  uint8_t* sf_rm;
  uint32_t* sf_pk;
  uint8_t* sf_tl;
  float* lse;
};

__device__ __forceinline__ float code_value(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(c));
  float f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float scale_value(uint32_t b) { return __uint_as_float(b == 0 ? 0x00400000u : b << 23); }

__global__ void __launch_bounds__(kThreads) split_kernel(const Args a) {
  extern __shared__ float sm[];
  float* q = sm;                    // [8][D]
  float* x = q + kHeads * a.D;      // [32][D]
  float* p = x + kTile * a.D;       // [8][32]
  __shared__ float m[kHeads], l[kHeads], f[kHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / (a.kv * a.blocks), kv = blockIdx.x / a.blocks % a.kv, h0 = blockIdx.x % a.blocks * kHeads;
  const int nh = min(kHeads, a.G - h0), head0 = kv * a.G + h0;
  const int64_t len = max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.lens[b]), static_cast<int64_t>(a.table_width) * a.page_size));
  const int64_t tiles = (len + kTile - 1) / kTile;
  const int64_t t0 = tiles * blockIdx.y / a.splits * kTile, t1 = min(len, tiles * (blockIdx.y + 1) / a.splits * kTile);
  for (int i = tid; i < kHeads * a.D; i += kThreads) {
    const int h = i / a.D;
    q[i] = h < nh ? __uint_as_float(static_cast<uint32_t>(a.q[b * a.ldq + (head0 + h) * a.ldqh + i % a.D]) << 16) : 0.f;
  }
  if (tid < kHeads) m[tid] = -INFINITY, l[tid] = 0.f;
  float o[kHeads][2] = {};
  __syncthreads();
  for (int64_t t = t0; t < t1; t += kTile) {
    for (int which = 0; which < 2; ++which) {
      const Cache& c = which == 0 ? a.k : a.v;
      if (which == 0 || !a.shared) {
        for (int i = tid; i < kTile * a.D; i += kThreads) {
          const int64_t pos = t + i / a.D;
          const int d = i % a.D;
          float v = 0.f;
          if (pos < t1) {
            const uint32_t page = a.table[b * a.ld_table + pos / a.page_size], at = pos % a.page_size;
            if (page < a.pages)
              v = code_value(c.data[page * c.page + at * c.token + kv * c.head + d]) *
                  scale_value(c.sf[page * c.sf_page + at * c.sf_token + kv * c.sf_head + d / 32]);
          }
          x[i] = v;
        }
        __syncthreads();
      }
      if (which == 0) {
        for (int i = warp; i < kHeads * kTile; i += kThreads / 32) {
          const int h = i / kTile, r = i % kTile;
          float s = 0.f;
          for (int d = lane; d < a.D; d += 32) s = fmaf(q[h * a.D + d], x[r * a.D + d], s);
          for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
          const int64_t pos = t + r;
          const bool there = pos < t1 && static_cast<uint32_t>(a.table[b * a.ld_table + pos / a.page_size]) < a.pages;
          if (lane == 0) p[i] = there ? s * a.scale : -INFINITY;
        }
        __syncthreads();
        if (warp < kHeads) {  // one warp per head
          const float s = p[warp * kTile + lane];
          float mx = s;
          for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float mn = fmaxf(m[warp], mx);
          const float e = s == -INFINITY ? 0.f : expf(s - mn);
          float sum = e;
          for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
          p[warp * kTile + lane] = e;
          __syncwarp();
          if (lane == 0) {
            f[warp] = m[warp] == -INFINITY ? 0.f : expf(m[warp] - mn);
            l[warp] = l[warp] * f[warp] + sum;
            m[warp] = mn;
          }
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int d = tid + j * kThreads;
      if (d < a.D)
        for (int h = 0; h < kHeads; ++h) {
          float acc = o[h][j] * f[h];
          for (int r = 0; r < kTile; ++r) acc = fmaf(p[h * kTile + r], x[r * a.D + d], acc);
          o[h][j] = acc;
        }
    }
    __syncthreads();
  }
  for (int h = 0; h < nh; ++h) {
    float* out = a.part + ((static_cast<int64_t>(b) * a.H + head0 + h) * a.splits + blockIdx.y) * (a.D + 2);
    if (tid == 0) out[0] = m[h], out[1] = l[h];
    for (int j = 0; j < 2; ++j)
      if (tid + j * kThreads < a.D) out[2 + tid + j * kThreads] = o[h][j];
  }
}

// One warp per (row, 32 elements of o); rows past the batch write the scale layouts' padding.
__global__ void __launch_bounds__(128) join_kernel(const Args a) {
  const int64_t groups = static_cast<int64_t>(a.H) * a.D / 32, w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t row = w / groups, g = w % groups;
  const int lane = threadIdx.x & 31;
  const int64_t B4 = (a.B + 3) / 4 * 4, B128 = (static_cast<int64_t>(a.B) + 127) / 128 * 128;
  if (row >= B128) return;
  uint32_t code = 0;
  if (row < a.B) {
    const int h = g * 32 / a.D, d = g * 32 % a.D + lane;
    const float* part = a.part + (row * a.H + h) * a.splits * (a.D + 2);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, part[s * (a.D + 2)]);
    for (int s = 0; s < a.splits; ++s) {
      const float* q = part + s * (a.D + 2);
      const float f = q[0] == -INFINITY ? 0.f : expf(q[0] - m);
      l = fmaf(q[1], f, l);
      o = fmaf(q[2 + d], f, o);
    }
    const uint32_t y = bf16x2_rn(l > 0.f ? o / l : 0.f, 0.f) & 0xFFFFu;
    code = ue8m0_from_bf16_amax(__reduce_max_sync(0xffffffffu, y & 0x7FFFu));
    const int64_t at = row * a.H * a.D + g * 32 + lane;
    if (a.o != nullptr) a.o[at] = static_cast<uint16_t>(y);
    if (a.oq != nullptr) a.oq[at] = static_cast<uint8_t>(e4m3x2(bf16_lo(y) * ue8m0_inverse(code), 0.f));
    if (a.lse != nullptr && d == 0) a.lse[row * a.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
  }
  if (lane != 0) return;
  if (a.sf_rm != nullptr && row < a.B) a.sf_rm[row * groups + g] = code;
  if (a.sf_pk != nullptr && row < B4) reinterpret_cast<uint8_t*>(a.sf_pk)[(g / 4 * B4 + row) * 4 + g % 4] = code;
  if (a.sf_tl != nullptr) a.sf_tl[tiled128x4_word_offset(row, g / 4, groups / 4) + g % 4] = code;
}

Cache cache_of(const mxq_kv_cache& c) {
  return {static_cast<const uint8_t*>(c.data), static_cast<const uint8_t*>(c.sf), c.page_stride, c.token_stride, c.head_stride,
          c.sf_page_stride, c.sf_token_stride, c.sf_head_stride};
}

int splits_of(int64_t B, int32_t q_heads, int32_t kv_heads) {
  const int64_t blocks = B * kv_heads * ((q_heads / kv_heads + kHeads - 1) / kHeads);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(64, 608 / blocks)));
}

}  // namespace

int64_t paged_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  return (B * q_heads * splits_of(B, q_heads, kv_heads) * (dim + 2) * 4 + 15) / 16 * 16;
}

cudaError_t launch_paged_attention(const PagedAttentionLaunch& l, cudaStream_t stream) {
  const mxq_kv_cache& k = *l.k;
  Args a{};
  a.q = static_cast<const uint16_t*>(l.q);
  a.ldq = l.ldq;
  a.ldqh = l.ldqh;
  a.k = cache_of(k);
  a.v = cache_of(l.v != nullptr ? *l.v : k);
  a.shared = l.v == nullptr;
  a.table = l.table;
  a.ld_table = l.ld_table;
  a.table_width = static_cast<uint32_t>(l.table_width);
  a.page_size = static_cast<uint32_t>(k.page_size);
  a.pages = static_cast<uint32_t>(k.pages);
  a.lens = l.lens;
  a.B = static_cast<int32_t>(l.B);
  a.H = l.q_heads;
  a.kv = k.heads;
  a.G = l.q_heads / k.heads;
  a.D = k.dim;
  a.blocks = (a.G + kHeads - 1) / kHeads;
  a.splits = splits_of(l.B, l.q_heads, k.heads);
  a.scale = l.scale;
  a.part = static_cast<float*>(l.workspace);
  a.o = static_cast<uint16_t*>(l.o);
  a.oq = static_cast<uint8_t*>(l.o_q);
  a.sf_rm = static_cast<uint8_t*>(l.sf_rowmajor);
  a.sf_pk = static_cast<uint32_t*>(l.sf_packed);
  a.sf_tl = static_cast<uint8_t*>(l.sf_tiled);
  a.lse = l.lse;
  const int bytes = ((kHeads + kTile) * a.D + kHeads * kTile) * 4;
  static PerDevice set;
  cudaError_t e = allow_smem(set, split_kernel, ((kHeads + kTile) * 512 + kHeads * kTile) * 4);
  if (e != cudaSuccess) return e;
  split_kernel<<<dim3(static_cast<unsigned>(a.B * a.kv * a.blocks), a.splits), kThreads, bytes, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t warps = (l.B + 127) / 128 * 128 * a.H * a.D / 32;
  join_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mxq
