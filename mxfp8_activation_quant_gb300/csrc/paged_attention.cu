// Attention over a paged MXFP8 cache: the join of the parts, and the host's side (the attention itself:
// mxq_paged_attention.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "mxq_paged_attention.cuh"

namespace mxq {

using namespace paged;

namespace {

// Adds the parts of the items that more than one CTA held, always in the CTAs' order of a warp's share:
//   o = sum_k (w_k / sum_k w_k) o_k, w_k = l_k 2^(ref_k - max ref), lse = ln 2 (max ref + log2 sum_k w_k);
// divided first, so that no partial sum is larger than the largest part (w_k is up to 2^15 for each token).
// With few items, which then have many parts, or where there is a block for each head and panel, a block takes 128 features of a head and
// its warps every eighth part; else a warp takes a head. The whole call with a block, with a warp (us): 64 heads of 512, 8 items 37.9, 42.6,
// 16 items 44.9, 35.9, 32 items 64.0, 33.7; 16 heads of 256 (32 blocks an item of 608), 16 items 18.6, 22.3, 24 items 21.9, 21.0; 8 heads of 128
// (8 blocks), 64 items 16.8, 17.4, 100 items 19.4, 17.5. Also the scale layouts' padding rows. Bound by the chain of loads (owner,
// statistics, parts) with few parts, 6.6 us alone (serialised, cold), and by L2 with many: 152 parts of 64 x 512, 20 MB, 9.8 us; 216 of them,
// 28 MB, 11 us.
// (Parts asked for before their weights are known: 13.1 us, for the registers.)
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxCtas = 512;
constexpr int kFewItems = 12;

struct JoinWork {
  int j0, h, parts, b, head;
};
__device__ __forceinline__ JoinWork join_work(const Args& a, const int16_t* owners, uint32_t owner, int h) {
  JoinWork w;
  w.j0 = owners[owner];
  w.h = h;
  const int2 own = a.owner[w.j0];
  const uint32_t item = own.x - 1, sub = item / a.B, kvh = sub / a.blocks;
  w.b = item - sub * a.B;
  const int h0 = (sub - kvh * a.blocks) * a.block_heads;
  w.parts = h < min(a.block_heads, a.G - h0) ? own.y - w.j0 + 1 : 0;
  w.head = kvh * a.G + h0 + h;
  return w;
}
// Part k: the first CTA's last segment, the others' first.
__device__ __forceinline__ int join_slot(const JoinWork& w, int k) { return k == 0 ? 2 * w.j0 + 1 : 2 * (w.j0 + k); }

// A warp's features 128 p + 4 lane .. + 3.
__device__ __forceinline__ void join_store(const Args& a, const JoinWork& w, int p, float4 v, int lane) {
  const uint2 y = make_uint2(bf16x2_rn(v.x, v.y), bf16x2_rn(v.z, v.w));
  const int64_t at = (static_cast<int64_t>(w.b) * a.H + w.head) * a.D + 128 * p + 4 * lane;
  if (a.o != nullptr) *reinterpret_cast<uint2*>(a.o + at) = y;
  if (a.oq != nullptr) {
    uint32_t amax = max(absmax_bf16x2(y.x), absmax_bf16x2(y.y));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const uint32_t code = ue8m0_from_bf16_amax(amax);
    const float s = ue8m0_inverse(code);
    *reinterpret_cast<uint32_t*>(a.oq + at) = e4m3x2(bf16_lo(y.x) * s, bf16_hi(y.x) * s) | (e4m3x2(bf16_lo(y.y) * s, bf16_hi(y.y) * s) << 16);
    uint32_t c = code;
    c |= __shfl_down_sync(0xffffffffu, code, 8) << 8;
    c |= __shfl_down_sync(0xffffffffu, code, 16) << 16;
    c |= __shfl_down_sync(0xffffffffu, code, 24) << 24;
    if (lane == 0) {
      const int64_t words = static_cast<int64_t>(a.H) * a.panels, word = static_cast<int64_t>(w.head) * a.panels + p;
      if (a.sf_rm != nullptr) *reinterpret_cast<uint32_t*>(a.sf_rm + (w.b * words + word) * 4) = c;
      if (a.sf_pk != nullptr) *reinterpret_cast<uint32_t*>(a.sf_pk + (word * ((a.B + 3) / 4 * 4) + w.b) * 4) = c;
      if (a.sf_tl != nullptr) *reinterpret_cast<uint32_t*>(a.sf_tl + tiled128x4_word_offset(w.b, word, words)) = c;
    }
  }
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ void join_add(float4& v, float w, const float4 f) {
  v.x = fmaf(w, f.x, v.x), v.y = fmaf(w, f.y, v.y), v.z = fmaf(w, f.z, v.z), v.w = fmaf(w, f.w, v.w);
}

__global__ void __launch_bounds__(kJoinThreads, 4) join_kernel(const __grid_constant__ Args a, int gp) {
  __shared__ int16_t owners[kMaxCtas];
  __shared__ uint32_t masks[kMaxCtas / 32];
  __shared__ float weight[kMaxCtas];
  __shared__ float4 acc[kJoinWarps][32];
  __shared__ float tops[kJoinWarps], sums[kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.sf_pk != nullptr || a.sf_tl != nullptr) {  // a word column per block and a row per thread
    const int words = a.H * a.panels, b4 = (a.B + 3) / 4 * 4, b128 = (a.B + 127) / 128 * 128, row = a.B + tid;
    if (row < b128)
#pragma unroll 1
      for (int w = blockIdx.x; w < words; w += gridDim.x) {
        if (a.sf_pk != nullptr && row < b4) *reinterpret_cast<uint32_t*>(a.sf_pk + (static_cast<int64_t>(w) * b4 + row) * 4) = 0;
        if (a.sf_tl != nullptr) *reinterpret_cast<uint32_t*>(a.sf_tl + tiled128x4_word_offset(row, w, words)) = 0;
      }
  }
  pdl_wait_primary();
  // the owners, in the same order in every block
#pragma unroll
  for (int u = 0; u < kMaxCtas / kJoinThreads; ++u) {
    const int i = u * kJoinThreads + tid;
    const uint32_t all = __ballot_sync(0xffffffffu, i < a.ctas && a.owner[i].x != 0);
    if (lane == 0) masks[i >> 5] = all;
  }
  __syncthreads();
  int count = 0;
#pragma unroll
  for (int k = 0; k < kMaxCtas / 32; ++k) {
    const uint32_t all = masks[k];
    if ((k & (kJoinWarps - 1)) == warp && (all >> lane & 1) != 0) owners[count + __popc(all & ((1u << lane) - 1))] = static_cast<int16_t>(32 * k + lane);
    count += __popc(all);
  }
  __syncthreads();
  const int heads = count * a.block_heads, NP = a.panels;
  if (count > kFewItems && heads * NP > static_cast<int>(gridDim.x)) {
#pragma unroll 1
    for (int i = blockIdx.x * kJoinWarps + warp; i < heads; i += gridDim.x * kJoinWarps) {
      const JoinWork w = join_work(a, owners, static_cast<uint32_t>(i) / a.block_heads, static_cast<uint32_t>(i) % a.block_heads);
      if (w.parts == 0) continue;
      float top = kLowRef, sum = 0.f;
#pragma unroll 1
      for (int k = lane; k < w.parts; k += 32) top = fmaxf(top, a.stat[join_slot(w, k) * gp + w.h].x);
      top = warp_max(top);
#pragma unroll 1
      for (int k = lane; k < w.parts; k += 32) {
        const float2 s = a.stat[join_slot(w, k) * gp + w.h];
        sum += s.y * ex2(s.x - top);
      }
      sum = warp_sum(sum);
      const float inv = sum > 0.f ? 1.0f / sum : 0.f;
      float4 v[4] = {};
#pragma unroll 1
      for (int k0 = 0; k0 < w.parts; k0 += 32) {
        float mine = 0.f;
        if (k0 + lane < w.parts) {
          const float2 s = a.stat[join_slot(w, k0 + lane) * gp + w.h];
          mine = s.y * ex2(s.x - top) * inv;
        }
        const int n = min(32, w.parts - k0);
#pragma unroll 2
        for (int k = 0; k < n; ++k) {
          const float4* x = reinterpret_cast<const float4*>(a.part + (static_cast<int64_t>(join_slot(w, k0 + k)) * gp + w.h) * a.D) + lane;
          const float f = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
          for (int p = 0; p < 4; ++p)
            if (p < NP) join_add(v[p], f, x[32 * p]);
        }
      }
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (p < NP) join_store(a, w, p, v[p], lane);
      if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(w.b) * a.H + w.head] = lse_of(top, sum);
    }
    return;
  }
#pragma unroll 1
  for (int i = blockIdx.x; i < heads * NP; i += gridDim.x) {
    const int h = i / NP, p = i - h * NP;
    const JoinWork w = join_work(a, owners, static_cast<uint32_t>(h) / a.block_heads, static_cast<uint32_t>(h) % a.block_heads);
    if (w.parts == 0) continue;  // block-uniform
    // at most two parts a thread
    const bool one = tid < w.parts, two = tid + kJoinThreads < w.parts;
    const float2 none = make_float2(kLowRef, 0.f);
    const float2 s0 = one ? a.stat[join_slot(w, tid) * gp + w.h] : none;
    const float2 s1 = two ? a.stat[join_slot(w, tid + kJoinThreads) * gp + w.h] : none;
    float top = warp_max(fmaxf(s0.x, s1.x));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, tops[k]);
    const float w0 = s0.y * ex2(s0.x - top), w1 = s1.y * ex2(s1.x - top);
    if (one) weight[tid] = w0;
    if (two) weight[tid + kJoinThreads] = w1;
    const float part_sum = warp_sum(w0 + w1);
    if (lane == 0) sums[warp] = part_sum;
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) sum += sums[k];
    const float inv = sum > 0.f ? 1.0f / sum : 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* const x = a.part + w.h * a.D + 128 * p + 4 * lane;
#pragma unroll 1
    for (int k0 = warp; k0 < w.parts; k0 += 10 * kJoinWarps) {  // ten loads in flight
      float4 f[10];
#pragma unroll
      for (int u = 0; u < 10; ++u) {
        const int k = k0 + u * kJoinWarps;
        f[u] = k < w.parts ? *reinterpret_cast<const float4*>(x + static_cast<int64_t>(join_slot(w, k)) * gp * a.D) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 10; ++u) {
        const int k = k0 + u * kJoinWarps;
        join_add(v, k < w.parts ? weight[k] * inv : 0.f, f[u]);
      }
    }
    acc[warp][lane] = v;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int k = 1; k < kJoinWarps; ++k) join_add(v, 1.0f, acc[k][lane]);
      join_store(a, w, p, v, lane);
      if (a.lse != nullptr && p == 0 && lane == 0) a.lse[static_cast<int64_t>(w.b) * a.H + w.head] = lse_of(top, sum);
    }
    __syncthreads();  // (the weights and sums of the next)
  }
}

// ---- host -----------------------------------------------------------------------------------
// SMs of the current device, asked for once per device.
int cached_sms() {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms();
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) known[dev].store(n = num_sms(), std::memory_order_relaxed);
  return n;
}

int padded_heads(int block_heads) { return block_heads <= 8 ? 8 : block_heads <= 16 ? 16 : block_heads <= 32 ? 32 : 64; }

// A cache as a 4-D tensor (feature, place, head, page) in boxes of 128 features x `box` places.
bool make_cache_map(CUtensorMap* m, const mxq_kv_cache& c, int box) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.heads),
                        static_cast<cuuint64_t>(c.pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride), static_cast<cuuint64_t>(c.head_stride),
                           static_cast<cuuint64_t>(c.page_stride)};
  cuuint32_t boxes[4] = {128u, static_cast<cuuint32_t>(box), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.data, dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, c.dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

// The workspace: parts, statistics, owners, queries.
struct Space {
  int64_t ctas, gp, stat, owner, q, total;
};
Space space_of(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  const int G = q_heads / kv_heads, blocks = (G + kMaxHeads - 1) / kMaxHeads;
  Space s;
  s.gp = padded_heads((G + blocks - 1) / blocks);
  s.ctas = std::min(kMaxCtas, cached_sms());
  s.stat = align256(2 * s.ctas * s.gp * dim * 4);
  s.owner = s.stat + align256(2 * s.ctas * s.gp * 8);
  s.q = s.owner + align256(s.ctas * 8);
  s.total = s.q + B * kv_heads * blocks * (dim / 128) * (s.gp * 256 + 512);
  return s;
}

}  // namespace

int64_t paged_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  return space_of(B, q_heads, kv_heads, dim).total;
}

int64_t paged_attention_units(int64_t B, int32_t q_heads, int32_t kv_heads, int64_t places) {
  const int G = q_heads / kv_heads;
  return B * kv_heads * ((G + kMaxHeads - 1) / kMaxHeads) * ((places + kUnit - 1) / kUnit);
}

cudaError_t launch_paged_attention(const PagedAttentionLaunch& l, cudaStream_t stream) {
  const mxq_kv_cache& k = *l.k;
  Args a{};
  a.q = static_cast<const uint16_t*>(l.q);
  a.ldq = l.ldq;
  a.ldqh = l.ldqh;
  a.k_sf = static_cast<const uint8_t*>(k.sf);
  a.k_sf_page = static_cast<uint32_t>(k.sf_page_stride);
  a.k_sf_token = static_cast<uint32_t>(k.sf_token_stride);
  a.k_sf_head = static_cast<uint32_t>(k.sf_head_stride);
  if (l.v != nullptr) {
    a.v_sf = static_cast<const uint8_t*>(l.v->sf);
    a.v_sf_page = static_cast<uint32_t>(l.v->sf_page_stride);
    a.v_sf_token = static_cast<uint32_t>(l.v->sf_token_stride);
    a.v_sf_head = static_cast<uint32_t>(l.v->sf_head_stride);
  }
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
  a.panels = k.dim / 128;
  a.blocks = (a.G + kMaxHeads - 1) / kMaxHeads;
  a.block_heads = (a.G + a.blocks - 1) / a.blocks;
  a.box = std::min(kUnit, k.page_size & -k.page_size);
  a.box_shift = __builtin_ctz(a.box);
  // 2^(31 + s) / d rounded up, s = floor(log2 d): off by less than d < 2^(s + 1), which t < 2^30 times stays below 2^(31 + s)
  const int s = 31 - __builtin_clz(k.page_size);
  a.page_mul = static_cast<uint32_t>((uint64_t(1) << (31 + s)) / k.page_size + 1);
  a.page_shift = s - 1;
  a.scale = l.scale;
  a.o = static_cast<uint16_t*>(l.o);
  a.oq = static_cast<uint8_t*>(l.o_q);
  a.sf_rm = static_cast<uint8_t*>(l.sf_rowmajor);
  a.sf_pk = static_cast<uint8_t*>(l.sf_packed);
  a.sf_tl = static_cast<uint8_t*>(l.sf_tiled);
  a.lse = l.lse;
  a.status = l.status;
  // scales are copied in the largest pieces that every token's start on a multiple of
  auto vec_of = [&](const mxq_kv_cache& c) {
    const uint64_t all = reinterpret_cast<uintptr_t>(c.sf) | c.sf_page_stride | c.sf_token_stride | c.sf_head_stride;
    return all % 16 == 0 ? 16 : 4;
  };
  a.sf_vec = std::min(vec_of(k), vec_of(l.v != nullptr ? *l.v : k));
  const Space sp = space_of(l.B, l.q_heads, k.heads, k.dim);
  a.ctas = static_cast<int32_t>(
      std::min(sp.ctas, paged_attention_units(l.B, l.q_heads, k.heads, static_cast<int64_t>(l.table_width) * k.page_size)));
  uint8_t* const ws = static_cast<uint8_t*>(l.workspace);
  a.part = reinterpret_cast<float*>(ws);
  a.stat = reinterpret_cast<float2*>(ws + sp.stat);
  a.owner = reinterpret_cast<int2*>(ws + sp.owner);
  a.q_ws = ws + sp.q;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, k, a.box)) return cudaErrorInvalidValue;
  if (l.v == nullptr) mv = mk;
  else if (!make_cache_map(&mv, *l.v, a.box)) return cudaErrorInvalidValue;
  const cudaError_t e = sp.gp == 8    ? launch_heads<8>(mk, mv, a, stream)
                        : sp.gp == 16 ? launch_heads<16>(mk, mv, a, stream)
                        : sp.gp == 32 ? launch_heads<32>(mk, mv, a, stream)
                                      : launch_heads<64>(mk, mv, a, stream);
  return e != cudaSuccess ? e : launch_behind(join_kernel, 4 * cached_sms(), kJoinThreads, 0, stream, a, static_cast<int>(sp.gp));
}

}  // namespace mxq
