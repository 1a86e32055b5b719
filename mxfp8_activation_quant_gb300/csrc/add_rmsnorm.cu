// Residual addition + RMSNorm with bf16 and MXFP8 outputs (add_rmsnorm_dual_out): one pass over
// the residual stream.
//
//   h = RNE_st(x + residual), y = RNE_bf16((h r) gamma), r = 1 / sqrt(mean h^2 + eps),
//   (y_q, scales) = MXFP8(y)
//
// HBM bound: 9 1/32 bytes per element with a bf16 stream and one scale layout (13 1/32 with fp32)
// against about 10 fp32 operations. One block per row, so that every element is read once and kept
// in registers between the sum of squares and the outputs; thread t owns the 8-element chunks t,
// t + NT, ... of the row, in 16-byte loads. NT is a multiple of 16, so a scale word's 16 chunks stay
// in 16 lanes of one warp.
//
// y is rounded from the exact value of the formula in fp32, rounded once: its group's scale and codes
// hang on the bf16 rounding, and a chain of fp32 roundings would fall one value in ten thousand on the
// other side. The sum of squares
// and r are held as unevaluated sums of two floats (error-free sums and products, Dekker 1971, Knuth
// 4.2.2); (h r) gamma is taken in fp32, within 4 ulp, and only where that lies within 4 ulp of a bf16
// midpoint (one value in 7000) it is taken again with its error terms. 8192 x 5120: 57 us without and
// 60.5 us with it. The two-float sum holds while it lies well inside fp32; a row whose sum of squares
// does not (|h| above about 1e19, infinities and NaN, or next to nothing with an eps as small) is taken
// in fp64 instead.
#include <cfloat>
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_moe_internal.h"
#include "mxq_scales.cuh"

namespace mxq {
namespace {

struct AddRmsArgs {
  const uint16_t* x;
  const uint8_t* res;  // row strides in bytes
  const uint16_t* gamma;
  float eps, h;
  int64_t T, H, ldx, ldr_b, ldro_b;
  uint8_t* res_out;
  uint16_t* y;
  uint8_t* yq;
  int64_t rows_total;
  bool far;  // y is more than the next kernel can find in L2
  QuantArgs q;
};

// The residual is read through the coherent path: in place, this kernel also writes it.
__device__ __forceinline__ uint4 ld_row_u4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// The stream is not read again before the next layer, and y is read next: the stream's stores may leave
// L2 first, y's too when it is larger than L2 anyway (8192 x 5120: 67.3 us in a loop with plain stores,
// 66.9 with the stream's set aside, 64.1 with all).
template <typename V>
__device__ __forceinline__ void put(V* p, const V v, bool far) {
  if (far)
    __stcs(p, v);
  else
    *p = v;
}

// The codes and scales of 8 values of y; a warp holds 256 of a row, `in`: these are in it.
__device__ __forceinline__ void store_codes(const AddRmsArgs& a, int64_t row, int64_t c, const uint4 y, int lane, bool in) {
  uint32_t amax = absmax8(y);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t code = ue8m0_from_bf16_amax(amax);
  if (in) put(reinterpret_cast<uint2*>(a.yq + row * a.H + c), quant8(y, ue8m0_inverse(code)), a.far);
  store_unit_scales(a.q, row, c, code, lane);
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return bf16x2_rn(bf16_lo(a) + bf16_lo(b), bf16_hi(a) + bf16_hi(b));
}

// Two floats in one register pair: one instruction does both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// (s, lo) += v, both halves; the error of every addition goes to lo. (a - b as fma(b, -1, a): exact.)
__device__ __forceinline__ void dd_add2(F2& s, F2& lo, F2 v, F2 minus1) {
  const F2 t = add2(s, v), d = fma2(s, minus1, t);
  const F2 e = add2(fma2(fma2(d, minus1, t), minus1, s), fma2(d, minus1, v));
  s = t;
  lo = add2(lo, e);
}

// a + b as a rounded sum and its error (any order of magnitudes)
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}
// (s, lo) += (v, v_lo)
__device__ __forceinline__ void dd_add(float& s, float& lo, float v, float v_lo) {
  float e;
  s = two_sum(s, v, e);
  lo = __fadd_rn(lo, __fadd_rn(e, v_lo));
}

// 1 / sqrt(sum / n + eps) in two parts, relative error below 2^-43: one Newton step whose residual
// 1 - m r^2 is formed from exact products.
__device__ __forceinline__ float2 dd_rsqrt_mean(float s, float lo, float n, float eps) {
  float e;
  const float q = __fdiv_rn(s, n);
  const float q_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, n, s), lo), n);
  const float m = two_sum(q, eps, e);
  const float m_lo = __fadd_rn(e, q_lo);
  const float r = rsqrtf(m);
  const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
  float t = __fmaf_rn(-m, p, 1.f);
  t = __fmaf_rn(-m, pe, t);
  t = __fmaf_rn(-m_lo, p, t);
  const float c = 0.5f * r * t;
  const float hi = __fadd_rn(r, c);
  return make_float2(hi, __fadd_rn(__fsub_rn(r, hi), c));
}

// Within 4 ulp of the midpoint of two bf16 values; of two values at once, the smaller distance (plus 4)
// of each half and `least`.
__device__ __forceinline__ bool near_midpoint(float y) { return ((__float_as_uint(y) - 0x7FFCu) & 0xFFFFu) <= 8u; }
__device__ __forceinline__ uint32_t midpoint_min2(float y0, float y1, uint32_t least) {
  const uint32_t low = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x5410);
  return __viaddmin_u16x2(low, 0x80048004u, least);  // - 0x7FFC in each half
}

// The sum of squares and n eps, at least: squares' errors below fp32's range then stay under 2^-43 of it.
constexpr float kLeastSum = 8.3e-25f;  // 2^-80

// (h r) g rounded once to fp32.
__device__ __forceinline__ float rounded_once(float h, float2 r, float g) {
  const float p = __fmul_rn(h, r.x), pe = __fmaf_rn(h, r.y, __fmaf_rn(h, r.x, -p));
  const float q = __fmul_rn(p, g), qe = __fmaf_rn(pe, g, __fmaf_rn(p, g, -q));
  return __fadd_rn(q, qe);
}

// One row of the block in fp64, from the stream as it has just been stored (each thread reads what it wrote).
template <bool F32, int NT>
__device__ __noinline__ void row_f64(const AddRmsArgs& a, int64_t row) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ double red[NT / 32];
  auto load = [&](int64_t i) {
    const uint8_t* h = a.res_out + row * a.ldro_b;
    return static_cast<double>(F32 ? reinterpret_cast<const float*>(h)[i]
                                   : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(h)[i]) << 16));
  };
  double ss = 0.0;
  for (int64_t c = 8 * tid; c < a.H; c += 8 * NT)
    for (int i = 0; i < 8; ++i) {
      const double h = load(c + i);
      ss += h * h;
    }
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  ss = 0.0;
  for (int i = 0; i < NT / 32; ++i) ss += red[i];
  const double r = 1.0 / sqrt(ss / static_cast<double>(a.h) + static_cast<double>(a.eps));
  for (int64_t c0 = 0; c0 < a.H; c0 += 8 * NT) {  // (whole warps: the scales are gathered by shuffles)
    const int64_t c = c0 + 8 * tid;
    uint32_t yw[4] = {};
    if (c < a.H) {
      for (int i = 0; i < 4; ++i) {
        float y[2];
        for (int j = 0; j < 2; ++j) {
          const float g = __uint_as_float(static_cast<uint32_t>(a.gamma[c + 2 * i + j]) << 16);
          y[j] = static_cast<float>(load(c + 2 * i + j) * r * static_cast<double>(g));
        }
        yw[i] = bf16x2_rn(y[0], y[1]);
      }
    }
    const uint4 y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
    if (a.y != nullptr && c < a.H) *reinterpret_cast<uint4*>(a.y + row * a.H + c) = y;
    if (a.yq != nullptr) store_codes(a, row, c, y, lane, c < a.H);
  }
}

// Blocks per SM that the registers have to leave room for, by the floats that a thread holds.
template <int CPT, bool F32, int NT>
constexpr int kMinBlocks = (CPT * (F32 ? 2 : 1) <= 4 ? 1280 : CPT * (F32 ? 2 : 1) <= 8 ? 800 : 320) / NT;

template <int CPT, bool F32, int NT>
__global__ void __launch_bounds__(NT, (kMinBlocks<CPT, F32, NT>)) add_rmsnorm_kernel(const AddRmsArgs a) {
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool vrow = row < a.T;  // (rows past T only zero the padding of the scale layouts)
  __shared__ float2 red[NT / 32];

  uint4 hb[F32 ? 1 : CPT];       // the stored h: packed bf16, or fp32
  float hf[F32 ? CPT * 8 : 1];
  const F2 minus1 = pack2(-1.f, -1.f);
  F2 ss2 = pack2(0.f, 0.f), lo2 = ss2;  // sum of squares and its error, even and odd elements
  if constexpr (!F32) {
    uint4 xv[CPT], rv[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t c = 8 * (tid + NT * j);
      const bool in = vrow && c < a.H;
      xv[j] = in ? ld_stream_u4(a.x + row * a.ldx + c) : make_uint4(0, 0, 0, 0);
      rv[j] = in ? ld_row_u4(a.res + row * a.ldr_b + 2 * c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t c = 8 * (tid + NT * j);
      hb[j] = make_uint4(add_bf16x2(xv[j].x, rv[j].x), add_bf16x2(xv[j].y, rv[j].y), add_bf16x2(xv[j].z, rv[j].z),
                         add_bf16x2(xv[j].w, rv[j].w));
      if (vrow && c < a.H) __stcs(reinterpret_cast<uint4*>(a.res_out + row * a.ldro_b + 2 * c), hb[j]);
      const uint32_t w[4] = {hb[j].x, hb[j].y, hb[j].z, hb[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 h = pack2(bf16_lo(w[i]), bf16_hi(w[i]));
        dd_add2(ss2, lo2, mul2(h, h), minus1);  // (squares of bf16 are exact)
      }
    }
  } else {
    uint4 xv[CPT], r0[CPT], r1[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t c = 8 * (tid + NT * j);
      const bool in = vrow && c < a.H;
      xv[j] = in ? ld_stream_u4(a.x + row * a.ldx + c) : make_uint4(0, 0, 0, 0);
      r0[j] = in ? ld_row_u4(a.res + row * a.ldr_b + 4 * c) : make_uint4(0, 0, 0, 0);
      r1[j] = in ? ld_row_u4(a.res + row * a.ldr_b + 4 * c + 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int64_t c = 8 * (tid + NT * j);
      const uint32_t w[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
      const uint32_t r[8] = {r0[j].x, r0[j].y, r0[j].z, r0[j].w, r1[j].x, r1[j].y, r1[j].z, r1[j].w};
      float* h = hf + 8 * j;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[2 * i] = bf16_lo(w[i]) + __uint_as_float(r[2 * i]);
        h[2 * i + 1] = bf16_hi(w[i]) + __uint_as_float(r[2 * i + 1]);
      }
      if (vrow && c < a.H) {
        float4* dst = reinterpret_cast<float4*>(a.res_out + row * a.ldro_b + 4 * c);
        __stcs(dst, make_float4(h[0], h[1], h[2], h[3]));
        __stcs(dst + 1, make_float4(h[4], h[5], h[6], h[7]));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 v = pack2(h[2 * i], h[2 * i + 1]), sq = mul2(v, v);
        lo2 = add2(lo2, fma2(v, v, fma2(sq, minus1, pack2(0.f, 0.f))));
        dd_add2(ss2, lo2, sq, minus1);
      }
    }
  }
  float ss = unpack2(ss2).x, ss_lo = unpack2(lo2).x;
  dd_add(ss, ss_lo, unpack2(ss2).y, unpack2(lo2).y);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, ss, o), v_lo = __shfl_xor_sync(0xffffffffu, ss_lo, o);
    dd_add(ss, ss_lo, v, v_lo);
  }
  if (lane == 0) red[warp] = make_float2(ss, ss_lo);
  __syncthreads();
  ss = ss_lo = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) dd_add(ss, ss_lo, red[i].x, red[i].y);
  const float size = fmaf(a.h, a.eps, ss);
  if (vrow && !(size >= kLeastSum && size <= FLT_MAX)) {  // the same in every thread
    row_f64<F32, NT>(a, row);
    return;
  }
  const float2 r = dd_rsqrt_mean(ss, ss_lo, a.h, a.eps);
  const F2 rr = pack2(r.x, r.x);

#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (static_cast<int64_t>(8) * NT * j >= a.H) break;  // block-uniform
    const int64_t c = 8 * (tid + NT * j);
    uint4 y = make_uint4(0, 0, 0, 0);
    if (vrow && c < a.H) {
      const uint4 g = *reinterpret_cast<const uint4*>(a.gamma + c);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
      float hv[8], yv[8];
      uint32_t least = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          hv[2 * i] = hf[8 * j + 2 * i];
          hv[2 * i + 1] = hf[8 * j + 2 * i + 1];
        } else {
          const uint32_t w = i == 0 ? hb[j].x : i == 1 ? hb[j].y : i == 2 ? hb[j].z : hb[j].w;
          hv[2 * i] = bf16_lo(w);
          hv[2 * i + 1] = bf16_hi(w);
        }
        const float2 v = unpack2(mul2(mul2(pack2(hv[2 * i], hv[2 * i + 1]), rr), pack2(bf16_lo(gw[i]), bf16_hi(gw[i]))));
        yv[2 * i] = v.x;
        yv[2 * i + 1] = v.y;
        least = midpoint_min2(v.x, v.y, least);
      }
      const bool near = min(least & 0xFFFFu, least >> 16) <= 8u;
      if (near) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (near_midpoint(yv[i])) yv[i] = rounded_once(hv[i], r, i & 1 ? bf16_hi(gw[i / 2]) : bf16_lo(gw[i / 2]));
      }
      uint32_t yw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) yw[i] = bf16x2_rn(yv[2 * i], yv[2 * i + 1]);
      y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
      if (a.y != nullptr) put(reinterpret_cast<uint4*>(a.y + row * a.H + c), y, a.far);
    }
    if (a.yq != nullptr) store_codes(a, row, c, y, lane, vrow && c < a.H);
  }
}

// The kernel of the least of CPTS 8-element chunks per thread that holds a row.
template <bool F32, int NT, int... CPTS>
cudaError_t launch_nt(const AddRmsArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.rows_total);
  const int64_t need = (a.H / 8 + NT - 1) / NT;
  bool done = false;
  ((!done && need <= CPTS ? (add_rmsnorm_kernel<CPTS, F32, NT><<<grid, NT, 0, stream>>>(a), done = true) : false), ...);
  return done ? cudaGetLastError() : cudaErrorInvalidValue;
}

// Threads per row. Few rows: a row is one block's latency, so 320 threads (1 x 5120 5.2 us, against 5.6
// with 256 and 6.5 with 160; 333 x 7168 in fp32 9.5 against 9.9 and 10.3). Many rows: more, smaller
// blocks hide one another's reductions (8192 x 5120 60.5 us with 160 threads in 8 blocks per SM,
// against 64.5 with 256 and 66.1 with 320), the fewest with at most four chunks a thread (4000 x 8096
// 52 us with 256 and 66 us with 160, whose eight chunks cost it its residency).
constexpr int64_t kFewRows = 512;
constexpr int64_t kFarBytes = int64_t(96) << 20;  // three quarters of L2

template <bool F32>
cudaError_t launch_type(const AddRmsArgs& a, cudaStream_t stream) {
  const int64_t chunks = a.H / 8;
  if (a.rows_total <= kFewRows) return launch_nt<F32, 320, 1, 2, 3, 4, 6, 8>(a, stream);
  if (chunks <= 2 * 64) return launch_nt<F32, 64, 1, 2>(a, stream);
  if (chunks <= 4 * 160) return launch_nt<F32, 160, 1, 2, 3, 4>(a, stream);
  if (chunks <= 4 * 256) return launch_nt<F32, 256, 3, 4>(a, stream);
  return chunks <= 4 * 320 ? launch_nt<F32, 320, 4>(a, stream) : launch_nt<F32, 512, 3, 4>(a, stream);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t launch_add_rmsnorm(const AddRmsnormLaunch& l, cudaStream_t stream) {
  AddRmsArgs a = {};
  a.x = static_cast<const uint16_t*>(l.x);
  a.res = static_cast<const uint8_t*>(l.residual);
  a.gamma = static_cast<const uint16_t*>(l.gamma);
  a.eps = l.eps;
  a.h = static_cast<float>(l.H);
  a.T = l.T;
  a.H = l.H;
  a.ldx = l.ldx;
  a.ldr_b = l.ldr * (l.fp32_stream ? 4 : 2);
  a.ldro_b = l.ldro * (l.fp32_stream ? 4 : 2);
  a.res_out = static_cast<uint8_t*>(l.residual_out);
  a.y = static_cast<uint16_t*>(l.y);
  a.yq = static_cast<uint8_t*>(l.yq);
  a.far = 3 * l.T * l.H > kFarBytes;
  a.q.M = l.T;
  a.q.K = l.H;
  a.q.sf_rm = static_cast<uint8_t*>(l.sf_rowmajor);
  a.q.sf_pk = static_cast<uint32_t*>(l.sf_packed);
  a.q.sf_tl = static_cast<uint8_t*>(l.sf_tiled);
  a.q.Kg = l.H / 32;
  a.q.Kw = ceil_div(a.q.Kg, 4);
  a.q.Mp4 = ceil_div(l.T, 4) * 4;
  a.q.Mp128 = ceil_div(l.T, 128) * 128;
  a.rows_total = l.sf_tiled ? a.q.Mp128 : (l.sf_packed ? a.q.Mp4 : l.T);
  if (a.rows_total > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return l.fp32_stream ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace mxq
