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

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return bf16x2_rn(bf16_lo(a) + bf16_lo(b), bf16_hi(a) + bf16_hi(b));
}

template <int CPT, bool F32, int NT>
__global__ void __launch_bounds__(NT) add_rmsnorm_kernel(const AddRmsArgs a) {
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool vrow = row < a.T;  // (rows past T only zero the padding of the scale layouts)
  __shared__ float red[NT / 32];

  uint4 hb[F32 ? 1 : CPT];       // the stored h: packed bf16, or fp32
  float hf[F32 ? CPT * 8 : 1];
  float ss = 0.f;
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
      if (vrow && c < a.H) *reinterpret_cast<uint4*>(a.res_out + row * a.ldro_b + 2 * c) = hb[j];
      const uint32_t w[4] = {hb[j].x, hb[j].y, hb[j].z, hb[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
        ss = fmaf(lo, lo, ss);
        ss = fmaf(hi, hi, ss);
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
        dst[0] = make_float4(h[0], h[1], h[2], h[3]);
        dst[1] = make_float4(h[4], h[5], h[6], h[7]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) red[warp] = ss;
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) total += red[i];
  const float r = rsqrtf(total / a.h + a.eps);

#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (static_cast<int64_t>(8) * NT * j >= a.H) break;  // block-uniform
    const int64_t c = 8 * (tid + NT * j);
    uint4 y = make_uint4(0, 0, 0, 0);
    if (vrow && c < a.H) {
      const uint4 g = *reinterpret_cast<const uint4*>(a.gamma + c);
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
      uint32_t yw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        if constexpr (F32) {
          lo = hf[8 * j + 2 * i];
          hi = hf[8 * j + 2 * i + 1];
        } else {
          const uint32_t w = i == 0 ? hb[j].x : i == 1 ? hb[j].y : i == 2 ? hb[j].z : hb[j].w;
          lo = bf16_lo(w);
          hi = bf16_hi(w);
        }
        yw[i] = bf16x2_rn((lo * r) * bf16_lo(gw[i]), (hi * r) * bf16_hi(gw[i]));
      }
      y = make_uint4(yw[0], yw[1], yw[2], yw[3]);
      if (a.y != nullptr) *reinterpret_cast<uint4*>(a.y + row * a.H + c) = y;
    }
    if (a.yq == nullptr) continue;
    uint32_t amax = absmax8(y);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = ue8m0_from_bf16_amax(amax);
    if (vrow && c < a.H) *reinterpret_cast<uint2*>(a.yq + row * a.H + c) = quant8(y, ue8m0_inverse(code));
    store_unit_scales(a.q, row, c, code, lane);
  }
}

template <bool F32, int NT>
cudaError_t launch_nt(const AddRmsArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.rows_total);
  switch ((a.H / 8 + NT - 1) / NT) {  // 8-element chunks per thread
    case 1: add_rmsnorm_kernel<1, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    case 2: add_rmsnorm_kernel<2, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    case 3: add_rmsnorm_kernel<3, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    case 4: add_rmsnorm_kernel<4, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    case 5: case 6: add_rmsnorm_kernel<6, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    case 7: case 8: add_rmsnorm_kernel<8, F32, NT><<<grid, NT, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
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
  return l.fp32_stream ? launch_nt<true, 256>(a, stream) : launch_nt<false, 256>(a, stream);
}

}  // namespace mxq
