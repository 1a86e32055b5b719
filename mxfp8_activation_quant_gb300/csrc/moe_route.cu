// The router of a mixture of experts (moe_route): scores, balance bias, group limit, top-k and
// renormalised weights, one warp per token.
//
// 4 E bytes read and 8 k written per token against E exponentials: at any T this is a matter of
// latency and instruction issue, so a token's E logits stay in one warp's registers (expert
// 32 i + lane in register i, no alignment asked of rows), the groups' values meet in shared
// memory, and each of the k picks is two warp reductions (largest key, then lowest index of it).
//
// Which experts are chosen does not depend on fp32 rounding. Without a bias the order of the
// choices is that of the logits, which is exact. Otherwise choices and group values are computed
// in fp32 with a known error bound; where two values whose order matters are nearer than the
// bound, the warp decides the row again in fp64 (about one row in a thousand at 256 experts with
// standard-normal logits).
#include <cfloat>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "mxq_device.cuh"
#include "mxq_moe_internal.h"

namespace mxq {
namespace {

constexpr int kWarps = 4;

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  const float* bias;
  int64_t T;
  int32_t E, k, groups, topk_groups, group_top, gsize;
  uint32_t gmul;  // expert e lies in group (e * gmul) >> 22
  int32_t softmax, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

// Order-preserving map of finite floats (and +inf) to positive integers; -inf and NaN give 0,
// "never chosen".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t k = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return v > -CUDART_INF_F ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t row, int e) {
  float v;
  if (BF16)
    v = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[row * a.ldl + e]) << 16);
  else
    v = static_cast<const float*>(a.logits)[row * a.ldl + e];
  return v > FLT_MAX ? FLT_MAX : v;
}

// fp32 score of one logit; for softmax `m` is the row's maximum and `inv` 1 / the sum.
__device__ __forceinline__ float score32(float l, bool softmax, float m, float inv) {
  return softmax ? expf(l - m) * inv : 1.f / (1.f + expf(-l));
}

// Relative error bounds of score32. expf is within 2 ulp (2^-22). Sigmoid: exp, sum and division
// stay below 2^-21.4. Softmax adds the rounding of l - m (|l - m| 2^-24 relative to a score that
// is itself e^-|l - m| of the largest), the sum of E terms in at most 37 additions, a reciprocal
// and a product: below 2^-18.4 for every score above 2^-24 of the largest.
constexpr float kSigmoidErr = 4.8e-7f;  // 2^-21
constexpr float kSoftmaxErr = 3.9e-6f;  // 2^-18

// Whether two fp32 values may be out of order: score_err bounds their scores' errors together,
// and each value carries up to three roundings of numbers no larger than `size`.
__device__ __forceinline__ bool too_near(float hi, float lo, float score_err, float size) {
  return hi - lo <= score_err + 4.8e-7f * size;
}

// One row decided in fp64. `d` holds E doubles per warp. Returns this lane's pick (lane r: slot r).
template <int VPL, bool BF16>
__device__ __noinline__ int route_row_f64(const RouteArgs& a, int64_t row, double* d, int lane) {
  double m = -CUDART_INF, sum = 0.0;
  if (a.softmax) {
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_logit<BF16>(a, row, e);
      if (l > -CUDART_INF_F) m = fmax(m, static_cast<double>(l));
    }
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int e = lane; e < a.E; e += 32) {
      const float l = load_logit<BF16>(a, row, e);
      if (l > -CUDART_INF_F) sum += exp(static_cast<double>(l) - m);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  for (int e = lane; e < a.E; e += 32) {
    const double l = load_logit<BF16>(a, row, e);
    double c = a.softmax ? exp(l - m) / sum : 1.0 / (1.0 + exp(-l));
    if (a.bias != nullptr) c += static_cast<double>(a.bias[e]);
    if (!(l > -CUDART_INF) || !(c > -CUDART_INF)) c = -CUDART_INF;
    d[e] = c;
  }
  __syncwarp();
  uint32_t kept = 0xFFFFFFFFu;
  if (a.groups > 1) {
    double v = -CUDART_INF;
    if (lane < a.groups) {
      double b0 = -CUDART_INF, b1 = -CUDART_INF;
      for (int i = 0; i < a.gsize; ++i) {
        const double c = d[lane * a.gsize + i];
        if (c > b0) {
          b1 = b0;
          b0 = c;
        } else if (c > b1) {
          b1 = c;
        }
      }
      v = b0;
      if (a.group_top == 2 && b1 > -CUDART_INF) v += b1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double u = __shfl_sync(0xffffffffu, v, g);
      rank += (u > v || (u == v && g < lane)) ? 1 : 0;
    }
    kept = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.topk_groups && v > -CUDART_INF);
  }
  // without a bias experts are ordered by their logits (scores may underflow to the same value)
  for (int e = lane; e < a.E; e += 32) {
    if (a.groups > 1 && !((kept >> ((e * a.gmul) >> 22)) & 1u)) d[e] = -CUDART_INF;
    else if (a.bias == nullptr && d[e] > -CUDART_INF) d[e] = static_cast<double>(load_logit<BF16>(a, row, e));
  }
  __syncwarp();
  int mine = -1;
  for (int r = 0; r < a.k; ++r) {
    double b = -CUDART_INF;
    int at = 0x7FFFFFFF;
    for (int e = lane; e < a.E; e += 32)
      if (d[e] > b) {
        b = d[e];
        at = e;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, b, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (ob > b || (ob == b && oa < at)) {
        b = ob;
        at = oa;
      }
    }
    if (!(b > -CUDART_INF)) break;
    if (lane == r) mine = at;
    if (lane == (at & 31)) d[at] = -CUDART_INF;
    __syncwarp();
  }
  return mine;
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  __shared__ double scratch[kWarps][VPL * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= a.T) return;  // whole warps; the block never synchronizes

  float c[VPL];  // logits, then choices
  uint32_t key[VPL];
  float m = -CUDART_INF_F, inv = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    c[i] = e < a.E ? load_logit<BF16>(a, row, e) : -CUDART_INF_F;
    if (!(c[i] > -CUDART_INF_F)) c[i] = -CUDART_INF_F;  // NaN too
  }
  if (a.softmax) {
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) mk = max(mk, order_key(c[i]));
    mk = __reduce_max_sync(0xffffffffu, mk);
    m = mk ? key_value(mk) : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += expf(c[i] - m);  // exp(-inf) = 0
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  const float rel = a.softmax ? kSoftmaxErr : kSigmoidErr;
  const bool sums = a.groups > 1 && a.group_top == 2;
  const bool values = a.bias != nullptr || sums;  // choices are computed, not only ordered
  float smax = 0.f, cmax = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = 32 * i + lane;
    const bool there = c[i] > -CUDART_INF_F;
    key[i] = order_key(c[i]);
    if (values) {
      const float s = there ? score32(c[i], a.softmax, m, inv) : 0.f;
      smax = fmaxf(smax, s);
      c[i] = there ? s + (a.bias != nullptr ? a.bias[e] : 0.f) : -CUDART_INF_F;
      if (a.bias != nullptr) key[i] = order_key(c[i]);
      if (there) cmax = fmaxf(cmax, fabsf(c[i]));
    }
  }

  bool near = false;
  if (a.groups > 1) {
    float* sc = reinterpret_cast<float*>(scratch[warp]);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (32 * i + lane < a.E) sc[32 * i + lane] = key[i] ? c[i] : -CUDART_INF_F;
    __syncwarp();
    float v = -CUDART_INF_F;
    if (lane < a.groups) {
      float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
      int i = lane % a.gsize;  // lanes start at different members: fewer bank conflicts
      for (int n = 0; n < a.gsize; ++n) {
        const float u = sc[lane * a.gsize + i];
        b1 = fmaxf(b1, fminf(b0, u));
        b0 = fmaxf(b0, u);
        i = i + 1 == a.gsize ? 0 : i + 1;
      }
      v = b0;
      if (a.group_top == 2 && b1 > -CUDART_INF_F) v += b1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float u = __shfl_sync(0xffffffffu, v, g);
      rank += (u > v || (u == v && g < lane)) ? 1 : 0;
    }
    const bool have = lane < a.groups && v > -CUDART_INF_F;
    const uint32_t kept = __ballot_sync(0xffffffffu, have && rank < a.topk_groups);
    if (values) {
      // the least kept value against the largest one left out
      smax = key_value(__reduce_max_sync(0xffffffffu, order_key(smax)));
      cmax = key_value(__reduce_max_sync(0xffffffffu, order_key(cmax)));
      const uint32_t in = __reduce_min_sync(0xffffffffu, have && rank < a.topk_groups ? order_key(v) : 0xFFFFFFFFu);
      const uint32_t out = __reduce_max_sync(0xffffffffu, have && rank >= a.topk_groups ? order_key(v) : 0u);
      if (out != 0u) near = too_near(key_value(in), key_value(out), 2.f * a.group_top * rel * smax, 2.f * cmax);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t g = (static_cast<uint32_t>(32 * i + lane) * a.gmul) >> 22;
      if (!((kept >> (g & 31u)) & 1u)) key[i] = 0u;
    }
  }

  // k picks, and the runner-up when the choices carry errors
  const int rounds = a.k + (a.bias != nullptr ? 1 : 0);
  int mine = -1;
  float my_c = -CUDART_INF_F, next_c = -CUDART_INF_F;
  int next = -1;
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
  for (int r = 0; r < rounds; ++r) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0u) break;
    int at = 0x7FFFFFFF;
    if (best == top) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == top) at = 32 * i + lane;
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (r == a.k) {
      next = at;
      next_c = key_value(top);
      break;
    }
    if (lane == r) {
      mine = at;
      my_c = key_value(top);
    }
    if ((at & 31) == lane) {
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (32 * i + lane == at) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
  }
  float s = mine >= 0 ? score32(load_logit<BF16>(a, row, mine), a.softmax, m, inv) : 0.f;
  if (a.bias != nullptr) {
    // neighbours in the order (lane r against slot r + 1, the last one against the runner-up)
    float s2 = __shfl_down_sync(0xffffffffu, s, 1), c2 = __shfl_down_sync(0xffffffffu, my_c, 1);
    if (lane == a.k - 1) {
      c2 = next_c;
      s2 = next >= 0 ? score32(load_logit<BF16>(a, row, next), a.softmax, m, inv) : 0.f;
    }
    const bool pair = mine >= 0 && lane < a.k && c2 > -CUDART_INF_F;
    near = __any_sync(0xffffffffu, near || (pair && too_near(my_c, c2, rel * (s + s2), fmaxf(fabsf(my_c), fabsf(c2)))));
  }
  if (near) {
    __syncwarp();  // the float scratch is read no more
    mine = route_row_f64<VPL, BF16>(a, row, scratch[warp], lane);
    s = mine >= 0 ? score32(load_logit<BF16>(a, row, mine), a.softmax, m, inv) : 0.f;
  }
  float w = s;
  if (a.renorm) {
    float sum = lane < a.k ? s : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = s / (sum + 1e-20f);
  }
  if (lane < a.k) {
    a.ids[row * a.k + lane] = mine;
    a.weights[row * a.k + lane] = w * a.scale;
  }
}

template <int VPL>
cudaError_t launch_vpl(const RouteArgs& a, bool bf16, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.T + kWarps - 1) / kWarps);
  if (bf16)
    route_kernel<VPL, true><<<grid, kWarps * 32, 0, stream>>>(a);
  else
    route_kernel<VPL, false><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteLaunch& l, cudaStream_t stream) {
  RouteArgs a = {};
  a.logits = l.logits;
  a.ldl = l.ldl;
  a.bias = l.bias;
  a.T = l.T;
  a.E = l.E;
  a.k = l.k;
  a.groups = l.groups;
  a.topk_groups = l.topk_groups;
  a.group_top = l.group_top;
  a.gsize = l.E / l.groups;
  a.gmul = (1u << 22) / static_cast<uint32_t>(a.gsize) + 1u;
  a.softmax = l.softmax;
  a.renorm = l.renormalize;
  a.scale = l.scale;
  a.ids = l.ids;
  a.weights = l.weights;
  if (l.E <= 64) return launch_vpl<2>(a, l.bf16_logits, stream);
  if (l.E <= 128) return launch_vpl<4>(a, l.bf16_logits, stream);
  if (l.E <= 256) return launch_vpl<8>(a, l.bf16_logits, stream);
  if (l.E <= 512) return launch_vpl<16>(a, l.bf16_logits, stream);
  return launch_vpl<32>(a, l.bf16_logits, stream);
}

}  // namespace mxq
