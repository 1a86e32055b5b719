// The router of a mixture of experts (moe_route): scores, balance bias, group limit, top-k and
// renormalised weights, one warp per token.
//
// 4 E bytes read and 8 k written per token against E exponentials: at any T this is a matter of
// latency and instruction issue, so a token's E logits stay in one warp's registers. Lane l holds
// experts VPL l .. VPL l + VPL - 1: a group is then a run of lanes wherever VPL divides its size
// (two shuffles at 8 groups of 32; otherwise its values meet in shared memory), the lowest lane
// holds the lowest index of a tie, and each of the k picks is one warp maximum and one ballot.
//
// Which experts are chosen does not depend on fp32 rounding. Without a bias the order of the
// choices is that of the logits, which is exact. Otherwise choices and group values are computed
// in fp32 with an error bound each, and values nearer than their bounds are compared in fp64: for
// sigmoid scores only the groups or picks in question, one value per lane (an fp64 exponential
// takes a warp about 0.7 us; the whole row's, which one row in 10^4 took at first, added 10 us to a
// launch), for softmax scores the sum as well. Three rows in a thousand have such picks at 256 experts
// with logits of deviation 1.6.
//
// 16384 tokens, 256 experts, 8 of 4 of 8 groups: 57 us with one expert per 32 in a lane and groups
// through shared memory, 30 us so.
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
  int32_t group_lanes;  // lanes that hold a group, a power of two; 0: groups do not end between lanes
  int32_t vec, bias_vec;  // rows, and the bias, are 16-byte aligned
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

// Error bounds of the fp32 scores that choices are made of. Sigmoid, 1 / (1 + __expf(-l)): __expf is
// within 2 + 1.173 |l| ulp, which the sigmoid's slope reduces to (2 s + 0.33) 2^-23, the sum and the
// quotient add 2.5 s 2^-23: below 6e-7 in all. Softmax, expf(l - m) / sum: the rounding of l - m
// (|l - m| 2^-24 relative to a score that is itself e^-|l - m| of the largest), expf within 2 ulp,
// the sum in at most 37 additions: below 3.9e-6 of the row's largest score.
constexpr float kSigmoidErr = 6.0e-7f;
constexpr float kSoftmaxErr = 3.9e-6f;

// A choice's exact value is within radius(c, err) of c: the score's error `err`, and kRel |c| for the rounding
// of the sum (2^-24) and of what is reckoned with the two. (A bias may lie far from the scores; the
// bound goes by the choice itself, so that one such expert does not widen the others'.) An infinite choice
// is that of an infinite bias: exact.
constexpr float kRel = 2.4e-7f;
__device__ __forceinline__ float radius(float c, float err) {
  return fabsf(c) <= FLT_MAX ? fmaf(kRel, fabsf(c), err) : 0.f;
}

// A group's value, the least of its terms, and the value's error bound: its terms' (which may cancel) and a
// rounding no larger than theirs. A sum of finite terms that leaves fp32 stands at the type's end.
struct GroupValue {
  float value, least, radius;
};
__device__ __forceinline__ GroupValue group_value(float b0, float b1, int top, float err) {
  GroupValue v = {b0, b0, radius(b0, err)};
  if (top == 2 && b1 > -CUDART_INF_F) {
    v.value = b0 <= FLT_MAX ? fminf(fmaxf(b0 + b1, -FLT_MAX), FLT_MAX) : b0;
    v.least = b1;
    v.radius = b0 <= FLT_MAX ? v.radius + radius(b1, err) : 0.f;
  }
  return v;
}
// order_key of the end of a range of finite values: past the type's end it stands there.
__device__ __forceinline__ uint32_t range_key(float v, float value) {
  return fabsf(value) <= FLT_MAX ? order_key(fminf(fmaxf(v, -FLT_MAX), FLT_MAX)) : order_key(value);
}

// The largest logit and the sum of the softmax in fp64, of one row by its warp.
template <bool BF16>
__device__ __noinline__ double2 softmax_f64(const RouteArgs& a, int64_t row, int lane) {
  double m = -CUDART_INF, sum = 0.0;
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
  return make_double2(m, sum);
}
// An expert's choice in fp64; `soft` from softmax_f64 where that is the score.
template <bool BF16>
__device__ __forceinline__ double choice_f64(const RouteArgs& a, int64_t row, int e, double2 soft) {
  const double l = load_logit<BF16>(a, row, e);
  const double s = a.softmax ? exp(l - soft.x) / soft.y : 1.0 / (1.0 + exp(-l));
  return a.bias != nullptr ? s + static_cast<double>(a.bias[e]) : s;
}

// One row decided in fp64. `d` holds E doubles per warp. Returns this lane's pick (lane r: slot r).
template <int VPL, bool BF16>
__device__ __noinline__ int route_row_f64(const RouteArgs& a, int64_t row, double* d, int lane) {
  const double2 soft = a.softmax ? softmax_f64<BF16>(a, row, lane) : make_double2(0.0, 0.0);
  for (int e = lane; e < a.E; e += 32) {
    const double l = load_logit<BF16>(a, row, e);
    double c = choice_f64<BF16>(a, row, e, soft);
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

// VPL consecutive logits of a row from expert e0, in vectors where `vec` says that they are aligned.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int e0, float (&c)[VPL]) {
  constexpr int kVec = BF16 ? 8 : 4;  // elements of 16 bytes
  if (VPL % kVec == 0 && a.vec && e0 + VPL <= a.E) {
    const char* src = static_cast<const char*>(a.logits) + (row * a.ldl + e0) * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < VPL / kVec; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BF16) {
          c[kVec * i + 2 * j] = bf16_lo(w[j]);
          c[kVec * i + 2 * j + 1] = bf16_hi(w[j]);
        } else {
          c[kVec * i + j] = __uint_as_float(w[j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = c[i] > FLT_MAX ? FLT_MAX : c[i];
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) c[i] = e0 + i < a.E ? load_logit<BF16>(a, row, e0 + i) : -CUDART_INF_F;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (!(c[i] > -CUDART_INF_F)) c[i] = -CUDART_INF_F;  // NaN too
}

// VPL consecutive biases from expert e0 (0 past the last).
template <int VPL>
__device__ __forceinline__ void load_bias(const RouteArgs& a, int e0, float (&v)[VPL]) {
  if (VPL % 4 == 0 && a.bias_vec && e0 + VPL <= a.E) {
#pragma unroll
    for (int i = 0; i < VPL / 4; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(a.bias + e0 + 4 * i);
      v[4 * i] = u.x;
      v[4 * i + 1] = u.y;
      v[4 * i + 2] = u.z;
      v[4 * i + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = e0 + i < a.E ? a.bias[e0 + i] : 0.f;
  }
}

template <int VPL, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  __shared__ double scratch[kWarps][VPL * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= a.T) return;  // whole warps; the block never synchronizes
  const int e0 = VPL * lane;

  float c[VPL];  // logits, then choices
  uint32_t key[VPL];
  load_logits<VPL, BF16>(a, row, e0, c);
  float m = -CUDART_INF_F, inv = 0.f;
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
  const bool sums = a.groups > 1 && a.group_top == 2;
  const bool values = a.bias != nullptr || sums;  // choices are computed, not only ordered
  if (values) {
    float bias[VPL] = {};
    if (a.bias != nullptr) load_bias<VPL>(a, e0, bias);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool there = c[i] > -CUDART_INF_F;
      const float s = a.softmax ? expf(c[i] - m) * inv : __fdividef(1.f, 1.f + __expf(-c[i]));
      key[i] = a.bias != nullptr ? 0u : order_key(c[i]);
      c[i] = there ? s + bias[i] : -CUDART_INF_F;
      if (a.bias != nullptr) key[i] = order_key(c[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = order_key(c[i]);
  }
  float err = kSigmoidErr;
  if (a.softmax) err = kSoftmaxErr * inv;  // the largest score is expf(0) * inv

  bool whole = false;  // decide the whole row in fp64
  double2 soft = make_double2(0.0, 0.0);  // softmax_f64, once it has been wanted
  if (a.groups > 1) {
    GroupValue v = {-CUDART_INF_F, -CUDART_INF_F, 0.f};  // of this lane's group
    int g, kept_lanes = a.group_lanes;
    if (kept_lanes > 0) {  // a group is a run of lanes
      float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float u = key[i] ? c[i] : -CUDART_INF_F;
        b1 = fmaxf(b1, fminf(b0, u));
        b0 = fmaxf(b0, u);
      }
      for (int o = 1; o < kept_lanes; o <<= 1) {
        const float o0 = __shfl_xor_sync(0xffffffffu, b0, o), o1 = __shfl_xor_sync(0xffffffffu, b1, o);
        b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
        b0 = fmaxf(b0, o0);
      }
      v = group_value(b0, b1, a.group_top, err);
      g = lane / kept_lanes;
    } else {  // through shared memory, lane g sums up group g
      float* sc = reinterpret_cast<float*>(scratch[warp]);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e0 + i < a.E) sc[e0 + i] = key[i] ? c[i] : -CUDART_INF_F;
      __syncwarp();
      if (lane < a.groups) {
        float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
        int i = lane % a.gsize;  // lanes start at different members: fewer bank conflicts
        for (int n = 0; n < a.gsize; ++n) {
          const float u = sc[lane * a.gsize + i];
          b1 = fmaxf(b1, fminf(b0, u));
          b0 = fmaxf(b0, u);
          i = i + 1 == a.gsize ? 0 : i + 1;
        }
        v = group_value(b0, b1, a.group_top, err);
      }
      g = lane;
      kept_lanes = 1;
    }
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const float u = __shfl_sync(0xffffffffu, v.value, h * kept_lanes);
      rank += (u > v.value || (u == v.value && h < g)) ? 1 : 0;
    }
    const bool have = g < a.groups && v.value > -CUDART_INF_F;
    bool keep = have && rank < a.topk_groups;
    if (values) {
      // the least that a kept value may be against the most that one left out may be
      const float lo = v.value - v.radius, hi = v.value + v.radius;
      const uint32_t ki = __reduce_min_sync(0xffffffffu, keep ? range_key(lo, v.value) : 0xFFFFFFFFu);
      const uint32_t ko = __reduce_max_sync(0xffffffffu, have && !keep ? range_key(hi, v.value) : 0u);
      if (ko != 0u && ki <= ko) {
        // Some groups lie too near to the border: they are ranked by their values in fp64, a lane for
        // each expert that may be among a group's largest.
        const bool border = have && (keep ? range_key(lo, v.value) <= ko : range_key(hi, v.value) >= ki);
        int* list = reinterpret_cast<int*>(reinterpret_cast<float*>(scratch[warp]) + VPL * 32);
        int n = 0;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int holder = a.group_lanes > 0 ? lane : min((e0 + i) / a.gsize, 31);
          const float thr = __shfl_sync(0xffffffffu, v.least - radius(v.least, err), holder);
          const bool mine = __shfl_sync(0xffffffffu, border, holder) && key[i] != 0u && c[i] + radius(c[i], err) >= thr;
          const uint32_t who = __ballot_sync(0xffffffffu, mine);
          const int at = n + __popc(who & ((1u << lane) - 1u));
          if (mine && at < 32) list[at] = e0 + i;
          n += __popc(who);
        }
        __syncwarp();
        if (n > 32) {
          whole = true;  // too many experts are in question
        } else {
          if (a.softmax) soft = softmax_f64<BF16>(a, row, lane);
          const int e = lane < n ? list[lane] : -1, eg = e >= 0 ? e / a.gsize : -1;
          double d = -CUDART_INF;
          if (e >= 0) d = choice_f64<BF16>(a, row, e, soft);
          double b0 = -CUDART_INF, b1 = -CUDART_INF;
          bool first = e >= 0;  // the lane that speaks for its group
          for (int r = 0; r < n; ++r) {
            const double u = __shfl_sync(0xffffffffu, d, r);
            if (__shfl_sync(0xffffffffu, eg, r) != eg) continue;
            if (r < lane) first = false;
            if (u > b0) {
              b1 = b0;
              b0 = u;
            } else if (u > b1) {
              b1 = u;
            }
          }
          const double value = a.group_top == 2 && b1 > -CUDART_INF ? b0 + b1 : b0;
          int above = 0;
          for (int r = 0; r < n; ++r) {
            const double u = __shfl_sync(0xffffffffu, value, r);
            const int h = __shfl_sync(0xffffffffu, eg, r);
            if (__shfl_sync(0xffffffffu, first, r)) above += (u > value || (u == value && h < eg)) ? 1 : 0;
          }
          // groups kept for certain, a bit each
          uint32_t kept = __reduce_or_sync(0xffffffffu, keep && !border ? 1u << g : 0u);
          const int room = a.topk_groups - __popc(kept);
          kept |= __reduce_or_sync(0xffffffffu, first && above < room ? 1u << eg : 0u);
          keep = have && ((kept >> g) & 1u);
        }
      }
    }
    if (a.group_lanes > 0) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!keep) key[i] = 0u;
    } else {
      const uint32_t kept = __ballot_sync(0xffffffffu, keep);
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!((kept >> (((static_cast<uint32_t>(e0 + i) * a.gmul) >> 22) & 31u)) & 1u)) key[i] = 0u;
    }
  }

  // k picks; with a bias one more, and on while the last two may be out of order
  int mine = -1, picks = 0;
  float last_lo = 0.f;
  bool near = false;  // some neighbours of the list may be out of order
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
  for (;; ++picks) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0u) break;
    if (a.bias != nullptr) {
      const float now = key_value(top);
      // (after an infinite choice last_lo is NaN, and its order is exact)
      const bool close = picks > 0 && last_lo <= fmaf(kRel, fabsf(now), now + err);
      if (picks >= a.k && !close) break;
      near |= close;
      last_lo = fmaf(-kRel, fabsf(now), now - err);
      if (picks == 32) {  // the list may go on
        whole = true;
        break;
      }
    } else if (picks >= a.k) {
      break;
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    int at = 0;
    if (lane == src) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i)
        if (key[i] == top) at = i;
      best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == at) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
    at = __shfl_sync(0xffffffffu, e0 + at, src);
    if (lane == picks) mine = at;
  }
  if (near && !whole) {
    // Everything outside the list is certainly below all of it: its order in fp64, a lane each.
    if (a.softmax && soft.y == 0.0) soft = softmax_f64<BF16>(a, row, lane);
    const double d = mine >= 0 ? choice_f64<BF16>(a, row, mine, soft) : -CUDART_INF;
    int rank = 0;
    for (int r = 0; r < picks; ++r) {
      const double u = __shfl_sync(0xffffffffu, d, r);
      const int e = __shfl_sync(0xffffffffu, mine, r);
      rank += (u > d || (u == d && e < mine)) ? 1 : 0;
    }
    int ordered = -1;
    for (int r = 0; r < picks; ++r) {
      const int e = __shfl_sync(0xffffffffu, mine, r), at = __shfl_sync(0xffffffffu, rank, r);
      if (at == lane) ordered = e;
    }
    mine = ordered;
  }
  if (whole) {
    __syncwarp();  // the float scratch is read no more
    mine = route_row_f64<VPL, BF16>(a, row, scratch[warp], lane);
  }
  if (lane >= a.k) mine = -1;
  const float s = mine >= 0 ? score32(load_logit<BF16>(a, row, mine), a.softmax, m, inv) : 0.f;
  float w = s;
  if (a.renorm) {
    float sum = s;
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
cudaError_t launch_vpl(RouteArgs a, bool bf16, cudaStream_t stream) {
  const int lanes = a.gsize % VPL == 0 ? a.gsize / VPL : 0;
  a.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
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
  const int64_t es = l.bf16_logits ? 2 : 4;
  a.vec = reinterpret_cast<uintptr_t>(l.logits) % 16 == 0 && l.ldl * es % 16 == 0;
  a.bias_vec = reinterpret_cast<uintptr_t>(l.bias) % 16 == 0;
  a.softmax = l.softmax;
  a.renorm = l.renormalize;
  a.scale = l.scale;
  a.ids = l.ids;
  a.weights = l.weights;
  if (l.E <= 32) return launch_vpl<1>(a, l.bf16_logits, stream);
  if (l.E <= 64) return launch_vpl<2>(a, l.bf16_logits, stream);
  if (l.E <= 128) return launch_vpl<4>(a, l.bf16_logits, stream);
  if (l.E <= 256) return launch_vpl<8>(a, l.bf16_logits, stream);
  if (l.E <= 512) return launch_vpl<16>(a, l.bf16_logits, stream);
  return launch_vpl<32>(a, l.bf16_logits, stream);
}

}  // namespace mxq
