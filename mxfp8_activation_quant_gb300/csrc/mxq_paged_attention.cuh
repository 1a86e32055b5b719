// Attention of one new token per sequence over a paged MXFP8 cache, split over the cache's length and
// joined.
//
// One persistent CTA per SM takes an equal share of all (sequence, cache head, block of query heads)
// items' tokens, in units of 64, in tiles of up to 128 tokens. For a tile:
//   S^T[t, h] = K_t . q_h    tcgen05.mma kind::mxf8f6f4, block-scaled, M = 128 tokens: cache rows go from TMA
//                            straight into the MMA. bf16 has 8 significant bits and E4M3 4, so q = hi + lo, both
//                            MXFP8 (lo's scales 2^-4 of hi's): N = 2 GP columns, added where S is read.
//   P = exp2(S - ref)        ref: a running reference, put 2^7 below the running maximum when it moves (with O and the
//                            sums; only when a score passes it by more than 2^15), so that a tile needs no maximum of its own and
//                            P fits fp16, whose largest is 2^16: the largest P is 2^7 or more, so one 2^-21 of it is still a normal
//                            number, and one of 2^-32 counts (with ref at the maximum, long tails of 2^-25 were lost from O, not
//                            from the sums)
//   O^T[d, h] += V^T P^T     kind::f16, M = 128 features a panel: ldmatrix transposes the E4M3 bytes, registers make
//                            them fp16 with their scales relative to the segment's pivot 2^E, and they
//                            are stored to TMEM as the A operand. (Dequantized rows in shared memory would
//                            cost 128 KB written and read a tile of 512 features, which alone takes
//                            2048 of the 2800 cycles in which HBM delivers the tile.)
// fp16 holds code * 2^(b - E) exactly for b in [E - 14, E + 7] (the factor is an fp16 of its own, and normal): a tile with a scale above
// raises E (O is rescaled with ref), one with a nonzero scale byte below takes P and V as bf16. Byte 0 does not ask for that: all-zero
// groups and tokens that take no part have it. Its factor is 0 once E passes 14, so what values it has, of at most 448 * 2^-127, then
// count as zeros.
//
// Warps: 0 the rows' loads, 1 and 2 MMAs (scores, outputs), 3 scales, 4-11 softmax (two a TMEM lane quarter, half of the
// heads each), 12-19 V^T (two a quarter; every second panel each) and the outputs (half of the heads each). Of few heads
// the softmax takes four warps; warp 8 then copies the scales and warp 9 loads the values' rows.
//
// A CTA that holds an item from start to end writes its outputs; the others' normalised parts go to the
// workspace (at most two a CTA), and join_kernel adds them up in the order of the CTAs.
//
// Measured, the whole call (captured, GB300) and the algorithmic bytes' rate:
//   128 sequences of 1024-4096 tokens, 8 cache heads x 8 query heads of 128: 132 us, 5300 GB/s (a copy: 6770). Bound by HBM;
//     a tile of 128 tokens takes 0.94 us, of which its bytes need 0.74. With 16 query heads a cache head 145 us, with 32 175: there the
//     softmax is as long as the rows.
//   64 sequences of 2048-8192 tokens, latent, 64 heads of 512: 79 us, 2300 GB/s; 1 sequence of 131072: 43 us. Bound by the
//     instructions: 3000 a scheduler and tile (softmax, conversion of V; issue slots 46 % busy), the waits of the chain TMA ->
//     scores -> softmax -> outputs between them, and their fetching: the roles' loops miss the instruction cache in one of
//     ten requests. Tensor cores 31 % busy. About 18 us are the queries, the first tile and the join.
// A kernel of fp32 FMAs over the same items, the first that was right, took 10900 and 30000 us.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_kv_internal.h"
#include "mxq_rings.h"
#include "mxq_tma.h"

namespace mxq {
namespace paged {

constexpr int kUnit = 64;         // tokens of the unit of work; a TMA box has no more
constexpr int kTile = 128;        // tokens of a tile
constexpr int kThreads = 640;     // (five warps a scheduler leave each thread 96 registers; a sixth anywhere, 80)
constexpr int kPanel = 128 * 128;  // bytes of 128 features of a tile
constexpr int kMaxHeads = 64;     // query heads of an item
constexpr float kLowRef = -3.4028235e38f;  // ref before the first token: the lowest finite number, so that every score is above
constexpr float kLead = 7.0f, kSlack = 15.0f;  // of the largest score over ref, in binary orders: where ref is put, and before it moves
constexpr int32_t kNoScore = static_cast<int32_t>(0x807FFFFFu);  // ordered(-infinity)

// TMEM columns for GP heads: O from 0, S (one buffer of 64 heads, two of fewer, and as many of K's scales, so that a tile's are
// not overwritten before its products are done), the queries' scales, and V^T in slots of 64 tokens x 128 features.
// Of 64 heads the products with lo are added to those with hi in the tensor core (twice the MMAs of half the width, and five slots
// for V^T instead of three: 64 latent sequences of 16384 x 256, 91.7 -> 84.0 us; of 512 features the same); their scales are rows 64 and on of the
// queries', two columns further. Fewer heads' would start on an odd column or within one, where no MMA may read scales.
template <int GP>
struct Columns {
  static constexpr int kBuffers = GP == 64 ? 1 : 2;
  static constexpr bool kAdd = GP == 64;
  static constexpr int kSWidth = kAdd ? GP : 2 * GP;
  static constexpr uint32_t kS = GP == 64 ? 256 : GP == 32 ? 128 : 64, kSfK = kS + (GP < 16 ? 64 : kBuffers * kSWidth),
                            kSfQ = kSfK + 16 * kBuffers, kV = (kSfQ + 16 + 31) / 32 * 32;
  static constexpr int kSlots = (512 - kV) / 32 < 8 ? (512 - kV) / 32 : 8;
  // A set of warps that is about to fill chunk c has filled one of c - 3 .. c - 1, so chunk c - 3 - kSlots is used up; its wait for
  // chunk c - kSlots tells a phase from the next only if c - 2 kSlots is too.
  static_assert(kSlots >= 3);
};
constexpr int kMaxVSlots = 8;

struct Args {
  const uint16_t* q;
  int64_t ldq, ldqh;
  const uint8_t* k_sf;
  const uint8_t* v_sf;  // null: the keys'
  uint32_t k_sf_page, k_sf_token, k_sf_head, v_sf_page, v_sf_token, v_sf_head;  // (below 2^31)
  const int32_t* table;
  int64_t ld_table;
  uint32_t table_width, page_size, pages;
  uint32_t page_mul, page_shift;  // t / page_size = umulhi(t, page_mul) >> page_shift for t < 2^30
  const int32_t* lens;
  int32_t B, H, kv, G, D, panels;
  int32_t blocks, block_heads;  // blocks of query heads per cache head, and their size
  int32_t box, box_shift;       // tokens of a TMA box, a power of two
  int32_t sf_vec;               // bytes of a copy of scales
  float scale;
  uint8_t* q_ws; // [items][panels][2 GP x 128] swizzled, [panels][512] scale atoms
  float* part;   // [2 * CTAs][GP][D]
  float2* stat;  // [2 * CTAs][GP]: ref, sum
  int2* owner;   // [CTAs]: 1 + the item whose first part is the CTA's last segment (0: none), the CTA of its last part
  uint16_t* o;
  uint8_t* oq;
  uint8_t* sf_rm;
  uint8_t* sf_pk;
  uint8_t* sf_tl;
  float* lse;
  int32_t* status;
  int32_t ctas;
};

constexpr int kMaxSfBufs = 6;
// Shared memory besides the buffers.
struct Misc {
  uint64_t ring_full[16], ring_empty[16], sf_raw[kMaxSfBufs], sf_full[kMaxSfBufs], sf_empty[kMaxSfBufs], s_full[2], s_empty[2],
      p_full[2], p_empty[2], v_full[kMaxVSlots], v_empty[kMaxVSlots], q_full, q_empty, o_full, o_empty, fin_full[2],
      fin_empty[2], done;
  alignas(16) float ref[kMaxHeads];
  alignas(16) float fac[kMaxHeads];
  int32_t red[kMaxHeads];
  int32_t sums[kThreads / 32];
  int32_t p_wide[2];  // whether the probabilities are bf16
  int32_t w0, w1, per_cta, rest;
  int32_t b0, kvh0, blk0, u0;
  // the softmax's own walk over the segments, for each half of the heads: units left, sequence, first unit, length, tiles of the segment
  int32_t left[2], b[2], u[2], len[2], tiles[2];
  uint32_t tmem;
  volatile int32_t dead;
};
// A buffer of scales: K atoms [panels][512], V bytes [panels][128 tokens][4 groups], then this.
constexpr int kWide = 1;  // values in bf16
struct TileInfo {
  uint32_t valid[4];
  int32_t pivot, flags;
  uint32_t there;  // bit l: tokens 4 l .. 4 l + 3 are on a page of the cache
  int32_t pad;
};
// A finished segment's sums and references.
struct Fin {
  float sum[4][kMaxHeads];
  float ref[kMaxHeads];
  int32_t pivot;
  int32_t pad[3];
};
// The kernel for GP heads (padded) and NP panels of 128 features: its buffers in shared memory, panels on 1024-byte
// boundaries (their swizzle), as many of them as there is room for.
constexpr int kSmemLimit = 227 * 1024;
template <int GP, int NP>
struct Sizes {
  static constexpr int kSfBufs = NP == 1 ? 6 : NP == 2 ? 4 : 3, kPBufs = 2;
  static constexpr int kQ = 0, kP = kQ + NP * GP * 256, kQSf = kP + kPBufs * kPanel, kSf = kQSf + NP * 512,
                       kSfBytes = NP * 1024 + static_cast<int>(sizeof(TileInfo)), kFin = kSf + kSfBufs * kSfBytes,
                       kMisc = kFin + 2 * static_cast<int>(sizeof(Fin)), kRing = (kMisc + static_cast<int>(sizeof(Misc)) + 1023) / 1024 * 1024;
  static constexpr int kRoom = (kSmemLimit - kRing) / kPanel, kSlots = kRoom < 16 ? kRoom : 16, kTotal = kRing + kSlots * kPanel;
  static constexpr int kValueSlots = value_ring(kSlots);  // of them, where the values are not the keys
  static_assert(kSlots >= 6 && kSfBufs <= kMaxSfBufs && scale_ring_ok(kSfBufs) && ring_ok(kSlots, Columns<GP>::kSlots) && ring_ok(kValueSlots, Columns<GP>::kSlots));
};

// ---- PTX ----------------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* desc, uint32_t bar, int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          dst),
      "l"(desc), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Two 16 x 16 byte matrices transposed; lanes 0-15 and 16-31 give their rows' addresses. Lane l gets, of each,
// columns l / 4 and 8 + l / 4, rows 4 (l % 4) .. + 3 a register.
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 lanes x 32 columns: lane l holds rows l / 4 and 8 + l / 4 of columns 4 i + l % 4 in r[2 i] and r[2 i + 1].
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem], 16-bit operands.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp32 accumulator, A and B both fp16 or both bf16, B with N contiguous (MN-major).
__device__ __forceinline__ constexpr uint32_t idesc_f16_mn(uint32_t N, bool bf16) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (1u << 16) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two E4M3 bytes (the low or the high half of w) as fp16x2.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t w) {
  float2 f;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(w));
  return f;
}
__device__ __forceinline__ uint32_t f16x2_rn(float first, float second) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(second), "f"(first));
  return r;
}
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// An arrival on `bar` (counted in its number) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// A named barrier among `count` threads that also tells whether any of them said so.
__device__ __forceinline__ bool named_barrier_or(uint32_t id, uint32_t count, bool said) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(id), "r"(count), "r"(said ? 1u : 0u) : "memory");
  return r != 0;
}
// What four E4M3 values leave of four bf16 (two words) times inv, times up, as E4M3.
__device__ __forceinline__ uint32_t rest4(uint32_t x01, uint32_t x23, uint32_t codes, float inv, float up) {
  uint32_t c0, c1;
  e4m3x4_f16(codes, c0, c1);
  const float2 f0 = f16x2_f32(c0), f1 = f16x2_f32(c1);
  return e4m3x2((bf16_lo(x01) * inv - f0.x) * up, (bf16_hi(x01) * inv - f0.y) * up) |
         (e4m3x2((bf16_lo(x23) * inv - f1.x) * up, (bf16_hi(x23) * inv - f1.y) * up) << 16);
}
__device__ __forceinline__ uint32_t fp16_fields(uint32_t bytes, uint32_t down) {
  return (__viaddmax_s16x2(bytes & 0x00FF00FFu, down, 0) << 2) | (__viaddmax_s16x2((bytes >> 8) & 0x00FF00FFu, down, 0) << 10);
}
// Two fp32 at a time.
__device__ __forceinline__ float2 add2(float a0, float a1, float b0, float b1) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b));
  return r;
}
// Bytes of ones where the low four bits are set.
__device__ __forceinline__ uint32_t byte_mask(uint32_t bits) { return (((bits & 15) * 0x00204081u) & 0x01010101u) * 0xFFu; }
// ln of sum * 2^ref
__device__ __forceinline__ float lse_of(float ref, float sum) {
  return sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;  // (NaN stays NaN)
}
// 2^(b - 127) as fp32; byte 255 is NaN.
__device__ __forceinline__ float pow2_byte(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}
// 2^e as fp32, e <= 127 (0 below the smallest subnormal).
__device__ __forceinline__ float pow2_of(int32_t e) {
  return __uint_as_float(e >= -126 ? static_cast<uint32_t>(e + 127) << 23 : e >= -149 ? 0x400000u >> (-127 - e) : 0u);
}
// Floats as integers of the same order (no NaN).
__device__ __forceinline__ int32_t ordered(float f) {
  const int32_t i = __float_as_int(f);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float of_ordered(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// Sums of l[0 .. N) over the warp's lanes: halves of the values change hands at each step, until lane i has that of
// value i / (32 / N) in l[0].
template <int O, int N, int M>
__device__ __forceinline__ void fold_sums(float (&l)[M], int lane) {
  if constexpr (N > 1) {
    const bool up = (lane & O) != 0;
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      const float first = l[j], second = l[j + N / 2];
      l[j] = (up ? second : first) + __shfl_xor_sync(0xffffffffu, up ? first : second, O);
    }
  } else {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], O);
  }
  if constexpr (O > 1) fold_sums<O / 2, (N > 1 ? N / 2 : 1)>(l, lane);
}

__device__ __forceinline__ int64_t wide_mul(uint32_t a, uint32_t b) { return static_cast<int64_t>(static_cast<uint64_t>(a) * b); }
// ---- work -----------------------------------------------------------------------------------
__device__ __forceinline__ int32_t length_of(const Args& a, int32_t len) {
  const int64_t cap = static_cast<int64_t>(a.table_width) * a.page_size;
  return len <= 0 ? 0 : static_cast<int32_t>(cap < len ? cap : len);
}
__device__ __forceinline__ uint32_t page_index(const Args& a, uint32_t t) { return __umulhi(t, a.page_mul) >> a.page_shift; }
// A sequence without tokens is one unit, which writes its zeros.
__device__ __forceinline__ int32_t units_of(int32_t len) { return len <= 0 ? 1 : (len - 1) / kUnit + 1; }

// Walks a CTA's segments: runs of units of one item. An item is (cache head, block of query heads, sequence), in that
// order: CTAs that work at the same time then read the heads of the same tokens, which lie side by side, and
// blocks of heads that share a cache head find it in L2 (128 sequences x 8 heads of 128, tokens before heads: 132 us;
// with the sequences outermost, 150).
struct Segments {
  const Args& a;
  int32_t left, next_len, b, k, blk_, u, len, units;
  // the current segment
  int32_t seg_b, kvh, blk, seg_len, u0, u1, seg_units;

  __device__ __forceinline__ Segments(const Args& args, const Misc& m)
      : a(args), left(m.w1 - m.w0), b(m.b0), k(m.kvh0), blk_(m.blk0), u(m.u0) {
    len = left > 0 ? length_of(a, a.lens[b]) : 0;
    units = units_of(len);
    next_len = left > 0 ? a.lens[b + 1 < a.B ? b + 1 : 0] : 0;
  }
  __device__ __forceinline__ bool next() {
    if (left <= 0) return false;
    if (u == units) {
      u = 0;
      if (++b == a.B) {
        b = 0;
        if (++blk_ == a.blocks) {
          blk_ = 0;
          ++k;
        }
      }
      len = length_of(a, next_len);
      units = units_of(len);
      next_len = a.lens[b + 1 < a.B ? b + 1 : 0];
    }
    seg_b = b;
    kvh = k;
    blk = blk_;
    seg_len = len;
    seg_units = units;
    u0 = u;
    u1 = u + min(units - u, left);
    left -= u1 - u;
    u = u1;
    return true;
  }
  __device__ __forceinline__ int tiles() const { return (u1 - u0 + 1) >> 1; }
  __device__ __forceinline__ int32_t start(int tile) const { return (u0 + 2 * tile) * kUnit; }
  // tokens of a tile (0 only in a sequence without any)
  __device__ __forceinline__ int32_t tokens(int tile) const {
    const int32_t n = min(u1 * kUnit, seg_len) - start(tile);
    return max(0, min(kTile, n));
  }
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == seg_units; }
  __device__ __forceinline__ int head0() const { return kvh * a.G + blk * a.block_heads; }
  __device__ __forceinline__ int heads() const { return min(a.block_heads, a.G - blk * a.block_heads); }
};

// Position in a ring of n barriers: the slot and the parity of its current use.
struct Ring {
  int n, slot = 0;
  uint32_t phase = 0;
  __device__ explicit Ring(int count) : n(count) {}
  __device__ void next() {
    if (++slot == n) slot = 0, phase ^= 1;
  }
};

// A bounded wait: half a million tries, of about two microseconds each; false once one has run out, after which nothing waits any
// more: results are void, and the status word is written at the end. Then
//  - every loop still ends: roles count their tiles from the lengths, not from what a wait guards (the softmax's warps meet at barriers
//    without a limit, so they must all count the same);
//  - no load is announced over one in flight: who has not waited for a panel, a chunk of V^T or the queries hands on and releases nothing
//    any more, but leaves, so that the barriers of the rings keep their meaning
// (both in tests/giveup_sim.cpp). Small on purpose: it is inlined thirty times, and the roles' loops have to fit the instruction cache
// together (with the library's usual wait, which reads a clock, they did not: 93 % hits, and its refills at 64 % of their peak).
constexpr uint32_t kWaitTries = 1u << 19;
__device__ __forceinline__ bool wait_bar(Misc& m, uint32_t bar, uint32_t parity) {
  uint32_t tries = 0;
#pragma unroll 1
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (++tries > kWaitTries || m.dead != 0) {
      m.dead = 1;
      return false;
    }
  }
}

// Whether the phase of that parity is over, without a wait: the loops' next phases are tested while this one's work is issued
// (128 sequences x 8 heads of 128: 130.4 -> 128.4 us; 64 sequences x 64 heads of 512 the same).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r) : "r"(bar), "r"(parity) : "memory");
  return r != 0;
}

// Copies of scales, a tile at a time: four tokens a lane (they lie on one page), as they lie in the cache, to where the
// check puts them in order. (Word by word straight to their places took 32 copies a lane for 512 features, 6000 cycles,
// and the scores waited for them.)
template <int GP, int NP>
struct ScaleCopies {
  using Z = Sizes<GP, NP>;
  const Args& a;
  Misc& m;
  Segments seg;
  Ring sf;
  const uint32_t sf0;
  const int lane;
  int i = 0, tiles = 0;
  uint32_t page = 0;
  const int32_t* row = nullptr;
  const uint8_t *k_base = nullptr, *v_base = nullptr;

  __device__ __forceinline__ ScaleCopies(const Args& args, Misc& misc, uint32_t sf_smem, int l)
      : a(args), m(misc), seg(args, misc), sf(Z::kSfBufs), sf0(sf_smem), lane(l) {}
  __device__ __forceinline__ uint32_t page_of(int tile) const {  // (2^32 - 1: none)
    return tile < tiles && 4 * lane < seg.tokens(tile) ? static_cast<uint32_t>(row[page_index(a, seg.start(tile) + 4 * lane)]) : 0xFFFFFFFFu;
  }
  // Few panels: word by word, K's where the MMA's scale atoms have them and V's to a table of tokens. More: token by
  // token in the widest pieces that every token's start is a multiple of; the check then puts them in order.
  static constexpr bool kInOrder = NP <= 2;
  __device__ __forceinline__ void copy(uint32_t buf, const uint8_t* ks, const uint8_t* vs, uint32_t v_step) const {
    if constexpr (kInOrder) {
      const uint32_t kd = buf + (lane & 7) * 64 + (lane >> 3) * 4, vd = buf + NP * 512 + lane * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          cp_async<4>(kd + p * 512 + 16 * k, ks + wide_mul(k, a.k_sf_token) + 4 * p);
          cp_async<4>(vd + p * 512 + 4 * k, vs + wide_mul(k, v_step) + 4 * p);
        }
      }
    } else {
      const uint32_t kd = buf + lane * 16 * NP, vd = kd + NP * 512;
      if (a.v_sf != nullptr) copy_tokens(kd, ks, a.k_sf_token);  // (as check_scales asks, whatever the addresses: two caches may share scales)
      copy_tokens(vd, vs, v_step);
    }
  }
  __device__ __forceinline__ void copy_tokens(uint32_t dst, const uint8_t* src, uint32_t step) const {
#pragma unroll
    for (int k = 0; k < 4; ++k, dst += 4 * NP, src += step) {
      if (NP == 4 && a.sf_vec == 16) {
        cp_async<16>(dst, src);
      } else {
#pragma unroll
        for (int p = 0; p < NP; ++p) cp_async<4>(dst + 4 * p, src + 4 * p);
      }
    }
  }
  __device__ __forceinline__ bool next(uint8_t* sf_area) {
    if (i == tiles) {
      if (!seg.next()) return false;
      i = 0;
      tiles = seg.tiles();
      row = a.table + seg.seg_b * a.ld_table;
      k_base = a.k_sf + wide_mul(seg.kvh, a.k_sf_head);
      v_base = a.v_sf + wide_mul(seg.kvh, a.v_sf_head);
      page = page_of(0);
    }
    const uint32_t next_page = page_of(i + 1);
    const uint32_t raw = smem_u32(&m.sf_raw[0]) + 8 * sf.slot;
    wait_bar(m, smem_u32(&m.sf_empty[0]) + 8 * sf.slot, sf.phase ^ 1);
    const uint32_t there = __ballot_sync(0xffffffffu, page < a.pages);
    if (page < a.pages) {
      const uint32_t t = seg.start(i) + 4 * lane, at = t - page_index(a, t) * a.page_size;
      const uint8_t* const ks = k_base + wide_mul(page, a.k_sf_page) + wide_mul(at, a.k_sf_token);
      // (tokens of the page behind the sequence's end are copied too, and not used)
      if (a.v_sf == nullptr) copy(sf0 + sf.slot * Z::kSfBytes, ks, ks, a.k_sf_token);
      else copy(sf0 + sf.slot * Z::kSfBytes, ks, v_base + wide_mul(page, a.v_sf_page) + wide_mul(at, a.v_sf_token), a.v_sf_token);
    }
    cp_async_arrive(raw);
    if (lane == 0) {
      reinterpret_cast<TileInfo*>(sf_area + sf.slot * Z::kSfBytes + NP * 1024)->there = there;
      mbar_arrive(raw);
    }
    sf.next();
    ++i;
    page = next_page;
    return true;
  }
};

// q as hi + lo, an item's panels as the kernel's shared memory holds them (rows of 128 bytes, swizzled; hi heads, then
// lo heads; then the scale atoms), so that they come by bulk copies. One block a panel: 8 values a lane, 16 lanes a head.
// In the attention kernel itself this took 5 us an item of 64 x 512, with loads that nothing overlaps.
constexpr int kQThreads = 256;
template <int GP>
__global__ void __launch_bounds__(kQThreads) query_kernel(const __grid_constant__ Args a) {
  pdl_launch_dependents();
  const uint32_t item = blockIdx.x / a.panels, p = blockIdx.x - item * a.panels;
  const uint32_t bk = item / a.blocks, blk = item - bk * a.blocks, b = bk / a.kv, kvh = bk - b * a.kv;
  const int heads = min(a.block_heads, a.G - static_cast<int>(blk) * a.block_heads), head0 = kvh * a.G + blk * a.block_heads;
  const int tid = threadIdx.x, col = (tid & 15) * 8;
  const uint16_t* const q = a.q + b * a.ldq + head0 * a.ldqh + 128 * p + col;
  uint8_t* const out = a.q_ws + static_cast<int64_t>(item) * (a.panels * (GP * 256 + 512));
  uint8_t* const panel = out + p * GP * 256;
  uint8_t* const atom = out + a.panels * GP * 256 + p * 512;
  constexpr int kRows = GP < 16 ? 1 : GP / 16;
  uint4 xs[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int h = (tid >> 4) + 16 * u;
    xs[u] = h < heads ? ld_stream_u4(q + h * a.ldqh) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int h = (tid >> 4) + 16 * u, r = GP + h;
    if (h >= GP) break;  // (whole warps)
    const uint4 x = xs[u];
    uint32_t amax = absmax8(x);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t code = ue8m0_from_bf16_amax(amax), low = code >= 4 ? code - 4 : 0;
    const float inv = ue8m0_inverse(code), up = __uint_as_float((127 + code - low) << 23);
    const uint2 hi = quant8(x, inv);
    const uint2 lo = make_uint2(rest4(x.x, x.y, hi.x, inv, up), rest4(x.z, x.w, hi.y, inv, up));
    const int at = (((col >> 4) ^ (h & 7)) << 4) + (col & 8);  // (GP is a multiple of 8: both rows swizzle alike)
    *reinterpret_cast<uint2*>(panel + h * 128 + at) = hi;
    *reinterpret_cast<uint2*>(panel + r * 128 + at) = lo;
    if ((tid & 3) == 0) {
      atom[(h & 31) * 16 + (h >> 5) * 4 + (col >> 5)] = static_cast<uint8_t>(code);
      atom[(r & 31) * 16 + (r >> 5) * 4 + (col >> 5)] = static_cast<uint8_t>(low);
    }
  }
}

// A tile's scales: V's bytes become 4 max(0, b - pivot + 15) (the exponent field of 2^(b - pivot) in fp16) where fp16
// holds them, else they stay; what takes no part is zero. In order they are where they belong; else both lie token by
// token, and K's words go to the MMA's scale atoms, V's to a table of tokens for each panel. `mine`: which of the lane's
// four tokens take part. Raises the pivot.
template <int NP, bool kInOrder>
__device__ __forceinline__ int32_t check_scales(uint8_t* buf, TileInfo* info, bool shared_kv, int lane, uint32_t mine, int32_t& pivot) {
  uint32_t k[4 * NP], v[4 * NP];  // [token][panel]
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(buf + NP * 512 + (kInOrder ? i * 512 + lane * 16 : (lane * NP + i) * 16));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) v[kInOrder ? t * NP + i : 4 * i + t] = w[t];
  }
  if constexpr (!kInOrder) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint4 x = shared_kv ? make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3])
                                : *reinterpret_cast<const uint4*>(buf + (lane * NP + i) * 16);
      k[4 * i] = x.x, k[4 * i + 1] = x.y, k[4 * i + 2] = x.z, k[4 * i + 3] = x.w;
    }
  }
  if (mine != 15u) {
#pragma unroll
    for (int i = 0; i < 4 * NP; ++i) v[i] = (mine >> (i / NP) & 1) != 0 ? v[i] : 0;
  }
  uint32_t hi = 0, lo = 0xFFFFFFFFu;  // largest byte, smallest nonzero byte - 1
#pragma unroll
  for (int i = 0; i < 4 * NP; ++i) {
    const uint32_t e = v[i] & 0x00FF00FFu, o = (v[i] >> 8) & 0x00FF00FFu;
    hi = __vimax3_u16x2(hi, e, o);
    lo = __viaddmin_u16x2(e, 0xFFFFFFFFu, lo);
    lo = __viaddmin_u16x2(o, 0xFFFFFFFFu, lo);
  }
  int32_t top = static_cast<int32_t>(max(hi & 0xFFFFu, hi >> 16)), least = static_cast<int32_t>(min(lo & 0xFFFFu, lo >> 16)) + 1;
  bool wide = false;
  if (__any_sync(0xffffffffu, mine != 15u || top > pivot + 7 || least < pivot - 14)) {  // seldom
    top = __reduce_max_sync(0xffffffffu, top);
    least = __reduce_min_sync(0xffffffffu, least);  // (65536: no nonzero one)
    if (top > pivot + 7) pivot = top;
    wide = least < pivot - 14;
    // token 32 w + 4 j + i: bit 4 j + i of word w
    uint32_t word = mine << (4 * (lane & 7));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if ((lane & 7) == 0) info->valid[lane >> 3] = word;
  } else if (lane < 4) {
    info->valid[lane] = 0xFFFFFFFFu;
  }
  // (the vote has every lane's loads behind it)
  const uint32_t down = static_cast<uint32_t>((15 - pivot) & 0xFFFF) * 0x10001u;
  uint8_t* const atom = buf + (lane & 7) * 64 + (lane >> 3) * 4;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if constexpr (!kInOrder) {
#pragma unroll
      for (int t = 0; t < 4; ++t) *reinterpret_cast<uint32_t*>(atom + p * 512 + t * 16) = k[t * NP + p];
    }
    uint4 x = make_uint4(v[p], v[NP + p], v[2 * NP + p], v[3 * NP + p]);
    if (!wide) x = make_uint4(fp16_fields(x.x, down), fp16_fields(x.y, down), fp16_fields(x.z, down), fp16_fields(x.w, down));
    *reinterpret_cast<uint4*>(buf + NP * 512 + p * 512 + lane * 16) = x;
  }
  return wide ? kWide : 0;
}

template <int GP, int NP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ Args a) {
  constexpr int GO = GP < 16 ? 16 : GP;   // columns of O a panel: an MMA has 16 at least
  constexpr int HPT = GO / 2;             // heads of an output thread
  // Warps of the softmax, and a thread's heads. With four of them others copy scales and load the values' rows: better where a tile's
  // softmax is short beside its rows. Eight warps, four (us): 64 sequences of 1024-4096 on 4 cache heads, 16 heads of 128 57.4, 49.1, of 512
  // 130.1, 124.9, 32 heads of 128 56.5, 70.7, of 384 106.9, 110.7, of 512 135.1, 135.1; latent of 2048-8192, 16 of 512 60.3, 53.9, 32 of 384
  // 52.8, 55.0, of 512 63.1, 61.6.
  constexpr int SW = GP <= 16 || GP <= 8 * NP ? 4 : 8;
  constexpr int SH = GP * 4 / SW;
  constexpr bool kCopier = SW == 4;       // then another copies the scales
  using Cols = Columns<GP>;
  constexpr int SB = Cols::kBuffers, kVSlots = Cols::kSlots;
  constexpr uint32_t kColS = Cols::kS, kColSfK = Cols::kSfK, kColSfQ = Cols::kSfQ, kColV = Cols::kV;
  extern __shared__ __align__(1024) uint8_t smem[];
  using Z = Sizes<GP, NP>;
  constexpr int sf_bytes = Z::kSfBytes;
  Misc& m = *reinterpret_cast<Misc*>(smem + Z::kMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool shared_kv = a.v_sf == nullptr;
  const int S = a.kv * a.blocks;
  const int ring_v = shared_kv ? Z::kSlots : Z::kValueSlots, ring_k = shared_kv ? Z::kSlots : Z::kSlots - ring_v;
#define BAR(x) smem_u32(&m.x)

  pdl_launch_dependents();
  if (warp == 1) {
    tmem_alloc(smem_u32(&m.tmem), 512);
    tmem_relinquish();
  }
  if (tid == 0) {
#pragma unroll 1
    for (int i = 0; i < Z::kSlots; ++i) {
      mbar_init(BAR(ring_full[i]), 1);
      mbar_init(BAR(ring_empty[i]), shared_kv ? 5 : i < ring_k ? 1 : 4);
    }
#pragma unroll 1
    for (int i = 0; i < kMaxSfBufs; ++i) {
      mbar_init(BAR(sf_raw[i]), 33), mbar_init(BAR(sf_full[i]), 1);
      mbar_init(BAR(sf_empty[i]), 1 + SW + (NP > 1 ? 8 : 4));
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(s_full[i]), 1), mbar_init(BAR(s_empty[i]), SW);
      mbar_init(BAR(p_full[i]), SW), mbar_init(BAR(p_empty[i]), 1);
      mbar_init(BAR(fin_full[i]), SW), mbar_init(BAR(fin_empty[i]), 8);
    }
#pragma unroll 1
    for (int i = 0; i < kVSlots; ++i) mbar_init(BAR(v_full[i]), 4), mbar_init(BAR(v_empty[i]), 1);
    mbar_init(BAR(q_full), 1), mbar_init(BAR(q_empty), 1);
    mbar_init(BAR(o_full), 1), mbar_init(BAR(o_empty), 8);
    mbar_init(BAR(done), 2);
    fence_mbar_init();
    m.dead = 0;
    m.w0 = m.w1 = 0;
    for (int i = 0; i < 2; ++i) m.left[i] = m.b[i] = m.u[i] = m.len[i] = 0;
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (tid < kMaxHeads) m.red[tid] = kNoScore;

  // The CTA's share: a scan of the sequences' units, a run of sequences per thread.
  {
    const int32_t per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int32_t sum = 0;
#pragma unroll 1
    for (int32_t b = b0; b < b1; ++b) sum += units_of(length_of(a, a.lens[b]));
    int32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) m.sums[warp] = inc;
    __syncthreads();
    // (every warp sums the warps' sums, a lane each)
    const int32_t theirs = lane < kThreads / 32 ? m.sums[lane] : 0;
    const int32_t once = __reduce_add_sync(0xffffffffu, theirs), total = once * S;  // the sequences', the items' units
    const int32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? theirs : 0) + inc - sum;
    // (no share is empty among the CTAs that have one: the parts of an item lie in consecutive CTAs)
    const int32_t per_cta = max(1, total / a.ctas), rest = total < a.ctas ? 0 : total - per_cta * a.ctas;
    const int32_t w0 = per_cta * static_cast<int32_t>(blockIdx.x) + min(static_cast<int32_t>(blockIdx.x), rest);
    const int32_t sub = w0 / once;
    int32_t at = w0 - sub * once;
    if (w0 < total && before <= at && at < before + sum) {  // one thread
      at -= before;
      int32_t b = b0, units = units_of(length_of(a, a.lens[b]));
#pragma unroll 1
      while (at >= units) {
        at -= units;
        units = units_of(length_of(a, a.lens[++b]));
      }
      m.b0 = b;
      m.kvh0 = sub / a.blocks;
      m.blk0 = sub - m.kvh0 * a.blocks;
      m.u0 = at;
      m.w0 = w0;
      m.w1 = w0 + per_cta + (static_cast<int32_t>(blockIdx.x) < rest ? 1 : 0);
      m.per_cta = per_cta;
      m.left[0] = m.left[1] = m.w1 - m.w0;
      m.b[0] = m.b[1] = b - 1;
      m.u[0] = m.u[1] = at;
      m.len[0] = m.len[1] = a.lens[b];
      m.rest = rest;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m.tmem;

  if (warp == 0 || (kCopier && warp == 9)) {
    // ---- rows: a panel of a tile per ring slot (with warps to spare, the values' come from one of their own) ----
    if (elect_one()) {
      Segments seg(a, m);
      const int kind0 = warp == 0 ? 0 : 1, kinds = shared_kv ? 1 - kind0 : kCopier ? kind0 + 1 : 2;  // kinds [kind0, kinds)
      Ring ring(kind0 == 0 ? ring_k : ring_v), other(ring_v);
      int used = 0, other_used = 0;
      const bool two = a.box == kUnit;  // two boxes a tile: their pages are looked up a tile ahead
#pragma unroll 1
      while (kind0 < kinds && m.dead == 0 && seg.next()) {
        const int tiles = seg.tiles(), kvh = seg.kvh;
        const int32_t* row = a.table + seg.seg_b * a.ld_table;
        auto page_at = [&](int32_t t, int32_t& place) {  // the page and the place in it of a box
          const uint32_t i = page_index(a, t);
          place = t - static_cast<int32_t>(i * a.page_size);
          return row[i];
        };
        int32_t page0 = 0, page1 = 0, place0 = 0, place1 = 0;
        auto look_up = [&](int tile) {
          const int32_t n = seg.tokens(tile), t = seg.start(tile);
          if (n > 0) page0 = page_at(t, place0);
          if (n > kUnit) page1 = page_at(t + kUnit, place1);
        };
        if (two) look_up(0);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const int32_t t = seg.start(i), boxes = (seg.tokens(i) + a.box - 1) >> a.box_shift, bytes = boxes << a.box_shift << 7;
          const int32_t p0 = page0, p1 = page1, at0 = place0, at1 = place1;
          if (two && i + 1 < tiles) look_up(i + 1);
#pragma unroll 1
          for (int kind = kind0; kind < kinds; ++kind) {
            const CUtensorMap* const map = kind == 0 ? &map_k : &map_v;
            const int slot0 = kind == 0 ? 0 : ring_k;
#pragma unroll 1
            for (int x = 0; x < 128 * NP; x += 128) {
              const int s = slot0 + ring.slot;
              const uint32_t full = BAR(ring_full[0]) + 8 * s;
              uint32_t dst = sbase + Z::kRing + s * kPanel;
              if (!wait_bar(m, BAR(ring_empty[0]) + 8 * s, ring.phase ^ 1)) break;
              mbar_arrive_expect_tx(full, bytes);
              if (two) {
                if (boxes > 0) tma_load_4d(dst, map, full, x, at0, kvh, p0);
                if (boxes > 1) tma_load_4d(dst + kUnit * 128, map, full, x, at1, kvh, p1);
              } else {
#pragma unroll 1
                for (int j = 0; j < boxes; ++j, dst += a.box << 7) {
                  int32_t at;
                  const int32_t page = page_at(t + (j << a.box_shift), at);
                  tma_load_4d(dst, map, full, x, at, kvh, page);
                }
              }
              ring.next();
              ++used;
            }
            if (!kCopier && kinds == 2) {  // (a reference to either ring would live in memory)
              const Ring r = ring;
              const int u = used;
              ring = other, other = r;
              used = other_used, other_used = u;
            }
          }
        }
      }
      // every load in flight lands before the CTA leaves
#pragma unroll 1
      for (int kind = kind0; kind < kinds; ++kind) {
        const int n = kind == 0 ? ring_k : ring_v, u = kind == kind0 ? used : other_used;
#pragma unroll 1
        for (int i = max(0, u - n); i < u; ++i)
          if (!mbar_wait_bounded(BAR(ring_full[(kind == 0 ? 0 : ring_k) + i % n]), (i / n) & 1)) m.dead = 1;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- the scores' MMAs ----
    // (A thread of their own: a wait behind a commit takes the issuing thread about 250 cycles, eight of which a tile's
    // other products need.)
    if (elect_one()) {
      Segments seg(a, m);
      Ring rk(ring_k), sf(Z::kSfBufs), s(SB), q_ring(1);
      bool first = true, ready = false;
#pragma unroll 1
      while (seg.next()) {
        const int tiles = seg.tiles();
        // this item's queries, once the last scores of the one before are done
        if (!wait_bar(m, BAR(q_empty), q_ring.phase ^ 1)) goto scores_over;
        if (first) pdl_wait_primary();
        first = false;
        const uint8_t* const q = a.q_ws + ((static_cast<int64_t>(seg.seg_b) * a.kv + seg.kvh) * a.blocks + seg.blk) * (NP * (GP * 256 + 512));
        mbar_arrive_expect_tx(BAR(q_full), NP * (GP * 256 + 512));
        bulk_load(sbase + Z::kQ, q, NP * GP * 256, BAR(q_full));
        bulk_load(sbase + Z::kQSf, q + NP * GP * 256, NP * 512, BAR(q_full));
        const bool landed = wait_bar(m, BAR(q_full), q_ring.phase);
        q_ring.next();
        if (!landed) goto scores_over;
        tc_fence_after();
#pragma unroll 1
        for (int p = 0; p < NP; ++p) tc_cp_sf_atom(tmem + kColSfQ + 4 * p, sdesc_sf_atom(sbase + Z::kQSf + 512 * p));
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          wait_bar(m, BAR(sf_full[0]) + 8 * sf.slot, sf.phase);
          wait_bar(m, BAR(s_empty[0]) + 8 * s.slot, s.phase ^ 1);
          tc_fence_after();
          const uint32_t sf_at = sbase + Z::kSf + sf.slot * sf_bytes;
          const uint32_t d = tmem + kColS + s.slot * Cols::kSWidth, sfk = tmem + kColSfK + 16 * s.slot;
#pragma unroll 1
          for (int p = 0; p < NP; ++p) {
            if (!ready && !wait_bar(m, BAR(ring_full[0]) + 8 * rk.slot, rk.phase)) goto scores_over;
            tc_fence_after();
            const int slot = rk.slot;
            rk.next();
            ready = mbar_test(BAR(ring_full[0]) + 8 * rk.slot, rk.phase);
            tc_cp_sf_atom(sfk + 4 * p, sdesc_sf_atom(sf_at + 512 * p));
            const uint64_t ad = sdesc_kmajor_sw128(sbase + Z::kRing + slot * kPanel);
            const uint64_t bd = sdesc_kmajor_sw128(sbase + Z::kQ + p * GP * 256);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              tc_mma_mxf8(d, ad + 2 * k, bd + 2 * k, idesc_mxf8(128, Cols::kSWidth, k, k), sfk + 4 * p, tmem + kColSfQ + 4 * p,
                          (p | k) != 0 ? 1u : 0u);
              if constexpr (Cols::kAdd)
                tc_mma_mxf8(d, ad + 2 * k, bd + GP * 8 + 2 * k, idesc_mxf8(128, GP, k, k), sfk + 4 * p, tmem + kColSfQ + 4 * p + 2, 1u);
            }
            tc_commit(BAR(ring_empty[0]) + 8 * slot);
          }
          tc_commit(BAR(s_full[0]) + 8 * s.slot);
          tc_commit(BAR(sf_empty[0]) + 8 * sf.slot);
          if (i + 1 == tiles) tc_commit(BAR(q_empty));
          sf.next();
          s.next();
        }
      }
    scores_over:
      tc_commit(BAR(done));
      if (!first && !mbar_wait_bounded(BAR(q_full), q_ring.phase ^ 1)) m.dead = 1;  // (no copy outlives the CTA)
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- the output's MMAs ----
    if (elect_one()) {
      Segments seg(a, m);
      Ring pr(Z::kPBufs), vr(kVSlots), o_ring(1);
      bool ready = false;
#pragma unroll 1
      while (seg.next()) {
        const int tiles = seg.tiles();
        wait_bar(m, BAR(o_empty), o_ring.phase ^ 1);
        o_ring.next();
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const int both = seg.tokens(i) > 64 ? 1 : 0, chunks = NP << both;
          wait_bar(m, BAR(p_full[0]) + 8 * pr.slot, pr.phase);
          const uint32_t idesc = m.p_wide[pr.slot] != 0 ? idesc_f16_mn(GO, true) : idesc_f16_mn(GO, false);
          const uint64_t p_desc = sdesc(sbase + Z::kP + pr.slot * kPanel, 1024, 1024, 2);
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            const int p = c >> both, h = c & both;
            if (!ready && !wait_bar(m, BAR(v_full[0]) + 8 * vr.slot, vr.phase)) goto outputs_over;
            tc_fence_after();
            const int slot = vr.slot;
            vr.next();
            ready = mbar_test(BAR(v_full[0]) + 8 * vr.slot, vr.phase);
            const uint64_t bd = p_desc + h * 512;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_f16_ts(tmem + p * GO, tmem + kColV + 32 * slot + 8 * k, bd + 128 * k, idesc, (i | h | k) != 0 ? 1u : 0u);
            tc_commit(BAR(v_empty[0]) + 8 * slot);
          }
          tc_commit(BAR(p_empty[0]) + 8 * pr.slot);
          pr.next();
        }
        tc_commit(BAR(o_full));
      }
    outputs_over:
      tc_commit(BAR(done));
      if (!mbar_wait_bounded(BAR(done), 0)) m.dead = 1;
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---- scales: the tokens that take part, the pivot, and whether fp16 holds them; four tokens a lane ----
    Segments seg(a, m);
    Ring sf(Z::kSfBufs);
    ScaleCopies<GP, NP> copies(a, m, sbase + Z::kSf, lane);
    // Without a warp for the copies they run two tiles ahead of the check; with three buffers right before it (a tile's
    // scales would otherwise wait for the tile two before it, and its scores with them).
    int more_copies = kCopier ? 0 : Z::kSfBufs >= 4 ? 3 : 1;
#pragma unroll 1
    while (seg.next()) {
      const int tiles = seg.tiles();
      int32_t pivot = 0;
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        uint8_t* const buf = smem + Z::kSf + sf.slot * sf_bytes;
        TileInfo* const info = reinterpret_cast<TileInfo*>(buf + NP * 1024);
        const int32_t n = seg.tokens(i) - 4 * lane;
        if constexpr (!kCopier) {
#pragma unroll 1
          do copies.next(smem + Z::kSf);
          while (--more_copies > 0);
          more_copies = 1;
        }
        wait_bar(m, BAR(sf_raw[0]) + 8 * sf.slot, sf.phase);
        const bool ok = (info->there >> lane) & 1;
        const uint32_t mine = !ok || n <= 0 ? 0u : n >= 4 ? 15u : (1u << n) - 1;  // these of the lane's tokens take part
        const int32_t flags = check_scales<NP, ScaleCopies<GP, NP>::kInOrder>(buf, info, shared_kv, lane, mine, pivot);
        if (lane == 0) info->pivot = pivot, info->flags = flags;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(sf_full[0]) + 8 * sf.slot);
        sf.next();
      }
    }
    cp_async_wait_all();
  } else if (kCopier && warp == 8) {
    ScaleCopies<GP, NP> copies(a, m, sbase + Z::kSf, lane);
#pragma unroll 1
    while (copies.next(smem + Z::kSf)) {
    }
    cp_async_wait_all();
  } else if (warp < 12) {
    // ---- softmax ----
    const int quarter = warp & 3, h0 = (warp - 4) / 4 * SH, st = tid - 128;
    const int hl = h0 + (st & 127), half_bar = 1 + (warp - 4) / 4;  // the warps of the same heads agree among themselves
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float c = a.scale * 1.4426950408889634f;
    const int t = 32 * quarter + lane;
    // the row of P of this thread's token: tokens 4 j + i of 16 are rows 2 j + i (i < 2) and 6 + 2 j + i
    const int prow = (t & ~15) + ((t >> 2) & 3) * 2 + (t & 1) + ((t & 2) << 2);
    // (where S has as many buffers as P, one position serves both)
    constexpr bool kOneRing = SB == Z::kPBufs;
    Ring sf(Z::kSfBufs), pr(Z::kPBufs), s_own(SB), fin(2);
    Ring& s = kOneRing ? pr : s_own;
    const int half = (warp - 4) / 4;
#pragma unroll 1
    while (warp < 4 + SW) {
      float l[SH];
#pragma unroll
      for (int i = 0; i < SH; ++i) l[i] = 0.f;
      // The segment's tiles, counted by one thread for the warps of the same heads (a walk of each thread's own would cost registers).
      if ((st & 127) == 0) {
        cp_async_wait_all();
        const int32_t left = m.left[half], b = m.b[half] + 1 == a.B ? 0 : m.b[half] + 1;
        const int32_t n = min(units_of(length_of(a, m.len[half])) - m.u[half], left);
        m.left[half] = left - n;
        m.b[half] = b;
        m.u[half] = 0;
        m.tiles[half] = (n + 1) >> 1;
        if (left > n) cp_async<4>(smem_u32(&m.len[half]), a.lens + (b + 1 == a.B ? 0 : b + 1));
      }
      // (the last segment's references were read before this barrier)
      named_barrier(half_bar, 128);
      if ((st & 127) < SH) m.ref[hl] = -kLowRef;
      uint32_t state = static_cast<uint32_t>(m.tiles[half]) << 8;  // tiles left, and the pivot in the low byte: one register
      named_barrier(half_bar, 128);
      if (state == 0) break;
      bool started = false;
      do {
        wait_bar(m, BAR(s_full[0]) + 8 * s.slot, s.phase);
        tc_fence_after();
        const uint32_t sc = t_lane + kColS + s.slot * Cols::kSWidth + h0;
        wait_bar(m, BAR(sf_full[0]) + 8 * sf.slot, sf.phase);
        const TileInfo* const info = reinterpret_cast<const TileInfo*>(smem + Z::kSf + sf.slot * sf_bytes + NP * 1024);
        const bool valid = (info->valid[quarter] >> lane) & 1;
        const int32_t new_pivot = info->pivot;
        const bool wide = (info->flags & kWide) != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(sf_empty[0]) + 8 * sf.slot);
        sf.next();
        // The probabilities with the references so far; where a score passes its reference by too much (a segment's first
        // tile: they all do), or the pivot moves, the references move first, and S is read again.
        float e[SH];
        bool move = !started;
        const bool ready = mbar_test(BAR(p_empty[0]) + 8 * pr.slot, pr.phase ^ 1);
        while (true) {
          if (move) {
#pragma unroll 1
            for (int j = 0; j < SH; j += 8) {
              uint32_t hi[8], lo[8];
              tmem_ld_x8(sc + j, hi);
              if constexpr (!Cols::kAdd) tmem_ld_x8(sc + GP + j, lo);
              tmem_ld_wait();
              int32_t mine = kNoScore;  // lane k: the largest score of head j + k
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float x = Cols::kAdd ? __uint_as_float(hi[k]) : __uint_as_float(hi[k]) + __uint_as_float(lo[k]);
                const int32_t top = __reduce_max_sync(0xffffffffu, valid ? ordered(x * c) : kNoScore);
                mine = lane == k ? top : mine;
              }
              if (lane < 8) atomicMax(&m.red[h0 + j + lane], mine);
            }
            named_barrier(half_bar, 128);
            if ((st & 127) < SH) {
              const float old = -m.ref[hl], now = fmaxf(old, fmaxf(kLowRef, of_ordered(m.red[hl]) - kLead));
              m.ref[hl] = -now;
              m.fac[hl] = ex2(old - now);
              m.red[hl] = kNoScore;
            }
            named_barrier(half_bar, 128);
            if (started) {
#pragma unroll
              for (int j = 0; j < SH; j += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&m.fac[h0 + j]);
                l[j] *= f.x, l[j + 1] *= f.y, l[j + 2] *= f.z, l[j + 3] *= f.w;
              }
              // every product so far is in O, and the next waits for P
              const int prev = pr.slot == 0 ? Z::kPBufs - 1 : pr.slot - 1;
              wait_bar(m, BAR(p_empty[0]) + 8 * prev, pr.slot == 0 ? pr.phase ^ 1 : pr.phase);
              tc_fence_after();
              const int down = static_cast<int>(state & 255) - new_pivot;  // <= 0
              const float pf = down < -126 ? 0.f : __uint_as_float((127 + down) << 23);
#pragma unroll 1
              for (int q = 0; q < NP * (SH / 8); ++q) {
                const int j = q % (SH / 8) * 8;
                const uint32_t col = t_lane + q / (SH / 8) * GO + h0 + j;
                uint32_t r[8];
                tmem_ld_x8(col, r);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * m.fac[h0 + j + k] * pf);
                tmem_st_x8(col, r);
              }
              tmem_st_wait();
            }
            state = (state & ~255u) | (new_pivot & 255);
          }
          constexpr int n = SH < 16 ? 8 : 16;
#pragma unroll
          for (int j = 0; j < SH; j += n) {
            uint32_t hi[n], lo[n];
            if constexpr (n == 8) tmem_ld_x8(sc + j, hi);
            else tmem_ld_x16(sc + j, hi);
            if constexpr (!Cols::kAdd) {
              if constexpr (n == 8) tmem_ld_x8(sc + GP + j, lo);
              else tmem_ld_x16(sc + GP + j, lo);
            }
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < n; k += 4) {
              const float4 r = *reinterpret_cast<const float4*>(&m.ref[h0 + j + k]);  // (minus the references)
              // (scaled as the references were, with a rounding of its own, so that the largest score's difference is 0
              // however large it is)
              float2 x0 = make_float2(__uint_as_float(hi[k]), __uint_as_float(hi[k + 1]));
              float2 x1 = make_float2(__uint_as_float(hi[k + 2]), __uint_as_float(hi[k + 3]));
              if constexpr (!Cols::kAdd) {
                x0 = add2(x0.x, x0.y, __uint_as_float(lo[k]), __uint_as_float(lo[k + 1]));
                x1 = add2(x1.x, x1.y, __uint_as_float(lo[k + 2]), __uint_as_float(lo[k + 3]));
              }
              x0 = mul2(x0, c), x1 = mul2(x1, c);
              const float2 d0 = add2(x0.x, x0.y, r.x, r.y), d1 = add2(x1.x, x1.y, r.z, r.w);
              e[j + k] = d0.x, e[j + k + 1] = d0.y, e[j + k + 2] = d1.x, e[j + k + 3] = d1.y;
            }
          }
          if (!__all_sync(0xffffffffu, valid)) {  // (what takes no part may be NaN)
#pragma unroll
            for (int j = 0; j < SH; ++j) e[j] = valid ? e[j] : -INFINITY;
          }
          float over = -INFINITY;
#pragma unroll
          for (int j = 0; j < SH; j += 2) over = fmaxf(over, fmaxf(e[j], e[j + 1]));
#pragma unroll
          for (int j = 0; j < SH; ++j) e[j] = ex2(e[j]);
          if (move) break;
          move = named_barrier_or(half_bar, 128, over > kSlack || ((state ^ new_pivot) & 255) != 0);
          if (!move) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(s_empty[0]) + 8 * s.slot);
        if constexpr (!kOneRing) s.next();
        if (!ready) wait_bar(m, BAR(p_empty[0]) + 8 * pr.slot, pr.phase ^ 1);
        uint8_t* const row = smem + Z::kP + pr.slot * kPanel + prow * 128;
#pragma unroll
        for (int j = 0; j < SH; j += 8) {
          const float* const f = e + j;
          uint4 v;
          if (wide) v = make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]), bf16x2_rn(f[6], f[7]));
          else v = make_uint4(f16x2_rn(f[0], f[1]), f16x2_rn(f[2], f[3]), f16x2_rn(f[4], f[5]), f16x2_rn(f[6], f[7]));
          *reinterpret_cast<uint4*>(row + ((((h0 + j) >> 3) ^ (prow & 7)) << 4)) = v;
        }
#pragma unroll
        for (int j = 0; j < SH; j += 2) {
          const float2 t2 = add2(l[j], l[j + 1], e[j], e[j + 1]);
          l[j] = t2.x, l[j + 1] = t2.y;
        }
        if (st == 0) m.p_wide[pr.slot] = wide;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(p_full[0]) + 8 * pr.slot);
        pr.next();
        started = true;
      } while ((state -= 256) >= 256);
      // sums over the quarter's tokens
      Fin& f = *reinterpret_cast<Fin*>(smem + Z::kFin + fin.slot * sizeof(Fin));
      wait_bar(m, BAR(fin_empty[fin.slot]), fin.phase ^ 1);
      fold_sums<16, SH>(l, lane);
      constexpr int kShare = 32 / SH;  // lanes that hold the same head
      if (lane % kShare == 0) f.sum[quarter][h0 + lane / kShare] = l[0];
      if (quarter == 0 && lane < SH) f.ref[h0 + lane] = -m.ref[h0 + lane];
      if (st == 0) f.pivot = static_cast<int32_t>(state);
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(fin_full[fin.slot]));
      fin.next();
    }
  } else {
    // ---- V^T and the outputs ----
    const int quarter = warp & 3, set = (warp - 12) / 4, h0 = set * HPT;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    Segments seg(a, m);
    Ring rv(ring_v), sf(Z::kSfBufs), fin(2), o_ring(1);
    const int slot0 = shared_kv ? 0 : ring_k;
    int v_slot = 0, turn = 0;  // of the next panel's first chunk; whose the panel is
    uint32_t v_phase = 0;
    const uint32_t pick = static_cast<uint32_t>(quarter) * 0x1010u | 0x4000u;  // a byte of each word, to bytes 1 and 3 (0 and 2 are masked)
    int2 owner = make_int2(0, 0);
#pragma unroll 1
    while (seg.next()) {
      const int tiles = seg.tiles();
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int halves = seg.tokens(i) > 64 ? 2 : 1;
        if (NP > 1 || turn == set) {
          wait_bar(m, BAR(sf_full[0]) + 8 * sf.slot, sf.phase);
          const uint8_t* const buf = smem + Z::kSf + sf.slot * sf_bytes;
          const TileInfo* const info = reinterpret_cast<const TileInfo*>(buf + NP * 1024);
          const bool wide = (info->flags & kWide) != 0;
          const int32_t pivot = info->pivot;
          // the scale bytes of four tokens a lane; the rows of its 16 tokens
          const uint8_t* const tab0 = buf + NP * 512 + 16 * (lane & 3);
          const uint32_t row_at = sbase + Z::kRing + (lane & 15) * 128 + (((2 * quarter + (lane >> 4)) ^ (lane & 7)) << 4);
#pragma unroll 1
          for (int p = 0; p < NP; ++p) {
            const int s = slot0 + rv.slot;
            int vs = v_slot;
            uint32_t vphase = v_phase;
            rv.next();
            v_slot += halves;
            if (v_slot >= kVSlots) v_slot -= kVSlots, v_phase ^= 1;
            turn ^= 1;
            if (turn == set) continue;  // (it was the other's)
            if (!__all_sync(0xffffffffu, wait_bar(m, BAR(ring_full[0]) + 8 * s, rv.slot == 0 ? rv.phase ^ 1 : rv.phase))) goto values_over;
#pragma unroll 1
            for (int h = 0; h < halves; ++h) {
              const uint32_t rows = row_at + s * kPanel + h * 8192, dst = t_lane + kColV + 32 * vs;
              const uint8_t* const tab = tab0 + p * 512 + h * 256;
              const uint32_t valid0 = info->valid[2 * h], valid1 = info->valid[2 * h + 1];
              if (!wide) {
                uint32_t r[4][4];
                uint4 sw[4];
                const bool tested = mbar_test(BAR(v_empty[0]) + 8 * vs, vphase ^ 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  ldmatrix_b8_trans_x2(rows + k * 2048, r[k]);
                  sw[k] = *reinterpret_cast<const uint4*>(tab + k * 64);
                }
                if ((valid0 & valid1) != 0xFFFFFFFFu) {  // tokens that take no part may be NaN
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t mask = byte_mask((k < 2 ? valid0 : valid1) >> (16 * (k & 1) + 4 * (lane & 3)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[k][j] &= mask;
                  }
                }
                uint32_t w0[16], w1[16];  // features 0-15 and 16-31 of the quarter's 32
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // this quarter's group: each byte to the top of an fp16
                  const uint32_t s01 = __byte_perm(sw[k].x, sw[k].y, pick) & 0xFF00FF00u, s23 = __byte_perm(sw[k].z, sw[k].w, pick) & 0xFF00FF00u;
                  uint32_t lo[4], hi[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    e4m3x4_f16(r[k][j], lo[j], hi[j]);
                    lo[j] = hmul2(lo[j], s01), hi[j] = hmul2(hi[j], s23);
                  }
                  w0[4 * k] = lo[0], w0[4 * k + 1] = lo[1], w0[4 * k + 2] = hi[0], w0[4 * k + 3] = hi[1];
                  w1[4 * k] = lo[2], w1[4 * k + 1] = lo[3], w1[4 * k + 2] = hi[2], w1[4 * k + 3] = hi[3];
                }
                if (!__all_sync(0xffffffffu, tested) && !__all_sync(0xffffffffu, wait_bar(m, BAR(v_empty[0]) + 8 * vs, vphase ^ 1))) goto values_over;
                tc_fence_after();
                tmem_st_16x128b_x8(dst, w0);
                tmem_st_16x128b_x8(dst + (16u << 16), w1);
              } else {  // the scales span more than fp16 holds: bf16
                if (!__all_sync(0xffffffffu, wait_bar(m, BAR(v_empty[0]) + 8 * vs, vphase ^ 1))) goto values_over;
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                  uint32_t r[4];
                  ldmatrix_b8_trans_x2(rows + k * 2048, r);
                  const uint4 sw = *reinterpret_cast<const uint4*>(tab + k * 64);
                  const uint32_t mask = byte_mask((k < 2 ? valid0 : valid1) >> (16 * (k & 1) + 4 * (lane & 3)));
                  const float f0 = pow2_of(((sw.x >> (8 * quarter)) & 0xFF) - pivot), f1 = pow2_of(((sw.y >> (8 * quarter)) & 0xFF) - pivot),
                              f2 = pow2_of(((sw.z >> (8 * quarter)) & 0xFF) - pivot), f3 = pow2_of(((sw.w >> (8 * quarter)) & 0xFF) - pivot);
                  uint32_t lo[4], hi[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    e4m3x4_f16(r[j] & mask, lo[j], hi[j]);
                    const float2 fl = f16x2_f32(lo[j]), fh = f16x2_f32(hi[j]);
                    lo[j] = bf16x2_rn(fl.x * f0, fl.y * f1);
                    hi[j] = bf16x2_rn(fh.x * f2, fh.y * f3);
                  }
                  tmem_st_16x128b_x2(dst + 8 * k, lo[0], lo[1], hi[0], hi[1]);
                  tmem_st_16x128b_x2(dst + (16u << 16) + 8 * k, lo[2], lo[3], hi[2], hi[3]);
                }
              }
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(BAR(v_full[0]) + 8 * vs);
              if (++vs == kVSlots) vs = 0, vphase ^= 1;
            }
            if (lane == 0) mbar_arrive(BAR(ring_empty[0]) + 8 * s);  // (after the warp's last barrier)
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(sf_empty[0]) + 8 * sf.slot);
        } else {
          turn ^= 1;
          rv.next();
          v_slot += halves;
          if (v_slot >= kVSlots) v_slot -= kVSlots, v_phase ^= 1;
        }
        sf.next();
      }
      // outputs: this thread's feature 128 p + 32 quarter + lane of its heads
      wait_bar(m, BAR(fin_full[fin.slot]), fin.phase);
      wait_bar(m, BAR(o_full), o_ring.phase);
      tc_fence_after();
      const Fin& f = *reinterpret_cast<const Fin*>(smem + Z::kFin + fin.slot * sizeof(Fin));
      // lane: the sum of head lane % HPT, its inverse in the values' unit, and its reference
      const int my = h0 + lane % HPT;
      const float sum = f.sum[0][my] + f.sum[1][my] + f.sum[2][my] + f.sum[3][my], ref = f.ref[my];
      const float inv = sum > 0.f ? 1.0f / sum : 0.f, unit = pow2_byte(f.pivot);
      const bool whole = seg.whole();
      const int heads = seg.heads(), head0 = seg.head0();
      const int part = 2 * blockIdx.x + (seg.u0 == 0 ? 1 : 0);
      if (!whole && seg.u0 == 0) {  // the item's first part, and this CTA's last segment
        const int32_t last = m.w1 + seg.seg_units - seg.u1 - 1, more = (m.per_cta + 1) * m.rest;  // the item's last unit
        const int32_t cta = last < more ? last / (m.per_cta + 1) : m.rest + (last - more) / m.per_cta;
        owner = make_int2(1 + (seg.kvh * a.blocks + seg.blk) * a.B + seg.seg_b, cta);
      }
      if (quarter == 0 && lane < HPT && my < heads) {
        if (!whole) a.stat[part * GP + my] = make_float2(ref, sum);
        else if (a.lse != nullptr)
          a.lse[static_cast<int64_t>(seg.seg_b) * a.H + head0 + my] = lse_of(ref, sum);
      }
      const int64_t row = seg.seg_b;
      const int mine = heads - h0;  // of this thread's heads there are so many
      if (!whole) {
        constexpr int CH = HPT < 16 ? 8 : 16;
#pragma unroll 1
        for (int i = 0; i < NP * (HPT / CH); ++i) {
          const int p = i / (HPT / CH), j = i % (HPT / CH) * CH;
          float* out = a.part + (static_cast<int64_t>(part) * GP + h0 + j) * a.D + 128 * p + 32 * quarter + lane;
          uint32_t r[CH];
          if constexpr (CH == 8) tmem_ld_x8(t_lane + p * GO + h0 + j, r);
          else tmem_ld_x16(t_lane + p * GO + h0 + j, r);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < CH; ++k, out += a.D) {
            const float v = __uint_as_float(r[k]) * __shfl_sync(0xffffffffu, inv, j + k) * unit;
            if (j + k < mine) *out = v;
          }
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < NP * (HPT / 8); ++i) {
          const int p = i / (HPT / 8), j = i % (HPT / 8) * 8, n = min(8, mine - j);
          if (n <= 0) continue;
          uint32_t r[8];
          tmem_ld_x8(t_lane + p * GO + h0 + j, r);
          tmem_ld_wait();
          const int64_t at = (row * a.H + head0 + h0 + j) * a.D + 128 * p + 32 * quarter + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k) r[k] = bf16x2_rn(__uint_as_float(r[k]) * __shfl_sync(0xffffffffu, inv, j + k) * unit, 0.f);
          if (a.o != nullptr) {
            uint16_t* out = a.o + at;
#pragma unroll
            for (int k = 0; k < 8; ++k, out += a.D)
              if (k < n) *out = static_cast<uint16_t>(r[k]);
          }
          if (a.oq != nullptr) {
            uint8_t* out = a.oq + at;
            uint32_t byte = 0;  // lane k: the scale byte of head k
#pragma unroll
            for (int k = 0; k < 8; ++k, out += a.D) {
              const uint32_t code = ue8m0_from_bf16_amax(__reduce_max_sync(0xffffffffu, r[k] & 0x7FFFu));
              if (k < n) *out = static_cast<uint8_t>(e4m3x2(bf16_lo(r[k]) * ue8m0_inverse(code), 0.f));
              byte = lane == k ? code : byte;
            }
            if (lane < n) {
              const int64_t word = static_cast<int64_t>(head0 + h0 + j + lane) * NP + p, words = static_cast<int64_t>(a.H) * NP;
              if (a.sf_rm != nullptr) a.sf_rm[(row * words + word) * 4 + quarter] = static_cast<uint8_t>(byte);
              if (a.sf_pk != nullptr) a.sf_pk[(word * ((a.B + 3) / 4 * 4) + row) * 4 + quarter] = static_cast<uint8_t>(byte);
              if (a.sf_tl != nullptr) a.sf_tl[tiled128x4_word_offset(row, word, words) + quarter] = static_cast<uint8_t>(byte);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(o_empty)), mbar_arrive(BAR(fin_empty[fin.slot]));
      o_ring.next();
      fin.next();
    }
  values_over:
    if (tid == 12 * 32) a.owner[blockIdx.x] = owner;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (tid == 0 && m.dead != 0 && a.status != nullptr) atomicCAS(a.status, 0, MXQ_ERR_TIMEOUT);
#undef BAR
}

// ---- host -----------------------------------------------------------------------------------
// Launches `kern` so that it may start before the kernel ahead of it ends.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), unsigned grid, int threads, int bytes, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int GP, int NP>
cudaError_t launch_panels(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, cudaStream_t stream) {
  static PerDevice set;
  const cudaError_t e = allow_smem(set, attention_kernel<GP, NP>, Sizes<GP, NP>::kTotal);
  return e != cudaSuccess ? e : launch_behind(attention_kernel<GP, NP>, a.ctas, kThreads, Sizes<GP, NP>::kTotal, stream, mk, mv, a);
}

// The queries' kernel and the attention for GP padded heads; each GP is compiled by a file of its own.
template <int GP>
cudaError_t launch_heads(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, cudaStream_t stream) {
  query_kernel<GP><<<static_cast<unsigned>(a.B * a.kv * a.blocks * a.panels), kQThreads, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  switch (a.panels) {
    case 1: return launch_panels<GP, 1>(mk, mv, a, stream);
    case 2: return launch_panels<GP, 2>(mk, mv, a, stream);
    case 3: return launch_panels<GP, 3>(mk, mv, a, stream);
    default: return launch_panels<GP, 4>(mk, mv, a, stream);
  }
}
extern template cudaError_t launch_heads<8>(const CUtensorMap&, const CUtensorMap&, const Args&, cudaStream_t);
extern template cudaError_t launch_heads<16>(const CUtensorMap&, const CUtensorMap&, const Args&, cudaStream_t);
extern template cudaError_t launch_heads<32>(const CUtensorMap&, const CUtensorMap&, const Args&, cudaStream_t);
extern template cudaError_t launch_heads<64>(const CUtensorMap&, const CUtensorMap&, const Args&, cudaStream_t);

}  // namespace paged
}  // namespace mxq
