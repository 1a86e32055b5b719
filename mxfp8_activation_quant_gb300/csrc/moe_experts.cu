// The experts' products of a mixture of experts (moe_experts_mxfp8):
//   plan     sorts the (token, slot) pairs by expert and cuts every expert's rows into token tiles
//   rows     gives each pair its row and copies its activation scales to its tile's slot, and with
//            many tokens per expert its activations too (all within plan for few pairs)
//   GEMM 1   (g, u) = W13_e x, a = MXFP8(bf16(silu(g) u)) in the epilogue; a tile's token rows come
//            from the copies, or with few tokens per expert straight from x, four rows per load
//   GEMM 2   y = W2_e a, fp32 per pair: y is a part of the sum over a token's experts
//   combine  out[t] = bf16(sum_j w[t, j] y[pair(t, j)]), fp32 sum in slot order
//
// Both GEMMs are one kernel template on CTA pairs (tcgen05 cta_group::2, kind::mxf8f6f4 block
// scaled), persistent, with the WEIGHTS on the MMA's M side: M = 256 weight rows (128 per CTA) and
// N = the token tile, up to 208 tokens in steps of 16. An expert's token count is ragged and its
// weight rows are not, so the ragged dimension sits where the MMA's size follows it exactly.
// Two accumulators of 208 TMEM columns alternate, so a tile's epilogue runs under the next tile's
// MMAs; the remaining 96 columns hold the scales of 6 stages.
//
// Up to about 208 tokens per expert the GEMMs stream the active experts' weights (33/32 B per
// element) and are HBM bound, beyond that tensor bound.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "mxq_device.cuh"
#include "mxq_internal.h"
#include "mxq_moe_internal.h"
#include "mxq_settle.h"
#include "mxq_tma.h"

namespace mxq {
namespace {

constexpr int kTileTokens = 208;   // most tokens of a tile (MMA N)
constexpr int kSlotRows = 256;     // scale rows reserved per tile: two F8_128x4 row tiles
constexpr int kPlanThreads = 1024;
constexpr int kMaxExperts = 1024;
constexpr int kStatusTimeout = 6;  // MXQ_ERR_TIMEOUT

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// One unit of work of a GEMM: a block of 256 weight rows of an expert against a token tile, rows
// [row0, row0 + n) of the expert-sorted pairs. The tile's scales lie in slot `tile` of the scale
// arrays: [tile][k-block][2 atoms of 128 rows][512 bytes].
struct __align__(16) Item {
  int32_t expert, row0, n, tile;
  int32_t block, tiles, pad[2];  // tiles: of the expert
};

// Where an expert's pairs go, and how many have been placed. (A cache line each: the counters of 64
// experts in 8 lines made 32768 atomics take 9 us longer.)
struct __align__(128) ExpertRows {
  int32_t row0, tile0, step, next;
};

// Whether the token rows are copied in expert order before GEMM 1. Reading them in place costs a gather of
// four rows per load for every block of 256 weight rows, copying them H bytes a pair once. us of the call
// in place / copied at 100, 160 and 400 tokens per expert: 5120 -> 2 x 1024 (64 experts, top 8) 228 / 230,
// 267 / 269, 499 / 463; 7168 -> 2 x 512 (32, top 8) 99 / 103, 140 / 141, 264 / 259; 2048 -> 2 x 768 (32, top 4)
// 46.0 / 44.7, 58.6 / 56.7, 99.5 / 95.2; 1024 -> 2 x 1024 35.9 / 34.0, 43.5 / 41.1, 77 / 72. So the sides cross
// between 60 (narrow rows, many blocks) and 300; what the one number gives away is at most 6 %.
inline bool copies_rows(int64_t P, int32_t E) { return P > static_cast<int64_t>(160) * E; }

struct Layout {  // byte offsets into the workspace
  int64_t max_tiles, blocks1, blocks2;
  int64_t n_items, experts, items1, items2, pair_row, row_token, xp, xsf, hq, hsf, y, total;
  Layout(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I) {
    const int64_t P = T * k;
    blocks1 = ceil_div(2 * I, 256);
    blocks2 = ceil_div(H, 256);
    max_tiles = P / kTileTokens + (E < P ? E : P);
    int64_t o = 0;
    auto take = [&](int64_t bytes) {
      const int64_t at = o;
      o += round_up(bytes, 256);
      return at;
    };
    n_items = take(8);
    experts = take(E * static_cast<int64_t>(sizeof(ExpertRows)));
    items1 = take(max_tiles * blocks1 * static_cast<int64_t>(sizeof(Item)));
    items2 = take(max_tiles * blocks2 * static_cast<int64_t>(sizeof(Item)));
    pair_row = take(P * 4);
    row_token = take(P * 4);
    xp = copies_rows(P, E) ? take(P * H) : o;
    xsf = take(max_tiles * kSlotRows * (H / 32));
    hq = take(P * I);
    hsf = take(max_tiles * kSlotRows * (I / 32));
    y = take(P * H * 4);
    total = o;
  }
};

// ------------------------------------------------------------------------------------------
// plan
// ------------------------------------------------------------------------------------------
struct PlanArgs {
  const int32_t* ids;
  int32_t P, E;
  int32_t blocks1, blocks2;  // weight-row blocks per expert of the two GEMMs
  int32_t* n_items;          // of the two GEMMs
  Item* items1;
  Item* items2;
  ExpertRows* experts;  // null: few pairs, placed here (and their scales copied)
  int32_t* pair_row;    // expert-sorted row of pair p, or -1
  int32_t* row_token;   // token of an expert-sorted row
  int32_t k;
  // activation scales, row-major or F8_128x4, of `words` k-blocks; their slots (256 rows per tile)
  const uint8_t* sf;
  int32_t sf_tiled, words;
  uint8_t* xsf;
};

// Byte offset of (row `slot` of the scale slots, k-block w) in a scale array of `kbs` k-blocks.
__device__ __forceinline__ int64_t slot_word_offset(int64_t slot, int w, int kbs) {
  const int64_t atom = ((slot >> 8) * kbs + w) * 2 + ((slot >> 7) & 1);
  return atom * 512 + (slot & 31) * 16 + ((slot >> 5) & 3) * 4;
}
__device__ __forceinline__ uint32_t sf_word(const uint8_t* sf, bool tiled, int64_t t, int w, int words) {
  return *reinterpret_cast<const uint32_t*>(sf + (tiled ? tiled128x4_word_offset(t, w, words) : (t * words + w) * 4));
}

__device__ __forceinline__ int2 add2(const int2 a, const int2 b) { return make_int2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ int2 shfl_up2(const int2 a, int d) {
  return make_int2(__shfl_up_sync(0xffffffffu, a.x, d), __shfl_up_sync(0xffffffffu, a.y, d));
}

// One block: counts per expert, the experts in falling order of their counts, scans of rows and
// tiles in that order, every pair's row, and the items of both GEMMs.
//
// SM pair p of NP takes items p, p + NP, ...: the pairs work on neighbouring items at any time, a
// few experts whose weights and tokens then stay in L2, and the falling order gives every round
// items of nearly the same cost and ends on the cheapest. (Contiguous shares of equal cost per
// pair balanced as well, but the 76 pairs' operands did not fit in L2 together: GEMM 1 at 4096
// tokens, 64 experts, 5120 -> 2 x 1024, took 588 us.)
//
// A row's place within its expert follows the order of shared-memory atomics; no result depends on
// it (a column of an MMA never meets another).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ int cnt[kMaxExperts], order[kMaxExperts];
  __shared__ int row0[kMaxExperts], tile0[kMaxExperts + 1];  // by rank
  __shared__ int rank_of[kMaxExperts], next[kMaxExperts], step[kMaxExperts];  // by expert
  __shared__ int2 part[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  cnt[tid] = 0;
  next[tid] = 0;
  __syncthreads();
  const bool quads = (reinterpret_cast<uintptr_t>(a.ids) & 15u) == 0;  // ids four at a time
  const int P4 = quads ? a.P / 4 : 0;
#pragma unroll 4
  for (int i = tid; i < P4; i += kPlanThreads) {
    const int4 e = reinterpret_cast<const int4*>(a.ids)[i];
    if (e.x >= 0 && e.x < a.E) atomicAdd(&cnt[e.x], 1);
    if (e.y >= 0 && e.y < a.E) atomicAdd(&cnt[e.y], 1);
    if (e.z >= 0 && e.z < a.E) atomicAdd(&cnt[e.z], 1);
    if (e.w >= 0 && e.w < a.E) atomicAdd(&cnt[e.w], 1);
  }
  for (int p = 4 * P4 + tid; p < a.P; p += kPlanThreads) {
    const int e = a.ids[p];
    if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < a.E) {
    const int mine = cnt[tid];
    int r = 0;
    for (int e = 0; e < a.E; ++e) r += (cnt[e] > mine || (cnt[e] == mine && e < tid)) ? 1 : 0;
    rank_of[tid] = r;
    order[r] = tid;
  }
  __syncthreads();
  const int expert = tid < a.E ? order[tid] : 0;  // thread r: the expert of rank r
  const int c = tid < a.E ? cnt[expert] : 0;
  const int nt = (c + kTileTokens - 1) / kTileTokens;
  const int per = nt > 0 ? ((c + nt - 1) / nt + 15) / 16 * 16 : 16;  // tokens per tile, at most 208
  int2 v = make_int2(c, nt);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int2 u = shfl_up2(v, d);
    if (lane >= d) v = add2(v, u);
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int2 s = part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int2 u = shfl_up2(s, d);
      if (lane >= d) s = add2(s, u);
    }
    part[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v = add2(v, part[warp - 1]);  // inclusive
  row0[tid] = v.x - c;
  tile0[tid + 1] = v.y;
  if (tid == 0) tile0[0] = 0;
  if (tid < a.E) step[expert] = per;
  __syncthreads();
  const int tiles = tile0[a.E];
  if (tid < 2) a.n_items[tid] = tiles * (tid == 0 ? a.blocks1 : a.blocks2);
  // items: an expert's weight-row blocks in turn, each with all of the expert's tiles
  for (int g = 0; g < 2; ++g) {
    const int F = g == 0 ? a.blocks1 : a.blocks2;
    Item* items = g == 0 ? a.items1 : a.items2;
    for (int i = tid; i < tiles * F; i += kPlanThreads) {
      int b = 0, t = a.E;  // the largest rank with F tile0 <= i (it has tiles)
      while (t - b > 1) {
        const int m = (b + t) >> 1;
        if (tile0[m] * F <= i) b = m;
        else t = m;
      }
      const int e = order[b], n_e = tile0[b + 1] - tile0[b], local = i - tile0[b] * F;
      const int block = local / n_e, j = local - block * n_e;
      const int left = cnt[e] - j * step[e];
      items[i] = {e, row0[b] + j * step[e], left < step[e] ? left : step[e], tile0[b] + j, block, n_e, {0, 0}};
    }
  }
  if (a.experts != nullptr) {
    if (tid < a.E) a.experts[expert] = {row0[tid], tile0[tid], per, 0};
    return;
  }
  // few pairs (at most one per thread): their scales too
  __syncthreads();  // cnt has been read: it takes the pairs' slots
  if (tid < a.P) {
    const int e = a.ids[tid];
    int row = -1, slot = -1;
    if (e >= 0 && e < a.E) {
      const int k = rank_of[e], r = atomicAdd(&next[e], 1), i = r / step[e];
      row = row0[k] + r;
      slot = (tile0[k] + i) * kSlotRows + r - i * step[e];
      a.row_token[row] = tid / a.k;
    }
    a.pair_row[tid] = row;
    cnt[tid] = slot;
  }
  __syncthreads();
  for (int i = tid; i < a.P * a.words; i += kPlanThreads) {
    const int p = i / a.words, w = i - p * a.words, slot = cnt[p];
    if (slot >= 0)
      *reinterpret_cast<uint32_t*>(a.xsf + slot_word_offset(slot, w, a.words)) = sf_word(a.sf, a.sf_tiled, p / a.k, w, a.words);
  }
}

// ------------------------------------------------------------------------------------------
// rows: a warp per token, or a block where its activations are copied. Lane j places the token's
// pair j (one atomic on its expert's counter);
// the token's scale words, and its activations if they are copied, are read once and written to
// each of its places.
// ------------------------------------------------------------------------------------------
struct RowsArgs {
  const int32_t* ids;
  int32_t E, k;
  int64_t T;
  ExpertRows* experts;
  int32_t* pair_row;
  int32_t* row_token;
  const uint8_t* sf;
  int32_t sf_tiled, words;
  uint8_t* xsf;
  const uint8_t* x;
  int64_t ldx, H;
  uint8_t* xp;
};
constexpr int kRowsThreads = 128;
// Most scale words that plan copies itself, in one block (one token of 5120 in 8 places has 320). us of the
// call so / with the kernel for rows, 5120 -> 2 x 1024, 2048 -> 2 x 640 and 7168 -> 2 x 512: 320 words
// 34.0 / 35.1, 64 17.8 / 18.9, 448 32.8 / 33.7; about 1500 equal (74.4 / 74.7, 38.0 / 38.1, 59.5 / 59.6); 5120
// 139 / 136, 6144 42.4 / 38.7, 7168 71.1 / 66.7.
constexpr int64_t kScalesInPlan = 2048;

template <bool COPY>
__global__ void __launch_bounds__(kRowsThreads) rows_kernel(const RowsArgs a) {
  constexpr int kTokens = COPY ? 1 : kRowsThreads / 32, kPer = kRowsThreads / kTokens;  // threads per token
  __shared__ int2 places[kTokens][32];  // row and scale slot
  const int lane = threadIdx.x & 31, sub = threadIdx.x / kPer, tid = threadIdx.x % kPer;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + sub;
  pdl_wait_primary();
  pdl_launch_dependents();
  const bool live = t < a.T;
  const int chunks = static_cast<int>(a.H / 16);
  for (int j0 = 0; j0 < a.k; j0 += 32) {
    const int kj = a.k - j0 < 32 ? a.k - j0 : 32;
    uint4 v[3];  // the first chunks, on their way while the places are found
    if (COPY) {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (kPer * i + tid < chunks) v[i] = ld_stream_u4(a.x + t * a.ldx + 16 * (kPer * i + tid));
    }
    if (tid < kj && live) {
      const int64_t p = t * a.k + j0 + lane;
      const int e = a.ids[p];
      int2 at = make_int2(-1, -1);
      if (e >= 0 && e < a.E) {
        const int4 x = *reinterpret_cast<const int4*>(a.experts + e);  // row0, tile0, step
        const int r = atomicAdd(&a.experts[e].next, 1), i = r / x.z;
        at = make_int2(x.x + r, (x.y + i) * kSlotRows + r - i * x.z);
        a.row_token[at.x] = static_cast<int>(t);
      }
      a.pair_row[p] = at.x;
      places[sub][lane] = at;
    }
    __syncthreads();
    if (live) {
      for (int w = tid; w < a.words; w += kPer) {
        const uint32_t u = sf_word(a.sf, a.sf_tiled, t, w, a.words);
        for (int j = 0; j < kj; ++j)
          if (places[sub][j].y >= 0)
            *reinterpret_cast<uint32_t*>(a.xsf + slot_word_offset(places[sub][j].y, w, a.words)) = u;
      }
      if (COPY)
        for (int c0 = 0; c0 < chunks; c0 += 3 * kPer) {
          if (c0 > 0) {
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (c0 + kPer * i + tid < chunks) v[i] = ld_stream_u4(a.x + t * a.ldx + 16 * (c0 + kPer * i + tid));
          }
          for (int j = 0; j < kj; ++j) {
            const int64_t r = places[sub][j].x;
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (c0 + kPer * i + tid < chunks)
                *reinterpret_cast<uint4*>(a.xp + r * a.H + 16 * (c0 + kPer * i + tid)) = v[i];
          }
        }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------
// grouped GEMM
// ------------------------------------------------------------------------------------------
constexpr int kGateUp = 0;        // GEMM 1, token rows from the copies
constexpr int kDown = 1;          // GEMM 2
constexpr int kGateUpInPlace = 2; // GEMM 1, token rows from x
// operand loads, MMA, 8 epilogue warps, scale copies, scale loads; in place: 3 more warps that load
// token rows
template <int MODE>
constexpr int kThreads = MODE == kGateUpInPlace ? 480 : 384;
constexpr int BM = 128;        // weight rows per CTA
constexpr int BK = 128;        // K bytes per stage
constexpr int STAGES = 6;
constexpr int kAccBlocks = 4;  // most 32-token blocks of a tile that one epilogue warp takes
constexpr int kPassTokens = 16;  // token rows of a staging buffer of GEMM 2
constexpr int kNextItems = 2;   // items of GEMM 2 whose weights a pair of GEMM 1 fetches into L2
constexpr int kRowLoaders = 4;  // threads that load token rows (in place)
constexpr int kSfKb = 4;      // k-blocks per scale chunk
constexpr int kSfChunks = 3;  // scale chunks in flight

template <int MODE>
struct GemmCfg {
  static constexpr int A_BYTES = BM * BK;
  static constexpr int B_BYTES = kTileTokens / 2 * BK;  // a CTA holds half of the tile's tokens
  static constexpr int SF_COLS = 12;                    // the CTA's weight rows, two token atoms
  static constexpr int SFA_BYTES = 512 * kSfKb, SFB_BYTES = 1024 * kSfKb;
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_SF = OFF_B + STAGES * B_BYTES;
  // epilogue staging, one row per token: 64 bf16 features of every token of the tile (gate-up), or 128
  // fp32 features of kPassTokens tokens, two buffers in turn for each half of the warps (down)
  static constexpr int EPI_BYTES = MODE == kDown ? 4 * kPassTokens * 512 : kTileTokens * 128;
  static constexpr int OFF_EPI = OFF_SF + kSfChunks * (SFA_BYTES + SFB_BYTES);
  static constexpr int OFF_BAR = OFF_EPI + EPI_BYTES;
  static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 2 * kSfChunks + 5) * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
  static constexpr int LOADERS = MODE == kGateUpInPlace ? kRowLoaders : 1;  // threads that load operands
  static constexpr int TMEM_SF = 2 * kTileTokens;  // first scale column
  static_assert(B_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(TMEM_SF + STAGES * SF_COLS <= 512, "TMEM");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

constexpr int kBoxes = 4;  // token-row boxes of the operand loads: 8, 40, 72 or 104 rows, one load
__device__ __forceinline__ int token_box(int half) { return (half + 23) >> 5; }  // the least of at least `half` rows
__device__ __forceinline__ int token_box_rows(int half) { return 32 * token_box(half) + 8; }
struct GemmMaps {
  CUtensorMap w, sfw;      // weights (128 rows) and their scale atoms
  CUtensorMap x[kBoxes];   // activations (in place: x[0], single rows)
  CUtensorMap sfx;         // a chunk of the tile's scale atoms
  CUtensorMap y16;         // down: fp32 output boxes of 128 features x kPassTokens rows
  CUtensorMap w_next;      // gate-up: the weights of GEMM 2
};

struct GemmArgs {
  const Item* items;
  const int32_t* n_items;
  int32_t kbs;       // 128-wide k-blocks
  int32_t rows;      // weight rows per expert
  const int32_t* row_token;  // gate-up in place
  // gate-up: GEMM 2's items, k-blocks, weight rows per expert and SM pairs
  const Item* next_items;
  const int32_t* next_n;
  int32_t next_kbs, next_rows, next_pairs;
  int32_t early;             // the plan is older than the kernel ahead
  // gate-up: E4M3 activations [pairs, rows / 2] and their scales by tile
  uint8_t* hq;
  uint8_t* hsf;
  // down: fp32 [pairs, rows]
  float* y;
  int32_t* status;
};

__device__ __forceinline__ void report(int32_t* status) {
  if (status != nullptr) atomicCAS(status, 0, kStatusTimeout);
}

// A ring position: slot and phase parity.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// The items of one SM pair: index pair, pair + pairs, ... The next one is loaded an item ahead.
struct Items {
  const Item* items;
  int at, stride, end;
  int4 t, t_next;  // expert, row0, n, tile
  int block, block_next, tiles, tiles_next;
  __device__ __forceinline__ Items(const GemmArgs& a, int pair, int pairs) {
    items = a.items;
    at = pair - pairs;
    stride = pairs;
    end = *a.n_items;
    t_next = make_int4(0, 0, 0, 0);
    block_next = tiles_next = 0;
    load();
    next();
  }
  __device__ __forceinline__ void load() {
    if (at + stride < end) {
      t_next = *reinterpret_cast<const int4*>(items + at + stride);
      const int2 b = *reinterpret_cast<const int2*>(&items[at + stride].block);
      block_next = b.x;
      tiles_next = b.y;
    }
  }
  __device__ __forceinline__ bool more() const { return at < end; }
  __device__ __forceinline__ void next() {
    at += stride;
    t = t_next;
    block = block_next;
    tiles = tiles_next;
    load();
  }
  __device__ __forceinline__ int expert() const { return t.x; }
  __device__ __forceinline__ int row0() const { return t.y; }
  __device__ __forceinline__ int n() const { return t.z; }
  __device__ __forceinline__ int tile() const { return t.w; }
  __device__ __forceinline__ int n16() const { return (t.z + 15) & ~15; }
};

// The token rows of a tile's half, four at a time: thread `part` of kRowLoaders takes quads part,
// part + kRowLoaders, ... Rows past the tile's last token repeat it (their columns are not used).
constexpr int kRowQuads = (kTileTokens / 2 / 4 + kRowLoaders - 1) / kRowLoaders;
__device__ __forceinline__ void load_quads(const GemmArgs& p, const Items& item, uint32_t rank, int part,
                                           int (&tok)[kRowQuads][4]) {
  const int half = item.n16() >> 1, first = half * static_cast<int>(rank), last = item.n() - 1;
#pragma unroll
  for (int i = 0; i < kRowQuads; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = first + 4 * (part + kRowLoaders * i) + j;
      tok[i][j] = p.row_token[item.row0() + (r < last ? r : last)];
    }
}
__device__ __forceinline__ void issue_quads(uint32_t dst, const CUtensorMap* tm, uint32_t bar, int x, int half, int part,
                                            const int (&tok)[kRowQuads][4]) {
#pragma unroll
  for (int i = 0; i < kRowQuads; ++i) {
    const int quad = part + kRowLoaders * i;
    if (4 * quad < half) tma_gather4_pair(dst + 512 * quad, tm, bar, x, tok[i][0], tok[i][1], tok[i][2], tok[i][3]);
  }
}

// silu(g) u. e^-|g| is taken as the square of e1 = e^(-|g| / 2): below zero silu(g) = g e1 e1 / (1 + e^-|g|)
// then stays in range as far as the product with u does (g / (1 + e^-g) is 0 from -88 on).
__device__ __forceinline__ float silu_times(float g, float u) {
  const float e1 = __expf(-0.5f * fabsf(g)), a = g < 0.f ? e1 : 1.f;
  return g * a * __fdividef(1.f, fmaf(e1, e1, 1.f)) * (a * u);
}

template <int MODE>
__global__ void __launch_bounds__(kThreads<MODE>, 1)
    experts_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs p) {
  using C = GemmCfg<MODE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - sraw);
  const uint32_t bar_full = sbase + C::OFF_BAR;
  const uint32_t bar_empty = bar_full + 8 * STAGES;
  const uint32_t bar_sff = bar_empty + 8 * STAGES;     // scale chunk landed
  const uint32_t bar_sfe = bar_sff + 8 * kSfChunks;    // scale chunk copied to TMEM
  const uint32_t bar_accf = bar_sfe + 8 * kSfChunks;  // two accumulators
  const uint32_t bar_acce = bar_accf + 16;
  const uint32_t bar_drain = bar_acce + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  // stages (chunks) that each thread has dealt with when it stops
  int* issued_cnt = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);  // [kRowLoaders]
  int* consumed_cnt = issued_cnt + kRowLoaders;
  int* staged_cnt = consumed_cnt + 1;
  int* sf_issued_cnt = consumed_cnt + 2;
  int* sf_consumed_cnt = consumed_cnt + 3;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const bool elected = elect_one();
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int nk = p.kbs;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.sfw);
    tma_prefetch_desc(&maps.x[0]);
    tma_prefetch_desc(&maps.sfx);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 2);  // operands landed, and scales in TMEM
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int c = 0; c < kSfChunks; ++c) {
      mbar_init(bar_sff + 8 * c, 1);
      mbar_init(bar_sfe + 8 * c, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accf + 8 * b, 1);
      mbar_init(bar_acce + 8 * b, 16);  // the epilogue warps of both CTAs
    }
    mbar_init(bar_drain, 2);  // the MMA thread and the scale-copy thread
    *abort_flag = 0;
    for (int i = 0; i < kRowLoaders + 4; ++i) issued_cnt[i] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before any load or commit can reach them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // A kernel of the call launches its dependents only once its own wait is over, so that they may read
  // what the kernels before it wrote at once. Where the plan is such (GEMM 2; GEMM 1 behind the kernel
  // for rows), the first weights and scales are fetched while the kernel ahead still runs, and only
  // the loads of what that one writes wait (one token: the call 43.9 -> 41.2 us).
  const bool early = MODE == kDown || p.early;
  if (!early) {
    pdl_wait_primary();
    pdl_launch_dependents();
  }
  Items item(p, pair, gridDim.x >> 1);

  if (warp == 0 && elected) {
    // ---------------- operand loads (both CTAs) ----------------
    const uint32_t full0 = mapa_shared(bar_full, 0);  // the even CTA's stage barriers
    int it = 0;
    Ring<STAGES> ring;
    bool first = true;
    // Weights that one tile alone reads leave L2 first and spare what the next kernels want there (one
    // token 40.8 -> 38.5 us, 333 tokens of the small model 46.5 -> 45, 777 tokens 210 -> 207); an
    // expert of several tiles reads them again (4096 tokens 518 -> 540 us with the policy for all).
    const uint64_t first_out = l2_evict_first();
    auto load_weights = [&](uint32_t dst, uint32_t fb, int kb, int w_row) {
      if (item.tiles == 1)
        tma_load_2d_pair_hint(dst, &maps.w, fb, kb * BK, w_row, first_out);
      else
        tma_load_2d_pair(dst, &maps.w, fb, kb * BK, w_row);
    };
    for (; item.more() && !*abort_flag; item.next()) {
      const int half = item.n16() >> 1;
      const uint32_t tx = 2u * static_cast<uint32_t>(C::A_BYTES + (MODE == kGateUpInPlace ? half : token_box_rows(half)) * BK);
      const CUtensorMap* tm_x = &maps.x[MODE == kGateUpInPlace ? 0 : token_box(half)];
      const int w_row = item.expert() * p.rows + item.block * (2 * BM) + BM * static_cast<int>(rank);
      const int x_row = item.row0() + half * static_cast<int>(rank);
      int tok[kRowQuads][4];
      if (MODE == kGateUpInPlace && !first) load_quads(p, item, rank, 0, tok);
      int kb = 0;
      if (first) {  // the ring is empty: stage i takes k-block i
        const int pre = nk < STAGES ? nk : STAGES;
        for (int i = 0; i < pre; ++i) {
          if (leader) mbar_arrive_expect_tx(bar_full + 8 * i, tx);
          load_weights(sbase + i * C::A_BYTES, full0 + 8 * i, i, w_row);
        }
        if (early) {
          pdl_wait_primary();
          pdl_launch_dependents();
        }
        if (MODE == kGateUpInPlace) load_quads(p, item, rank, 0, tok);
        for (; kb < pre; ++kb, ++it, ring.next()) {
          if (MODE == kGateUpInPlace)
            issue_quads(sbase + C::OFF_B + kb * C::B_BYTES, tm_x, full0 + 8 * kb, kb * BK, half, 0, tok);
          else
            tma_load_2d_pair(sbase + C::OFF_B + kb * C::B_BYTES, tm_x, full0 + 8 * kb, kb * BK, x_row);
        }
        first = false;
      }
      for (; kb < nk; ++kb, ++it, ring.next()) {
        const int s = ring.slot;
        if (!mbar_wait_bounded(bar_empty + 8 * s, ring.phase ^ 1)) {
          *abort_flag = 1;
          report(p.status);
          break;
        }
        const uint32_t fb = full0 + 8 * s;
        if (leader) mbar_arrive_expect_tx(bar_full + 8 * s, tx);
        load_weights(sbase + s * C::A_BYTES, fb, kb, w_row);
        if (MODE == kGateUpInPlace)
          issue_quads(sbase + C::OFF_B + s * C::B_BYTES, tm_x, fb, kb * BK, half, 0, tok);
        else
          tma_load_2d_pair(sbase + C::OFF_B + s * C::B_BYTES, tm_x, fb, kb * BK, x_row);
      }
    }
    issued_cnt[0] = it;
    if (MODE != kDown && item.end <= item.stride && !*abort_flag && pair < p.next_pairs) {
      // One round of items: with the last loads on their way HBM idles until GEMM 2 begins, so the weights
      // of this pair's first items there are fetched into L2 (one token 38.8 -> 37.5 us; with more
      // rounds other pairs are still loading, and nothing was gained).
      const int n = *p.next_n;
      for (int j = 0; j < kNextItems; ++j) {
        const int at = pair + j * p.next_pairs;
        if (at >= n) break;
        const int row = p.next_items[at].expert * p.next_rows + p.next_items[at].block * (2 * BM) + BM * static_cast<int>(rank);
        for (int kb = 0; kb < p.next_kbs; ++kb) tma_prefetch_2d(&maps.w_next, kb * BK, row);
      }
    }
    if (first && early) {  // no item: the grid still ends after GEMM 1
      pdl_wait_primary();
      pdl_launch_dependents();
    }
  } else if (MODE == kGateUpInPlace && warp >= 12 && elected) {
    // ---------------- token rows (both CTAs; with warp 0, every fourth quad of rows each) ----------------
    const uint32_t full0 = mapa_shared(bar_full, 0);
    if (early) pdl_wait_primary();
    int it = 0;
    Ring<STAGES> ring;
    for (; item.more() && !*abort_flag; item.next()) {
      const int half = item.n16() >> 1;
      int tok[kRowQuads][4];
      load_quads(p, item, rank, warp - 11, tok);
      for (int kb = 0; kb < nk; ++kb, ++it, ring.next()) {
        const int s = ring.slot;
        if (!mbar_wait_bounded(bar_empty + 8 * s, ring.phase ^ 1)) {
          *abort_flag = 1;
          report(p.status);
          break;
        }
        issue_quads(sbase + C::OFF_B + s * C::B_BYTES, &maps.x[0], full0 + 8 * s, kb * BK, half, warp - 11, tok);
      }
    }
    issued_cnt[warp - 11] = it;
  } else if (warp == 11 && elected) {
    // ---------------- scale loads (both CTAs) ----------------
    // The scales of kSfKb k-blocks at a time, in a ring of their own that runs ahead of the operands
    const uint32_t full0 = mapa_shared(bar_sff, 0);
    int ic = 0;
    Ring<kSfChunks> ring;
    bool first = early;
    for (; item.more() && !*abort_flag; item.next()) {
      const int w_row = item.expert() * p.rows + item.block * (2 * BM) + BM * static_cast<int>(rank);
      const int w_atom = (w_row >> 7) * nk;
      const int x_atom = item.tile() * nk * 2;
      int kb = 0;
      if (first) {
        const int chunks = (nk + kSfKb - 1) / kSfKb, pre = chunks < kSfChunks ? chunks : kSfChunks;
        const uint32_t dst = sbase + C::OFF_SF;
        for (int i = 0; i < pre; ++i) {
          if (leader) mbar_arrive_expect_tx(bar_sff + 8 * i, 2u * (C::SFA_BYTES + C::SFB_BYTES));
          tma_load_2d_pair(dst + i * (C::SFA_BYTES + C::SFB_BYTES), &maps.sfw, full0 + 8 * i, 0, w_atom + i * kSfKb);
        }
        pdl_wait_primary();
        for (; ic < pre; kb += kSfKb, ++ic, ring.next())
          tma_load_2d_pair(dst + ic * (C::SFA_BYTES + C::SFB_BYTES) + C::SFA_BYTES, &maps.sfx, full0 + 8 * ic, 0,
                           x_atom + 2 * kb);
        first = false;
      }
      for (; kb < nk; kb += kSfKb, ++ic, ring.next()) {
        const int c = ring.slot;
        if (!mbar_wait_bounded(bar_sfe + 8 * c, ring.phase ^ 1)) {
          *abort_flag = 1;
          report(p.status);
          break;
        }
        if (leader) mbar_arrive_expect_tx(bar_sff + 8 * c, 2u * (C::SFA_BYTES + C::SFB_BYTES));
        const uint32_t dst = sbase + C::OFF_SF + c * (C::SFA_BYTES + C::SFB_BYTES);
        // (k-blocks past the last read the following atoms, or zeros past the arrays' ends)
        tma_load_2d_pair(dst, &maps.sfw, full0 + 8 * c, 0, w_atom + kb);
        tma_load_2d_pair(dst + C::SFA_BYTES, &maps.sfx, full0 + 8 * c, 0, x_atom + 2 * kb);
      }
    }
    *sf_issued_cnt = ic;
  } else if (warp == 1 && elected) {
    // ---------------- MMA issuer (even CTA) ----------------
    if (leader) {
      int it = 0, ti = 0;
      Ring<STAGES> ring;
      for (; item.more() && !*abort_flag; item.next(), ++ti) {
        const int b = ti & 1;
        if (!mbar_wait_bounded(bar_acce + 8 * b, ((ti >> 1) & 1) ^ 1)) {
          *abort_flag = 1;
          report(p.status);
          break;
        }
        tc_fence_after();
        const uint32_t n16 = static_cast<uint32_t>(item.n16());
        bool ok = true;
        for (int kb = 0; kb < nk; ++kb, ++it, ring.next()) {
          const int s = ring.slot;
          if (!mbar_wait_bounded(bar_full + 8 * s, ring.phase)) {
            *abort_flag = 1;
            report(p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sfa_t = tmem + C::TMEM_SF + s * C::SF_COLS;
          const uint64_t ad = sdesc_kmajor_sw128(sbase + s * C::A_BYTES);
          const uint64_t bd = sdesc_kmajor_sw128(sbase + C::OFF_B + s * C::B_BYTES);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            tc_mma_mxf8_pair(tmem + kTileTokens * b, ad + 2 * k, bd + 2 * k, idesc_mxf8(2 * BM, n16, k, k), sfa_t,
                             sfa_t + 4, (kb | k) != 0 ? 1u : 0u);
          tc_commit_pair(bar_empty + 8 * s, 0x3);
        }
        tc_commit_pair(bar_accf + 8 * b, 0x3);
        if (!ok) break;
      }
      *consumed_cnt = it;
    }
  } else if (warp == 10) {
    // ---------------- scale copies (even CTA) ----------------
    // A stage's scale columns are free with the stage; its scales have landed long before its
    // operands, so the copies run under the operands' loads. They count on the stage's own barrier,
    // which spares the MMA thread a second wait of 65 cycles for each of its 352 (176 tokens).
    if (leader && elected) {
      int ic = 0, staged = 0;
      Ring<STAGES> ring;
      Ring<kSfChunks> chunk;
      bool ok = true;
      for (; item.more() && ok && !*abort_flag; item.next()) {
        const bool two = item.n16() > 128;
        // two k-blocks at a time: a wait behind a commit takes this thread 250 cycles
        for (int kb = 0; kb < nk && ok; kb += 2) {
          const int cnt = nk - kb < 2 ? 1 : 2;
          Ring<STAGES> last = ring;
          if (cnt == 2) last.next();  // (its slot is freed after the one before)
          if ((kb % kSfKb == 0 && !mbar_wait_bounded(bar_sff + 8 * chunk.slot, chunk.phase)) ||
              !mbar_wait_bounded(bar_empty + 8 * last.slot, last.phase ^ 1)) {
            *abort_flag = 1;
            report(p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t src = sbase + C::OFF_SF + chunk.slot * (C::SFA_BYTES + C::SFB_BYTES);
#pragma unroll
          for (int g = 0; g < 2; ++g)
            if (g < cnt) {
              const int j = kb % kSfKb + g;
              const uint32_t dst = tmem + C::TMEM_SF + ring.slot * C::SF_COLS;
              tc_cp_sf_atom_pair(dst, sdesc_sf_atom(src + 512 * j));
              tc_cp_sf_atom_pair(dst + 4, sdesc_sf_atom(src + C::SFA_BYTES + 1024 * j));
              if (two) tc_cp_sf_atom_pair(dst + 8, sdesc_sf_atom(src + C::SFA_BYTES + 1024 * j + 512));
              tc_commit_pair(bar_full + 8 * ring.slot, 0x1);
              ++staged;
              ring.next();
            }
          if (kb % kSfKb + 2 == kSfKb || kb + 2 >= nk) {
            tc_commit_pair(bar_sfe + 8 * chunk.slot, 0x3);
            ++ic;
            chunk.next();
          }
        }
      }
      *staged_cnt = staged;
      *sf_consumed_cnt = ic;
    }
  } else if (warp >= 2 && warp < 10) {
    // ---------------- epilogue (both CTAs) ----------------
    // TMEM lane = weight row, column = token. The warps turn the tile through shared memory (one
    // row per token). Warp q = warp % 4 owns TMEM lanes 32 q .. 32 q + 31; of the tile's 32-token
    // blocks, warps 2..5 take the even ones and 6..9 the odd ones. Every warp runs every item's
    // barriers, also after an abort.
    const int q = warp & 3, odd = (warp - 2) >> 2, et = static_cast<int>(threadIdx.x) - 64;
    const uint32_t acce0 = mapa_shared(bar_acce, 0);
    const uint32_t stage = sbase + C::OFF_EPI;
    int ti = 0, pass = 0;
    for (; item.more(); item.next(), ++ti) {
      const int b = ti & 1, n = item.n();
      bool ok = !*abort_flag;
      if (ok && !mbar_wait_bounded(bar_accf + 8 * b, (ti >> 1) & 1)) {
        *abort_flag = 1;
        report(p.status);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      // Several loads of columns in flight before one wait: a tcgen05.ld behind running MMAs takes
      // long. (32-token blocks odd, odd + 2, ... of the tile; columns past n are not used.)
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * q) << 16) + kTileTokens * b + 32 * odd;
      auto release = [&] {  // the MMAs may overwrite this accumulator now
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(bar_acce + 8 * b);
          else
            mbar_arrive_remote_relaxed(acce0 + 8 * b);
        }
      };
      if constexpr (MODE != kDown) {
        if (ok) {
          tc_fence_after();
          // rows alternate gate, up: lane pairs (2 i, 2 i + 1) hold feature 16 q + i. Of two tokens
          // the even lane finishes the first and the odd lane the second.
          const int up = lane & 1, f = 16 * q + (lane >> 1);
#pragma unroll
          for (int h2 = 0; h2 < kAccBlocks / 2; ++h2) {
            uint32_t acc[2][32];
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (64 * (2 * h2 + i) + 32 * odd < n) tmem_ld_x32(t_lane + 64 * (2 * h2 + i), acc[i]);
            tmem_ld_wait();
            if (h2 == kAccBlocks / 2 - 1) release();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t0 = 64 * (2 * h2 + i) + 32 * odd;
              if (t0 >= n) break;
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float a0 = __uint_as_float(acc[i][2 * c]), a1 = __uint_as_float(acc[i][2 * c + 1]);
                const float o = __shfl_xor_sync(0xffffffffu, up ? a0 : a1, 1);
                const float g = up ? o : a0, u = up ? a1 : o;
                const float h = silu_times(g, u);
                const int tok = t0 + 2 * c + up;
                // 16-byte pieces of a 128-byte row are XOR-swizzled by the row
                const uint32_t at = stage + tok * 128 + (((f >> 3) ^ (2 * (tok & 3))) << 4) + (f & 7) * 2;
                if (tok < kTileTokens)
                  asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(bf16x2_rn(h, 0.f)))
                               : "memory");
              }
            }
          }
        }
        named_barrier(1, 256);
        if (ok) {
          // one thread = one token and one 32-feature group: the rule of mxfp8_quantize
          const int64_t ld = p.rows / 2;
          const int f0 = item.block * 128 + static_cast<int>(rank) * 64;
          for (int i = et; i < 2 * n; i += 256) {
            const int tok = i >> 1, g = i & 1;
            uint4 v[4];
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = ld_smem_v4(stage + tok * 128 + (((4 * g + j) ^ (2 * (tok & 3))) << 4));
              amax = max(amax, absmax8(v[j]));
            }
            const uint32_t code = ue8m0_from_bf16_amax(amax);
            const float s = ue8m0_inverse(code);
            const uint2 q0 = quant8(v[0], s), q1 = quant8(v[1], s), q2 = quant8(v[2], s), q3 = quant8(v[3], s);
            const int f = f0 + 32 * g;
            uint4* dst = reinterpret_cast<uint4*>(p.hq + (item.row0() + tok) * ld + f);
            dst[0] = make_uint4(q0.x, q0.y, q1.x, q1.y);
            dst[1] = make_uint4(q2.x, q2.y, q3.x, q3.y);
            p.hsf[slot_word_offset(static_cast<int64_t>(item.tile()) * kSlotRows + tok, f >> 7, static_cast<int>(ld >> 7)) +
                  ((f >> 5) & 3)] = static_cast<uint8_t>(code);
          }
        }
        named_barrier(1, 256);
      } else {
        uint32_t acc[kAccBlocks][32];
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kAccBlocks; ++i)
            if (64 * i + 32 * odd < n) tmem_ld_x32(t_lane + 64 * i, acc[i]);
          tmem_ld_wait();
          release();
        }
        const int f0 = item.block * (2 * BM) + static_cast<int>(rank) * BM;
        const bool live = ok && f0 < p.rows;  // the last block of an odd number of 128-row tiles has one half
        const bool issuer = (et & 127) == 0;
        const uint32_t group = stage + static_cast<uint32_t>(odd) * (2 * kPassTokens * 512);
        // A half of the warps passes kPassTokens tokens at a time through its two buffers, which leave by
        // TMA; the last tokens of a tile go from the registers, 128 bytes of a token a store. A buffer is
        // written again two passes later; its rows have been read out before the barrier between. (4096
        // tokens: GEMM 2 179 us, and 204 us with all rows from the registers.)
#pragma unroll
        for (int i = 0; i < 2 * kAccBlocks; ++i) {
          const int t0 = 64 * (i >> 1) + 32 * odd + kPassTokens * (i & 1), tn = n - t0;
          const uint32_t* v = acc[i >> 1] + kPassTokens * (i & 1);
          if (tn >= kPassTokens) {
            const uint32_t buf = group + static_cast<uint32_t>(pass) * (kPassTokens * 512);
            if (live) {
              const uint32_t at = buf + (32 * q + lane) * 4;
#pragma unroll
              for (int c = 0; c < kPassTokens; ++c) st_smem_u32(at + 512 * c, v[c]);
              fence_proxy_async_smem();
            }
            if (issuer) bulk_wait_read();  // this thread's copy out of the other buffer
            named_barrier(1 + odd, 128);
            if (issuer && live) {
              tma_store_2d(&maps.y16, buf, f0, item.row0() + t0);
              bulk_commit();
            }
            pass ^= 1;
          } else if (tn > 0 && live) {
            float* dst = p.y + static_cast<int64_t>(item.row0() + t0) * p.rows + f0 + 32 * q + lane;
#pragma unroll
            for (int c = 0; c < kPassTokens; ++c)
              if (c < tn) dst[static_cast<int64_t>(c) * p.rows] = __uint_as_float(v[c]);
          }
        }
      }
    }
    if (MODE == kDown) bulk_wait_all();  // the copies have left shared memory and are written
  }
  __syncwarp();

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs have left their loops: issue counts and abort flags are final
  if (leader && warp == 0 && lane == 0) {
    const int peer_abort = ld_dsmem_s32(mapa_shared(smem_u32(const_cast<int*>(abort_flag)), 1));
    if (*abort_flag || peer_abort) {
      // Some loads of either CTA may be in flight for stages that the MMA thread (chunks that the
      // scale copies) did not take. The loaders stop at different stages: the barriers are brought
      // to wait for what was issued, and then waited for (bounded).
      auto settle = [](uint32_t bar, uint32_t phase, Owed o) {
        if (o.bytes > 0) mbar_expect_tx(bar, static_cast<uint32_t>(o.bytes));
        if (o.bytes < 0) mbar_complete_tx(bar, static_cast<uint32_t>(-o.bytes));
        for (int i = 0; i < o.arrivals; ++i) mbar_arrive(bar);
        (void)mbar_wait_bounded(bar, phase);
      };
      int count[2][C::LOADERS], hi = 0;
      for (int l = 0; l < C::LOADERS; ++l) {
        count[0][l] = issued_cnt[l];
        count[1][l] = ld_dsmem_s32(mapa_shared(smem_u32(issued_cnt + l), 1));
        hi = max(hi, max(count[0][l], count[1][l]));
      }
      for (int i = *consumed_cnt; i < hi; ++i) {  // (at most STAGES: the ring lets none further ahead)
        const int half = ((p.items[pair + i / nk * static_cast<int>(gridDim.x >> 1)].n + 15) & ~15) >> 1;
        const int rows = MODE == kGateUpInPlace ? half : token_box_rows(half);
        settle(bar_full + 8 * (i % STAGES), (i / STAGES) & 1, owed_operands(i, count, *staged_cnt, C::A_BYTES, rows * BK));
      }
      const int sf0 = *sf_issued_cnt, sf1 = ld_dsmem_s32(mapa_shared(smem_u32(sf_issued_cnt), 1));
      for (int i = *sf_consumed_cnt; i < max(sf0, sf1); ++i)
        settle(bar_sff + 8 * (i % kSfChunks), (i / kSfChunks) & 1, owed_scales(i, sf0, sf1, C::SFA_BYTES + C::SFB_BYTES));
      *abort_flag = 1;
    }
  }
  __syncthreads();
  if (leader && (warp == 1 || warp == 10) && elected && *abort_flag) {
    tc_commit_pair(bar_drain, 0x1);  // arrives once every MMA / copy this thread issued has completed
    if (warp == 1) (void)mbar_wait_bounded(bar_drain, 0);
  }
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs and copies are over before either CTA frees TMEM or leaves
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------------
// combine: out[t] = bf16(sum_j w[t, j] y[row(t, j)]), 4 columns per thread
// ------------------------------------------------------------------------------------------
struct CombineArgs {
  const float* y;
  const float* weights;
  const int32_t* pair_row;
  int32_t k;
  int64_t H, ldo;
  uint16_t* out;
};
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineArgs a) {
  // (the rows and weights are known before GEMM 2 ends: see there)
  __shared__ int rows[64];
  __shared__ float ws[64];
  const int64_t t = blockIdx.x;
  for (int j = threadIdx.x; j < a.k; j += kCombineThreads) {
    rows[j] = a.pair_row[t * a.k + j];
    ws[j] = a.weights[t * a.k + j];
  }
  __syncthreads();
  pdl_wait_primary();
  const int64_t c = 4 * (static_cast<int64_t>(blockIdx.y) * kCombineThreads + threadIdx.x);
  if (c >= a.H) return;
  float s[4] = {};
  for (int j0 = 0; j0 < a.k; j0 += 4) {  // four rows in flight
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = j0 + j < a.k ? rows[j0 + j] : -1;
      v[j] = r >= 0 ? ld_stream_u4(a.y + r * a.H + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j0 + j >= a.k || rows[j0 + j] < 0) continue;  // (the weight of an empty slot may be anything)
      const float w = ws[j0 + j];
      s[0] = fmaf(w, __uint_as_float(v[j].x), s[0]);
      s[1] = fmaf(w, __uint_as_float(v[j].y), s[1]);
      s[2] = fmaf(w, __uint_as_float(v[j].z), s[2]);
      s[3] = fmaf(w, __uint_as_float(v[j].w), s[3]);
    }
  }
  *reinterpret_cast<uint2*>(a.out + t * a.ldo + c) = make_uint2(bf16x2_rn(s[0], s[1]), bf16x2_rn(s[2], s[3]));
}

// ------------------------------------------------------------------------------------------
// host
// ------------------------------------------------------------------------------------------
// A launch that may begin while the preceding kernel drains (its griddepcontrol.wait orders it).
template <typename K, typename... Args>
cudaError_t launch_dependent(K kern, dim3 grid, int threads, int smem, int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attrs;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int MODE>
cudaError_t launch_gemm_mode(const mxq_mx_tensor& w, const void* act, int64_t act_ld, const void* act_sf,
                             int64_t act_rows, int64_t K,
                             int64_t max_tiles, int64_t most, int pairs, const GemmArgs& ga, const mxq_mx_tensor* next,
                             cudaStream_t stream) {
  using C = GemmCfg<MODE>;
  auto kern = experts_gemm_kernel<MODE>;
  static PerDevice smem_set;
  const cudaError_t attr_err = allow_smem(smem_set, kern, C::SMEM_BYTES);
  if (attr_err != cudaSuccess) return attr_err;
  GemmMaps maps = {};
  if (!make_map(&maps.w, w.data, w.rows, K, w.ld, BM) || !make_sf_map(&maps.sfw, w.sf, w.rows / 128 * (K / 128), kSfKb) ||
      !make_sf_map(&maps.sfx, act_sf, max_tiles * 2 * (K / 128), 2 * kSfKb))
    return cudaErrorInvalidValue;
  // (encoding a map costs the host about a microsecond: only those that tiles of `most` tokens use)
  const int64_t half = round_up(most < kTileTokens ? most : kTileTokens, 16) / 2;
  for (int i = 0; i < kBoxes; ++i)
    if (MODE == kGateUpInPlace ? i == 0 && !make_map(&maps.x[i], act, act_rows, K, act_ld, 1)
                               : half > 32 * i - 24 && !make_map(&maps.x[i], act, act_rows, K, act_ld, 32 * i + 8))
      return cudaErrorInvalidValue;
  if (MODE == kDown && most >= kPassTokens && !make_f32_map(&maps.y16, ga.y, act_rows, ga.rows, ga.rows, kPassTokens))
    return cudaErrorInvalidValue;
  if (next != nullptr && !make_map(&maps.w_next, next->data, next->rows, next->cols, next->ld, BM))
    return cudaErrorInvalidValue;
  return launch_dependent(kern, dim3(static_cast<unsigned>(2 * pairs), 1, 1), kThreads<MODE>, C::SMEM_BYTES, 2, stream, maps, ga);
}

}  // namespace

int64_t experts_workspace_bytes(int64_t T, int32_t k, int32_t E, int64_t H, int64_t I) {
  return Layout(T, k, E, H, I).total;
}

cudaError_t launch_experts(const ExpertsLaunch& l, cudaStream_t stream) {
  const int sm_pairs = num_sms() / 2;
  const Layout lay(l.T, l.k, l.E, l.H, l.I);
  uint8_t* ws = static_cast<uint8_t*>(l.workspace);
  const int64_t P = l.T * l.k;
  auto pairs_for = [&](int64_t blocks) {
    const int64_t items = lay.max_tiles * blocks;
    return static_cast<int>(items < sm_pairs ? items : sm_pairs);
  };
  PlanArgs pa = {};
  pa.ids = l.ids;
  pa.P = static_cast<int32_t>(P);
  pa.E = l.E;
  pa.blocks1 = static_cast<int32_t>(lay.blocks1);
  pa.blocks2 = static_cast<int32_t>(lay.blocks2);
  pa.n_items = reinterpret_cast<int32_t*>(ws + lay.n_items);
  pa.items1 = reinterpret_cast<Item*>(ws + lay.items1);
  pa.items2 = reinterpret_cast<Item*>(ws + lay.items2);
  pa.pair_row = reinterpret_cast<int32_t*>(ws + lay.pair_row);
  pa.row_token = reinterpret_cast<int32_t*>(ws + lay.row_token);
  pa.k = l.k;
  pa.sf = static_cast<const uint8_t*>(l.x->sf);
  pa.sf_tiled = l.x->sf_layout == MXQ_SF_TILED_128X4;
  pa.words = static_cast<int32_t>(l.H / 128);
  pa.xsf = ws + lay.xsf;
  const bool copy = copies_rows(P, l.E);
  const bool in_plan = !copy && P <= kPlanThreads && P * pa.words <= kScalesInPlan;
  pa.experts = in_plan ? nullptr : reinterpret_cast<ExpertRows*>(ws + lay.experts);
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(pa);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  uint8_t* xp = ws + lay.xp;
  if (!in_plan) {
    const RowsArgs ra = {l.ids, l.E, l.k, l.T, pa.experts, pa.pair_row, pa.row_token, pa.sf, pa.sf_tiled, pa.words, pa.xsf,
                         static_cast<const uint8_t*>(l.x->data), l.x->ld, l.H, xp};
    e = launch_dependent(copy ? rows_kernel<true> : rows_kernel<false>,
                         dim3(static_cast<unsigned>(copy ? l.T : ceil_div(l.T, kRowsThreads / 32)), 1, 1), kRowsThreads, 0, 1,
                         stream, ra);
    if (e != cudaSuccess) return e;
  }

  GemmArgs g1 = {};
  g1.items = pa.items1;
  g1.n_items = pa.n_items;
  g1.kbs = static_cast<int32_t>(l.H / BK);
  g1.rows = static_cast<int32_t>(2 * l.I);
  g1.row_token = pa.row_token;
  g1.early = in_plan ? 0 : 1;
  g1.hq = ws + lay.hq;
  g1.hsf = ws + lay.hsf;
  g1.status = l.status;
  const int pairs1 = pairs_for(lay.blocks1);
  g1.next_items = pa.items2;
  g1.next_n = pa.n_items + 1;
  g1.next_kbs = static_cast<int32_t>(l.I / BK);
  g1.next_rows = static_cast<int32_t>(l.H);
  g1.next_pairs = pairs_for(lay.blocks2);
  e = copy ? launch_gemm_mode<kGateUp>(*l.w13, xp, l.H, pa.xsf, P, l.H, lay.max_tiles, P, pairs1, g1, l.w2, stream)
           : launch_gemm_mode<kGateUpInPlace>(*l.w13, l.x->data, l.x->ld, pa.xsf, l.T, l.H, lay.max_tiles, P, pairs1, g1,
                                              l.w2, stream);
  if (e != cudaSuccess) return e;

  GemmArgs g2 = {};
  g2.items = pa.items2;
  g2.n_items = pa.n_items + 1;
  g2.kbs = static_cast<int32_t>(l.I / BK);
  g2.rows = static_cast<int32_t>(l.H);
  g2.y = reinterpret_cast<float*>(ws + lay.y);
  g2.status = l.status;
  e = launch_gemm_mode<kDown>(*l.w2, g1.hq, l.I, g1.hsf, P, l.I, lay.max_tiles, P, pairs_for(lay.blocks2), g2, nullptr, stream);
  if (e != cudaSuccess) return e;

  CombineArgs ca = {g2.y, l.weights, pa.pair_row, l.k, l.H, l.ldo, static_cast<uint16_t*>(l.out)};
  return launch_dependent(combine_kernel,
                          dim3(static_cast<unsigned>(l.T), static_cast<unsigned>(ceil_div(l.H, 4 * kCombineThreads)), 1),
                          kCombineThreads, 0, 1, stream, ca);
}

}  // namespace mxq
