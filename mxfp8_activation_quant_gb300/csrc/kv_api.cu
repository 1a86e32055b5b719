// C ABI of the paged key-value cache: argument checks on the host, then the launches of
// mxq_kv_internal.h. The operators are documented in include/mxq_kv.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "mxq_internal.h"
#include "mxq_kv_internal.h"

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;  // a tensor map's

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Strides of dimensions of size 1 become those of a dense array, so that nothing looks at the caller's.
void settle(mxq_kv_cache* c) {
  const int64_t row = c->dim, sf_row = c->dim / 32;
  if (c->heads == 1) c->head_stride = row, c->sf_head_stride = sf_row;
  if (c->page_size == 1) c->token_stride = row * c->heads, c->sf_token_stride = sf_row * c->heads;
  if (c->pages == 1) c->page_stride = row * c->heads * c->page_size, c->sf_page_stride = sf_row * c->heads * c->page_size;
}

// Whether rows of `row` bytes at these strides overlap. The strides are taken from the smallest up, each at
// least the span of what lies below it.
bool overlaps(const mxq_kv_cache& c, int64_t page, int64_t token, int64_t head, int64_t row) {
  std::pair<int64_t, int64_t> d[3] = {{page, c.pages}, {token, c.page_size}, {head, c.heads}};
  std::sort(d, d + 3);
  int64_t span = row;
  for (const auto& [stride, n] : d) {
    if (n == 1) continue;
    if (stride < span) return true;
    if (stride > (int64_t(1) << 62) / n) return true;  // (no address space holds it)
    span += stride * (n - 1);
  }
  return false;
}

// Checks a cache and gives it back with settled strides.
mxq_status check_cache(const mxq_kv_cache* in, mxq_kv_cache* out) {
  if (in == nullptr || in->data == nullptr || in->sf == nullptr) return MXQ_ERR_INVALID_ARG;
  if (in->pages <= 0 || in->page_size <= 0 || in->heads <= 0 || in->dim <= 0) return MXQ_ERR_INVALID_ARG;
  if (in->dim % 32 != 0 || in->dim > 1024 || in->heads > 1024 || in->page_size > 65536 ||
      in->pages >= (int64_t(1) << 31) || in->pages * in->page_size >= (int64_t(1) << 31))
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  *out = *in;
  settle(out);
  for (int64_t s : {out->page_stride, out->token_stride, out->head_stride})
    if (s < 0 || s >= kMaxStride) return MXQ_ERR_UNSUPPORTED_SHAPE;
  for (int64_t s : {out->sf_page_stride, out->sf_token_stride, out->sf_head_stride})
    if (s < 0 || s >= (int64_t(1) << 31)) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (!al16(out->data) || !al4(out->sf) || out->page_stride % 16 != 0 || out->token_stride % 16 != 0 ||
      out->head_stride % 16 != 0)
    return MXQ_ERR_MISALIGNED;
  if (out->dim % 128 == 0 && (out->sf_page_stride % 4 != 0 || out->sf_token_stride % 4 != 0 || out->sf_head_stride % 4 != 0))
    return MXQ_ERR_MISALIGNED;
  if (overlaps(*out, out->page_stride, out->token_stride, out->head_stride, out->dim) ||
      overlaps(*out, out->sf_page_stride, out->sf_token_stride, out->sf_head_stride, out->dim / 32))
    return MXQ_ERR_INVALID_ARG;
  return MXQ_OK;
}

mxq_status check_rows(const void* x, int64_t* ld, int64_t* ldh, int64_t T, const mxq_kv_cache& c) {
  if (x == nullptr) return MXQ_ERR_INVALID_ARG;
  if (c.heads == 1) *ldh = c.dim;
  if (T == 1) *ld = static_cast<int64_t>(c.heads) * *ldh;
  if (*ldh < c.dim || *ld < c.dim || *ld >= kMaxStride || *ldh >= kMaxStride) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (!al16(x) || *ld % 8 != 0 || *ldh % 8 != 0) return MXQ_ERR_MISALIGNED;
  return MXQ_OK;
}

mxq_status check_table(const void* table, int64_t* ld, int32_t width, int64_t B) {
  if (table == nullptr || width <= 0) return MXQ_ERR_INVALID_ARG;
  if (B == 1) *ld = width;
  if (*ld < width || *ld >= kMaxStride) return MXQ_ERR_UNSUPPORTED_SHAPE;
  return al4(table) ? MXQ_OK : MXQ_ERR_MISALIGNED;
}

bool attention_shape_ok(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  return B >= 1 && q_heads >= 1 && kv_heads >= 1 && q_heads <= 4096 && q_heads % kv_heads == 0 && B <= 65536 / kv_heads &&
         (dim == 128 || dim == 256 || dim == 384 || dim == 512);
}

}  // namespace

extern "C" {

mxq_status kv_write_mxfp8(const void* k_bf16, int64_t ldk, int64_t ldkh, const mxq_kv_cache* k_cache, const void* v_bf16,
                          int64_t ldv, int64_t ldvh, const mxq_kv_cache* v_cache, const void* slots_i32, int64_t T,
                          void* stream) {
  if (slots_i32 == nullptr || T <= 0 || (v_bf16 == nullptr) != (v_cache == nullptr)) return MXQ_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 31)) return MXQ_ERR_UNSUPPORTED_SHAPE;
  mxq::KvWriteLaunch l{};
  l.tensors = v_cache != nullptr ? 2 : 1;
  for (int i = 0; i < l.tensors; ++i) {
    mxq::KvTensor& t = l.t[i];
    t.rows = i == 0 ? k_bf16 : v_bf16;
    t.ld = i == 0 ? ldk : ldv;
    t.ldh = i == 0 ? ldkh : ldvh;
    mxq_status st = check_cache(i == 0 ? k_cache : v_cache, &t.c);
    if (st != MXQ_OK) return st;
    if ((st = check_rows(t.rows, &t.ld, &t.ldh, T, t.c)) != MXQ_OK) return st;
  }
  if (l.tensors == 2 && (l.t[0].c.pages != l.t[1].c.pages || l.t[0].c.page_size != l.t[1].c.page_size))
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (!al4(slots_i32)) return MXQ_ERR_MISALIGNED;
  l.slots = static_cast<const int32_t*>(slots_i32);
  l.T = T;
  return mxq::from_cuda(mxq::launch_kv_write(l, static_cast<cudaStream_t>(stream)));
}

mxq_status kv_read_bf16(const mxq_kv_cache* k_cache, const mxq_kv_cache* v_cache, const void* block_table_i32,
                        int64_t ld_table, int32_t table_width, const void* cu_rows_i32, const void* starts_i32, int64_t B,
                        int64_t rows, void* k_out, void* v_out, void* stream) {
  if (cu_rows_i32 == nullptr || B <= 0 || rows <= 0 || (v_out == nullptr) != (v_cache == nullptr)) return MXQ_ERR_INVALID_ARG;
  if (B >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31)) return MXQ_ERR_UNSUPPORTED_SHAPE;
  mxq::KvReadLaunch l{};
  l.tensors = v_cache != nullptr ? 2 : 1;
  for (int i = 0; i < l.tensors; ++i) {
    mxq::KvTensor& t = l.t[i];
    t.rows = i == 0 ? k_out : v_out;
    mxq_status st = check_cache(i == 0 ? k_cache : v_cache, &t.c);
    if (st != MXQ_OK) return st;
    t.ldh = t.c.dim;
    t.ld = static_cast<int64_t>(t.c.heads) * t.c.dim;
    if ((st = check_rows(t.rows, &t.ld, &t.ldh, rows, t.c)) != MXQ_OK) return st;
  }
  if (l.tensors == 2 && (l.t[0].c.pages != l.t[1].c.pages || l.t[0].c.page_size != l.t[1].c.page_size))
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  const mxq_status st = check_table(block_table_i32, &ld_table, table_width, B);
  if (st != MXQ_OK) return st;
  if (!al4(cu_rows_i32) || !al4(starts_i32)) return MXQ_ERR_MISALIGNED;
  l.table = static_cast<const int32_t*>(block_table_i32);
  l.ld_table = ld_table;
  l.table_width = table_width;
  l.cu = static_cast<const int32_t*>(cu_rows_i32);
  l.starts = static_cast<const int32_t*>(starts_i32);
  l.B = B;
  l.rows = rows;
  return mxq::from_cuda(mxq::launch_kv_read(l, static_cast<cudaStream_t>(stream)));
}

int64_t mxq_paged_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  return attention_shape_ok(B, q_heads, kv_heads, dim) ? mxq::paged_attention_workspace_bytes(B, q_heads, kv_heads, dim) : 0;
}

mxq_status paged_attention_mxfp8(const void* q_bf16, int64_t ldq, int64_t ldqh, const mxq_kv_cache* k_cache,
                                 const mxq_kv_cache* v_cache, const void* block_table_i32, int64_t ld_table,
                                 int32_t table_width, const void* seq_lens_i32, int64_t B, int32_t q_heads, float scale,
                                 void* o_bf16, void* o_q, void* o_sf_packed_i32, void* o_sf_rowmajor, void* o_sf_128x4,
                                 void* lse_f32, void* workspace, int64_t workspace_bytes, void* status, void* stream) {
  if (q_bf16 == nullptr || seq_lens_i32 == nullptr || workspace == nullptr) return MXQ_ERR_INVALID_ARG;
  const bool scales = o_sf_packed_i32 != nullptr || o_sf_rowmajor != nullptr || o_sf_128x4 != nullptr;
  if ((o_bf16 == nullptr && o_q == nullptr) || (o_q != nullptr) != scales) return MXQ_ERR_INVALID_ARG;
  if (B <= 0 || q_heads <= 0 || !(scale >= -1e38f && scale <= 1e38f)) return MXQ_ERR_INVALID_ARG;  // (times log2(e) it is finite too)
  mxq_kv_cache k, v;
  mxq_status st = check_cache(k_cache, &k);
  if (st != MXQ_OK) return st;
  if (v_cache != nullptr) {
    if ((st = check_cache(v_cache, &v)) != MXQ_OK) return st;
    if (v.pages != k.pages || v.page_size != k.page_size || v.heads != k.heads || v.dim != k.dim)
      return MXQ_ERR_UNSUPPORTED_SHAPE;
  }
  if (!attention_shape_ok(B, q_heads, k.heads, k.dim) || k.page_size % 16 != 0) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_table(block_table_i32, &ld_table, table_width, B)) != MXQ_OK) return st;
  const int64_t places = static_cast<int64_t>(table_width) * k.page_size;
  if (places > (int64_t(1) << 30) || mxq::paged_attention_units(B, q_heads, k.heads, places) >= (int64_t(1) << 30))
    return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (q_heads == 1) ldqh = k.dim;
  if (B == 1) ldq = static_cast<int64_t>(q_heads) * ldqh;
  if (ldqh < k.dim || ldq < k.dim || ldq >= kMaxStride || ldqh >= kMaxStride) return MXQ_ERR_UNSUPPORTED_SHAPE;
  if (!al16(q_bf16) || ldq % 8 != 0 || ldqh % 8 != 0 || !al16(o_bf16) || !al16(o_q) || !al16(o_sf_packed_i32) ||
      !al16(o_sf_rowmajor) || !al16(o_sf_128x4) || !al4(lse_f32) || !al4(seq_lens_i32) || !al16(workspace) || !al16(status))
    return MXQ_ERR_MISALIGNED;
  if (workspace_bytes < mxq::paged_attention_workspace_bytes(B, q_heads, k.heads, k.dim)) return MXQ_ERR_INVALID_ARG;
  mxq::PagedAttentionLaunch l{q_bf16, ldq, ldqh, &k, v_cache != nullptr ? &v : nullptr,
                              static_cast<const int32_t*>(block_table_i32), ld_table, table_width,
                              static_cast<const int32_t*>(seq_lens_i32), B, q_heads, scale, o_bf16, o_q, o_sf_packed_i32,
                              o_sf_rowmajor, o_sf_128x4, static_cast<float*>(lse_f32), workspace,
                              static_cast<int32_t*>(status)};
  return mxq::from_cuda(mxq::launch_paged_attention(l, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
