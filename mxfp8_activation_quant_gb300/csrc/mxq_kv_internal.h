// Internal launcher interface of the paged key-value cache (host side). Arguments are validated by the
// C ABI layer (kv_api.cu) before any of these is called.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxq_kv.h"

namespace mxq {

// One tensor of kv_write_mxfp8 / kv_read_bf16.
struct KvTensor {
  mxq_kv_cache c;
  const void* rows;    // bf16 [T, heads, dim]; written by kv_read_bf16
  int64_t ld, ldh;     // row strides in elements
};

struct KvWriteLaunch {
  KvTensor t[2];       // keys, values
  int tensors;
  const int32_t* slots;
  int64_t T;
};
cudaError_t launch_kv_write(const KvWriteLaunch& a, cudaStream_t stream);

struct KvReadLaunch {
  KvTensor t[2];
  int tensors;
  const int32_t* table;
  int64_t ld_table;
  int32_t table_width;
  const int32_t* cu;
  const int32_t* starts;
  int64_t B, rows;
};
cudaError_t launch_kv_read(const KvReadLaunch& a, cudaStream_t stream);

struct PagedAttentionLaunch {
  const void* q;
  int64_t ldq, ldqh;
  const mxq_kv_cache* k;
  const mxq_kv_cache* v;  // null: the keys
  const int32_t* table;
  int64_t ld_table;
  int32_t table_width;
  const int32_t* lens;
  int64_t B;
  int32_t q_heads;
  float scale;
  void* o;
  void* o_q;
  void* sf_packed;
  void* sf_rowmajor;
  void* sf_tiled;
  float* lse;
  void* workspace;
  int32_t* status;
};
cudaError_t launch_paged_attention(const PagedAttentionLaunch& a, cudaStream_t stream);
// Pieces of work, of 64 tokens, at tables of `places` tokens.
int64_t paged_attention_units(int64_t B, int32_t q_heads, int32_t kv_heads, int64_t places);
int64_t paged_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim);

}  // namespace mxq
