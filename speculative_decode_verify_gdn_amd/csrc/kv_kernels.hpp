// kv_kernels.hpp -- internal launch interface of the attention layers' paged
// key/value cache and attention (kv_api.cpp to the gfx950 kernels), and the
// device-side view of a sequence that they share.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_verify.h"

namespace gdn {

// Where a round's new tokens are.
struct KvBatch {
  const int32_t* q_start;  // [B+1], or nullptr: sequence b has rows b*T .. b*T+T-1
  const int32_t* seq_len;  // [B]
  int B, T, N;
  int page_shift;  // log2(page_size)
  int n_pages, max_blocks;
};

// One sequence's new tokens: rows s .. s+n-1, behind ctx cached tokens.
struct KvSpan {
  int s, n, ctx;
  bool ok;  // otherwise n = 0
};

// The rows alone (kv_commit's copies run beside the update of seq_len).
__device__ __forceinline__ KvSpan kv_rows(const KvBatch& k, int b) {
  KvSpan r;
  if (k.q_start) {
    r.s = k.q_start[b];
    const int e = k.q_start[b + 1];
    r.ok = r.s >= 0 && e >= r.s && e <= k.N && e - r.s <= k.T;
    r.n = r.ok ? e - r.s : 0;
  } else {
    r.s = b * k.T;
    r.n = k.T;
    r.ok = true;
  }
  r.ctx = 0;
  return r;
}

__device__ __forceinline__ KvSpan kv_span(const KvBatch& k, int b) {
  KvSpan r = kv_rows(k, b);
  r.ctx = k.seq_len[b];
  const int room = k.max_blocks << k.page_shift;  // <= 2^30
  if (r.ctx < 0 || r.ctx > room - r.n) {
    r.ok = false;
    r.n = 0;
    r.ctx = 0;
  }
  return r;
}

// The kernels' own division by the page size, rounded up.
__device__ __forceinline__ int kv_blocks(const KvBatch& k, int tokens) {
  return (tokens + (1 << k.page_shift) - 1) >> k.page_shift;
}

struct KvReserveArgs {
  KvBatch k;
  int32_t* block_table;
  const int32_t* free_pages;
  const int32_t* n_free;
  int32_t* n_left;
  int32_t* slots;
  int32_t* dev_err;
};

struct KvAppendArgs {
  const void* k;
  const void* v;
  int64_t k_ld, v_ld;
  const int32_t* slots;
  void* k_cache;
  void* v_cache;
  int32_t* dev_err;
  int L, N, H, page_shift, n_pages;
};

struct KvCommitArgs {
  KvBatch k;
  const int32_t* path;  // or nullptr: no copies
  const int32_t* n_keep;
  const int32_t* done;  // or nullptr
  const int32_t* slots;
  int32_t* seq_len_out;
  const int32_t* block_table;
  int32_t* free_pages;
  const int32_t* n_left;
  int32_t* n_free;
  const void* kk;
  const void* vv;
  int64_t k_ld, v_ld;
  void* k_cache;
  void* v_cache;
  int32_t* dev_err;
  int L, H;
};

struct AttnArgs {
  KvBatch k;
  const int32_t* block_table;
  const int32_t* parent;  // [N] or nullptr
  const void* q;
  int64_t q_ld;
  float scale;
  const void* k_cache;
  const void* v_cache;
  void* o;
  void* ws;
  int32_t* dev_err;
  int L, Hq, Hkv;
};

// dtype: 0 fp32, 1 bf16; hipErrorInvalidValue for an uninstantiated head size.
hipError_t launch_kv_reserve(const KvReserveArgs& a, hipStream_t s);
hipError_t launch_kv_append(const KvAppendArgs& a, int head_dim, int dtype, hipStream_t s);
hipError_t launch_kv_commit(const KvCommitArgs& a, int head_dim, int dtype, hipStream_t s);
hipError_t launch_attn(const AttnArgs& a, int head_dim, int dtype, hipStream_t s);
// Bytes of the workspace that launch_attn uses, for sequences of at most `rows`
// query rows to a key head.
size_t attn_workspace(long long rows, int head_dim, int dtype);

}  // namespace gdn
