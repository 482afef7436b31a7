// kv_api.cpp -- the C ABI of the attention layers' paged key/value cache and
// attention: host-side validation and dispatch, as gdn_api.cpp for the GDN
// layers.  Declared in include/gdn_verify.h.

#include <cmath>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_verify.h"
#include "kv_kernels.hpp"

namespace {

using gdn::KvBatch;

constexpr int kMaxTree = 64;
constexpr int32_t kMaxTokens = 1 << 24;

// Structural checks shared by every call that takes a kv_shape.
gdn_status check_kv(const kv_shape* s) {
  if (!s) return GDN_ERR_INVALID_ARG;
  if (s->n_layers < 1 || s->batch < 1 || s->n_q_heads < 1 || s->n_kv_heads < 1 ||
      s->n_pages < 1 || s->max_blocks < 1 || s->head_dim < 1 || s->page_size < 1)
    return GDN_ERR_INVALID_ARG;
  if (s->n_q_heads % s->n_kv_heads != 0) return GDN_ERR_INVALID_ARG;
  if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (s->head_dim != 64 && s->head_dim != 128 && s->head_dim != 256) return GDN_ERR_UNSUPPORTED;
  if (s->page_size < 16 || s->page_size > 256 || (s->page_size & (s->page_size - 1)))
    return GDN_ERR_UNSUPPORTED;
  // slots and positions are 32-bit; grids stay within their limits
  if (static_cast<long long>(s->n_pages) * s->page_size >= (1LL << 31)) return GDN_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->max_blocks) * s->page_size > (1LL << 30))
    return GDN_ERR_UNSUPPORTED;
  if (s->batch >= 65536) return GDN_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->n_layers) * s->n_kv_heads >= 65536) return GDN_ERR_UNSUPPORTED;
  if (static_cast<long long>(s->n_layers) * s->batch > (1LL << 23)) return GDN_ERR_UNSUPPORTED;
  if (s->n_q_heads >= 65536) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_batch(const kv_shape* s, int32_t T, int32_t n_tokens, const int32_t* q_start) {
  const gdn_status st = check_kv(s);
  if (st != GDN_OK) return st;
  if (T < 1 || n_tokens < 1) return GDN_ERR_INVALID_ARG;
  if (!q_start && static_cast<long long>(s->batch) * T > n_tokens) return GDN_ERR_INVALID_ARG;
  if (n_tokens > kMaxTokens || T > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int log2i(int x) { return 31 - __builtin_clz(static_cast<unsigned>(x)); }

KvBatch kv_batch(const kv_shape* s, int32_t T, int32_t n_tokens, const int32_t* q_start,
                 const int32_t* seq_len) {
  KvBatch k{};
  k.q_start = q_start;
  k.seq_len = seq_len;
  k.B = s->batch;
  k.T = T;
  k.N = n_tokens;
  k.page_shift = log2i(s->page_size);
  k.n_pages = s->n_pages;
  k.max_blocks = s->max_blocks;
  return k;
}

// Rows of `heads` heads, ld elements apart: whole 16-byte pieces, and no
// further apart than 64-bit offsets of 2^24 rows and 2^16 layers reach.
bool ld_ok(const kv_shape* s, int64_t ld, int heads) {
  const int per = s->dtype == GDN_BF16 ? 8 : 4;
  return ld >= static_cast<int64_t>(heads) * s->head_dim && ld % per == 0 && ld <= (1LL << 20);
}

// Query rows of a key head are counted in 32 bits.
bool rows_ok(const kv_shape* s, int32_t n_tokens) {
  return static_cast<long long>(n_tokens) * (s->n_q_heads / s->n_kv_heads) <= (1LL << 30);
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

gdn_status launch_status(hipError_t e) {
  if (e == hipSuccess) return GDN_OK;
  if (e == hipErrorInvalidValue) return GDN_ERR_UNSUPPORTED;
  return GDN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

gdn_status kv_reserve(const kv_shape* shape, int32_t T, int32_t n_tokens, const int32_t* q_start,
                      const int32_t* seq_len, int32_t* block_table, const int32_t* free_pages,
                      const int32_t* n_free, int32_t* n_left, int32_t* slots, int32_t* dev_err,
                      void* stream) {
  const gdn_status st = check_batch(shape, T, n_tokens, q_start);
  if (st != GDN_OK) return st;
  if (!seq_len || !block_table || !free_pages || !n_free || !n_left || !slots)
    return GDN_ERR_INVALID_ARG;
  if (n_free == n_left) return GDN_ERR_INVALID_ARG;  // workgroups still read one
  gdn::KvReserveArgs a{};
  a.k = kv_batch(shape, T, n_tokens, q_start, seq_len);
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.n_left = n_left;
  a.slots = slots;
  a.dev_err = dev_err;
  return launch_status(gdn::launch_kv_reserve(a, static_cast<hipStream_t>(stream)));
}

gdn_status kv_append(const kv_shape* shape, int32_t n_tokens, const void* k, int64_t k_ld,
                     const void* v, int64_t v_ld, const int32_t* slots, void* k_cache,
                     void* v_cache, int32_t* dev_err, void* stream) {
  const gdn_status st = check_kv(shape);
  if (st != GDN_OK) return st;
  if (n_tokens < 1) return GDN_ERR_INVALID_ARG;
  if (n_tokens > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (!k || !v || !slots || !k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
  if (!ld_ok(shape, k_ld, shape->n_kv_heads) || !ld_ok(shape, v_ld, shape->n_kv_heads))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(k) || !aligned(v) || !aligned(k_cache) || !aligned(v_cache))
    return GDN_ERR_INVALID_ARG;
  gdn::KvAppendArgs a{};
  a.k = k;
  a.v = v;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.dev_err = dev_err;
  a.L = shape->n_layers;
  a.N = n_tokens;
  a.H = shape->n_kv_heads;
  a.page_shift = log2i(shape->page_size);
  a.n_pages = shape->n_pages;
  return launch_status(gdn::launch_kv_append(a, shape->head_dim, shape->dtype,
                                             static_cast<hipStream_t>(stream)));
}

size_t attn_verify_workspace_bytes(const kv_shape* shape, int32_t T, int32_t n_tokens) {
  if (check_kv(shape) != GDN_OK || T < 1 || n_tokens < 1 || n_tokens > kMaxTokens ||
      T > kMaxTokens || !rows_ok(shape, n_tokens))
    return 0;
  return gdn::attn_workspace(
      static_cast<long long>(T) * (shape->n_q_heads / shape->n_kv_heads), shape->head_dim,
      shape->dtype);
}

gdn_status attn_verify(const kv_shape* shape, int32_t T, int32_t n_tokens, const int32_t* q_start,
                       const int32_t* seq_len, const int32_t* block_table, const int32_t* parent,
                       const void* q, int64_t q_ld, float scale, const void* k_cache,
                       const void* v_cache, void* o, void* workspace, size_t workspace_bytes,
                       int32_t* dev_err, void* stream) {
  const gdn_status st = check_batch(shape, T, n_tokens, q_start);
  if (st != GDN_OK) return st;
  if (!seq_len || !block_table || !q || !k_cache || !v_cache || !o) return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(scale * 1.4426950408889634f)) return GDN_ERR_INVALID_ARG;  // exp2's factor
  if (!ld_ok(shape, q_ld, shape->n_q_heads)) return GDN_ERR_INVALID_ARG;
  if (!aligned(q) || !aligned(k_cache) || !aligned(v_cache) || !aligned(o))
    return GDN_ERR_INVALID_ARG;
  if (parent && T > kMaxTree) return GDN_ERR_UNSUPPORTED;
  if (!rows_ok(shape, n_tokens)) return GDN_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace) ||
      workspace_bytes < attn_verify_workspace_bytes(shape, T, n_tokens))
    return GDN_ERR_WORKSPACE;
  gdn::AttnArgs a{};
  a.k = kv_batch(shape, T, n_tokens, q_start, seq_len);
  a.block_table = block_table;
  a.parent = parent;
  a.q = q;
  a.q_ld = q_ld;
  a.scale = scale;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.o = o;
  a.ws = workspace;
  a.dev_err = dev_err;
  a.L = shape->n_layers;
  a.Hq = shape->n_q_heads;
  a.Hkv = shape->n_kv_heads;
  return launch_status(gdn::launch_attn(a, shape->head_dim, shape->dtype,
                                        static_cast<hipStream_t>(stream)));
}

gdn_status kv_commit(const kv_shape* shape, int32_t T, int32_t n_tokens, const int32_t* q_start,
                     const int32_t* path, const int32_t* n_keep, const int32_t* done,
                     const int32_t* slots, const int32_t* seq_len, int32_t* seq_len_out,
                     const int32_t* block_table, int32_t* free_pages, const int32_t* n_left,
                     int32_t* n_free, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                     void* k_cache, void* v_cache, int32_t* dev_err, void* stream) {
  const gdn_status st = check_batch(shape, T, n_tokens, q_start);
  if (st != GDN_OK) return st;
  if (!n_keep || !slots || !seq_len || !seq_len_out || !block_table || !free_pages || !n_left ||
      !n_free)
    return GDN_ERR_INVALID_ARG;
  if (path) {
    if (T > kMaxTree) return GDN_ERR_UNSUPPORTED;
    if (!k || !v || !k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
    if (!ld_ok(shape, k_ld, shape->n_kv_heads) || !ld_ok(shape, v_ld, shape->n_kv_heads))
      return GDN_ERR_INVALID_ARG;
    if (!aligned(k) || !aligned(v) || !aligned(k_cache) || !aligned(v_cache))
      return GDN_ERR_INVALID_ARG;
  }
  gdn::KvCommitArgs a{};
  a.k = kv_batch(shape, T, n_tokens, q_start, seq_len);
  a.path = path;
  a.n_keep = n_keep;
  a.done = done;
  a.slots = slots;
  a.seq_len_out = seq_len_out;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.n_left = n_left;
  a.n_free = n_free;
  a.kk = k;
  a.vv = v;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.dev_err = dev_err;
  a.L = shape->n_layers;
  a.H = shape->n_kv_heads;
  return launch_status(gdn::launch_kv_commit(a, shape->head_dim, shape->dtype,
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
