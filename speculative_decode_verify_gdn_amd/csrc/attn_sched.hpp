// attn_sched.hpp -- how the attention kernels divide a batch of unequal
// sequences among workgroups, on the device (the lengths are only known there).
//
// An item is one tile of R query rows (the rows of a key head: G query heads of
// each token, token by token) against all its keys.  Items are laid on a line,
// each as long as it costs (its keys, and as many more as its start and end are
// worth), in the order layer, sequence, key head, tile.  Active workgroup w takes the part
// [w, w+1) * total / active of the line, so every workgroup has the same amount
// of work whatever the lengths are, and at most two items of a workgroup are
// shared with others: the one that its part begins within (its fragment goes to
// place 2w of the workspace) and the one that it ends within (place 2w + 1).
// k_attn_join adds the fragments of a shared item in order of w.
#pragma once

#include "attn_parts.hpp"
#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {

struct AttnSched {
  long long total;   // length of the line over all layers
  long long layer;   // over one layer
  int active;        // workgroups that take part
};

// A shared item as its first workgroup describes it for the join: last = -1 if
// there is none.
struct AttnJoin {
  int last;  // last workgroup with a fragment
  int rows;  // rows of the tile
  int skip;  // the tile's first row within its first token
  int pad;
  long long out;  // of that token's first query head of the tile's key head, in o
};

// One item, and where it lies.
struct AttnItem {
  int layer, b, h, tile;
  long long at, cost;  // start on the line, length
};

// ITEM: what an item costs beside its keys, in keys (its queries, the first loads'
// latency, keys that only some rows see, the outputs or fragments).
template <int R, int ITEM>
struct AttnLine {
  // Cost of the first i tiles of one head: a tile costs its cached tokens, the
  // new ones up to its end at `per` a tile, and ITEM.
  static __device__ __forceinline__ long long upto(const KvSpan& r, int per, int i) {
    return static_cast<long long>(i) * (r.ctx + ITEM) +
           ((static_cast<long long>(i) * (i + 1) * per) >> 1);
  }
  static __device__ __forceinline__ int tiles(const KvSpan& r, int G) {
    return (r.n * G + R - 1) / R;  // n * G <= 2^30
  }
  static __device__ __forceinline__ long long sequence(const KvSpan& r, int G, int H) {
    return H * upto(r, per(G), tiles(r, G));
  }
  // tokens of a tile, at least one
  static __device__ __forceinline__ int per(int G) { return G >= R ? 1 : R / G; }
};

// a * b / c, rounded the same way for everyone who asks: monotone in a, 0 at
// a = 0 and b at a = c.
__device__ __forceinline__ long long part_of(long long a, long long b, long long c) {
  if (a >= c) return b;
  return static_cast<long long>(static_cast<double>(a) * static_cast<double>(b) /
                                static_cast<double>(c));
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long long lane_of(long long x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(x), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(x >> 32), lane);
  return static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ long long uni(long long x) { return lane_of(x, 0); }

// v plus the v of the lanes that DPP control C (row mask M) takes it from.
template <int C, int M>
__device__ __forceinline__ long long dpp_add(long long v) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), C, M, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), C, M, 0xf, false);
  return v + static_cast<long long>(static_cast<uint64_t>(hi) << 32 | lo);
}
// Inclusive prefix sum over a wave: within rows of 16, then rows 0 and 2 into
// 1 and 3, then the first half into the second.
__device__ __forceinline__ long long wave_scan(long long v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  return dpp_add<0x143, 0xc>(v);
}

// The line's length, and the sequence and place where this workgroup's part
// begins, found by every wave for itself (64 sequences a step, no barrier: what
// a call of few keys waits for is this chain of latencies).  Uniform.
struct AttnStart {
  AttnSched s;
  int wg;            // this workgroup's number on the line
  long long lo, hi;  // its part; empty if it has none
  int layer, b;      // of the first item
  long long seq_at;  // where sequence b begins
  KvSpan span;       // of sequence b
};

// NEAR: neighbours on the line to one XCD.  idle: as attn_active has it.
template <typename Line, bool NEAR>
__device__ AttnStart attn_start(const AttnArgs& p, int G, int n_wg, long long grain, int idle) {
  const KvBatch& k = p.k;
  const int lane = threadIdx.x % kWave;
  long long sum = 0, v = 0, upto = 0;
  KvSpan r{};
  bool bad = false;
  auto step = [&](int c) {
    v = 0;
    if (c + lane < k.B) {
      r = kv_span(k, c + lane);
      bad |= !r.ok;
      v = Line::sequence(r, G, p.Hkv);
    }
    upto = wave_scan(v);
  };
  for (int c = 0; c < k.B; c += kWave) {
    step(c);
    upto += sum;
    sum = lane_of(upto, kWave - 1);
  }
  if (blockIdx.x == 0 && __any(bad) && threadIdx.x == 0 && p.dev_err)
    atomicOr(p.dev_err, GDN_DEV_ERR_LENGTH);
  AttnStart a{};
  a.s.layer = sum;
  a.s.total = sum * p.L;
  a.s.active = uni(attn_active(a.s.total, n_wg, grain, p.Hkv * p.L, idle));
  const int block = blockIdx.x;
  const int wg = a.wg = NEAR ? attn_spread(block, a.s.active, kNumXcd) : block;
  if (wg >= a.s.active) return a;
  a.lo = uni(part_of(wg, a.s.total, a.s.active));
  a.hi = uni(part_of(wg + 1, a.s.total, a.s.active));
  a.layer = p.L == 1 ? 0 : static_cast<int>(a.lo / sum);
  const long long x = a.lo - a.layer * sum;
  long long before = 0;
  for (int c = 0;; c += kWave) {
    if (k.B > kWave) {  // one step's values are still in registers
      step(c);
      upto += before;
      before = lane_of(upto, kWave - 1);
    }
    const unsigned long long who = __ballot(upto - v <= x && x < upto);
    if (who || c + kWave >= k.B) {
      const int at = who ? __builtin_ctzll(who) : 0;
      a.b = c + at;
      a.seq_at = a.layer * sum + lane_of(upto - v, at);
      a.span.s = __builtin_amdgcn_readlane(r.s, at);
      a.span.n = __builtin_amdgcn_readlane(r.n, at);
      a.span.ctx = __builtin_amdgcn_readlane(r.ctx, at);
      a.span.ok = true;
      return a;
    }
  }
}

// The item at place x of the line, x within the sequence (layer, b) that begins
// at seq_at.
template <typename Line>
__device__ AttnItem attn_item(const AttnArgs& p, int G, int layer, int b, const KvSpan& span,
                              long long seq_at, long long x) {
  AttnItem it;
  it.layer = layer;
  it.b = b;
  const int nt = Line::tiles(span, G), per = Line::per(G);
  const long long head = Line::upto(span, per, nt);
  const long long off = x - seq_at;
  int h = p.Hkv == 1 ? 0
                     : uni(static_cast<int>(static_cast<double>(off) / static_cast<double>(head)));
  if (h * head > off) --h;
  if ((h + 1) * head <= off) ++h;
  it.h = h;
  const long long in = off - h * head;
  int lo = 0, hi = nt - 1;  // the last tile that begins at or before `in`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (Line::upto(span, per, mid) <= in)
      lo = mid;
    else
      hi = mid - 1;
  }
  it.tile = lo;
  const long long a = Line::upto(span, per, lo);
  it.at = seq_at + h * head + a;
  it.cost = Line::upto(span, per, lo + 1) - a;
  return it;
}

// The workgroup whose part holds place x.
__device__ __forceinline__ int attn_owner(const AttnSched& s, long long x) {
  int w = static_cast<int>(part_of(x, s.active, s.total));
  if (w >= s.active) w = s.active - 1;
  while (w > 0 && part_of(w, s.total, s.active) > x) --w;
  while (w + 1 < s.active && part_of(w + 1, s.total, s.active) <= x) ++w;
  return w;
}

}  // namespace gdn
