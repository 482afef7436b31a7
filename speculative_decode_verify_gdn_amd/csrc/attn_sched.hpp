// attn_sched.hpp -- how the attention kernels divide a batch of unequal
// sequences among workgroups, on the device (the lengths are only known there).
//
// An item is one tile of R query rows (the rows of a key head: G query heads of
// each token, token by token) against all its keys.  Items are laid on a line,
// each as long as it costs (its keys, and kItemCost for its start and end), in
// the order layer, sequence, key head, tile.  Active workgroup w takes the part
// [w, w+1) * total / active of the line, so every workgroup has the same amount
// of work whatever the lengths are, and at most two items of a workgroup are
// shared with others: the one that its part begins within (its fragment goes to
// place 2w of the workspace) and the one that it ends within (place 2w + 1).
// k_attn_join adds the fragments of a shared item in order of w.
#pragma once

#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {

constexpr int kItemCost = 64;  // keys' worth of an item's own work

struct AttnSched {
  long long total;   // length of the line over all layers
  long long layer;   // over one layer
  int active;        // workgroups that take part
};

// A shared item as its first workgroup describes it for the join: last = -1 if
// there is none.
struct AttnJoin {
  int last;        // last workgroup with a fragment
  int rows;        // rows of the tile
  int row0;        // first row of the tile within the sequence's rows
  int tok0;        // first token of the sequence
  int layer, head;
};

// One item, and where it lies.
struct AttnItem {
  int layer, b, h, tile;
  long long at, cost;  // start on the line, length
  KvSpan span;
};

template <int R>
struct AttnLine {
  // Cost of the first i tiles of one head: with c = ctx + kItemCost,
  // sum over tiles of (c + tokens up to the tile's end).
  static __device__ __forceinline__ long long upto(const KvSpan& r, int G, int i) {
    return static_cast<long long>(i) * (r.ctx + kItemCost) +
           static_cast<long long>(R) * i * (i + 1) / (2 * G);
  }
  static __device__ __forceinline__ int tiles(const KvSpan& r, int G) {
    return static_cast<int>((static_cast<long long>(r.n) * G + R - 1) / R);
  }
  static __device__ __forceinline__ long long sequence(const KvSpan& r, int G, int H) {
    return H * upto(r, G, tiles(r, G));
  }
};

// a * b / c, rounded the same way for everyone who asks: monotone in a, 0 at
// a = 0 and b at a = c.
__device__ __forceinline__ long long part_of(long long a, long long b, long long c) {
  if (a >= c) return b;
  return static_cast<long long>(static_cast<double>(a) * static_cast<double>(b) /
                                static_cast<double>(c));
}

template <int NT>
__device__ __forceinline__ long long sched_scan(long long v, long long* lds, long long& total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const long long o = __shfl_up(v, off, kWave);
    if (lane >= off) v += o;
  }
  __syncthreads();
  if (lane == kWave - 1) lds[wave] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w) {
    if (w < wave) before += lds[w];
    total += lds[w];
  }
  return v + before;
}

// The line's length, and the sequence and place where this workgroup's part
// begins.  lds: NT/64 + 2 long longs.  Every thread returns the same values.
struct AttnStart {
  AttnSched s;
  long long lo, hi;  // this workgroup's part; empty if it has none
  int layer, b;      // of the first item
  long long seq_at;  // where sequence b begins
};

template <int R, int NT>
__device__ AttnStart attn_start(const AttnArgs& p, int G, int wg, int n_wg, long long grain,
                                long long* lds) {
  const KvBatch& k = p.k;
  const int tid = threadIdx.x;
  long long* found = lds + NT / kWave;
  long long sum = 0, v = 0, upto = 0;
  bool bad = false;
  for (int c = 0; c < k.B; c += NT) {
    v = 0;
    if (c + tid < k.B) {
      const KvSpan r = kv_span(k, c + tid);
      bad |= !r.ok;
      v = AttnLine<R>::sequence(r, G, p.Hkv);
    }
    long long total;
    upto = sum + sched_scan<NT>(v, lds, total);
    sum += total;
  }
  if (bad && wg == 0 && p.dev_err) atomicOr(p.dev_err, GDN_DEV_ERR_LENGTH);
  AttnStart a;
  a.s.layer = sum;
  a.s.total = sum * p.L;
  const long long want = (a.s.total + grain - 1) / grain;
  a.s.active = static_cast<int>(want < n_wg ? want : n_wg);
  a.lo = a.hi = 0;
  a.layer = a.b = 0;
  a.seq_at = 0;
  if (wg >= a.s.active) return a;
  a.lo = part_of(wg, a.s.total, a.s.active);
  a.hi = part_of(wg + 1, a.s.total, a.s.active);
  a.layer = static_cast<int>(a.lo / sum);
  const long long x = a.lo - a.layer * sum;
  if (k.B <= NT) {  // the one chunk is still in registers
    if (upto - v <= x && x < upto) {
      found[0] = tid;
      found[1] = upto - v;
    }
  } else {
    long long before = 0;
    for (int c = 0; c < k.B; c += NT) {
      v = 0;
      if (c + tid < k.B) v = AttnLine<R>::sequence(kv_span(k, c + tid), G, p.Hkv);
      long long total;
      upto = before + sched_scan<NT>(v, lds, total);
      if (upto - v <= x && x < upto) {
        found[0] = c + tid;
        found[1] = upto - v;
      }
      before += total;
    }
  }
  __syncthreads();
  a.b = static_cast<int>(found[0]);
  a.seq_at = a.layer * sum + found[1];
  return a;
}

// The item at place x of the line, x within the sequence (layer, b) that begins
// at seq_at.
template <int R>
__device__ AttnItem attn_item(const AttnArgs& p, int G, int layer, int b, long long seq_at,
                              long long x) {
  AttnItem it;
  it.layer = layer;
  it.b = b;
  it.span = kv_span(p.k, b);
  const int nt = AttnLine<R>::tiles(it.span, G);
  const long long head = AttnLine<R>::upto(it.span, G, nt);
  const long long off = x - seq_at;
  it.h = static_cast<int>(off / head);
  const long long in = off - it.h * head;
  int lo = 0, hi = nt - 1;  // the last tile that begins at or before `in`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (AttnLine<R>::upto(it.span, G, mid) <= in)
      lo = mid;
    else
      hi = mid - 1;
  }
  it.tile = lo;
  const long long a = AttnLine<R>::upto(it.span, G, lo);
  it.at = seq_at + it.h * head + a;
  it.cost = AttnLine<R>::upto(it.span, G, lo + 1) - a;
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
