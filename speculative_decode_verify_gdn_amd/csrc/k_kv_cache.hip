// k_kv_cache.hip -- the paged key/value cache of a hybrid stack's attention
// layers, for gfx950: pages and slots for a round's new tokens (k_kv_reserve),
// their keys and values written into the slots (k_kv_append), and the end of a
// round (k_kv_commit).
//
// Pages are counted on the device because the lengths are only known there:
// a sequence of len tokens holds ceil(len / page) pages, and its new ones are
// found by a prefix sum over the batch.  No atomics take part in that, so the
// same inputs give the same pages every time.

#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {
namespace {

constexpr int kNT = 256;

// Inclusive prefix sum over the workgroup's kNT threads, and the total.
__device__ __forceinline__ long long block_scan(long long v, long long* lds, long long& total) {
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
  for (int w = 0; w < kNT / kWave; ++w) {
    if (w < wave) before += lds[w];
    total += lds[w];
  }
  return v + before;
}

// Pages a sequence holds (have) and will hold with its new tokens (want).
struct Need {
  int have, want;
};
__device__ __forceinline__ Need kv_need(const KvBatch& k, const KvSpan& r) {
  return {kv_blocks(k, r.ctx), kv_blocks(k, r.ctx + r.n)};
}

// One workgroup per (sequence, kChunk new tokens).  Each finds the pages taken
// by the sequences before its own from the lengths (a few loads per thread: a
// batch of 256 is one step), so no workgroup waits for another and the call is
// one launch; the last sequence's workgroup sees the whole batch and writes
// what is left.  Latency is all there is to it: 5 us of kernel, for 32 sequences of
// 8 drafts as for 256 of up to 2,048 tokens (a call through the binding takes 10 us).
constexpr int kChunk = 2048;

// Slot -1 for every row that lies in no well-formed sequence.  With the starts as
// they should be these are the rows before the first and behind the last one.  If any
// sequence is left out they may lie anywhere, so all rows are looked at, kClaimRows at
// a time: the sequences mark theirs, and those without a mark are cleared (no row of a
// sequence, which its own workgroup writes).  `odd` is uniform.  It costs such a call
// 5 us for 256 sequences of 17,000 rows together, 150 for three of 120,000.
constexpr int kClaimRows = 65536;
__device__ void clear_rows_of_none(const KvBatch& k, int32_t* slots, bool odd) {
  __shared__ uint32_t claimed[kClaimRows / 32];
  const int tid = threadIdx.x;
  if (!odd) {
    const int lo = k.q_start ? k.q_start[0] : 0, hi = k.q_start ? k.q_start[k.B] : k.B * k.T;
    for (int i = tid; i < lo; i += kNT) slots[i] = -1;
    for (int i = hi + tid; i < k.N; i += kNT) slots[i] = -1;
    return;
  }
  for (int base = 0; base < k.N; base += kClaimRows) {
    const int end = min(base + kClaimRows, k.N);
    for (int i = tid; i < kClaimRows / 32; i += kNT) claimed[i] = 0;
    __syncthreads();
    for (int s = tid; s < k.B; s += kNT) {
      const KvSpan r = kv_rows(k, s);
      const int lo = max(r.s, base) - base, hi = min(r.s + r.n, end) - base;
      for (int w = lo / 32; r.n > 0 && w * 32 < hi; ++w) {
        const int a = max(lo - w * 32, 0), e = min(hi - w * 32, 32);  // bits a .. e-1
        atomicOr(&claimed[w], (~0u >> (32 - (e - a))) << a);
      }
    }
    __syncthreads();
    for (int i = base + tid; i < end; i += kNT)
      if (!((claimed[(i - base) / 32] >> (i & 31)) & 1)) slots[i] = -1;
    __syncthreads();
  }
}

__global__ __launch_bounds__(kNT) void k_kv_reserve(KvReserveArgs p) {
  __shared__ long long lds[kNT / kWave];
  __shared__ long long sh_before;
  const KvBatch& k = p.k;
  const int b = blockIdx.x, tid = threadIdx.x;
  const KvSpan me = kv_span(k, b);
  const int first = blockIdx.y * kChunk;
  if (first > 0 && first >= me.n) return;
  const int raw_free = *p.n_free;
  const bool free_ok = raw_free >= 0 && raw_free <= k.n_pages;
  const long long n_free = free_ok ? raw_free : 0;
  long long carry = 0;
  long long taken = 0;  // pages of the served sequences among this thread's
  bool odd = false;     // one of them is left out
  for (int c = 0; c <= b; c += kNT) {
    const int s = c + tid;
    int need = 0;
    if (s <= b) {
      const KvSpan r = kv_span(k, s);
      const Need n = kv_need(k, r);
      need = n.want - n.have;
      odd |= !r.ok;
    }
    long long total;
    const long long upto = carry + block_scan(need, lds, total);
    if (s == b) sh_before = upto - need;
    if (upto <= n_free) taken += need;
    carry += total;
  }
  __syncthreads();
  const Need nd = kv_need(k, me);
  const long long before = sh_before;
  const int need = nd.want - nd.have;
  const bool served = need == 0 || before + need <= n_free;
  int err = 0;
  if (first == 0 && tid == 0) {
    if (!me.ok) err |= GDN_DEV_ERR_LENGTH;
    if (!served || !free_ok) err |= GDN_DEV_ERR_NO_PAGES;
  }
  // page of block j, or -1
  auto page_of = [&](int j) {
    int pg;
    if (j < nd.have)
      pg = p.block_table[static_cast<size_t>(b) * k.max_blocks + j];
    else
      pg = p.free_pages[n_free - 1 - before - (j - nd.have)];
    if (pg < 0 || pg >= k.n_pages) {
      err |= GDN_DEV_ERR_PAGE;
      pg = -1;
    }
    return pg;
  };
  if (served && first == 0)
    for (int j = nd.have + tid; j < nd.want; j += kNT)
      p.block_table[static_cast<size_t>(b) * k.max_blocks + j] = page_of(j);
  const int end = me.n < first + kChunk ? me.n : first + kChunk;
  for (int i = first + tid; i < end; i += kNT) {
    int slot = -1;
    if (served) {
      const int at = me.ctx + i;
      const int pg = page_of(at >> k.page_shift);
      if (pg >= 0) slot = (pg << k.page_shift) + (at & ((1 << k.page_shift) - 1));
    }
    p.slots[me.s + i] = slot;
  }
  if (first == 0 && !me.ok) {  // rows in order, but not the length
    const KvSpan r = kv_rows(k, b);
    for (int i = tid; i < r.n; i += kNT) p.slots[r.s + i] = -1;
  }
  if (first == 0 && b == k.B - 1) {
    long long total;
    block_scan(taken + (odd ? 1LL << 40 : 0), lds, total);  // taken <= n_free < 2^31
    if (tid == 0) *p.n_left = static_cast<int32_t>(n_free - (total & 0xffffffffLL));
    clear_rows_of_none(k, p.slots, total >> 40 != 0);
  }
  if (err && p.dev_err) atomicOr(p.dev_err, err);
}

// Copy-bound: every byte of k and v is read once and written once.  A
// workgroup takes 64 tokens of one key head.  Keys are copied in 16-byte
// pieces.  Values change their order: the eight tokens of a channel lie side by
// side in the cache, so lanes take tokens and each lane writes its 16 bytes of
// channels one by one: eight lanes complete a piece, and the L2 the lines.  17,000
// tokens of 4 heads of 128 channels (bf16): 16.4 us, 3.9 TB/s of the 4.8 that a
// copy reaches; 256 tokens 6 us, which is latency.
template <typename T, int D>
__global__ __launch_bounds__(kNT) void k_kv_append(KvAppendArgs p) {
  constexpr int E = 16 / sizeof(T);  // elements of a 16-byte piece
  __shared__ int slot[64];
  const int h = blockIdx.y % p.H, l = blockIdx.y / p.H;
  const int t0 = blockIdx.x * 64, tid = threadIdx.x;
  const int total = p.n_pages << p.page_shift, ps = 1 << p.page_shift;
  if (tid < 64) {
    int s = t0 + tid < p.N ? p.slots[t0 + tid] : -1;
    if (s < -1 || s >= total) {
      if (p.dev_err) atomicOr(p.dev_err, GDN_DEV_ERR_PAGE);
      s = -1;
    }
    slot[tid] = s;
  }
  __syncthreads();
  const size_t head = static_cast<size_t>(ps) * D;  // elements of a page's head
  T* kc = static_cast<T*>(p.k_cache) + static_cast<size_t>(l) * p.n_pages * p.H * head + h * head;
  T* vc = static_cast<T*>(p.v_cache) + static_cast<size_t>(l) * p.n_pages * p.H * head + h * head;
  const T* k = static_cast<const T*>(p.k) + static_cast<size_t>(l) * p.N * p.k_ld + h * D;
  const T* v = static_cast<const T*>(p.v) + static_cast<size_t>(l) * p.N * p.v_ld + h * D;
  for (int i = tid; i < 64 * (D / E); i += kNT) {
    const int t = i / (D / E), c = i % (D / E), s = slot[t];
    if (s < 0) continue;
    const u32x4 x = *reinterpret_cast<const u32x4*>(k + (t0 + t) * p.k_ld + c * E);
    *reinterpret_cast<u32x4*>(kc + static_cast<size_t>(s >> p.page_shift) * p.H * head +
                              (s & (ps - 1)) * D + c * E) = x;
  }
  const int t = tid % 64, s = slot[t];
  if (s < 0) return;
  const int off = s & (ps - 1);
  T* vd = vc + static_cast<size_t>(s >> p.page_shift) * p.H * head + (off / 8) * (D * 8) + off % 8;
  for (int c = tid / 64; c < D / E; c += kNT / 64) {
    T e[E];
    *reinterpret_cast<u32x4*>(e) = *reinterpret_cast<const u32x4*>(v + (t0 + t) * p.v_ld + c * E);
#pragma unroll
    for (int i = 0; i < E; ++i) vd[(c * E + i) * 8] = e[i];
  }
}

// One workgroup per (sequence, layer) puts the accepted path's rows into the
// slots of the first tokens, read from the round's k and v, so that no copy
// depends on another; one more workgroup counts lengths and pages.  The two
// touch nothing in common.  A wave has several rows of a head on their way at once.
// A row of k is a few 16-byte pieces, a lane each.  A row of v lies in the cache with
// 8 slots between two channels, so neighbouring lanes take neighbouring channels
// and a store touches as few lines as it can (64 trees over ten layers: 29 us with
// 16-byte pieces of v, 25 so, 12 with the pages dealt out as below.  The copies of 12
// MB take those 12 by themselves, the counts 5: loads of the path, its slots and its
// rows that wait for each other, and 2-byte stores 16 bytes apart).
template <typename T, int D>
__device__ void commit_rows(const KvCommitArgs& p, int b, int l) {
  constexpr int E = 16 / sizeof(T);   // elements of a piece
  constexpr int P = D / E;            // pieces of a row
  constexpr int RW = kWave / P;       // rows of a wave
  constexpr int C = D / kWave;        // channels of v of a lane
  const KvBatch& k = p.k;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const KvSpan r = kv_rows(k, b);
  const int n = p.n_keep[b];
  if (n <= 0 || n > r.n) return;  // n <= T <= 64: a wave holds the path
  int node = lane < n ? p.path[static_cast<size_t>(b) * k.T + lane] : 0;
  int slot = lane < n ? p.slots[r.s + lane] : -1;
  if (__any(node < 0 || node >= r.n)) return;
  if (__shfl(slot, 0, kWave) < 0) return;  // not served: commit_counts keeps nothing of it
  if (slot >= k.n_pages << k.page_shift) slot = -1;
  const int ps = 1 << k.page_shift;
  const size_t head = static_cast<size_t>(ps) * D;
  const size_t layer = static_cast<size_t>(l) * k.n_pages * p.H * head;
  const T* kk = static_cast<const T*>(p.kk) + static_cast<size_t>(l) * k.N * p.k_ld;
  const T* vv = static_cast<const T*>(p.vv) + static_cast<size_t>(l) * k.N * p.v_ld;
  T* kc = static_cast<T*>(p.k_cache) + layer;
  T* vc = static_cast<T*>(p.v_cache) + layer;
  const int c = lane % P * E, rows = n * p.H;
  for (int i0 = wave * RW; i0 < rows; i0 += kNT / kWave * RW) {
    T vx[RW][C];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int i = min(i0 + j, rows - 1), h = i / n;
      const int from = __shfl(node, i - h * n, kWave);
      const T* src = vv + (r.s + from) * p.v_ld + h * D + lane * C;
#pragma unroll
      for (int e = 0; e < C; ++e) vx[j][e] = src[e];
    }
    const int i = min(i0 + lane / P, rows - 1), h = i / n;  // the last row may be done twice
    const int from = __shfl(node, i - h * n, kWave), s = __shfl(slot, i - h * n, kWave);
    const u32x4 kx = *reinterpret_cast<const u32x4*>(kk + (r.s + from) * p.k_ld + h * D + c);
    if (s >= 0)
      *reinterpret_cast<u32x4*>(kc + (static_cast<size_t>(s >> k.page_shift) * p.H + h) * head +
                                static_cast<size_t>(s & (ps - 1)) * D + c) = kx;
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int i = min(i0 + j, rows - 1), h = i / n;
      const int s = __shfl(slot, i - h * n, kWave);
      if (s < 0) continue;
      const int off = s & (ps - 1);
      T* dst = vc + (static_cast<size_t>(s >> k.page_shift) * p.H + h) * head +
               static_cast<size_t>(off / 8) * (D * 8) + off % 8 + lane * C * 8;
#pragma unroll
      for (int e = 0; e < C; ++e) dst[e * 8] = vx[j][e];
    }
  }
}

__device__ void commit_counts(const KvCommitArgs& p) {
  __shared__ long long lds[kNT / kWave];
  const KvBatch& k = p.k;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int raw_left = *p.n_left;
  const bool left_ok = raw_left >= 0 && raw_left <= k.n_pages;
  long long top = left_ok ? raw_left : 0;
  int err = !left_ok && tid == 0 ? GDN_DEV_ERR_NO_PAGES : 0;
  for (int c = 0; c < k.B; c += kNT) {
    const int b = c + tid;
    int from = 0, to = 0;  // blocks that go back
    if (b < k.B) {
      const KvSpan r = kv_span(k, b);
      int keep = p.n_keep[b];
      bool served = r.ok;
      if (!r.ok) {
        err |= GDN_DEV_ERR_LENGTH;
        keep = 0;
      } else {
        if (keep < 0 || keep > r.n) {
          err |= GDN_DEV_ERR_N_KEEP;
          keep = 0;
        }
        if (r.n > 0 && p.slots[r.s] < 0) {
          served = false;
          if (keep > 0) err |= GDN_DEV_ERR_NO_PAGES;
          keep = 0;
        }
        if (p.path) {
          const int32_t* path = p.path + static_cast<size_t>(b) * k.T;
          bool bad = false;
          for (int i = 0; i < keep; i += 8)  // loads that wait for no other
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int node = path[min(i + j, keep - 1)];
              bad |= node < 0 || node >= r.n;
            }
          if (bad) {
            err |= GDN_DEV_ERR_PATH;
            keep = 0;
          }
        }
      }
      if (r.ok) {
        const bool ends = p.done && p.done[b] != 0;
        const int len = ends ? 0 : r.ctx + keep;
        from = kv_blocks(k, len);
        to = kv_blocks(k, served ? r.ctx + r.n : r.ctx);
        p.seq_len_out[b] = len;
      } else if (p.seq_len_out != k.seq_len) {
        p.seq_len_out[b] = k.seq_len[b];
      }
    }
    long long total;
    const long long upto = block_scan(to - from, lds, total);
    // a wave deals its sequences' pages out to its lanes, one each at a time:
    // sixty-four trees give one or two pages each, a sequence that ends thousands
    // (64 trees of 64 tokens, ten layers: a sequence at a time 25 us, so 12 us)
    const long long first = __shfl(upto - (to - from), 0, kWave);  // of the wave
    const long long mine = upto - first, all = __shfl(mine, kWave - 1, kWave);
    for (long long q0 = 0; q0 < all; q0 += kWave) {
      const long long q = min(q0 + lane, all - 1);  // the last page may be done twice
      int who = 0;  // the first sequence whose pages end behind q
#pragma unroll
      for (int step = kWave / 2; step; step /= 2)
        if (__shfl(mine, who + step - 1, kWave) <= q) who += step;
      const int e = __shfl(to, who, kWave);
      const long long end = __shfl(mine, who, kWave);
      const int j = e - static_cast<int>(end - q);
      const int pg = p.block_table[static_cast<size_t>(c + tid - lane + who) * k.max_blocks + j];
      if (pg < 0 || pg >= k.n_pages) err |= GDN_DEV_ERR_PAGE;
      if (top + first + q < k.n_pages)
        p.free_pages[top + first + q] = pg;
      else
        err |= GDN_DEV_ERR_NO_PAGES;
    }
    top += total;
  }
  __syncthreads();  // every thread has read n_left
  if (tid == 0) *p.n_free = static_cast<int32_t>(top < k.n_pages ? top : k.n_pages);
  if (err && p.dev_err) atomicOr(p.dev_err, err);
}

template <typename T, int D>
__global__ __launch_bounds__(kNT) void k_kv_commit(KvCommitArgs p) {
  if (blockIdx.x == 0) {
    commit_counts(p);
    return;
  }
  const int u = blockIdx.x - 1;
  commit_rows<T, D>(p, u % p.k.B, u / p.k.B);
}

template <typename T, int D>
hipError_t append_t(const KvAppendArgs& a, hipStream_t s) {
  k_kv_append<T, D><<<dim3((a.N + 63) / 64, a.L * a.H), kNT, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t commit_t(const KvCommitArgs& a, hipStream_t s) {
  const unsigned rows = a.path ? static_cast<unsigned>(a.L) * a.k.B : 0u;
  k_kv_commit<T, D><<<1 + rows, kNT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_reserve(const KvReserveArgs& a, hipStream_t s) {
  k_kv_reserve<<<dim3(a.k.B, (a.k.T + kChunk - 1) / kChunk), kNT, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a, int head_dim, int dtype, hipStream_t s) {
  if (dtype == 1) {
    if (head_dim == 64) return append_t<uint16_t, 64>(a, s);
    if (head_dim == 128) return append_t<uint16_t, 128>(a, s);
    if (head_dim == 256) return append_t<uint16_t, 256>(a, s);
  } else {
    if (head_dim == 64) return append_t<float, 64>(a, s);
    if (head_dim == 128) return append_t<float, 128>(a, s);
    if (head_dim == 256) return append_t<float, 256>(a, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_kv_commit(const KvCommitArgs& a, int head_dim, int dtype, hipStream_t s) {
  if (dtype == 1) {
    if (head_dim == 64) return commit_t<uint16_t, 64>(a, s);
    if (head_dim == 128) return commit_t<uint16_t, 128>(a, s);
    if (head_dim == 256) return commit_t<uint16_t, 256>(a, s);
  } else {
    if (head_dim == 64) return commit_t<float, 64>(a, s);
    if (head_dim == 128) return commit_t<float, 128>(a, s);
    if (head_dim == 256) return commit_t<float, 256>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
