// k_attn.hip -- attention of a round's new tokens over the paged cache, for
// gfx950 (attn_verify).
//
//   o_r = sum_j softmax_j(scale * q_r . k_j) v_j
//
// in one pass over the keys with the running maximum m, sum l and output O of
// each row: a step with scores s rescales l and O by exp(m - m') and adds
// exp(s - m') (times v).  Two such triples over disjoint keys join the same way
// (the waves of a workgroup, then the fragments of an item).  No triple is left out of
// a sum, whatever its weight: an infinity in its O must reach the row (0 * inf is NaN).
// Only a row whose whole l is 0, all its scores -inf, is written as 0.
//
// Everything is computed transposed, S^T = K Q^T and O^T = V^T P^T, so that a
// lane owns one query row: its column of a 16x16 result tile.  Maximum, sum
// and rescaling are then per lane, and the exponentials of S^T are, in the
// registers where they lie, the B operand of the second product: the key that
// a result row stands for is free to choose, and is chosen so that a lane's
// eight probabilities belong to eight consecutive keys, which the value cache
// stores side by side.  No operand is shuffled between lanes.
//
// Three kernels.  Few rows (k_attn_stream): keys and values go from the cache to
// registers and are used once; their bytes bound it.  Many rows in
// bf16 (k_attn_tile): they pass through LDS, where several waves read them, and
// the matrix products bound it.  k_attn_join adds up the items that workgroups
// share.
//
// Rounding: scores, maxima, sums and outputs are fp32, and the sum l takes every
// probability as it is.  As an operand beside bf16 values a probability becomes the
// bf16 nearest to it and, in a second product, the bf16 nearest to what is left
// (2^-16 of it), so that the output's own rounding is the only one that shows:
// 0.0017 of the result, as with probabilities in fp32.  The bytes that bound the
// kernels of up to 64 rows hide nearly all of that (24 long contexts 89.1 and 90.3 us
// without and with it, drafts 63.6 and 64.0).  Tiles of 128 rows are bound by their
// products and take the first operand alone, off by 2^-8 of it (0.0023 of the result):
// with both, the prompts take 850 us instead of 612, the trees 208 instead of 178.

#include <type_traits>

#include "attn_sched.hpp"
#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 8.f;

// ---- element types: 32 keys of K and V as MFMA operands

template <typename T>
struct Frag;

// bf16, v_mfma_f32_16x16x32_bf16.  Result row m of score tile t (0, 1) is key
// 8 (m / 4) + 4 t + m % 4 of the 32, so lane group g holds keys 8g .. 8g+7.
template <>
struct Frag<uint16_t> {
  static constexpr int kPerK = 32;  // channels of one score product
  static constexpr int kPad = 8;    // of a Q row in LDS
  typedef bf16x8 K;                 // 8 channels of a key
  typedef bf16x8 V;                 // 8 keys of a channel
  static constexpr int kVLoads = 1;
  // An exponent of all ones, plus one in its last place, carries into the sign.
  static constexpr uint32_t kExp = 0x7f807f80u, kOne = 0x00800080u, kTop = 0x80008000u;
  static __device__ __forceinline__ uint32_t spread(uint32_t top) { return (top >> 15) * 0xffffu; }
  // The words of 8 keys of which the bits say which to keep.
  static __device__ __forceinline__ u32x4 keep(uint32_t there) {
    u32x4 m;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[j] = ((there >> (2 * j)) & 1) * 0xffffu + ((there >> (2 * j + 1)) & 1) * 0xffff0000u;
    return m;
  }
  static __device__ __forceinline__ int key_of(int t, int g, int i) { return 8 * g + 4 * t + i; }
  // the key whose row lane c feeds to tile t
  static __device__ __forceinline__ int row_key(int t, int c) {
    return 8 * (c >> 2) + 4 * t + (c & 3);
  }
  static __device__ __forceinline__ floatx4 score(K k, K q, floatx4 s) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q, s, 0, 0, 0);
  }
};

// fp32, v_mfma_f32_16x16x4_f32: four products per 16-byte load, product i of
// channels 16 j + 4 g + i; result row m of tile t is key 16 t + m, so lane
// group g holds keys 16 t + 4g .. 4g+3.
template <>
struct Frag<float> {
  static constexpr int kPerK = 16;
  static constexpr int kPad = 4;
  typedef floatx4 K;
  typedef floatx4 V;
  static constexpr int kVLoads = 2;
  static constexpr uint32_t kExp = 0x7f800000u, kOne = 0x00800000u, kTop = 0x80000000u;
  static __device__ __forceinline__ uint32_t spread(uint32_t top) { return (top >> 31) * ~0u; }
  static __device__ __forceinline__ u32x4 keep(uint32_t there) {
    u32x4 m;
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = ((there >> j) & 1) * ~0u;
    return m;
  }
  static __device__ __forceinline__ int key_of(int t, int g, int i) { return 16 * t + 4 * g + i; }
  static __device__ __forceinline__ int row_key(int t, int c) { return 16 * t + c; }
  static __device__ __forceinline__ floatx4 score(K k, K q, floatx4 s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x4f32(k[i], q[i], s, 0, 0, 0);
    return s;
  }
};

// O^T += V^T P^T over 32 keys; p[t] holds tile t's probabilities.
__device__ __forceinline__ floatx4 weigh(const bf16x8* v, const floatx4* p, floatx4 o) {
  bf16x8 w, rest;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = p[i / 4][i % 4];
    w[i] = static_cast<__bf16>(x);
    rest[i] = static_cast<__bf16>(x - static_cast<float>(w[i]));
  }
  o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], w, o, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], rest, o, 0, 0, 0);
}
__device__ __forceinline__ floatx4 weigh(const floatx4* v, const floatx4* p, floatx4 o) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o = __builtin_amdgcn_mfma_f32_16x16x4f32(v[t][i], p[t][i], o, 0, 0, 0);
  return o;
}

__device__ __forceinline__ bool not_finite(float x) {
  return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ uint16_t to_out(float x, uint16_t) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ float to_out(float x, float) { return x; }

// Over the four lanes that hold a row's keys (c, c+16, c+32, c+48): halves
// exchanged, then rows of 16.
__device__ __forceinline__ floatx2 swap32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return floatx2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ floatx2 swap16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return floatx2{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
// x, as far as the compiler knows any number: what is computed from it is not
// moved out of a rare branch into registers that the loop around it needs.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ float row_max(float x) {
  const floatx2 a = swap32(x);
  const floatx2 b = swap16(fmaxf(a[0], a[1]));
  return fmaxf(b[0], b[1]);
}
__device__ __forceinline__ float row_sum(float x) {
  const floatx2 a = swap32(x);
  const floatx2 b = swap16(a[0] + a[1]);
  return b[0] + b[1];
}

// Ancestors (and self) of every node of a sequence's tree, as bits; false if
// the array is malformed.  lds: 64 masks and one flag.
struct TreeLds {
  uint64_t mask[64];
  int parent[64];
  int bad;
};
__device__ bool tree_masks(const int32_t* parent, int n, TreeLds& t) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) t.bad = 0;
  __syncthreads();
  if (tid < n) {
    const int q = parent[tid];
    t.parent[tid] = q;
    if (q < -1 || q >= tid) t.bad = 1;
  }
  __syncthreads();
  if (t.bad) return false;
  if (tid < n) {
    uint64_t m = 0;
    for (int u = tid; u >= 0; u = t.parent[u]) m |= 1ull << u;
    t.mask[tid] = m;
  }
  __syncthreads();
  return true;
}

// Fragments in the workspace: 2 n_wg places of R rows of D sums, then of R
// (m, l) pairs, then n_wg descriptions for the join.  Between places lie 256 bytes
// more: the join reads the same row of many of them, and at a distance of a power
// of two they would all come from one memory channel (61 to 92 us for one sequence
// of 60,000 keys and 64 rows).
template <int R, int D>
struct Places {
  static constexpr size_t kPlace = static_cast<size_t>(R) * D + 64;
  float* o;
  floatx2* ml;
  AttnJoin* join;
  __device__ __host__ Places(void* ws, int n_wg) {
    o = static_cast<float*>(ws);
    ml = reinterpret_cast<floatx2*>(o + 2 * n_wg * kPlace);
    join = reinterpret_cast<AttnJoin*>(ml + static_cast<size_t>(2 * n_wg) * R);
  }
  __device__ __forceinline__ float* row(int place, int r) const {
    return o + place * kPlace + static_cast<size_t>(r) * D;
  }
};
size_t places_bytes(int rows, int head_dim, int n_wg) {
  return static_cast<size_t>(2 * n_wg) * ((static_cast<size_t>(rows) * head_dim + 64) * 4 + rows * 8) +
         static_cast<size_t>(n_wg) * sizeof(AttnJoin);
}

// What a row sees of `count` consecutive keys from `base` on, as bits: in a
// chain the keys below lim; in a tree the cached ones (below ctx) and those of
// its ancestors, whose bits `mask` holds from ctx on.
__device__ __forceinline__ uint32_t chain_sees(int lim, int base, int count) {
  return (1u << min(max(lim - base, 0), count)) - 1u;
}
__device__ __forceinline__ uint32_t tree_sees(uint64_t mask, int ctx, int base, int count) {
  const int in = base - ctx;  // place among the new tokens
  uint64_t m = in >= 64 ? 0 : in >= 0 ? mask >> in : in <= -32 ? ~0ull : ~(~mask << -in);
  return static_cast<uint32_t>(m) & ((1u << count) - 1u);
}

// Token of row `row` of a tile that begins `skip` rows into token 0 of it, with
// inv = 1/G: exact for the small numbers at hand (skip + row < 2^17).
__device__ __forceinline__ int tile_token(int skip, int row, float inv) {
  return static_cast<int>((static_cast<float>(skip + row) + 0.5f) * inv);
}

// ---- few query rows: the waves of a workgroup take different keys
//
// R = 16 NT rows; each wave streams 32 keys at a time straight from the cache
// into MFMA operands (no LDS, no barrier until the item ends) and keeps all the
// rows' sums.  32 query heads of 24 contexts of 500 to 32,000 tokens, 4 key heads
// of 128 channels: 81 us, 5.0 TB/s; a large copy reaches 4.8.  A single short sequence is
// latency: 10 us for 800 tokens.
template <typename T, int D, int NT>
struct Stream {
  static constexpr int W = 4;            // waves
  static constexpr int R = 16 * NT;
  static constexpr int kStep = 32 * W;   // keys of one step of the workgroup
  static constexpr int QLD = D + Frag<T>::kPad;
  static constexpr int kC = D < 128 ? D : 128;  // channels joined at a time
  // (24 long contexts in bf16: 89 us with 64, 86 with 128; 16 in 32 bits, whose keys
  // take longer: 27.4 and 28.5)
  typedef AttnLine<R, sizeof(T) == 2 ? 128 : 64> Line;
  struct Lds {
    union {  // one after the other
      T q[R * QLD];
      float join[W][R][kC + 4];
    };
    float m[W][R], l[W][R], inv[R];
    TreeLds tree;
    int any_odd;
  };
};

template <typename T, int D, int NT>
__global__ __launch_bounds__(256, 1) void k_attn_stream(AttnArgs p, int n_wg, long long grain) {
  using St = Stream<T, D, NT>;
  using Line = typename St::Line;
  using F = Frag<T>;
  constexpr int W = St::W, R = St::R, QLD = St::QLD;
  constexpr int KJ = D / F::kPerK;  // score products per tile
  constexpr int MT = D / 16;        // output tiles
  constexpr int VE = 16 / sizeof(T);  // keys of a V operand
  __shared__ typename St::Lds sh;
  const KvBatch& k = p.k;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, g = lane / 16;
  const int G = p.Hq / p.Hkv;
  const float inv_g = 1.f / static_cast<float>(G);
  const Places<R, D> places(p.ws, n_wg);
  // Single tokens, 512 workgroups: with 60 heads 480 take 90.5 us against 93.9 for all,
  // with 384 heads 384 take 87 against 86, with 300 heads 300 take 151 against 129.
  const AttnStart st = attn_start<Line, false>(p, G, n_wg, grain, n_wg / 4);
  const int wg = st.wg;
  AttnJoin join;
  join.last = -1;
  // scores are compared unscaled (a negative scale turns q's sign); at least
  // the smallest normal, so that a masked -inf stays -inf at scale 0
  const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 1.17549435e-38f);
  const int ps = 1 << k.page_shift;
  const size_t head_sz = static_cast<size_t>(ps) * D;
  int err = 0;

  long long x = st.lo, seq_at = st.seq_at;
  int layer = st.layer, b = st.b;
  KvSpan r = st.span;
  while (x < st.hi) {
    const AttnItem it = attn_item<Line>(p, G, layer, b, r, seq_at, x);
    const long long end = it.at + it.cost;
    const long long till = end < st.hi ? end : st.hi;
    const int row0 = it.tile * R;
    const int rows = min(R, r.n * G - row0);
    const int tok_first = row0 / G;
    const int skip = row0 - tok_first * G;
    const int tok_last = tok_first + tile_token(skip, rows - 1, inv_g);
    const int len = r.ctx + (p.parent ? r.n : tok_last + 1);
    const int steps = (len + St::kStep - 1) / St::kStep;
    const int s0 = x == it.at ? 0 : uni(static_cast<int>(part_of(x - it.at, steps, it.cost)));
    const int s1 =
        till == end ? steps : uni(static_cast<int>(part_of(till - it.at, steps, it.cost)));
    const bool whole = it.at >= st.lo && end <= st.hi;
    bool good = true;
    if (p.parent) {
      good = tree_masks(p.parent + r.s, r.n, sh.tree);
      if (!good) err |= GDN_DEV_ERR_PARENT;
    }
    if (good) {
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * k.max_blocks;
      // Page numbers of 32 steps at a time, a lane each: the wave's keys of
      // step first + lane/2, the half lane%2 of them (16 keys lie in one page).
      auto pages_from = [&](int first) {
        const long long key =
            (static_cast<long long>(first) + (lane >> 1)) * St::kStep + wave * 32 + (lane & 1) * 16;
        int pg = -1;
        if (first + (lane >> 1) < s1 && key < len) {
          pg = table[key >> k.page_shift];
          if (pg < 0 || pg >= k.n_pages) {
            err |= GDN_DEV_ERR_PAGE;
            pg = -2;
          }
        }
        return pg;
      };
      int pgs = pages_from(s0), pgn = -1, batch = s0;
      // Q rows, zero behind the last one
      const T* q = static_cast<const T*>(p.q) +
                   (static_cast<size_t>(it.layer) * k.N + r.s + tok_first) * p.q_ld +
                   static_cast<size_t>(it.h) * G * D;
      constexpr int CH = D / VE;  // 16-byte pieces of a row
      constexpr int QN = (R * CH + W * kWave - 1) / (W * kWave);
      u32x4 qv[QN];
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        const int at = tid + i * W * kWave, row = at / CH, ch = at % CH;
        qv[i] = u32x4{0, 0, 0, 0};
        if (row < rows) {
          const int tok = tile_token(skip, row, inv_g), qh = skip + row - tok * G;
          qv[i] = *reinterpret_cast<const u32x4*>(q + tok * p.q_ld + qh * D + ch * VE);
        }
      }
      const T* kc = static_cast<const T*>(p.k_cache) +
                    (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const T* vc = static_cast<const T*>(p.v_cache) +
                    (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const size_t page_sz = static_cast<size_t>(p.Hkv) * head_sz;

      typename F::K kf[2][KJ];
      typename F::V vf[MT][F::kVLoads];
      int h0 = 0, h1 = 0;  // the current step's page numbers, below 0 where nothing is
      auto step_pages = [&](int s, int& a, int& e) {
        if (s - batch == 32) {
          pgs = pgn;
          batch = s;
        }
        if (s == batch) pgn = pages_from(batch + 32);
        a = __builtin_amdgcn_readlane(pgs, 2 * (s - batch));
        e = __builtin_amdgcn_readlane(pgs, 2 * (s - batch) + 1);
      };
      // Loads of a step: absent pages read page 0 and are masked afterwards.
      auto load_k = [&](int s, int a, int e) {
        const int kb = s * St::kStep + wave * 32;
        const T* b0 = kc + static_cast<size_t>(max(a, 0)) * page_sz +
                      static_cast<size_t>(kb & (ps - 1)) * D;
        const T* b1 = kc + static_cast<size_t>(max(e, 0)) * page_sz +
                      static_cast<size_t>((kb + 16) & (ps - 1)) * D;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int key = F::row_key(t, c);
          const T* row = (key < 16 ? b0 : b1) + (key & 15) * D + g * VE;
#pragma unroll
          for (int j = 0; j < KJ; ++j)
            kf[t][j] = *reinterpret_cast<const typename F::K*>(row + j * F::kPerK);
        }
      };
      auto load_v = [&](int s, int a, int e) {
        const int kb = s * St::kStep + wave * 32;
#pragma unroll
        for (int u = 0; u < F::kVLoads; ++u) {
          const int key = F::key_of(u, g, 0);  // the first of the lane's keys
          const T* base = vc + static_cast<size_t>(max(key < 16 ? a : e, 0)) * page_sz +
                          static_cast<size_t>((((kb + key) & (ps - 1)) >> 3)) * (D * 8) + (key & 7);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            vf[t][u] = *reinterpret_cast<const typename F::V*>(base + (t * 16 + c) * 8);
        }
      };
      if (s0 < s1) {
        step_pages(s0, h0, h1);
        load_k(s0, h0, h1);
        load_v(s0, h0, h1);
      }
      __syncthreads();  // the last item's LDS is free
      if (tid == 0) sh.any_odd = 0;
#pragma unroll
      for (int i = 0; i < QN; ++i) {
        const int at = tid + i * W * kWave, row = at / CH, ch = at % CH;
        if (p.scale < 0.f)
#pragma unroll
          for (int j = 0; j < 4; ++j) qv[i][j] ^= sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
        if (row < R) *reinterpret_cast<u32x4*>(&sh.q[row * QLD + ch * VE]) = qv[i];
      }
      floatx4 o[NT][MT];
      float m[NT], l[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n] = kNegInf;
        l[n] = 0.f;
#pragma unroll
        for (int t = 0; t < MT; ++t) o[n][t] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      for (int s = s0; s < s1; ++s) {
        const int kb = s * St::kStep + wave * 32;
        const int a = h0, e = h1;
        floatx4 sc[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sc[n][0] = floatx4{0.f, 0.f, 0.f, 0.f};
          sc[n][1] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < KJ; ++j) {
            const typename F::K qf = *reinterpret_cast<const typename F::K*>(
                &sh.q[(n * 16 + c) * QLD + j * F::kPerK + g * VE]);
            sc[n][0] = F::score(kf[0][j], qf, sc[n][0]);
            sc[n][1] = F::score(kf[1][j], qf, sc[n][1]);
          }
        }
        if (s + 1 < s1) {
          step_pages(s + 1, h0, h1);
          load_k(s + 1, h0, h1);
        }
        // any key that some row does not see, or that is not there
        if (kb + 32 > r.ctx + (p.parent ? 0 : tok_first + 1) || a < 0 || e < 0) {
          uint32_t odd = 0;
#pragma unroll
          for (int u = 0; u < F::kVLoads; ++u) {
            // the lane's keys: base .. base + VE - 1, those of tile u (bf16: of both)
            const int first = F::key_of(u, g, 0), base = kb + first;
            const uint32_t there = (first < 16 ? a : e) < 0 ? 0u : chain_sees(len, base, VE);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int tok = tok_first + tile_token(skip, min(n * 16 + c, rows - 1), inv_g);
              const uint32_t sees =
                  there & (p.parent ? tree_sees(sh.tree.mask[tok], r.ctx, base, VE)
                                    : chain_sees(r.ctx + tok + 1, base, VE));
#pragma unroll
              for (int i = 0; i < VE; ++i) {
                const int t = VE == 8 ? i / 4 : u;
                sc[n][t][i % 4] = (sees >> i) & 1 ? sc[n][t][i % 4] : kNegInf;
              }
            }
            // Values that are not there become 0, and so do infinities and NaN:
            // 0 * inf would take them to rows that do not see them.
            const u32x4 keep = F::keep(there);
            uint32_t bad = 0;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const u32x4 w = __builtin_bit_cast(u32x4, vf[t][u]) & keep;
              vf[t][u] = __builtin_bit_cast(typename F::V, w);
#pragma unroll
              for (int j = 0; j < 4; ++j) bad |= ((w[j] & F::kExp) + F::kOne) & F::kTop;
            }
            if (__any(bad)) {
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                u32x4 w = __builtin_bit_cast(u32x4, vf[t][u]);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] &= ~F::spread(((w[j] & F::kExp) + F::kOne) & F::kTop);
                vf[t][u] = __builtin_bit_cast(typename F::V, w);
              }
              odd |= bad;
            }
          }
          if (odd) sh.any_odd = 1;  // rare: rows that do see them get them in the end
        }
        // m is the maximum so far, or a number at most kSlack below it in
        // powers of two: sums stay far from overflow and their precision is the
        // same, and the rescaling of all outputs is left out while no row's
        // maximum rises by more.
        float top[NT];
        bool rise = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float z = fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3]));
          z = fmaxf(z, fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
          top[n] = row_max(z);
          rise |= (top[n] - m[n]) * c2 > kSlack;
        }
        if (__any(rise)) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float M = fmaxf(top[n], m[n]);
            // a row that has seen no key yet has nothing to rescale
            const float back = m[n] == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m[n] - M) * c2);
            m[n] = M;
            l[n] *= back;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[n][t][i] *= back;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float at = m[n] == kNegInf ? 0.f : m[n];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = __builtin_amdgcn_exp2f((sc[n][t][i] - at) * c2);
              sc[n][t][i] = w;
              l[n] += w;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < MT; ++t) o[n][t] = weigh(vf[t], sc[n], o[n][t]);
        if (s + 1 < s1) load_v(s + 1, h0, h1);
      }

      // join the four waves: maxima and sums of every row, then the outputs of
      // kC channels at a time
      __syncthreads();  // Q's place is free for the outputs
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float sum = row_sum(l[n]);
        if (g == 0) {
          sh.m[wave][n * 16 + c] = m[n];
          sh.l[wave][n * 16 + c] = sum;
        }
      }
      __syncthreads();
      const int place = 2 * wg + (it.at < st.lo ? 0 : 1);
      const long long out =
          ((static_cast<long long>(it.layer) * k.N + r.s + tok_first) * p.Hq + it.h * G) * D;
      float mine[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sh.m[w][n * 16 + c]);
        mine[n] = m[n] == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m[n] - M) * c2);
      }
      if (tid < rows) {
        float M = kNegInf, L = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sh.m[w][tid]);
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (sh.m[w][tid] != kNegInf || sh.l[w][tid] != sh.l[w][tid])
            L += sh.l[w][tid] * __builtin_amdgcn_exp2f((sh.m[w][tid] - M) * c2);
        sh.inv[tid] = L == 0.f ? 0.f : 1.f / L;
        if (!whole) places.ml[static_cast<size_t>(place) * R + tid] = floatx2{M, L};
      }
#pragma unroll
      for (int ch = 0; ch < D / St::kC; ++ch) {
        if (ch) __syncthreads();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < St::kC / 16; ++t) {
            floatx4 v = o[n][ch * (St::kC / 16) + t];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= mine[n];
            *reinterpret_cast<floatx4*>(&sh.join[wave][n * 16 + c][t * 16 + 4 * g]) = v;
          }
        __syncthreads();
#pragma unroll 2
        for (int i = tid; i < rows * (St::kC / 4); i += W * kWave) {
          const int rr = i / (St::kC / 4), d = i % (St::kC / 4) * 4, dd = ch * St::kC + d;
          floatx4 v = *reinterpret_cast<const floatx4*>(&sh.join[0][rr][d]);
#pragma unroll
          for (int w = 1; w < W; ++w) {
            const floatx4 y = *reinterpret_cast<const floatx4*>(&sh.join[w][rr][d]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += y[j];
          }
          const int tok = tile_token(skip, rr, inv_g);
          if (sh.any_odd) {
            const int from = max(s0 * St::kStep, r.ctx & ~31), to = min(len, s1 * St::kStep);
#pragma unroll 1
            for (int key = from; key < to; ++key) {
              const bool sees = p.parent ? tree_sees(sh.tree.mask[tok_first + tok], r.ctx, key, 1)
                                         : key <= r.ctx + tok_first + tok;
              const int pg = table[key >> k.page_shift];
              if (!sees || pg < 0 || pg >= k.n_pages) continue;
              const T* e = vc + static_cast<size_t>(pg) * page_sz +
                           static_cast<size_t>((key & (ps - 1)) >> 3) * (D * 8) + dd * 8 + (key & 7);
#pragma unroll 1
              for (int j = 0; j < 4; ++j) {
                const float y = ld_in(e, j * 8);
                const float was = j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3];
                const float now = not_finite(y) ? was + y : was;
                v[0] = j == 0 ? now : v[0];
                v[1] = j == 1 ? now : v[1];
                v[2] = j == 2 ? now : v[2];
                v[3] = j == 3 ? now : v[3];
              }
            }
          }
          if (whole) {
            const float inv = sh.inv[rr];
            T* dst = static_cast<T*>(p.o) + out +
                     (static_cast<long long>(tok) * p.Hq + skip + rr - tok * G) * D + dd;
            T e4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e4[j] = to_out(inv == 0.f ? 0.f : v[j] * inv, T{});
            __builtin_memcpy(__builtin_assume_aligned(dst, 4 * sizeof(T)), e4, sizeof(e4));
          } else {
            *reinterpret_cast<floatx4*>(places.row(place, rr) + dd) = v;
          }
        }
      }
      if (!whole && it.at >= st.lo) {
        join.last = attn_owner(st.s, end - 1);
        join.rows = rows;
        join.skip = skip;
        join.out = out;
      }
    }
    x = till;
    if (x < st.hi) {  // the next item, of this sequence or of the next that has any
      long long seq_end = seq_at + Line::sequence(r, G, p.Hkv);
      while (x >= seq_end) {
        seq_at = seq_end;
        if (++b == k.B) {
          b = 0;
          ++layer;
        }
        r = kv_span(k, b);
        seq_end = seq_at + Line::sequence(r, G, p.Hkv);
      }
    }
  }
  if (tid == 0) places.join[wg] = join;
  if (err && p.dev_err) atomicOr(p.dev_err, err);
}

// ---- many query rows: the waves of a workgroup take different rows
//
// Keys pass through LDS, a tile at a time, and every wave multiplies with all of
// them.  Two forms of a wave:
//
// Rows32: 32 rows, products of v_mfma_f32_32x32x16_bf16.  Result row m = 8a + 4h + r
// (h = lane / 32; register 4a + r) stands for key 16 (a / 2) + 8h + 4 (a % 2) + r of
// its 32: then the eight registers of a = 2s, 2s + 1 are eight consecutive keys, the
// operand of product step s.
//
// Rows16: 16 rows, products of v_mfma_f32_16x16x32_bf16 and keys in the stream
// kernel's order.  An operand from LDS feeds half as many products, but a wave's
// sums and queries take half the registers.
//
// A tile of the line has 64 rows, four waves of 16, where no sequence has more;
// else 128: four waves of 32, or with 256 channels eight of 16 (with 32 rows of 256
// channels only one wave would fit on a SIMD, and it waits for every load by
// itself: 289 against 235 us for 64 trees of 64 nodes, 16 query heads).
//
// Three prompts of about 3,000 tokens behind 1,000 cached ones, 32 query heads of
// 128 channels: 580 to 640 us by card, 930 to 840 TFLOP/s; a large matrix product
// reaches 1,189.  The rest is the vector work of the softmax, which the matrix pipe
// hides in part.  64-row tiles of 32 drafted chunks: 54 us for 198 MB; the bytes alone
// take 41.  64 trees of 512 rows to a key head of 256 channels: 160 us and more, for
// which four tiles sweep the same keys, in turn and from memory: 6.0e6 L2 misses, 765
// MB in lines of 128 bytes, for 254 MB of operands.
//
// LDS: keys row by row, 16-byte pieces of a row permuted by the key so that the
// rows that are read together fall on different banks; values as in the cache,
// where an operand's channels lie in a row anyway.  While one tile is multiplied,
// the next one is loaded into another buffer, from memory to LDS without a
// register in between.
typedef float floatx16 __attribute__((ext_vector_type(16)));

// One wave's products.  A lane has one row, and of a tile's keys kGroups times
// eight consecutive ones: from kEvery * i + 8 * part on.
template <int D, int KT>
struct Rows32 {
  static constexpr int kRows = 32;
  static constexpr int kGroups = KT / 16, kEvery = 16;
  static constexpr int QJ = D / 16, DT = D / 32;  // score products, output tiles
  static constexpr int kQ = 16;                   // channels of a score product
  typedef floatx16 Acc;
  static constexpr int kAcc = 16;
  static __device__ __forceinline__ int row_key(int c) {
    return 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);
  }
  // LDS serves 16 rows at once, whose keys differ in four bits, 256 bytes (two rows
  // of 64 channels) from each other or in the same ones: 16 different pieces.
  static __device__ __forceinline__ int swizzle(int key) {
    return D == 64 ? (key >> 1) & 7 : key & 15;
  }
  static constexpr int kSwizzlePeriod = 16;  // keys after which it repeats
  static constexpr int kScoreTiles = KT / 32;
  static __device__ __forceinline__ Acc mul(bf16x8 a, bf16x8 b, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // the keys of score tile t begin here
  static __device__ __forceinline__ constexpr int tile_key(int t) { return 32 * t; }
  // score tile and register of key e of group i
  static __device__ __forceinline__ constexpr int tile_of(int i, int) { return i / 2; }
  static __device__ __forceinline__ constexpr int reg_of(int i, int e) { return 8 * (i % 2) + e; }
  // channel of register r of an output tile, behind 4 * part
  static __device__ __forceinline__ constexpr int channel(int r) { return 8 * (r / 4) + r % 4; }
  static __device__ __forceinline__ float top(float x) {
    const floatx2 a = swap32(x);
    return fmaxf(a[0], a[1]);
  }
  static __device__ __forceinline__ float sum(float x) {
    const floatx2 a = swap32(x);
    return a[0] + a[1];
  }
};

template <int D, int KT>
struct Rows16 {
  static constexpr int kRows = 16;
  static constexpr int kGroups = KT / 32, kEvery = 32;
  static constexpr int QJ = D / 32, DT = D / 16;
  static constexpr int kQ = 32;
  typedef floatx4 Acc;
  static constexpr int kAcc = 4;
  static __device__ __forceinline__ int row_key(int c) { return 8 * (c >> 2) + (c & 3); }
  // a score tile's keys differ in bits 0, 1, 3 and 4
  static __device__ __forceinline__ int swizzle(int key) {
    return D == 64 ? (key >> 1 & 1) | (key >> 2 & 6) : (key & 3) | (key >> 1 & 12);
  }
  static constexpr int kSwizzlePeriod = 32;
  static constexpr int kScoreTiles = KT / 16;
  static __device__ __forceinline__ Acc mul(bf16x8 a, bf16x8 b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ constexpr int tile_key(int t) { return t / 2 * 32 + t % 2 * 4; }
  static __device__ __forceinline__ constexpr int tile_of(int i, int e) { return 2 * i + e / 4; }
  static __device__ __forceinline__ constexpr int reg_of(int, int e) { return e % 4; }
  static __device__ __forceinline__ constexpr int channel(int r) { return r; }
  static __device__ __forceinline__ float top(float x) { return row_max(x); }
  static __device__ __forceinline__ float sum(float x) { return row_sum(x); }
};

template <int D, int ROWS>
struct Tile {
  static constexpr bool kNarrow = ROWS == 64 || D == 256;  // Rows16
  static constexpr int R = ROWS;
  static constexpr bool kRest = ROWS == 64;  // what a probability's rounding leaves counts too
  // With 256 channels and 64 rows the tile is halved: two workgroups' LDS fit on a CU.
  static constexpr int kKeys = D == 256 && ROWS == 64 ? 32 : 64;
  typedef typename std::conditional<kNarrow, Rows16<D, kKeys>, Rows32<D, kKeys>>::type Mma;
  static constexpr int W = ROWS / Mma::kRows;
  static constexpr int kPieces = D / 8;                         // 16-byte pieces of a key
  static constexpr int kLoads = kKeys * kPieces / (W * kWave);  // of a wave, K and V each
  static constexpr int kKeysPerLoad = W * kWave / kPieces;      // of the workgroup
  // (64 keys' worth for all: prompts 634 us, trees 219, drafts 63; so 605, 202, 61)
  typedef AttnLine<ROWS, ROWS == 64 ? 256 : 448> Line;
};

// 16 bytes per lane, from a uniform address and the lane's own offset in bytes to
// lane * 16 behind the wave's place.
__device__ __forceinline__ void to_lds(const char* from, uint32_t bytes, u32x4* to) {
  __builtin_amdgcn_global_load_lds(
      (const __attribute__((address_space(1))) void*)(from + bytes),
      (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
// A barrier for what the waves read from LDS: their reads have returned, and
// loads into LDS that are still under way stay so (__syncthreads would wait for
// those too).
__device__ __forceinline__ void lds_barrier() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// N products whose operands read(n) fetches from LDS kAhead products ahead, in this
// order whatever the compiler would prefer: no product waits for its operand, and
// no more registers hold operands than that.
// (Four ahead: prompts 637 us, trees 222; eight: 633 and 219.)
constexpr int kAhead = 8;
template <int N, typename Read, typename Mul>
__device__ __forceinline__ void products(Read read, Mul mul) {
  static_assert(N % kAhead == 0, "the ring comes round");
  bf16x8 f[kAhead];
#pragma unroll
  for (int n = 0; n < kAhead; ++n) f[n] = read(n);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    mul(n, f[n % kAhead]);
    if (n + kAhead < N) f[n % kAhead] = read(n + kAhead);
    __builtin_amdgcn_sched_barrier(0);
  }
}
// Until the wave's loads into LDS have arrived.
__device__ __forceinline__ void lds_loads_done() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt 0
}

template <int D, int ROWS>
__global__ __launch_bounds__((Tile<D, ROWS>::W * kWave), 2) void k_attn_tile(AttnArgs p, int n_wg,
                                                                           long long grain) {
  using Tl = Tile<D, ROWS>;
  using Line = typename Tl::Line;
  using Mm = typename Tl::Mma;
  typedef typename Mm::Acc Acc;
  using F = Frag<uint16_t>;
  constexpr int W = Tl::W, R = Tl::R, KT = Tl::kKeys, P = Tl::kPieces, NL = Tl::kLoads;
  constexpr int KB = Mm::kScoreTiles, QJ = Mm::QJ, DT = Mm::DT, NG = Mm::kGroups;
  constexpr int MR = Mm::kRows, PT = kWave / MR;  // rows of a wave, lanes of a row
  // separate objects, so that the compiler sees that loads into one buffer do
  // not touch what is read from the other
  constexpr int kBuf = 2 * KT * P;
  __shared__ u32x4 lds0[kBuf], lds1[kBuf];  // keys, then values
  auto buf = [&](int i) { return i == 0 ? lds0 : lds1; };
  __shared__ TreeLds tree;
  __shared__ int any_odd;
  const KvBatch& k = p.k;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = uni(tid / kWave);
  const int c = lane % MR, h = lane / MR;  // row, part
  const int G = p.Hq / p.Hkv;
  const float inv_g = 1.f / static_cast<float>(G);
  const Places<R, D> places(p.ws, n_wg);
  // Of 64 rows, whole heads save fragments of bandwidth-bound work: with 60 heads 480 of
  // 512 workgroups take 84 us against 112, with 300 heads 300 take 153 against 163.  Of
  // 128 rows work is lost with them: with 68 heads 204 of 256 take 250 us against 194,
  // with 6 heads 252 take 319 against 304.
  const AttnStart st = attn_start<Line, true>(p, G, n_wg, grain, ROWS == 64 ? n_wg : 0);
  const int wg = st.wg;
  AttnJoin join;
  join.last = -1;
  const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 1.17549435e-38f);
  const int ps = 1 << k.page_shift;
  const size_t head_sz = static_cast<size_t>(ps) * D;
  const size_t page_sz = static_cast<size_t>(p.Hkv) * head_sz;
  // The lane's offset in a load of keys: its key behind the wave's first, and the
  // piece that belongs at its place; the same for every KP-th load of the wave.
  constexpr int KP = Mm::kSwizzlePeriod > Tl::kKeysPerLoad ? Mm::kSwizzlePeriod / Tl::kKeysPerLoad : 1;
  uint32_t k_off[KP];
#pragma unroll
  for (int j = 0; j < KP; ++j) {
    const int key = (j * W + wave) * kWave / P + lane / P;
    k_off[j] = (lane / P * D + (lane % P ^ Mm::swizzle(key)) * 8) * 2;
  }
  // the key whose row lane c feeds to a score tile, and its piece h; piece PT j + h
  // is at k_at ^ PT j (tile keys leave the permutation as it is)
  const int row_key = Mm::row_key(c);
  const int k_at = row_key * P + (h ^ Mm::swizzle(row_key));
  const int v_at = h * D + c;
  int err = 0;

  long long x = st.lo, seq_at = st.seq_at;
  int layer = st.layer, b = st.b;
  KvSpan r = st.span;
  while (x < st.hi) {
    const AttnItem it = attn_item<Line>(p, G, layer, b, r, seq_at, x);
    const long long end = it.at + it.cost;
    const long long till = end < st.hi ? end : st.hi;
    const int row0 = it.tile * R;
    const int rows = min(R, r.n * G - row0);
    const int tok_first = row0 / G;
    const int skip = row0 - tok_first * G;
    const int tok_last = tok_first + tile_token(skip, rows - 1, inv_g);
    const int len = r.ctx + (p.parent ? r.n : tok_last + 1);
    const int steps = (len + KT - 1) / KT;
    const int s0 = x == it.at ? 0 : uni(static_cast<int>(part_of(x - it.at, steps, it.cost)));
    const int s1 =
        till == end ? steps : uni(static_cast<int>(part_of(till - it.at, steps, it.cost)));
    const bool whole = it.at >= st.lo && end <= st.hi;
    bool good = true;
    if (p.parent) {
      good = tree_masks(p.parent + r.s, r.n, tree);
      if (!good) err |= GDN_DEV_ERR_PARENT;
    }
    if (good) {
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * k.max_blocks;
      // Pages of 64 sixteens of keys at a time, a lane each: the next ones' numbers
      // (below 0: none), and the offset in bytes of the current ones' keys in a
      // cache, which is that of their values too.
      int pgn, batch = s0 * (KT / 16), off_lo, off_hi;
      unsigned long long gone_all;
      auto has_key = [&](int first16) {
        const long long key = (static_cast<long long>(first16) + lane) * 16;
        return key < len && key < static_cast<long long>(s1) * KT;
      };
      // As they stand in the table, or any entry where there is no key: nothing
      // here depends on the number, so that nothing waits for it before its turn.
      auto pages_from = [&](int first16) {
        return table[has_key(first16) ? ((first16 + lane) * 16) >> k.page_shift : 0];
      };
      auto enter = [&](int first16, int pg) {
        batch = first16;
        const bool bad = pg < 0 || pg >= k.n_pages;
        const bool none = bad || !has_key(first16);
        if (none && has_key(first16)) err |= GDN_DEV_ERR_PAGE;
        gone_all = __ballot(none);
        const long long off =
            (static_cast<long long>(none ? 0 : pg) * static_cast<long long>(page_sz) +
             (((first16 + lane) * 16) & (ps - 1)) * D) * 2;
        off_lo = static_cast<int>(off);
        off_hi = static_cast<int>(off >> 32);
        pgn = pages_from(first16 + 64);
      };
      enter(batch, pages_from(batch));
      const uint16_t* kc = static_cast<const uint16_t*>(p.k_cache) +
                           (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const uint16_t* vc = static_cast<const uint16_t*>(p.v_cache) +
                           (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const char* kw = reinterpret_cast<const char*>(kc + wave * kWave / P % 16 * D);
      const char* vw =
          reinterpret_cast<const char*>(vc + (wave * kWave / D % 2 * D + wave * kWave % D) * 8);
      // Sixteens without a page of the tile last sent, looked at when it is multiplied
      // (only then does a page number that is not one count).
      uint32_t gone_sent = 0;
      // Sends the tile of step s on its way into the buffers: load j of a wave
      // fills 64 pieces in a row, of keys (and of values: eight keys of a channel
      // to a piece) that lie in one sixteen.
      auto fetch = [&](int s, u32x4* kl) {
        u32x4* const vl = kl + KT * P;
        const int at = s * (KT / 16);
        if (at - batch == 64) enter(at, pgn);
        gone_sent = static_cast<uint32_t>(gone_all >> (at - batch)) & ((1u << (KT / 16)) - 1u);
        const int six0 = at - batch + wave * kWave / P / 16;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int six = six0 + j * Tl::kKeysPerLoad / 16;
          const uint32_t lo = __builtin_amdgcn_readlane(off_lo, six);
          const uint32_t hi = __builtin_amdgcn_readlane(off_hi, six);
          const size_t off = (static_cast<size_t>(hi) << 32 | lo) +
                             j * Tl::kKeysPerLoad % 16 * D * 2;
          const int i0 = (j * W + wave) * kWave;
          to_lds(kw + off, opaque(k_off[j % KP]), kl + i0);
          to_lds(vw + off, opaque(lane * 16), vl + i0);
        }
      };
      __syncthreads();  // the last item's LDS is free
      if (tid == 0) any_odd = 0;
      if (s0 < s1) fetch(s0, buf(0));
      // the lane's row
      const int myrow = min(wave * MR + c, rows - 1);
      const int tok = tile_token(skip, myrow, inv_g);
      bf16x8 qf[QJ];
      {
        const uint16_t* q =
            static_cast<const uint16_t*>(p.q) +
            (static_cast<size_t>(it.layer) * k.N + r.s + tok_first + tok) * p.q_ld +
            static_cast<size_t>(it.h * G + skip + myrow - tok * G) * D + h * 8;
#pragma unroll
        for (int j = 0; j < QJ; ++j) {
          u32x4 w = *reinterpret_cast<const u32x4*>(q + j * Mm::kQ);
          if (p.scale < 0.f)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] ^= 0x80008000u;
          qf[j] = __builtin_bit_cast(bf16x8, w);
        }
      }
      // keys that all rows see, and those that any of the wave's does
      const int wave_tok1 = tok_first + tile_token(skip, min(wave * MR + MR - 1, rows - 1), inv_g);
      const int all_see = r.ctx + (p.parent ? 0 : tok_first + 1);
      const int any_sees = wave * MR >= rows ? 0 : p.parent ? len : r.ctx + wave_tok1 + 1;

      Acc o[DT];
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] = Acc{};
      float m = kNegInf, l = 0.f;
      auto scores = [&](Acc* sc, const u32x4* kl) {
        const int ka = opaque(k_at);  // the operands' places are worked out anew: few registers
        products<KB * QJ>(
            [&](int n) {
              return __builtin_bit_cast(
                  bf16x8, kl[(ka ^ PT * (n % QJ)) + Mm::tile_key(n / QJ) * P]);
            },
            [&](int n, bf16x8 kf) {
              Acc& z = sc[n / QJ];
              if (n % QJ == 0) z = Acc{};
              z = Mm::mul(kf, qf[n % QJ], z);
            });
      };
      // Raises the maximum where it has to, then turns scores into probabilities.
      auto weights = [&](const Acc* sc, bf16x8* pf, bf16x8* rest) {
        float top = sc[0][0];
#pragma unroll
        for (int t = 0; t < KB; ++t)
#pragma unroll
          for (int i = 0; i < Mm::kAcc; ++i) top = fmaxf(top, sc[t][i]);
        top = Mm::top(top);
        if (__any((top - m) * c2 > kSlack)) {
          const float M = fmaxf(top, m);
          const float back = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m - M) * c2);
          m = M;
          l *= back;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < Mm::kAcc; ++i) o[t][i] *= back;
        }
        const float at = m == kNegInf ? 0.f : m * c2;
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float w =
                __builtin_amdgcn_exp2f(fmaf(sc[Mm::tile_of(i, e)][Mm::reg_of(i, e)], c2, -at));
            l += w;
            pf[i][e] = static_cast<__bf16>(w);
            if (Tl::kRest) rest[i][e] = static_cast<__bf16>(w - static_cast<float>(pf[i][e]));
          }
      };
      auto values = [&](const bf16x8* pf, const bf16x8* rest, const u32x4* vl) {
        products<NG * DT>(
            [&](int n) {
              return __builtin_bit_cast(
                  bf16x8, vl[v_at + n / DT * (Mm::kEvery / 8) * D + n % DT * MR]);
            },
            [&](int n, bf16x8 vf) {
              o[n % DT] = Mm::mul(vf, pf[n / DT], o[n % DT]);
              if (Tl::kRest) o[n % DT] = Mm::mul(vf, rest[n / DT], o[n % DT]);
            });
      };
      // A tile that every row sees all of.
      auto plain = [&](const u32x4* kl) {
        const u32x4* const vl = kl + KT * P;
        if (any_sees == 0) return;  // a wave without rows
        Acc sc[KB];
        bf16x8 pf[NG], rest[NG];
        scores(sc, kl);
        weights(sc, pf, rest);
        values(pf, rest, vl);
      };
      // A tile with keys that some row does not see or that are not there.
      // Values that are not there, infinities and NaN are left out, as in the
      // stream kernel: the workgroup puts zeros in their places first.
      auto edge = [&](int kb, uint32_t gone, u32x4* kl) {
        u32x4* const vl = kl + KT * P;
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int at = i * W * kWave + opaque(tid), first = at / D * 8;
          const uint32_t there =
              (gone >> (first / 16)) & 1 ? 0u : chain_sees(len, kb + first, 8);
          u32x4 w = vl[at] & F::keep(there);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = ((w[e] & F::kExp) + F::kOne) & F::kTop;
            bad |= y;
            w[e] &= ~F::spread(y);
          }
          vl[at] = w;
        }
        if (bad) any_odd = 1;
        lds_barrier();
        if (kb >= any_sees) return;
        Acc sc[KB];
        bf16x8 pf[NG], rest[NG];
        scores(sc, kl);
        // the first of the lane's eight keys of group i, and those of them that are there
        auto base_of = [&](int i) { return kb + Mm::kEvery * i + opaque(8 * h); };
        auto there_of = [&](int i, int base) {
          return (gone >> ((base - kb) / 16)) & 1 ? 0u : chain_sees(len, base, 8);
        };
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const int base = base_of(i);
          uint32_t sees = there_of(i, base);
          sees &= p.parent ? tree_sees(tree.mask[tok_first + tok], r.ctx, base, 8)
                           : chain_sees(r.ctx + tok_first + tok + 1, base, 8);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float z = sc[Mm::tile_of(i, e)][Mm::reg_of(i, e)];
            sc[Mm::tile_of(i, e)][Mm::reg_of(i, e)] = (sees >> e) & 1 ? z : kNegInf;
          }
        }
        weights(sc, pf, rest);
        values(pf, rest, vl);
      };

      lds_loads_done();
      lds_barrier();
      int s = s0, at = 0;  // at: the buffer of tile s
      while (s < s1 && (s + 1) * KT <= all_see && gone_sent == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (s + 1 < s1) fetch(s + 1, buf(1 - i));
          plain(buf(i));
          lds_loads_done();
          lds_barrier();
          ++s;
          at = 1 - i;
          if (!(s < s1 && (s + 1) * KT <= all_see && gone_sent == 0)) break;
        }
      }
      for (; s < s1; ++s) {
        const uint32_t gone = gone_sent;
        if (s + 1 < s1) fetch(s + 1, buf(1 - at));
        edge(s * KT, gone, buf(at));
        lds_loads_done();
        lds_barrier();
        at = 1 - at;
      }
      if (any_odd) {  // rare: to the rows that do see them
        const int from = max(s0 * KT, r.ctx & ~(KT - 1)), to = min(len, s1 * KT);
#pragma unroll 1
        for (int key = from; key < to; ++key) {
          const bool sees = p.parent ? tree_sees(tree.mask[tok_first + tok], r.ctx, key, 1) != 0
                                     : key <= r.ctx + tok_first + tok;
          const int pg = table[key >> k.page_shift];
          if (pg < 0 || pg >= k.n_pages) continue;
          const uint16_t* e = vc + pg * page_sz +
                              static_cast<size_t>((key & (ps - 1)) >> 3) * (D * 8) + (key & 7) +
                              opaque(h * 32);
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < Mm::kAcc; ++i) {
              const float y = ld_in(e, (t * MR + Mm::channel(i)) * 8);
              if (sees && not_finite(y)) o[t][i] += y;
              __builtin_amdgcn_sched_barrier(0);  // one at a time: no registers to spare
            }
        }
      }

      l = Mm::sum(l);
      if (wave * MR + c < rows) {
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* dst =
              static_cast<uint16_t*>(p.o) +
              ((static_cast<long long>(it.layer) * k.N + r.s + tok_first + tok) * p.Hq + it.h * G +
               skip + myrow - tok * G) * D + opaque(4 * h);
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int a = 0; a < Mm::kAcc / 4; ++a) {
              uint16_t e4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                e4[i] = to_out(l == 0.f ? 0.f : o[t][4 * a + i] * inv, uint16_t{});
              __builtin_memcpy(__builtin_assume_aligned(dst + t * MR + 8 * a, 8), e4, 8);
            }
        } else {
          const int place = 2 * wg + (it.at < st.lo ? 0 : 1), row = wave * MR + opaque(c);
          if (h == 0) places.ml[static_cast<size_t>(place) * R + row] = floatx2{m, l};
          float* const dst = places.row(place, row) + 4 * h;
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int a = 0; a < Mm::kAcc / 4; ++a) {
              floatx4 v;
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = o[t][4 * a + i];
              *reinterpret_cast<floatx4*>(dst + t * MR + 8 * a) = v;
            }
        }
      }
      if (!whole && it.at >= st.lo) {
        join.last = attn_owner(st.s, end - 1);
        join.rows = rows;
        join.skip = skip;
        join.out =
            ((static_cast<long long>(it.layer) * k.N + r.s + tok_first) * p.Hq + it.h * G) * D;
      }
    }
    x = till;
    if (x < st.hi) {  // the next item, of this sequence or of the next that has any
      long long seq_end = seq_at + Line::sequence(r, G, p.Hkv);
      while (x >= seq_end) {
        seq_at = seq_end;
        if (++b == k.B) {
          b = 0;
          ++layer;
        }
        r = kv_span(k, b);
        seq_end = seq_at + Line::sequence(r, G, p.Hkv);
      }
    }
  }
  if (tid == 0) places.join[wg] = join;
  if (err && p.dev_err) atomicOr(p.dev_err, err);
}

// Adds the fragments of the item that workgroup blockIdx.x began and did not
// end, in order of their keys.  Four fragments or fewer: a wave has RB rows, all
// their fragments in flight at once.  More (a long context and few rows): a
// workgroup has RB rows, wave w fragments w, w + 4, ... of each, and the four
// partial results are added in order.
template <int E>
struct Partial {
  float m, l, o[E];
  __device__ __forceinline__ void clear() {
    m = kNegInf;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
  }
  // A sum that has seen no key but those of score -inf has no weight.
  __device__ __forceinline__ void add(const Partial& y, float c2) {
    const float M = fmaxf(m, y.m);
    const float a = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m - M) * c2);
    const float b = y.m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((y.m - M) * c2);
    l = l * a + y.l * b;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * a + y.o[i] * b;
    m = M;
  }
};

constexpr int kMostWg = 512;
constexpr int kFew = 4;
constexpr int kJoinWg = 1024;  // workgroups, all resident at once

// The tasks (an item's RB or 4 RB rows) are counted by every workgroup for itself
// from the n_wg descriptions, and dealt out in turn: a grid of n_wg by rows, most
// of which have nothing to do, costs more than that (7 against 3 us).
template <typename T, int D, int R, int RB>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p, int n_wg) {
  const Places<R, D> places(p.ws, n_wg);
  constexpr int E = D / kWave;
  __shared__ float weight[RB][kMostWg];  // of a fragment, over l of them all
  __shared__ float all[RB];              // that l
  __shared__ float part[3][RB][D];
  __shared__ int upto[kMostWg];  // tasks of the items that workgroups 0 .. w began
  __shared__ int wave_sum_[2][4];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uni(tid / kWave);
  const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 1.17549435e-38f);
  const float inv_g = 1.f / static_cast<float>(p.Hq / p.Hkv);
  int scan[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = i * 256 + tid;
    int tasks = 0;
    if (w < n_wg) {
      const AttnJoin j = places.join[w];
      if (j.last >= 0) {
        const int per = j.last - w + 1 <= kFew ? 4 * RB : RB;
        tasks = (j.rows + per - 1) / per;
      }
    }
    scan[i] = static_cast<int>(wave_scan(tasks));
    if (lane == kWave - 1) wave_sum_[i][wave] = scan[i];
  }
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w == wave) upto[i * 256 + tid] = before + scan[i];
      before += wave_sum_[i][w];
    }
  __syncthreads();
  for (int task = blockIdx.x; task < before; task += gridDim.x) {
    int w0 = 0, hi = kMostWg - 1;  // the first with more tasks up to it
    while (w0 < hi) {
      const int mid = (w0 + hi) / 2;
      if (upto[mid] > task)
        hi = mid;
      else
        w0 = mid + 1;
    }
    w0 = uni(w0);
    const AttnJoin j = places.join[w0];
    const int n = j.last - w0 + 1;
    const bool few = n <= kFew;
    int row0 = (task - (w0 ? upto[w0 - 1] : 0)) * (few ? 4 * RB : RB);
    auto place = [&](int f) { return 2 * (w0 + f) + (f == 0 ? 1 : 0); };
    auto load = [&](int f, int row) {  // fragment f of a row that is there
      Partial<E> y;
      const floatx2 ml = places.ml[static_cast<size_t>(place(f)) * R + row];
      y.m = ml[0];
      y.l = ml[1];
#pragma unroll
      for (int i = 0; i < E; ++i) y.o[i] = places.row(place(f), row)[lane * E + i];
      return y;
    };
    auto write = [&](const Partial<E>& y, int row) {
      const int G = p.Hq / p.Hkv, tok = tile_token(j.skip, row, inv_g);
      T* out = static_cast<T*>(p.o) + j.out +
               (static_cast<long long>(tok) * p.Hq + j.skip + row - tok * G) * D + lane * E;
      const float inv = y.l == 0.f ? 0.f : 1.f / y.l;
      T e[E];
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = to_out(y.l == 0.f ? 0.f : y.o[i] * inv, T{});
      __builtin_memcpy(__builtin_assume_aligned(out, E * sizeof(T)), e, sizeof(e));
    };
    if (few) {
      row0 += wave * RB;
      Partial<E> y[RB][kFew];
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int f = 0; f < kFew; ++f) {
          y[i][f].clear();
          if (f < n && row0 + i < j.rows) y[i][f] = load(f, row0 + i);
        }
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (row0 + i >= j.rows) continue;
#pragma unroll
        for (int f = 1; f < kFew; ++f) y[i][0].add(y[i][f], c2);
        write(y[i][0], row0 + i);
      }
      continue;
    }
    // the weights first, a lane to a fragment, so that the long sums wait for loads only
    for (int i = wave; i < RB; i += 4) {
      const floatx2* ml = places.ml + min(row0 + i, j.rows - 1);
      float M = kNegInf;
      for (int f = lane; f < n; f += kWave) M = fmaxf(M, ml[static_cast<size_t>(place(f)) * R][0]);
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor(M, off, kWave));
      float L = 0.f;
      for (int f = lane; f < n; f += kWave) {
        const floatx2 y = ml[static_cast<size_t>(place(f)) * R];
        // a fragment without keys has no weight; l may be NaN where m is still -inf
        const float w = y[0] == kNegInf ? 0.f : __builtin_amdgcn_exp2f((y[0] - M) * c2);
        if (w != 0.f || y[1] != y[1]) L += y[1] == y[1] ? y[1] * w : y[1];
        weight[i][f] = w;
      }
      L = wave_sum(L);
      if (lane == 0) all[i] = L;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      for (int f = lane; f < n; f += kWave) weight[i][f] *= inv;
    }
    __syncthreads();
    float o[RB][E] = {};
#pragma unroll 2
    for (int f = wave; f < n; f += 4)
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const float* from = places.row(place(f), min(row0 + i, j.rows - 1));
        const float w = weight[i][f];
#pragma unroll
        for (int e = 0; e < E; ++e) o[i][e] += from[lane * E + e] * w;
      }
    if (wave > 0)
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) part[wave - 1][i][lane * E + e] = o[i][e];
    __syncthreads();
    if (wave == 0)
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        if (row0 + i >= j.rows) continue;
        Partial<E> y;
        y.l = all[i] == 0.f ? 0.f : 1.f;  // the weights are over it already
#pragma unroll
        for (int e = 0; e < E; ++e) {
          y.o[e] = o[i][e];
#pragma unroll
          for (int w = 0; w < 3; ++w) y.o[e] += part[w][i][lane * E + e];
        }
        write(y, row0 + i);
      }
    __syncthreads();  // the LDS is free for the next task
  }
}

// A workgroup has at least this many keys' cost.  In bf16 256: for the stream kernel
// level with 128 (one sequence of 800 tokens); for the tile kernel 8 drafts behind
// 16,000 tokens take 24.1 us with 256, 28.2 with 192, 29.4 with 128, a prompt of 300
// tokens 29, 32 and 38, 4 sequences of 8 drafts 20.4, 19.9 and 24.2, 8 drafts behind
// 1,000 tokens 17.5, 16.6 and 16.0.  In 32 bits, where a key's products take sixteen
// times as long, fewer: 90 rows of three heads 47 us with 256, 24 with 64.
constexpr long long grain_of(int size) { return size == 2 ? 256 : 64; }
constexpr int kCus = 256;
static_assert(2 * kCus <= kMostWg, "the join counts no more");

// The kernel and tile for sequences of at most `rows` query rows, and how many
// workgroups: two to a CU, or one where LDS or registers hold no second.  (With 64
// channels in bf16 three or four would fit; the join counts no more than 512.)
struct AttnPlan {
  int tile;  // rows of the tile kernel's tile, or 0: the stream kernel
  int nt;    // its 16s of rows
  int wgs;
  int rows() const { return tile ? tile : 16 * nt; }
};

// Rows of the stream kernel's tile in 16s: with bf16 it takes 16 rows at most, and
// the tile kernel more (32 rounds of 64 rows and about 3,000 keys: 92 us by the stream
// kernel with 64 rows' sums in one wave's registers, 68 by tiles when they were taken).
// In 32 bits 32 rows; with 256 channels 16, whose sums and operands already spill 140
// bytes a lane.
constexpr int stream_most(int head_dim, int size) { return size == 2 || head_dim == 256 ? 1 : 2; }
AttnPlan attn_plan(long long rows, int head_dim, int size) {
  AttnPlan a{0, 1, 2 * kCus};
  if (size == 2 && rows > 16) {
    a.tile = rows > 64 ? 128 : 64;
    // LDS for one workgroup on a CU (64 trees: 186 us; two parts for each 202)
    if (a.tile == 128 && head_dim == 256) a.wgs = kCus;
    return a;
  }
  const int most = stream_most(head_dim, size);
  const int want = rows <= 16 ? 1 : 2;
  a.nt = want < most ? want : most;
  // registers for one wave on a SIMD only
  if (a.nt * head_dim * size > 256) a.wgs = kCus;
  return a;
}

template <typename T, int D, int R>
hipError_t join_t(const AttnArgs& a, int wgs, hipStream_t s) {
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  constexpr int RB = R < 64 ? R / 16 : 4;
  k_attn_join<T, D, R, RB><<<kJoinWg, 256, 0, s>>>(a, wgs);
  return hipGetLastError();
}

template <typename T, int D, int NT>
hipError_t stream_t(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  k_attn_stream<T, D, NT><<<p.wgs, 256, 0, s>>>(a, p.wgs, grain_of(sizeof(T)));
  return join_t<T, D, 16 * NT>(a, p.wgs, s);
}

template <int D, int ROWS>
hipError_t tile_t(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  k_attn_tile<D, ROWS><<<p.wgs, Tile<D, ROWS>::W * kWave, 0, s>>>(a, p.wgs, grain_of(2));
  return join_t<uint16_t, D, ROWS>(a, p.wgs, s);
}

template <typename T, int D>
hipError_t attn_t(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.k.T) * (a.Hq / a.Hkv);
  const AttnPlan p = attn_plan(rows, D, sizeof(T));
  if constexpr (sizeof(T) == 2) {
    if (p.tile == 128) return tile_t<D, 128>(a, p, s);
    if (p.tile == 64) return tile_t<D, 64>(a, p, s);
  } else {
    constexpr int most = stream_most(D, sizeof(T));
    if constexpr (most >= 2)
      if (p.nt == 2) return stream_t<T, D, 2>(a, p, s);
  }
  return stream_t<T, D, 1>(a, p, s);
}

}  // namespace

hipError_t launch_attn(const AttnArgs& a, int head_dim, int dtype, hipStream_t s) {
  if (dtype == 1) {
    if (head_dim == 64) return attn_t<uint16_t, 64>(a, s);
    if (head_dim == 128) return attn_t<uint16_t, 128>(a, s);
    if (head_dim == 256) return attn_t<uint16_t, 256>(a, s);
  } else {
    if (head_dim == 64) return attn_t<float, 64>(a, s);
    if (head_dim == 128) return attn_t<float, 128>(a, s);
    if (head_dim == 256) return attn_t<float, 256>(a, s);
  }
  return hipErrorInvalidValue;
}

// The most that any call of as many rows or fewer needs: narrow tiles on more
// workgroups can take a little more than wide ones on fewer.
size_t attn_workspace(long long rows, int head_dim, int dtype) {
  size_t most = 0;
  for (long long r : {1LL, 17LL, 65LL}) {  // the least rows of each plan
    if (r > rows) break;
    const AttnPlan p = attn_plan(r, head_dim, dtype == 1 ? 2 : 4);
    const size_t bytes = places_bytes(p.rows(), head_dim, p.wgs);
    if (bytes > most) most = bytes;
  }
  return most;
}

}  // namespace gdn
