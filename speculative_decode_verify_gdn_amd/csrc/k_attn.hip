// k_attn.hip -- attention of a round's new tokens over the paged cache, for
// gfx950 (attn_verify).
//
//   o_r = sum_j softmax_j(scale * q_r . k_j) v_j
//
// in one pass over the keys with the running maximum m, sum l and output O of
// each row: a step with scores s rescales l and O by exp(m - m') and adds
// exp(s - m') (times v).  Two such triples over disjoint keys join the same way
// (the waves of a workgroup, then the fragments of an item).
//
// Everything is computed transposed, S^T = K Q^T and O^T = V^T P^T, so that a
// lane owns one query row: its column of a 16x16 result tile.  Maximum, sum
// and rescaling are then per lane, and the exponentials of S^T are, in the
// registers where they lie, the B operand of the second product: the key that
// a result row stands for is free to choose, and is chosen so that a lane's
// eight probabilities belong to eight consecutive keys, which the value cache
// stores side by side.  No operand is shuffled or passes through LDS but Q.

#include <algorithm>

#include "attn_sched.hpp"
#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

// ---- element types: 32 keys of K and V as MFMA operands

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

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
  const floatx4 a = p[0], b = p[1];
  bf16x8 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = static_cast<__bf16>(a[i]);
    w[i + 4] = static_cast<__bf16>(b[i]);
  }
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], w, o, 0, 0, 0);
}
__device__ __forceinline__ floatx4 weigh(const floatx4* v, const floatx4* p, floatx4 o) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o = __builtin_amdgcn_mfma_f32_16x16x4f32(v[t][i], p[t][i], o, 0, 0, 0);
  return o;
}

__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t bits(__bf16 x) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, x)) << 16;
}
__device__ __forceinline__ bool not_finite(uint32_t b) { return (b & 0x7f800000u) == 0x7f800000u; }

__device__ __forceinline__ uint16_t to_out(float x, uint16_t) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ float to_out(float x, float) { return x; }

// Maximum over the four lanes that hold a row's keys (c, c+16, c+32, c+48).
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, kWave));
  return fmaxf(x, __shfl_xor(x, 32, kWave));
}
__device__ __forceinline__ float row_sum(float x) {
  x += __shfl_xor(x, 16, kWave);
  return x + __shfl_xor(x, 32, kWave);
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
// (m, l) pairs, then n_wg descriptions for the join.
template <int R, int D>
struct Places {
  float* o;
  floatx2* ml;
  AttnJoin* join;
  __device__ __host__ Places(void* ws, int n_wg) {
    o = static_cast<float*>(ws);
    ml = reinterpret_cast<floatx2*>(o + static_cast<size_t>(2 * n_wg) * R * D);
    join = reinterpret_cast<AttnJoin*>(ml + static_cast<size_t>(2 * n_wg) * R);
  }
  static size_t bytes(int n_wg) {
    return static_cast<size_t>(2 * n_wg) * R * (D + 2) * sizeof(float) +
           static_cast<size_t>(n_wg) * sizeof(AttnJoin);
  }
};

// ---- few query rows: the waves of a workgroup take different keys
//
// R = 16 NT rows; each wave streams 32 keys at a time straight from the cache
// into MFMA operands (no LDS, no barrier until the item ends) and keeps all the
// rows' sums.  Bound by the cache's bytes while R is small.
template <typename T, int D, int NT>
struct Stream {
  static constexpr int W = 4;            // waves
  static constexpr int R = 16 * NT;
  static constexpr int kStep = 32 * W;   // keys of one step of the workgroup
  static constexpr int QLD = D + Frag<T>::kPad;
  static constexpr int kC = D < 128 ? D : 128;  // channels joined at a time
  struct Lds {
    T q[R * QLD];
    float join[W][16][kC + 4];
    float m[W][R], l[W][R];
    TreeLds tree;
    long long scan[W + 2];
  };
};

template <typename T, int D, int NT>
__global__ __launch_bounds__(256, 1) void k_attn_stream(AttnArgs p, int n_wg, long long grain) {
  using St = Stream<T, D, NT>;
  using F = Frag<T>;
  constexpr int W = St::W, R = St::R, QLD = St::QLD;
  constexpr int KJ = D / F::kPerK;  // score products per tile
  constexpr int MT = D / 16;        // output tiles
  __shared__ typename St::Lds sh;
  const KvBatch& k = p.k;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int c = lane % 16, g = lane / 16;
  const int G = p.Hq / p.Hkv;
  const int wg = blockIdx.x;
  const Places<R, D> places(p.ws, n_wg);
  const AttnStart st = attn_start<R, W * kWave>(p, G, wg, n_wg, grain, sh.scan);
  AttnJoin join;
  join.last = -1;
  const float sgn = p.scale < 0.f ? -1.f : 1.f;
  // scores are compared unscaled; at least the smallest normal, so that a
  // masked -inf stays -inf at scale 0
  const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 1.17549435e-38f);
  const int ps = 1 << k.page_shift;
  const size_t head_sz = static_cast<size_t>(ps) * D;
  int err = 0;

  long long x = st.lo, seq_at = st.seq_at;
  int layer = st.layer, b = st.b;
  while (x < st.hi) {
    const AttnItem it = attn_item<R>(p, G, layer, b, seq_at, x);
    const KvSpan& r = it.span;
    const long long end = it.at + it.cost;
    const long long till = end < st.hi ? end : st.hi;
    const int rows_all = r.n * G;
    const int row0 = it.tile * R;
    const int rows = min(R, rows_all - row0);
    const int tok_first = row0 / G;
    const int tok_last = (row0 + rows - 1) / G;
    const int len = r.ctx + (p.parent ? r.n : tok_last + 1);
    const int steps = (len + St::kStep - 1) / St::kStep;
    const int s0 = static_cast<int>(part_of(x - it.at, steps, it.cost));
    const int s1 = static_cast<int>(part_of(till - it.at, steps, it.cost));
    const bool whole = it.at >= st.lo && end <= st.hi;
    bool good = true;
    if (p.parent) {
      good = tree_masks(p.parent + r.s, r.n, sh.tree);
      if (!good) err |= GDN_DEV_ERR_PARENT;
    }
    __syncthreads();  // the last item's LDS is free
    if (good) {
      // Q rows, zero behind the last one
      constexpr int E = 16 / sizeof(T);
      const T* q = static_cast<const T*>(p.q) +
                   (static_cast<size_t>(it.layer) * k.N + r.s) * p.q_ld +
                   static_cast<size_t>(it.h) * G * D;
      for (int i = tid; i < R * (D / E); i += W * kWave) {
        const int row = i / (D / E), ch = i % (D / E);
        T e[E] = {};
        if (row < rows) {
          const int tok = (row0 + row) / G, qh = (row0 + row) % G;
          *reinterpret_cast<u32x4*>(e) =
              *reinterpret_cast<const u32x4*>(q + tok * p.q_ld + qh * D + ch * E);
          if (sgn < 0.f)
#pragma unroll
            for (int j = 0; j < E; ++j) {
              if constexpr (sizeof(T) == 2)
                e[j] ^= 0x8000;
              else
                e[j] = -e[j];
            }
        }
        *reinterpret_cast<u32x4*>(&sh.q[row * QLD + ch * E]) = *reinterpret_cast<u32x4*>(e);
      }
      // what each of the lane's rows may see: keys below lim, and bits of amask
      // for the new tokens of a tree
      int lim[NT];
      uint64_t amask[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = min(n * 16 + c, rows - 1);
        const int tok = (row0 + row) / G;
        lim[n] = p.parent ? r.ctx : r.ctx + tok + 1;
        amask[n] = p.parent ? sh.tree.mask[tok] : 0;
      }
      __syncthreads();

      floatx4 o[NT][MT];
      float m[NT], l[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n] = kNegInf;
        l[n] = 0.f;
#pragma unroll
        for (int t = 0; t < MT; ++t) o[n][t] = floatx4{0.f, 0.f, 0.f, 0.f};
      }
      const T* kc = static_cast<const T*>(p.k_cache) +
                    (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const T* vc = static_cast<const T*>(p.v_cache) +
                    (static_cast<size_t>(it.layer) * k.n_pages * p.Hkv + it.h) * head_sz;
      const int32_t* table = p.block_table + static_cast<size_t>(it.b) * k.max_blocks;
      const size_t page_sz = static_cast<size_t>(p.Hkv) * head_sz;

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
      typename F::K kf[2][KJ];
      typename F::V vf[MT][F::kVLoads];
      int pgs = pages_from(s0), pgn = -1, batch = s0;
      int h0 = 0, h1 = 0;  // the current step's page numbers, -1 where nothing is
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
          const T* row = (key < 16 ? b0 : b1) + (key & 15) * D + g * (16 / sizeof(T));
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
                &sh.q[(n * 16 + c) * QLD + j * F::kPerK + g * (16 / sizeof(T))]);
            sc[n][0] = F::score(kf[0][j], qf, sc[n][0]);
            sc[n][1] = F::score(kf[1][j], qf, sc[n][1]);
          }
        }
        if (s + 1 < s1) {
          step_pages(s + 1, h0, h1);
          load_k(s + 1, h0, h1);
        }
        // any key that some row does not see, or that is not there
        const bool edge = kb + 32 > r.ctx + (p.parent ? 0 : tok_first + 1) || a < 0 || e < 0;
        if (edge) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int kk = F::key_of(t, g, i), key = kb + kk;
              const bool there = key < len && (kk < 16 ? a : e) >= 0;
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                bool live = there && key < lim[n];
                if (there && key >= r.ctx && ((amask[n] >> (key - r.ctx)) & 1)) live = true;
                if (!live) sc[n][t][i] = kNegInf;
              }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top = fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3]));
          top = fmaxf(top, fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
          top = fmaxf(row_max(top), m[n]);
          // a row that has seen no key yet: any finite number will do
          const float at = top == kNegInf ? 0.f : top;
          const float back = __builtin_amdgcn_exp2f((m[n] - at) * c2);
          m[n] = top;
          float add = 0.f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float w = __builtin_amdgcn_exp2f((sc[n][t][i] - at) * c2);
              sc[n][t][i] = w;
              add += w;
            }
          l[n] = l[n] * back + add;
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][t][i] *= back;
        }
        if (edge) {
          // Values that are not there become 0.  An infinity or NaN that only
          // some rows see would reach the others as 0 * inf: the product is
          // taken without it, and it is added to the rows that do see it.
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            bool odd = false;
            constexpr int VE = 16 / sizeof(T);
#pragma unroll
            for (int u = 0; u < F::kVLoads; ++u)
#pragma unroll
              for (int i = 0; i < VE; ++i) {
                const int kk = F::key_of(u, g, 0) + i;
                if (!(kb + kk < len && (kk < 16 ? a : e) >= 0)) vf[t][u][i] = 0;
                odd |= not_finite(bits(vf[t][u][i]));
              }
            if (__any(odd)) {
#pragma unroll 1
              for (int kind = 0; kind < 3; ++kind) {
                const float what = kind == 0   ? __builtin_inff()
                                   : kind == 1 ? -__builtin_inff()
                                               : __builtin_nanf("");
                typename F::V is[F::kVLoads];
#pragma unroll
                for (int u = 0; u < F::kVLoads; ++u)
#pragma unroll
                  for (int i = 0; i < VE; ++i) {
                    const uint32_t w = bits(vf[t][u][i]);
                    const bool hit = kind == 0   ? w == 0x7f800000u
                                     : kind == 1 ? w == 0xff800000u
                                                 : (w & 0x7fffffffu) > 0x7f800000u;
                    is[u][i] = hit ? 1.f : 0.f;
                  }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  floatx4 seen[2];
#pragma unroll
                  for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
                    for (int i = 0; i < 4; ++i) seen[t2][i] = sc[n][t2][i] > 0.f ? 1.f : 0.f;
                  const floatx4 cnt = weigh(is, seen, floatx4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (cnt[i] > 0.f) o[n][t][i] += what;
                }
              }
#pragma unroll
              for (int u = 0; u < F::kVLoads; ++u)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                  if (not_finite(bits(vf[t][u][i]))) vf[t][u][i] = 0;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int t = 0; t < MT; ++t) o[n][t] = weigh(vf[t], sc[n], o[n][t]);
        if (s + 1 < s1) load_v(s + 1, h0, h1);
      }

      // join the four waves: maxima first, then 16 rows and kC channels at a time
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
      T* out = static_cast<T*>(p.o) + ((static_cast<size_t>(it.layer) * k.N + r.s) * p.Hq +
                                       static_cast<size_t>(it.h) * G) * D;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 16 >= rows) break;
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sh.m[w][n * 16 + c]);
        const float mine = m[n] == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m[n] - M) * c2);
#pragma unroll
        for (int ch = 0; ch < D / St::kC; ++ch) {
          __syncthreads();
#pragma unroll
          for (int t = 0; t < St::kC / 16; ++t) {
            floatx4 v = o[n][ch * (St::kC / 16) + t];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mine == 0.f ? 0.f : v[i] * mine;
            *reinterpret_cast<floatx4*>(&sh.join[wave][c][t * 16 + 4 * g]) = v;
          }
          __syncthreads();
          for (int i = tid; i < 16 * St::kC / 4; i += W * kWave) {
            const int row = i / (St::kC / 4), d = i % (St::kC / 4) * 4;
            const int rr = n * 16 + row;
            if (rr >= rows) continue;
            floatx4 v = *reinterpret_cast<const floatx4*>(&sh.join[0][row][d]);
#pragma unroll
            for (int w = 1; w < W; ++w) {
              const floatx4 y = *reinterpret_cast<const floatx4*>(&sh.join[w][row][d]);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] += y[j];
            }
            float Mr = kNegInf, L = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) Mr = fmaxf(Mr, sh.m[w][rr]);
#pragma unroll
            for (int w = 0; w < W; ++w)
              if (sh.m[w][rr] != kNegInf || sh.l[w][rr] != sh.l[w][rr])
                L += sh.l[w][rr] * __builtin_amdgcn_exp2f((sh.m[w][rr] - Mr) * c2);
            if (whole) {
              const int tok = (row0 + rr) / G, qh = (row0 + rr) % G;
              T* dst = out + (static_cast<size_t>(tok) * p.Hq + qh) * D + ch * St::kC + d;
              T e4[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) e4[j] = to_out(L == 0.f ? 0.f : v[j] / L, T{});
              __builtin_memcpy(__builtin_assume_aligned(dst, 4 * sizeof(T)), e4, sizeof(e4));
            } else {
              *reinterpret_cast<floatx4*>(
                  &places.o[(static_cast<size_t>(place) * R + rr) * D + ch * St::kC + d]) = v;
              if (d == 0 && ch == 0) places.ml[static_cast<size_t>(place) * R + rr] = floatx2{Mr, L};
            }
          }
        }
      }
      if (!whole && it.at >= st.lo) {
        join.last = attn_owner(st.s, end - 1);
        join.rows = rows;
        join.row0 = row0;
        join.tok0 = r.s;
        join.layer = it.layer;
        join.head = it.h;
      }
    }
    x = till;
    if (x < st.hi) {  // the next item, of this sequence or of the next that has any
      long long seq_end = seq_at + AttnLine<R>::sequence(r, G, p.Hkv);
      while (x >= seq_end) {
        seq_at = seq_end;
        if (++b == k.B) {
          b = 0;
          ++layer;
        }
        seq_end = seq_at + AttnLine<R>::sequence(kv_span(k, b), G, p.Hkv);
      }
    }
  }
  if (tid == 0) places.join[wg] = join;
  if (err && p.dev_err) atomicOr(p.dev_err, err);
}

// Adds the fragments of the item that workgroup blockIdx.x began and did not
// end, in order.  A wave per fragment modulo four, a workgroup per row.
template <typename T, int D, int R>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs p, int n_wg) {
  const Places<R, D> places(p.ws, n_wg);
  const int w0 = blockIdx.x, row = blockIdx.y;
  const AttnJoin j = places.join[w0];
  if (j.last < 0 || row >= j.rows) return;
  constexpr int E = D / kWave;
  __shared__ float sh_m[4], sh_l[4], sh_o[4][D];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const float c2 = fmaxf(fabsf(p.scale) * kLog2e, 1.17549435e-38f);
  float m = kNegInf, l = 0.f, o[E] = {};
#pragma unroll 4
  for (int w = w0 + wave; w <= j.last; w += 4) {
    const size_t at = static_cast<size_t>(2 * w + (w == w0 ? 1 : 0)) * R + row;
    const floatx2 ml = places.ml[at];
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = places.o[at * D + lane * E + i];
    if (ml[0] == kNegInf && ml[1] == ml[1]) continue;  // a fragment without keys
    const float M = fmaxf(m, ml[0]);
    const float back = m == kNegInf ? 0.f : __builtin_amdgcn_exp2f((m - M) * c2);
    const float add = __builtin_amdgcn_exp2f((ml[0] - M) * c2);
    m = M;
    l = l * back + ml[1] * add;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = (back == 0.f ? 0.f : o[i] * back) + (add == 0.f ? 0.f : v[i] * add);
  }
  if (lane == 0) {
    sh_m[wave] = m;
    sh_l[wave] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) sh_o[wave][lane * E + i] = o[i];
  __syncthreads();
  float M = kNegInf, L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sh_m[w]);
  float f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = sh_m[w] == kNegInf && sh_l[w] == sh_l[w] ? 0.f : __builtin_amdgcn_exp2f((sh_m[w] - M) * c2);
    if (f[w] != 0.f || sh_l[w] != sh_l[w]) L += sh_l[w] * f[w];
  }
  const int G = p.Hq / p.Hkv;
  const int tok = (j.row0 + row) / G, qh = (j.row0 + row) % G;
  T* out = static_cast<T*>(p.o) +
           ((static_cast<size_t>(j.layer) * p.k.N + j.tok0 + tok) * p.Hq +
            static_cast<size_t>(j.head) * G + qh) * D;
  if (static_cast<int>(threadIdx.x) < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (f[w] != 0.f) v += sh_o[w][threadIdx.x] * f[w];
    out[threadIdx.x] = to_out(L == 0.f ? 0.f : v / L, T{});
  }
}

// Workgroups of the stream kernel: two per CU, each with at least kGrain keys.
constexpr int kStreamWg = 512;
constexpr long long kGrain = 512;

// Rows of a tile: the fewest 16s that hold a sequence's rows, at most 64 (32
// with 256 channels, whose sums take the registers).
int stream_nt(long long rows, int head_dim) {
  if (rows <= 16) return 1;
  if (rows <= 32 || head_dim == 256) return 2;
  return 4;
}

template <typename T, int D, int NT>
hipError_t stream_t(const AttnArgs& a, hipStream_t s) {
  constexpr int R = 16 * NT;
  k_attn_stream<T, D, NT><<<kStreamWg, 256, 0, s>>>(a, kStreamWg, kGrain);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_attn_join<T, D, R><<<dim3(kStreamWg, R), 256, 0, s>>>(a, kStreamWg);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t attn_t(const AttnArgs& a, hipStream_t s) {
  const long long rows = static_cast<long long>(a.k.T) * (a.Hq / a.Hkv);
  const int nt = stream_nt(rows, D);
  if (nt == 1) return stream_t<T, D, 1>(a, s);
  if (nt == 2) return stream_t<T, D, 2>(a, s);
  if constexpr (D < 256) return stream_t<T, D, 4>(a, s);
  return hipErrorInvalidValue;
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

size_t attn_workspace(int L, int B, int T, int N, int Hq, int Hkv, int head_dim, int dtype,
                      long long max_tokens) {
  const int R = 16 * stream_nt(static_cast<long long>(T) * (Hq / Hkv), head_dim);
  return static_cast<size_t>(2 * kStreamWg) * R * (head_dim + 2) * sizeof(float) +
         static_cast<size_t>(kStreamWg) * sizeof(AttnJoin);
}

}  // namespace gdn
