// k_attn.hip -- attention of a round's new tokens over the paged cache.
//
// One wave per (query row, layer): keys in steps of 64, a key per lane for
// the scores, a channel per lane for the sum over values, with the running
// maximum and sum of the softmax.

#include "gdn_common.hpp"
#include "kv_kernels.hpp"

namespace gdn {
namespace {

__device__ __forceinline__ uint16_t to_out(float x, uint16_t) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}
__device__ __forceinline__ float to_out(float x, float) { return x; }

// Ancestors (and self) of node v as a bit mask; 0 where the array is malformed.
__device__ __forceinline__ uint64_t ancestors(const int32_t* parent, int v) {
  uint64_t m = 0;
  for (int u = v; u >= 0;) {
    m |= 1ull << u;
    const int q = parent[u];
    if (q < -1 || q >= u) return 0;
    u = q;
  }
  return m;
}

template <typename T, int D>
__global__ __launch_bounds__(kWave) void k_attn_row(AttnArgs p) {
  __shared__ float qs[D];
  __shared__ float ps[kWave];
  const KvBatch& k = p.k;
  const int i = blockIdx.x, hq = blockIdx.y % p.Hq, l = blockIdx.y / p.Hq;
  const int h = hq / (p.Hq / p.Hkv), lane = threadIdx.x;
  int b = 0;
  KvSpan r{};
  for (; b < k.B; ++b) {
    r = kv_span(k, b);
    if (!r.ok && lane == 0 && p.dev_err) atomicOr(p.dev_err, GDN_DEV_ERR_LENGTH);
    if (r.n > 0 && i >= r.s && i < r.s + r.n) break;
  }
  if (b == k.B) return;
  const int own = i - r.s;
  uint64_t mask = 0;
  if (p.parent) {
    bool bad = false;
    for (int v = lane; v < r.n; v += kWave) {
      const int q = p.parent[r.s + v];
      bad |= q < -1 || q >= v;
    }
    if (__any(bad)) {
      if (p.dev_err && lane == 0) atomicOr(p.dev_err, GDN_DEV_ERR_PARENT);
      return;
    }
    mask = ancestors(p.parent + r.s, own);
  }
  const int psz = 1 << k.page_shift;
  const size_t head = static_cast<size_t>(psz) * D;
  const size_t layer = static_cast<size_t>(l) * k.n_pages * p.Hkv * head;
  const T* q = static_cast<const T*>(p.q) + (static_cast<size_t>(l) * k.N + i) * p.q_ld + hq * D;
  for (int d = lane; d < D; d += kWave) qs[d] = ld_in(q, d) * p.scale;
  __syncthreads();
  const int total = r.ctx + (p.parent ? r.n : own + 1);
  float m = -__builtin_inff(), sum = 0.f, acc[D / kWave] = {};
  for (int c = 0; c < total; c += kWave) {
    const int j = c + lane;
    bool live = j < total;
    if (live && p.parent && j >= r.ctx) live = (mask >> (j - r.ctx)) & 1;
    int pg = 0;
    if (live) {
      pg = p.block_table[static_cast<size_t>(b) * k.max_blocks + (j >> k.page_shift)];
      if (pg < 0 || pg >= k.n_pages) {
        if (p.dev_err) atomicOr(p.dev_err, GDN_DEV_ERR_PAGE);
        live = false;
        pg = 0;
      }
    }
    const size_t page = layer + (static_cast<size_t>(pg) * p.Hkv + h) * head;
    const int off = j & (psz - 1);
    float z = -__builtin_inff();
    if (live) {
      z = 0.f;
      const T* kr = static_cast<const T*>(p.k_cache) + page + static_cast<size_t>(off) * D;
      for (int d = 0; d < D; ++d) z = fmaf(qs[d], ld_in(kr, d), z);
    }
    float top = z;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
    const float M = fmaxf(m, top);
    const float e = live && M > -__builtin_inff() ? expf(z - M) : (live && z != z ? z : 0.f);
    const float back = M > -__builtin_inff() ? expf(m - M) : 1.f;
    sum = sum * back + wave_sum(e);
    m = M;
    ps[lane] = e;
    const uint64_t who = __ballot(live);
    __syncthreads();
    for (int x = 0; x < D / kWave; ++x) acc[x] *= back;
    for (int t = 0; t < kWave; ++t) {
      if (!((who >> t) & 1)) continue;
      const size_t pt = layer + (static_cast<size_t>(__shfl(pg, t, kWave)) * p.Hkv + h) * head;
      const int ot = (c + t) & (psz - 1);
      const T* vr = static_cast<const T*>(p.v_cache) + pt + static_cast<size_t>(ot / 8) * (D * 8) +
                    ot % 8;
      for (int x = 0; x < D / kWave; ++x)
        acc[x] = fmaf(ps[t], ld_in(vr, static_cast<size_t>(x * kWave + lane) * 8), acc[x]);
    }
    __syncthreads();
  }
  T* o = static_cast<T*>(p.o) + ((static_cast<size_t>(l) * k.N + i) * p.Hq + hq) * D;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  for (int x = 0; x < D / kWave; ++x) o[x * kWave + lane] = to_out(acc[x] * inv, T{});
}

template <typename T, int D>
hipError_t attn_t(const AttnArgs& a, hipStream_t s) {
  k_attn_row<T, D><<<dim3(a.k.N, a.L * a.Hq), kWave, 0, s>>>(a);
  return hipGetLastError();
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

size_t attn_workspace(int, int, int, int, int, int, int, int, long long) { return 16; }

}  // namespace gdn
