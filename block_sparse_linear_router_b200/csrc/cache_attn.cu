// Attention of a step's new tokens over the paged 8-bit cache: one warp per (token, query head), one
// key per lane at a time, an online softmax over groups of 32 keys.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "device.cuh"
#include "window.cuh"

namespace sla2 {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

template <class T, int D>
__global__ void __launch_bounds__(128) cache_attn_kernel(CacheShape s, CacheAttnArgs a) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h = blockIdx.y * 4 + warp;
  if (h >= s.Hq) return;
  int b = 0;
  while (b + 1 < s.B && __ldg(s.cu + b + 1) <= t) ++b;
  Span sp;
  if (!step_span(s, b, &sp)) {
    flag_bad_index(s);
    return;
  }
  if (t < sp.t0 || t >= sp.t0 + sp.n) return;
  const int i = sp.len + (t - sp.t0), hk = h / s.g;
  const T* q = static_cast<const T*>(a.q.p) + (long long)t * a.q.st + h * a.q.sh;
  for (int c = lane; c < D; c += 32) sq[warp][c] = Half16<T>::f(q[c]) * a.scale * LOG2E;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  auto keys = [&](int j0, int j1) {
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      float x = -INFINITY, vs = 0.f;
      int pid = -1;
      if (j < j1) {
        const int pi = j >> s.lpage;
        pid = pi < s.max_pages ? __ldg(s.table + (size_t)b * s.max_pages + pi) : -1;
        if (pid >= 0 && pid < s.num_pages) {
          const size_t ph = (size_t)pid * s.Hkv + hk;
          const int8_t* kc = s.kc + (ph * s.page + (j & (s.page - 1))) * D;
          x = 0.f;
          for (int c = 0; c < D; ++c) x = fmaf(sq[warp][c], (float)kc[c], x);
          x *= s.ks[ph];
          vs = s.vs[ph];
        } else {
          pid = -1;
          flag_bad_index(s);
        }
      }
      float mx = x;
      for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
      const float mn = fmaxf(m, mx);
      if (mn == -INFINITY) continue;
      const float corr = exp2f(m - mn), p = exp2f(x - mn);
      float ps = p;
      for (int off = 16; off; off >>= 1) ps += __shfl_xor_sync(~0u, ps, off);
      l = l * corr + ps;
      m = mn;
      for (int c = 0; c < D / 32; ++c) o[c] *= corr;
      for (int u = 0; u < 32 && jb + u < j1; ++u) {
        const float pt = __shfl_sync(~0u, p * vs, u);
        const int pd = __shfl_sync(~0u, pid, u);
        if (pd < 0) continue;
        const int8_t* vc = s.vc + (((size_t)pd * s.Hkv + hk) * s.page + ((jb + u) & (s.page - 1))) * D;
        for (int c = 0; c < D / 32; ++c) o[c] = fmaf(pt, (float)vc[c * 32 + lane], o[c]);
      }
    }
  };
  const int lo = a.W <= i ? i - a.W + 1 : 0;
  keys(0, a.S < lo ? a.S : lo);
  keys(lo, i + 1);
  T* out = static_cast<T*>(a.out.p) + (long long)t * a.out.st + h * a.out.sh;
  for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = Half16<T>::r(m > -INFINITY ? o[c] / l : 0.f);
}

template <class T, int D>
cudaError_t launch_t(const CacheShape& s, const CacheAttnArgs& a, cudaStream_t st) {
  cache_attn_kernel<T, D><<<dim3(s.T, (s.Hq + 3) / 4), 128, 0, st>>>(s, a);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attention_workspace(const CacheShape&) { return 256; }

cudaError_t launch_cache_attention(const CacheShape& s, int fp16, const CacheAttnArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
