// Sliding-window attention with sinks, forward: one warp per query row, one key per lane at a time,
// an online softmax over groups of 32 keys.
#include "device.cuh"
#include "window.cuh"

namespace sla2 {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <class T, int D>
__global__ void __launch_bounds__(128) window_fwd_kernel(WindowShape s, WindowFwdArgs a) {
  __shared__ float sq[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + warp, h = blockIdx.y % s.Hq, b = blockIdx.y / s.Hq;
  if (i >= s.N) return;
  const int n = window_len(s, b);
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + h * a.q.sh + i * a.q.sn;
  const T* K = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / s.g) * a.k.sh;
  const T* V = static_cast<const T*>(a.v.p) + b * a.v.sb + (h / s.g) * a.v.sh;
  for (int c = lane; c < D; c += 32) sq[warp][c] = i < n ? Half16<T>::f(q[c]) * s.scale * LOG2E : 0.f;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  auto keys = [&](int j0, int j1) {
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      float x = -INFINITY;
      if (j < j1) {
        x = 0.f;
        for (int c = 0; c < D; ++c) x = fmaf(sq[warp][c], Half16<T>::f(K[j * a.k.sn + c]), x);
      }
      float mx = x;
      for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
      const float mn = fmaxf(m, mx), corr = exp2f(m - mn), p = exp2f(x - mn);
      float ps = p;
      for (int off = 16; off; off >>= 1) ps += __shfl_xor_sync(~0u, ps, off);
      l = l * corr + ps;
      m = mn;
      for (int c = 0; c < D / 32; ++c) o[c] *= corr;
      for (int t = 0; t < 32 && jb + t < j1; ++t) {
        const float pt = __shfl_sync(~0u, p, t);
        for (int c = 0; c < D / 32; ++c) o[c] = fmaf(pt, Half16<T>::f(V[(jb + t) * a.v.sn + c * 32 + lane]), o[c]);
      }
    }
  };
  if (i < n) {
    const int lo = i - s.W + 1 > 0 ? i - s.W + 1 : 0;
    const int hi = s.causal ? i + 1 : (s.W < n - i ? i + s.W : n);
    keys(0, s.S < lo ? s.S : lo);                          // sinks before the window
    keys(lo, hi);
    if (!s.causal) keys(hi, s.S < n ? s.S : n);            // sinks behind it
  }
  T* out = static_cast<T*>(a.out.p) + b * a.out.sb + h * a.out.sh + i * a.out.sn;
  for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = Half16<T>::r(i < n ? o[c] / l : 0.f);
  if (a.lse && lane == 0) a.lse[((long long)b * s.Hq + h) * s.N + i] = i < n ? (m + log2f(l)) * LN2 : -INFINITY;
}

template <class T, int D>
cudaError_t launch_t(const WindowShape& s, const WindowFwdArgs& a, cudaStream_t st) {
  window_fwd_kernel<T, D><<<dim3((s.N + 3) / 4, s.B * s.Hq), 128, 0, st>>>(s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_forward(const WindowShape& s, int fp16, const WindowFwdArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
