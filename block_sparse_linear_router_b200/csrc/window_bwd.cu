// Gradients of sliding-window attention with sinks. With P = exp(scale Q K^T - lse) on the visible
// pairs, delta = rowsum(dO * O) and dS = scale P (dO V^T - delta):
//   dQ = dS K,  dK = dS^T Q,  dV = P^T dO.
// One warp per query row for dQ (which also leaves delta), one per key row for dK and dV.
#include "device.cuh"
#include "window.cuh"

namespace sla2 {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

template <class T, int D>
__device__ __forceinline__ float dot(const float* x, const T* y) {
  float r = 0.f;
  for (int c = 0; c < D; ++c) r = fmaf(x[c], Half16<T>::f(y[c]), r);
  return r;
}

template <class T, int D>
__global__ void __launch_bounds__(128) window_dq_kernel(WindowShape s, WindowBwdArgs a) {
  __shared__ float sq[4][D], so[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 4 + warp, h = blockIdx.y % s.Hq, b = blockIdx.y / s.Hq;
  if (i >= s.N) return;
  const int n = window_len(s, b);
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + h * a.q.sh + i * a.q.sn;
  const T* o = static_cast<const T*>(a.out.p) + b * a.out.sb + h * a.out.sh + i * a.out.sn;
  const T* dO = static_cast<const T*>(a.dout.p) + b * a.dout.sb + h * a.dout.sh + i * a.dout.sn;
  const T* K = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / s.g) * a.k.sh;
  const T* V = static_cast<const T*>(a.v.p) + b * a.v.sb + (h / s.g) * a.v.sh;
  const long long row = ((long long)b * s.Hq + h) * s.N + i;
  float delta = 0.f, dq[D / 32] = {};
  if (i < n) {
    for (int c = lane; c < D; c += 32) {
      sq[warp][c] = Half16<T>::f(q[c]);
      so[warp][c] = Half16<T>::f(dO[c]);
      delta = fmaf(so[warp][c], Half16<T>::f(o[c]), delta);
    }
    for (int off = 16; off; off >>= 1) delta += __shfl_xor_sync(~0u, delta, off);
  }
  __syncwarp();
  const float lse2 = a.lse[row] * LOG2E;
  auto keys = [&](int j0, int j1) {
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      float ds = 0.f;
      if (j < j1) {
        const float p = exp2f(dot<T, D>(sq[warp], K + j * a.k.sn) * (s.scale * LOG2E) - lse2);
        ds = p * (dot<T, D>(so[warp], V + j * a.v.sn) - delta) * s.scale;
      }
      for (int t = 0; t < 32 && jb + t < j1; ++t) {
        const float x = __shfl_sync(~0u, ds, t);
        for (int c = 0; c < D / 32; ++c) dq[c] = fmaf(x, Half16<T>::f(K[(jb + t) * a.k.sn + c * 32 + lane]), dq[c]);
      }
    }
  };
  if (i < n) {
    const int lo = i - s.W + 1 > 0 ? i - s.W + 1 : 0;
    const int hi = s.causal ? i + 1 : (s.W < n - i ? i + s.W : n);
    keys(0, s.S < lo ? s.S : lo);
    keys(lo, hi);
    if (!s.causal) keys(hi, s.S < n ? s.S : n);
  }
  T* out = static_cast<T*>(a.dq.p) + b * a.dq.sb + h * a.dq.sh + i * a.dq.sn;
  for (int c = 0; c < D / 32; ++c) out[c * 32 + lane] = Half16<T>::r(dq[c]);
  if (lane == 0) a.delta[row] = delta;
}

template <class T, int D>
__global__ void __launch_bounds__(128) window_dkdv_kernel(WindowShape s, WindowBwdArgs a) {
  __shared__ float sk[4][D], sv[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 4 + warp, hk = blockIdx.y % s.Hkv, b = blockIdx.y / s.Hkv;
  if (j >= s.N) return;
  const int n = window_len(s, b);
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + hk * a.k.sh + j * a.k.sn;
  const T* v = static_cast<const T*>(a.v.p) + b * a.v.sb + hk * a.v.sh + j * a.v.sn;
  float dk[D / 32] = {}, dv[D / 32] = {};
  if (j < n) {
    for (int c = lane; c < D; c += 32) {
      sk[warp][c] = Half16<T>::f(k[c]);
      sv[warp][c] = Half16<T>::f(v[c]);
    }
    __syncwarp();
    // the queries that see key j
    int lo = s.causal ? j : (j - s.W + 1 > 0 ? j - s.W + 1 : 0), hi = s.W < n - j ? j + s.W : n;
    if (j < s.S) {
      lo = s.causal ? j : 0;
      hi = n;
    }
    for (int h = hk * s.g; h < (hk + 1) * s.g; ++h) {
      const T* Q = static_cast<const T*>(a.q.p) + b * a.q.sb + h * a.q.sh;
      const T* dO = static_cast<const T*>(a.dout.p) + b * a.dout.sb + h * a.dout.sh;
      const long long row = ((long long)b * s.Hq + h) * s.N;
      for (int ib = lo; ib < hi; ib += 32) {
        const int i = ib + lane;
        float p = 0.f, ds = 0.f;
        if (i < hi) {
          p = exp2f(dot<T, D>(sk[warp], Q + i * a.q.sn) * (s.scale * LOG2E) - a.lse[row + i] * LOG2E);
          ds = p * (dot<T, D>(sv[warp], dO + i * a.dout.sn) - a.delta[row + i]) * s.scale;
        }
        for (int t = 0; t < 32 && ib + t < hi; ++t) {
          const float x = __shfl_sync(~0u, p, t), y = __shfl_sync(~0u, ds, t);
          for (int c = 0; c < D / 32; ++c) {
            dv[c] = fmaf(x, Half16<T>::f(dO[(ib + t) * a.dout.sn + c * 32 + lane]), dv[c]);
            dk[c] = fmaf(y, Half16<T>::f(Q[(ib + t) * a.q.sn + c * 32 + lane]), dk[c]);
          }
        }
      }
    }
  }
  T* dk_o = static_cast<T*>(a.dk.p) + b * a.dk.sb + hk * a.dk.sh + j * a.dk.sn;
  T* dv_o = static_cast<T*>(a.dv.p) + b * a.dv.sb + hk * a.dv.sh + j * a.dv.sn;
  for (int c = 0; c < D / 32; ++c) {
    dk_o[c * 32 + lane] = Half16<T>::r(dk[c]);
    dv_o[c * 32 + lane] = Half16<T>::r(dv[c]);
  }
}

template <class T, int D>
cudaError_t launch_t(const WindowShape& s, const WindowBwdArgs& a, cudaStream_t st) {
  window_dq_kernel<T, D><<<dim3((s.N + 3) / 4, s.B * s.Hq), 128, 0, st>>>(s, a);
  window_dkdv_kernel<T, D><<<dim3((s.N + 3) / 4, s.B * s.Hkv), 128, 0, st>>>(s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_backward(const WindowShape& s, int fp16, const WindowBwdArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
