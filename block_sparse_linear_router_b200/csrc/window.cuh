// Shared by the sliding-window attention kernels (window_fwd.cu, window_bwd.cu) and their C entry
// points (window_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace sla2 {

// A [B][H][N][d] tensor of 16-bit elements, strides in elements.
struct View4 {
  void* p;
  long long sb, sh, sn;
};

struct WindowShape {
  int B, Hq, Hkv, g, N, d;   // g = Hq / Hkv query heads share a key head
  int W, S, causal;          // window and sinks, both at most N
  float scale;
  const int32_t* lens;       // device [B] or nullptr
  unsigned* status;
  unsigned long long budget_ns;
};

__device__ __forceinline__ int window_len(const WindowShape& s, int b) {
  if (!s.lens) return s.N;
  const int n = __ldg(s.lens + b);
  return n < 0 ? 0 : (n > s.N ? s.N : n);
}

// TMA map of a 16-bit [B][H][N][d] view: boxes of `cols` (64 or 32) elements x `rows` tokens, swizzled
// over their width; implemented in window_api.cu.
bool make_tmap_4d(CUtensorMap* m, const View4& v, int B, int H, int N, int d, int cols, int rows);

struct WindowFwdArgs {
  View4 q, k, v, out;
  float* lse;                // [B][Hq][N] or nullptr
};
cudaError_t launch_window_forward(const WindowShape& s, int fp16, const WindowFwdArgs& a, cudaStream_t st);

struct WindowBwdArgs {
  View4 q, k, v, out, dout, dq, dk, dv;
  const float* lse;          // [B][Hq][N]
  float* delta;              // workspace, fp32 [3][B][Hq][N]: rowsum(dO * O), and two parts of what it is off by
  uint32_t* sizes;           // workspace: window_backward_sizes bytes
  uint8_t* pieces;           // workspace: window_backward_pieces bytes
};
size_t window_backward_sizes(const WindowShape& s);
size_t window_backward_pieces(const WindowShape& s);
cudaError_t launch_window_backward(const WindowShape& s, int fp16, const WindowBwdArgs& a, cudaStream_t st);

template <class T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float f(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 r(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Half16<__half> {
  static __device__ __forceinline__ float f(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half r(float x) { return __float2half_rn(x); }
};

}  // namespace sla2
