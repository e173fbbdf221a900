// Shared by the kernels of the paged 8-bit cache (cache_append.cu, cache_attn.cu) and their C entry
// points (cache_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace sla2 {

constexpr unsigned SLA2_DEV_BAD_INDEX = 6u;   // same value as SLA2_ERR_BAD_INDEX

// A [T][H][d] tensor of 16-bit elements, strides in elements.
struct View3 {
  void* p;
  long long st, sh;
};

struct CacheShape {
  int num_pages, Hkv, page, lpage, d;   // lpage = log2(page)
  int8_t *kc, *vc;                      // [num_pages][Hkv][page][d]
  float *ks, *vs;                       // [num_pages][Hkv]
  int B, T, Hq, g, max_pages;
  const int32_t *table, *lens, *cu;
  unsigned* status;
  int sms;
};

// Rows [t0, t0 + n) are the new tokens of sequence b, at positions len and up. Returns false, n = 0,
// where the arrays' values are out of range.
struct Span {
  int t0, n, len;
};
__device__ __forceinline__ bool step_span(const CacheShape& s, int b, Span* o) {
  const int c0 = __ldg(s.cu + b), c1 = __ldg(s.cu + b + 1), len = __ldg(s.lens + b);
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= s.T && len >= 0 && len <= 0x7fffffff - (c1 - c0);
  *o = {c0, ok ? c1 - c0 : 0, len};
  return ok;
}
__device__ __forceinline__ void flag_bad_index(const CacheShape& s) {
  if (s.status) atomicExch(s.status, SLA2_DEV_BAD_INDEX);
}
// The span of sequence b, for a block whose threads go through the sequences in order (b = threadIdx.x, then blockDim.x
// further on each call; n = 0 from s.B on). Sequences are left out from the first one on whose offsets go down or
// reach outside the token rows: those behind it may claim rows of those before. `cut` keeps that from call to call.
// report: this block sets the status word.
__device__ __forceinline__ Span block_span(const CacheShape& s, int b, bool* cut, bool report) {
  __shared__ int from;
  Span sp{0, 0, 0};
  bool off = false;
  if (b < s.B) {
    if (!step_span(s, b, &sp)) {
      const int c0 = __ldg(s.cu + b), c1 = __ldg(s.cu + b + 1);
      off = c0 < 0 || c1 < c0 || c1 > s.T;
      if (report) flag_bad_index(s);
    }
  }
  if (*cut) {
    sp.n = 0;
  } else if (__syncthreads_or(off)) {
    if (threadIdx.x == 0) from = 0x7fffffff;
    __syncthreads();
    if (off) atomicMin(&from, b);
    __syncthreads();
    if (b >= from) sp.n = 0;
    *cut = true;
  }
  return sp;
}

struct AppendArgs {
  View3 k, v, q, q_out, k_out;   // q.p, k_out.p may be NULL
  const float *cos, *sin;
  int rope_rows, rope_dim, interleaved;
};
cudaError_t launch_cache_append(const CacheShape& s, int fp16, const AppendArgs& a, cudaStream_t st);

constexpr int CACHE_UNIT = 32;   // keys that attention takes at a time
struct CacheAttnArgs {
  View3 q, out;
  int W, S;
  int end;                       // units that a row of the page table reaches
  float scale;
  void* workspace;
};
size_t cache_attention_workspace(const CacheShape& s);
cudaError_t launch_cache_attention(const CacheShape& s, int fp16, const CacheAttnArgs& a, cudaStream_t st);

}  // namespace sla2
