// C entry points of sliding-window attention (declared in include/sla2.h): argument checks, the
// workspace layout and the launches.
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "sla2.h"
#include "kernels.cuh"
#include "window.cuh"

using namespace sla2;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

sla2_status check_window(const sla2_window_desc* d, WindowShape* s) {
  if (!d) return SLA2_ERR_INVALID_ARG;
  if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->N < 1 || d->d < 1 || d->Hq % d->Hkv) return SLA2_ERR_INVALID_ARG;
  if (d->window < 1 || d->sinks < 0 || (d->causal != 0 && d->causal != 1) || (d->dtype != 0 && d->dtype != 1))
    return SLA2_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return SLA2_ERR_INVALID_ARG;
  if (d->d != 64 && d->d != 128) return SLA2_ERR_UNSUPPORTED;
  const long long BH = (long long)d->B * d->Hq;
  if (BH > 0x7fffffffLL / d->N) return SLA2_ERR_UNSUPPORTED;
  s->B = d->B;
  s->Hq = d->Hq;
  s->Hkv = d->Hkv;
  s->g = d->Hq / d->Hkv;
  s->N = d->N;
  s->d = d->d;
  s->W = d->window < d->N ? d->window : d->N;
  s->S = d->sinks < d->N ? d->sinks : d->N;
  s->causal = d->causal;
  s->scale = d->scale;
  s->lens = d->lens;
  s->status = d->status;
  s->budget_ns = wait_budget_ns();
  return SLA2_OK;
}

// The view's strides, those of extents of 1 replaced by ones that the checks and the tensor maps take.
bool view_ok(const sla2_view* v, int B, int H, int N, int d, View4* o) {
  if (!v || !v->data || !aligned16(v->data)) return false;
  *o = {v->data, B > 1 ? v->stride_b : d, H > 1 ? v->stride_h : d, N > 1 ? v->stride_n : d};
  for (long long st : {o->sb, o->sh, o->sn})
    if (st < d || st % 8 || st >= (1LL << 39)) return false;     // 2^40 bytes: a tensor map's limit
  return true;
}

#define SLA2_TRY(expr)                                   \
  do {                                                   \
    if ((expr) != cudaSuccess) return SLA2_ERR_CUDA;     \
  } while (0)

cudaError_t clear_status(unsigned* status, cudaStream_t st) {
  return status ? cudaMemsetAsync(status, 0, sizeof(unsigned), st) : cudaSuccess;
}

// the driver's encoder, looked up once through the runtime
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

size_t delta_bytes(const WindowShape& s) { return align256((size_t)s.B * s.Hq * s.N * 12); }   // and what it is off by, twice
size_t sizes_bytes(const WindowShape& s) { return align256(window_backward_sizes(s)); }
size_t bwd_workspace(const WindowShape& s) { return delta_bytes(s) + sizes_bytes(s) + align256(window_backward_pieces(s)); }

}  // namespace

bool sla2::make_tmap_4d(CUtensorMap* m, const View4& v, int B, int H, int N, int d, int cols, int rows) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)v.sn * 2, (cuuint64_t)v.sh * 2, (cuuint64_t)v.sb * 2};
  const cuuint32_t box[4] = {(cuuint32_t)cols, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, v.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" {

sla2_status sla2_window_forward(const sla2_window_desc* desc, const sla2_view* q, const sla2_view* k,
                                const sla2_view* v, const sla2_view* out, float* lse, void* stream) {
  WindowShape s;
  const sla2_status r = check_window(desc, &s);
  if (r != SLA2_OK) return r;
  WindowFwdArgs a{};
  if (!view_ok(q, s.B, s.Hq, s.N, s.d, &a.q) || !view_ok(k, s.B, s.Hkv, s.N, s.d, &a.k) ||
      !view_ok(v, s.B, s.Hkv, s.N, s.d, &a.v) || !view_ok(out, s.B, s.Hq, s.N, s.d, &a.out))
    return SLA2_ERR_INVALID_ARG;
  if (a.out.p == a.q.p || a.out.p == a.k.p || a.out.p == a.v.p) return SLA2_ERR_INVALID_ARG;
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SLA2_TRY(clear_status(s.status, st));
  SLA2_TRY(launch_window_forward(s, desc->dtype, a, st));
  return SLA2_OK;
}

size_t sla2_window_backward_workspace_size(const sla2_window_desc* desc) {
  WindowShape s;
  if (check_window(desc, &s) != SLA2_OK) return 0;
  return bwd_workspace(s);
}

sla2_status sla2_window_backward(const sla2_window_desc* desc, const sla2_view* q, const sla2_view* k,
                                 const sla2_view* v, const sla2_view* out, const float* lse, const sla2_view* dout,
                                 const sla2_view* dq, const sla2_view* dk, const sla2_view* dv, void* stream) {
  WindowShape s;
  const sla2_status r = check_window(desc, &s);
  if (r != SLA2_OK) return r;
  WindowBwdArgs a{};
  if (!view_ok(q, s.B, s.Hq, s.N, s.d, &a.q) || !view_ok(k, s.B, s.Hkv, s.N, s.d, &a.k) ||
      !view_ok(v, s.B, s.Hkv, s.N, s.d, &a.v) || !view_ok(out, s.B, s.Hq, s.N, s.d, &a.out) ||
      !view_ok(dout, s.B, s.Hq, s.N, s.d, &a.dout) || !view_ok(dq, s.B, s.Hq, s.N, s.d, &a.dq) ||
      !view_ok(dk, s.B, s.Hkv, s.N, s.d, &a.dk) || !view_ok(dv, s.B, s.Hkv, s.N, s.d, &a.dv) || !lse)
    return SLA2_ERR_INVALID_ARG;
  for (const void* o : {a.dq.p, a.dk.p, a.dv.p})
    for (const void* i : {a.q.p, a.k.p, a.v.p, a.out.p, a.dout.p})
      if (o == i) return SLA2_ERR_INVALID_ARG;
  if (a.dq.p == a.dk.p || a.dq.p == a.dv.p || a.dk.p == a.dv.p) return SLA2_ERR_INVALID_ARG;
  if (!desc->workspace || desc->workspace_bytes < bwd_workspace(s) ||
      (reinterpret_cast<uintptr_t>(desc->workspace) & 255u))
    return SLA2_ERR_WORKSPACE;
  a.lse = lse;
  a.delta = static_cast<float*>(desc->workspace);
  a.sizes = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(desc->workspace) + delta_bytes(s));
  a.pieces = static_cast<uint8_t*>(desc->workspace) + delta_bytes(s) + sizes_bytes(s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SLA2_TRY(clear_status(s.status, st));
  SLA2_TRY(launch_window_backward(s, desc->dtype, a, st));
  return SLA2_OK;
}

}  // extern "C"
