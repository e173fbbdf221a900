// C entry points of the paged 8-bit cache (declared in include/sla2.h): argument checks and launches.
#include <cmath>

#include "sla2.h"
#include "cache.cuh"
#include "kernels.cuh"

using namespace sla2;

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

sla2_status check_step(const sla2_cache* c, const sla2_step* t, CacheShape* s) {
  if (!c || !t) return SLA2_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->page < 1 || c->d < 1) return SLA2_ERR_INVALID_ARG;
  if (t->B < 1 || t->T < 1 || t->Hq < 1 || t->max_pages < 1 || t->Hq % c->Hkv || (t->dtype != 0 && t->dtype != 1))
    return SLA2_ERR_INVALID_ARG;
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !t->page_table || !t->kv_lens || !t->cu_new)
    return SLA2_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes)) return SLA2_ERR_INVALID_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SLA2_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return SLA2_ERR_UNSUPPORTED;
  if (c->Hkv > 65535 || t->Hq > 65535 || t->B > (1 << 24) || t->T > (1 << 30)) return SLA2_ERR_UNSUPPORTED;
  // rows of the token arrays and of the codes are counted in 32 bits
  if ((long long)t->T * t->Hq > 0x7fffffffLL || (long long)c->num_pages * c->Hkv > 0x7fffffffLL / c->page)
    return SLA2_ERR_UNSUPPORTED;
  s->num_pages = c->num_pages;
  s->Hkv = c->Hkv;
  s->page = c->page;
  s->lpage = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  s->d = c->d;
  s->kc = c->k_codes;
  s->vc = c->v_codes;
  s->ks = c->k_scale;
  s->vs = c->v_scale;
  s->B = t->B;
  s->T = t->T;
  s->Hq = t->Hq;
  s->g = t->Hq / c->Hkv;
  s->max_pages = t->max_pages;
  s->table = t->page_table;
  s->lens = t->kv_lens;
  s->cu = t->cu_new;
  s->status = t->status;
  s->sms = SM_COUNT;
  return SLA2_OK;
}

// The view's strides, those of extents of 1 replaced by ones that the checks take.
bool view_ok(const sla2_view* v, int T, int H, int d, View3* o) {
  if (!v || !v->data || !aligned16(v->data)) return false;
  *o = {v->data, T > 1 ? v->stride_n : d, H > 1 ? v->stride_h : d};
  return o->st >= d && o->sh >= d && o->st % 8 == 0 && o->sh % 8 == 0 && o->st < (1LL << 39) && o->sh < (1LL << 39);
}

#define SLA2_TRY(expr)                                   \
  do {                                                   \
    if ((expr) != cudaSuccess) return SLA2_ERR_CUDA;     \
  } while (0)

cudaError_t clear_status(unsigned* status, cudaStream_t st) {
  return status ? cudaMemsetAsync(status, 0, sizeof(unsigned), st) : cudaSuccess;
}

}  // namespace

extern "C" {

sla2_status sla2_cache_append(const sla2_cache* cache, const sla2_step* step, const sla2_view* k, const sla2_view* v,
                              const sla2_view* q, const sla2_view* q_out, const sla2_view* k_out, const float* cos,
                              const float* sin, int rope_rows, int rope_dim, int interleaved, void* stream) {
  CacheShape s;
  const sla2_status r = check_step(cache, step, &s);
  if (r != SLA2_OK) return r;
  AppendArgs a{};
  if (!view_ok(k, s.T, s.Hkv, s.d, &a.k) || !view_ok(v, s.T, s.Hkv, s.d, &a.v)) return SLA2_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return SLA2_ERR_INVALID_ARG;
  if (q && (!view_ok(q, s.T, s.Hq, s.d, &a.q) || !view_ok(q_out, s.T, s.Hq, s.d, &a.q_out))) return SLA2_ERR_INVALID_ARG;
  if (k_out && !view_ok(k_out, s.T, s.Hkv, s.d, &a.k_out)) return SLA2_ERR_INVALID_ARG;
  for (const void* o : {a.q_out.p, a.k_out.p})
    if (o && (o == a.k.p || o == a.v.p || o == a.q.p)) return SLA2_ERR_INVALID_ARG;
  if (a.q_out.p && a.q_out.p == a.k_out.p) return SLA2_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return SLA2_ERR_INVALID_ARG;
  if ((cos == nullptr) != (sin == nullptr) || (cos == nullptr) != (rope_dim == 0)) return SLA2_ERR_INVALID_ARG;
  if (rope_dim < 0 || rope_dim > s.d || rope_dim % 16 || (rope_dim && rope_rows < 1)) return SLA2_ERR_INVALID_ARG;
  if (!aligned16(cos) || !aligned16(sin)) return SLA2_ERR_INVALID_ARG;
  a.cos = cos;
  a.sin = sin;
  a.rope_rows = rope_rows;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SLA2_TRY(clear_status(s.status, st));
  SLA2_TRY(launch_cache_append(s, step->dtype, a, st));
  return SLA2_OK;
}

size_t sla2_cache_attention_workspace_size(const sla2_cache* cache, const sla2_step* step) {
  CacheShape s;
  if (check_step(cache, step, &s) != SLA2_OK) return 0;
  return cache_attention_workspace(s);
}

sla2_status sla2_cache_attention(const sla2_cache* cache, const sla2_step* step, const sla2_view* q,
                                 const sla2_view* out, int window, int sinks, float scale, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  CacheShape s;
  const sla2_status r = check_step(cache, step, &s);
  if (r != SLA2_OK) return r;
  CacheAttnArgs a{};
  if (!view_ok(q, s.T, s.Hq, s.d, &a.q) || !view_ok(out, s.T, s.Hq, s.d, &a.out) || a.q.p == a.out.p)
    return SLA2_ERR_INVALID_ARG;
  if (window < 1 || sinks < 0 || !(scale > 0.f) || !std::isfinite(scale)) return SLA2_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < cache_attention_workspace(s) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SLA2_ERR_WORKSPACE;
  a.W = window;
  a.S = sinks;
  const long long end = ((long long)s.max_pages * s.page + CACHE_UNIT - 1) / CACHE_UNIT;
  a.end = (int)(end < 0x7fffffff ? end : 0x7fffffff);
  a.scale = scale;
  a.workspace = workspace;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SLA2_TRY(clear_status(s.status, st));
  SLA2_TRY(launch_cache_attention(s, step->dtype, a, st));
  return SLA2_OK;
}

}  // extern "C"
