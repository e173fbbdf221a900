// Appends the new tokens of a step to the paged 8-bit cache, rotating keys (and queries) on the way.
//
// One CTA per (page that a sequence touches, key head). It holds the page's new rows in registers as
// the 16-bit values that are to be quantised, takes their largest magnitude, settles the page's scale
// s = max(s of the tokens already there, max|y| / 127), rescales the earlier codes if the scale grew,
// and writes the new ones. The query heads of the key head's group are rotated by the same CTA.
//
// The result is defined to the bit: the rotation is taken in 64 bits (its products of a 16-bit and a
// 32-bit number are exact there) and rounded to 32 bits and to the type; codes are the rounding of
// the true quotient y / s. The quotient is formed in 32 bits first; its error is at most
// 127 * 1.5 * 2^-23 < 3e-5, so wherever it lies further than 1e-4 from a border between two codes
// the code is certain, and the others are divided in 64 bits.
//
// A step's page for the CTA x: sequence b owns the CTAs from cu[b] / page + 2 b on, which leaves at
// least new / page + 2 of them to each, as many as its tokens can touch; the search for b is a count
// over all sequences, one pass for the whole CTA.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "device.cuh"

namespace sla2 {

namespace {

constexpr int THREADS = 256;

template <class T>
__device__ __forceinline__ float to_f(uint16_t x);
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(uint16_t x) {
  return __uint_as_float((uint32_t)x << 16);
}
template <>
__device__ __forceinline__ float to_f<__half>(uint16_t x) {
  return __half2float(__ushort_as_half(x));
}
template <class T>
__device__ __forceinline__ uint16_t to_t(float x);
template <>
__device__ __forceinline__ uint16_t to_t<__nv_bfloat16>(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <>
__device__ __forceinline__ uint16_t to_t<__half>(float x) {
  return __half_as_ushort(__float2half_rn(x));
}
template <class T>
constexpr uint32_t INF_BITS = 0x7f80u;
template <>
constexpr uint32_t INF_BITS<__half> = 0x7c00u;

union Chunk {     // 8 elements of a row
  uint4 v;
  uint16_t e[8];
};

// Elements [8c, 8c + 8) of a row, rotated for position `pos`.
template <class T>
__device__ __forceinline__ Chunk rotated(const uint16_t* row, int c, int pos, const AppendArgs& a) {
  Chunk x;
  x.v = *reinterpret_cast<const uint4*>(row + c * 8);
  if (c * 8 >= a.rope_dim) return x;
  Chunk y;
  const int half = a.rope_dim / 2;
  const float* cr = a.cos + (size_t)pos * half;
  const float* sr = a.sin + (size_t)pos * half;
  if (a.interleaved) {
    const float4 cv = __ldg(reinterpret_cast<const float4*>(cr + c * 4));
    const float4 sv = __ldg(reinterpret_cast<const float4*>(sr + c * 4));
    const float cs[4] = {cv.x, cv.y, cv.z, cv.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double p = to_f<T>(x.e[2 * i]), q = to_f<T>(x.e[2 * i + 1]);
      y.e[2 * i] = to_t<T>((float)fma(p, (double)cs[i], -(q * (double)sn[i])));
      y.e[2 * i + 1] = to_t<T>((float)fma(q, (double)cs[i], p * (double)sn[i]));
    }
  } else {
    const bool hi = c * 8 >= half;
    const int o = hi ? c * 8 - half : c * 8;
    Chunk w;
    w.v = *reinterpret_cast<const uint4*>(row + (hi ? o : o + half));
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      *reinterpret_cast<float4*>(cs + i) = __ldg(reinterpret_cast<const float4*>(cr + o + i));
      *reinterpret_cast<float4*>(sn + i) = __ldg(reinterpret_cast<const float4*>(sr + o + i));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double p = to_f<T>(x.e[i]), q = (double)to_f<T>(w.e[i]) * (double)(hi ? sn[i] : -sn[i]);
      y.e[i] = to_t<T>((float)fma(p, (double)cs[i], q));
    }
  }
  return y;
}

__device__ __forceinline__ uint32_t code_of(float y, float s, float inv) {
  if (!(s > 0.f)) return 0u;                       // zero, or NaN: the values read are 0 or NaN whatever the code
  const float q = y * inv, c = rintf(q);
  int r = (int)c;
  if (!(fabsf(q - c) < 0.4999f)) r = (int)rint((double)y / (double)s);
  return (uint32_t)(r < -127 ? -127 : (r > 127 ? 127 : r)) & 0xffu;
}

// One tensor's part: the new rows' chunks are in x[0..n), of `rows` rows from slot c0 on.
template <class T, int D, int MAXC>
__device__ __forceinline__ void put(const Chunk (&x)[MAXC], int nch, int c0, int8_t* codes, float* scale, int* red) {
  constexpr int CPR = D / 8;
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < MAXC; ++u) {
    if (u * THREADS + (int)threadIdx.x < nch) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = x[u].e[e] & 0x7fffu;
        m = m > w ? m : w;
      }
    }
  }
  const float s_old = c0 > 0 ? *scale : 0.f;
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = (int)m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = m > (uint32_t)red[w] ? m : (uint32_t)red[w];
  const float s_new = __fdiv_rn(to_f<T>((uint16_t)m), 127.f);
  float s = fmaxf(s_old, s_new);
  if (m >= INF_BITS<T> || s_old != s_old) s = __uint_as_float(0x7fffffffu);
  if (c0 > 0 && s > s_old) {
    // earlier codes to the new scale, 16 at a time
    const double ratio = (double)s_old / (double)s;
    for (int i = threadIdx.x; i < c0 * (D / 16); i += THREADS) {
      uint4* p = reinterpret_cast<uint4*>(codes) + i;
      uint4 v = *p;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = (int)(int8_t)(w[j] >> (8 * e));
          r |= ((uint32_t)__double2int_rn((double)c * ratio) & 0xffu) << (8 * e);
        }
        w[j] = r;
      }
      *p = v;
    }
  }
  const float inv = __fdiv_rn(1.f, s);
#pragma unroll
  for (int u = 0; u < MAXC; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < nch) {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e >> 2] |= code_of(to_f<T>(x[u].e[e]), s, inv) << (8 * (e & 3));
      *reinterpret_cast<uint2*>(codes + (size_t)(c0 + i / CPR) * D + (i % CPR) * 8) = make_uint2(w[0], w[1]);
    }
  }
  __syncthreads();     // every thread has read the old scale (and `red` may be written again)
  if (threadIdx.x == 0) *scale = s;
}

template <class T, int D>
__global__ void __launch_bounds__(THREADS) cache_append_kernel(CacheShape s, AppendArgs a) {
  constexpr int CPR = D / 8, MAXC = 128 * CPR / THREADS;    // chunks a row; chunks a thread at 128 rows
  __shared__ int red[THREADS / 32];
  // the sequence whose CTAs this one belongs to
  int before = 0;
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const int b = b0 + (int)threadIdx.x;
    before += __syncthreads_count(b < s.B && (long long)(__ldg(s.cu + b) >> s.lpage) + 2LL * b <= (long long)blockIdx.x);
  }
  const int b = before > 0 ? before - 1 : 0, h = blockIdx.y;
  Span sp;
  if (!step_span(s, b, &sp)) {
    if (threadIdx.x == 0) flag_bad_index(s);
    return;
  }
  const int r = (int)blockIdx.x - (sp.t0 >> s.lpage) - 2 * b;
  const int pi = (sp.len >> s.lpage) + r;                   // page of the sequence
  const long long p0 = (long long)pi << s.lpage;            // its first position
  if (r < 0 || p0 >= (long long)sp.len + sp.n) return;
  const int first = r == 0 ? sp.len : (int)p0;              // positions [first, last) of this page are new
  int last = (int)(p0 + s.page < (long long)sp.len + sp.n ? p0 + s.page : (long long)sp.len + sp.n);
  const int pid = pi < s.max_pages ? __ldg(s.table + (size_t)b * s.max_pages + pi) : -1;
  const bool turn = a.rope_dim > 0;
  if (pid < 0 || pid >= s.num_pages || (turn && last > a.rope_rows)) {
    if (threadIdx.x == 0) flag_bad_index(s);
    if (pid < 0 || pid >= s.num_pages) return;
    last = last < a.rope_rows ? last : a.rope_rows;
    if (last <= first) return;
  }
  const int c0 = first - (int)p0, nch = (last - first) * CPR;
  const size_t ph = (size_t)pid * s.Hkv + h;
  const int t = sp.t0 + (first - sp.len);                   // row of the first token
  const uint16_t* k = static_cast<const uint16_t*>(a.k.p) + (size_t)t * a.k.st + h * a.k.sh;
  const uint16_t* v = static_cast<const uint16_t*>(a.v.p) + (size_t)t * a.v.st + h * a.v.sh;
  Chunk x[MAXC];
#pragma unroll
  for (int u = 0; u < MAXC; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < nch) {
      x[u] = rotated<T>(k + (size_t)(i / CPR) * a.k.st, i % CPR, first + i / CPR, a);
      if (a.k_out.p)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out.p) + (size_t)(t + i / CPR) * a.k_out.st +
                                  h * a.k_out.sh + (i % CPR) * 8) = x[u].v;
    }
  }
  put<T, D, MAXC>(x, nch, c0, s.kc + ph * s.page * D, s.ks + ph, red);
#pragma unroll
  for (int u = 0; u < MAXC; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < nch) x[u].v = *reinterpret_cast<const uint4*>(v + (size_t)(i / CPR) * a.v.st + (i % CPR) * 8);
  }
  put<T, D, MAXC>(x, nch, c0, s.vc + ph * s.page * D, s.vs + ph, red);
  if (a.q.p) {
    for (int i = threadIdx.x; i < nch * s.g; i += THREADS) {
      const int tok = i / (CPR * s.g), hq = h * s.g + (i / CPR) % s.g, c = i % CPR;
      const uint16_t* q = static_cast<const uint16_t*>(a.q.p) + (size_t)(t + tok) * a.q.st + hq * a.q.sh;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out.p) + (size_t)(t + tok) * a.q_out.st + hq * a.q_out.sh +
                                c * 8) = rotated<T>(q, c, first + tok, a).v;
    }
  }
}

template <class T, int D>
cudaError_t launch_t(const CacheShape& s, const AppendArgs& a, cudaStream_t st) {
  cache_append_kernel<T, D><<<dim3((s.T >> s.lpage) + 2 * s.B, s.Hkv), THREADS, 0, st>>>(s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheShape& s, int fp16, const AppendArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
