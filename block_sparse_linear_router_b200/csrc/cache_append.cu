// Appends the new tokens of a step to the paged 8-bit cache, rotating keys (and queries) on the way.
//
// A CTA of kind K or V takes one page that a sequence touches, of one key head. It holds the page's
// new rows in registers as the 16-bit values that are to be quantised, takes their largest magnitude,
// settles the page's scale s = max(s of the tokens already there, max|y| / 127), rescales the earlier
// codes if the scale grew, and writes the new ones. A CTA of kind Q rotates 32 rows of that page's
// tokens, of the query heads of one key head. The three kinds are CTAs of their own so that a single
// token waits for one chain of loads, not for three in turn.
//
// The result is defined to the bit: the rotation is taken in 64 bits (its products of a 16-bit and a
// 32-bit number are exact there) and rounded to 32 bits and to the type; codes are the rounding of
// the true quotient y / s. Both are formed in 32 bits first, with a bound on the error, and again in
// 64 bits only where the bound does not settle the rounding: conversions to and from 64 bits run at
// an eighth of the rate of 32-bit arithmetic, and with all values in 64 bits they were the bound.
//
// Bytes are the floor: 12306 new tokens of five prompts, 12 query and 4 key heads of 128, fp16, half of
// the channels turned, 32.2 us, 3.6 TB/s of 117 MB. The arithmetic of both roundings fills 2.4 of 4 issue
// slots; with nothing left to 64 bits it would be 29 us. All in 64 bits and one CTA for the three kinds:
// 56.5 us. 32 sequences with a new token each, 8 key heads: 6.4 us, the latency of a chain of four loads.
//
// A step's page for the CTA x: sequence b owns the CTAs from min(cu[b], cu[b] / page + 2 b) on. That
// leaves it at least min(new, new / page + 2), as many as the pages that its tokens can touch. The
// search for b is one pass over all sequences, each thread asking whether x is its sequence's; where
// offsets ascend that is one at most, and sequences behind a pair that does not are left out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "device.cuh"

namespace sla2 {

namespace {

// With 512 threads five prompts of 12306 tokens take 34 us, with 256 and no more than three blocks an
// SM 33.3, with four of them 32.4: what is waited for is loads, so warps count more than a few spills.
constexpr int THREADS = 256, BLOCKS = 4;

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
__device__ __forceinline__ float2 unpack_t(uint32_t x) {
  return make_float2(to_f<T>((uint16_t)x), to_f<T>((uint16_t)(x >> 16)));
}
template <class T>
__device__ __forceinline__ uint32_t pack_t(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_t<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack_t<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <class T>
constexpr uint32_t INF_BITS = 0x7f80u;
template <>
constexpr uint32_t INF_BITS<__half> = 0x7c00u;

constexpr int QROWS = 32;      // rows of a CTA of kind Q

struct Pair {                  // two chunks of 8 elements of a row, the elements that turn with each other
  uint32_t w[8];
};

// The columns of pair p's two chunks: those that turn with each other, and past rope_dim the next two.
struct Columns {
  int c0, c1;
  bool turn;
};
template <bool INTER>
__device__ __forceinline__ Columns columns(int p, int rope_dim) {
  const int half = rope_dim >> 4;        // pairs that turn
  if (INTER || p >= half) return {p * 16, p * 16 + 8, p < half};
  return {p * 8, (p + half) * 8, true};
}
__device__ __forceinline__ Pair load_pair(const uint16_t* row, const Columns& c) {
  Pair x;
  *reinterpret_cast<uint4*>(x.w) = *reinterpret_cast<const uint4*>(row + c.c0);
  *reinterpret_cast<uint4*>(x.w + 4) = *reinterpret_cast<const uint4*>(row + c.c1);
  return x;
}
__device__ __forceinline__ void store_pair(uint16_t* row, const Columns& c, const Pair& x) {
  *reinterpret_cast<uint4*>(row + c.c0) = *reinterpret_cast<const uint4*>(x.w);
  *reinterpret_cast<uint4*>(row + c.c1) = *reinterpret_cast<const uint4*>(x.w + 4);
}

struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ Angles load_angles(int p, int pos, const AppendArgs& a) {
  Angles g;
  const size_t o = (size_t)pos * (a.rope_dim >> 1) + p * 8;
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(g.c + i) = __ldg(reinterpret_cast<const float4*>(a.cos + o + i));
    *reinterpret_cast<float4*>(g.s + i) = __ldg(reinterpret_cast<const float4*>(a.sin + o + i));
  }
  return g;
}

// Two angles' outputs again, in 64 bits: first members p c - q s in a's halves, second ones q c + p s in b's.
template <class T>
__device__ __noinline__ uint2 turned64(float2 p, float2 q, float2 c, float2 s) {
  const uint32_t a0 = to_t<T>((float)fma((double)p.x, (double)c.x, -((double)q.x * (double)s.x)));
  const uint32_t a1 = to_t<T>((float)fma((double)p.y, (double)c.y, -((double)q.y * (double)s.y)));
  const uint32_t b0 = to_t<T>((float)fma((double)q.x, (double)c.x, (double)p.x * (double)s.x));
  const uint32_t b1 = to_t<T>((float)fma((double)q.y, (double)c.y, (double)p.y * (double)s.y));
  return make_uint2(a0 | a1 << 16, b0 | b1 << 16);
}

// Numbers below and above t = p c + (a product, whose rounding is m). With r = fl(p c + m), t is within
// 2^-24 (|m| + |r|) + 2^-149 of r, and r -+ err round by 2^-24 |r| more; err holds both, and 2^-12 of
// itself for its own rounding.
__device__ __forceinline__ float2 bracket(float p, float c, float m) {
  const float r = fmaf(p, c, m), err = fmaf(fabsf(m), 0x1.001p-24f, fmaf(fabsf(r), 0x1.001p-23f, 1e-43f));
  return make_float2(r - err, r + err);
}

// The pair turned: p c - q s and q c + p s, in 32 bits where that settles the result. Rounding to a
// type is monotone: where the numbers around t round to the same finite value, so does t, by way of
// 64 and of 32 bits as well; one word in a thousand or so is left to 64 bits. INTER: elements 2i and
// 2i + 1 are the members of angle i, else element i of the first chunk and of the second.
template <class T, bool INTER>
__device__ __forceinline__ Pair turned(const Pair& x, const Angles& g) {
  Pair y;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t u = INTER ? x.w[i] : x.w[i >> 1], v = INTER ? x.w[i + 1] : x.w[4 + (i >> 1)];
    const float2 uf = unpack_t<T>(u), vf = unpack_t<T>(v);
    const float2 p = INTER ? make_float2(uf.x, vf.x) : uf, q = INTER ? make_float2(uf.y, vf.y) : vf;
    const float2 c = make_float2(g.c[i], g.c[i + 1]), s = make_float2(g.s[i], g.s[i + 1]);
    const float2 a0 = bracket(p.x, c.x, -(q.x * s.x)), a1 = bracket(p.y, c.y, -(q.y * s.y));
    const float2 b0 = bracket(q.x, c.x, p.x * s.x), b1 = bracket(q.y, c.y, p.y * s.y);
    uint32_t a, b, a2, b2;     // the words that go out
    if (INTER) {
      a = pack_t<T>(a0.x, b0.x), b = pack_t<T>(a1.x, b1.x);
      a2 = pack_t<T>(a0.y, b0.y), b2 = pack_t<T>(a1.y, b1.y);
    } else {
      a = pack_t<T>(a0.x, a1.x), b = pack_t<T>(b0.x, b1.x);
      a2 = pack_t<T>(a0.y, a1.y), b2 = pack_t<T>(b0.y, b1.y);
    }
    const uint32_t top = __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
    if (a != a2 || b != b2 || (top >> 16) >= INF_BITS<T> || (top & 0xffffu) >= INF_BITS<T>) {
      const uint2 t = turned64<T>(p, q, c, s);
      a = INTER ? __byte_perm(t.x, t.y, 0x5410) : t.x;
      b = INTER ? __byte_perm(t.x, t.y, 0x7632) : t.y;
    }
    y.w[INTER ? i : i >> 1] = a;
    y.w[INTER ? i + 1 : 4 + (i >> 1)] = b;
  }
  return y;
}

// To the nearest whole number, |x| < 2^22, ties to even: the low bits of the sum hold it.
constexpr float MAGIC = 12582912.f;      // 1.5 * 2^23
// A quotient within 127 that is off by 127 * 2^-23 < 1.6e-5 at most is rounded for certain this near to a whole number.
constexpr float SURE = 0.49998f;

// The code of y in 64 bits.
__device__ __noinline__ uint32_t code64(float y, float s) {
  const int r = (int)rint((double)y / (double)s);
  return (uint32_t)(r < -127 ? -127 : (r > 127 ? 127 : r)) & 0xffu;
}
// Codes of 4 elements. y / s is formed as y (1 / s), two roundings of 2^-24. |y| is at most 127 s but for
// the rounding of s, so no code leaves -127..127.
template <class T>
__device__ __forceinline__ uint32_t codes_of(uint32_t x0, uint32_t x1, float s, float inv) {
  if (!(s > 0.f)) return 0u;       // zero, or NaN: the values read are 0 or NaN whatever the code
  const float2 u = unpack_t<T>(x0), v = unpack_t<T>(x1);
  const float y[4] = {u.x, u.y, v.x, v.y};
  uint32_t w[4];
  bool sure = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = y[e] * inv, m = q + MAGIC;
    sure = sure && fabsf(q - (m - MAGIC)) < SURE;
    w[e] = __float_as_uint(m);
  }
  uint32_t r = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  if (!sure) {
    r = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) r |= code64(y[e], s) << (8 * e);
  }
  return r;
}

// Four codes at the scale s_old as codes at the larger scale s, the rounding of c s_old / s.
__device__ __noinline__ uint32_t rescaled64(uint32_t w, float s_old, float s) {
  uint32_t r = 0u;
  const double ratio = (double)s_old / (double)s;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r |= ((uint32_t)__double2int_rn((double)(int)(int8_t)(w >> (8 * e)) * ratio) & 0xffu) << (8 * e);
  return r;
}
// `ratio` is the quotient in 32 bits: two roundings again.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio, float s_old, float s) {
  uint32_t r = 0u;
  bool sure = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = (float)(int)(int8_t)(w >> (8 * e)) * ratio, m = q + MAGIC;
    sure = sure && fabsf(q - (m - MAGIC)) < SURE;
    r |= (__float_as_uint(m) & 0xffu) << (8 * e);
  }
  return sure ? r : rescaled64(w, s_old, s);
}

// The first CTA of sequence b.
__device__ __forceinline__ int first_cta(const CacheShape& s, int b, const Span& sp) {
  const long long o = (long long)(sp.t0 >> s.lpage) + 2LL * b;
  return (int)(o < sp.t0 ? o : sp.t0);
}

template <class T, int D, bool INTER>
__global__ void __launch_bounds__(THREADS, BLOCKS) cache_append_kernel(CacheShape s, AppendArgs a) {
  constexpr int PPR = D / 16, MAXP = 128 * PPR / THREADS;    // pairs a row; pairs a thread at 128 rows
  __shared__ uint32_t red[THREADS / 32];
  __shared__ int who;
  const int h = blockIdx.y, kind = blockIdx.z;               // 0: keys, 1: values, 2 and up: 32 rows of queries each
  // the sequence whose CTAs this one belongs to
  bool found = false, cut = false;
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const Span sp = block_span(s, b0 + (int)threadIdx.x, &cut, blockIdx.x == 0 && h == 0 && kind == 0);
    const int r = (int)blockIdx.x - first_cta(s, b0 + (int)threadIdx.x, sp);
    const bool mine = sp.n > 0 && r >= 0 && r <= ((sp.len + sp.n - 1) >> s.lpage) - (sp.len >> s.lpage);
    if (mine) who = b0 + (int)threadIdx.x;
    found |= __syncthreads_or(mine) != 0;
  }
  if (!found) return;
  const int b = who;
  Span sp;
  step_span(s, b, &sp);
  const int r = (int)blockIdx.x - first_cta(s, b, sp);
  const long long pi = (long long)(sp.len >> s.lpage) + r;  // page of the sequence
  const long long p0 = pi << s.lpage;                       // its first position
  const int first = r == 0 ? sp.len : (int)p0;              // positions [first, last) of this page are new
  int last = (int)(p0 + s.page < (long long)sp.len + sp.n ? p0 + s.page : (long long)sp.len + sp.n);
  const int pid = pi < s.max_pages ? __ldg(s.table + (size_t)b * s.max_pages + pi) : -1;
  if (pid < 0 || pid >= s.num_pages || (a.rope_dim > 0 && last > a.rope_rows)) {
    if (threadIdx.x == 0) flag_bad_index(s);
    if (pid < 0 || pid >= s.num_pages) return;
    last = last < a.rope_rows ? last : a.rope_rows;
    if (last <= first) return;
  }
  const int t = sp.t0 + (first - sp.len);                   // row of the first token
  if (kind >= 2) {
    // queries: one pair of a row, and as many of the heads as there are threads left for
    const int f = (kind - 2) * QROWS, rows = last - first - f < QROWS ? last - first - f : QROWS, n = rows * PPR;
    if (n <= 0) return;
    const int i = (int)threadIdx.x % n, step = THREADS / n;
    const Columns c = columns<INTER>(i % PPR, a.rope_dim);
    const int row = f + i / PPR;
    const size_t tok = (size_t)t + row;
    Angles g{};
    if (c.turn) g = load_angles(i % PPR, first + row, a);
    int hq = (int)threadIdx.x / n;
    if (hq >= step) return;
    const uint16_t* src = static_cast<const uint16_t*>(a.q.p) + tok * a.q.st + h * s.g * a.q.sh;
    uint16_t* dst = static_cast<uint16_t*>(a.q_out.p) + tok * a.q_out.st + h * s.g * a.q_out.sh;
    Pair x{};
    if (hq < s.g) x = load_pair(src + hq * a.q.sh, c);
    while (hq < s.g) {
      const int next = hq + step;
      Pair y{};
      if (next < s.g) y = load_pair(src + next * a.q.sh, c);
      if (c.turn) x = turned<T, INTER>(x, g);
      store_pair(dst + hq * a.q_out.sh, c, x);
      x = y;
      hq = next;
    }
    return;
  }
  const int c0 = first - (int)p0, n = (last - first) * PPR;
  const size_t ph = (size_t)pid * s.Hkv + h;
  const View3 in = kind ? a.v : a.k;
  int8_t* codes = (kind ? s.vc : s.kc) + ph * s.page * D;
  float* scale = (kind ? s.vs : s.ks) + ph;
  const float s_old = c0 > 0 ? *scale : 0.f;
  const uint16_t* src = static_cast<const uint16_t*>(in.p) + (size_t)t * in.st + h * in.sh;
  Pair x[MAXP];
#pragma unroll
  for (int u = 0; u < MAXP; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < n) x[u] = load_pair(src + (size_t)(i / PPR) * in.st, columns<INTER>(i % PPR, a.rope_dim));
  }
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < MAXP; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < n) {
      const Columns c = columns<INTER>(i % PPR, a.rope_dim);
      if (kind == 0) {
        if (c.turn) x[u] = turned<T, INTER>(x[u], load_angles(i % PPR, first + i / PPR, a));
        if (a.k_out.p)
          store_pair(static_cast<uint16_t*>(a.k_out.p) + (size_t)(t + i / PPR) * a.k_out.st + h * a.k_out.sh, c, x[u]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) m = __vmaxu2(m, x[u].w[e] & 0x7fff7fffu);
    }
  }
  m = m >> 16 > (m & 0xffffu) ? m >> 16 : m & 0xffffu;
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();                                           // every thread has read the old scale, too
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = m > red[w] ? m : red[w];
  const float s_new = __fdiv_rn(to_f<T>((uint16_t)m), 127.f);
  float sc = fmaxf(s_old, s_new);
  if (m >= INF_BITS<T> || s_old != s_old) sc = __uint_as_float(0x7fffffffu);
  if (threadIdx.x == 0) *scale = sc;
  if (c0 > 0 && sc > s_old) {
    // earlier codes to the new scale, 16 at a time
    const float ratio = __fdiv_rn(s_old, sc);
    for (int i = threadIdx.x; i < c0 * (D / 16); i += THREADS) {
      uint4* p = reinterpret_cast<uint4*>(codes) + i;
      uint4 v = *p;
      v.x = rescaled(v.x, ratio, s_old, sc);
      v.y = rescaled(v.y, ratio, s_old, sc);
      v.z = rescaled(v.z, ratio, s_old, sc);
      v.w = rescaled(v.w, ratio, s_old, sc);
      *p = v;
    }
  }
  const float inv = __fdiv_rn(1.f, sc);
#pragma unroll
  for (int u = 0; u < MAXP; ++u) {
    const int i = u * THREADS + (int)threadIdx.x;
    if (i < n) {
      const Columns c = columns<INTER>(i % PPR, a.rope_dim);
      int8_t* to = codes + (size_t)(c0 + i / PPR) * D;
      *reinterpret_cast<uint2*>(to + c.c0) =
          make_uint2(codes_of<T>(x[u].w[0], x[u].w[1], sc, inv), codes_of<T>(x[u].w[2], x[u].w[3], sc, inv));
      *reinterpret_cast<uint2*>(to + c.c1) =
          make_uint2(codes_of<T>(x[u].w[4], x[u].w[5], sc, inv), codes_of<T>(x[u].w[6], x[u].w[7], sc, inv));
    }
  }
}

template <class T, int D>
cudaError_t launch_t(const CacheShape& s, const AppendArgs& a, cudaStream_t st) {
  const int most = (s.T >> s.lpage) + 2 * s.B;
  const dim3 grid(most < s.T ? most : s.T, s.Hkv, a.q.p ? 2 + (s.page + QROWS - 1) / QROWS : 2);
  if (a.interleaved)
    cache_append_kernel<T, D, true><<<grid, THREADS, 0, st>>>(s, a);
  else
    cache_append_kernel<T, D, false><<<grid, THREADS, 0, st>>>(s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheShape& s, int fp16, const AppendArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
