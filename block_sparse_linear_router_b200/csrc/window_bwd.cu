// Gradients of sliding-window attention with sinks. With P = exp(scale Q K^T - lse) on the visible
// pairs, delta = rowsum(dO * O) and dS = P (dO V^T - delta):
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
// Kernels: delta; dQ, a query tile (128 rows) per item, over the key tiles that it sees; dK and dV, key tile
// (128 keys) by key tile, over the query tiles that see it; and the sum of what two CTAs have of one key
// tile. S and dO V^T are formed in both of the middle two (seven products instead of five): nothing is
// then summed across CTAs, so there are no atomics, and a gradient is the same bits from run to run. The
// sum over the query heads that share a key head is part of the key tile's item.
//
// Roundings to 16 bits: P and dS as operands, and O, which delta is formed from. Were dS rounded for both of
// its products and delta taken as it is, dQ and dK would be off by 1.5 times what rounding them alone
// costs (bf16, windows of 8 to 400 keys; 2.2 times at 2 keys). So dQ takes dS as the sum of two
// 16-bit numbers (its fourth product: 168 us without, 217 with it), and adds up each row's dS: their sum
// is zero but for delta's error, which dK then takes away. dQ and dK are off by 1.1 and 1.4 times the
// rounding alone from 8 keys on, whatever the size of dO, where the logits' standard deviation is 1. dQ keeps
// delta's error, which weighs more the more a row's weight sits on few keys: at 2 it is off by 1.3 times, at 4
// by 2.1, at 8 by 3.2 (dK by 1.4 throughout). A product of P and K, another sixth of dQ's kernel, would take it away.
//
// 16384 tokens, 12 heads of 128, window 1024, 64 sinks, causal, bf16, each alone: delta 25 us (4 TB/s), dQ
// 221 us (720 TFLOP/s of three products' visible pairs, tensor pipe busy 63%), dK and dV 283 us (750 TFLOP/s
// of four products, 50%), the sum 12 us; 615 to 627 us with the forward pass. fp16: delta and the largest rows 46 us,
// dQ 228, dK and dV 305. What bounds the large two is a step's chain from S to dS, which two waits a step and
// single-tile buffers do not hide whole; of d = 128 tensor memory (512 columns) has no room for a second key
// tile's accumulators (of d = 64, pipe busy 27%, it would have one for dP). Without the exponentials dK and dV
// take 7% less, without their loads 2%.
//
// delta and what dQ adds to it are written by kernels that a reader's launch may overlap with: they are read through L2
// (ld.cg) behind griddepcontrol.wait, not as data that no kernel writes (ld.nc).
//
// Both tensor-core kernels are persistent, one CTA of 384 threads per SM:
//   warps 0-7  thread t of a warpgroup owns TMEM lane t % 128, the warpgroups split the 128 columns of
//              S and dP; P and dS go back over their own columns as 16-bit A operands.
//   warp 8     TMA producer. Rows behind a sequence's end may hold anything: a tile that has some is
//              completed by the producer, which zeroes them before it hands the tile on.
//   warp 9     tcgen05 issuer.
//   warp 10    (dK, dV) brings each query tile's lse and delta into shared memory.
#include "device.cuh"
#include "kernels.cuh"
#include "window.cuh"
#include "window_tile.cuh"

namespace sla2 {

namespace {

constexpr int THREADS = 384;
constexpr int MIN_SHARE = 4;               // steps of dK, dV that a CTA takes at least

template <class T>
__device__ __forceinline__ float2 unpack16(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack16<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 unpack16<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}

// delta: one row per D / 8 lanes, 16 bytes of each tensor a lane; zero behind the sequence's end.
// Of rows that see FEW keys at most (a narrow window, a short sequence, the first rows of a causal one), delta = sum of
// P (dO V^T) over them instead. O has been rounded, and with few keys dP - delta is the difference of numbers
// that are nearly the same: at 2 keys dQ was off by 1.9 times what rounding it costs, so by as much as that.
constexpr int FEW = 8;
// The keys that row i sees in order: `before` sinks, the window's from lo to hi, and sinks behind those.
struct RowKeys {
  int before, lo, hi, after;
  __device__ __forceinline__ RowKeys(const WindowShape& s, int n, int i) {
    const int sinks = s.S < n ? s.S : n;
    lo = i - s.W + 1 > 0 ? i - s.W + 1 : 0;
    hi = s.causal ? i : (s.W < n - i ? i + s.W - 1 : n - 1);
    before = sinks < lo ? sinks : lo;
    after = !s.causal && sinks > hi + 1 ? sinks - hi - 1 : 0;
  }
  __device__ __forceinline__ int count() const { return before + (hi - lo + 1) + after; }
  __device__ __forceinline__ int at(int u) const { return u < before ? u : lo + (u - before); }      // behind hi sinks follow
};
inline bool narrow(const WindowShape& s) { return (long long)s.W * (s.causal ? 1 : 2) - (s.causal ? 0 : 1) + s.S <= FEW; }      // every row
// Where the window is not narrow itself, such rows are among the first FEW of a sequence and, if it is not causal, the last.
__device__ __forceinline__ bool few_keys(const WindowShape& s, int n, int i) {
  return (i < FEW || (!s.causal && i >= n - FEW)) && RowKeys(s, n, i).count() <= FEW;
}

template <class T>
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  const uint32_t us[4] = {a.x, a.y, a.z, a.w}, ws[4] = {b.x, b.y, b.z, b.w};
  float x = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = unpack16<T>(us[e]), q = unpack16<T>(ws[e]);
    x = fmaf(p.x, q.x, fmaf(p.y, q.y, x));
  }
  return x;
}
template <int LPR>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int off = LPR / 2; off; off >>= 1) x += __shfl_xor_sync(~0u, x, off);
  return x;
}

// The scale of the logits stays out of dS and goes into dQ and dK in fp32. fp16's dS is also multiplied by a power of
// two, `up`, that takes a bound on it, 2 |dO_i| |V_j| of the largest rows of a key head and its query heads, to
// between 2^13 and 2^15; 1 / up goes into the gradients with the scale. With scale P (dP - delta) as it is,
// gradients of dout around 1e-3 were off by 16 times their rounding, of 1e-5 by 26%, since dS lay below fp16's
// normal range, and a large dout made it infinite. bf16 has fp32's range: up is 1 and nothing is looked for.
// The largest rows: `warps` warps (8: a thread block; 1 where a key head has few rows) have one of `chunks` parts of a
// key head's rows, and write the squares of its largest |dO_i| and |V_j| to sizes[b][hk][0, 1][chunk]; who
// needs them reads a key head's 2 x chunks words, a lane each.
// fp16's P for dV is 2^15 P, too, and up 2^-15 of itself there: weights of 1 / 83679 lay between two of fp16's
// smallest numbers, and dV was off by 0.25%.
template <class T>
constexpr bool SIZED = std::is_same<T, __half>::value;
template <class T>
constexpr float P_UP = SIZED<T> ? 15.f : 0.f;        // log2
constexpr float P_DOWN = 1.f / 32768.f;
__device__ __forceinline__ float one_over(float power_of_two) { return __uint_as_float((254u << 23) - __float_as_uint(power_of_two)); }
struct Sizes {
  uint32_t o, v;                             // of this lane's chunk
  __device__ __forceinline__ float up() const {
    const float x = __uint_as_float(__reduce_max_sync(~0u, o)) * __uint_as_float(__reduce_max_sync(~0u, v));
    const int e2 = (int)(__float_as_uint(x) >> 23) - 127;
    const int e = 14 - ((e2 + 2) >> 1);      // |dO| |V| < 2^((e2 + 1) / 2); e from -51 to 77
    return __uint_as_float((uint32_t)(127 + e) << 23);
  }
};
struct SizesAt {
  uint32_t* p;
  int chunks, warps;                         // at most 32; 1 or 8
  __device__ __forceinline__ Sizes read(const WindowShape& s, int b, int hk, int lane) const {
    const uint32_t* at = p + ((long long)b * s.Hkv + hk) * 2 * chunks + lane;
    return lane < chunks ? Sizes{__ldcg(at), __ldcg(at + chunks)} : Sizes{0u, 0u};
  }
};
template <class T, int D>
__device__ __forceinline__ void find_sizes(const WindowShape& s, const View4& dout, const View4& v, const SizesAt& to, unsigned block) {
  constexpr int LPR = D / 8;
  __shared__ uint32_t red[2][8];
  const unsigned unit = (block * 8 + threadIdx.x / 32) / to.warps;
  const unsigned word = unit / to.chunks, chunk = unit - word * to.chunks, b = word / s.Hkv, hk = word - b * s.Hkv;
  uint32_t mo = 0, mv = 0;
  if (b < (unsigned)s.B) {
    const int n = window_len(s, b), t = threadIdx.x % (32 * to.warps), step = 32 * to.warps / LPR;
    const int r0 = (int)((long long)n * chunk / to.chunks), r1 = (int)((long long)n * (chunk + 1) / to.chunks);
    auto rows = [&](const View4& x, int h) {
      const T* p = static_cast<const T*>(x.p) + b * x.sb + h * x.sh + t % LPR * 8;
      float most = 0.f;
#pragma unroll 4
      for (int r = r0; r < r1; r += step) {
        const int i = r + t / LPR < r1 ? r + t / LPR : r0;
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(p + i * x.sn));
        most = fmaxf(most, sum_lanes<LPR>(dot8<T>(y, y)));
      }
      return __float_as_uint(most);
    };
    mv = rows(v, hk);
    for (int h = 0; h < s.g; ++h) mo = max(mo, rows(dout, hk * s.g + h));
  }
  mo = __reduce_max_sync(~0u, mo);
  mv = __reduce_max_sync(~0u, mv);
  if (to.warps == 8) {
    if (threadIdx.x % 32 == 0) red[0][threadIdx.x / 32] = mo, red[1][threadIdx.x / 32] = mv;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) mo = max(mo, red[0][w]), mv = max(mv, red[1][w]);
  }
  if (threadIdx.x % (32 * to.warps) == 0 && b < (unsigned)s.B) {
    uint32_t* at = to.p + (long long)word * 2 * to.chunks + chunk;
    at[0] = mo;
    at[to.chunks] = mv;
  }
}
SizesAt sizes_at(const WindowShape& s, uint32_t* p) {      // enough blocks for the device, of 64 rows or more
  const long long heads = (long long)s.B * s.Hkv, rows = (long long)s.N * s.g, want = (592 + heads - 1) / heads, most = (rows + 63) / 64;
  const long long c = want < most ? want : most;
  return {p, c > 32 ? 32 : (int)c, rows > 64 ? 8 : 1};
}
unsigned size_blocks(const WindowShape& s, const SizesAt& a) { return (unsigned)(((long long)s.B * s.Hkv * a.chunks * a.warps + 7) / 8); }

// delta of the row i of (b, h), a warp's 32 / (D / 8) rows side by side; `live`: this one sees few keys.
template <class T, int D>
__device__ __forceinline__ void few_delta(const WindowShape& s, const View4& q, const View4& k, const View4& v, const View4& dout,
                                          const float* lse, float* delta, int b, int h, int i, int n, bool live) {
  constexpr int LPR = D / 8;
  const int c = threadIdx.x % LPR;
  auto chunk = [&](const View4& t, int h, int i) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(t.p) + b * t.sb + h * t.sh + i * t.sn) + c);
  };
  const long long row = ((long long)b * s.Hq + h) * s.N + i;
  const RowKeys keys(s, n, i);
  const int count = live ? keys.count() : 0, most = __reduce_max_sync(~0u, count);
  const uint4 qc = live ? chunk(q, h, i) : make_uint4(0, 0, 0, 0), oc = live ? chunk(dout, h, i) : make_uint4(0, 0, 0, 0);
  const float nl = live ? -lse[row] * W_LOG2E : 0.f;
  float x = 0.f;
  for (int u = 0; u < most; ++u) {
    float dot = 0.f, dp = 0.f;
    if (u < count) {
      dot = dot8<T>(qc, chunk(k, h / s.g, keys.at(u)));
      dp = dot8<T>(oc, chunk(v, h / s.g, keys.at(u)));
    }
    dot = sum_lanes<LPR>(dot);
    dp = sum_lanes<LPR>(dp);
    if (u < count) x = fmaf(ex2_approx(fmaf(dot, s.scale * W_LOG2E, nl)), dp, x);
  }
  if (live && c == 0) delta[row] = x;
}

// The first `few` blocks take the rows that see few keys, where others see more; the next, up to `blocks`, look for the
// largest rows (fp16). Beside the sums of the others each of the three costs them registers or a branch a row: 24 us of
// 16384 tokens and 12 heads of 128 as it is, 31 to 40 with the rows of few keys in line.
template <class T, int D, bool NARROW>
__global__ void __launch_bounds__(256, NARROW ? 1 : SIZED<T> ? 5 : 8)
    window_delta_kernel(WindowShape s, View4 q, View4 k, View4 v, View4 o, View4 dout, const float* lse, float* delta, SizesAt sizes,
                        unsigned few, unsigned blocks) {
  constexpr int LPR = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!NARROW && blockIdx.x < few) {
    const int ends = s.causal ? FEW : 2 * FEW;
    const unsigned long long slot = (unsigned long long)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const unsigned bh = (unsigned)(slot / ends), e = (unsigned)(slot % ends);
    const bool in = bh < (unsigned)(s.B * s.Hq);
    const int b = in ? bh / s.Hq : 0, h = in ? bh - b * s.Hq : 0, n = window_len(s, b);
    const int i = e < FEW ? e : n - 2 * FEW + (int)e;
    few_delta<T, D>(s, q, k, v, dout, lse, delta, b, h, i, n, in && i < n && (e < FEW || i >= FEW) && few_keys(s, n, i));
    return;
  }
  if (SIZED<T> && blockIdx.x < blocks) {
    find_sizes<T, D>(s, dout, v, sizes, blockIdx.x - few);
    return;
  }
  const unsigned N = s.N, row = (blockIdx.x - blocks) * (256 / LPR) + threadIdx.x / LPR, bhu = row / N;
  const int c = threadIdx.x % LPR;
  const bool in = row < (unsigned)(s.B * s.Hq) * N;        // below 2^31
  const int bh = in ? bhu : 0, i = row - bhu * N, b = bh / s.Hq, h = bh - b * s.Hq;
  const int n = window_len(s, b);
  const bool live = in && i < n;
  if (NARROW) {
    few_delta<T, D>(s, q, k, v, dout, lse, delta, b, h, i, n, live);
    if (in && !live && c == 0) delta[row] = 0.f;
    return;
  }
  auto chunk = [&](const View4& t) {
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(t.p) + b * t.sb + h * t.sh + i * t.sn) + c);
  };
  float x = 0.f;
  if (live) x = dot8<T>(chunk(o), chunk(dout));
  x = sum_lanes<LPR>(x);
  if (in && c == 0 && !(live && few_keys(s, n, i))) delta[row] = x;
}

template <int D>
struct Cfg {
  static constexpr int SLABS = D / 64;
  static constexpr int TILE = WT * D * 2;
  static constexpr int NST = D == 128 ? 5 : 8;             // ring of single tiles: Q, dO, Q, dO, ... (dQ: K, V, ...)
  static constexpr int NAUX = 2;                           // lse / delta rows of a query tile (dK, dV)
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_AUX = OFF_RING + NST * TILE;
  static constexpr int OFF_BAR = OFF_AUX + NAUX * 1024;
  static constexpr int NBAR = 4 + 2 * NST + 2 * NAUX + 12;
  static constexpr int OFF_MISC = OFF_BAR + ((8 * NBAR + 15) / 16) * 16;
  static constexpr int SMEM = OFF_MISC + 16;               // the base is 1024-byte aligned
  static_assert(SMEM <= 232448, "dynamic shared memory per CTA (227 KB)");
};

// Lane q of four gets chunk q of each of their rows: x[k] of it becomes x[q] of lane k.
__device__ __forceinline__ void transpose4(uint4 (&x)[4], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
      uint4& lo = x[k];
      uint4& hi = x[k | bit];
      uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
      uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t y = __shfl_xor_sync(~0u, up ? a[e] : b[e], bit);
        if (up)
          a[e] = y;
        else
          b[e] = y;
      }
    }
  }
}
__device__ __forceinline__ void scale_all(uint32_t (&x)[32], float f) {
#pragma unroll
  for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
}
// 32 columns of this thread's accumulator row to the tensor's row `dst` (zeros if not live). Four lanes write 64
// bytes of a row together: with a row a lane each store touched 32 lines, and the stores of a tile
// took 4096 cycles.
template <class T>
__device__ __forceinline__ void store_row(T* dst, long long stride, int row, int N, const uint32_t (&o)[32], bool live, int lane) {
  uint4 x[4];
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t* w = reinterpret_cast<uint32_t*>(x + ch);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = live ? pack16<T>(__uint_as_float(o[ch * 8 + 2 * e]), __uint_as_float(o[ch * 8 + 2 * e + 1])) : 0u;
  }
  transpose4(x, lane);
  const int q = lane & 3;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (row - q + k < N) *reinterpret_cast<uint4*>(dst + (k - q) * stride + q * 8) = x[k];
}

// ------------------------------------------------------------------ dK, dV
// The steps (a key tile of one key head, a query tile of one of its query heads) form one line, key
// tile by key tile, and every CTA takes an equal, contiguous share of it: key tiles that hold a sink
// are seen by every query behind them, others by a window's worth. A key tile that one CTA has whole
// is written there; pieces of others go to the workspace in fp32 and are summed, in order, by a
// kernel of their own.
//
// TMEM columns: [0, 128) S^T, then dP^T of the same step (rows: keys, columns: queries), [128, 192) P,
// [192, 256) dS, both as 16-bit operands, [256, 256 + D) dV, [384, 384 + D) dK. The warps take a
// tile of S into registers at once, so that dP = V dO^T may follow it in the same columns while P is
// formed, and S of the next step while dS is; dV += P^T dO and dK += dS^T Q of the step before run
// beside dP. (With P over S and dS over dP, S of the next step waited for P, and a step took
// 3500 cycles; the four products take 2150.)

// Query tiles [lo, hi) that see a key of tile t.
__device__ __forceinline__ void query_tiles(const WindowShape& s, int n, int t, int* lo, int* hi) {
  const int c0 = t * WT, c1 = (c0 + WT < n ? c0 + WT : n) - 1;      // keys [c0, c1]
  if (c0 >= n) {
    *lo = *hi = 0;
    return;
  }
  const bool sink = c0 < s.S;
  const int first = s.causal ? c0 : (sink || c0 - s.W + 1 < 0 ? 0 : c0 - s.W + 1);
  const int last = sink || s.W >= n - c1 ? n - 1 : c1 + s.W - 1;
  *lo = first / WT;
  *hi = last / WT + 1;
}

// A CTA's way along its share: steps [u0, u1) of the key tile t of (b, hk), `steps` in all, step u being
// query head hk g + u / nt and query tile lo + u % nt.
struct Walk {
  int y, b, t, hk, n, lo, nt, steps, u0, u1;
  long long left;                          // steps of the share from u0 on
  __device__ __forceinline__ void tile(const WindowShape& s, int tiles) {
    b = y / tiles;
    t = y % tiles;
    n = window_len(s, b);
    int hi;
    query_tiles(s, n, t, &lo, &hi);
    nt = hi - lo;
    steps = nt * s.g;
  }
  __device__ __forceinline__ void clip() { u1 = (long long)(steps - u0) < left ? steps : u0 + (int)left; }
  __device__ __forceinline__ bool next(const WindowShape& s, int tiles) {
    left -= u1 - u0;
    if (left <= 0) return false;
    u0 = 0;
    if (++hk == s.Hkv) {
      hk = 0;
      do {
        ++y;
        tile(s, tiles);
      } while (steps == 0);                // left > 0: there is one
    }
    clip();
    return true;
  }
};

struct Join {
  int on, y, hk, last;                     // pieces: of this CTA (the second), and of those up to `last` (the first)
};
template <int D>
constexpr size_t PIECE = (size_t)2 * WT * D * 4;   // dV, dK: [D / 4][128 rows] of 4 columns each

template <class T, int D>
__global__ void __launch_bounds__(THREADS, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                       View4 dk, View4 dv, WindowShape s, const float* __restrict__ lse, const float* delta,
                       const float* rho, SizesAt sizes, uint8_t* pieces) {
  using C = Cfg<D>;
  constexpr uint32_t F = kind16<T>();
  constexpr uint32_t IDESC_S = make_idesc(1, F, F, 128, 128);
  constexpr uint32_t IDESC_G = make_idesc(1, F, F, 128, D) | (1u << 16);     // B (Q or dO) read MN-major
  extern __shared__ __align__(1024) uint8_t base[];       // no room to round up: the swizzled tiles need it as it is
  if (smem_u32(base) & 1023u) {
    if (threadIdx.x == 0 && s.status) atomicExch(s.status, SLA2_DEV_TIMEOUT);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + C::OFF_BAR);
  uint64_t* k_full = bar;
  uint64_t* k_free = bar + 1;
  uint64_t* v_full = bar + 2;
  uint64_t* v_free = bar + 3;
  uint64_t* full = bar + 4;
  uint64_t* empty = full + C::NST;
  uint64_t* aux_full = empty + C::NST;
  uint64_t* aux_empty = aux_full + C::NAUX;
  uint64_t* s_full = aux_empty + C::NAUX;
  uint64_t* s_read = s_full + 1;
  uint64_t* dp_full = s_full + 2;
  uint64_t* dp_read = s_full + 3;
  uint64_t* p_free = s_full + 5;
  uint64_t* ds_full = s_full + 6;           // of a key tile's last step
  uint64_t* ds_free = s_full + 7;
  uint64_t* acc_full = s_full + 8;
  uint64_t* acc_free = s_full + 9;
  uint64_t* fix = s_full + 10;
  uint64_t* drain = s_full + 11;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC + 4);
  float* powers = reinterpret_cast<float*>(base + C::OFF_MISC + 8);          // `up` of the aux rows (fp16)
  long long* scan = reinterpret_cast<long long*>(base + C::OFF_AUX);         // before the aux rows are in use
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int tiles = (s.N + WT - 1) / WT, ny = s.B * tiles;
  Join* joins = reinterpret_cast<Join*>(pieces + 2 * gridDim.x * PIECE<D>);
  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_free, 1);
    mbar_init(v_full, 1);
    mbar_init(v_free, 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < C::NAUX; ++i) {
      mbar_init(aux_full + i, 1);
      mbar_init(aux_empty + i, 8);
    }
    mbar_init(s_full, 1);
    mbar_init(s_read, 8);
    mbar_init(dp_full, 1);
    mbar_init(dp_read, 8);
    mbar_init(p_free, 1);
    mbar_init(ds_full, 8);
    mbar_init(ds_free, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 8);
    mbar_init(fix, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    joins[blockIdx.x].on = 0;
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }

  // ---- the line's length and this CTA's share of it
  Walk walk{};
  long long total = 0, share = 0, begin = 0;
  for (int pass = 0; pass < 2; ++pass) {
    long long before = 0;
    for (int y0 = 0; y0 < ny; y0 += THREADS) {
      const int y = y0 + (int)threadIdx.x;
      long long mine = 0;
      if (y < ny) {
        Walk w;
        w.y = y;
        w.tile(s, tiles);
        mine = (long long)w.steps * s.Hkv;
      }
      long long sum = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(~0u, sum, off);
        if (lane >= off) sum += v;
      }
      if (lane == 31) scan[warp] = sum;
      __syncthreads();
      long long block = 0, ahead = before;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w == warp) ahead = before + block;
        block += scan[w];
      }
      ahead += sum - mine;
      if (pass == 1 && mine > 0 && ahead <= begin && begin < ahead + mine) {
        scan[16] = y;
        scan[17] = ahead;
      }
      before += block;
      __syncthreads();
    }
    if (pass == 0) {
      total = before;
      share = (total + gridDim.x - 1) / gridDim.x;
      if (share < MIN_SHARE) share = MIN_SHARE;
      begin = share * blockIdx.x;
      if (begin >= total) break;
    }
  }
  bool work = begin < total;
  if (work) {
    walk.y = (int)scan[16];
    const long long off = begin - scan[17];
    walk.tile(s, tiles);
    walk.hk = (int)(off / walk.steps);
    walk.u0 = (int)(off % walk.steps);
    walk.left = total - begin < share ? total - begin : share;
    walk.clip();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");                   // delta and what dQ adds to it are there
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const Waiter wait{abort_flag, s.status, s.budget_ns};

  if (warp >= 8) {
    if (warp == 8) {
      int r = 0, kv = 0, fixes = 0;
      if (lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&tdo);
      }
      auto load = [&](const CUtensorMap* m, int row, int h, int b, int zero) {   // rows from `zero` on are zeroed
        const int st = r % C::NST;
        if (r >= C::NST) wait(empty + st, r / C::NST - 1);
        if (wait.aborted()) return;
        uint8_t* dst = base + C::OFF_RING + st * C::TILE;
        uint64_t* on = zero < WT ? fix : full + st;
        if (lane == 0) {
          mbar_arrive_expect_tx(on, C::TILE);
          for (int sl = 0; sl < C::SLABS; ++sl) tma_load_4d(dst + sl * (WT * 128), m, on, sl * 64, row, h, b);
        }
        __syncwarp();
        ++r;
        if (zero < WT) {
          wait(fix, fixes++);
          zero_rows(dst, C::SLABS, zero, lane);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + st);
        }
      };
      // keys behind the end are rows of their own: nothing reads what becomes of them
      auto load_kv = [&](const CUtensorMap* m, uint8_t* dst, uint64_t* on, uint64_t* free) {
        if (kv > 0) wait(free, kv - 1);
        if (wait.aborted()) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(on, C::TILE);
          for (int sl = 0; sl < C::SLABS; ++sl)
            tma_load_4d(dst + sl * (WT * 128), m, on, sl * 64, walk.t * WT, walk.hk, walk.b);
        }
        __syncwarp();
      };
      for (bool more = work; more; more = walk.next(s, tiles), ++kv) {
        load_kv(&tk, base, k_full, k_free);
        for (int u = walk.u0; u < walk.u1; ++u) {
          const int i0 = (walk.lo + u % walk.nt) * WT, h = walk.hk * s.g + u / walk.nt;
          const int zero = walk.n < s.N && walk.n - i0 < WT ? walk.n - i0 : WT;      // behind N zeros come by themselves
          load(&tq, i0, h, walk.b, zero);
          if (u == walk.u0) load_kv(&tv, base + C::TILE, v_full, v_free);            // S needs K and Q alone
          load(&tdo, i0, h, walk.b, zero);
        }
      }
      if (wait.aborted() && lane == 0) {     // copies in flight land before shared memory is released
        for (int i = r > C::NST ? r - C::NST : 0; i < r; ++i) mbar_wait_drain(full + i % C::NST, (i / C::NST) & 1, W_DRAIN_NS);
        if (fixes > 0) mbar_wait_drain(fix, (fixes - 1) & 1, W_DRAIN_NS);
        // the loop leaves kv one ahead; a load that was not made any more completes nothing and only costs the limit
        if (kv > 0) mbar_wait_drain(k_full, (kv - 1) & 1, W_DRAIN_NS);
        if (kv > 0) mbar_wait_drain(v_full, (kv - 1) & 1, W_DRAIN_NS);
      }
      __syncwarp();
    } else if (warp == 9) {
      // The warps arrive on s_read of a step after their dS of the step before is written, and on dp_read
      // after their P is: two waits a step are all that the products need.
      const uint32_t kt = smem_u32(base), ring = smem_u32(base + C::OFF_RING);
      const uint32_t kd = kmajor(kt), vd = kmajor(kt + C::TILE), lead = elect_one();
      int g = 0, kv = 0;                     // steps and key tiles of this CTA so far
      Slot<C::NST> q, o;                     // of Q and dO of step g: every other place of the ring
      o.next();
      auto tile = [&](const Slot<C::NST>& t) { return ring + (uint32_t)t.at * C::TILE; };
      auto issue_s = [&](bool ends) {        // of the step at q; ends: the last that reads this K
        const uint32_t qd = kmajor(tile(q));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) mma_ss(lead, tmem, kmajor_step(kd, ks), kmajor_step(qd, ks), IDESC_S, ks > 0);
        commit(lead, s_full);
        if (ends) commit(lead, k_free);
      };
      bool more = work;
      int steps = uniform(walk.u1 - walk.u0);
      if (more) {
        wait(k_full, 0);
        wait(full + q.at, q.round);
        tc_fence_after();
        issue_s(steps == 1);
      }
      for (; more; ++kv) {
        const int n = steps;
        more = walk.next(s, tiles);
        steps = uniform(walk.u1 - walk.u0);  // of the next key tile, if there is one
        Slot<C::NST> q1 = q, o1 = o;         // of the step before
        for (int u = 0; u < n; ++u, ++g) {
          // S(g) has been read: dP(g) over it, and dK(g - 1) behind
          const uint32_t dod = kmajor(tile(o)), qm = mnmajor(tile(q1));
          if (u == 0) wait(v_full, kv);
          wait(full + o.at, o.round);
          wait(s_read, g);
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) mma_ss(lead, tmem, kmajor_step(vd, ks), kmajor_step(dod, ks), IDESC_S, ks > 0);
          commit(lead, dp_full);
          if (u == n - 1) commit(lead, v_free);
          if (u > 0) {
#pragma unroll
            for (int ks = 0; ks < WT / 16; ++ks)
              mma_ts(lead, tmem + 384, tmem + 192 + ks * 8, mnmajor_step(qm, ks), IDESC_G, u > 1 || ks > 0);
            commit(lead, ds_free);
            commit(lead, empty + q1.at);
          }
          q1 = q;
          o1 = o;
          q.next();
          q.next();
          o.next();
          o.next();
          // dP(g) has been read: S(g + 1) over it, and dV(g) behind. The first dV and dK of a key
          // tile overwrite the accumulators: those of the one before have been read
          const uint32_t dom = mnmajor(tile(o1));
          const bool ends = u == n - 1;
          if (!ends) wait(full + q.at, q.round);
          wait(dp_read, g);
          tc_fence_after();
          if (!ends) issue_s(u == n - 2);
          if (u == 0 && kv > 0) {
            wait(acc_free, kv - 1);
            tc_fence_after();
          }
#pragma unroll
          for (int ks = 0; ks < WT / 16; ++ks)
            mma_ts(lead, tmem + 256, tmem + 128 + ks * 8, mnmajor_step(dom, ks), IDESC_G, u > 0 || ks > 0);
          commit(lead, p_free);
          commit(lead, empty + o1.at);
        }
        // the last dK of the key tile
        const uint32_t qm = mnmajor(tile(q1));
        wait(ds_full, kv);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < WT / 16; ++ks)
          mma_ts(lead, tmem + 384, tmem + 192 + ks * 8, mnmajor_step(qm, ks), IDESC_G, n > 1 || ks > 0);
        commit(lead, ds_free);
        commit(lead, empty + q1.at);
        commit(lead, acc_full);
        if (more) {                          // the first S of the next
          wait(k_full, kv + 1);
          wait(full + q.at, q.round);
          tc_fence_after();
          issue_s(steps == 1);
        }
      }
      if (wait.aborted()) {                  // MMAs in flight end before the tensor memory is released
        commit(lead, drain);
        mbar_wait_drain(drain, 0, W_DRAIN_NS);
      }
      __syncwarp();
    } else if (warp == 10) {
      const long long rows = (long long)s.B * s.Hq * s.N;
      int g = 0;
      for (bool more = work; more; more = walk.next(s, tiles)) {
        const float up = SIZED<T> ? sizes.read(s, walk.b, walk.hk, lane).up() * P_DOWN : 1.f;
        for (int u = walk.u0; u < walk.u1; ++u, ++g) {
          const int sl = g % C::NAUX, i = walk.lo + u % walk.nt;
          if (g >= C::NAUX) wait(aux_empty + sl, g / C::NAUX - 1);
          float* dst = reinterpret_cast<float*>(base + C::OFF_AUX + sl * 1024);
          const long long row = ((long long)walk.b * s.Hq + walk.hk * s.g + u / walk.nt) * s.N + i * WT;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e * 32 + lane;
            const bool in = i * WT + r < walk.n;
            dst[r] = in ? fmaf(-__ldg(lse + row + r), W_LOG2E, P_UP<T>) : -INFINITY;     // P is zero behind the end
            dst[WT + r] = in ? -(__ldcg(delta + row + r) + (__ldcg(rho + row + r) + __ldcg(rho + rows + row + r))) * up : 0.f;
          }
          if (SIZED<T> && lane == 0) powers[sl] = up;
          __syncwarp();
          if (lane == 0) mbar_arrive(aux_full + sl);
        }
      }
    }
  } else {
    const int half = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t x_c = lanes + half * 64, p_c = lanes + 128 + half * 32, ds_c = lanes + 192 + half * 32;
    const float sc = s.scale * W_LOG2E;
    const uint64_t sc2 = f2_pack(sc, sc);
    int g = 0, kv = 0;
    for (bool more = work; more; more = walk.next(s, tiles), ++kv) {
      float up = 1.f;
      const int j = walk.t * WT + r, n = walk.n;
      // the queries [q0, q1) see key j
      const int q0 = s.causal ? j : (j < s.S ? 0 : j - s.W + 1);
      const int q1 = j < s.S || s.W >= n - j ? n : j + s.W;
      for (int u = walk.u0; u < walk.u1; ++u, ++g) {
        const float* aux = reinterpret_cast<const float*>(base + C::OFF_AUX + (g % C::NAUX) * 1024) + half * 64;
        wait(aux_full + g % C::NAUX, g / C::NAUX);
        wait(s_full, g);
        tc_fence_after();
        uint32_t v[64];
        tmem_ld32(x_c, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld32(x_c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_read);
        const int i0 = (walk.lo + u % walk.nt) * WT + half * 64;
        const int c0 = walk.t * WT, c1 = c0 + WT - 1;
        const bool whole = (i0 >= c1 || (!s.causal && (c1 < s.S || i0 > c1 - s.W))) && (c1 < s.S || i0 + 63 < c0 + s.W);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t w = below(q1 - i0 - c * 32) & ~below(q0 - i0 - c * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(w >> e & 1u)) v[c * 32 + e] = 0xff800000u;
          }
        }
        uint64_t p[32];
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 m = *reinterpret_cast<const float4*>(aux + e);
          float x0, x1, x2, x3;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, f2_pack(m.x, m.y)), x0, x1);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), sc2, f2_pack(m.z, m.w)), x2, x3);
          x0 = ex2_approx(x0);
          x1 = ex2_approx(x1);
          x2 = ex2_approx(x2);
          x3 = ex2_approx(x3);
          pk[e / 2] = pack16<T>(x0, x1);
          pk[e / 2 + 1] = pack16<T>(x2, x3);
          p[e / 2] = f2_pack(x0, x1);
          p[e / 2 + 1] = f2_pack(x2, x3);
        }
        if (g > 0) {                         // the dV that read P of the step before
          wait(p_free, g - 1);
          tc_fence_after();
        }
        tmem_st32(p_c, pk);
        tmem_wait_st();
        wait(dp_full, g);
        tc_fence_after();
        tmem_ld32(x_c, *reinterpret_cast<uint32_t(*)[32]>(v));
        tmem_ld32(x_c + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_read);
        if (SIZED<T>) up = powers[g % C::NAUX];
        const uint64_t up2 = f2_pack(up, up);
        auto sub = [&](uint32_t a, uint32_t b, float da, float db) {       // up (dP - delta)
          const uint64_t y = f2_pack(__uint_as_float(a), __uint_as_float(b)), m = f2_pack(da, db);
          return SIZED<T> ? f2_fma(y, up2, m) : f2_add(y, m);
        };
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
          const float4 m = *reinterpret_cast<const float4*>(aux + WT + e);
          float x0, x1, x2, x3;
          f2_unpack(f2_mul(p[e / 2], sub(v[e], v[e + 1], m.x, m.y)), x0, x1);
          f2_unpack(f2_mul(p[e / 2 + 1], sub(v[e + 2], v[e + 3], m.z, m.w)), x2, x3);
          pk[e / 2] = pack16<T>(x0, x1);
          pk[e / 2 + 1] = pack16<T>(x2, x3);
        }
        if (g > 0) {                         // the dK that read dS of the step before
          wait(ds_free, g - 1);
          tc_fence_after();
        }
        tmem_st32(ds_c, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (u == walk.u1 - 1) mbar_arrive(ds_full);
          mbar_arrive(aux_empty + g % C::NAUX);
        }
      }
      // dV (warpgroup 0) and dK (1) of the key tile
      wait(acc_full, kv);
      tc_fence_after();
      const uint32_t acc = lanes + 256 + half * 128;
      const float out_scale = (half ? s.scale * one_over(up) : 1.f) * (SIZED<T> ? P_DOWN : 1.f);
      if (walk.u0 == 0 && walk.u1 == walk.steps) {
        const View4& o = half ? dk : dv;
        T* dst = static_cast<T*>(o.p) + walk.b * o.sb + walk.hk * o.sh + j * o.sn;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(acc + c * 32, x);
          tmem_wait_ld();
          scale_all(x, out_scale);
          store_row<T>(dst + c * 32, o.sn, j, s.N, x, j < walk.n, lane);
        }
      } else {
        float4* dst = reinterpret_cast<float4*>(pieces + (2 * blockIdx.x + (walk.u0 == 0 ? 1 : 0)) * PIECE<D>) +
                      half * (D / 4) * WT + r;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(acc + c * 32, o);
          tmem_wait_ld();
          scale_all(o, out_scale);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            dst[(c * 8 + e / 4) * WT] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                                    __uint_as_float(o[e + 3]));
        }
        if (walk.u0 == 0 && threadIdx.x == 0)      // begins here: joined with what the next CTAs have of it
          joins[blockIdx.x] = {1, walk.y, walk.hk,
                               (int)((begin + share - walk.left + walk.steps - 1) / share)};
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
    }
    // key tiles behind a sequence's end: zeros
    if (s.lens) {
      for (int x = blockIdx.x; x < ny * s.Hkv; x += gridDim.x) {
        const int y = x / s.Hkv, b = y / tiles, t = y % tiles;
        if (t * WT < window_len(s, b)) continue;
        const int j = t * WT + r;
        const View4& o = half ? dk : dv;
        T* dst = static_cast<T*>(o.p) + b * o.sb + x % s.Hkv * o.sh + j * o.sn;
        if (j < s.N)
          for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums the pieces of the key tile that begins in CTA blockIdx.x of the kernel above and ends in a later
// one; blockIdx.y: 32 columns of dV or dK.
template <class T, int D>
__global__ void __launch_bounds__(256) window_join_kernel(WindowShape s, View4 dk, View4 dv, const uint8_t* pieces) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join j = reinterpret_cast<const Join*>(pieces + 2 * gridDim.x * PIECE<D>)[blockIdx.x];
  if (!j.on) return;
  const int tiles = (s.N + WT - 1) / WT, b = j.y / tiles, t = j.y % tiles;
  const int r = threadIdx.x & 127, row = t * WT + r;
  const int which = blockIdx.y / (D / 32), c4 = blockIdx.y % (D / 32) * 8 + (threadIdx.x >> 7) * 4;   // dV first
  if (row >= s.N) return;
  float4 x[4] = {};
  if (row < window_len(s, b)) {
    for (int k = blockIdx.x; k <= j.last; ++k) {
      const float4* p = reinterpret_cast<const float4*>(pieces + (2 * k + (k == (int)blockIdx.x ? 1 : 0)) * PIECE<D>) +
                        (which * (D / 4) + c4) * WT + r;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 y = p[e * WT];
        x[e].x += y.x;
        x[e].y += y.y;
        x[e].z += y.z;
        x[e].w += y.w;
      }
    }
  }
  const View4& o = which ? dk : dv;
  T* dst = static_cast<T*>(o.p) + b * o.sb + j.hk * o.sh + row * o.sn + c4 * 4;
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    *reinterpret_cast<uint4*>(dst + e * 4) = make_uint4(pack16<T>(x[e].x, x[e].y), pack16<T>(x[e].z, x[e].w),
                                                        pack16<T>(x[e + 1].x, x[e + 1].y), pack16<T>(x[e + 1].z, x[e + 1].w));
}

// CTAs of the dK, dV kernel: as many as there are shares of MIN_SHARE steps, at most (lengths are not
// known here: those of full sequences).
int dkdv_ctas(const WindowShape& s) {
  const long long tiles = (s.N + WT - 1) / WT, sinks = (s.S + WT - 1) / WT;
  const long long near = (s.causal ? 1 : 2) * ((long long)(s.W + WT - 1) / WT) + 2;
  const long long per_head = sinks * tiles + (tiles - sinks) * (near < tiles ? near : tiles);
  const long long shares = ((long long)s.B * s.Hq * per_head + MIN_SHARE - 1) / MIN_SHARE;
  return shares < SM_COUNT ? (int)shares : SM_COUNT;
}

// ------------------------------------------------------------------ dQ
// TMEM columns: [0, 128), [128, 256) S (two buffers; rows: queries, columns: keys), [256, 384) dP, then
// dS, [384, 384 + D) dQ. The steps of a CTA's query tiles follow one another without a break: S runs one
// step ahead of the warps, in the other buffer, and once dS(g) is written the products go out together:
// dQ += dS(g) K(g), dP(g + 1) over dS(g), S(g + 2) over S(g). A finished dQ is stored beside the next
// tile's first step.
// RAGGED: items with rows before their sequence's end come first, so that every CTA has as many of them as
// the next. It counts through the sequences for each item, so it is for RAGGED_MAX of them at most. A backward pass of
// padded sequences without it / with it, us: 2 of 4096 tokens, 24 heads of 64 186 / 183; 3 of them 295 / 285; 4, 16 heads
// 252 / 250; 5, 12 heads 216 / 221; 8, 8 heads 260 / 275; 16 of 2048, 8 heads 239 / 276. All of one length: 2% more.
constexpr int RAGGED_MAX = 4;
template <class T, int D, bool RAGGED>
__global__ void __launch_bounds__(THREADS, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                     const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo, View4 dq, WindowShape s,
                     const float* __restrict__ lse, const float* delta, float* rho,
                     SizesAt sizes, int items) {
  using C = Cfg<D>;
  constexpr uint32_t F = kind16<T>();
  constexpr uint32_t IDESC_S = make_idesc(1, F, F, 128, 128);
  constexpr uint32_t IDESC_G = make_idesc(1, F, F, 128, D) | (1u << 16);     // B (K) read MN-major
  extern __shared__ __align__(1024) uint8_t base[];       // no room to round up: the swizzled tiles need it as it is
  if (smem_u32(base) & 1023u) {
    if (threadIdx.x == 0 && s.status) atomicExch(s.status, SLA2_DEV_TIMEOUT);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + C::OFF_BAR);
  uint64_t* q_full = bar;
  uint64_t* q_free = bar + 1;
  uint64_t* o_full = bar + 2;                // dO
  uint64_t* o_free = bar + 3;
  uint64_t* full = bar + 4;
  uint64_t* empty = full + C::NST;
  uint64_t* s_full = empty + C::NST;         // [2]
  uint64_t* dp_full = s_full + 2;
  uint64_t* ds_full = s_full + 3;
  uint64_t* acc_full = s_full + 4;
  uint64_t* acc_free = s_full + 5;
  uint64_t* fix = s_full + 6;
  uint64_t* drain = s_full + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC + 4);
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_full + 1, 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(acc_full, 1);
    mbar_init(acc_free, 8);
    mbar_init(fix, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");                   // delta is there
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const Waiter wait{abort_flag, s.status, s.budget_ns};
  const int BH = s.B * s.Hq, tiles = (s.N + WT - 1) / WT;
  // A query tile: rows [a, a + 128) of (b, h), in a sequence of n tokens. The last rows come first: where
  // the attention is causal they see most.
  struct Tile {
    int a, b, h, n;
  };
  auto tile_of = [&](int x) {
    Tile t;
    if (!RAGGED) {
      t.a = (tiles - 1 - x / BH) * WT;
      t.b = x % BH / s.Hq;
      t.h = x % BH % s.Hq;
      t.n = window_len(s, t.b);
      return t;
    }
    t.h = x % s.Hq;
    t.a = x / s.Hq;                          // counts through the sequences' tiles
    for (t.b = 0;; ++t.b) {
      t.n = window_len(s, t.b);
      const int live = (t.n + WT - 1) / WT;
      if (t.a < live) {
        t.a = (live - 1 - t.a) * WT;
        return t;
      }
      t.a -= live;
      if (t.b == s.B - 1) break;
    }
    for (t.b = 0;; ++t.b) {                  // those behind the ends
      t.n = window_len(s, t.b);
      const int live = (t.n + WT - 1) / WT, dead = tiles - live;
      if (t.a < dead || t.b == s.B - 1) {
        t.a = (live + t.a) * WT;
        return t;
      }
      t.a -= dead;
    }
  };

  if (warp == 8) {
    int r = 0, fixes = 0, qn = 0;
    if (lane == 0) {
      tma_prefetch_desc(&tq);
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      tma_prefetch_desc(&tdo);
    }
    auto copy = [&](const CUtensorMap* m, uint8_t* dst, uint64_t* on, int row, int h, int b) {
      if (lane == 0) {
        mbar_arrive_expect_tx(on, C::TILE);
        for (int sl = 0; sl < C::SLABS; ++sl) tma_load_4d(dst + sl * (WT * 128), m, on, sl * 64, row, h, b);
      }
      __syncwarp();
    };
    auto load = [&](const CUtensorMap* m, int row, int h, int b, int zero) {   // rows from `zero` on are zeroed
      const int st = r % C::NST;
      if (r >= C::NST) wait(empty + st, r / C::NST - 1);
      if (wait.aborted()) return;
      uint8_t* dst = base + C::OFF_RING + st * C::TILE;
      copy(m, dst, zero < WT ? fix : full + st, row, h, b);
      ++r;
      if (zero < WT) {
        wait(fix, fixes++);
        zero_rows(dst, C::SLABS, zero, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + st);
      }
    };
    for (int x = blockIdx.x; x < items; x += gridDim.x) {
      const Tile t = tile_of(x);
      const TileList tl = key_tiles(s, t.n, t.a, t.a + WT);
      const int nt = tl.count();
      if (nt == 0) continue;
      if (qn > 0) wait(q_free, qn - 1);
      if (wait.aborted()) break;
      copy(&tq, base, q_full, t.a, t.h, t.b);
      for (int u = 0; u < nt; ++u) {
        const int k0 = tl.at(u) * WT;
        const int zero = t.n < s.N && t.n - k0 < WT ? t.n - k0 : WT;           // behind N zeros come by themselves
        load(&tk, k0, t.h / s.g, t.b, zero);
        if (u == 0) {                        // S needs Q and K alone
          if (qn > 0) wait(o_free, qn - 1);
          copy(&tdo, base + C::TILE, o_full, t.a, t.h, t.b);
          ++qn;
        }
        load(&tv, k0, t.h / s.g, t.b, zero);
      }
    }
    if (wait.aborted() && lane == 0) {       // copies in flight land before shared memory is released
      for (int i = r > C::NST ? r - C::NST : 0; i < r; ++i) mbar_wait_drain(full + i % C::NST, (i / C::NST) & 1, W_DRAIN_NS);
      if (fixes > 0) mbar_wait_drain(fix, (fixes - 1) & 1, W_DRAIN_NS);
      if (qn > 0) mbar_wait_drain(q_full, (qn - 1) & 1, W_DRAIN_NS);
      if (qn > 0) mbar_wait_drain(o_full, (qn - 1) & 1, W_DRAIN_NS);
    }
    __syncwarp();
  } else if (warp == 9) {
    // whole warp, one lane issues
    const uint32_t qt = smem_u32(base), ring = smem_u32(base + C::OFF_RING), lead = elect_one();
    const uint32_t qd = kmajor(qt), dod = kmajor(qt + C::TILE);
    // where one of the three products is: step u of nt of the CTA's item `n`, its tile in the ring
    struct Cursor {
      int x, u, nt, n;
      Slot<C::NST> at;
    };
    auto settle = [&](Cursor& c) {           // to an item that has steps, from c.x on
      for (; c.x < items; c.x += gridDim.x) {
        const Tile t = tile_of(c.x);
        c.nt = uniform(key_tiles(s, t.n, t.a, t.a + WT).count());
        if (c.nt > 0) return;
      }
    };
    auto step = [&](Cursor& c) {
      c.at.next();
      c.at.next();
      if (++c.u < c.nt) return;
      c.u = 0;
      ++c.n;
      c.x += gridDim.x;
      settle(c);
    };
    Cursor cs{(int)blockIdx.x, 0, 0, 0, {}};
    settle(cs);
    Cursor cp = cs, cq = cs;
    cp.at.next();                            // V behind K
    int j = 0;                               // S so far
    auto issue_s = [&]() {
      const uint32_t kd = kmajor(ring + (uint32_t)cs.at.at * C::TILE);
      if (cs.u == 0) wait(q_full, cs.n);
      wait(full + cs.at.at, cs.at.round);
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_ss(lead, tmem + (uint32_t)(j & 1) * 128, kmajor_step(qd, ks), kmajor_step(kd, ks), IDESC_S, ks > 0);
      commit(lead, s_full + (j & 1));
      if (cs.u == cs.nt - 1) commit(lead, q_free);
      ++j;
      step(cs);
    };
    auto issue_dp = [&]() {
      const uint32_t vd = kmajor(ring + (uint32_t)cp.at.at * C::TILE);
      if (cp.u == 0) wait(o_full, cp.n);
      wait(full + cp.at.at, cp.at.round);
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) mma_ss(lead, tmem + 256, kmajor_step(dod, ks), kmajor_step(vd, ks), IDESC_S, ks > 0);
      commit(lead, dp_full);
      commit(lead, empty + cp.at.at);
      if (cp.u == cp.nt - 1) commit(lead, o_free);
      step(cp);
    };
    if (cs.x < items) {
      issue_s();
      issue_dp();
      if (cs.x < items) issue_s();
    }
    for (int g = 0; cq.x < items; ++g) {
      const uint32_t km = mnmajor(ring + (uint32_t)cq.at.at * C::TILE);
      if (cq.u == 0 && cq.n > 0) wait(acc_free, cq.n - 1);
      wait(ds_full, g);
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < WT / 16; ++ks)
#pragma unroll
        for (int lo = 0; lo < 2; ++lo)
          mma_ts(lead, tmem + 384, tmem + 256 + (ks >> 2) * 64 + lo * 32 + (ks & 3) * 8, mnmajor_step(km, ks), IDESC_G,
                 cq.u > 0 || ks > 0 || lo > 0);
      commit(lead, empty + cq.at.at);
      if (cq.u == cq.nt - 1) commit(lead, acc_full);
      step(cq);
      if (cp.x < items) issue_dp();
      if (cs.x < items) issue_s();
    }
    if (wait.aborted()) {                    // MMAs in flight end before the tensor memory is released
      commit(lead, drain);
      mbar_wait_drain(drain, 0, W_DRAIN_NS);
    }
    __syncwarp();
  } else if (warp < 8) {
    const int half = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t dpc = lanes + 256 + half * 64;
    const float sc = s.scale * W_LOG2E;
    const uint64_t sc2 = f2_pack(sc, sc);
    int g = 0, qn = 0;
    auto row_of = [&](const Tile& t) {
      return static_cast<T*>(dq.p) + t.b * dq.sb + t.h * dq.sh + (long long)(t.a + r) * dq.sn + half * (D / 2);
    };
    float out_scale = s.scale;                             // of the tile to be finished
    auto finish = [&](const Tile& t, int i) {              // dQ of the CTA's i-th tile: half of the columns a warpgroup
      wait(acc_full, i);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32];
        tmem_ld32(lanes + 384 + half * (D / 2) + c * 32, x);
        tmem_wait_ld();
        scale_all(x, out_scale);
        store_row<T>(row_of(t) + c * 32, dq.sn, t.a + r, s.N, x, t.a + r < t.n, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_free);
    };
    auto stats = [&](const Tile& t) {                      // -lse and -delta of this thread's row
      const long long at = ((long long)t.b * s.Hq + t.h) * s.N + t.a + r;
      return t.a + r < t.n ? make_float2(-__ldg(lse + at) * W_LOG2E, -__ldcg(delta + at)) : make_float2(-INFINITY, 0.f);
    };
    Tile last{};
    auto sizes_of = [&](const Tile& t) { return SIZED<T> ? sizes.read(s, t.b, t.h / s.g, lane) : Sizes{}; };
    float2 st = (int)blockIdx.x < items ? stats(tile_of(blockIdx.x)) : make_float2(0.f, 0.f);
    Sizes sz = (int)blockIdx.x < items ? sizes_of(tile_of(blockIdx.x)) : Sizes{};
    for (int x = blockIdx.x; x < items; x += gridDim.x) {
      const Tile t = tile_of(x);
      const TileList tl = key_tiles(s, t.n, t.a, t.a + WT);
      const int nt = tl.count(), row = t.a + r;
      const float up = SIZED<T> ? sz.up() : 1.f;
      const uint64_t nl2 = f2_pack(st.x, st.x), nd2 = f2_pack(st.y * up, st.y * up), up2 = f2_pack(up, up);
      uint64_t sum2 = f2_pack(0.f, 0.f);     // of this row's dS
      if (x + (int)gridDim.x < items) {      // on its way while this tile is worked on
        const Tile next = tile_of(x + gridDim.x);
        st = stats(next);
        sz = sizes_of(next);
      }
      if (nt == 0) {
        if (row < s.N)
          for (int c = 0; c < D / 2; c += 8) *reinterpret_cast<uint4*>(row_of(t) + c) = make_uint4(0, 0, 0, 0);
        continue;
      }
      for (int u = 0; u < nt; ++u, ++g) {
        const int kt = tl.at(u);
        wait(s_full + (g & 1), g >> 1);
        tc_fence_after();
        uint64_t p[32];
        const bool whole = all_visible(s, t.n, t.a, kt);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          tmem_ld32(lanes + (g & 1) * 128 + half * 64 + c * 32, v);
          tmem_wait_ld();
          if (!whole) {
            const uint32_t w = key_mask(s, t.n, row, kt * WT + half * 64 + c * 32);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(w >> e & 1u)) v[e] = 0xff800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc2, nl2), x0, x1);
            p[c * 16 + e / 2] = f2_pack(ex2_approx(x0), ex2_approx(x1));
          }
        }
        if (u == 0 && qn > 0) finish(last, qn - 1);
        wait(dp_full, g);
        tc_fence_after();
        // dS as the sum of two 16-bit numbers, so that dQ's own rounding is the only one of its size: [0, 32) of
        // the half's columns for the first, [32, 64) for the rest
        uint32_t low[16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32], pk[16], rest[16];
          tmem_ld32(dpc + c * 32, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint64_t dp = f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            const uint64_t ds = f2_mul(p[c * 16 + e / 2], SIZED<T> ? f2_fma(dp, up2, nd2) : f2_add(dp, nd2));
            sum2 = f2_add(sum2, ds);
            float x0, x1;
            f2_unpack(ds, x0, x1);
            pk[e / 2] = pack16<T>(x0, x1);
            const float2 y = unpack16<T>(pk[e / 2]);
            rest[e / 2] = pack16<T>(x0 - y.x, x1 - y.y);
          }
          tmem_st16(dpc + c * 16, pk);
          if (c == 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) low[e] = rest[e];
          } else {
            tmem_st16(dpc + 32, low);
            tmem_st16(dpc + 48, rest);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      // What delta is off by: the row's dS sum to zero. delta comes from O as it was rounded, and where few keys are
      // seen that is most of dS's error; dK takes it into account. One array for each half of the columns.
      {
        float x0, x1;
        f2_unpack(sum2, x0, x1);
        if (row < t.n) rho[(half * (long long)s.B * s.Hq + (long long)t.b * s.Hq + t.h) * s.N + row] = (x0 + x1) * one_over(up);
      }
      last = t;
      if (SIZED<T>) out_scale = s.scale * one_over(up);
      ++qn;
    }
    if (qn > 0) finish(last, qn - 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class T, int D>
cudaError_t launch_t(const WindowShape& s, const WindowBwdArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  CUtensorMap tq, tk, tv, tdo;
  if (!make_tmap_4d(&tq, a.q, s.B, s.Hq, s.N, D, 64, WT) || !make_tmap_4d(&tk, a.k, s.B, s.Hkv, s.N, D, 64, WT) ||
      !make_tmap_4d(&tv, a.v, s.B, s.Hkv, s.N, D, 64, WT) || !make_tmap_4d(&tdo, a.dout, s.B, s.Hq, s.N, D, 64, WT))
    return cudaErrorInvalidValue;
  auto dkdv = window_dkdv_kernel<T, D>;
  const bool ragged = s.lens && s.B <= RAGGED_MAX;
  auto dq = ragged ? window_dq_kernel<T, D, true> : window_dq_kernel<T, D, false>;
  cudaError_t e;
  static unsigned long long done[3] = {0, 0, 0};
  if ((e = allow_smem(dkdv, C::SMEM, done)) != cudaSuccess || (e = allow_smem(dq, C::SMEM, done + 1 + ragged)) != cudaSuccess) return e;
  const long long rows = (long long)s.B * s.Hq * s.N;
  const SizesAt sizes = sizes_at(s, a.sizes);
  constexpr int STEP = 256 / (D / 8);        // rows of a block
  const unsigned few = narrow(s) ? 0 : (unsigned)(((long long)s.B * s.Hq * FEW * (s.causal ? 1 : 2) + STEP - 1) / STEP);
  const unsigned first = few + (SIZED<T> ? size_blocks(s, sizes) : 0);
  const auto delta = narrow(s) ? window_delta_kernel<T, D, true> : window_delta_kernel<T, D, false>;
  delta<<<first + (unsigned)((rows + STEP - 1) / STEP), 256, 0, st>>>(s, a.q, a.k, a.v, a.out, a.dout, a.lse, a.delta, sizes, few, first);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int ctas = dkdv_ctas(s), nq = (s.N + WT - 1) / WT * s.B * s.Hq;
  // each sets up while the one before runs
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(nq < SM_COUNT ? nq : SM_COUNT);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  float* rho = a.delta + rows;
  if ((e = cudaLaunchKernelEx(&cfg, dq, tq, tk, tv, tdo, a.dq, s, (const float*)a.lse, (const float*)a.delta, rho, sizes, nq)) != cudaSuccess)
    return e;
  cfg.gridDim = dim3(ctas);
  if ((e = cudaLaunchKernelEx(&cfg, dkdv, tq, tk, tv, tdo, a.dk, a.dv, s, (const float*)a.lse, (const float*)a.delta, (const float*)rho,
                              sizes, (uint8_t*)a.pieces)) != cudaSuccess)
    return e;
  cfg.gridDim = dim3(ctas, 2 * (D / 32));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, window_join_kernel<T, D>, s, a.dk, a.dv, (const uint8_t*)a.pieces);
}

}  // namespace

size_t window_backward_sizes(const WindowShape& s) { return (size_t)s.B * s.Hkv * 2 * sizes_at(s, nullptr).chunks * 4; }
size_t window_backward_pieces(const WindowShape& s) {
  return dkdv_ctas(s) * (2 * (s.d == 128 ? PIECE<128> : PIECE<64>) + sizeof(Join));
}

cudaError_t launch_window_backward(const WindowShape& s, int fp16, const WindowBwdArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
