// What the tensor-core kernels of sliding-window attention share: the key tiles that a range of
// query rows sees, the mask words of a row, 4-D TMA copies and 16-bit packing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device.cuh"
#include "window.cuh"

namespace sla2 {

constexpr int WT = 128;                    // rows of a query tile, keys of a key tile
constexpr float W_LOG2E = 1.4426950408889634f, W_LN2 = 0.6931471805599453f;

// The tiles, in ascending order, that hold what a range of rows sees: [0, head) of the sinks before
// the window, then [lo, hi].
struct TileList {
  int head, lo, hi, sinks;                 // sinks: tiles that hold a sink
  __device__ __forceinline__ int count() const { return hi < lo ? head : head + hi - lo + 1; }
  __device__ __forceinline__ int at(int u) const { return u < head ? u : lo + (u - head); }
  __device__ __forceinline__ bool has(int t) const { return t <= hi && (t >= lo || t < head); }
};

// Key tiles for the query rows [a, e) of a sequence of n tokens (empty for a >= e).
__device__ __forceinline__ TileList key_tiles(const WindowShape& s, int n, int a, int e) {
  TileList t;
  if (e > n) e = n;
  t.sinks = ((s.S < n ? s.S : n) + WT - 1) / WT;
  if (a >= e) {
    t.head = 0;
    t.lo = 1;
    t.hi = -1;
    return t;
  }
  const int first = a - s.W + 1 > 0 ? a - s.W + 1 : 0;
  const int last = s.causal ? e - 1 : (s.W < n - e + 1 ? e + s.W - 2 : n - 1);
  t.lo = first / WT;
  t.hi = last / WT;
  if (!s.causal && t.sinks - 1 > t.hi) t.hi = t.sinks - 1;
  t.head = t.sinks < t.lo ? t.sinks : t.lo;
  return t;
}

// Does every row of [a, a + 128) see every key of tile t?
__device__ __forceinline__ bool all_visible(const WindowShape& s, int n, int a, int t) {
  const int c0 = t * WT, c1 = c0 + WT - 1;
  if (c1 >= n) return false;
  if (s.causal && c1 > a) return false;
  if (c1 < s.S) return true;
  return c0 >= a + WT - s.W && (s.causal || c1 < a + s.W);
}

__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : (x >= 32 ? ~0u : (1u << x) - 1u); }

// Which of the keys [c, c + 32) the row i sees (i < n).
__device__ __forceinline__ uint32_t key_mask(const WindowShape& s, int n, int i, int c) {
  const int lo = i - s.W + 1, hi = s.causal ? i + 1 : (s.W < n - i ? i + s.W : n);
  const int sk = s.causal && s.S > i + 1 ? i + 1 : (s.S < n ? s.S : n);
  return (below(hi - c) & ~below(lo - c)) | below(sk - c);
}

template <class T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) {
  return cvt_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <class T>
constexpr uint32_t kind16() {              // kind::f16 operand format
  return std::is_same<T, __half>::value ? 0u : 1u;
}

// [B][H][N][d] tiles: coordinates (element, token, head, batch); x a multiple of 64, all >= 0.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int n, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(n), "r"(h), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int n, int h, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(n), "r"(h), "r"(b)
               : "memory");
}

// Waits (whole warp) until the phase of `bar` with the given parity has completed. If the budget runs out
// the status word is set and every later wait of the block returns at once: the roles then run their loops
// to the end on whatever the buffers hold. All addresses are in bounds whatever the data, so nothing
// hangs or faults, and no wait needs a vote and a branch (the issuing warp lost 400 cycles a batch
// of products to those).
struct Waiter {
  int* abort_flag;
  unsigned* status;
  unsigned long long budget_ns;
  __device__ __forceinline__ void operator()(uint64_t* bar, int phase) const {
    if (!mbar_try_wait(bar, phase & 1)) slow(bar, phase & 1);
    __syncwarp();
  }
  __device__ __forceinline__ void slow(uint64_t* bar, uint32_t parity) const {
    volatile int* f = abort_flag;
    if (!*f) mbar_wait(bar, parity, f, status, budget_ns);
  }
  __device__ __forceinline__ bool aborted() const { return *static_cast<volatile int*>(abort_flag) != 0; }
};

// x, the same in all lanes, known as such to the compiler
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(~0u, x, 0); }

// Operand tiles of 128 rows stored as 128-byte-swizzled slabs of 64 columns. The low word of their
// matrix descriptors for the tile's address (the same in all lanes), to which a K step adds a
// constant: kmajor reads the tile's rows as M or N and its columns as K, mnmajor its rows as K (16 a
// step) and its columns as N.
__device__ __forceinline__ uint32_t kmajor(uint32_t tile) { return (uint32_t)uniform((int)(tile >> 4 | 1u << 16)); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t tile) {
  return (uint32_t)uniform((int)(tile >> 4 | (uint32_t)(WT * 128 >> 4) << 16));
}
__device__ __forceinline__ uint64_t tile_desc(uint32_t lo) {
  // stride 1024 bytes between groups of 8 rows, version 1, 128-byte swizzle
  return (uint64_t)(1024u >> 4 | 1u << 14 | LAYOUT_SW128 << 29) << 32 | lo;
}
__device__ __forceinline__ uint64_t kmajor_step(uint32_t lo, int ks) {
  return tile_desc(lo + (uint32_t)(((ks >> 2) * (WT * 128) + (ks & 3) * 32) >> 4));
}
__device__ __forceinline__ uint64_t mnmajor_step(uint32_t lo, int ks) { return tile_desc(lo + (uint32_t)(ks * 2048 >> 4)); }

// Zeroes the rows [r0, 128) of a tile of `slabs` 64-column slabs (whole warp).
__device__ __forceinline__ void zero_rows(uint8_t* tile, int slabs, int r0, int lane) {
  for (int sl = 0; sl < slabs; ++sl)
    for (int o = r0 * 128 + lane * 16; o < WT * 128; o += 512)
      *reinterpret_cast<uint4*>(tile + sl * (WT * 128) + o) = make_uint4(0, 0, 0, 0);
}

// One lane of a converged warp, always the same one. The issuing warp runs its loop as a whole, without
// branches, and predicates its MMAs and commits on this: with the loop inside a branch on the lane,
// descriptors are no longer known to be the same for the warp and each MMA first moves them to uniform
// registers (115 cycles an MMA of 128 x 128 x 16 where the tensor pipe takes 64); with branches around
// the MMAs, each batch pays for leaving and joining the warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p;
}
// kind::f16 MMAs (A from shared or tensor memory) and commits of the lane that has `lead` set
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// A place in a ring of N slots and the parity of its round.
template <int N>
struct Slot {
  int at = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      round ^= 1;
    }
  }
};

// Moves registers between warpgroups (every warp of a warpgroup; the shares must add up to what the
// block was launched with).
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}

constexpr uint64_t W_DRAIN_NS = 20000000ull;   // for copies and MMAs in flight after an abort

}  // namespace sla2
