// Attention of a step's new tokens over the paged 8-bit cache.
//
// The bound is the cache's bytes: 2 d per visible key and key head, read once. The work is cut to that:
// every (sequence, key head, block of query rows) is an item of so many units of 32 keys, the items of
// all sequences form one line, and each CTA (one per SM) takes an equal, contiguous share of it,
// whatever the lengths are. A CTA finds its share by a scan over the lengths, so the host needs to
// know none of them. An item that one CTA holds whole is finished there; the pieces of others are
// joined by a second kernel, launched so that it is resident by the time the first one ends.
//
// Each of a CTA's 8 to 16 warps has a ring of units of its own (K and V tiles by TMA, scales by cp.async)
// and its own running maximum and sum; they meet at the end of an item. Rows are few (query heads
// that share a key head, times new tokens), so keys take the 16-row side of the warp-wide products and
// rows the 8-column side: S = K Q^T, O^T = V^T P^T. tcgen05 wants 128 rows and would leave 120 empty;
// the tensor pipe is busy 19% of the time here, as it is.
//
// 64 sequences of up to 8192 tokens, 8 key heads of 128, 4 query heads each, one new token each: 171 us,
// 4.75 TB/s of the codes (the loads alone, with nothing done to them: 135 us). What is left is
// instructions, 850 a unit and warp, at two of four issue slots: with 8 warps 220 us, with 12 warps
// 183, with whole-number products for S 176 (both sides of each at one time). A warp of its own for the
// loads was slower (191), units of 64 keys were for short lengths (window of 4096: 51 against 46).
//
// S is formed in whole numbers, from the codes as they are: a query row becomes 16-bit numbers of its own
// scale, the high and the low bytes of which multiply the codes by two 8-bit products (which the tensor
// path runs at twice the rate of fp16 ones, and which need no conversion of K). For P V weights are
// rounded to fp16 and codes become fp16 exactly (the byte next to 0x64 is 1024 + code + 128; one
// subtraction). Page scales stay out of the products: S is multiplied by k's afterwards, and a page's
// P V joins O in fp32 times v's.
// The order of keys and channels inside a product is free: it is chosen so that a thread reads its
// share in 16-byte pieces and the swizzled rows meet no bank twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "device.cuh"
#include "kernels.cuh"
#include "window.cuh"
#include "window_tile.cuh"

namespace sla2 {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int UNIT = CACHE_UNIT;
// Units that a CTA takes at least. One sequence of 1001 keys, 12 heads of 64: 12.5 us with 4 or 8, 17 with
// 2 (more pieces to join) or 12 (a lone CTA's warps one after the other's latency).
constexpr int MIN_SHARE = 4;
constexpr float LOW = -3.0e38f;          // a maximum that nothing has been seen for
constexpr int NONE = -0x7fffffff - 1;    // no page needed
constexpr float LAZY = 8.f;              // log2 of how far a row's maximum may grow before O is rescaled
// log2 of the weight of a row's largest key: fp16 has the room above (2^(UP + LAZY) < 65504), and needs it
// below. With it at 0, of 200000 keys 17 nats below one the weights were off by 44%.
constexpr float UP = 7.f;

template <int D, int NT>
struct Cfg {
  static constexpr int RB = 8 * NT;                      // query rows of an item
  // Warps and their registers: 168 a thread for 12, 128 for 16, 255 for 8. Of 16 rows, 10 or 11 warps spill:
  // 63 us for 24 windows of 4160 keys, 8 warps 46.
  static constexpr int WARPS = NT == 2 ? 8 : D == 128 ? 12 : 16;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int OWN = NT == 2 ? WARPS : WARPS / 2; // warps that have room for O in shared memory
  static constexpr int NST = 2;
  static constexpr int TILE = UNIT * D;                  // codes of a unit, K or V
  static constexpr int STAGE = 2 * TILE;
  static constexpr int OFF_O = WARPS * NST * STAGE;
  static constexpr int OFF_ML = OFF_O + OWN * RB * D * 4;
  static constexpr int OFF_SC = OFF_ML + OWN * RB * 8;   // scales of a stage: k, v of its two halves
  static constexpr int OFF_BAR = OFF_SC + WARPS * NST * 16;
  static constexpr int OFF_MISC = OFF_BAR + WARPS * NST * 8;
  static constexpr int SMEM = OFF_MISC + 192 + WARPS * 16 + 1024;
  static_assert(SMEM <= 232448, "dynamic shared memory per CTA (227 KB)");
  // workspace: what a CTA may leave (the end of an item that began before it, and the beginning of
  // one that ends after it), then a line per CTA on the item that begins in it and is to be joined
  static constexpr size_t PIECE = (size_t)RB * (D + 2) * 4;
};

struct Join {
  int on, b, hk, rb, last;               // pieces: of this CTA (the second), and of those up to `last` (the first)
};

// The units of an item: [0, head) of the sinks before the window, then from lo on.
struct Units {
  int head, lo, count;
  int first, last;                       // keys of the window, over all of the item's rows
  __device__ __forceinline__ int at(int u) const { return u < head ? u : lo + (u - head); }
};
template <int RB>
__device__ __forceinline__ Units item_units(const CacheShape& s, const CacheAttnArgs& a, const Span& sp, int rb) {
  const int rows = sp.n * s.g;
  const int q0 = rb * RB / s.g, q1 = ((rb + 1) * RB < rows ? (rb + 1) * RB - 1 : rows - 1) / s.g;
  const int p0 = sp.len + q0, p1 = sp.len + q1;
  const int first = a.W <= p0 ? p0 - a.W + 1 : 0;
  // Units [0, a.end) are what the table reaches. A length behind it is wrong, and its items have the table's units
  // and one behind them, whose page there is not: the row is written and the fault seen, at no more
  // than the table's cost.
  Units u;
  u.first = first;
  u.last = p1;
  u.lo = first / UNIT;
  const int sinks = a.S < first ? (int)(((unsigned)a.S + UNIT - 1) / UNIT) : u.lo;
  u.head = min(min(sinks, u.lo), a.end);
  u.count = u.head + max(min(p1 / UNIT, a.end) - u.lo, 0) + 1;
  return u;
}
template <int RB>
__device__ __forceinline__ int sequence_blocks(const CacheShape& s, const Span& sp) {
  return (int)(((long long)sp.n * s.g + RB - 1) / RB);
}
template <int RB>
__device__ __forceinline__ long long sequence_units(const CacheShape& s, const CacheAttnArgs& a, const Span& sp) {
  long long t = 0;
  const int blocks = sequence_blocks<RB>(s, sp);
  for (int rb = 0; rb < blocks; ++rb) t += item_units<RB>(s, a, sp, rb).count;
  return t;
}

// A place on the line of units: unit u of the item (b, hk, rb); `left` units of the CTA's share from
// here on. All lanes hold the same.
template <int RB>
struct Place {
  int b, hk, rb, u;
  long long left;
  Span sp;
  Units un;
  __device__ __forceinline__ void item(const CacheShape& s, const CacheAttnArgs& a) { un = item_units<RB>(s, a, sp, rb); }
  // to the first unit of the next item (left > 0: there is one)
  __device__ __forceinline__ void next_item(const CacheShape& s, const CacheAttnArgs& a) {
    u = 0;
    if ((long long)(++rb) * RB >= (long long)sp.n * s.g) {
      rb = 0;
      if (++hk == s.Hkv) {
        hk = 0;
        do {
          ++b;
          step_span(s, b, &sp);
        } while (sp.n == 0 && b + 1 < s.B);
      }
    }
    item(s, a);
  }
  __device__ __forceinline__ int piece() const { return (int)((long long)(un.count - u) < left ? un.count - u : left); }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// bytes 0 and 1 (sel 0x4140) or 2 and 3 (0x4342) of offset codes (code + 128) as two fp16 codes
__device__ __forceinline__ uint32_t codes_f16(uint32_t u, uint32_t sel) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(prmt(u, 0x64646464u, sel)), "r"(0x64806480u));
  return r;
}
// c (+)= a b
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool fresh) {
  if (fresh)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, bool fresh) {
  if (fresh)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void copy4_async(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// arrives on `bar` when this thread's cp.async copies so far have landed
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 16-byte chunk c of row t of a tile (rows of 128 or 64 bytes, swizzled over their width)
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int t, int c) {
  return D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
}
// the key of 16 that a product's row r (< 8) stands for; row r + 8: 8 more
template <int D>
__device__ __forceinline__ int key_of(int r) {
  return D == 128 ? ((r & 1) << 2) | (r >> 1) : r;
}

// Channels 4c .. 4c + 3 of a row of an item: the weighted sum over the weights' sum (a row that has seen
// nothing is zero).
template <class T>
__device__ __forceinline__ void store_out(const CacheShape& s, const CacheAttnArgs& a, const Span& sp, int hk, int rho, int c,
                                          float4 x, float sum) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* dst = static_cast<T*>(a.out.p) + (long long)(sp.t0 + rho / s.g) * a.out.st + (hk * s.g + rho % s.g) * a.out.sh;
  T y[4] = {Half16<T>::r(x.x * inv), Half16<T>::r(x.y * inv), Half16<T>::r(x.z * inv), Half16<T>::r(x.w * inv)};
  *reinterpret_cast<uint2*>(dst + c * 4) = *reinterpret_cast<const uint2*>(y);
}

// SOLO: an item is a warp's alone, from its first unit to its last, for tables of a few units a sequence.
template <class T, int D, int NT, bool SOLO>
__global__ void __launch_bounds__(Cfg<D, NT>::THREADS, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, CacheShape s,
                      CacheAttnArgs a, unsigned long long budget_ns) {
  using C = Cfg<D, NT>;
  constexpr int RB = C::RB, KC = D / 64, MT = D / 16, VW = D / 32;   // K chunks a lane, channel tiles, V words a lane and key
  constexpr int WARPS = C::WARPS, THREADS = C::THREADS, OWN = C::OWN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, q = lane & 3;
  uint8_t* ring = base + warp * C::NST * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + C::OFF_BAR) + warp * C::NST;
  float* scales = reinterpret_cast<float*>(base + C::OFF_SC) + warp * C::NST * 4;
  float* Osm = reinterpret_cast<float*>(base + C::OFF_O);
  float2* ML = reinterpret_cast<float2*>(base + C::OFF_ML);
  long long* scan = reinterpret_cast<long long*>(base + C::OFF_MISC);      // [WARPS], then what was found
  int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC + 184);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int i = 0; i < C::NST; ++i) mbar_init(full + i, 5);      // the copies' issuer and four scales
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }

  // ---- the line's length and this CTA's share of it
  Place<RB> at;
  long long total = 0, share = 0, begin = 0;
  Join* joins = reinterpret_cast<Join*>(static_cast<uint8_t*>(a.workspace) + 2 * gridDim.x * C::PIECE);
  if constexpr (SOLO) {
    // a line of items; warps take equal numbers of them, the first warps of all CTAs first
    long long* found = reinterpret_cast<long long*>(base + C::OFF_MISC + 192);      // [WARPS][2]
    for (int pass = 0; pass < 2; ++pass) {
      long long before = 0;
      bool cut = false;
      for (int b0 = 0; b0 < s.B; b0 += THREADS) {
        const int b = b0 + (int)threadIdx.x;
        const Span sp = block_span(s, b, &cut, blockIdx.x == 0);
        const long long mine = (long long)s.Hkv * sequence_blocks<RB>(s, sp);
        long long sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long x = __shfl_up_sync(~0u, sum, off);
          if (lane >= off) sum += x;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        long long block = 0, first = before;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          if (w == warp) first = before + block;
          block += scan[w];
        }
        first += sum - mine;
        if (pass == 1 && mine > 0)
          for (int w = 0; w < WARPS; ++w) {
            const long long x = share * ((long long)w * gridDim.x + blockIdx.x);
            if (first <= x && x < first + mine) {
              found[2 * w] = b;
              found[2 * w + 1] = x - first;
            }
          }
        before += block;
        __syncthreads();
      }
      if (pass == 0) {
        total = before;
        share = (total + (long long)gridDim.x * WARPS - 1) / ((long long)gridDim.x * WARPS);
      }
    }
    begin = share * ((long long)warp * gridDim.x + blockIdx.x);
    if (begin >= total) return;          // the CTA has no barrier from here on
    at.b = (int)found[2 * warp];
    step_span(s, at.b, &at.sp);
    const int blocks = sequence_blocks<RB>(s, at.sp);
    at.hk = (int)(found[2 * warp + 1] / blocks);
    at.rb = (int)(found[2 * warp + 1] % blocks);
    at.item(s, a);
    at.u = 0;
    at.left = total - begin < share ? total - begin : share;      // items here, units otherwise
  } else {
    for (int pass = 0; pass < 2; ++pass) {
      long long before = 0, ahead = 0, mine = 0;
      bool cut = false;
      for (int b0 = 0; b0 < s.B; b0 += THREADS) {
        const int b = b0 + (int)threadIdx.x;
        const Span sp = block_span(s, b, &cut, blockIdx.x == 0);
        mine = s.Hkv * sequence_units<RB>(s, a, sp);
        long long sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long x = __shfl_up_sync(~0u, sum, off);
          if (lane >= off) sum += x;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        long long block = 0;
        ahead = before;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          if (w == warp) ahead = before + block;
          block += scan[w];
        }
        ahead += sum - mine;                                        // units before sequence b
        if (pass == 1 && mine > 0 && ahead <= begin && begin < ahead + mine) {
          scan[WARPS] = b;
          scan[WARPS + 1] = ahead;
        }
        before += block;
        __syncthreads();
      }
      if (pass == 0) {
        total = before;
        share = (total + gridDim.x - 1) / gridDim.x;
        if (share < MIN_SHARE) share = MIN_SHARE;
        begin = share * blockIdx.x;
        if (begin >= total) break;                                  // the whole CTA
        if (s.B <= THREADS) {                                       // one round: what it found still stands
          if (mine > 0 && ahead <= begin && begin < ahead + mine) {
            scan[WARPS] = (int)threadIdx.x;
            scan[WARPS + 1] = ahead;
          }
          __syncthreads();
          break;
        }
      }
    }
    if (begin >= total) {
      if (threadIdx.x == 0) joins[blockIdx.x].on = 0;
      return;
    }
    at.b = (int)scan[WARPS];
    long long found = begin - scan[WARPS + 1];
    step_span(s, at.b, &at.sp);
    {
      const long long per_head = sequence_units<RB>(s, a, at.sp);
      at.hk = (int)(found / per_head);
      found -= at.hk * per_head;
      at.rb = 0;
      at.item(s, a);
      while (found >= at.un.count) {
        found -= at.un.count;
        ++at.rb;
        at.item(s, a);
      }
      at.u = (int)found;
    }
    at.left = (total - begin < share ? total - begin : share);
  }
  constexpr int WSTEP = SOLO ? 1 : WARPS;
  const int w0 = SOLO ? 0 : warp;        // this warp's units of a piece: w0, w0 + WSTEP, ...
  bool bad = false;
  auto piece = [&](const Place<RB>& p) { return SOLO ? p.un.count : p.piece(); };
  bool join_mine = false;

  // ---- loads: this warp's units of its share, in order, as far ahead as the ring holds
  Place<RB> ahead = at;
  int ahead_n = piece(ahead), ahead_w = w0;   // units of the piece, and which of them is this warp's next
  int issued = 0, used = 0;
  int t0_next = 0, pid[2];               // the next unit's first key, and the pages of its two halves
  bool have = true;                      // is there a next unit?
  const Waiter wait{abort_flag, s.status, budget_ns};
  const bool two = s.page == 16;         // a unit takes two pages
  auto page_at = [&](int p) {
    return p < s.max_pages ? max(__ldg(s.table + (size_t)ahead.b * s.max_pages + p), -1) : -1;
  };
  auto find = [&]() {                    // to this warp's next unit
    while (ahead_w >= ahead_n) {
      ahead_w = w0;
      ahead.left -= SOLO ? 1 : ahead_n;
      if (ahead.left <= 0) {
        have = false;
        return;
      }
      ahead.next_item(s, a);
      ahead_n = piece(ahead);
    }
    t0_next = ahead.un.at(ahead.u + ahead_w) * UNIT;
    const int p0 = t0_next >> s.lpage;
    if (two) {
      // keys [t, t + 16) hold one that some row sees; where none does their page is not asked for
      auto needed = [&](int t) { return t <= ahead.un.last && (t < a.S || t + 16 > ahead.un.first); };
      pid[0] = needed(t0_next) ? page_at(p0) : NONE;
      pid[1] = needed(t0_next + 16) ? page_at(p0 + 1) : NONE;
    } else {
      pid[0] = page_at(p0);
    }
  };
  auto issue = [&]() {
    if (!have || wait.aborted()) return;
    const int st = issued % C::NST;
    uint8_t* dst = ring + st * C::STAGE;
    if (!two) pid[1] = pid[0];
    const bool v0 = (unsigned)pid[0] < (unsigned)s.num_pages, v1 = (unsigned)pid[1] < (unsigned)s.num_pages;
    bad |= (!v0 && pid[0] != NONE) || (!v1 && pid[1] != NONE);
    if (lane == 0) {
      const int y = (pid[0] * s.Hkv + ahead.hk) * s.page + (t0_next & (s.page - 1));
      mbar_arrive_expect_tx(full + st, two ? C::TILE * (v0 + v1) : C::STAGE * v0);
      if (v0) {
        tma_load_2d(dst, &tk, full + st, 0, y);
        tma_load_2d(dst + C::TILE, &tv, full + st, 0, y);
      }
      if (two && v1) {
        const int z = (pid[1] * s.Hkv + ahead.hk) * s.page;
        tma_load_2d(dst + C::TILE / 2, &tk, full + st, 0, z);
        tma_load_2d(dst + C::TILE + C::TILE / 2, &tv, full + st, 0, z);
      }
    }
    if (lane < 4) {                      // k of the halves, v of the halves; a page left out: a scale below zero
      float* d = scales + st * 4 + lane;
      if (lane & 1 ? v1 : v0) {
        copy4_async(smem_u32(d), (lane < 2 ? s.ks : s.vs) + (size_t)(lane & 1 ? pid[1] : pid[0]) * s.Hkv + ahead.hk);
        copies_arrive(full + st);
      } else {
        *d = -1.f;
        mbar_arrive(full + st);
      }
    }
    __syncwarp();
    ++issued;
    ahead_w += WSTEP;
    find();
  };
  find();
  __syncwarp();
  for (int i = 0; i < C::NST; ++i) issue();

  const int f = D == 128 ? r & 1 : (r >> 1) & 1;         // which of a pair of keys is read first
  const uint32_t mix_lo = f ? 0x1504u : 0x5140u, mix_hi = f ? 0x3726u : 0x7362u;
  uint32_t k_at[KC], v_at[2];                             // where this lane reads in a tile (8 rows on: + 8 D)
#pragma unroll
  for (int i = 0; i < KC; ++i) k_at[i] = chunk_at<D>(key_of<D>(r), q + 4 * i);
#pragma unroll
  for (int g = 0; g < 2; ++g)
    v_at[g] = D == 128 ? chunk_at<D>(key_of<D>(2 * q + (g ^ f)), r)
                       : chunk_at<D>(key_of<D>(2 * q + (g ^ f)), r >> 1) + (r & 1) * 8;

  while (true) {
    // ---- a piece of an item
    const int n = piece(at);
    const bool starts = at.u == 0, ends = at.u + n == at.un.count;
    const int rows = at.sp.n * s.g - at.rb * RB;         // rows of this block (those behind it see nothing)
    // A row of Q as whole numbers v in [-32639, 32639] of steps of its largest magnitude / 32639 (off by half a
    // step, 2^-16 of that magnitude, at most), v = 256 hi + lo with both in 8 bits.
    uint32_t qh[NT][KC * 4], ql[NT][KC * 4];
    float qs[NT][2];                                      // of the rows 2q, 2q + 1 of each 8
    int pos[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = t * 8 + r, rho = at.rb * RB + row;
      uint4 w[KC * 2];
      const T* src = static_cast<const T*>(a.q.p) + (long long)(at.sp.t0 + rho / s.g) * a.q.st + (at.hk * s.g + rho % s.g) * a.q.sh;
#pragma unroll
      for (int i = 0; i < KC; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[i * 2 + e] = row < rows ? __ldg(reinterpret_cast<const uint4*>(src + 16 * (q + 4 * i) + 8 * e)) : make_uint4(0, 0, 0, 0);
      const uint32_t* ws = reinterpret_cast<const uint32_t*>(w);
      float x[KC * 16];
      uint32_t mb = 0;
#pragma unroll
      for (int i = 0; i < KC * 8; ++i) {
        if (std::is_same<T, __half>::value) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(ws + i));
          x[2 * i] = y.x;
          x[2 * i + 1] = y.y;
        } else {
          x[2 * i] = bf16_lo(ws[i]);
          x[2 * i + 1] = bf16_hi(ws[i]);
        }
        mb = max(mb, max(__float_as_uint(x[2 * i]) & 0x7fffffffu, __float_as_uint(x[2 * i + 1]) & 0x7fffffffu));
      }
      mb = max(mb, __shfl_xor_sync(~0u, mb, 1));
      mb = max(mb, __shfl_xor_sync(~0u, mb, 2));
      // scaled by a power of two first: its largest magnitude into [1, 2) (where 2^-e is a normal number)
      const int e = min(max((int)(mb >> 23), 1), 252) - 127;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float top = __uint_as_float(mb) * down, inv = mb > 0 && mb < 0x7f800000u ? 32639.f / top : 0.f;
#pragma unroll
      for (int i = 0; i < KC * 4; ++i) {
        qh[t][i] = ql[t][i] = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int v = min(max(__float2int_rn(x[4 * i + c] * down * inv), -32639), 32639), hi = (v + 128) >> 8;
          qh[t][i] |= (uint32_t)(hi & 0xff) << (8 * c);
          ql[t][i] |= (uint32_t)((v - hi * 256) & 0xff) << (8 * c);
        }
      }
      // what is not finite makes the row NaN
      const float sc = mb < 0x7f800000u ? top * (up / 32639.f) * a.scale * LOG2E : NAN;
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        qs[t][e2] = __shfl_sync(~0u, sc, 4 * (2 * q + e2));
        const int row2 = t * 8 + 2 * q + e2;
        pos[t][e2] = row2 < rows ? at.sp.len + (at.rb * RB + row2) / s.g : -1;
      }
    }
    const int p_lo = at.sp.len + at.rb * RB / s.g, p_hi = at.sp.len + min(at.rb * RB + RB - 1, at.sp.n * s.g - 1) / s.g;
    float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = LOW;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
    }
    for (int w = w0; w < n; w += WSTEP) {
      const int t0 = at.un.at(at.u + w) * UNIT, st = used % C::NST;
      wait(full + st, used / C::NST);
      ++used;
      const uint8_t* kt = ring + st * C::STAGE;
      const uint8_t* vt = kt + C::TILE;
      const float4 sc4 = *reinterpret_cast<const float4*>(scales + st * 4);
      const float ks[2] = {sc4.x, sc4.y}, vs[2] = {sc4.z, sc4.w};
      float x[NT][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        int hi[NT][4], lo[NT][4];
#pragma unroll
        for (int i = 0; i < KC; ++i) {
          const uint4 k0 = *reinterpret_cast<const uint4*>(kt + k_at[i] + h * 16 * D);
          const uint4 k1 = *reinterpret_cast<const uint4*>(kt + k_at[i] + h * 16 * D + 8 * D);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16832(hi[t], k0.x, k1.x, k0.y, k1.y, qh[t][i * 4], qh[t][i * 4 + 1], i == 0);
            mma16832(lo[t], k0.x, k1.x, k0.y, k1.y, ql[t][i * 4], ql[t][i * 4 + 1], i == 0);
            mma16832(hi[t], k0.z, k1.z, k0.w, k1.w, qh[t][i * 4 + 2], qh[t][i * 4 + 3], false);
            mma16832(lo[t], k0.z, k1.z, k0.w, k1.w, ql[t][i * 4 + 2], ql[t][i * 4 + 3], false);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][h][e] = (float)(hi[t][e] * 256 + lo[t][e]);     // below 2^30
      }
      // ---- softmax: x[t][h][2 e + c] is key h * 16 + e * 8 + key_of(r), row t * 8 + 2 q + c. Rows behind
      // the block's last are not looked at by anybody
      if (!(t0 + UNIT - 1 <= p_lo && (t0 + UNIT <= a.S || t0 > p_hi - a.W) && !(ks[0] < 0.f) && !(ks[1] < 0.f))) {
        // some row does not see some key of the unit
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = t0 + h * 16 + e * 8 + key_of<D>(r);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (!(j <= pos[t][c] && (j > pos[t][c] - a.W || j < a.S)) || ks[h] < 0.f) x[t][h][2 * e + c] = -INFINITY;
          }
      }
      float kf[2] = {ks[0], ks[1]};
      if (!(ks[0] + ks[1] < INFINITY)) {                  // a page that is not finite reaches the rows that see it, and no others
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!(ks[h] < INFINITY)) {
            kf[h] = 1.f;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (x[t][h][e] != -INFINITY) x[t][h][e] = NAN;
          }
      }
      // Raw products to logits: by a factor that is not 0, which would make -inf a NaN (one below the smallest
      // normal number stands for logits of 0: a page of zeros, a page left out)
      float f[NT][2][2];
      bool grow = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          f[t][c][0] = kf[0] * qs[t][c];
          f[t][c][0] = f[t][c][0] < 1.2e-38f ? 1.2e-38f : f[t][c][0];
          f[t][c][1] = f[t][c][0];
          if (two) {
            f[t][c][1] = kf[1] * qs[t][c];
            f[t][c][1] = f[t][c][1] < 1.2e-38f ? 1.2e-38f : f[t][c][1];
          }
          const float mx = fmaxf(fmaxf(x[t][0][c], x[t][0][2 + c]) * f[t][c][0], fmaxf(x[t][1][c], x[t][1][2 + c]) * f[t][c][1]);
          grow |= mx > m[t][c] + (LAZY + UP);
        }
      if (__any_sync(~0u, grow)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(x[t][0][c], x[t][0][2 + c]) * f[t][c][0], fmaxf(x[t][1][c], x[t][1][2 + c]) * f[t][c][1]);
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16)) - UP;
            if (mx > m[t][c]) {
              const float corr = ex2_approx(m[t][c] - mx);       // 0 for the first keys seen
              m[t][c] = mx;
              l[t][c] *= corr;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[t][i][c] *= corr;
                o[t][i][2 + c] *= corr;
              }
            }
          }
      }
      float y[NT][2][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[t][h][e] = ex2_approx(fmaf(x[t][h][e], f[t][e & 1][h], -m[t][e & 1]));
            l[t][e & 1] += y[t][h][e];
          }
      if (!(vs[0] + vs[1] < INFINITY)) {                  // as with k's pages
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (!(vs[h] < INFINITY)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) y[t][h][e] = x[t][h][e] == -INFINITY ? 0.f : NAN;
          }
      }
      uint32_t p[NT][2][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[t][h][e] = transpose8(pack16<__half>(y[t][h][2 * e], y[t][h][2 * e + 1]));
      // ---- O += v's scale x (P V), channel tile by channel tile
      uint32_t v[2][2][2][VW];                            // half, keys e * 8 + (two of a pair), in the order read
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint8_t* src = vt + v_at[g] + (h * 16 + e * 8) * D;
            uint32_t y[4];
            if (D == 128)
              *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(src);
            else
              *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(src);
#pragma unroll
            for (int j = 0; j < VW; ++j) v[h][e][g][j] = y[j] ^ 0x80808080u;
          }
      const float v0 = vs[0] < INFINITY ? fmaxf(vs[0], 0.f) : 1.f, v1 = vs[1] < INFINITY ? fmaxf(vs[1], 0.f) : 1.f;
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        // channels 4j .. 4j + 3 of this lane's: bytes of a pair's two keys side by side
        uint32_t af[2][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t mix = z ? mix_hi : mix_lo;
            const uint32_t y0 = prmt(v[h][0][0][j], v[h][0][1][j], mix), y1 = prmt(v[h][1][0][j], v[h][1][1][j], mix);
            af[h][z][0] = codes_f16(y0, 0x4140u);
            af[h][z][1] = codes_f16(y0, 0x4342u);
            af[h][z][2] = codes_f16(y1, 0x4140u);
            af[h][z][3] = codes_f16(y1, 0x4342u);
          }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            float pv[4];
            mma16816(pv, af[0][z], p[t][0][0], p[t][0][1], true);
            if (two) {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][2 * j + z][e] = fmaf(v0, pv[e], o[t][2 * j + z][e]);
              mma16816(pv, af[1][z], p[t][1][0], p[t][1][1], true);
            } else {
              mma16816(pv, af[1][z], p[t][1][0], p[t][1][1], false);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][2 * j + z][e] = fmaf(v1, pv[e], o[t][2 * j + z][e]);
          }
      }
      __syncwarp();                                       // the stage has been read
      issue();
    }
    // ---- the warps' parts meet: o[t][i][2 z + c] is channel D / 8 * r + 2 i + z, row t * 8 + 2 q + c
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[t][c] += __shfl_xor_sync(~0u, l[t][c], 4);
        l[t][c] += __shfl_xor_sync(~0u, l[t][c], 8);
        l[t][c] += __shfl_xor_sync(~0u, l[t][c], 16);
      }
    if constexpr (SOLO) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = t * 8 + 2 * q + c, rho = at.rb * RB + row;
          if (row >= rows) continue;
          const float inv = l[t][c] == 0.f ? 0.f : 1.f / l[t][c];
          T* dst = static_cast<T*>(a.out.p) + (long long)(at.sp.t0 + rho / s.g) * a.out.st + (at.hk * s.g + rho % s.g) * a.out.sh +
                   r * (D / 8);
#pragma unroll
          for (int i = 0; i < MT; i += 4) {
            T y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = Half16<T>::r(o[t][i + e / 2][2 * (e & 1) + c] * inv);
            *reinterpret_cast<uint4*>(dst + 2 * i) = *reinterpret_cast<const uint4*>(y);
          }
        }
      if (--at.left <= 0) break;
      at.next_item(s, a);
      continue;
    }
    if (OWN < WARPS && n > OWN) {                         // the second half of the warps hand theirs to the first
      float4* swap = reinterpret_cast<float4*>(Osm) + (warp % OWN) * (RB * D / 4) + lane;
      if (warp >= OWN && warp < n) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
            swap[(t * MT + i) * 32] = make_float4(o[t][i][0], o[t][i][1], o[t][i][2], o[t][i][3]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (r == 0) ML[(warp - OWN) * RB + t * 8 + 2 * q + c] = make_float2(m[t][c], l[t][c]);
        }
      }
      __syncthreads();
      if (warp < OWN && warp + OWN < n) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f0[2], f1[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float2 ml = ML[warp * RB + t * 8 + 2 * q + c];
            const float M = fmaxf(m[t][c], ml.x);
            f0[c] = ex2_approx(m[t][c] - M);
            f1[c] = ex2_approx(ml.x - M);
            m[t][c] = M;
            l[t][c] = l[t][c] * f0[c] + ml.y * f1[c];
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const float4 y = swap[(t * MT + i) * 32];
            o[t][i][0] = o[t][i][0] * f0[0] + y.x * f1[0];
            o[t][i][1] = o[t][i][1] * f0[1] + y.y * f1[1];
            o[t][i][2] = o[t][i][2] * f0[0] + y.z * f1[0];
            o[t][i][3] = o[t][i][3] * f0[1] + y.w * f1[1];
          }
        }
      }
      __syncthreads();
    }
    const int parts = n < OWN ? n : OWN;
    if (warp < parts) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = warp * RB + t * 8 + 2 * q + c;
          if (r == 0) ML[row] = make_float2(m[t][c], l[t][c]);
          float* dst = Osm + row * D + r * (D / 8);
#pragma unroll
          for (int i = 0; i < MT; i += 2)
            *reinterpret_cast<float4*>(dst + 2 * i) =
                make_float4(o[t][i][c], o[t][i][2 + c], o[t][i + 1][c], o[t][i + 1][2 + c]);
        }
    }
    __syncthreads();
    const bool alone = starts && ends;
    uint8_t* piece = static_cast<uint8_t*>(a.workspace) + (2 * blockIdx.x + (starts ? 1 : 0)) * C::PIECE;
    for (int i = threadIdx.x; i < RB * (D / 4); i += THREADS) {
      const int row = i / (D / 4), c = i % (D / 4);
      if (row >= rows) continue;
      float M = LOW, L = 0.f;
      for (int w = 0; w < parts; ++w) M = fmaxf(M, ML[w * RB + row].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < parts; ++w) {
        const float2 ml = ML[w * RB + row];
        const float fac = ex2_approx(ml.x - M);
        const float4 y = *reinterpret_cast<const float4*>(Osm + (w * RB + row) * D + c * 4);
        L += ml.y * fac;
        acc.x = fmaf(y.x, fac, acc.x);
        acc.y = fmaf(y.y, fac, acc.y);
        acc.z = fmaf(y.z, fac, acc.z);
        acc.w = fmaf(y.w, fac, acc.w);
      }
      if (alone) {
        store_out<T>(s, a, at.sp, at.hk, at.rb * RB + row, c, acc, L);
      } else {
        *reinterpret_cast<float4*>(piece + (row * D + c * 4) * 4) = acc;
        if (c == 0) *reinterpret_cast<float2*>(piece + RB * D * 4 + row * 8) = make_float2(M, L);
      }
    }
    if (starts && !ends) {
      join_mine = true;
      if (threadIdx.x == 0)
        joins[blockIdx.x] = {1, at.b, at.hk, at.rb, (int)((begin + share - at.left + (at.un.count - at.u) - 1) / share)};
    }
    at.left -= n;
    if (at.left <= 0) break;
    at.next_item(s, a);
    __syncthreads();                                      // shared parts have been read
  }
  if (!SOLO && !join_mine && threadIdx.x == 0) joins[blockIdx.x].on = 0;
  if (bad && lane == 0) flag_bad_index(s);
  if (wait.aborted())                                     // copies in flight land before shared memory is released
    for (int i = issued > C::NST ? issued - C::NST : 0; i < issued; ++i)
      mbar_wait_drain(full + i % C::NST, (i / C::NST) & 1, W_DRAIN_NS);
}

// Joins the pieces of the item that begins in CTA blockIdx.x of the kernel above and ends in a later one;
// blockIdx.y: 32 channels. First every piece's factor, for all rows at once, then sums without a chain,
// each fourth piece a group of threads.
template <class T, int D, int NT>
__global__ void __launch_bounds__(256 * NT) cache_join_kernel(CacheShape s, CacheAttnArgs a) {
  using C = Cfg<D, NT>;
  constexpr int RB = C::RB, G = 4;
  __shared__ float fac[SM_COUNT * RB], sum[RB];
  __shared__ float4 part[G][64 * NT];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join j = reinterpret_cast<const Join*>(static_cast<const uint8_t*>(a.workspace) + 2 * gridDim.x * C::PIECE)[blockIdx.x];
  if (!j.on) return;
  Span sp;
  step_span(s, j.b, &sp);
  const int rows = sp.n * s.g - j.rb * RB, parts = j.last - (int)blockIdx.x + 1;
  const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
  auto piece = [&](int k) { return ws + (2 * ((int)blockIdx.x + k) + (k == 0 ? 1 : 0)) * C::PIECE; };
  auto ml = [&](int k, int row) { return *reinterpret_cast<const float2*>(piece(k) + RB * D * 4 + row * 8); };
  {
    const int row = threadIdx.x / 32, z = threadIdx.x % 32;        // a warp a row
    float M = LOW, L = 0.f;
    for (int k = z; k < parts; k += 32) M = fmaxf(M, ml(k, row).x);
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, off));
    for (int k = z; k < parts; k += 32) {
      const float2 y = ml(k, row);
      const float f = ex2_approx(y.x - M);
      fac[k * RB + row] = f;
      L += y.y * f;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(~0u, L, off);
    if (z == 0) sum[row] = L;
  }
  __syncthreads();
  const int t = threadIdx.x % (64 * NT), grp = threadIdx.x / (64 * NT), row = t / 8, c = blockIdx.y * 8 + t % 8;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = grp; k < parts; k += G) {
    const float4 y = *reinterpret_cast<const float4*>(piece(k) + (row * D + c * 4) * 4);
    const float x = fac[k * RB + row];
    acc.x = fmaf(y.x, x, acc.x);
    acc.y = fmaf(y.y, x, acc.y);
    acc.z = fmaf(y.z, x, acc.z);
    acc.w = fmaf(y.w, x, acc.w);
  }
  part[grp][t] = acc;
  __syncthreads();
  if (grp == 0 && row < rows) {
#pragma unroll
    for (int i = 1; i < G; ++i) {
      const float4 y = part[i][t];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
    store_out<T>(s, a, sp, j.hk, j.rb * RB + row, c, acc, sum[row]);
  }
}

// Tables of up to so many units a sequence: an item a warp, and nothing to join. 94 sequences of 58 tokens, 12 key
// heads of 128, 8 query heads each: 49 us with an item a CTA, 12 so; 8 key heads, 256 sequences of 250: 114, so
// 45; 32 of 250: 26, so 19; 32 of 500: 29, but 33.
constexpr int SOLO_UNITS = 8;

template <class T, int D, int NT, bool SOLO>
cudaError_t launch_s(const CacheShape& s, const CacheAttnArgs& a, cudaStream_t st) {
  using C = Cfg<D, NT>;
  auto kern = cache_attn_kernel<T, D, NT, SOLO>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(kern, C::SMEM, &done);
  if (e != cudaSuccess) return e;
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)s.num_pages * s.Hkv * s.page;
  const uint32_t box = s.page < UNIT ? s.page : UNIT;
  if (!make_tmap_2d(&tk, s.kc, 1, D, rows, D, box, D) || !make_tmap_2d(&tv, s.vc, 1, D, rows, D, box, D))
    return cudaErrorInvalidValue;
  kern<<<s.sms, C::THREADS, C::SMEM, st>>>(tk, tv, s, a, wait_budget_ns());
  if ((e = cudaGetLastError()) != cudaSuccess || SOLO) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.sms, D / 32);
  cfg.blockDim = dim3(256 * NT);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<T, D, NT>, s, a);
}

template <class T, int D, int NT>
cudaError_t launch_t(const CacheShape& s, const CacheAttnArgs& a, cudaStream_t st) {
  return (long long)s.max_pages * s.page <= SOLO_UNITS * UNIT ? launch_s<T, D, NT, true>(s, a, st) : launch_s<T, D, NT, false>(s, a, st);
}

// Items of 16 rows where a sequence has more than 8 on average (any choice is right for any lengths).
// 32 sequences of 4096 tokens, 4 key heads of 128, by the rows of a sequence, in blocks of 8 / of 16: 8 rows
// 44 / 54 us, 12 rows 71 / 57, 16 rows 71 / 56, 24 rows 96 / 95, 32 rows 121 / 95.
bool wide(const CacheShape& s) { return (long long)s.T * s.g > 8LL * s.B; }

template <class T, int D>
cudaError_t launch_d(const CacheShape& s, const CacheAttnArgs& a, cudaStream_t st) {
  return wide(s) ? launch_t<T, D, 2>(s, a, st) : launch_t<T, D, 1>(s, a, st);
}

template <int D>
size_t workspace_d(const CacheShape& s) {
  return s.sms * (2 * (wide(s) ? Cfg<D, 2>::PIECE : Cfg<D, 1>::PIECE) + sizeof(Join));
}

}  // namespace

size_t cache_attention_workspace(const CacheShape& s) {
  return ((s.d == 128 ? workspace_d<128>(s) : workspace_d<64>(s)) + 255) & ~size_t(255);
}

cudaError_t launch_cache_attention(const CacheShape& s, int fp16, const CacheAttnArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_d<__half, 128>(s, a, st) : launch_d<__half, 64>(s, a, st);
  return s.d == 128 ? launch_d<__nv_bfloat16, 128>(s, a, st) : launch_d<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
