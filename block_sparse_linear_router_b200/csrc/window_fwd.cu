// Sliding-window attention with sinks, forward: O = softmax(scale Q K^T over the visible keys) V.
//
// Persistent CTAs (one per SM) walk items of 256 query rows of one head, as two streams of 128 rows
// that share the K and V tiles (128 keys each) that either of them sees. 384 threads:
//   warps 0-3, 4-7  softmax of stream 0, 1: thread t owns query row t (= TMEM lane t). One pass with
//             the running maximum m and sum l; P = 2^(s - m) goes back into TMEM over its own S as
//             16-bit values, the A operand of PV. m only moves when a row's maximum has grown by more
//             than 2^8: until then P stays below 2^8 (fp16: 2^15), which both types hold, and O needs no
//             rescaling.
//   warp 8    TMA producer: Q of each stream (one item ahead), K and V tiles into a ring. The rows of
//             a V tile behind the sequence's end may hold anything (0 x NaN is NaN): such a tile is
//             completed by the producer, which zeroes them before it hands the tile on.
//   warp 9    tcgen05 issuer. Per tile and stream: O += P V of the previous tile, in two halves as P
//             comes, then S = Q K^T of this one (an issuer's products run in its order, so S may
//             overwrite that P). While one stream's S is in its softmax, the other stream's products run.
//             Of d = 64 a tile's keys come as two parts of 64, each with its S and its place: one part's
//             S and P V run while the other is in the softmax; warp 10 then issues for stream 1.
//   warp 11 (and 10)  only give their registers to the softmax warps.
// What bounds it: of 256 rows and a key tile of d = 128 the four products take 2048 cycles of the tensor
// pipe and the 32768 exponentials as many of the special function units, so a step cannot take less.
// 32768 tokens, 12 heads of 128, window 2048, 64 sinks, causal, bf16: 390 us (a few calls; 458 in a row of them that
// lasts, at the 1.63 GHz that the power limit leaves), 1055 TFLOP/s of the visible pairs, 3500 cycles a step, tensor pipe and special function units busy 55% each. Without the
// exponentials a step takes 3 to 8% less, without the maxima as well 6 to 8%, without loads 9%: it is the
// hand-overs between the roles, two chains of them a step, that are not hidden. Of d = 64, parts and two
// issuers: 3 x 24 heads of 4096 tokens, window 512, 102 us, without them 113. Of d = 128, tiles in two
// parts: 464 us, in one 398 (a product of 64 keys reads more from shared memory than that delivers); two
// issuers: 176 us for 4 x 16 heads of 4999 tokens, window 512 both ways, one 157. Parts of the
// exponentials as a polynomial on the fma pipe were slower (spills).
// TMEM columns: [0, 128) S and P of stream 0, [128, 256) of stream 1, [256, 384) and [384, 512) their O.
#include "device.cuh"
#include "kernels.cuh"
#include "window.cuh"
#include "window_tile.cuh"

namespace sla2 {

namespace {

constexpr int HALF = WT / 2;               // keys of a half tile
constexpr float LAZY = 8.f;                // log2 of how far a row maximum may grow before O is rescaled
// P is 2^UP at a row's maximum, in O and in the sum alike. fp16 has the room above (2^(UP + LAZY) < 65504) and needs it
// below: with 0, the weights of 32767 keys 17 nats below one were off by 44%.
template <class T>
constexpr float UP = std::is_same<T, __half>::value ? 7.f : 0.f;

template <int D>
struct Cfg {
  static constexpr int SLABS = D / 64;
  static constexpr int TILE = WT * D * 2;
  static constexpr int NST = D == 128 ? 4 : 8;
  static constexpr int PARTS = D == 64 ? 2 : 1;            // of a tile's keys, each with an S of its own
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_OUT = OFF_RING + NST * TILE;     // 8 warps x 32 rows x 128 bytes
  static constexpr int OFF_BAR = OFF_OUT + 8 * 4096;
  static constexpr int ISSUERS = D == 64 ? 2 : 1;
  // q_full[2], q_free[2], full[NST], empty[NST], s_full[4], p_full[4], pv_done[4], o_full[2], o_free[2], fix, drain
  static constexpr int NBAR = 4 + 2 * NST + 12 + 4 + 3;
  static constexpr int OFF_MISC = OFF_BAR + ((8 * NBAR + 15) / 16) * 16;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static_assert(SMEM <= 232448, "dynamic shared memory per CTA (227 KB)");
};

struct Item {
  int b, h, a, n;                          // rows [a, a + 256) of a sequence of n tokens
};

__device__ __forceinline__ Item item_at(const WindowShape& s, int x) {
  Item it;
  const int BH = s.B * s.Hq, pairs = (s.N + 2 * WT - 1) / (2 * WT);
  const int bh = x % BH;
  it.b = bh / s.Hq;
  it.h = bh % s.Hq;
  it.a = (pairs - 1 - x / BH) * (2 * WT);  // the last rows first: where the attention is causal they see most
  it.n = window_len(s, it.b);
  return it;
}
// key tiles of stream i of an item, and of both together
__device__ __forceinline__ TileList stream_tiles(const WindowShape& s, const Item& it, int i) {
  return key_tiles(s, it.n, it.a + i * WT, it.a + (i + 1) * WT);
}
__device__ __forceinline__ TileList item_tiles(const WindowShape& s, const Item& it) {
  return key_tiles(s, it.n, it.a, it.a + 2 * WT);
}

template <class T, int D>
__global__ void __launch_bounds__(384, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, WindowShape s,
                      float* lse, int items) {
  using C = Cfg<D>;
  constexpr uint32_t IDESC_QK = make_idesc(1, kind16<T>(), kind16<T>(), 128, WT / C::PARTS);
  constexpr uint32_t IDESC_PV = make_idesc(1, kind16<T>(), kind16<T>(), 128, D) | (1u << 16);   // B = V, MN-major
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + C::OFF_BAR);
  uint64_t* q_full = bar;
  uint64_t* q_free = bar + 2;
  uint64_t* full = bar + 4;
  uint64_t* empty = full + C::NST;
  uint64_t* s_full = empty + C::NST;
  uint64_t* p_full = s_full + 4;             // [stream][half], as s_full and pv_done
  uint64_t* pv_done = s_full + 8;
  uint64_t* o_full = s_full + 12;
  uint64_t* o_free = s_full + 14;
  uint64_t* fix = s_full + 16;
  uint64_t* drain = s_full + 17;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::OFF_MISC);
  int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC + 4);
  const int warp = __shfl_sync(~0u, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_free + i, 1);
      mbar_init(o_full + i, 1);
      mbar_init(o_free + i, 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, C::ISSUERS);
    }
    mbar_init(fix, 1);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
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
  const uint32_t tmem = __shfl_sync(~0u, *tmem_slot, 0);
  const Waiter wait{abort_flag, s.status, s.budget_ns};

  // registers: launched with 384 x 168; 256 x 216 + 128 x 72 is the same sum
  if (warp >= 8) {
    regs_dec<72>();
    if (warp == 8) {
      // ------------------------------------------------------------ TMA producer (whole warp)
      int r = 0, fixes = 0, qn[2] = {0, 0};
      if (lane == 0) {
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&to);
      }
      // tile t of K or V into the next ring place; rows from `zero` on are zeroed (128: none)
      auto load = [&](const CUtensorMap* m, const Item& it, int t, int zero) {
        const int st = r % C::NST;
        if (r >= C::NST) wait(empty + st, r / C::NST - 1);
        if (wait.aborted()) return;
        uint8_t* dst = base + C::OFF_RING + st * C::TILE;
        uint64_t* b = zero < WT ? fix : full + st;
        if (lane == 0) {
          mbar_arrive_expect_tx(b, C::TILE);
          for (int sl = 0; sl < C::SLABS; ++sl)
            tma_load_4d(dst + sl * (WT * 128), m, b, sl * 64, t * WT, it.h / s.g, it.b);
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
      auto load_q = [&](const Item& it, int i) {
        if (it.a + i * WT >= it.n) return;
        if (qn[i] > 0) wait(q_free + i, qn[i] - 1);
        if (wait.aborted()) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full + i, C::TILE);
          for (int sl = 0; sl < C::SLABS; ++sl)
            tma_load_4d(base + i * C::TILE + sl * (WT * 128), &tq, q_full + i, sl * 64, it.a + i * WT, it.h, it.b);
        }
        __syncwarp();
        ++qn[i];
      };
      for (int x = blockIdx.x; x < items; x += gridDim.x) {
        const Item it = item_at(s, x);
        const TileList both = item_tiles(s, it);
        const int nt = both.count();
        for (int u = 0; u < nt; ++u) {
          const int t = both.at(u);
          load(&tk, it, t, WT);
          if (u == 0) {
            load_q(it, 0);
            load_q(it, 1);
          }
          // behind N the copy itself fills in zeros
          load(&tv, it, t, it.n < s.N && it.n - t * WT < WT ? it.n - t * WT : WT);
        }
      }
      if (wait.aborted() && lane == 0) {     // copies in flight land before shared memory is released
        for (int i = r > C::NST ? r - C::NST : 0; i < r; ++i) mbar_wait_drain(full + i % C::NST, (i / C::NST) & 1, W_DRAIN_NS);
        if (fixes > 0) mbar_wait_drain(fix, (fixes - 1) & 1, W_DRAIN_NS);
        for (int i = 0; i < 2; ++i)
          if (qn[i] > 0) mbar_wait_drain(q_full + i, (qn[i] - 1) & 1, W_DRAIN_NS);
      }
      __syncwarp();
    } else if (warp < 9 + C::ISSUERS) {
      // ------------------------------------------------------------ MMA issuers (whole warp, one lane issues)
      constexpr int NI = 2 / C::ISSUERS;     // streams of an issuer: i0 and up
      const int me = warp - 9, i0 = me * NI;
      const uint32_t q_addr = smem_u32(base), ring = smem_u32(base + C::OFF_RING), lead = elect_one();
      uint32_t qd[NI];
      bool on[NI], first[NI], last[NI];      // the PV that a stream's last S still needs
      int qn[NI], pn[NI], done[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        qd[j] = kmajor(q_addr + (i0 + j) * C::TILE);
        on[j] = first[j] = last[j] = false;
        qn[j] = pn[j] = done[j] = 0;
      }
      Slot<C::NST> kp, vp;                   // of K and V of the next tile: every other place of the ring
      vp.next();
      Slot<C::NST> v1 = vp;                  // of V of the tile before
      bool begun = false;                    // has this CTA had a tile before?
      // O += P V of a half of the tile before, stream i0 + j
      auto pv = [&](int j, int hf) {
        const int i = i0 + j;
        const uint32_t vd = mnmajor(ring + (uint32_t)v1.at * C::TILE);
        if (hf == 0 && first[j] && done[j] > 0) wait(o_free + i, done[j] - 1);
        wait(p_full + 2 * i + hf, pn[j]);
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_ts(lead, tmem + 256 + i * 128, tmem + i * 128 + hf * HALF + ks * 8, mnmajor_step(vd, hf * 4 + ks), IDESC_PV,
                 !first[j] || hf > 0 || ks > 0);
        if (C::PARTS == 2) commit(lead, pv_done + 2 * i + hf);
        if (hf == 1) {
          ++pn[j];
          if (last[j]) {
            commit(lead, o_full + i);
            ++done[j];
          }
        }
      };
      for (int x = blockIdx.x; x < items; x += gridDim.x) {
        const Item it = item_at(s, x);
        const TileList both = item_tiles(s, it);
        TileList own[NI];
        bool fresh[NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          own[j] = stream_tiles(s, it, i0 + j);
          fresh[j] = true;
        }
        const int nt = uniform(both.count());
        for (int u = 0; u < nt; ++u) {
          const int t = uniform(both.at(u));
          const uint32_t kd = kmajor(ring + (uint32_t)kp.at * C::TILE);
          // every tile is waited for, used or not: a place is freed by all issuers, once a round
          if (begun) wait(full + v1.at, v1.round);
          if (C::ISSUERS == 2) wait(full + kp.at, kp.round);
#pragma unroll
          for (int part = 0; part < C::PARTS; ++part)
#pragma unroll
            for (int j = 0; j < NI; ++j) {
              const int i = i0 + j;
              const bool qk = own[j].has(t);
              if (on[j]) {
                pv(j, part);
                if (C::PARTS == 1) pv(j, 1);
              }
              if (part == C::PARTS - 1) {
                on[j] = qk;
                first[j] = fresh[j];
                last[j] = t == own[j].hi;
              }
              if (!qk) continue;
              if (part == 0 && fresh[j]) wait(q_full + i, qn[j]++);
              if (C::ISSUERS == 1) wait(full + kp.at, kp.round);
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                mma_ss(lead, tmem + i * 128 + part * HALF, kmajor_step(qd[j], ks),
                       kmajor_step(kd + part * (HALF * 128 >> 4), ks), IDESC_QK, ks > 0);
              commit(lead, s_full + 2 * i + part);
              if (part == C::PARTS - 1) {
                if (t == own[j].hi) commit(lead, q_free + i);
                fresh[j] = false;
              }
            }
          if (begun) commit(lead, empty + v1.at);
          commit(lead, empty + kp.at);
          begun = true;
          v1 = vp;
          kp.next();
          kp.next();
          vp.next();
          vp.next();
        }
      }
      if (begun) wait(full + v1.at, v1.round);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          if (on[j]) pv(j, hf);
      if (wait.aborted()) {                  // MMAs in flight end before the tensor memory is released
        commit(lead, drain + me);
        mbar_wait_drain(drain + me, 0, W_DRAIN_NS);
      }
      __syncwarp();
    }
  } else {
    regs_inc<216>();
    // ------------------------------------------------------------ softmax warps
    const int i = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t sp = lanes + i * 128, oc = lanes + 256 + i * 128;
    uint8_t* stage = base + C::OFF_OUT + warp * 4096;
    const float sc = s.scale * W_LOG2E;
    int sn = 0, on = 0;
    for (int x = blockIdx.x; x < items; x += gridDim.x) {
      const Item it = item_at(s, x);
      const TileList own = stream_tiles(s, it, i);
      const int a = it.a + i * WT, row = a + r, nt = own.count();
      float m = -INFINITY, l = 0.f;
      for (int u = 0; u < nt; ++u) {
        const int t = own.at(u);
        const bool whole = all_visible(s, it.n, a, t);
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
          constexpr int CH = 4 / C::PARTS;   // chunks of 32 columns
          const uint32_t sh = sp + part * HALF;
          wait(s_full + 2 * i + part, sn);
          tc_fence_after();
          uint32_t v[CH][32];
#pragma unroll
          for (int c = 0; c < CH; ++c) tmem_ld32(sh + c * 32, v[c]);
          tmem_wait_ld();
          if (!whole) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const uint32_t w = key_mask(s, it.n, row, t * WT + part * HALF + c * 32);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(w >> e & 1u)) v[c][e] = 0xff800000u;       // -inf
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            constexpr int M = 8 * CH;        // columns of a quarter
            const uint32_t* x = v[c * M / 32] + c * M % 32;
            mx[c] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
            for (int e = 2; e < M; e += 2) mx[c] = fmax3(mx[c], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
          const float m_old = m;
          if (top > m + LAZY || m == -INFINITY) m = top;
          const float mu = m == -INFINITY ? 0.f : m;             // a row that has seen nothing yet
          if (__any_sync(~0u, m != m_old)) {
            const float corr = ex2_approx(m_old - mu);
            l *= corr;
            if (u > 0 || part > 0) {
              // Of one part, S is complete, and so is every product issued before it; of two, the last product
              // that adds to O was issued behind this S
              if (C::PARTS == 2) {
                wait(pv_done + 2 * i + (part ^ 1), part ? sn : sn - 1);
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(oc + c * 16, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                tmem_st16(oc + c * 16, o);
              }
            }
          }
          const float off = UP<T> > 0.f ? UP<T> - mu : -mu;
          const uint64_t sc2 = f2_pack(sc, sc), mu2 = f2_pack(off, off);
          uint64_t l2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              const uint64_t y = f2_fma(f2_pack(__uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1])), sc2, mu2);
              f2_unpack(y, x0, x1);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              l2[(e >> 1) & 1] = f2_add(l2[(e >> 1) & 1], f2_pack(x0, x1));
              pk[e >> 1] = pack16<T>(x0, x1);
            }
            tmem_st16(sh + (C::PARTS == 2 || c < 2 ? c * 16 : HALF + (c - 2) * 16), pk);
            if (c & 1) {                     // 64 keys: the products of a half may begin
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_full + 2 * i + (C::PARTS == 2 ? part : c >> 1));
            }
          }
          float y0, y1;
          f2_unpack(f2_add(l2[0], l2[1]), y0, y1);
          l += y0 + y1;
        }
        ++sn;
      }
      // ---- the item's rows: O / l, zero behind the sequence's end
      const bool live = row < it.n;
      const float inv = live ? 1.f / l : 0.f;
      if (nt > 0) {
        wait(o_full + i, on++);
        tc_fence_after();
      }
#pragma unroll 1
      for (int sl = 0; sl < C::SLABS; ++sl) {
        if (lane == 0) bulk_wait_read0();                        // the staging rows are free again
        __syncwarp();
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t o[32];
          if (nt > 0) {
            tmem_ld32(oc + sl * 64 + hf * 32, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = live ? pack16<T>(__uint_as_float(o[ch * 8 + 2 * e]) * inv, __uint_as_float(o[ch * 8 + 2 * e + 1]) * inv) : 0u;
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((hf * 4 + ch) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (nt > 0 && sl == C::SLABS - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free + i);
        }
        fence_proxy_async_smem();
        __syncwarp();
        const int row0 = a + (warp & 3) * 32;
        if (lane == 0 && row0 < s.N) {
          tma_store_4d(&to, stage, sl * 64, row0, it.h, it.b);
          bulk_commit();
        }
      }
      if (lse && row < s.N)
        lse[((long long)it.b * s.Hq + it.h) * s.N + row] = live ? ((UP<T> > 0.f ? m - UP<T> : m) + log2f(l)) * W_LN2 : -INFINITY;
    }
    if (lane == 0) bulk_wait0();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class T, int D>
cudaError_t launch_t(const WindowShape& s, const WindowFwdArgs& a, cudaStream_t st) {
  auto kern = window_fwd_kernel<T, D>;
  static unsigned long long done = 0;
  cudaError_t e = allow_smem(kern, Cfg<D>::SMEM, &done, 168);
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_4d(&tq, a.q, s.B, s.Hq, s.N, D, 64, WT) || !make_tmap_4d(&tk, a.k, s.B, s.Hkv, s.N, D, 64, WT) ||
      !make_tmap_4d(&tv, a.v, s.B, s.Hkv, s.N, D, 64, WT) || !make_tmap_4d(&to, a.out, s.B, s.Hq, s.N, D, 64, 32))
    return cudaErrorInvalidValue;
  const int items = s.B * s.Hq * ((s.N + 2 * WT - 1) / (2 * WT));
  kern<<<items < SM_COUNT ? items : SM_COUNT, 384, Cfg<D>::SMEM, st>>>(tq, tk, tv, to, s, a.lse, items);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_forward(const WindowShape& s, int fp16, const WindowFwdArgs& a, cudaStream_t st) {
  if (fp16) return s.d == 128 ? launch_t<__half, 128>(s, a, st) : launch_t<__half, 64>(s, a, st);
  return s.d == 128 ? launch_t<__nv_bfloat16, 128>(s, a, st) : launch_t<__nv_bfloat16, 64>(s, a, st);
}

}  // namespace sla2
