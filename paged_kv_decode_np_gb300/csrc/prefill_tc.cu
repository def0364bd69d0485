// prefill_tc.cu -- np_paged_prefill for bf16 on the tensor cores (tcgen05),
// compiled once per head_dim (-DNPK_D).
//
// A tile is 128 (token, head) rows of one kv head, token-major: the GQA
// group's heads of one chunk token are neighbouring rows, so one fetch of K
// and V serves G heads and a one-token row fills G rows.  Per kv tile of BN
// tokens and q tile w:
//     S_w = Q_w K^T            tcgen05.mma, both operands in shared memory
//     P_w = 2^(c S_w - m)      fp32 -> bf16, into tensor memory
//     O_w += P_w V             tcgen05.mma, A = P_w from tensor memory
// Roles: MT warpgroups of softmax (one thread a row: no shuffles), one warp
// that issues the mma, one that loads q and K, one that loads V.  With two q
// tiles (head_dim <= 128) the tensor cores work on one while the other's softmax runs:
//     ... PV_0(j), S_0(j+1) | PV_1(j), S_1(j+1) ...
// and the two share every K and V tile, 128 operations a byte of it in
// shared memory.  In a unit of one tile (a row with few tokens; always at
// head_dim 256, whose O takes 256 of the 512 columns) S(j+1) runs under softmax j.
//
// Tensor memory: one S, two P, O.  mma of different shapes or accumulators have
// no order among themselves, so none may write what an earlier one still reads:
// - S is free once the softmax has read it, into registers, at its beginning
//   (s_read; the issuing warp waits for that of the S before, whichever tile's);
// - a P (a q tile's; of one tile alone, that of every other kv tile) is written
//   after its tile's S(j) is complete, whose commit covers every P V that was
//   issued before S(j) and with that all uses of this P.
// (With P over its S, as one buffer a tile, S(j+1) has to wait for P V(j): mixed
// batch 254 us, chunk 1024 of 131072 3490 us, prompts 267 us; so 242, 3250, 240.)
//
// The running maximum is replaced only where it would grow by more than 2^8
// (m need not be the maximum, only near it: p <= 256 keeps its relative
// precision in bf16 and its sum in fp32); then the row's warp rescales O in
// tensor memory itself, which is rare after the first tiles.  P is rounded
// to bf16 for its product with V (half a step of each weight); l sums the
// unrounded p.
//
// K and V land in shared memory as [8 tokens][64-dim slab][token][128 bytes] in
// the 128-byte swizzle, which is both K^T's K-major and V's N-major operand
// layout: 8-token groups are SL KB apart, a group's slabs 1 KB.  With head_dim
// a multiple of 64 and block_size a multiple of 8 one tiled copy moves
// box_tokens of a block, all slabs (TILED: the map's dimensions are 64 dims,
// token of 8, slab, 8-token group, kv head, in the order the box lands); other
// shapes take 16-byte asynchronous copies token by token, swizzled by hand.
//
// Bound: the chain S -> softmax -> P V of a q tile, ~3200 cycles a kv tile (1500
// of them the softmax) against 2048 of mma for the pair (head_dim 128).  1024
// tokens over 131072 positions, 64 / 8 heads: 3.2-3.46 ms by the box, 1270-1370
// TFLOP/s; a shorter one under the profiler has the tensor pipe 65 % active.  Six
// prompts of 581-2750 tokens, 40 / 8 heads: 240-256 us, 710-760 TFLOP/s; 62
// one-token rows and two chunks of 512 over 1024-8192 positions: 240-246 us, 5.0
// TB/s.  The roles' code is kept small on purpose: unrolling a loader's loop or
// another copy of the mma sequence cost 5 to 20 % in instruction fetch.
#include <limits.h>

#include "prefill.cuh"
#include "tcgen05.cuh"

#ifndef NPK_D
#error "compiled per head_dim"
#endif

namespace npk {

template <int D>
struct TcCfg {
  static constexpr int SL = D > 64 ? D / 64 : 1;    // 64-dim slabs
  static constexpr int MT = D == 256 ? 1 : 2;       // q tiles of a unit
  static constexpr int BN = D == 256 ? 64 : 128;    // kv tile
  static constexpr int SLOT = SL * BN * 128;        // bytes of a K or V tile
  static constexpr int QT = SL * 128 * 128;         // bytes of a q tile
  static constexpr int FIT = (227 * 1024 - 2048 - MT * QT) / SLOT;
  static constexpr int NS = FIT < 8 ? FIT : 8;      // slots of the K/V ring
  static constexpr int RING = MT * QT;              // offset of the ring
  static constexpr int BARS = RING + NS * SLOT;     // offset of the barriers
  static constexpr int SMEM = 1024 + BARS + 512;    // + up to 1024 of alignment
  static constexpr int THREADS = 128 * (MT + 1);    // whole warpgroups: setmaxnreg is theirs
  static constexpr int BM = 128 * MT;
  // tensor memory columns: S at 0 (BN), the two P (BN / 2 each), O
  static constexpr uint32_t P0 = BN, O0 = 256;
  // A loader waits for the slot's last use only, and skips the other loaders'
  // phases: its tile before, at most 3 positions back, waited for a slot that was
  // freed after the use before that.
  static_assert(NS >= 4, "ring");
  // One block an SM: a second would wait for the first's tensor memory.
  static_assert(2 * (SMEM + 1024) > 228 * 1024, "one block an SM");
};

// Barriers, by index from the barrier area's start (8 bytes each).
template <int D>
struct TcBars {
  static constexpr int NS = TcCfg<D>::NS;
  static constexpr int q_full = 0, q_empty = 1, kv_full = 2, kv_empty = 2 + NS;
  // s_*, o_full: by q tile; p_full: by P buffer.  Four warps arrive on s_read and
  // p_full, each once a phase: what a warp arrives for next was issued after a
  // wait for the phase before (S(j+1) after s_read of S(j); the S of a P buffer's
  // next use after the P V of this one).
  // A wait that skips phases could take an earlier one of the same parity for its
  // own.  q_*, s_*, p_full, o_full and tail_full: who waits, waits for every phase.
  // The two others are never two phases behind what is waited for:
  // - kv_empty: a loader skips the others' tiles of a slot (the lag: TcCfg::NS);
  // - pv_done, waited for only where O is rescaled: phase j - 1 at tile j, whose
  //   S(j) is complete; S(j) was issued after P V(j - 2), so that phase j - 2 is
  //   complete with it, and P V(j) is not issued before this warp's P(j).
  static constexpr int s_full = 2 + 2 * NS, s_read = s_full + 2, p_full = s_read + 2;
  static constexpr int o_full = p_full + 2;
  static constexpr int pv_done = o_full + 2;  // one-tile units: one phase a kv tile
  static constexpr int drain = pv_done + 1, tail_full = drain + 1, count = tail_full + 1;
};

// kv tiles of the current segment that q tile t sees, from kv0 on
template <int D>
__device__ __forceinline__ int tc_tiles(const PrefillParams& p, const PrefillWalk& w, int t) {
  const int64_t first = ((int64_t)w.m * TcCfg<D>::MT + t) * p.tile_tokens;
  if (first >= w.g.n) return 0;
  const int nk = prefill_kv_tiles(p, w.g, first + p.tile_tokens);
  const int end = nk < w.kv1 ? nk : w.kv1;
  return end > w.kv0 ? end - w.kv0 : 0;
}

// The current segment's unit has one q tile with tokens.
template <int D>
__device__ __forceinline__ bool tc_single(const PrefillParams& p, const PrefillWalk& w) {
  return TcCfg<D>::MT == 1 || ((int64_t)w.m * TcCfg<D>::MT + 1) * p.tile_tokens >= w.g.n;
}

// mbar_wait of a warp that may have nothing to do for a long while beside a block
// that works on: the limit runs from the last tile the block has made.
__device__ __forceinline__ bool tc_wait_beside(uint32_t bar, uint32_t parity, volatile int* abort,
                                               volatile uint32_t* tiles) {
  if (mbar_try_wait(bar, parity)) return true;
  long long t0 = clock64();
  uint32_t seen = *tiles;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      const long long t = clock64();
      if (t - t0 > kWaitLimitCycles) {
        const uint32_t now = *tiles;
        if (now == seen) {
          *abort = 1;
          return false;
        }
        seen = now;
        t0 = t;
      }
    }
  }
}

struct RingPos {
  int slot;
  uint32_t phase;
  template <int NS>
  __device__ __forceinline__ void step() {
    if (++slot == NS) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

template <int D, bool TILED>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillParams p) {
  using C = TcCfg<D>;
  using B = TcBars<D>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int MT = C::MT, BN = C::BN, SL = C::SL, NS = C::NS;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t ring = base + C::RING;
  const uint32_t bars = base + C::BARS;
  auto bar = [&](int i) { return bars + 8u * i; };
  volatile uint32_t* tail = reinterpret_cast<volatile uint32_t*>(smem + C::BARS + 8 * B::count);
  volatile int* abort = reinterpret_cast<volatile int*>(tail + 1);
  volatile uint32_t* tiles = tail + 2;  // kv tiles of one-tile units so far (tc_wait_beside)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int LOAD = 4 * MT, ISSUER = 4 * MT + 3;  // three warps load, or two (TILED)

  if (threadIdx.x == 0) {
    for (int i = 0; i < B::count; ++i)
      mbar_init(bar(i), i >= B::s_read && i < B::o_full ? 4 : 1);  // s_read, p_full: four warps
    *abort = 0;
    *tiles = 0;
    fence_mbar_init();
  }
  if (warp == ISSUER) tmem_alloc(smem_u32(const_cast<uint32_t*>(tail)), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tail;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may wait

  bool ok = true;
  PrefillWalk w;

  // Registers: a softmax thread holds a row of S (BN values).  With 384 threads
  // each has 168 at launch; 2 x 208 + 88 = 3 x 168.
  if (warp < 4 * MT) {
    if constexpr (MT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    w.start(p, blockIdx.x);
    // ============================================================= softmax
    const int t = warp >> 2;                         // q tile
    const int row = (warp & 3) * 32 + lane;          // its row: tensor memory lane
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = lanes + C::O0 + t * D;
    const int tt = row / p.group, h = row - tt * p.group;
    constexpr int OC = D < 32 ? 16 : 32;             // columns of O at a time
    uint32_t used = 0;            // S tiles so far
    uint32_t pv = 0, oc = 0;      // phases of pv_done; of this tile's o_full
    while (ok && w.next(p)) {
      const int64_t first = ((int64_t)w.m * MT + t) * p.tile_tokens;
      if (first >= w.g.n) {  // no tokens in this tile
        w.advance();
        continue;
      }
      const bool single = tc_single<D>(p, w);
      const int n = tc_tiles<D>(p, w, t);
      const int64_t tok = first + tt;
      const bool live = tt < p.tile_tokens && tok < w.g.n;
      const bool idle = !__any_sync(FULL, live);  // none of the warp's rows is stored
      // the last position the row sees; rows that are not stored need no mask
      const int lim = live ? (int)((int64_t)w.g.c - w.g.n + tok) : INT_MAX;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        const int pb = single ? (j & 1) : t;  // P buffer
        // (tile 1's warps pass over the units of one tile before, a share's worth of them)
        ok = __all_sync(FULL, tc_wait_beside(bar(B::s_full + t), used & 1u, abort, tiles));
        if (!ok) break;
        ++used;
        if (idle) {  // P of these rows is whatever is there: it moves their own O only
          if (lane == 0) {
            mbar_arrive(bar(B::s_read + t));
            mbar_arrive(bar(B::p_full + pb));
          }
          continue;
        }
        tmem_fence_after();
        const uint32_t p_at = lanes + C::P0 + pb * (BN / 2);
        const int rel = lim - (w.kv0 + j) * BN;  // last visible column
        const bool masked = __any_sync(FULL, rel < BN - 1);
        uint32_t r[BN];  // the row of S
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld32(lanes + c, r + c);
        tmem_wait_ld();
        tmem_pin<BN>(r);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::s_read + t));
        if (masked) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c > rel) r[c] = 0xff800000u;  // -inf
        }
        float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < BN; c += 8) {
          x0 = fmaxf(fmaxf(x0, __uint_as_float(r[c])), __uint_as_float(r[c + 1]));
          x1 = fmaxf(fmaxf(x1, __uint_as_float(r[c + 2])), __uint_as_float(r[c + 3]));
          x2 = fmaxf(fmaxf(x2, __uint_as_float(r[c + 4])), __uint_as_float(r[c + 5]));
          x3 = fmaxf(fmaxf(x3, __uint_as_float(r[c + 6])), __uint_as_float(r[c + 7]));
        }
        const float mt = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * p.qscale;
        const bool grow = mt > m + 8.f;  // also the first visible tile: m = -inf
        if (__any_sync(FULL, grow)) {
          const float f = grow ? ex2(m - mt) : 1.f;
          if (grow) m = mt;
          l *= f;
          if (j > 0) {
            // PV(j - 1) must be complete.  With two q tiles it is: S(j) was
            // issued after it.  With one, S(j) was issued before it.
            if (single) {
              ok = __all_sync(FULL, mbar_wait(bar(B::pv_done), (pv + (uint32_t)j - 1u) & 1u, abort));
              if (!ok) break;
              tmem_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + c, o);
              tmem_wait_ld();
              tmem_pin<16>(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_at + c, o);
            }
            tmem_wait_st();
          }
        }
        const float ref = m == -INFINITY ? 0.f : -m;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < BN; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a = __uint_as_float(r[c + e]), b = __uint_as_float(r[c + e + 1]);
            fma2(a, b, p.qscale, ref);
            a = ex2(a);
            b = ex2(b);
            add2(l0, l1, a, b);
            const __nv_bfloat162 hh = __floats2bfloat162_rn(a, b);
            pk[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          tmem_st16(p_at + (c >> 1), pk);
        }
        l += l0 + l1;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::p_full + pb));
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(FULL, mbar_wait(bar(B::o_full + t), oc & 1u, abort));
        if (!ok) break;
        ++oc;
        tmem_fence_after();
      }
      if (single) pv += (uint32_t)n;
      if (idle) {
        tmem_fence_before();
        w.advance();
        continue;
      }
      // ---- the row's result: out, or this block's partial of a cut unit
      const bool whole = w.whole();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                           ((w.g.q0 + tok) * p.q_heads + (int64_t)w.kvh * p.group + h) * D;
      float* part = p.parts + (size_t)(2 * blockIdx.x + (w.kv0 > 0 ? 0 : 1)) *
                                  prefill_part_floats(C::BM, D);
      const int urow = t * 128 + row;
      if (!whole) {
        part[urow] = m;
        part[C::BM + urow] = l;
      }
      // (rolled, as is the mma's loop over all of a unit: four roles share the
      // instruction caches.  Prompts 260 us unrolled, 240 so)
#pragma unroll 1
      for (int c = 0; c < D; c += OC) {
        uint32_t o[OC];
        if (n > 0) {
          if constexpr (OC == 32) tmem_ld32(o_at + c, o);
          else tmem_ld16(o_at + c, o);
          tmem_wait_ld();
          tmem_pin<OC>(o);
        } else {  // a later piece of the unit, past what this tile sees
#pragma unroll
          for (int e = 0; e < OC; ++e) o[e] = 0u;
        }
        if (whole) {
          if (live) {
#pragma unroll
            for (int e = 0; e < OC; e += 8) {
              float x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(o[e + i]) * inv;
              Storage<__nv_bfloat16>::store<8>(out + c + e, x);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < OC; e += 4)
            *reinterpret_cast<uint4*>(part + 2 * C::BM + ((size_t)((c + e) / 4) * C::BM + urow) * 4) =
                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      tmem_fence_before();  // O is read before the next unit's first P is reported
      w.advance();
    }
  } else {
   if constexpr (MT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
   w.start(p, blockIdx.x);
   if (warp < LOAD + (TILED ? 2 : 3)) {
    // =============================================================== loads
    // TILED: one warp copies q and the K tiles, another the V tiles (a copy costs
    // its issuing thread tens of cycles, and a tile is up to 16 of them).  Token
    // by token, 64 copies of the whole warp a tile and some 70 cycles each: three
    // warps take the tiles in turn, the first one q too.
    const int id = warp - LOAD;
    const int G = p.group;
    uint32_t seg = 0, seq0 = 0;  // segments; ring tiles before this segment
    int64_t last = -1;  // the last tile's ring position (for the drain)
    uint32_t tails = 0; // TILED: phases of tail_full
    int pending = -1;   // token by token: the slot whose copies are in flight

    // the pool slot of the row's position t, its block id checked
    auto pool_slot = [&](unsigned t) {
      const unsigned j = t / (unsigned)p.block_size;
      int64_t b = p.block_tables[(int64_t)w.r * p.max_blocks_per_row + j];
      if (b < 0 || b >= p.num_blocks) {
        set_flag(p.err, NP_FLAG_BLOCK_ID);
        b = 0;
      }
      return b * p.block_size + (t - j * p.block_size);
    };
    // TILED: the pool slot of lane i's box of kv tile kt, read a tile ahead
    auto look_up = [&](int kt) {
      const int off = lane * p.box_tokens;
      return off < BN && kt * BN + off < w.g.c ? (int32_t)pool_slot((unsigned)(kt * BN + off)) : 0;
    };
    // token by token: the pending tile's copies are complete, for the mma too
    auto report = [&]() {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kv_full + pending));
    };
    // V rows past the context are zeroed, whatever their slots hold: 0 x NaN is
    // NaN.  (K's only make scores that are masked.)
    auto clear_tail = [&](uint32_t slot, int valid) {
      const int from = max(valid, 0);
      unsigned char* to = smem + C::RING + slot * C::SLOT;
      for (int e = from * SL * 8 + lane; e < BN * SL * 8; e += 32)
        *reinterpret_cast<uint4*>(to + tc_kv_at<SL>(e / (SL * 8), e % (SL * 8))) =
            make_uint4(0u, 0u, 0u, 0u);
    };
    // copies kv tile kt of K or V to position `seq` of the ring; at: look_up(kt)
    auto load_tile = [&](bool isv, int kt, uint32_t seq, int32_t at) {
      const uint32_t slot = seq % NS;
      const int valid = min(BN, w.g.c - kt * BN);  // <= 0: a row without history
      // token by token: byte offsets of tokens lane, 32 + lane, ..., on their way
      // while the slot is waited for
      constexpr int TOK = TILED ? 1 : BN / 32;
      int64_t mine[TOK];
      if constexpr (!TILED) {
#pragma unroll
        for (int x = 0; x < TOK; ++x)
          mine[x] = x * 32 + lane < valid
                        ? pool_slot((unsigned)(kt * BN + x * 32 + lane)) * p.kv_heads * (D * 2)
                        : -1;
      }
      if (seq >= NS) {
        const uint32_t phase = (seq / NS - 1u) & 1u;
        if (!TILED && pending >= 0 &&
            !__all_sync(FULL, mbar_try_wait(bar(B::kv_empty + slot), phase))) {
          cp_async_wait<0>();  // not yet: the mma may need the pending tile first
          report();
          pending = -1;
        }
        ok = __all_sync(FULL, mbar_wait(bar(B::kv_empty + slot), phase, abort));
        if (!ok) return;
      }
      const uint32_t dst = ring + slot * C::SLOT;
      if constexpr (TILED) {
        // a context's last V tile lands on a barrier of this warp's, which
        // clears its tail and then reports it
        const bool tail = isv && valid < BN;
        const uint32_t fb = bar(tail ? B::tail_full : B::kv_full + slot);
        const int bt = p.box_tokens;
        const int nbox = valid > 0 ? (valid + bt - 1) / bt : 0;
        if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(nbox * SL * bt) * 128u);
        const CUtensorMap* map = isv ? &p.tm_v : &p.tm_k;
        __syncwarp();
        for (int i = 0; i < nbox; ++i)
          tma_load_5d_warp(dst + (uint32_t)(i * bt) * (SL * 128u), map,
                           __shfl_sync(FULL, at, i) >> 3, w.kvh, fb);
        if (tail) {
          ok = __all_sync(FULL, mbar_wait(fb, tails & 1u, abort));
          ++tails;
          if (!ok) {
            mbar_wait_drain(fb, (tails - 1u) & 1u);
            return;
          }
          clear_tail(slot, valid);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::kv_full + slot));
        }
        last = seq;
      } else {
        constexpr int CH = D / 8;      // 16-byte pieces of a token
        constexpr int PER = 32 / CH;   // tokens a warp copies at a time
        static_assert(CH <= 32, "a token's pieces fit a warp");
        const char* src = static_cast<const char*>(isv ? p.v_pool : p.k_pool) + (int64_t)w.kvh * D * 2 +
                          lane % CH * 16;
        // lane: piece ch of the tokens sub, sub + PER, ...; where token 8 a + b + sub
        // (b a multiple of PER) goes, tc_kv_at, is a sum of what depends on a, on
        // b and on the lane, but for the swizzle: b's bits flip the lane's
        const int ch = lane % CH, sub = lane / CH;
        const uint32_t to = dst + (uint32_t)(((sub >> 3) * SL + (ch >> 3)) * 1024 + (sub & 7) * 128);
        const uint32_t swz = (uint32_t)(((ch & 7) ^ (sub & 7)) << 4);
        // (rolled: four roles share the instruction caches)
#pragma unroll 1
        for (int r0 = 0; r0 < valid; r0 += 32) {
#pragma unroll 8
          for (int i = 0; i < 32; i += PER) {
            const int64_t at = __shfl_sync(FULL, mine[0], i + sub);
            if (at >= 0)
              cp_async16(to + (uint32_t)(((r0 + i) >> 3) * (SL * 1024) + (i & 7) * 128) +
                             (swz ^ (uint32_t)((i & 7) << 4)),
                         src + at);
          }
#pragma unroll
          for (int x = 0; x + 1 < TOK; ++x) mine[x] = mine[x + 1];
        }
        if (isv && valid < BN) clear_tail(slot, valid);
        cp_async_commit();
        if (pending >= 0) {  // one tile's copies stay in flight
          cp_async_wait<1>();
          report();
        }
        pending = (int)slot;
      }
    };

    while (ok && w.next(p)) {
      int32_t ahead = TILED ? look_up(w.kv0) : 0;
      const bool single = tc_single<D>(p, w);
      if (id == 0) {
        // ---- q
        if (seg > 0) {
          ok = __all_sync(FULL, mbar_wait(bar(B::q_empty), (seg - 1) & 1u, abort));
          if (!ok) break;
        }
        const int qt = single ? 1 : 2;
        if constexpr (D >= 64) {  // (tiled copies whatever the pools take)
          if (lane == 0)
            mbar_arrive_expect_tx(bar(B::q_full), (uint32_t)(qt * SL * G * p.tile_tokens) * 128u);
          __syncwarp();
          for (int i = 0; i < qt * SL; ++i)
            tma_load_3d_warp(base + (uint32_t)i * 16384u, &p.tm_q, (i % SL) * 64, w.kvh * G,
                             w.g.q0 + (w.m * MT + i / SL) * p.tile_tokens, bar(B::q_full));
        } else {
          constexpr int CH = D / 8;
          for (int e = lane; e < qt * 128 * CH; e += 32) {
            const int row = e / CH, ch = e % CH;  // row of the unit
            const int t = row >> 7, in = row & 127;
            const int tt = in / G, h = in - tt * G;
            const int tok = (w.m * MT + t) * p.tile_tokens + tt;
            if (tt < p.tile_tokens && tok < w.g.n)
              cp_async16(base + (uint32_t)t * C::QT + (uint32_t)((ch >> 3) * 128 + in) * 128u +
                             (uint32_t)(((ch & 7) ^ (in & 7)) << 4),
                         static_cast<const char*>(p.q) +
                             (((int64_t)(w.g.q0 + tok) * p.q_heads + w.kvh * G + h) * D + ch * 8) * 2);
          }
          cp_async_commit();
          cp_async_wait<0>();  // nothing else is in flight at a segment's start
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::q_full));
        }
      }
      ++seg;
      // ---- this warp's tiles, at their positions in the order the mma takes
      // them: K0 V0 K1 V1 ... with two q tiles, K0 K1 V0 K2 V1 ... V with one
      const int n = w.kv1 - w.kv0;
      if constexpr (TILED) {
        const bool isv = id == 1;
        for (int j = 0; j < n && ok; ++j) {
          const int32_t at = ahead;
          if (j + 1 < n) ahead = look_up(w.kv0 + j + 1);
          uint32_t seq;
          if (!single) seq = 2u * j + (isv ? 1u : 0u);
          else if (isv) seq = j + 1 < n ? 2u * j + 2u : 2u * n - 1u;
          else seq = j == 0 ? 0u : 2u * j - 1u;
          load_tile(isv, w.kv0 + j, seq0 + seq, at);
        }
      } else {
        for (int s = 0; s < 2 * n && ok; ++s) {
          if ((seq0 + (uint32_t)s) % 3u != (uint32_t)id) continue;
          bool isv = s & 1;
          int j = s >> 1;
          if (single) {
            isv = s == 2 * n - 1 || (s > 0 && !isv);
            j = s == 0 ? 0 : (s == 2 * n - 1 ? n - 1 : (isv ? s / 2 - 1 : (s + 1) / 2));
          }
          load_tile(isv, w.kv0 + j, seq0 + (uint32_t)s, 0);
        }
      }
      seq0 += 2u * n;
      if constexpr (!TILED) {  // all of it is reported before the next q waits for it
        cp_async_wait<0>();
        if (pending >= 0) report();
        pending = -1;
      }
      w.advance();
    }
    if (*abort) {  // never leave copies in flight (bounded)
      if (D >= 64 && id == 0 && seg > 0) mbar_wait_drain(bar(B::q_full), (seg - 1) & 1u);
      if constexpr (TILED) {
        // the last NS positions up to this warp's last tile: those of the other
        // warp's that never came run into the wait's limit
        for (int64_t q = last > NS ? last - NS : 0; q <= last; ++q)
          mbar_wait_drain(bar(B::kv_full + (int)(q % NS)), (uint32_t)(q / NS) & 1u);
      } else {
        cp_async_wait<0>();
      }
    }
   } else if (warp == ISSUER) {
    // ================================================================= mma
    // The whole warp runs the role, its lanes alike; one of them issues.
    constexpr uint32_t PV = umma_idesc_bf16(128, D, true);
    constexpr uint32_t QHI = umma_desc_hi(1024), KVHI = umma_desc_hi(SL * 1024);
    const uint32_t QK = umma_idesc_bf16(128, BN, false, p.negate != 0);
    RingPos pos{0, 0};
    uint32_t seg = 0;
    uint32_t done0 = 0, done1 = 0;  // phases of each p_full so far
    int s_bar = -1;                 // s_read of the last S issued, and its phase
    uint32_t s_phase = 0, issued0 = 0, issued1 = 0;

    auto wait = [&](int b, uint32_t phase) {
      ok = ok && __all_sync(FULL, mbar_wait(bar(b), phase, abort));
      return ok;
    };
    auto issue_s = [&](int t, int slot) {  // S = Q_t K^T, once the S before has been read
      if (s_bar >= 0 && !wait(s_bar, s_phase)) return false;
      s_bar = B::s_read + t;
      s_phase = (t ? issued1++ : issued0++) & 1u;
      tmem_fence_after();
      const uint32_t q = umma_desc_lo(base + (uint32_t)t * C::QT, 16);
      const uint32_t k = umma_desc_lo(ring + (uint32_t)slot * C::SLOT, 16);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        umma_ss(tmem, q + ((ks >> 2) * 16384u + (ks & 3) * 32u) / 16u, QHI,
                k + ((ks >> 2) * 1024u + (ks & 3) * 32u) / 16u, KVHI, QK, ks > 0);
      umma_commit(bar(B::s_full + t));
      return true;
    };
    auto issue_pv = [&](int t, int pb, int slot, bool acc) {  // O_t += P V, P in buffer pb
      tmem_fence_after();
      const uint32_t pa = tmem + C::P0 + pb * (BN / 2);
      const uint32_t v = umma_desc_lo(ring + (uint32_t)slot * C::SLOT, 1024);
#pragma unroll
      for (int ks = 0; ks < BN / 16; ++ks)
        umma_ts(tmem + C::O0 + t * D, pa + ks * 8, v + ks * (SL * 128u), KVHI, PV,
                ks > 0 ? 1u : (acc ? 1u : 0u));
    };

    while (ok && w.next(p)) {
      const int n = w.kv1 - w.kv0;
      if (!wait(B::q_full, seg & 1u)) break;
      ++seg;
      if (!tc_single<D>(p, w)) {
        const int n0 = tc_tiles<D>(p, w, 0);  // <= n: the unit's last tokens see the most
#pragma unroll 1
        for (int j = -1; j < n; ++j) {  // P V_t(j), S_t(j + 1)
          const int vslot = pos.slot;
          const uint32_t vphase = pos.phase;
          if (j >= 0) pos.template step<NS>();
          const int kslot = pos.slot;
          const uint32_t kphase = pos.phase;
          if (j + 1 < n) pos.template step<NS>();
          if (j < n0) {
            if (j >= 0) {
              if (!wait(B::kv_full + vslot, vphase) || !wait(B::p_full, done0 & 1u)) break;
              ++done0;
              issue_pv(0, 0, vslot, j > 0);
            }
            if (j + 1 < n0) {
              if (!wait(B::kv_full + kslot, kphase) || !issue_s(0, kslot)) break;
            } else if (j >= 0) {
              umma_commit(bar(B::o_full));
            }
          }
          if (j >= 0) {
            if (!wait(B::kv_full + vslot, vphase) || !wait(B::p_full + 1, done1 & 1u)) break;
            ++done1;
            issue_pv(1, 1, vslot, j > 0);
            umma_commit(bar(B::kv_empty + vslot));
          }
          if (j + 1 < n) {
            if (!wait(B::kv_full + kslot, kphase) || !issue_s(1, kslot)) break;
            umma_commit(bar(B::kv_empty + kslot));
            if (j + 2 == n) umma_commit(bar(B::q_empty));
          } else {
            umma_commit(bar(B::o_full + 1));
          }
        }
      } else {
        for (int j = -1; j < n; ++j) {
          if (j + 1 < n) {  // S(j + 1)
            const int slot = pos.slot;
            if (!wait(B::kv_full + slot, pos.phase) || !issue_s(0, slot)) break;
            pos.template step<NS>();
            umma_commit(bar(B::kv_empty + slot));
            if (j + 2 == n) umma_commit(bar(B::q_empty));
          }
          if (j >= 0) {  // O += P(j) V(j)
            const int slot = pos.slot;
            const uint32_t phase = pos.phase;
            pos.template step<NS>();
            if (!wait(B::kv_full + slot, phase) ||
                !wait(B::p_full + (j & 1), (j & 1 ? done1 : done0) & 1u))
              break;
            if (j & 1) ++done1;
            else ++done0;
            issue_pv(0, j & 1, slot, j > 0);
            umma_commit(bar(B::pv_done));
            umma_commit(bar(B::kv_empty + slot));
            if (MT == 2 && lane == 0) *tiles = *tiles + 1u;
            if (j + 1 == n) umma_commit(bar(B::o_full));
          }
        }
      }
      w.advance();
    }
    // nothing of this block is left running in the tensor cores (bounded)
    umma_commit(bar(B::drain));
    mbar_wait_drain(bar(B::drain), 0u);
    __syncwarp();
   }
  }
  if (!ok && lane == 0) set_flag(p.err, NP_FLAG_TIMEOUT);
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == ISSUER) {
    tmem_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool TILED>
static np_status launch(const PrefillParams& p, cudaStream_t s) {
  static unsigned long long allowed = 0;
  const np_status rc = allow_smem(prefill_tc_kernel<D, TILED>, TcCfg<D>::SMEM, &allowed);
  if (rc != NP_OK) return rc;
  return launch_dependent(prefill_tc_kernel<D, TILED>, p.ctas, 1, TcCfg<D>::THREADS, TcCfg<D>::SMEM, s,
                          p);
}

#define NPK_CAT2(a, b) a##b
#define NPK_CAT(a, b) NPK_CAT2(a, b)

np_status NPK_CAT(prefill_tc_d, NPK_D)(const PrefillParams& p, bool tiled, cudaStream_t s) {
#if NPK_D >= 64
  if (tiled) return launch<NPK_D, true>(p, s);
#endif
  return launch<NPK_D, false>(p, s);
}

}  // namespace npk
