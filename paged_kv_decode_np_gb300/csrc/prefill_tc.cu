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
// An 8-bit cache (Q8, compiled apart) comes in one of two ways.
// Tiled copies (Q8T): a tile's bytes land in rings of their own, one for K and one for V,
// from which four warps widen a quarter of each tile to fp16, which holds every code:
// two or three instructions for four codes, where bf16 takes ten.  A tile's largest
// exponents (of its blocks' scales; one for K, one for V) stay apart from its values: K's
// is a factor of the tile's scores, V's is added to the exponents of its weights and
// taken back in l, as 2^(x + b) v and 2^x are a weight's two shares.  Blocks of smaller
// scales are multiplied by what they are below the largest, 2^-kWide at most, which is
// exact.  In a tile whose scales lie further apart (it is wide) the codes stay as they are,
// and the softmax takes the exponents group by group: a largest one that belongs to
// positions without weight, or not yet seen, would push the others' values out of fp16's
// range, and their weights too (tc_wide_tile).  q is fp16 as well, each row times a power of two
// that brings its largest element to 2^14 .. 2^15; the same four warps turn it in place.
// 1024 tokens of 65536, 64 / 8 heads: 1.83 ms, 1190 TFLOP/s, 60 us of it for telling wide
// tiles from others (the bf16 pools' kernel: 1.50); the four warps take ~1000 cycles a tile and the softmax 10 % longer beside
// them.  (Widened to bf16 by six instructions a pair, all pieces unrolled 3.63 ms: their
// fetching stalled everybody; rolled 2.93.)
// Token by token, six warps widen to bf16 with the scales multiplied in, exactly: they
// take the 8-token groups of the tiles in turn, each group through a ring of the warp's
// own, filled by asynchronous copies of which every lane reads back its own alone.
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

#include "cache8.cuh"
#include "prefill.cuh"
#include "tcgen05.cuh"

#ifndef NPK_D
#error "compiled per head_dim"
#endif

namespace npk {

// How K and V come: bf16 token by token, bf16 by tiled copies; 8 bits (+ form) the same two ways
enum : int { kTokens = 0, kTiled = 1, kQ8 = 2, kQ8Tiled = 4 };
// How far the exponents of a tile's scales lie apart at most that are one factor's.  (Weights
// lose as many bits at fp16's small end; a cache of tokens of one model is within two.  All
// tiles wide: chunk 1024 of 65536 4.74 ms for 1.83.)
constexpr int kWide = 4;
// How far V's may be from 0 in such a tile.  2^(x - m) is also l's term, times 2^-b: no number below
// 2^-126, which m 60 above the largest score (another tile's b) and b = -20 reach for terms
// below 2^-40 of the largest only, as does the factor of l where m grows.  Wide tiles form l's
// terms without b.
constexpr int kFar = 20;
// 0: bf16, 1: 8 bits token by token, 2: 8 bits by tiled copies
__host__ __device__ constexpr int tc_kind(int kv) { return kv >= kQ8Tiled ? 2 : kv >= kQ8 ? 1 : 0; }

template <int D, int KIND = 0>
struct TcCfg {
  static constexpr bool Q8 = KIND > 0;
  static constexpr int SL = D > 64 ? D / 64 : 1;    // 64-dim slabs
  static constexpr int MT = D == 256 ? 1 : 2;       // q tiles of a unit
  static constexpr int BN = D == 256 ? 64 : 128;    // kv tile
  static constexpr int SLOT = SL * BN * 128;        // bytes of a K or V tile
  static constexpr int QT = SL * 128 * 128;         // bytes of a q tile
  // Q8: warps that widen, the lanes' 16-byte pieces of an 8-token group; token by token:
  // bytes of a group (and its scales) and how many of them a warp's ring holds; tiled:
  // bytes of a raw tile (and its scales), tiles of the raw ring
  static constexpr int CONV = KIND == 2 ? 4 : 6;
  static constexpr int PI = D >= 64 ? D / 64 : 1;
  static constexpr int GB = PI * 512 + 128;
  static constexpr int SG = D == 256 ? 2 : D == 128 ? 4 : 8;
  static constexpr int RT = BN * D, RS = 2;  // (of K, and as many of V)
  static constexpr int STG = KIND == 2 ? 2 * RS * RT : KIND == 1 ? CONV * SG * GB : 0;
  static constexpr int FIT = (227 * 1024 - 2048 - MT * QT - STG) / SLOT;
  static constexpr int NS = FIT < 8 ? FIT : 8;      // slots of the K/V ring
  static constexpr int RING = MT * QT;              // offset of the ring
  static constexpr int RAW_T = RING + NS * SLOT;    // offset of the raw rings
  static constexpr int BARS = RAW_T + (KIND == 2 ? STG : 0);  // offset of the barriers
  static constexpr int RAW = BARS + 512;            // offset of the widening warps' rings
  // Q8T: raw rings (1024-byte aligned: swizzled copies), then barriers, a ring of the
  // tiles' exponents (TE bytes a tile: how far the groups' are below the tile's, K's and
  // V's, 0 where it is wide; the tile's K and V exponent and whether it is wide; a wide
  // one's groups, K's and V's), the exponents of q's rows by segment parity
  static constexpr int TEK = 2 * (BN / 8), TEW = TEK + 4;
  static constexpr int TE = (TEW + 2 * (BN / 8) + 3) / 4 * 4, TILES = RS + NS + 3 <= 8 ? 8 : 16;
  static constexpr int EXPS = BARS + 512, QEXP = EXPS + TILES * TE;
  static constexpr int SMEM = 1024 + (KIND == 2 ? QEXP + 2 * 128 * MT : RAW + STG);  // + up to 1024 of alignment
  static constexpr int THREADS = 128 * (MT + (Q8 ? 2 : 1));  // whole warpgroups: setmaxnreg is theirs
  static constexpr int BM = 128 * MT;
  // tensor memory columns: S at 0 (BN), the two P (BN / 2 each), O
  static constexpr uint32_t P0 = BN, O0 = 256;
  // A loader waits for the slot's last use only, and skips the other loaders'
  // phases: its tile before, at most 3 positions back, waited for a slot that was
  // freed after the use before that.
  // (Q8: all widening warps take part in every tile.)
  static_assert(NS >= (KIND == 2 ? 3 : 4), "ring");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // One block an SM: a second would wait for the first's tensor memory.
  static_assert(2 * (SMEM + 1024) > 228 * 1024, "one block an SM");
};

// Barriers, by index from the barrier area's start (8 bytes each).
template <int D, int KIND = 0>
struct TcBars {
  static constexpr int NS = TcCfg<D, KIND>::NS;
  static constexpr int q_full = 0, q_empty = 1, kv_full = 2, kv_empty = 2 + NS;
  // s_*, o_full: by q tile; p_full: by P buffer.  Four warps arrive on s_read and
  // p_full, each once a phase: what a warp arrives for next was issued after a
  // wait for the phase before (S(j+1) after s_read of S(j); the S of a P buffer's
  // next use after the P V of this one).
  // A wait that skips phases could take an earlier one of the same parity for its
  // own.  q_*, s_*, p_full, o_full and tail_full: who waits, waits for every phase.
  // The two others are never two phases behind what is waited for:
  // - kv_empty: a loader skips the others' tiles of a slot (the lag: TcCfg::NS; Q8:
  //   each of the six warps has groups of every tile, and waits for every phase);
  // - pv_done, waited for only where O is rescaled: phase j - 1 at tile j, whose
  //   S(j) is complete; S(j) was issued after P V(j - 2), so that phase j - 2 is
  //   complete with it, and P V(j) is not issued before this warp's P(j).
  static constexpr int s_full = 2 + 2 * NS, s_read = s_full + 2, p_full = s_read + 2;
  static constexpr int o_full = p_full + 2;
  static constexpr int pv_done = o_full + 2;  // one-tile units: one phase a kv tile
  static constexpr int drain = pv_done + 1, tail_full = drain + 1;
  // Q8T: raw tiles, K's ring and V's; q as it came.  Who waits, waits for every phase.
  static constexpr int raw_full = tail_full + 1, raw_empty = raw_full + 4, q_raw = raw_empty + 4;
  static constexpr int count = KIND == 2 ? q_raw + 1 : raw_full;
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

// The kv tile at position s of a segment's 2 n tiles, in the order the mma takes them:
// K0 V0 K1 V1 ... with two q tiles, K0 K1 V0 K2 V1 ... V with one.
__device__ __forceinline__ int tc_tile_at(int s, int n, bool single, bool& isv) {
  isv = s & 1;
  if (!single) return s >> 1;
  isv = s == 2 * n - 1 || (s > 0 && !isv);
  return s == 0 ? 0 : (s == 2 * n - 1 ? n - 1 : (isv ? s / 2 - 1 : (s + 1) / 2));
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

// A wide tile of the softmax, 16 columns at a time: x = c S 2^-k + b - v with the groups'
// k and v in its place, its maximum, then weights 2^(x - m) and l's terms 2^(x - b + v - m).
// Returns m and l.  (A function of its own: in line, its code made tiles that never run it a
// fifth slower, chunk 1024 of 65536 2.21 ms.)
template <int D>
__device__ __noinline__ float2 tc_wide_tile(uint32_t s_at, uint32_t p_at, uint32_t o_at,
                                            const volatile unsigned char* te, float row_scale, uint32_t tx,
                                            int rel, bool any_o, float m, float l) {
  constexpr int BN = TcCfg<D, 2>::BN;
  const float c = row_scale * pow2f((signed char)(tx & 0xffu)), b = (float)(signed char)(tx >> 8);
  float most = -INFINITY;
#pragma unroll 1
  for (int d = 0; d < BN; d += 16) {
    uint32_t y[16];
    tmem_ld16(s_at + d, y);
    tmem_wait_ld();
    tmem_pin<16>(y);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float cg = c * pow2f(-(int)te[d / 8 + g]), vg = b - (float)te[BN / 8 + d / 8 + g];
#pragma unroll
      for (int e = 8 * g; e < 8 * g + 8; ++e) {
        const float x = d + e <= rel ? fmaf(__uint_as_float(y[e]), cg, vg) : -INFINITY;
        most = fmaxf(most, x);
        y[e] = __float_as_uint(x);
      }
    }
    tmem_st16(s_at + d, y);
  }
  tmem_wait_st();
  const bool grow = most > m + 14.f;
  if (__any_sync(0xffffffffu, grow)) {
    const float fe = grow ? m - (most - 6.f) : 0.f, f = ex2(fe);
    if (grow) m = most - 6.f;
    l = scaled_down(l, fe);
#pragma unroll 1
    for (int d = 0; any_o && d < D; d += 16) {
      uint32_t o[16];
      tmem_ld16(o_at + d, o);
      tmem_wait_ld();
      tmem_pin<16>(o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st16(o_at + d, o);
    }
    tmem_wait_st();
  }
  const float ref = m == -INFINITY ? 0.f : -m;
#pragma unroll 1
  for (int d = 0; d < BN; d += 16) {
    uint32_t y[16], pk[8];
    tmem_ld16(s_at + d, y);
    tmem_wait_ld();
    tmem_pin<16>(y);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const float lg = (float)te[BN / 8 + (d + e) / 8] - b + ref;
      const float u = __uint_as_float(y[e]), v = __uint_as_float(y[e + 1]);
      l += ex2(u + lg) + ex2(v + lg);
      const __half2 hh = __floats2half2_rn(ex2(u + ref), ex2(v + ref));
      pk[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
    }
    tmem_st8(p_at + (d >> 1), pk);
  }
  tmem_wait_st();
  return make_float2(m, l);
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

template <int D, int KV>
__global__ void __launch_bounds__(TcCfg<D, tc_kind(KV)>::THREADS, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillParams p) {
  constexpr bool TILED = KV == kTiled, Q8 = KV >= kQ8, Q8T = KV >= kQ8Tiled;
  using C = TcCfg<D, tc_kind(KV)>;
  using B = TcBars<D, tc_kind(KV)>;
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
  // three warps load, or two (TILED); Q8: six widen, one loads q; Q8T: four widen, one
  // loads K, one V, one q
  constexpr int LOAD = 4 * MT, ISSUER = C::THREADS / 32 - 1;
  constexpr int CONV = Q8 ? C::CONV : 0, RAWER = LOAD + CONV, LOADERS = Q8 ? 1 : TILED ? 2 : 3;
  constexpr int Q0 = RAWER + (Q8T ? 2 : 0);  // the first loader

  if (threadIdx.x == 0) {
    for (int i = 0; i < B::count; ++i)
      mbar_init(bar(i), i >= B::s_read && i < B::o_full ? 4  // s_read, p_full: four warps
                        : Q8 && i >= B::kv_full && i < B::kv_empty ? (Q8T ? CONV : BN / 8)
                        : Q8T && ((i >= B::raw_empty && i < B::q_raw) || i == B::q_full) ? CONV : 1);
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
  // each has 168 at launch; 2 x 208 + 88 = 3 x 168.  512 threads (Q8): 128 each, 2 x 192 +
  // 2 x 64 = 4 x 128.
  if (warp < 4 * MT) {
    if constexpr (MT == 2 && !Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if constexpr (MT == 2 && Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    w.start(p, blockIdx.x);
    // ============================================================= softmax
    const int t = warp >> 2;                         // q tile
    const int row = (warp & 3) * 32 + lane;          // its row: tensor memory lane
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = lanes + C::O0 + t * D;
    const int tt = row / p.group, h = row - tt * p.group;
    constexpr int OC = D < 32 ? 16 : 32;             // columns of O at a time
    uint32_t used = 0;            // S tiles so far
    uint32_t seen = 0, segs = 0;  // Q8T: kv tiles and segments so far, whosever they were
    uint32_t pv = 0, oc = 0;      // phases of pv_done; of this tile's o_full
    while (ok && w.next(p)) {
      const int64_t first = ((int64_t)w.m * MT + t) * p.tile_tokens;
      const uint32_t tile0 = seen;
      seen += (uint32_t)(w.kv1 - w.kv0);
      ++segs;
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
      // Q8T: x = c S + b, weights 2^(x - m) with m 6 below the largest x (fp16's range)
      constexpr float ABOVE = Q8T ? 14.f : 8.f, BELOW = Q8T ? 6.f : 0.f;
      float row_scale = p.qscale;
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
        const volatile unsigned char* te = smem + C::EXPS + (tile0 + (uint32_t)j) % C::TILES * C::TE;
        uint32_t tx = 0;
        if constexpr (Q8T) {
          // (before S is given back: the next segment's exponents may come after that)
          if (j == 0)
            row_scale *= pow2f(-(int)*reinterpret_cast<volatile signed char*>(
                smem + C::QEXP + (segs & 1u) * (128 * MT) + t * 128 + row));
          tx = *reinterpret_cast<const volatile uint32_t*>(te + C::TEK);
          if (__builtin_expect(tx >> 16 != 0u, 0)) {  // uniform
            if (single && j > 0) {  // as below
              ok = __all_sync(FULL, mbar_wait(bar(B::pv_done), (pv + (uint32_t)j - 1u) & 1u, abort));
              if (!ok) break;
              tmem_fence_after();
            }
            const float2 ml = tc_wide_tile<D>(lanes, p_at, o_at, te + C::TEW, row_scale, tx, rel, j > 0, m, l);
            m = ml.x;
            l = ml.y;
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(B::s_read + t));
              mbar_arrive(bar(B::p_full + pb));
            }
            continue;
          }
        }
        uint32_t r[BN];  // the row of S
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld32(lanes + c, r + c);
        tmem_wait_ld();
        tmem_pin<BN>(r);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::s_read + t));
        float c = p.qscale, b = 0.f, back = 1.f;
        if constexpr (Q8T) {
          const int ke = (signed char)(tx & 0xffu), ve = (signed char)(tx >> 8);
          c = fmaxf(row_scale * pow2f(ke), 1.2e-38f);  // (a masked score is -inf before it is scaled)
          b = (float)ve;
          back = pow2f(-ve);
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < BN; ++e)
            if (e > rel) r[e] = 0xff800000u;  // -inf
        }
        float x0 = -INFINITY, x1 = -INFINITY, x2 = -INFINITY, x3 = -INFINITY;
#pragma unroll
        for (int e = 0; e < BN; e += 8) {
          x0 = fmaxf(fmaxf(x0, __uint_as_float(r[e])), __uint_as_float(r[e + 1]));
          x1 = fmaxf(fmaxf(x1, __uint_as_float(r[e + 2])), __uint_as_float(r[e + 3]));
          x2 = fmaxf(fmaxf(x2, __uint_as_float(r[e + 4])), __uint_as_float(r[e + 5]));
          x3 = fmaxf(fmaxf(x3, __uint_as_float(r[e + 6])), __uint_as_float(r[e + 7]));
        }
        const float most = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
        const float mt = Q8T ? fmaf(most, c, b) : most * c;
        const bool grow = mt > m + ABOVE;  // also the first visible tile: m = -inf
        if (__any_sync(FULL, grow)) {
          const float f = grow ? ex2(m - (mt - BELOW)) : 1.f;
          if (grow) m = mt - BELOW;
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
            for (int d = 0; d < D; d += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + d, o);
              tmem_wait_ld();
              tmem_pin<16>(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(o_at + d, o);
            }
            tmem_wait_st();
          }
        }
        const float ref = m == -INFINITY ? 0.f : b - m;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int k = 0; k < BN; k += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float u = __uint_as_float(r[k + e]), v = __uint_as_float(r[k + e + 1]);
            fma2(u, v, c, ref);
            u = ex2(u);
            v = ex2(v);
            add2(l0, l1, u, v);
            if constexpr (Q8T) {
              const __half2 hh = __floats2half2_rn(u, v);
              pk[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
            } else {
              const __nv_bfloat162 hh = __floats2bfloat162_rn(u, v);
              pk[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
            }
          }
          tmem_st16(p_at + (k >> 1), pk);
        }
        l = Q8T ? fmaf(l0 + l1, back, l) : l + (l0 + l1);
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
   if constexpr (MT == 2 && !Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
   if constexpr (MT == 2 && Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
   w.start(p, blockIdx.x);
   if (warp < LOAD + CONV) {
    // =============================================================== widen
    if constexpr (Q8T) {
      // q of each segment, then tile by tile, a quarter of the rows and tokens each.
      // Bytes past the context are whatever they are.  K's only make scores that are
      // masked; V's meet weights of 0, which e4m3's NaN would not stand: zeros instead.
      constexpr int GW = BN / 8 / CONV;  // 8-token groups of a warp
      constexpr int RS = C::RS, PI = C::PI, FORM = KV - kQ8Tiled;
      const int wc = warp - LOAD, tok = lane & 7, c0 = lane >> 3;
      uint32_t seq = 0, tile = 0, segs = 0;  // positions in the ring; kv tiles; segments
      while (ok && w.next(p)) {
        const bool single = tc_single<D>(p, w);
        const int n = w.kv1 - w.kv0;
        ok = __all_sync(FULL, mbar_wait(bar(B::q_raw), segs & 1u, abort));
        if (!ok) break;
        ++segs;
        for (int t = 0; t < (single ? 1 : 2); ++t) {
          // a lane's row; rows that hold no (token, head) are left as they are
          const int row = wc * 32 + lane;
          const int64_t first = ((int64_t)w.m * MT + t) * p.tile_tokens;
          const int live = (int)min((int64_t)p.tile_tokens, w.g.n - first) * p.group;
          if (wc * 32 >= live) continue;
          const uint32_t at = base + (uint32_t)t * C::QT + (uint32_t)row * 128u;
          auto piece = [&](int i) { return at + (uint32_t)((i >> 3) * 16384 + (((i & 7) ^ (row & 7)) << 4)); };
          uint32_t big = 0;
#pragma unroll 2
          for (int i = 0; i < D / 8; ++i) {
            uint32_t x[4];
            lds<4>(piece(i), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) big = __vmaxu2(big, x[e] & 0x7fff7fffu);
          }
          big = max(big & 0xffffu, big >> 16);
          const int e = min(14 + 127 - (int)(big >> 7), 120);
          const float f = pow2f(e);
#pragma unroll 1
          for (int i = 0; i < D / 8; ++i) {
            uint32_t x[4];
            lds<4>(piece(i), x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float lo, hi;
              widen_bf16x2(x[k], lo, hi);
              const __half2 h = __floats2half2_rn(lo * f, hi * f);
              x[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            sts4(piece(i), x);
          }
          smem[C::QEXP + (segs & 1u) * (128 * MT) + t * 128 + row] = (unsigned char)(signed char)e;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::q_full));
#pragma unroll 1
        for (int s = 0; s < 2 * n; ++s, ++seq) {
          bool isv;
          const int j = tc_tile_at(s, n, single, isv);
          const uint32_t slot = seq % NS, te = (tile + (uint32_t)j) % C::TILES;
          const uint32_t own = tile + (uint32_t)j, rs = own % RS + (isv ? RS : 0);
          ok = mbar_wait(bar(B::raw_full + rs), (own / RS) & 1u, abort);
          if (ok && seq >= NS) ok = mbar_wait(bar(B::kv_empty + slot), (seq / NS - 1u) & 1u, abort);
          ok = __all_sync(FULL, ok);
          if (!ok) break;
          // The lane's piece k of group i of the warp's: token r, 16-byte piece ch = c0 + 4 k.
          // In the raw tile groups are 8 D bytes apart (in boxes: box_tokens tokens, in
          // slabs of 128 bytes, swizzled), in the widened one SL KB.
          const int r0 = wc * GW * 8 + tok;
          const uint32_t from = base + C::RAW_T + rs * (uint32_t)C::RT;
          const uint32_t to = ring + slot * C::SLOT + (uint32_t)(wc * GW * SL * 1024 + tok * 128);
          auto raw = [&](int i, uint32_t (&q)[PI][4]) {
            const int r = r0 + 8 * i;
#pragma unroll
            for (int k = 0; k < PI; ++k) {
              const int ch = c0 + 4 * k;
              uint32_t at;
              if constexpr (D == 64) at = (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
              else if constexpr (D == 128) at = (uint32_t)(r * 128 + ((ch ^ tok) << 4));
              else {
                const int b = r & ~(p.box_tokens - 1);
                at = (uint32_t)(b * 256 + ((k >> 1) * p.box_tokens + r - b) * 128 + (((ch & 7) ^ tok) << 4));
              }
              lds<4>(from + at, q[k]);
            }
          };
          uint32_t below;  // how far the groups' scales are below the tile's, a byte each (0: wide)
          {
            const uint32_t at = base + C::EXPS + te * C::TE + (isv ? BN / 8 : 0) + wc * GW;
            if constexpr (GW == 4) lds<1>(at, &below);
            else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(below) : "r"(at));
          }
          const int valid = FORM == NP_E4M3 && isv ? w.g.c - (w.kv0 + j) * BN : BN;
          uint32_t q[PI][4];
          raw(0, q);
          // (a group's pieces unrolled, the groups rolled: four roles share the instruction
          // caches.  Chunk 1024 of 65536 2073 us with the pieces rolled too)
#pragma unroll 1
          for (int i = 0; i < GW; ++i) {
            uint32_t q1[PI][4];
            raw(min(i + 1, GW - 1), q1);  // on its way meanwhile
            const Below8<FORM> f(below & 0xffu);
            below >>= 8;
            if (FORM == NP_E4M3 && r0 + 8 * i >= valid) {
#pragma unroll
              for (int k = 0; k < PI; ++k) q[k][0] = q[k][1] = q[k][2] = q[k][3] = 0u;
            }
#pragma unroll
            for (int k = 0; k < PI; ++k) {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) f.widen(q[k][e], y[2 * e], y[2 * e + 1]);
              const int ch = 2 * (c0 + 4 * k);  // 16-byte piece of the widened token
              const uint32_t at = to + (uint32_t)(i * SL * 1024 + k * 1024) + (((ch & 7) ^ tok) << 4);
              sts4(at, y);
              sts4(at ^ 16u, y + 4);
#pragma unroll
              for (int e = 0; e < 4; ++e) q[k][e] = q1[k][e];
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(B::raw_empty + rs));
            mbar_arrive(bar(B::kv_full + slot));
          }
        }
        tile += (uint32_t)n;
        w.advance();
      }
    } else if constexpr (Q8) {
      constexpr int GPT = BN / 8;       // groups of a tile
      constexpr int CPT = D / 16;       // 16-byte pieces of a token
      constexpr int SG = C::SG, PI = C::PI, FORM = KV - kQ8;
      const int wc = warp - LOAD;
      const int tok = lane & 7, c0 = lane >> 3;  // token of a group; its pieces c0, c0 + 4, ..
      const uint32_t raw = base + C::RAW + (uint32_t)(wc * SG) * C::GB;
      const int64_t row = (int64_t)p.kv_heads * D;
      uint32_t seq0 = 0;                // ring tiles before this segment
      while (ok && w.next(p)) {
        const bool single = tc_single<D>(p, w);
        const int n = w.kv1 - w.kv0, NG = 2 * n * GPT;
        // the group to copy next: its tokens' blocks are looked up a group ahead
        int xl = wc, put = 0;
        bool on = false, isv = false;
        int32_t block = 0, inner = 0;
        auto look_up = [&]() {
          const int j = tc_tile_at(xl / GPT, n, single, isv);
          const int t = (w.kv0 + j) * BN + xl % GPT * 8 + tok;
          on = t < w.g.c;
          block = inner = 0;
          if (on) {
            const int b = (int)((unsigned)t / (unsigned)p.block_size);
            inner = t - b * p.block_size;
            block = p.block_tables[(int64_t)w.r * p.max_blocks_per_row + b];
          }
        };
        auto issue = [&]() {
          if (xl < NG) {
            if (block < 0 || block >= p.num_blocks) {
              set_flag(p.err, NP_FLAG_BLOCK_ID);
              block = 0;
            }
            const uint32_t to = raw + (uint32_t)put * C::GB;
            const char* src = static_cast<const char*>(isv ? p.v_pool : p.k_pool) +
                              ((int64_t)block * p.block_size + inner) * row + w.kvh * D;
#pragma unroll
            for (int i = 0; i < PI; ++i)
              if (CPT >= 4 || c0 < CPT) copy16(to + i * 512 + lane * 16, src + (c0 + 4 * i) * 16, on);
            copy4(to + PI * 512 + lane * 4,
                  (isv ? p.v_scale : p.k_scale) + (int64_t)block * p.kv_heads + w.kvh, on);
            put = put + 1 == SG ? 0 : put + 1;
            xl += CONV;
            if (xl < NG) look_up();
          }
          cp_async_commit();
        };
        look_up();  // (a segment has two tiles at least, a tile more groups than warps)
#pragma unroll 1
        for (int i = 0; i < SG - 1; ++i) issue();
        int get = 0, was = -1;
        for (int x = wc; x < NG; x += CONV) {
          cp_async_wait<SG - 2>();
          issue();  // to where the group before lay
          const int s = x / GPT;
          const uint32_t seq = seq0 + (uint32_t)s, slot = seq % NS;
          if (s != was) {
            was = s;
            if (seq >= NS) {
              ok = __all_sync(FULL, mbar_wait(bar(B::kv_empty + slot), (seq / NS - 1u) & 1u, abort));
              if (!ok) break;
            }
          }
          const uint32_t from = raw + (uint32_t)get * C::GB;
          get = get + 1 == SG ? 0 : get + 1;
          uint32_t bits;
          lds<1>(from + PI * 512 + lane * 4, &bits);
          const Scaled8<FORM> sc(scale_exp(bits));
          unsigned char* dst = smem + C::RING + slot * C::SLOT;
#pragma unroll
          for (int i = 0; i < PI; ++i) {
            if (CPT < 4 && c0 >= CPT) break;
            uint32_t q[4], y[8];
            lds<4>(from + i * 512 + lane * 16, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) sc.widen(q[k], y[2 * k], y[2 * k + 1]);
            if (sc.large()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) sc.widen_large(y[2 * k], y[2 * k + 1]);
            }
            const int r = x % GPT * 8 + tok, ch = 2 * (c0 + 4 * i);
            *reinterpret_cast<uint4*>(dst + tc_kv_at<SL>(r, ch)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(dst + tc_kv_at<SL>(r, ch + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B::kv_full + slot));
        }
        cp_async_wait<0>();
        seq0 += 2u * n;
        w.advance();
      }
    }
   } else if (Q8T && warp < Q0) {
    // ============================================================ raw tiles
    // One warp copies K's tiles, the other V's; lane i looks after 8-token group i, whose
    // block is looked up two tiles ahead.  K's warp also brings the tile's exponents, of
    // K and V, a tile ahead (TcCfg::TE).  An entry is written TILES tiles after the one it
    // replaces, whose readers are done: K's tile is at most RS + NS tiles before one whose
    // scores have been read, and the softmax of the tile two before that is over.
    if constexpr (Q8T) {
      constexpr int RS = C::RS;
      static_assert(RS + NS + 3 <= C::TILES, "ring of exponents");
      const bool isv = warp != RAWER;
      const CUtensorMap* map = isv ? &p.tm_v : &p.tm_k;
      const int ring0 = isv ? RS : 0;
      const int per = p.box_tokens / 8;  // groups of a box
      const int bs = p.block_size, step = BN / bs, rest = BN % bs;
      const bool mine = lane < BN / 8;
      uint32_t tile = 0;  // kv tiles so far
      while (ok && w.next(p)) {
        const int n = w.kv1 - w.kv0;
        // the lane's group: position, its place among the row's blocks and in its block, two
        // tiles ahead of the copies
        int t = w.kv0 * BN + lane * 8;
        int j = (int)((unsigned)t / (unsigned)bs), in = t - j * bs;
        const int32_t* row = p.block_tables + (int64_t)w.r * p.max_blocks_per_row;
        auto look_up = [&]() -> int32_t {
          const int32_t b = mine && t < w.g.c ? row[j] : 0;
          t += BN;
          j += step;
          in += rest;
          if (in >= bs) {
            in -= bs;
            ++j;
          }
          return b;
        };
        auto checked = [&](int32_t b) {
          if (b < 0 || b >= p.num_blocks) {
            set_flag(p.err, NP_FLAG_BLOCK_ID);
            b = 0;
          }
          return b;
        };
        auto scale = [&](const float* s, int32_t b) { return __float_as_uint(s[(int64_t)b * p.kv_heads + w.kvh]); };
        int in0 = in;
        int32_t b0 = checked(look_up());
        int in1 = in;
        int32_t b1 = look_up();
        uint32_t ks = 0, vs = 0;
        if (!isv) {
          ks = scale(p.k_scale, b0);
          vs = scale(p.v_scale, b0);
        }
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++tile) {
          const int in2 = in;
          const int32_t b2 = look_up();
          b1 = checked(b1);
          const uint32_t ks0 = ks, vs0 = vs;
          if (!isv) {
            ks = scale(p.k_scale, b1);
            vs = scale(p.v_scale, b1);
          }
          const uint32_t rs = tile % RS + ring0;
          if (tile >= RS) {
            ok = __all_sync(FULL, mbar_wait(bar(B::raw_empty + rs), (tile / RS - 1u) & 1u, abort));
            if (!ok) break;
          }
          const int valid = min(w.g.c - (w.kv0 + i) * BN, BN);  // <= 0: a row without history
          if (!isv) {
            const bool on = mine && lane * 8 < valid;
            const int ke = on ? scale_exp(ks0) : kScaleMin, ve = on ? scale_exp(vs0) : kScaleMin;
            const int kt = __reduce_max_sync(FULL, ke), vt = __reduce_max_sync(FULL, ve);
            const int kd = on ? kt - ke : 0, vd = on ? vt - ve : 0;  // (past the context: masked)
            const bool far = on && (unsigned)(ve + kFar) > 2u * kFar;
            const bool wide = __any_sync(FULL, kd > kWide || vd > kWide || far);
            unsigned char* te = smem + C::EXPS + tile % C::TILES * C::TE;
            if (mine) {
              te[lane] = (unsigned char)(wide ? 0 : kd);
              te[BN / 8 + lane] = (unsigned char)(wide ? 0 : vd);
              if (wide) {
                te[C::TEW + lane] = (unsigned char)kd;
                te[C::TEW + BN / 8 + lane] = (unsigned char)vd;
              }
            }
            if (lane == 0)
              *reinterpret_cast<uint32_t*>(te + C::TEK) = (kt & 0xff) | (vt & 0xff) << 8 | (wide ? 0x10000 : 0);
            __syncwarp();
          }
          const int nbox = valid <= 0 ? 0 : (valid + p.box_tokens - 1) / p.box_tokens;
          if (lane == 0) mbar_arrive_expect_tx(bar(B::raw_full + rs), (uint32_t)(nbox * p.box_tokens * D));
          __syncwarp();
          // (each by the lane of its first group: a loop of elected copies takes twice the time)
          if (mine && lane % per == 0 && lane * 8 < valid)
            tma_load_4d_lane(base + C::RAW_T + rs * (uint32_t)C::RT + (uint32_t)(lane * 8 * D), map,
                             b0 * bs + in0, w.kvh, bar(B::raw_full + rs));
          __syncwarp();
          b0 = b1;
          b1 = b2;
          in0 = in1;
          in1 = in2;
        }
        w.advance();
      }
      if (*abort)  // never leave copies in flight (bounded)
        for (uint32_t q = tile > RS ? tile - RS : 0; q < tile; ++q)
          mbar_wait_drain(bar(B::raw_full + (int)(q % RS) + ring0), (q / RS) & 1u);
    }
   } else if (warp < Q0 + LOADERS) {
    // =============================================================== loads
    // TILED: one warp copies q and the K tiles, another the V tiles (a copy costs
    // its issuing thread tens of cycles, and a tile is up to 16 of them).  Token
    // by token, 64 copies of the whole warp a tile and some 70 cycles each: three
    // warps take the tiles in turn, the first one q too.
    const int id = warp - Q0;
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
          const uint32_t qb = bar(Q8T ? B::q_raw : B::q_full);
          if (lane == 0) mbar_arrive_expect_tx(qb, (uint32_t)(qt * SL * G * p.tile_tokens) * 128u);
          __syncwarp();
          for (int i = 0; i < qt * SL; ++i)
            tma_load_3d_warp(base + (uint32_t)i * 16384u, &p.tm_q, (i % SL) * 64, w.kvh * G,
                             w.g.q0 + (w.m * MT + i / SL) * p.tile_tokens, qb);
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
      if constexpr (Q8) {
      } else if constexpr (TILED) {
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
      if constexpr (!TILED && !Q8) {  // all of it is reported before the next q waits for it
        cp_async_wait<0>();
        if (pending >= 0) report();
        pending = -1;
      }
      w.advance();
    }
    if (*abort) {  // never leave copies in flight (bounded)
      if (D >= 64 && id == 0 && seg > 0) mbar_wait_drain(bar(Q8T ? B::q_raw : B::q_full), (seg - 1) & 1u);
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
    constexpr uint32_t PV = umma_idesc_bf16(128, D, true, false, Q8T);
    constexpr uint32_t QHI = umma_desc_hi(1024), KVHI = umma_desc_hi(SL * 1024);
    const uint32_t QK = umma_idesc_bf16(128, BN, false, p.negate != 0, Q8T);
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

template <int D, int KV>
static np_status launch(const PrefillParams& p, cudaStream_t s) {
  static unsigned long long allowed = 0;
  using C = TcCfg<D, tc_kind(KV)>;
  const np_status rc = allow_smem(prefill_tc_kernel<D, KV>, C::SMEM, &allowed);
  if (rc != NP_OK) return rc;
  return launch_dependent(prefill_tc_kernel<D, KV>, p.ctas, 1, C::THREADS, C::SMEM, s, p);
}

#define NPK_CAT2(a, b) a##b
#define NPK_CAT(a, b) NPK_CAT2(a, b)

#ifdef NPK_Q8
np_status NPK_CAT(prefill_tcq8_d, NPK_D)(const PrefillParams& p, np_form8 form, bool tiled, cudaStream_t s) {
#if NPK_D >= 64
  if (tiled)
    return form == NP_E4M3 ? launch<NPK_D, kQ8Tiled + NP_E4M3>(p, s) : launch<NPK_D, kQ8Tiled + NP_INT8>(p, s);
#endif
  return form == NP_E4M3 ? launch<NPK_D, kQ8 + NP_E4M3>(p, s) : launch<NPK_D, kQ8 + NP_INT8>(p, s);
}
#else
np_status NPK_CAT(prefill_tc_d, NPK_D)(const PrefillParams& p, bool tiled, cudaStream_t s) {
#if NPK_D >= 64
  if (tiled) return launch<NPK_D, kTiled>(p, s);
#endif
  return launch<NPK_D, kTokens>(p, s);
}
#endif

}  // namespace npk
