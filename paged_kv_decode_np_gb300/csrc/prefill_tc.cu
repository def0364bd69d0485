// prefill_tc.cu -- np_paged_prefill for bf16 on the tensor cores (tcgen05),
// compiled once per head_dim (-DNPK_D).
//
// A tile is 128 (token, head) rows of one kv head, token-major: the GQA
// group's heads of one chunk token are neighbouring rows, so one fetch of K
// and V serves G heads and a one-token row fills G rows.  Per kv tile of BN
// tokens and q tile w:
//     S_w = Q_w K^T            tcgen05.mma, both operands in shared memory
//     P_w = 2^(c S_w - m)      fp32 -> bf16, into the tensor memory of S_w
//     O_w += P_w V             tcgen05.mma, A = P_w from tensor memory
// Roles: MT warpgroups of softmax (one thread a row: no shuffles), one warp
// that issues the mma, one that loads.  With two q tiles (head_dim <= 128)
// the tensor cores work on one while the other's softmax runs:
//     ... PV_0(j), S_0(j+1) | PV_1(j), S_1(j+1) ...
// and the two share every K and V tile, 128 operations a byte of it in
// shared memory.  head_dim 256 has tensor memory for one O only (256
// columns): S is double-buffered instead, S(j+1) running under softmax j.
//
// The running maximum is replaced only where it would grow by more than 2^8
// (m need not be the maximum, only near it: p <= 256 keeps its relative
// precision in bf16 and its sum in fp32); then the row's warp rescales O in
// tensor memory itself, which is rare after the first tiles.  P is rounded
// to bf16 for its product with V (half a step of each weight); l sums the
// unrounded p.
//
// K and V land in shared memory as [64-dim slab][token][128 bytes] in the
// 128-byte swizzle, which is both K^T's K-major and V's N-major operand
// layout.  With head_dim a multiple of 64 and block_size a multiple of 8 a
// tiled copy moves box_tokens of a block (TILED); other shapes take 16-byte
// asynchronous copies token by token, swizzled by hand.
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
  static constexpr uint32_t O0 = 256;               // tensor memory column of O_0
  static_assert(NS >= 4, "ring");
};

// Barriers, by index from the barrier area's start (8 bytes each).
template <int D>
struct TcBars {
  static constexpr int NS = TcCfg<D>::NS;
  static constexpr int q_full = 0, q_empty = 1, kv_full = 2, kv_empty = 2 + NS;
  static constexpr int s_full = 2 + 2 * NS, p_full = s_full + 2, o_full = p_full + 2;
  static constexpr int pv_done = o_full + 1;  // MT == 1: one phase a kv tile
  static constexpr int drain = o_full + 2, count = drain + 1;
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int LOADER = 4 * MT, ISSUER = 4 * MT + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < B::count; ++i)
      mbar_init(bar(i), i >= B::p_full && i < B::p_full + 2 ? 4 : 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == ISSUER) tmem_alloc(smem_u32(const_cast<uint32_t*>(tail)), 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tail;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is complete

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
    uint32_t it = 0, oc = 0;
    while (ok && w.next(p)) {
      const int64_t first = ((int64_t)w.m * MT + t) * p.tile_tokens;
      if (first >= w.g.n) {  // no tokens in this tile
        w.advance();
        continue;
      }
      const int n = tc_tiles<D>(p, w, t);
      const int64_t tok = first + tt;
      const bool live = tt < p.tile_tokens && tok < w.g.n;
      // the last position the row sees; rows that are not stored need no mask
      const int lim = live ? (int)((int64_t)w.g.c - w.g.n + tok) : INT_MAX;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t buf = MT == 2 ? (uint32_t)t : (it & 1u);
        const uint32_t phase = MT == 2 ? (it & 1u) : ((it >> 1) & 1u);
        ok = __all_sync(FULL, mbar_wait(bar(B::s_full + buf), phase, abort));
        if (!ok) break;
        tmem_fence_after();
        const uint32_t s_at = lanes + buf * BN;
        uint32_t r[BN];
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld32(s_at + c, r + c);
        tmem_wait_ld();
        tmem_pin<BN>(r);
        float* s = reinterpret_cast<float*>(r);
        const int rel = lim - (w.kv0 + j) * BN;  // last visible column
        if (__any_sync(FULL, rel < BN - 1)) {
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = c <= rel ? s[c] : -INFINITY;
        }
        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
        for (int c = 4; c < BN; c += 4) {
          x0 = fmaxf(x0, s[c]);
          x1 = fmaxf(x1, s[c + 1]);
          x2 = fmaxf(x2, s[c + 2]);
          x3 = fmaxf(x3, s[c + 3]);
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
            if constexpr (MT == 1) {
              ok = __all_sync(FULL, mbar_wait(bar(B::pv_done), (it - 1) & 1u, abort));
              if (!ok) break;
              tmem_fence_after();
            }
#pragma unroll
            for (int c = 0; c < D; c += OC) {
              uint32_t o[OC];
              if constexpr (OC == 32) tmem_ld32(o_at + c, o);
              else tmem_ld16(o_at + c, o);
              tmem_wait_ld();
              tmem_pin<OC>(o);
#pragma unroll
              for (int e = 0; e < OC; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              if constexpr (OC == 32) tmem_st32(o_at + c, o);
              else tmem_st16(o_at + c, o);
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
            float a = s[c + e], b = s[c + e + 1];
            fma2(a, b, p.qscale, ref);
            a = ex2(a);
            b = ex2(b);
            add2(l0, l1, a, b);
            const __nv_bfloat162 hh = __floats2bfloat162_rn(a, b);
            pk[e >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          tmem_st16(s_at + (c >> 1), pk);
        }
        l += l0 + l1;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::p_full + buf));
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(FULL, mbar_wait(bar(B::o_full + t), oc & 1u, abort));
        if (!ok) break;
        ++oc;
        tmem_fence_after();
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
#pragma unroll
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
   if (warp == LOADER) {
    // =============================================================== loads
    RingPos pos{0, 0};
    int issued = 0;       // tiles issued so far (saturates: only 0..NS and "more" matter)
    RingPos told{0, 0};   // token-by-token copies: the next tile to report
    int untold = 0;
    const int G = p.group;
    uint32_t seg = 0;

    // reports the oldest unreported tile: its copies are complete
    auto tell = [&]() {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B::kv_full + told.slot));
      told.template step<NS>();
      --untold;
    };
    // copies K or V of kv tile kt into the ring's next slot
    auto load_tile = [&](bool isv, int kt) {
      if (issued >= NS) {
        ok = __all_sync(FULL, mbar_wait(bar(B::kv_empty + pos.slot), pos.phase ^ 1u, abort));
        if (!ok) return;
      } else {
        ++issued;
      }
      const int t0 = kt * BN;
      const int valid = min(BN, w.g.c - t0);  // <= 0: a row without history
      const uint32_t dst = ring + (uint32_t)pos.slot * C::SLOT;
      const int32_t* table = p.block_tables + (int64_t)w.r * p.max_blocks_per_row;
      if constexpr (TILED) {
        const uint32_t fb = bar(B::kv_full + pos.slot);
        const int bt = p.box_tokens;
        const int nbox = valid > 0 ? (valid + bt - 1) / bt : 0;
        if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(nbox * SL * bt) * 128u);
        __syncwarp();
        for (int i = lane; i < nbox * SL; i += 32) {
          const int box = i / SL, slab = i % SL;
          const unsigned t = (unsigned)(t0 + box * bt);
          const unsigned j = t / (unsigned)p.block_size;
          int64_t b = table[j];
          if (b < 0 || b >= p.num_blocks) {
            set_flag(p.err, NP_FLAG_BLOCK_ID);
            b = 0;
          }
          const int32_t slot = (int32_t)(b * p.block_size + (t - j * p.block_size));
          tma_load_3d_plain(dst + (uint32_t)(slab * BN + box * bt) * 128u, isv ? &p.tm_v : &p.tm_k,
                      slab * 64, slot, w.kvh, fb);
        }
      } else {
        constexpr int CH = D / 8;           // 16-byte pieces of a token
        constexpr int PER = 32 / CH > 0 ? 32 / CH : 1;  // tokens a warp copies at a time
        const char* src = static_cast<const char*>(isv ? p.v_pool : p.k_pool);
        for (int r0 = 0; r0 < valid; r0 += 32) {
          int64_t at = -1;  // element offset of token r0 + lane
          if (r0 + lane < valid) {
            const unsigned t = (unsigned)(t0 + r0 + lane);
            const unsigned j = t / (unsigned)p.block_size;
            int64_t b = table[j];
            if (b < 0 || b >= p.num_blocks) {
              set_flag(p.err, NP_FLAG_BLOCK_ID);
              b = 0;
            }
            at = ((b * p.block_size + (t - j * p.block_size)) * p.kv_heads + w.kvh) * D;
          }
          if constexpr (CH <= 32) {
            const int ch = lane % CH, sub = lane / CH;
#pragma unroll 4
            for (int i = 0; i < 32; i += PER) {
              const int row = r0 + i + sub;
              const int64_t a = __shfl_sync(FULL, at, i + sub);
              if (a >= 0)
                cp_async16(dst + (uint32_t)((ch >> 3) * BN + row) * 128u +
                               (uint32_t)(((ch & 7) ^ (row & 7)) << 4),
                           src + (a + ch * 8) * 2);
            }
          }
        }
        cp_async_commit();
        if (++untold > 2) {
          cp_async_wait<2>();
          tell();
        }
      }
      pos.template step<NS>();
    };

    while (ok && w.next(p)) {
      // ---- q
      if (seg > 0) {
        ok = __all_sync(FULL, mbar_wait(bar(B::q_empty), (seg - 1) & 1u, abort));
        if (!ok) break;
      }
      int qt = 0;
      for (int t = 0; t < MT; ++t)
        if (((int64_t)w.m * MT + t) * p.tile_tokens < w.g.n) ++qt;
      if constexpr (TILED) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B::q_full), (uint32_t)(qt * SL * G * p.tile_tokens) * 128u);
          for (int t = 0; t < qt; ++t)
            for (int s = 0; s < SL; ++s)
              tma_load_3d_plain(base + (uint32_t)(t * SL + s) * 16384u, &p.tm_q, s * 64, w.kvh * G,
                          w.g.q0 + (w.m * MT + t) * p.tile_tokens, bar(B::q_full));
        }
        __syncwarp();
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
      ++seg;
      // ---- K and V tiles in the order the mma takes them
      const int n = w.kv1 - w.kv0;
      if constexpr (MT == 2) {
        for (int j = 0; j < n && ok; ++j) {
          load_tile(false, w.kv0 + j);
          if (ok) load_tile(true, w.kv0 + j);
        }
      } else {
        load_tile(false, w.kv0);
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) load_tile(false, w.kv0 + j + 1);
          if (ok) load_tile(true, w.kv0 + j);
        }
      }
      if constexpr (!TILED) {  // all of it is reported before the next q waits for it
        cp_async_wait<0>();
        while (untold > 0) tell();
      }
      w.advance();
    }
    if (*abort) {  // never leave copies in flight (bounded)
      if constexpr (TILED) {
        if (seg > 0) mbar_wait_drain(bar(B::q_full), (seg - 1) & 1u);
        RingPos d = pos;  // the tile before pos, and back
        for (int i = 0; i < NS && i < issued; ++i) {
          if (--d.slot < 0) {
            d.slot = NS - 1;
            d.phase ^= 1u;
          }
          mbar_wait_drain(bar(B::kv_full + d.slot), d.phase);
        }
      } else {
        cp_async_wait<0>();
      }
    }
   } else if (warp == ISSUER) {
    // ================================================================= mma
    constexpr uint32_t PV = umma_idesc_bf16(128, D, true);
    const uint32_t QK = umma_idesc_bf16(128, BN, false, p.negate != 0);
    RingPos pos{0, 0};
    uint32_t seg = 0;
    uint32_t done[2] = {0u, 0u};  // tiles of each S buffer so far: phase of p_full
    uint32_t it = 0;              // MT == 1: tiles so far

    auto wait = [&](int b, uint32_t phase) {
      ok = ok && __all_sync(FULL, mbar_wait(bar(b), phase, abort));
      return ok;
    };
    auto issue_s = [&](int t, int buf, uint32_t k) {  // S_buf = Q_t K^T
      if (lane == 0) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t q = base + (uint32_t)t * C::QT + (ks >> 2) * 16384u + (ks & 3) * 32u;
          const uint32_t kk = k + (uint32_t)(ks >> 2) * (BN * 128u) + (ks & 3) * 32u;
          umma_ss(tmem + buf * BN, umma_desc(q, 16, 1024), umma_desc(kk, 16, 1024), QK, ks > 0);
        }
        umma_commit(bar(B::s_full + buf));
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int buf, uint32_t v, bool acc) {  // O_t += P_buf V
      tmem_fence_after();
      if (lane == 0) {
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks)
          umma_ts(tmem + C::O0 + t * D, tmem + buf * BN + ks * 8,
                  umma_desc(v + ks * 2048u, BN * 128, 1024), PV, acc || ks > 0);
      }
      __syncwarp();
    };
    // V rows past the context are whatever their slots held: zeroed, for 0 x
    // NaN is NaN
    auto clear_tail = [&](uint32_t v, int kt) {
      const int valid = max(0, min(BN, w.g.c - kt * BN));
      if (valid == BN) return;
      unsigned char* at = smem + (v - base);
      for (int e = lane; e < SL * (BN - valid) * 8; e += 32) {
        const int slab = e / ((BN - valid) * 8), x = e % ((BN - valid) * 8);
        *reinterpret_cast<uint4*>(at + (slab * BN + valid) * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      __syncwarp();
    };

    while (ok && w.next(p)) {
      const int n = w.kv1 - w.kv0;
      if (!wait(B::q_full, seg & 1u)) break;
      ++seg;
      if constexpr (MT == 2) {
        const int n0 = tc_tiles<D>(p, w, 0), n1 = tc_tiles<D>(p, w, 1);
        // n == max(n0, n1): the unit's last tokens see the most
        uint32_t kaddr = ring + (uint32_t)pos.slot * C::SLOT;
        int kslot = pos.slot;
        if (!wait(B::kv_full + kslot, pos.phase)) break;
        pos.template step<NS>();
        if (n0 > 0) issue_s(0, 0, kaddr);
        if (n1 > 0) issue_s(1, 1, kaddr);
        if (lane == 0) {
          umma_commit(bar(B::kv_empty + kslot));
          if (n == 1) umma_commit(bar(B::q_empty));
        }
        for (int j = 0; j < n && ok; ++j) {
          const int vslot = pos.slot;
          const uint32_t vphase = pos.phase;
          const uint32_t vaddr = ring + (uint32_t)vslot * C::SLOT;
          pos.template step<NS>();
          bool have_v = false, have_k = false;
          kslot = pos.slot;
          kaddr = ring + (uint32_t)kslot * C::SLOT;
          const uint32_t kphase = pos.phase;
          if (j + 1 < n) pos.template step<NS>();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t == 0 ? n0 : n1;
            if (j >= nt) continue;
            if (!wait(B::p_full + t, done[t] & 1u)) break;
            ++done[t];
            if (!have_v) {
              if (!wait(B::kv_full + vslot, vphase)) break;
              clear_tail(vaddr, w.kv0 + j);
              have_v = true;
            }
            issue_pv(t, t, vaddr, j > 0);
            // the last tile that reads this V frees it
            if (lane == 0 && (t == 1 || j >= n1)) umma_commit(bar(B::kv_empty + vslot));
            if (j + 1 < nt) {
              if (!have_k) {
                if (!wait(B::kv_full + kslot, kphase)) break;
                have_k = true;
              }
              issue_s(t, t, kaddr);
              if (lane == 0 && (t == 1 || j + 1 >= n1)) {
                umma_commit(bar(B::kv_empty + kslot));
                if (j + 2 == n) umma_commit(bar(B::q_empty));
              }
            } else if (lane == 0) {
              umma_commit(bar(B::o_full + t));
            }
            __syncwarp();
          }
        }
      } else {
        const uint32_t first = it;
        for (int j = -1; j < n && ok; ++j) {
          if (j + 1 < n) {  // S(j + 1)
            const int slot = pos.slot;
            if (!wait(B::kv_full + slot, pos.phase)) break;
            pos.template step<NS>();
            issue_s(0, (first + j + 1) & 1u, ring + (uint32_t)slot * C::SLOT);
            if (lane == 0) {
              umma_commit(bar(B::kv_empty + slot));
              if (j + 2 == n) umma_commit(bar(B::q_empty));
            }
          }
          if (j >= 0) {  // O += P(j) V(j)
            const uint32_t buf = it & 1u;
            const int slot = pos.slot;
            const uint32_t phase = pos.phase;
            pos.template step<NS>();
            if (!wait(B::p_full + buf, (it >> 1) & 1u)) break;
            if (!wait(B::kv_full + slot, phase)) break;
            ++it;
            clear_tail(ring + (uint32_t)slot * C::SLOT, w.kv0 + j);
            issue_pv(0, buf, ring + (uint32_t)slot * C::SLOT, j > 0);
            if (lane == 0) {
              umma_commit(bar(B::pv_done));
              umma_commit(bar(B::kv_empty + slot));
              if (j + 1 == n) umma_commit(bar(B::o_full));
            }
          }
        }
      }
      w.advance();
    }
    // nothing of this block is left running in the tensor cores (bounded)
    if (lane == 0) {
      umma_commit(bar(B::drain));
      mbar_wait_drain(bar(B::drain), 0u);
    }
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
  if (cudaFuncSetAttribute(prefill_tc_kernel<D, TILED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           TcCfg<D>::SMEM) != cudaSuccess)
    return NP_ERR_CUDA;
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
