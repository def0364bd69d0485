// prefill_tc32.cu -- np_paged_prefill for fp32 pools on the bf16 tensor cores,
// head_dim 16 to 128, compiled once per head_dim (-DNPK_D).
//
// An fp32 number is the sum of three bf16 numbers, exactly: its first 8
// significant bits, the next 8, the last 8 (each cut off, not rounded, so the
// remainders are exact; sums never overflow).  A product of two such sums is
// nine bf16 products, exact in fp32; the three smallest (below 2^-22 of the
// whole) are left out:
//     a b = a0 b0 + (a0 b1 + a1 b0) + (a1 b1 + a0 b2 + a2 b0)
// so S = Q K^T and O = P V are six tensor-core products each, added in fp32,
// the small ones first (an accumulator's rounding is relative to what it
// holds).  Six times the work of bf16 is still several times the rate of the
// FMA pipes.  O is accumulated over the kv tiles in
// registers: a tile's P V is 24 steps of the tensor cores' accumulator, and
// the sum over a long history is rounded to nearest.
//
// A unit is one tile of 128 (token, head) rows; a kv tile is 64 tokens.  Roles:
//   4 warps of softmax (one thread a row): q in three parts to tensor memory,
//     S from there, P in three parts back to it, O of the tile before added up;
//   4 warps that copy K, 4 that copy V: fp32 from global memory to registers
//     half a tile ahead, split, to shared memory in the mma's layout;
//   1 warp that issues:  S(j+1), P V(j), S(j+2), P V(j+1) ...
// A 128 x 64 mma takes as long as a 128 x 128 one, so S has 128 columns: a kv
// tile's parts lie one after the other, and q_i times [K_0; K_1] gives q_i K_0 in
// the first 64 columns and q_i K_1 in the others (q_2 K_1 comes for nothing);
// q_0 K_2 joins the latter, and the softmax adds the two.  Four mma a 16-dim
// step instead of six.  Successive mma run in order only where they share their
// accumulator and their shape, and q_0 K_2 is 64 wide over half of the columns:
// it is issued once the others are complete (their own commit), and the next
// tile's first mma once the softmax has read these (s_empty).  P and q's first two parts are A operands in tensor
// memory, which has no room for q's third: that one is in shared memory.
//
// Bound: the softmax warps, one a scheduler (~5400 cycles of work in ~6600 a kv
// tile), and behind them the mma (56 of them, 64 cycles each, and ~420 for the
// wait between the shapes: ~4000).  Eight chunks of 71-184 tokens over 833-2031
// positions, 32 / 8 heads of 128: 167 us, 143 TFLOP/s of fp32 products (950 us on
// the FMA pipes); without the wait 162; with all products 64 columns wide, no
// wait and half the adding up, 173.  Error against exact values 3e-7 of their norm.
//
// An 8-bit cache (FORM, compiled apart): a code times its scale, a power of two, is
// one bf16 number, so K and V are their first part alone: q's three parts times K into
// one S of 64 columns, P's three parts times V, exact products all of them.  Eight chunks of
// 64-192 tokens over 512-2048 positions: 118 us (954 on the FMA pipes), 2.5e-7 off.
#include <limits.h>

#include <type_traits>

#include "cache8.cuh"
#include "prefill.cuh"
#include "tcgen05.cuh"

#ifndef NPK_D
#error "compiled per head_dim"
#endif

namespace npk {

template <int D>
struct Tc32Cfg {
  static constexpr int SL = D > 64 ? D / 64 : 1;  // 64-dim slabs
  static constexpr int BN = 64;
  static constexpr int PART = SL * BN * 128;      // bytes of a K or V part
  static constexpr int NS = D == 128 ? 2 : 4;     // K tiles, V tiles in shared memory
  static constexpr int K0 = SL * 128 * 128;       // after q's third part
  static constexpr int V0 = K0 + NS * 3 * PART;
  static constexpr int BARS = V0 + NS * 3 * PART;
  static constexpr int SMEM = 1024 + BARS + 256;
  static constexpr int THREADS = 512;
  // tensor memory: S (128 columns), P (three parts of 32), q (two of D / 2), O
  static constexpr uint32_t P0 = 128, Q0 = 224, O0 = 384;
  static_assert(SMEM <= 227 * 1024 && Q0 + D <= O0, "shared and tensor memory");
  static_assert(2 * (SMEM + 1024) > 228 * 1024, "one block an SM");
};

struct Tc32Bars {
  static constexpr int k_full = 0, k_empty = 4, v_full = 8, v_empty = 12;  // of NS <= 4 slots
  static constexpr int q_full = 16, s_full = 17, s_empty = 18, p_full = 19, pv_done = 20;
  static constexpr int s_part = 21;  // the products with [K_0; K_1] are complete
  static constexpr int drain = 22, count = 23;
};

// The parts of a product, the small ones first: (a part, b part).
__device__ constexpr int kPartA[6] = {0, 2, 1, 0, 1, 0};
__device__ constexpr int kPartB[6] = {2, 0, 1, 1, 0, 0};

// x = y0 + y1 + y2, bf16 numbers in the upper halves
__device__ __forceinline__ void split3(float x, uint32_t& y0, uint32_t& y1, uint32_t& y2) {
  y0 = __float_as_uint(x) & 0xffff0000u;
  const float r = x - __uint_as_float(y0);
  y1 = __float_as_uint(r) & 0xffff0000u;
  y2 = __float_as_uint(r - __uint_as_float(y1));  // 8 bits are left: its lower half is zero
}

__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
  return __byte_perm(lo, hi, 0x7632);
}

// 8 fp32 values to 16 bytes of each part
__device__ __forceinline__ void split8(const float4& a, const float4& b, uint4 (&o)[3]) {
  const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t y[8][3], w[3][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(x[i], y[i][0], y[i][1], y[i][2]);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[k][i] = upper_halves(y[2 * i][k], y[2 * i + 1][k]);
    o[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
  }
}

// FORM: the pools' 8-bit form, or -1 for fp32
template <int D, int FORM>
__global__ void __launch_bounds__(Tc32Cfg<D>::THREADS, 1)
    prefill_tc32_kernel(const __grid_constant__ PrefillParams p) {
  using C = Tc32Cfg<D>;
  using B = Tc32Bars;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int BN = C::BN, SL = C::SL, NS = C::NS;
  constexpr bool Q8 = FORM >= 0;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t bars = base + C::BARS;
  auto bar = [&](int i) { return bars + 8u * i; };
  volatile uint32_t* tail = reinterpret_cast<volatile uint32_t*>(smem + C::BARS + 8 * B::count);
  volatile int* abort = reinterpret_cast<volatile int*>(tail + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int ISSUER = 12;  // warps 0-3 softmax, 4-7 K, 8-11 V

  if (threadIdx.x == 0) {
    for (int i = 0; i < B::count; ++i) {
      const bool warps4 = (i >= B::k_full && i < B::k_empty) || (i >= B::v_full && i < B::v_empty) ||
                          i == B::q_full || i == B::s_empty || i == B::p_full;
      mbar_init(bar(i), warps4 ? 4 : 1);
    }
    *abort = 0;
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
  auto wait = [&](int b, uint32_t phase) {
    ok = ok && __all_sync(FULL, mbar_wait(bar(b), phase, abort));
    return ok;
  };

  // Registers: 512 threads have 128 each at launch; 240 + 2 x 96 + 80 = 4 x 128.
  if (warp < 4) {
    // ============================================================= softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    w.start(p, blockIdx.x);
    const int row = warp * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const int tt = row / p.group, h = row - tt * p.group;
    uint32_t it = 0;  // kv tiles so far
    while (ok && w.next(p)) {
      const int n = w.kv1 - w.kv0;
      const int64_t tok = (int64_t)w.m * p.tile_tokens + tt;
      const bool live = tt < p.tile_tokens && tok < w.g.n;
      const bool idle = !__any_sync(FULL, live);  // none of the warp's rows is stored
      const int lim = live ? (int)((int64_t)w.g.c - w.g.n + tok) : INT_MAX;
      // ---- q of the row, zeros without a token.  The last segment's S are
      // complete (this warp has waited for each), so its q may go.
      float acc[D];
      if (!idle) {
        const float* q = static_cast<const float*>(p.q) +
                         ((w.g.q0 + tok) * p.q_heads + (int64_t)w.kvh * p.group + h) * D;
#pragma unroll
        for (int c = 0; c < D; c += 4) {  // the whole row in flight
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (live) x = *reinterpret_cast<const float4*>(q + c);
          acc[c] = x.x;
          acc[c + 1] = x.y;
          acc[c + 2] = x.z;
          acc[c + 3] = x.w;
        }
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t k[3][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t x[3], y[3];
            split3(acc[c + 2 * e], x[0], x[1], x[2]);
            split3(acc[c + 2 * e + 1], y[0], y[1], y[2]);
#pragma unroll
            for (int i = 0; i < 3; ++i) k[i][e] = upper_halves(x[i], y[i]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_st8(lanes + C::Q0 + i * (D / 2) + (c >> 1), k[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i)  // the third part: 16-byte pieces c / 8 + i
            *reinterpret_cast<uint4*>(smem + (c >> 6) * 16384 + row * 128 +
                                      ((((c >> 3) + i) & 7) ^ (row & 7)) * 16) =
                make_uint4(k[2][4 * i], k[2][4 * i + 1], k[2][4 * i + 2], k[2][4 * i + 3]);
        }
        tmem_wait_st();
        tmem_fence_before();
        fence_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar(B::q_full));

      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int c = 0; c < D; ++c) acc[c] = 0.f;
      // acc = (acc + O of the tile before) * f
      auto add_o = [&](float f) {
        constexpr int OC = D < 32 ? 16 : (D < 64 ? 32 : 64);  // columns at a time
#pragma unroll
        for (int c = 0; c < D; c += OC) {
          uint32_t o[OC];
          if constexpr (OC == 16) {
            tmem_ld16(lanes + C::O0 + c, o);
          } else {
#pragma unroll
            for (int e = 0; e < OC; e += 32) tmem_ld32(lanes + C::O0 + c + e, o + e);
          }
          tmem_wait_ld();
          tmem_pin<OC>(o);
#pragma unroll
          for (int e = 0; e < OC; ++e) acc[c + e] = (acc[c + e] + __uint_as_float(o[e])) * f;
        }
      };
      for (int j = 0; j < n; ++j, ++it) {
        if (!wait(B::s_full, it & 1u)) break;
        tmem_fence_after();
        if (idle) {  // P of these rows is whatever tensor memory holds: it moves their own O only
          if (lane == 0) mbar_arrive(bar(B::s_empty));
          if (j > 0 && !wait(B::pv_done, (it - 1) & 1u)) break;
          if (lane == 0) mbar_arrive(bar(B::p_full));
          continue;
        }
        uint32_t r[BN];
        tmem_ld32(lanes, r);  // q K_0 of all parts; q K_1 and q K_2 are BN columns on
        tmem_ld32(lanes + 32, r + 32);
        tmem_wait_ld();
        tmem_pin<BN>(r);
        if constexpr (!Q8) {
#pragma unroll
          for (int c = 0; c < BN; c += 32) {
            uint32_t y[32];
            tmem_ld32(lanes + BN + c, y);
            tmem_wait_ld();
            tmem_pin<32>(y);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              r[c + e] = __float_as_uint(__uint_as_float(r[c + e]) + __uint_as_float(y[e]));
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::s_empty));
        const int rel = lim - (w.kv0 + j) * BN;  // last visible column
        if (__any_sync(FULL, rel < BN - 1)) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (c > rel) r[c] = 0xff800000u;  // -inf
        }
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < BN; c += 4) {
          x0 = fmaxf(fmaxf(x0, __uint_as_float(r[c])), __uint_as_float(r[c + 1]));
          x1 = fmaxf(fmaxf(x1, __uint_as_float(r[c + 2])), __uint_as_float(r[c + 3]));
        }
        const float mn = fmaxf(m, fmaxf(x0, x1) * p.qscale);
        const float ref = mn == -INFINITY ? 0.f : -mn;
        const float f = ex2(m + ref);
        m = mn;
        float l0 = 0.f, l1 = 0.f;
#pragma unroll
        for (int c = 0; c < BN; c += 2) {
          const float a = ex2(fmaf(__uint_as_float(r[c]), p.qscale, ref));
          const float b = ex2(fmaf(__uint_as_float(r[c + 1]), p.qscale, ref));
          l0 += a;
          l1 += b;
          r[c] = __float_as_uint(a);
          r[c + 1] = __float_as_uint(b);
        }
        l = fmaf(l, f, l0 + l1);
        if (j > 0) {  // P V of the tile before is complete: P may go, O is there
          if (!wait(B::pv_done, (it - 1) & 1u)) break;
          tmem_fence_after();
        }
#pragma unroll
        for (int c = 0; c < BN; c += 16) {  // 16 weights: 8 columns of each part
          uint32_t k[3][8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t a[3], b[3];
            split3(__uint_as_float(r[c + 2 * e]), a[0], a[1], a[2]);
            split3(__uint_as_float(r[c + 2 * e + 1]), b[0], b[1], b[2]);
#pragma unroll
            for (int i = 0; i < 3; ++i) k[i][e] = upper_halves(a[i], b[i]);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) tmem_st8(lanes + C::P0 + i * 32 + (c >> 1), k[i]);
        }
        if (j > 0) add_o(f);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B::p_full));
      }
      if (!wait(B::pv_done, (it - 1) & 1u)) break;
      tmem_fence_after();
      if (!idle) {
        add_o(1.f);
        // ---- the row's result: out, or this block's partial of a cut unit
        if (w.whole()) {
          if (live) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            float* out = static_cast<float*>(p.out) +
                         ((w.g.q0 + tok) * p.q_heads + (int64_t)w.kvh * p.group + h) * D;
#pragma unroll
            for (int c = 0; c < D; c += 4)
              *reinterpret_cast<float4*>(out + c) =
                  make_float4(acc[c] * inv, acc[c + 1] * inv, acc[c + 2] * inv, acc[c + 3] * inv);
          }
        } else {
          float* part =
              p.parts + (size_t)(2 * blockIdx.x + (w.kv0 > 0 ? 0 : 1)) * prefill_part_floats(128, D);
          part[row] = m;
          part[128 + row] = l;
#pragma unroll
          for (int c = 0; c < D; c += 4)
            *reinterpret_cast<float4*>(part + 256 + ((size_t)(c / 4) * 128 + row) * 4) =
                make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        }
      }
      tmem_fence_before();  // O is read before the next unit's first P is reported
      w.advance();
    }
  } else if (warp < ISSUER) {
    // =============================================================== loads
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    w.start(p, blockIdx.x);
    const bool isv = warp >= 8;
    const int wl = warp & 3;                 // warp of its group of four
    constexpr int PT = D / 8;                // 8-dim pieces of a token
    constexpr int TW = 32 / PT;              // tokens a warp takes at a time
    constexpr int NP = PT / 2;               // times: 16 tokens of the 64 are a warp's
    constexpr int HP = NP > 1 ? NP / 2 : 1;  // as many times at once: half a tile
    const int piece = lane % PT, sub = lane / PT;
    using E = typename std::conditional<Q8, uint8_t, float>::type;
    const E* pool = static_cast<const E*>(isv ? p.v_pool : p.k_pool);
    const float* scales = isv ? p.v_scale : p.k_scale;
    const int64_t token = (int64_t)p.kv_heads * D;
    const int full = isv ? B::v_full : B::k_full, empty = isv ? B::v_empty : B::k_empty;
    uint32_t it = 0;
    float4 x[HP][2];   // fp32: the pieces; 8 bits: codes and exponent of each
    uint2 codes[HP];
    int exps[HP];
    struct Token {     // lane i: element offset of the warp's token i, -1 past the context; its scale
      int64_t at;
      uint32_t scale;
    };
    // token i of the warp's 16 (i = pass * TW + sub) is row pass * 4 TW + wl TW + sub
    auto row_of = [&](int pass, int s) { return (pass * 4 + wl) * TW + s; };
    auto look_up = [&](int kt) {  // of kv tile kt
      Token k{-1, 0u};
      if (lane < 16) {
        const int64_t t = (int64_t)kt * BN + row_of(lane / TW, lane % TW);
        if (t < w.g.c) {
          const unsigned j = (unsigned)t / (unsigned)p.block_size;
          int64_t b = p.block_tables[(int64_t)w.r * p.max_blocks_per_row + j];
          if (b < 0 || b >= p.num_blocks) {
            set_flag(p.err, NP_FLAG_BLOCK_ID);
            b = 0;
          }
          k.at = (b * p.block_size + ((unsigned)t - j * p.block_size)) * token + (int64_t)w.kvh * D;
          if constexpr (Q8) k.scale = __float_as_uint(scales[b * p.kv_heads + w.kvh]);
        }
      }
      return k;
    };
    auto fetch = [&](const Token& k, int first) {  // passes first .. first + HP - 1; zeros past the context
#pragma unroll
      for (int i = 0; i < HP; ++i) {
        const int64_t a = __shfl_sync(FULL, k.at, (first + i) * TW + sub);
        if constexpr (Q8) {
          exps[i] = scale_exp(__shfl_sync(FULL, k.scale, (first + i) * TW + sub));
          codes[i] = a >= 0 ? *reinterpret_cast<const uint2*>(pool + a + piece * 8) : make_uint2(0u, 0u);
          continue;
        }
        x[i][0] = x[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a >= 0) {
          const float4* src = reinterpret_cast<const float4*>(pool + a + piece * 8);
          x[i][0] = src[0];
          x[i][1] = src[1];
        }
      }
    };
    // brings this warp's tokens of a tile into L2: the registers hold half a tile
    // ahead, too little for HBM's latency.  Lines of 128 bytes, two a lane.
    auto prefetch = [&](const Token& k) {
      constexpr int LE = 128 / (int)sizeof(E);              // elements of a line
      constexpr int LINES = D / LE > 0 ? D / LE : 1;        // of a token
#pragma unroll
      for (int i = 0; i < (16 * LINES + 31) / 32; ++i) {
        const int x = i * 32 + lane;
        const int64_t a = __shfl_sync(FULL, k.at, (x / LINES) & 15);
        if (x < 16 * LINES && a >= 0)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(pool + a + (x % LINES) * LE));
      }
    };
    while (ok && w.next(p)) {
      const int n = w.kv1 - w.kv0;
      Token at = look_up(w.kv0);
      Token ahead = n > 1 ? look_up(w.kv0 + 1) : Token{-1, 0u};
      fetch(at, 0);
      if (n > 1) prefetch(ahead);
      for (int j = 0; j < n; ++j, ++it) {
        const uint32_t slot = it % NS, use = it / NS;
        const Token ahead2 = j + 2 < n ? look_up(w.kv0 + j + 2) : Token{-1, 0u};
        if (use > 0 && !wait(empty + slot, (use - 1) & 1u)) break;
        unsigned char* dst = smem + (isv ? C::V0 : C::K0) + slot * (3 * C::PART);
#pragma unroll 1
        for (int first = 0; first < NP; first += HP) {
#pragma unroll
          for (int i = 0; i < HP; ++i) {
            unsigned char* d = dst + tc_kv_at<SL>(row_of(first + i, sub), piece);
            if constexpr (Q8) {
              const Scaled8<FORM> sc(exps[i]);
              uint4 o;
              sc.widen(codes[i].x, o.x, o.y);
              sc.widen(codes[i].y, o.z, o.w);
              if (sc.large()) {
                sc.widen_large(o.x, o.y);
                sc.widen_large(o.z, o.w);
              }
              *reinterpret_cast<uint4*>(d) = o;
            } else {
              uint4 o[3];
              split8(x[i][0], x[i][1], o);
#pragma unroll
              for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(d + k * C::PART) = o[k];
            }
          }
          if (first + HP < NP) fetch(at, first + HP);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(full + slot));
        at = ahead;
        ahead = ahead2;
        if (j + 1 < n) fetch(at, 0);
        if (j + 2 < n) prefetch(ahead);
      }
      w.advance();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    w.start(p, blockIdx.x);
    if (warp == ISSUER) {
      // =============================================================== mma
      // The whole warp runs the role, its lanes alike; one of them issues.
      constexpr uint32_t PV = umma_idesc_bf16(128, D, true);
      constexpr uint32_t QHI = umma_desc_hi(1024), KVHI = umma_desc_hi(SL * 1024);
      const uint32_t QK1 = umma_idesc_bf16(128, BN, false, p.negate != 0);      // one part of K
      const uint32_t QK2 = umma_idesc_bf16(128, 2 * BN, false, p.negate != 0);  // two
      uint32_t it = 0, seg = 0;  // kv tiles whose P V is issued; segments
      while (ok && w.next(p)) {
        const int n = w.kv1 - w.kv0;
        if (!wait(B::q_full, seg & 1u)) break;
        ++seg;
        for (int j = -1; j < n; ++j) {
          if (j + 1 < n) {  // S(j + 1), once S(j) has been read
            const uint32_t t = it + (j < 0 ? 0u : 1u), slot = t % NS;
            if (!wait(B::k_full + slot, (t / NS) & 1u)) break;
            if (t > 0 && !wait(B::s_empty, (t - 1u) & 1u)) break;
            tmem_fence_after();
            const uint32_t k = umma_desc_lo(base + C::K0 + slot * (3 * C::PART), 16);
            const uint32_t q2 = umma_desc_lo(base, 16);
            // 16 dims of K parts from `part` on
            auto kd = [&](int part, int ks) {
              return k + (uint32_t)(part * C::PART + (ks >> 2) * 1024 + (ks & 3) * 32) / 16;
            };
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)  // q2 [K0; K1]  (8 bits: K0)
              umma_ss(tmem, q2 + ((ks >> 2) * 16384 + (ks & 3) * 32) / 16, QHI, kd(0, ks), KVHI,
                      Q8 ? QK1 : QK2, ks > 0);
#pragma unroll
            for (int i = 1; i >= 0; --i)  // q1 [K0; K1], q0 [K0; K1]
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)
                umma_ts(tmem, tmem + C::Q0 + i * (D / 2) + ks * 8, kd(0, ks), KVHI, Q8 ? QK1 : QK2, 1);
            if constexpr (!Q8) {
              umma_commit(bar(B::s_part));  // another shape follows on their columns
              if (!wait(B::s_part, t & 1u)) break;
              tmem_fence_after();
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks)  // q0 K2
                umma_ts(tmem + BN, tmem + C::Q0 + ks * 8, kd(2, ks), KVHI, QK1, 1);
            }
            umma_commit(bar(B::s_full));
            umma_commit(bar(B::k_empty + slot));
          }
          if (j >= 0) {  // O = P(j) V(j)
            const uint32_t slot = it % NS;
            if (!wait(B::p_full, it & 1u) || !wait(B::v_full + slot, (it / NS) & 1u)) break;
            tmem_fence_after();
            const uint32_t v = umma_desc_lo(base + C::V0 + slot * (3 * C::PART), 1024);
#pragma unroll
            for (int x = 0; x < (Q8 ? 3 : 6); ++x)
#pragma unroll
              for (int ks = 0; ks < BN / 16; ++ks)
                umma_ts(tmem + C::O0, tmem + C::P0 + (Q8 ? 2 - x : kPartA[x]) * 32 + ks * 8,
                        v + ((Q8 ? 0 : kPartB[x]) * C::PART + ks * (2 * SL * 1024)) / 16, KVHI, PV,
                        x > 0 || ks > 0);
            umma_commit(bar(B::pv_done));
            umma_commit(bar(B::v_empty + slot));
            ++it;
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

#define NPK_CAT2(a, b) a##b
#define NPK_CAT(a, b) NPK_CAT2(a, b)

template <int FORM>
static np_status launch(const PrefillParams& p, cudaStream_t s) {
  constexpr int bytes = Tc32Cfg<NPK_D>::SMEM;
  static unsigned long long allowed = 0;
  const np_status rc = allow_smem(prefill_tc32_kernel<NPK_D, FORM>, bytes, &allowed);
  if (rc != NP_OK) return rc;
  return launch_dependent(prefill_tc32_kernel<NPK_D, FORM>, p.ctas, 1, Tc32Cfg<NPK_D>::THREADS, bytes, s,
                          p);
}

#ifdef NPK_Q8
np_status NPK_CAT(prefill_tc32q8_d, NPK_D)(const PrefillParams& p, np_form8 form, cudaStream_t s) {
  return form == NP_E4M3 ? launch<NP_E4M3>(p, s) : launch<NP_INT8>(p, s);
}
#else
np_status NPK_CAT(prefill_tc32_d, NPK_D)(const PrefillParams& p, cudaStream_t s) { return launch<-1>(p, s); }
#endif

}  // namespace npk
