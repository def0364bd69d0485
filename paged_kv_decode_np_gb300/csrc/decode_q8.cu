// decode_q8.cu -- np_paged_decode_q8: the decode read of an 8-bit cache, compiled
// once per head_dim and form (-DNPK_D, -DNPK_FORM).
//
// Per row, kv head and its MR = G Q (query token, head) rows, with codes k, v and
// exponents a, b of their scales:
//     y_j = c (q . k_j) 2^a_j - M                  (log2 units; c = scale log2 e)
//     O  = sum_j 2^(y_j + b_j) v_j,   l = sum_j 2^y_j,   out = O / l
// so V's scale is a power of two at the weight, and its product stays a product
// of codes.  M is a whole number, the largest y + M + b rounded up, and replaced only where
// one passes it by more than 8; y then has one rounding, and M's changes are exact powers
// of two.  Weights are taken 2^6 larger: they stay within fp16's 2^15, and what is too small
// for its subnormals is below 2^-30 of the largest.  The exponential is l's term and the
// weight its product with 2^(b + 6), not the other way round: M is at most 60 above the
// largest score and 2^y leaves fp32's range only below 2^-66 of the largest term of l, while
// 2^(y + b) may be 2^-120 of O's largest where V's scales lie that far apart.
//
// The products are m16n8k16 mma (fp16 in, fp32 out) with the cache as the A
// operand -- 16 tokens x 16 dims of K, 16 dims x 16 tokens of V -- and the rows
// as B's 8 columns, so that a code is widened once for 8 rows.  Codes are exact
// in fp16; q is scaled by a power of two; fp32 q and weights take two fp16
// parts each, two mma to a sum.  S comes out with a lane's values on tokens
// lane/4, lane/4 + 8 and rows 2 (lane%4), + 1; movmatrix turns it into B of the
// second product.
//
// A warp is a reader of its own: it owns a ring of stages in shared memory, a
// stage holding the K, V and scales of CT tokens of one kv head, filled by its own
// 16-byte asynchronous copies (which zero what lies past the context) and waited for
// by nobody else.  No barrier is on the way but the join of a head's warps at a
// row's end.  A block's HG kv heads have WPH warps each, which take the block's
// chunks of CT tokens in turn.
//
// The work: rows (times groups of HG kv heads) laid end to end in chunks, an
// equal share per block, one block an SM, from the context lengths on the device.
// A row inside one block is stored directly; one that is cut leaves partials
// that a second launch joins in block order.
//
// Bound: HBM on long rows (16 rows of 32768-131072 positions, 64 / 8 heads: 458 us, 6.8
// TB/s).  Shorter ones pay what runs once: about 5 us until the first chunk is there, 3 at
// each row's end, 6 for the join (64 rows of 1024-8192: 100 us, 82 at the copy rate; 8 fp32
// rows of 512-2048: 20, latency throughout).  More than eight rows a head take two column
// tiles, whose sums leave registers for eight warps only: 4 query tokens of 4 heads, int8,
// 125 us against 86; the issue slots are half used and each warp waits for its own
// products.  Why warps that read for themselves: the loop's copies, widening and products
// overlap across 16 warps without a barrier, and a stage is 4 KB, so that three of them a
// warp keep 130 KB an SM on the way.  Measured against: table look-ups in line with the copies
// and each row of a segment's end by itself 110 us (64 rows); copies of chunks inside one
// block in a branch of their own 159 us for 146 (4 tokens: the branch keeps the copies from
// being scheduled among the products); join with one block an SM 137 us for 125.
#include <type_traits>

#include "cache8.cuh"
#include "decode_q8.cuh"
#include "tcgen05.cuh"  // cp_async_*

#ifndef NPK_D
#error "compiled per head_dim and form"
#endif

namespace npk {

constexpr float kAbove = 8.f;
constexpr int kWeightExp = 6;


// Geometry of a stage.  Rows of D bytes; 128-byte lines; 16-byte pieces of a line are
// swizzled so that both products' reads are free of bank conflicts.
template <int D, int NT>
struct Q8Geo {
  static constexpr int WARPS = q8_warps(D, NT);
  static constexpr int CT = 16 * NT;              // tokens of a stage
  static constexpr int MR = 8 * NT;               // rows of the exchange at a row's end
  static constexpr int LD = D + 4;                // floats of an exchanged O row
  static constexpr int DATA = 2 * CT * D + 8 * CT;
  static constexpr int SWAP = (MR * LD + 2 * MR) * 4;
  static constexpr int STAGE = ((DATA > SWAP ? DATA : SWAP) + 127) / 128 * 128;
  static constexpr int FIT = 224 * 1024 / (WARPS * STAGE);
  static constexpr int NS = FIT < 8 ? FIT : 8;    // stages of a warp's ring
  static constexpr int SMEM = WARPS * NS * STAGE;
  static_assert(NS >= 3, "ring");
  // byte of piece `ch` of row `r`
  __device__ __forceinline__ static uint32_t at(int r, int ch) {
    if constexpr (D >= 128) return (uint32_t)(r * D + ((ch ^ (r & 7)) << 4));
    else if constexpr (D == 16) return (uint32_t)(r << 4);
    else {
      constexpr int PL = 128 / D, PP = D / 16;  // rows of a line, pieces of a row
      const int line = r / PL, c = (r % PL) * PP + ch;
      return (uint32_t)(line * 128 + ((c ^ (2 * (line & 3))) << 4));
    }
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the same without a sum before it
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// the part of (lo, hi) that `packed` leaves
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t packed) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_half(lo - f.x, hi - f.y);
}

// Row r's query tokens: the first one's place in q and out, how many, and whether the
// row is read here at all.
struct Q8Row {
  int32_t q0, n;
};
__device__ __forceinline__ Q8Row q8_row(const DecodeQ8Params& p, int r) {
  if (p.query_starts == nullptr) return {r * p.query_len, p.query_len};
  const int32_t a = min(max(p.query_starts[r], 0), p.tokens);
  const int32_t n = min(max(p.query_starts[r + 1], a), p.tokens) - a;
  return {a, n <= p.query_len ? n : 0};
}

// Row r's context, 0 where it is not read here.
__device__ __forceinline__ int32_t q8_len(const DecodeQ8Params& p, int r) {
  const int64_t cap = (int64_t)p.max_blocks * p.block_size;
  const int32_t c = p.lens[r];
  if (p.query_starts != nullptr && q8_row(p, r).n == 0) return 0;
  return c < 0 ? 0 : (c > cap ? (int32_t)cap : c);
}

// A block's walk over its share, by each of its warps: segment by segment (a run of
// one row's chunks), in each the chunks that are this warp's.
template <int CT>
struct Q8Walk {
  int hgi, r;          // the segment's kv head group and row
  int32_t c;           // its context
  int32_t c0;          // its first chunk (of the row)
  int32_t g0, g1;      // its chunks among the block's
  int32_t total;       // the block's chunks

  __device__ __forceinline__ void fill(const DecodeQ8Params& p) {
    c = q8_len(p, r);
    g1 = min(total, g0 + (c + CT - 1) / CT - c0);
  }
  __device__ __forceinline__ void start(const DecodeQ8Params& p, int hgi_, int r_, int32_t c0_, int32_t n) {
    hgi = hgi_;
    r = r_;
    c0 = c0_;
    g0 = 0;
    g1 = 0;
    total = n;
    if (total > 0) fill(p);
  }
  __device__ __forceinline__ bool live() const { return g0 < total; }
  __device__ __forceinline__ void next(const DecodeQ8Params& p) {  // the next segment with chunks
    g0 = g1;
    c0 = 0;
    while (g0 < total && g1 == g0) {
      if (++r == p.rows) {
        r = 0;
        ++hgi;
      }
      fill(p);
    }
  }
};

// MANY (fp32): a warp may sum many chunks.  An mma's sum truncates, and hundreds in a row
// add that up, so each chunk's O is summed by itself and then added with rounding.  64 rows
// of 15000 positions (470 chunks a warp): 4.9e-6 of the result off without and 5.0e-7 with,
// 322 and 469 us; 94 chunks: 1.3e-6 and 3.7e-7, 109 and 151 us.  The launch goes by what the
// tables may hold, not by what they do (lengths are the device's): 64 rows of 1024-8192 take
// the 151 us under tables of 131072 tokens, 8 rows of 512-2048 21.8 for 20.3.
template <typename T, int D, int FORM, int NT, bool MANY>
__global__ void __launch_bounds__(32 * Q8Geo<D, NT>::WARPS, 1)
    decode_q8_kernel(const __grid_constant__ DecodeQ8Params p) {
  using Geo = Q8Geo<D, NT>;
  using F = Form8<FORM>;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int WARPS = Geo::WARPS, CT = Geo::CT, NS = Geo::NS, MR = Geo::MR, LD = Geo::LD;
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int PARTS = F32 ? 2 : 1;            // fp16 parts of q and of the weights
  static_assert(!F32 || NT == 1, "fp32 rows fit one tile");
  constexpr int KW = D >= 64 ? 4 : D / 16;      // 4-byte words of a K read
  constexpr int KJ = D / 16 / KW;               // K reads of a token
  constexpr int VB = D >= 128 ? 16 : D / 8;     // bytes of a V read
  constexpr int VJ = D == 256 ? 2 : 1;          // V reads of a token
  extern __shared__ __align__(128) unsigned char q8_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int HG = p.head_group, WPH = WARPS / HG;
  const int hl = warp % HG, wi = warp / HG;     // kv head of the group, warp of the head
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this block's share: chunks [u0, u1) of all rows' chunks (W, < 2^31), which each
  // thread counts for a run of rows.  (What runs once is fetched once, from L2: it is
  // kept short, 32-bit and rolled.)
  __shared__ int warp_sum[WARPS];
  __shared__ int last_stage[WARPS];
  __shared__ int found[3];  // the first chunk's kv head group, row, place in the row
  int W, Pe, each, over;
  // floor(b W / Pe), Pe <= 160
  auto start_of = [&](int b) { return b < Pe ? each * b + over * b / Pe : W; };
  {
    const int per = (p.rows + 32 * WARPS - 1) / (32 * WARPS);
    const int ra = min(p.rows, (int)threadIdx.x * per), rb = min(p.rows, ra + per);
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    int own = 0;
    bool empty = false;
#pragma unroll 1
    for (int r = ra; r < rb; ++r) {
      const int32_t c = p.lens[r];
      if (blockIdx.x == 0) {
        if (c < 0 || c > cap) set_flag(p.err, NP_FLAG_CONTEXT);
        if (p.query_starts != nullptr) {
          const int32_t a = p.query_starts[r], b = p.query_starts[r + 1];
          if (a < 0 || b < a || b > p.tokens) set_flag(p.err, NP_FLAG_QUERY);
        }
      }
      const int n = (q8_len(p, r) + CT - 1) / CT;
      own += n;
      empty |= n == 0;
    }
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULL, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    if (__syncthreads_or(empty)) {  // rows without history: zeros
#pragma unroll 1
      for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
        if (q8_len(p, r) != 0) continue;
        const Q8Row qr = q8_row(p, r);
        T* o = static_cast<T*>(p.out) + (int64_t)qr.q0 * p.q_heads * D;
        for (int i = threadIdx.x; i < qr.n * p.q_heads * D; i += 32 * WARPS) o[i] = T(0.f);
      }
    }
    int before = x - own, all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    W = all * (p.kv_heads / HG);
    Pe = max(1, min((W + p.least - 1) / p.least, (int)gridDim.x));
    each = W / Pe;
    over = W - each * Pe;
    const int u0 = start_of(blockIdx.x);
    if (u0 < W) {
      const int lap = u0 / all, at = u0 - lap * all;
      if (before <= at && at < before + own) {  // one thread's
        int run = before, r = ra;
#pragma unroll 1
        for (;; ++r) {
          const int n = (q8_len(p, r) + CT - 1) / CT;
          if (at < run + n) break;
          run += n;
        }
        found[0] = lap;
        found[1] = r;
        found[2] = at - run;
      }
    }
    if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);  // (unless its last row is cut, below)
    __syncthreads();
  }
  const int u0 = start_of(blockIdx.x);
  const int32_t chunks = start_of(blockIdx.x + 1) - u0;
  if (wi >= WPH || chunks == 0) return;  // (warps beyond the heads' have nothing to do)

  unsigned char* ring = q8_smem + (size_t)warp * NS * Geo::STAGE;
  const uint32_t ring_u = smem_u32(ring);
  // ---- q of a segment, as it is stored: column n of tile nt is row n + 8 nt of the head's
  // (query token, head) rows; a lane holds dims 16 (piece) + 4 word .. + 3 of column g
  Q8Walk<CT> w;
  w.start(p, found[0], found[1], found[2], chunks);
  // (in the registers of O, which hold nothing then)
  using Raw = typename std::conditional<F32, uint4, uint2>::type;  // 4 elements
  float o[NT][D / 16][4];
  Q8Row qr{0, 0};
  auto load_q = [&]() {
    qr = q8_row(p, w.r);
    const int kvh = w.hgi * HG + hl;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g;
      const bool on = row < p.group * qr.n;
      const int qi = on ? row / p.group : 0, h = on ? row - qi * p.group : 0;
      const T* src = static_cast<const T*>(p.q) +
                     ((int64_t)(qr.q0 + qi) * p.q_heads + (int64_t)kvh * p.group + h) * D;
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const int d = D >= 128 ? 16 * (2 * t4 + (j & 1) + 8 * (j >> 1)) + 4 * k : t4 * (4 * KW) + 4 * k;
          Raw x = {};
          if (on) x = *reinterpret_cast<const Raw*>(src + d);
          const int i = j * KW + k;
          if constexpr (F32) {
            o[nt][i][0] = __uint_as_float(x.x);
            o[nt][i][1] = __uint_as_float(x.y);
            o[nt][i][2] = __uint_as_float(x.z);
            o[nt][i][3] = __uint_as_float(x.w);
          } else {
            o[nt][i / 2][i % 2 * 2] = __uint_as_float(x.x);
            o[nt][i / 2][i % 2 * 2 + 1] = __uint_as_float(x.y);
          }
        }
    }
  };

  // ---- loads: chunk by chunk ahead of the reads.  Lane i < CT looks after token i.  Its
  // block is looked up two chunks before the copies.
  Q8Walk<CT> ld = w;
  int32_t lg = wi;  // the next chunk to look up, of the block's
  struct Ahead {
    int32_t block, inner, kvh;  // inner < 0: no token of the row
  };
  auto look_up = [&]() -> Ahead {
    Ahead a{0, -1, -1};
    while (ld.live() && lg >= ld.g1) ld.next(p);
    if (!ld.live()) return a;
    a.kvh = ld.hgi * HG + hl;
    const int32_t t = (ld.c0 + (lg - ld.g0)) * CT + (lane % CT);
    if (t < ld.c) {
      const int32_t j = (int32_t)((uint32_t)t / (uint32_t)p.block_size);
      a.inner = t - j * p.block_size;
      a.block = p.tables[(int64_t)ld.r * p.max_blocks + j];
    }
    lg += WPH;
    return a;
  };
  auto issue = [&](int slot, Ahead x) {
    if (x.kvh >= 0) {
      const uint32_t st = ring_u + (uint32_t)slot * Geo::STAGE;
      const bool held = x.inner >= 0;
      if (!held) x.inner = 0;
      if (x.block < 0 || x.block >= p.num_blocks) {
        set_flag(p.err, NP_FLAG_BLOCK_ID);
        x.block = 0;
      }
      const int64_t at = ((int64_t)x.block * p.block_size + x.inner) * p.kv_heads + x.kvh;
      if (lane < CT) {  // NT 1: 16 lanes; their scales
        const int64_t sc = (int64_t)x.block * p.kv_heads + x.kvh;
        copy4(st + 2 * CT * D + 4 * lane, p.k_scale + sc, held);
        copy4(st + 2 * CT * D + 4 * (CT + lane), p.v_scale + sc, held);
      }
      constexpr int LT = D / 16;                    // lanes of a token
      constexpr int TP = 32 / LT < CT ? 32 / LT : CT;  // tokens of a step
      const int sub = lane / LT, ch = lane % LT;
      const unsigned live = __ballot_sync(FULL, held);
#pragma unroll
      for (int i = 0; i < CT; i += TP) {
        const int tok = (i + sub) % CT;             // (D 16, NT 1: half the lanes repeat)
        const int64_t off = __shfl_sync(FULL, at, tok) * D + ch * 16;
        const bool on = (live >> tok) & 1u;
        if (TP * LT == 32 || lane < TP * LT) {
          copy16(st + Geo::at(tok, ch), p.k_pool + off, on);
          copy16(st + CT * D + Geo::at(tok, ch), p.v_pool + off, on);
        }
      }
    }
    cp_async_commit();
  };
  Ahead a0{0, -1, -1}, a1{0, -1, -1};
  int32_t cg = wi;        // this warp's next chunk
  int slot = 0;           // its stage
  uint32_t qf[NT][PARTS][KJ * KW][2];
  float qs[NT][2];        // scale of rows 2 t4, + 1
  int32_t lim[NT][2];     // the first position each does not see
  int32_t all_see = 0;    // positions before it: every row
  // of rows 2 t4, + 1: -M, what y + b may not pass (-inf: no M yet), the sum
  float off[NT][2], top[NT][2], l[NT][2];
  int last = -1;          // the stage read last in this segment; -1: none yet
  bool first = true;

  // q to fp16, sums to zero
  auto begin = [&]() {
    const int rows_used = p.group * qr.n;  // MR at most
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool on = nt * 8 + g < rows_used;
      float x[KJ * KW][4];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < KJ * KW; ++i) {
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = o[nt][i][e];
        } else {
          widen_bf16x2(__float_as_uint(o[nt][i / 2][i % 2 * 2]), x[i][0], x[i][1]);
          widen_bf16x2(__float_as_uint(o[nt][i / 2][i % 2 * 2 + 1]), x[i][2], x[i][3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[i][e]));
      }
      big = fmaxf(big, __shfl_xor_sync(FULL, big, 1));
      big = fmaxf(big, __shfl_xor_sync(FULL, big, 2));
      // the row's largest element to [2^14, 2^15)
      const int e = min(14 + 127 - (int)(__float_as_uint(big) >> 23), 120);
      const float f = pow2f(e);
      const float s = on ? p.qscale * pow2f(-e) : 0.f;
      qs[nt][0] = __shfl_sync(FULL, s, 8 * t4);
      qs[nt][1] = __shfl_sync(FULL, s, 8 * t4 + 4);
#pragma unroll
      for (int i = 0; i < KJ * KW; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float a = x[i][2 * c] * f, b = x[i][2 * c + 1] * f;
          qf[nt][0][i][c] = pack_half(a, b);
          if constexpr (F32) qf[nt][1][i][c] = pack_rest(a, b, qf[nt][0][i][c]);
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row2 = nt * 8 + 2 * t4 + c;
        lim[nt][c] = row2 < rows_used ? w.c - qr.n + row2 / p.group + 1 : w.c;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
      off[nt][0] = off[nt][1] = 0.f;
      top[nt][0] = top[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
    all_see = w.c - qr.n + 1;
  };

  // The segment's end: each of the head's warps puts m, l and O into the stage it read
  // last (which nothing is on its way into), then each joins some of the rows.
  auto finish = [&]() {
    const Q8Row now = q8_row(p, w.r);
    const int32_t q0 = now.q0, kvh = w.hgi * HG + hl, rows_used = p.group * now.n;
    __syncwarp();
    if (last >= 0) {
      float* e = reinterpret_cast<float*>(ring + (size_t)last * Geo::STAGE);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = l[nt][c];
          x += __shfl_xor_sync(FULL, x, 4);
          x += __shfl_xor_sync(FULL, x, 8);
          x += __shfl_xor_sync(FULL, x, 16);
          const int row = nt * 8 + 2 * t4 + c;
          if (g == 0) {
            e[row] = top[nt][c] == -INFINITY ? -INFINITY : -off[nt][c];
            e[MR + row] = x * pow2f(kWeightExp);  // (as O is)
          }
          float* orow = e + 2 * MR + row * LD;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int j = i / (VB / 2), d = j * 128 + g * VB + 2 * (i % (VB / 2));
            *reinterpret_cast<float2*>(orow + d) = make_float2(o[nt][i][c], o[nt][i][2 + c]);
          }
        }
    }
    if (lane == 0) last_stage[warp] = last;
    const bool whole = w.c0 == 0 && w.g1 - w.g0 >= (w.c + CT - 1) / CT;
    if (threadIdx.x == 0 && w.g1 == w.total && w.c0 == 0 && !whole) {
      // The share ends in this row, which begins here: it is cut, and its last block is the
      // one with its last chunk.
      const int end = u0 + w.g0 + (w.c + CT - 1) / CT;
      int to = min((int)((float)end * (float)Pe / (float)W), Pe - 1);
      while (to + 1 < Pe && start_of(to + 1) < end) ++to;
      while (start_of(to) >= end) --to;
      p.cuts[blockIdx.x] = make_int4(w.hgi * p.rows + w.r, blockIdx.x, to, first ? 0 : 1);
    }
    w.next(p);
    if (w.live()) load_q();  // the next segment's, on its way meanwhile
    if (WPH > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + hl), "r"(32 * WPH) : "memory");
    else __syncwarp();
    {
      float* part = p.parts + (((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * HG + hl) * q8_entry_floats(D);
      // lane i: the stage that warp i of the head read last, -1: it had no chunk here
      int at = -1;
      if (lane < WPH) {
        const int wr = hl + lane * HG, st = last_stage[wr];
        at = st < 0 ? -1 : (wr * NS + st) * Geo::STAGE;
      }
      const unsigned has = __ballot_sync(FULL, at >= 0);
      // lane r: row r's maximum and sum
      float M = -INFINITY, L = 0.f;
      const int mine = lane < MR ? lane : 0;
      for (unsigned k = has; k != 0; k &= k - 1) {
        const float* e = reinterpret_cast<const float*>(q8_smem + __shfl_sync(FULL, at, __ffs(k) - 1));
        const float mx = fmaxf(M, e[mine]), ref = mx == -INFINITY ? 0.f : mx;
        L = scaled_down(e[MR + mine], e[mine] - ref) + scaled_down(L, M - ref);
        M = mx;
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      if (!whole && wi == 0 && lane < rows_used) {
        part[lane] = M;
        part[kQ8Rows + lane] = L;
      }
      // rows in turn over the head's warps, LR lanes a row, 4 (or 2 x 4) dims a lane, RU rows
      // of a lane side by side
      constexpr int LR = D >= 128 ? 32 : D / 4, RP = 32 / LR, DV = D == 256 ? 2 : 1;
      constexpr int RU = D == 256 ? 2 : 4;
      const int d = lane % LR * 4;
#pragma unroll 1
      for (int r0 = wi * RP + lane / LR; r0 - lane / LR < rows_used; r0 += RU * WPH * RP) {
        float ref[RU], f0[RU], acc[RU][DV][4];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int row = min(r0 + u * WPH * RP, MR - 1);
          const float Mr = __shfl_sync(FULL, M, row), iv = __shfl_sync(FULL, inv, row);
          ref[u] = Mr == -INFINITY ? 0.f : Mr;
          f0[u] = whole ? iv : 1.f;
#pragma unroll
          for (int v = 0; v < DV; ++v) acc[u][v][0] = acc[u][v][1] = acc[u][v][2] = acc[u][v][3] = 0.f;
        }
#pragma unroll 1
        for (unsigned k = has; k != 0; k &= k - 1) {
          const float* e = reinterpret_cast<const float*>(q8_smem + __shfl_sync(FULL, at, __ffs(k) - 1));
#pragma unroll
          for (int u = 0; u < RU; ++u) {
            const int row = min(r0 + u * WPH * RP, MR - 1);
            const float f = ex2(e[row] - ref[u]) * f0[u];
#pragma unroll
            for (int v = 0; v < DV; ++v) {
              const float4 x = *reinterpret_cast<const float4*>(e + 2 * MR + row * LD + d + 128 * v);
              acc[u][v][0] = fmaf(f, x.x, acc[u][v][0]);
              acc[u][v][1] = fmaf(f, x.y, acc[u][v][1]);
              acc[u][v][2] = fmaf(f, x.z, acc[u][v][2]);
              acc[u][v][3] = fmaf(f, x.w, acc[u][v][3]);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const int row = r0 + u * WPH * RP;
          if (row >= rows_used) continue;
          if (whole) {
            // rows are the query tokens' heads of this kv head: a token's lie side by side
            const int qi = row / p.group;
            T* out = static_cast<T*>(p.out) +
                     ((int64_t)(q0 + qi) * p.q_heads + (int64_t)(kvh - qi) * p.group + row) * D;
#pragma unroll
            for (int v = 0; v < DV; ++v) Storage<T>::template store<4>(out + d + 128 * v, acc[u][v]);
          } else {
#pragma unroll
            for (int v = 0; v < DV; ++v)
              Storage<float>::store<4>(part + 2 * kQ8Rows + row * D + d + 128 * v, acc[u][v]);
          }
        }
      }
    }
    if (WPH > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + hl), "r"(32 * WPH) : "memory");
    else __syncwarp();
    first = false;
    last = -1;
  };

  load_q();  // (on its way while the first chunks are looked up)
#pragma unroll 1
  for (int it = -2; it < NS - 1; ++it) {
    const Ahead a2 = look_up();
    if (it >= 0) issue(it, a0);
    a0 = a1;
    a1 = a2;
  }
  while (w.live()) {
    begin();
    for (; cg < w.g1; cg += WPH) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      {
        const Ahead a2 = look_up();
        issue(slot == 0 ? NS - 1 : slot - 1, a0);  // into the stage read before
        a0 = a1;
        a1 = a2;
      }
      const uint32_t st = ring_u + (uint32_t)slot * Geo::STAGE;
      last = slot;
      slot = slot + 1 == NS ? 0 : slot + 1;
      const int32_t t0 = (w.c0 + (cg - w.g0)) * CT;
#pragma unroll
      for (int sub = 0; sub < CT; sub += 16) {
        // ---- S
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        float rest[4] = {0.f, 0.f, 0.f, 0.f};  // fp32: of q's second part
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          uint32_t a[KW], b[KW];
          if constexpr (D >= 128) {
            const int ch = 2 * t4 + (j & 1) + 8 * (j >> 1);
            lds<KW>(st + Geo::at(sub + g, ch), a);
            lds<KW>(st + Geo::at(sub + g + 8, ch), b);
          } else {
            const int ch = t4 * KW / 4, in = t4 * KW % 4 * 4;
            lds<KW>(st + Geo::at(sub + g, ch) + in, a);
            lds<KW>(st + Geo::at(sub + g + 8, ch) + in, b);
          }
#pragma unroll
          for (int k = 0; k < KW; ++k) {
            const uint32_t a0 = F::half_lo(a[k]), a2 = F::half_hi(a[k]);
            const uint32_t a1 = F::half_lo(b[k]), a3 = F::half_hi(b[k]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(s[nt], a0, a1, a2, a3, qf[nt][0][j * KW + k][0], qf[nt][0][j * KW + k][1]);
              if constexpr (F32)
                mma_f16(rest, a0, a1, a2, a3, qf[nt][1][j * KW + k][0], qf[nt][1][j * KW + k][1]);
            }
          }
        }
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] += rest[e];
        }
        // ---- softmax: rows of S are tokens g and g + 8
        uint32_t sc[4];
        lds<1>(st + 2 * CT * D + 4 * (sub + g), &sc[0]);
        lds<1>(st + 2 * CT * D + 4 * (sub + g + 8), &sc[1]);
        lds<1>(st + 2 * CT * D + 4 * (CT + sub + g), &sc[2]);
        lds<1>(st + 2 * CT * D + 4 * (CT + sub + g + 8), &sc[3]);
        const float ka = pow2f(scale_exp(sc[0])), kb = pow2f(scale_exp(sc[1]));
        const int ea = scale_exp(sc[2]), eb = scale_exp(sc[3]);
        const float va = (float)ea, vb = (float)eb, wa = pow2f(ea + kWeightExp), wb = pow2f(eb + kWeightExp);
        const bool edge = t0 + sub + 16 > all_see;  // uniform
        // y, with one rounding; M is a whole number
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            s[nt][c] = fmaf(s[nt][c], ka * qs[nt][c], off[nt][c]);
            s[nt][2 + c] = fmaf(s[nt][2 + c], kb * qs[nt][c], off[nt][c]);
            if (edge) {
              if (t0 + sub + g >= lim[nt][c]) s[nt][c] = -INFINITY;
              if (t0 + sub + g + 8 >= lim[nt][c]) s[nt][2 + c] = -INFINITY;
            }
            grow |= fmaxf(s[nt][c] + va, s[nt][2 + c] + vb) > top[nt][c];
          }
        }
        if (__any_sync(FULL, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = fmaxf(s[nt][c] + va, s[nt][2 + c] + vb);
              x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
              x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
              x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
              if (x > top[nt][c]) {
                x = ceilf(x);
                const float f = top[nt][c] == -INFINITY ? 0.f : ex2(-x);
                l[nt][c] = top[nt][c] == -INFINITY ? 0.f : scaled_down(l[nt][c], -x);
                off[nt][c] -= x;
                top[nt][c] = kAbove;
                s[nt][c] -= x;
                s[nt][2 + c] -= x;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  o[nt][i][c] *= f;
                  o[nt][i][2 + c] *= f;
                }
              }
            }
          }
        }
        uint32_t pf[NT][PARTS][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            s[nt][c] = ex2(s[nt][c]);
            s[nt][2 + c] = ex2(s[nt][2 + c]);
            l[nt][c] += s[nt][c] + s[nt][2 + c];
            s[nt][c] *= wa;
            s[nt][2 + c] *= wb;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x = pack_half(s[nt][2 * k], s[nt][2 * k + 1]);
            pf[nt][0][k] = transpose8(x);
            if constexpr (F32) pf[nt][1][k] = transpose8(pack_rest(s[nt][2 * k], s[nt][2 * k + 1], x));
          }
        }
        // ---- O += V^T P: a lane's dims are VB bytes of tokens 2 t4, + 1, + 8, + 9
        auto add = [&](float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                       const uint32_t (&w)[PARTS][2]) {
          if constexpr (F32) {
            if constexpr (MANY) {
              float x[4];
              mma_f16_first(x, a0, a1, a2, a3, w[1][0], w[1][1]);
              mma_f16(x, a0, a1, a2, a3, w[0][0], w[0][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) c[e] += x[e];
            } else {
              mma_f16(c, a0, a1, a2, a3, w[1][0], w[1][1]);
              mma_f16(c, a0, a1, a2, a3, w[0][0], w[0][1]);
            }
          } else {
            mma_f16(c, a0, a1, a2, a3, w[0][0], w[0][1]);
          }
        };
#pragma unroll
        for (int j = 0; j < VJ; ++j) {
          uint32_t x[4][(VB + 3) / 4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = sub + 2 * t4 + (k & 1) + 8 * (k >> 1);
            const int byte = j * 128 + g * VB;
            const uint32_t at = st + CT * D + Geo::at(tok, byte >> 4) + (byte & 15);
            if constexpr (VB == 2) {
              uint16_t y;
              asm volatile("ld.shared.u16 %0, [%1];" : "=h"(y) : "r"(at));
              x[k][0] = y;
            } else {
              lds<VB / 4>(at, x[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < (VB + 3) / 4; ++k) {
            const uint32_t p01 = __byte_perm(x[0][k], x[1][k], 0x5140), p23 = __byte_perm(x[2][k], x[3][k], 0x5140);
            const uint32_t a0 = F::half_lo(p01), a1 = F::half_hi(p01);
            const uint32_t a2 = F::half_lo(p23), a3 = F::half_hi(p23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) add(o[nt][j * (VB / 2) + 2 * k], a0, a1, a2, a3, pf[nt]);
            if constexpr (VB >= 4) {
              const uint32_t q01 = __byte_perm(x[0][k], x[1][k], 0x7362),
                             q23 = __byte_perm(x[2][k], x[3][k], 0x7362);
              const uint32_t b0 = F::half_lo(q01), b1 = F::half_hi(q01);
              const uint32_t b2 = F::half_lo(q23), b3 = F::half_hi(q23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) add(o[nt][j * (VB / 2) + 2 * k + 1], b0, b1, b2, b3, pf[nt]);
            }
          }
        }
      }
    }
    finish();
  }
  cp_async_wait<0>();
}

// The join: one warp per (cut row, kv head, (query token, head) row), over the blocks
// that hold a piece, in block order: 32 pieces' m and l in one round, then their rows of O,
// eight loads in flight.  Bound by the latency of those rounds (the partials are in L2).
constexpr int kQ8JoinThreads = 256;
constexpr int kQ8JoinGrid = 4;  // blocks an SM: 64 rows 102, 100, 99, 101 us with 1, 2, 4, 6

template <typename T, int D>
__global__ void __launch_bounds__(kQ8JoinThreads) decode_q8_join_kernel(const __grid_constant__
                                                                        DecodeQ8Params p) {
  __shared__ int4 list[kQ8MaxCtas];
  __shared__ int cuts;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int WARPS = kQ8JoinThreads / 32, U = 8;
  constexpr int LR = D >= 128 ? 32 : D / 4, DV = D == 256 ? 2 : 1;  // lanes of a row, 4 (2 x 4) dims each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int HG = p.head_group, MR = p.group * p.query_len;  // rows at most
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {
    int4 c[kQ8MaxCtas / 32];
#pragma unroll
    for (int i = 0; i < kQ8MaxCtas / 32; ++i)
      c[i] = 32 * i + lane < p.ctas ? __ldcg(p.cuts + 32 * i + lane) : make_int4(-1, 0, 0, 0);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kQ8MaxCtas / 32; ++i) {
      const unsigned m = __ballot_sync(FULL, c[i].x >= 0);
      if (c[i].x >= 0) list[n + __popc(m & ((1u << lane) - 1u))] = c[i];
      n += __popc(m);
    }
    if (lane == 0) cuts = n;
  }
  __syncthreads();
  const int tasks = cuts * HG * MR;
  const int d = lane % LR * 4;
  for (int task = blockIdx.x + warp * gridDim.x; task < tasks; task += WARPS * gridDim.x) {
    const int row = task % MR, hl = task / MR % HG;
    const int4 c = list[task / MR / HG];
    const int r = c.x % p.rows, kvh = c.x / p.rows * HG + hl;
    const Q8Row qr = q8_row(p, r);
    if (row >= p.group * qr.n) continue;
    auto entry = [&](int b) {
      return p.parts + (((size_t)b * 2 + (b == c.y ? c.w : 0)) * HG + hl) * q8_entry_floats(D);
    };
    float M = -INFINITY, L = 0.f, acc[DV][4];
#pragma unroll
    for (int v = 0; v < DV; ++v) acc[v][0] = acc[v][1] = acc[v][2] = acc[v][3] = 0.f;
    for (int b0 = c.y; b0 <= c.z; b0 += 32) {
      const int n = min(32, c.z - b0 + 1);
      float m = -INFINITY, l = 0.f;
      if (lane < n) {
        const float* e = entry(b0 + lane);
        m = __ldcg(e + row);
        l = __ldcg(e + kQ8Rows + row);
      }
      float4 x[U][DV];
      auto fetch = [&](int u0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* e = entry(b0 + min(u0 + u, n - 1)) + 2 * kQ8Rows + row * D + d;
#pragma unroll
          for (int v = 0; v < DV; ++v) x[u][v] = __ldcg(reinterpret_cast<const float4*>(e + 128 * v));
        }
      };
      fetch(0);  // (with m and l on their way)
      float mx = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, o));
      mx = fmaxf(mx, M);
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float f = ex2(M - ref), a = ex2(m - ref);
      float sum = scaled_down(l, m - ref);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
      L = scaled_down(L, M - ref) + sum;
      M = mx;
#pragma unroll
      for (int v = 0; v < DV; ++v) {
        acc[v][0] *= f;
        acc[v][1] *= f;
        acc[v][2] *= f;
        acc[v][3] *= f;
      }
#pragma unroll 1
      for (int u0 = 0; u0 < n; u0 += U) {
        if (u0 > 0) fetch(u0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float g = u0 + u < n ? __shfl_sync(FULL, a, (u0 + u) & 31) : 0.f;
#pragma unroll
          for (int v = 0; v < DV; ++v) {
            acc[v][0] = fmaf(g, x[u][v].x, acc[v][0]);
            acc[v][1] = fmaf(g, x[u][v].y, acc[v][1]);
            acc[v][2] = fmaf(g, x[u][v].z, acc[v][2]);
            acc[v][3] = fmaf(g, x[u][v].w, acc[v][3]);
          }
        }
      }
    }
    if (lane >= LR) continue;  // (narrow heads: the other lanes repeat)
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const int qi = row / p.group, h = row - qi * p.group;
    T* out = static_cast<T*>(p.out) + ((int64_t)(qr.q0 + qi) * p.q_heads + (int64_t)kvh * p.group + h) * D;
#pragma unroll
    for (int v = 0; v < DV; ++v) {
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = acc[v][e] * inv;
      Storage<T>::template store<4>(out + d + 128 * v, y);
    }
  }
}

template <typename T, int D, int FORM, int NT, bool MANY>
static np_status launch(const DecodeQ8Params& p, cudaStream_t s) {
  using Geo = Q8Geo<D, NT>;
  static unsigned long long allowed = 0;
  np_status rc = allow_smem(decode_q8_kernel<T, D, FORM, NT, MANY>, Geo::SMEM, &allowed);
  if (rc != NP_OK) return rc;
  decode_q8_kernel<T, D, FORM, NT, MANY><<<p.ctas, 32 * Geo::WARPS, Geo::SMEM, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NP_ERR_CUDA;
  return launch_dependent(decode_q8_join_kernel<T, D>, kQ8JoinGrid * p.ctas, 1, kQ8JoinThreads, 0, s, p);
}

#define NPK_CAT2(a, b) a##b
#define NPK_CAT(a, b) NPK_CAT2(a, b)

#if NPK_FORM == 0
#define NPK_NAME NPK_CAT(NPK_CAT(decode_q8_d, NPK_D), _e4m3)
#else
#define NPK_NAME NPK_CAT(NPK_CAT(decode_q8_d, NPK_D), _int8)
#endif

np_status NPK_NAME(const DecodeQ8Params& p, np_dtype dtype, cudaStream_t s) {
  if (dtype == NP_F32) {
    // chunks that a warp may have to sum, from the tables' size
    const int64_t most = (int64_t)p.rows * p.max_blocks * p.block_size / 16 * (p.kv_heads / p.head_group) /
                         ((int64_t)p.ctas * (q8_warps(NPK_D, 1) / p.head_group));
    return most > 128 ? launch<float, NPK_D, NPK_FORM, 1, true>(p, s)
                      : launch<float, NPK_D, NPK_FORM, 1, false>(p, s);
  }
  return p.group * p.query_len <= 8 ? launch<__nv_bfloat16, NPK_D, NPK_FORM, 1, false>(p, s)
                                    : launch<__nv_bfloat16, NPK_D, NPK_FORM, 2, false>(p, s);
}

}  // namespace npk
