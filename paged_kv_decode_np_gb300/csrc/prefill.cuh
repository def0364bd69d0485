// prefill.cuh -- what the kernels of np_paged_prefill share: parameters, the
// division of the work over thread blocks, and the workspace.
//
// The operation, per row r with chunk length n (its newest positions) and
// context length c, kv head k with its G query heads: chunk token i attends
// to positions t <= c - n + i.  A *unit* is BM (token, head) rows of one kv
// head -- U = MT * (BMT / G) chunk tokens times their G heads, packed token-major as MT
// tiles of BMT rows -- against the positions its last token sees, in kv tiles of BN
// tokens: nk(m) = max(1, ceil((c - n + min(n, (m + 1) U)) / BN)) tiles.
//
// All units, in the order (row, kv head, m), are laid end to end as one
// stream, a cost per kv tile and a fixed cost each, and the stream is cut into one
// equal share per thread block: every SM has the same amount of work whatever
// the mix of long and short chunks, causal triangles and histories.  A block walks its share; a
// unit that lies inside one block is normalised and stored directly, a unit
// cut by a share's end leaves a partial (m, l, unnormalised O in fp32) per
// block that touched it, and a second launch joins them in block order
// (deterministic, no atomics).  A block cuts at most two units, so the
// workspace has a fixed size.
//
// Three launches: the plan (one block: the shares' ends), the attention, the
// join.  The plan's scan over the rows would cost each attention block the
// same time if it were repeated there, and needs registers that the
// attention has no room for.
#pragma once

#include <cuda.h>
#include <math.h>

#include "np_common.cuh"

namespace npk {

constexpr int kPrefillMaxCtas = 160;
constexpr int kPrefillMaxRows = 4096;

struct PrefillParams {
  CUtensorMap tm_q, tm_k, tm_v;  // bf16 tensor-core kernel with tiled copies only
  void* out;
  const void* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_starts;
  int32_t* err;
  int4* plan;    // [ctas + 1] {row, kv head, m, kv tile}: where each block's share begins
  int4* cuts;    // [ctas] {row (-1: none), kv head, m, last block}: units cut by a share's end
  float* parts;  // [ctas][2] partials
  int64_t num_blocks;
  int32_t block_size, kv_heads, q_heads, group, max_blocks_per_row;
  int32_t rows, tokens, ctas, head_dim;
  int32_t tile_tokens;  // chunk tokens of one BMT-row tile: BMT / G
  int32_t tile_rows;    // BMT
  int32_t tiles;        // MT
  int32_t bn;           // kv tile
  // what the plan counts: for a kv tile of a unit whose tiles all have tokens,
  // of one with a single such tile, for beginning a unit; the least share of a block
  int32_t full_cost, single_cost, unit_cost, min_share;
  int32_t box_tokens;   // tokens per tiled copy
  float qscale;         // |scale| * log2(e)
  int32_t negate;       // scale < 0
};

// The tiles of a type and head_dim, and what the plan counts for them.
// Measured, us, {full, single, unit cost, least share}.  bf16, two q tiles: a batch
// of 62 one-token rows and two chunks of 512 takes 242 with {3, 2, 8, 8}, 304
// with {1, 1, 2, 4}, 275 with {2, 1, 6, 6}; six prompts of 581-2750 tokens 227,
// 230, 227, and 239 with {1, 1, 1, 3}; 16 tokens over 1000 positions 16.7, with
// a least share of 16 20.5.  One q tile (head_dim 256, 16 chunks): {1, 1, 2, 4}
// 72, {1, 1, 1, 3} 75, {3, 2, 8, 8} 89.  fp32 (head_dim 128; eight chunks of
// 71-184 over 833-2031 positions, and 32 over 900): unit cost 3 183, 1 187, 8
// 190; least share 2 23, 4 28, 6 31.
inline void prefill_tiling(PrefillParams& p, np_dtype dtype) {
  const bool two = dtype == NP_BF16 && p.head_dim <= 128;
  p.tiles = two ? 2 : 1;
  p.tile_rows = dtype == NP_F32 && p.head_dim == 256 ? 64 : 128;
  p.bn = two ? 128 : 64;
  p.tile_tokens = p.tile_rows / p.group;
  p.full_cost = two ? 3 : 1;
  p.single_cost = two ? 2 : 1;
  p.unit_cost = two ? 8 : (dtype == NP_BF16 ? 2 : 3);
  p.min_share = two ? 8 : (dtype == NP_BF16 ? 4 : 2);
}

// floats of one partial: m[BM], l[BM], O[D/4][BM][4]
__host__ __device__ inline size_t prefill_part_floats(int bm, int d) { return (size_t)bm * (d + 2); }

struct PrefillRow {
  int32_t q0;  // first chunk token in q and out
  int32_t n;   // chunk tokens
  int32_t c;   // context, the chunk included
};

// The arithmetic of the shares and of the walk is for the host too: it is
// tested there, as it stands, against brute force.
#define NPK_HD __host__ __device__ __forceinline__

NPK_HD void prefill_flag(const PrefillParams& p, int32_t bit) {
#ifdef __CUDA_ARCH__
  set_flag(p.err, bit);
#else
  if (p.err) *p.err |= bit;
#endif
}

// Row r's chunk and context, clamped into what the arrays hold.
NPK_HD PrefillRow prefill_row(const PrefillParams& p, int r, bool flag = false) {
  PrefillRow g;
  const int32_t a = p.query_starts[r], b = p.query_starts[r + 1];
  const int64_t cap = (int64_t)p.max_blocks_per_row * p.block_size;
  int32_t c = p.context_lens[r];
  const int32_t a2 = min(max(a, 0), p.tokens);
  const int32_t b2 = min(max(b, a2), p.tokens);
  if (flag && (a2 != a || b2 != b)) prefill_flag(p, NP_FLAG_QUERY);
  if (c < 0 || c > cap) {
    if (flag) prefill_flag(p, NP_FLAG_CONTEXT);
    c = c < 0 ? 0 : (int32_t)cap;
  }
  g.q0 = a2;
  g.n = b2 - a2;
  g.c = c;
  return g;
}

NPK_HD int prefill_units(const PrefillParams& p, int n) {
  const int u = p.tile_tokens * p.tiles;
  return n / u + (n % u != 0);
}

// positions [0, end) are seen by the first `tok` chunk tokens
NPK_HD int prefill_end(const PrefillRow& g, int64_t tok) {
  const int64_t e = (int64_t)g.c - g.n + (tok < g.n ? tok : g.n);
  return e < 0 ? 0 : (int)e;
}

// kv tiles of the first `tok` chunk tokens (at least one: a unit that sees
// nothing still has its zeros to write)
NPK_HD int prefill_kv_tiles(const PrefillParams& p, const PrefillRow& g, int64_t tok) {
  const int e = prefill_end(g, tok);
  const int nk = e / p.bn + (e % p.bn != 0);
  return nk < 1 ? 1 : nk;
}

// sum over i < n of floor((a i + b) / m), for a, b >= 0, m > 0: the lattice
// points under a line, counted by Euclid's reduction of (a, m).  T holds
// a n + b; a 64-bit division takes several times a 32-bit one.
template <typename T>
NPK_HD int64_t floor_sum_in(T n, T m, T a, T b) {
  int64_t s = 0;
  while (n > 0) {
    const T qa = a / m, qb = b / m;
    s += (int64_t)n * (n - 1) / 2 * qa + (int64_t)n * qb;
    a -= qa * m;
    b -= qb * m;
    const T y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const T t = m;
    m = a;
    a = t;
  }
  return s;
}

NPK_HD int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  // the first step leaves a < m and b < m; later ones only shrink
  if (n < (1 << 20) && m <= 1024 && a <= 1024 && b < (1ll << 31))
    return floor_sum_in<uint32_t>((uint32_t)n, (uint32_t)m, (uint32_t)a, (uint32_t)b);
  return floor_sum_in<int64_t>(n, m, a, b);
}

// what a kv tile of a row's unit a costs
NPK_HD int prefill_tile_cost(const PrefillParams& p, const PrefillRow& g, int a) {
  return ((int64_t)a * p.tiles + 1) * p.tile_tokens >= g.n ? p.single_cost : p.full_cost;
}

// cost of a row's first k units (of one kv head), k <= units
NPK_HD int64_t prefill_row_prefix(const PrefillParams& p, const PrefillRow& g, int units, int k) {
  if (k <= 0) return 0;
  const int64_t U = (int64_t)p.tile_tokens * p.tiles;
  int64_t cost = (int64_t)k * p.unit_cost;
  if (k == units) {  // the last unit ends with the chunk, not U tokens on
    --k;
    cost += (int64_t)prefill_kv_tiles(p, g, g.n) * prefill_tile_cost(p, g, k);
  }
  const int64_t base = (int64_t)g.c - g.n;
  const int64_t z0 = base < 0 ? -base / U : 0;  // units that see nothing: one tile each
  const int z = z0 < k ? (int)z0 : k;
  return cost + (z + floor_sum(k - z, p.bn, U, base + (z + 1) * U + p.bn - 1)) * p.full_cost;
}

// cost of all units of row r, every kv head's
NPK_HD int64_t prefill_row_cost(const PrefillParams& p, int r) {
  const PrefillRow g = prefill_row(p, r, true);
  const int units = prefill_units(p, g.n);
  return prefill_row_prefix(p, g, units, units) * p.kv_heads;
}

// Where block b's share begins; pre[r]: work before row r, pre[rows]: all of it.
NPK_HD int4 prefill_share_start(const PrefillParams& p, const int64_t* pre, int b) {
  const int64_t W = pre[p.rows];
  // blocks that share the work: a share holds min_share at least
  const int64_t want = (W + p.min_share - 1) / p.min_share;
  const int Pe = (int)(want < 1 ? 1 : (want < p.ctas ? want : p.ctas));
  const int64_t share = W / Pe;
  const int64_t x = b >= Pe ? W : share * b + (W % Pe) * b / Pe;
  if (x >= W) return make_int4(p.rows, 0, 0, 0);
  int lo = 0, hi = p.rows;  // the last row with pre[row] <= x: it has work there
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid;
  }
  const PrefillRow g = prefill_row(p, lo);
  const int units = prefill_units(p, g.n);
  const int64_t wh = (pre[lo + 1] - pre[lo]) / p.kv_heads;
  int kvh = (int)((x - pre[lo]) / wh);
  const int64_t in = (x - pre[lo]) - kvh * wh;
  int a = 0, e = units;  // the last unit that begins at or before `in`
  while (e - a > 1) {
    const int mid = (a + e) >> 1;
    if (prefill_row_prefix(p, g, units, mid) <= in) a = mid;
    else e = mid;
  }
  const int64_t s0 = prefill_row_prefix(p, g, units, a);
  const int nk = prefill_kv_tiles(p, g, (int64_t)(a + 1) * p.tile_tokens * p.tiles);
  const int cost = prefill_tile_cost(p, g, a);
  int off = ((int)(in - s0) - p.unit_cost) / cost;  // <= 0: within the fixed cost
  // An end that lies near a unit's own start or end is moved there: the partials
  // it saves cost more than the imbalance.  Within 1/8, 1/16, 1/32 of a share, or
  // not at all, us: mixed batch 249, 240, 244, 244; 16 wide chunks 78, 74, 77, 77;
  // fp32 chunks 182, 166, 165, 165; six prompts 239, 243, 243, 242.
  if (off <= 0 || (int64_t)off * cost * 16 <= share) {
    off = 0;
  } else if ((int64_t)(nk - off) * cost * 16 <= share) {
    off = 0;
    // the unit after: of this head, the next head, or the next row
    if (++a >= units) {
      a = 0;
      if (++kvh >= p.kv_heads) {
        kvh = 0;
        ++lo;
      }
    }
  }
  return make_int4(lo, kvh, a, off);
}

// The unit that the end of block b's share cuts, if the share holds its first
// tile, with the last block that has a piece of it; row -1: none.
NPK_HD int4 prefill_share_cut(const PrefillParams& p, const int4* pos, int b) {
  auto same = [](const int4& u, const int4& v) { return u.x == v.x && u.y == v.y && u.z == v.z; };
  const int4 s = pos[b], e = pos[b + 1];
  if (e.w <= 0 || (same(s, e) && s.w != 0)) return make_int4(-1, 0, 0, 0);
  int last = b + 1;  // the last block whose share begins in the unit
  while (last + 1 <= p.ctas && same(pos[last + 1], e)) ++last;
  return make_int4(e.x, e.y, e.z, last);
}

// A block's walk over its share: one segment is a run of kv tiles [kv0, kv1)
// of one unit.  Every role of the block walks it by itself.
struct PrefillWalk {
  int r, kvh, m;
  int off;      // first kv tile of the next segment
  int4 end;     // where the next block's share begins
  PrefillRow g;
  int units;
  // the current segment
  int kv0, kv1, nk;

  NPK_HD void start(const PrefillParams& p, int cta) {
    const int4 a = p.plan[cta];
    end = p.plan[cta + 1];
    r = a.x;
    kvh = a.y;
    m = a.z;
    off = a.w;
    units = 0;
    if (r < p.rows) {
      g = prefill_row(p, r);
      units = prefill_units(p, g.n);
    }
  }
  // the next segment; false at the share's end
  NPK_HD bool next(const PrefillParams& p) {
    if (r >= p.rows) return false;
    while (m >= units) {  // past the kv head's last unit
      m = 0;
      if (++kvh < p.kv_heads && units > 0) break;
      kvh = 0;
      if (++r >= p.rows) return false;
      g = prefill_row(p, r);
      units = prefill_units(p, g.n);
    }
    const bool last = r == end.x && kvh == end.y && m == end.z;  // the unit that the share ends in
    if (last ? off >= end.w
             : r > end.x || (r == end.x && (kvh > end.y || (kvh == end.y && m > end.z))))
      return false;
    nk = prefill_kv_tiles(p, g, (int64_t)(m + 1) * p.tile_tokens * p.tiles);
    kv0 = off;
    kv1 = last ? end.w : nk;
    return true;
  }
  // past the current segment (its fields stay valid until next())
  NPK_HD void advance() {
    off = 0;
    ++m;
  }
  NPK_HD bool whole() const { return kv0 == 0 && kv1 == nk; }
};

// prefill_plan.cu
np_status launch_prefill_plan(const PrefillParams& p, cudaStream_t s);
np_status launch_prefill_join(const PrefillParams& p, np_dtype dtype, cudaStream_t s);
// prefill_simt.cu
np_status launch_prefill_simt(const PrefillParams& p, cudaStream_t s);

// prefill_tc.cu, per head_dim
np_status prefill_tc_d16(const PrefillParams& p, bool tiled, cudaStream_t s);
np_status prefill_tc_d32(const PrefillParams& p, bool tiled, cudaStream_t s);
np_status prefill_tc_d64(const PrefillParams& p, bool tiled, cudaStream_t s);
np_status prefill_tc_d128(const PrefillParams& p, bool tiled, cudaStream_t s);
np_status prefill_tc_d256(const PrefillParams& p, bool tiled, cudaStream_t s);

// prefill_tc32.cu, per head_dim
np_status prefill_tc32_d16(const PrefillParams& p, cudaStream_t s);
np_status prefill_tc32_d32(const PrefillParams& p, cudaStream_t s);
np_status prefill_tc32_d64(const PrefillParams& p, cudaStream_t s);
np_status prefill_tc32_d128(const PrefillParams& p, cudaStream_t s);

// The opt-in shared-memory limit of a kernel, a per-device attribute: set at
// its first launch on a device.  `done`: one word per kernel, bit d for device d.
template <typename K>
np_status allow_smem(K kern, size_t bytes, unsigned long long* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NP_ERR_CUDA;
  if (dev < 64 && ((__atomic_load_n(done, __ATOMIC_ACQUIRE) >> dev) & 1ull)) return NP_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
      cudaSuccess)
    return NP_ERR_CUDA;
  if (dev < 64) __atomic_fetch_or(done, 1ull << dev, __ATOMIC_ACQ_REL);
  return NP_OK;
}

// Launches `kern` so that it may become resident while the launch before it
// still runs; its griddepcontrol.wait holds it until that one is complete.
template <typename K, typename... A>
np_status launch_dependent(K kern, unsigned grid_x, unsigned grid_y, unsigned threads, size_t smem,
                           cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? NP_OK : NP_ERR_CUDA;
}

}  // namespace npk
