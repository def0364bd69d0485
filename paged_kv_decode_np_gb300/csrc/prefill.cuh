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

// floats of one partial: m[BM], l[BM], O[D/4][BM][4]
__host__ __device__ inline size_t prefill_part_floats(int bm, int d) { return (size_t)bm * (d + 2); }

struct PrefillRow {
  int32_t q0;  // first chunk token in q and out
  int32_t n;   // chunk tokens
  int32_t c;   // context, the chunk included
};

// Row r's chunk and context, clamped into what the arrays hold.
__device__ __forceinline__ PrefillRow prefill_row(const PrefillParams& p, int r, bool flag = false) {
  PrefillRow g;
  const int32_t a = p.query_starts[r], b = p.query_starts[r + 1];
  const int64_t cap = (int64_t)p.max_blocks_per_row * p.block_size;
  int32_t c = p.context_lens[r];
  const int32_t a2 = min(max(a, 0), p.tokens);
  const int32_t b2 = min(max(b, a2), p.tokens);
  if (flag && (a2 != a || b2 != b)) set_flag(p.err, NP_FLAG_QUERY);
  if (c < 0 || c > cap) {
    if (flag) set_flag(p.err, NP_FLAG_CONTEXT);
    c = c < 0 ? 0 : (int32_t)cap;
  }
  g.q0 = a2;
  g.n = b2 - a2;
  g.c = c;
  return g;
}

__device__ __forceinline__ int prefill_units(const PrefillParams& p, int n) {
  const int u = p.tile_tokens * p.tiles;
  return n / u + (n % u != 0);
}

// positions [0, end) are seen by the first `tok` chunk tokens
__device__ __forceinline__ int prefill_end(const PrefillRow& g, int64_t tok) {
  const int64_t e = (int64_t)g.c - g.n + (tok < g.n ? tok : g.n);
  return e < 0 ? 0 : (int)e;
}

// kv tiles of the first `tok` chunk tokens (at least one: a unit that sees
// nothing still has its zeros to write)
__device__ __forceinline__ int prefill_kv_tiles(const PrefillParams& p, const PrefillRow& g,
                                                int64_t tok) {
  const int e = prefill_end(g, tok);
  const int nk = e / p.bn + (e % p.bn != 0);
  return nk < 1 ? 1 : nk;
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

  __device__ __forceinline__ void start(const PrefillParams& p, int cta) {
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
  __device__ __forceinline__ bool next(const PrefillParams& p) {
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
  __device__ __forceinline__ void advance() {
    off = 0;
    ++m;
  }
  __device__ __forceinline__ bool whole() const { return kv0 == 0 && kv1 == nk; }
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
