// block_map.cu -- np_block_map: block tables, slots, positions and query starts
// of a batch from its requests' lengths.
//
// Per row: kept positions b = min(c, kept), c' = b + n, have = ceil(c / bs), need =
// ceil(c' / bs).  The free list is a stack: everything freed is put on its end
// first, then what is needed is taken from its end, both at places that prefix
// sums over the rows give, so no row waits for another and no atomics decide
// who gets which block.
//
// Bound: latency (a few KB).  One block of 1024 threads scans the rows (up to
// four a thread) and moves the blocks; the moves and the tokens are dealt over
// the threads one by one, each finding its row by bisection of the prefix sums
// in shared memory, so that one long prompt among many rows is no thread's
// alone.
#include "host_checks.h"
#include "prefill.cuh"

namespace npk {

constexpr int kMapThreads = 1024;
constexpr int kMapMaxRows = 4096;
constexpr int kMapPer = kMapMaxRows / kMapThreads;  // rows of a thread

struct MapParams {
  int32_t* tables;
  int32_t* lens;
  const int32_t* fresh;
  const int32_t* kept;
  int32_t* list;
  int32_t* count;
  int32_t* starts;
  int64_t* slots;
  int32_t* positions;
  int32_t* err;
  int64_t num_blocks;
  int32_t rows, block_size, max_blocks, tokens;
  int32_t token_cap;  // num_tokens, or what int32 holds without a slot mapping
  int32_t apart;      // the tokens are a launch of their own
};

// the last i with a[i] <= x, of n + 1 ascending entries with a[0] = 0 <= x < a[n]
__device__ __forceinline__ int map_row(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) {
  return (int32_t)(((uint32_t)a + (uint32_t)b - 1u) / (uint32_t)b);  // a < 2^31, b < 2^31
}

// Slots and positions of tokens i0, i0 + stride, .. below `end`, of `tokens` in all: four
// at a time, their table entries on the way together.
__device__ __forceinline__ void map_tokens(const MapParams& p, const int32_t* tok, const int32_t* base,
                                           int32_t tokens, int i0, int stride, int end) {
#pragma unroll 1
  for (; i0 < end; i0 += 4 * stride) {
    int32_t pos[4], in[4], b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * stride;
      b[u] = -1;
      pos[u] = in[u] = 0;
      if (i < tokens && i < end) {
        const int r = map_row(tok, p.rows, i);
        pos[u] = base[r] + (i - tok[r]);
        const int32_t j = (int32_t)((uint32_t)pos[u] / (uint32_t)p.block_size);
        in[u] = pos[u] - j * p.block_size;
        b[u] = p.tables[(int64_t)r * p.max_blocks + j];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * stride;
      if (i >= end) break;
      const bool good = b[u] >= 0 && b[u] < p.num_blocks;
      if (i < tokens && !good) set_flag(p.err, NP_FLAG_BLOCK_ID);
      p.slots[i] = good ? (int64_t)b[u] * p.block_size + in[u] : -1;
      if (p.positions) p.positions[i] = pos[u];
    }
  }
}

struct MapSum {
  int64_t tok, take, back;
  __device__ __forceinline__ MapSum operator+(const MapSum& o) const {
    return {tok + o.tok, take + o.take, back + o.back};
  }
};

__device__ __forceinline__ MapSum map_shfl_up(const MapSum& s, int o) {
  constexpr unsigned FULL = 0xffffffffu;
  return {__shfl_up_sync(FULL, s.tok, o), __shfl_up_sync(FULL, s.take, o),
          __shfl_up_sync(FULL, s.back, o)};
}

__global__ void __launch_bounds__(kMapThreads) block_map_kernel(const __grid_constant__ MapParams p) {
  extern __shared__ __align__(16) int32_t map_smem[];
  int32_t* tok = map_smem;                  // [rows + 1] new tokens before each row
  int32_t* take = tok + kMapMaxRows + 1;    // blocks taken before each row
  int32_t* back = take + kMapMaxRows + 1;   // blocks given back before each row
  int32_t* base = back + kMapMaxRows + 1;   // [rows] kept positions
  __shared__ MapSum warp_sum[kMapThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (p.rows + kMapThreads - 1) / kMapThreads;
  const int64_t cap = (int64_t)p.max_blocks * p.block_size;  // < 2^31
  int32_t have[kMapPer], keep[kMapPer], fresh[kMapPer];
  int flags = 0;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    have[i] = keep[i] = fresh[i] = 0;
    const int r = tid * per + i;
    if (i >= per || r >= p.rows) continue;
    int32_t c = p.lens[r], n = p.fresh[r], k = p.kept ? p.kept[r] : c;
    if (c < 0 || c > cap) {
      flags |= NP_FLAG_CONTEXT;
      c = c < 0 ? 0 : (int32_t)cap;
    }
    if (n < 0 || (p.kept && k < 0)) flags |= NP_FLAG_QUERY;
    n = max(n, 0);
    k = min(max(k, 0), c);
    if (n > cap - k) {
      flags |= NP_FLAG_CONTEXT;
      n = 0;
    }
    have[i] = ceil_div(c, p.block_size);
    keep[i] = k;
    fresh[i] = n;
  }
  int32_t held = p.count[0];
  if (held < 0 || held > p.num_blocks) {
    flags |= NP_FLAG_BLOCKS;
    held = held < 0 ? 0 : (int32_t)p.num_blocks;
  }

  // what row i of this thread adds to the sums
  auto of_row = [&](int i) -> MapSum {
    const int32_t d = ceil_div(keep[i] + fresh[i], p.block_size) - have[i];
    return {fresh[i], max(d, 0), max(-d, 0)};
  };
  // the sums before this thread's rows, and all rows'
  auto scan = [&](MapSum& all) -> MapSum {
    MapSum own{0, 0, 0};
#pragma unroll
    for (int i = 0; i < kMapPer; ++i) own = own + of_row(i);  // rows that are not there: 0
    MapSum x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const MapSum y = map_shfl_up(x, o);
      if (lane >= o) x = x + y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      MapSum y = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const MapSum z = map_shfl_up(y, o);
        if (lane >= o) y = y + z;
      }
      warp_sum[lane] = y;
    }
    __syncthreads();
    all = warp_sum[kMapThreads / 32 - 1];
    MapSum before{x.tok - own.tok, x.take - own.take, x.back - own.back};
    return warp > 0 ? before + warp_sum[warp - 1] : before;
  };

  MapSum all;
  MapSum at = scan(all);
  if (all.tok > p.token_cap || all.take > held + all.back) {  // uniform
    // Rows past the first that does not fit get nothing new: the sums with what
    // they wanted only grow.  (What they give back more for it comes on top of
    // what was counted on here.)
    MapSum run = at;
    bool drop[kMapPer];
#pragma unroll
    for (int i = 0; i < kMapPer; ++i) {
      run = run + of_row(i);
      const bool no = run.tok > p.token_cap, out = run.take > held + all.back;
      drop[i] = no || out;
      if (fresh[i] > 0) flags |= (no ? NP_FLAG_QUERY : 0) | (out ? NP_FLAG_BLOCKS : 0);
    }
#pragma unroll
    for (int i = 0; i < kMapPer; ++i)
      if (drop[i]) fresh[i] = 0;
    at = scan(all);
  }
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int r = tid * per + i;
    if (i < per && r < p.rows) {
      tok[r] = (int32_t)at.tok;
      take[r] = (int32_t)at.take;
      back[r] = (int32_t)at.back;
      base[r] = keep[i];
      p.starts[r] = (int32_t)at.tok;
      p.lens[r] = keep[i] + fresh[i];
    }
    at = at + of_row(i);
  }
  const int32_t tokens = (int32_t)all.tok, taken = (int32_t)all.take, given = (int32_t)all.back;
  // the list after what is put there; what has no room (a count that was wrong) is dropped
  const int64_t full = (int64_t)held + given;
  if (full > p.num_blocks) flags |= NP_FLAG_BLOCKS;
  int32_t top = (int32_t)min(full, p.num_blocks);
  if (tid == 0) {
    tok[p.rows] = tokens;
    take[p.rows] = taken;
    back[p.rows] = given;
    p.starts[p.rows] = tokens;
  }
  __syncthreads();
  auto need_of = [&](int r) { return ceil_div(base[r] + (tok[r + 1] - tok[r]), p.block_size); };
  bool lost = false;
  for (int32_t e = tid; e < given; e += kMapThreads) {
    const int r = map_row(back, p.rows, e);
    int32_t* t = p.tables + (int64_t)r * p.max_blocks + need_of(r) + (e - back[r]);
    const int64_t to = (int64_t)held + given - 1 - e;
    const int32_t b = *t;
    lost |= b < 0 || b >= p.num_blocks;
    if (to < p.num_blocks) p.list[to] = b;
    *t = -1;
  }
  if (__syncthreads_or(lost)) {
    // What is no block does not stay in the list: one warp moves the others up.
    if (lost) flags |= NP_FLAG_BLOCK_ID;
    __shared__ int32_t left;
    if (warp == 0) {
      int32_t to = held;
      for (int32_t i0 = held; i0 < top; i0 += 32) {  // (at most num_blocks of them)
        const int32_t i = i0 + lane, b = i < top ? p.list[i] : -1;
        const bool good = b >= 0 && b < p.num_blocks;
        const unsigned m = __ballot_sync(0xffffffffu, good);  // every lane has read its entry
        if (good) p.list[to + __popc(m & ((1u << lane) - 1u))] = b;
        to += __popc(m);
        __syncwarp();
      }
      if (lane == 0) left = to;
    }
    __syncthreads();
    top = left;
  }
  if (tid == 0) p.count[0] = max(top - taken, 0);
  for (int32_t e = tid; e < taken; e += kMapThreads) {
    const int r = map_row(take, p.rows, e);
    const int32_t n = take[r + 1] - take[r];
    const int32_t from = top - 1 - e;
    int32_t b = from >= 0 ? p.list[from] : -1;
    if (b < 0 || b >= p.num_blocks) {
      flags |= NP_FLAG_BLOCK_ID;
      b = -1;
    }
    p.tables[(int64_t)r * p.max_blocks + need_of(r) - n + (e - take[r])] = b;
  }
  if (flags) set_flag(p.err, flags);
  __syncthreads();
  if (!p.apart) map_tokens(p, tok, base, tokens, tid, kMapThreads, p.tokens);
}

// The tokens of long steps: kMapFill a block, from what the first launch left.
constexpr int kMapFill = 2048, kMapFillThreads = 512;

__global__ void __launch_bounds__(kMapFillThreads) block_map_fill_kernel(const __grid_constant__
                                                                         MapParams p) {
  extern __shared__ __align__(16) int32_t map_smem[];
  int32_t* tok = map_smem;                 // [rows + 1]
  int32_t* base = tok + kMapMaxRows + 1;   // [rows]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int r = threadIdx.x; r <= p.rows; r += kMapFillThreads) {
    tok[r] = p.starts[r];
    if (r < p.rows) base[r] = p.lens[r] - (p.starts[r + 1] - p.starts[r]);
  }
  __syncthreads();
  const int first = blockIdx.x * kMapFill;
  map_tokens(p, tok, base, tok[p.rows], first + (int)threadIdx.x, kMapFillThreads,
             min(p.tokens, first + kMapFill));
}

np_status launch_block_map(MapParams& p, cudaStream_t s) {
  constexpr size_t smem = (size_t)(4 * (kMapMaxRows + 1)) * 4;
  static unsigned long long allowed = 0;
  const np_status rc = allow_smem(block_map_kernel, smem, &allowed);
  if (rc != NP_OK) return rc;
  // Long steps' tokens over many blocks: us of a step and its undoing, 64 rows, one
  // launch / two: 2000 tokens 9.5 / 10.9, 4000 10.9 / 10.7, 8000 13.6 / 10.7, 18000 17.6 / 10.7.
  p.apart = p.tokens > 2 * kMapFill;
  block_map_kernel<<<1, kMapThreads, smem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return NP_ERR_CUDA;
  if (!p.apart) return NP_OK;
  constexpr size_t fill = (size_t)(2 * (kMapMaxRows + 1)) * 4;
  return launch_dependent(block_map_fill_kernel, (unsigned)((p.tokens + kMapFill - 1) / kMapFill), 1,
                          kMapFillThreads, fill, s, p);
}

}  // namespace npk

extern "C" np_status np_block_map_packed(const np_block_map_args* a) {
  using namespace npk;
  if (!a) return NP_ERR_INVALID_ARG;
  if (a->rows < 0 || a->num_tokens < 0 || a->block_size <= 0 || a->max_blocks_per_row <= 0 ||
      a->num_blocks <= 0)
    return NP_ERR_INVALID_ARG;
  int64_t cap = 0, tab = 0, slots = 0;
  if (!mul_fits(a->max_blocks_per_row, a->block_size, &cap) ||
      !mul_fits(a->num_blocks, a->block_size, &slots) ||
      !mul_fits(a->rows, (int64_t)a->max_blocks_per_row * 4, &tab))
    return NP_ERR_OUT_OF_RANGE;
  if (a->rows > kMapMaxRows || cap > INT32_MAX - 1024) return NP_ERR_UNSUPPORTED;
  // every block of every row's table has its number among 32-bit prefix sums, and every
  // block and token in loops that step past the last by less than 4096
  if ((int64_t)a->rows * a->max_blocks_per_row > INT32_MAX - 4096 || a->num_blocks > INT32_MAX - 4096 ||
      a->num_tokens > INT32_MAX - 4096)
    return NP_ERR_UNSUPPORTED;
  if (a->rows == 0 && a->num_tokens == 0) return NP_OK;
  if (!a->query_starts || !a->free_blocks || !a->free_count || (a->num_tokens > 0 && !a->slot_mapping) ||
      (a->num_tokens == 0 && a->slot_mapping) || (a->positions && !a->slot_mapping) ||
      (a->rows > 0 && (!a->block_tables || !a->context_lens || !a->new_lens)))
    return NP_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(a->block_tables), static_cast<const void*>(a->context_lens),
                        static_cast<const void*>(a->new_lens), static_cast<const void*>(a->kept_lens),
                        static_cast<const void*>(a->free_blocks), static_cast<const void*>(a->free_count),
                        static_cast<const void*>(a->query_starts), static_cast<const void*>(a->positions),
                        static_cast<const void*>(a->err_word)})
    if (!aligned_to(x, 4)) return NP_ERR_INVALID_ARG;
  if (!aligned_to(a->slot_mapping, 8)) return NP_ERR_INVALID_ARG;
  const int64_t row_bytes = 4ll * a->rows;
  const Span spans[] = {{a->block_tables, tab},          {a->context_lens, row_bytes},
                        {a->free_blocks, 4 * a->num_blocks}, {a->free_count, 4},
                        {a->query_starts, row_bytes + 4}, {a->slot_mapping, 8ll * a->num_tokens},
                        {a->positions, 4ll * a->num_tokens}, {a->new_lens, row_bytes},
                        {a->kept_lens == a->context_lens ? nullptr : a->kept_lens, row_bytes}};
  if (any_overlap(spans, 7)) return NP_ERR_INVALID_ARG;
  MapParams p{};
  p.tables = a->block_tables;
  p.lens = a->context_lens;
  p.fresh = a->new_lens;
  p.kept = a->kept_lens;
  p.list = a->free_blocks;
  p.count = a->free_count;
  p.starts = a->query_starts;
  p.slots = a->slot_mapping;
  p.positions = a->positions;
  p.err = a->err_word;
  p.num_blocks = a->num_blocks;
  p.rows = a->rows;
  p.block_size = a->block_size;
  p.max_blocks = a->max_blocks_per_row;
  p.tokens = a->num_tokens;
  p.token_cap = a->slot_mapping ? a->num_tokens : INT32_MAX;
  return launch_block_map(p, reinterpret_cast<cudaStream_t>(a->stream));
}

extern "C" np_status np_block_map(int32_t* block_tables, int32_t max_blocks_per_row,
                                  int32_t* context_lens, const int32_t* new_lens,
                                  const int32_t* kept_lens, int32_t rows, int32_t block_size,
                                  int32_t* free_blocks, int32_t* free_count, int64_t num_blocks,
                                  int32_t* query_starts, int64_t* slot_mapping, int32_t* positions,
                                  int32_t num_tokens, int32_t* err_word, np_stream_t stream) {
  np_block_map_args a{};
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.new_lens = new_lens;
  a.kept_lens = kept_lens;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.query_starts = query_starts;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.err_word = err_word;
  a.stream = stream;
  a.num_blocks = num_blocks;
  a.max_blocks_per_row = max_blocks_per_row;
  a.rows = rows;
  a.block_size = block_size;
  a.num_tokens = num_tokens;
  return np_block_map_packed(&a);
}
