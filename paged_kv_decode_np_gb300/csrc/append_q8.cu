// append_q8.cu -- np_kv_append_q8: new tokens' K and V rounded into the 8-bit
// pools, with one power-of-two scale per (block of tokens, kv head).
//
// A run is the call's tokens of one block, side by side in the slot mapping.
// For a run, a kv head and K or V:
//   A  = max |x|,  e = least with A <= QMAX 2^e
//   e' = e where the run holds the block's first slot, else max(e_old, e)
//   older codes of the block: rne(code 2^(e_old - e')) where e' > e_old
//   new codes: rne(x 2^-e')
// One warp does that: it reads the run's values (a 16-byte vector a lane and
// step), keeps them in registers where they fit (32 tokens of 128 bf16 dims),
// takes the maximum, and writes the codes.  No two warps touch the same block
// and head, so there is nothing to wait for and nothing atomic.
//
// Bound: the chain of a run's loads, maximum, scale and stores; enough runs side by side
// reach half of the copy rate (16384 tokens, 8 heads of 128, bf16, blocks of 32: 28 us as
// calls, 3.6 TB/s; 22.4 replayed, when L2 still holds part of it), decode batches are latency
// (64 tokens 2.7 us where no scale grows, 256 3.9).  Where one grows, the block's other slots
// are read, rounded and written one by one: with 6 % of a decode batch's (block, head) pairs,
// about what its steps have, 64 tokens take 8.6 us in blocks of 16 and 26 in blocks of 64.  A
// block of the grid takes `window` tokens: every warp finds by itself which of them begin runs, and
// they deal out (run, head, K or V).  The first token's values are on their way before the
// run's length is known.  (A shared list of the runs, 16 tokens in registers and the rest one by
// one: 32, 3.5 and 7.4 us.)
#include "cache8.cuh"
#include "decode_launch.h"
#include "host_checks.h"

namespace npk {

constexpr int kAppend8Warps = 8;

struct Append8Params {
  uint8_t* pool[2];
  float* scale[2];
  const void* src[2];
  int64_t stride[2];  // elements between tokens
  const int64_t* slots;
  int32_t* err;
  int64_t num_slots;
  int32_t block_size, kv_heads, tokens, window;
};

__device__ __forceinline__ int64_t block_of(const Append8Params& p, int64_t slot) {
  return p.num_slots <= 0x7fffffffll ? (int64_t)((uint32_t)slot / (uint32_t)p.block_size)
                                     : slot / p.block_size;
}

// The largest |x| of a vector joins `top`, as bits (bf16: two at a time); what is not
// finite is past any number.
template <typename T>
__device__ __forceinline__ uint32_t largest(uint32_t top, const uint4& r) {
  for (uint32_t w : {r.x, r.y, r.z, r.w}) {
    if constexpr (sizeof(T) == 2) top = __vmaxu2(top, w & 0x7fff7fffu);
    else top = max(top, w & 0x7fffffffu);
  }
  return top;
}

template <typename T, int D, int FORM, int STEPS>
__device__ __forceinline__ void append8_run(const Append8Params& p, int t0, int h, int kv, int lane) {
  constexpr unsigned FULL = 0xffffffffu;
  using F = Form8<FORM>;
  constexpr int V = 16 / (int)sizeof(T);         // values of a vector
  constexpr int LT = D / V;                      // lanes of a token (2 to 64)
  constexpr int PT = LT <= 32 ? 1 : LT / 32;     // vectors of a lane and token
  constexpr int TP = LT <= 32 ? 32 / LT : 1;     // tokens of a step
  constexpr int U = STEPS / PT;                  // steps whose values stay in registers
  const int sub = LT <= 32 ? lane / LT : 0;
  const int col = (LT <= 32 ? lane % LT : lane) * V;

  const T* src = static_cast<const T*>(p.src[kv]) + (int64_t)h * D + col;
  const int64_t stride = p.stride[kv];
  uint4 held[U][PT];
  auto load = [&](int i, int n, uint4* r) {  // token i + sub, of n
#pragma unroll
    for (int k = 0; k < PT; ++k)
      r[k] = i + sub < n
                 ? *reinterpret_cast<const uint4*>(src + (t0 + i + sub) * stride + k * 32 * V)
                 : make_uint4(0u, 0u, 0u, 0u);
  };
  load(0, p.tokens - t0, held[0]);  // (before it is known whose they are)

  // the run's length, and whether it holds the block's first slot
  const int64_t blk = block_of(p, p.slots[t0]), start = blk * p.block_size;
  float* sp = p.scale[kv] + blk * p.kv_heads + h;
  const int e_old = scale_exp(__float_as_uint(*sp));
  int n = 0;
  bool anew = false;
#pragma unroll 1
  for (int i0 = 0;; i0 += 32) {
    const int64_t s = t0 + i0 + lane < p.tokens ? p.slots[t0 + i0 + lane] : -1;
    const bool in = s >= start && s < start + p.block_size && s < p.num_slots;
    const unsigned m = __ballot_sync(FULL, in);
    const int run = m == FULL ? 32 : __ffs(~m) - 1;
    anew |= __any_sync(FULL, in && lane < run && s == start);
    n += run;
    if (run < 32) break;
  }
#pragma unroll
  for (int u = 1; u < U; ++u)
    if (u * TP < n) load(u * TP, n, held[u]);
  if (sub >= n) {
#pragma unroll
    for (int k = 0; k < PT; ++k) held[0][k] = make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * TP < n) {
#pragma unroll
      for (int k = 0; k < PT; ++k) top = largest<T>(top, held[u][k]);
    }
  // (runs that do not fit are read in batches, and again for their codes: from L2)
  auto batches = [&](auto use) {
#pragma unroll 1
    for (int i = U * TP; i < n; i += 4 * TP) {
      uint4 r[4][PT];
#pragma unroll
      for (int u = 0; u < 4; ++u) load(i + u * TP, n, r[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) use(i + u * TP, r[u]);
    }
  };
  batches([&](int, const uint4* r) {
#pragma unroll
    for (int k = 0; k < PT; ++k) top = largest<T>(top, r[k]);
  });
  if constexpr (sizeof(T) == 2) top = max(top << 16, top & 0xffff0000u);
  top = __reduce_max_sync(FULL, top);
  auto widen = [&](const uint4& r, float* x) {
    Storage<T>::template load<V>(reinterpret_cast<const T*>(&r), x);
  };
  if (top >= 0x7f800000u) {  // something is not finite: the largest of what is
    if (lane == 0) set_flag(p.err, NP_FLAG_VALUE);
    top = 0;
#pragma unroll 1
    for (int i = 0; i < n; i += TP) {
      uint4 r[PT];
      load(i, n, r);
#pragma unroll
      for (int k = 0; k < PT; ++k) {
        float x[V];
        widen(r[k], x);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const uint32_t a = __float_as_uint(x[e]) & 0x7fffffffu;
          if (a < 0x7f800000u) top = max(top, a);
        }
      }
    }
    top = __reduce_max_sync(FULL, top);
  }
  int e = top < 0x00800000u ? kScaleMin : min(max(F::need(top), kScaleMin), kScaleMax);
  if (!anew) e = max(e, e_old);

  uint8_t* pool = p.pool[kv] + (int64_t)h * D;
  const int64_t row = (int64_t)p.kv_heads * D;  // bytes of a slot, all heads
  if (!anew && e > e_old) {
    // the codes of the block's other slots, to the new scale
    const float f = pow2f(max(e_old - e, -126));
#pragma unroll 1
    for (int o = 0; o < p.block_size; ++o) {
      bool mine = false;  // written by this run
      for (int i = lane; i < n; i += 32) mine |= p.slots[t0 + i] == start + o;
      if (__any_sync(FULL, mine)) continue;
      uint8_t* at = pool + (start + o) * row;
      for (int d = 4 * lane; d < D; d += 128) {
        float x[4];
        widen8x4<FORM>(*reinterpret_cast<const uint32_t*>(at + d), x);
        *reinterpret_cast<uint32_t*>(at + d) =
            F::code2(x[0] * f, x[1] * f) | (F::code2(x[2] * f, x[3] * f) << 16);
      }
    }
  }
  if (lane == 0) *sp = pow2f(e);

  const float f = pow2f(-e);
  auto store = [&](int i, const uint4* r) {
    if (i + sub >= n) return;
    uint8_t* at = pool + p.slots[t0 + i + sub] * row + col;
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      float x[V];
      widen(r[k], x);
      uint32_t w[V / 4];
#pragma unroll
      for (int q = 0; q < V / 4; ++q)
        w[q] = F::code2(x[4 * q] * f, x[4 * q + 1] * f) | (F::code2(x[4 * q + 2] * f, x[4 * q + 3] * f) << 16);
      if constexpr (V == 8) *reinterpret_cast<uint2*>(at + k * 32 * V) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(at + k * 32 * V) = w[0];
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * TP < n) store(u * TP, held[u]);
  batches(store);
}

template <typename T, int D, int FORM, int STEPS>
__global__ void __launch_bounds__(32 * kAppend8Warps, STEPS == 16 ? 2 : STEPS == 8 ? 3 : 4) append8_kernel(const __grid_constant__
                                                                     Append8Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // which of this block's tokens begin a run: every warp looks for itself
  const int t = blockIdx.x * p.window + lane;
  const bool live = lane < p.window && t < p.tokens;
  const int64_t s = live ? p.slots[t] : -1;
  const int64_t before = live && t > 0 ? p.slots[t - 1] : -1;
  if (s >= p.num_slots && blockIdx.y == 0 && warp == 0) set_flag(p.err, NP_FLAG_SLOT);
  const bool in = s >= 0 && s < p.num_slots;
  const bool joined = before >= 0 && before < p.num_slots && in && block_of(p, before) == block_of(p, s);
  unsigned leads = __ballot_sync(0xffffffffu, in && !joined);
  const int per = 2 * p.kv_heads, step = gridDim.y * kAppend8Warps;
  const int tasks = __popc(leads) * per;
  int at = 0;  // the run of the lowest bit of `leads`
  for (int i = blockIdx.y * kAppend8Warps + warp; i < tasks; i += step) {
    const int x = i / per, rest = i - x * per;
    for (; at < x; ++at) leads &= leads - 1;
    // neighbouring warps: neighbouring heads of the same tokens
    const int kv = rest >= p.kv_heads ? 1 : 0;
    append8_run<T, D, FORM, STEPS>(p, blockIdx.x * p.window + __ffs(leads) - 1, rest - kv * p.kv_heads, kv, lane);
  }
}

template <typename T, int D, int FORM, int STEPS>
static np_status launch_append8(Append8Params& p, cudaStream_t s) {
  // few tokens: few of them a block, so that all warps find work.  us of 16384 tokens with
  // 4, 8, 16, 32 a block: 39, 29, 25, 22; of 2000 tokens with 4, 8, 16: 8.3, 6.2, 7.2.
  p.window = p.tokens >= 4096 ? 32 : p.tokens >= 512 ? 8 : 1;
  const unsigned x = (unsigned)((p.tokens + p.window - 1) / p.window);
  const int tasks = 2 * p.kv_heads;  // of one run
  unsigned y = (unsigned)((tasks + kAppend8Warps - 1) / kAppend8Warps);
  if (y > 64) y = 64;
  append8_kernel<T, D, FORM, STEPS><<<dim3(x, y), 32 * kAppend8Warps, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? NP_OK : NP_ERR_CUDA;
}

// How many steps of a run's values stay in registers: those of a whole block, 8 or 16;
// few tokens (decode batches) are mostly runs of one.  us, 8 / 16 steps: 16000 tokens in
// blocks of 16 22.0 / 29.4, of 64 over 30 / 24.6; 256 rows 2 / 16 steps 3.9 / 7.4.
template <typename T, int D, int FORM>
static np_status launch_append8_steps(Append8Params& p, cudaStream_t s) {
  if (p.tokens < 512) return launch_append8<T, D, FORM, 2>(p, s);
  return (int64_t)p.block_size * D * (int)sizeof(T) > 8 * 512 ? launch_append8<T, D, FORM, 16>(p, s)
                                                              : launch_append8<T, D, FORM, 8>(p, s);
}

template <typename T, int FORM>
static np_status launch_append8_dim(Append8Params& p, int32_t d, cudaStream_t s) {
  switch (d) {
    case 16: return launch_append8_steps<T, 16, FORM>(p, s);
    case 32: return launch_append8_steps<T, 32, FORM>(p, s);
    case 64: return launch_append8_steps<T, 64, FORM>(p, s);
    case 128: return launch_append8_steps<T, 128, FORM>(p, s);
    case 256: return launch_append8_steps<T, 256, FORM>(p, s);
  }
  return NP_ERR_UNSUPPORTED;
}

}  // namespace npk

extern "C" np_status np_kv_append_q8_packed(const np_kv_append_q8_args* a) {
  using namespace npk;
  if (!a) return NP_ERR_INVALID_ARG;
  const int es = a->dtype == NP_F32 ? 4 : (a->dtype == NP_BF16 ? 2 : 0);
  if (es == 0 || (a->form != NP_E4M3 && a->form != NP_INT8)) return NP_ERR_UNSUPPORTED;
  const int d = a->head_dim;
  if (a->num_blocks <= 0 || a->block_size <= 0 || a->kv_heads <= 0 || a->num_tokens < 0 || d <= 0)
    return NP_ERR_INVALID_ARG;
  if (d != 16 && d != 32 && d != 64 && d != 128 && d != 256) return NP_ERR_UNSUPPORTED;
  if (a->kv_heads > 4096) return NP_ERR_UNSUPPORTED;  // far above any model's
  if (a->num_tokens > INT32_MAX - 4096) return NP_ERR_UNSUPPORTED;  // loops step past the last
  const int64_t row = (int64_t)a->kv_heads * d;
  int64_t slots = 0, pool = 0, scales = 0, kn = 0, vn = 0;
  if (!mul_fits(a->num_blocks, a->block_size, &slots) || !mul_fits(slots, row, &pool) ||
      !mul_fits(a->num_blocks, 4ll * a->kv_heads, &scales))
    return NP_ERR_OUT_OF_RANGE;
  if (a->num_tokens == 0) return NP_OK;
  if (a->k_stride < 0 || a->v_stride < 0) return NP_ERR_INVALID_ARG;
  if (!mul_fits(a->num_tokens - 1, a->k_stride, &kn) || !mul_fits(a->num_tokens - 1, a->v_stride, &vn) ||
      !mul_fits(kn, es, &kn) || !mul_fits(vn, es, &vn))
    return NP_ERR_OUT_OF_RANGE;
  kn += row * es;
  vn += row * es;
  if (!a->k_pool || !a->v_pool || !a->k_scale || !a->v_scale || !a->k_new || !a->v_new || !a->slot_mapping)
    return NP_ERR_INVALID_ARG;
  if (a->num_tokens > 1 && (a->k_stride < row || a->k_stride * es % 16 != 0 || a->v_stride < row ||
                            a->v_stride * es % 16 != 0))
    return NP_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(a->k_pool), static_cast<const void*>(a->v_pool), a->k_new,
                        a->v_new})
    if (!aligned_to(x, 16)) return NP_ERR_INVALID_ARG;
  if (!aligned_to(a->k_scale, 4) || !aligned_to(a->v_scale, 4) || !aligned_to(a->slot_mapping, 8) ||
      !aligned_to(a->err_word, 4))
    return NP_ERR_INVALID_ARG;
  const Span spans[] = {{a->k_pool, pool}, {a->v_pool, pool}, {a->k_scale, scales}, {a->v_scale, scales},
                        {a->k_new, kn},    {a->v_new, vn},    {a->slot_mapping, 8ll * a->num_tokens}};
  if (any_overlap(spans, 4)) return NP_ERR_INVALID_ARG;
  Append8Params p{};
  p.pool[0] = static_cast<uint8_t*>(a->k_pool);
  p.pool[1] = static_cast<uint8_t*>(a->v_pool);
  p.scale[0] = a->k_scale;
  p.scale[1] = a->v_scale;
  p.src[0] = a->k_new;
  p.src[1] = a->v_new;
  p.stride[0] = a->k_stride;
  p.stride[1] = a->v_stride;
  p.slots = a->slot_mapping;
  p.err = a->err_word;
  p.num_slots = slots;
  p.block_size = a->block_size;
  p.kv_heads = a->kv_heads;
  p.tokens = a->num_tokens;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(a->stream);
  if (a->form == NP_E4M3)
    return a->dtype == NP_BF16 ? launch_append8_dim<__nv_bfloat16, NP_E4M3>(p, d, s)
                               : launch_append8_dim<float, NP_E4M3>(p, d, s);
  return a->dtype == NP_BF16 ? launch_append8_dim<__nv_bfloat16, NP_INT8>(p, d, s)
                             : launch_append8_dim<float, NP_INT8>(p, d, s);
}

extern "C" np_status np_kv_append_q8(void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                                     np_form8 form, int64_t num_blocks, int32_t block_size,
                                     int32_t kv_heads, int32_t head_dim, const void* k_new,
                                     const void* v_new, np_dtype dtype, int64_t k_stride,
                                     int64_t v_stride, const int64_t* slot_mapping, int32_t num_tokens,
                                     int32_t* err_word, np_stream_t stream) {
  np_kv_append_q8_args a{};
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_new = k_new;
  a.v_new = v_new;
  a.slot_mapping = slot_mapping;
  a.err_word = err_word;
  a.stream = stream;
  a.num_blocks = num_blocks;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.form = form;
  a.dtype = dtype;
  a.block_size = block_size;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.num_tokens = num_tokens;
  return np_kv_append_q8_packed(&a);
}
