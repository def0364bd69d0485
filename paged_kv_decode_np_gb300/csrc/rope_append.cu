// rope_append.cu -- np_rope_append: the new tokens' q and k are normalised
// per head (optional), rotated by their positions, and q goes to its buffer
// while k and v go to the tokens' slots of the paged pools: one pass.
//
// For a head row x in R^D with weight w and pairs (x0, x1)_j, j < rot/2:
//   x  <- x * w / sqrt(mean(x^2) + eps)                  (rows with a weight)
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin           (angle of pair j at
//                                                         the position of its axis)
// Everything is fp32; a result is rounded to the storage type once, at its
// store.
//
// Bound: HBM (each q, k, v element is read once and written once; ~10
// operations per element).  So the layout is chosen for wide accesses: a
// thread owns two 16-byte vectors of a head -- with pairs in halves, dims
// [j, j+V) and [j + rot/2, +V); with interleaved pairs, 2V consecutive dims;
// past rot_dim, 2V consecutive dims that pass through -- so both members of
// each of its V pairs are in its registers and no exchange is needed.  The
// D / 2V threads of a head (1 to 32, a power of two) add their squares with
// xor-shuffles.  A thread keeps its V cosines and sines in registers and
// walks over the token's heads with them, two heads' loads in flight.
#include <math.h>

#include "decode_launch.h"
#include "np_common.cuh"

namespace npk {

constexpr int kRopeMaxAxes = 4;
constexpr int kRopeThreads = 256;

struct RopeParams {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  void* k_pool;
  void* v_pool;
  const int64_t* slots;
  const int32_t* positions;  // [axes, tokens]
  const float* table;        // [max_positions, rot]: cosines, then sines
  const void* q_weight;
  const void* k_weight;
  int32_t* err;
  int64_t num_slots;
  int32_t tokens, q_heads, kv_heads;
  int32_t rot, max_positions, axes, interleaved;
  int32_t section_end[kRopeMaxAxes];  // first pair past each axis' section
  float eps;
  int32_t head_lanes;        // heads a token's threads take at a time
  int32_t block_tokens;      // tokens per block
};

// position of axis a of token t, clamped into the table
__device__ __forceinline__ int32_t rope_position(const RopeParams& p, int a, int64_t t) {
  int32_t x = p.positions[(int64_t)a * p.tokens + t];
  if (x < 0 || x >= p.max_positions) {
    set_flag(p.err, NP_FLAG_POSITION);
    x = x < 0 ? 0 : p.max_positions - 1;
  }
  return x;
}

template <typename T, int D, bool NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__
                                                                   RopeParams p) {
  constexpr int V = 16 / (int)sizeof(T);  // elements per vector
  constexpr int TPH = D / (2 * V);        // threads per head
  constexpr unsigned FULL = 0xffffffffu;
  using S = Storage<T>;
  const int per_token = TPH * p.head_lanes;
  const int tl = threadIdx.x / per_token;  // token within the block
  const int i = threadIdx.x - tl * per_token;
  const int part = i % TPH;                // which 2V dims of a head
  const int hl = i / TPH;                  // first head
  const int64_t t = (int64_t)blockIdx.x * p.block_tokens + tl;
  const bool live = tl < p.block_tokens && t < p.tokens;
  const int heads = p.q_heads + 2 * p.kv_heads;

  // dims of the thread's two vectors, and its first pair (-1: pass through)
  const int half = p.rot >> 1;
  int da, db, pair;
  if (part * V >= half) {
    da = part * 2 * V;
    db = da + V;
    pair = -1;
  } else if (p.interleaved) {
    da = part * 2 * V;
    db = da + V;
    pair = part * V;
  } else {
    da = part * V;
    db = da + half;
    pair = da;
  }

  const int64_t slot = live ? p.slots[t] : -1;
  if (live && slot >= p.num_slots && i == 0) set_flag(p.err, NP_FLAG_SLOT);
  const bool keep = slot >= 0 && slot < p.num_slots;

  // source and destination of head h (q heads, then k, then v): false where
  // nothing is read or written
  auto where = [&](int h, const T*& src, T*& dst) -> bool {
    if (!live || h >= heads) return false;
    if (h < p.q_heads) {
      src = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)h * D;
      dst = static_cast<T*>(p.q_out) + (t * p.q_heads + h) * D;
      return true;
    }
    if (!keep) return false;
    const bool isv = h >= p.q_heads + p.kv_heads;
    const int hk = h - p.q_heads - (isv ? p.kv_heads : 0);
    src = isv ? static_cast<const T*>(p.v) + t * p.v_stride : static_cast<const T*>(p.k) + t * p.k_stride;
    src += (int64_t)hk * D;
    dst = static_cast<T*>(isv ? p.v_pool : p.k_pool) + (slot * p.kv_heads + hk) * D;
    return true;
  };

  float c[V], s[V];
  if (live && pair >= 0) {
    if (p.axes == 1) {
      const float* row = p.table + (int64_t)rope_position(p, 0, t) * p.rot + pair;
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        Storage<float>::load<4>(row + e, c + e);
        Storage<float>::load<4>(row + half + e, s + e);
      }
    } else {
      int a = 0;
      while (pair >= p.section_end[a]) ++a;  // section_end[axes - 1] == half > pair
      const float* row = p.table + (int64_t)rope_position(p, a, t) * p.rot;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (pair + e >= p.section_end[a]) {
          while (pair + e >= p.section_end[a]) ++a;
          row = p.table + (int64_t)rope_position(p, a, t) * p.rot;
        }
        c[e] = row[pair + e];
        s[e] = row[half + pair + e];
      }
    }
  }

  auto finish = [&](int h, const uint4 (&raw)[2], T* dst, bool on) {
    if (h >= p.q_heads + p.kv_heads) {  // v: the bits as they are
      if (on) {
        *reinterpret_cast<uint4*>(dst + da) = raw[0];
        *reinterpret_cast<uint4*>(dst + db) = raw[1];
      }
      if (!NORM) return;
    }
    float x[2 * V];
    S::template load<V>(reinterpret_cast<const T*>(&raw[0]), x);
    S::template load<V>(reinterpret_cast<const T*>(&raw[1]), x + V);
    if (NORM) {
      // the whole warp takes part: a head's lanes are aligned to TPH
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) sq = fmaf(x[e], x[e], sq);
#pragma unroll
      for (int o = TPH / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(FULL, sq, o);
      if (h >= p.q_heads + p.kv_heads) return;
      const void* w = h < p.q_heads ? p.q_weight : p.k_weight;
      if (on && w != nullptr) {
        const float r = 1.f / sqrtf(sq * (1.f / D) + p.eps);
        float wv[2 * V];
        S::template load<V>(static_cast<const T*>(w) + da, wv);
        S::template load<V>(static_cast<const T*>(w) + db, wv + V);
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) x[e] = x[e] * r * wv[e];
      }
    }
    if (!on) return;
    if (pair >= 0) {
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x0 = x[2 * e], x1 = x[2 * e + 1];
          x[2 * e] = x0 * c[e] - x1 * s[e];
          x[2 * e + 1] = x1 * c[e] + x0 * s[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float x0 = x[e], x1 = x[V + e];
          x[e] = x0 * c[e] - x1 * s[e];
          x[V + e] = x1 * c[e] + x0 * s[e];
        }
      }
    }
    S::template store<V>(dst + da, x);
    S::template store<V>(dst + db, x + V);
  };

  // Two heads at a time, both loaded before either is stored (q_out may be q).
  // The trip count is the block's, so every lane reaches the shuffles.
  for (int h0 = 0; h0 < heads; h0 += 2 * p.head_lanes) {
    const int ha = h0 + hl, hb = ha + p.head_lanes;
    const T *sa = nullptr, *sb = nullptr;
    T *oa = nullptr, *ob = nullptr;
    const bool na = where(ha, sa, oa), nb = where(hb, sb, ob);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 xa[2] = {zero, zero}, xb[2] = {zero, zero};
    if (na) {
      xa[0] = *reinterpret_cast<const uint4*>(sa + da);
      xa[1] = *reinterpret_cast<const uint4*>(sa + db);
    }
    if (nb) {
      xb[0] = *reinterpret_cast<const uint4*>(sb + da);
      xb[1] = *reinterpret_cast<const uint4*>(sb + db);
    }
    finish(ha, xa, oa, na);
    finish(hb, xb, ob, nb);
  }
}

template <typename T, int D>
static np_status launch_rope(RopeParams& p, cudaStream_t stream) {
  constexpr int TPH = D / (2 * (16 / (int)sizeof(T)));
  const int heads = p.q_heads + 2 * p.kv_heads;
  // Threads of a block.  Few tokens: a token's heads side by side, so that a
  // call is one round of loads (64 tokens of 48 heads of 128 bf16 dims: 2.6 us
  // with 256 threads, 3.4 with 64, 5.0 with 32).  Many: one warp a token, which
  // walks its heads with the token's cosines, sines, slot and position read
  // once by few threads (16384 tokens of 80 heads: 102 us, 6.6 TB/s, with 32;
  // 114 with 128; 136 with 256).  At the borders, us with 32 / 128 / 256 threads,
  // bf16, 128 dims, 80 heads: 511 tokens 12.5 / 7.1 / 6.6, 1000 14.0 / 9.7 / 11.2,
  // 2048 18.4 / 17.2 / 20.4, 4096 29.2 / 32.0 / 37.7; 10 heads: 511 3.2 / 2.7 / 2.8,
  // 2048 5.3 / 6.0 / 6.3, 4096 6.8 / 9.3 / 9.6; with norms, 80 heads: 2048 21.3 /
  // 21.7 / 32.1, 16384 123 / 145 / 236 (86 registers: 23 blocks of a warp an SM).
  // Three heads leave lanes idle in a warp a token: 2048 3.1 / 2.7 / 2.9, 16384
  // 13.1 / 11.2 / 12.2, where 128 threads would be right.
  const int cap = p.tokens >= 2048 ? 32 : (p.tokens >= 512 ? 128 : kRopeThreads);
  // heads a token's threads take at a time: all of them in the fewest equal
  // rounds that fit a block
  const int most = cap / TPH;
  const int rounds = (heads + most - 1) / most;
  p.head_lanes = (heads + rounds - 1) / rounds;
  const int per_token = TPH * p.head_lanes;
  p.block_tokens = cap / per_token;
  if (p.block_tokens > p.tokens) p.block_tokens = p.tokens;
  const int threads = (p.block_tokens * per_token + 31) / 32 * 32;
  const unsigned blocks = (unsigned)(((int64_t)p.tokens + p.block_tokens - 1) / p.block_tokens);
  if (p.q_weight || p.k_weight)
    rope_append_kernel<T, D, true><<<blocks, threads, 0, stream>>>(p);
  else
    rope_append_kernel<T, D, false><<<blocks, threads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? NP_OK : NP_ERR_CUDA;
}

template <typename T>
static np_status launch_rope_dim(RopeParams& p, int32_t head_dim, cudaStream_t stream) {
  switch (head_dim) {
    case 16: return launch_rope<T, 16>(p, stream);
    case 32: return launch_rope<T, 32>(p, stream);
    case 64: return launch_rope<T, 64>(p, stream);
    case 128: return launch_rope<T, 128>(p, stream);
    case 256: return launch_rope<T, 256>(p, stream);
  }
  return NP_ERR_UNSUPPORTED;
}

}  // namespace npk

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// a*b without int64 overflow (a, b >= 0)
bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

// [p, p + n) and [q, q + m) share a byte
bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

}  // namespace

extern "C" np_status np_rope_append(
    void* q_out, const void* q, const void* k_new, const void* v_new, int64_t q_stride,
    int64_t k_stride, int64_t v_stride, const int64_t* slot_mapping, void* k_pool, void* v_pool,
    np_dtype dtype, int64_t num_blocks, int32_t block_size, int32_t q_heads, int32_t kv_heads,
    int32_t head_dim, const float* cos_sin, int32_t max_positions, int32_t rot_dim,
    const int32_t* positions, int32_t num_axes, const int32_t* sections, int32_t interleaved,
    const void* q_weight, const void* k_weight, float eps, int32_t num_tokens, int32_t* err_word,
    np_stream_t stream) {
  const int es = dtype == NP_F32 ? 4 : (dtype == NP_BF16 ? 2 : 0);
  if (es == 0) return NP_ERR_UNSUPPORTED;
  if (num_blocks <= 0 || block_size <= 0 || q_heads < 0 || kv_heads <= 0 || num_tokens < 0 ||
      max_positions <= 0 || rot_dim <= 0 || num_axes <= 0 || head_dim <= 0 || !(eps >= 0.f) ||
      !isfinite(eps) || (interleaved != 0 && interleaved != 1))
    return NP_ERR_INVALID_ARG;
  if (head_dim != 16 && head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
    return NP_ERR_UNSUPPORTED;
  if (rot_dim > head_dim) return NP_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || num_axes > npk::kRopeMaxAxes) return NP_ERR_UNSUPPORTED;
  // heads per token: a block walks them; far above any model's
  if (q_heads > 4096 || kv_heads > 4096) return NP_ERR_UNSUPPORTED;
  npk::RopeParams p{};
  if (num_axes == 1 && !sections) {
    p.section_end[0] = rot_dim / 2;
  } else {
    if (!sections) return NP_ERR_INVALID_ARG;
    int64_t end = 0;
    for (int a = 0; a < num_axes; ++a) {
      if (sections[a] < 0) return NP_ERR_INVALID_ARG;
      end += sections[a];
      if (end > rot_dim / 2) return NP_ERR_INVALID_ARG;
      p.section_end[a] = (int32_t)end;
    }
    if (end != rot_dim / 2) return NP_ERR_INVALID_ARG;
  }
  const int64_t q_row = (int64_t)q_heads * head_dim, kv_row = (int64_t)kv_heads * head_dim;
  int64_t slots = 0, pool = 0, out_n = 0, qn = 0, kn = 0, vn = 0;
  if (!mul_ok(num_blocks, block_size, &slots) || !mul_ok(slots, kv_row * es, &pool))
    return NP_ERR_OUT_OF_RANGE;
  if (num_tokens == 0) return NP_OK;
  if (q_stride < 0 || k_stride < 0 || v_stride < 0) return NP_ERR_INVALID_ARG;
  if (!mul_ok(num_tokens, q_row * es, &out_n) || !mul_ok(num_tokens - 1, q_stride, &qn) ||
      !mul_ok(num_tokens - 1, k_stride, &kn) || !mul_ok(num_tokens - 1, v_stride, &vn) ||
      !mul_ok(qn, es, &qn) || !mul_ok(kn, es, &kn) || !mul_ok(vn, es, &vn))
    return NP_ERR_OUT_OF_RANGE;
  qn += q_row * es;
  kn += kv_row * es;
  vn += kv_row * es;
  if (!k_new || !v_new || !slot_mapping || !k_pool || !v_pool || !cos_sin || !positions)
    return NP_ERR_INVALID_ARG;
  if (q_heads > 0 ? (!q || !q_out) : (q || q_out || q_weight)) return NP_ERR_INVALID_ARG;
  // a token's row starts 16-byte aligned; rows do not run into one another
  if (num_tokens > 1 &&
      ((q_heads > 0 && (q_stride < q_row || q_stride * es % 16 != 0)) || k_stride < kv_row ||
       k_stride * es % 16 != 0 || v_stride < kv_row || v_stride * es % 16 != 0))
    return NP_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(q_out), q, k_new, v_new,
                        static_cast<const void*>(k_pool), static_cast<const void*>(v_pool),
                        static_cast<const void*>(cos_sin), q_weight, k_weight})
    if (x && !aligned(x, 16)) return NP_ERR_INVALID_ARG;
  if (!aligned(slot_mapping, 8) || !aligned(positions, 4) || (err_word && !aligned(err_word, 4)))
    return NP_ERR_INVALID_ARG;
  // what is written lies apart from what is read, but for q_out being q itself
  const bool in_place = q && q == q_out && (num_tokens == 1 || q_stride == q_row);
  if ((!in_place && overlap(q_out, out_n, q, qn)) || overlap(q_out, out_n, k_new, kn) ||
      overlap(q_out, out_n, v_new, vn))
    return NP_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(k_pool), static_cast<const void*>(v_pool)})
    if (overlap(x, pool, q, qn) || overlap(x, pool, k_new, kn) || overlap(x, pool, v_new, vn) ||
        overlap(x, pool, q_out, out_n))
      return NP_ERR_INVALID_ARG;
  if (overlap(k_pool, pool, v_pool, pool)) return NP_ERR_INVALID_ARG;

  p.q_out = q_out;
  p.q = q;
  p.k = k_new;
  p.v = v_new;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.slots = slot_mapping;
  p.positions = positions;
  p.table = cos_sin;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.err = err_word;
  p.num_slots = slots;
  p.tokens = num_tokens;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.rot = rot_dim;
  p.max_positions = max_positions;
  p.axes = num_axes;
  p.interleaved = interleaved;
  p.eps = eps;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == NP_BF16 ? npk::launch_rope_dim<__nv_bfloat16>(p, head_dim, st)
                          : npk::launch_rope_dim<float>(p, head_dim, st);
}

extern "C" np_status np_rope_append_packed(const np_rope_append_args* a) {
  if (!a) return NP_ERR_INVALID_ARG;
  return np_rope_append(a->q_out, a->q, a->k_new, a->v_new, a->q_stride, a->k_stride, a->v_stride,
                        a->slot_mapping, a->k_pool, a->v_pool, static_cast<np_dtype>(a->dtype),
                        a->num_blocks, a->block_size, a->q_heads, a->kv_heads, a->head_dim, a->cos_sin,
                        a->max_positions, a->rot_dim, a->positions, a->num_axes,
                        a->has_sections ? a->sections : nullptr, a->interleaved, a->q_weight,
                        a->k_weight, a->eps, a->num_tokens, a->err_word, a->stream);
}
