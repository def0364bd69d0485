// prefill_simt.cuh -- np_paged_prefill and np_paged_prefill_q8 on the FMA pipes: fp32
// at head_dim 256.  (Narrower heads: prefill_tc32.cu, whose tiles of 128 rows and 64 tokens do
// not fit in shared memory in three bf16 parts at this width.  Smaller ones
// would: 64 rows and 32 tokens, 192 KB; not built.)
//
// A unit is one tile of 64 (token, head) rows; a kv tile is 64 tokens.  256
// threads form S = Q K^T as 4 x 4 microtiles from shared memory (rows 4 ty +
// i, tokens tx + 16 j), run the online softmax with each row spread over the
// 16 lanes of its ty, and add P V as 4 rows x (D / 16) dims.  Everything is
// fp32.  Bound: the FMA pipes behind shared memory (8 16-byte reads for 64
// products); eight chunks of 71-184 tokens over 833-2031 positions, 8 / 1
// heads: 447 us, 27 TFLOP/s.
#pragma once

#include "cache8.cuh"
#include "prefill.cuh"

namespace npk {

constexpr int kSimtThreads = 256;
constexpr int kSimtRows = 64;
constexpr int kSimtBn = 64;

constexpr int kSimtD = 256;

struct SimtSmem {
  static constexpr int D = kSimtD;
  static constexpr int LD = D + 4;        // rows start on different banks
  static constexpr int LP = kSimtBn + 4;
  static constexpr size_t floats = (size_t)(kSimtRows + 2 * kSimtBn) * LD + (size_t)kSimtRows * LP;
  static constexpr size_t bytes = floats * 4 + kSimtBn * 8;
};

// FORM: the pools' 8-bit form, or -1 for fp32.
template <int FORM>
__global__ void __launch_bounds__(kSimtThreads, 1) prefill_simt_kernel(const __grid_constant__
                                                                       PrefillParams p) {
  using S = Storage<float>;
  using M = SimtSmem;
  constexpr int D = kSimtD;
  constexpr unsigned FULL = 0xffffffffu;
  constexpr int V = 4;        // values of an access
  constexpr int NG = D / 64;  // groups of 4 dims a thread owns: 4 tx + 64 j
  extern __shared__ __align__(16) unsigned char smem[];
  float* qs = reinterpret_cast<float*>(smem);
  float* ks = qs + kSimtRows * M::LD;
  float* vs = ks + kSimtBn * M::LD;
  float* ps = vs + kSimtBn * M::LD;
  int64_t* slot = reinterpret_cast<int64_t*>(ps + kSimtRows * M::LP);

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const float qscale = p.negate ? -p.qscale : p.qscale;
  const int G = p.group;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is complete
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may wait
  PrefillWalk w;
  w.start(p, blockIdx.x);
  while (w.next(p)) {
    // ---- q of the unit: row = token * G + head; rows past the chunk are zero
    const int tok0 = w.m * p.tile_tokens;
    __syncthreads();
    for (int e = threadIdx.x; e < kSimtRows * (D / V); e += kSimtThreads) {
      const int row = e / (D / V), d = (e % (D / V)) * V;
      const int tt = row / G, h = row % G;
      float x[V];
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = 0.f;
      if (tt < p.tile_tokens && tok0 + tt < w.g.n)
        S::template load<V>(static_cast<const float*>(p.q) +
                            ((int64_t)(w.g.q0 + tok0 + tt) * p.q_heads + w.kvh * G + h) * D + d,
                            x);
#pragma unroll
      for (int k = 0; k < V; ++k) qs[row * M::LD + d + k] = x[k];
    }
    // the last position each of this thread's rows sees
    int lim[4];
    float m_run[4], l_run[4], o[4][NG][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tt = (4 * ty + i) / G;
      lim[i] = tt < p.tile_tokens && tok0 + tt < w.g.n ? w.g.c - w.g.n + tok0 + tt : -1;
      m_run[i] = -INFINITY;
      l_run[i] = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }
    for (int kt = w.kv0; kt < w.kv1; ++kt) {
      const int t0 = kt * kSimtBn;
      __syncthreads();  // the last tile's readers are done
      if (threadIdx.x < kSimtBn) {
        const int64_t t = (int64_t)t0 + threadIdx.x;
        int64_t sl = -1;
        if (t < w.g.c) {
          const int64_t j = t / p.block_size;
          int64_t b = p.block_tables[(int64_t)w.r * p.max_blocks_per_row + j];
          if (b < 0 || b >= p.num_blocks) {
            set_flag(p.err, NP_FLAG_BLOCK_ID);
            b = 0;
          }
          sl = b * p.block_size + (t - j * p.block_size);
        }
        slot[threadIdx.x] = sl;
      }
      __syncthreads();
      for (int e = threadIdx.x; e < kSimtBn * (D / V); e += kSimtThreads) {
        const int row = e / (D / V), d = (e % (D / V)) * V;
        const int64_t sl = slot[row];
        float x[V], y[V];
#pragma unroll
        for (int k = 0; k < V; ++k) x[k] = y[k] = 0.f;
        if (sl >= 0) {
          const int64_t at = (sl * p.kv_heads + w.kvh) * D + d;
          if constexpr (FORM < 0) {
            Storage<float>::load<V>(static_cast<const float*>(p.k_pool) + at, x);
            Storage<float>::load<V>(static_cast<const float*>(p.v_pool) + at, y);
          } else {
            const int64_t sc = sl / p.block_size * p.kv_heads + w.kvh;
            const float a = pow2f(scale_exp(__float_as_uint(p.k_scale[sc])));
            const float b = pow2f(scale_exp(__float_as_uint(p.v_scale[sc])));
            widen8x4<FORM>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.k_pool) + at), x);
            widen8x4<FORM>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.v_pool) + at), y);
#pragma unroll
            for (int k = 0; k < V; ++k) {
              x[k] *= a;
              y[k] *= b;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
          ks[row * M::LD + d + k] = x[k];
          vs[row * M::LD + d + k] = y[k];
        }
      }
      __syncthreads();
      // ---- S
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = *reinterpret_cast<const float4*>(&qs[(4 * ty + i) * M::LD + d]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          b[j] = *reinterpret_cast<const float4*>(&ks[(tx + 16 * j) * M::LD + d]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
            s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
            s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
            s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
          }
      }
      // ---- softmax
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = t0 + tx + 16 * j <= lim[i] ? s[i][j] * qscale : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int of = 8; of > 0; of >>= 1) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, of));
        const float mn = fmaxf(m_run[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m_run[i] - ref);
        m_run[i] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = ex2(s[i][j] - ref);
          sum += e;
          ps[(4 * ty + i) * M::LP + tx + 16 * j] = e;
        }
        l_run[i] = fmaf(l_run[i], alpha, sum);
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][j][e] *= alpha;
      }
      __syncwarp();  // a row's probabilities stay within its warp
      // ---- O += P V
#pragma unroll 2
      for (int k = 0; k < kSimtBn; k += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pr[i] = *reinterpret_cast<const float4*>(&ps[(4 * ty + i) * M::LP + k]);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int d = 4 * tx + 64 * j;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const float4 v = *reinterpret_cast<const float4*>(&vs[(k + kk) * M::LD + d]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float pk = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
              o[i][j][0] = fmaf(pk, v.x, o[i][j][0]);
              o[i][j][1] = fmaf(pk, v.y, o[i][j][1]);
              o[i][j][2] = fmaf(pk, v.z, o[i][j][2]);
              o[i][j][3] = fmaf(pk, v.w, o[i][j][3]);
            }
          }
        }
      }
    }
    // ---- the rows' results: out, or this block's partial of a cut unit
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int of = 8; of > 0; of >>= 1) l_run[i] += __shfl_xor_sync(FULL, l_run[i], of);
      const int row = 4 * ty + i, tt = row / G, h = row % G;
      if (w.whole()) {
        if (tt >= p.tile_tokens || tok0 + tt >= w.g.n) continue;
        const float inv = l_run[i] > 0.f ? 1.f / l_run[i] : 0.f;
        float* out = static_cast<float*>(p.out) +
                     ((int64_t)(w.g.q0 + tok0 + tt) * p.q_heads + w.kvh * G + h) * D;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int d = 4 * tx + 64 * j;
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = o[i][j][e] * inv;
          S::template store<4>(out + d, y);
        }
      } else {
        float* part = p.parts + (size_t)(2 * blockIdx.x + (w.kv0 > 0 ? 0 : 1)) *
                                    prefill_part_floats(kSimtRows, D);
        if (tx == 0) {
          part[row] = m_run[i];
          part[kSimtRows + row] = l_run[i];
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int g = tx + 16 * j;  // dims 4 g .. 4 g + 3
          *reinterpret_cast<float4*>(part + 2 * kSimtRows + ((size_t)g * kSimtRows + row) * 4) =
              make_float4(o[i][j][0], o[i][j][1], o[i][j][2], o[i][j][3]);
        }
      }
    }
    w.advance();
  }
}

template <int FORM>
np_status launch_simt(const PrefillParams& p, cudaStream_t s) {
  constexpr size_t bytes = SimtSmem::bytes;
  static_assert(bytes <= 227 * 1024, "shared memory");
  static unsigned long long allowed = 0;
  const np_status rc = allow_smem(prefill_simt_kernel<FORM>, bytes, &allowed);
  if (rc != NP_OK) return rc;
  return launch_dependent(prefill_simt_kernel<FORM>, p.ctas, 1, kSimtThreads, bytes, s, p);
}

}  // namespace npk
