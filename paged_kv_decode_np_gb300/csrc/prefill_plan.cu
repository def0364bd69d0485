// prefill_plan.cu -- the shares of np_paged_prefill's thread blocks, and the
// join of the units that a share's end cuts.
#include "prefill.cuh"

namespace npk {

constexpr int kPlanThreads = 256;

// One block.  Scans the rows' work (costs of kv tiles and of beginning units),
// cuts the stream into equal shares and writes where each block's begins
// (row, kv head, unit, kv tile), and which units the shares' ends cut.
__global__ void __launch_bounds__(kPlanThreads) prefill_plan_kernel(const __grid_constant__
                                                                    PrefillParams p) {
  __shared__ int64_t pre[kPrefillMaxRows + 1];  // work before each row
  __shared__ int64_t warp_sum[kPlanThreads / 32];
  __shared__ int4 pos[kPrefillMaxCtas + 1];
  constexpr unsigned FULL = 0xffffffffu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the attention may become resident: it waits for this block before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (p.rows + kPlanThreads - 1) / kPlanThreads;  // rows a thread
  int64_t sum = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < p.rows) {
      pre[r] = sum;  // within the thread's rows for now
      sum += prefill_row_cost(p, r);
    }
  }
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    constexpr int WARPS = kPlanThreads / 32;
    int64_t y = lane < WARPS ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int64_t u = __shfl_up_sync(FULL, y, o);
      if (lane >= o) y += u;
    }
    if (lane < WARPS) warp_sum[lane] = y;
  }
  __syncthreads();
  const int64_t run = x - sum + (warp > 0 ? warp_sum[warp - 1] : 0);
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    if (r < p.rows) pre[r] += run;
  }
  if (tid == 0) pre[p.rows] = warp_sum[kPlanThreads / 32 - 1];
  __syncthreads();
  if (tid <= p.ctas) p.plan[tid] = pos[tid] = prefill_share_start(p, pre, tid);
  __syncthreads();
  if (tid < p.ctas) p.cuts[tid] = prefill_share_cut(p, pos, tid);
}

np_status launch_prefill_plan(const PrefillParams& p, cudaStream_t s) {
  prefill_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? NP_OK : NP_ERR_CUDA;
}

// The join: block (b, y) merges rows [32 y, 32 y + 32) of the unit that block
// b's share began and its end cuts.  Piece b lies in b's slot 1, the pieces
// of blocks b + 1 .. last in their slot 0.
//     out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// Bound by latency (a unit's partials are some hundred KB in L2), so it is a
// few rounds of independent loads: the pieces' list, then every (piece, row)'s
// m and l, then the O -- a thread holds one row's 4 dims of D / 32 groups,
// consecutive lanes consecutive rows, four pieces in flight.  The result goes
// through shared memory so that the stores are coalesced.
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) prefill_join_kernel(const __grid_constant__
                                                                    PrefillParams p) {
  // every (piece, row)'s m and l; then the results [32][D + 4]
  __shared__ __align__(16) float buf[2 * kPrefillMaxCtas * 32];
  static_assert(32 * (D + 4) <= 2 * kPrefillMaxCtas * 32, "results fit");
  float(*ms)[32] = reinterpret_cast<float(*)[32]>(buf);
  float(*ls)[32] = ms + kPrefillMaxCtas;
  __shared__ int piece[kPrefillMaxCtas];  // the partials, in block order
  __shared__ int pieces;
  // The plan is complete: every block of the attention waited for it before it let
  // this launch start.  Its results are read from L2, where they are: this block
  // has not waited for anything yet that would make an older line in L1 go.
  const int b = blockIdx.x;
  const int4 cut = __ldcg(p.cuts + b);
  if (cut.x < 0) {
    // (this launch must not end before the attention: what comes after waits for it)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (threadIdx.x < 32) {
    // a share may be empty: it begins where the next one does and left nothing
    int n = 0;
    for (int i0 = b; i0 <= cut.w; i0 += 32) {
      const int i = i0 + threadIdx.x;
      bool has = false;
      if (i <= cut.w) {
        const int4 s = __ldcg(p.plan + i), e = __ldcg(p.plan + i + 1);
        has = s.x != e.x || s.y != e.y || s.z != e.z || s.w != e.w;
      }
      const unsigned m = __ballot_sync(0xffffffffu, has);
      if (has) piece[n + __popc(m & ((1u << threadIdx.x) - 1u))] = i == b ? 2 * b + 1 : 2 * i;
      n += __popc(m);
    }
    if (threadIdx.x == 0) pieces = n;
  }
  const PrefillRow gr = prefill_row(p, cut.x);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention is complete
  const int bm = p.tile_rows * p.tiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int WARPS = kJoinThreads / 32;
  const int row = blockIdx.y * 32 + lane;  // < bm
  const size_t pf = prefill_part_floats(bm, D);
  const int np = pieces;
  for (int i = warp; i < np; i += WARPS) {
    const float* q = p.parts + (size_t)piece[i] * pf;
    ms[i][lane] = q[row];
    ls[i][lane] = q[bm + row];
  }
  __syncthreads();
  float M = -INFINITY;
  for (int i = 0; i < np; ++i) M = fmaxf(M, ms[i][lane]);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int i = 0; i < np; ++i) L = fmaf(ex2(ms[i][lane] - ref), ls[i][lane], L);
  const float inv = L > 0.f ? 1.f / L : 0.f;
  constexpr int GW = D / 4 < WARPS ? 1 : D / 4 / WARPS;  // groups of 4 dims a warp
  const bool some = warp * GW < D / 4;
  float acc[GW][4];
#pragma unroll
  for (int g = 0; g < GW; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[g][e] = 0.f;
  if (some) {
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const float* q = p.parts + (size_t)piece[i] * pf + 2 * bm + ((size_t)(warp * GW) * bm + row) * 4;
      const float w = ex2(ms[i][lane] - ref);
#pragma unroll
      for (int g = 0; g < GW; ++g) {
        const float4 o = *reinterpret_cast<const float4*>(q + (size_t)g * bm * 4);
        acc[g][0] = fmaf(w, o.x, acc[g][0]);
        acc[g][1] = fmaf(w, o.y, acc[g][1]);
        acc[g][2] = fmaf(w, o.z, acc[g][2]);
        acc[g][3] = fmaf(w, o.w, acc[g][3]);
      }
    }
  }
  __syncthreads();  // m and l are no longer read
  float(*tile)[D + 4] = reinterpret_cast<float(*)[D + 4]>(buf);
  if (some) {
#pragma unroll
    for (int g = 0; g < GW; ++g)
      *reinterpret_cast<float4*>(&tile[lane][4 * (warp * GW + g)]) =
          make_float4(acc[g][0] * inv, acc[g][1] * inv, acc[g][2] * inv, acc[g][3] * inv);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * (D / 4); e += kJoinThreads) {
    const int rr = e / (D / 4), d = (e % (D / 4)) * 4;
    const int urow = blockIdx.y * 32 + rr;           // row of the unit
    const int mt = urow / p.tile_rows, in = urow % p.tile_rows;
    const int tt = in / p.group, h = in % p.group;
    const int64_t tok = ((int64_t)cut.z * p.tiles + mt) * p.tile_tokens + tt;
    if (tt >= p.tile_tokens || tok >= gr.n) continue;
    T* o = static_cast<T*>(p.out) + ((gr.q0 + tok) * p.q_heads + (int64_t)cut.y * p.group + h) * D;
    Storage<T>::template store<4>(o + d, &tile[rr][d]);
  }
}

template <typename T>
static np_status launch_join_t(const PrefillParams& p, cudaStream_t s) {
  const unsigned gy = (unsigned)(p.tile_rows * p.tiles / 32);
  switch (p.head_dim) {
    case 16: return launch_dependent(prefill_join_kernel<T, 16>, p.ctas, gy, kJoinThreads, 0, s, p);
    case 32: return launch_dependent(prefill_join_kernel<T, 32>, p.ctas, gy, kJoinThreads, 0, s, p);
    case 64: return launch_dependent(prefill_join_kernel<T, 64>, p.ctas, gy, kJoinThreads, 0, s, p);
    case 128: return launch_dependent(prefill_join_kernel<T, 128>, p.ctas, gy, kJoinThreads, 0, s, p);
    case 256: return launch_dependent(prefill_join_kernel<T, 256>, p.ctas, gy, kJoinThreads, 0, s, p);
  }
  return NP_ERR_UNSUPPORTED;
}

np_status launch_prefill_join(const PrefillParams& p, np_dtype dtype, cudaStream_t s) {
  return dtype == NP_BF16 ? launch_join_t<__nv_bfloat16>(p, s) : launch_join_t<float>(p, s);
}

}  // namespace npk
