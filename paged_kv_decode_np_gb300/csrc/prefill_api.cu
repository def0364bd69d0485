// prefill_api.cu -- np_paged_prefill: argument validation, the workspace's
// layout and the launches.
#include <limits.h>

#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled_v12000

#include "prefill.cuh"

namespace {

using npk::PrefillParams;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

constexpr float kLog2e = 1.4426950408889634f;

// Plan and cut list, then the partials of kPrefillMaxCtas blocks.
constexpr size_t kPlanBytes = (2 * npk::kPrefillMaxCtas + 1) * sizeof(int4);

// rows of the largest unit any kernel of this head_dim takes
int unit_rows(int32_t head_dim) { return head_dim == 256 ? 128 : 256; }

std::atomic<int> g_sms[64];

int sm_count() {
  int dev = 0, s = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64) s = g_sms[dev].load();
  if (s == 0) {
    if (cudaDeviceGetAttribute(&s, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) g_sms[dev].store(s);
  }
  return s;
}

// The driver's tensor map encoder, through the runtime (no libcuda link).
PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A bf16 tensor of N dims (innermost first, byte strides of dims 1 ..), copied
// in the given box in the 128-byte swizzle.
template <int N>
bool encode_map(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[N],
                const cuuint64_t (&strides)[N - 1], const cuuint32_t (&box)[N]) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint32_t estr[N];
  for (int i = 0; i < N; ++i) estr[i] = 1u;
  auto encode = [&] {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, N, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // A host thread that has launched nothing yet has no context, which the driver's
  // encoder wants: the runtime binds the current device's, and it is tried again.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// bf16: the tensor-core kernel of this head_dim
np_status launch_tc(PrefillParams& p, int64_t slots, cudaStream_t s) {
  const int d = p.head_dim;
  // a masked score is -inf before it is scaled: no 0 x inf
  p.qscale = fmaxf(p.qscale, 1e-30f);
  npk::prefill_tiling(p, NP_BF16);
  // Tiled copies: boxes of whole 8-row swizzle atoms inside one block, slot
  // coordinates in int32.  box_tokens: the largest power of two that divides
  // the block size, at most a kv tile.
  int bt = 1;
  while (bt < p.bn && p.block_size % (2 * bt) == 0) bt *= 2;
  p.box_tokens = bt;
  bool tiled = bt >= 8 && slots <= INT32_MAX;
  if (d >= 64) {
    const cuuint64_t row = (cuuint64_t)p.kv_heads * d * 2, head = (cuuint64_t)d * 2;
    const cuuint32_t slabs = (cuuint32_t)d / 64;
    const cuuint64_t q_dims[3] = {(cuuint64_t)d, (cuuint64_t)p.q_heads, (cuuint64_t)p.tokens};
    const cuuint64_t q_strides[2] = {head, (cuuint64_t)p.q_heads * head};
    const cuuint32_t q_box[3] = {64u, (cuuint32_t)p.group, (cuuint32_t)p.tile_tokens};
    if (!encode_map(&p.tm_q, p.q, q_dims, q_strides, q_box)) return NP_ERR_CUDA;
    // 64 dims, token of 8, slab, group of 8 tokens, kv head
    const cuuint64_t kv_dims[5] = {64u, 8u, slabs, (cuuint64_t)slots / 8, (cuuint64_t)p.kv_heads};
    const cuuint64_t kv_strides[4] = {row, 128u, 8 * row, head};
    const cuuint32_t kv_box[5] = {64u, 8u, slabs, (cuuint32_t)bt / 8, 1u};
    tiled = tiled && encode_map(&p.tm_k, p.k_pool, kv_dims, kv_strides, kv_box) &&
            encode_map(&p.tm_v, p.v_pool, kv_dims, kv_strides, kv_box);
  } else {
    tiled = false;
  }
  np_status rc = npk::launch_prefill_plan(p, s);
  if (rc != NP_OK) return rc;
  switch (d) {
    case 16: return npk::prefill_tc_d16(p, tiled, s);
    case 32: return npk::prefill_tc_d32(p, tiled, s);
    case 64: return npk::prefill_tc_d64(p, tiled, s);
    case 128: return npk::prefill_tc_d128(p, tiled, s);
    case 256: return npk::prefill_tc_d256(p, tiled, s);
  }
  return NP_ERR_UNSUPPORTED;
}

// fp32: three bf16 parts on the tensor cores; head_dim 256 on the FMA pipes
np_status launch_f32(PrefillParams& p, cudaStream_t s) {
  npk::prefill_tiling(p, NP_F32);
  if (p.head_dim <= 128) p.qscale = fmaxf(p.qscale, 1e-30f);
  const np_status rc = npk::launch_prefill_plan(p, s);
  if (rc != NP_OK) return rc;
  switch (p.head_dim) {
    case 16: return npk::prefill_tc32_d16(p, s);
    case 32: return npk::prefill_tc32_d32(p, s);
    case 64: return npk::prefill_tc32_d64(p, s);
    case 128: return npk::prefill_tc32_d128(p, s);
    case 256: return npk::launch_prefill_simt(p, s);
  }
  return NP_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" size_t np_paged_prefill_workspace_bytes(int32_t head_dim) {
  if (head_dim != 16 && head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
    return 0;
  return round_up(kPlanBytes, 256) +
         2 * npk::kPrefillMaxCtas * npk::prefill_part_floats(unit_rows(head_dim), head_dim) * 4;
}

namespace {

// The checks of a call; *run: whether there is something to launch.
np_status check_prefill(const np_paged_prefill_args& a, bool* run) {
  *run = false;
  const int es = a.dtype == NP_F32 ? 4 : (a.dtype == NP_BF16 ? 2 : 0);
  if (es == 0) return NP_ERR_UNSUPPORTED;
  if (a.rows < 0 || a.num_tokens < 0 || a.q_heads <= 0 || a.kv_heads <= 0 ||
      a.q_heads % a.kv_heads != 0 || a.num_blocks <= 0 || a.block_size <= 0 ||
      a.max_blocks_per_row <= 0 || a.head_dim <= 0 || !isfinite(a.scale * kLog2e))
    return NP_ERR_INVALID_ARG;
  const int d = a.head_dim;
  if (d != 16 && d != 32 && d != 64 && d != 128 && d != 256) return NP_ERR_UNSUPPORTED;
  if (a.q_heads / a.kv_heads > (a.dtype == NP_BF16 ? 16 : 8)) return NP_ERR_UNSUPPORTED;
  int64_t slots = 0, pool = 0, cap = 0, qn = 0, tab = 0;
  if (!mul_ok(a.num_blocks, a.block_size, &slots) ||
      !mul_ok(slots, (int64_t)a.kv_heads * d * es, &pool) ||
      !mul_ok(a.num_tokens, (int64_t)a.q_heads * d * es, &qn) ||
      !mul_ok(a.max_blocks_per_row, a.block_size, &cap) || !mul_ok(a.rows, a.max_blocks_per_row, &tab))
    return NP_ERR_OUT_OF_RANGE;
  // positions are int32 with some kv tiles to spare
  if (cap > INT32_MAX - 1024 || a.num_tokens > INT32_MAX - 512) return NP_ERR_UNSUPPORTED;
  if (a.rows > npk::kPrefillMaxRows) return NP_ERR_UNSUPPORTED;
  if (a.rows == 0 || a.num_tokens == 0) return NP_OK;
  if (!a.out || !a.q || !a.k_pool || !a.v_pool || !a.block_tables || !a.context_lens || !a.query_starts)
    return NP_ERR_INVALID_ARG;
  if (!aligned(a.out, 16) || !aligned(a.q, 16) || !aligned(a.k_pool, 16) || !aligned(a.v_pool, 16) ||
      !aligned(a.block_tables, 4) || !aligned(a.context_lens, 4) || !aligned(a.query_starts, 4) ||
      (a.err_word && !aligned(a.err_word, 4)))
    return NP_ERR_INVALID_ARG;
  if (overlap(a.out, qn, a.q, qn) || overlap(a.out, qn, a.k_pool, pool) ||
      overlap(a.out, qn, a.v_pool, pool))
    return NP_ERR_INVALID_ARG;
  if (!a.workspace || a.workspace_bytes < 0 ||
      (size_t)a.workspace_bytes < np_paged_prefill_workspace_bytes(d) || !aligned(a.workspace, 256))
    return NP_ERR_WORKSPACE;
  *run = true;
  return NP_OK;
}

}  // namespace

extern "C" np_status np_paged_prefill_check(const np_paged_prefill_args* a) {
  bool run;
  return a ? check_prefill(*a, &run) : NP_ERR_INVALID_ARG;
}

extern "C" np_status np_paged_prefill_packed(const np_paged_prefill_args* a) {
  if (!a) return NP_ERR_INVALID_ARG;
  bool run;
  const np_status st = check_prefill(*a, &run);
  if (st != NP_OK || !run) return st;
  const int sms = sm_count();
  if (sms <= 0) return NP_ERR_CUDA;

  PrefillParams p{};
  p.out = a->out;
  p.q = a->q;
  p.k_pool = a->k_pool;
  p.v_pool = a->v_pool;
  p.block_tables = a->block_tables;
  p.context_lens = a->context_lens;
  p.query_starts = a->query_starts;
  p.err = a->err_word;
  p.plan = static_cast<int4*>(a->workspace);
  p.cuts = p.plan + npk::kPrefillMaxCtas + 1;
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a->workspace) + round_up(kPlanBytes, 256));
  p.num_blocks = a->num_blocks;
  p.block_size = a->block_size;
  p.kv_heads = a->kv_heads;
  p.q_heads = a->q_heads;
  p.group = a->q_heads / a->kv_heads;
  p.max_blocks_per_row = a->max_blocks_per_row;
  p.rows = a->rows;
  p.tokens = a->num_tokens;
  p.ctas = sms < npk::kPrefillMaxCtas ? sms : npk::kPrefillMaxCtas;
  p.head_dim = a->head_dim;
  p.qscale = fabsf(a->scale) * kLog2e;
  p.negate = a->scale < 0.f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(a->stream);
  const np_dtype dtype = static_cast<np_dtype>(a->dtype);
  const np_status rc =
      dtype == NP_BF16 ? launch_tc(p, a->num_blocks * a->block_size, s) : launch_f32(p, s);
  return rc == NP_OK ? npk::launch_prefill_join(p, dtype, s) : rc;
}

extern "C" np_status np_paged_prefill(void* out, const void* q, const void* k_pool,
                                      const void* v_pool, np_dtype dtype, int64_t num_blocks,
                                      int32_t block_size, int32_t kv_heads, int32_t head_dim,
                                      const int32_t* block_tables, int32_t max_blocks_per_row,
                                      const int32_t* context_lens, const int32_t* query_starts,
                                      int32_t rows, int32_t num_tokens, int32_t q_heads,
                                      float scale, void* workspace, size_t workspace_bytes,
                                      int32_t* err_word, np_stream_t stream) {
  np_paged_prefill_args a{};
  a.out = out;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_starts = query_starts;
  a.workspace = workspace;
  a.err_word = err_word;
  a.stream = stream;
  a.num_blocks = num_blocks;
  a.workspace_bytes = workspace_bytes > (size_t)INT64_MAX ? INT64_MAX : (int64_t)workspace_bytes;
  a.dtype = dtype;
  a.block_size = block_size;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.max_blocks_per_row = max_blocks_per_row;
  a.rows = rows;
  a.num_tokens = num_tokens;
  a.q_heads = q_heads;
  a.scale = scale;
  return np_paged_prefill_packed(&a);
}
