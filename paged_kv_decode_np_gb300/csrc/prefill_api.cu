// prefill_api.cu -- np_paged_prefill: argument validation, the workspace's
// layout and the launches.
#include <limits.h>

#include <mutex>

#include <cudaTypedefs.h>  // PFN_cuTensorMapEncodeTiled_v12000

#include "decode_q8.cuh"
#include "host_checks.h"
#include "prefill.cuh"

namespace {

using npk::aligned_to;
using npk::mul_fits;
using npk::overlaps;
using npk::PrefillParams;
using npk::sm_count;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr float kLog2e = 1.4426950408889634f;

// Plan and cut list, then the partials of kPrefillMaxCtas blocks.
constexpr size_t kPlanBytes = (2 * npk::kPrefillMaxCtas + 1) * sizeof(int4);
// The decode read's partials and cuts use the same workspace (np_paged_prefill_q8).
static_assert(npk::kQ8MaxCtas <= npk::kPrefillMaxCtas && 8 * npk::kQ8Rows <= 128 &&
                  npk::kQ8MaxCtas * sizeof(int4) <= kPlanBytes,
              "workspace");

// rows of the largest unit any kernel of this head_dim takes
int unit_rows(int32_t head_dim) { return head_dim == 256 ? 128 : 256; }

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

// A tensor of N dims (innermost first, byte strides of dims 1 ..) of bf16 or of another
// type, copied in the given box in the 128-byte swizzle or another.
template <int N>
bool encode_map(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[N],
                const cuuint64_t (&strides)[N - 1], const cuuint32_t (&box)[N],
                CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tmap_encoder();
  if (!enc) return false;
  cuuint32_t estr[N];
  for (int i = 0; i < N; ++i) estr[i] = 1u;
  auto encode = [&] {
    return enc(m, type, N, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // A host thread that has launched nothing yet has no context, which the driver's
  // encoder wants: the runtime binds the current device's, and it is tried again.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// q's map of the tensor-core kernel, head_dim a multiple of 64
bool encode_q(PrefillParams& p) {
  const cuuint64_t d = (cuuint64_t)p.head_dim, head = d * 2;
  const cuuint64_t q_dims[3] = {d, (cuuint64_t)p.q_heads, (cuuint64_t)p.tokens};
  const cuuint64_t q_strides[2] = {head, (cuuint64_t)p.q_heads * head};
  const cuuint32_t q_box[3] = {64u, (cuuint32_t)p.group, (cuuint32_t)p.tile_tokens};
  return encode_map(&p.tm_q, p.q, q_dims, q_strides, q_box);
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
    if (!encode_q(p)) return NP_ERR_CUDA;
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

// An 8-bit cache: on the tensor cores, but for fp32 at head_dim 256.
np_status launch_q8(PrefillParams& p, np_dtype dtype, np_form8 form, cudaStream_t s) {
  if (dtype == NP_F32) {
    npk::prefill_tiling(p, NP_F32);
    if (p.head_dim <= 128) p.qscale = fmaxf(p.qscale, 1e-30f);
    const np_status rc = npk::launch_prefill_plan(p, s);
    if (rc != NP_OK) return rc;
    switch (p.head_dim) {
      case 16: return npk::prefill_tc32q8_d16(p, form, s);
      case 32: return npk::prefill_tc32q8_d32(p, form, s);
      case 64: return npk::prefill_tc32q8_d64(p, form, s);
      case 128: return npk::prefill_tc32q8_d128(p, form, s);
      case 256: return npk::launch_prefill_q8_simt(p, form, s);
    }
    return NP_ERR_UNSUPPORTED;
  }
  p.qscale = fmaxf(p.qscale, 1e-30f);  // (as above)
  npk::prefill_tiling(p, NP_BF16);
  const int d = p.head_dim;
  bool tiled = false;
  if (d >= 64) {
    if (!encode_q(p)) return NP_ERR_CUDA;
    // Tiled copies: boxes of whole 8-token groups inside one block, slots in int32.
    int bt = 1;
    while (bt < p.bn && p.block_size % (2 * bt) == 0) bt *= 2;
    p.box_tokens = bt;
    const int64_t slots = p.num_blocks * p.block_size;
    if (bt >= 8 && slots <= INT32_MAX) {
      // up to 128 bytes of a token, slot, 128-byte slab, kv head
      const cuuint64_t wide = d < 128 ? d : 128, slabs = d / wide;
      const cuuint64_t dims[4] = {wide, (cuuint64_t)slots, slabs, (cuuint64_t)p.kv_heads};
      const cuuint64_t strides[3] = {(cuuint64_t)p.kv_heads * d, 128u, (cuuint64_t)d};
      const cuuint32_t box[4] = {(cuuint32_t)wide, (cuuint32_t)bt, (cuuint32_t)slabs, 1u};
      const CUtensorMapSwizzle swizzle = d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
      tiled = encode_map(&p.tm_k, p.k_pool, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8, swizzle) &&
              encode_map(&p.tm_v, p.v_pool, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8, swizzle);
    }
  }
  const np_status rc = npk::launch_prefill_plan(p, s);
  if (rc != NP_OK) return rc;
  switch (d) {
    case 16: return npk::prefill_tcq8_d16(p, form, tiled, s);
    case 32: return npk::prefill_tcq8_d32(p, form, tiled, s);
    case 64: return npk::prefill_tcq8_d64(p, form, tiled, s);
    case 128: return npk::prefill_tcq8_d128(p, form, tiled, s);
    case 256: return npk::prefill_tcq8_d256(p, form, tiled, s);
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

// The checks of a call; *run: whether there is something to launch.  pool_es: bytes of
// a pool's element (0: the dtype's).
np_status check_prefill(const np_paged_prefill_args& a, bool* run, int pool_es = 0) {
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
  if (!mul_fits(a.num_blocks, a.block_size, &slots) ||
      !mul_fits(slots, (int64_t)a.kv_heads * d * (pool_es ? pool_es : es), &pool) ||
      !mul_fits(a.num_tokens, (int64_t)a.q_heads * d * es, &qn) ||
      !mul_fits(a.max_blocks_per_row, a.block_size, &cap) || !mul_fits(a.rows, a.max_blocks_per_row, &tab))
    return NP_ERR_OUT_OF_RANGE;
  // positions are int32 with some kv tiles to spare
  if (cap > INT32_MAX - 1024 || a.num_tokens > INT32_MAX - 512) return NP_ERR_UNSUPPORTED;
  if (a.rows > npk::kPrefillMaxRows) return NP_ERR_UNSUPPORTED;
  if (a.rows == 0 || a.num_tokens == 0) return NP_OK;
  if (!a.out || !a.q || !a.k_pool || !a.v_pool || !a.block_tables || !a.context_lens || !a.query_starts)
    return NP_ERR_INVALID_ARG;
  if (!aligned_to(a.out, 16) || !aligned_to(a.q, 16) || !aligned_to(a.k_pool, 16) ||
      !aligned_to(a.v_pool, 16) || !aligned_to(a.block_tables, 4) || !aligned_to(a.context_lens, 4) ||
      !aligned_to(a.query_starts, 4) ||
      (a.err_word && !aligned_to(a.err_word, 4)))
    return NP_ERR_INVALID_ARG;
  if (overlaps({a.out, qn}, {a.q, qn}) || overlaps({a.out, qn}, {a.k_pool, pool}) ||
      overlaps({a.out, qn}, {a.v_pool, pool}))
    return NP_ERR_INVALID_ARG;
  if (!a.workspace || a.workspace_bytes < 0 ||
      (size_t)a.workspace_bytes < np_paged_prefill_workspace_bytes(d) || !aligned_to(a.workspace, 256))
    return NP_ERR_WORKSPACE;
  *run = true;
  return NP_OK;
}

}  // namespace

extern "C" np_status np_paged_prefill_check(const np_paged_prefill_args* a) {
  bool run;
  return a ? check_prefill(*a, &run) : NP_ERR_INVALID_ARG;
}

namespace {

// A checked call's parameters, but for the tiling; false: no device.
bool fill_params(const np_paged_prefill_args* a, PrefillParams& p) {
  const int sms = sm_count();
  if (sms <= 0) return false;
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
  return true;
}

}  // namespace

extern "C" np_status np_paged_prefill_packed(const np_paged_prefill_args* a) {
  if (!a) return NP_ERR_INVALID_ARG;
  bool run;
  const np_status st = check_prefill(*a, &run);
  if (st != NP_OK || !run) return st;
  PrefillParams p{};
  if (!fill_params(a, p)) return NP_ERR_CUDA;
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

// ---------------------------------------------------------- 8-bit caches --
namespace {

np_paged_prefill_args plain_args(const np_read_q8_args& a) {
  np_paged_prefill_args b{};
  b.out = a.out;
  b.q = a.q;
  b.k_pool = a.k_pool;
  b.v_pool = a.v_pool;
  b.block_tables = a.block_tables;
  b.context_lens = a.context_lens;
  b.query_starts = a.query_starts;
  b.workspace = a.workspace;
  b.err_word = a.err_word;
  b.stream = a.stream;
  b.num_blocks = a.num_blocks;
  b.workspace_bytes = a.workspace_bytes;
  b.dtype = a.dtype;
  b.block_size = a.block_size;
  b.kv_heads = a.kv_heads;
  b.head_dim = a.head_dim;
  b.max_blocks_per_row = a.max_blocks_per_row;
  b.rows = a.rows;
  b.num_tokens = a.num_tokens;
  b.q_heads = a.q_heads;
  b.scale = a.scale;
  return b;
}

np_status check_prefill_q8(const np_read_q8_args& a, bool* run) {
  *run = false;
  if (a.form != NP_E4M3 && a.form != NP_INT8) return NP_ERR_UNSUPPORTED;
  if (a.query_len != 0) return NP_ERR_INVALID_ARG;
  const np_status st = check_prefill(plain_args(a), run, 1);
  if (st != NP_OK || !*run) return st;
  *run = false;
  int64_t scales = 0;
  if (!mul_fits(a.num_blocks, 4ll * a.kv_heads, &scales)) return NP_ERR_OUT_OF_RANGE;
  if (!a.k_scale || !a.v_scale || !aligned_to(a.k_scale, 4) || !aligned_to(a.v_scale, 4))
    return NP_ERR_INVALID_ARG;
  const int64_t out = (int64_t)a.num_tokens * a.q_heads * a.head_dim * (a.dtype == NP_BF16 ? 2 : 4);
  if (overlaps({a.out, out}, {a.k_scale, scales}) || overlaps({a.out, out}, {a.v_scale, scales}))
    return NP_ERR_INVALID_ARG;
  *run = true;
  return NP_OK;
}

}  // namespace

extern "C" np_status np_paged_prefill_q8_check(const np_read_q8_args* a) {
  bool run;
  return a ? check_prefill_q8(*a, &run) : NP_ERR_INVALID_ARG;
}

extern "C" np_status np_paged_prefill_q8_packed(const np_read_q8_args* a) {
  if (!a) return NP_ERR_INVALID_ARG;
  bool run;
  const np_status st = check_prefill_q8(*a, &run);
  if (st != NP_OK || !run) return st;
  const np_paged_prefill_args b = plain_args(*a);
  PrefillParams p{};
  if (!fill_params(&b, p)) return NP_ERR_CUDA;
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(a->stream);
  const np_dtype dtype = static_cast<np_dtype>(a->dtype);
  const np_form8 form = static_cast<np_form8>(a->form);
  // Rows with few tokens go to the decode read's kernel: their (token, head) rows fit
  // one fetch of its tile.  Two launches more (5 to 15 us), so where rows are short on
  // average.  us, replayed, bf16 / fp32, all rows here -> the short ones there (heads 32 / 8,
  // histories of 1024-8192): 62 rows of one token and two of 512 (17 a row) 288 / 772 -> 193 /
  // 315; 30 and two of 900 (57) 242 / 650 -> 206 / 413; 64 of two 219 / 552 -> 107 / 120; 64
  // of 4, 8, 16 and 48, none short: 218-304 -> 224-313.  Past the border: 30 and two of 1024
  // (65) 285 / 680, 208 / 446 if they went there; 14 and two of 1024 (129) 237 / 658, 224 /
  // 523; 12 and four of 400 (101) 224 / 648, 227 / 516; 3 and one of 300 (76) 51 / 99, 66 / 109:
  // few rows lose by it, many gain, and the average does not tell them apart.
  const int few = (p.group <= 8 ? 8 : 16) / p.group;
  if ((p.rows > 1 ? p.tokens < 64ll * p.rows : p.tokens <= few) &&
      npk::q8_work_fits(p.rows, p.kv_heads, (int64_t)p.max_blocks_per_row * p.block_size)) {
    p.skip_tokens = few;
    npk::DecodeQ8Params d{};
    d.out = p.out;
    d.q = p.q;
    d.k_pool = static_cast<const uint8_t*>(p.k_pool);
    d.v_pool = static_cast<const uint8_t*>(p.v_pool);
    d.k_scale = p.k_scale;
    d.v_scale = p.v_scale;
    d.tables = p.block_tables;
    d.lens = p.context_lens;
    d.err = p.err;
    // (the workspace is the attention's after the join: the plan is launched when that is over)
    d.parts = static_cast<float*>(a->workspace);
    d.cuts = reinterpret_cast<int4*>(static_cast<char*>(a->workspace) + npk::q8_parts_bytes(p.head_dim));
    d.num_blocks = p.num_blocks;
    d.block_size = p.block_size;
    d.kv_heads = p.kv_heads;
    d.q_heads = p.q_heads;
    d.group = p.group;
    d.max_blocks = p.max_blocks_per_row;
    d.query_starts = p.query_starts;
    d.tokens = p.tokens;
    d.rows = p.rows;
    d.query_len = few;
    d.qscale = a->scale * kLog2e;
    const np_status rc = npk::launch_decode_q8(d, p.head_dim, dtype, form, p.ctas, s);
    if (rc != NP_OK || p.tokens <= few) return rc;  // (no row has more than all the tokens)
  }
  const np_status rc = launch_q8(p, dtype, form, s);
  return rc == NP_OK ? npk::launch_prefill_join(p, dtype, s) : rc;
}

extern "C" np_status np_paged_prefill_q8(void* out, const void* q, np_dtype dtype, const void* k_pool,
                                         const void* v_pool, const float* k_scale, const float* v_scale,
                                         np_form8 form, int64_t num_blocks, int32_t block_size,
                                         int32_t kv_heads, int32_t head_dim, const int32_t* block_tables,
                                         int32_t max_blocks_per_row, const int32_t* context_lens,
                                         const int32_t* query_starts, int32_t rows, int32_t num_tokens,
                                         int32_t q_heads, float scale, void* workspace,
                                         size_t workspace_bytes, int32_t* err_word, np_stream_t stream) {
  np_read_q8_args a{};
  a.out = out;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_starts = query_starts;
  a.workspace = workspace;
  a.err_word = err_word;
  a.stream = stream;
  a.num_blocks = num_blocks;
  a.workspace_bytes = workspace_bytes > (size_t)INT64_MAX ? INT64_MAX : (int64_t)workspace_bytes;
  a.form = form;
  a.dtype = dtype;
  a.block_size = block_size;
  a.kv_heads = kv_heads;
  a.head_dim = head_dim;
  a.max_blocks_per_row = max_blocks_per_row;
  a.rows = rows;
  a.num_tokens = num_tokens;
  a.q_heads = q_heads;
  a.scale = scale;
  return np_paged_prefill_q8_packed(&a);
}
