// decode_q8_api.cu -- np_paged_decode_q8: argument validation and the launches.
#include <limits.h>

#include "decode_q8.cuh"
#include "host_checks.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool head_dim_ok(int32_t d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

np_status check_decode_q8(const np_read_q8_args& a, bool* run) {
  using namespace npk;
  *run = false;
  const int es = a.dtype == NP_F32 ? 4 : (a.dtype == NP_BF16 ? 2 : 0);
  if (es == 0 || (a.form != NP_E4M3 && a.form != NP_INT8)) return NP_ERR_UNSUPPORTED;
  if (a.rows < 0 || a.query_len <= 0 || a.q_heads <= 0 || a.kv_heads <= 0 || a.q_heads % a.kv_heads != 0 ||
      a.num_blocks <= 0 || a.block_size <= 0 || a.max_blocks_per_row <= 0 || a.head_dim <= 0 ||
      !isfinite(a.scale * kLog2e))
    return NP_ERR_INVALID_ARG;
  if (!head_dim_ok(a.head_dim)) return NP_ERR_UNSUPPORTED;
  const int64_t d = a.head_dim;
  if ((int64_t)(a.q_heads / a.kv_heads) * a.query_len > (a.dtype == NP_BF16 ? 16 : 8)) return NP_ERR_UNSUPPORTED;
  int64_t slots = 0, pool = 0, scales = 0, cap = 0, tab = 0, qn = 0;
  if (!mul_fits(a.num_blocks, a.block_size, &slots) || !mul_fits(slots, a.kv_heads * d, &pool) ||
      !mul_fits(a.num_blocks, 4ll * a.kv_heads, &scales) || !mul_fits(a.max_blocks_per_row, a.block_size, &cap) ||
      !mul_fits(a.rows, 4ll * a.max_blocks_per_row, &tab) ||
      !mul_fits((int64_t)a.rows * a.query_len, a.q_heads * d * es, &qn))
    return NP_ERR_OUT_OF_RANGE;
  if (a.rows > 65535 || cap > INT32_MAX - 1024) return NP_ERR_UNSUPPORTED;
  if (!q8_work_fits(a.rows, a.kv_heads, cap)) return NP_ERR_UNSUPPORTED;
  if (a.rows == 0) return NP_OK;
  if (!a.out || !a.q || !a.k_pool || !a.v_pool || !a.k_scale || !a.v_scale || !a.block_tables || !a.context_lens)
    return NP_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(a.out), a.q, a.k_pool, a.v_pool})
    if (!aligned_to(x, 16)) return NP_ERR_INVALID_ARG;
  if (!aligned_to(a.k_scale, 4) || !aligned_to(a.v_scale, 4) || !aligned_to(a.block_tables, 4) ||
      !aligned_to(a.context_lens, 4) || !aligned_to(a.err_word, 4))
    return NP_ERR_INVALID_ARG;
  const Span spans[] = {{a.out, qn}, {a.q, qn}, {a.k_pool, pool}, {a.v_pool, pool}, {a.k_scale, scales},
                        {a.v_scale, scales}, {a.block_tables, tab}, {a.context_lens, 4ll * a.rows}};
  if (any_overlap(spans, 1)) return NP_ERR_INVALID_ARG;
  if (!a.workspace || a.workspace_bytes < 0 || (size_t)a.workspace_bytes < q8_workspace_bytes(a.head_dim) ||
      !aligned_to(a.workspace, 256))
    return NP_ERR_WORKSPACE;
  *run = true;
  return NP_OK;
}

}  // namespace

namespace npk {

np_status launch_decode_q8(DecodeQ8Params& p, int32_t head_dim, np_dtype t, np_form8 form, int sms,
                           cudaStream_t s) {
  p.ctas = sms < kQ8MaxCtas ? sms : kQ8MaxCtas;
  // kv heads of a block: the largest divisor that its warps have room for
  const int tiles = t == NP_BF16 && p.group * p.query_len > 8 ? 2 : 1;
  const int warps = q8_warps(head_dim, tiles);
  p.head_group = 1;
  for (int h = 2; h <= 8 && h <= warps; ++h)
    if (p.kv_heads % h == 0) p.head_group = h;
  // Two chunks a warp at least, us with 1, 2, 3, 4: 8 fp32 rows of 512-2048 21.6, 20.3, 21.2,
  // 22.2; one row of 4000 23.0, 17.1, 17.2, 17.0; 16 of 300-600 16.0, 16.9, 17.7, 19.1.
  p.least = 2 * (warps / p.head_group);
  const bool e4m3 = form == NP_E4M3;
  switch (head_dim) {
    case 16: return e4m3 ? decode_q8_d16_e4m3(p, t, s) : decode_q8_d16_int8(p, t, s);
    case 32: return e4m3 ? decode_q8_d32_e4m3(p, t, s) : decode_q8_d32_int8(p, t, s);
    case 64: return e4m3 ? decode_q8_d64_e4m3(p, t, s) : decode_q8_d64_int8(p, t, s);
    case 128: return e4m3 ? decode_q8_d128_e4m3(p, t, s) : decode_q8_d128_int8(p, t, s);
    case 256: return e4m3 ? decode_q8_d256_e4m3(p, t, s) : decode_q8_d256_int8(p, t, s);
  }
  return NP_ERR_UNSUPPORTED;
}

}  // namespace npk

extern "C" size_t np_paged_decode_q8_workspace_bytes(int32_t head_dim) {
  return head_dim_ok(head_dim) ? npk::q8_workspace_bytes(head_dim) : 0;
}

extern "C" np_status np_paged_decode_q8_check(const np_read_q8_args* a) {
  bool run;
  return a ? check_decode_q8(*a, &run) : NP_ERR_INVALID_ARG;
}

extern "C" np_status np_paged_decode_q8_packed(const np_read_q8_args* a) {
  if (!a) return NP_ERR_INVALID_ARG;
  bool run;
  const np_status st = check_decode_q8(*a, &run);
  if (st != NP_OK || !run) return st;
  const int sms = npk::sm_count();
  if (sms <= 0) return NP_ERR_CUDA;
  npk::DecodeQ8Params p{};
  p.out = a->out;
  p.q = a->q;
  p.k_pool = static_cast<const uint8_t*>(a->k_pool);
  p.v_pool = static_cast<const uint8_t*>(a->v_pool);
  p.k_scale = a->k_scale;
  p.v_scale = a->v_scale;
  p.tables = a->block_tables;
  p.lens = a->context_lens;
  p.err = a->err_word;
  p.parts = static_cast<float*>(a->workspace);
  p.cuts = reinterpret_cast<int4*>(static_cast<char*>(a->workspace) + npk::q8_parts_bytes(a->head_dim));
  p.num_blocks = a->num_blocks;
  p.block_size = a->block_size;
  p.kv_heads = a->kv_heads;
  p.q_heads = a->q_heads;
  p.group = a->q_heads / a->kv_heads;
  p.max_blocks = a->max_blocks_per_row;
  p.rows = a->rows;
  p.query_len = a->query_len;
  p.qscale = a->scale * kLog2e;
  return npk::launch_decode_q8(p, a->head_dim, static_cast<np_dtype>(a->dtype), static_cast<np_form8>(a->form),
                               sms, reinterpret_cast<cudaStream_t>(a->stream));
}

extern "C" np_status np_paged_decode_q8(void* out, const void* q, np_dtype dtype, const void* k_pool,
                                        const void* v_pool, const float* k_scale, const float* v_scale,
                                        np_form8 form, int64_t num_blocks, int32_t block_size,
                                        int32_t kv_heads, int32_t head_dim, const int32_t* block_tables,
                                        int32_t max_blocks_per_row, const int32_t* context_lens,
                                        int32_t rows, int32_t query_len, int32_t q_heads, float scale,
                                        void* workspace, size_t workspace_bytes, int32_t* err_word,
                                        np_stream_t stream) {
  np_read_q8_args a{};
  a.out = out;
  a.q = q;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
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
  a.query_len = query_len;
  a.q_heads = q_heads;
  a.scale = scale;
  return np_paged_decode_q8_packed(&a);
}
