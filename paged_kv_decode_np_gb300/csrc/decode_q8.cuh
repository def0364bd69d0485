// decode_q8.cuh -- what the launches of np_paged_decode_q8 share.
#pragma once

#include "prefill.cuh"  // allow_smem, launch_dependent

namespace npk {

constexpr int kQ8MaxCtas = 160;
constexpr int kQ8Rows = 16;  // (query token, head) rows a kv head's fetch serves

// A cut row's partial of one kv head: m[16] l[16] O[16][D], fp32.
__host__ __device__ constexpr size_t q8_entry_floats(int d) { return (size_t)kQ8Rows * (d + 2); }
constexpr size_t q8_parts_bytes(int d) { return (size_t)kQ8MaxCtas * 2 * 8 * q8_entry_floats(d) * 4; }
constexpr size_t q8_workspace_bytes(int d) { return q8_parts_bytes(d) + kQ8MaxCtas * sizeof(int4); }

struct DecodeQ8Params {
  void* out;
  const void* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* tables;
  const int32_t* lens;
  int32_t* err;
  float* parts;  // [ctas][first row, last row][head_group] entries
  int4* cuts;    // [ctas] {row of the stream, first block, last block, slot}; x = -1: none
  int64_t num_blocks;
  int32_t block_size, kv_heads, q_heads, group, max_blocks;
  // Chunks (np_paged_prefill_q8): row r's query tokens are query_starts[r] .. [r + 1] of
  // `tokens`, and only rows with at most query_len of them are read; else NULL, and
  // every row has query_len.
  const int32_t* query_starts;
  int32_t tokens;
  int32_t rows, query_len, head_group, ctas;
  int32_t least;  // chunks a block takes at least
  float qscale;   // scale * log2(e)
};

// decode_q8.cu, per head_dim and form
#define NPK_Q8_DECLARE(d)                                                            \
  np_status decode_q8_d##d##_e4m3(const DecodeQ8Params& p, np_dtype dtype, cudaStream_t s); \
  np_status decode_q8_d##d##_int8(const DecodeQ8Params& p, np_dtype dtype, cudaStream_t s);
NPK_Q8_DECLARE(16)
NPK_Q8_DECLARE(32)
NPK_Q8_DECLARE(64)
NPK_Q8_DECLARE(128)
NPK_Q8_DECLARE(256)
#undef NPK_Q8_DECLARE

// The launches for a head_dim and form, after everything that they need but head_group,
// least and ctas is in p (decode_q8_api.cu).
// Whether all rows' chunks (of 16 tokens, per kv head) can be counted in an int32: 2^30 at
// most, with tables of `cap` tokens.  rows < 2^16, cap < 2^31.
constexpr bool q8_work_fits(int64_t rows, int64_t kv_heads, int64_t cap) {
  const int64_t chunks = rows * ((cap + 15) / 16);  // < 2^43
  return chunks == 0 || kv_heads <= (1ll << 30) / chunks;
}
np_status launch_decode_q8(DecodeQ8Params& p, int32_t head_dim, np_dtype dtype, np_form8 form, int sms,
                           cudaStream_t s);

// the warps of a thread block, which bound the kv heads it takes (head_group)
__host__ __device__ constexpr int q8_warps(int d, int tiles) {
  return d == 256 ? (tiles == 2 ? 4 : 8) : (tiles == 2 ? 8 : 16);
}

}  // namespace npk
