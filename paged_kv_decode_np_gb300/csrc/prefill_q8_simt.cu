// prefill_q8_simt.cu -- np_paged_prefill_q8 on the FMA pipes.
#include "prefill_simt.cuh"

namespace npk {

template <typename T, int FORM>
static np_status by_dim(const PrefillParams& p, cudaStream_t s) {
  switch (p.head_dim) {
    case 16: return launch_simt<T, 16, FORM>(p, s);
    case 32: return launch_simt<T, 32, FORM>(p, s);
    case 64: return launch_simt<T, 64, FORM>(p, s);
    case 128: return launch_simt<T, 128, FORM>(p, s);
    case 256: return launch_simt<T, 256, FORM>(p, s);
  }
  return NP_ERR_UNSUPPORTED;
}

np_status launch_prefill_q8_simt(const PrefillParams& p, np_dtype dtype, np_form8 form, cudaStream_t s) {
  if (dtype == NP_BF16)
    return form == NP_E4M3 ? by_dim<__nv_bfloat16, NP_E4M3>(p, s) : by_dim<__nv_bfloat16, NP_INT8>(p, s);
  return form == NP_E4M3 ? by_dim<float, NP_E4M3>(p, s) : by_dim<float, NP_INT8>(p, s);
}

}  // namespace npk
