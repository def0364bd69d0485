// prefill_q8_simt.cu -- np_paged_prefill_q8 on the FMA pipes: fp32 q.
#include "prefill_simt.cuh"

namespace npk {

template <int FORM>
static np_status by_dim(const PrefillParams& p, cudaStream_t s) {
  switch (p.head_dim) {
    case 16: return launch_simt<float, 16, FORM>(p, s);
    case 32: return launch_simt<float, 32, FORM>(p, s);
    case 64: return launch_simt<float, 64, FORM>(p, s);
    case 128: return launch_simt<float, 128, FORM>(p, s);
    case 256: return launch_simt<float, 256, FORM>(p, s);
  }
  return NP_ERR_UNSUPPORTED;
}

np_status launch_prefill_q8_simt(const PrefillParams& p, np_form8 form, cudaStream_t s) {
  return form == NP_E4M3 ? by_dim<NP_E4M3>(p, s) : by_dim<NP_INT8>(p, s);
}

}  // namespace npk
