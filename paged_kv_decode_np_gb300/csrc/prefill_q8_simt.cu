// prefill_q8_simt.cu -- np_paged_prefill_q8 on the FMA pipes: fp32 q, head_dim 256.
#include "prefill_simt.cuh"

namespace npk {

np_status launch_prefill_q8_simt(const PrefillParams& p, np_form8 form, cudaStream_t s) {
  return form == NP_E4M3 ? launch_simt<NP_E4M3>(p, s) : launch_simt<NP_INT8>(p, s);
}

}  // namespace npk
