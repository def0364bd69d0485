// prefill_simt.cu -- np_paged_prefill on the FMA pipes: fp32 pools of head_dim 256.
#include "prefill_simt.cuh"

namespace npk {

np_status launch_prefill_simt(const PrefillParams& p, cudaStream_t s) {
  return launch_simt<-1>(p, s);
}

}  // namespace npk
