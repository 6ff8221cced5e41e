// paged_attention_prefill on tcgen05 (prefill_umma.cuh).
#include "prefill_umma.cuh"

namespace pa {

cudaError_t launch_prefill_umma(const AttnArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  return launch_um<false>(a, dt, s, launches);
}

}  // namespace pa
