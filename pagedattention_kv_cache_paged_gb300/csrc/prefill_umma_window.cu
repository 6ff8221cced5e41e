// paged_attention_window's chunks on tcgen05 (prefill_umma.cuh); a unit of its own for the compiler's time.
#include "prefill_umma.cuh"

namespace pa {

cudaError_t launch_prefill_umma_window(const AttnArgs& a, pa_dtype dt, cudaStream_t s, int* launches) {
  return launch_um<true>(a, dt, s, launches);
}

}  // namespace pa
