// Sliding-window instances of the tcgen05 forward: dense and packed bf16.
#include "fwd_bf16_sm103.cuh"

namespace fa {

cudaError_t launch_fwd_window(const FwdParams& p, cudaStream_t stream, const char** why) {
  return p.d == 128 ? launch<128, false, false, true>(p, stream, why)
                    : launch<64, false, false, true>(p, stream, why);
}

}  // namespace fa
